// Attention of a tree of drafted tokens over the quantized cache (sm_103a).
//
// "W4A16 + KV cache quantization combined accuracy": softmax(q K^T / sqrt(d)) V for
// every node of a drafted tree at once.  Node n of sequence b sees the sequence's
// cached tokens, itself and its ancestors.  The gh query heads of a kv head and the
// N nodes give gh * N query columns against the same Keys and Values, so the two
// products are matrix products and run on the tensor cores (tcgen05), transposed:
//
//   S^T [128 tokens x columns] = K [128 x 128 channels] Q^T     A = K from tensor memory, B = Q from shared memory
//   O^T [128 channels x columns] += V^T [128 x 128 tokens] P^T  A = V^T from tensor memory, B = P from shared memory
//
// The cache tile is the 128-row operand (M), the query columns are the free one (N):
// no row of M is padding however few columns there are, a token is a tensor-memory
// lane (its mask is a per-thread predicate) and a column's statistics are the same
// in all lanes.  The codes of the cache are stored in the register order of a 16 x 16
// operand fragment, which is also what tcgen05.st's 16x128b shape takes: dequantized
// fragments go straight from registers to tensor memory.
//
// A CTA works on 128 cache tokens ("block") and NT = 32, 64 or 128 columns at a time (the fewest that
// hold all columns; chunks of 128 beyond that), its warps in roles joined by mbarriers:
//   loader warp     cache bytes -> shared-memory slots, a block each (one bulk copy from a contiguous
//                   store, one per block-table entry from a paged one; bf16 rows: cp.async)
//   prep warps      (integer layers) a slot's fp32 scales and zero points -> f16 pairs, checked for range
//   dequant warps   slots -> K and V^T as f16 in tensor memory, a warpgroup for each
//   MMA warp        the tcgen05.mma of both products (scores of the next block before the outputs of this one)
//   softmax warps   scores -> P in one pass with the maxima so far, sums in fp32; a warpgroup for NT / 2
//                   columns (NT / 4 of 128)
// The blocks of all (sequence, kv head, column chunk) items are divided over one CTA per SM, whole items
// where a cut would save few blocks (kCutBlocks, tree_ctas); an item cut between CTAs is merged by the
// last CTA to finish it, in CTA order (the result does not depend on which one that is).
//
// What bounds it: neither HBM nor the tensor cores but the warps' instructions, about 8 cycles each for
// the 5 to 7 warps of a scheduler (ncu, 16 sequences x 8 kv heads x 8192 INT4 tokens, 128 columns: issue
// slots 61 % busy, tensor pipe 29 %, DRAM 16 %; 8600 warp instructions per block, of them about 3700
// softmax, 3300 dequantization).  GB300, one launch: those 119 us (579 TFLOP/s, 0.31 of a measured bf16
// GEMM); the same tokens in FP8 with 64 columns 71 us (3.87 TB/s, 0.57 of a measured copy); 128 heads of
// 32768 INT2 tokens with 32 columns 293 us.
//
// Roundings.  The tensor cores take f16 operands, each half an f16 step (2^-11, relative) off at most: P,
// the bf16 queries (exact from 2^-14 up), bf16 Keys and Values, and those of integer layers, s m + c with
// an exact centred code m and s, c = s (2^(b-1) - z) rounded to f16 first.  (fp32 scales cost the
// dequantization twice the instructions and gained a factor of 1.7 in the error.)  FP8 codes are exact in
// f16; their tensor scales enter in fp32.  Sums, maxima and the merge are fp32.  A running maximum may be
// stale by up to 8 in the exponent (P below 2^8, well inside f16).
#pragma once

#include <mutex>

#include "kvq_common.cuh"

namespace kvq {

// ---------------------------------------------------------------------------
// tcgen05 wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tc_alloc512(uint32_t smem_dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_dst) : "memory");
}
__device__ __forceinline__ void tc_dealloc512(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(taddr));
}
__device__ __forceinline__ void tc_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The loads' registers pass through the wait, so that nothing reads them before it.
__device__ __forceinline__ void tc_wait_ld(float (&x)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7])
               :
               : "memory");
}
template <int N>
__device__ __forceinline__ void tc_wait_ld(float (&x)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(x[i]));
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], f16 operands, fp32 accumulate, M = 128
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 lanes in fragment order: four, two or one 16 x 16 f16 fragments (4 registers each) side by side
__device__ __forceinline__ void tc_st_frags(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void tc_st_frags(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]));
}
__device__ __forceinline__ void tc_st_frags(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
// 32 lanes x 16 columns, one lane per thread
__device__ __forceinline__ void tc_ld16(uint32_t taddr, float* x) {
  uint32_t* u = reinterpret_cast<uint32_t*>(x);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_ld8(uint32_t taddr, float* x) {
  uint32_t* u = reinterpret_cast<uint32_t*>(x);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tc_st8(uint32_t taddr, const float* x) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(x);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]));
}

// Shared-memory matrix descriptor: start address, leading and stride byte offsets (16-byte
// units), descriptor version 1, swizzle mode (2: 128 B, 4: 64 B, 6: 32 B).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         (1ull << 46) | ((uint64_t)swizzle << 61);
}
// Instruction descriptor of kind::f16: fp32 D, f16 A and B, M = 128, N = n; b_mn: B stored with N contiguous
__host__ __device__ constexpr uint32_t mma_idesc(int n, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float warp_max(float v) {  // (NaN only where all are)
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// one lane of the warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}
// v f; a sum that is still 0 stays so whatever f is
__device__ __forceinline__ float scaled(float v, float f) { return v == 0.f ? 0.f : v * f; }
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_any(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %3, 0; bar.red.or.pred q, %1, %2, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------------------
// shapes
// ---------------------------------------------------------------------------
constexpr int kBlk = 128;  // cache tokens per block

template <int NT>
struct TreeShape {
  // warps: 4 K, 4 V, then a softmax warpgroup per kSub columns, then loader, MMA, two prep warps.  128 columns take
  // four softmax warpgroups: two of 64 columns each leave a scheduler too few warps to issue from (152 -> 136 us for
  // the 70B-shaped INT4 layer); their registers leave the others few.
  static constexpr int kGroups = NT == 128 ? 4 : 2, kSub = NT / kGroups;
  static constexpr int kSmWarps = 4 * kGroups, kIo = 8 + kSmWarps;
  static constexpr int kWarps = kIo + 4, kThreads = 32 * kWarps;
  // registers a thread: at launch, then by role (the roles' warpgroups together stay within the launch's)
  static constexpr int kRegLaunch = NT == 128 ? 72 : 96;
  static constexpr int kRegDq = NT == 128 ? 56 : 80, kRegSm = NT == 128 ? 88 : 128, kRegIo = NT == 128 ? 40 : 64;
  static_assert(2 * kRegDq + kGroups * kRegSm + kRegIo <= (kWarps / 4) * kRegLaunch, "register split");
  static constexpr int kQBytes = NT * 256;         // queries (f16): [two 64-channel halves][NT rows of 128 bytes]
  static constexpr int kPBytes = kBlk * NT * 2;    // one buffer of P (f16)
  static constexpr int kFixed = kQBytes + 2 * kPBytes;
  // tensor memory: K and V twice 64 columns each, outputs NT, scores NT, twice where there is room (128 columns: one
  // buffer of scores and two of K and V; the other way round every dequantization waits for a product: 181 -> 172 us)
  static constexpr int kSb = NT == 128 ? 1 : 2;
  static constexpr uint32_t kTmK = 0, kTmV = 128, kTmS = 256, kTmO = 256 + kSb * NT;
  static_assert(kTmO + NT <= 512, "tensor memory");
  // P rows (one per token): NT <= 64 columns in one row of 2 NT bytes, 128 as two 64-column regions, in the
  // swizzle of that row length (B operand with the columns contiguous)
  static constexpr int kPRow = NT == 32 ? 64 : 128;
  static constexpr uint32_t kPSwizzle = NT == 32 ? 4 : 2, kPMask = NT == 32 ? 3 : 7;
  // Blocks that a cut has to save a CTA before it pays (it costs partial results and the merge).  Break-even, GB300:
  // 32 columns, 28 INT2 and 22 FP8 blocks; 64 columns, 14 of FP8; 128 columns, 16 to 20 of INT4 (32 and 128 items of
  // 1280 to 49152 tokens; 128 FP8 items of 32768 tokens 248 us whole, 223 cut, of 8192 71 whole, 74 cut)
  static constexpr unsigned kCutBlocks = NT == 32 ? 24 : 16;
};

constexpr int kMaxSlots = 12;
constexpr long long kTreeWait = kWaitLimitCycles;

// One cut of an item: blocks [blk0, blk1) of (sequence b, kv head h, column chunk ch)
struct TreeSeg {
  int b, h, ch, blk0, blk1, nblk, nq;
  int n_sink, qn, r;  // the sequence's tokens: sink, quantized, window
  unsigned item0;     // first unit of the item
};

// A warp's position in its CTA's units
struct TreeCursor {
  unsigned u, end;
  int b;
};

struct TreeSmem {  // small shared state, after the big buffers
  // (barriers, in the order that the set-up initialises them in)
  unsigned long long slot_full[kMaxSlots], slot_ready[kMaxSlots], slot_empty[kMaxSlots];
  unsigned long long k_full[2], k_empty[2], v_full[2], v_empty[2];
  unsigned long long s_full[2], s_free[2], p_full[2], p_free[2], q_full, drain;
  int tile_at[kMaxSlots][8], head_at[kMaxSlots][8];  // integer layers: byte offsets of a slot's tiles, of their Key scales
  uint32_t slot_ok[kMaxSlots];  // quantized slots: which of the four tiles were copied
  uint32_t tmem;
  int abort;
  int last;                       // merge: this CTA finished the item
  alignas(16) float neg[128];     // minus the running maximum of each column (log2 domain; 0 until one is set)
  alignas(16) float fall[128];    // what a change of the maxima scales sums by; epilogue: 1 / sum
  alignas(16) float red[4][128];  // the four warps' maxima or sums
  int row[128];                   // epilogue: the columns' rows of the output, -1: none
  int unset[4];
  unsigned long long anc[64];     // a node's ancestors and itself
  unsigned long long wild;        // nodes whose drafted Values f16 does not hold
  int par[64];
  unsigned units, ctas;           // blocks of the launch, CTAs that share them
  float kscale, vunit;            // FP8: the Keys' tensor scale, the unit of the Values (else 1)
  int whole;                      // an item a CTA
  TreeCursor cur[28];             // per warp
  TreeSeg seg[28];
};

// node n's ancestors and itself; par[n] < n, or -1
__device__ __forceinline__ unsigned long long tree_ancestors(const int* par, int n) {
  unsigned long long a = 0;
  for (; n >= 0; n = par[n]) a |= 1ull << n;
  return a;
}

__device__ __forceinline__ void tree_cursor(const TreeParams& p, const int* pre, unsigned lo, unsigned hi, TreeCursor& c) {
  c.u = lo;
  c.end = hi;
  int a = 0, z = p.batch - 1;  // the last sequence whose first unit is <= lo
  const unsigned hc = (unsigned)(p.L.H * p.chunks);
  while (a < z) {
    const int m = (a + z + 1) >> 1;
    if ((unsigned)pre[m] * hc <= lo) a = m;
    else z = m - 1;
  }
  c.b = a;
}

// Record of tile t (t / tiles per record): t < 2^32 / tpg by the host's check, so that the
// rounded-up reciprocal's excess (below tpg / 2^32 of t) does not reach the next integer
__device__ __forceinline__ int tile_record(const TreeParams& p, int t) {
  return p.tpg_inv ? (int)__umulhi((unsigned)t, p.tpg_inv) : t;
}

// A quantized slot holds one block's bytes as they lie in memory, behind kPreHdr bytes (integer layers) for the
// header of a record that began in an earlier block: [header] tile tile .. [header] tile ..
struct TileMap {
  int t0, r0, own;  // first tile, its record, whether that record begins here
  __device__ __forceinline__ TileMap(const TreeParams& p, int blk) {
    t0 = blk * 8;
    r0 = tile_record(p, t0);
    own = r0 * p.L.tpg == t0;
  }
  // bytes to tile j (0 .. 7) of the block, given its record's number behind r0
  __device__ __forceinline__ int tile(const TreeParams& p, int j, int e) const {
    return p.slot_hdr + j * p.L.tile_bytes + (e + own) * p.L.hdr_bytes;
  }
  // bytes to the header of record r0 + e
  __device__ __forceinline__ int header(const TreeParams& p, int e) const {
    return e + own == 0 ? 0 : tile(p, e == 0 ? 0 : (r0 + e) * p.L.tpg - t0, e) - p.L.hdr_bytes;
  }
  __device__ __forceinline__ int record(const TreeParams& p, int j) const { return tile_record(p, t0 + j) - r0; }
};

// First unit of CTA c of W: floor(U c / W) without a 64-bit division (U = q W + r, c <= W < 2^16)
__device__ __forceinline__ unsigned tree_unit(unsigned U, unsigned W, unsigned c) {
  const unsigned q = U / W, r = U - q * W;
  return q * c + r * c / W;
}

// The warp's next cut, in shared memory (roles keep few of its fields in registers); false behind the last.
__device__ __forceinline__ bool tree_next(const TreeParams& p, const int* pre, const int* lens, TreeCursor& c,
                                          TreeSeg& s) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0 && c.u < c.end) {
    const unsigned hc = (unsigned)(p.L.H * p.chunks);
    int b = c.b;
#pragma unroll 1
    while (b + 1 < p.batch && (unsigned)pre[b + 1] * hc <= c.u) ++b;
    c.b = b;
    const unsigned nblk = (unsigned)(pre[b + 1] - pre[b]);
    const unsigned off = c.u - (unsigned)pre[b] * hc, item = off / nblk, blk0 = off - item * nblk;
    const unsigned left = c.end - c.u, n = left < nblk - blk0 ? left : nblk - blk0;
    const int T = lens[b], qn = lens[p.batch + b], n_sink = T < p.L.S ? T : p.L.S;
    s.b = b;
    s.h = (int)(item / (unsigned)p.chunks);
    s.ch = (int)(item % (unsigned)p.chunks);
    s.blk0 = (int)blk0;
    s.blk1 = (int)(blk0 + n);
    s.nblk = (int)nblk;
    s.nq = (qn + kBlk - 1) / kBlk;
    s.n_sink = n_sink;
    s.qn = qn;
    s.r = T - n_sink - qn;
    s.item0 = c.u - blk0;
    c.u += n;
  } else if ((threadIdx.x & 31) == 0) {
    s.blk1 = -1;
  }
  __syncwarp();
  return *const_cast<volatile int*>(&s.blk1) >= 0;
}

// Wait for a barrier phase; false when the bound ran out here or elsewhere in the CTA.
__device__ __forceinline__ bool tree_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool tree_wait(unsigned long long* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  const uint32_t a = smem_addr(bar);
  if (__builtin_expect(tree_try(a, parity), 1)) return true;
  const long long t0 = clock64();
  while (!tree_try(a, parity)) {
    if (__builtin_expect(*abort != 0, 0)) return false;
    if (__builtin_expect(clock64() - t0 > kTreeWait, 0)) {
      *abort = 1;
      report(status, KVQ_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}

// ---------------------------------------------------------------------------
// dequantization of 16-token tiles to f16 operand fragments
// ---------------------------------------------------------------------------
template <int FMT>
struct TreeFmt {
  static constexpr bool kFp8 = FMT == KVQ_FMT_FP8_E4M3 || FMT == KVQ_FMT_FP8_E5M2;
  static constexpr int kBits = kFp8 ? 8 : FMT;
  static constexpr int kWords = kBits * 2;  // 32-bit operand words per lane and matrix
  static constexpr int kRb = 16 * kBits;    // bytes of a token row of codes
};

template <int FMT>
__device__ __forceinline__ void fp8_pairs(uint32_t w, uint32_t& a, uint32_t& b) {
  if constexpr (FMT == KVQ_FMT_FP8_E5M2) e5m2x4_to_f16x4(w, a, b);
  else e4m3x4_to_f16x4(w, a, b);
}

// Integer codes n as n - 2^(b-1), a pair per register, exact: placed in the mantissa of 1024
// (1024 + n 2^o, one ulp is 1), then one fma takes the 2^o and the offset out.  Register REG of step s.
template <int FMT, int REG>
__device__ __forceinline__ uint32_t centred(const uint32_t* w, int s) {
  constexpr uint32_t kMagic = 0x64006400u;  // 1024, 1024
  uint32_t x;
  if constexpr (FMT == KVQ_FMT_INT8) {  // bytes (REG & 1), (REG & 1) + 2 of word 2s + REG / 2
    x = __byte_perm(w[2 * s + (REG >> 1)], kMagic, (REG & 1) ? 0x7351 : 0x7250);
    return hadd2(x, 0xE480E480u);  // - 1152
  } else if constexpr (FMT == KVQ_FMT_INT4) {  // bits 4 REG, 4 REG + 16 of word s
    x = (REG >> 1) ? w[s] >> 8 : w[s];
    if constexpr ((REG & 1) == 0) return hadd2(lop3_and_or(x, 0x000F000Fu, kMagic), 0xE408E408u);  // - 1032
    else return hfma2(lop3_and_or(x, 0x00F000F0u, kMagic), 0x2C002C00u, 0xD480D480u);               // / 16 - 72
  } else {  // bits 8 (s & 1) + 2 REG, + 16 of word s / 2
    x = w[s >> 1] >> (8 * (s & 1));
    constexpr uint32_t kMul[4] = {0x3C003C00u, 0x34003400u, 0x2C002C00u, 0x24002400u};  // 2^-2REG
    constexpr uint32_t kAdd[4] = {0xE402E402u, 0xDC08DC08u, 0xD420D420u, 0xCC80CC80u};  // -(2^(10 - 2REG) + 2)
    return hfma2(lop3_and_or(x, 0x00030003u << (2 * REG), kMagic), kMul[REG], kAdd[REG]);
  }
}

// Scales as the dequantization reads them (f16 pairs, written over the fp32 ones by the prep warps): a value is
// s m + c with m the centred code and c = s (2^(b-1) - z).  K: 16 bytes per four channels {s01, s23, c01, c23};
// V: per group of channels, 16 bytes per q {s of tokens 2q, 2q+1; of 2q+8, 2q+9; c of both}.

// K fragments of N steps of a tile from their words and scales (rows = tokens; register pairs = channels
// 16s + 4q + {0,1}, {2,3})
template <int FMT, int N>
__device__ __forceinline__ void k_frags(const uint32_t* w, const uint4* scales, uint32_t (&r)[4 * N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if constexpr (TreeFmt<FMT>::kFp8) {
      fp8_pairs<FMT>(w[2 * j], r[4 * j], r[4 * j + 1]);
      fp8_pairs<FMT>(w[2 * j + 1], r[4 * j + 2], r[4 * j + 3]);
    } else {
      const uint4 sc = scales[j];
      r[4 * j] = hfma2(centred<FMT, 0>(w, j), sc.x, sc.z);
      r[4 * j + 1] = hfma2(centred<FMT, 1>(w, j), sc.x, sc.z);
      r[4 * j + 2] = hfma2(centred<FMT, 2>(w, j), sc.y, sc.w);
      r[4 * j + 3] = hfma2(centred<FMT, 3>(w, j), sc.y, sc.w);
    }
  }
}

// V^T fragment of step s (rows = channels 16s + .., register pairs = tokens 2q + {0,1}, then + 8)
template <int FMT>
__device__ __forceinline__ void v_frag(const uint32_t* w, int s, const uint4& sc, uint32_t* r) {
  if constexpr (TreeFmt<FMT>::kFp8) {
    fp8_pairs<FMT>(w[2 * s], r[0], r[1]);
    fp8_pairs<FMT>(w[2 * s + 1], r[2], r[3]);
    if constexpr (FMT == KVQ_FMT_FP8_E5M2) {  // units of 256 scales: exact, and leaves room above the codes
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = hfma2(r[i], 0x1C001C00u, 0x80008000u);
    }
  } else {
    r[0] = hfma2(centred<FMT, 0>(w, s), sc.x, sc.z);
    r[1] = hfma2(centred<FMT, 1>(w, s), sc.x, sc.z);
    r[2] = hfma2(centred<FMT, 2>(w, s), sc.y, sc.w);
    r[3] = hfma2(centred<FMT, 3>(w, s), sc.y, sc.w);
  }
}

// the lane's operand words for steps N i .. N i + N - 1 of a code matrix (word w of a lane lies at byte
// ((w / 4) * 32 + lane) * 16 + (w % 4) * 4)
template <int FMT, int N>
__device__ __forceinline__ void load_words(const uint8_t* codes, int lane, int i, uint32_t (&w)[N * TreeFmt<FMT>::kWords / 8]) {
  constexpr int kN = N * TreeFmt<FMT>::kWords / 8;  // 1, 2, 4 or 8
  if constexpr (kN >= 4) {
#pragma unroll
    for (int k = 0; k < kN / 4; ++k) {
      const uint4 v = *reinterpret_cast<const uint4*>(codes + ((i * (kN / 4) + k) * 32 + lane) * 16);
      w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
    }
  } else if constexpr (kN == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(codes + ((i >> 1) * 32 + lane) * 16 + (i & 1) * 8);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(codes + lane * 16 + i * 4);
  }
}

// largest magnitude that a group of scale s and zero point z stands for
__device__ __forceinline__ float group_reach(float s, float z, float levels) {
  return fabsf(s) * fmaxf(fabsf(z), fabsf(levels - z));
}
// four groups' scales and zero points as f16 pairs {s01, s23, c01, c23} with c = s (half - z); `worst` gets the largest
// magnitude that they stand for where that may be more than f16 holds (s m + c with |m| <= half) and `used`
__device__ __forceinline__ uint4 f16_scales(const float4& s, const float4& z, float half, float levels, bool used,
                                            float& worst) {
  const float4 c = make_float4(s.x * (half - z.x), s.y * (half - z.y), s.z * (half - z.z), s.w * (half - z.w));
  const float most = fmaxf(fmaxf(fmaf(fabsf(s.x), half, fabsf(c.x)), fmaf(fabsf(s.y), half, fabsf(c.y))),
                           fmaxf(fmaf(fabsf(s.z), half, fabsf(c.z)), fmaf(fabsf(s.w), half, fabsf(c.w))));
  if (__builtin_expect(most >= 65000.f && used, 0))
    worst = fmaxf(worst, fmaxf(fmaxf(group_reach(s.x, z.x, levels), group_reach(s.y, z.y, levels)),
                               fmaxf(group_reach(s.z, z.z, levels), group_reach(s.w, z.w, levels))));
  return make_uint4(pack_f16(s.x, s.y), pack_f16(s.z, s.w), pack_f16(c.x, c.y), pack_f16(c.z, c.w));
}
// f16 pair of tokens t, t + 1: all ones where the token is below n
__device__ __forceinline__ uint32_t pair_mask(int t, int n) {
  return (t < n ? 0xFFFFu : 0u) | (t + 1 < n ? 0xFFFF0000u : 0u);
}
__device__ __forceinline__ void put_out(const TreeParams& p, int row, int c, float v) {
  const long long at = (long long)row * 128 + c;
  if (p.out_bf16) reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(p.out)[at] = v;
}

// bf16 rows in a slot: token row of 256 bytes, its 16-byte chunks permuted so that the
// operand reads below are free of bank conflicts (K: 8-byte reads of 4 rows x 2 chunks;
// V: ldmatrix over 8 rows)
__device__ __forceinline__ int krow_chunk(int row, int c) { return row * 256 + ((c ^ ((row & 3) << 1)) << 4); }
__device__ __forceinline__ int vrow_chunk(int row, int c) { return row * 256 + ((c ^ (row & 7)) << 4); }

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  const float2 f = unpack_bf16(w);
  return pack_f16(f.x, f.y);
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float mul) {
  const float2 f = unpack_bf16(w);
  return pack_f16(f.x * mul, f.y * mul);
}
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int FMT, int NT>
__global__ void __launch_bounds__(TreeShape<NT>::kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  using Sh = TreeShape<NT>;
  using F = TreeFmt<FMT>;
  constexpr int SUB = Sh::kSub;
  constexpr uint32_t kAll = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const LayerDesc& L = p.L;
  const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31;
  uint8_t* const Qs = smem;
  uint8_t* const Ps = smem + Sh::kQBytes;
  uint8_t* const slots = smem + Sh::kFixed;
  TreeSmem& S = *reinterpret_cast<TreeSmem*>(slots + (size_t)p.nslots * p.slot_bytes);
  int* const pre = reinterpret_cast<int*>(&S + 1);  // [batch + 1] blocks before
  int* const lens = pre + p.batch + 1;              // [batch] tokens
  int* const quants = lens + p.batch;               // [batch] those in the quantized store

  // ---- set-up: barriers, tensor memory, the batch's block counts ----
  // (a thread per barrier and 32-bit divisions below: this code runs once, and every instruction of it is fetched
  // from beyond the SM, so a small call costs what its length costs)
  if (tid < 3 * kMaxSlots) {
    const int kind = tid / kMaxSlots;  // slot_full, slot_ready, slot_empty
    mbar_init(smem_addr(S.slot_full + tid), kind == 0 ? 32 : (kind == 1 ? 1 : 8));
  } else if (tid < 3 * kMaxSlots + 18) {
    const int i = tid - 3 * kMaxSlots;  // k_full k_empty v_full v_empty s_full s_free p_full p_free (two each) q_full drain
    const int kind = i >> 1;
    mbar_init(smem_addr(S.k_full + i), kind == 0 || kind == 2 ? 4 : (kind == 5 || kind == 6 || i == 16 ? Sh::kSmWarps : 1));
  } else if (tid < 3 * kMaxSlots + 22) {
    S.unset[tid - 3 * kMaxSlots - 18] = 0;
  } else if (tid == 3 * kMaxSlots + 22) {
    S.abort = 0;
  }
  if (tid < 64) fence_barrier_init();
  if (warp == Sh::kIo + 1) {
    tc_alloc512(smem_addr(&S.tmem));
    tc_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  if (tid == 0) {
    S.kscale = F::kFp8 ? *p.C.k_tscale : 1.f;
    S.vunit = F::kFp8 ? *p.C.v_tscale * (FMT == KVQ_FMT_FP8_E5M2 ? 256.f : 1.f) : 1.f;
  }
#pragma unroll 1
  for (int b = tid; b < p.batch; b += Sh::kThreads) {
    int T = p.seq_lens[b];
    if (T > p.most_tokens) {
      if (blockIdx.x == 0) report(p.status, KVQ_DEV_CAPACITY);
      T = p.most_tokens;
    }
    const TokenSplit ts = split_tokens(T < 0 ? 0 : T, L);
    lens[b] = ts.n_sink + ts.qn + ts.r;
    quants[b] = ts.qn;
    pre[b + 1] = (ts.qn + kBlk - 1) / kBlk + (ts.n_sink + ts.r + p.N + kBlk - 1) / kBlk;
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0, least = 0x7FFFFFFF, most = 0;
    if (lane == 0) pre[0] = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      int v = b0 + lane < p.batch ? pre[b0 + lane + 1] : 0;
      if (b0 + lane < p.batch) least = min(least, v), most = max(most, v);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += x;
      }
      if (b0 + lane < p.batch) pre[b0 + lane + 1] = run + v;
      run += __shfl_sync(kAll, v, 31);
    }
    least = __reduce_min_sync(kAll, least);
    most = __reduce_max_sync(kAll, most);
    if (lane == 0) {
      const unsigned items = (unsigned)(p.batch * L.H * p.chunks), U = (unsigned)run * (unsigned)(L.H * p.chunks);
      S.units = U;
      S.whole = items <= gridDim.x && (unsigned)most <= U / gridDim.x + Sh::kCutBlocks;
      S.ctas = tree_ctas(gridDim.x, U, items, least == most, Sh::kCutBlocks);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(kAll, S.tmem, 0);
  volatile int* const abort = &S.abort;
  TreeCursor& cur = S.cur[warp];
  TreeSeg& sg = S.seg[warp];
  if (lane == 0) {
    const unsigned U = S.units, W = S.ctas, c = blockIdx.x, hc = (unsigned)(L.H * p.chunks);
    unsigned lo = U, hi = U;
    if (S.whole) {  // an item a CTA
      if (c < (unsigned)p.batch * hc) {
        const unsigned b = c / hc, n = (unsigned)(pre[b + 1] - pre[b]);
        lo = (unsigned)pre[b] * hc + (c - b * hc) * n;
        hi = lo + n;
      }
    } else if (c < W) {
      lo = tree_unit(U, W, c);
      hi = tree_unit(U, W, c + 1);
    }
    tree_cursor(p, pre, lo, hi, cur);
  }
  __syncwarp();

  // (each role's branch begins with its register count, which the compiler then allocates by)
  if (warp >= Sh::kIo) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::kRegIo));
    if (warp == Sh::kIo) {
      // ======================= loader =======================
      int slot = 0;
      uint32_t ph = 1;  // the first pass over the slots finds them empty
      int used = 0;
      unsigned rows = 0;  // slots that last held bf16 rows
      bool ok = true;
      // half-warps copy the K and the V row of a bf16 token
      const int kv = lane >> 4;
      const __nv_bfloat16* const sink = reinterpret_cast<const __nv_bfloat16*>(kv ? p.C.sink_v : p.C.sink_k);
      const __nv_bfloat16* const ring = reinterpret_cast<const __nv_bfloat16*>(kv ? p.C.resid_v : p.C.resid_k);
      const __nv_bfloat16* const draft = reinterpret_cast<const __nv_bfloat16*>(kv ? p.v_draft : p.k_draft);
      while (ok && tree_next(p, pre, lens, cur, sg)) {
        const long long pair = (long long)sg.b * L.H + sg.h;
        const int blk1 = sg.blk1, nq = sg.nq, qn = sg.qn;
        for (int blk = sg.blk0; ok && blk < blk1; ++blk) {
          if (blk < nq) {
            const TileMap map(p, blk);
            const int tiles = min(8, ((qn + 15) >> 4) - map.t0);  // of this block
            const uint32_t bar = smem_addr(&S.slot_full[slot]);
            const uint32_t dst = smem_addr(slots + (size_t)slot * p.slot_bytes);
            // paged: lane e owns the block's record r0 + e; contiguous: lane 0 owns all of them, one run of bytes
            const int e = lane, first = e == 0 ? 0 : (map.r0 + e) * L.tpg - map.t0;
            const uint8_t* rec = nullptr;
            uint32_t bytes = 0, okmask = 0;
            int n = 0;  // tiles that the lane copies
            if (L.paged ? first < tiles : lane == 0) {
              rec = record_addr(L, p.C, sg.b, sg.h, map.r0 + e, p.status);
              n = L.paged ? min(tiles, (map.r0 + e + 1) * L.tpg - map.t0) - first : tiles;
              const int heads = L.paged ? (e + map.own > 0) : map.record(p, tiles - 1) + map.own;
              bytes = (uint32_t)(n * L.tile_bytes + heads * L.hdr_bytes);
              okmask = ((1u << n) - 1u) << first;
            }
            if (!rec) bytes = okmask = 0;
            const bool pre = rec && e == 0 && !map.own && L.hdr_bytes;  // the header lies before the block's bytes
            okmask = __reduce_or_sync(kAll, okmask);
            const uint32_t total = __reduce_add_sync(kAll, bytes + (pre ? (uint32_t)L.hdr_bytes : 0u));
            if (!(ok = tree_wait(&S.slot_empty[slot], ph, abort, p.status))) break;
            if (F::kFp8 && (rows >> slot) & 1u) {  // those writes come before the bulk copy (integer layers: prep fences)
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              rows &= ~(1u << slot);
            }
            if (lane == 0) {
              S.slot_ok[slot] = okmask;
              mbar_arrive_expect_tx(bar, total);
            }
            __syncwarp();
            if (rec) {
              if (pre) bulk_copy_g2s(dst, rec, L.hdr_bytes, bar);
              const int within = e == 0 ? map.t0 - map.r0 * L.tpg : 0;
              bulk_copy_g2s(dst + (e + map.own > 0 ? map.tile(p, first, e) - L.hdr_bytes : p.slot_hdr),
                            rec + (within ? L.hdr_bytes + (long long)within * L.tile_bytes : 0), bytes, bar);
            }
            if (lane != 0) mbar_arrive(bar);
            if (++slot == p.nslots) { slot = 0; ph ^= 1; }
            ++used;
          } else {
            const int x0 = (blk - nq) * kBlk, n_sink = sg.n_sink;
            const int nsr = n_sink + sg.r, nrow = nsr + p.N;
            for (int part = 0; part < kBlk; part += p.bf_tokens) {
              if (!(ok = tree_wait(&S.slot_empty[slot], ph, abort, p.status))) break;
              const uint32_t dst = smem_addr(slots + (size_t)slot * p.slot_bytes) + (kv ? p.bf_tokens * 256 : 0);
              const int c = lane & 15;
              // runs of rows that follow one another in memory: sink, ring up to its end, ring, drafts; then zeros
              for (int i = 0; i < p.bf_tokens;) {
                const int x = x0 + part + i;
                const __nv_bfloat16* src = draft;
                int n = p.bf_tokens - i;
                uint32_t size = 16;
                if (x < n_sink) {
                  src = sink + (pair * L.S + x) * L.d;
                  n = min(n, n_sink - x);
                } else if (x < nsr) {
                  const int at = (int)((unsigned)(qn + (x - n_sink)) % (unsigned)L.W);
                  src = ring + (pair * L.W + at) * L.d;
                  n = min(n, min(nsr - x, L.W - at));
                } else if (x < nrow) {
                  src = draft + (pair * p.N + (x - nsr)) * L.d;
                  n = min(n, nrow - x);
                } else {
                  size = 0;  // rows behind the list
                }
                src += c * 8;
                const int step = size ? L.d : 0;
#pragma unroll 8
                for (const int end = i + n; i < end; ++i, src += step) {
                  const uint32_t to = dst + (kv ? vrow_chunk(i, c) : krow_chunk(i, c));
                  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(size));
                }
              }
              asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                               smem_addr(&S.slot_full[slot]))
                           : "memory");
              rows |= 1u << slot;
              if (++slot == p.nslots) { slot = 0; ph ^= 1; }
              ++used;
            }
          }
        }
      }
      // every copy must have landed before the CTA ends (bounded; the consumers waited for all of
      // them unless the launch was given up)
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (*abort) {
        for (int i = 0; i < p.nslots && i < used; ++i) {
          const int n = used - 1 - i;  // the slot's last use
          mbar_wait_bounded(smem_addr(&S.slot_full[n % p.nslots]), (n / p.nslots) & 1, kTreeWait);
        }
      }
    } else if (warp == Sh::kIo + 1) {
      // ======================= MMA =======================
      // (the whole warp walks, so that the operands of the one-thread instructions stay uniform)
      constexpr uint32_t kIdQk = mma_idesc(NT, 0), kIdPv = mma_idesc(NT, 1);
      const uint64_t dq = smem_desc(smem_addr(Qs), 16, 1024, 2);
      const uint64_t dp = smem_desc(smem_addr(Ps), kBlk * 128, 8 * Sh::kPRow, Sh::kPSwizzle);
      uint32_t g = 0, nseg = 0;  // blocks and cuts so far
      bool ok = true;
      while (ok && tree_next(p, pre, lens, cur, sg)) {
        const int nb = __shfl_sync(kAll, sg.blk1 - sg.blk0, 0);
        ok = __all_sync(kAll, tree_wait(&S.q_full, nseg & 1, abort, p.status));
        ++nseg;
#pragma unroll 1
        for (int i = 0; ok && i <= nb; ++i) {
          if (i < nb) {
            const uint32_t kb = g & 1, kph = (g >> 1) & 1, sb = Sh::kSb == 2 ? g & 1 : 0;
            ok = tree_wait(&S.k_full[kb], kph, abort, p.status);
            if (ok && g >= Sh::kSb) ok = tree_wait(&S.s_free[sb], ((g / Sh::kSb) - 1) & 1, abort, p.status);
            if (!__all_sync(kAll, ok)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int s = 0; s < 8; ++s)
                tc_mma_ts(tm + Sh::kTmS + sb * NT, tm + Sh::kTmK + kb * 64 + 8 * s,
                          dq + (uint32_t)(((s >> 2) * NT * 128 + (s & 3) * 32) >> 4), kIdQk, s > 0);
              tc_commit(smem_addr(&S.s_full[sb]));
              tc_commit(smem_addr(&S.k_empty[kb]));
            }
            __syncwarp();
          }
          if (i > 0) {
            const uint32_t pg = g - 1, vb = pg & 1, pb = vb, ph = (pg >> 1) & 1;
            ok = tree_wait(&S.v_full[vb], ph, abort, p.status);
            if (ok) ok = tree_wait(&S.p_full[pb], ph, abort, p.status);
            if (!__all_sync(kAll, ok)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                tc_mma_ts(tm + Sh::kTmO, tm + Sh::kTmV + vb * 64 + 8 * j,
                          dp + (uint32_t)((pb * Sh::kPBytes + j * 16 * Sh::kPRow) >> 4), kIdPv,
                          (i > 1 || j > 0) ? 1u : 0u);
              tc_commit(smem_addr(&S.p_free[pb]));
              tc_commit(smem_addr(&S.v_empty[vb]));
            }
            __syncwarp();
          }
          if (i < nb) ++g;
        }
      }
      if (!ok && elect_one()) {  // given up: let the products in flight end before the tensor memory is freed
        tc_commit(smem_addr(&S.drain));
        mbar_wait_bounded(smem_addr(&S.drain), 0, kTreeWait);
      }
      __syncwarp();
    } else if (!F::kFp8) {
      // ======================= prep: scales to f16, two warps, the even and the odd slots =======================
      constexpr float kL = (float)((1 << F::kBits) - 1), kHalf = (float)(1 << (F::kBits - 1));
      int slot = 0;
      uint32_t ph = 0;
      bool ok = true;
      float worst = 0.f;  // largest magnitude that any group stands for
      const int ngv = L.ngv, lg = 31 - __clz(ngv);
      constexpr int kTwo = NT == 128 ? 1 : 2;  // (registers)
      while (ok && tree_next(p, pre, lens, cur, sg)) {
        const int blk1 = sg.blk1, nq = sg.nq;
        for (int blk = sg.blk0; ok && blk < blk1; ++blk) {
          const bool quant = blk < nq;
          const int parts = quant ? 1 : kBlk / p.bf_tokens;
          for (int i = 0; i < parts; ++i) {
            // A warp owns slots, not turns: having seen every phase of a slot's barrier it cannot take an older
            // phase of the same parity for the one it waits for.
            if (((slot ^ warp) & 1) == 0) {
              if (!(ok = tree_wait(&S.slot_full[slot], ph, abort, p.status))) break;
              if (quant) {
                const uint32_t okmask = S.slot_ok[slot];
                uint8_t* const src = slots + (size_t)slot * p.slot_bytes;
                const TileMap map(p, blk);
                const int nh = map.record(p, 31 - __clz(okmask | 1u)) + 1;
                // where the dequantization finds the tiles and their Key scales
                if (lane < 8) {
                  const int e = map.record(p, lane);
                  S.tile_at[slot][lane] = map.tile(p, lane, e);
                  S.head_at[slot][lane] = map.header(p, e);
                }
                __syncwarp();
                // kTwo at a time: all read, then all written over
#pragma unroll 1
                for (int e0 = 0; e0 < nh; e0 += kTwo) {  // (a header whose tiles were not copied holds anything, and is not used)
                  uint8_t* hdr[kTwo];
                  uint4 out[kTwo];
#pragma unroll
                  for (int k = 0; k < kTwo; ++k) {
                    const int e = min(e0 + k, nh - 1);
                    hdr[k] = src + map.header(p, e);
                    const float4 sc = reinterpret_cast<const float4*>(hdr[k])[lane];
                    const float4 z = reinterpret_cast<const float4*>(hdr[k] + 512)[lane];
                    const int ti = e == 0 ? 0 : (map.r0 + e) * L.tpg - map.t0;  // its first tile of the block
                    out[k] = f16_scales(sc, z, kHalf, kL, (okmask >> ti) & 1u, worst);
                  }
                  __syncwarp();
#pragma unroll
                  for (int k = 0; k < kTwo; ++k) reinterpret_cast<uint4*>(hdr[k])[lane] = out[k];
                }
                // Values: a lane per (tile, q, group), the tokens 2q, 2q + 1, 2q + 8, 2q + 9; whole tiles at a time
#pragma unroll 1
                for (int at0 = lane; at0 < 32 * ngv; at0 += 32 * kTwo) {
                  uint8_t* to[kTwo];
                  uint4 out[kTwo];
#pragma unroll
                  for (int k = 0; k < kTwo; ++k) {
                    const int at = ngv == 1 ? at0 : at0 + 32 * k;
                    const int ti = at >> (2 + lg), within = at & (4 * ngv - 1), vq = within >> lg, j = within & (ngv - 1);
                    uint8_t* const base = src + S.tile_at[slot][ti] + 32 * F::kRb;
                    const float* const f = reinterpret_cast<const float*>(base) + 2 * vq * ngv + j;
                    to[k] = base + j * 64 + vq * 16;
                    out[k] = make_uint4(0u, 0u, 0u, 0u);  // (a tile that was not copied: all its Values zero)
                    if ((okmask >> ti) & 1u) {
                      const float4 sc = make_float4(f[0], f[ngv], f[8 * ngv], f[9 * ngv]);
                      const float4 z = make_float4(f[16 * ngv], f[17 * ngv], f[24 * ngv], f[25 * ngv]);
                      out[k] = f16_scales(sc, z, kHalf, kL, true, worst);
                    }
                  }
                  __syncwarp();
#pragma unroll
                  for (int k = 0; k < kTwo; ++k) *reinterpret_cast<uint4*>(to[k]) = out[k];
                }
              }
              // (these writes come before the slot's next bulk copy)
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&S.slot_ready[slot]));
            }
            if (++slot == p.nslots) { slot = 0; ph ^= 1; }
          }
        }
      }
      if (__any_sync(kAll, worst >= 65520.f) && lane == 0) report(p.status, KVQ_DEV_RANGE);
    }
  } else if (warp < 8) {
    // ======================= dequantization =======================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::kRegDq));
    const int wq = warp & 3;  // tensor-memory lanes 32 wq ..
    const bool isV = warp >= 4;
    const int r = lane >> 2, q = lane & 3;
    const uint32_t tlane = tm + ((uint32_t)(32 * wq) << 16) + (isV ? Sh::kTmV : Sh::kTmK);
    unsigned long long* const full = isV ? S.v_full : S.k_full;
    unsigned long long* const empty = isV ? S.v_empty : S.k_empty;
    unsigned long long* const ready = F::kFp8 ? S.slot_full : S.slot_ready;
    // fragments in registers at a time (K: steps of a tile; V: tiles)
    constexpr int kSteps = NT == 128 ? 2 : 4, kTiles = NT == 128 ? 1 : 2;
    int slot = 0;
    uint32_t ph = 0, g = 0;
    bool ok = true, bad = false;
    // byte offsets of the warp's first operand word and of its channels' scales in a tile (V)
    const int lgv = F::kFp8 ? 7 : 31 - __clz(L.Gv);
    const int vcode = 16 * F::kRb + (F::kBits == 8 ? (wq * 32 + lane) * 16
                                                   : F::kBits == 4 ? ((wq >> 1) * 32 + lane) * 16 + (wq & 1) * 8 : lane * 16 + wq * 4);
    const int vs0 = 32 * F::kRb + ((32 * wq) >> lgv) * 64 + q * 16, vs1 = 32 * F::kRb + ((32 * wq + 16) >> lgv) * 64 + q * 16;
    while (ok && tree_next(p, pre, lens, cur, sg)) {
      const int blk1 = sg.blk1, nq = sg.nq, qn = sg.qn;
#pragma unroll 1
      for (int blk = sg.blk0; ok && blk < blk1; ++blk, ++g) {
        const int buf = (int)(g & 1);
        // the buffer's previous use has been read
        if (!(ok = tree_wait(&empty[buf], ((g >> 1) & 1) ^ 1, abort, p.status))) break;
        tc_fence_after();
        const uint32_t tt = tlane + buf * 64;
        if (blk < nq) {
          if (!(ok = tree_wait(&ready[slot], ph, abort, p.status))) break;
          const uint8_t* const src = slots + (size_t)slot * p.slot_bytes;
          const uint32_t okmask = S.slot_ok[slot];
          if (!isV) {
            // tile 2 wq + e, kSteps steps at a time; the next ones' words and scales on their way meanwhile
            constexpr int kPer = 8 / kSteps;
            uint32_t w[2][kSteps * F::kWords / 8];
            uint4 sc[2][kSteps];
            auto fetch = [&](int ei, int to) {
              const int ti = 2 * wq + ei / kPer, i = ei % kPer;
              load_words<FMT, kSteps>(src + (F::kFp8 ? ti * L.tile_bytes : S.tile_at[slot][ti]), lane, i, w[to]);
              if constexpr (!F::kFp8) {
                const uint4* const s = reinterpret_cast<const uint4*>(src + S.head_at[slot][ti]) + 4 * kSteps * i + q;
#pragma unroll
                for (int j = 0; j < kSteps; ++j) sc[to][j] = s[4 * j];
              }
            };
            fetch(0, 0);
#pragma unroll 2
            for (int ei = 0; ei < 2 * kPer; ++ei) {
              if (ei + 1 < 2 * kPer) fetch(ei + 1, (ei + 1) & 1);
              uint32_t f[4 * kSteps];
              k_frags<FMT, kSteps>(w[ei & 1], sc[ei & 1], f);
              tc_st_frags(tt + ((uint32_t)(16 * (ei / kPer)) << 16) + 8 * kSteps * (ei % kPer), f);
            }
          } else {
              // kTiles tiles at a time, channels 32 wq .. and 32 wq + 16 ..  (Tiles that were not copied, behind the
              // last one or of a bad block, read as zeros: P is 0 there, so V must be finite.)
#pragma unroll 2
              for (int tp = 0; tp < 8; tp += kTiles) {
                uint32_t f[2][4 * kTiles];
#pragma unroll
                for (int u = 0; u < kTiles; ++u) {
                  const uint8_t* const tile = src + (F::kFp8 ? (tp + u) * L.tile_bytes : S.tile_at[slot][tp + u]);
                  uint32_t w[4];  // the words of steps 2 wq and 2 wq + 1
                  if constexpr (F::kBits == 8) {
                    const uint4 v = *reinterpret_cast<const uint4*>(tile + vcode);
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                  } else if constexpr (F::kBits == 4) {
                    const uint2 v = *reinterpret_cast<const uint2*>(tile + vcode);
                    w[0] = v.x, w[1] = v.y;
                  } else {
                    w[0] = *reinterpret_cast<const uint32_t*>(tile + vcode);
                    w[1] = w[0] >> 8;
                  }
                  uint4 s0 = make_uint4(0, 0, 0, 0), s1 = s0;  // scales of the two steps' channels
                  if constexpr (!F::kFp8) {
                    s0 = *reinterpret_cast<const uint4*>(tile + vs0);
                    s1 = *reinterpret_cast<const uint4*>(tile + vs1);
                  }
                  v_frag<FMT>(w, 0, s0, f[0] + 4 * u);
                  v_frag<FMT>(w + (F::kBits == 8 ? 2 : 1), 0, s1, f[1] + 4 * u);
                  if constexpr (F::kFp8) {
                    // tokens behind the last one: zeros whatever the store, or an uncopied tile of the slot, holds
                    const int nv = (okmask >> (tp + u)) & 1u ? qn - 16 * (8 * blk + tp + u) : 0;
                    if (__builtin_expect(nv < 16, 0)) {
                      const uint32_t m0 = pair_mask(2 * q, nv), m1 = pair_mask(2 * q + 8, nv);
#pragma unroll
                      for (int e = 0; e < 2; ++e) {
                        f[e][4 * u] &= m0, f[e][4 * u + 1] &= m0;
                        f[e][4 * u + 2] &= m1, f[e][4 * u + 3] &= m1;
                      }
                    }
                  }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  tc_st_frags(tt + ((uint32_t)(16 * e) << 16) + 8 * tp, f[e]);
              }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&S.slot_empty[slot]));
          if (++slot == p.nslots) { slot = 0; ph ^= 1; }
        } else {
          uint32_t top = 0;
          const bool drafts = (blk - nq) * kBlk + kBlk > sg.n_sink + sg.r;
          const float vinv = F::kFp8 && isV ? 1.f / S.vunit : 1.f;
#pragma unroll 1
          for (int part = 0; part < kBlk; part += p.bf_tokens) {
            if (!(ok = tree_wait(&ready[slot], ph, abort, p.status))) break;
            const uint8_t* const src = slots + (size_t)slot * p.slot_bytes;
            if (!isV) {
              if (32 * wq >= part && 32 * wq < part + p.bf_tokens) {
#pragma unroll 1
                for (int ei = 0; ei < 16 / kSteps; ++ei) {  // 16 rows, kSteps steps
                  const int e = ei / (8 / kSteps), i = ei % (8 / kSteps);
                  const int row = 32 * wq - part + 16 * e + r;
                  uint32_t f[4 * kSteps];
#pragma unroll
                  for (int j = 0; j < kSteps; ++j) {
                    const int c = 2 * (kSteps * i + j) + (q >> 1);
                    const uint2 a = *reinterpret_cast<const uint2*>(src + krow_chunk(row, c) + (q & 1) * 8);
                    const uint2 b = *reinterpret_cast<const uint2*>(src + krow_chunk(row + 8, c) + (q & 1) * 8);
                    top = abs_max2(abs_max2(abs_max2(abs_max2(top, a.x), a.y), b.x), b.y);
                    f[4 * j] = bf16x2_to_f16x2(a.x);
                    f[4 * j + 1] = bf16x2_to_f16x2(b.x);
                    f[4 * j + 2] = bf16x2_to_f16x2(a.y);
                    f[4 * j + 3] = bf16x2_to_f16x2(b.y);
                  }
                  tc_st_frags(tt + ((uint32_t)(16 * e) << 16) + 8 * kSteps * i, f);
                }
              }
            } else {
              const uint32_t vbase = smem_addr(src) + p.bf_tokens * 256;
              const int row0 = (lane & 7) + ((lane >> 4) << 3), cc = (lane >> 3) & 1;
#pragma unroll 1
              for (int t4 = 0; t4 < p.bf_tokens; t4 += 16 * kTiles) {  // kTiles fragments of 16 tokens at a time
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int c = 2 * (2 * wq + e) + cc;
                  uint32_t f[4 * kTiles];
#pragma unroll
                  for (int u = 0; u < kTiles; ++u) {
                    uint32_t a[4];
                    ldmatrix_x4_trans(vbase + vrow_chunk(t4 + 16 * u + row0, c), a[0], a[1], a[2], a[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      top = abs_max2(top, a[i]);
                      f[4 * u + i] = F::kFp8 ? bf16x2_to_f16x2(a[i], vinv) : bf16x2_to_f16x2(a[i]);
                    }
                  }
                  if (drafts) {
                    // a drafted Value that f16 does not hold: zero, so that the nodes that do not see
                    // its token do not get 0 * NaN (those that do get NaN through P)
#pragma unroll
                    for (int i = 0; i < 4 * kTiles; ++i) {
                      if ((f[i] & 0x7C00u) == 0x7C00u) f[i] &= 0xFFFF0000u;
                      if ((f[i] & 0x7C000000u) == 0x7C000000u) f[i] &= 0xFFFFu;
                    }
                  }
                  tc_st_frags(tt + ((uint32_t)(16 * e) << 16) + ((part + t4) >> 1), f);
                }
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&S.slot_empty[slot]));
            if (++slot == p.nslots) { slot = 0; ph ^= 1; }
          }
          // a bf16 value that f16 does not hold (65504 is the last one)
          if (!(__uint_as_float(max(top & 0xFFFFu, top >> 16) << 16) * fabsf(vinv) < 65520.f)) bad = true;
        }
        if (!ok) break;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&full[buf]));
      }
    }
    if (__any_sync(kAll, bad) && lane == 0) report(p.status, KVQ_DEV_RANGE);
  } else {
    // ======================= softmax, epilogue =======================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Sh::kRegSm));
    constexpr int kAllSm = 128 * Sh::kGroups;
    const int h = (warp - 8) >> 2;        // the warpgroup's columns: kSub h ..
    const int wq = warp & 3;
    const int tok = 32 * wq + lane;       // the thread's tensor-memory lane: token of the scores, channel of the outputs
    const int th = tid - 256;             // over all groups
    const uint32_t tlane = tm + ((uint32_t)(32 * wq) << 16);
    float* const neg = S.neg + h * SUB;
    const int barid = 1 + h;
    uint32_t g = 0;
    while (tree_next(p, pre, lens, cur, sg)) {
      // ---- the drafted tokens, where this cut reaches a block of theirs ----
      named_sync(5, kAllSm);  // (the previous cut's epilogue has read S.neg)
      if (th < NT) S.neg[th] = 0.f;
      if (th < 64 && sg.blk1 > sg.nq + (sg.n_sink + sg.r) / kBlk) {
        bool wild = false;
        if (th < p.N) {
          int up = p.parents[(long long)sg.b * p.N + th];
          if (up < -1 || up >= th) {
            report(p.status, KVQ_DEV_BAD_TREE);
            up = -1;
          }
          S.par[th] = up;
          const float vinv = F::kFp8 ? 1.f / S.vunit : 1.f;
          const uint4* v = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.v_draft) +
                                                          (((long long)sg.b * L.H + sg.h) * p.N + th) * L.d);
          uint32_t m = 0;
#pragma unroll 8
          for (int i = 0; i < 16; ++i) {
            const uint4 a = v[i];
            m = abs_max2(abs_max2(abs_max2(abs_max2(m, a.x), a.y), a.z), a.w);
          }
          wild = !(__uint_as_float(max(m & 0xFFFFu, m >> 16) << 16) * fabsf(vinv) < 65520.f);
        }
        const uint32_t w = __ballot_sync(kAll, wild);
        if (lane == 0) reinterpret_cast<uint32_t*>(&S.wild)[wq] = w;
      }
      // ---- the queries, f16, channels in the Key fragments' order within every 16 ----
      {
        uint32_t m = 0;
        const int g16 = th & 7;
#pragma unroll 1
        for (int row = th >> 3; row < NT; row += kAllSm / 8) {
          const int col = sg.ch * NT + row;
          uint4 a = make_uint4(0, 0, 0, 0), b = a;
          if (col < p.gh * p.N) {
            const int n = col / p.gh, hh = col - n * p.gh;
            const uint4* src = reinterpret_cast<const uint4*>(
                reinterpret_cast<const __nv_bfloat16*>(p.q) +
                (((long long)sg.b * p.N + n) * p.Hq + (long long)sg.h * p.gh + hh) * L.d + 16 * g16);
            a = src[0];
            b = src[1];
          }
          m = abs_max2(abs_max2(abs_max2(abs_max2(m, a.x), a.y), a.z), a.w);
          m = abs_max2(abs_max2(abs_max2(abs_max2(m, b.x), b.y), b.z), b.w);
          uint8_t* const dst = Qs + (g16 >> 2) * (NT * 128) + row * 128;
          const int c = 2 * (g16 & 3);
          *reinterpret_cast<uint4*>(dst + ((c ^ (row & 7)) << 4)) = make_uint4(
              bf16x2_to_f16x2(a.x), bf16x2_to_f16x2(a.z), bf16x2_to_f16x2(b.x), bf16x2_to_f16x2(b.z));
          *reinterpret_cast<uint4*>(dst + (((c + 1) ^ (row & 7)) << 4)) = make_uint4(
              bf16x2_to_f16x2(a.y), bf16x2_to_f16x2(a.w), bf16x2_to_f16x2(b.y), bf16x2_to_f16x2(b.w));
        }
        if (max(m & 0xFFFFu, m >> 16) >= 0x4780u) report(p.status, KVQ_DEV_RANGE);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&S.q_full));
      named_sync(5, kAllSm);
      if (th < p.N && sg.blk1 > sg.nq + (sg.n_sink + sg.r) / kBlk) S.anc[th] = tree_ancestors(S.par, th);
      named_sync(5, kAllSm);

      constexpr int kCh = NT == 64 ? 32 : 16;  // columns in registers at a time
      float l[SUB];
#pragma unroll
      for (int j = 0; j < SUB; ++j) l[j] = 0.f;
      bool unset = true;  // some column has no maximum yet (uniform over the warpgroup)
      bool has = false;   // column `tok` has one

      const int blk0 = sg.blk0, blk1 = sg.blk1, nq = sg.nq;
      const int nplain = L.paged ? 0 : sg.qn / kBlk;  // leading blocks whose tokens all count
#pragma unroll 1
      for (int blk = blk0; blk < blk1; ++blk, ++g) {
        const uint32_t sb = Sh::kSb == 2 ? g & 1 : 0, pb = g & 1;
        const uint32_t ts = tlane + Sh::kTmS + sb * NT + h * SUB, to = tlane + Sh::kTmO + h * SUB;
        // ---- which of the half's columns see the thread's token ----
        const bool quant = blk < nq;
        bool masked = false, spoilt = false;
        unsigned long long allow = ~0ull;
        if (__builtin_expect(blk >= nplain, 0)) {
          bool valid;
          if (quant) {
            const int x = blk * kBlk + tok;
            valid = x < sg.qn;
            if (L.paged && valid) {
              const int e = p.C.block_table[(long long)sg.b * L.mbps + x / L.P];
              valid = e >= 0 && e < L.num_blocks;
            }
            allow = valid ? ~0ull : 0ull;
          } else {
            const int nsr = sg.n_sink + sg.r, x = (blk - nq) * kBlk + tok;
            valid = x < nsr;
            if (!valid) allow = 0;
            if (x >= nsr && x < nsr + p.N) {  // a drafted token: its descendants' columns
              const int m = x - nsr;
              spoilt = (S.wild >> m) & 1ull;
              int n = (sg.ch * NT + h * SUB) / p.gh, k = sg.ch * NT + h * SUB - n * p.gh;
              for (int j = 0; j < SUB; ++j) {
                if (n < p.N && ((S.anc[n] >> m) & 1ull)) allow |= 1ull << j;
                if (++k == p.gh) { k = 0; ++n; }
              }
            }
          }
          masked = __any_sync(kAll, !valid);
        }
        // log2 units per unit of the scores (a scale of 0 as one that no score survives: masks stay infinite)
        float c = F::kFp8 && quant ? p.scale_log2 * S.kscale : p.scale_log2;
        if (c == 0.f) c = 1e-37f;
        tree_wait(&S.s_full[sb], (g / Sh::kSb) & 1, abort, p.status);
        if (g > 1) tree_wait(&S.p_free[pb], ((g >> 1) - 1) & 1, abort, p.status);  // P's buffer has been read
        tc_fence_after();
        if (masked) {  // into the scores themselves
#pragma unroll 1
          for (int c0 = 0; c0 < SUB; c0 += 8) {
            const uint32_t w = (uint32_t)(allow >> c0);
            float x[8];
            tc_ld8(ts + c0, x);
            tc_wait_ld(x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (w >> j) & 1u ? (spoilt ? NAN : x[j]) : (c > 0.f ? -INFINITY : INFINITY);
            tc_st8(ts + c0, x);
          }
          tc_wait_st();
        }
        auto load = [&](int c0, float (&x)[kCh]) {
#pragma unroll
          for (int j = 0; j < kCh; j += 16) tc_ld16(ts + c0 + j, x + j);
          tc_wait_ld(x);
        };
        // Columns c0 .. of the scores as exponents (log2) relative to the columns' maxima so far, and their largest
        auto exponents = [&](int c0, float (&x)[kCh], float& top) {
          float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
          for (int j = 0; j < kCh; j += 4) {
            const float4 m4 = *reinterpret_cast<const float4*>(neg + c0 + j);
            const float2 a = fma_f32x2(make_float2(x[j], x[j + 1]), make_float2(c, c), make_float2(m4.x, m4.y));
            const float2 b = fma_f32x2(make_float2(x[j + 2], x[j + 3]), make_float2(c, c), make_float2(m4.z, m4.w));
            x[j] = a.x;
            x[j + 1] = a.y;
            x[j + 2] = b.x;
            x[j + 3] = b.y;
          }
#pragma unroll
          for (int j = 0; j < kCh; j += 4) {
            t0 = fmaxf(fmaxf(x[j], x[j + 1]), t0);
            t1 = fmaxf(fmaxf(x[j + 2], x[j + 3]), t1);
          }
          top = fmaxf(top, fmaxf(t0, t1));
        };
        uint8_t* const P = Ps + pb * Sh::kPBytes + h * SUB / 64 * (kBlk * 128);
        auto put_p = [&](int col, const float* e) {  // eight columns
          const uint32_t at = (uint32_t)(tok * Sh::kPRow + (h * SUB % 64 + col) * 2);
          *reinterpret_cast<uint4*>(P + (at ^ (((at >> 7) & Sh::kPMask) << 4))) =
              make_uint4(pack_f16(e[0], e[1]), pack_f16(e[2], e[3]), pack_f16(e[4], e[5]), pack_f16(e[6], e[7]));
        };
        // P and the sums in one pass, with the maxima as they are; whether one rose too far shows at its end.
        // (a power beyond what the sums could give back is cut to kCap; its column is done over)
        constexpr float kCap = 1.2676506e30f;  // 2^100
        bool fresh = unset, again = false;     // the block's column maxima first; the pass for a second time
        float x[kCh];
#pragma unroll 1
        while (true) {
          if (__builtin_expect(fresh, 0)) {
            // ---- the block's column maxima ----
            float top = -INFINITY;
#pragma unroll 1
            for (int c0 = 0; c0 < SUB; c0 += kCh) {
              load(c0, x);
              exponents(c0, x, top);
              float mine = 0.f;
#pragma unroll
              for (int j = 0; j < kCh; ++j) {
                const float v = warp_max(x[j]);
                if (lane == j) mine = v;
              }
              if (lane < kCh) S.red[wq][h * SUB + c0 + lane] = mine;
            }
            named_sync(barid, 128);
            if (tok < SUB) {
              const int j = h * SUB + tok;
              // d: the block's maximum relative to the column's so far; its first one is taken as it is
              const float d = fmaxf(fmaxf(S.red[0][j], S.red[1][j]), fmaxf(S.red[2][j], S.red[3][j]));
              float rise = fmaxf(d, 0.f);
              if (!has) {
                has = d != -INFINITY;
                rise = has && d == d ? d : 0.f;  // (not a number: in the sum, where a merge keeps it)
              }
              neg[tok] -= rise;
              S.fall[j] = exp2_approx(-rise);
              if (!has) S.unset[h] = 1;
            }
            named_sync(barid, 128);
            unset = S.unset[h] != 0;
            if (blk > blk0) {  // what the sums and O hold so far (O: behind the previous block's product)
#pragma unroll
              for (int j = 0; j < SUB; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&S.fall[h * SUB + j]);
                l[j] = scaled(l[j], f.x);
                l[j + 1] = scaled(l[j + 1], f.y);
                l[j + 2] = scaled(l[j + 2], f.z);
                l[j + 3] = scaled(l[j + 3], f.w);
              }
              tree_wait(&S.p_free[(g - 1) & 1], ((g - 1) >> 1) & 1, abort, p.status);
              tc_fence_after();
#pragma unroll 1
              for (int j0 = 0; j0 < SUB; j0 += 8) {
                float o[8];
                tc_ld8(to + j0, o);
                tc_wait_ld(o);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = scaled(o[j], S.fall[h * SUB + j0 + j]);
                tc_st8(to + j0, o);
              }
              tc_wait_st();
            }
            named_sync(barid, 128);  // (fall and unset have been read)
            if (tok == 0) S.unset[h] = 0;
          }
          float top = -INFINITY;
#pragma unroll
          for (int c0 = 0; c0 < SUB; c0 += kCh) {
            load(c0, x);
            exponents(c0, x, top);
            const bool hot = __any_sync(kAll, top > 99.f);
#pragma unroll
            for (int j = 0; j < kCh; ++j) x[j] = exp2_approx(x[j]);
            if (__builtin_expect(hot, 0)) {
#pragma unroll
              for (int j = 0; j < kCh; ++j) x[j] = fminf(x[j], kCap);
            }
#pragma unroll
            for (int j = 0; j < kCh; j += 2) {
              const float2 n = add_f32x2(make_float2(l[c0 + j], l[c0 + j + 1]), make_float2(x[j], x[j + 1]));
              l[c0 + j] = n.x;
              l[c0 + j + 1] = n.y;
            }
#pragma unroll
            for (int j = 0; j < kCh; j += 8) put_p(c0 + j, x + j);
          }
          if (__builtin_expect(!named_any(barid, 128, top > 8.f) || again, 1)) break;
          // ---- a maximum rose by more than 8: the block over, with new maxima.  Its share is taken out of the
          // sums again (what that rounds is scaled down with them: at most 2^-24 of the new sum) ----
#pragma unroll
          for (int c0 = 0; c0 < SUB; c0 += kCh) {
            load(c0, x);
            exponents(c0, x, top);
#pragma unroll
            for (int j = 0; j < kCh; ++j) l[c0 + j] -= fminf(exp2_approx(x[j]), kCap);
          }
          named_sync(barid, 128);  // (the old maxima have been read)
          fresh = again = true;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&S.s_free[sb]));
          mbar_arrive(smem_addr(&S.p_full[pb]));
        }
      }

      // ---- epilogue: column sums, then O ----
      // a lane's sums of all columns -> all lanes' sum of one column (32 columns: lane; 16: lane / 2):
      // each step halves the columns a lane keeps and adds the partner's for those
#pragma unroll
      for (int w = SUB / 2, bit = 16; bit > 0; w >>= 1, bit >>= 1) {
        const bool up = (lane & bit) != 0;
        if (w == 0) l[0] += __shfl_xor_sync(kAll, l[0], bit);
#pragma unroll
        for (int j = 0; j < w; ++j) {
          const float keep = up ? l[j + w] : l[j], give = up ? l[j] : l[j + w];
          l[j] = keep + __shfl_xor_sync(kAll, give, bit);
        }
      }
      if (SUB == 32 || (lane & 1) == 0) S.red[wq][h * SUB + (SUB == 32 ? lane : lane >> 1)] = l[0];
      tree_wait(&S.p_free[(g - 1) & 1], ((g - 1) >> 1) & 1, abort, p.status);
      tc_fence_after();
      named_sync(barid, 128);
      const bool whole = sg.blk0 == 0 && sg.blk1 == sg.nblk;
      const float vunit = S.vunit;
      // a cut item is the CTA's first (place 0) or its last (place 1)
      const long long place = ((long long)blockIdx.x * 2 + (sg.blk0 > 0 ? 0 : 1)) * NT;
      if (tok < SUB) {
        const int j = h * SUB + tok, col = sg.ch * NT + j;
        const float sum = (S.red[0][j] + S.red[1][j]) + (S.red[2][j] + S.red[3][j]);
        int row = -1;
        if (col < p.gh * p.N) {
          const int n = col / p.gh;
          row = (sg.b * p.N + n) * p.Hq + sg.h * p.gh + (col - n * p.gh);
          if (!whole) {
            p.ws_ml[(place + j) * 2] = sum == 0.f ? -INFINITY : -S.neg[j];
            p.ws_ml[(place + j) * 2 + 1] = sum;
          } else if (p.lse) {
            p.lse[row] = sum == 0.f ? -INFINITY : (log2f(sum) - S.neg[j]) * 0.69314718055994531f;
          }
        }
        S.row[j] = row;
        S.fall[j] = sum == 0.f ? 0.f : vunit / sum;
      }
      named_sync(barid, 128);
#pragma unroll 1
      for (int j0 = 0; j0 < SUB; j0 += 8) {
        float o[8];
        tc_ld8(tlane + Sh::kTmO + h * SUB + j0, o);
        tc_wait_ld(o);
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
          const int j = h * SUB + j0 + jj, row = S.row[j];
          if (row < 0) continue;
          if (!whole) p.ws_o[(place + j) * L.d + tok] = o[jj];
          else put_out(p, row, tok, S.fall[j] == 0.f ? 0.f : o[jj] * S.fall[j]);
        }
      }
      tc_fence_before();
      if (!whole) {
        // ---- the last CTA to finish the item merges its parts, in CTA order ----
        __threadfence();
        named_sync(5, kAllSm);
        const unsigned U = S.units, W = S.ctas, a0 = sg.item0, a1 = a0 + (unsigned)sg.nblk;
        // the CTAs whose ranges meet [a0, a1)
        const unsigned most = U / W + 1;  // units of a CTA, at most
        unsigned c0 = a0 / most, c1 = (a1 - 1) / most;
        while (tree_unit(U, W, c0 + 1) <= a0) ++c0;
        while (tree_unit(U, W, c1 + 1) <= a1 - 1) ++c1;
        if (th == 0) {
          unsigned* const ctr = p.counters + ((long long)sg.b * L.H + sg.h) * p.chunks + sg.ch;
          const unsigned n = atomicAdd(ctr, 1u);
          S.last = n + 1 == c1 - c0 + 1;
          if (S.last) *ctr = 0u;
        }
        named_sync(5, kAllSm);
        if (S.last) {
          __threadfence();
          const long long p0 = ((long long)c0 * 2 + (tree_unit(U, W, c0) > a0 ? 0 : 1)) * NT;  // (its first part)
          // each column's maximum and sum over the parts
          if (th < NT && S.row[th] >= 0) {
            float m = -INFINITY, sum = 0.f;
#pragma unroll 2
            for (unsigned cc = c0; cc <= c1; ++cc)
              m = fmaxf(m, __ldcg(p.ws_ml + ((cc == c0 ? p0 : (long long)cc * 2 * NT) + th) * 2));
            if (m != -INFINITY) {
#pragma unroll 2
              for (unsigned cc = c0; cc <= c1; ++cc) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + (cc == c0 ? p0 : (long long)cc * 2 * NT) + th);
                sum += ml.y * exp2_approx(ml.x - m);
              }
            }
            S.neg[th] = m == -INFINITY ? 0.f : -m;
            S.fall[th] = sum == 0.f ? 0.f : vunit / sum;
            if (p.lse) p.lse[S.row[th]] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
          }
          named_sync(5, kAllSm);
          // a warp per four columns, four channels a lane: their loads are in flight together
#pragma unroll 1
          for (int j = (warp - 8) * 4; j < NT; j += Sh::kSmWarps * 4) {
            float4 acc[4];
            float neg4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              neg4[k] = S.neg[j + k];
            }
#pragma unroll 2
            for (unsigned cc = c0; cc <= c1; ++cc) {
              const long long at = (cc == c0 ? p0 : (long long)cc * 2 * NT) + j;
              float4 o[4];
              float w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // (columns behind the last one: what lies there is not used)
                w[k] = __ldcg(p.ws_ml + (at + k) * 2);
                o[k] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + (at + k) * L.d) + lane);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float f = exp2_approx(w[k] + neg4[k]);
                if (w[k] == -INFINITY) continue;  // (no token of that part)
                acc[k].x = fmaf(o[k].x, f, acc[k].x);
                acc[k].y = fmaf(o[k].y, f, acc[k].y);
                acc[k].z = fmaf(o[k].z, f, acc[k].z);
                acc[k].w = fmaf(o[k].w, f, acc[k].w);
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = S.row[j + k];
              const float inv = S.fall[j + k];
              if (row < 0) continue;
              const float4 v = inv == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                          : make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
              const long long to = (long long)row * 32 + lane;  // in units of four channels
              if (p.out_bf16) reinterpret_cast<uint2*>(p.out)[to] = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
              else reinterpret_cast<float4*>(p.out)[to] = v;
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Sh::kIo + 1) tc_dealloc512(tm);
}

template <int FMT, int NT>
cudaError_t launch_tree_nt(const TreeParams& p, int ctas, int smem, cudaStream_t stream) {
  static std::mutex mu;
  static int set_for[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || set_for[dev] < smem) {
      e = cudaFuncSetAttribute(tree_kernel<FMT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      cudaFuncAttributes fa;  // the register split draws on what the launch brings
      e = cudaFuncGetAttributes(&fa, tree_kernel<FMT, NT>);
      if (e != cudaSuccess) return e;
      if (fa.numRegs < TreeShape<NT>::kRegLaunch) return cudaErrorInvalidConfiguration;
      if (dev >= 0 && dev < 64) set_for[dev] = smem;
    }
  }
  return launch_pdl(tree_kernel<FMT, NT>, dim3(ctas), dim3(TreeShape<NT>::kThreads), (size_t)smem, stream, p);
}

template <int FMT>
cudaError_t launch_tree_fmt(const TreeParams& p, int nt, int ctas, int smem, cudaStream_t stream) {
  switch (nt) {
    case 32: return launch_tree_nt<FMT, 32>(p, ctas, smem, stream);
    case 64: return launch_tree_nt<FMT, 64>(p, ctas, smem, stream);
    default: return launch_tree_nt<FMT, 128>(p, ctas, smem, stream);
  }
}

}  // namespace kvq
