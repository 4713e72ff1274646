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
// A CTA works on 128 cache tokens at a time ("block") and at most 2 * SUB columns, in
// two halves of SUB columns whose score, softmax and output steps alternate:
//   loader warp     cache bytes -> shared-memory slots (bulk copies; bf16 rows: cp.async)
//   dequant warps   slots -> K, V^T as f16 in tensor memory (two buffers each)
//   one MMA thread  the tcgen05.mma of both products
//   softmax warps   scores -> P (one warpgroup per half), running maximum and sum in fp32
// The blocks of all (sequence, kv head, column chunk) items are divided evenly over one
// CTA per SM; an item cut between CTAs is merged by the last CTA to finish it, in CTA
// order (the result does not depend on which one that is).
//
// Roundings: dequantized Keys and Values to f16 (codes of FP8 layers are exact in f16,
// their scale enters in fp32), queries bf16 -> f16 (exact from 2^-14 up), P to f16, each
// at most 2^-12 relative (2^-11 where half an f16 step is counted at the low end of a
// binade); everything else is fp32.  A running maximum that is stale by at most 2^8 in
// the exponent is kept (P then stays below 2^8, well inside f16).
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
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
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
// 16 lanes x 16 columns in fragment order: four 16 x 16 f16 fragments (4 registers each) side by side
__device__ __forceinline__ void tc_st_frag4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
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
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
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

template <int SUB>
struct TreeShape {
  // 64-column halves are bound by the softmax warps and need their registers; narrower ones by
  // the dequantization, which then gets a warpgroup for K and one for V
  static constexpr int kDq = SUB == 64 ? 4 : 8;
  static constexpr int kWarps = kDq + 8 + 4;  // (the last warpgroup: MMA, loader, two idle)
  static constexpr int kThreads = 32 * kWarps;
  // registers a thread: at launch, then by role (the roles' warpgroups together stay within the launch's)
  static constexpr int kRegLaunch = SUB == 64 ? 128 : 96;
  static constexpr int kRegDq = SUB == 64 ? 112 : 88, kRegSm = SUB == 64 ? 168 : 112, kRegIo = 64;
  static_assert(kDq / 4 * kRegDq + 2 * kRegSm + kRegIo <= (kWarps / 4) * kRegLaunch, "register split");
  static constexpr int kQBytes = SUB * 256;        // one half's queries (f16, two 64-channel halves)
  static constexpr int kPBytes = kBlk * SUB * 2;   // one half's P (f16, token rows)
  static constexpr int kFixed = 2 * kQBytes + 2 * kPBytes;
};

// tensor-memory columns
constexpr uint32_t kTmK = 0, kTmV = 128, kTmS = 256, kTmO = 384;

constexpr int kMaxSlots = 12;
constexpr long long kTreeWait = kWaitLimitCycles;

struct TreeSmem {  // small shared state, after the big buffers
  unsigned long long slot_full[kMaxSlots], slot_empty[kMaxSlots];
  unsigned long long k_full[2], k_empty[2], v_full[2], v_empty[2];
  unsigned long long s_full[2], s_free[2], p_full[2], p_free[2], q_full[2], drain;
  uint32_t slot_ok[kMaxSlots];  // quantized slots: which of the four tiles were copied
  uint32_t tmem;
  int abort;
  int last;      // merge: this CTA finished the item
  alignas(16) float m[2][64];   // running maximum of each column (log2 domain; 0 until one is set)
  alignas(16) float red[2][4][64];
  alignas(16) float rise[2][64], fall[2][64];  // change of the maxima and what it scales sums by
  int unset[2];
  unsigned long long anc[2][64];  // a node's ancestors and itself
  unsigned long long wild[2];     // nodes whose drafted Values f16 does not hold
  int par[2][64];
};

// One cut of an item: blocks [blk0, blk1) of (sequence b, kv head h, column chunk ch)
struct TreeSeg {
  int b, h, ch, blk0, blk1, nblk, nq, T;
  long long item0;  // first unit of the item
  TokenSplit ts;
};

// node n's ancestors and itself; par[n] < n, or -1
__device__ __forceinline__ unsigned long long tree_ancestors(const int* par, int n) {
  unsigned long long a = 0;
  for (; n >= 0; n = par[n]) a |= 1ull << n;
  return a;
}

struct TreeCursor {
  long long u, end;
  int b;
};

__device__ __forceinline__ TreeCursor tree_cursor(const TreeParams& p, const int* pre, long long lo, long long hi) {
  TreeCursor c;
  c.u = lo;
  c.end = hi;
  int a = 0, z = p.batch - 1;  // the last sequence whose first unit is <= lo
  const long long hc = (long long)p.L.H * p.chunks;
  while (a < z) {
    const int m = (a + z + 1) >> 1;
    if ((long long)pre[m] * hc <= lo) a = m;
    else z = m - 1;
  }
  c.b = a;
  return c;
}

__device__ __forceinline__ bool tree_next(const TreeParams& p, const int* pre, const int* lens, TreeCursor& c,
                                          TreeSeg& s) {
  if (c.u >= c.end) return false;
  const long long hc = (long long)p.L.H * p.chunks;
  while (c.b + 1 < p.batch && (long long)pre[c.b + 1] * hc <= c.u) ++c.b;
  s.b = c.b;
  s.nblk = pre[c.b + 1] - pre[c.b];
  const long long off = c.u - (long long)pre[c.b] * hc;
  const long long item = off / s.nblk;
  s.blk0 = (int)(off - item * s.nblk);
  s.h = (int)(item / p.chunks);
  s.ch = (int)(item - (long long)s.h * p.chunks);
  const long long left = c.end - c.u;
  s.blk1 = left < s.nblk - s.blk0 ? s.blk0 + (int)left : s.nblk;
  s.item0 = c.u - s.blk0;
  s.T = lens[c.b];
  s.ts = split_tokens(s.T, p.L);
  s.nq = (s.ts.qn + kBlk - 1) / kBlk;
  c.u += s.blk1 - s.blk0;
  return true;
}

// Wait for a barrier phase; false when the bound ran out here or elsewhere in the CTA.
__device__ __forceinline__ bool tree_wait(unsigned long long* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  const uint32_t a = smem_addr(bar);
  if (mbar_try_wait(a, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(a, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kTreeWait) {
      *abort = 1;
      report(status, KVQ_DEV_TIMEOUT);
      return false;
    }
  }
}

// ---------------------------------------------------------------------------
// dequantization of 16-token tiles to f16 operand fragments
// ---------------------------------------------------------------------------
// the code at bit OFF (< 23 - BITS) of w, exact in fp32: placed in the mantissa of 2^23, then
// (2^23 + code 2^OFF) 2^-OFF - 2^(23-OFF) in one exact fma
template <int BITS, int OFF>
__device__ __forceinline__ float2 codes_f32(uint32_t lo, uint32_t hi) {
  constexpr uint32_t kMask = ((1u << BITS) - 1u) << OFF;
  constexpr float kMul = 1.0f / (float)(1u << OFF), kAdd = -8388608.0f / (float)(1u << OFF);
  const float a = __uint_as_float(lop3_and_or(lo, kMask, 0x4B000000u));
  const float b = __uint_as_float(lop3_and_or(hi, kMask, 0x4B000000u));
  return fma_f32x2(make_float2(a, b), make_float2(kMul, kMul), make_float2(kAdd, kAdd));
}

// the code pair (half 0, half 1) of register REG of step s's fragment; w: the lane's operand words
template <int FMT, int REG>
__device__ __forceinline__ float2 frag_codes(const uint32_t* w, int s) {
  if constexpr (FMT == KVQ_FMT_INT4) {
    return codes_f32<4, 4 * REG>(w[s], w[s] >> 16);
  } else if constexpr (FMT == KVQ_FMT_INT2) {
    const uint32_t x = w[s >> 1];
    return (s & 1) ? codes_f32<2, 8 + 2 * REG>(x, x >> 16) : codes_f32<2, 2 * REG>(x, x >> 16);
  } else {
    const uint32_t x = w[2 * s + (REG >> 1)];
    return codes_f32<8, 0>(x >> (8 * (REG & 1)), x >> (8 * (REG & 1) + 16));
  }
}

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

// K fragments of steps 4i .. 4i+3 of a tile (rows = tokens; register pairs = channels 16s + 4q + {0,1}, {2,3})
template <int FMT>
__device__ __forceinline__ void k_frags(const uint32_t* w, const float* hdr, int i, int q, uint32_t (&r)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int s = 4 * i + j;
    if constexpr (TreeFmt<FMT>::kFp8) {
      fp8_pairs<FMT>(w[2 * s], r[4 * j], r[4 * j + 1]);
      fp8_pairs<FMT>(w[2 * s + 1], r[4 * j + 2], r[4 * j + 3]);
    } else {
      const float4 sc = *reinterpret_cast<const float4*>(hdr + 16 * s + 4 * q);
      const float4 z = *reinterpret_cast<const float4*>(hdr + 128 + 16 * s + 4 * q);
      const float2 s01 = make_float2(sc.x, sc.y), s23 = make_float2(sc.z, sc.w);
      const float2 n01 = make_float2(-sc.x * z.x, -sc.y * z.y), n23 = make_float2(-sc.z * z.z, -sc.w * z.w);
      const float2 a = fma_f32x2(frag_codes<FMT, 0>(w, s), s01, n01), b = fma_f32x2(frag_codes<FMT, 1>(w, s), s01, n01);
      const float2 c = fma_f32x2(frag_codes<FMT, 2>(w, s), s23, n23), d = fma_f32x2(frag_codes<FMT, 3>(w, s), s23, n23);
      r[4 * j] = pack_f16(a.x, a.y);
      r[4 * j + 1] = pack_f16(b.x, b.y);
      r[4 * j + 2] = pack_f16(c.x, c.y);
      r[4 * j + 3] = pack_f16(d.x, d.y);
    }
  }
}

// V^T fragment of step s (rows = channels 16s + .., register pairs = tokens 2q + {0,1}, then + 8)
template <int FMT>
__device__ __forceinline__ void v_frag(const uint32_t* w, int s, float4 sc, float4 nz, uint32_t* r) {
  if constexpr (TreeFmt<FMT>::kFp8) {
    fp8_pairs<FMT>(w[2 * s], r[0], r[1]);
    fp8_pairs<FMT>(w[2 * s + 1], r[2], r[3]);
    if constexpr (FMT == KVQ_FMT_FP8_E5M2) {  // units of 256 scales: exact, and leaves room above the codes
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = hfma2(r[i], 0x1C001C00u, 0x80008000u);
    }
  } else {
    const float2 s01 = make_float2(sc.x, sc.y), s23 = make_float2(sc.z, sc.w);
    const float2 n01 = make_float2(nz.x, nz.y), n23 = make_float2(nz.z, nz.w);
    const float2 a = fma_f32x2(frag_codes<FMT, 0>(w, s), s01, n01), b = fma_f32x2(frag_codes<FMT, 1>(w, s), s01, n01);
    const float2 c = fma_f32x2(frag_codes<FMT, 2>(w, s), s23, n23), d = fma_f32x2(frag_codes<FMT, 3>(w, s), s23, n23);
    r[0] = pack_f16(a.x, a.y);
    r[1] = pack_f16(b.x, b.y);
    r[2] = pack_f16(c.x, c.y);
    r[3] = pack_f16(d.x, d.y);
  }
}

// all operand words of the lane for one code matrix
template <int FMT>
__device__ __forceinline__ void load_words(const uint8_t* codes, int lane, uint32_t (&w)[TreeFmt<FMT>::kWords]) {
#pragma unroll
  for (int i = 0; i < TreeFmt<FMT>::kWords / 4; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(codes + (i * 32 + lane) * 16);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
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
template <int FMT, int SUB>
__global__ void __launch_bounds__(TreeShape<SUB>::kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  using Sh = TreeShape<SUB>;
  using F = TreeFmt<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const LayerDesc& L = p.L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* const Qs = smem;                      // [2 halves][SUB rows]
  uint8_t* const Ps = smem + 2 * Sh::kQBytes;    // [2 halves][128 tokens][SUB]
  uint8_t* const slots = smem + Sh::kFixed;
  TreeSmem& S = *reinterpret_cast<TreeSmem*>(slots + (size_t)p.nslots * p.slot_bytes);
  int* const pre = reinterpret_cast<int*>(&S + 1);  // [batch + 1] blocks before
  int* const lens = pre + p.batch + 1;                                               // [batch] tokens

  pdl_wait();
  pdl_trigger();

  // ---- set-up: barriers, tensor memory, the batch's block counts ----
  if (tid == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(smem_addr(&S.slot_full[i]), 32);
      mbar_init(smem_addr(&S.slot_empty[i]), Sh::kDq);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&S.k_full[i]), 4);
      mbar_init(smem_addr(&S.k_empty[i]), 1);
      mbar_init(smem_addr(&S.v_full[i]), 4);
      mbar_init(smem_addr(&S.v_empty[i]), 1);
      mbar_init(smem_addr(&S.s_full[i]), 1);
      mbar_init(smem_addr(&S.s_free[i]), 4);
      mbar_init(smem_addr(&S.p_full[i]), 4);
      mbar_init(smem_addr(&S.p_free[i]), 1);
      mbar_init(smem_addr(&S.q_full[i]), 4);
    }
    mbar_init(smem_addr(&S.drain), 1);
    S.abort = 0;
    S.unset[0] = S.unset[1] = 0;
    fence_barrier_init();
  }
  if (warp == Sh::kDq + 8) {
    tc_alloc512(smem_addr(&S.tmem));
    tc_relinquish();
  }
  for (int b = tid; b < p.batch; b += Sh::kThreads) {
    long long T = p.seq_lens[b];
    const long long cap = max_tokens(L);
    if (T > cap) {
      if (blockIdx.x == 0) report(p.status, KVQ_DEV_CAPACITY);
      T = cap;
    }
    if (T < 0) T = 0;
    const TokenSplit ts = split_tokens((int)T, L);
    lens[b] = (int)T;
    pre[b + 1] = (ts.qn + kBlk - 1) / kBlk + (ts.n_sink + ts.r + p.N + kBlk - 1) / kBlk;
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    if (lane == 0) pre[0] = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      int v = b0 + lane < p.batch ? pre[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (b0 + lane < p.batch) pre[b0 + lane + 1] = run + v;
      run += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = S.tmem;
  volatile int* const abort = &S.abort;

  const long long U = (long long)pre[p.batch] * L.H * p.chunks;
  const long long W = tree_ctas(gridDim.x, U);
  const long long cta = blockIdx.x;
  const long long lo = cta < W ? U * cta / W : U, hi = cta < W ? U * (cta + 1) / W : U;
  TreeCursor cur = tree_cursor(p, pre, lo, hi);
  TreeSeg sg;

  if (warp >= Sh::kDq + 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::kRegIo));
  else if (warp < Sh::kDq) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::kRegDq));
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Sh::kRegSm));

  if (warp == Sh::kDq + 9) {
    // ======================= loader =======================
    int slot = 0;
    uint32_t ph = 1;  // the first pass over the slots finds them empty
    int used = 0;
    bool ok = true;
    const __nv_bfloat16* sink[2] = {reinterpret_cast<const __nv_bfloat16*>(p.C.sink_k),
                                    reinterpret_cast<const __nv_bfloat16*>(p.C.sink_v)};
    const __nv_bfloat16* ring[2] = {reinterpret_cast<const __nv_bfloat16*>(p.C.resid_k),
                                    reinterpret_cast<const __nv_bfloat16*>(p.C.resid_v)};
    const __nv_bfloat16* draft[2] = {reinterpret_cast<const __nv_bfloat16*>(p.k_draft),
                                     reinterpret_cast<const __nv_bfloat16*>(p.v_draft)};
    while (ok && tree_next(p, pre, lens, cur, sg)) {
      const long long pair = (long long)sg.b * L.H + sg.h;
      for (int blk = sg.blk0; ok && blk < sg.blk1; ++blk) {
        if (blk < sg.nq) {
          const int ntile = (sg.ts.qn + 15) >> 4;
          for (int half = 0; half < 2; ++half) {
            if (!(ok = tree_wait(&S.slot_empty[slot], ph, abort, p.status))) break;
            const int t0 = blk * 8 + half * 4;
            // lane i < 4 owns tile t0 + i; a run of tiles of one record is one copy
            const int t = t0 + lane;
            uint32_t bytes = 0, hbytes = 0;
            const uint8_t* rec = nullptr;
            int run = 0, within = 0;
            if (lane < 4 && t < ntile) {
              const int r = t / L.tpg;
              within = t - r * L.tpg;
              if (lane == 0 || within == 0) {
                rec = record_addr(L, p.C, sg.b, sg.h, r, p.status);
                run = min(min(L.tpg - within, 4 - lane), ntile - t);
                if (rec) {
                  bytes = (uint32_t)(run * L.tile_bytes);
                  hbytes = (uint32_t)L.hdr_bytes;
                }
              }
            }
            uint32_t okmask = rec ? (((1u << run) - 1u) << lane) : 0u;
            okmask = __reduce_or_sync(0xffffffffu, okmask);
            const uint32_t total = __reduce_add_sync(0xffffffffu, bytes + hbytes);
            const uint32_t bar = smem_addr(&S.slot_full[slot]);
            uint8_t* const dst = slots + (size_t)slot * p.slot_bytes;
            if (lane == 0) {
              S.slot_ok[slot] = okmask;
              mbar_arrive_expect_tx(bar, total);
            }
            __syncwarp();
            if (rec) {
              if (hbytes) bulk_copy_g2s(smem_addr(dst + (t / L.tpg - t0 / L.tpg) * 1024), rec, hbytes, bar);
              bulk_copy_g2s(smem_addr(dst + p.slot_hdr + lane * L.tile_bytes),
                            rec + L.hdr_bytes + (long long)within * L.tile_bytes, bytes, bar);
            }
            if (lane != 0) mbar_arrive(bar);
            if (++slot == p.nslots) { slot = 0; ph ^= 1; }
            ++used;
          }
        } else {
          const int x0 = (blk - sg.nq) * kBlk;
          const int nsr = sg.ts.n_sink + sg.ts.r, nrow = nsr + p.N;
          for (int part = 0; part < kBlk; part += p.bf_tokens) {
            if (!(ok = tree_wait(&S.slot_empty[slot], ph, abort, p.status))) break;
            uint8_t* const dst = slots + (size_t)slot * p.slot_bytes;
            const int c = lane & 15;
#pragma unroll 4
            for (int i = 0; i < p.bf_tokens; ++i) {  // half-warps copy the K and the V row of a token
              const int kv = lane >> 4;
              const int x = x0 + part + i;
              const __nv_bfloat16* src = draft[kv];
              uint32_t n = 16;
              if (x < sg.ts.n_sink) src = sink[kv] + (pair * L.S + x) * L.d;
              else if (x < nsr) src = ring[kv] + (pair * L.W + (sg.ts.qn + (x - sg.ts.n_sink)) % L.W) * L.d;
              else if (x < nrow) src = draft[kv] + (pair * p.N + (x - nsr)) * L.d;
              else n = 0;  // rows behind the list: zeros
              const uint32_t to = smem_addr(dst) + (kv ? p.bf_tokens * 256 + vrow_chunk(i, c) : krow_chunk(i, c));
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src + c * 8), "r"(n)
                           : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                             smem_addr(&S.slot_full[slot]))
                         : "memory");
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
  } else if (warp == Sh::kDq + 8) {
    // ======================= MMA issue (one thread) =======================
    if (lane == 0) {
      constexpr uint32_t kIdQk = mma_idesc(SUB, 0), kIdPv = mma_idesc(SUB, 1);
      constexpr uint32_t kSwP = SUB == 64 ? 2 : (SUB == 32 ? 4 : 6);
      constexpr uint32_t kPRow = SUB * 2;
      uint64_t dq[2], dp[2];
      for (int h = 0; h < 2; ++h) {
        dq[h] = smem_desc(smem_addr(Qs + h * Sh::kQBytes), 16, 1024, 2);
        dp[h] = smem_desc(smem_addr(Ps + h * Sh::kPBytes), 8 * kPRow, 8 * kPRow, kSwP);
      }
      long long g = 0;  // blocks so far
      uint32_t nseg = 0;
      bool ok = true;
      while (ok && tree_next(p, pre, lens, cur, sg)) {
        const int nb = sg.blk1 - sg.blk0;
        for (int h = 0; h < 2 && ok; ++h) ok = tree_wait(&S.q_full[h], nseg & 1, abort, p.status);
        ++nseg;
        for (int i = 0; ok && i <= nb; ++i) {
          if (i < nb) {
            const int kb = (int)(g & 1);
            if (!(ok = tree_wait(&S.k_full[kb], (uint32_t)(g >> 1) & 1, abort, p.status))) break;
            for (int h = 0; h < 2; ++h) {
              if (g > 0 && !(ok = tree_wait(&S.s_free[h], (uint32_t)(g - 1) & 1, abort, p.status))) break;
              tc_fence_after();
#pragma unroll
              for (int s = 0; s < 8; ++s)
                tc_mma_ts(tm + kTmS + h * 64, tm + kTmK + kb * 64 + 8 * s,
                          dq[h] + (uint64_t)(((s >> 2) * SUB * 128 + (s & 3) * 32) >> 4), kIdQk, s > 0);
              tc_commit(smem_addr(&S.s_full[h]));
            }
            if (!ok) break;
            tc_commit(smem_addr(&S.k_empty[kb]));
          }
          if (i > 0) {
            const long long pg = g - 1;
            const int vb = (int)(pg & 1);
            if (!(ok = tree_wait(&S.v_full[vb], (uint32_t)(pg >> 1) & 1, abort, p.status))) break;
            for (int h = 0; h < 2; ++h) {
              if (!(ok = tree_wait(&S.p_full[h], (uint32_t)pg & 1, abort, p.status))) break;
              tc_fence_after();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                tc_mma_ts(tm + kTmO + h * 64, tm + kTmV + vb * 64 + 8 * j,
                          dp[h] + (uint64_t)((j * 16 * kPRow) >> 4), kIdPv, (i > 1 || j > 0) ? 1u : 0u);
              tc_commit(smem_addr(&S.p_free[h]));
            }
            if (!ok) break;
            tc_commit(smem_addr(&S.v_empty[vb]));
          }
          if (i < nb) ++g;
        }
      }
      if (!ok) {  // given up: let the products in flight end before the tensor memory is freed
        tc_commit(smem_addr(&S.drain));
        mbar_wait_bounded(smem_addr(&S.drain), 0, kTreeWait);
      }
    }
    __syncwarp();
  } else if (warp < Sh::kDq) {
    // ======================= dequantization =======================
    const int wq = warp & 3;                       // tensor-memory lanes 32 wq ..
    const bool doK = warp < 4, doV = Sh::kDq == 4 || warp >= 4;
    const int r = lane >> 2, q = lane & 3;
    const uint32_t tlane = tm + ((uint32_t)(32 * wq) << 16);
    int slot = 0;
    uint32_t ph = 0;
    long long g = 0;
    bool ok = true;
    uint32_t bad = 0;
    float vinv = 1.f;
    if constexpr (F::kFp8) vinv = 1.f / (*p.C.v_tscale * (FMT == KVQ_FMT_FP8_E5M2 ? 256.f : 1.f));
    while (ok && tree_next(p, pre, lens, cur, sg)) {
      for (int blk = sg.blk0; ok && blk < sg.blk1; ++blk, ++g) {
        const int buf = (int)(g & 1);
        const uint32_t eph = ((uint32_t)(g >> 1) & 1) ^ 1;  // the buffer's previous use has been read
        if (doK) ok = tree_wait(&S.k_empty[buf], eph, abort, p.status);
        if (ok && doV) ok = tree_wait(&S.v_empty[buf], eph, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tk = tlane + kTmK + buf * 64, tv = tlane + kTmV + buf * 64;
        if (blk < sg.nq) {
          for (int half = 0; half < 2; ++half) {
            if (!(ok = tree_wait(&S.slot_full[slot], ph, abort, p.status))) break;
            const uint8_t* const src = slots + (size_t)slot * p.slot_bytes;
            const uint32_t okmask = S.slot_ok[slot];
            const int t0 = blk * 8 + half * 4;
            if (doK && (wq >> 1) == half) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int ti = 2 * (wq & 1) + e;  // tile of the slot
                if ((okmask >> ti) & 1u) {
                  const float* hdr = nullptr;
                  if constexpr (!F::kFp8) {
                    hdr = reinterpret_cast<const float*>(src + ((t0 + ti) / L.tpg - t0 / L.tpg) * 1024);
                    // a Key beyond f16: its scale group says so
                    const float4 sc = *reinterpret_cast<const float4*>(hdr + 4 * lane);
                    const float4 z = *reinterpret_cast<const float4*>(hdr + 128 + 4 * lane);
                    constexpr float kL = (float)((1 << F::kBits) - 1);
                    const float m = fmaxf(fmaxf(fabsf(sc.x) * fmaxf(fabsf(z.x), fabsf(kL - z.x)),
                                                fabsf(sc.y) * fmaxf(fabsf(z.y), fabsf(kL - z.y))),
                                          fmaxf(fabsf(sc.z) * fmaxf(fabsf(z.z), fabsf(kL - z.z)),
                                                fabsf(sc.w) * fmaxf(fabsf(z.w), fabsf(kL - z.w))));
                    if (m >= 65520.f) bad = 1;
                  }
                  uint32_t w[F::kWords];
                  load_words<FMT>(src + p.slot_hdr + ti * L.tile_bytes, lane, w);
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    uint32_t f[16];
                    k_frags<FMT>(w, hdr, i, q, f);
                    tc_st_frag4(tk + ((uint32_t)(16 * e) << 16) + 32 * i, f);
                  }
                }
              }
            }
            if (doV) {
              const int ngv = F::kFp8 ? 1 : L.ngv;
#pragma unroll
              for (int e = 0; e < 2; ++e) {  // channels 32 wq + 16 e ..
                const int s = 2 * wq + e;
                uint32_t f[16];
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                  if ((okmask >> ti) & 1u) {
                    const uint8_t* tile = src + p.slot_hdr + ti * L.tile_bytes;
                    const uint8_t* codes = tile + 16 * F::kRb;
                    // the words of step s only
                    uint32_t w2[2];
                    if constexpr (F::kBits == 8) {
                      const uint2 v = *reinterpret_cast<const uint2*>(codes + ((s >> 1) * 32 + lane) * 16 + (s & 1) * 8);
                      w2[0] = v.x;
                      w2[1] = v.y;
                    } else if constexpr (F::kBits == 4) {
                      w2[0] = *reinterpret_cast<const uint32_t*>(codes + ((s >> 2) * 32 + lane) * 16 + (s & 3) * 4);
                    } else {
                      w2[0] = *reinterpret_cast<const uint32_t*>(codes + lane * 16 + (s >> 1) * 4) >> (8 * (s & 1));
                    }
                    float4 sc = make_float4(1.f, 1.f, 1.f, 1.f), nz = make_float4(0.f, 0.f, 0.f, 0.f);
                    if constexpr (!F::kFp8) {
                      const float* vs = reinterpret_cast<const float*>(tile + 32 * F::kRb) + (16 * s) / L.Gv;
                      const float* vz = vs + 16 * ngv;
                      sc = make_float4(vs[(2 * q) * ngv], vs[(2 * q + 1) * ngv], vs[(2 * q + 8) * ngv],
                                       vs[(2 * q + 9) * ngv]);
                      const float4 z = make_float4(vz[(2 * q) * ngv], vz[(2 * q + 1) * ngv], vz[(2 * q + 8) * ngv],
                                                   vz[(2 * q + 9) * ngv]);
                      nz = make_float4(-sc.x * z.x, -sc.y * z.y, -sc.z * z.z, -sc.w * z.w);
                      constexpr float kL = (float)((1 << F::kBits) - 1);
                      const float m = fmaxf(fmaxf(fmaxf(fabsf(nz.x), fabsf(fmaf(kL, sc.x, nz.x))),
                                                  fmaxf(fabsf(nz.y), fabsf(fmaf(kL, sc.y, nz.y)))),
                                            fmaxf(fmaxf(fabsf(nz.z), fabsf(fmaf(kL, sc.z, nz.z))),
                                                  fmaxf(fabsf(nz.w), fabsf(fmaf(kL, sc.w, nz.w)))));
                      if (m >= 65520.f) bad = 1;
                    }
                    v_frag<FMT>(w2, 0, sc, nz, f + 4 * ti);
                    if constexpr (F::kFp8) {
                      // tokens behind the last one of a partly filled tile: zeros whatever the store holds
                      const int nv = sg.ts.qn - 16 * (t0 + ti);
                      if (nv < 16) {
                        if (2 * q >= nv) f[4 * ti] = f[4 * ti + 1] = 0u;
                        else if (2 * q + 1 >= nv) { f[4 * ti] &= 0xFFFFu; f[4 * ti + 1] &= 0xFFFFu; }
                        if (2 * q + 8 >= nv) f[4 * ti + 2] = f[4 * ti + 3] = 0u;
                        else if (2 * q + 9 >= nv) { f[4 * ti + 2] &= 0xFFFFu; f[4 * ti + 3] &= 0xFFFFu; }
                      }
                    }
                  } else {  // not in the store (behind the last tile, or a bad block): P is 0 there, so V must be finite
                    f[4 * ti] = f[4 * ti + 1] = f[4 * ti + 2] = f[4 * ti + 3] = 0u;
                  }
                }
                tc_st_frag4(tv + ((uint32_t)(16 * e) << 16) + 32 * half, f);
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&S.slot_empty[slot]));
            if (++slot == p.nslots) { slot = 0; ph ^= 1; }
          }
        } else {
          uint32_t km = 0, vm = 0;
          const bool drafts = (blk - sg.nq) * kBlk + kBlk > sg.ts.n_sink + sg.ts.r;
          for (int part = 0; part < kBlk; part += p.bf_tokens) {
            if (!(ok = tree_wait(&S.slot_full[slot], ph, abort, p.status))) break;
            const uint8_t* const src = slots + (size_t)slot * p.slot_bytes;
            if (doK && 32 * wq >= part && 32 * wq < part + p.bf_tokens) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int row = 32 * wq - part + 16 * e + r;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t f[16];
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const int c = 2 * (4 * i + j) + (q >> 1);
                    const uint2 a = *reinterpret_cast<const uint2*>(src + krow_chunk(row, c) + (q & 1) * 8);
                    const uint2 b = *reinterpret_cast<const uint2*>(src + krow_chunk(row + 8, c) + (q & 1) * 8);
                    km = abs_max2(abs_max2(abs_max2(abs_max2(km, a.x), a.y), b.x), b.y);
                    f[4 * j] = bf16x2_to_f16x2(a.x);
                    f[4 * j + 1] = bf16x2_to_f16x2(b.x);
                    f[4 * j + 2] = bf16x2_to_f16x2(a.y);
                    f[4 * j + 3] = bf16x2_to_f16x2(b.y);
                  }
                  tc_st_frag4(tk + ((uint32_t)(16 * e) << 16) + 32 * i, f);
                }
              }
            }
            if (doV) {
              const uint32_t vbase = smem_addr(src) + p.bf_tokens * 256;
              const int row0 = (lane & 7) + ((lane >> 4) << 3), cc = (lane >> 3) & 1;
              for (int t4 = 0; t4 < p.bf_tokens; t4 += 32) {  // two fragments of 16 tokens at a time
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int c = 2 * (2 * wq + e) + cc;
                  uint32_t f[8];
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    uint32_t a[4];
                    ldmatrix_x4_trans(vbase + vrow_chunk(t4 + 16 * u + row0, c), a[0], a[1], a[2], a[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      vm = abs_max2(vm, a[i]);
                      uint32_t v = F::kFp8 ? bf16x2_to_f16x2(a[i], vinv) : bf16x2_to_f16x2(a[i]);
                      if (drafts) {
                        if ((v & 0x7C00u) == 0x7C00u) v &= 0xFFFF0000u;
                        if ((v & 0x7C000000u) == 0x7C000000u) v &= 0xFFFFu;
                      }
                      f[4 * u + i] = v;
                    }
                  }
                  asm volatile(
                      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                          tv + ((uint32_t)(16 * e) << 16) + ((part + t4) >> 1)),
                      "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3]), "r"(f[4]), "r"(f[5]), "r"(f[6]), "r"(f[7])
                      : "memory");
                }
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&S.slot_empty[slot]));
            if (++slot == p.nslots) { slot = 0; ph ^= 1; }
          }
          // a bf16 value that f16 does not hold (65504 is the last one)
          const float kx = __uint_as_float(max(km & 0xFFFFu, km >> 16) << 16);
          const float vx = __uint_as_float(max(vm & 0xFFFFu, vm >> 16) << 16) * fabsf(vinv);
          if (!(kx < 65520.f) || !(vx < 65520.f)) bad = 1;
        }
        if (!ok) break;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (doK) mbar_arrive(smem_addr(&S.k_full[buf]));
          if (doV) mbar_arrive(smem_addr(&S.v_full[buf]));
        }
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) report(p.status, KVQ_DEV_RANGE);
  } else if (warp < Sh::kDq + 8) {
    // ======================= softmax, epilogue =======================
    const int h = (warp - Sh::kDq) >> 2;    // column half
    const int tok = tid - 32 * Sh::kDq - 128 * h;  // 0 .. 127: the thread's tensor-memory lane
    const int wq = tok >> 5;
    const uint32_t tlane = tm + ((uint32_t)(32 * wq) << 16);
    const uint32_t ts_ = tlane + kTmS + h * 64, to_ = tlane + kTmO + h * 64;
    uint8_t* const Q = Qs + h * Sh::kQBytes;
    uint8_t* const P = Ps + h * Sh::kPBytes;
    float* const ms = S.m[h];
    const int barid = 1 + h;
    const float vunit = F::kFp8 ? *p.C.v_tscale * (FMT == KVQ_FMT_FP8_E5M2 ? 256.f : 1.f) : 1.f;
    const float cq = F::kFp8 ? p.scale_log2 * *p.C.k_tscale : p.scale_log2;
    long long g = 0;
    uint32_t bad = 0;
    while (tree_next(p, pre, lens, cur, sg)) {
      const int col0 = (sg.ch * 2 + h) * SUB;  // first column of this half
      const int C = p.gh * p.N;
      // ---- the drafted tokens, where this segment reaches a block of theirs ----
      const bool has_tree = sg.blk1 > sg.nq + (sg.ts.n_sink + sg.ts.r) / kBlk;
      bool wild = false;
      if (has_tree && tok < p.N) {
        int up = p.parents[(long long)sg.b * p.N + tok];
        if (up < -1 || up >= tok) {
          report(p.status, KVQ_DEV_BAD_TREE);
          up = -1;
        }
        S.par[h][tok] = up;
        // (its Values are replaced by zeros, see the dequantization: the nodes that do not see them
        // must not get 0 * NaN; the ones that do get NaN through P)
        const uint4* v = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.v_draft) +
                                                        (((long long)sg.b * L.H + sg.h) * p.N + tok) * L.d);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint4 a = v[i];
          m = abs_max2(abs_max2(abs_max2(abs_max2(m, a.x), a.y), a.z), a.w);
        }
        wild = !(__uint_as_float(max(m & 0xFFFFu, m >> 16) << 16) * fabsf(1.f / vunit) < 65520.f);
      }
      // ---- the half's queries, f16, channels in the Key fragments' order within every 16 ----
      for (int i = tok; i < SUB * 8; i += 128) {
        const int row = i >> 3, g16 = i & 7;
        const int col = col0 + row;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (col < C) {
          const int n = col / p.gh, hh = col - n * p.gh;
          const uint4* src = reinterpret_cast<const uint4*>(
              reinterpret_cast<const __nv_bfloat16*>(p.q) +
              (((long long)sg.b * p.N + n) * p.Hq + (long long)sg.h * p.gh + hh) * L.d + 16 * g16);
          a = src[0];
          b = src[1];
        }
        uint32_t m = abs_max2(abs_max2(abs_max2(abs_max2(0u, a.x), a.y), a.z), a.w);
        m = abs_max2(abs_max2(abs_max2(abs_max2(m, b.x), b.y), b.z), b.w);
        if (max(m & 0xFFFFu, m >> 16) >= 0x4780u) bad = 1;
        const uint4 lo4 = make_uint4(bf16x2_to_f16x2(a.x), bf16x2_to_f16x2(a.z), bf16x2_to_f16x2(b.x),
                                     bf16x2_to_f16x2(b.z));
        const uint4 hi4 = make_uint4(bf16x2_to_f16x2(a.y), bf16x2_to_f16x2(a.w), bf16x2_to_f16x2(b.y),
                                     bf16x2_to_f16x2(b.w));
        uint8_t* const dst = Q + (g16 >> 2) * (SUB * 128) + row * 128;
        const int c = 2 * (g16 & 3);
        *reinterpret_cast<uint4*>(dst + ((c ^ (row & 7)) << 4)) = lo4;
        *reinterpret_cast<uint4*>(dst + (((c + 1) ^ (row & 7)) << 4)) = hi4;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&S.q_full[h]));
      named_sync(barid, 128);  // (also: the previous segment's epilogue has read ms)
      if (tok < SUB) ms[tok] = 0.f;
      if (has_tree) {
        if (tok < p.N) S.anc[h][tok] = tree_ancestors(S.par[h], tok);
        if (tok < 64) {
          const uint32_t w = __ballot_sync(0xffffffffu, wild);
          if (lane == 0) reinterpret_cast<uint32_t*>(&S.wild[h])[wq] = w;
        }
      }
      named_sync(barid, 128);

      float l[SUB];
#pragma unroll
      for (int j = 0; j < SUB; ++j) l[j] = 0.f;
      bool unset = true;  // some column has no maximum yet (uniform over the warpgroup)
      bool has = false;   // column `tok` has one

      for (int blk = sg.blk0; blk < sg.blk1; ++blk, ++g) {
        const bool first = blk == sg.blk0;
        // which of the block's tokens count
        const bool quant = blk < sg.nq;
        bool valid = true, tree = false, spoilt = false;
        unsigned long long desc = 0;
        if (quant) {
          const int x = blk * kBlk + tok;
          valid = x < sg.ts.qn;
          if (L.paged && valid) {
            const int e = p.C.block_table[(long long)sg.b * L.mbps + x / L.P];
            valid = e >= 0 && e < L.num_blocks;
          }
        } else {
          const int nsr = sg.ts.n_sink + sg.ts.r;
          const int x = (blk - sg.nq) * kBlk + tok;
          valid = x < nsr;
          tree = (blk - sg.nq) * kBlk + kBlk > nsr;  // (uniform) drafted nodes in this block
          if (tree && !valid && x < nsr + p.N) {
            for (int n = x - nsr; n < p.N; ++n) desc |= ((S.anc[h][n] >> (x - nsr)) & 1ull) << n;
            spoilt = (S.wild[h] >> (x - nsr)) & 1ull;
            valid = true;
          } else if (valid) {
            desc = ~0ull;
          }
        }
        const float c = quant ? cq : p.scale_log2;
        tree_wait(&S.s_full[h], (uint32_t)g & 1, abort, p.status);
        tc_fence_after();
        float x[SUB];
#pragma unroll
        for (int j = 0; j < SUB; j += 16) tc_ld16(ts_ + j, x + j);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&S.s_free[h]));
        // x: the exponent (log2) relative to the column's maximum so far
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < SUB; j += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(ms + j);
          const float2 a = fma_f32x2(make_float2(x[j], x[j + 1]), make_float2(c, c), make_float2(-m4.x, -m4.y));
          const float2 b = fma_f32x2(make_float2(x[j + 2], x[j + 3]), make_float2(c, c), make_float2(-m4.z, -m4.w));
          x[j] = a.x;
          x[j + 1] = a.y;
          x[j + 2] = b.x;
          x[j + 3] = b.y;
        }
        if (__any_sync(0xffffffffu, !valid || tree)) {
          if (tree && valid) {
            int n = col0 / p.gh, k = col0 - n * p.gh;
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
              if (n < 64) {
                if (!((desc >> n) & 1ull)) x[j] = -INFINITY;
                else if (spoilt) x[j] = NAN;
              }
              if (++k == p.gh) { k = 0; ++n; }
            }
          }
          if (!valid) {
#pragma unroll
            for (int j = 0; j < SUB; ++j) x[j] = -INFINITY;
          }
        }
#pragma unroll
        for (int j = 0; j < SUB; ++j) top = fmaxf(top, x[j]);
        const bool slow = named_any(barid, 128, unset || !(top <= 8.f));
        // the product of the previous block has read P (and written O)
        if (g > 0) tree_wait(&S.p_free[h], (uint32_t)(g - 1) & 1, abort, p.status);
        if (slow) {
          // new column maxima over the block's 128 tokens
#pragma unroll
          for (int j = 0; j < SUB; ++j) {
            float v = x[j];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            if (lane == 0) S.red[h][wq][j] = v;
          }
          named_sync(barid, 128);
          if (tok < SUB) {
            // d: the block's maximum relative to the column's so far; its first one is taken as it is
            const float d = fmaxf(fmaxf(S.red[h][0][tok], S.red[h][1][tok]), fmaxf(S.red[h][2][tok], S.red[h][3][tok]));
            float rise = fmaxf(d, 0.f);
            if (!has) {
              has = d != -INFINITY;
              rise = has ? d : 0.f;
            }
            ms[tok] += rise;
            S.rise[h][tok] = rise;
            S.fall[h][tok] = exp2_approx(-rise);
            if (!has) S.unset[h] = 1;
          }
          named_sync(barid, 128);
          unset = S.unset[h] != 0;
#pragma unroll
          for (int j = 0; j < SUB; j += 4) {
            const float4 d = *reinterpret_cast<const float4*>(&S.rise[h][j]);
            const float4 f = *reinterpret_cast<const float4*>(&S.fall[h][j]);
            x[j] -= d.x;
            x[j + 1] -= d.y;
            x[j + 2] -= d.z;
            x[j + 3] -= d.w;
            l[j] = scaled(l[j], f.x);
            l[j + 1] = scaled(l[j + 1], f.y);
            l[j + 2] = scaled(l[j + 2], f.z);
            l[j + 3] = scaled(l[j + 3], f.w);
          }
          if (!first) {  // what O holds so far
            tc_fence_after();
#pragma unroll 1
            for (int j0 = 0; j0 < SUB; j0 += 8) {
              float o[8];
              tc_ld8(to_ + j0, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] = scaled(o[j], S.fall[h][j0 + j]);
              tc_st8(to_ + j0, o);
            }
            tc_wait_st();
          }
          named_sync(barid, 128);  // (rise, fall and unset have been read)
          if (tok == 0) S.unset[h] = 0;
        }
#pragma unroll
        for (int j = 0; j < SUB; j += 8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float a = exp2_approx(x[j + i]), b = exp2_approx(x[j + i + 1]);
            l[j + i] += a;
            l[j + i + 1] += b;
            w[i >> 1] = pack_f16(a, b);
          }
          const uint32_t at = (uint32_t)(tok * SUB * 2 + j * 2);
          constexpr uint32_t kM = SUB == 64 ? 7 : (SUB == 32 ? 3 : 1);
          *reinterpret_cast<uint4*>(P + (at ^ (((at >> 7) & kM) << 4))) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&S.p_full[h]));
      }

      // ---- epilogue: column sums, then O ----
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        float v = l[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) S.red[h][wq][j] = v;
      }
      tree_wait(&S.p_free[h], (uint32_t)(g - 1) & 1, abort, p.status);
      tc_fence_after();
      named_sync(barid, 128);
      const bool whole = sg.blk0 == 0 && sg.blk1 == sg.nblk;
      const int which = sg.blk0 > 0 ? 0 : 1;  // a cut item is the CTA's first (slot 0) or its last (slot 1)
      const long long slotid = cta * 2 + which;
      const int NT = 2 * SUB;
#pragma unroll 1
      for (int j0 = 0; j0 < SUB; j0 += 16) {
        float o[16];
        tc_ld16(to_ + j0, o);
        tc_wait_ld();
#pragma unroll
        for (int jj = 0; jj < 16; ++jj) {
          const int j = j0 + jj, col = col0 + j;
          const float sum = (S.red[h][0][j] + S.red[h][1][j]) + (S.red[h][2][j] + S.red[h][3][j]);
          if (col < C) {
            if (whole) {
              const int n = col / p.gh, hh = col - n * p.gh;
              const long long row = ((long long)sg.b * p.N + n) * p.Hq + (long long)sg.h * p.gh + hh;
              const float v = sum == 0.f ? 0.f : o[jj] * (vunit / sum);
              if (p.out_bf16) reinterpret_cast<__nv_bfloat16*>(p.out)[row * L.d + tok] = __float2bfloat16_rn(v);
              else reinterpret_cast<float*>(p.out)[row * L.d + tok] = v;
              if (p.lse && tok == 0)
                p.lse[row] = sum == 0.f ? -INFINITY : (ms[j] + log2f(sum)) * 0.69314718055994531f;
            } else {
              p.ws_o[(slotid * NT + h * SUB + j) * L.d + tok] = o[jj];
              if (tok == 0) {
                p.ws_ml[(slotid * NT + h * SUB + j) * 2] = sum == 0.f ? -INFINITY : ms[j];
                p.ws_ml[(slotid * NT + h * SUB + j) * 2 + 1] = sum;
              }
            }
          }
        }
      }
      tc_fence_before();
      if (!whole) {
        // ---- the last CTA to finish the item merges its parts, in CTA order ----
        __threadfence();
        named_sync(3, 256);
        const long long a0 = sg.item0, a1 = sg.item0 + sg.nblk;
        // the CTAs whose ranges meet [a0, a1)
        long long c0 = a0 * W / U, c1 = (a1 - 1) * W / U;
        while (U * (c0 + 1) / W <= a0) ++c0;
        while (U * c0 / W > a0) --c0;
        while (U * (c1 + 1) / W <= a1 - 1) ++c1;
        while (U * c1 / W > a1 - 1) --c1;
        unsigned* const ctr = p.counters + ((long long)sg.b * L.H + sg.h) * p.chunks + sg.ch;
        if (h == 0 && tok == 0) {
          const unsigned n = atomicAdd(ctr, 1u);
          S.last = n + 1 == (unsigned)(c1 - c0 + 1);
          if (S.last) *ctr = 0u;
        }
        named_sync(3, 256);
        if (S.last) {
          __threadfence();
          for (int j = 0; j < SUB; ++j) {
            const int col = col0 + j;
            if (col >= C) break;
            float m = -INFINITY, sum = 0.f, acc = 0.f;
            for (long long cc = c0; cc <= c1; ++cc) {
              const long long sl = (cc * 2 + (U * cc / W > a0 ? 0 : 1)) * NT + h * SUB + j;
              const float mi = __ldcg(p.ws_ml + sl * 2), li = __ldcg(p.ws_ml + sl * 2 + 1);
              if (mi == -INFINITY) continue;
              const float oi = __ldcg(p.ws_o + sl * L.d + tok);
              const float mn = fmaxf(m, mi);
              const float fa = m == -INFINITY ? 0.f : exp2_approx(m - mn), fb = exp2_approx(mi - mn);
              sum = sum * fa + li * fb;
              acc = acc * fa + oi * fb;
              m = mn;
            }
            const int n = col / p.gh, hh = col - n * p.gh;
            const long long row = ((long long)sg.b * p.N + n) * p.Hq + (long long)sg.h * p.gh + hh;
            const float v = sum == 0.f ? 0.f : acc * (vunit / sum);
            if (p.out_bf16) reinterpret_cast<__nv_bfloat16*>(p.out)[row * L.d + tok] = __float2bfloat16_rn(v);
            else reinterpret_cast<float*>(p.out)[row * L.d + tok] = v;
            if (p.lse && tok == 0)
              p.lse[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
          }
        }
      }
    }
    if (bad) report(p.status, KVQ_DEV_RANGE);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Sh::kDq + 8) tc_dealloc512(tm);
}

template <int FMT, int SUB>
cudaError_t launch_tree_sub(const TreeParams& p, int ctas, int smem, cudaStream_t stream) {
  static std::mutex mu;
  static int set_for[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || set_for[dev] < smem) {
      e = cudaFuncSetAttribute(tree_kernel<FMT, SUB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      cudaFuncAttributes fa;  // the register split draws on what the launch brings
      e = cudaFuncGetAttributes(&fa, tree_kernel<FMT, SUB>);
      if (e != cudaSuccess) return e;
      if (fa.numRegs < TreeShape<SUB>::kRegLaunch) return cudaErrorInvalidConfiguration;
      if (dev >= 0 && dev < 64) set_for[dev] = smem;
    }
  }
  return launch_pdl(tree_kernel<FMT, SUB>, dim3(ctas), dim3(TreeShape<SUB>::kThreads), (size_t)smem, stream, p);
}

template <int FMT>
cudaError_t launch_tree_fmt(const TreeParams& p, int sub, int ctas, int smem, cudaStream_t stream) {
  switch (sub) {
    case 16: return launch_tree_sub<FMT, 16>(p, ctas, smem, stream);
    case 32: return launch_tree_sub<FMT, 32>(p, ctas, smem, stream);
    default: return launch_tree_sub<FMT, 64>(p, ctas, smem, stream);
  }
}

}  // namespace kvq
