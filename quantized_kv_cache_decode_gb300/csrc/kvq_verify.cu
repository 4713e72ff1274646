// Verification of drafted trees against the target's probabilities (sm_103a).
//
// From the root, with w = p (the target's row after the last accepted node) and W = 1,
// the children c of that node are tried in index order; token x is accepted when
//   u_c W q(x) < w(x),   and otherwise   w <- max(w - W q, 0),  W <- sum_x w(x)
// (q: the drafter's row, or all weight on x when the children were chosen).  That is
// rejection sampling against the remaining distribution w / W, kept unnormalised: the
// test and the final draw only need w and W to a common factor.  When no child is left
// the next token is the first x with cumsum(w)(x) > u_0 sum(w).
//
// The tests need single entries, which are read for all nodes at once up front; only a
// rejection and the final draw need whole rows.  One cluster of CTAs takes a sequence,
// each a contiguous slice of the vocabulary; the walk itself runs in every CTA alike
// (one thread's arithmetic on shared memory), and the slices' sums are exchanged through
// distributed shared memory.  Whether a token is drawn must not depend on rounding, so
// everything runs in pairs of fp32 numbers (hi + lo, about 45 bits), in a fixed order: one
// fp64 instruction holds a warp scheduler of this GPU for 64 cycles, a pair's sum for 10.
//
// Bound by latency: the first reads, one sum per rejection that a sibling follows and one for
// the draw, each a pass over the row's slices and a cluster barrier.  GB300: 32 sequences of 16
// nodes over 128256 tokens 40 us (the longest walk: three sums of 3 to 10 us), one chain of 6
// over 32000 tokens 10 us.
#include <cooperative_groups.h>

#include "kvq_common.cuh"

namespace kvq {
namespace cg = cooperative_groups;

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kMaxCluster = 8;
constexpr unsigned kAllLanes = 0xffffffffu;

// a + b of unevaluated pairs (hi + lo), about 45 bits
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  Two s = two_sum(a.hi, b.hi);
  const float lo = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo));
  const float hi = __fadd_rn(s.hi, lo);
  return Two{hi, __fsub_rn(lo, __fsub_rn(hi, s.hi))};
}
__device__ __forceinline__ Two mul(Two a, float b) {
  const float ph = __fmul_rn(a.hi, b), pl = __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -ph));
  const float hi = __fadd_rn(ph, pl);
  return Two{hi, __fsub_rn(pl, __fsub_rn(hi, ph))};
}
__device__ __forceinline__ bool less(Two a, Two b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ Two shfl_xor(Two a, int o) {
  return Two{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Two shfl(Two a, int lane) {
  return Two{__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
// sum over the lanes up to this one
__device__ __forceinline__ Two prefix(Two a, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two b{__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
    if (lane >= o) a = add(b, a);
  }
  return a;
}
// max(w - W q, 0)
__device__ __forceinline__ Two minus_part(Two w, Two W, float q) {
  const float ph = __fmul_rn(W.hi, q);
  const float pl = __fmaf_rn(W.lo, q, __fmaf_rn(W.hi, q, -ph));
  const Two r = add(w, Two{-ph, -pl});
  return r.hi > 0.f ? r : Two{0.f, 0.f};
}

constexpr int kRun = 1024;  // entries of a run: what a warp looks a token up in at a time

struct VerShared {
  int tok[64], par[64], path[64];
  float p[64], q[64], u[64];   // entries of the parent's rows at the node's token, the node's number
  Two W[64];                   // W before the r-th rejection at the current node
  int rejected[64];            // those nodes' tokens
  Two part[2][kMaxCluster];    // the cluster's slice sums (two buffers, used in turn)
  int at, n_rej, done;         // where the walk stands: the last accepted node, rejections there, no child left
  int owner;                   // slice that holds the next token, -1: none does
  Two before, want;            // the sum in front of that slice; what the running sum has to pass
  int sel, found;              // the owner's warp range that holds it; whether a run passed `want`
  Two warp[kVerWarps];
  Two run[kRun + 32];          // the weights of the run that holds the next token
};

// w at index x of the rows (target's entry p, drafter's q) after the first n_rej rejections
__device__ __forceinline__ Two weight(const VerShared& S, float p, float q, int x, bool drafted, int n_rej) {
  Two w{p, 0.f};
  if (n_rej == 0) return w;
  if (drafted) {
    // (W = 1 before the first one: an exact difference)
    w = two_sum(p, -q);
    if (!(w.hi > 0.f)) w = Two{0.f, 0.f};
    for (int r = 1; r < n_rej; ++r) w = minus_part(w, S.W[r], q);
  } else {
    for (int r = 0; r < n_rej; ++r)
      if (S.rejected[r] == x) w = minus_part(w, S.W[r], 1.f);
  }
  return w;
}

// Two running sums of pairs (packed fp32 operations, each rounded by itself): hi + w.hi exactly in two parts,
// the small one into lo, whose own roundings are 2^-48 of the sum
struct Sum2 {
  float2 hi, lo;
};
__device__ __forceinline__ void gather(Sum2& acc, float2 hi, float2 lo) {
  const float2 s = add_f32x2(acc.hi, hi), b = sub_f32x2(s, acc.hi);
  const float2 e = add_f32x2(sub_f32x2(acc.hi, sub_f32x2(s, b)), sub_f32x2(hi, b));
  acc.hi = s;
  acc.lo = add_f32x2(acc.lo, add_f32x2(e, lo));
}
// max(p - q, 0) into the sums: for p > q >= 0 the difference and what it rounds off are exact in three operations
__device__ __forceinline__ void gather_difference(Sum2& acc, float2 p, float2 q) {
  float2 hi = sub_f32x2(p, q), lo = sub_f32x2(sub_f32x2(p, hi), q);
  if (!(hi.x > 0.f)) hi.x = lo.x = 0.f;
  if (!(hi.y > 0.f)) hi.y = lo.y = 0.f;
  gather(acc, hi, lo);
}

// the same after n_rej rejections
__device__ __forceinline__ void remains(Sum2& acc, float2 p, float2 q, const VerShared& S, int n_rej) {
  float2 hi = sub_f32x2(p, q), lo = sub_f32x2(sub_f32x2(p, hi), q);
  if (!(hi.x > 0.f)) hi.x = lo.x = 0.f;
  if (!(hi.y > 0.f)) hi.y = lo.y = 0.f;
  for (int r = 1; r < n_rej; ++r) {  // minus_part, two entries at a time
    const Two W = S.W[r];
    const float2 Wh = make_float2(W.hi, W.hi), Wl = make_float2(W.lo, W.lo);
    const float2 ph = mul_f32x2(Wh, q), nph = make_float2(-ph.x, -ph.y);
    const float2 pl = fma_f32x2(Wl, q, fma_f32x2(Wh, q, nph));
    const float2 s = add_f32x2(hi, nph), b = sub_f32x2(s, hi);
    const float2 e = add_f32x2(sub_f32x2(hi, sub_f32x2(s, b)), sub_f32x2(nph, b));
    const float2 l = add_f32x2(e, sub_f32x2(lo, pl));
    hi = add_f32x2(s, l);
    lo = sub_f32x2(l, sub_f32x2(hi, s));
    if (!(hi.x > 0.f)) hi.x = lo.x = 0.f;
    if (!(hi.y > 0.f)) hi.y = lo.y = 0.f;
  }
  gather(acc, hi, lo);
}

// Sums of w: S.warp gets the CTA's warps' ranges, S.part[buf] all slices (behind a cluster barrier).
// A warp takes a contiguous range; its lanes hold every 32nd group of four entries, each component
// summed by itself (four independent chains), so loads are wide and in flight together.  No rejection and
// the first one of drawn children, the usual cases, have loops of their own.
__device__ void cluster_sum(VerShared& S, cg::cluster_group& cl, const float* tp, const float* dp, int lo, int hi,
                              int len, int n_rej, int& buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int a = min(lo + warp * len, hi), z = min(a + len, hi);
  const bool wide = ((reinterpret_cast<uintptr_t>(tp) | reinterpret_cast<uintptr_t>(dp)) & 15u) == 0;  // (a is a multiple of 4)
  const int n4 = wide ? (z - a) >> 2 : 0;
  const float4* t4 = reinterpret_cast<const float4*>(tp + a);
  const float4* d4 = reinterpret_cast<const float4*>(dp + a);
  Sum2 s[2] = {};
  if (n_rej == 0) {
    const float2 none = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int i = lane; i < n4; i += 32) {
      const float4 p = __ldg(t4 + i);
      gather(s[0], make_float2(p.x, p.y), none);
      gather(s[1], make_float2(p.z, p.w), none);
    }
  } else if (n_rej == 1 && dp) {
#pragma unroll 4
    for (int i = lane; i < n4; i += 32) {
      const float4 p = __ldg(t4 + i), q = __ldg(d4 + i);
      gather_difference(s[0], make_float2(p.x, p.y), make_float2(q.x, q.y));
      gather_difference(s[1], make_float2(p.z, p.w), make_float2(q.z, q.w));
    }
  } else if (dp) {
#pragma unroll 2
    for (int i = lane; i < n4; i += 32) {
      const float4 p = __ldg(t4 + i), q = __ldg(d4 + i);
      remains(s[0], make_float2(p.x, p.y), make_float2(q.x, q.y), S, n_rej);
      remains(s[1], make_float2(p.z, p.w), make_float2(q.z, q.w), S, n_rej);
    }
  } else {  // chosen children: only the rejected tokens' entries differ from the target's
#pragma unroll 4
    for (int i = lane; i < n4; i += 32) {
      const float4 p = __ldg(t4 + i);
      const int x = a + 4 * i;
      bool hit = false;
      for (int r = 0; r < n_rej; ++r) hit |= (S.rejected[r] >> 2) == (x >> 2);
      Two w[4] = {{p.x, 0.f}, {p.y, 0.f}, {p.z, 0.f}, {p.w, 0.f}};
      if (hit)
        for (int k = 0; k < 4; ++k) w[k] = weight(S, w[k].hi, 0.f, x + k, false, n_rej);
      gather(s[0], make_float2(w[0].hi, w[1].hi), make_float2(w[0].lo, w[1].lo));
      gather(s[1], make_float2(w[2].hi, w[3].hi), make_float2(w[2].lo, w[3].lo));
    }
  }
  // what wide loads do not cover: a tail below four entries, or rows that are not 16-byte aligned
#pragma unroll 4
  for (int x = a + 4 * n4 + lane; x < z; x += 32) {
    const Two w = weight(S, tp[x], dp && n_rej ? dp[x] : 0.f, x, dp != nullptr, n_rej);
    gather(s[0], make_float2(w.hi, 0.f), make_float2(w.lo, 0.f));
  }
  Two t = add(add(Two{s[0].hi.x, s[0].lo.x}, Two{s[0].hi.y, s[0].lo.y}), add(Two{s[1].hi.x, s[1].lo.x}, Two{s[1].hi.y, s[1].lo.y}));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t = add(t, shfl_xor(t, o));
  buf ^= 1;
  if (lane == 0) S.warp[warp] = t;
  __syncthreads();
  if (warp == 0) {
    Two v = lane < kVerWarps ? S.warp[lane] : Two{0.f, 0.f};
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = add(v, shfl_xor(v, o));
    v = shfl(v, 0);
    if (lane < (int)cl.num_blocks()) cl.map_shared_rank(&S, lane)->part[buf][cl.block_rank()] = v;
  }
  cl.sync();
}

// (two CTAs an SM: with one, a batch of 32 sequences takes two turns, 52 instead of 43 us)
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(const VerifyParams p) {
  __shared__ VerShared S;
  pdl_wait();
  pdl_trigger();
  cg::cluster_group cl = cg::this_cluster();
  const int n_cta = (int)cl.num_blocks(), me = (int)cl.block_rank();
  const int b = blockIdx.x / n_cta;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // contiguous slices and, within them, warps' ranges, all multiples of 4 but the last
  const int slice = ((p.V + n_cta - 1) / n_cta + 3) & ~3, len = ((slice + kVerWarps - 1) / kVerWarps + 3) & ~3;
  const int lo = min(me * slice, p.V), hi = min(lo + slice, p.V);
  const float* const trow = p.target + (long long)b * p.N * p.tstride;
  const float* const drow = p.draft ? p.draft + (long long)b * p.N * p.dstride : nullptr;
  if (tid == 0) S.path[0] = 0;
  if (tid < p.N) {
    const int tok = p.tokens[(long long)b * p.N + tid];
    int par = p.parents[(long long)b * p.N + tid];
    float tp = 0.f, dp = 1.f;
    bool bad = par < -1 || par >= tid;
    if (bad || tid == 0) par = -1;
    if (par >= 0) {
      if (tok < 0 || tok >= p.V) {
        bad = true;
        par = -1;
      } else {
        tp = trow[par * p.tstride + tok];
        if (drow) dp = drow[par * p.dstride + tok];
      }
    }
    if (bad && me == 0) report(p.status, KVQ_DEV_BAD_TREE);
    S.tok[tid] = tok;
    S.par[tid] = par;
    S.p[tid] = tp;
    S.q[tid] = dp;
    S.u[tid] = p.uniforms[(long long)b * p.N + tid];
  }
  cl.sync();  // (every CTA of the cluster runs before another writes to its shared memory)

  // ---- the walk: by one thread of every CTA, on the same numbers; all threads for the sums it asks for ----
  int n = 1, at = 0, count = 1, n_rej = 0, buf = 0;
  Two W{1.f, 0.f};
  bool redone = false, stale = false;  // stale: W is from before the last rejection
  while (true) {
    if (tid == 0) {
      bool sum = false;
      for (; n < p.N; ++n) {
        if (S.par[n] != at) continue;
        if (stale) {  // another child behind a rejected one
          sum = true;
          break;
        }
        bool accept;
        if (n_rej == 0) {  // W = 1: u q < p, exactly, from the product's two parts
          const float ph = __fmul_rn(S.u[n], S.q[n]), pl = __fmaf_rn(S.u[n], S.q[n], -ph);
          const Two d = two_sum(ph, -S.p[n]);
          accept = __fadd_rn(d.hi, __fadd_rn(d.lo, pl)) < 0.f;
        } else {
          // w at the node's token after the rejections so far
          Two w{S.p[n], 0.f};
          const float q = S.q[n];
          for (int r = 0; r < n_rej; ++r)
            if (drow || S.rejected[r] == S.tok[n]) w = minus_part(w, S.W[r], q);
          accept = less(mul(mul(W, q), S.u[n]), w);
        }
        if (accept) {
          S.path[count++] = n;
          at = n;
          n_rej = 0;
          W = Two{1.f, 0.f};
          stale = false;
        } else {
          S.W[n_rej] = W;
          S.rejected[n_rej++] = S.tok[n];
          stale = true;
        }
      }
      S.at = at;
      S.n_rej = n_rej;
      S.done = !sum;
    }
    __syncthreads();
    const int row = S.at, rej = S.n_rej;
    const bool done = S.done != 0;
    cluster_sum(S, cl, trow + row * p.tstride, drow ? drow + row * p.dstride : nullptr, lo, hi, len, rej, buf);
    if (tid == 0) {
      Two total{0.f, 0.f};
      for (int i = 0; i < n_cta; ++i) total = add(total, S.part[buf][i]);
      if (!done) {
        W = total;
        stale = false;
      } else {
        const bool fine = total.hi > 0.f && total.hi < 3e38f;
        S.owner = -1;
        if (!fine && rej > 0 && !redone) {  // nothing left: the target's row
          n_rej = 0;
          redone = true;
          S.owner = -2;
        } else if (fine) {
          // the slice in which the running sum passes `want`: the first, or the last with any weight
          const Two want = mul(total, S.u[0]);
          Two run{0.f, 0.f};
          for (int i = 0; i < n_cta; ++i) {
            const Two v = S.part[buf][i];
            if (v.hi > 0.f) {
              S.owner = i;
              S.before = run;
            }
            run = add(run, v);
            if (less(want, run)) break;
          }
          S.want = want;
        }
      }
    }
    __syncthreads();
    if (done && S.owner != -2) break;
  }

  // ---- the next token ----
  const float* const tp = trow + S.at * p.tstride;
  const float* const dp = drow ? drow + S.at * p.dstride : nullptr;
  n_rej = S.n_rej;
  const int owner = S.owner;
  if (tid == 0) S.par[0] = count;
  __syncthreads();
  if (tid < p.N && me == 0) p.path[(long long)b * p.N + tid] = tid < S.par[0] ? S.path[tid] : -1;
  if (tid == 0 && me == 0) {
    p.n_accepted[b] = count;
    if (owner < 0) {
      p.next_token[b] = -1;
      report(p.status, KVQ_DEV_BAD_PROBS);
    }
  }
  if (me == owner) {  // (uniform over the CTA)
    if (tid == 0) {
      Two run = S.before;
      const Two want = S.want;
      for (int i = 0; i < kVerWarps; ++i) {
        const Two s = S.warp[i];
        if (s.hi > 0.f) {
          S.sel = i;
          S.before = run;
        }
        run = add(run, s);
        if (less(want, run)) break;
      }
    }
    __syncthreads();
    // runs of 1024 entries of that warp's range: the first that passes `want`, else the last with any weight
    const int a = min(lo + S.sel * len, hi), z = min(a + len, hi);
    const Two want = S.want;
    int pick = -1;
    Two c = S.before;
    for (int r0 = a; r0 < z; r0 += kRun) {
#pragma unroll
      for (int i = 0; i < kRun / kVerThreads; ++i) {
        const int at = i * kVerThreads + tid, x = r0 + at;
        Two w{0.f, 0.f};
        if (x < z) w = weight(S, tp[x], dp && n_rej ? dp[x] : 0.f, x, dp != nullptr, n_rej);
        S.run[33 * (at >> 5) + lane] = w;
      }
      __syncthreads();
      if (warp == 0) {
        Two s{0.f, 0.f};  // a lane sums 32 neighbours
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
          s = add(s, S.run[33 * lane + i]);
        }
        const Two incl = prefix(s, lane);
        const unsigned has = __ballot_sync(kAllLanes, s.hi > 0.f);
        const unsigned past = __ballot_sync(kAllLanes, s.hi > 0.f && less(want, add(c, incl)));
        if (has) {
          // within 32 neighbours: the same among the lanes
          const int row = past ? __ffs(past) - 1 : 31 - __clz(has);
          const Two w = S.run[33 * row + lane];
          const Two base = row > 0 ? add(c, shfl(incl, row > 0 ? row - 1 : 0)) : c;
          const Two sum = add(base, prefix(w, lane));
          const unsigned any = __ballot_sync(kAllLanes, w.hi > 0.f);
          const unsigned over = __ballot_sync(kAllLanes, w.hi > 0.f && less(want, sum));
          pick = r0 + 32 * row + (over ? __ffs(over) - 1 : 31 - __clz(any));
        }
        c = add(c, shfl(incl, 31));
        if (lane == 0) S.found = past != 0;
      }
      __syncthreads();
      if (S.found) break;
    }
    if (tid == 0) p.next_token[b] = pick;
  }
  cl.sync();  // no CTA leaves while another may still write to its shared memory
}

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // CTAs of a sequence: as many as the GPU holds at once, slices of at least 2048 entries
  int n = kMaxCluster;
  while (n > 1 && ((long long)p.batch * n > 2LL * sms || p.V / n < 2048)) n /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * n));
  cfg.blockDim = dim3(kVerThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = n;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel, p);
}

}  // namespace kvq
