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
// distributed shared memory.  Whether a token is drawn must not depend on rounding: sums
// run in pairs of fp32 numbers (an fp64 sum of a row would be bound by the GPU's two fp64
// operations a clock and SM), thread sums are joined in a fixed order, and the few scalars
// are fp64.
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
// max(w - W q, 0)
__device__ __forceinline__ Two minus_part(Two w, Two W, float q) {
  const float ph = __fmul_rn(W.hi, q);
  const float pl = __fmaf_rn(W.lo, q, __fmaf_rn(W.hi, q, -ph));
  const Two r = add(w, Two{-ph, -pl});
  return r.hi > 0.f ? r : Two{0.f, 0.f};
}

struct VerShared {
  int tok[64], par[64], path[64];
  float p[64], q[64], u[64];   // entries of the parent's rows at the node's token, the node's number
  double W[64];                // W before the r-th rejection at the current node
  Two W2[64];
  int rejected[64];            // those nodes' tokens
  double part[2][kMaxCluster]; // the cluster's slice sums (two buffers, used in turn)
  double warp[kVerWarps];
  int last[kMaxCluster];       // highest index with w > 0 in each slice, or -1
  int n_rej, at;
};

// w at index x of the rows (p, q) after the first n_rej rejections
__device__ __forceinline__ Two weight(const VerShared& S, const float* tp, const float* dp, int x, int n_rej) {
  Two w{tp[x], 0.f};
  if (n_rej) {
    if (dp) {
      const float q = dp[x];
      for (int r = 0; r < n_rej; ++r) w = minus_part(w, S.W2[r], q);
    } else {
      for (int r = 0; r < n_rej; ++r)
        if (S.rejected[r] == x) w = minus_part(w, S.W2[r], 1.f);
    }
  }
  return w;
}

// Sum of w over the whole vocabulary; S.warp keeps the CTA's warp sums, S.part[buf] the slices'.
__device__ double cluster_sum(VerShared& S, cg::cluster_group& cl, const float* tp, const float* dp, int lo, int hi,
                              int n_rej, int& buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = (hi - lo + kVerWarps - 1) / kVerWarps;  // indices of a warp
  const int a = min(lo + warp * len, hi), z = min(a + len, hi);
  Two s{0.f, 0.f};
#pragma unroll 8
  for (int x = a + lane; x < z; x += 32) s = add(s, weight(S, tp, dp, x, n_rej));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Two b{__shfl_xor_sync(kAllLanes, s.hi, o), __shfl_xor_sync(kAllLanes, s.lo, o)};
    s = add(s, b);
  }
  buf ^= 1;
  if (lane == 0) S.warp[warp] = (double)s.hi + (double)s.lo;
  __syncthreads();
  const int n = (int)cl.num_blocks(), me = (int)cl.block_rank();
  if (threadIdx.x < (unsigned)n) {
    double t = 0.0;
    for (int i = 0; i < kVerWarps; ++i) t += S.warp[i];
    cl.map_shared_rank(&S, threadIdx.x)->part[buf][me] = t;
  }
  cl.sync();
  double t = 0.0;
  for (int i = 0; i < n; ++i) t += S.part[buf][i];
  return t;
}

__global__ void __launch_bounds__(kVerThreads) verify_kernel(const VerifyParams p) {
  __shared__ VerShared S;
  pdl_wait();
  pdl_trigger();
  cg::cluster_group cl = cg::this_cluster();
  const int n_cta = (int)cl.num_blocks(), me = (int)cl.block_rank();
  const int b = blockIdx.x / n_cta;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slice = (p.V + n_cta - 1) / n_cta;
  const int lo = min(me * slice, p.V), hi = min(lo + slice, p.V);
  const float* const trow = p.target + (long long)b * p.N * p.tstride;
  const float* const drow = p.draft ? p.draft + (long long)b * p.N * p.dstride : nullptr;
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

  // ---- the walk: the same in every thread of the cluster ----
  int at = 0, count = 1, n_rej = 0, buf = 0;
  double W = 1.0;
  if (tid == 0) S.path[0] = 0;
  for (int n = 1; n < p.N; ++n) {
    if (S.par[n] != at) continue;
    // w at the node's token after the rejections so far
    double w = S.p[n];
    const double q = S.q[n];
    for (int r = 0; r < n_rej; ++r)
      if (drow || S.rejected[r] == S.tok[n]) w = fmax(w - S.W[r] * q, 0.0);
    if ((double)S.u[n] * (W * q) < w) {
      if (tid == 0) S.path[count] = n;
      ++count;
      at = n;
      n_rej = 0;
      W = 1.0;
    } else {
      __syncthreads();  // (the lists of an earlier node have been read)
      if (tid == 0) {
        S.W[n_rej] = W;
        S.W2[n_rej] = Two{(float)W, (float)(W - (double)(float)W)};
        S.rejected[n_rej] = S.tok[n];
      }
      __syncthreads();
      ++n_rej;
      W = cluster_sum(S, cl, trow + at * p.tstride, drow ? drow + at * p.dstride : nullptr, lo, hi, n_rej, buf);
    }
  }

  // ---- the next token ----
  const float* const tp = trow + at * p.tstride;
  const float* const dp = drow ? drow + at * p.dstride : nullptr;
  double total = cluster_sum(S, cl, tp, dp, lo, hi, n_rej, buf);
  if (!(total > 0.0) || !(total < 1e300)) {  // nothing left (or no number): the target's row
    n_rej = 0;
    __syncthreads();
    total = cluster_sum(S, cl, tp, dp, lo, hi, 0, buf);
  }
  const bool none = !(total > 0.0) || !(total < 1e300);
  const double want = (double)S.u[0] * total;
  // the slice in which the running sum passes `want`: the first, or the last with any weight
  int owner = -1;
  double before = 0.0;
  {
    double run = 0.0;
    for (int i = 0; i < n_cta; ++i) {
      const double next = run + S.part[buf][i];
      if (S.part[buf][i] > 0.0) {
        owner = i;
        before = run;
      }
      if (next > want) break;
      run = next;
    }
  }
  if (tid < p.N && me == 0) p.path[(long long)b * p.N + tid] = tid < count ? S.path[tid] : -1;
  if (tid == 0 && me == 0) {
    p.n_accepted[b] = count;
    if (none) {
      p.next_token[b] = -1;
      report(p.status, KVQ_DEV_BAD_PROBS);
    }
  }
  if (!none && me == owner && warp == 0) {
    // the same among the slice's warps, then among the lanes of the warp's range, then in the lane's
    const int len = (hi - lo + kVerWarps - 1) / kVerWarps;
    int wsel = -1;
    double run = before, wbefore = before;
    for (int i = 0; i < kVerWarps; ++i) {
      const double s = S.warp[i];
      if (s > 0.0) {
        wsel = i;
        wbefore = run;
      }
      if (run + s > want) break;
      run += s;
    }
    const int a = min(lo + wsel * len, hi), z = min(a + len, hi);
    const int each = (z - a + 31) / 32;
    const int la = min(a + lane * each, z), lz = min(la + each, z);
    double s = 0.0;
    for (int x = la; x < lz; ++x) {
      const Two w = weight(S, tp, dp, x, n_rej);
      s += (double)w.hi + (double)w.lo;
    }
    double incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double v = __shfl_up_sync(kAllLanes, incl, o);
      if (lane >= o) incl += v;
    }
    const double mine = wbefore + (incl - s);
    const unsigned has = __ballot_sync(kAllLanes, s > 0.0);
    const unsigned past = __ballot_sync(kAllLanes, s > 0.0 && mine + s > want);
    const int sel = past ? __ffs(past) - 1 : 31 - __clz(has);
    if (lane == sel) {
      double c = mine;
      int pick = -1;
      for (int x = la; x < lz; ++x) {
        const Two w = weight(S, tp, dp, x, n_rej);
        const double v = (double)w.hi + (double)w.lo;
        if (v > 0.0) {
          pick = x;
          c += v;
          if (c > want) break;
        }
      }
      p.next_token[b] = pick;
    }
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
