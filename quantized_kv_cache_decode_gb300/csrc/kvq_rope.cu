// Queries and keys of a fused projection, normed per head and rotated to their
// positions, keys and values laid out for the cache's append (sm_103a).
//
// "KV Cache Quantization Analysis", section 3 (Keys and RoPE): channel pair
// (i, i + 64) of a head is turned by t * base^(-2i/128) at position t.  Section 5:
// K and V go to the cache right after they are computed.
//   y = w x / sqrt(mean(x^2) + eps),  y'_i = y_i cos - y_{i+64} sin,  y'_{i+64} = y_{i+64} cos + y_i sin
//
// Bound by memory: every head is 256 bytes in and 256 bytes out.  Eight lanes hold a head,
// two 16-byte pieces each (channels 8j.. and 64 + 8j..: both halves of its eight pairs), so
// the sum of squares is three shuffles and the rotation none; a warp takes four heads at a
// time and loads the next four meanwhile.  The eight angles of a lane serve all heads of a
// token that its warp takes; a few tokens (a decode step) are spread over the SMs a warp per
// four heads instead.  GB300: 32768 tokens of 64 + 16 heads 224 us, 6.0 TB/s (0.88 of a
// measured copy); a step of 16 tokens 2.7 us in a captured graph.
#include "kvq_common.cuh"

namespace kvq {

constexpr int kRopeWarps = 8;

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// A warp takes `per` groups of four heads of one token, `parts` warps a token.
__global__ void __launch_bounds__(32 * kRopeWarps) norm_rope_kernel(const __grid_constant__ NormRopeParams p, int per,
                                                                    int parts) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, j = lane & 7, sub = lane >> 3;
  const long long task = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const long long row = task / parts;
  if (row >= p.rows) return;
  const int part = (int)(task - row * parts);
  const int heads = p.Hq + 2 * p.H, rotated = p.rotate_keys ? p.Hq + p.H : p.Hq;
  const int h0 = part * per * 4;
  const long long b = row / p.n_tokens;
  const int t = (int)(row - b * p.n_tokens);
  float cs[8], sn[8];
  if (p.rotate && h0 < rotated) {
    // the angle in turns is position * turn mod 1, in 64-bit fixed point: its top 32 bits, signed,
    // are the angle in units of 2^-31 half turns
    const unsigned long long pos = (unsigned long long)(long long)p.positions[row];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int top = (int)(uint32_t)((pos * p.turn[8 * j + i]) >> 32);
      sincospif((float)top * 4.656612873077393e-10f, &sn[i], &cs[i]);
    }
  }
  const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.qkv) + row * p.row_stride);
  const long long base = (b * p.H) * p.n_tokens + t;  // row of kv head 0 in k_out and v_out
  uint4 a = make_uint4(0, 0, 0, 0), c = a;
  auto load = [&](int g) {  // head h0 + 4 g + sub
    const int h = h0 + 4 * g + sub;
    if (g < per && h < heads) {
      a = __ldcs(src + h * 16 + j);
      c = __ldcs(src + h * 16 + 8 + j);
    }
  };
  load(0);
#pragma unroll 2
  for (int g = 0; g < per; ++g) {
    const int h = h0 + 4 * g + sub;
    const uint4 a0 = a, c0 = c;
    load(g + 1);  // the next heads on their way
    if (__all_sync(0xffffffffu, h >= heads)) break;
    const bool isq = h < p.Hq, isk = !isq && h < p.Hq + p.H;
    uint4 lo = a0, hi = c0;
    if (__any_sync(0xffffffffu, isq || isk)) {
      const uint4* w = reinterpret_cast<const uint4*>(isq ? p.q_weight : p.k_weight);
      float x[8], y[8];
      bf16x8_to_f32(a0, x);
      bf16x8_to_f32(c0, y);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      // squares that leave fp32 (bf16 does not end at 2^64): such a head's sum again, of values scaled
      // by a power of two that the quotient loses
      float mean = ss * (1.0f / 128.0f) + p.eps;
      const bool far = w && !(mean <= 0x1p100f && mean >= 0x1p-90f);
      if (__any_sync(0xffffffffu, far)) {
        const float s = !far ? 1.0f : (mean < 1.0f ? 0x1p100f : 0x1p-70f);
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= s;
          y[i] *= s;
          ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        mean = ss * (1.0f / 128.0f) + p.eps * s * s;
      }
      if (isq || isk) {
        if (w) {
          const float r = 1.0f / sqrtf(mean);
          float u[8], v[8];
          bf16x8_to_f32(__ldg(w + j), u);
          bf16x8_to_f32(__ldg(w + 8 + j), v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = x[i] * r * u[i];
            y[i] = y[i] * r * v[i];
          }
        }
        if (p.rotate && h < rotated) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float xi = x[i];
            x[i] = xi * cs[i] - y[i] * sn[i];
            y[i] = y[i] * cs[i] + xi * sn[i];
          }
        }
        lo = f32_to_bf16x8(x);
        hi = f32_to_bf16x8(y);
      }
    }
    if (h < heads) {
      uint4* dst;
      if (isq) {
        dst = reinterpret_cast<uint4*>(p.q_out) + (row * p.Hq + h) * 16;
      } else {
        const int hk = isk ? h - p.Hq : h - p.Hq - p.H;
        dst = reinterpret_cast<uint4*>(isk ? p.k_out : p.v_out) + (base + (long long)hk * p.n_tokens) * 16;
      }
      dst[j] = lo;
      dst[8 + j] = hi;
    }
  }
}

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
  const int groups = (p.Hq + 2 * p.H + 3) / 4;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // few tokens: a warp per four heads, so that all SMs take part; many: more heads per warp share the angles
  int parts = groups;
  while (parts > 1 && p.rows * (parts / 2) >= 32LL * sms) parts /= 2;
  const int per = (groups + parts - 1) / parts;
  parts = (groups + per - 1) / per;
  const long long blocks = (p.rows * parts + kRopeWarps - 1) / kRopeWarps;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  return launch_pdl(norm_rope_kernel, dim3((unsigned)blocks), dim3(32 * kRopeWarps), 0, stream, p, per, parts);
}

}  // namespace kvq
