// Head norms with rotary positions: queries (and keys) after their projection,
// one pass.  The attention calls take q normed and rotated ([S] eq. 5 applies
// RoPE_t(N_k(.)) to keys; the query side is the same map with its own gain):
//   y = x * rsqrt(mean_d x_d^2 + eps) * gain
//   (o_i, o_{i+64}) = (y_i cos a - y_{i+64} sin a, y_i sin a + y_{i+64} cos a),  a = p base^(-2i/128)
// per token at position p and per 128-wide head, half-split pairs.
//
// Bound by memory: 4 bytes per element (bf16 in and out) against about 10
// flops.  Half a warp owns a head: lane i of 16 holds elements 4i .. 4i+3 and
// their partners 64 + 4i .. 64 + 4i+3, so a pair never leaves its thread, every
// access is 8 bytes of a contiguous 128, and the mean is four shuffles.  The
// angles of a token are shared by all of its heads: a CTA forms them once, in
// turns p * (base^(-2i/128) / 2 pi) in 64 bits, drops the whole turns and calls
// sincospif on the rest, so a far position loses nothing to the range
// reduction.
#include <math.h>

#include "common.cuh"

namespace fsq {
namespace {

constexpr int kHalf = FSQ_HEAD_DIM / 2;
constexpr int kNT = 256;
constexpr int kSlots = kNT / 16;  // heads a CTA works on at once
constexpr int kUnroll = 4;        // heads of one half-warp whose loads are in flight together

struct NormRopeParams {
  double turn[kHalf];  // base^(-2i/128) / (2 pi)
  const uint16_t *x[2];
  uint16_t *y[2];
  int64_t ldx[2], ldy[2];
  const uint16_t *gain[2];
  int heads[2];
  int64_t n_tok, pos0;
  const int32_t *positions;
  float eps;
};

__device__ __forceinline__ float2 bf16x2_f32(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t f32_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// TT tokens per CTA (grid x), hpc heads of each (grid y).
template <int TT>
__global__ void __launch_bounds__(kNT) norm_rope_kernel(const __grid_constant__ NormRopeParams p, int hpc) {
  __shared__ float2 cs[TT][kHalf];  // (cos, sin)
  __shared__ __align__(16) float gain[2][FSQ_HEAD_DIM];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * TT;
  const int nt = (int)min((int64_t)TT, p.n_tok - t0);
  const int heads = p.heads[0] + p.heads[1];
  const int h0 = blockIdx.y * hpc, nh = min(hpc, heads - h0);
  pdl_wait();  // x may come from the kernel before this one
  {
    const int w = tid / FSQ_HEAD_DIM, d = tid % FSQ_HEAD_DIM;  // kNT == 2 * FSQ_HEAD_DIM
    gain[w][d] = p.gain[w] ? bf16_to_f32(p.gain[w][d]) : 1.f;
  }
  for (int i = tid; i < nt * kHalf; i += kNT) {
    const int t = i / kHalf, k = i % kHalf;
    const int64_t pos = p.pos0 + (p.positions ? (int64_t)p.positions[t0 + t] : t0 + t);
    double a = (double)pos * p.turn[k];
    a -= rint(a);
    float s, c;
    sincospif(2.f * (float)a, &s, &c);
    cs[t][k] = make_float2(c, s);
  }
  __syncthreads();
  const int slot = tid / 16, l = tid % 16;
  const int items = nt * nh;
  for (int i0 = slot; i0 < items; i0 += kSlots * kUnroll) {
    uint2 lo[kUnroll], hi[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int it = i0 + u * kSlots;
      lo[u] = hi[u] = make_uint2(0u, 0u);
      if (it < items) {
        const int t = it / nh, h = h0 + it % nh, w = h >= p.heads[0];
        const uint16_t *src = p.x[w] + (t0 + t) * p.ldx[w] + (int64_t)(w ? h - p.heads[0] : h) * FSQ_HEAD_DIM;
        lo[u] = *reinterpret_cast<const uint2 *>(src + 4 * l);
        hi[u] = *reinterpret_cast<const uint2 *>(src + kHalf + 4 * l);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int it = i0 + u * kSlots;
      const float2 a0 = bf16x2_f32(lo[u].x), a1 = bf16x2_f32(lo[u].y);
      const float2 b0 = bf16x2_f32(hi[u].x), b1 = bf16x2_f32(hi[u].y);
      float ss = a0.x * a0.x + a0.y * a0.y + a1.x * a1.x + a1.y * a1.y;
      ss += b0.x * b0.x + b0.y * b0.y + b1.x * b1.x + b1.y * b1.y;
#pragma unroll
      for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (it < items) {
        const int t = it / nh, h = h0 + it % nh, w = h >= p.heads[0];
        const float r = rsqrtf(fmaf(ss, 1.f / FSQ_HEAD_DIM, p.eps));
        const float4 ga = *reinterpret_cast<const float4 *>(&gain[w][4 * l]);
        const float4 gb = *reinterpret_cast<const float4 *>(&gain[w][kHalf + 4 * l]);
        const float4 c01 = *reinterpret_cast<const float4 *>(&cs[t][4 * l]);
        const float4 c23 = *reinterpret_cast<const float4 *>(&cs[t][4 * l + 2]);
        const float x0 = a0.x * r * ga.x, x1 = a0.y * r * ga.y, x2 = a1.x * r * ga.z, x3 = a1.y * r * ga.w;
        const float y0 = b0.x * r * gb.x, y1 = b0.y * r * gb.y, y2 = b1.x * r * gb.z, y3 = b1.y * r * gb.w;
        uint16_t *dst = p.y[w] + (t0 + t) * p.ldy[w] + (int64_t)(w ? h - p.heads[0] : h) * FSQ_HEAD_DIM;
        *reinterpret_cast<uint2 *>(dst + 4 * l) =
            make_uint2(f32_bf16x2(x0 * c01.x - y0 * c01.y, x1 * c01.z - y1 * c01.w),
                       f32_bf16x2(x2 * c23.x - y2 * c23.y, x3 * c23.z - y3 * c23.w));
        *reinterpret_cast<uint2 *>(dst + kHalf + 4 * l) =
            make_uint2(f32_bf16x2(x0 * c01.y + y0 * c01.x, x1 * c01.w + y1 * c01.z),
                       f32_bf16x2(x2 * c23.y + y2 * c23.x, x3 * c23.w + y3 * c23.z));
      }
    }
  }
}

constexpr int kTokBig = 8;  // tokens per CTA once they fill the SMs several times over

}  // namespace

cudaError_t launch_norm_rope(const uint16_t *q, int64_t ldq, int n_q, const uint16_t *q_gain, uint16_t *q_out,
                             int64_t ldqo, const uint16_t *k, int64_t ldk, int n_k, const uint16_t *k_gain,
                             uint16_t *k_out, int64_t ldko, int64_t n_tok, const int32_t *positions, int64_t pos0,
                             float eps, float rope_base, cudaStream_t st) {
  NormRopeParams p;
  double fine[8];  // base^(-2i/128) = base^(-16 (i / 8) / 128) base^(-2 (i % 8) / 128)
  for (int i = 0; i < 8; ++i) fine[i] = pow((double)rope_base, -2.0 * i / FSQ_HEAD_DIM);
  for (int i = 0; i < kHalf; i += 8) {
    const double coarse = pow((double)rope_base, -2.0 * i / FSQ_HEAD_DIM) / (2.0 * 3.14159265358979323846);
    for (int k = 0; k < 8; ++k) p.turn[i + k] = coarse * fine[k];
  }
  p.x[0] = q, p.x[1] = k;
  p.y[0] = q_out, p.y[1] = k_out;
  p.ldx[0] = ldq, p.ldx[1] = ldk;
  p.ldy[0] = ldqo, p.ldy[1] = ldko;
  p.gain[0] = q_gain, p.gain[1] = k_gain;
  p.heads[0] = n_q, p.heads[1] = n_k;
  p.n_tok = n_tok;
  p.pos0 = pos0;
  p.positions = positions;
  p.eps = eps;
  const int heads = n_q + n_k;
  if (n_tok >= (int64_t)kTokBig * kNumSMs)
    return launch_pdl(norm_rope_kernel<kTokBig>, dim3((unsigned)((n_tok + kTokBig - 1) / kTokBig)), dim3(kNT), 0, st,
                      p, heads);
  // few tokens: a CTA per token and 16 heads, so that the work spreads over the SMs
  return launch_pdl(norm_rope_kernel<1>, dim3((unsigned)n_tok, (unsigned)((heads + kSlots - 1) / kSlots)), dim3(kNT),
                    0, st, p, kSlots);
}

}  // namespace fsq
