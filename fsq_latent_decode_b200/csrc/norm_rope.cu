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
// angles of a token are shared by all of its heads and formed once, in turns
// p * (base^(-2i/128) / 2 pi) in 64 bits: without its whole turns the rest goes to
// sincospif, so a far position loses nothing to the range reduction.  The first
// heads are loaded before the angles are formed, the next before these are stored.
// The kernel may not let its dependents start early: the attention kernels behind
// it read the q that it writes before their own wait.
// Measured: 61 us for 16383 tokens of 40 heads read out of a fused projection (336
// MB: 5.5 TB/s, 84 % of the measured copy); one token of 40 heads 1.8 us.
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

// A warp works on one token, two heads at a time.  WIDE: a CTA has 8 tokens, a
// warp all heads of one.  Otherwise a CTA has 16 heads of one token (grid y), a
// warp two of them.
template <bool WIDE>
__global__ void __launch_bounds__(kNT) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int W = kNT / 32, TT = WIDE ? W : 1;
  __shared__ __align__(16) float2 cs[TT][kHalf];  // (cos, sin)
  __shared__ __align__(16) float gain[2][FSQ_HEAD_DIM];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t tok = (int64_t)blockIdx.x * TT + (WIDE ? warp : 0);
  const int heads = p.heads[0] + p.heads[1];
  const int l = lane % 16, side = lane / 16;  // the half-warp's head of a pair
  const int first = WIDE ? 0 : 2 * (blockIdx.y * W + warp), last = WIDE ? heads : min(heads, first + 2);
  constexpr int U = WIDE ? kUnroll : 1;
  const bool there = tok < p.n_tok;
  const uint16_t *x0 = p.x[0] + tok * p.ldx[0] + 4 * l, *x1 = p.x[1] + tok * p.ldx[1] + 4 * l - p.heads[0] * FSQ_HEAD_DIM;
  uint16_t *y0 = p.y[0] + tok * p.ldy[0] + 4 * l, *y1 = p.y[1] + tok * p.ldy[1] + 4 * l - p.heads[0] * FSQ_HEAD_DIM;
  uint2 lo[U], hi[U];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + 2 * u;
      lo[u] = hi[u] = make_uint2(0u, 0u);
      if (there && h < last) {
        const uint16_t *src = (h >= p.heads[0] ? x1 : x0) + h * FSQ_HEAD_DIM;
        lo[u] = *reinterpret_cast<const uint2 *>(src);
        hi[u] = *reinterpret_cast<const uint2 *>(src + kHalf);
      }
    }
  };
  pdl_wait();  // x may come from the kernel before this one
  load(first + side);
  {
    const int w = tid / FSQ_HEAD_DIM, d = tid % FSQ_HEAD_DIM;  // kNT == 2 * FSQ_HEAD_DIM
    gain[w][d] = p.gain[w] ? bf16_to_f32(p.gain[w][d]) : 1.f;
  }
  if (there)
    for (int k = WIDE ? lane : tid; k < kHalf; k += WIDE ? 32 : kNT) {
      const int64_t pos = p.pos0 + (p.positions ? (int64_t)p.positions[tok] : tok);
      double a = (double)pos * p.turn[k];
      a -= rint(a);
      float s, c;
      sincospif(2.f * (float)a, &s, &c);
      cs[WIDE ? warp : 0][k] = make_float2(c, s);
    }
  __syncthreads();
  if (!there) return;
  const float4 c01 = *reinterpret_cast<const float4 *>(&cs[WIDE ? warp : 0][4 * l]);
  const float4 c23 = *reinterpret_cast<const float4 *>(&cs[WIDE ? warp : 0][4 * l + 2]);
  for (int h0 = first + side; h0 - side < last; h0 += 2 * U) {
    uint2 ol[U], oh[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = h0 + 2 * u >= p.heads[0];
      const float2 a0 = bf16x2_f32(lo[u].x), a1 = bf16x2_f32(lo[u].y);
      const float2 b0 = bf16x2_f32(hi[u].x), b1 = bf16x2_f32(hi[u].y);
      float ss = a0.x * a0.x + a0.y * a0.y + a1.x * a1.x + a1.y * a1.y;
      ss += b0.x * b0.x + b0.y * b0.y + b1.x * b1.x + b1.y * b1.y;
#pragma unroll
      for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(fmaf(ss, 1.f / FSQ_HEAD_DIM, p.eps));
      const float4 ga = *reinterpret_cast<const float4 *>(&gain[w][4 * l]);
      const float4 gb = *reinterpret_cast<const float4 *>(&gain[w][kHalf + 4 * l]);
      const float x0 = a0.x * r * ga.x, x1 = a0.y * r * ga.y, x2 = a1.x * r * ga.z, x3 = a1.y * r * ga.w;
      const float y0 = b0.x * r * gb.x, y1 = b0.y * r * gb.y, y2 = b1.x * r * gb.z, y3 = b1.y * r * gb.w;
      ol[u] = make_uint2(f32_bf16x2(x0 * c01.x - y0 * c01.y, x1 * c01.z - y1 * c01.w),
                         f32_bf16x2(x2 * c23.x - y2 * c23.y, x3 * c23.z - y3 * c23.w));
      oh[u] = make_uint2(f32_bf16x2(x0 * c01.y + y0 * c01.x, x1 * c01.w + y1 * c01.z),
                         f32_bf16x2(x2 * c23.y + y2 * c23.x, x3 * c23.w + y3 * c23.z));
    }
    if (h0 - side + 2 * U < last) load(h0 + 2 * U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + 2 * u;
      if (h < last) {
        uint16_t *dst = (h >= p.heads[0] ? y1 : y0) + h * FSQ_HEAD_DIM;
        *reinterpret_cast<uint2 *>(dst) = ol[u];
        *reinterpret_cast<uint2 *>(dst + kHalf) = oh[u];
      }
    }
  }
}

constexpr int kWideFrom = 8 * kNumSMs;  // tokens from which CTAs of 8 fill the SMs

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
  if (n_tok >= kWideFrom)
    return launch_pdl(norm_rope_kernel<true>, dim3((unsigned)((n_tok + kNT / 32 - 1) / (kNT / 32))), dim3(kNT), 0, st, p);
  // few tokens: the heads of one over several CTAs, so that the work spreads over the SMs
  return launch_pdl(norm_rope_kernel<false>, dim3((unsigned)n_tok, (unsigned)((n_q + n_k + kSlots - 1) / kSlots)),
                    dim3(kNT), 0, st, p);
}

}  // namespace fsq
