// Absorbed queries for the tensor-core kernels that hold them in fp16: per (kv
// head j, batch row b) and head h of the group,
//   q'_h[g] = c sum_d W_k[j d_h + d][g] q_h[d],  c = scale log2 e.
// Bound by latency (64 KB of W_k per CTA at G = 256): a thread loads its
// coordinate pair's 32 rows of a quarter of the head dimension at once, the
// quarters meet in shared memory, and four warps per head take the head's
// largest weight, by whose power of two the caller scales.
#pragma once
#include <type_traits>

#include "common.cuh"

namespace fsq {
namespace tc {

constexpr int kAbsorbThreads = 512, kAbsorbHeads = 4;  // heads worked on together
constexpr int kAbsorbSlices = 4, kAbsorbRows = FSQ_HEAD_DIM / kAbsorbSlices;

template <int MAXG>
struct AbsorbSmem {
  float4 q[FSQ_HEAD_DIM];  // four heads of one d
  float part[kAbsorbSlices][kAbsorbHeads][MAXG];
  float top[kAbsorbHeads][4];
};

// store(h, g, v, e): head h (of the whole call), coordinate g, q' and the
// exponent of the head's largest weight (0 for a head of zeros and for one that
// is not finite, whose results are not finite either); for every g < Gs, 0 from
// G on.  scale(h, e) once per head; if store returns a float, scale(h, e, sum) with
// the head's sum of them.  Every thread of the CTA calls this.
template <int MAXG, class Store, class Scale>
__device__ __forceinline__ void absorb_heads(AbsorbSmem<MAXG> &sm, const uint16_t *__restrict__ q,
                                             const uint16_t *__restrict__ W_kv, int n_q, int n_kv, int G, int Gs,
                                             float c, int j, int64_t b, Store store, Scale scale) {
  constexpr int D = FSQ_HEAD_DIM;
  const int tid = threadIdx.x, lane = tid & 31;
  const int grp = n_q / n_kv;
  const int slice = tid / 128, cp = tid % 128;
  for (int h0 = 0; h0 < grp; h0 += kAbsorbHeads) {
    const int nh = min(kAbsorbHeads, grp - h0);
    // element (h, d) of the four heads; rows of missing heads are zero
    {
      const int h = tid / D, d = tid % D;
      reinterpret_cast<float *>(sm.q)[d * 4 + h] = h < nh ? bf16_to_f32(q[(b * n_q + j * grp + h0 + h) * D + d]) : 0.f;
    }
#pragma unroll 1
    for (int x0 = 0; x0 < G / 2; x0 += 128) {
      const int x = x0 + cp;
      const bool in = x < G / 2;
      uint32_t w[kAbsorbRows];
      const uint16_t *src = W_kv + ((int64_t)j * D + slice * kAbsorbRows) * G + 2 * x;
#pragma unroll
      for (int d = 0; d < kAbsorbRows; ++d) w[d] = in ? *reinterpret_cast<const uint32_t *>(src + (int64_t)d * G) : 0u;
      if (x0 == 0) __syncthreads();  // q, written while the first loads are on their way
      float v[kAbsorbHeads][2] = {};
#pragma unroll
      for (int d = 0; d < kAbsorbRows; ++d) {
        const float4 qv = sm.q[slice * kAbsorbRows + d];
        const float lo = __uint_as_float(w[d] << 16), hi = __uint_as_float(w[d] & 0xFFFF0000u);
        v[0][0] = fmaf(lo, qv.x, v[0][0]), v[0][1] = fmaf(hi, qv.x, v[0][1]);
        v[1][0] = fmaf(lo, qv.y, v[1][0]), v[1][1] = fmaf(hi, qv.y, v[1][1]);
        v[2][0] = fmaf(lo, qv.z, v[2][0]), v[2][1] = fmaf(hi, qv.z, v[2][1]);
        v[3][0] = fmaf(lo, qv.w, v[3][0]), v[3][1] = fmaf(hi, qv.w, v[3][1]);
      }
      if (in) {
#pragma unroll
        for (int h = 0; h < kAbsorbHeads; ++h)
          *reinterpret_cast<float2 *>(&sm.part[slice][h][2 * x]) = make_float2(v[h][0], v[h][1]);
      }
    }
    __syncthreads();
    // a head per 128 threads
    const int h = tid / 128, w4 = (tid / 32) % 4;
    constexpr int PER = (MAXG + 127) / 128;
    float v[PER], top = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int g = cp + 128 * i;
      v[i] = 0.f;
      if (g < G) {
        v[i] = c * ((sm.part[0][h][g] + sm.part[1][h][g]) + (sm.part[2][h][g] + sm.part[3][h][g]));
        top = fmaxf(top, fabsf(v[i]));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sm.top[h][w4] = top;
    __syncthreads();
    top = fmaxf(fmaxf(sm.top[h][0], sm.top[h][1]), fmaxf(sm.top[h][2], sm.top[h][3]));
    const int e = top > 0.f && top < INFINITY ? ilogbf(top) : 0;
    constexpr bool SUM = !std::is_void<decltype(store(0, 0, 0.f, 0))>::value;
    float sum = 0.f;
    if (h < nh) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int g = cp + 128 * i;
        if (g < Gs) {
          if constexpr (SUM) sum += store(j * grp + h0 + h, g, v[i], e);
          else store(j * grp + h0 + h, g, v[i], e);
        }
      }
    }
    if constexpr (SUM) {
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      __syncthreads();  // sm.top has been read
      if (lane == 0) sm.top[h][w4] = sum;
      __syncthreads();
      if (h < nh && cp == 0) scale(j * grp + h0 + h, e, (sm.top[h][0] + sm.top[h][1]) + (sm.top[h][2] + sm.top[h][3]));
    } else {
      if (h < nh && cp == 0) scale(j * grp + h0 + h, e);
    }
    __syncthreads();
  }
}

}  // namespace tc
}  // namespace fsq
