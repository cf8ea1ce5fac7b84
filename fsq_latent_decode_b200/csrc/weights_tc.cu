// Attention weight of every cached token, summed over the query heads and added
// to a running total (what an eviction ranks tokens by):
//   acc[b][t] += sum_h softmax_t(scale q_h . W_k z_t)
//
// The weights need each head's log-sum-exp over the whole row first, so the
// scores are formed twice, by the same kernel in two modes: kLse leaves (max,
// sum) per split and head, kAdd folds those and adds the weights.  Storing the
// scores instead would cost 8 n_q bytes per token, more than a code row.
// kAdd goes through its tiles backwards: the last codes of the first pass are
// still in L2.
//
// The result is a running fp32 sum over many steps, so scores are exact to fp32:
// Q' = W_k^T q * scale * log2 e is held as two fp16 terms per head (22 bits),
// scaled by a power of two, against exact fp16 levels.
//   S [128 tokens x 2 n_q] = Z [128 x G] . [Q'_hi ; Q'_lo]^T      score = S_hi + S_lo
// A token is a TMEM lane, so a softmax thread owns its tokens: kLse keeps
// (reference, sum) per head and thread, the first token's score as the
// reference, moved only when a score exceeds it by 2^64; no exchange until the
// split ends.  kAdd sums a token's heads in one thread.
//
// Bound by memory: R bytes of codes per token and pass (kAdd: 8 bytes of acc
// more).  Per 128-token tile: the packed rows come by TMA as 128-byte rows in
// swizzled order (rows of whole 16-byte pieces; a thread then reads its own
// token without bank conflicts) or by a plain bulk copy; each dequantising
// thread unpacks its token's row into Z in TMEM, the A operand (read from shared
// memory, A would take twice its bandwidth); B is Q' in shared memory.
//
// Warps: 0 copies, 1 issues the MMAs, 4-7 and 8-11 take the scores of every other
// 8 heads, 12-19 (12-15 with many heads) dequantise.  Every wait is bounded (FSQ_ERR_TIMEOUT).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include <mutex>

#include "common.cuh"
#include "f16_codes.cuh"
#include "query_f16.cuh"
#include "tc_decode.cuh"
#include "tc_ptx.cuh"

namespace fsq {
namespace tc {
namespace weights {

constexpr int kTile = 128;
// Dequantising warps: eight, two per TMEM quarter, where a score thread keeps few
// heads (640 threads have at most 96 registers each), else four.
template <int NC>
struct Shape {
  static constexpr int DQ = NC <= 2 ? 8 : 4, THREADS = (12 + DQ) * 32;
};
constexpr int kAtom = 64;
constexpr int kMaxQ = 64;             // query heads
constexpr int kMaxStages = 8, kMaxZ = 4, kMaxS = 4;
constexpr int kMiscBytes = 4096;
constexpr size_t kSmemMax = 227 * 1024;
constexpr int kTop = 12;              // Q' is scaled to a largest weight of 2^12 .. 2^13: its lo terms stay normal
constexpr float kFar = 64.f;          // a score above the reference by more than 2^64 moves it
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainNs = 1000000000ull;
enum Mode { kLse, kAdd };

struct Plan {
  int Gp, NA, R, N, stages, nz, ns;  // N: score columns (16 per 8 heads)
  bool tma;
  uint32_t q_bytes, stage_bytes, off_misc, total, col_s;
};
__host__ __device__ inline Plan plan_of(int n_q, int G, int bits) {
  Plan p;
  p.Gp = (G + 15) / 16 * 16;
  p.NA = (G + kAtom - 1) / kAtom;
  p.R = G * bits / 8;
  p.N = (n_q + 7) / 8 * 16;
  p.tma = p.R % 16 == 0;
  p.q_bytes = (uint32_t)(p.NA * p.N * 128);
  // (+16: without TMA, a token's last group may read past its row)
  p.stage_bytes = (uint32_t)(kTile * p.R + (p.tma ? 0 : 16) + 1023) / 1024 * 1024;
  p.stages = (int)((kSmemMax - kMiscBytes - p.q_bytes) / p.stage_bytes);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.off_misc = p.q_bytes + p.stages * p.stage_bytes;
  p.total = p.off_misc + kMiscBytes;
  // TMEM: Z buffers of Gp / 2 columns from 0, S buffers of N columns behind them
  const int zc = p.Gp / 2;
  p.nz = (512 - (zc + 2 * p.N <= 512 ? 2 : 1) * p.N) / zc;
  if (p.nz > kMaxZ) p.nz = kMaxZ;
  p.col_s = p.nz * zc;
  p.ns = (int)(512 - p.col_s) / p.N;
  if (p.ns > kMaxS) p.ns = kMaxS;
  return p;
}

// TMA boxes of a tile of R 128-byte lines: at most 256 lines each, whole swizzle
// atoms of 8.  R is a multiple of 16, so boxes of 8 lines always serve.
__host__ __device__ inline int boxes_of(int R) {
  for (int n = 1; n < R / 8; ++n)
    if (R % (8 * n) == 0 && R / n <= 256) return n;
  return R / 8;
}

struct Params {
  const uint8_t *codes;
  int64_t bstride, T;
  const int32_t *seq_lens;
  const uint8_t *qbuf;   // per batch row: Q' in the score MMA's B layout
  const float *sig;      // [B][n_q] score scales
  float2 *part;          // [B][S][n_q] (max, sum) per split
  float *acc;
  int64_t acc_stride;
  uint32_t *err;
  int n_q, G, S, k;      // splits per row, tiles per split
  uint32_t stall_ns;
};

struct Misc {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t z_ready[kMaxZ], z_free[kMaxZ], s_full[kMaxS], s_free[kMaxS];
  uint64_t q_full, done, never;
  uint32_t tmem_base, abort;
  __align__(16) float sig[kMaxQ];
  __align__(16) float neg[kMaxQ];  // kAdd: -(log-sum-exp)
  union {
    float2 red[4][kMaxQ];          // kLse: per quarter of the lanes
    float sum[2][kTile];           // kAdd: the second group's share of a token
  };
};
static_assert(sizeof(Misc) <= kMiscBytes, "Misc block exceeds its reservation");

// Pieces [first, pieces) of one token's row -> Z columns; load(u) gives the 16 bytes of piece u.
template <int BITS, class F>
__device__ __forceinline__ void fill_pieces(uint32_t z, int first, int pieces, F load) {
  constexpr int PER = 128 / BITS / 2;  // columns of a piece: 8, 16, 32
#pragma unroll 1
  for (int u0 = first; u0 < pieces; u0 += 4) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u0 + u < pieces) v[u] = load(u0 + u);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (u0 + u >= pieces) break;
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint32_t o[PER];
#pragma unroll
      for (int e = 0; e < PER / 4; ++e) {
        uint4 l;
        if constexpr (BITS == 8) l = levels8<8>(w[2 * e], w[2 * e + 1]);
        else if constexpr (BITS == 4) l = levels8<4>(w[e], 0u);
        else l = levels8<2>(w[e / 2] >> (16 * (e & 1)), 0u);
        o[4 * e] = l.x, o[4 * e + 1] = l.y, o[4 * e + 2] = l.z, o[4 * e + 3] = l.w;
      }
      const uint32_t at = z + (u0 + u) * PER;
      if constexpr (PER == 8) tmem_st8(at, o);
      else if constexpr (PER == 16) tmem_st16(at, o);
      else tmem_st32(at, o);
    }
  }
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint4 v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// NC: 8-head chunks a score thread takes (of every other chunk)
template <int BITS, int NC, Mode MODE>
__global__ void __launch_bounds__(Shape<NC>::THREADS, 1) weights_split_tc(const __grid_constant__ CUtensorMap tmap, Params p) {
  constexpr int kDqWarps = Shape<NC>::DQ;
  const Plan pl = plan_of(p.n_q, p.G, BITS);
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc &ms = *reinterpret_cast<Misc *>(smem + pl.off_misc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.G, Gp = pl.Gp, NA = pl.NA, R = pl.R, N = pl.N, stages = pl.stages, nz = pl.nz, ns = pl.ns, n_q = p.n_q;
  const int split = blockIdx.x;
  const int64_t b = blockIdx.y;
  // the query prologue has waited for whatever wrote the codes and the lengths
  pdl_wait();
  const int64_t t0 = (int64_t)split * p.k * kTile;
  const int64_t t1 = min(row_len(p.seq_lens, b, p.T, p.err, MODE == kLse && split == 0 && tid == 0),
                         t0 + (int64_t)p.k * kTile);
  float2 *part = p.part + (b * p.S + split) * n_q;
  if (t1 <= t0) {  // wholly behind the row's length
    if (MODE == kLse && tid < n_q) part[tid] = make_float2(-INFINITY, 0.f);
    return;
  }
  // a first pass that gave up leaves no sums to divide by: nothing is added
  if (MODE == kAdd && __syncthreads_or(*p.err == (uint32_t)(-FSQ_ERR_TIMEOUT))) return;
  const int n_tiles = (int)((t1 - t0 + kTile - 1) / kTile);
  auto tile_of = [&](int i) { return MODE == kAdd ? n_tiles - 1 - i : i; };
  auto rows_of = [&](int i) { return (int)min((int64_t)kTile, t1 - t0 - (int64_t)tile_of(i) * kTile); };
  const uint8_t *src = p.codes + b * p.bstride + t0 * R;
  volatile uint32_t *abort = &ms.abort;
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&ms.full[i], 1);
      mbar_init(&ms.empty[i], kDqWarps);
    }
    for (int i = 0; i < kMaxZ; ++i) {
      mbar_init(&ms.z_ready[i], kDqWarps);
      mbar_init(&ms.z_free[i], 1);
    }
    for (int i = 0; i < kMaxS; ++i) {
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.s_free[i], 8);
    }
    mbar_init(&ms.q_full, 1);
    mbar_init(&ms.done, 1);
    mbar_init(&ms.never, 1);  // completed by nothing: the test-only stall waits on it
    ms.abort = 0u;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&ms.tmem_base, 512);
    tmem_relinquish();
  }
  if (tid < n_q) ms.sig[tid] = p.sig[b * n_q + tid];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tm = 0;  // all 512 columns are this CTA's
  if (MODE == kLse) pdl_trigger();
  auto fail = [&]() {
    record_error(p.err, FSQ_ERR_TIMEOUT);
    *abort = 1u;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = l2_evict_normal();
    if (lane == 0) {
      mbar_arrive_expect_tx(&ms.q_full, pl.q_bytes);
      bulk_g2s(smem, p.qbuf + (size_t)b * pl.q_bytes, pl.q_bytes, &ms.q_full);
    }
    bool ok = true;
    const int boxes = pl.tma ? boxes_of(R) : 0;
    int issued = 0;
    Ring c;
    for (int i = 0; i < n_tiles; ++i, c.next(stages)) {
      if (!warp_wait(&ms.empty[c.slot], c.par ^ 1u, abort, kWaitNs)) {
        ok = false;
        break;
      }
      uint8_t *dst = smem + pl.q_bytes + c.slot * pl.stage_bytes;
      if (lane == 0) {
        if (rows_of(i) < kTile) {
          mbar_arrive(&ms.full[c.slot]);  // the dequantising threads read a ragged tile themselves
        } else {
          mbar_arrive_expect_tx(&ms.full[c.slot], (uint32_t)(kTile * R));
          if (pl.tma) {
            const int row0 = (int)(t0 / kTile + tile_of(i)) * R;
            for (int x = 0; x < boxes; ++x)
              tma_load_3d(dst + x * (R / boxes) * 128, &tmap, 0, row0 + x * (R / boxes), (int)b, &ms.full[c.slot], pol);
          } else {
            bulk_g2s_hint(dst, src + (int64_t)tile_of(i) * kTile * R, (uint32_t)(kTile * R), &ms.full[c.slot], pol);
          }
        }
      }
      issued = i + 1;
    }
    if (!ok) {
      if (lane == 0) fail();
      for (int i = max(0, issued - stages); i < issued; ++i)
        drain_bar(&ms.full[i % stages], (uint32_t)(i / stages) & 1u, kDrainNs);
      drain_bar(&ms.q_full, 0, kDrainNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (whole warp, one lane issues)
    const uint32_t id_s = idesc_f16(kTile, N, 0, 0);
    const uint32_t b0 = swz_lo(smem_u32(smem), 16), el = elect_one();
    Ring z, s;
    bool ok = warp_wait(&ms.q_full, 0, abort, kWaitNs);
    for (int i = 0; ok && i < n_tiles; ++i, z.next(nz), s.next(ns)) {
      ok = warp_wait(&ms.z_ready[z.slot], z.par, &ms.s_free[s.slot], s.par ^ 1u, abort, kWaitNs);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tm + pl.col_s + s.slot * N, a = tm + z.slot * (Gp / 2);
#pragma unroll
      for (int k = 0; k < (FSQ_MAX_G + 15) / 16; ++k) {  // atoms of 64 coordinates: four MMAs each
        if (16 * k >= Gp) break;
        mma_ts_warp(el, d, a + 8 * k, b0 + (k >> 2) * (N * 8) + 2 * (k & 3), id_s, k > 0 ? 1u : 0u);
      }
      if (el) {
        tc_commit(&ms.s_full[s.slot]);
        tc_commit(&ms.z_free[z.slot]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) fail();
    // every issued MMA finishes before TMEM is freed
    tc_commit_elect(&ms.done);
    mbar_wait_fixed(&ms.done, 0, kDrainNs);
  } else if (warp >= 12) {
    // ------------------------------------------------------------ dequantisation: thread = token
    const int t = 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    // a warp's share of the row's pieces or groups
    constexpr int PARTS = kDqWarps / 4;
    const int dq = (warp - 12) >> 2;
    auto lo_of = [&](int n) { return (n + PARTS - 1) / PARTS * dq; };
    auto hi_of = [&](int n) { return min(n, (n + PARTS - 1) / PARTS * (dq + 1)); };
    const int units = (G + 7) / 8, align = R % 4 == 0 ? 4 : R % 2 == 0 ? 2 : 1;
    if (dq == 0 && 4 * units < Gp / 2)  // the group behind the last one stays zero
      for (int i = 0; i < nz; ++i) tmem_st4(tm + lanes + i * (Gp / 2) + 4 * units, make_uint4(0u, 0u, 0u, 0u));
    Ring c, z;
    for (int i = 0; i < n_tiles; ++i, c.next(stages), z.next(nz)) {
      if (!warp_wait(&ms.full[c.slot], c.par, &ms.z_free[z.slot], z.par ^ 1u, abort, kWaitNs)) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const uint8_t *stage = smem + pl.q_bytes + c.slot * pl.stage_bytes;
      const uint32_t zt = tm + lanes + z.slot * (Gp / 2);
      const int rows = rows_of(i);
      // a ragged tile's rows from memory, the last one again for those behind it
      const uint8_t *row = src + ((int64_t)tile_of(i) * kTile + min(t, rows - 1)) * R;
      if (pl.tma) {
        if (rows == kTile) {
          const uint32_t o0 = (uint32_t)(t * R);
          fill_pieces<BITS>(zt, lo_of(R / 16), hi_of(R / 16), [&](int u) {
            const uint32_t o = o0 + 16u * u;  // chunk (o / 16) % 8 of 128-byte row o / 128, swizzled
            return *reinterpret_cast<const uint4 *>(stage + (o ^ (((o >> 7) & 7u) << 4)));
          });
        } else {
          fill_pieces<BITS>(zt, lo_of(R / 16), hi_of(R / 16), [&](int u) { return *reinterpret_cast<const uint4 *>(row + 16 * u); });
        }
      } else {
        const bool whole = rows == kTile;
        if (whole) row = stage + t * R;
#pragma unroll 4
        for (int u = lo_of(units); u < hi_of(units); ++u) {
          uint4 v;
          if (whole || u + 1 < units) {
            v = group8<BITS>(row, u, align);
          } else {  // the last group may reach past the row, and there past the cache: byte by byte
            uint32_t w[2] = {0u, 0u};
            for (int x = 0; x < BITS && u * BITS + x < R; ++x) w[x / 4] |= (uint32_t)row[u * BITS + x] << (8 * (x & 3));
            v = levels8<BITS>(w[0], w[1]);
          }
          tmem_st4(zt + 4 * u, v);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.z_ready[z.slot]);
        mbar_arrive(&ms.empty[c.slot]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scores: thread = token, chunks wg, wg + 2, ..
    const int wg = (warp - 4) >> 2, q4 = warp & 3;
    const int r = 32 * q4 + lane;
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    const int chunks = N / 16;
    bool ok = true;
    // test-only stall: a wait that runs out on purpose (nothing completes `never`)
    if (p.stall_ns != 0u && !warp_wait(&ms.never, 0, abort, p.stall_ns)) ok = false;
    if constexpr (MODE == kAdd) {
      // each head's log-sum-exp over the row's splits: a warp per head
      for (int h = warp - 4; h < n_q; h += 8) {
        float m = -INFINITY, l = 0.f;
        for (int s = lane; s < p.S; s += 32) {
          const float2 v = p.part[(b * p.S + s) * n_q + h];
          const float mn = fmaxf(m, v.x);
          if (mn > -INFINITY) {
            l = l * exp2f(m - mn) + v.y * exp2f(v.x - mn);
            m = mn;
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const float om = __shfl_xor_sync(0xffffffffu, m, o), ol = __shfl_xor_sync(0xffffffffu, l, o);
          const float mn = fmaxf(m, om);
          if (mn > -INFINITY) {
            l = l * exp2f(m - mn) + ol * exp2f(om - mn);
            m = mn;
          }
        }
        if (lane == 0) ms.neg[h] = -(m + log2f(l));
      }
      named_bar(5, 256);
    }
    float ref[MODE == kLse ? 8 * NC : 1], sum[MODE == kLse ? 8 * NC : 1];
    float *acc = p.acc + b * p.acc_stride + t0;
    Ring s;
    for (int i = 0; i < n_tiles; ++i, s.next(ns)) {
      const bool valid = r < rows_of(i);
      float old = 0.f;
      if (MODE == kAdd && wg == 0 && valid) old = acc[(int64_t)tile_of(i) * kTile + r];
      ok = ok && warp_wait(&ms.s_full[s.slot], s.par, abort, kWaitNs);
      tc_fence_after();
      float w4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int ch = 2 * c + wg;
        if (ch >= chunks) break;  // uniform
        uint32_t v[16];
        tmem_ld16(tm + lanes + pl.col_s + s.slot * N + 16 * ch, v);
        float sg[8], ng[8];
        *reinterpret_cast<float4 *>(sg) = *reinterpret_cast<const float4 *>(&ms.sig[8 * ch]);
        *reinterpret_cast<float4 *>(sg + 4) = *reinterpret_cast<const float4 *>(&ms.sig[8 * ch + 4]);
        if (MODE == kAdd) {
          *reinterpret_cast<float4 *>(ng) = *reinterpret_cast<const float4 *>(&ms.neg[8 * ch]);
          *reinterpret_cast<float4 *>(ng + 4) = *reinterpret_cast<const float4 *>(&ms.neg[8 * ch + 4]);
        }
        tmem_ld_wait();
        if constexpr (MODE == kAdd) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = fmaf(__uint_as_float(v[e]) + __uint_as_float(v[8 + e]), sg[e], ng[e]);
            if (8 * ch + e < n_q) w4[e & 3] += ex2_approx(x);
          }
        } else {
          float d[8], far = -INFINITY;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = (__uint_as_float(v[e]) + __uint_as_float(v[8 + e])) * sg[e];
            if (i == 0) {
              ref[8 * c + e] = x;
              sum[8 * c + e] = 0.f;
            }
            d[e] = x - ref[8 * c + e];
            far = fmaxf(far, d[e]);
          }
          if (valid) {
            if (far > kFar) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (d[e] > kFar) {
                  sum[8 * c + e] *= exp2f(-d[e]);
                  ref[8 * c + e] += d[e];
                  d[e] = 0.f;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[8 * c + e] += ex2_approx(d[e]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.s_free[s.slot]);
      if constexpr (MODE == kAdd) {
        const float w = (w4[0] + w4[1]) + (w4[2] + w4[3]);
        if (wg == 1) ms.sum[i & 1][r] = w;
        if (named_bar_or(1 + q4, 64, !ok)) {
          ok = false;
          break;
        }
        if (wg == 0 && valid) acc[(int64_t)tile_of(i) * kTile + r] = old + (w + ms.sum[i & 1][r]);
      } else if (!ok) {
        break;  // the whole warp
      }
    }
    if (!ok) fail();
    if constexpr (MODE == kLse) {
      // fold the 128 lanes of every head
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int ch = 2 * c + wg;
        if (ch >= chunks) break;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float l = sum[8 * c + e], m = l == 0.f ? -INFINITY : ref[8 * c + e];  // NaN sums keep their reference
#pragma unroll
          for (int o = 16; o; o >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, m, o), ol = __shfl_xor_sync(0xffffffffu, l, o);
            const float mn = fmaxf(m, om);
            if (mn > -INFINITY) {
              l = l * exp2f(m - mn) + ol * exp2f(om - mn);
              m = mn;
            }
          }
          if (lane == 0) ms.red[q4][8 * ch + e] = make_float2(m, l);
        }
      }
      named_bar(5, 256);
      const int h = tid - 4 * 32;
      if (h < n_q) {
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = ms.red[k][h];
          const float mn = fmaxf(m, v.x);
          if (mn > -INFINITY) {
            l = l * exp2f(m - mn) + v.y * exp2f(v.x - mn);
            m = mn;
          }
        }
        part[h] = make_float2(m, l);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

// ---------------------------------------------------------------- prologue
// Per (kv head j, batch row b): q'_h[g] = c sum_d W_k[j d_h + d][g] q_h[d] (c =
// scale log2 e), scaled by the power of two that brings the head's largest
// weight into [2^kTop, 2^(kTop + 1)), as fp16 hi + lo in the score MMA's B layout: head h
// is rows 16 (h / 8) + h % 8 (hi) and 8 further (lo) of 128-byte-swizzled atoms.
// Also clears the error word.
template <int BITS>
__global__ void __launch_bounds__(kAbsorbThreads, 1) weights_query(const uint16_t *__restrict__ q,
                                                                const uint16_t *__restrict__ W_kv, int n_q, int n_kv,
                                                                int G, int NA, int N, float c,
                                                                uint8_t *__restrict__ qbuf, float *__restrict__ sig,
                                                                uint32_t *err) {
  __shared__ AbsorbSmem<FSQ_MAX_G> sm;
  const int64_t b = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && b == 0 && threadIdx.x == 0) *err = 0u;
  uint8_t *dst = qbuf + b * ((int64_t)NA * N * 128);
  auto at = [&](int n, int g) {  // row n, physical coordinate g
    return dst + (g >> 6) * N * 128 + n * 128 + ((((g & 63) >> 3) ^ (n & 7)) << 4) + (g & 7) * 2;
  };
  // heads that pad the last chunk of 8 are zero
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < (N / 2 - n_q) * NA * kAtom; i += kAbsorbThreads) {
      const int h = n_q + i / (NA * kAtom), n = (h >> 3) * 16 + (h & 7);
      *reinterpret_cast<uint16_t *>(at(n, i % (NA * kAtom))) = 0;
      *reinterpret_cast<uint16_t *>(at(n + 8, i % (NA * kAtom))) = 0;
    }
  absorb_heads(
      sm, q, W_kv, n_q, n_kv, G, NA * kAtom, c, blockIdx.x, b,
      [&](int h, int g, float v, int e) {
        const int ph = (g & ~7) | order_of<BITS>(g & 7), n = (h >> 3) * 16 + (h & 7);
        const float s = scalbnf(v, kTop - e);
        const __half hi = __float2half_rn(s);
        *reinterpret_cast<__half *>(at(n, ph)) = hi;
        *reinterpret_cast<__half *>(at(n + 8, ph)) = __float2half_rn(s - __half2float(hi));
      },
      [&](int h, int e) { sig[b * n_q + h] = scalbnf(1.f, e - kTop); });
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, []() {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

template <int BITS, int NC>
cudaError_t launch_nc(const CUtensorMap &map, const Params &p, int64_t B, const Plan &pl, void *const *prof,
                      cudaStream_t st) {
  // one CTA per SM: each takes all of TMEM
  const size_t smem = pl.total > 120 * 1024 ? pl.total : 120 * 1024;
  auto lse = weights_split_tc<BITS, NC, kLse>;
  auto add = weights_split_tc<BITS, NC, kAdd>;
  cudaError_t e = ensure_smem_limit((const void *)lse, smem);
  if (e == cudaSuccess) e = ensure_smem_limit((const void *)add, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.S, (unsigned)B);
  record_prof_event(prof[0], st);
  e = launch_pdl(lse, grid, dim3(Shape<NC>::THREADS), smem, st, map, p);
  if (e == cudaSuccess) e = launch_pdl(add, grid, dim3(Shape<NC>::THREADS), smem, st, map, p);
  record_prof_event(prof[1], st);
  return e;
}

template <int BITS>
cudaError_t launch_t(const uint16_t *q, const uint16_t *W_kv, int n_kv, float scale, const Params &p, int64_t B,
                     uint8_t *qbuf, float *sig, void *const *prof, cudaStream_t st) {
  const Plan pl = plan_of(p.n_q, p.G, BITS);
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  const int64_t lines = p.T / kTile * pl.R;  // 128-byte rows of the whole tiles; a ragged one is read without TMA
  if (pl.tma && lines > 0) {
    // the packed rows as lines of 128 bytes, [B][lines][128]
    PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const int boxes = boxes_of(pl.R);
    const cuuint64_t dims[3] = {128, (cuuint64_t)lines, (cuuint64_t)B};
    const cuuint64_t strides[2] = {128, (cuuint64_t)p.bstride};
    const cuuint32_t box[3] = {128, (cuuint32_t)(pl.R / boxes), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(p.codes), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  cudaError_t e = launch_pdl(weights_query<BITS>, dim3(n_kv, (unsigned)B), dim3(kAbsorbThreads), 0, st, q, W_kv, p.n_q, n_kv, p.G,
                             pl.NA, pl.N, scale * kLog2e, qbuf, sig, p.err);
  if (e != cudaSuccess) return e;
  switch ((pl.N / 16 + 1) / 2) {
    case 1: return launch_nc<BITS, 1>(map, p, B, pl, prof, st);
    case 2: return launch_nc<BITS, 2>(map, p, B, pl, prof, st);
    case 3: return launch_nc<BITS, 3>(map, p, B, pl, prof, st);
    default: return launch_nc<BITS, 4>(map, p, B, pl, prof, st);
  }
}

}  // namespace weights
}  // namespace tc

bool weights_supported(int n_q, int G, int bits) {
  if (n_q > tc::weights::kMaxQ) return false;
  const tc::weights::Plan p = tc::weights::plan_of(n_q, G, bits);
  return p.stages >= 1 && p.nz >= 1 && p.ns >= 1;
}
int weights_tile_tokens() { return tc::weights::kTile; }
size_t weights_query_bytes(int n_q, int G, int bits) { return tc::weights::plan_of(n_q, G, bits).q_bytes; }

cudaError_t launch_weights(const uint16_t *q, int64_t B, int n_q, int n_kv, const uint8_t *codes, int64_t bstride,
                           int64_t T, const int32_t *seq_lens, int G, int bits, const uint16_t *W_kv, float scale, int S,
                           int k, float *acc, int64_t acc_stride, uint8_t *qbuf, float *sig, float *part, uint32_t *err,
                           uint32_t stall_ns, void *const *prof, cudaStream_t st) {
  tc::weights::Params p{codes, bstride, T, seq_lens, qbuf, sig, (float2 *)part, acc, acc_stride, err,
                        n_q, G, S, k, stall_ns};
  return bits == 2   ? tc::weights::launch_t<2>(q, W_kv, n_kv, scale, p, B, qbuf, sig, prof, st)
         : bits == 4 ? tc::weights::launch_t<4>(q, W_kv, n_kv, scale, p, B, qbuf, sig, prof, st)
                     : tc::weights::launch_t<8>(q, W_kv, n_kv, scale, p, B, qbuf, sig, prof, st);
}

}  // namespace fsq
