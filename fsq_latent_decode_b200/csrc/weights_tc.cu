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
// The result is a running fp32 sum over many steps, so scores keep an fp32 sum's
// precision: Q' = W_k^T q * scale * log2 e is held as two fp16 terms per head (22
// bits), scaled by a power of two.  2- and 8-bit codes enter as signed levels.  4-bit
// codes enter as they lie in their word, as the mantissa of an fp16 subnormal (n 2^-24
// times the power of two of its place, which Q' takes off): one LOP3 per pair, where
// levels take two instructions (203 against 234 us in the case below).  Their offset
// 8 sum_g q'_g, which can be hundreds of times a score where W_k has a component that
// all coordinates share, may not cost precision: the hi term is an integer of 11
// bits in units of a grid (10 above G = 512), so that S_hi, below 2^24 of them, is
// exact, and 8 sum_g hi_g leaves it, exactly, before S_lo joins.
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
// Warps: 0 copies, 1 and 2 issue the MMAs of every other tile, 4-7 and 8-11 take
// the scores, 12-19 (12-15 with many heads) dequantise.  A warp's way through a
// tile is a chain of waits and loads, so two of each kind run side by side.
// Every wait is bounded (FSQ_ERR_TIMEOUT).
//
// Measured: 199-203 us a call (graph replay; 218 us in a loop of calls) for 16 rows of
// 131072 tokens at G = 256 and 32 heads (two passes over 268 MB: 2.7 TB/s).  A tile of 128 tokens takes about 1500
// cycles: 3.1k (kAdd) to 3.8k (kLse) instructions on four schedulers and each
// role's chain of waits; its codes' DRAM time would be 710.
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
// Dequantising warps: two per TMEM quarter, which halve a token's row, where a
// score thread keeps few heads (640 threads have at most 96 registers each), else
// one.
template <int NC>
struct Shape {
  static constexpr int PARTS = NC <= 2 ? 2 : 1, DQ = 4 * PARTS, THREADS = (12 + DQ) * 32;
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

// n buffers that tiles take in turn.  Warps that take every other tile wait on
// barriers whose every phase is theirs (a barrier's parity tells only
// neighbouring phases apart): n is a power of two, and one buffer has two barriers,
// for even and odd tiles.
struct Slots {
  int n, nb, lb;  // buffers, barriers (a power of two: 2^lb)
  __host__ __device__ explicit Slots(int fit = 1, int most = 1) {
    n = 1;
    while (2 * n <= fit && 2 * n <= most) n *= 2;
    nb = n < 2 ? 2 : n;
    for (lb = 1; (1 << lb) < nb; ++lb) {
    }
  }
  __device__ __forceinline__ int buf(int i) const { return i & (n - 1); }
  __device__ __forceinline__ int bar(int i) const { return i & (nb - 1); }
  __device__ __forceinline__ uint32_t par(int i) const { return (uint32_t)(i >> lb) & 1u; }
};

struct Plan {
  int Gp, NA, R, N;   // N: score columns, 16 (hi, lo) per 8 heads, 32 NC in all
  Slots st, z, s;    // code stages in shared memory; Z and S buffers in TMEM
  bool tma;
  bool fits;
  uint32_t q_bytes, stage_bytes, off_misc, total, col_s;
};
__host__ __device__ inline Plan plan_of(int n_q, int G, int bits) {
  Plan p;
  p.Gp = (G + 15) / 16 * 16;
  p.NA = (G + kAtom - 1) / kAtom;
  p.R = G * bits / 8;
  p.N = (n_q + 15) / 16 * 32;
  p.tma = p.R % 16 == 0;
  p.q_bytes = (uint32_t)(p.NA * p.N * 128);
  // (+16: without TMA, a token's last group may read past its row)
  p.stage_bytes = (uint32_t)(kTile * p.R + (p.tma ? 0 : 16) + 1023) / 1024 * 1024;
  const int fit = (int)((kSmemMax - kMiscBytes - p.q_bytes) / p.stage_bytes);
  p.st = Slots(fit, kMaxStages);
  p.off_misc = p.q_bytes + p.st.n * p.stage_bytes;
  p.total = p.off_misc + kMiscBytes;
  // TMEM: Z buffers of Gp / 2 columns from 0, S buffers of N columns behind them
  const int zc = p.Gp / 2, zfit = (512 - (zc + 2 * p.N <= 512 ? 2 : 1) * p.N) / zc;
  p.z = Slots(zfit, kMaxZ);
  p.col_s = p.z.n * zc;
  p.s = Slots((int)(512 - p.col_s) / p.N, kMaxS);
  p.fits = fit >= 1 && zfit >= 1;
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
  const float2 *sig;     // [B][n_q] score scales, and the offset that S_hi sheds first (negated)
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
  uint64_t q_full, done[2], never;
  uint32_t tmem_base, abort;
  __align__(16) float sig[kMaxQ];
  __align__(16) float off[kMaxQ];
  __align__(16) float neg[kMaxQ];  // kAdd: -(log-sum-exp)
  float2 red[4][kMaxQ];            // kLse: per quarter of the lanes
};
static_assert(sizeof(Misc) <= kMiscBytes, "Misc block exceeds its reservation");

// Eight codes -> four words of the score's A operand, in levels8's order.  BITS = 4:
// word k holds codes k and k + 4 as subnormals, times 2^(place_of(k) - 24); else levels.
constexpr bool raw_codes(int bits) { return bits == 4; }
__host__ __device__ constexpr int place_of(int k) { return 4 * (k & 1); }
__host__ __device__ constexpr int grid_bits(int G) { return 15 * G < 1 << 13 ? 10 : 9; }  // 15 G 2^(bits + 1) <= 2^24
template <int BITS>
__device__ __forceinline__ uint4 codes8(uint32_t w, uint32_t w2) {
  if constexpr (raw_codes(BITS)) {
    const uint32_t v = w >> 8;
    return make_uint4(w & 0x000F000Fu, w & 0x00F000F0u, v & 0x000F000Fu, v & 0x00F000F0u);
  } else {
    return levels8<BITS>(w, w2);
  }
}

// The 16-byte pieces [first, pieces) of one token's row -> Z columns; load(u) gives piece u.
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
        if constexpr (BITS == 8) l = codes8<8>(w[2 * e], w[2 * e + 1]);
        else if constexpr (BITS == 4) l = codes8<4>(w[e], 0u);
        else l = codes8<2>(w[e / 2] >> (16 * (e & 1)), 0u);
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
  const Plan pl = plan_of(p.n_q, p.G, BITS);
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc &ms = *reinterpret_cast<Misc *>(smem + pl.off_misc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.G, Gp = pl.Gp, NA = pl.NA, R = pl.R, n_q = p.n_q;
  const Slots st = pl.st, zb = pl.z, sb = pl.s;
  constexpr int N = 32 * NC;  // pl.N
  constexpr int PARTS = Shape<NC>::PARTS, kDqWarps = Shape<NC>::DQ;
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
      mbar_init(&ms.s_free[i], MODE == kAdd ? 4 : 8);
    }
    mbar_init(&ms.q_full, 1);
    mbar_init(&ms.done[0], 1);
    mbar_init(&ms.done[1], 1);
    mbar_init(&ms.never, 1);  // completed by nothing: the test-only stall waits on it
    ms.abort = 0u;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&ms.tmem_base, 512);
    tmem_relinquish();
  }
  if (tid < kMaxQ) {
    const float2 v = tid < n_q ? p.sig[b * n_q + tid] : make_float2(0.f, 0.f);
    ms.sig[tid] = v.x;
    ms.off[tid] = v.y;
  }
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
    for (int i = 0; i < n_tiles; ++i) {
      if (i >= st.n && !warp_wait(&ms.empty[st.bar(i - st.n)], st.par(i - st.n), abort, kWaitNs)) {
        ok = false;
        break;
      }
      uint8_t *dst = smem + pl.q_bytes + st.buf(i) * pl.stage_bytes;
      uint64_t *full = &ms.full[st.bar(i)];
      if (lane == 0) {
        if (rows_of(i) < kTile) {
          mbar_arrive(full);  // the dequantising threads read a ragged tile themselves
        } else {
          mbar_arrive_expect_tx(full, (uint32_t)(kTile * R));
          if (pl.tma) {
            const int row0 = (int)(t0 / kTile + tile_of(i)) * R;
            for (int x = 0; x < boxes; ++x)
              tma_load_3d(dst + x * (R / boxes) * 128, &tmap, 0, row0 + x * (R / boxes), (int)b, full, pol);
          } else {
            bulk_g2s_hint(dst, src + (int64_t)tile_of(i) * kTile * R, (uint32_t)(kTile * R), full, pol);
          }
        }
      }
      issued = i + 1;
    }
    if (!ok) {
      if (lane == 0) fail();
      for (int i = max(0, issued - st.n); i < issued; ++i) drain_bar(&ms.full[st.bar(i)], st.par(i), kDrainNs);
      drain_bar(&ms.q_full, 0, kDrainNs);
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------------ MMA issuers (whole warps, one lane issues):
    // they take turns at the tiles, so that one's waits and commits (100-200
    // cycles each) pass while the tensor core has the other's MMAs
    constexpr uint32_t id_s = idesc_f16(kTile, N, 0, 0);
    const uint32_t b0 = swz_lo(smem_u32(smem), 16), el = elect_one();
    bool ok = warp_wait(&ms.q_full, 0, abort, kWaitNs);
    with_count<1, (FSQ_MAX_G + 15) / 16>(Gp / 16, [&](auto ks) {
    for (int i = warp - 1; ok && i < n_tiles; i += 2) {
      ok = (i < sb.n || warp_wait(&ms.s_free[sb.bar(i - sb.n)], sb.par(i - sb.n), abort, kWaitNs)) &&
           warp_wait(&ms.z_ready[zb.bar(i)], zb.par(i), abort, kWaitNs);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tm + pl.col_s + sb.buf(i) * N, a = tm + zb.buf(i) * (Gp / 2);
#pragma unroll
      for (int k = 0; k < decltype(ks)::value; ++k)  // atoms of 64 coordinates: four MMAs each
        mma_ts_warp(el, d, a + 8 * k, b0 + (k >> 2) * (N * 8) + 2 * (k & 3), id_s, k > 0 ? 1u : 0u);
      if (el) {
        tc_commit(&ms.s_full[sb.bar(i)]);
        tc_commit(&ms.z_free[zb.bar(i)]);
      }
      __syncwarp();
    }
    });
    if (!ok && lane == 0) fail();
    // every issued MMA finishes before TMEM is freed
    tc_commit_elect(&ms.done[warp - 1]);
    mbar_wait_fixed(&ms.done[warp - 1], 0, kDrainNs);
  } else if (warp >= 12) {
    // ------------------------------------------------------------ dequantisation: thread = token
    const int t = 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const int part = (warp - 12) >> 2;
    auto lo_of = [&](int n) { return (n + PARTS - 1) / PARTS * part; };  // this warp's share of n
    auto hi_of = [&](int n) { return min(n, (n + PARTS - 1) / PARTS * (part + 1)); };
    const int units = (G + 7) / 8, align = R % 4 == 0 ? 4 : R % 2 == 0 ? 2 : 1;
    if (part == 0 && 4 * units < Gp / 2)  // the group behind the last one stays zero
      for (int i = 0; i < zb.n; ++i) tmem_st4(tm + lanes + i * (Gp / 2) + 4 * units, make_uint4(0u, 0u, 0u, 0u));
    for (int i = 0; i < n_tiles; ++i) {
      if (!(i < zb.n || warp_wait(&ms.z_free[zb.bar(i - zb.n)], zb.par(i - zb.n), abort, kWaitNs)) ||
          !warp_wait(&ms.full[st.bar(i)], st.par(i), abort, kWaitNs)) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const uint8_t *stage = smem + pl.q_bytes + st.buf(i) * pl.stage_bytes;
      const uint32_t zt = tm + lanes + zb.buf(i) * (Gp / 2);
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
            uint32_t w[2];
            group_words<BITS>(row, u, align, w);
            v = codes8<BITS>(w[0], w[1]);
          } else {  // the last group may reach past the row, and there past the cache: byte by byte
            uint32_t w[2] = {0u, 0u};
            for (int x = 0; x < BITS && u * BITS + x < R; ++x) w[x / 4] |= (uint32_t)row[u * BITS + x] << (8 * (x & 3));
            v = codes8<BITS>(w[0], w[1]);
          }
          tmem_st4(zt + 4 * u, v);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.z_ready[zb.bar(i)]);
        mbar_arrive(&ms.empty[st.bar(i)]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scores: thread = token, chunks wg, wg + 2, ..
    const int wg = (warp - 4) >> 2, q4 = warp & 3;
    const int r = 32 * q4 + lane;
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
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
      if (tid - 4 * 32 < kMaxQ - n_q) ms.neg[n_q + tid - 4 * 32] = -INFINITY;  // heads that pad the last chunk
      named_bar(5, 256);
    }
    float2 ref[MODE == kLse ? 4 * NC : 1], sum[MODE == kLse ? 4 * NC : 1];  // of two heads each; ref holds its negative
    float *acc = p.acc + b * p.acc_stride + t0;
    // kLse: the groups halve the heads of every tile, for whose sums a thread has
    // no more registers.  kAdd: they take turns at the tiles.  A chunk's scores are
    // loaded while the one before is worked on.
    constexpr int STEP = MODE == kAdd ? 2 : 1, CH = MODE == kAdd ? 2 * NC : NC;
    auto chunk_of = [&](int c) { return MODE == kAdd ? c : 2 * c + wg; };
    uint32_t v[2][16];
    int i = MODE == kAdd ? wg : 0;
    auto fetch = [&](int tile, int c, uint32_t *to) {
      tmem_ld16(tm + lanes + pl.col_s + sb.buf(tile) * N + 16 * chunk_of(c), to);
    };
    auto arrived = [&](int tile) {
      ok = ok && warp_wait(&ms.s_full[sb.bar(tile)], sb.par(tile), abort, kWaitNs);
      tc_fence_after();
    };
    if (i < n_tiles) {
      arrived(i);
      fetch(i, 0, v[0]);
    }
    for (; ok && i < n_tiles; i += STEP) {
      const bool valid = r < rows_of(i);
      float *to = acc + (int64_t)tile_of(i) * kTile + r;
      float old = 0.f;
      if (MODE == kAdd && valid) old = *to;
      float2 w2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int ch = chunk_of(c);
        uint32_t(&x16)[16] = v[CH % 2 ? 0 : c & 1];
        tmem_ld_wait16(x16);
        float2 x[4];  // S_hi + S_lo of two heads each
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = make_float2(__uint_as_float(x16[2 * e]), __uint_as_float(x16[2 * e + 1]));
          if constexpr (raw_codes(BITS)) x[e] = __fadd2_rn(x[e], *reinterpret_cast<const float2 *>(&ms.off[8 * ch + 2 * e]));
          x[e] = __fadd2_rn(x[e], make_float2(__uint_as_float(x16[8 + 2 * e]), __uint_as_float(x16[9 + 2 * e])));
        }
        if (c + 1 < CH) {
          fetch(i, c + 1, v[CH % 2 ? 0 : (c + 1) & 1]);
        } else {
          // the tile's scores are in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.s_free[sb.bar(i)]);
          if (i + STEP < n_tiles) {
            arrived(i + STEP);
            fetch(i + STEP, 0, v[0]);
          }
        }
        float sg[8], ng[8];
        *reinterpret_cast<float4 *>(sg) = *reinterpret_cast<const float4 *>(&ms.sig[8 * ch]);
        *reinterpret_cast<float4 *>(sg + 4) = *reinterpret_cast<const float4 *>(&ms.sig[8 * ch + 4]);
        if constexpr (MODE == kAdd) {
          *reinterpret_cast<float4 *>(ng) = *reinterpret_cast<const float4 *>(&ms.neg[8 * ch]);
          *reinterpret_cast<float4 *>(ng + 4) = *reinterpret_cast<const float4 *>(&ms.neg[8 * ch + 4]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 d = __ffma2_rn(x[e], make_float2(sg[2 * e], sg[2 * e + 1]), make_float2(ng[2 * e], ng[2 * e + 1]));
            w2[e & 1] = __fadd2_rn(w2[e & 1], make_float2(ex2_approx(d.x), ex2_approx(d.y)));
          }
        } else {
          if (i == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              ref[4 * c + e] = make_float2(-x[e].x * sg[2 * e], -x[e].y * sg[2 * e + 1]);
              sum[4 * c + e] = make_float2(0.f, 0.f);
            }
          }
          float2 d[4];
          float far = -INFINITY;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[e] = __ffma2_rn(x[e], make_float2(sg[2 * e], sg[2 * e + 1]), ref[4 * c + e]);
            far = fmax3f(far, d[e].x, d[e].y);
          }
          if (valid) {
            if (far > kFar) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (d[e].x > kFar) sum[4 * c + e].x *= exp2f(-d[e].x), ref[4 * c + e].x -= d[e].x, d[e].x = 0.f;
                if (d[e].y > kFar) sum[4 * c + e].y *= exp2f(-d[e].y), ref[4 * c + e].y -= d[e].y, d[e].y = 0.f;
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sum[4 * c + e] = __fadd2_rn(sum[4 * c + e], make_float2(ex2_approx(d[e].x), ex2_approx(d[e].y)));
          }
        }
      }
      if (MODE == kAdd && valid) *to = old + ((w2[0].x + w2[0].y) + (w2[1].x + w2[1].y));
    }
    if (!ok) fail();
    if constexpr (MODE == kLse) {
      // fold the 128 lanes of every head
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int ch = 2 * c + wg;
        if (ch >= N / 16) break;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 s2 = sum[4 * c + e / 2], r2 = ref[4 * c + e / 2];
          float l = e % 2 ? s2.y : s2.x, m = l == 0.f ? -INFINITY : -(e % 2 ? r2.y : r2.x);  // NaN sums keep their reference
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
                                                                uint8_t *__restrict__ qbuf, float2 *__restrict__ sig,
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
        float s = scalbnf(v, kTop - e), hi;
        if constexpr (raw_codes(BITS)) hi = scalbnf(rintf(scalbnf(s, grid_bits(G) - kTop)), kTop - grid_bits(G));
        else hi = __half2float(__float2half_rn(s));
        const int place = raw_codes(BITS) ? place_of((ph & 7) / 2) : 0;
        *reinterpret_cast<__half *>(at(n, ph)) = __float2half_rn(scalbnf(hi, -place));
        *reinterpret_cast<__half *>(at(n + 8, ph)) = __float2half_rn(scalbnf(s - hi, -place));
        return raw_codes(BITS) ? hi : 0.f;
      },
      [&](int h, int e, float sum) {
        constexpr int unit = raw_codes(BITS) ? 24 : 0;
        sig[b * n_q + h] = make_float2(scalbnf(1.f, e - kTop + unit), raw_codes(BITS) ? -scalbnf(sum, 3 - unit) : 0.f);
      });
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
                     uint8_t *qbuf, float2 *sig, void *const *prof, cudaStream_t st) {
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
  switch (pl.N / 32) {
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
  return p.fits;
}
int weights_tile_tokens() { return tc::weights::kTile; }
size_t weights_query_bytes(int n_q, int G, int bits) { return tc::weights::plan_of(n_q, G, bits).q_bytes; }

cudaError_t launch_weights(const uint16_t *q, int64_t B, int n_q, int n_kv, const uint8_t *codes, int64_t bstride,
                           int64_t T, const int32_t *seq_lens, int G, int bits, const uint16_t *W_kv, float scale, int S,
                           int k, float *acc, int64_t acc_stride, uint8_t *qbuf, float *sig, float *part, uint32_t *err,
                           uint32_t stall_ns, void *const *prof, cudaStream_t st) {
  tc::weights::Params p{codes, bstride, T, seq_lens, qbuf, (float2 *)sig, (float2 *)part, acc, acc_stride, err,
                        n_q, G, S, k, stall_ns};
  return bits == 2   ? tc::weights::launch_t<2>(q, W_kv, n_kv, scale, p, B, qbuf, (float2 *)sig, prof, st)
         : bits == 4 ? tc::weights::launch_t<4>(q, W_kv, n_kv, scale, p, B, qbuf, (float2 *)sig, prof, st)
                     : tc::weights::launch_t<8>(q, W_kv, n_kv, scale, p, B, qbuf, (float2 *)sig, prof, st);
}

}  // namespace fsq
