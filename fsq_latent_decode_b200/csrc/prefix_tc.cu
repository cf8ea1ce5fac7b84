// Decode attention of a batch whose rows share a long prefix of cached tokens,
// on the tensor cores (tcgen05 / TMEM), absorbed form ([S] eq. 6).
//
// Every row b attends to the T_p shared tokens and then to its own.  One latent
// serves all heads, and a shared token serves all rows too, so the shared part
// is a dense attention of the B n_q absorbed queries against one code stream:
//   S [128 queries x 64 tokens] = Q' Z^T       Q' = W_k^T q * scale * log2 e
//   O [128 queries x G]         += P Z         P = 2^(S - m)
// A tile of 128 query rows (whole batch rows: floor(128 / n_q) of them) reads a
// token once for all of its rows.  A row's own tokens run through the same
// kernel with that row's n_q queries as the only live ones.  The partials
// (m, l, O) of all token ranges go to the split merge, which applies W_v.
//
// Per 64-token tile: bulk copy of the packed rows -> the codes become fp16
// levels in shared memory, token rows of 64 coordinates in 128-byte-swizzled
// atoms.  Read along the coordinates an atom is a K-major operand (Z^T of the
// scores), read along the tokens an MN-major one (Z of the pooling): one copy,
// no transpose.  A code pair costs one LOP3, which drops the codes into the
// mantissas of 1024.0, and one HFMA2, which takes the offset (and the code's
// place in the word) off: the levels are exact, of both signs, so long sums do
// not drift one way.  Pairs come out as codes k and k + 4 of a group of eight;
// Q' and the result use that order.
//
// Q' is two fp16 terms, hi and lo (22 significant bits: the scores keep fp32's
// precision, also where they spread over hundreds of powers of two), each row
// scaled by a power of two to its largest weight.  The lo products go into S first,
// while its sums are small.  P is fp16, in a window of its range (kTau).
//
// Q' lives in TMEM as the A operand: read from shared memory, both operands of
// a score MMA need more than its bandwidth (48 cycles instead of 32).  TMEM
// columns: O [0, Gp), Q' hi (Gp / 2), Q' lo (Gp / 2), two P buffers of 32 (fp16),
// then as many 64-column S buffers as fit.  From Gp = 208 on they do not: there lo
// stays in shared memory after all, and the ring gives up two of its six tiles.  A
// softmax warp frees S as soon as it holds it in registers, so the next scores run
// while this tile's exponentials do.  Shared memory is a ring of dequantised tiles,
// deep enough that a tile waits in it from its scores to its pooling while the next
// ones are made.
//
// Warps (16): 0 copies, 1 and 2 issue the MMAs, 4-7 and 8-11 take the softmax of
// every other tile (lane = query row) and 12-13 and 14-15 its dequantisation: a
// warp's way through a tile is a chain of waits and loads about twice as long as
// the tensor core's, so two of them run side by side.  The two softmax warps of a
// row agree on its reference tile by tile (`decided`).  Warps that take turns at
// the tiles wait on barriers whose every phase is theirs (an even number of
// stages and tile buffers; scores announced by the tile's parity): a barrier's
// parity tells only neighbouring phases apart.  (For the same reason S has two
// buffers at most: S(i + 2) is announced after S(i) has been read.)
// Every wait is bounded (FSQ_ERR_TIMEOUT), as in the other decode kernels.
//
// Measured: 107 us a call for 16 rows of 32 heads on 131072 shared tokens at G = 256
// (69 GFLOP: 645 TFLOP/s, 39 % of the measured matrix rate; with the lo products
// 102 GFLOP), about 90 of them in this kernel; with hi alone, 96.  A tile keeps the
// tensor core busy for 1792 cycles (lo 768, hi 512, pooling 512); the four schedulers
// need about 1300 (4.8k instructions: dequantisation, exponentials, hand-offs).
#include "common.cuh"
#include "f16_codes.cuh"
#include "query_f16.cuh"
#include "tc_decode.cuh"
#include "tc_ptx.cuh"

namespace fsq {
namespace tc {
namespace prefix {

constexpr int kRows = 128;                         // query rows of a tile
constexpr int kTile = 64;                          // tokens of a tile
constexpr int kThreads = 512;                      // 128 registers a thread: a softmax thread holds 64 scores
constexpr int kAtom = 64;                          // coordinates of a swizzled atom row (128 bytes)
constexpr int kAtomBytes = kTile * 128;            // 64 coordinates of a tile
constexpr int kMaxG = 256;                         // O, Q' hi, two P and one S buffer fill TMEM
constexpr int kLoTmem = 192;                       // widest Gp whose Q' lo fits beside them
constexpr int kQAtomBytes = kRows * 128;           // 64 coordinates of Q' lo in shared memory
constexpr int kTop = 12;                           // Q' is scaled to a largest weight of 2^12 .. 2^13: its lo terms stay normal
constexpr int kMaxStages = 6, kMaxZ = 6, kMaxS = 2;
constexpr int kDqWarps = 2;                        // of a group; the two groups take turns
constexpr int kMiscBytes = 2048;
constexpr size_t kSmemMax = 227 * 1024;
// P is fp16: a row's weights are 2^(s - m), its reference m moves when a score
// exceeds it by kTau, so P stays below 2^15 (fp16 ends at 2^16), and m is set
// `lift` below the maximum of the tile that sets it.  Of n tokens of a split none
// loses more than 2^-25 - lift of the largest weight to fp16's smallest step, all
// together n 2^-25 - lift: lift is the smallest that keeps this at 2^-13, 0 up to
// 4096 tokens.  (The sum l takes the rounded weights, so that what rounding does
// to a weight, it does above and below the fraction bar.)  Scores climb some powers
// of two beyond a tile's first maximum, and moving O holds the whole CTA up for
// longer than a tile takes, so the window above is as wide as the tail lets it be.
constexpr float kTau = 15.f;
constexpr int kTailBits = 12, kMaxLift = 10;
static_assert(kTile == 1 << 6, "prefix_split_tiles counts tiles of 64 tokens");
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainNs = 1000000000ull;

// Shared-memory and TMEM plan of a CTA.
struct Plan {
  int Gp, NA, R, stages, nz, ns;
  uint32_t z_bytes, stage_bytes, off_l, off_c, off_misc, total, col_q, col_l, col_p, col_s;
};
__host__ __device__ inline Plan plan_of(int G, int bits) {
  Plan p;
  p.Gp = (G + 15) / 16 * 16;
  p.NA = (G + kAtom - 1) / kAtom;
  p.R = G * bits / 8;
  const bool tmem = p.Gp <= kLoTmem;  // Q' lo
  p.nz = tmem ? kMaxZ : kMaxZ - 2;
  p.z_bytes = (uint32_t)(p.NA * kAtomBytes);
  p.off_l = p.nz * p.z_bytes;
  p.off_c = p.off_l + (tmem ? 0 : p.NA * kQAtomBytes);
  // +16: the last token's last group may read past its row
  p.stage_bytes = (uint32_t)(kTile * p.R + 16 + 127) / 128 * 128;
  p.stages = (int)((kSmemMax - kMiscBytes - p.off_c) / p.stage_bytes);
  p.stages = p.stages > kMaxStages ? kMaxStages : p.stages / 2 * 2;
  p.off_misc = p.off_c + p.stages * p.stage_bytes;
  p.total = p.off_misc + kMiscBytes;
  p.col_q = p.Gp;
  p.col_l = p.col_q + p.Gp / 2;
  p.col_p = p.col_l + (tmem ? p.Gp / 2 : 0);
  p.col_s = p.col_p + 2 * (kTile / 2);
  p.ns = (int)(512 - p.col_s) / kTile;
  if (p.ns > kMaxS) p.ns = kMaxS;
  return p;
}

struct Params {
  const uint8_t *shared;    // [Tp] rows
  const uint8_t *codes;     // own rows
  int64_t bstride, Tp, T;
  const int32_t *seq_lens;
  // Q', fp16 [QT][hi, lo], physical order: [8 NA chunks of 8][128 rows], so that a
  // warp reads a chunk of its rows at once; lo in swizzled atoms where it stays in
  // shared memory
  const uint8_t *qbuf;
  const float *sig;         // [B n_q] score scales
  float *part;              // [B][S][n_q][2 + G]
  uint32_t *err;
  int B, n_q, G, rpt;       // rpt: batch rows per query tile
  int QT, Sp, Ss, k;        // query tiles, splits of the prefix and of a row's own tokens, tiles per split
  float lift;               // of a split's first maximum above the reference
  uint32_t stall_ns;
};

struct Misc {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t z_ready[kMaxZ], z_free[kMaxZ];  // z_free: the tile's pooling is done
  uint64_t s_full[2], s_free[kMaxS], p_ready[2];  // s_full, p_ready: even and odd tiles
  uint64_t q_ready, l_full, done[2], never;
  uint32_t tmem_base, abort;
  uint64_t decided[2][4];                  // per softmax warp: the tile's reference stands
  float m[kRows];                          // the rows' references
};
static_assert(sizeof(Misc) <= kMiscBytes, "Misc block exceeds its reservation");

// (x, y) += v, in fp32
__device__ __forceinline__ void add_f16x2(float2 &a, __half2 v) {
  asm("{\n\t.reg .f16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32.f16 %0, x, %0;\n\tadd.rn.f32.f16 %1, y, %1;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(*reinterpret_cast<const uint32_t *>(&v)));
}

// 16-byte chunk c (8 coordinates) of token row t in the swizzled atoms
__device__ __forceinline__ uint32_t z_at(int t, int c) {
  return (uint32_t)((c >> 3) * kAtomBytes + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}

template <int BITS>
__global__ void __launch_bounds__(kThreads, 1) prefix_split_tc(Params p) {
  const Plan pl = plan_of(p.G, BITS);
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc &ms = *reinterpret_cast<Misc *>(smem + pl.off_misc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.G, Gp = pl.Gp, NA = pl.NA, R = pl.R, stages = pl.stages, nz = pl.nz, ns = pl.ns;
  const uint32_t z_a = smem_u32(smem);
  // this CTA's work: a query tile and a token range of the prefix, or a row's own range
  const int nshare = p.QT * p.Sp;
  const bool own = (int)blockIdx.x >= nshare;
  const int item = own ? (int)blockIdx.x - nshare : (int)blockIdx.x;
  const int row = own ? item / p.Ss : 0;                       // batch row of an own range
  const int qt = own ? row / p.rpt : item % p.QT;
  const int split = own ? item % p.Ss : item / p.QT;           // within its kind
  const int slot = own ? p.Sp + split : split;                 // within the row's partials
  const int b_lo = own ? row : qt * p.rpt, b_hi = own ? row + 1 : min(p.B, (qt + 1) * p.rpt);
  const int r_lo = (b_lo - qt * p.rpt) * p.n_q, r_hi = (b_hi - qt * p.rpt) * p.n_q;  // live query rows of the tile
  const int S = p.Sp + p.Ss;
  int64_t len = own ? p.T : p.Tp;
  bool bad_len = false;
  if (own && p.seq_lens) {
    // written before this call; the query prologue has waited for that
    pdl_wait();
    const int64_t v = p.seq_lens[row];
    len = v < 0 ? 0 : (v > p.T ? p.T : v);
    bad_len = v != len;
  }
  const int64_t t0 = (int64_t)split * p.k * kTile, t1 = min(len, t0 + (int64_t)p.k * kTile);
  const int n_tiles = t1 > t0 ? (int)((t1 - t0 + kTile - 1) / kTile) : 0;
  const uint8_t *src = (own ? p.codes + (int64_t)row * p.bstride : p.shared) + t0 * R;
  // part[b][slot][h] of query row r (live rows only)
  auto record = [&](int r) {
    const int b = qt * p.rpt + r / p.n_q, h = r % p.n_q;
    return p.part + (((int64_t)b * S + slot) * p.n_q + h) * (2 + G);
  };
  if (n_tiles == 0) {  // nothing of this row here: an empty partial, which the merge weighs by 2^-inf = 0
    pdl_wait();
    if (bad_len && split == 0 && tid == 0) record_error(p.err, FSQ_ERR_INVALID_ARG);
    for (int i = tid; i < p.n_q * (2 + G); i += kThreads) {
      float *out = record(r_lo + i / (2 + G));
      out[i % (2 + G)] = i % (2 + G) == 0 ? -INFINITY : 0.f;
    }
    return;
  }
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
      mbar_init(&ms.s_free[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.p_ready[i], 4);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&ms.decided[i / 4][i % 4], 1);
    mbar_init(&ms.q_ready, 8);
    mbar_init(&ms.l_full, 1);
    mbar_init(&ms.done[0], 1);
    mbar_init(&ms.done[1], 1);
    mbar_init(&ms.never, 1);  // completed by nothing: the test-only stall waits on it
    ms.abort = 0u;
    fence_mbar_init();
  }
  if (tid < kRows) ms.m[tid] = -INFINITY;
  if (warp == 0) {
    tmem_alloc(&ms.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tm = 0;  // all 512 columns are this CTA's
  pdl_trigger();  // the merge kernel may start staging W_v
  auto fail = [&]() {
    record_error(p.err, FSQ_ERR_TIMEOUT);
    *abort = 1u;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    pdl_wait();  // for the query prologue, which waited for whatever wrote the codes
    if (bad_len && split == 0 && lane == 0) record_error(p.err, FSQ_ERR_INVALID_ARG);
    // Q' lo, of the whole tile: what rows without a query get, they alone see
    if (Gp > kLoTmem && lane == 0) {
      mbar_arrive_expect_tx(&ms.l_full, NA * kQAtomBytes);
      bulk_g2s(smem + pl.off_l, p.qbuf + (int64_t)(2 * qt + 1) * (NA * kQAtomBytes), NA * kQAtomBytes, &ms.l_full);
    }
    // a row's own tokens are read once; the tiles of the prefix by every query tile
    const uint64_t pol = own ? l2_evict_first() : l2_evict_normal();
    bool ok = true;
    int issued = 0;
    Ring c;
    for (int i = 0; i < n_tiles; ++i, c.next(stages)) {
      const int st = c.slot;
      if (!warp_wait(&ms.empty[st], c.par ^ 1u, abort, kWaitNs)) {
        ok = false;
        break;
      }
      uint8_t *dst = smem + pl.off_c + st * pl.stage_bytes;
      const int nb = (int)min((int64_t)kTile, t1 - (t0 + (int64_t)i * kTile)) * R;
      const uint8_t *s = src + (int64_t)i * kTile * R;
      // whole 16-byte pieces by bulk copy, the last bytes of the range one by
      // one; what lies behind them in the stage decodes to finite levels
      if (lane < nb % 16) dst[nb / 16 * 16 + lane] = s[nb / 16 * 16 + lane];
      __syncwarp();
      if (lane == 0) {
        const uint32_t bulk = (uint32_t)(nb / 16 * 16);
        if (bulk) {
          mbar_arrive_expect_tx(&ms.full[st], bulk);
          bulk_g2s_hint(dst, s, bulk, &ms.full[st], pol);
        } else {
          mbar_arrive(&ms.full[st]);
        }
      }
      issued = i + 1;
    }
    if (!ok) {
      if (lane == 0) fail();
      for (int i = max(0, issued - stages); i < issued; ++i)
        drain_bar(&ms.full[i % stages], (uint32_t)(i / stages) & 1u, kDrainNs);
      if (Gp > kLoTmem) drain_bar(&ms.l_full, 0, kDrainNs);
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------------ MMA issuers (whole warps, one lane issues):
    // one of the scores, one of the pooling.  Every wait costs a warp 100-200
    // cycles even when its phase is complete; with two warps the tensor core has
    // the other's MMAs meanwhile.  All hazards between them are barriers': S(i)
    // overwrites scores that the softmax has loaded, P(i) follows S(i), and a
    // tile is freed by its pooling.
    constexpr uint32_t id_s = idesc_f16(kRows, kTile, 0, 0);
    const uint32_t id_o = idesc_f16(kRows, Gp, 0, 1), el = elect_one();
    bool ok = true;
    if (warp == 1) {
      ok = warp_wait(&ms.q_ready, 0, abort, kWaitNs) && (Gp <= kLoTmem || warp_wait(&ms.l_full, 0, abort, kWaitNs));
      with_count<1, kMaxG / 16>(Gp / 16, [&](auto ks) {
      constexpr bool LO_SMEM = 16 * decltype(ks)::value > kLoTmem;
      const uint32_t lo_s = swz_lo(z_a + pl.off_l, 16);
      Ring z, s;
      for (int i = 0; ok && i < n_tiles; ++i, z.next(nz), s.next(ns)) {
        ok = warp_wait(&ms.s_free[s.slot], s.par ^ 1u, &ms.z_ready[z.slot], z.par, abort, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tm + pl.col_s + s.slot * kTile, a = tm + pl.col_q, lo = tm + pl.col_l;
        const uint32_t b = swz_lo(z_a + z.slot * pl.z_bytes, 16);
#pragma unroll
        for (int k = 0; k < decltype(ks)::value; ++k) {
          const uint32_t bk = b + (((k >> 2) * kAtomBytes + (k & 3) * 32) >> 4);
          if constexpr (LO_SMEM)
            mma_ss_warp(el, d, lo_s + (((k >> 2) * kQAtomBytes + (k & 3) * 32) >> 4), bk, id_s, k > 0 ? 1u : 0u);
          else mma_ts_warp(el, d, lo + 8 * k, bk, id_s, k > 0 ? 1u : 0u);
        }
#pragma unroll
        for (int k = 0; k < decltype(ks)::value; ++k)
          mma_ts_warp(el, d, a + 8 * k, b + (((k >> 2) * kAtomBytes + (k & 3) * 32) >> 4), id_s, 1u);
        if (el) tc_commit(&ms.s_full[i & 1]);
        __syncwarp();
      }
      });
    } else {
      Ring z, pr;
      for (int i = 0; i < n_tiles; ++i, z.next(nz), pr.next(2)) {
        ok = warp_wait(&ms.p_ready[pr.slot], pr.par, abort, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = tm + pl.col_p + pr.slot * (kTile / 2);
        const uint32_t b = swz_lo(z_a + z.slot * pl.z_bytes, kAtomBytes);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts_warp(el, tm, a + 8 * k, b + ((k * 2048) >> 4), id_o, k > 0 || i > 0 ? 1u : 0u);
        if (el) tc_commit(&ms.z_free[z.slot]);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) fail();
    // every issued MMA finishes before TMEM is freed
    tc_commit_elect(&ms.done[warp - 1]);
    mbar_wait_fixed(&ms.done[warp - 1], 0, kDrainNs);
  } else if (warp >= 12) {
    // ------------------------------------------------------------ dequantisation
    const int grp = (warp - 12) / kDqWarps, dt = tid - (12 + kDqWarps * grp) * 32;
    const int align = R % 16 == 0 ? 16 : R % 4 == 0 ? 4 : R % 2 == 0 ? 2 : 1;
    const int units = (G + 7) / 8;   // groups of 8 coordinates that hold codes
    // the groups behind them stay zero
    static_assert(kMaxZ % 2 == 0 && kMaxStages % 2 == 0, "a group always takes the same stages and tile buffers");
    for (int i = dt; i < kTile * (8 * NA - units) * (nz / 2); i += kDqWarps * 32) {
      const int t = i % kTile, x = i / kTile;
      *reinterpret_cast<uint4 *>(smem + (2 * (x % (nz / 2)) + grp) * pl.z_bytes + z_at(t, units + x / (nz / 2))) =
          make_uint4(0u, 0u, 0u, 0u);
    }
    Ring cr, zr;
    for (int i = 0; i < n_tiles; ++i, cr.next(stages), zr.next(nz)) {
      if ((i & 1) != grp) continue;
      if (!warp_wait(&ms.full[cr.slot], cr.par, &ms.z_free[zr.slot], zr.par ^ 1u, abort, kWaitNs)) {
        if (lane == 0) fail();
        break;
      }
      const uint8_t *c = smem + pl.off_c + cr.slot * pl.stage_bytes;
      uint8_t *z = smem + zr.slot * pl.z_bytes;
      if (align == 16) {
        // 16 bytes of a row at a time, in order, so that the reads are contiguous
        // over the warp.  Eight lanes then hold neighbouring pieces of one token,
        // whose chunks of the same rank share banks: each lane takes its NE chunks
        // in another order, and the eight writes of a step cover all banks.
        constexpr int NE = 16 / BITS;                  // chunks (groups of 8 coordinates) of a piece
        const int ppr = R / 16;
        const uint32_t inv = (65536u + ppr - 1) / ppr;  // x / ppr for x < 64 * 16
#pragma unroll 4
        for (int x = dt; x < kTile * ppr; x += kDqWarps * 32) {
          const int t = (int)(((uint32_t)x * inv) >> 16), piece = x - t * ppr;
          const uint4 v = *reinterpret_cast<const uint4 *>(c + 16 * x);
          // chunk e ^ rot is the lane's e-th; its place: atom, row, and the
          // chunk's number swizzled by the row
          const int c0 = NE * piece, rot = (c0 >> 3) & (NE - 1);
          const uint32_t at = (uint32_t)((c0 >> 3) * kAtomBytes + t * 128 + (((c0 & 7) ^ (t & 7) ^ rot) << 4));
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if constexpr (BITS == 2) {
            if (rot & 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = __funnelshift_r(w[e], w[e], 16);
            }
          }
          constexpr int ONE = BITS == 8 ? 0 : BITS == 4 ? 1 : 2, TWO = BITS == 8 ? 1 : BITS == 4 ? 2 : 4;  // rot bits
          if (rot & ONE) {
            uint32_t f = w[0];
            w[0] = w[1], w[1] = f;
            f = w[2], w[2] = w[3], w[3] = f;
          }
          if (rot & TWO) {
            const uint32_t f = w[0], g = w[1];
            w[0] = w[2], w[1] = w[3], w[2] = f, w[3] = g;
          }
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            uint4 l;
            if constexpr (BITS == 8) l = levels8<8>(w[2 * e], w[2 * e + 1]);
            else if constexpr (BITS == 4) l = levels8<4>(w[e], 0u);
            else l = levels8<2>(w[e / 2] >> (16 * (e & 1)), 0u);
            *reinterpret_cast<uint4 *>(z + (at ^ (uint32_t)(e << 4))) = l;
          }
        }
      } else {
        // a group at a time; the lanes hold neighbouring tokens
#pragma unroll 4
        for (int x = dt; x < kTile * units; x += kDqWarps * 32) {
          const int t = x % kTile, u = x / kTile;
          uint32_t w[2];
          group_words<BITS>(c + t * R, u, align, w);
          *reinterpret_cast<uint4 *>(z + z_at(t, u)) = levels8<BITS>(w[0], w[1]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.z_ready[zr.slot]);
        mbar_arrive(&ms.empty[cr.slot]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax: lane = query row, every other tile
    const int wg = (warp - 4) >> 2, q4 = warp & 3;
    const int r = 32 * q4 + lane;
    const bool busy = 32 * q4 < r_hi && 32 * q4 + 32 > r_lo;  // this warp has live rows
    const bool live = r >= r_lo && r < r_hi;
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    bool ok = true;
    pdl_wait();  // Q' and sig come from the query prologue
    float sig = 0.f;
    {
      // half of the row's Q' into TMEM, lo as far as it fits; rows without a query are zero
      const uint8_t *qr = p.qbuf + (int64_t)qt * (2 * NA * kQAtomBytes) + r * 16;
      if (live) sig = p.sig[(int64_t)qt * p.rpt * p.n_q + r];
#pragma unroll 1
      for (int term = 0; term < (Gp > kLoTmem ? 1 : 2); ++term, qr += NA * kQAtomBytes) {
#pragma unroll 4
        for (int c = 8 * wg; c < Gp / 2; c += 16) {  // columns: two coordinates each
          uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
          if (live) {
            a = *reinterpret_cast<const uint4 *>(qr + (c >> 2) * (16 * kRows));
            b = *reinterpret_cast<const uint4 *>(qr + ((c >> 2) + 1) * (16 * kRows));
          }
          const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          tmem_st8(tm + lanes + (term ? pl.col_l : pl.col_q) + c, v);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.q_ready);
    }
    // test-only stall: a wait that runs out on purpose (nothing completes `never`)
    if (p.stall_ns != 0u && !warp_wait(&ms.never, 0, abort, p.stall_ns)) ok = false;
    float m = -INFINITY, l = 0.f;  // the reference that l is relative to, which the other warp may have moved since
    Ring sr, zo, zp;               // S buffer of the tile; the tile before it; the one before that
    if (wg == 1) sr.next(ns), zp.next(nz);
    else zo.next(nz);
    for (int i = wg; ok && i < n_tiles; i += 2) {
      ok = warp_wait(&ms.s_full[wg], (uint32_t)(i >> 1) & 1u, abort, kWaitNs);
      tc_fence_after();
      uint32_t s[64];
      float top = -INFINITY;
      if (busy) {
        const uint32_t ts = tm + lanes + pl.col_s + sr.slot * kTile;
        tmem_ld32(ts, s);
        tmem_ld32(ts + 32, s + 32);
        tmem_ld_wait16(s);
        tmem_held16(s + 16);
        tmem_held16(s + 32);
        tmem_held16(s + 48);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.s_free[sr.slot]);
      sr.next(ns);
      sr.next(ns);
      if (busy) {
        const int valid = (int)min((int64_t)kTile, t1 - (t0 + (int64_t)i * kTile));
        if (valid < kTile) {
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (c >= valid) s[c] = 0xFF800000u;  // -inf
        }
        float t2[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kTile; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            t2[e] = fmax3f(t2[e], __uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1]));
        top = fmaxf(fmaxf(t2[0], t2[1]), fmaxf(t2[2], t2[3])) * sig;
      }
      // the row's reference after the tile before this one, which the other warp has decided
      if (i > 0) ok = warp_wait(&ms.decided[wg ^ 1][q4], (uint32_t)((i - 1) >> 1) & 1u, abort, kWaitNs) && ok;
      const float was = *(volatile float *)&ms.m[r];
      const bool raise = live && (top > was + kTau || (i == 0 && top > was));
      const float now = raise ? top - p.lift : was;
      if (raise) *(volatile float *)&ms.m[r] = now;
      const bool move = __any_sync(0xffffffffu, raise) && i > 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.decided[wg][q4]);
      if (m != now) l *= exp2f(m - now);
      m = now;
      // P(i - 2) has been pooled (a warp without live rows waits too: its arrival
      // for this tile must not count for that one)
      if (i > 1) ok = warp_wait(&ms.z_free[zp.slot], zp.par, abort, kWaitNs) && ok;
      tc_fence_after();
      if (busy) {
        const uint32_t tp = tm + lanes + pl.col_p + wg * (kTile / 2);
        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 sig2 = make_float2(sig, sig), off2 = make_float2(-now, -now);
#pragma unroll
        for (int c0 = 0; c0 < kTile / 2; c0 += 8) {
          uint32_t h[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * (c0 + c)]), __uint_as_float(s[2 * (c0 + c) + 1])),
                                        sig2, off2);
            const __half2 v = __floats2half2_rn(ex2_approx(x.x), ex2_approx(x.y));
            add_f16x2(l2[c & 1], v);
            h[c] = *reinterpret_cast<const uint32_t *>(&v);
          }
          tmem_st8(tp + c0, h);
        }
        l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
        if (move) {
          // O holds every earlier tile once the last pooling is done
          const float f = raise ? exp2f(was - now) : 1.f;
          ok = warp_wait(&ms.z_free[zo.slot], zo.par, abort, kWaitNs) && ok;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < Gp; c += 32) {
            uint32_t a[32];
            const bool two = c + 16 < Gp;
            tmem_ld16(tm + lanes + c, a);
            if (two) tmem_ld16(tm + lanes + c + 16, a + 16);
            tmem_ld_wait16(a);
            tmem_held16(a + 16);
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * f);
            tmem_st16(tm + lanes + c, a);
            if (two) tmem_st16(tm + lanes + c + 16, a + 16);
          }
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.p_ready[wg]);
      if (i > 0) zo.next(nz), zo.next(nz);
      if (i > 1) zp.next(nz), zp.next(nz);
    }
    // ---- epilogue: O through shared memory (the tiles are spent) to the partials
    if (ok) {
      const int z = (n_tiles - 1) % nz;
      ok = warp_wait(&ms.z_free[z], (uint32_t)((n_tiles - 1) / nz) & 1u, abort, kWaitNs);
    }
    if (!ok) fail();
    // behind the staged O, which the Z tiles leave room for: per group (reference, sum) of a row
    float2 *sums = reinterpret_cast<float2 *>(smem + pl.off_c) - 2 * kRows;
    sums[wg * kRows + r] = make_float2(m, l);
    if (!named_bar_or(5, 256, !ok)) {
      tc_fence_after();
      float *stage = reinterpret_cast<float *>(smem);  // [128][Gp + 1]: conflict-free both ways
      const int ld = Gp + 1;
      if (busy) {
#pragma unroll 1
        for (int c = 16 * wg; c < Gp; c += 32) {
          uint32_t a[16];
          tmem_ld16(tm + lanes + c, a);
          tmem_ld_wait16(a);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int g = c + (e & 8) + (BITS == 8 ? (e & 7) : ((e & 1) << 2) + ((e & 7) >> 1));
            stage[r * ld + g] = __uint_as_float(a[e]);
          }
        }
      }
      named_bar(5, 256);
      for (int rr = r_lo + (warp - 4); rr < r_hi; rr += 8) {
        float *out = record(rr) + 2;
        const float *from = stage + rr * ld;
        float v[kMaxG / 32];
#pragma unroll
        for (int x = 0; x < kMaxG / 32; ++x) v[x] = 32 * x + lane < G ? from[32 * x + lane] : 0.f;
#pragma unroll
        for (int x = 0; x < kMaxG / 32; ++x)
          if (32 * x + lane < G) out[32 * x + lane] = v[x];
      }
      if (live && wg == 0) {
        float *out = record(r);
        const float2 a = sums[r], c = sums[kRows + r];
        const float last = ms.m[r];
        out[0] = last;
        out[1] = a.y * exp2f(a.x - last) + (n_tiles > 1 ? c.y * exp2f(c.x - last) : 0.f);
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
// weight into [2^kTop, 2^(kTop + 1)), as two rows of fp16, hi and lo, in physical
// order of their tile's chunks; sig_h takes the power back.  Also clears the error word.
template <int BITS>
__global__ void __launch_bounds__(kAbsorbThreads, 1) prefix_query(const uint16_t *__restrict__ q,
                                                               const uint16_t *__restrict__ W_kv, int n_q, int n_kv,
                                                               int G, int NA, int rpt, float c, uint8_t *__restrict__ qbuf,
                                                               float *__restrict__ sig, uint32_t *err) {
  __shared__ AbsorbSmem<kMaxG> sm;
  const int64_t b = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && b == 0 && threadIdx.x == 0) *err = 0u;
  uint8_t *tile = qbuf + b / rpt * (2 * NA * kQAtomBytes);
  const int r0 = (int)(b % rpt) * n_q;
  const bool atoms = (G + 15) / 16 * 16 > kLoTmem;  // of lo
  absorb_heads(
      sm, q, W_kv, n_q, n_kv, G, NA * kAtom, c, blockIdx.x, b,
      [&](int h, int g, float v, int e) {
        const int r = r0 + h, ch = g >> 3, x = 2 * order_of<BITS>(g & 7);
        const float s = scalbnf(v, kTop - e);
        const __half hi = __float2half_rn(s);
        const int at = (ch * kRows + r) * 16 + x;
        *reinterpret_cast<__half *>(tile + at) = hi;
        *reinterpret_cast<__half *>(tile + NA * kQAtomBytes + (atoms ? (ch >> 3) * kQAtomBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4) + x : at)) =
            __float2half_rn(s - __half2float(hi));
      },
      [&](int h, int e) { sig[b * n_q + h] = scalbnf(1.f, e - kTop); });
}

// ---------------------------------------------------------------- split merge
// Per (kv head j, batch row b): the group's heads, four at a time,
//   m = max_s m_s,  w_s = 2^(m_s - m),  abar_h = sum_s w_s O_s / sum_s w_s l_s,  o_h = W_v^(j) abar_h.
// Bound by latency (35 splits of 4 heads at G = 256: 140 KB of partials and 64 KB
// of W_v per CTA).  W_v^(j) comes into shared memory before the wait for the
// split kernel; a thread sums one coordinate pair of one head over its share of
// the splits, the first eight of them loaded while a warp per head forms w_s; a
// warp then takes eight rows of W_v, the heads' sums in registers, and one
// butterfly folds the 32 results over its lanes.
constexpr int kMergeThreads = 512, kMergeHeads = 4, kMergeRows = FSQ_HEAD_DIM / (kMergeThreads / 32);
constexpr int kMergeAhead = 8;
constexpr int kMaxSplits = 2048;  // of a row

// VEC: coordinates that are moved at once (8, or 2 where G is not a multiple of 8)
template <int VEC>
__global__ void __launch_bounds__(kMergeThreads, 1) prefix_merge(const float *__restrict__ part, int S, int n_q, int n_kv,
                                                                 int G, const uint16_t *__restrict__ W_kv, void *o,
                                                                 int out_fp32) {
  constexpr int D = FSQ_HEAD_DIM, STEPS = kMaxG / (32 * VEC);
  extern __shared__ __align__(16) uint8_t msm[];
  uint16_t *wv = reinterpret_cast<uint16_t *>(msm);                                // [D][G]
  float2 *wts = reinterpret_cast<float2 *>(msm + sizeof(uint16_t) * D * G);        // [kMergeHeads][S]: (m, l), then w in x
  __shared__ float2 sum[kMergeThreads];
  __shared__ __align__(16) float abar[kMergeHeads][kMaxG];
  const int j = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.y;
  const int grp = n_q / n_kv;
  {
    const uint16_t *src = W_kv + (int64_t)(n_kv + j) * D * G;
    for (int i = tid; i < D * G / VEC; i += kMergeThreads) {
      const uint32_t at = (uint32_t)__cvta_generic_to_shared(wv + i * VEC);
      if constexpr (VEC == 8) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(src + i * VEC) : "memory");
      else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(src + i * VEC) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  pdl_wait();
  const int64_t hs = 2 + G, ss = (int64_t)n_q * hs;  // floats of a record, of a split
  for (int h0 = 0; h0 < grp; h0 += kMergeHeads) {
    const int nh = min(kMergeHeads, grp - h0);
    const float *rec = part + (b * S * n_q + (int64_t)j * grp + h0) * hs;
    const int pairs = G / 2, items = nh * pairs, nsub = min(16, max(1, kMergeThreads / items));  // items <= 4 * 128
    const int it = tid % items, sub = tid / items, h = it / pairs, x = it % pairs;
    const float *src = rec + h * hs + 2 + 2 * x;
    float2 first[kMergeAhead];
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k) {
      const int s = sub + k * nsub;
      first[k] = sub < nsub && s < S ? *reinterpret_cast<const float2 *>(src + s * ss) : make_float2(0.f, 0.f);
    }
    if (warp < nh) {  // a warp per head: the splits' weights
      float m = -INFINITY, l = 0.f;
      for (int s = lane; s < S; s += 32) {
        const float2 v = *reinterpret_cast<const float2 *>(rec + s * ss + warp * hs);
        wts[warp * S + s] = v;
        m = fmaxf(m, v.x);
      }
#pragma unroll
      for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      for (int s = lane; s < S; s += 32) {
        const float2 v = wts[warp * S + s];
        const float e = exp2f(v.x - m);  // 0 for an empty split
        wts[warp * S + s].x = e;
        l = fmaf(e, v.y, l);
      }
#pragma unroll
      for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
      const float inv = 1.f / l;
      for (int s = lane; s < S; s += 32) wts[warp * S + s].x *= inv;
    }
    __syncthreads();
    float2 a = make_float2(0.f, 0.f);
    if (sub < nsub) {
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k) {
        const int s = sub + k * nsub;
        const float e = s < S ? wts[h * S + s].x : 0.f;
        a.x = fmaf(e, first[k].x, a.x);
        a.y = fmaf(e, first[k].y, a.y);
      }
#pragma unroll 8
      for (int s = sub + kMergeAhead * nsub; s < S; s += nsub) {
        const float2 v = *reinterpret_cast<const float2 *>(src + s * ss);
        const float e = wts[h * S + s].x;
        a.x = fmaf(e, v.x, a.x);
        a.y = fmaf(e, v.y, a.y);
      }
    }
    if (nsub > 1) {
      sum[tid] = a;
      __syncthreads();
      if (sub == 0)
        for (int k = 1; k < nsub; ++k) {
          a.x += sum[k * items + it].x;
          a.y += sum[k * items + it].y;
        }
    }
    if (sub == 0) *reinterpret_cast<float2 *>(&abar[h][2 * x]) = a;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float av[kMergeHeads][STEPS][VEC];
#pragma unroll
    for (int k = 0; k < kMergeHeads; ++k)
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int g = 32 * VEC * i + VEC * lane + e;
          av[k][i][e] = k < nh && g < G ? abar[k][g] : 0.f;
        }
    // 32 results a warp: row warp * kMergeRows + r of head k at 4 r + k
    static_assert(kMergeRows * kMergeHeads == 32, "a lane per result");
    float acc[32];
#pragma unroll
    for (int r = 0; r < kMergeRows; ++r) {
#pragma unroll
      for (int k = 0; k < kMergeHeads; ++k) acc[4 * r + k] = 0.f;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int g = 32 * VEC * i + VEC * lane;
        uint32_t w[VEC / 2] = {};
        if (g < G) {
          const uint16_t *row = wv + (warp * kMergeRows + r) * G + g;
          if constexpr (VEC == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(row);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
          } else {
            w[0] = *reinterpret_cast<const uint32_t *>(row);
          }
        }
#pragma unroll
        for (int e = 0; e < VEC; e += 2)
#pragma unroll
          for (int k = 0; k < kMergeHeads; ++k) {
            acc[4 * r + k] = fmaf(__uint_as_float(w[e / 2] << 16), av[k][i][e], acc[4 * r + k]);
            acc[4 * r + k] = fmaf(__uint_as_float(w[e / 2] & 0xFFFF0000u), av[k][i][e + 1], acc[4 * r + k]);
          }
      }
    }
    // butterfly: every step hands the other half of the results over; lane x ends with result x
#pragma unroll
    for (int k = 16; k; k >>= 1) {
      const bool up = lane & k;
#pragma unroll
      for (int i = 0; i < k; ++i) {
        const float give = up ? acc[i] : acc[i + k], keep = up ? acc[i + k] : acc[i];
        acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, k);
      }
    }
    if (lane % 4 < nh) {
      const int64_t at = ((b * n_q + (int64_t)j * grp + h0 + lane % 4) * D) + warp * kMergeRows + lane / 4;
      if (out_fp32) reinterpret_cast<float *>(o)[at] = acc[0];
      else reinterpret_cast<uint16_t *>(o)[at] = f32_to_bf16_rn(acc[0]);
    }
    __syncthreads();
  }
}

template <int BITS>
cudaError_t launch_t(const uint16_t *q, const uint16_t *W_kv, int n_kv, float scale, const Params &p, uint8_t *qbuf,
                     float *sig, void *o, int out_fp32, void *const *prof, cudaStream_t st) {
  const Plan pl = plan_of(p.G, BITS);
  cudaError_t e = launch_pdl(prefix_query<BITS>, dim3(n_kv, (unsigned)p.B), dim3(kAbsorbThreads), 0, st, q, W_kv, p.n_q, n_kv,
                             p.G, pl.NA, p.rpt, scale * kLog2e, qbuf, sig, p.err);
  if (e != cudaSuccess) return e;
  // one CTA per SM: each takes all of TMEM
  const size_t smem = pl.total > 120 * 1024 ? pl.total : 120 * 1024;
  e = ensure_smem_limit((const void *)prefix_split_tc<BITS>, smem);
  if (e != cudaSuccess) return e;
  record_prof_event(prof[0], st);
  e = launch_pdl(prefix_split_tc<BITS>, dim3((unsigned)(p.QT * p.Sp + p.B * p.Ss)), dim3(kThreads), smem, st, p);
  record_prof_event(prof[1], st);
  if (e != cudaSuccess) return e;
  const int S = p.Sp + p.Ss;
  auto merge = p.G % 8 == 0 ? prefix_merge<8> : prefix_merge<2>;
  const size_t msm = sizeof(uint16_t) * FSQ_HEAD_DIM * p.G + sizeof(float2) * kMergeHeads * S;
  e = ensure_smem_limit((const void *)merge, msm);
  if (e != cudaSuccess) return e;
  return launch_pdl(merge, dim3(n_kv, (unsigned)p.B), dim3(kMergeThreads), msm, st, (const float *)p.part, S, p.n_q,
                    n_kv, p.G, W_kv, o, out_fp32);
}

}  // namespace prefix
}  // namespace tc

bool prefix_supported(int n_q, int G) { return n_q <= tc::prefix::kRows && G <= tc::prefix::kMaxG; }
int prefix_rows_per_tile(int n_q) { return tc::prefix::kRows / n_q; }
int prefix_max_splits() { return tc::prefix::kMaxSplits; }
int prefix_tile_tokens() { return tc::prefix::kTile; }
int prefix_split_tiles() { return 1 << (tc::prefix::kTailBits + tc::prefix::kMaxLift - 6); }
size_t prefix_query_bytes(int G) {  // Q' of a query tile, hi and lo
  return (size_t)((G + tc::prefix::kAtom - 1) / tc::prefix::kAtom) * tc::prefix::kQAtomBytes * 2;
}

cudaError_t launch_prefix(const uint16_t *q, int64_t B, int n_q, int n_kv, const uint8_t *shared, int64_t Tp,
                          const uint8_t *codes, int64_t bstride, int64_t T, const int32_t *seq_lens, int G, int bits,
                          const uint16_t *W_kv, float scale, int QT, int Sp, int Ss, int k, uint8_t *qbuf, float *sig,
                          float *part, uint32_t *err, void *o, int out_fp32, uint32_t stall_ns,
                          void *const *prof, cudaStream_t st) {
  int lift = 0;
  while (lift < tc::prefix::kMaxLift && (int64_t)k * tc::prefix::kTile > (int64_t)1 << (tc::prefix::kTailBits + lift)) ++lift;
  tc::prefix::Params p{shared, codes, bstride, Tp, T, seq_lens, qbuf, sig, part, err,
                       (int)B, n_q, G, prefix_rows_per_tile(n_q), QT, Sp, Ss, k, (float)lift, stall_ns};
  return bits == 2   ? tc::prefix::launch_t<2>(q, W_kv, n_kv, scale, p, qbuf, sig, o, out_fp32, prof, st)
         : bits == 4 ? tc::prefix::launch_t<4>(q, W_kv, n_kv, scale, p, qbuf, sig, o, out_fp32, prof, st)
                     : tc::prefix::launch_t<8>(q, W_kv, n_kv, scale, p, qbuf, sig, o, out_fp32, prof, st);
}

}  // namespace fsq
