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
// Q' is fp16, each row scaled by a power of two to its largest weight: 11
// significant bits, finer than the bf16 of q and W_k it comes from.  P is fp16
// with the running maximum at 2^6, so weights down to 2^-30 of it count.
//
// Q' lives in TMEM as the A operand: read from shared memory, both operands of
// a score MMA would need more than its bandwidth.  TMEM columns: O [0, Gp), Q'
// (Gp / 2), then as many 64-column S buffers as fit, two at G = 256; P (fp16)
// overlays the first half of its S.  Shared memory is a ring of dequantised
// tiles, deep enough that a tile waits in it from its scores to its pooling
// while the next ones are made.
//
// Warps (16): 0 copies, 1 issues the MMAs, 4-7 and 8-11 the softmax of tokens
// 0-31 and 32-63 of a tile (lane = query row), 12-15 dequantise.  The rescale
// of a row's accumulator is decided by the two warps that hold its row.
// Every wait is bounded (FSQ_ERR_TIMEOUT), as in the other decode kernels.
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
constexpr int kThreads = 512;
constexpr int kAtom = 64;                          // coordinates of a swizzled atom row (128 bytes)
constexpr int kAtomBytes = kTile * 128;            // 64 coordinates of a tile
constexpr int kMaxG = 256;                         // O, Q' and two S buffers fill TMEM
constexpr int kMaxStages = 6, kMaxZ = 6, kMaxS = 4;
constexpr int kDqWarps = 4;
constexpr int kMiscBytes = 2048;
constexpr size_t kSmemMax = 227 * 1024;
// A row's reference m enters P as 2^kLift and moves when a score exceeds it by
// 2^kTau, so P stays below 2^15 (fp16 ends at 2^16) and weights count down to
// 2^-26 of the reference.  Random scores climb a few powers of two beyond a
// tile's first maximum; moving O costs 1.5k cycles of a tile's 1.3k, so the
// window is as wide as fp16 lets it be (kTau = 8: 97 us at G = 256, 131072
// shared tokens, 16 rows; 13: see the table).
constexpr float kTau = 13.f;
constexpr float kLift = 2.f;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainNs = 1000000000ull;

// Shared-memory and TMEM plan of a CTA.
struct Plan {
  int Gp, NA, R, stages, nz, ns;
  uint32_t z_bytes, stage_bytes, off_c, off_misc, total, col_q, col_s;
};
__host__ __device__ inline Plan plan_of(int G, int bits) {
  Plan p;
  p.Gp = (G + 15) / 16 * 16;
  p.NA = (G + kAtom - 1) / kAtom;
  p.R = G * bits / 8;
  p.nz = kMaxZ;
  p.z_bytes = (uint32_t)(p.NA * kAtomBytes);
  p.off_c = p.nz * p.z_bytes;
  // +16: the last token's last group may read past its row
  p.stage_bytes = (uint32_t)(kTile * p.R + 16 + 127) / 128 * 128;
  p.stages = (int)((kSmemMax - kMiscBytes - p.off_c) / p.stage_bytes);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.off_misc = p.off_c + p.stages * p.stage_bytes;
  p.total = p.off_misc + kMiscBytes;
  p.col_q = p.Gp;
  p.col_s = p.col_q + p.Gp / 2;
  p.ns = (int)(512 - p.col_s) / kTile;
  if (p.ns > kMaxS) p.ns = kMaxS;
  return p;
}

struct Params {
  const uint8_t *shared;    // [Tp] rows
  const uint8_t *codes;     // own rows
  int64_t bstride, Tp, T;
  const int32_t *seq_lens;
  const uint8_t *qbuf;      // Q', fp16 [B n_q][NA 64], physical order
  const float *sig;         // [B n_q] score scales
  float *part;              // [B][S][n_q][2 + G]
  uint32_t *err;
  int B, n_q, G, rpt;       // rpt: batch rows per query tile
  int QT, Sp, Ss, k;        // query tiles, splits of the prefix and of a row's own tokens, tiles per split
  uint32_t stall_ns;
};

struct Misc {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t z_ready[kMaxZ], z_free[kMaxZ];  // z_free: the tile's pooling is done
  uint64_t s_full[kMaxS], p_ready[kMaxS];
  uint64_t q_ready, done, never;
  uint32_t tmem_base, abort;
  float mx[2][kRows];
};
static_assert(sizeof(Misc) <= kMiscBytes, "Misc block exceeds its reservation");

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
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.p_ready[i], 8);
    }
    mbar_init(&ms.q_ready, 8);
    mbar_init(&ms.done, 1);
    mbar_init(&ms.never, 1);  // completed by nothing: the test-only stall waits on it
    ms.abort = 0u;
    fence_mbar_init();
  }
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
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (whole warp, one lane issues)
    constexpr uint32_t id_s = idesc_f16(kRows, kTile, 0, 0);
    const uint32_t id_o = idesc_f16(kRows, Gp, 0, 1), el = elect_one();
    Ring zs, zp, ss, sp, old;  // tile and S buffer of the next scores; of the next pooling; tile whose S is overwritten
    auto scores = [&](int i) -> bool {
      if (i >= ns) {  // this S buffer holds P(i - ns): its pooling must be done
        if (!warp_wait(&ms.z_free[old.slot], old.par, abort, kWaitNs)) return false;
        old.next(nz);
      }
      if (!warp_wait(&ms.z_ready[zs.slot], zs.par, abort, kWaitNs)) return false;
      tc_fence_after();
      const uint32_t d = tm + pl.col_s + ss.slot * kTile, a = tm + pl.col_q;
      const uint32_t b = swz_lo(z_a + zs.slot * pl.z_bytes, 16);
#pragma unroll
      for (int k = 0; k < kMaxG / 16; ++k) {
        if (16 * k >= Gp) break;
        mma_ts_warp(el, d, a + 8 * k, b + (((k >> 2) * kAtomBytes + (k & 3) * 32) >> 4), id_s, k > 0 ? 1u : 0u);
      }
      if (el) tc_commit(&ms.s_full[ss.slot]);
      __syncwarp();
      zs.next(nz);
      ss.next(ns);
      return true;
    };
    bool ok = warp_wait(&ms.q_ready, 0, abort, kWaitNs) && scores(0);
    for (int i = 0; ok && i < n_tiles; ++i) {
      if (i + 1 < n_tiles) ok = scores(i + 1);
      ok = ok && warp_wait(&ms.p_ready[sp.slot], sp.par, abort, kWaitNs);
      if (!ok) break;
      tc_fence_after();
      const uint32_t a = tm + pl.col_s + sp.slot * kTile;
      const uint32_t b = swz_lo(z_a + zp.slot * pl.z_bytes, kAtomBytes);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_ts_warp(el, tm, a + 8 * k, b + ((k * 2048) >> 4), id_o, k > 0 || i > 0 ? 1u : 0u);
      if (el) tc_commit(&ms.z_free[zp.slot]);
      __syncwarp();
      zp.next(nz);
      sp.next(ns);
    }
    if (!ok && lane == 0) fail();
    // every issued MMA finishes before TMEM is freed
    tc_commit_elect(&ms.done);
    mbar_wait_fixed(&ms.done, 0, kDrainNs);
  } else if (warp >= 12) {
    // ------------------------------------------------------------ dequantisation
    const int dt = tid - 12 * 32;
    const int align = R % 16 == 0 ? 16 : R % 4 == 0 ? 4 : R % 2 == 0 ? 2 : 1;
    const int units = (G + 7) / 8;   // groups of 8 coordinates that hold codes
    // the groups behind them stay zero
    for (int i = dt; i < kTile * (8 * NA - units) * nz; i += kDqWarps * 32) {
      const int t = i % kTile, x = i / kTile;
      *reinterpret_cast<uint4 *>(smem + (x % nz) * pl.z_bytes + z_at(t, units + x / nz)) = make_uint4(0u, 0u, 0u, 0u);
    }
    Ring cr, zr;
    for (int i = 0; i < n_tiles; ++i, cr.next(stages), zr.next(nz)) {
      if (!warp_wait(&ms.full[cr.slot], cr.par, &ms.z_free[zr.slot], zr.par ^ 1u, abort, kWaitNs)) {
        if (lane == 0) fail();
        break;
      }
      const uint8_t *c = smem + pl.off_c + cr.slot * pl.stage_bytes;
      uint8_t *z = smem + zr.slot * pl.z_bytes;
      if (align == 16) {
        // 16 bytes of a row at a time, in order: the reads are contiguous over
        // the warp and the swizzle spreads the writes over the banks
        const int ppr = R / 16;
        const uint32_t inv = (65536u + ppr - 1) / ppr;  // x / ppr for x < 64 * 16
#pragma unroll 4
        for (int x = dt; x < kTile * ppr; x += kDqWarps * 32) {
          const int t = (int)(((uint32_t)x * inv) >> 16), piece = x - t * ppr;
          const uint4 v = *reinterpret_cast<const uint4 *>(c + 16 * x);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if constexpr (BITS == 8) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4 *>(z + z_at(t, 2 * piece + e)) = levels8<8>(w[2 * e], w[2 * e + 1]);
          } else if constexpr (BITS == 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4 *>(z + z_at(t, 4 * piece + e)) = levels8<4>(w[e], 0u);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4 *>(z + z_at(t, 8 * piece + e)) = levels8<2>(w[e / 2] >> (16 * (e & 1)), 0u);
          }
        }
      } else {
        // a token's even or odd groups per thread
        const int t = dt % kTile;
        const uint8_t *rowp = c + t * R;
#pragma unroll 4
        for (int u = dt / kTile; u < units; u += kDqWarps * 32 / kTile)
          *reinterpret_cast<uint4 *>(z + z_at(t, u)) = group8<BITS>(rowp, u, align);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.z_ready[zr.slot]);
        mbar_arrive(&ms.empty[cr.slot]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax: lane = query row, 32 tokens
    const int wg = (warp - 4) >> 2, q4 = warp & 3;
    const int r = 32 * q4 + lane;
    const bool busy = 32 * q4 < r_hi && 32 * q4 + 32 > r_lo;  // this warp has live rows
    const bool live = r >= r_lo && r < r_hi;
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    const int pair = 1 + q4;  // barrier of the two warps of these rows
    bool ok = true;
    pdl_wait();  // Q' and sig come from the query prologue
    float sig = 0.f;
    {
      // half of the row's Q' into TMEM; rows without a query are zero
      const uint8_t *qr = p.qbuf + ((int64_t)qt * p.rpt * p.n_q + r) * (NA * 128);
      if (live) sig = p.sig[(int64_t)qt * p.rpt * p.n_q + r];
#pragma unroll 4
      for (int c = 8 * wg; c < Gp / 2; c += 16) {  // columns: two coordinates each
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (live) {
          a = *reinterpret_cast<const uint4 *>(qr + 4 * c);
          b = *reinterpret_cast<const uint4 *>(qr + 4 * c + 16);
        }
        const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        tmem_st8(tm + lanes + pl.col_q + c, v);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.q_ready);
    }
    // test-only stall: a wait that runs out on purpose (nothing completes `never`)
    if (p.stall_ns != 0u && !warp_wait(&ms.never, 0, abort, p.stall_ns)) ok = false;
    float m = -INFINITY, l = 0.f;
    Ring sr, zo;  // S buffer of the tile; tile before it
    for (int i = 0; i < n_tiles; ++i, sr.next(ns)) {
      ok = ok && warp_wait(&ms.s_full[sr.slot], sr.par, abort, kWaitNs);
      tc_fence_after();
      uint32_t s[32];
      float top = -INFINITY;
      const uint32_t ts = tm + lanes + pl.col_s + sr.slot * kTile;
      if (busy) {
        tmem_ld32(ts + 32 * wg, s);
        tmem_ld_wait();
        const int valid = (int)min((int64_t)kTile, t1 - (t0 + (int64_t)i * kTile)) - 32 * wg;  // tokens of this half
        if (valid < 32) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c >= valid) s[c] = 0xFF800000u;  // -inf
        }
        float t2[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 32; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            t2[e] = fmax3f(t2[e], __uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1]));
        top = fmaxf(fmaxf(t2[0], t2[1]), fmaxf(t2[2], t2[3])) * sig;
        if (!live) top = -INFINITY;
      }
      // both warps have read S before P overwrites it; they decide together
      if (named_bar_or(pair, 64, !ok || top > m + kTau || (i == 0 && live))) {
        ms.mx[wg][r] = top;
        if (named_bar_or(pair, 64, !ok)) {
          ok = false;
          break;
        }
        const float mn = fmaxf(m, fmaxf(ms.mx[0][r], ms.mx[1][r]));
        const float f = mn == m ? 1.f : exp2f(m - mn);
        l *= f;
        m = mn;
        if (i > 0 && busy) {
          // O holds every earlier tile once the last pooling is done
          if (!warp_wait(&ms.z_free[zo.slot], zo.par, abort, kWaitNs)) ok = false;
          tc_fence_after();
#pragma unroll 1
          for (int c = 16 * wg; c < Gp; c += 64) {  // the warps take turns at 16 columns, two turns at once
            uint32_t a[32];
            const bool two = c + 32 < Gp;
            tmem_ld16(tm + lanes + c, a);
            if (two) tmem_ld16(tm + lanes + c + 32, a + 16);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * f);
            tmem_st16(tm + lanes + c, a);
            if (two) tmem_st16(tm + lanes + c + 32, a + 16);
          }
        }
      }
      if (busy) {
        const float off = kLift - m;
        uint32_t h[16];
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float e0 = ex2_approx(fmaf(__uint_as_float(s[2 * c]), sig, off));
          const float e1 = ex2_approx(fmaf(__uint_as_float(s[2 * c + 1]), sig, off));
          l4[(2 * c) & 3] += e0;
          l4[(2 * c + 1) & 3] += e1;
          const __half2 v = __floats2half2_rn(e0, e1);
          h[c] = *reinterpret_cast<const uint32_t *>(&v);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        tmem_st16(ts + 16 * wg, h);
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.p_ready[sr.slot]);
      if (i > 0) zo.next(nz);
    }
    // ---- epilogue: O through shared memory (the tiles are spent) to the partials
    if (ok) {
      const int z = (n_tiles - 1) % nz;
      ok = warp_wait(&ms.z_free[z], (uint32_t)((n_tiles - 1) / nz) & 1u, abort, kWaitNs);
    }
    if (!ok) fail();
    ms.mx[wg][r] = l;
    if (!named_bar_or(5, 256, !ok)) {
      tc_fence_after();
      float *stage = reinterpret_cast<float *>(smem);  // [128][Gp + 1]: conflict-free both ways
      const int ld = Gp + 1;
      if (busy) {
#pragma unroll 1
        for (int c = 16 * wg; c < Gp; c += 32) {
          uint32_t a[16];
          tmem_ld16(tm + lanes + c, a);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int g = c + (e & 8) + (BITS == 8 ? (e & 7) : ((e & 1) << 2) + ((e & 7) >> 1));
            stage[r * ld + g] = __uint_as_float(a[e]);
          }
        }
      }
      named_bar(5, 256);
      for (int rr = r_lo + (warp - 4); rr < r_hi; rr += 8) {
        float *out = record(rr);
        for (int g = lane; g < G; g += 32) out[2 + g] = stage[rr * ld + g];
      }
      if (live && wg == 0) {
        float *out = record(r);
        out[0] = m - kLift;
        out[1] = ms.mx[0][r] + ms.mx[1][r];
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
// weight into [1, 2), as a row of fp16 in physical order; sig_h takes the power
// back.  Also clears the error word.
template <int BITS>
__global__ void __launch_bounds__(kAbsorbThreads, 1) prefix_query(const uint16_t *__restrict__ q,
                                                               const uint16_t *__restrict__ W_kv, int n_q, int n_kv,
                                                               int G, int NA, float c, uint8_t *__restrict__ qbuf,
                                                               float *__restrict__ sig, uint32_t *err) {
  __shared__ AbsorbSmem<kMaxG> sm;
  const int64_t b = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && b == 0 && threadIdx.x == 0) *err = 0u;
  absorb_heads(
      sm, q, W_kv, n_q, n_kv, G, NA * kAtom, c, blockIdx.x, b,
      [&](int h, int g, float v, int e) {
        reinterpret_cast<__half *>(qbuf)[(b * n_q + h) * (NA * kAtom) + ((g & ~7) | order_of<BITS>(g & 7))] =
            __float2half_rn(scalbnf(v, -e));
      },
      [&](int h, int e) { sig[b * n_q + h] = scalbnf(1.f, e); });
}

// ---------------------------------------------------------------- split merge
// Per (kv head j, batch row b): the group's heads, four at a time,
//   m = max_s m_s,  w_s = 2^(m_s - m),  abar_h = sum_s w_s O_s / sum_s w_s l_s,  o_h = W_v^(j) abar_h.
// A thread sums one coordinate pair of one head over its share of the splits
// (the loads of eight splits are in flight together); a warp then takes eight
// rows of W_v, loaded into registers before the wait for the split kernel.
constexpr int kMergeThreads = 512, kMergeHeads = 4, kMergeRows = FSQ_HEAD_DIM / (kMergeThreads / 32);
constexpr int kMaxSplits = 2048;  // of a row

// VEC: coordinates a lane reads of a W_v row at once (4, or 2 where G is not a multiple of 4)
template <int VEC>
__global__ void __launch_bounds__(kMergeThreads, 1) prefix_merge(const float *__restrict__ part, int S, int n_q, int n_kv,
                                                              int G, const uint16_t *__restrict__ W_kv, void *o,
                                                              int out_fp32) {
  constexpr int D = FSQ_HEAD_DIM, STEPS = kMaxG / (32 * VEC);
  extern __shared__ __align__(16) float wts[];  // [kMergeHeads][S]: w_s / sum
  __shared__ float2 sum[kMergeThreads];
  __shared__ __align__(16) float abar[kMergeHeads][kMaxG];
  const int j = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.y;
  const int grp = n_q / n_kv;
  // rows kMergeRows * warp .. of W_v^(j); coordinates 32 VEC i + VEC lane ..
  uint32_t w[kMergeRows][STEPS][VEC / 2];
#pragma unroll
  for (int r = 0; r < kMergeRows; ++r)
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int g = 32 * VEC * i + VEC * lane;
      const uint16_t *src = W_kv + ((int64_t)(n_kv + j) * D + warp * kMergeRows + r) * G + g;
      if constexpr (VEC == 4) {
        const uint2 v = g < G ? *reinterpret_cast<const uint2 *>(src) : make_uint2(0u, 0u);
        w[r][i][0] = v.x, w[r][i][1] = v.y;
      } else {
        w[r][i][0] = g < G ? *reinterpret_cast<const uint32_t *>(src) : 0u;
      }
    }
  pdl_wait();
  const int64_t hs = 2 + G, ss = (int64_t)n_q * hs;  // floats of a record, of a split
  for (int h0 = 0; h0 < grp; h0 += kMergeHeads) {
    const int nh = min(kMergeHeads, grp - h0);
    const float *rec = part + (b * S * n_q + (int64_t)j * grp + h0) * hs;
    if (warp < nh) {  // a warp per head: the splits' weights
      float m = -INFINITY, l = 0.f;
      for (int s = lane; s < S; s += 32) m = fmaxf(m, rec[s * ss + warp * hs]);
#pragma unroll
      for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      for (int s = lane; s < S; s += 32) {
        const float2 ml = *reinterpret_cast<const float2 *>(rec + s * ss + warp * hs);
        const float e = exp2f(ml.x - m);  // 0 for an empty split
        wts[warp * S + s] = e;
        l = fmaf(e, ml.y, l);
      }
#pragma unroll
      for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
      const float inv = 1.f / l;
      for (int s = lane; s < S; s += 32) wts[warp * S + s] *= inv;
    }
    __syncthreads();
    const int pairs = G / 2, items = nh * pairs, nsub = min(16, max(1, kMergeThreads / items));
    {
      const int it = tid % items, sub = tid / items, h = it / pairs, x = it % pairs;  // items <= 4 * 128
      float2 a = make_float2(0.f, 0.f);
      if (sub < nsub) {
        const float *src = rec + h * hs + 2 + 2 * x;
#pragma unroll 8
        for (int s = sub; s < S; s += nsub) {
          const float2 v = *reinterpret_cast<const float2 *>(src + s * ss);
          const float e = wts[h * S + s];
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
    }
    __syncthreads();
    // lane 4 r + h keeps row r of head h
    static_assert(kMergeRows * kMergeHeads == 32, "a lane per result");
    float mine = 0.f;
#pragma unroll
    for (int r = 0; r < kMergeRows; ++r) {
      float acc[kMergeHeads] = {};
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int g = 32 * VEC * i + VEC * lane;
        if (g >= G) break;
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float lo = __uint_as_float(w[r][i][e / 2] << 16), hi = __uint_as_float(w[r][i][e / 2] & 0xFFFF0000u);
#pragma unroll
          for (int h = 0; h < kMergeHeads; ++h) {
            const float2 a = *reinterpret_cast<const float2 *>(&abar[h][g + e]);
            acc[h] = fmaf(lo, a.x, fmaf(hi, a.y, acc[h]));
          }
        }
      }
#pragma unroll
      for (int h = 0; h < kMergeHeads; ++h) {
        float v = acc[h];
#pragma unroll
        for (int k = 16; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
        if (lane == 4 * r + h) mine = v;
      }
    }
    if (lane % 4 < nh) {
      const int64_t at = ((b * n_q + (int64_t)j * grp + h0 + lane % 4) * D) + warp * kMergeRows + lane / 4;
      if (out_fp32) reinterpret_cast<float *>(o)[at] = mine;
      else reinterpret_cast<uint16_t *>(o)[at] = f32_to_bf16_rn(mine);
    }
    __syncthreads();
  }
}

template <int BITS>
cudaError_t launch_t(const uint16_t *q, const uint16_t *W_kv, int n_kv, float scale, const Params &p, uint8_t *qbuf,
                     float *sig, void *o, int out_fp32, void *const *prof, cudaStream_t st) {
  const Plan pl = plan_of(p.G, BITS);
  cudaError_t e = launch_pdl(prefix_query<BITS>, dim3(n_kv, (unsigned)p.B), dim3(kAbsorbThreads), 0, st, q, W_kv, p.n_q, n_kv,
                             p.G, pl.NA, scale * kLog2e, qbuf, sig, p.err);
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
  auto merge = p.G % 4 == 0 ? prefix_merge<4> : prefix_merge<2>;
  return launch_pdl(merge, dim3(n_kv, (unsigned)p.B), dim3(kMergeThreads), sizeof(float) * kMergeHeads * S, st,
                    (const float *)p.part, S, p.n_q, n_kv, p.G, W_kv, o, out_fp32);
}

}  // namespace prefix
}  // namespace tc

bool prefix_supported(int n_q, int G) { return n_q <= tc::prefix::kRows && G <= tc::prefix::kMaxG; }
int prefix_rows_per_tile(int n_q) { return tc::prefix::kRows / n_q; }
int prefix_max_splits() { return tc::prefix::kMaxSplits; }
int prefix_tile_tokens() { return tc::prefix::kTile; }
size_t prefix_query_bytes(int G) {  // Q' of one query head
  return (size_t)((G + tc::prefix::kAtom - 1) / tc::prefix::kAtom) * tc::prefix::kAtom * 2;
}

cudaError_t launch_prefix(const uint16_t *q, int64_t B, int n_q, int n_kv, const uint8_t *shared, int64_t Tp,
                          const uint8_t *codes, int64_t bstride, int64_t T, const int32_t *seq_lens, int G, int bits,
                          const uint16_t *W_kv, float scale, int QT, int Sp, int Ss, int k, uint8_t *qbuf, float *sig,
                          float *part, uint32_t *err, void *o, int out_fp32, uint32_t stall_ns,
                          void *const *prof, cudaStream_t st) {
  tc::prefix::Params p{shared, codes, bstride, Tp, T, seq_lens, qbuf, sig, part, err,
                       (int)B, n_q, G, prefix_rows_per_tile(n_q), QT, Sp, Ss, k, stall_ns};
  return bits == 2   ? tc::prefix::launch_t<2>(q, W_kv, n_kv, scale, p, qbuf, sig, o, out_fp32, prof, st)
         : bits == 4 ? tc::prefix::launch_t<4>(q, W_kv, n_kv, scale, p, qbuf, sig, o, out_fp32, prof, st)
                     : tc::prefix::launch_t<8>(q, W_kv, n_kv, scale, p, qbuf, sig, o, out_fp32, prof, st);
}

}  // namespace fsq
