// Eviction from the code cache by accumulated attention weight.
//
// Row b holds L_b tokens with weights acc[b][t].  It keeps its last n_recent
// tokens and, of the others, the n_keep - n_recent with the largest weight
// (equal weights: the lowest index first); the kept rows move to the front of
// the row in their order.  Rows of at most n_keep tokens keep everything.
//
// Two kernels:
//  evict_select   one thread-block cluster per row finds the weight of the last
//                 token that stays, by a radix select over order-preserving
//                 32-bit keys (digits of 11, 11 and 10 bits: histograms in
//                 shared memory, added up over the cluster; up to 131072 tokens
//                 the keys stay in registers), then writes one keep bit per token
//                 and each chunk's position in the packed row.
//  evict_compact  one CTA per chunk of tokens copies its kept rows, weights and
//                 indices to their places.
//
// Bound by memory: 4 bytes of weight per token, twice the code bytes of every
// kept token.  In place, a chunk's destination lies at or before its source,
// in the sources of at most two earlier chunks: a chunk loads its kept rows
// into registers or shared memory, publishes that it has, waits until the
// chunks it overwrites have published the same, and stores.  Chunks are taken in
// ascending order from a counter, and a chunk publishes before it waits, so the
// chunks waited for are always running or done: the wait ends whatever the
// scheduling.  It is bounded all the same (FSQ_ERR_TIMEOUT; the row is then left as it is,
// part moved).
//
// Measured, 16 rows of 131072 tokens cut to 65536, 128-byte rows: select 34 us,
// compaction 56 us (277 MB: 5.0 TB/s); one row of 2048: 7.2 and 2.9 us.  The select
// is a chain of about twenty barriers and dependent reads, not bandwidth.
#include <cooperative_groups.h>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace fsq {
namespace evict {

constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kHeld = 32;              // most words of a select warp whose keys stay in registers
constexpr int kCopyNT = 256;           // threads of a compaction CTA
constexpr int kCopyBytes = 32 * 1024;  // code bytes of a chunk
constexpr uint64_t kWaitNs = 1000000000ull;

// Tokens per chunk: a power of two of at least 32 tokens (whole keep words, and
// a chunk's first row 16-byte aligned) with at most kCopyBytes of codes, or 32.
__host__ __device__ inline int chunk_tokens(int R) {
  int c = 1024;
  while (c > 32 && c * R > kCopyBytes) c >>= 1;
  return c;
}

struct Plan {
  int R, chunk;
  int64_t nchunk, words;  // per row
  size_t off_rows, off_bits, off_off, off_flag, off_ticket, total;
};
inline Plan plan_of(int64_t B, int64_t T, int R) {
  Plan p;
  p.R = R;
  p.chunk = chunk_tokens(R);
  p.nchunk = (T + p.chunk - 1) / p.chunk;
  p.words = p.nchunk * (p.chunk / 32);
  size_t off = kWsHeader;
  p.off_rows = off;  // per row: length before, length after, whether the given length was out of range
  off = align_up(off + 3 * sizeof(int32_t) * (size_t)B, 256);
  p.off_bits = off;
  off = align_up(off + sizeof(uint32_t) * (size_t)(B * p.words), 256);
  p.off_off = off;
  off = align_up(off + sizeof(int32_t) * (size_t)(B * p.nchunk), 256);
  p.off_flag = off;
  off = align_up(off + sizeof(uint32_t) * (size_t)(B * p.nchunk), 256);
  p.off_ticket = off;
  off = align_up(off + sizeof(uint32_t), 256);
  p.total = off;
  return p;
}

// Order-preserving key: larger weight, larger key; -0 equals +0; NaN is below
// every number.
__device__ __forceinline__ uint32_t key_of(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

struct SelectParams {
  const float *acc;
  int64_t acc_stride;
  const int32_t *lens;
  int64_t T, n_keep, n_recent;
  int32_t *rows;    // [B][3]
  uint32_t *bits;   // [B][words]
  int32_t *off;     // [B][nchunk]
  uint32_t *flag;   // [B][nchunk]
  uint32_t *ticket;
  uint32_t *err;
  int32_t *lens_out, *kept;
  int64_t nchunk, words;
  int chunk;
};

// Exclusive prefix of `v` over the CTA's NT threads; *total: the sum.  red has
// NT / 32 entries; two barriers.
template <int NT>
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t *red, uint32_t *total) {
  static_assert(NT / 32 <= 32, "reads one warp total per lane");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += n;
  }
  if (lane == 31) red[warp] = s;
  __syncthreads();
  const uint32_t w = lane < NT / 32 ? red[lane] : 0u;
  uint32_t ws = w;
#pragma unroll
  for (int o = 1; o < NT / 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(0xffffffffu, ws, o);
    if (lane >= o) ws += n;
  }
  *total = __shfl_sync(0xffffffffu, ws, NT / 32 - 1);
  const uint32_t before = __shfl_sync(0xffffffffu, ws - w, warp);
  __syncthreads();
  return before + s - v;
}

// The CTA's segment is `per` 32-token words per warp, a warp's words in a row.
// HELD: per <= HELD and the keys stay in registers; 0: they are read again
// (from L2) in each pass.  Latency counts: every CTA sums all bins of the cluster
// itself, so that a pass has one cluster barrier, and each pass has a histogram of
// its own; one CTA's worth of tokens takes 256 threads, whose barriers are quick.
template <int NT, int HELD>
__global__ void __launch_bounds__(NT, 1024 / NT) evict_select(SelectParams p, int per) {
  constexpr int NW = NT / 32, BPT = kBins / NT;  // bins per thread
  cg::cluster_group cl = cg::this_cluster();
  const int CS = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  __shared__ __align__(16) uint32_t hist[3][kBins];  // per pass: this CTA's keys by digit
  __shared__ uint32_t found[3];                       // digit, keys still to keep inside it, keys inside it
  __shared__ uint32_t total[2][kMaxCluster];          // per rank: ties, kept tokens of its segment (written by the ranks)
  __shared__ uint32_t red[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.x / CS;
  auto sync = [&]() {
    if (CS > 1) cl.sync();
    else __syncthreads();
  };
  // A CTA's shared memory may be touched by the others only once it runs, which the
  // cluster's first barrier tells: arrived at here, waited for behind the loads
  // below, before any remote access, whichever of them a row's length leads to.
  if (CS > 1) cl.barrier_arrive();
  pdl_wait();
  const int64_t given = p.lens ? p.lens[b] : p.T;
  const int64_t L = given < 0 ? 0 : (given > p.T ? p.T : given);
  const int64_t after = min(L, p.n_keep);
  const int64_t w0 = ((int64_t)rank * NW + warp) * per;  // this warp's first word
  const float *acc = p.acc + b * p.acc_stride;
  // the segment's chunks (a power of two of words, at most 32 of them)
  const int cw = p.chunk / 32;
  for (int64_t c = (int64_t)rank * NW * per / cw + tid; c < min(p.nchunk, ((int64_t)(rank + 1) * NW * per + cw - 1) / cw);
       c += NT)
    p.flag[b * p.nchunk + c] = 0u;
  if (blockIdx.x == 0 && tid == 0) {
    *p.ticket = 0u;
    *p.err = 0u;
  }
  const bool cut = L > p.n_keep;
  const int64_t N = cut ? L - p.n_recent : 0;  // candidates
  const uint32_t need = cut ? (uint32_t)(p.n_keep - p.n_recent) : 0u;  // of which stay
  uint32_t held[HELD ? HELD : 1];
  if constexpr (HELD > 0) {
    float v[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int64_t t = (w0 + i) * 32 + lane;
      v[i] = i < per && t < N ? acc[t] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = key_of(v[i]);
  }
  // f(i, token, key) for this thread's candidates
  auto each = [&](auto f) {
    if constexpr (HELD > 0) {
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (i < per) f(i, (w0 + i) * 32 + lane, held[i]);
    } else {
      for (int i = 0; i < per; ++i) {
        const int64_t t = (w0 + i) * 32 + lane;
        f(i, t, t < N ? key_of(acc[t]) : 0u);
      }
    }
  };
  if (CS > 1) cl.barrier_wait();
  uint32_t limit = 0, ties = need, equal = need;  // key of the last one that stays; how many of the keys equal to it do, of how many
  if (need > 0) {
    int shift = 32;
    for (int i = tid; i < 3 * kBins; i += NT) hist[0][i] = 0u;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bitsn = pass < 2 ? 11 : 10, bins = 1 << bitsn;  // the last pass leaves the upper half of the bins empty
      const uint32_t above = shift == 32 ? 0u : (0xFFFFFFFFu << shift);
      shift -= bitsn;
      uint32_t *h = hist[pass];
      each([&](int, int64_t t, uint32_t k) {
        if (t < N && (k & above) == limit) atomicAdd(&h[(k >> shift) & (bins - 1)], 1u);
      });
      sync();
      // BPT bins a thread, from the top
      const int hi = kBins - BPT * (tid + 1);
      uint32_t m[BPT] = {};
#pragma unroll
      for (int r0 = 0; r0 < kMaxCluster; r0 += 4) {  // four CTAs' bins in flight
        uint4 v[4][BPT / 4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int x = 0; x < BPT / 4; ++x)
            v[r][x] = r0 + r < CS ? *reinterpret_cast<const uint4 *>(cl.map_shared_rank(h, r0 + r) + hi + 4 * x)
                                  : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int x = 0; x < BPT / 4; ++x)
            m[4 * x] += v[r][x].x, m[4 * x + 1] += v[r][x].y, m[4 * x + 2] += v[r][x].z, m[4 * x + 3] += v[r][x].w;
      }
      uint32_t mine = 0, sum;
#pragma unroll
      for (int x = 0; x < BPT; ++x) mine += m[x];
      uint32_t n = block_prefix<NT>(mine, red, &sum);  // keys in the bins above this thread's
      if (n < ties && ties <= n + mine) {  // one thread
#pragma unroll
        for (int x = BPT - 1; x >= 0; --x) {
          if (n < ties && ties <= n + m[x]) {
            found[0] = (uint32_t)(hi + x);
            found[1] = ties - n;
            found[2] = m[x];
          }
          n += m[x];
        }
      }
      __syncthreads();
      limit |= found[0] << shift;
      ties = found[1];
      equal = found[2];
      __syncthreads();
    }
  }
  // ties before this warp's tokens, where not all of them stay
  uint32_t eq_before = 0;
  if (ties < equal) {
    uint32_t eq = 0, sum;
    each([&](int, int64_t t, uint32_t k) { eq += t < N && k == limit ? 1u : 0u; });
    eq = block_prefix<NT>(eq, red, &sum);
    eq_before = __shfl_sync(0xffffffffu, eq, 0);
    if (CS > 1) {
      if (tid < CS) cl.map_shared_rank(total[0], tid)[rank] = sum;
      cl.sync();
      for (int r = 0; r < rank; ++r) eq_before += total[0][r];
    }
  }
  // keep words: a candidate above the limit, or equal to it and among the first
  // `ties`; every token from N to L.  Lane i keeps the i-th word of a round of 32.
  uint32_t kept = 0;  // of the warp, so far
  uint32_t mine = 0;
  auto flush = [&](int64_t word0, int n) {  // words word0 .. word0 + n - 1 are in lanes 0 .. n - 1
    const int64_t w = word0 + lane;
    uint32_t c = lane < n ? __popc(mine) : 0u, s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += v;
    }
    if (lane < n && w < p.words) {
      p.bits[b * p.words + w] = mine;
      if (w % cw == 0) p.off[b * p.nchunk + w / cw] = (int32_t)(kept + s - c);  // within the warp, so far
    }
    kept += __shfl_sync(0xffffffffu, s, 31);
  };
  auto keep_word = [&](int i, int64_t t, uint32_t k) {
    const bool same = need > 0 && t < N && k == limit;
    const uint32_t eq = __ballot_sync(0xffffffffu, same);
    const bool first = same && eq_before + __popc(eq & ((1u << lane) - 1u)) < ties;
    eq_before += __popc(eq);
    const uint32_t word = __ballot_sync(0xffffffffu, t < L && (t >= N || first || (need > 0 && k > limit)));
    if (lane == (i & 31)) mine = word;
    if (HELD == 0 && ((i & 31) == 31 || i == per - 1)) flush(w0 + (i & ~31), (i & 31) + 1);
  };
  each(keep_word);
  if constexpr (HELD > 0) flush(w0, per);  // per <= 32; outside the unrolled loop, whose code has to fit its cache
  uint32_t sum;
  uint32_t base = block_prefix<NT>(lane == 0 ? kept : 0u, red, &sum);  // kept tokens of the warps before this one
  base = __shfl_sync(0xffffffffu, base, 0);
  if (CS > 1) {
    if (tid < CS) cl.map_shared_rank(total[1], tid)[rank] = sum;
    cl.sync();  // also: every CTA of the cluster has read lens[b], which lens_out may alias, and the others' histograms
    for (int r = 0; r < rank; ++r) base += total[1][r];
  }
  for (int64_t w = (w0 + cw - 1) / cw * cw + (int64_t)lane * cw; w < min(p.words, w0 + per); w += 32 * cw)
    p.off[b * p.nchunk + w / cw] += (int32_t)base;
  if (rank == 0 && tid == 0) {
    p.rows[3 * b] = (int32_t)L;
    p.rows[3 * b + 1] = (int32_t)after;
    p.rows[3 * b + 2] = given != L ? 1 : 0;
    if (p.lens_out) p.lens_out[b] = (int32_t)after;
  }
  if (p.kept)
    for (int64_t i = after + (int64_t)rank * NT + tid; i < p.n_keep; i += (int64_t)CS * NT) p.kept[b * p.n_keep + i] = -1;
}

struct CopyParams {
  const uint8_t *codes;
  uint8_t *out;
  int64_t bstride, ostride;
  const float *acc;
  float *acc_out;
  int64_t acc_stride, acc_ostride;
  int32_t *kept;
  const int32_t *rows;
  const uint32_t *bits;
  const int32_t *off;
  uint32_t *flag, *ticket, *err;
  int64_t B, T, n_keep, nchunk, words;
  int R, chunk, in_place;
};

__device__ __forceinline__ uint32_t load_acquire(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(uint32_t *p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// U: bytes that are moved at once (the largest power of two up to 16 dividing
// a row).  Rows of whole 16-byte pieces are loaded one by one, only the kept
// ones, into registers; others come with their whole chunk into shared memory
// (aligned, contiguous loads), and the packed bytes are put together there.
template <int U>
__global__ void __launch_bounds__(kCopyNT, 4) evict_compact(CopyParams p) {
  extern __shared__ __align__(16) uint8_t stage[];  // U < 16: the chunk's code bytes
  __shared__ uint16_t list[1024];                   // kept tokens of the chunk
  __shared__ uint32_t order;
  __shared__ int go;
  const int tid = threadIdx.x;
  pdl_wait();
  uint32_t job = blockIdx.x;
  if (p.in_place) {
    if (tid == 0) order = atomicAdd(p.ticket, 1u);
    __syncthreads();
    job = order;
  }
  // rows side by side, chunks ascending
  const int64_t c = job / (uint32_t)p.B, b = job - c * (uint32_t)p.B;
  const int64_t t0 = (int64_t)c * p.chunk;
  // all that does not depend on one another in flight together: the row's lengths,
  // the chunk's place, its keep words (lane = word, in every warp) and its weights
  const int nw = p.chunk / 32, lane = tid & 31;
  const int64_t L = p.rows[3 * b], after = p.rows[3 * b + 1];
  const int bad = p.rows[3 * b + 2];
  const int64_t dst = p.off[b * p.nchunk + c];
  const uint32_t word = lane < nw ? p.bits[b * p.words + t0 / 32 + lane] : 0u;
  const float *acc = p.acc + b * p.acc_stride + t0;
  float av[4];  // of tokens tid + k kCopyNT; chunk <= 4 kCopyNT
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = tid + k * kCopyNT;
    av[k] = t < p.chunk && t0 + t < p.T ? acc[t] : 0.f;
  }
  if (c == 0 && tid == 0 && bad) record_error(p.err, FSQ_ERR_INVALID_ARG);  // the word is clear by now
  if (t0 >= L) return;  // nothing here; nobody waits for a chunk behind the last token
  const bool still = p.in_place && L == after;  // nothing moves
  // every warp: kept tokens before each word; then the chunk's kept tokens, ascending
  uint32_t upto = __popc(word);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  const int n = (int)__shfl_sync(0xffffffffu, upto, 31);
  int rank[4] = {-1, -1, -1, -1};  // of this thread's tokens among the kept ones, -1: not kept
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k * kCopyNT >= p.chunk) break;  // uniform
    const int t = tid + k * kCopyNT, w = t / 32;  // w < 32: the warp's word
    const uint32_t bits = __shfl_sync(0xffffffffu, word, w), to = __shfl_sync(0xffffffffu, upto, w);
    if (t < p.chunk && ((bits >> lane) & 1u)) {
      rank[k] = (int)(to - __popc(bits >> lane));
      list[rank[k]] = (uint16_t)t;
      if (p.kept) p.kept[b * p.n_keep + dst + rank[k]] = (int32_t)(t0 + t);
    }
  }
  if (still) return;
  __syncthreads();
  // ---- load
  constexpr int kRegs = kCopyBytes / 16 / kCopyNT;  // 16-byte pieces of a thread
  const uint8_t *src = p.codes + b * p.bstride + t0 * p.R;
  const int rows_here = (int)min((int64_t)p.chunk, L - t0);
  uint4 v[U == 16 ? kRegs : 1];
  if constexpr (U == 16) {
    const int ppr = p.R / 16;       // pieces per row
    const uint32_t inv = (65536u + ppr - 1) / ppr;  // x / ppr for x < 2048 (kCopyBytes / 16) and ppr <= 50; rows end at 36
#pragma unroll
    for (int k = 0; k < kRegs; ++k) {
      if (k * kCopyNT >= n * ppr) break;  // uniform: no index arithmetic for rows that go
      const int i = tid + k * kCopyNT;
      const int r = (int)((uint32_t)i * inv >> 16);
      if (i < n * ppr) v[k] = *reinterpret_cast<const uint4 *>(src + (int64_t)list[r] * p.R + (i - r * ppr) * 16);
    }
  } else {
    const int nb = rows_here * p.R;  // the row's bytes may end inside a 16-byte piece
    for (int i = tid; i < nb / 16; i += kCopyNT)
      *reinterpret_cast<uint4 *>(stage + 16 * i) = *reinterpret_cast<const uint4 *>(src + 16 * i);
    for (int i = nb / 16 * 16 + tid; i < nb; i += kCopyNT) stage[i] = src[i];
  }
  if (tid == 0) go = 1;
  __syncthreads();
  if (p.in_place) {
    // publish that this chunk is loaded, then wait for the chunks its destination covers
    if (tid == 0) {
      __threadfence();
      uint32_t *flag = p.flag + b * p.nchunk;
      store_release(flag + c, 1u);
      if (n > 0) {
        const uint64_t start = ptx::globaltimer_ns();
        for (int64_t d = dst / p.chunk; d <= (dst + n - 1) / p.chunk && d < c && go; ++d)
          while (load_acquire(flag + d) == 0u)
            if (ptx::globaltimer_ns() - start > kWaitNs) {
              record_error(p.err, FSQ_ERR_TIMEOUT);
              go = 0;
              break;
            }
      }
    }
    __syncthreads();
    if (!go) return;
  }
  // ---- store
  uint8_t *to = p.out + b * p.ostride + dst * p.R;
  if constexpr (U == 16) {
    const int ppr = p.R / 16;
#pragma unroll
    for (int k = 0; k < kRegs; ++k) {
      if (k * kCopyNT >= n * ppr) break;
      const int i = tid + k * kCopyNT;
      if (i < n * ppr) *reinterpret_cast<uint4 *>(to + (int64_t)i * 16) = v[k];
    }
  } else {
    // whole aligned 16-byte pieces of the destination, and the bytes at both ends
    const int nb = n * p.R;
    const int head = min(nb, (int)((16u - (uint32_t)((uintptr_t)to & 15u)) & 15u));
    auto byte_at = [&](int i) { return stage[(int)list[i / p.R] * p.R + i % p.R]; };
    for (int i = tid; i < head; i += kCopyNT) to[i] = byte_at(i);
    const int np = (nb - head) / 16;
    for (int i = tid; i < np; i += kCopyNT) {
      const int at = head + 16 * i;
      int r = at / p.R, x = at - r * p.R;  // x is a multiple of U, as the destination's offset and R are
      uint32_t w[4];
      const uint8_t *row = stage + (int)list[r] * p.R;
#pragma unroll
      for (int e = 0; e < 16 / U; ++e) {
        if constexpr (U == 8) {
          const uint2 q = *reinterpret_cast<const uint2 *>(row + x);
          w[2 * e] = q.x;
          w[2 * e + 1] = q.y;
        } else if constexpr (U == 4) {
          w[e] = *reinterpret_cast<const uint32_t *>(row + x);
        } else if constexpr (U == 2) {
          const uint32_t q = *reinterpret_cast<const uint16_t *>(row + x);
          w[e / 2] = (e % 2) ? (w[e / 2] | (q << 16)) : q;
        } else {
          const uint32_t q = row[x];
          w[e / 4] = (e % 4) ? (w[e / 4] | (q << (8 * (e % 4)))) : q;
        }
        x += U;
        if (x == p.R && e + 1 < 16 / U) {
          x = 0;
          row = stage + (int)list[++r] * p.R;
        }
      }
      *reinterpret_cast<uint4 *>(to + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    for (int i = head + 16 * np + tid; i < nb; i += kCopyNT) to[i] = byte_at(i);
  }
  float *ao = p.acc_out + b * p.acc_ostride;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (rank[k] >= 0) ao[dst + rank[k]] = av[k];
  // in place, the freed positions start from zero weight; they are this chunk's own
  if (p.in_place)
    for (int t = tid; t < rows_here; t += kCopyNT)
      if (t0 + t >= after) ao[t0 + t] = 0.f;
}

template <int U>
cudaError_t launch_copy(const CopyParams &p, cudaStream_t st) {
  const size_t smem = U < 16 ? align_up((size_t)p.chunk * p.R, 16) : 0;
  cudaError_t e = ensure_smem_limit((const void *)evict_compact<U>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(evict_compact<U>, dim3((unsigned)(p.B * p.nchunk)), dim3(kCopyNT), smem, st, p);
}

}  // namespace evict

size_t evict_workspace_bytes(int64_t B, int64_t T, int R) { return evict::plan_of(B, T, R).total; }
int64_t evict_jobs(int64_t B, int64_t T, int R) { return B * evict::plan_of(B, T, R).nchunk; }

cudaError_t launch_evict(const uint8_t *codes, int64_t bstride, const float *acc, int64_t acc_stride,
                         const int32_t *lens, int64_t B, int64_t T, int64_t n_keep, int64_t n_recent, int R,
                         uint8_t *out, int64_t ostride, float *acc_out, int64_t acc_ostride, int32_t *lens_out,
                         int32_t *kept, uint8_t *ws, cudaStream_t st) {
  using namespace evict;
  const Plan pl = plan_of(B, T, R);
  SelectParams sp{acc, acc_stride, lens, T, n_keep, n_recent, (int32_t *)(ws + pl.off_rows),
                  (uint32_t *)(ws + pl.off_bits), (int32_t *)(ws + pl.off_off), (uint32_t *)(ws + pl.off_flag),
                  (uint32_t *)(ws + pl.off_ticket), (uint32_t *)ws, lens_out, kept, pl.nchunk, pl.words, pl.chunk};
  // words per warp: 256 threads while that keeps the keys in registers, then CTAs
  // of 512 that do.  (Two of those share an SM, so that 16 clusters of 8 run at once
  // whatever the GPCs' sizes; of 1024 threads some waited for a second wave.)
  const int64_t words = pl.words;  // whole chunks
  const int nt = words <= 8 * 8 ? 256 : 512, nw = nt / 32;
  int cs = 1;
  while (nt == 512 && cs < kMaxCluster && words > (int64_t)cs * nw * (cs < 4 ? 8 : kHeld)) cs *= 2;
  const int per = (int)((words + nw * cs - 1) / (nw * cs));
  auto select = nt == 256      ? evict_select<256, 8>
                : per <= 16    ? evict_select<512, 16>
                : per <= kHeld ? evict_select<512, kHeld>
                               : evict_select<512, 0>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * cs));
  cfg.blockDim = dim3(nt);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, select, sp, per);
  if (e != cudaSuccess) return e;
  CopyParams cp{codes, out, bstride, ostride, acc, acc_out, acc_stride, acc_ostride, kept, sp.rows, sp.bits, sp.off,
                sp.flag, sp.ticket, (uint32_t *)ws, B, T, n_keep, pl.nchunk, pl.words, R, pl.chunk, out == codes};
  if (R % 16 == 0 && pl.chunk * R <= kCopyBytes) return launch_copy<16>(cp, st);
  if (R % 8 == 0) return launch_copy<8>(cp, st);
  if (R % 4 == 0) return launch_copy<4>(cp, st);
  if (R % 2 == 0) return launch_copy<2>(cp, st);
  return launch_copy<1>(cp, st);
}

}  // namespace fsq
