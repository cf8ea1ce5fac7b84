// C ABI of the library: argument validation, launch planning, dispatch.
// Every check that can fail runs before any CUDA call, so invalid requests
// return synchronously without touching the device.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "common.cuh"

namespace fsq {
cudaError_t launch_encode_pack(const uint16_t *x, int64_t n_tok, int64_t ldx, int64_t C, const uint16_t *E, int G,
                               int levels, const float *th, uint8_t *codes, int64_t ldc, int64_t per_row,
                               int64_t row_stride, uint32_t *status, uint32_t stall_ns, cudaStream_t s);
cudaError_t launch_quantize_pack_f32(const float *u, int64_t n_tok, int G, int levels, const float *th,
                                     uint8_t *codes, int64_t ldc, cudaStream_t s);
cudaError_t launch_absorbed_simt(const uint16_t *q, const uint8_t *codes, int64_t bstride, int64_t B, int n_new,
                                 int64_t T, const int32_t *seq_lens, int n_q, int n_kv, int d_h, int G, int bits,
                                 const uint16_t *W_kv, float scale, int S, int64_t tps, float *qa, float *part,
                                 uint32_t *err, MergeScratch ms, void *o, int out_fp32, void *const *prof,
                                 cudaStream_t st);
cudaError_t launch_expand_simt(const uint16_t *q, const uint8_t *codes, int64_t bstride, int64_t B, int n_new,
                               int64_t T, const int32_t *seq_lens, int n_q, int n_kv, int d_h, int G, int bits,
                               const uint16_t *W_kv, float scale, int S, int64_t tps, int rope_knorm,
                               float rope_base, const uint16_t *gain, float eps, float *part, uint32_t *err, void *o,
                               int out_fp32, void *const *prof, cudaStream_t st);
size_t absorbed_simt_smem(int n_q, int G);
size_t expand_simt_smem(int G);
bool expand_tc_supported(int n_q, int n_kv, int G);
size_t expand_tc_stage_bytes(int G, int variant_expand);
cudaError_t launch_expand_tc(const uint16_t *q, const uint8_t *codes, int64_t bstride, int64_t B, int n_new,
                             int64_t T, const int32_t *seq_lens, int n_q, int n_kv, int d_h, int G, const uint16_t *W_kv,
                             float scale, int S, int64_t tps, int hybrid, int rope, float rope_base,
                             const uint16_t *gain, float eps, uint8_t *wk, uint8_t *wv, float *ck, float *cv,
                             uint8_t *qs, float *part, uint32_t *err, MergeScratch ms, void *o, int out_fp32,
                             uint32_t stall_ns, void *const *prof, cudaStream_t st);
int simt_max_nq();
int simt_max_grp();
int absorbed_tc_width(int n_q, int n_kv, int G, int levels);
bool absorbed_gen_supported(int n_q, int n_kv, int G, int levels);
size_t absorbed_gen_qbuf_bytes(int n_q, int G);
int absorbed_gen_ctas_per_sm(int n_q, int G, int levels);
cudaError_t launch_absorbed_gen(const uint16_t *q, const uint8_t *codes, int64_t bstride, int64_t R, int n_new,
                                int64_t T, const int32_t *seq_lens, int n_q, int n_kv, int d_h, int G, int levels,
                                const uint16_t *W_kv, float scale, int S, int64_t tps, uint8_t *qbuf, float *part,
                                uint32_t *err, MergeScratch ms, void *o, int out_fp32, uint32_t stall_ns,
                                void *const *prof, cudaStream_t st);
size_t absorbed_tc_qphys_bytes(int n_q, int G);
cudaError_t launch_absorbed_tc(const uint16_t *q, const uint8_t *codes, int64_t bstride, int64_t B, int n_new,
                               int64_t T, const int32_t *seq_lens, int n_q, int n_kv, int d_h, int G, int levels,
                               const uint16_t *W_kv, float scale, int S, int64_t tps, uint8_t *qphys, float *corr,
                               float *part, uint32_t *err, MergeScratch ms, void *o, int out_fp32,
                               uint32_t stall_ns, void *const *prof, cudaStream_t st);
bool prefix_supported(int n_q, int G);
int prefix_rows_per_tile(int n_q);
int prefix_max_splits();
int prefix_tile_tokens();
int prefix_split_tiles();
size_t prefix_query_bytes(int G);
cudaError_t launch_prefix(const uint16_t *q, int64_t B, int n_q, int n_kv, const uint8_t *shared, int64_t Tp,
                          const uint8_t *codes, int64_t bstride, int64_t T, const int32_t *seq_lens, int G, int bits,
                          const uint16_t *W_kv, float scale, int QT, int Sp, int Ss, int k, uint8_t *qbuf, float *sig,
                          float *part, uint32_t *err, void *o, int out_fp32, uint32_t stall_ns,
                          void *const *prof, cudaStream_t st);
bool weights_supported(int n_q, int G, int bits);
int weights_tile_tokens();
size_t weights_query_bytes(int n_q, int G, int bits);
cudaError_t launch_weights(const uint16_t *q, int64_t B, int n_q, int n_kv, const uint8_t *codes, int64_t bstride,
                           int64_t T, const int32_t *seq_lens, int G, int bits, const uint16_t *W_kv, float scale, int S,
                           int k, float *acc, int64_t acc_stride, uint8_t *qbuf, float *sig, float *part, uint32_t *err,
                           uint32_t stall_ns, void *const *prof, cudaStream_t st);
cudaError_t launch_norm_rope(const uint16_t *q, int64_t ldq, int n_q, const uint16_t *q_gain, uint16_t *q_out,
                             int64_t ldqo, const uint16_t *k, int64_t ldk, int n_k, const uint16_t *k_gain,
                             uint16_t *k_out, int64_t ldko, int64_t n_tok, const int32_t *positions, int64_t pos0,
                             float eps, float rope_base, cudaStream_t st);
size_t evict_workspace_bytes(int64_t B, int64_t T, int R);
cudaError_t launch_evict(const uint8_t *codes, int64_t bstride, const float *acc, int64_t acc_stride,
                         const int32_t *lens, int64_t B, int64_t T, int64_t n_keep, int64_t n_recent, int R,
                         uint8_t *out, int64_t ostride, float *acc_out, int64_t acc_ostride, int32_t *lens_out,
                         int32_t *kept, uint8_t *ws, cudaStream_t st);

namespace {

constexpr int kMaxSplits = 1024;
constexpr int64_t kMaxGridRows = 65535;  // grid rows of a call: batch rows x queries per row (grid y)
constexpr bool kEnableTc = true;  // tensor-core absorbed kernel (being validated)

constexpr size_t kMaxDynSmem = 227 * 1024;  // dynamic shared memory a CTA may request

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// Level count of a levels field (0 selects 16); 0 when unsupported.
int levels_of(int levels) {
  if (levels == 0) return FSQ_LEVELS;
  return bits_of_levels(levels) ? levels : 0;
}

// Latent widths that pack into whole bytes and whole coordinate pairs.
bool width_ok(int G, int L) { return G >= 2 && G <= FSQ_MAX_G && G % 2 == 0 && (L != 4 || G % 4 == 0); }

// Every level of eq. (2) must lie in {-L/2 .. L/2-1}.
fsq_status check_quant(fsq_quant_params qp) {
  const int L = levels_of(qp.levels);
  if (!L) return FSQ_ERR_UNSUPPORTED;
  const float top = 0.5f * (float)L;
  if (!(qp.delta > 0.f) || !(qp.h > qp.delta)) return FSQ_ERR_INVALID_ARG;
  if (!(qp.h - qp.delta <= top - 0.5f) || !(qp.h + qp.delta <= top + 0.5f)) return FSQ_ERR_INVALID_ARG;
  return FSQ_OK;
}

// Smallest float not below x (x finite).
float ceil_to_float(double x) {
  float f = (float)x;
  if ((double)f < x) f = nextafterf(f, INFINITY);
  return f;
}

// The L-1 thresholds of eq. (2) at L = levels_of(qp.levels).
void make_thresholds(fsq_quant_params qp, float *out) {
  const int L = levels_of(qp.levels);
  const double h = qp.h, dl = qp.delta;
  const double a = atanh(dl / h);
  for (int k = 0; k < L - 1; ++k) {
    const double m = (double)(k - L / 2);     // boundary between levels m and m+1
    const double arg = (m + 0.5 + dl) / h;    // tanh(u + a) at u~ = m + 1/2
    if (arg >= 1.0) out[k] = INFINITY;
    else if (arg <= -1.0) out[k] = -INFINITY;
    else out[k] = ceil_to_float(atanh(arg) - a);
  }
}

struct Plan {
  int variant;
  int levels;     // L of the codes
  bool gen;       // generic tensor-core absorbed kernel
  bool tc;        // tensor-core kernel (absorbed, expand or hybrid form)
  int S;          // splits per batch row
  int64_t tps;    // tokens per split
  MergePlan mp;   // split merge of the absorbed and hybrid forms
  size_t off_qa, off_corr, off_part, off_mslab, off_mcnt, total;
  size_t off_wk, off_wv, off_ck, off_cv;  // staged decoder slices of the tensor-core expand / hybrid forms
};

fsq_status plan_decode(int64_t B, int64_t T, int n_q, int n_kv, int d_h, int G, const fsq_attn_opts &op, Plan *p) {
  if (B < 0 || T < 1 || n_q < 1 || n_kv < 1 || d_h < 1 || G < 2) return FSQ_ERR_INVALID_ARG;
  if (n_q % n_kv) return FSQ_ERR_INVALID_ARG;
  const int L = levels_of(op.levels);
  if (!L || !width_ok(G, L) || d_h != FSQ_HEAD_DIM) return FSQ_ERR_UNSUPPORTED;
  if (op.variant < FSQ_VARIANT_AUTO || op.variant > FSQ_VARIANT_HYBRID) return FSQ_ERR_INVALID_ARG;
  if (op.num_splits < 0) return FSQ_ERR_INVALID_ARG;
  if (op.rope_knorm != 0 && op.rope_knorm != 1) return FSQ_ERR_INVALID_ARG;
  int variant = op.variant;
  // the tensor-core kernels read 16-level codes
  const bool xtc_shape = kEnableTc && L == 16 && expand_tc_supported(n_q, n_kv, G);
  if (variant == FSQ_VARIANT_AUTO)
    variant = !op.rope_knorm ? FSQ_VARIANT_ABSORBED : (xtc_shape ? FSQ_VARIANT_HYBRID : FSQ_VARIANT_EXPAND);
  if (variant == FSQ_VARIANT_ABSORBED && op.rope_knorm) return FSQ_ERR_UNSUPPORTED;
  if (variant == FSQ_VARIANT_ABSORBED && n_q > simt_max_nq()) return FSQ_ERR_UNSUPPORTED;
  if (variant == FSQ_VARIANT_HYBRID && !xtc_shape) return FSQ_ERR_UNSUPPORTED;
  if (variant == FSQ_VARIANT_EXPAND && !xtc_shape && n_q / n_kv > simt_max_grp()) return FSQ_ERR_UNSUPPORTED;
  if (op.rope_knorm && !(op.rope_base > 1.f && op.knorm_eps >= 0.f)) return FSQ_ERR_INVALID_ARG;

  const int64_t Bc = B > 0 ? B : 1;
  const bool xtc = (variant == FSQ_VARIANT_EXPAND || variant == FSQ_VARIANT_HYBRID) && xtc_shape;
  // the absorbed tensor-core kernel reads rows of Gn nibbles: 16-level codes,
  // or 256-level codes read as two nibbles each (Gn = 2G)
  const int Gn = (kEnableTc && variant == FSQ_VARIANT_ABSORBED) ? absorbed_tc_width(n_q, n_kv, G, L) : 0;
  // other absorbed shapes: the generic tensor-core kernel (codes unpacked to fp16 in shared memory)
  const bool gen = !Gn && kEnableTc && variant == FSQ_VARIANT_ABSORBED && absorbed_gen_supported(n_q, n_kv, G, L);
  const bool tc = Gn > 0 || xtc || gen;
  // the CUDA-core kernels hold a tile of latents (and, in the expand form, W_kv^(j)) in shared memory
  if (!tc && variant == FSQ_VARIANT_ABSORBED && absorbed_simt_smem(n_q, G) > kMaxDynSmem) return FSQ_ERR_UNSUPPORTED;
  if (!tc && variant == FSQ_VARIANT_EXPAND && expand_simt_smem(G) > kMaxDynSmem) return FSQ_ERR_UNSUPPORTED;
  const int64_t ctas_per_row = (variant == FSQ_VARIANT_EXPAND || variant == FSQ_VARIANT_HYBRID) ? n_kv : 1;
  int64_t S = op.num_splits;
  if (S == 0) {
    if (tc) {
      // one wave of CTAs: one per SM (each holds all of TMEM), or as many as
      // an SM holds of the generic kernel
      const int per_sm = gen ? absorbed_gen_ctas_per_sm(n_q, G, L) : 1;
      S = (int64_t)kNumSMs * per_sm / (Bc * ctas_per_row);
      if (S < 1) S = 1;
    } else {
      const int64_t target = 2 * kNumSMs;
      S = (target + Bc * ctas_per_row - 1) / (Bc * ctas_per_row);
      const int64_t max_by_len = (T + 255) / 256;
      if (S > max_by_len) S = max_by_len;
    }
  }
  if (S < 1) S = 1;
  if (S > kMaxSplits) S = kMaxSplits;
  if (S > T) S = T;
  int64_t tps = (T + S - 1) / S;
  if (tc) tps = (tps + 127) / 128 * 128;  // whole 128-token tiles, 16-byte aligned split starts
  S = (T + tps - 1) / tps;  // no empty splits
  p->variant = variant;
  p->levels = L;
  p->tc = tc;
  p->gen = gen;
  p->S = (int)S;
  p->tps = tps;
  const int acc_len = variant == FSQ_VARIANT_EXPAND ? d_h : (Gn ? Gn : G);  // floats per partial after (m, l)
  size_t off = kWsHeader;
  p->off_qa = off;
  if (xtc) off = align_up(off + (size_t)Bc * n_kv * 16 * d_h * 2, 256);  // staged queries
  else if (gen) off = align_up(off + absorbed_gen_qbuf_bytes(n_q, G) * (size_t)Bc, 256);
  else if (tc) off = align_up(off + absorbed_tc_qphys_bytes(n_q, Gn) * (size_t)Bc, 256);
  else if (variant == FSQ_VARIANT_ABSORBED) off = align_up(off + sizeof(float) * (size_t)Bc * n_q * G, 256);
  p->off_corr = off;
  if (tc && !xtc && !gen) off = align_up(off + 2 * sizeof(float) * (size_t)Bc * n_q, 256);  // per-head scales / offsets
  p->off_wk = p->off_wv = p->off_ck = p->off_cv = off;
  if (xtc) {
    const size_t slice = expand_tc_stage_bytes(G, 0);
    p->off_wk = off;
    off = align_up(off + slice * n_kv, 256);
    p->off_wv = off;
    if (variant == FSQ_VARIANT_EXPAND) off = align_up(off + slice * n_kv, 256);
    p->off_ck = off;
    off = align_up(off + sizeof(float) * d_h * n_kv, 256);
    p->off_cv = off;
    off = align_up(off + sizeof(float) * d_h * n_kv, 256);
  }
  p->off_part = off;
  off = align_up(off + sizeof(float) * (size_t)Bc * S * n_q * (2 + acc_len), 256);
  if (variant == FSQ_VARIANT_ABSORBED || variant == FSQ_VARIANT_HYBRID) p->mp = merge_plan((int)S, Bc, n_q, n_kv, acc_len);
  p->off_mslab = off;
  off = align_up(off + p->mp.slab_bytes, 256);
  p->off_mcnt = off;
  off = align_up(off + p->mp.cnt_bytes, 256);
  p->total = off;
  return FSQ_OK;
}

// Shared-prefix attention: query tiles, splits, workspace.
struct PrefixPlan {
  int levels, QT, Sp, Ss, k;  // k: tiles of a split, of the prefix and of a row's own tokens alike
  size_t off_q, off_sig, off_part, total;
};

fsq_status plan_prefix(int64_t B, int64_t Tp, int64_t T, int n_q, int n_kv, int d_h, int G, const fsq_attn_opts &op,
                       PrefixPlan *p) {
  if (B < 0 || Tp < 1 || T < 0 || n_q < 1 || n_kv < 1 || d_h < 1 || G < 2) return FSQ_ERR_INVALID_ARG;
  if (n_q % n_kv) return FSQ_ERR_INVALID_ARG;
  if (op.variant < FSQ_VARIANT_AUTO || op.variant > FSQ_VARIANT_HYBRID || op.num_splits < 0) return FSQ_ERR_INVALID_ARG;
  if (op.rope_knorm != 0 && op.rope_knorm != 1) return FSQ_ERR_INVALID_ARG;
  const int L = levels_of(op.levels);
  if (!L || !width_ok(G, L) || d_h != FSQ_HEAD_DIM || !prefix_supported(n_q, G)) return FSQ_ERR_UNSUPPORTED;
  if (op.rope_knorm || op.variant > FSQ_VARIANT_ABSORBED || B > kMaxGridRows) return FSQ_ERR_UNSUPPORTED;
  const int64_t tile = prefix_tile_tokens(), Bc = B > 0 ? B : 1;
  const int64_t nt = (Tp + tile - 1) / tile, no = (T + tile - 1) / tile, most = nt > no ? nt : no;
  if (most > INT32_MAX / 2) return FSQ_ERR_UNSUPPORTED;
  const int64_t rpt = prefix_rows_per_tile(n_q), QT = (Bc + rpt - 1) / rpt;
  // Tiles per split.  Every CTA costs its tiles and a fixed start and end, runs
  // of CTAs beyond one per SM follow one another, and every split of a row
  // leaves a partial that is written and merged: the cheapest k by these rates
  // (measured at G = 256, n_q = 32: 0.6 us a tile, 5 us a CTA, partials at 3 TB/s).
  int64_t k = 0;
  if (op.num_splits > 0) {
    const int64_t s = op.num_splits < nt ? op.num_splits : nt;
    k = (nt + s - 1) / s;
  } else {
    double best = 0;
    int64_t last = 0;
    for (int s = 1; s <= kNumSMs; ++s) {
      const int64_t kk = (most + s - 1) / s;
      if (kk == last) continue;
      last = kk;
      const int64_t sp = (nt + kk - 1) / kk, so = (no + kk - 1) / kk, ctas = QT * sp + Bc * so;
      const double cost = (double)((ctas + kNumSMs - 1) / kNumSMs) * (0.6 * kk + 5.0) +
                          8e-6 / 3.0 * (double)(sp + so) * Bc * n_q * (G + 2);
      if (s == 1 || cost < best) best = cost, k = kk;
      if (kk == 1) break;
    }
  }
  // fp16 weights hold a split's tail up to this length
  if (k > prefix_split_tiles()) k = prefix_split_tiles();
  // a row's partials fit the merge
  while ((nt + k - 1) / k + (no + k - 1) / k > prefix_max_splits()) k *= 2;
  const int64_t Sp = (nt + k - 1) / k, Ss = (no + k - 1) / k;
  if (QT * Sp + Bc * Ss > INT32_MAX) return FSQ_ERR_UNSUPPORTED;
  p->levels = L;
  p->QT = (int)QT;
  p->Sp = (int)Sp;
  p->Ss = (int)Ss;
  p->k = (int)k;
  size_t off = kWsHeader;
  p->off_q = off;
  off = align_up(off + prefix_query_bytes(G) * (size_t)QT, 256);
  p->off_sig = off;
  off = align_up(off + sizeof(float) * (size_t)Bc * n_q, 256);
  p->off_part = off;
  off = align_up(off + sizeof(float) * (size_t)Bc * (Sp + Ss) * n_q * (2 + G), 256);
  p->total = off;
  return FSQ_OK;
}

// Attention weights: splits and workspace.
struct WeightsPlan {
  int levels, S, k;  // splits per row, tiles per split
  size_t off_q, off_sig, off_part, total;
};

fsq_status plan_weights(int64_t B, int64_t T, int n_q, int n_kv, int d_h, int G, const fsq_attn_opts &op,
                        WeightsPlan *p) {
  if (B < 0 || T < 1 || n_q < 1 || n_kv < 1 || d_h < 1 || G < 2) return FSQ_ERR_INVALID_ARG;
  if (n_q % n_kv) return FSQ_ERR_INVALID_ARG;
  if (op.variant < FSQ_VARIANT_AUTO || op.variant > FSQ_VARIANT_HYBRID || op.num_splits < 0) return FSQ_ERR_INVALID_ARG;
  if (op.rope_knorm != 0 && op.rope_knorm != 1) return FSQ_ERR_INVALID_ARG;
  const int L = levels_of(op.levels);
  if (!L || !width_ok(G, L) || d_h != FSQ_HEAD_DIM || !weights_supported(n_q, G, bits_of_levels(L)))
    return FSQ_ERR_UNSUPPORTED;
  if (op.rope_knorm || op.variant > FSQ_VARIANT_ABSORBED || B > kMaxGridRows) return FSQ_ERR_UNSUPPORTED;
  const int bits = bits_of_levels(L);
  if (T > ((int64_t)1 << 37) / (G * bits / 8 > 0 ? G * bits / 8 : 1)) return FSQ_ERR_UNSUPPORTED;
  const int64_t nt = (T + weights_tile_tokens() - 1) / weights_tile_tokens(), Bc = B > 0 ? B : 1;
  if (nt > INT32_MAX / 2) return FSQ_ERR_UNSUPPORTED;
  int64_t k = 0;
  if (op.num_splits > 0) {
    const int64_t s = op.num_splits < nt ? op.num_splits : nt;
    k = (nt + s - 1) / s;
  } else {
    // one CTA per SM runs at a time; a CTA costs its tiles and the start and end of about four
    int64_t best = 0, last = 0;
    for (int s = 1; s <= kNumSMs; ++s) {
      const int64_t kk = (nt + s - 1) / s;
      if (kk == last) continue;
      last = kk;
      const int64_t ctas = Bc * ((nt + kk - 1) / kk);
      const int64_t cost = (ctas + kNumSMs - 1) / kNumSMs * (kk + 4);
      if (s == 1 || cost < best) best = cost, k = kk;
      if (kk == 1) break;
    }
  }
  p->levels = L;
  p->k = (int)k;
  p->S = (int)((nt + k - 1) / k);
  size_t off = kWsHeader;
  p->off_q = off;
  off = align_up(off + weights_query_bytes(n_q, G, bits) * (size_t)Bc, 256);
  p->off_sig = off;
  off = align_up(off + 2 * sizeof(float) * (size_t)Bc * n_q, 256);
  p->off_part = off;
  off = align_up(off + 2 * sizeof(float) * (size_t)Bc * p->S * n_q, 256);
  p->total = off;
  return FSQ_OK;
}

fsq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FSQ_OK : FSQ_ERR_CUDA; }

}  // namespace
}  // namespace fsq

using namespace fsq;

extern "C" {

void fsq_attn_opts_default(fsq_attn_opts *opts) {
  if (!opts) return;
  memset(opts, 0, sizeof(*opts));
  opts->variant = FSQ_VARIANT_AUTO;
  opts->scale = 0.f;
  opts->num_splits = 0;
  opts->rope_knorm = 0;
  opts->rope_base = 1.0e6f;
  opts->knorm_gain = nullptr;
  opts->knorm_eps = 1.0e-6f;
  opts->out_fp32 = 0;
  opts->prof_events[0] = opts->prof_events[1] = nullptr;
  opts->seq_lens = nullptr;
  opts->debug_stall_ns = 0;
  opts->levels = FSQ_LEVELS;
}

fsq_status fsq_thresholds(fsq_quant_params qp, float *theta_out) {
  if (!theta_out) return FSQ_ERR_INVALID_ARG;
  fsq_status st = check_quant(qp);
  if (st != FSQ_OK) return st;
  make_thresholds(qp, theta_out);
  return FSQ_OK;
}

fsq_status fsq_encode_pack(const uint16_t *x, int64_t n_tok, int64_t ldx, int64_t C, const uint16_t *E, int G,
                           fsq_quant_params qp, uint8_t *codes, int64_t ldc_bytes, const fsq_encode_opts *opts,
                           fsq_stream_t stream) {
  if (n_tok < 0 || C < 1 || G < 2) return FSQ_ERR_INVALID_ARG;
  fsq_status st = check_quant(qp);
  if (st != FSQ_OK) return st;
  const int L = levels_of(qp.levels);
  if (!width_ok(G, L) || C % 64) return FSQ_ERR_UNSUPPORTED;
  if (ldx < C || ldc_bytes < (int64_t)G * bits_of_levels(L) / 8) return FSQ_ERR_INVALID_ARG;
  if (n_tok == 0) return FSQ_OK;
  if (!x || !E || !codes) return FSQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(E) || ldx % 8) return FSQ_ERR_MISALIGNED;
  uint32_t *status = opts ? opts->status_word : nullptr;
  if ((uintptr_t)status & 3u) return FSQ_ERR_MISALIGNED;
  const int64_t per_row = opts ? opts->tokens_per_row : 0;
  const int64_t row_stride = opts ? opts->row_stride_bytes : 0;
  if (per_row < 0 || (per_row > 0 && row_stride < 0)) return FSQ_ERR_INVALID_ARG;
  float th[kMaxLevels - 1];
  make_thresholds(qp, th);
  return from_cuda(launch_encode_pack(x, n_tok, ldx, C, E, G, L, th, codes, ldc_bytes, per_row, row_stride, status,
                                      opts ? opts->debug_stall_ns : 0u, (cudaStream_t)stream));
}

fsq_status fsq_quantize_pack_f32(const float *u, int64_t n_tok, int G, fsq_quant_params qp, uint8_t *codes,
                                 int64_t ldc_bytes, fsq_stream_t stream) {
  if (n_tok < 0 || G < 2) return FSQ_ERR_INVALID_ARG;
  fsq_status st = check_quant(qp);
  if (st != FSQ_OK) return st;
  const int L = levels_of(qp.levels);
  if (!width_ok(G, L)) return FSQ_ERR_UNSUPPORTED;
  if (ldc_bytes < (int64_t)G * bits_of_levels(L) / 8) return FSQ_ERR_INVALID_ARG;
  if (n_tok == 0) return FSQ_OK;
  if (!u || !codes) return FSQ_ERR_INVALID_ARG;
  if (!aligned16(u)) return FSQ_ERR_MISALIGNED;
  float th[kMaxLevels - 1];
  make_thresholds(qp, th);
  return from_cuda(launch_quantize_pack_f32(u, n_tok, G, L, th, codes, ldc_bytes, (cudaStream_t)stream));
}

size_t fsq_decode_attn_workspace_size(int64_t B, int64_t T, int n_q, int n_kv, int d_h, int G,
                                      const fsq_attn_opts *opts) {
  return fsq_decode_attn_multi_workspace_size(B, 1, T, n_q, n_kv, d_h, G, opts);
}

size_t fsq_decode_attn_multi_workspace_size(int64_t B, int n_new, int64_t T, int n_q, int n_kv, int d_h, int G,
                                            const fsq_attn_opts *opts) {
  fsq_attn_opts op;
  if (opts) op = *opts;
  else fsq_attn_opts_default(&op);
  Plan p;
  if (n_new < 1 || B < 0 || B * n_new > kMaxGridRows) return 0;
  if (plan_decode(B * n_new, T, n_q, n_kv, d_h, G, op, &p) != FSQ_OK) return 0;
  return p.total;
}

const char *fsq_decode_attn_kernel(int64_t B, int n_new, int64_t T, int n_q, int n_kv, int d_h, int G,
                                   const fsq_attn_opts *opts) {
  fsq_attn_opts op;
  if (opts) op = *opts;
  else fsq_attn_opts_default(&op);
  Plan p;
  if (n_new < 1 || B < 0 || B * n_new > kMaxGridRows) return nullptr;
  if (plan_decode(B * n_new, T, n_q, n_kv, d_h, G, op, &p) != FSQ_OK) return nullptr;
  if (p.variant == FSQ_VARIANT_HYBRID) return "hybrid_split_tc";
  if (p.variant == FSQ_VARIANT_EXPAND) return p.tc ? "expand_split_tc" : "expand_split_simt";
  if (p.gen) return "absorbed_split_gen";
  return p.tc ? "absorbed_split_tc" : "absorbed_split_simt";
}

fsq_status fsq_decode_attn(const uint16_t *q, int64_t B, int n_q, int d_h, const uint8_t *codes,
                           int64_t code_batch_stride_bytes, int64_t T, int G, const uint16_t *W_kv, int n_kv,
                           const fsq_attn_opts *opts, void *workspace, size_t workspace_bytes, void *o,
                           fsq_stream_t stream) {
  return fsq_decode_attn_multi(q, B, 1, n_q, d_h, codes, code_batch_stride_bytes, T, G, W_kv, n_kv, opts, workspace,
                               workspace_bytes, o, stream);
}

// The queries of a cache row run as n_new consecutive grid rows of the same
// kernels (R = B * n_new rows); only the split kernels map a grid row to its
// cache row and causal length.
fsq_status fsq_decode_attn_multi(const uint16_t *q, int64_t B, int n_new, int n_q, int d_h, const uint8_t *codes,
                                 int64_t code_batch_stride_bytes, int64_t T, int G, const uint16_t *W_kv, int n_kv,
                                 const fsq_attn_opts *opts, void *workspace, size_t workspace_bytes, void *o,
                                 fsq_stream_t stream) {
  fsq_attn_opts op;
  if (opts) op = *opts;
  else fsq_attn_opts_default(&op);
  if (n_new < 1 || B < 0) return FSQ_ERR_INVALID_ARG;
  if (B * n_new > kMaxGridRows) return FSQ_ERR_UNSUPPORTED;
  const int64_t R = B * n_new;
  Plan p;
  fsq_status st = plan_decode(R, T, n_q, n_kv, d_h, G, op, &p);
  if (st != FSQ_OK) return st;
  if (B == 0) return FSQ_OK;
  if (!q || !codes || !W_kv || !o) return FSQ_ERR_INVALID_ARG;
  const int bits = bits_of_levels(p.levels);
  if (code_batch_stride_bytes < T * ((int64_t)G * bits / 8)) return FSQ_ERR_INVALID_ARG;
  if (!aligned16(codes) || code_batch_stride_bytes % 16) return FSQ_ERR_MISALIGNED;
  if (!aligned16(q) || !aligned16(W_kv) || !aligned16(o)) return FSQ_ERR_MISALIGNED;
  if ((uintptr_t)op.seq_lens & 3u) return FSQ_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < p.total) return FSQ_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255u) return FSQ_ERR_MISALIGNED;
  const float scale = op.scale > 0.f ? op.scale : 1.f / sqrtf((float)d_h);
  char *ws = (char *)workspace;
  uint32_t *err = (uint32_t *)ws;
  float *part = (float *)(ws + p.off_part);
  cudaStream_t s = (cudaStream_t)stream;
  MergeScratch ms{nullptr, nullptr, 0};
  if (p.mp.cnt_bytes) ms = {(float *)(ws + p.off_mslab), (uint32_t *)(ws + p.off_mcnt), (int)(R * n_kv)};
  cudaError_t e;
  if (p.tc && (p.variant == FSQ_VARIANT_EXPAND || p.variant == FSQ_VARIANT_HYBRID)) {
    e = launch_expand_tc(q, codes, code_batch_stride_bytes, R, n_new, T, op.seq_lens, n_q, n_kv, d_h, G, W_kv, scale,
                         p.S, p.tps, p.variant == FSQ_VARIANT_HYBRID, op.rope_knorm, op.rope_base, op.knorm_gain,
                         op.knorm_eps, (uint8_t *)(ws + p.off_wk), (uint8_t *)(ws + p.off_wv),
                         (float *)(ws + p.off_ck), (float *)(ws + p.off_cv), (uint8_t *)(ws + p.off_qa), part, err,
                         ms, o, op.out_fp32, op.debug_stall_ns, op.prof_events, s);
  } else if (p.gen) {
    e = launch_absorbed_gen(q, codes, code_batch_stride_bytes, R, n_new, T, op.seq_lens, n_q, n_kv, d_h, G, p.levels,
                            W_kv, scale, p.S, p.tps, (uint8_t *)(ws + p.off_qa), part, err, ms, o, op.out_fp32,
                            op.debug_stall_ns, op.prof_events, s);
  } else if (p.tc) {
    e = launch_absorbed_tc(q, codes, code_batch_stride_bytes, R, n_new, T, op.seq_lens, n_q, n_kv, d_h, G, p.levels,
                           W_kv, scale, p.S, p.tps, (uint8_t *)(ws + p.off_qa), (float *)(ws + p.off_corr), part, err,
                           ms, o, op.out_fp32, op.debug_stall_ns, op.prof_events, s);
  } else if (p.variant == FSQ_VARIANT_ABSORBED) {
    e = launch_absorbed_simt(q, codes, code_batch_stride_bytes, R, n_new, T, op.seq_lens, n_q, n_kv, d_h, G, bits,
                             W_kv, scale, p.S, p.tps, (float *)(ws + p.off_qa), part, err, ms, o, op.out_fp32,
                             op.prof_events, s);
  } else {
    e = launch_expand_simt(q, codes, code_batch_stride_bytes, R, n_new, T, op.seq_lens, n_q, n_kv, d_h, G, bits,
                           W_kv, scale, p.S, p.tps, op.rope_knorm, op.rope_base, op.knorm_gain, op.knorm_eps, part,
                           err, o, op.out_fp32, op.prof_events, s);
  }
  return from_cuda(e);
}

size_t fsq_decode_attn_prefix_workspace_size(int64_t B, int64_t T_prefix, int64_t T, int n_q, int n_kv, int d_h, int G,
                                             const fsq_attn_opts *opts) {
  fsq_attn_opts op;
  if (opts) op = *opts;
  else fsq_attn_opts_default(&op);
  PrefixPlan p;
  return plan_prefix(B, T_prefix, T, n_q, n_kv, d_h, G, op, &p) == FSQ_OK ? p.total : 0;
}

fsq_status fsq_decode_attn_prefix(const uint16_t *q, int64_t B, int n_q, int d_h, const uint8_t *prefix_codes,
                                  int64_t T_prefix, const uint8_t *codes, int64_t code_batch_stride_bytes, int64_t T,
                                  int G, const uint16_t *W_kv, int n_kv, const fsq_attn_opts *opts, void *workspace,
                                  size_t workspace_bytes, void *o, fsq_stream_t stream) {
  fsq_attn_opts op;
  if (opts) op = *opts;
  else fsq_attn_opts_default(&op);
  PrefixPlan p;
  const fsq_status st = plan_prefix(B, T_prefix, T, n_q, n_kv, d_h, G, op, &p);
  if (st != FSQ_OK) return st;
  if (B == 0) return FSQ_OK;
  if (!q || !prefix_codes || !W_kv || !o || (T > 0 && !codes)) return FSQ_ERR_INVALID_ARG;
  const int bits = bits_of_levels(p.levels);
  if (T > 0 && code_batch_stride_bytes < T * ((int64_t)G * bits / 8)) return FSQ_ERR_INVALID_ARG;
  if (!aligned16(prefix_codes) || (T > 0 && (!aligned16(codes) || code_batch_stride_bytes % 16)))
    return FSQ_ERR_MISALIGNED;
  if (!aligned16(q) || !aligned16(W_kv) || !aligned16(o)) return FSQ_ERR_MISALIGNED;
  if ((uintptr_t)op.seq_lens & 3u) return FSQ_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < p.total) return FSQ_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255u) return FSQ_ERR_MISALIGNED;
  char *ws = (char *)workspace;
  return from_cuda(launch_prefix(q, B, n_q, n_kv, prefix_codes, T_prefix, codes, code_batch_stride_bytes, T,
                                 op.seq_lens, G, bits, W_kv, op.scale > 0.f ? op.scale : 1.f / sqrtf((float)d_h), p.QT,
                                 p.Sp, p.Ss, p.k, (uint8_t *)(ws + p.off_q), (float *)(ws + p.off_sig),
                                 (float *)(ws + p.off_part), (uint32_t *)ws, o, op.out_fp32, op.debug_stall_ns,
                                 op.prof_events, (cudaStream_t)stream));
}

size_t fsq_attn_weights_workspace_size(int64_t B, int64_t T, int n_q, int n_kv, int d_h, int G,
                                       const fsq_attn_opts *opts) {
  fsq_attn_opts op;
  if (opts) op = *opts;
  else fsq_attn_opts_default(&op);
  WeightsPlan p;
  return plan_weights(B, T, n_q, n_kv, d_h, G, op, &p) == FSQ_OK ? p.total : 0;
}

fsq_status fsq_attn_weights(const uint16_t *q, int64_t B, int n_q, int d_h, const uint8_t *codes,
                            int64_t code_batch_stride_bytes, int64_t T, int G, const uint16_t *W_kv, int n_kv,
                            const fsq_attn_opts *opts, float *acc, int64_t acc_stride, void *workspace,
                            size_t workspace_bytes, fsq_stream_t stream) {
  fsq_attn_opts op;
  if (opts) op = *opts;
  else fsq_attn_opts_default(&op);
  WeightsPlan p;
  const fsq_status st = plan_weights(B, T, n_q, n_kv, d_h, G, op, &p);
  if (st != FSQ_OK) return st;
  if (B == 0) return FSQ_OK;
  if (!q || !codes || !W_kv || !acc) return FSQ_ERR_INVALID_ARG;
  const int bits = bits_of_levels(p.levels);
  if (code_batch_stride_bytes < T * ((int64_t)G * bits / 8) || acc_stride < T) return FSQ_ERR_INVALID_ARG;
  if (!aligned16(codes) || code_batch_stride_bytes % 16 || !aligned16(q) || !aligned16(W_kv)) return FSQ_ERR_MISALIGNED;
  if (((uintptr_t)op.seq_lens | (uintptr_t)acc) & 3u) return FSQ_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < p.total) return FSQ_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255u) return FSQ_ERR_MISALIGNED;
  char *ws = (char *)workspace;
  return from_cuda(launch_weights(q, B, n_q, n_kv, codes, code_batch_stride_bytes, T, op.seq_lens, G, bits, W_kv,
                                  op.scale > 0.f ? op.scale : 1.f / sqrtf((float)d_h), p.S, p.k, acc, acc_stride,
                                  (uint8_t *)(ws + p.off_q), (float *)(ws + p.off_sig), (float *)(ws + p.off_part),
                                  (uint32_t *)ws, op.debug_stall_ns, op.prof_events, (cudaStream_t)stream));
}

fsq_status fsq_qk_norm_rope(const uint16_t *q, int64_t ldq, int n_q, const uint16_t *q_gain, uint16_t *q_out,
                            int64_t ldq_out, const uint16_t *k, int64_t ldk, int n_k, const uint16_t *k_gain,
                            uint16_t *k_out, int64_t ldk_out, int64_t n_tok, int d_h, const int32_t *positions,
                            int64_t pos0, float eps, float rope_base, fsq_stream_t stream) {
  if (n_tok < 0 || n_q < 1 || n_k < 0 || d_h < 1) return FSQ_ERR_INVALID_ARG;
  if (d_h != FSQ_HEAD_DIM || (int64_t)n_q + n_k > kMaxGridRows || n_tok > INT32_MAX) return FSQ_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || !(rope_base > 1.f) || isinf(eps) || isinf(rope_base)) return FSQ_ERR_INVALID_ARG;
  if (n_tok == 0) return FSQ_OK;
  const int64_t wq = (int64_t)n_q * d_h, wk = (int64_t)n_k * d_h;
  if (!q || !q_out || (n_k && (!k || !k_out))) return FSQ_ERR_INVALID_ARG;
  if (n_tok > 1 && (ldq < wq || ldq_out < wq || (n_k && (ldk < wk || ldk_out < wk)))) return FSQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(q_out) || ldq % 8 || ldq_out % 8) return FSQ_ERR_MISALIGNED;
  if (n_k && (!aligned16(k) || !aligned16(k_out) || ldk % 8 || ldk_out % 8)) return FSQ_ERR_MISALIGNED;
  if (!aligned16(q_gain) || (n_k && !aligned16(k_gain)) || ((uintptr_t)positions & 3u)) return FSQ_ERR_MISALIGNED;
  // two tensors of interleaved heads (one projection's q and k) span the same
  // bytes without sharing any, so spans are only told apart within a token
  const bool q_same = q_out == q && (ldq_out == ldq || n_tok == 1), k_same = k_out == k && (ldk_out == ldk || n_tok == 1);
  auto clash = [&](const uint16_t *a, int64_t lda, int64_t wa, const uint16_t *b, int64_t ldb, int64_t wb) {
    const int64_t na = ((n_tok - 1) * lda + wa) * 2, nb = ((n_tok - 1) * ldb + wb) * 2;
    if (!overlap(a, na, b, nb)) return false;
    if (lda != ldb || n_tok == 1) return true;
    // equal strides: token rows meet if the offset between them, modulo the stride, is within a row
    int64_t d = (int64_t)(((intptr_t)b - (intptr_t)a) / 2) % lda;
    if (d < 0) d += lda;
    return d < wa || lda - d < wb;
  };
  if (!q_same && clash(q, ldq, wq, q_out, ldq_out, wq)) return FSQ_ERR_INVALID_ARG;
  if (n_k) {
    if (!k_same && clash(k, ldk, wk, k_out, ldk_out, wk)) return FSQ_ERR_INVALID_ARG;
    if (clash(q, ldq, wq, k_out, ldk_out, wk) || clash(k, ldk, wk, q_out, ldq_out, wq) ||
        clash(q_out, ldq_out, wq, k_out, ldk_out, wk))
      return FSQ_ERR_INVALID_ARG;
  }
  return from_cuda(launch_norm_rope(q, ldq, n_q, q_gain, q_out, ldq_out, k, ldk, n_k, k_gain, k_out, ldk_out, n_tok,
                                    positions, pos0, eps, rope_base, (cudaStream_t)stream));
}

size_t fsq_cache_evict_workspace_size(int64_t B, int64_t T, int G, int levels) {
  const int L = levels_of(levels);
  if (B < 0 || T < 0 || T > INT32_MAX || !L || !width_ok(G, L)) return 0;
  if (B > 0 && (T + 31) / 32 > INT32_MAX / B) return 0;
  return evict_workspace_bytes(B, T, G * bits_of_levels(L) / 8);
}

fsq_status fsq_cache_evict(const uint8_t *codes, int64_t code_batch_stride_bytes, const float *acc,
                           int64_t acc_stride, const int32_t *seq_lens, int64_t B, int64_t T, int64_t n_keep,
                           int64_t n_recent, int G, int levels, uint8_t *codes_out, int64_t out_stride_bytes,
                           float *acc_out, int64_t acc_out_stride, int32_t *lens_out, int32_t *kept, void *workspace,
                           size_t workspace_bytes, fsq_stream_t stream) {
  if (B < 0 || T < 0 || n_keep < 1 || n_recent < 0 || n_recent > n_keep || G < 2) return FSQ_ERR_INVALID_ARG;
  const int L = levels_of(levels);
  if (!L || !width_ok(G, L) || T > INT32_MAX || n_keep > INT32_MAX) return FSQ_ERR_UNSUPPORTED;
  if (B > 0 && (T + 31) / 32 > INT32_MAX / B) return FSQ_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return FSQ_OK;
  if (!codes || !acc || !codes_out || !acc_out) return FSQ_ERR_INVALID_ARG;
  const int64_t R = (int64_t)G * bits_of_levels(L) / 8, rows_out = T < n_keep ? T : n_keep;
  if (code_batch_stride_bytes < T * R || acc_stride < T) return FSQ_ERR_INVALID_ARG;
  if (out_stride_bytes < rows_out * R || acc_out_stride < rows_out) return FSQ_ERR_INVALID_ARG;
  if (!aligned16(codes) || !aligned16(codes_out) || code_batch_stride_bytes % 16 || out_stride_bytes % 16)
    return FSQ_ERR_MISALIGNED;
  if (((uintptr_t)acc | (uintptr_t)acc_out | (uintptr_t)seq_lens | (uintptr_t)lens_out | (uintptr_t)kept) & 3u)
    return FSQ_ERR_MISALIGNED;
  const bool in_place = codes == codes_out;
  if (in_place != (acc == acc_out)) return FSQ_ERR_INVALID_ARG;
  if (in_place && (code_batch_stride_bytes != out_stride_bytes || acc_stride != acc_out_stride))
    return FSQ_ERR_INVALID_ARG;
  if (!in_place &&
      (overlap(codes, (B - 1) * code_batch_stride_bytes + T * R, codes_out, (B - 1) * out_stride_bytes + rows_out * R) ||
       overlap(acc, ((B - 1) * acc_stride + T) * 4, acc_out, ((B - 1) * acc_out_stride + rows_out) * 4)))
    return FSQ_ERR_INVALID_ARG;
  // lengths and indices: rows read their length and write the new one at different times
  const int64_t len_bytes = 4 * B, kept_bytes = n_keep > INT64_MAX / 4 / B ? INT64_MAX : 4 * B * n_keep;
  if ((seq_lens && lens_out && seq_lens != lens_out && overlap(seq_lens, len_bytes, lens_out, len_bytes)) ||
      (kept && seq_lens && overlap(kept, kept_bytes, seq_lens, len_bytes)) ||
      (kept && lens_out && overlap(kept, kept_bytes, lens_out, len_bytes)))
    return FSQ_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < evict_workspace_bytes(B, T, (int)R)) return FSQ_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255u) return FSQ_ERR_MISALIGNED;
  return from_cuda(launch_evict(codes, code_batch_stride_bytes, acc, acc_stride, seq_lens, B, T, n_keep, n_recent,
                                (int)R, codes_out, out_stride_bytes, acc_out, acc_out_stride, lens_out, kept,
                                (uint8_t *)workspace, (cudaStream_t)stream));
}

fsq_status fsq_workspace_status(const void *workspace, size_t workspace_bytes, fsq_stream_t stream) {
  if (!workspace || workspace_bytes < sizeof(uint32_t)) return FSQ_ERR_INVALID_ARG;
  if ((uintptr_t)workspace & 3u) return FSQ_ERR_MISALIGNED;
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, workspace, sizeof(v), cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return FSQ_ERR_CUDA;
  return v == 0 ? FSQ_OK : (fsq_status)(-(int)v);
}

const char *fsq_status_string(fsq_status s) {
  switch (s) {
    case FSQ_OK: return "ok";
    case FSQ_ERR_INVALID_ARG: return "invalid argument";
    case FSQ_ERR_UNSUPPORTED: return "unsupported shape or option";
    case FSQ_ERR_MISALIGNED: return "pointer or stride not 16-byte aligned";
    case FSQ_ERR_WORKSPACE: return "workspace missing or too small";
    case FSQ_ERR_CUDA: return "CUDA error";
    case FSQ_ERR_TIMEOUT: return "device wait timed out";
  }
  return "unknown status";
}

int fsq_format_version(void) { return FSQ_FORMAT_VERSION; }

}  // extern "C"
