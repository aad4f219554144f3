// Internal interface between the C-ABI layer (flce_api.cu) and the kernels
// (flce_kernels.cu).  Not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#if defined(__CUDACC__)
#define FLCE_HOST_DEVICE __host__ __device__
#else
#define FLCE_HOST_DEVICE
#endif

namespace flce {

// Tile shape of every tensor-core kernel: 128 rows (TMEM lanes) x 256 columns
// (TMEM columns of one accumulator), K staged 64 bf16 (one 128-byte swizzle row)
// at a time.
constexpr int kBM = 128;
constexpr int kBN = 256;
constexpr int kBK = 64;
constexpr int kStages = 6;    // 32 KiB per stage and CTA (own A rows + own half of B)
constexpr int kThreads = 192;  // warp 0: TMA producer, warp 1: MMA issuer, warps 2-5: epilogue
constexpr int kMaxSplit = 32;  // most vocabulary splits of the forward pass
constexpr int kPairRows = 2 * kBM;  // every launch runs on CTA pairs: a pair tile has 256 rows
constexpr int kBoxB = kBN / 2;      // rows of the B operand each CTA of a pair stages (K-major box)

// Grid of a tensor-core launch: CTA pairs, at most one CTA per SM.
inline int pair_grid(int sms, long long pair_work) {
  long long pairs = sms / 2;
  if (pair_work < pairs) pairs = pair_work;
  if (pairs < 1) pairs = 1;
  return static_cast<int>(2 * pairs);
}

// Vocabulary chunk width of the backward pass (a multiple of kBN).  The
// workspace holds one chunk of G, N x chunk bf16.
inline int chunk_width(int64_t n) { return n <= 16384 ? 8192 : 4096; }

// Token log probabilities' backward: chunk width and dX parts.  A wide chunk while its G
// (n x chunk bf16) stays within 128 MiB, so that few rows need few launches; and where the
// dX tiles are too few for the GPU's 76 CTA pairs, each tile's sum over the vocabulary cut
// into parts (at least 512 ids, 64 MiB together), added up in order at the end: 256 x 4096 x
// 128256 in 753 us, 1424 without either; 100 x 512 x 60000 in 87, 385 without.
//   A part is `part_k` ids in every chunk.  The first chunk is the widest: it fills all
// `parts`, the ones that exist, and stores them; a later chunk adds to as many or fewer.
struct ScorePlan {
  int chunk, parts, part_k;
  // of a chunk of cw ids
  int splits(int cw) const { return (cw + part_k - 1) / part_k; }
};
inline ScorePlan score_plan(int64_t n, int64_t h, int64_t v) {
  constexpr int64_t kPairs = 76;
  const int64_t whole = (v + 255) / 256 * 256;
  const int64_t fit = (int64_t{1} << 26) / std::max<int64_t>(n, 1) / 256 * 256;
  const int64_t wide = std::min<int64_t>({fit, int64_t{1} << 17, whole});
  const int64_t chunk = std::max<int64_t>(std::min<int64_t>(chunk_width(n), whole), wide);
  const int64_t first = std::min(chunk, v);
  const int64_t tiles = (n + kPairRows - 1) / kPairRows * ((h + kBN - 1) / kBN);
  int64_t parts = tiles < kPairs ? (2 * kPairs + tiles - 1) / std::max<int64_t>(tiles, 1) : 1;
  parts = std::min<int64_t>({parts, first / 512, (int64_t{1} << 24) / std::max<int64_t>(n * h, 1)});
  // fewer than 4 parts save less than the launch that adds them up costs
  if (parts < 4) return ScorePlan{static_cast<int>(chunk), 1, static_cast<int>(chunk)};
  const int part_k = static_cast<int>((first + kBK * parts - 1) / (kBK * parts)) * kBK;
  return ScorePlan{static_cast<int>(chunk), static_cast<int>((first + part_k - 1) / part_k), part_k};
}

enum Mode : int {
  kModeForward = 0,
  kModeGrad = 1,
  kModeBwd = 2,
  kModeFwdStore = 3,
  kModeTopk = 4,
  kModeScore = 5,      // forward with the entropy's sum, at a temperature
  kModeScoreTop = 6,   // the same with each row's best logits
  kModeGradScore = 7,  // G of the gradients of token log probabilities and entropies
  kModeScoreTopWide = 8,  // kModeScoreTop with eight epilogue warps (see score_subranges)
};

// Forward-store: a row's p~ is stored relative to its reference logit (log2
// units) unless a tile's p~ sum exceeds 2^kRefSpan; then relative to the
// tile's max.
constexpr float kRefSpan = 64.f;

constexpr int kTopkMax = 16;     // largest k of flce_topk / of soft targets per row
constexpr int kTopkSplit = 16;   // most vocabulary splits of the top-k pass (bounds its partial buffer)
constexpr int kScoreSplitMax = 80;  // most vocabulary splits of the score pass (see score_splits)

// Output format of the dX / dW tiles of a kModeBwd launch.
enum OutMode : int {
  kOutF32Store = 0,      // fp32 stored to dx_f32 / dw_f32
  kOutF32Add = 1,        // fp32 added at L2 to dx_f32 / dw_f32
  kOutBF16 = 2,          // bf16 through `out`/`out2`
  kOutF32AccToBF16 = 3,  // dW only: read the fp32 accumulator through `out2`, add, write bf16 through `out3`
};

// Everything a tensor-core launch needs besides its tensor maps.
struct TcParams {
  int n, h, v;
  int ignore_index;
  uint64_t timeout_ns;
  int* status;
  // forward: row pair tiles (256 rows) x vocabulary splits
  int row_tiles, vocab_tiles, vsplit;
  float* part_m;  // [vsplit][n] running max, log2 units
  float* part_l;  // [vsplit][n] running sum of 2^(t - m)
  float* tgt;     // [n] target logit z_{i, y_i}
  const int32_t* labels;
  int shift, seq_len;   // shift = 1: row i is scored against labels[i + 1]; each sequence's last row is ignored
  const float* grad_rows;  // grad (reduction none): per-row upstream gradient, or null
  // grad / bwd: one vocabulary chunk [c0, c0 + cw)
  int c0, cw;
  const float* lse;
  const float* scale;  // device scalar s
  int grad_n_tiles;    // grad: vocabulary tiles in the chunk
  // bwd: dX tiles then dW tiles
  int dx_tiles, dw_tiles;
  int h_tiles;          // ceil(h / kBN)
  int dw_m_tiles;       // ceil(cw / kPairRows)
  int dx_out, dw_out;   // OutMode of the dX and dW tiles
  float* dx_f32;        // bwd: the fp32 dX accumulator [n, h] for kOutF32Store / kOutF32Add dX tiles (else null)
  float* dw_f32;        // bwd: the fp32 dW accumulator [v, h] for kOutF32Store / kOutF32Add dW tiles (else null)
  int dx_k, dw_k;       // K extents: dX tiles run over dx_k vocabulary ids, dW tiles over dw_k rows
  int dx_first;         // 1: dX tiles are listed first (they are the long ones)
  // bwd with dx_splits > 1: each dX tile's K is cut into that many parts of dx_split_k ids (a
  // multiple of kBK), part s a tile of its own that goes to dx_f32 + s n h
  int dx_splits, dx_split_k;
  int* tile_counter;    // bwd: global tile counter, zero at launch
  // row chunk of the forward-store pass: rows [r0, row_end) (row_end 0 means n)
  int r0, row_end;
  float* mtile;         // forward-store: per (chunk row, vocabulary tile) reference exponent, log2 units
  const float* mref;    // forward-store: per row of X its reference logit, log2 units
  const float* rowscale;  // bwd: per chunk row factor f_i of the stored G / (s f_i) (null: the buffer holds G)
  int b2_r0;            // bwd: first row of the dW B operand's tensor map
  int* zero_words;      // if set: two ints the launch sets to 0 once its predecessors are done
  // top-k pass: per (split, row) the best topk_k (logit, id) pairs, [vsplit][n][kTopkMax]
  float* topk_val;
  int32_t* topk_idx;
  int topk_k;
  uint64_t* topk_keys;  // score modes: the same as candidate keys, [n][vsplit][topk_k]
  unsigned* topk_thr;   // top-k: per row the best 16th-best value any range has reached (ordered key), zeroed
  int units_group;      // forward modes: row tiles per unit group (see units_group_rows)
  // element counts of the buffers above that are indexed by computed offsets (checked in
  // builds with FLCE_DEBUG_CHECKS): part_m / part_l, mtile, topk_val / topk_idx, rowscale
  int64_t part_count, mtile_count, topk_count, rowscale_count;
  // score modes and their gradient: log2 e / temperature, 1 / temperature, the third
  // partial of each (split, row), per-row upstream gradients (either may be null; those of
  // the log probabilities are in grad_rows) and entropies
  float zscale, inv_temp;
  float* part_s;        // sum of 2^(t - m) (t - m)
  const float* grad_ent;
  const float* entropy;
  int soft_grad;        // grad: soft targets (every row valid, no one-hot; grad_rows carries s Q_i)
};

// Unit order of the forward modes: units (row tile, vocabulary range) run row
// tile fastest within a group of this many row tiles, then range, then group.
// A group's X panels (256 rows x H bf16 each) fit in 48 MB, so they stay in
// L2 while the pairs of a wave share each W tile: W is read from memory about
// once per group instead of once per row tile.
inline int units_group_rows(int row_tiles, int64_t h) {
  const int64_t panel = static_cast<int64_t>(kPairRows) * h * 2;
  int64_t g = (int64_t{48} << 20) / panel;
  if (g < 1) g = 1;
  return static_cast<int>(g < row_tiles ? g : row_tiles);
}

// First vocabulary tile of range sp when vocab_tiles tiles are cut into vsplit
// ranges: the first (vocab_tiles % vsplit) ranges take one tile more than the
// rest, so the units handed out last (the highest ranges) are the smaller ones.
FLCE_HOST_DEVICE inline int range_begin(int sp, int vocab_tiles, int vsplit) {
  const int base = vocab_tiles / vsplit;
  const int rem = vocab_tiles % vsplit;
  return sp * base + (sp < rem ? sp : rem);
}

// The (row tile, range) of unit u in that order.
FLCE_HOST_DEVICE inline void unit_coords(int u, int row_tiles, int vsplit, int group, int* rt, int* sp) {
  const int per_group = group * vsplit;
  const int g = u / per_group;
  const int g0 = g * group;
  const int rows_g = row_tiles - g0 < group ? row_tiles - g0 : group;  // the last group may be short
  const int local = u - g * per_group;
  *rt = g0 + local % rows_g;
  *sp = local / rows_g;
}

struct TcMaps {
  CUtensorMap a;   // forward/grad: X (K-major, box 64x128); bwd: G K-major (dX)
  CUtensorMap b;   // forward/grad: W (K-major, box 64x256); bwd: W MN-major (dX)
  CUtensorMap out; // grad: G store (bf16 box 64x32); bwd: dX fp32 accumulator (box 32x32)
  CUtensorMap a2;  // bwd: G MN-major (dW A operand, box 64x64)
  CUtensorMap b2;  // bwd: X MN-major (dW B operand, box 64x64)
  CUtensorMap out2;// bwd: dW output (bf16 box 64x32, or the fp32 accumulator, box 32x32)
  CUtensorMap out3;// bwd, kOutF32AccToBF16: dW bf16 store (box 64x32)
};

// Launchers (asynchronous on `stream`; return the launch error, if any).
cudaError_t launch_tc(int mode, const TcMaps& maps, const TcParams& p, int grid, cudaStream_t stream);
// Labels as the kernels read them: with shift, row i takes labels[i + 1] and
// the last row of each sequence of seq_len rows is ignored.
struct LabelView {
  const int32_t* labels;   // hard labels (may be null when soft targets are given)
  int ignore_index;
  int shift, seq_len;
  // soft targets: per row soft_k (vocabulary id, probability) pairs; soft_k = 0 for hard labels
  const int32_t* soft_idx;
  const float* soft_prob;
  int soft_k;
};

cudaError_t launch_fwd_finalize_rows(int r0, int rows, int n, int v, int vsplit, LabelView lv, const float* part_m,
                                     const float* part_l, const float* tgt, float* lse, float* loss_rows,
                                     double* blk_loss, int* blk_valid, int* status, cudaStream_t stream);
// Fused path.  label_prep: label check, the rows' references (log2 units: the
// target logit, or for soft targets the q-weighted mean target logit, whose
// q-weighted sum goes to tgt; +inf for rows without a gradient) and, through
// the last block, n_valid and s.
cudaError_t launch_label_prep(int n, int h, int v, int reduction, LabelView lv, const void* X, const void* W,
                              float* mref, float* tgt, int* blk_cnt, int* ticket, int* n_valid, float* scale,
                              int* status, cudaStream_t stream);
// finalize_ref, rows [r0, r0 + rows) of one chunk: lse, losses and the loss
// partials (one per kRefRowsPerBlock rows, index r0 / kRefRowsPerBlock + b),
// the row factors f_i, the chunk buffer's target entries, xs = f x, and the
// list of rows a tile stored relative to its own max (fix_list / fix_count).
constexpr int kRefRowsPerBlock = 8;
cudaError_t launch_finalize_ref(int r0, int rows, int n, int h, int v, int vp, int vsplit, LabelView lv,
                                const float* part_m, const float* part_l, const float* tgt, const float* mref,
                                float* lse, float* loss_rows, double* blk_loss, int* blk_valid,
                                float* rowscale, const void* X, void* xs, void* P, int* fix_list, int* fix_count,
                                int* status, cudaStream_t stream);
// The listed rows' full fix-up (G / s in place), `grid` blocks.
cudaError_t launch_fixup_list(const int* fix_list, const int* fix_count, int r0, int v, int vp, int vtiles,
                              LabelView lv, const float* lse, const float* mtile, void* P, int grid,
                              cudaStream_t stream);
// nsub: the (max, sum) pairs and candidate lists per row, vocabulary sub-ranges.
cudaError_t launch_topk_finalize(int n, int nsub, int k, const float* part_m, const float* part_l,
                                 const float* cand_val, const int32_t* cand_idx, float* lse, float* out_val,
                                 int32_t* out_idx, cudaStream_t stream);
cudaError_t launch_label_scan_view(int n, int v, LabelView lv, double* blk_loss, int* blk_valid, int* status,
                                   cudaStream_t stream);
cudaError_t launch_reduce_final(int nblk, const double* blk_loss, const int* blk_valid, int reduction,
                                const float* grad_loss, float* loss_out, int* n_valid_out, float* scale_out,
                                cudaStream_t stream);
cudaError_t launch_convert_bf16(const float* src, void* dst, int64_t count, cudaStream_t stream);
// dX from its parts: dst[i] = bf16(sum of src[s * count + i] in the order of s); count a multiple of 8.
cudaError_t launch_sum_parts_bf16(const float* src, int parts, void* dst, int64_t count, cudaStream_t stream);
// fp32 -> bf16 (round to nearest even) of any count; src and dst 16-byte aligned.
cudaError_t launch_f32_to_bf16(const float* src, void* dst, int64_t count, cudaStream_t stream);

// Soft targets on the bounded path: per row s Q_i (the grad launch's
// coefficient), and a vocabulary chunk's target entries G_ij -= s q_k in place.
cudaError_t launch_soft_rowcoef(int n, int k, const float* soft_prob, const float* scale, float* coef,
                               cudaStream_t stream);
cudaError_t launch_soft_chunk_targets(int n, int k, const int32_t* soft_idx, const float* soft_prob,
                                      const float* scale, int c0, int cw, int64_t pitch, void* G, int v, int* status,
                                      cudaStream_t stream);

// Token log probabilities: per row, from the splits' partials, lse, the log probability of
// its label (0 where ignored), the entropy (any but lse may be null) and, for k > 0, the k
// best of the candidates with their log probabilities.  zscale, inv_temp as in TcParams.
//
// Most splits of an n-row score pass: enough that one row tile's ranges occupy every CTA
// pair (76 on this GPU), 16 (as for the top-k pass) from ten row tiles on.
constexpr int kScoreSub = 2;  // most sub-ranges that a score launch reports for each vocabulary split
// Those that it does: two, of eight epilogue warps, but with alternatives only where a tile's
// contraction is too short to hide the epilogue of four.  Four warps and eight (us), 777 rows x
// 40009 ids, k = 16: H = 256 101 and 94, 1024 110 and 103, 1544 123 and 128, 4096 206 and 214;
// 8192 x 32000, k = 8: H = 256 360 and 300, 1024 398 and 382, 2048 626 and 634, 4096 1227 and 1253.
inline int score_subranges(int64_t h, int k) { return k == 0 || h <= 1024 ? 2 : 1; }
inline int score_splits(int64_t n) {
  const int64_t row_tiles = (n + kPairRows - 1) / kPairRows;
  const int64_t s = row_tiles > 0 ? 2 * kScoreSplitMax / row_tiles : kScoreSplitMax;
  return static_cast<int>(s < 16 ? 16 : s > kScoreSplitMax ? kScoreSplitMax : s);
}
cudaError_t launch_score_finalize(int n, int v, int nsplit, int k, LabelView lv, float zscale, const float* part_m,
                                  const float* part_l, const float* part_s, const float* tgt,
                                  const uint64_t* cand_keys, float* logprob, float* entropy, float* lse,
                                  int32_t* top_ids, float* top_logprobs, int* status, cudaStream_t stream);

// The same for a few rows (flce_decode.cu): CTAs own vocabulary ranges, at most kDecodeCtas
// of them.  X and W are read through K-major maps: x
// with a_rows (n rounded up to a multiple of 8) rows a box, w[i] with 256 >> i.
constexpr int kDecodeRows = 128;  // most rows
int decode_copies(int64_t n, int64_t h, int64_t v, int k);
constexpr int kDecodeCtas = 160;
constexpr int kDecodeBoxes = 5;   // 256 rows to 16
constexpr int kDecodeSlots = 24;  // most candidates of a part
struct DecodeMaps {
  CUtensorMap x, w[kDecodeBoxes];
};
struct DecodeParams {
  int n, h, v, k;
  int a_rows;
  int copies;  // of X on the MMA's 128 rows: 4, 2 or 1; each reports a part of the CTA's range
  int parts;   // per token
  int slots;   // candidates a part may report, at least k
  int ignore_index, shift, seq_len;
  float zscale;
  uint64_t timeout_ns;
  const int32_t* tokens;
  float *part_m, *part_l, *part_s;  // [n][parts]
  uint64_t* cand;                   // [n][parts][slots]
  float* tgt;                       // [n]
  int* err;                         // [CTAs] error codes
  int* status;
  int64_t part_count;               // elements of each part array (debug builds)
};
cudaError_t launch_decode(const DecodeMaps& maps, const DecodeParams& p, int ctas, float* logprob, float* entropy,
                          float* lse, int32_t* top_ids, float* top_logprobs, cudaStream_t stream);

// Vocabulary shards.  A shard's kernels read labels in shard-local form: -1 for an
// ignored row (the shard calls run with ignore_index -1), y - v0 for a label the
// shard holds, kNotOwned for a valid label held by another shard (it never equals
// a column index, so no tile gathers it and no one-hot entry is subtracted).
constexpr int kNotOwned = 0x7fffffff;
cudaError_t launch_shard_labels(int n, int64_t v_total, int64_t v0, int64_t vs, LabelView lv, int32_t* lab_local,
                                int* status, cudaStream_t stream);
// Per row: the shard's lse (natural log) from the split partials, and its target
// logit where the shard holds the label (0 elsewhere).
cudaError_t launch_shard_finalize(int n, int vsplit, const float* part_m, const float* part_l, const float* tgt,
                                  const int32_t* lab_local, float* lse_part, float* tgt_part, cudaStream_t stream);
// Per row: lse = log sum_r exp(lse_parts[r]), z = sum_r tgt_parts[r] (parts in index
// order), the loss row against the global labels, and per-block partials.
cudaError_t launch_shard_combine(int n, int parts, int64_t v_total, LabelView lv, const float* lse_parts,
                                 const float* tgt_parts, float* lse, float* loss_rows, double* blk_loss,
                                 int* blk_valid, int* status, cudaStream_t stream);
cudaError_t launch_scale_bf16(void* x, int64_t count, const float* g, cudaStream_t stream);
cudaError_t launch_timeout_selftest(int* status, uint64_t limit_ns, cudaStream_t stream);
// One thread tests index 1 against a buffer of one element: builds with
// FLCE_DEBUG_CHECKS record kErrBounds (and touch no memory), release builds nothing.
cudaError_t launch_bounds_selftest(int* status, cudaStream_t stream);

// Layer norm (flce_norm.cu).
struct NormParams {
  int64_t n;
  int h;
  int64_t x_pitch;
  float eps;
  bool x_f32, w_f32;  // else bf16
};
size_t norm_partial_floats(int64_t n, int64_t h);  // of the backward pass's workspace
cudaError_t launch_norm_forward(const NormParams& q, const void* x, const void* weight, const void* bias, void* y,
                                float* mean, float* rstd, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormParams& q, const void* dy, const void* x, const void* weight,
                                 const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                                 float* part, cudaStream_t stream);

// Embedding (flce_embed.cu).
constexpr int kEmbedRangeBits = 9;
constexpr int kEmbedRanges = 1 << kEmbedRangeBits;  // of the vocabulary, a block's each in the sort
constexpr int64_t kEmbedIdsMost = 1 << 20;   // rows of a matrix
constexpr int kEmbedStretches = 304;         // of the positions: two blocks for each SM
constexpr int64_t kEmbedFew = 16384;         // tokens up to which one launch sorts them
// Tokens of the sorted order that a warp sums at once.  Few tokens or short rows need small tiles to
// occupy the GPU, many leave fewer parts in large ones: 131072 x 4096 in 259 us with 64, 286 with 32
// (frequent ids: 328, 390), 131072 x 1001 in 126, 128 (235, 314), 32768 x 512 in 40, 36 (44, 46).
constexpr int kEmbedTile = 32, kEmbedTileMany = 64;
FLCE_HOST_DEVICE inline int embed_tile(int64_t n, int64_t h) {
  return n >= 32768 && n * ((h + 255) / 256) >= 131072 ? kEmbedTileMany : kEmbedTile;
}
// The sorted order is one of ids' keys.  One launch's blocks take consecutive ids; in two launches a
// range is every kEmbedRanges-th id: vocabularies put their frequent ids side by side, and a block
// with all of them was the end of the sort (131072 tokens, the first 98 of 50000 ids a third of
// them: 168 us).
struct EmbedKeys {
  int bits;  // range: the id's low bits
  int per;   // ids of a range
  FLCE_HOST_DEVICE int of(int id) const { return (id & ((1 << bits) - 1)) * per + (id >> bits); }
  FLCE_HOST_DEVICE int id(int key) const { return (key % per << bits) + key / per; }
  FLCE_HOST_DEVICE int count() const { return per << bits; }  // some of ids past the vocabulary's end
};
FLCE_HOST_DEVICE inline EmbedKeys embed_keys(int64_t n, int64_t v) {
  const int bits = n <= kEmbedFew ? 0 : kEmbedRangeBits;
  return EmbedKeys{bits, static_cast<int>((v + (int64_t{1} << bits) - 1) >> bits)};
}
struct EmbedParams {
  int64_t n;
  int h;
  int64_t v;
  float scale;
  bool w_f32, y_f32;  // else bf16
};
// The tokens other than the padding id in the order of (key, position): their positions and
// ids, start[keys + 1] of each key's, and the parts of the rows whose tokens lie in several tiles.
struct EmbedSorted {
  int32_t* start;
  int32_t* order;
  int32_t* sorted_id;
  void* tokens;    // [n] (id, position), by stretch and range
  int32_t* off;    // [kEmbedRanges + 1][kEmbedStretches]
  int32_t* bad;    // [kEmbedStretches]
  float* part;
  int* status;
};
// Parts of n tokens with rows of h elements: two, of whole groups of 256, for each tile of the
// sorted order.
FLCE_HOST_DEVICE inline int64_t embed_part_floats(int64_t n, int64_t h) {
  const int64_t tile = embed_tile(n, h);
  return n > tile ? 2 * ((n + tile - 1) / tile) * ((h + 255) / 256 * 256) : 0;
}
cudaError_t launch_embed_forward(const EmbedParams& q, const int32_t* ids, const void* w, void* y, int* status,
                                 cudaStream_t stream);
cudaError_t launch_embed_sort(const EmbedParams& q, int pad, const int32_t* ids, const EmbedSorted& o, int sms,
                              cudaStream_t stream);
cudaError_t launch_embed_backward(const EmbedParams& q, const void* dy, const EmbedSorted& o, void* dw, bool add,
                                  cudaStream_t stream);

// AdamW (flce_adamw.cu).  The tensors travel as a kernel argument, so a step needs no
// table in device memory; an argument holds at most 32764 bytes.
constexpr int kAdamwBlock = 256;   // elements of one 8-bit scale
constexpr int kAdamwChunk = 4096;  // elements of one thread block
struct AdamwTensor {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t count;
  float decay;     // 1 - lr wd
  float rate;      // lr / (1 - beta1^step)
  uint32_t flags;  // kAdamwParamF32 | ...
  uint32_t chunk0; // chunks of the tensors before this one
};
enum : uint32_t { kAdamwParamF32 = 1, kAdamwGradF32 = 2, kAdamwAligned = 4 };
constexpr int kAdamwManyTensors = 400;
constexpr int kAdamwFewTensors = 16;
template <int N>
struct AdamwArgs {
  AdamwTensor t[N];
  int tensors;
  uint32_t chunks;
  float beta1, omb1, beta2, omb2;  // omb = 1 - beta
  float inv_root_bc2;              // 1 / sqrt(1 - beta2^step)
  float eps;
  uint32_t step_key;               // of the 8-bit rounding's hash
  const float* grad_scale;
};
static_assert(sizeof(AdamwArgs<kAdamwManyTensors>) <= 32764, "kernel argument limit");
template <int N>
cudaError_t launch_adamw(const AdamwArgs<N>& a, int state_bits, cudaStream_t stream);

// Muon (flce_muon.cu).  Matrices of one shape form a group, [matrix][rows][pitch] in the workspace; a
// call runs in rounds of as many groups and matrices as the kernels' arguments hold.
constexpr int kMuonGroups = 12, kMuonMatrices = 256;
// Most calls of latency's kind have one or a few matrices: kernels whose arguments hold no more take
// 1 KB where the others take 17 KB (with fewer maps 45 us of the host for 52, 128 x 128).
constexpr int kMuonFewGroups = 2, kMuonFewMatrices = 16;
constexpr int kMuonChunk = 8192;     // elements of one block of the momentum's pass
constexpr int kMuonStrip = 4096;     // and of the passes between a tensor and X
constexpr int kMuonExactRows = 128;  // up to this many rows or columns: pairs of fp16, steps on X X^T alone
constexpr int kMuonSplitBlocks = 8;  // of 64 elements, of one part of their X X^T
constexpr int kMuonSplitsMost = 64;
// The steps on X X^T go on until singular values may have grown this much, then X is read again: an
// error d of an eigenvalue grows with the square of what singular values do, and counts as
// |b| / a d 144^2 then in the weakest directions' factor.  d is up to 2^-22 by its pair and 5e-8 by fp32 sums:
// 2e-3 to 7e-3 of these directions.  The usual coefficients reach 141 before the fifth step, 485
// before a sixth, which on 128 x 128 with strong directions is off by 1e-3, an eighth step
// by 2e-2 and a twelfth by infinities (simulated); with reads every five steps by 4e-4, 5e-4, 9e-4
// (measured).  A read is three launches, 20 us of the 101 of 6 steps there.
constexpr double kMuonReadGrowth = 144.0;
// Larger matrices' iterates are pairs too, but for the last: a rounding to one fp16 leaves 2e-4 of
// X's norm in its weak directions, which the remaining steps multiply by up to their slopes at 0.  Iterates are
// single from where these products add up to at most 16 (usual coefficients: the last two, 3.4 + 11.9; the
// first three are pairs however gentle the steps).  Of 300 x 777 with eight directions over 0.2% of noise
// the result is off by 3e-3 after five usual steps (2e-3 with all as pairs), 2e-3 after six, 7e-4 after
// eight; with three pairs for any number of steps by 7e-3 and 9e-3, without noise 0.2 after eight
// (simulated).  A pair costs P X 10 us of 45 more for 40M elements.
constexpr int kMuonPairSteps = 3;
constexpr double kMuonPairGrowth = 16.0;
constexpr float kMuonXScale = 16384.f, kMuonAScale = 8192.f;
// The largest singular value of X and shift of A's diagonal that coefficients may lead to: A, P A
// and X stay below fp16's 65504.  (Schedules of steep first steps reach 2.)
constexpr double kMuonMostX = 2.1, kMuonMostShift = 3.0;
static_assert((kMuonMostX * kMuonMostX + kMuonMostShift) * kMuonAScale < 65000 && kMuonMostX * kMuonXScale < 65000, "fp16");
enum MuonMode : int { kMuonGram, kMuonPoly, kMuonApply };
enum : uint32_t {
  kMuonParamF32 = 1,
  kMuonGradF32 = 2,
  kMuonAligned = 4  // gradient and momentum: four elements at a time from the start on
};
// One launch's view of a group: out = alpha a b, + gamma (and in kPoly alpha diag) on the diagonal,
// + beta lo; [m, n].  Operands in boxes of 64 columns by 128 and by 64 rows.
struct MuonGroup {
  CUtensorMap a128, a64, b128, b64;
  CUtensorMap a_lo128, a_lo64, b_lo128, b_lo64;  // what their rounding to fp16 left (segments = 3)
  CUtensorMap out, out_lo;
  float* diag;  // [matrix][m], for the square: what rounding the diagonal left (null: nothing)
  float alpha, beta, gamma;
  float* part;  // kGram of a matrix of few rows: alpha a b of each split of the contraction, [matrix][split][128][128]
  int m, n;
  int kblocks, segments;  // 64-element steps of the contraction; 3 for hi hi + hi lo + lo hi, else 1
  int split_blocks;       // of one split of kGram's parts
  int tile0, tiles_each, row_tiles, col_tiles;
  int tall;               // X has more rows than columns
  int lo_in, write_lo;    // add beta times out_lo's old values; write out_lo
};
template <int G>
struct MuonArgs {
  MuonGroup g[G];
  int groups, tiles;
  uint64_t timeout_ns;
  int* status;
};
static_assert(sizeof(MuonArgs<kMuonGroups>) <= 32764, "kernel argument limit");
// The steps of the matrices of at most kMuonExactRows rows between two reads of X, from X X^T to
// the product Q of their P, a block each.
struct MuonChainGroup {
  const float* part;   // X X^T in kGram's parts, in units of 1 / kMuonAScale
  int splits;
  __half *q, *q_lo;    // [matrix][r][pitch]
  int r, pitch;
  int block0;
};
struct MuonChain {
  MuonChainGroup g[kMuonGroups];
  float a[16], b[16], c[16];  // of each step
  float p_scale, q_scale[16];
  int groups, blocks, steps;
  uint64_t timeout_ns;
  int* status;
};
struct MuonSource {
  const void* grad;
  float* momentum;  // or null: the gradient itself is what is orthogonalised
  __half *hi, *lo;  // X, rows of `pitch` elements
  int rows, cols, pitch;
  uint32_t flags;
  int vec;  // columns at a time that every tensor's rows allow: 4, 2 or 1
};
template <int N>
struct MuonSources {
  // the first block of work of each source, and the number of blocks behind the last: apart from
  // the sources, so that a search stays within a few lines of the constant cache
  uint32_t chunk0[N + 1], strip0[N + 1];
  MuonSource s[N];
  int count;
  float mu, omm;  // momentum and 1 - momentum
  int nesterov;
  float eps;
  const float* grad_scale;
  float* part;   // a sum of squares for each chunk
  int* status;
  int first;     // the momentum's pass clears the status word
};
static_assert(sizeof(MuonSources<kMuonMatrices>) <= 32764, "kernel argument limit");
// Where X goes: out (bf16), or w <- w decay - rate X on the weights.
struct MuonTarget {
  const __half *hi, *lo;  // (lo may be null)
  void* out;
  void* param;
  float* master;
  float decay, rate;
  int rows, cols, pitch;
  uint32_t flags;
  int vec;
};
template <int N>
struct MuonTargets {
  uint32_t strip0[N + 1];
  MuonTarget t[N];
  int count;
  int* status;
};
static_assert(sizeof(MuonTargets<kMuonMatrices>) <= 32764, "kernel argument limit");
int64_t muon_strips(int64_t rows, int64_t cols, int vec);  // blocks of the scale's or the weights' launch for one matrix
// N: kMuonMatrices or kMuonFewMatrices; G: kMuonGroups or kMuonFewGroups.
template <int N>
cudaError_t launch_muon_momentum(const MuonSources<N>& a, cudaStream_t stream);
template <int N>
cudaError_t launch_muon_scale(const MuonSources<N>& a, int sms, cudaStream_t stream);
template <int N>
cudaError_t launch_muon_weights(const MuonTargets<N>& a, int sms, cudaStream_t stream);
cudaError_t launch_muon_chain(const MuonChain& a, cudaStream_t stream);
// bn: columns of a tile, 256 or 128.
template <int G>
cudaError_t launch_muon_product(int mode, int bn, const MuonArgs<G>& a, int sms, cudaStream_t stream);

// Limit of every bounded wait in the kernels, in nanoseconds: FLCE_TIMEOUT_NS
// from the environment (read once), else 4 s.
uint64_t timeout_ns();

int tc_smem_bytes();
int tc_topk_subranges();  // vocabulary sub-ranges the top-k launch reports per range
constexpr int kFinalizeThreads = 256;

}  // namespace flce
