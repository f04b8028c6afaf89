// Causal attention of packed query rows over the paged cache: what its kernels share.
//
// Row (t, h) of sequence b, at position pos = len_b - n_b + t, attends to tokens 0..pos:
//   x_u = sm_scale q . k_u,  lse = log sum_u exp(x_u),  out = sum_u exp(x_u - lse) v_u.
// The group's G query heads read the same keys, so a tile's rows are (token, head) pairs of
// one KV head, token-major: kRows rows are kRows / G consecutive tokens. A tile's keys are cut
// into key tiles, and these into S splits of whole key tiles when there are too few row tiles
// to fill the GPU; each split then leaves (m, l, acc) of its rows in the workspace, and a merge
// kernel joins them.
#pragma once

#include "packed_rows.cuh"

namespace skv {

struct PrefillArgs {
  const void* q;
  int64_t q_stride;       // elements between tokens
  void* out;              // [total][Hq][D] of the cache's type
  float* lse;             // [total][Hq], or NULL
  float* part_acc;        // [total][Hq][S][D] when S > 1
  float* part_ml;         // [total][Hq][S][2]: m in base 2 (-inf: no keys), l
  float scale_log2;       // sm_scale * log2(e)
  int Hq, G, S;
};

// A block's share: rows of `n_tok` tokens from packed row `row0` on, of KV head g, over the
// key tiles [kt0, kt1). Row r is token r / G; it sees keys up to pos0 + r / G.
struct PrefillItem {
  int b, g, s;
  int row0, n_tok, pos0, len;
  int kt0, kt1;
};

// Block x of the grid: KV heads vary fastest, then the row tiles, a sequence's last tile (the
// one with the most keys) first, so that the longest blocks start early. False: no work (a
// number past a sequence's tiles, or a sequence that was left out).
__device__ __forceinline__ bool prefill_item(const DevCtx& ctx, const kv_cache_desc& d,
                                             const PackedRows& pr, const PrefillArgs& a,
                                             int tile_tokens, int key_tile, PrefillItem* it) {
  const int item = blockIdx.x / d.num_kv_heads;
  it->g = blockIdx.x % d.num_kv_heads;
  it->s = blockIdx.y;
  int base;
  it->b = find_sequence(pr, d.batch, tile_tokens, 1, item, &base);
  const SeqRows sr = seq_rows(ctx, d, pr, it->b);
  const int tiles = (int)(((int64_t)sr.n + tile_tokens - 1) / tile_tokens);
  const int tile = tiles - 1 - (item - base);
  if (tile < 0) return false;
  const int t0 = tile * tile_tokens;
  it->len = sr.len;
  it->row0 = sr.row0 + t0;
  it->n_tok = min(tile_tokens, sr.n - t0);
  it->pos0 = sr.len - sr.n + t0;
  const int keys = it->pos0 + it->n_tok;
  const int kts = (int)(((int64_t)keys + key_tile - 1) / key_tile);
  it->kt0 = (int)((int64_t)kts * it->s / a.S);
  it->kt1 = (int)((int64_t)kts * (it->s + 1) / a.S);
  return true;
}

// The row of an empty sequence in the form of one row per sequence: zeros and lse = -inf, as
// a merge of empty splits gives.
template <typename T, int D>
__device__ __forceinline__ void empty_row(const PrefillArgs& a, int row, int g) {
  const int64_t at = (int64_t)row * a.Hq + g * a.G;
  T* out = static_cast<T*>(a.out) + at * D;
  for (int i = threadIdx.x; i < a.G * D; i += blockDim.x) out[i] = T{};
  if (a.lse != nullptr && threadIdx.x < a.G) a.lse[at + threadIdx.x] = -INFINITY;
}

// Launchers. prefill_tile_tokens: tokens of one row tile, for the grid and the split rule.
int prefill_tile_tokens(int dtype, int G);
cudaError_t launch_prefill(const kv_cache_desc& d, const int32_t* cu, int total,
                           const PrefillArgs& a, DevCtx ctx, cudaStream_t s);
cudaError_t launch_prefill_simt(const kv_cache_desc& d, const PackedRows& pr,
                                const PrefillArgs& a, DevCtx ctx, cudaStream_t s);
cudaError_t launch_prefill_mma(const kv_cache_desc& d, const PackedRows& pr,
                               const PrefillArgs& a, DevCtx ctx, cudaStream_t s);
constexpr int kPrefillSimtRows = 64, kPrefillMmaRows = 256;      // rows of a tile

}  // namespace skv
