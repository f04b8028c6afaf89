// Causal attention of packed query rows over the paged cache: what its kernels share.
//
// Row (t, h) of sequence b, at position pos = len_b - n_b + t, attends to tokens 0..pos:
//   x_u = sm_scale q . k_u,  lse = log sum_u exp(x_u),  out = sum_u exp(x_u - lse) v_u.
// The group's G query heads read the same keys, so a tile's rows are (token, head) pairs of
// one KV head, token-major: a tile of R rows is R / G consecutive tokens.
//
// Division of the work. An item is one row tile of one KV head; it costs its key tiles plus a
// fixed part. The items of the whole batch, in the order (sequence, KV head, row tile), form
// one line of cost units, and each of the NC blocks takes an equal piece of the line,
// whatever the lengths: a prompt of one sequence, a ragged batch and single tokens over long
// caches are all divided evenly, and the host needs to know no length. An item that a piece's
// border cuts is computed in parts: each block leaves its rows' (m, l, acc) in the workspace
// (a block has at most two such parts, its first and its last) and notes where its piece begins
// (BorderNote), from which a merge kernel, whose blocks are the borders, joins the parts. Every
// block finds its own piece from the lengths: one pass over the batch's offsets, a scan, and
// closed forms inside the sequence.
#pragma once

#include "packed_rows.cuh"

namespace skv {

// Where block c's piece of the line begins: the item there (by its first packed row and KV head)
// and the block's key tiles of it. 0 < kt0 < nk: the border cuts the item, whose part before
// it is block c - 1's last unless block c - 1 notes the same item with kt0 > 0.
struct BorderNote {
  int row0, n_tok, g;
  int kt0, kt1, nk;
};

struct PrefillArgs {
  const void* q;
  int64_t q_stride;       // elements between tokens
  void* out;              // [total][Hq][D] of the cache's type
  float* lse;             // [total][Hq], or NULL
  float* part_acc;        // [2 NC][part_rows][D], when NC > 1
  float* part_ml;         // [2 NC][part_rows][2]: m in base 2 (-inf: no keys), l
  BorderNote* notes;      // [NC]
  float scale_log2;       // sm_scale * log2(e)
  int Hq, G, log_g;
  int NC;                 // blocks the work is divided among
  int part_rows;          // rows of a part: a tile's, or all there are
};

// Tile sizes of a kernel: R rows by KT keys, and what an item costs: two units per key tile, one
// where the item has at most WIDE rows, and a fixed part of kItemCost units (bf16: an item's start
// and end are 5000 to 9000 cycles, a unit 1300; 3, 4, 5 and 8 give 240, 242, 247 and 257 us for
// sixteen ragged prompts, and 351, 345, 345 and 350 for one of 8192 tokens in pages of 64).
template <int R, int KT, int WIDE> struct TileShape {
  static constexpr int rows = R, keys = KT, narrow = WIDE;
};
constexpr int kItemCost = 4;
constexpr int kMinPart = 2;      // a border leaves an item at least this many key tiles

// One sequence's rows as items, the same for each of its KV heads.
template <typename S> struct SeqItems {
  int row0, n, len;
  int tq_log;      // log2 of the tokens of a row tile

  __device__ __forceinline__ SeqItems(const SeqRows& s, int log_g)
      : row0(s.row0), n(s.n), len(s.len), tq_log(__ffs(S::rows) - 1 - log_g) {}
  __device__ __forceinline__ int tiles() const {
    return (int)(((int64_t)n + (1 << tq_log) - 1) >> tq_log);
  }
  __device__ __forceinline__ int tokens(int tile) const {
    return min(1 << tq_log, n - (tile << tq_log));
  }
  __device__ __forceinline__ int key_tiles(int tile) const {
    const int64_t keys = (int64_t)(len - n) + (tile << tq_log) + tokens(tile);
    return (int)((keys + S::keys - 1) / S::keys);
  }
  __device__ __forceinline__ int unit(int tile, int log_g) const {
    return (tokens(tile) << log_g) > S::narrow ? 2 : 1;
  }
  // Cost of the first x tiles. All but the sequence's last tile are full: FULL units for each
  // of ceil((past + (j + 1) TQ) / KT) key tiles.
  __device__ __forceinline__ int64_t cost(int x, int log_g) const {
    constexpr int FULL = S::rows > S::narrow ? 2 : 1;
    const int nt = tiles();
    int64_t c = (int64_t)kItemCost * x;
    if (x == nt && x > 0) {
      --x;
      c += (int64_t)unit(x, log_g) * key_tiles(x);
    }
    const int a = len - n + S::keys - 1;            // sum of floor((a + j TQ) / KT), j = 1..x
    if ((1 << tq_log) >= S::keys) {
      const int64_t r = (1 << tq_log) / S::keys;
      return c + FULL * (x * (int64_t)(a / S::keys) + r * ((int64_t)x * (x + 1) / 2));
    }
    const int r_log = (__ffs(S::keys) - 1) - tq_log, r = 1 << r_log;
    const int rest = (a & (S::keys - 1)) >> tq_log;
    // floor((rest + j) / r) summed over j = 1..x; below r the terms are zero
    const int64_t y = (int64_t)rest + x + 1, q = y >> r_log;
    const int64_t steps = r * (q * (q - 1) / 2) + q * (y & (r - 1));
    return c + FULL * (x * (int64_t)(a / S::keys) + steps);
  }
};

// An item, or this block's part of it: rows of `n_tok` tokens from packed row `row0` on, of KV
// head g; row r is token r / G and sees keys up to pos0 + r / G; key tiles [kt0, kt1).
struct PrefillItem {
  int b, g;
  int row0, n_tok, pos0;
  int kt0, kt1;
  int part;             // workspace part, or -1: the block has the whole item
};

// a / b for a >= 0, b > 0, in 32 bits where they fit: a 64-bit division is a quarter of a
// microsecond of dependent instructions, and a block's start has several.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Key tiles of an item before border `y` of the line; the item starts at x and costs `unit`
// per key tile. Borders that would leave a few tiles on one side move to the item's end.
__device__ __forceinline__ int tiles_before(int64_t y, int64_t x, int nk, int unit) {
  const int64_t k = (y - x - kItemCost + unit - 1) >> (unit - 1);       // unit is 1 or 2
  if (k >= nk) return nk;
  return k < kMinPart ? 0 : nk - k < kMinPart ? nk : (int)k;
}

// Walks the items of the piece [lo, hi) of the line. Every warp that works on the items walks
// them by itself; the lengths of the next sequence are fetched ahead.
template <typename S> class ItemWalk {
 public:
  __device__ __forceinline__ ItemWalk(const kv_cache_desc& d, const PackedRows& pr,
                                      const PrefillArgs& a, const DevCtx& ctx, int64_t lo,
                                      int64_t hi, int b, int64_t before, int block)
      : d_(d), pr_(pr), a_(a), ctx_(ctx), lo_(lo), hi_(hi), x_(before), b_(b), g_(0), tile_(-1),
        block_(block), seq_(seq_rows(ctx, d, pr, b), a.log_g), next_(fetch(b + 1)) {
    // the last item that starts at or before lo
    const int64_t head = seq_.cost(seq_.tiles(), a.log_g);
    if (head > 0) {
      g_ = (int)divide(lo - x_, head);
      x_ += g_ * head;
      int t = 0, end = seq_.tiles();
      while (end - t > 1) {
        const int mid = (t + end) >> 1;
        if (x_ + seq_.cost(mid, a.log_g) <= lo) t = mid;
        else end = mid;
      }
      x_ += seq_.cost(t, a.log_g);
      tile_ = t - 1;
    }
  }

  // The next item with key tiles for this block; false when the piece is done.
  __device__ __forceinline__ bool next(PrefillItem* it) {
    for (;;) {
      ++tile_;
      while (tile_ >= seq_.tiles()) {
        tile_ = 0;
        if (seq_.n > 0 && ++g_ < d_.num_kv_heads) continue;
        g_ = 0;
        if (++b_ >= d_.batch) return false;
        seq_ = next_;
        next_ = fetch(b_ + 1);
      }
      if (x_ >= hi_) return false;
      const int nk = seq_.key_tiles(tile_), unit = seq_.unit(tile_, a_.log_g);
      const int64_t x = x_;
      x_ += kItemCost + (int64_t)unit * nk;
      it->kt0 = tiles_before(lo_, x, nk, unit);
      it->kt1 = tiles_before(hi_, x, nk, unit);
      if (it->kt0 >= it->kt1) continue;
      it->b = b_;
      it->g = g_;
      const int t0 = tile_ << seq_.tq_log;
      it->row0 = seq_.row0 + t0;
      it->n_tok = seq_.tokens(tile_);
      it->pos0 = seq_.len - seq_.n + t0;
      it->part = it->kt0 > 0 ? 2 * block_ : it->kt1 < nk ? 2 * block_ + 1 : -1;
      return true;
    }
  }

  // What a merge has to know of the place where the piece begins.
  __device__ __forceinline__ BorderNote border() const {
    const int t = tile_ + 1;
    BorderNote n{0, 0, 0, 0, 0, 0};
    if (t >= seq_.tiles()) return n;
    n.row0 = seq_.row0 + (t << seq_.tq_log);
    n.n_tok = seq_.tokens(t);
    n.g = g_;
    n.nk = seq_.key_tiles(t);
    n.kt0 = tiles_before(lo_, x_, n.nk, seq_.unit(t, a_.log_g));
    n.kt1 = tiles_before(hi_, x_, n.nk, seq_.unit(t, a_.log_g));
    return n;
  }

 private:
  __device__ __forceinline__ SeqItems<S> fetch(int b) const {
    if (b < d_.batch) return SeqItems<S>(seq_rows(ctx_, d_, pr_, b), a_.log_g);
    return SeqItems<S>(SeqRows{0, 0, 0}, a_.log_g);
  }
  const kv_cache_desc& d_;
  const PackedRows& pr_;
  const PrefillArgs& a_;
  const DevCtx& ctx_;
  int64_t lo_, hi_, x_;
  int b_, g_, tile_, block_;
  SeqItems<S> seq_, next_;
};

// The whole line's cost, and the sequence that border number `i` of NC falls into with the
// cost before that sequence. Called by the whole block; `sh` is shared scratch.
struct LineScratch {
  int64_t sums[32];
  int64_t total, before;
  int b;
};
struct LinePlace {
  int64_t total, before;
  int b;
  int64_t lo, hi;         // block i's piece: floor(total i / NC) up to the next block's
};

template <typename S>
__device__ __forceinline__ LinePlace find_place(const DevCtx& ctx, const kv_cache_desc& d,
                                                const PackedRows& pr, const PrefillArgs& a,
                                                int i, LineScratch* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (d.batch + blockDim.x - 1) / blockDim.x;
  const int b0 = tid * per, b1 = min(d.batch, b0 + per);
  auto cost_of = [&](int b) -> int64_t {
    const SeqItems<S> s(seq_rows(ctx, d, pr, b), a.log_g);
    return s.cost(s.tiles(), a.log_g) * d.num_kv_heads;
  };
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += cost_of(b);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) sh->sums[warp] = upto;
  if (tid == 0) sh->b = -1;
  __syncthreads();
  int64_t before = upto - mine, total = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    if (w < warp) before += sh->sums[w];
    total += sh->sums[w];
  }
  const int64_t each = divide(total, a.NC);
  const int rest = (int)(total - each * a.NC);
  const int64_t lo = each * i + rest * i / a.NC;       // rest * i < 2^20
  const int64_t hi = each * (i + 1) + rest * (i + 1) / a.NC;
  const int64_t y = lo;                      // < total: some thread holds it, unless all is empty
  if (mine > 0 && y >= before && y < before + mine) {
    int b = b0;
    for (; b < b1 - 1; ++b) {
      const int64_t c = cost_of(b);
      if (y < before + c) break;
      before += c;
    }
    sh->b = b;
    sh->before = before;
  }
  __syncthreads();
  return LinePlace{total, sh->before, sh->b, lo, hi};
}

// Launchers.
using MmaShape = TileShape<256, 128, 128>;       // bf16, tensor cores
using FewShape = TileShape<128, 128, 128>;       // the same for batches of few rows
using SimtShape = TileShape<128, 64, 0>;         // fp32, CUDA cores
int prefill_tile_rows(int dtype);
cudaError_t launch_prefill(const kv_cache_desc& d, const int32_t* cu, int total,
                           const PrefillArgs& a, DevCtx ctx, cudaStream_t s);
cudaError_t launch_prefill_simt(const kv_cache_desc& d, const PackedRows& pr,
                                const PrefillArgs& a, DevCtx ctx, cudaStream_t s);
cudaError_t launch_prefill_mma(const kv_cache_desc& d, const PackedRows& pr,
                               const PrefillArgs& a, DevCtx ctx, cudaStream_t s);

// What every kernel does once: flags offsets that do not start at zero, and gives the row of
// an empty sequence (in the form of one row per sequence) zeros and lse = -inf, as a merge of
// empty splits would.
template <typename T, int D>
__device__ __forceinline__ void finish_empty(const DevCtx& ctx, const kv_cache_desc& d,
                                             const PackedRows& pr, const PrefillArgs& a) {
  if (pr.cu != nullptr) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && pr.cu[0] != 0) flag(ctx, KV_DEVERR_BAD_LEN);
    return;
  }
  for (int b = blockIdx.x; b < d.batch; b += gridDim.x) {
    if (d.seq_lens[b] != 0) continue;                // of a bad length: left out
    T* out = static_cast<T*>(a.out) + (int64_t)b * a.Hq * D;
    for (int i = threadIdx.x; i < a.Hq * D; i += blockDim.x) out[i] = T{};
    if (a.lse != nullptr)
      for (int i = threadIdx.x; i < a.Hq; i += blockDim.x) a.lse[(int64_t)b * a.Hq + i] = -INFINITY;
  }
}

}  // namespace skv
