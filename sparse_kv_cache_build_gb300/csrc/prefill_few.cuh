// Attention of few rows (single tokens in a window, small trees) for bf16 caches, with the keys in
// the tensor core's 128 rows and the query rows in its columns.
//
// An item has at most 32 rows (32 / G tokens of one KV head). Held as rows of the scores they would
// leave three quarters of the tensor memory's lanes, and of the exponentials' units, without work:
// one warp would have a row's 128 exponentials to do for every tile. So the products are turned
// round:
//   S^T = K Q^T    128 keys x 32 rows; thread k of the softmax warpgroup holds key k's scores
//   P^T            2^(scale_log2 S - m) as two bf16 parts, side by side in shared memory: 64
//                  columns; what rounding to the first leaves goes to the second
//   O^T += V^T P^T D x 64: V's tile read transposed, both parts in one product
// and a tile costs a thread as many exponentials as there are rows. At D = 64 a product of 128 rows
// takes the tile's halves of 64 keys side by side, V^T above, P^T beside each other; the blocks
// off the diagonal are not used.
//
// Reference of the softmax: the largest score so far, as of when it last grew by more than 2^8
// over the one in use, common to the four warps: one vote per tile says whether any score asks for
// a new one. Sums are kept per thread (over its keys) and joined at an item's end.
//
// Measured: 32 single tokens of 32/8 heads in a window of 1024 (134 MB) 36 us, of which the keys
// and values stream in 20 at the copy rate; 6 are a block's start (its place in the line, the
// first item, the table's entries, the first pages: dependent reads, and code that runs once),
// the rest the items' ends and the merge. In a window of 4096 102 us, 79 at the copy rate. A tile
// takes its warpgroup 1700 cycles with 8 rows, 2200 with 32, against 2800 that its bytes take
// when all SMs stream. The same by the kernel that holds rows as rows: 43 and 108 us.
//
// One warp issues the products, a tile's scores before the product with the values of the tile
// before; one feeds K and V tiles through a ring by TMA, in the order in which the products take
// them; one walks the items and loads their rows. Rows, scores, P and O are held twice, so that the
// next tile, and the next item, begin while the last one is at work.
#pragma once

#include <atomic>

#include "prefill_tma.cuh"

namespace skv {
namespace {

constexpr int kFewThreads = 224;       // softmax warpgroup, products, loads, items
constexpr int kFewMma = 4, kFewLoad = 5, kFewItem = 6;
constexpr int kFewItems = 4;           // items known ahead
constexpr int kFewKeys = SwapShape::keys, kFewTileRows = SwapShape::rows;
// Sequences up to which one warp finds the block's place: against the whole block's search, which
// has the others fetch its code and wait at its barriers, 12.5 -> 12.2 us for one sequence and 34.3
// -> 33.9 for 32 (32/8 heads, a window of 1000).
constexpr int kFewAlone = 256;
constexpr float kFewLazy = 8.f;        // log2 of the growth that forces a rescale

template <int D> struct FewCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = HALVES * 128 * 128;
  static constexpr int STAGES = D == 128 ? 5 : 10;
  static constexpr int Q_BYTES = HALVES * kFewTileRows * 128;
  static constexpr int P_BYTES = 128 * 128;                     // 128 keys x 64 columns
  static constexpr size_t OFF_RING = 0;                         // from a 1024-aligned base
  static constexpr size_t OFF_P = (size_t)STAGES * TILE_BYTES;
  static constexpr size_t OFF_Q = OFF_P + 2 * P_BYTES;
  static constexpr size_t OFF_LINE = OFF_Q + 2 * Q_BYTES;       // ancestors: 32 rows x 32 words
  static constexpr size_t OFF_RED = OFF_LINE + 4096;            // [4][32], m, factors, sums [32]
  static constexpr size_t OFF_ITEMS = OFF_RED + 7 * 128;
  static constexpr size_t OFF_BAR = OFF_ITEMS + kFewItems * 48;
  static constexpr int BARS = 2 * STAGES + 13 + 2 * kFewItems;
  static constexpr size_t OFF_TMEM = OFF_BAR + 8 * BARS;
  static constexpr size_t SMEM = OFF_TMEM + 16 + 1024;          // + alignment slack
  static_assert(SMEM <= 227 * 1024 - sizeof(LineScratch), "shared memory");
  static_assert(sizeof(MaskedItem) <= 48, "items");
  static constexpr int O_COLS = D == 128 ? 64 : 128;
  static constexpr int COL_S = 0, COL_O = 64;                   // TMEM: two S, two O
  static constexpr int TMEM_COLS = 512;
  static_assert(COL_O + 2 * O_COLS <= TMEM_COLS, "tensor memory");
};

// The softmax warpgroup's own barrier, with a vote.
__device__ __forceinline__ bool group_any(bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any) : "r"((uint32_t)x) : "memory");
  return any != 0;
}
__device__ __forceinline__ void group_sync() {
  asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
}

// Joins the lanes' 32 values each: lane r ends with row r's.
template <typename F> __device__ __forceinline__ float join_lanes(float* v, F join) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float mine = up ? v[i + o] : v[i], theirs = up ? v[i] : v[i + o];
      v[i] = join(mine, __shfl_xor_sync(0xffffffffu, theirs, o));
    }
  }
  return v[0];
}

template <int D, Mask M>
__global__ void __launch_bounds__(kFewThreads, 1)
prefill_few_kernel(const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ kv_cache_desc d,
                   const __grid_constant__ PackedRows pr, const __grid_constant__ PrefillArgs a,
                   const __grid_constant__ DevCtx ctx) {
  using C = FewCfg<D>;
  using Shape = SwapShape::With<M>;
  using Item = ItemOf<Shape>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ LineScratch scratch;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);   // [STAGES] a tile has landed
  uint64_t* empty = full + C::STAGES;            // [STAGES] its product is done
  uint64_t* s_full = empty + C::STAGES;          // [2] S^T is in TMEM
  uint64_t* p_full = s_full + 2;                 // [2] P^T is in shared memory, O rescaled
  uint64_t* pv_done = p_full + 2;                // [2] its product is done
  uint64_t* q_full = pv_done + 2;                // [2] rows are in shared memory
  uint64_t* q_free = q_full + 2;                 // [2] their last scores are done
  uint64_t* o_free = q_free + 2;                 // [2] O has been read
  uint64_t* drained = o_free + 2;                // no product in flight
  uint64_t* item_full = drained + 1;             // [kFewItems] an item is in shared memory
  uint64_t* item_free = item_full + kFewItems;   // [kFewItems] every warp is done with it
  Item* items = reinterpret_cast<Item*>(sm + C::OFF_ITEMS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_TMEM);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int log_g = a.log_g;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full + w, 1);
      mbar_init(p_full + w, 4);
      mbar_init(pv_done + w, 1);
      mbar_init(q_full + w, 1);
      mbar_init(q_free + w, 1);
      mbar_init(o_free + w, 4);
    }
    mbar_init(drained, 1);
    for (int i = 0; i < kFewItems; ++i) {
      mbar_init(item_full + i, 1);
      mbar_init(item_free + i, 6);               // four softmax warps, products, loads
    }
    fence_mbar_init();
  }
  if (warp == kFewMma) tc::alloc(tmem_slot, C::TMEM_COLS);
  tc::fence_before();
  pdl_trigger();
  pdl_wait();
  finish_empty<bf16_t, D>(ctx, d, pr, a);
  // Only the warp that walks the items needs the block's place in the line; it looks for it alone
  // where the batch is small, while the others wait for the first item.
  const bool alone = d.batch <= kFewAlone;
  LinePlace at{0, 0, 0, 0, 0};
  if (!alone) at = find_place<Shape>(ctx, d, pr, a, blockIdx.x, &scratch);
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  auto item_ready = [&](int j) {
    return wait_bounded(item_full + j % kFewItems, (j / kFewItems) & 1, ctx.wait_ns);
  };
  auto item_done = [&](int j) {
    __syncwarp();
    if (lane == 0) arrive(item_free + j % kFewItems);
  };

  if (warp < 4) {
    // ---- softmax: thread tid has key tid of every tile. The warps take the same way at every
    // vote; one that gave up a wait says so at the next.
    float* red = reinterpret_cast<float*>(sm + C::OFF_RED);     // [4][32]
    float* ref_sh = red + 128;                                  // [32] reference of a row
    float* factor_sh = ref_sh + 32;                             // [32] what it changed by
    float* sum_sh = factor_sh + 32;                             // [32] a row's sum
    uint32_t* line = reinterpret_cast<uint32_t*>(sm + C::OFF_LINE);
    const uint32_t lanes = (uint32_t)warp << 21;                // TMEM lane 32 * warp
    bool ok = true;
    int c = 0;                                                  // tiles so far

    for (int j = 0;; ++j) {
      ok = item_ready(j);
      if (group_any(!ok)) {
        ok = false;
        break;
      }
      const Item it = items[j % kFewItems];
      if (it.kt0 >= it.kt1) break;
      const int rows = it.n_tok << log_g, chunks = (rows + 7) >> 3;
      const uint32_t to = tmem + lanes + C::COL_O + (j & 1) * C::O_COLS +
                          (D == 64 && tid >= 64 ? 64 : 0);
      if (warp == 0) ref_sh[lane] = -INFINITY;
      if constexpr (M == Mask::kTree) {
        // The rows' lines of ancestors as bits by their index among the sequence's rows; a row's
        // words are turned by its number.
        const int t0 = it.pos0 - it.past;
        const int i = t0 + min(lane >> log_g, it.n_tok - 1);
        if (warp == 0) {
          const int32_t* up = a.parents + it.row0 - t0;
          for (int k = 0; k <= i >> 5; ++k) prefetch_l1(up + 32 * k);
          for (int k = 0; k < kTreeNodes / 32; ++k) line[lane * 32 + (k ^ lane)] = 0;
          for (int v = i; v >= 0;) {
            line[lane * 32 + (v >> 5 ^ lane)] |= 1u << (v & 31);
            const int next = __ldg(up + v);
            if (next >= v || next < -1) {
              flag(ctx, KV_DEVERR_BAD_SEL);
              break;
            }
            v = next;
          }
        }
        group_sync();
      }
      float ref[kFewTileRows], sum[kFewTileRows];
#pragma unroll
      for (int r = 0; r < kFewTileRows; ++r) {
        ref[r] = -INFINITY;
        sum[r] = 0.f;
      }
      const int n = it.kt1 - it.kt0;
      for (int i = 0; i < n; ++i, ++c) {
        const int u0 = (it.kt0 + i) * kFewKeys, key = u0 + tid;
        ok = ok && wait_bounded(s_full + (c & 1), (c >> 1) & 1, ctx.wait_ns);
        float x[kFewTileRows];                       // q . k, or -inf where the row does not see it
        bool grow = false;
        if (ok) {
          tc::fence_after();
          uint32_t s[kFewTileRows];
          tc::ld32(tmem + lanes + C::COL_S + (c & 1) * 32, s);
          tc::wait_ld();
          tc::after_wait(s);
          // whether every row sees the whole tile
          const bool all = M == Mask::kTree
              ? u0 + kFewKeys <= it.past
              : u0 + kFewKeys - 1 <= it.pos0 &&
                    (it.pos0 + it.n_tok - 1 - u0 < a.window || u0 + kFewKeys <= a.sinks);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q >= chunks) {
#pragma unroll
              for (int e = 8 * q; e < 8 * q + 8; ++e) x[e] = -INFINITY;
              continue;
            }
#pragma unroll
            for (int e = 8 * q; e < 8 * q + 8; ++e) {
              x[e] = __uint_as_float(s[e]);
              if (!all) {
                const int pos = it.pos0 + (e >> log_g);
                bool sees = key <= pos;
                if constexpr (M == Mask::kWindow) {
                  sees = sees && (pos - key < a.window || key < a.sinks);
                } else {
                  const int node = key - it.past;
                  if (sees && node >= 0)
                    sees = line[e * 32 + ((node >> 5) ^ e)] >> (node & 31) & 1u;
                }
                if (!sees) x[e] = -INFINITY;
              }
              if (e >= rows) x[e] = -INFINITY;               // nobody's row
              grow |= fmaf(x[e], a.scale_log2, -ref[e]) > kFewLazy;   // NaN for no key so far
            }
          }
        }
        if (group_any(grow || !ok)) {
          if (group_any(!ok)) {
            ok = false;
            break;
          }
          float v[kFewTileRows];
#pragma unroll
          for (int r = 0; r < kFewTileRows; ++r) v[r] = x[r];
          red[warp * 32 + lane] = join_lanes(v, [](float p, float q) { return fmaxf(p, q); });
          group_sync();
          if (warp == 0) {
            const float top = a.scale_log2 * fmaxf(fmaxf(red[lane], red[32 + lane]),
                                                   fmaxf(red[64 + lane], red[96 + lane]));
            const float old = ref_sh[lane], now = top > old + kFewLazy ? top : old;
            ref_sh[lane] = now;
            factor_sh[lane] = now == -INFINITY ? 1.f : exp2f(old - now);
          }
          group_sync();
          // the product of the tile before is done: O holds what is to be scaled
          if (i > 0) ok = wait_bounded(pv_done + ((c - 1) & 1), ((c - 1) >> 1) & 1, ctx.wait_ns);
          float factor[kFewTileRows];
#pragma unroll
          for (int r = 0; r < kFewTileRows; ++r) {
            ref[r] = ref_sh[r];
            factor[r] = factor_sh[r];
            sum[r] *= factor[r];
          }
          if (ok && i > 0) {
            tc::fence_after();
#pragma unroll 1
            for (int part = 0; part < 64; part += 32) {
              uint32_t o[32];
              tc::ld32(to + part, o);
              tc::wait_ld();
              tc::after_wait(o);
#pragma unroll
              for (int r = 0; r < 32; ++r)
                o[r] = __float_as_uint(__uint_as_float(o[r]) * factor[r]);
              tc::st32(to + part, o);
            }
            tc::wait_st();
          }
        }
        // the product that read this buffer last is done
        if (c >= 2 && ok)
          ok = wait_bounded(pv_done + (c & 1), ((c >> 1) - 1) & 1, ctx.wait_ns);
        if (!ok) continue;
        uint8_t* p_row = sm + C::OFF_P + (c & 1) * C::P_BYTES + tid * 128;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q >= chunks) break;
          uint32_t high[4], low[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 8 * q + 2 * e;
            const float m0 = ref[r] == -INFINITY ? 0.f : ref[r];
            const float m1 = ref[r + 1] == -INFINITY ? 0.f : ref[r + 1];
            const float p0 = tc::exp2_approx(fmaf(x[r], a.scale_log2, -m0));
            const float p1 = tc::exp2_approx(fmaf(x[r + 1], a.scale_log2, -m1));
            sum[r] += p0;
            sum[r + 1] += p1;
            high[e] = tc::pack_bf16(p0, p1);
            low[e] = tc::pack_bf16(p0 - bf16_lo(high[e]), p1 - bf16_hi(high[e]));
          }
          *reinterpret_cast<uint4*>(p_row + ((q ^ (tid & 7)) << 4)) =
              make_uint4(high[0], high[1], high[2], high[3]);
          *reinterpret_cast<uint4*>(p_row + (((4 + q) ^ (tid & 7)) << 4)) =
              make_uint4(low[0], low[1], low[2], low[3]);
        }
        tc::fence_async_smem();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) arrive(p_full + (c & 1));
      }
      // ---- output: lane d of O^T is column d of the rows
      ok = ok && wait_bounded(pv_done + ((c - 1) & 1), ((c - 1) >> 1) & 1, ctx.wait_ns);
      red[warp * 32 + lane] = join_lanes(sum, [](float p, float q) { return p + q; });
      if (group_any(!ok)) {
        ok = false;
        break;
      }
      tc::fence_after();
      const bool whole = it.part < 0;
      if (warp == 0) {
        const float l = red[lane] + red[32 + lane] + red[64 + lane] + red[96 + lane];
        const float m = ref_sh[lane];
        sum_sh[lane] = whole ? 1.f / l : 1.f;      // every row of a whole item sees itself: l > 0
        if (lane < rows) {
          if (whole && a.lse != nullptr)
            a.lse[(int64_t)(it.row0 + (lane >> log_g)) * a.Hq + it.g * a.G + (lane & (a.G - 1))] =
                (m + log2f(l)) * kLn2;
          if (!whole) {                            // m = -inf: the part has no key for this row
            float* ml = a.part_ml + 2 * ((int64_t)it.part * a.part_rows + lane);
            ml[0] = m;
            ml[1] = l;
          }
        }
      }
      float o[kFewTileRows];
      {
        uint32_t part[32];
        tc::ld32(to, part);
        tc::wait_ld();
        tc::after_wait(part);
#pragma unroll
        for (int r = 0; r < 32; ++r) o[r] = __uint_as_float(part[r]);
        tc::ld32(to + 32, part);
        tc::wait_ld();
        tc::after_wait(part);
#pragma unroll
        for (int r = 0; r < 32; ++r) o[r] += __uint_as_float(part[r]);
      }
      tc::fence_before();
      // The second half of the keys at D = 64, handed over where P was.
      float* other = reinterpret_cast<float*>(sm + C::OFF_P);   // [32][64]
      if (D == 64 && tid >= 64) {
#pragma unroll
        for (int r = 0; r < 32; ++r) other[r * 64 + tid - 64] = o[r];
      }
      group_sync();
      if (tid < D) {
#pragma unroll
        for (int r = 0; r < 32; ++r) {
          if (r >= rows) break;
          float y = o[r];
          if (D == 64) y += other[r * 64 + tid];
          y *= sum_sh[r];
          if (whole) {
            const int64_t row = (int64_t)(it.row0 + (r >> log_g)) * a.Hq + it.g * a.G +
                                (r & (a.G - 1));
            uint16_t bits;
            asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(bits) : "f"(y));
            static_cast<uint16_t*>(a.out)[row * D + tid] = bits;
          } else {
            a.part_acc[((int64_t)it.part * a.part_rows + r) * D + tid] = y;
          }
        }
      }
      __syncwarp();
      if (lane == 0) arrive(o_free + (j & 1));
      item_done(j);
    }
    if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
  } else if (warp == kFewMma) {
    // ---- products: tile c's values after tile c + 1's scores
    bool ok = true;
    int c = 0, slot = 0;
    auto wait = [&](uint64_t* x, int parity) {
      ok = ok && wait_bounded(x, parity, ctx.wait_ns);
    };
    const uint64_t k_desc = tc::smem_desc(uniform(smem_addr(sm + C::OFF_RING)), 16);
    const uint64_t v_desc =
        tc::smem_desc(uniform(smem_addr(sm + C::OFF_RING)), D == 128 ? 16384 : 8192);
    const uint64_t q_desc = tc::smem_desc(uniform(smem_addr(sm + C::OFF_Q)), 16);
    const uint64_t p_desc = tc::smem_desc(uniform(smem_addr(sm + C::OFF_P)), 8192);
    // Scores of tile number `tile` of the block with item j's rows.
    auto scores = [&](int tile, int j, bool first, bool last) {
      if (first) wait(q_full + (j & 1), (j >> 1) & 1);
      const int stage = slot % C::STAGES;
      wait(full + stage, (slot / C::STAGES) & 1);
      ++slot;
      if (!ok) return;
      tc::fence_after();
      if (tc::elect()) {
        constexpr uint32_t id = tc::idesc(kFewTileRows, false);
        const uint64_t kd = k_desc + (uint64_t)(stage * (C::TILE_BYTES >> 4));
        const uint64_t qd = q_desc + (uint64_t)((j & 1) * (C::Q_BYTES >> 4));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(tmem + C::COL_S + (tile & 1) * 32,
                     kd + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                     qd + (((k >> 2) * kFewTileRows * 128 + (k & 3) * 32) >> 4), id, k > 0);
        tc::commit(s_full + (tile & 1));
        if (last) tc::commit(q_free + (j & 1));
        tc::commit(empty + stage);
      }
      __syncwarp();
    };
    auto tiles_of = [&](int j) {
      const Item& it = items[j % kFewItems];
      return uniform(it.kt1 - it.kt0);
    };
    ok = item_ready(0);
    int n = ok ? tiles_of(0) : 0, next = 0;
    const bool any = n > 0;
    if (any) scores(0, 0, true, n == 1);
#pragma unroll 1
    for (int j = 0; ok && n > 0; ++j) {
      // keys there are from the item's first tile on: V rows behind them become zeros
      const int keys = uniform(items[j % kFewItems].end - items[j % kFewItems].kt0 * kFewKeys);
#pragma unroll 1
      for (int i = 0; ok && i < n; ++i, ++c) {
        if (i + 1 < n) {
          scores(c + 1, j, false, i + 2 == n);
        } else {
          ok = item_ready(j + 1);
          if (!ok) break;
          next = tiles_of(j + 1);
          if (next > 0) scores(c + 1, j + 1, true, next == 1);
        }
        wait(p_full + (c & 1), (c >> 1) & 1);
        const int stage = slot % C::STAGES;
        wait(full + stage, (slot / C::STAGES) & 1);
        ++slot;
        if (i == 0 && j >= 2) wait(o_free + (j & 1), ((j >> 1) - 1) & 1);
        if (!ok) break;
        const int valid = keys - i * kFewKeys;
        if (valid < kFewKeys) {
          uint8_t* tile = sm + C::OFF_RING + stage * C::TILE_BYTES;
          for (int x = valid * 8 + lane; x < kFewKeys * 8; x += 32)
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h)
              *reinterpret_cast<uint4*>(tile + h * 16384 + x * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_async_smem();
          __syncwarp();
        }
        tc::fence_after();
        if (tc::elect()) {
          constexpr uint32_t id = tc::idesc(C::O_COLS, true, true);
          const uint64_t vd = v_desc + (uint64_t)(stage * (C::TILE_BYTES >> 4));
          const uint64_t pd = p_desc + (uint64_t)((c & 1) * (C::P_BYTES >> 4));
#pragma unroll
          for (int k = 0; k < (D == 128 ? 8 : 4); ++k)
            tc::mma_ss(tmem + C::COL_O + (j & 1) * C::O_COLS, vd + k * (2048 >> 4),
                       pd + k * (2048 >> 4), id, i > 0 || k > 0);
          tc::commit(empty + stage);
          tc::commit(pv_done + (c & 1));
        }
        __syncwarp();
      }
      item_done(j);
      n = next;
      next = 0;
    }
    // No product may be in flight when the TMEM goes.
    __syncwarp();
    if (any) {
      if (tc::elect()) tc::commit(drained);
      __syncwarp();
      (void)wait_bounded(drained, 0, kDrainNs);
    }
    if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
  } else if (warp == kFewLoad) {
    // ---- loads: one page half (64 columns) per lane; K of a tile, then V of the tile before
    const int PS = d.page_size, per_tile = kFewKeys / PS;
    const int copies = per_tile * C::HALVES;
    const int page = lane % per_tile, half = lane / per_tile;
    const uint32_t box_bytes = (uint32_t)PS * 128;
    const uint32_t dst = smem_addr(sm + C::OFF_RING) + half * 16384 + page * box_bytes;
    bool ok = true, behind = false;
    int used = 0, before = -1;                       // slots filled; the last K tile's pool rows
    auto load = [&](const CUtensorMap* map, int row) {
      const int stage = used % C::STAGES;
      if (used >= C::STAGES)
        ok = ok && wait_bounded(empty + stage, (used / C::STAGES - 1) & 1, ctx.wait_ns);
      if (!ok) return;
      const int boxes = __popc(__ballot_sync(0xffffffffu, row >= 0));
      if (lane == 0) mbar_arrive_expect_tx(full + stage, boxes * box_bytes);
      __syncwarp();
      if (row >= 0) tma_page(dst + stage * C::TILE_BYTES, map, half * 64, row, full + stage);
      ++used;
    };
#pragma unroll 1
    for (int j = 0;; ++j) {
      ok = ok && item_ready(j);
      if (!ok) break;
      const Item it = items[j % kFewItems];
      if (it.kt0 >= it.kt1) break;
      item_done(j);
      const int32_t* table = d.page_table + (int64_t)it.b * d.page_table_stride;
      const int pages = (int)(((int64_t)it.end + PS - 1) / PS);
      // the table's entries 32 at a time, one to a lane, and those ahead
      auto entries = [&](int chunk) {
        int p = chunk * 32 + lane;
        int P = -1;
        if (p < pages) {
          if constexpr (M == Mask::kWindow) p += p < a.sink_pages ? 0 : it.skip;
          P = __ldg(table + p);
          if (P < 0 || P >= d.num_phys_pages) {
            flag(ctx, KV_DEVERR_BAD_PAGE);
            P = -1;
          }
        }
        return P;
      };
      int chunk = it.kt0 * per_tile / 32;
      int e1 = entries(chunk), e2 = entries(chunk + 1);
#pragma unroll 1
      for (int t = it.kt0; ok && t < it.kt1; ++t) {
        const int first = t * per_tile;
        if (first / 32 > chunk) {
          e1 = e2;
          e2 = entries(++chunk + 1);
        }
        const int P = __shfl_sync(0xffffffffu, e1, (first + page) & 31);
        const int row = P >= 0 && lane < copies ? (P * d.num_kv_heads + it.g) * PS : -1;
        load(&map_k, row);
        if (behind) load(&map_v, before);
        before = row;
        behind = true;
      }
    }
    if (behind) load(&map_v, before);
    if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
    // no copy may be in flight when the block's shared memory goes
    for (int s = max(0, used - C::STAGES); s < used; ++s)
      (void)wait_bounded(full + s % C::STAGES, (s / C::STAGES) & 1, kDrainNs);
  } else {
    // ---- the block's items, one ahead of their rows, and after the last an item without key
    // tiles. Waits for an item's end are for work and count the limit once per key tile.
    if (alone) at = find_place_warp<Shape>(ctx, d, pr, a, blockIdx.x);
    const bool none = at.total == 0;                 // less than a unit of the line: no item either
    ItemWalk<Shape> walk(d, pr, a, ctx, at.lo, none ? at.lo : at.hi, none ? 0 : at.b,
                         none ? 0 : at.before, blockIdx.x);
    ItemWalk<Shape> start = walk;                    // for the note that a merge reads
    bool ok = true;
    int loaded = 0;
    Item it, next{};
    int open[kFewItems] = {};                        // key tiles of the last items published
    auto patience = [&]() {
      unsigned long long tiles = 1;
#pragma unroll
      for (int i = 0; i < kFewItems; ++i) tiles += open[i];
      return ctx.wait_ns <= ~0ull / tiles ? ctx.wait_ns * tiles : ~0ull;
    };
    // One place in the code publishes, after the rows of the item before are on their way.
#pragma unroll 1
    for (int j = -1;; ++j) {
      it = next;
      if (j >= 0) {
        if (j >= 2) ok = wait_bounded(q_free + (j & 1), ((j >> 1) - 1) & 1, patience());
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full + (j & 1), C::Q_BYTES);
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h)
            tma_rows(smem_addr(sm + C::OFF_Q) + (j & 1) * C::Q_BYTES + h * kFewTileRows * 128,
                     &map_q, 64 * h, it.g * a.G, it.row0, q_full + (j & 1));
        }
        __syncwarp();
        ++loaded;
      }
      if (none || !walk.next(&next)) next.kt0 = next.kt1 = 0;
      if (j + 1 >= kFewItems)
        ok = wait_bounded(item_free + (j + 1) % kFewItems, ((j + 1) / kFewItems - 1) & 1,
                          patience());
      if (!ok) break;
#pragma unroll
      for (int i = 0; i + 1 < kFewItems; ++i) open[i] = open[i + 1];
      open[kFewItems - 1] = next.kt1 - next.kt0;
      if (lane == 0) {
        items[(j + 1) % kFewItems] = next;
        arrive(item_full + (j + 1) % kFewItems);
      }
      __syncwarp();
      if (next.kt0 >= next.kt1) break;
    }
    if (lane == 0 && a.notes != nullptr)
      a.notes[blockIdx.x] = none ? BorderNote{0, 0, 0, 0, 0, 0} : start.border();
    if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
    for (int j = max(0, loaded - 2); j < loaded; ++j)
      (void)wait_bounded(q_full + (j & 1), (j >> 1) & 1, kDrainNs);
  }
  __syncwarp();
  __syncthreads();
  tc::fence_after();
  if (warp == kFewMma) tc::dealloc(tmem, C::TMEM_COLS);
}

template <int D, Mask M>
cudaError_t launch_few_t(const kv_cache_desc& d, const PackedRows& pr, const PrefillArgs& a,
                         DevCtx ctx, cudaStream_t s) {
  using C = FewCfg<D>;
  CUtensorMap mk, mv, mq;
  if (!pool_tensor_map(&mk, d.k_pool, d) || !pool_tensor_map(&mv, d.v_pool, d) ||
      !rows_tensor_map(&mq, a.q, a.q_stride, a.Hq, D, pr.total, a.G, kFewTileRows / a.G))
    return cudaErrorInvalidValue;
  auto kern = prefill_few_kernel<D, M>;
  // set once per device; setting it twice from two threads is harmless
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(1, std::memory_order_release);
  }
  return launch_pdl(kern, dim3(a.NC), dim3(kFewThreads), C::SMEM, s, mk, mv, mq, d, pr, a, ctx);
}

}  // namespace

template <Mask M>
cudaError_t launch_prefill_few(const kv_cache_desc& d, const PackedRows& pr,
                               const PrefillArgs& a, DevCtx ctx, cudaStream_t s) {
  return d.head_dim == 128 ? launch_few_t<128, M>(d, pr, a, ctx, s)
                           : launch_few_t<64, M>(d, pr, a, ctx, s);
}

}  // namespace skv
