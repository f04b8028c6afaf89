// Causal prompt attention for bf16 caches on the tensor cores.
//
// A block takes 256 rows (256 / G tokens of one KV head) as two tiles of 128, one per softmax
// warpgroup, and walks their keys 128 at a time:
//   S = Q K^T    128 x 128 x D,   Q and K from shared memory, S in TMEM
//   P = 2^(scale_log2 S - m)      one thread per row: its warpgroup reads S from TMEM, keeps
//                                 m and l in registers and writes P back over S as bf16
//   O += P V     128 x D x 128,   P from TMEM, V from shared memory, O in TMEM
// One warp issues the products, the two warpgroups' in turn:
//   ... P0 V(j), Q0 K(j+1) | P1 V(j), Q1 K(j+1) | P0 V(j+1), Q0 K(j+2) | ...
// so that one warpgroup's softmax runs under the other's products. P is handed over in two
// halves, so that half of P V runs under the softmax of the other half. A second warp waits for
// what the products need beside P (their K and V tiles, rows, O), so that the issuing warp waits
// once per half. One warp feeds K and V tiles through a ring by TMA, page by page (a page of one
// KV head is PS dense rows of the pool); one works out the items and loads their rows. Whole
// rows of the output leave by TMA.
//
// An item with at most 128 rows (single tokens, drafts, a prompt's tail) gives both warpgroups
// the same rows and alternating key tiles instead, and joins their (m, l, O) at the end: the
// same pipeline, with the softmax still under the other warpgroup's products.
//
// A block walks its share of the batch's items (prefill.cuh) without stopping between them:
// loads and products run ahead into the next item while a warpgroup writes its output.
//
// What bounds it. Long prompts: a tile's round trip. The two tiles of a key tile cost 2048
// cycles of products at D = 128 and take about 2600; a warpgroup's own chain (scores, about 1400
// cycles of softmax, half of P V) is as long, so neither side waits for the other alone. With
// pages of 16 tokens a K or V tile is sixteen copies of 2 KB, whose issue then bounds the rate:
// a prompt of 8192 tokens of 32/8 heads takes 0.41 ms with pages of 16, 0.33 with 32, 0.35 with
// 64. Short items: instruction fetches, as what lies between items is long code that few warps
// run (32 prompts of 400 tokens: a stall of 4.2 per instruction issued, 0.2 on a long prompt);
// hence the rolled loops there, which took them from 127 us to 111.
// Measured, D = 128: a prompt of 16384 tokens, 64/8 heads, pages of 64: 2.69 ms, 1.64 PFLOP/s,
// 84% of the measured library product's rate; 8192 tokens, 32/8 heads, pages of 16: 0.42 ms,
// 67%. At D = 64 the products are half as long and the chain is not: 465 TFLOP/s over prompts of
// 1 to 4096 tokens of 16 heads without sharing. A single token over 32768: 37 us, of which the
// keys and values stream in 18 at the measured copy rate; the start of the blocks (8), their
// last output (4) and the merge (5) remain. Single tokens of 32 sequences over 1K to 4K: 73 us,
// 68% of the copy rate over the call, and over 16K 360 us, 88%.
//
// Other masks (M). A window's items count their keys without the skipped pages (prefill.cuh): the
// pipeline is the causal one, the loading warp adds the skipped pages to the table's index, and a
// tile on either border of the window gets its mask from three compares to 32 columns. A tree's
// rows follow their parents to bits of their ancestors, kept in the warp's output buffer while
// the tiles run. With these masks the loading warp does not wait for a sequence's last V tile:
// the warp that is ahead of the products zeroes what is behind the end, and items inside a
// sequence need no zeros at all, as the tokens after them are cached and finite. Measured, D =
// 128, 32/8 heads, pages of 16, a prompt of 8192 tokens in windows of 128, 1024 and 8192 tokens:
// 65, 152 and 408 us (causal 407); 16384 tokens of 64/8 heads in pages of 64, window 4096: 1.18
// to 1.32 ms, up to 1.65 PFLOP/s. Short windows: an item's start and end, 9000 cycles (the output
// alone 5000, half of it fetching its instructions), against 1300 to 2600 a tile. Trees of 26
// nodes of 8 heads to a group over 16 sequences of 700 to 9700 tokens: 84 us, 61% of the copy
// rate over the call.
//
// Measured and dropped, at 16384 tokens unless said: one S for both warpgroups and P beside it,
// scores a tile ahead (the hand-over of S bounds it); two threads per row, 640 threads (3.5 ms);
// the maximum beside the first half's exponentials (3.07 ms); P handed over at 96 of 128 keys,
// or at 64 with the wait for its store put off by 16 or 32 keys (2.69 to 2.71 ms against 2.70,
// D = 64 slower by up to 4%); polling without suspension in the issuing warp (8192 tokens 0.60
// ms against 0.42); at D = 64 P beside each warpgroup's own S and scores a tile ahead (145 us
// against 109: with one more hand-over per tile the issuing warp, 1600 cycles a tile among the
// softmax's instructions, is the bound); the copies of a tile's pages issued by one thread, page
// after page (0.55 ms for 8192 tokens) or written out (0.38 against 0.41, but pages of 32 and 64
// and ragged batches 10 to 18% slower); both products' warpgroups in one loop (short items 9%
// faster, long prompts 4% slower); V tiles zeroed behind the sequence's end only (8192 tokens 1%
// slower).
//
// The running maximum is lazy: O and l are rescaled only when a row's maximum grows by more
// than 2^8, so that almost no tile pays for it. O / l does not depend on the reference m, as each
// term of both carries the same factor 2^-m; any m within 8 of the maximum keeps P below 2^8, and
// every sum is float32.
// Rows see keys up to their own position; the tiles on that border are masked. Keys of slots
// past the item's last key never reach a sum: their scores are masked, and their rows of the
// V tile are zeroed in shared memory (a zero probability times a NaN would not vanish).
//
// Rounding: P is rounded to bf16 for the second product (relative 2^-8 each, independent), as
// the tensor core takes bf16 operands; its sum l is taken over the unrounded values. Batches of
// few rows (FEW: at most 32 to a sequence) multiply V by P in two parts, its rounding and the
// rounding of what that leaves, 2^-17 together: with one warp of each warpgroup at work the
// tensor core idles, and the second part fits where S was, beside the first. Up to 32 rows that
// costs under 1% (16 sequences over 4133 tokens, 4 to 32 rows: 62.5 to 62.8 us against 62.0 to
// 62.3; one token over 32768: 37.2 against 36.4), from 64 rows on 8% and more (72.9 against 67.1;
// 128 rows 76.9 against 71.9). The mean is what the host knows: 31 single tokens and a chunk of
// 128, four heads to a group, have 20 rows to a sequence and pay 9% (125.7 us against 115.3).
// It is an instance of its own, whose tiles have 128 rows: with code for both in one kernel long
// prompts took 3 to 13% more, ragged batches 12 to 17% and heads of 64 35 to 55%, in registers
// and instruction fetches.
#pragma once

#include <atomic>
#include <type_traits>

#include "prefill_tma.cuh"

namespace skv {
namespace {

constexpr int kThreads = 384;          // two softmax warpgroups, then products and loads
constexpr int kMmaWarp = 8, kLoadWarp = 9, kItemWarp = 10, kReadyWarp = 11;
constexpr int kItems = 4;              // items known ahead
constexpr int kKeys = MmaShape::keys;
constexpr int kTmemCols = 512;
constexpr int kRegsSoftmax = 216, kRegsOther = 72;     // (2 * 216 + 72) * 128 = 384 * 168
constexpr int kFewRows = 32;           // mean rows per sequence up to which P has two parts
constexpr float kLazy = 8.f;           // log2 of the growth that forces a rescale

template <int D> struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = HALVES * 128 * 128;         // 128 rows of D bf16
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr size_t OFF_Q = 0;                            // from a 1024-aligned base
  static constexpr size_t OFF_RING = 2 * TILE_BYTES;
  static constexpr size_t OFF_OUT = OFF_RING + (size_t)STAGES * TILE_BYTES;   // 4 KB a warp
  static constexpr size_t OFF_BAR = OFF_OUT + 8 * 4096;
  static constexpr int BARS = 2 * STAGES + 17 + 2 * kItems;
  static constexpr size_t OFF_MISC = OFF_BAR + 8 * BARS;        // TMEM base, items, [2][128] (m, l)
  static constexpr size_t OFF_ITEMS = OFF_MISC + 8;
  static constexpr size_t OFF_ML = OFF_ITEMS + kItems * 48;
  static_assert(sizeof(MaskedItem) <= 48, "items");
  static constexpr size_t SMEM = OFF_ML + 1024 + 1024;          // + alignment slack
  static_assert(SMEM <= 227 * 1024 - sizeof(LineScratch), "shared memory");
  static constexpr int COL_O = 0, COL_S = 2 * D;                // TMEM: two O, two S with P over it
};

// An item's plan: which key tiles each warpgroup takes and where they lie in the ring, counted
// from the item's first slot.
// AHEAD (a window at D = 64, whose ring holds four tiles of keys and values): where the second row
// tile's window begins behind the first key tile, the second warpgroup begins with the second one
// and stays a tile ahead. Both then have as many tiles, where the first's rows end a tile earlier,
// and the next item's scores can follow at once.
template <bool AHEAD> struct Plan {
  bool wide;      // two row tiles; else one, with the key tiles dealt out in turn
  int n;          // key tiles of the item (or of the block's part of it)
  int n0, n1;     // key tiles of each warpgroup
  int ahead;      // key tiles that the second warpgroup leaves out at the start: 0 or 1

  __device__ __forceinline__ Plan(const PrefillItem& it, const PrefillArgs& a, bool few) {
    const int log_g = a.log_g;
    wide = !few && (it.n_tok << log_g) > 128;
    n = it.kt1 - it.kt0;
    ahead = 0;
    if (wide) {
      // the first tile's rows end earlier: its last keys may lie a tile before the item's
      n0 = max(0, min(n, (it.pos0 + (127 >> log_g)) / kKeys + 1 - it.kt0));
      n1 = n;
      if (AHEAD) {
        ahead = a.sinks <= it.kt0 * kKeys &&
                it.pos0 + (128 >> log_g) - a.window + 1 >= (it.kt0 + 1) * kKeys;
        n1 -= ahead;
      }
    } else {
      n0 = (n + 1) / 2;
      n1 = n / 2;
    }
  }
  __device__ __forceinline__ int tiles(int w) const { return w == 0 ? n0 : n1; }
  __device__ __forceinline__ int tile(int w, int i) const {
    return wide ? i + (AHEAD && w == 1 ? ahead : 0) : 2 * i + w;
  }
  // Whether warpgroup w is the last to read tile t's keys, or values.
  __device__ __forceinline__ bool last_reader(int w, int t) const {
    if (AHEAD && wide && ahead) return w == 0 || t >= n0;
    return !wide || w == 1;
  }
  // Ring slots in the order of first use: K0 V0 K1 V1 ..., or (dealt out) K0 K1 V0 K2 V1 K3 ...
  __device__ __forceinline__ int k_slot(int t) const {
    return wide ? 2 * t : t < 2 ? t : 2 * t - 1;
  }
  __device__ __forceinline__ int v_slot(int t) const {
    return wide || t == n - 1 ? 2 * t + 1 : 2 * t + 2;
  }
};

// The reverse, for 32 rows of the output: from shared memory, one group of copies per call.
__device__ __forceinline__ void tma_store_rows(const CUtensorMap* map, const void* src, int x,
                                               int head, int token) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
      "cp.async.bulk.commit_group;"
      ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(token), "r"(smem_addr(src))
      : "memory");
}

// The ancestors of a drafted row, itself too, as bits by their index among the sequence's rows:
// 32 words of the row's lane in its warp's output buffer, which is free while the tiles run. The
// words are turned by the lane, so that a warp's lanes hit all banks with the same word of each.
struct Ancestors {
  uint32_t* words;
  int last;                                      // the row's own word: those after it are zero

  __device__ __forceinline__ uint32_t& at(int k) const {
    return words[k ^ (threadIdx.x & 31)];
  }
  // Row `i` of the sequence whose parents are `up`: follows its line to the first node.
  __device__ __forceinline__ void walk(const DevCtx& ctx, const int32_t* up, int i) {
    last = i >> 5;
    for (int k = 0; k <= last; ++k) {
      prefetch_l1(up + 32 * k);
      at(k) = 0;
    }
    for (int v = i; v >= 0;) {
      at(v >> 5) |= 1u << (v & 31);
      const int next = __ldg(up + v);
      if (next >= v || next < -1) {
        flag(ctx, KV_DEVERR_BAD_SEL);
        break;
      }
      v = next;
    }
  }
  // Bits of the 32 tokens from row index `first` on; tokens before the rows are seen by all.
  __device__ __forceinline__ uint32_t seen(int first) const {
    const int k = first >> 5;
    const uint32_t low = k < 0 ? ~0u : k > last ? 0u : at(k);
    const uint32_t high = k + 1 < 0 ? ~0u : k + 1 > last ? 0u : at(k + 1);
    return __funnelshift_r(low, high, first & 31);
  }
};

// The lowest n bits.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}

template <int D, bool FEW, Mask M>
__global__ void __launch_bounds__(kThreads, 1)
prefill_mma_kernel(const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_out,
                   const __grid_constant__ kv_cache_desc d,
                   const __grid_constant__ PackedRows pr, const __grid_constant__ PrefillArgs a,
                   const __grid_constant__ DevCtx ctx) {
  using C = Cfg<D>;
  using Shape = typename std::conditional<FEW, FewShape, MmaShape>::type::template With<M>;
  using Item = ItemOf<Shape>;
  using Plan = skv::Plan<M == Mask::kWindow && C::STAGES >= 8>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ LineScratch scratch;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~(uintptr_t)1023);
  uint8_t* ring = sm + C::OFF_RING;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint64_t* full = bar;                          // [STAGES] a K or V tile has landed
  uint64_t* empty = bar + C::STAGES;             // [STAGES] its last product is done
  uint64_t* s_full = bar + 2 * C::STAGES;        // [2] S of a warpgroup is in TMEM
  uint64_t* p_half = s_full + 2;                 // [2] P of its first 64 keys is there, O rescaled
  uint64_t* p_full = p_half + 2;                 // [2] all of its P is in TMEM
  uint64_t* o_done = p_full + 2;                 // [2] its last product of an item is done
  uint64_t* q_full = o_done + 2;                 // [2] its rows are in shared memory
  uint64_t* q_free = q_full + 2;                 // [2] its last scores of an item are done
  uint64_t* o_free = q_free + 2;                 // [2] its O has been read
  uint64_t* joined = o_free + 2;                 // the second warpgroup's (m, l) are written
  uint64_t* v_land = joined + 1;                 // the last V tile, before its tail is zeroed
  uint64_t* drained = v_land + 1;                // no product in flight
  uint64_t* item_full = drained + 1;             // [kItems] an item is in shared memory
  uint64_t* item_free = item_full + kItems;      // [kItems] every warp is done with it
  Item* items = reinterpret_cast<Item*>(sm + C::OFF_ITEMS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  float* box = reinterpret_cast<float*>(sm + C::OFF_ML);          // [2][128]: m, l
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int log_g = a.log_g;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full + w, 1);
      mbar_init(p_full + w, 5);                  // the softmax warps', and the ready warp's
      mbar_init(q_full + w, 1);
      mbar_init(q_free + w, 1);
      mbar_init(p_half + w, 5);
      mbar_init(o_done + w, 1);
      mbar_init(o_free + w, 4);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(item_full + i, 1);
      mbar_init(item_free + i, 11);              // eight softmax warps, products, loads, ready
    }
    mbar_init(joined, 4);
    mbar_init(v_land, 1);
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  pdl_trigger();
  pdl_wait();
  finish_empty<bf16_t, D>(ctx, d, pr, a);
  const LinePlace at = find_place<Shape>(ctx, d, pr, a, blockIdx.x, &scratch);
  const int64_t lo = at.lo, hi = at.hi;
  if (at.total == 0 || lo >= hi) {                 // nothing, or less than a unit of the line
    if (tid == 0 && a.notes != nullptr)
      a.notes[blockIdx.x] =
          at.total == 0 ? BorderNote{0, 0, 0, 0, 0, 0}
                        : ItemWalk<Shape>(d, pr, a, ctx, lo, hi, at.b, at.before, 0).border();
    return;
  }
  if (warp == kMmaWarp) tc::alloc(tmem_slot, kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  // Item number j of the block, for the warp that asks; the last one has no key tiles.
  auto item_ready = [&](int j) {
    return wait_bounded(item_full + j % kItems, (j / kItems) & 1, ctx.wait_ns);
  };
  auto item_done = [&](int j) {
    __syncwarp();
    if (lane == 0) arrive(item_free + j % kItems);
  };

  if (warp < 8) {
    tc::more_regs<kRegsSoftmax>();
    const int w = warp >> 2, r = tid & 127;                       // warpgroup, TMEM lane
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // TMEM lane 32 * (warp % 4)
    const uint32_t ts = tmem + lanes + C::COL_S + w * 128, to = tmem + lanes + C::COL_O + w * D;
    const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
    bool ok = true;
    int tiles_seen = 0, items_seen = 0, joins_seen = 0;           // for the barriers' phases

    for (int j = 0;; ++j) {
      ok = item_ready(j);
      if (!ok) break;
      // What the tiles need of the item; it is read again for the output (its registers are
      // short while a row's 128 scores are held).
      int n, row, seen, warp_seen, step;
      int left = 0;          // kWindow: sinks from the tile's first key on; kTree: earlier tokens
      Ancestors line;
      bool idle;
      {
        const Item it = items[j % kItems];
        if (it.kt0 >= it.kt1) break;
        const Plan plan(it, a, FEW);
        n = plan.tiles(w);
        row = plan.wide ? w * 128 + r : r;
        idle = row - lane >= it.n_tok << log_g;                   // no row in this warp
        // the last key that the row sees, and the warp's first row, from the first tile's first
        const int u0 = (it.kt0 + plan.tile(w, 0)) * kKeys;
        seen = it.pos0 + (row >> log_g) - u0;
        warp_seen = it.pos0 + ((row - lane) >> log_g) - u0;
        step = plan.wide ? kKeys : 2 * kKeys;
        if (M == Mask::kWindow) left = a.sinks - u0;
        if constexpr (M == Mask::kTree) {
          left = it.past - u0;
          // the copy that left from the warp's buffer has read it
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
          const int t0 = it.pos0 - it.past;                       // the item's first row
          line.words = reinterpret_cast<uint32_t*>(sm + C::OFF_OUT + warp * 4096) + lane * 32;
          line.last = -1;
          if (!idle && n > 0)
            line.walk(ctx, a.parents + it.row0 - t0, t0 + min(row >> log_g, it.n_tok - 1));
        }
      }
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n; ++i) {
        ok = wait_bounded(s_full + w, tiles_seen & 1, ctx.wait_ns);
        if (!ok) break;
        ++tiles_seen;
        tc::fence_after();
        uint32_t s[128];
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, ref2;
        if (!idle) {
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::ld32(ts + 32 * c, s + 32 * c);
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::after_wait(s + 32 * c);
          // every row of the warp sees the whole tile
          const bool all =
              M == Mask::kTree ? left >= kKeys
                               : warp_seen >= kKeys - 1 &&
                                     (M == Mask::kCausal || left >= kKeys ||
                                      warp_seen + (31 >> log_g) < a.window);
          if (!all) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t keep;
              if constexpr (M == Mask::kCausal) {
                if (warp_seen >= 32 * q + 31) continue;
                const int last = seen - 32 * q;
                keep = last >= 31 ? ~0u : last < 0 ? 0u : (2u << last) - 1u;
              } else if constexpr (M == Mask::kWindow) {
                const int upto = seen + 1 - 32 * q;
                keep = low_bits(upto) & (~low_bits(upto - a.window) | low_bits(left - 32 * q));
              } else {
                keep = line.seen(32 * q - left);
              }
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if ((keep >> c & 1u) == 0u) s[32 * q + c] = 0xff800000u;
            }
          }
          seen -= step;
          warp_seen -= step;
          if (M != Mask::kCausal) left -= step;
          float top[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            top[c] = __uint_as_float(s[32 * c]);
#pragma unroll
            for (int e = 1; e + 1 < 32; e += 2)
              top[c] = tc::max3(top[c], __uint_as_float(s[32 * c + e]),
                                __uint_as_float(s[32 * c + e + 1]));
            top[c] = fmaxf(top[c], __uint_as_float(s[32 * c + 31]));
          }
          const float now = tc::max3(fmaxf(top[0], top[1]), top[2], top[3]) * a.scale_log2;
          if (__any_sync(0xffffffffu, now > m + kLazy)) {
            // s_full follows the products before it: O is complete up to tile i - 1
            const float next = now > m + kLazy ? now : m;
            const float f = next == -INFINITY ? 1.f : exp2f(m - next);
            m = next;
            l *= f;
            if (i > 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tc::ld16(to + c, o);
                tc::wait_ld();
                tc::after_wait16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tc::st16(to + c, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;             // no key of this row yet
          ref2 = make_float2(-ref, -ref);
        }
        constexpr int STEP = FEW ? 16 : 32;
        uint32_t p[64 / 32 * STEP], low[STEP];
        auto exps = [&](int first) {                              // P of 64 keys from `first` on
#pragma unroll
          for (int c = first / 2; c < first / 2 + 32; c += STEP) {
            uint32_t* high = p + c % (64 / 32 * STEP);
#pragma unroll
            for (int e = 0; e < STEP; ++e) {
              const int k = 2 * (c + e);
              float2 x = make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1]));
              x = tc::fma2(x, scale2, ref2);
              x.x = tc::exp2_approx(x.x);
              x.y = tc::exp2_approx(x.y);
              sum[e & 1] = tc::add2(sum[e & 1], x);
              high[e] = tc::pack_bf16(x.x, x.y);
              if (FEW) low[e] = tc::pack_bf16(x.x - bf16_lo(high[e]), x.y - bf16_hi(high[e]));
            }
            if constexpr (FEW) {
              tc::st16(ts + c, high);
              tc::st16(ts + 64 + c, low);
            } else {
              tc::st32(ts + c, high);
            }
          }
        };
        auto hand_over = [&](uint64_t* to_whom) {
          if (!idle) tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) arrive(to_whom + w);
        };
        if (!idle) exps(0);
        hand_over(p_half);
        if (!idle) exps(64);
        hand_over(p_full);
        sum[0] = tc::add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
      }
      if (!ok) break;
      // ---- output
      const PrefillItem it = items[j % kItems];
      const Plan plan(it, a, FEW);
      const int rows = it.n_tok << log_g, warp_row = row - lane;
      const bool join = !plan.wide && plan.n1 > 0;
      if (n > 0) ok = wait_bounded(o_done + w, items_seen & 1, ctx.wait_ns);
      if (!ok) break;
      if (join && w == 1) {
        box[r] = m;
        box[128 + r] = l;
        __syncwarp();
        if (lane == 0) arrive(joined);
      }
      if (n > 0) ++items_seen;
      if (join && w == 0) {
        // the other warpgroup's last product: it has one for each of this one's joins
        ok = wait_bounded(joined, joins_seen & 1, ctx.wait_ns);
        if (!ok) break;
        ++joins_seen;
      }
      if (!idle && (plan.wide || w == 0)) {
        tc::fence_after();
        float f0 = 1.f, f1 = 0.f;
        if (join) {
          const float m1 = box[r];
          const float both = fmaxf(m, m1);
          f0 = m == -INFINITY ? 0.f : exp2f(m - both);
          f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - both);
          l = l * f0 + box[128 + r] * f1;
          m = both;
        }
        const bool mine = row < rows, whole = it.part < 0;
        const int64_t at_row = (int64_t)(it.row0 + (row >> log_g)) * a.Hq + it.g * a.G +
                               (row & (a.G - 1));
        const int64_t at_part = (int64_t)it.part * a.part_rows + row;
        if (whole) {                               // every row sees its own token: l > 0
          const float inv = 1.f / l;
          f0 *= inv;
          f1 *= inv;
        }
        // Through 4 KB of the warp's own shared memory, 128 bytes of each of its 32 rows at a
        // time, so that eight lanes write one row's 128 bytes: a lane per row would touch 32
        // lines with every store (6000 cycles an item; this way 1500).
        uint8_t* stage = sm + C::OFF_OUT + warp * 4096;
        auto columns = [&](int c, float* o) {      // 32 columns from c on, scaled and joined
          uint32_t raw[32];
          tc::ld32(to + c, raw);
          tc::wait_ld();
          tc::after_wait(raw);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(raw[e]) * f0;
          if (join) {
            tc::ld32(to + D + c, raw);
            tc::wait_ld();
            tc::after_wait(raw);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(raw[e]), f1, o[e]);
          }
        };
        // Whole rows of a full warp leave by TMA while the warp goes on.
        const bool by_tma = it.part < 0 && warp_row + 32 <= rows;
        auto put = [&](int chunk, uint32_t x, uint32_t y, uint32_t z, uint32_t u) {
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((chunk ^ (lane & 7)) << 4)) =
              make_uint4(x, y, z, u);
        };
        auto flush = [&](uint8_t* base, uint32_t row_bytes, bool packed) {
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int k = 4 * e + (lane >> 3), chunk = lane & 7, out_row = warp_row + k;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + k * 128 +
                                                            ((chunk ^ (k & 7)) << 4));
            const uint32_t index =
                packed ? (uint32_t)((out_row >> log_g) * a.Hq + (out_row & (a.G - 1))) : out_row;
            if (out_row < rows)
              *reinterpret_cast<uint4*>(base + (uint64_t)index * row_bytes + chunk * 16) = v;
          }
          __syncwarp();
        };
        if (n > 0) {
          uint8_t* out = whole ? reinterpret_cast<uint8_t*>(
              static_cast<uint16_t*>(a.out) + ((int64_t)it.row0 * a.Hq + it.g * a.G) * D)
                               : reinterpret_cast<uint8_t*>(
              a.part_acc + (int64_t)it.part * a.part_rows * D);
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();                            // the copy before has read the buffer
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            columns(c, o);
            if (!whole) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                put(e, __float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
                    __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3]));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                put((c >> 3 & 4) + e, tc::pack_bf16(o[8 * e], o[8 * e + 1]),
                    tc::pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                    tc::pack_bf16(o[8 * e + 4], o[8 * e + 5]),
                    tc::pack_bf16(o[8 * e + 6], o[8 * e + 7]));
              if ((c & 32) == 0) continue;         // 128 bytes of a row are 64 columns
            }
            if (!by_tma) {
              flush(whole ? out + (c - 32) * 2 : out + c * 4, whole ? D * 2 : D * 4, whole);
              continue;
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_rows(&map_out, stage, c - 32, it.g * a.G, it.row0 + (warp_row >> log_g));
              if (c + 32 < D) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            __syncwarp();
          }
        }
        if (mine && whole && a.lse != nullptr) a.lse[at_row] = (m + log2f(l)) * kLn2;
        if (mine && !whole) {                      // m = -inf: the part has no key for this row
          a.part_ml[2 * at_part] = m;
          a.part_ml[2 * at_part + 1] = l;
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) {
        if (plan.wide ? n > 0 : w == 0) arrive(o_free + w);
        if (join && w == 0) arrive(o_free + 1);
      }
      item_done(j);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
  } else {
    tc::fewer_regs<kRegsOther>();
    auto uniform_plan = [&](int j) {
      Plan plan(items[j % kItems], a, FEW);
      if (!FEW) plan.wide = uniform(plan.wide);
      plan.n = uniform(plan.n);
      plan.n0 = uniform(plan.n0);
      plan.n1 = uniform(plan.n1);
      plan.ahead = uniform(plan.ahead);
      return plan;
    };
    // The next item's first scores can be issued with the last of this one's products.
    auto runs_on = [](const Plan& plan, const Plan& next) {
      return plan.wide && plan.n0 == plan.n1 && next.wide && next.n0 > 0 && next.n1 > 0;
    };
    if (warp == kMmaWarp) {
      // ---- products. The time between two batches of them is lost to the tensor core, so this
      // warp waits for as little as it can: for P, whose barriers the ready warp joins.
      bool ok = true;
      int base = 0;                                  // ring slots of the items before
      int items0 = 0, items1 = 0, tiles0 = 0, tiles1 = 0;           // for the barriers' phases
      // The first try stands alone: inside the loop of the slow path it costs 4% of a long prompt.
      auto wait = [&](uint64_t* x, int parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(x, parity))) return;
        ok = wait_bounded(x, parity, ctx.wait_ns) && ok;
      };
      const uint64_t q_desc = tc::smem_desc(uniform(smem_addr(sm + C::OFF_Q)), 16);
      const uint64_t k_desc = tc::smem_desc(uniform(smem_addr(ring)), 16);
      const uint64_t v_desc = tc::smem_desc(uniform(smem_addr(ring)), 16384);
      // Scores of warpgroup w's tile in ring slot `slot`; `done`: w is its last reader; `last`:
      // of the item.
      auto scores = [&](int w, int slot, bool done, bool last) {
        const int stage = slot % C::STAGES;
        constexpr uint32_t id = tc::idesc(kKeys, false);
        const uint64_t qd = q_desc + (uint64_t)(w * (C::TILE_BYTES >> 4));
        const uint64_t kd = k_desc + (uint64_t)(stage * (C::TILE_BYTES >> 4));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int step = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
          tc::mma_ss(tmem + C::COL_S + w * 128, qd + step, kd + step, id, k > 0);
        }
        tc::commit(s_full + w);
        if (last) tc::commit(q_free + w);
        if (done) tc::commit(empty + stage);
      };
      constexpr int kUnroll = FEW ? 1 : 2;
      bool early = false;          // this item's first scores were issued with the last's end
      ok = item_ready(0);
      Plan plan = uniform_plan(0), next = plan;
      const bool any = ok && plan.n > 0;
#pragma unroll 1
      for (int j = 0; ok && plan.n > 0; ++j) {
        const int most = max(plan.n0, plan.n1);
        if (!early) {
#pragma unroll 1
          for (int w = 0; w < 2; ++w) {
            if (!ok || plan.tiles(w) == 0) continue;
            const int t = plan.tile(w, 0), slot = base + plan.k_slot(t);
            wait(q_full + w, (w == 0 ? items0 : items1) & 1);
            wait(full + slot % C::STAGES, (slot / C::STAGES) & 1);
            if (!ok) continue;
            tc::fence_after();
            if (tc::elect()) scores(w, slot, plan.last_reader(w, t), plan.tiles(w) == 1);
            __syncwarp();
          }
        }
        early = false;
#pragma unroll 1
        for (int i = 0; ok && i < most; ++i) {
          if (i == most - 1) {                         // what follows
            ok = item_ready(j + 1);
            if (!ok) break;
            next = uniform_plan(j + 1);
            early = runs_on(plan, next);
          }
          // written out for both warpgroups: as a loop it costs a long prompt 4%
#pragma unroll kUnroll
          for (int w = 0; w < 2; ++w) {
            if (!ok || i >= plan.tiles(w)) continue;
            const int t = plan.tile(w, i), slot = base + plan.v_slot(t);
            const int tiles = w == 0 ? tiles0++ : tiles1++;
            const bool more = i + 1 < plan.tiles(w), go_on = more || early;
            const int k_slot = more ? base + plan.k_slot(plan.tile(w, i + 1))
                                    : base + 2 * plan.n + next.k_slot(next.tile(w, 0));
            const bool done = plan.last_reader(w, t);
            const bool last = more ? i + 2 == plan.tiles(w) : next.tiles(w) == 1;
            constexpr uint32_t id = tc::idesc(D, true);
            const uint64_t vd = v_desc + (uint64_t)(slot % C::STAGES * (C::TILE_BYTES >> 4));
            auto values = [&](int h) {
#pragma unroll
              for (int k = 4 * h; k < 4 * h + 4; ++k)
                tc::mma_ts(tmem + C::COL_O + w * D, tmem + C::COL_S + w * 128 + k * 8,
                           vd + k * (2048 >> 4), id, i > 0 || k > 0);
              if constexpr (FEW) {
#pragma unroll
                for (int k = 4 * h; k < 4 * h + 4; ++k)          // what P's rounding left
                  tc::mma_ts(tmem + C::COL_O + w * D, tmem + C::COL_S + w * 128 + 64 + k * 8,
                             vd + k * (2048 >> 4), id, 1);
              }
            };
            wait(p_half + w, tiles & 1);
            if (!ok) continue;
            tc::fence_after();
            if (tc::elect()) values(0);
            __syncwarp();
            wait(p_full + w, tiles & 1);
            if (!ok) continue;
            tc::fence_after();
            if (tc::elect()) {
              values(1);
              if (!more) tc::commit(o_done + w);
              if (done) tc::commit(empty + slot % C::STAGES);
              if (go_on)
                scores(w, k_slot,
                       more ? plan.last_reader(w, plan.tile(w, i + 1))
                            : next.last_reader(w, next.tile(w, 0)), last);
            }
            __syncwarp();
          }
        }
        item_done(j);
        items0 += plan.n0 > 0;
        items1 += plan.n1 > 0;
        base += 2 * plan.n;
        plan = next;
      }
      // No product may be in flight when the TMEM goes: this warp may have ended well while a
      // softmax warp, which waits for the last ones, gave up.
      __syncwarp();
      if (any) {
        if (tc::elect()) tc::commit(drained);
        __syncwarp();
        (void)wait_bounded(drained, 0, kDrainNs);
      }
      if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
    } else if (warp == kReadyWarp) {
      // ---- what the products need beside P: this warp walks the same batches a little ahead,
      // waits for their V and K tiles, rows and O, and adds its arrival to the softmax warps'
      // at p_half and p_full.
      bool ok = true;
      int base = 0, items0 = 0, items1 = 0, tiles0 = 0, tiles1 = 0;
      auto wait = [&](uint64_t* x, int parity) {
        ok = wait_bounded(x, parity, ctx.wait_ns) && ok;
      };
      auto wait_slot = [&](int slot) {
        wait(full + slot % C::STAGES, (slot / C::STAGES) & 1);
      };
      auto say = [&](uint64_t* x) {
        __syncwarp();
        if (lane == 0) arrive(x);
      };
      ok = item_ready(0);
      Plan plan = uniform_plan(0), next = plan;
#pragma unroll 1
      for (int j = 0; ok && plan.n > 0; ++j) {
        const int most = max(plan.n0, plan.n1);
        bool early = false;
        int it_end = 0;                                // keys there are from the item's first tile on
        if constexpr (M != Mask::kCausal) {
          const Item& it = items[j % kItems];
          it_end = it.end - it.kt0 * kKeys;
        }
#pragma unroll 1
        for (int i = 0; ok && i < most; ++i) {
          if (i == most - 1) {
            ok = item_ready(j + 1);
            if (!ok) break;
            next = uniform_plan(j + 1);
            early = runs_on(plan, next);
          }
#pragma unroll 1
          for (int w = 0; w < 2; ++w) {
            if (!ok || i >= plan.tiles(w)) continue;
            const int tiles = w == 0 ? tiles0++ : tiles1++, before = w == 0 ? items0 : items1;
            const bool more = i + 1 < plan.tiles(w);
            // The tile's scores are there: so is every tile before, whose barriers' phases (of
            // two kinds) could otherwise be taken for those waited for here.
            wait(s_full + w, tiles & 1);
            const int v_slot = base + plan.v_slot(plan.tile(w, i));
            wait_slot(v_slot);
            if constexpr (M != Mask::kCausal) {
              // the V rows behind the sequence's end become zeros, before the first product reads them
              const int valid = it_end - plan.tile(w, i) * kKeys;
              // (by whoever comes to them first)
              if (ok && valid < kKeys &&
                  (!plan.wide || (plan.ahead ? w == 1 : w == 0 || i >= plan.n0))) {
                uint8_t* tile = ring + v_slot % C::STAGES * C::TILE_BYTES;
                for (int x = valid * 8 + lane; x < kKeys * 8; x += 32)
#pragma unroll
                  for (int h = 0; h < C::HALVES; ++h)
                    *reinterpret_cast<uint4*>(tile + h * 16384 + x * 16) = make_uint4(0, 0, 0, 0);
                tc::fence_async_smem();
              }
            }
            if (i == 0 && before > 0) wait(o_free + w, (before - 1) & 1);     // it has been read
            if (!ok) continue;
            say(p_half + w);
            if (more || early) {
              if (!more) wait(q_full + w, (before + 1) & 1);
              wait_slot(more ? base + plan.k_slot(plan.tile(w, i + 1))
                             : base + 2 * plan.n + next.k_slot(next.tile(w, 0)));
              if (!ok) continue;
            }
            say(p_full + w);
          }
        }
        item_done(j);
        items0 += plan.n0 > 0;
        items1 += plan.n1 > 0;
        base += 2 * plan.n;
        plan = next;
      }
      __syncwarp();
      if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
    } else if (warp == kLoadWarp) {
      // ---- loads: one page half (64 columns) per lane
      const int PS = d.page_size, per_tile = kKeys / PS;
      const int copies = per_tile * C::HALVES;
      const int page = lane % per_tile, half = lane / per_tile;
      const uint32_t box_bytes = (uint32_t)PS * 128;
      const uint32_t dst = smem_addr(ring) + half * 16384 + page * box_bytes;
      bool ok = true;
      int used = 0, tails = 0;                         // slots filled
      for (int j = 0;; ++j) {
        ok = ok && item_ready(j);
        if (!ok) break;
        const Item it = items[j % kItems];
        if (it.kt0 >= it.kt1) break;
        item_done(j);
        const Plan plan(it, a, FEW);
        const int32_t* table = d.page_table + (int64_t)it.b * d.page_table_stride;
        // Keys from here on are nobody's. (With another mask: the sequence's end, as all its tokens
        // are cached and finite; only the tile that ends the sequence then needs zeros.)
        int keys = it.pos0 + it.n_tok;
        if constexpr (M != Mask::kCausal) keys = it.end;
        const int pages = (int)(((int64_t)keys + PS - 1) / PS);
        // The table's entries 32 at a time, one to a lane: those of the tile being loaded, the
        // ones before (V tiles come up to two tiles after their K tile) and the ones ahead.
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
        int e0 = -1, e1 = entries(chunk), e2 = entries(chunk + 1);
        auto load = [&](bool values, int t) {
          if (!ok) return;
          const int first = (it.kt0 + t) * per_tile;
          if (first / 32 > chunk) {
            e0 = e1;
            e1 = e2;
            e2 = entries(++chunk + 1);
          }
          int P = __shfl_sync(0xffffffffu, first / 32 == chunk ? e1 : e0, (first + page) & 31);
          if (lane >= copies) P = -1;
          const int slot = used;
          const int stage = slot % C::STAGES;
          if (slot >= C::STAGES)
            ok = wait_bounded(empty + stage, (slot / C::STAGES - 1) & 1, ctx.wait_ns);
          if (!ok) return;
          // the item's last key lies inside this tile: the V rows after it become zeros
          // (with another mask: by the ready warp)
          const int valid = min(kKeys, keys - (it.kt0 + t) * kKeys);
          const bool tail = M == Mask::kCausal && values && valid < kKeys;
          uint64_t* land = tail ? v_land : full + stage;
          const int boxes = __popc(__ballot_sync(0xffffffffu, P >= 0));
          if (lane == 0) mbar_arrive_expect_tx(land, boxes * box_bytes);
          __syncwarp();
          if (P >= 0)
            tma_page(dst + stage * C::TILE_BYTES, values ? &map_v : &map_k, half * 64,
                     (P * d.num_kv_heads + it.g) * PS, land);
          ++used;
          if (!tail) return;
          ok = wait_bounded(v_land, tails & 1, ctx.wait_ns);
          // given up: what follows is for nobody, but the copy must not outlive the block
          if (!ok) (void)wait_bounded(v_land, tails & 1, kDrainNs);
          ++tails;
          uint8_t* tile = ring + stage * C::TILE_BYTES;
          for (int i = valid * 8 + lane; i < kKeys * 8; i += 32)
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h)
              *reinterpret_cast<uint4*>(tile + h * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) arrive(full + stage);
        };
        if (plan.wide) {
#pragma unroll 1
          for (int t = 0; t < plan.n; ++t) {
            load(false, t);
            load(true, t);
          }
        } else {
#pragma unroll 1
          for (int t = -2; t < plan.n; ++t) {
            if (t >= 0) load(true, t);
            if (t + 2 < plan.n) load(false, t + 2);
          }
        }
      }
      if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
      // no copy may be in flight when the block's shared memory goes
      for (int slot = max(0, used - C::STAGES); slot < used; ++slot)
        (void)wait_bounded(full + slot % C::STAGES, (slot / C::STAGES) & 1, kDrainNs);
    } else if (warp == kItemWarp) {
      // ---- the block's items, one ahead of their rows, and after the last an item without key
      // tiles; a warpgroup's rows are loaded as soon as the item before is done with them
      // Its waits are for work, not for copies: an item takes as long as it has keys (11 ms over
      // 2^20), so the limit counts per key tile of the items not known to be done.
      ItemWalk<Shape> walk(d, pr, a, ctx, lo, hi, at.b, at.before, blockIdx.x);
      if (lane == 0 && a.notes != nullptr) a.notes[blockIdx.x] = walk.border();
      bool ok = true;
      int loaded[2] = {0, 0};
      Item it, next{};
      int open[kItems] = {};                         // key tiles of the last items published
      auto patience = [&]() {
        unsigned long long tiles = 1;
#pragma unroll
        for (int i = 0; i < kItems; ++i) tiles += open[i];
        return ctx.wait_ns <= ~0ull / tiles ? ctx.wait_ns * tiles : ~0ull;
      };
      auto publish = [&](int j) {
        if (!walk.next(&next)) next.kt0 = next.kt1 = 0;
        if (j >= kItems)
          ok = wait_bounded(item_free + j % kItems, (j / kItems - 1) & 1, patience());
#pragma unroll
        for (int i = 0; i + 1 < kItems; ++i) open[i] = open[i + 1];
        open[kItems - 1] = next.kt1 - next.kt0;
        if (ok && lane == 0) {
          items[j % kItems] = next;
          arrive(item_full + j % kItems);
        }
      };
#pragma unroll 1
      for (int j = -1;; ++j) {
        it = next;
        publish(j + 1);
        if (!ok) break;
        const Plan plan(it, a, FEW);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!ok || plan.tiles(w) == 0) continue;
          if (loaded[w] > 0)
            ok = wait_bounded(q_free + w, (loaded[w] - 1) & 1, patience());
          if (!ok) continue;
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full + w, C::TILE_BYTES);
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h)
              tma_rows(smem_addr(sm + C::OFF_Q) + w * C::TILE_BYTES + h * 16384, &map_q, 64 * h,
                       it.g * a.G, it.row0 + (plan.wide ? (w * 128) >> log_g : 0), q_full + w);
          }
          __syncwarp();
          ++loaded[w];
        }
        if (next.kt0 >= next.kt1) break;
      }
      if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (loaded[w] > 0) (void)wait_bounded(q_full + w, (loaded[w] - 1) & 1, kDrainNs);
    }
    __syncwarp();
  }
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(tmem, kTmemCols);
}

template <int D, bool FEW, Mask M>
cudaError_t launch_t(const kv_cache_desc& d, const PackedRows& pr, const PrefillArgs& a,
                     DevCtx ctx, cudaStream_t s) {
  using C = Cfg<D>;
  CUtensorMap mk, mv, mq, mo;
  if (!pool_tensor_map(&mk, d.k_pool, d) || !pool_tensor_map(&mv, d.v_pool, d) ||
      !rows_tensor_map(&mq, a.q, a.q_stride, a.Hq, D, pr.total, a.G, 128 / a.G) ||
      !rows_tensor_map(&mo, a.out, (int64_t)a.Hq * D, a.Hq, D, pr.total, a.G, 32 / a.G))
    return cudaErrorInvalidValue;
  auto kern = prefill_mma_kernel<D, FEW, M>;
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
  return launch_pdl(kern, dim3(a.NC), dim3(kThreads), C::SMEM, s, mk, mv, mq, mo, d, pr, a, ctx);
}

}  // namespace

template <Mask M>
cudaError_t launch_prefill_mma(const kv_cache_desc& d, const PackedRows& pr,
                               const PrefillArgs& a, DevCtx ctx, cudaStream_t s) {
  // one share promises a row the same bits whatever the batch, so the batch chooses nothing there
  const bool few = a.NC > 1 && (int64_t)pr.total * a.G <= (int64_t)kFewRows * d.batch;
  // Up to 16 rows to a sequence at D = 128, 8 at D = 64, another mask's keys take the rows' place.
  // Measured against the instance of few rows, 32 sequences of 32/8 heads of 128 in a window of
  // 1000: 4, 8, 16 and 32 rows 34, 35, 37 and 41 us (41 to 42); 16 heads of 64: 45, 46, 55 and 73
  // (58, 60, 60 and 61), trees over 6000 tokens 101, 105, 127 and 167 (104, 106, 111 and 114).
  // Smaller batches were not measured, and the mean counts sequences without rows too.
  if constexpr (M != Mask::kCausal) {
    if (few && (int64_t)pr.total * a.G * 8 <= (int64_t)d.head_dim * d.batch)
      return launch_prefill_few<M>(d, pr, a, ctx, s);
  }
  if (few)
    return d.head_dim == 128 ? launch_t<128, true, M>(d, pr, a, ctx, s)
                             : launch_t<64, true, M>(d, pr, a, ctx, s);
  return d.head_dim == 128 ? launch_t<128, false, M>(d, pr, a, ctx, s)
                           : launch_t<64, false, M>(d, pr, a, ctx, s);
}

}  // namespace skv
