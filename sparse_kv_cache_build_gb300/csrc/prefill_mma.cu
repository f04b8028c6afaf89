// Causal prompt attention for bf16 caches on the tensor cores.
//
// A block takes 256 rows (256 / G tokens of one KV head) as two tiles of 128, one per softmax
// warpgroup, and walks their keys 128 at a time:
//   S = Q K^T    128 x 128 x D,   Q and K from shared memory, S in TMEM
//   P = 2^(scale_log2 S - m)      one thread per row: its warpgroup reads S from TMEM, keeps
//                                 m and l in registers and writes P back over S as bf16
//   O += P V     128 x D x 128,   P from TMEM, V from shared memory, O in TMEM
// One thread issues the products, alternating between the two tiles, so that one tile's
// softmax runs under the other's products:
//   ... P0 V(j), Q0 K(j+1) | P1 V(j), Q1 K(j+1) | P0 V(j+1), ...
// One warp feeds K and V tiles through a ring by TMA, page by page (a page of one KV head is
// PS dense rows of the pool).
//
// A block with at most 128 rows (single tokens, drafts, a prompt's tail) gives both warpgroups
// the same rows and alternating key tiles instead, and joins their (m, l, O) at the end: the
// same pipeline, with the softmax still under the other warpgroup's products.
//
// The running maximum is lazy: O and l are rescaled only when a row's maximum grows by more
// than 2^8, so that almost no tile pays for it; P stays below 2^8 and every sum is float32.
// Rows see keys up to their own position; the tiles on that border are masked. Keys of slots
// past the item's last key never reach a sum: their scores are masked, and their rows of the
// V tile are zeroed in shared memory (a zero probability times a NaN would not vanish).
//
// Rounding: P is rounded to bf16 for the second product (relative 2^-8 each, independent), as
// the tensor core takes bf16 operands; its sum l is taken over the unrounded values.
#include <atomic>

#include "prefill.cuh"
#include "tcgen05.cuh"

namespace skv {
namespace {

constexpr int kThreads = 384;          // two softmax warpgroups, then products and loads
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kRows = kPrefillMmaRows;  // rows of a block, two tiles
constexpr int kKeys = 128;             // keys of a tile
constexpr int kTmemCols = 512;
constexpr int kRegsSoftmax = 216, kRegsOther = 72;     // (2 * 216 + 72) * 128 = 384 * 168
constexpr float kLazy = 8.f;           // log2 of the growth that forces a rescale

template <int D> struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = HALVES * 128 * 128;         // 128 rows of D bf16
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr size_t OFF_Q = 0;                            // from a 1024-aligned base
  static constexpr size_t OFF_RING = 2 * TILE_BYTES;
  static constexpr size_t OFF_BAR = OFF_RING + (size_t)STAGES * TILE_BYTES;
  static constexpr int BARS = 2 * STAGES + 9;
  static constexpr size_t OFF_MISC = OFF_BAR + 8 * BARS;
  static constexpr size_t SMEM = OFF_MISC + 16 + 1024;          // + alignment slack
  static_assert((size_t)STAGES * TILE_BYTES >= 128 * (size_t)(D + 2) * 4, "join buffer");
};

// The block's plan: which key tiles each warpgroup takes and where they lie in the ring.
struct Plan {
  bool wide;      // two row tiles; else one, with the key tiles dealt out in turn
  int n;          // key tiles of the block
  int n0, n1;     // key tiles of each warpgroup

  __device__ __forceinline__ int tiles(int w) const { return w == 0 ? n0 : n1; }
  __device__ __forceinline__ int tile(int w, int i) const { return wide ? i : 2 * i + w; }
  // Ring slots in the order of first use: K0 V0 K1 V1 ..., or (dealt out) K0 K1 V0 K2 V1 K3 ...
  __device__ __forceinline__ int k_slot(int t) const {
    return wide ? 2 * t : t < 2 ? t : 2 * t - 1;
  }
  __device__ __forceinline__ int v_slot(int t) const {
    return wide || t == n - 1 ? 2 * t + 1 : 2 * t + 2;
  }
};

__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prefill_mma_kernel(const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, kv_cache_desc d, PackedRows pr,
                   PrefillArgs a, int log_g, DevCtx ctx) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~(uintptr_t)1023);
  uint8_t* ring = sm + C::OFF_RING;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint64_t* full = bar;                          // [STAGES] a K or V tile has landed
  uint64_t* empty = bar + C::STAGES;             // [STAGES] its last product is done
  uint64_t* s_full = bar + 2 * C::STAGES;        // [2] S of a warpgroup is in TMEM
  uint64_t* p_full = s_full + 2;                 // [2] its P is in TMEM, O rescaled
  uint64_t* o_done = p_full + 2;                 // [2] its last product is done
  uint64_t* q_full = o_done + 2;                 // the rows are in shared memory
  uint64_t* v_land = q_full + 1;                 // the last V tile, before its tail is zeroed
  uint64_t* drained = v_land + 1;                // after a timeout: no product in flight
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full + w, 1);
      mbar_init(p_full + w, 4);                  // one arrival per softmax warp
      mbar_init(o_done + w, 1);
    }
    mbar_init(q_full, 8);
    mbar_init(v_land, 1);
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0) check_packed_rows(ctx, d, pr);
  PrefillItem it;
  if (!prefill_item(ctx, d, pr, a, kRows >> log_g, kKeys, &it)) {
    if (pr.cu == nullptr && a.S == 1) empty_row<bf16_t, D>(a, it.b, it.g);
    return;
  }
  if (warp == kMmaWarp) tc::alloc(tmem_slot, kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;

  const int rows = it.n_tok << log_g;
  Plan plan;
  plan.wide = rows > 128;
  plan.n = it.kt1 - it.kt0;
  if (plan.wide) {
    // the first tile's rows end earlier: its last keys may lie a tile before the block's
    const int last0 = it.pos0 + (127 >> log_g);
    plan.n0 = max(0, min(plan.n, last0 / kKeys + 1 - it.kt0));
    plan.n1 = plan.n;
  } else {
    plan.n0 = (plan.n + 1) / 2;
    plan.n1 = plan.n / 2;
  }
  const int keys = it.pos0 + it.n_tok;           // keys from here on are nobody's

  if (warp < 8) {
    tc::more_regs<kRegsSoftmax>();
    const int w = warp >> 2, r = tid & 127;      // warpgroup, TMEM lane
    // ---- the rows, into 128-byte swizzled shared rows (zeros past the block's last row)
    {
      constexpr int CH = D / 8;                  // 16-byte chunks of a row
      const int total = (plan.wide ? 256 : 128) * CH;
      const uint16_t* q = static_cast<const uint16_t*>(a.q);
      for (int i = tid; i < total; i += 256) {
        const int row = i / CH, c = i % CH;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < rows)
          v = *reinterpret_cast<const uint4*>(
              q + (int64_t)(it.row0 + (row >> log_g)) * a.q_stride +
              (int64_t)(it.g * a.G + (row & (a.G - 1))) * D + c * 8);
        uint8_t* dst = sm + C::OFF_Q + (row >> 7) * C::TILE_BYTES + (c >> 3) * 16384 +
                       (row & 127) * 128 + (((c & 7) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(dst) = v;
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) arrive(q_full);
    }
    // ---- softmax
    const int row = plan.wide ? w * 128 + r : r;
    const int last = it.pos0 + (row >> log_g);                    // the row's last key
    const int warp_row = row - lane;
    const bool idle = warp_row >= rows;                           // no row in this warp
    const int warp_first = it.pos0 + (warp_row >> log_g);         // its first row's last key
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // TMEM lane 32 * (warp % 4)
    const uint32_t ts = tmem + lanes + w * 128, to = tmem + lanes + 256 + w * 128;
    const int n = plan.tiles(w);
    const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      ok = mbar_wait_bounded(s_full + w, i & 1, ctx.wait_ns);
      if (!ok) break;
      tc::fence_after();
      if (!idle) {
        const int u0 = (it.kt0 + plan.tile(w, i)) * kKeys;
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld32(ts + 32 * c, s + 32 * c);
        tc::wait_ld();
        if (warp_first - u0 < kKeys - 1) {                        // on the border
          const int seen = last - u0;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > seen) s[c] = 0xff800000u;
        }
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          top[c] = __uint_as_float(s[c]);
#pragma unroll
          for (int e = 4; e < 128; e += 4) top[c] = fmaxf(top[c], __uint_as_float(s[e + c]));
        }
        const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
        if (__any_sync(0xffffffffu, now > m + kLazy)) {
          // s_full(i) follows the products before it: O is complete up to tile i - 1
          const float next = now > m + kLazy ? now : m;
          const float f = next == -INFINITY ? 1.f : exp2f(m - next);
          m = next;
          l *= f;
          if (i > 0) {
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc::ld32(to + c, o);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tc::st32(to + c, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;               // no key of this row yet
        const float2 ref2 = make_float2(-ref, -ref);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float2 x = make_float2(__uint_as_float(s[64 * h + 2 * e]),
                                   __uint_as_float(s[64 * h + 2 * e + 1]));
            x = tc::fma2(x, scale2, ref2);
            x.x = tc::exp2_approx(x.x);
            x.y = tc::exp2_approx(x.y);
            sum[e & 1] = tc::add2(sum[e & 1], x);
            p[e] = tc::pack_bf16(x.x, x.y);
          }
          tc::st32(ts + 32 * h, p);
        }
        sum[0] = tc::add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        tc::wait_st();
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) arrive(p_full + w);
    }
    // ---- output
    if (ok && n > 0) ok = mbar_wait_bounded(o_done + w, 0, ctx.wait_ns);
    const bool join = !plan.wide && plan.n1 > 0;
    if (join) {
      // the ring is free once both warpgroups' products are done
      if (ok) ok = mbar_wait_bounded(o_done + (w ^ 1), 0, ctx.wait_ns);
      tc::fence_after();
      float* box = reinterpret_cast<float*>(ring);                // [D + 2][128]
      if (w == 1 && ok && !idle) {
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc::ld32(to + c, o);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) box[(c + e) * 128 + r] = __uint_as_float(o[e]);
        }
        box[D * 128 + r] = m;
        box[(D + 1) * 128 + r] = l;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if (!ok) {
      if (lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
    } else if (!idle && (plan.wide || w == 0)) {
      tc::fence_after();
      const float* box = reinterpret_cast<const float*>(ring);
      float f0 = 1.f, f1 = 0.f;
      if (join) {
        const float m1 = box[D * 128 + r];
        const float both = fmaxf(m, m1);
        f0 = m == -INFINITY ? 0.f : exp2f(m - both);
        f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - both);
        l = l * f0 + box[(D + 1) * 128 + r] * f1;
        m = both;
      }
      const int64_t at = (int64_t)(it.row0 + (row >> log_g)) * a.Hq + it.g * a.G +
                         (row & (a.G - 1));
      const bool mine = row < rows;
      if (a.S == 1) f0 /= l, f1 /= l;            // every row sees its own token: l > 0
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t raw[32];
        float o[32];
        if (n > 0) {
          tc::ld32(to + c, raw);
          tc::wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          o[e] = n > 0 ? __uint_as_float(raw[e]) * f0 : 0.f;
          if (join) o[e] = fmaf(box[(c + e) * 128 + r], f1, o[e]);
        }
        if (!mine) continue;
        if (a.S == 1) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * D + c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(tc::pack_bf16(o[8 * e], o[8 * e + 1]),
                                tc::pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                tc::pack_bf16(o[8 * e + 4], o[8 * e + 5]),
                                tc::pack_bf16(o[8 * e + 6], o[8 * e + 7]));
        } else {
          float4* dst = reinterpret_cast<float4*>(a.part_acc + (at * a.S + it.s) * D + c);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (mine) {
        if (a.S == 1) {
          if (a.lse != nullptr) a.lse[at] = (m + log2f(l)) * kLn2;
        } else {
          a.part_ml[(at * a.S + it.s) * 2] = m;
          a.part_ml[(at * a.S + it.s) * 2 + 1] = l;
        }
      }
    }
    tc::fence_before();
  } else {
    tc::fewer_regs<kRegsOther>();
    if (warp == kMmaWarp && lane == 0 && plan.n > 0) {
      // ---- products
      constexpr uint32_t id_s = tc::idesc(kKeys, false), id_o = tc::idesc(D, true);
      const uint32_t q_addr = smem_addr(sm + C::OFF_Q), ring_addr = smem_addr(ring);
      bool ok = mbar_wait_bounded(q_full, 0, ctx.wait_ns);
      auto landed = [&](int slot) {
        return mbar_wait_bounded(full + slot % C::STAGES, (slot / C::STAGES) & 1, ctx.wait_ns);
      };
      auto scores = [&](int w, int i) {
        const int slot = plan.k_slot(plan.tile(w, i));
        ok = ok && landed(slot);
        if (!ok) return;
        tc::fence_after();
        const uint32_t qa = q_addr + (plan.wide ? w * C::TILE_BYTES : 0);
        const uint32_t ka = ring_addr + (slot % C::STAGES) * C::TILE_BYTES;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
          tc::mma_ss(tmem + w * 128, tc::smem_desc(qa + off, 16), tc::smem_desc(ka + off, 16),
                     id_s, k > 0);
        }
        tc::commit(s_full + w);
        if (!plan.wide || w == 1) tc::commit(empty + slot % C::STAGES);
      };
      auto values = [&](int w, int i) {
        const int slot = plan.v_slot(plan.tile(w, i));
        ok = ok && mbar_wait_bounded(p_full + w, i & 1, ctx.wait_ns) && landed(slot);
        if (!ok) return;
        tc::fence_after();
        const uint32_t va = ring_addr + (slot % C::STAGES) * C::TILE_BYTES;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          tc::mma_ts(tmem + 256 + w * 128, tmem + w * 128 + k * 8,
                     tc::smem_desc(va + k * 2048, 16384), id_o, i > 0 || k > 0);
        if (!plan.wide || w == 1) tc::commit(empty + slot % C::STAGES);
        if (i + 1 == plan.tiles(w)) tc::commit(o_done + w);
      };
      for (int w = 0; w < 2; ++w)
        if (plan.tiles(w) > 0) scores(w, 0);
      for (int i = 0; ok && i < max(plan.n0, plan.n1); ++i)
        for (int w = 0; w < 2; ++w) {
          if (i < plan.tiles(w)) values(w, i);
          if (i + 1 < plan.tiles(w)) scores(w, i + 1);
        }
      if (!ok) {
        flag(ctx, KV_DEVERR_TIMEOUT);
        tc::commit(drained);
        (void)mbar_wait_bounded(drained, 0, ctx.wait_ns);
      }
    } else if (warp == kLoadWarp) {
      // ---- loads: one page half (64 columns) per lane
      const int PS = d.page_size, per_tile = kKeys / PS;
      const int copies = per_tile * C::HALVES;
      const int page = lane % per_tile, half = lane / per_tile;
      const uint32_t box = (uint32_t)PS * 128;
      const uint32_t dst = smem_addr(ring) + half * 16384 + page * box;
      const int32_t* table = d.page_table + (int64_t)it.b * d.page_table_stride;
      bool ok = true;
      int used = 0;
      auto load = [&](const CUtensorMap* map, int t, int slot, bool values) {
        if (!ok) return;
        const int stage = slot % C::STAGES;
        const int64_t key = (int64_t)(it.kt0 + t) * kKeys + page * PS;   // of the lane's page
        int P = -1;
        const bool wanted = lane < copies && key < keys;
        if (wanted) {
          P = __ldg(table + (int)(key / PS));
          if (P < 0 || P >= d.num_phys_pages) {
            flag(ctx, KV_DEVERR_BAD_PAGE);
            P = -1;
          }
        }
        if (slot >= C::STAGES)
          ok = mbar_wait_bounded(empty + stage, (slot / C::STAGES - 1) & 1, ctx.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        // the item's last key lies inside this tile: the V rows after it become zeros
        const int valid = (int)min((int64_t)kKeys, (int64_t)keys - (int64_t)(it.kt0 + t) * kKeys);
        const bool tail = values && valid < kKeys;
        uint64_t* land = tail ? v_land : full + stage;
        const int boxes = __popc(__ballot_sync(0xffffffffu, P >= 0));
        if (lane == 0) mbar_arrive_expect_tx(land, boxes * box);
        __syncwarp();
        if (P >= 0)
          tma_page(dst + stage * C::TILE_BYTES, map, half * 64,
                   (P * d.num_kv_heads + it.g) * PS, land);
        used = slot + 1;
        if (!tail) return;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(v_land, 0, ctx.wait_ns));
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
        for (int t = 0; t < plan.n; ++t) {
          load(&map_k, t, plan.k_slot(t), false);
          load(&map_v, t, plan.v_slot(t), true);
        }
      } else {
        for (int t = 0; t < min(2, plan.n); ++t) load(&map_k, t, plan.k_slot(t), false);
        for (int t = 0; t < plan.n; ++t) {
          load(&map_v, t, plan.v_slot(t), true);
          if (t + 2 < plan.n) load(&map_k, t + 2, plan.k_slot(t + 2), false);
        }
      }
      if (!ok && lane == 0) flag(ctx, KV_DEVERR_TIMEOUT);
      // no copy may be in flight when the block's shared memory goes
      for (int slot = max(0, used - C::STAGES); slot < used; ++slot)
        (void)mbar_wait_bounded(full + slot % C::STAGES, (slot / C::STAGES) & 1, ctx.wait_ns);
    }
    __syncwarp();
  }
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(tmem, kTmemCols);
}

template <int D>
cudaError_t launch_t(const kv_cache_desc& d, const PackedRows& pr, const PrefillArgs& a,
                     DevCtx ctx, cudaStream_t s) {
  using C = Cfg<D>;
  CUtensorMap mk, mv;
  if (!pool_tensor_map(&mk, d.k_pool, d) || !pool_tensor_map(&mv, d.v_pool, d))
    return cudaErrorInvalidValue;
  auto kern = prefill_mma_kernel<D>;
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
  const int log_g = a.G == 1 ? 0 : a.G == 2 ? 1 : a.G == 4 ? 2 : 3;
  const long items = work_numbers(pr.cu, pr.total, d.batch, kRows / a.G, 1);
  dim3 grid((unsigned)(items * d.num_kv_heads), a.S);
  return launch_pdl(kern, grid, dim3(kThreads), C::SMEM, s, mk, mv, d, pr, a, log_g, ctx);
}

}  // namespace

cudaError_t launch_prefill_mma(const kv_cache_desc& d, const PackedRows& pr,
                               const PrefillArgs& a, DevCtx ctx, cudaStream_t s) {
  return d.head_dim == 128 ? launch_t<128>(d, pr, a, ctx, s) : launch_t<64>(d, pr, a, ctx, s);
}

}  // namespace skv
