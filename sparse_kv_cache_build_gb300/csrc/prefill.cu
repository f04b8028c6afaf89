// Attention of packed rows: the choice of kernel, and the join of the items its blocks shared.
#include <type_traits>

#include "prefill.cuh"

namespace skv {
namespace {

constexpr int kMergeWarps = 8;
constexpr int kMergeUnits = 4;           // (row, strip) units per warp at most

// V consecutive floats, read as one word.
template <int V> union Strip {
  using Few = typename std::conditional<V == 2, float2, float>::type;
  using Raw = typename std::conditional<V == 4, float4, Few>::type;
  Raw raw;
  float f[V];
  __device__ __forceinline__ Strip() {}
};

template <typename T> __device__ __forceinline__ void store1(T* p, float v);
template <> __device__ __forceinline__ void store1<bf16_t>(bf16_t* p, float v) {
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(p->bits) : "f"(v));
}
template <> __device__ __forceinline__ void store1<float>(float* p, float v) { *p = v; }

// Border number c = blockIdx.x + 1 between blocks c - 1 and c: if it cuts an item, and is the
// first that does, joins the item's parts row by row:
//   out = sum_p acc_p 2^(m_p - M) / L,  M = max_p m_p,  L = sum_p l_p 2^(m_p - M).
// The parts are those of blocks c - 1, c, ... up to the one that reaches the item's end. One
// warp takes 32 V columns of a row; notes, then (m, l) and accumulators together, are the only
// dependent reads, with several parts in flight. Few rows (single tokens: many parts each) take
// V = 1, so that four warps share a row (one token over 32K: 4.6 us from the last part to the
// output, against 7 us); tiles of rows take V = D / 32 (8192 tokens 429 us a call, against 464 us
// with V = 1, whose warps are four times as many). A part without keys for a row (m = -inf) has
// no accumulator: what lies there is read and not used.
template <typename T, int D, int V>
__global__ void __launch_bounds__(kMergeWarps * 32)
prefill_merge_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int STRIPS = D / (32 * V), BATCH = V == 4 ? 8 : 16;
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // lane i: the note of block c - 1 + i
  const BorderNote none{0, 0, 0, 0, 0, 0};
  BorderNote n = c - 1 + lane < a.NC ? a.notes[c - 1 + lane] : none;
  const int row0 = __shfl_sync(0xffffffffu, n.row0, 1), g = __shfl_sync(0xffffffffu, n.g, 1);
  const int n_tok = __shfl_sync(0xffffffffu, n.n_tok, 1);
  auto continues = [&](const BorderNote& x) {
    return x.row0 == row0 && x.g == g && x.kt0 > 0 && x.kt0 < x.nk;
  };
  const uint32_t first = __ballot_sync(0xffffffffu, continues(n));
  if ((first & 3u) != 2u) return;
  const int units = (n_tok << a.log_g) * STRIPS;
  for (int unit = blockIdx.y * kMergeWarps + warp; unit < units;
       unit += gridDim.y * kMergeWarps) {
    const int row = unit / STRIPS, col = ((unit % STRIPS) * 32 + lane) * V;
    float M = -INFINITY, L = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    bool more = true;
    for (int j0 = c - 1; more; j0 += 32) {
      const int j = j0 + lane;
      BorderNote x = n;
      if (j0 > c - 1) x = j < a.NC ? a.notes[j] : none;
      const bool head = j == c - 1, part = head || continues(x);
      const uint32_t run = __ballot_sync(0xffffffffu, part);
      const int parts = run == 0xffffffffu ? 32 : __ffs(~run) - 1;       // the lanes before a gap
      more = parts == 32;
      // block c - 1 ends with this item, the others begin with it
      const int64_t mine = (int64_t)(head ? 2 * j + 1 : 2 * j) * a.part_rows + row;
      float m = -INFINITY, l = 0.f;
      if (lane < parts && (head || x.kt1 > x.kt0)) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + mine);
        m = ml.x;
        l = ml.y;
      }
      for (int e0 = 0; e0 < parts; e0 += BATCH) {
        Strip<V> v[BATCH];
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
          const int64_t from = __shfl_sync(0xffffffffu, mine, (e0 + e) & 31);
          if (e0 + e < parts)
            v[e].raw = __ldcg(reinterpret_cast<const typename Strip<V>::Raw*>(
                a.part_acc + from * D + col));
        }
        if (e0 == 0) {
          float now = fmaxf(M, m);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
          const float ref = now == -INFINITY ? 0.f : now;
          const float keep = exp2f(M - ref);
          M = now;
          m = exp2f(m - ref);                      // now the part's weight
          float sum = l * m;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          L = fmaf(L, keep, sum);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] *= keep;
        }
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
          const float w = __shfl_sync(0xffffffffu, m, (e0 + e) & 31);
          if (e0 + e < parts && w != 0.f)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(v[e].f[i], w, acc[i]);
        }
      }
    }
    const int64_t out_row = (int64_t)(row0 + (row >> a.log_g)) * a.Hq + g * a.G +
                            (row & (a.G - 1));
    T* dst = static_cast<T*>(a.out) + out_row * D + col;
#pragma unroll
    for (int i = 0; i < V; ++i) store1<T>(dst + i, acc[i] / L);        // L > 0: its own token
    if (col == 0 && a.lse != nullptr) a.lse[out_row] = (M + log2f(L)) * kLn2;
  }
}

constexpr int kMergeFewRows = 64;

template <typename T, int D, int V>
cudaError_t merge_v(const PrefillArgs& a, cudaStream_t s) {
  // Few rows with many parts: a unit per warp, as four one after the other are the call's end (eight
  // drafts over 8192 tokens, 8/2 heads of 64: 29 -> 17 us).
  const int units = a.part_rows * (D / (32 * V)), per_warp = V == 1 ? 1 : kMergeUnits;
  return launch_pdl(prefill_merge_kernel<T, D, V>,
                    dim3(a.NC - 1, ceil_div(units, kMergeWarps * per_warp)),
                    dim3(kMergeWarps * 32), 0, s, a);
}
template <typename T, int D>
cudaError_t merge_t(const PrefillArgs& a, cudaStream_t s) {
  return a.part_rows < kMergeFewRows ? merge_v<T, D, 1>(a, s) : merge_v<T, D, D / 32>(a, s);
}

}  // namespace

int prefill_tile_rows(int dtype) { return dtype == KV_BF16 ? MmaShape::rows : SimtShape::rows; }

cudaError_t launch_prefill(const kv_cache_desc& d, const int32_t* cu, int total,
                           const PrefillArgs& a, DevCtx ctx, cudaStream_t s) {
  const PackedRows pr{cu, total};
  const bool bf = d.dtype == KV_BF16;
  cudaError_t e;
  if (a.mask == Mask::kCausal)
    e = bf ? launch_prefill_mma<Mask::kCausal>(d, pr, a, ctx, s)
           : launch_prefill_simt<Mask::kCausal>(d, pr, a, ctx, s);
  else if (a.mask == Mask::kWindow)
    e = bf ? launch_prefill_mma<Mask::kWindow>(d, pr, a, ctx, s)
           : launch_prefill_simt<Mask::kWindow>(d, pr, a, ctx, s);
  else
    e = bf ? launch_prefill_mma<Mask::kTree>(d, pr, a, ctx, s)
           : launch_prefill_simt<Mask::kTree>(d, pr, a, ctx, s);
  if (e != cudaSuccess || a.NC == 1) return e;
  if (bf) return d.head_dim == 128 ? merge_t<bf16_t, 128>(a, s) : merge_t<bf16_t, 64>(a, s);
  return d.head_dim == 128 ? merge_t<float, 128>(a, s) : merge_t<float, 64>(a, s);
}

}  // namespace skv
