// Causal prompt attention: the choice of kernel, and the join of the items its blocks shared.
#include "prefill.cuh"

namespace skv {
namespace {

constexpr int kMergeWarps = 8;
constexpr int kMergeRowGroups = 8;       // blocks per border, each with a share of the rows

template <typename T> __device__ __forceinline__ void store2(T* p, float a, float b);
template <> __device__ __forceinline__ void store2<bf16_t>(bf16_t* p, float a, float b) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  *reinterpret_cast<uint32_t*>(p) = w;
}
template <> __device__ __forceinline__ void store2<float>(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

// Border number c = blockIdx.x + 1 between blocks c - 1 and c: if it cuts an item, and is the
// first that does, joins the item's parts row by row:
//   out = sum_p acc_p 2^(m_p - M) / L,  M = max_p m_p,  L = sum_p l_p 2^(m_p - M).
// The parts are those of blocks c - 1, c, ... up to the one that reaches the item's end. One
// warp per row, lanes over the parts for (m, l) and over the columns for the accumulators,
// whose loads are independent of one another. A part without keys for a row (m = -inf) has no
// accumulator to read.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
prefill_merge_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int PAIRS = D / 64;            // column pairs per lane
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const BorderNote it = a.notes[c], before = a.notes[c - 1];
  auto continues = [&](const BorderNote& n) {
    return n.row0 == it.row0 && n.g == it.g && n.kt0 > 0 && n.kt0 < n.nk;
  };
  if (!continues(it) || continues(before)) return;
  const int rows = it.n_tok << a.log_g;
  for (int row = blockIdx.y * kMergeWarps + warp; row < rows;
       row += kMergeRowGroups * kMergeWarps) {
    float M = -INFINITY, L = 0.f;
    float2 acc[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) acc[p] = make_float2(0.f, 0.f);
    bool more = true;
    for (int j0 = c - 1; more; j0 += 32) {
      // block c - 1 ends with this item, the others begin with it
      const int j = j0 + lane;
      BorderNote n = it;
      if (j >= c && j < a.NC) n = a.notes[j];
      const bool part = j == c - 1 || (j < a.NC && continues(n));
      const int parts = __popc(__ballot_sync(0xffffffffu, part));       // the first lanes
      more = parts == 32;
      const int64_t mine = (int64_t)(j == c - 1 ? 2 * j + 1 : 2 * j) * a.part_rows + row;
      float m = -INFINITY, l = 0.f;
      if (part && (j == c - 1 || n.kt1 > n.kt0)) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + mine);
        m = ml.x;
        l = ml.y;
      }
      float now = fmaxf(M, m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
      if (now == -INFINITY) continue;
      const float keep = exp2f(M - now), w = exp2f(m - now);
      M = now;
      float sum = l * w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      L = fmaf(L, keep, sum);
#pragma unroll
      for (int p = 0; p < PAIRS; ++p) {
        acc[p].x *= keep;
        acc[p].y *= keep;
      }
#pragma unroll 8
      for (int e = 0; e < parts; ++e) {
        const float we = __shfl_sync(0xffffffffu, w, e);
        const int64_t from = __shfl_sync(0xffffffffu, mine, e);
        float2 v[PAIRS];
#pragma unroll
        for (int p = 0; p < PAIRS; ++p)          // no keys, or nothing left of them: not read
          v[p] = we == 0.f ? make_float2(0.f, 0.f)
                           : __ldcg(reinterpret_cast<const float2*>(a.part_acc + from * D) + lane +
                                    32 * p);
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
          acc[p].x = fmaf(v[p].x, we, acc[p].x);
          acc[p].y = fmaf(v[p].y, we, acc[p].y);
        }
      }
    }
    const int64_t out_row = (int64_t)(it.row0 + (row >> a.log_g)) * a.Hq + it.g * a.G +
                            (row & (a.G - 1));
    const float inv = 1.f / L;                     // every row sees its own token: L > 0
    T* dst = static_cast<T*>(a.out) + out_row * D + 2 * lane;
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) store2<T>(dst + 64 * p, acc[p].x * inv, acc[p].y * inv);
    if (lane == 0 && a.lse != nullptr) a.lse[out_row] = (M + log2f(L)) * kLn2;
  }
}

template <typename T, int D>
cudaError_t merge_t(const PrefillArgs& a, cudaStream_t s) {
  return launch_pdl(prefill_merge_kernel<T, D>, dim3(a.NC - 1, kMergeRowGroups),
                    dim3(kMergeWarps * 32), 0, s, a);
}

}  // namespace

int prefill_tile_rows(int dtype) { return dtype == KV_BF16 ? MmaShape::rows : SimtShape::rows; }
int prefill_blocks_per_sm(int dtype) { return dtype == KV_BF16 ? 1 : 2; }

cudaError_t launch_prefill(const kv_cache_desc& d, const int32_t* cu, int total,
                           const PrefillArgs& a, DevCtx ctx, cudaStream_t s) {
  const PackedRows pr{cu, total};
  const bool bf = d.dtype == KV_BF16;
  cudaError_t e = bf ? launch_prefill_mma(d, pr, a, ctx, s) : launch_prefill_simt(d, pr, a, ctx, s);
  if (e != cudaSuccess || a.NC == 1) return e;
  if (bf) return d.head_dim == 128 ? merge_t<bf16_t, 128>(a, s) : merge_t<bf16_t, 64>(a, s);
  return d.head_dim == 128 ? merge_t<float, 128>(a, s) : merge_t<float, 64>(a, s);
}

}  // namespace skv
