// Causal prompt attention: the choice of kernel, and the merge of its splits.
#include "prefill.cuh"

namespace skv {
namespace {

template <typename T> __device__ __forceinline__ void store_out(T* p, float a, float b);
template <> __device__ __forceinline__ void store_out<bf16_t>(bf16_t* p, float a, float b) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  *reinterpret_cast<uint32_t*>(p) = w;
}
template <> __device__ __forceinline__ void store_out<float>(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

// out = sum_s acc_s 2^(m_s - M) / L with M = max m_s, L = sum_s l_s 2^(m_s - M). One block of
// D/2 threads per (row, head), two columns each: with few rows the blocks are few, and a
// block's partials are all loaded before the first is used. Splits without keys for a row
// (m = -inf) carry no weight and their accumulators are not read.
constexpr int kMergeBatch = 8;

template <typename T, int D>
__global__ void __launch_bounds__(D / 2)
prefill_merge_kernel(kv_cache_desc d, PackedRows pr, PrefillArgs a, DevCtx ctx) {
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, h = blockIdx.y, c = 2 * threadIdx.x;
  int base;
  const int b = find_sequence(pr, d.batch, 1, 0, row, &base);
  const SeqRows sr = seq_rows(ctx, d, pr, b);
  const int64_t at = (int64_t)row * a.Hq + h;
  T* dst = static_cast<T*>(a.out) + at * D + c;
  if (row >= sr.row0 + sr.n || row < sr.row0) {
    // not a row of any sequence: left as it was, but for an empty sequence's own row
    if (pr.cu == nullptr) {
      store_out<T>(dst, 0.f, 0.f);
      if (c == 0 && a.lse != nullptr) a.lse[at] = -INFINITY;
    }
    return;
  }
  const float* ml = a.part_ml + at * a.S * 2;
  const float* acc = a.part_acc + at * a.S * D + c;
  float M = -INFINITY;
  for (int s = 0; s < a.S; ++s) M = fmaxf(M, ml[2 * s]);
  float L = 0.f, x = 0.f, y = 0.f;
  for (int s0 = 0; s0 < a.S; s0 += kMergeBatch) {
    float2 v[kMergeBatch];
    float w[kMergeBatch];
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      const int s = s0 + i;
      const float m = s < a.S ? ml[2 * s] : -INFINITY;
      w[i] = m == -INFINITY ? 0.f : exp2f(m - M);
      v[i] = m == -INFINITY ? make_float2(0.f, 0.f)
                            : *reinterpret_cast<const float2*>(acc + (int64_t)s * D);
      if (m != -INFINITY) L = fmaf(ml[2 * s + 1], w[i], L);
    }
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      x = fmaf(v[i].x, w[i], x);
      y = fmaf(v[i].y, w[i], y);
    }
  }
  const float inv = 1.f / L;             // every row sees its own token: L > 0
  store_out<T>(dst, x * inv, y * inv);
  if (c == 0 && a.lse != nullptr) a.lse[at] = (M + log2f(L)) * kLn2;
}

template <typename T, int D>
cudaError_t merge_t(const kv_cache_desc& d, const PackedRows& pr, const PrefillArgs& a,
                    DevCtx ctx, cudaStream_t s) {
  return launch_pdl(prefill_merge_kernel<T, D>, dim3(pr.total, a.Hq), dim3(D / 2), 0, s, d, pr,
                    a, ctx);
}

}  // namespace

int prefill_tile_tokens(int dtype, int G) {
  return (dtype == KV_BF16 ? kPrefillMmaRows : kPrefillSimtRows) / G;
}

cudaError_t launch_prefill(const kv_cache_desc& d, const int32_t* cu, int total,
                           const PrefillArgs& a, DevCtx ctx, cudaStream_t s) {
  const PackedRows pr{cu, total};
  cudaError_t e = d.dtype == KV_BF16 ? launch_prefill_mma(d, pr, a, ctx, s)
                                     : launch_prefill_simt(d, pr, a, ctx, s);
  if (e != cudaSuccess || a.S == 1) return e;
  if (d.dtype == KV_BF16)
    return d.head_dim == 128 ? merge_t<bf16_t, 128>(d, pr, a, ctx, s)
                             : merge_t<bf16_t, 64>(d, pr, a, ctx, s);
  return d.head_dim == 128 ? merge_t<float, 128>(d, pr, a, ctx, s)
                           : merge_t<float, 64>(d, pr, a, ctx, s);
}

}  // namespace skv
