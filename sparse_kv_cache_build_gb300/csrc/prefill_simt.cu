// Causal prompt attention for fp32 caches, on the CUDA cores.
//
// One block takes 64 rows and walks their keys 64 at a time, with the running maximum and sum
// of the softmax per row. 256 threads hold 4 x 4 of the 64 x 64 scores and 4 x D/16 of the
// output each; the operands come from shared memory as 16-byte reads (rows padded by four
// floats, so that the sixteen keys of a warp's read fall into different banks), the
// probabilities go through the key tile's buffer once its scores are done.
#include "prefill.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int R = SimtShape::rows, KT = SimtShape::keys;

template <int D> struct SimtCfg {
  static constexpr int LD = D + 4;                   // padded row, floats
  static constexpr int PLD = KT + 4;
  static constexpr size_t SMEM = sizeof(float) * 3 * R * LD;
  static_assert(R * PLD <= KT * LD, "the probabilities fit the key buffer");
};

// Copies R rows of D elements into padded shared rows; row(i) gives the source of row i, or NULL
// for zeros.
template <int D, typename F>
__device__ __forceinline__ void stage_rows(float* dst, F row) {
  constexpr int CPR = D / 4;                         // 16-byte chunks of a row
  for (int i = threadIdx.x; i < R * CPR; i += kThreads) {
    const int r = i / CPR, c = (i % CPR) * 4;
    const float* src = row(r);
    *reinterpret_cast<float4*>(dst + r * SimtCfg<D>::LD + c) =
        src != nullptr ? *reinterpret_cast<const float4*>(src + c)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

__device__ __forceinline__ void store4(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
prefill_simt_kernel(const __grid_constant__ kv_cache_desc d, const __grid_constant__ PackedRows pr,
                    const __grid_constant__ PrefillArgs a, const __grid_constant__ DevCtx ctx) {
  using C = SimtCfg<D>;
  constexpr int LD = C::LD, PLD = C::PLD, NC = D / 64;
  extern __shared__ __align__(16) float sm[];
  __shared__ LineScratch scratch;
  float* sq = sm;
  float* sk = sq + R * LD;
  float* sv = sk + KT * LD;
  pdl_trigger();
  pdl_wait();
  finish_empty<float, D>(ctx, d, pr, a);
  const LinePlace at = find_place<SimtShape>(ctx, d, pr, a, blockIdx.x, &scratch);
  const int64_t lo = at.lo, hi = at.hi;
  if (at.total == 0) {
    if (threadIdx.x == 0 && a.notes != nullptr) a.notes[blockIdx.x] = BorderNote{0, 0, 0, 0, 0, 0};
    return;
  }
  ItemWalk<SimtShape> walk(d, pr, a, ctx, lo, hi, at.b, at.before, blockIdx.x);
  if (threadIdx.x == 0 && a.notes != nullptr) a.notes[blockIdx.x] = walk.border();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int Hkv = d.num_kv_heads, PS = d.page_size;
  const float* q = static_cast<const float*>(a.q);
  const float* kp = static_cast<const float*>(d.k_pool);
  const float* vp = static_cast<const float*>(d.v_pool);

  PrefillItem it;
  while (walk.next(&it)) {
    const int32_t* table = d.page_table + (int64_t)it.b * d.page_table_stride;
    const int rows = it.n_tok << a.log_g, keys = it.pos0 + it.n_tok;
    __syncthreads();                         // the item before has read its rows
    stage_rows<D>(sq, [&](int r) -> const float* {
      return r < rows ? q + (it.row0 + (r >> a.log_g)) * a.q_stride +
                            (int64_t)(it.g * a.G + (r & (a.G - 1))) * D
                      : nullptr;
    });
    float m[4], l[4], o[4][4 * NC];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 4 * NC; ++j) o[i][j] = 0.f;
    }

    for (int kt = it.kt0; kt < it.kt1; ++kt) {
      const int u0 = kt * KT;
      // keys past the item's last are zeros: whatever their slots hold stays out of the sums
      auto row_of = [&](const float* pool, int i) -> const float* {
        if (i >= keys - u0) return nullptr;
        const int u = u0 + i;
        const int P = table[u / PS];
        if (P < 0 || P >= d.num_phys_pages) {
          flag(ctx, KV_DEVERR_BAD_PAGE);
          return nullptr;
        }
        return pool + (((int64_t)P * Hkv + it.g) * PS + u % PS) * D;
      };
      __syncthreads();
      stage_rows<D>(sk, [&](int i) { return row_of(kp, i); });
      stage_rows<D>(sv, [&](int i) { return row_of(vp, i); });
      __syncthreads();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = *reinterpret_cast<const float4*>(sq + (ty * 4 + i) * LD + c);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * LD + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
            s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
            s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
            s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
          }
      }
      __syncthreads();                     // the key buffer takes the probabilities
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int last = it.pos0 + ((ty * 4 + i) >> a.log_g);      // the row's last key
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = tx + 16 * j <= last - u0 ? s[i][j] * a.scale_log2 : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float now = fmaxf(m[i], top);
        const float ref = now == -INFINITY ? 0.f : now;     // no key of this row yet
        const float keep = exp2f(m[i] - ref);
        m[i] = now;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(s[i][j] - ref);
          sum += p;
          sk[(ty * 4 + i) * PLD + tx + 16 * j] = p;
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        l[i] = fmaf(l[i], keep, sum);
#pragma unroll
        for (int j = 0; j < 4 * NC; ++j) o[i][j] *= keep;
      }
      __syncwarp();                        // a row's sixteen writers are one half warp
#pragma unroll 4
      for (int u = 0; u < KT; u += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[i] = *reinterpret_cast<const float4*>(sk + (ty * 4 + i) * PLD + u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(sv + (u + e) * LD + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
              o[i][4 * c] = fmaf(w, v.x, o[i][4 * c]);
              o[i][4 * c + 1] = fmaf(w, v.y, o[i][4 * c + 1]);
              o[i][4 * c + 2] = fmaf(w, v.z, o[i][4 * c + 2]);
              o[i][4 * c + 3] = fmaf(w, v.w, o[i][4 * c + 3]);
            }
          }
        }
      }
    }

#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= rows) continue;
      if (it.part >= 0) {
        const int64_t at_part = (int64_t)it.part * a.part_rows + r;
        float* acc = a.part_acc + at_part * D;
#pragma unroll
        for (int c = 0; c < NC; ++c) store4(acc + 64 * c + 4 * tx, o[i] + 4 * c);
        if (tx == 0) {
          a.part_ml[2 * at_part] = m[i];
          a.part_ml[2 * at_part + 1] = l[i];
        }
        continue;
      }
      const int64_t row = (int64_t)(it.row0 + (r >> a.log_g)) * a.Hq + it.g * a.G + (r & (a.G - 1));
      const float inv = 1.f / l[i];                 // every row sees its own token: l > 0
#pragma unroll
      for (int j = 0; j < 4 * NC; ++j) o[i][j] *= inv;
      float* dst = static_cast<float*>(a.out) + row * D;
#pragma unroll
      for (int c = 0; c < NC; ++c) store4(dst + 64 * c + 4 * tx, o[i] + 4 * c);
      if (tx == 0 && a.lse != nullptr) a.lse[row] = (m[i] + log2f(l[i])) * kLn2;
    }
  }
}

template <int D>
cudaError_t launch_t(const kv_cache_desc& d, const PackedRows& pr, const PrefillArgs& a,
                     DevCtx ctx, cudaStream_t s) {
  auto kern = prefill_simt_kernel<D>;
  const size_t smem = SimtCfg<D>::SMEM;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.NC), dim3(kThreads), smem, s, d, pr, a, ctx);
}

}  // namespace

cudaError_t launch_prefill_simt(const kv_cache_desc& d, const PackedRows& pr,
                                const PrefillArgs& a, DevCtx ctx, cudaStream_t s) {
  return d.head_dim == 128 ? launch_t<128>(d, pr, a, ctx, s) : launch_t<64>(d, pr, a, ctx, s);
}

}  // namespace skv
