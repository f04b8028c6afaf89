// Causal prompt attention for fp32 caches, on the CUDA cores.
//
// A block takes 128 rows of an item and walks their keys 64 at a time, with the running maximum
// and sum of the softmax per row; it walks its share of the batch's items (prefill.cuh).
//
// What bounds it is the float32 multiply-add rate (two tiles of 128 x 64 x D products a step),
// so everything else is kept off the issue slots. 256 threads hold 8 x 4 of the 128 x 64 scores
// and 8 x D/16 of the output each, so that twelve 16-byte reads of shared memory feed 128
// multiply-adds, issued as packed pairs. Scores pair the even and odd columns of the head (two
// partial sums, joined at the end), the output pairs neighbouring columns. Rows are padded by
// four floats so that the sixteen keys of a warp's read fall into different banks. The
// probabilities take the place of the key tile just used; the next tiles arrive by asynchronous
// copies meanwhile.
//
// Measured: 4096 tokens of 8 query over 2 KV heads, D = 64: 491 us, 35 TFLOP/s (the causal
// multiply-adds alone would take 230 at one per lane and clock). Reads of shared memory keep
// their pipe 70% busy and the multiply-adds theirs 55%; 512 threads with 8 x 2 scores each, for
// more warps to hide the one under the other, took 515. Tensor cores would take six bf16
// products for each float32 product to keep its precision: 53 us of them for that call at the
// measured rate of the library product, so it is not the arithmetic that speaks against them; such
// a kernel has not been built.
//
// Every item computes 128 rows, however few it has, so single tokens cost as much as rows for 128:
// 16 single tokens over 4096 each take 131 us at 8/2 heads of 64 and 846 at 32/8 heads of 128
// (the bytes: 10 and 79), one over 32768 422 (40). kv_decode_step reads them at 18, 99 and 46, and
// is the call for float32 caches there; a form for few rows has not been built.
#include "prefill.cuh"
#include "tcgen05.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int R = SimtShape::rows, KT = SimtShape::keys;
constexpr int RPT = R / 16, KPT = KT / 16;           // rows and keys of a thread

template <int D> struct SimtCfg {
  static constexpr int LD = D + 4;                   // padded row, floats
  static constexpr size_t SMEM = sizeof(float) * ((R + 4 * KT) * LD + (D == 64 ? R * KT : 0));
  static_assert(D == 64 || R * KT <= KT * LD, "the probabilities fit the key tile");
};

__device__ __forceinline__ void copy16(float* dst, const float* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               ::"r"(smem_addr(dst)), "l"(src), "r"(have ? 16 : 0) : "memory");
}

// Copies `rows` rows of D elements into padded shared rows; row(i) gives the source of row i, or
// NULL for zeros.
template <int D, typename F>
__device__ __forceinline__ void stage_rows(float* dst, int rows, const float* any, F row) {
  constexpr int CPR = D / 4;                         // 16-byte chunks of a row
  for (int i = threadIdx.x; i < rows * CPR; i += kThreads) {
    const int r = i / CPR, c = (i % CPR) * 4;
    const float* src = row(r);
    copy16(dst + r * SimtCfg<D>::LD + c, src != nullptr ? src + c : any, src != nullptr);
  }
}

__device__ __forceinline__ float2 lo(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi(float4 v) { return make_float2(v.z, v.w); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prefill_simt_kernel(const __grid_constant__ kv_cache_desc d, const __grid_constant__ PackedRows pr,
                    const __grid_constant__ PrefillArgs a, const __grid_constant__ DevCtx ctx) {
  constexpr int LD = SimtCfg<D>::LD, NC = D / 64;
  extern __shared__ __align__(16) float sm[];
  __shared__ LineScratch scratch;
  float* sq = sm;
  float* ring = sq + R * LD;                 // K, V, K, V
  float* own_p = ring + 4 * KT * LD;         // at D = 64; over the K tile at D = 128
  pdl_trigger();
  pdl_wait();
  finish_empty<float, D>(ctx, d, pr, a);
  const LinePlace at = find_place<SimtShape>(ctx, d, pr, a, blockIdx.x, &scratch);
  const int64_t lo_place = at.lo, hi_place = at.hi;
  if (at.total == 0) {
    if (threadIdx.x == 0 && a.notes != nullptr) a.notes[blockIdx.x] = BorderNote{0, 0, 0, 0, 0, 0};
    return;
  }
  ItemWalk<SimtShape> walk(d, pr, a, ctx, lo_place, hi_place, at.b, at.before, blockIdx.x);
  if (threadIdx.x == 0 && a.notes != nullptr) a.notes[blockIdx.x] = walk.border();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int Hkv = d.num_kv_heads, PS = d.page_size;
  const float* q = static_cast<const float*>(a.q);
  const float* kp = static_cast<const float*>(d.k_pool);
  const float* vp = static_cast<const float*>(d.v_pool);
  const int turn = 16 * (ty & 1);            // the two rows of a warp's read in different banks

  PrefillItem it;
  while (walk.next(&it)) {
    const int32_t* table = d.page_table + (int64_t)it.b * d.page_table_stride;
    const int rows = it.n_tok << a.log_g, keys = it.pos0 + it.n_tok;
    // keys past the item's last are zeros: whatever their slots hold stays out of the sums
    auto stage_tile = [&](int kt, int buf) {
      const int u0 = kt * KT;
      float* dst = ring + 2 * buf * KT * LD;
      for (int which = 0; which < 2; ++which) {
        const float* pool = which == 0 ? kp : vp;
        stage_rows<D>(dst + which * KT * LD, KT, pool, [&](int i) -> const float* {
          if (i >= keys - u0) return nullptr;
          const int u = u0 + i;
          const int P = table[u / PS];
          if (P < 0 || P >= d.num_phys_pages) {
            flag(ctx, KV_DEVERR_BAD_PAGE);
            return nullptr;
          }
          return pool + (((int64_t)P * Hkv + it.g) * PS + u % PS) * D;
        });
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    stage_rows<D>(sq, R, q, [&](int r) -> const float* {
      return r < rows ? q + (it.row0 + (r >> a.log_g)) * a.q_stride +
                            (int64_t)(it.g * a.G + (r & (a.G - 1))) * D
                      : nullptr;
    });
    stage_tile(it.kt0, 0);
    float m[RPT], l[RPT];
    float2 o[RPT][2 * NC];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 2 * NC; ++j) o[i][j] = make_float2(0.f, 0.f);
    }

    for (int kt = it.kt0; kt < it.kt1; ++kt) {
      const int buf = (kt - it.kt0) & 1, u0 = kt * KT;
      if (kt + 1 < it.kt1) {
        stage_tile(kt + 1, buf ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
      const float* sk = ring + 2 * buf * KT * LD;
      const float* sv = sk + KT * LD;
      float* sp = D == 128 ? ring + 2 * buf * KT * LD : own_p;
      float2 s2[RPT][KPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < KPT; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 y[KPT];
#pragma unroll
        for (int j = 0; j < KPT; ++j)
          y[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * LD + c);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(sq + (ty * RPT + i) * LD + c);
#pragma unroll
          for (int j = 0; j < KPT; ++j) {
            s2[i][j] = tc::fma2(lo(x), lo(y[j]), s2[i][j]);
            s2[i][j] = tc::fma2(hi(x), hi(y[j]), s2[i][j]);
          }
        }
      }
      if (D == 128) __syncthreads();         // the key tile's buffer takes the probabilities
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int row = ty * RPT + i;
        const int last = it.pos0 + (row >> a.log_g);        // the row's last key
        float s[KPT], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
          s[j] = (s2[i][j].x + s2[i][j].y) * a.scale_log2;
          if (tx + 16 * j > last - u0) s[j] = -INFINITY;
          top = fmaxf(top, s[j]);
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float now = fmaxf(m[i], top);
        const float ref = now == -INFINITY ? 0.f : now;     // no key of this row yet
        const float keep = exp2f(m[i] - ref);
        m[i] = now;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
          const float p = exp2f(s[j] - ref);
          sum += p;
          sp[row * KT + ((tx + 16 * j + turn) & (KT - 1))] = p;
        }
        l[i] = fmaf(l[i], keep, sum);        // this thread's keys only: joined at the end
#pragma unroll
        for (int j = 0; j < 2 * NC; ++j) {
          o[i][j].x *= keep;
          o[i][j].y *= keep;
        }
      }
      __syncwarp();                          // a row's sixteen writers are one half warp
#pragma unroll 2
      for (int u = 0; u < KT; u += 4) {
        float4 p[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
          p[i] = *reinterpret_cast<const float4*>(sp + (ty * RPT + i) * KT +
                                                  ((u + turn) & (KT - 1)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float4 v[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c)
            v[c] = *reinterpret_cast<const float4*>(sv + (u + e) * LD + 64 * c + 4 * tx);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float w = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
            const float2 ww = make_float2(w, w);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              o[i][2 * c] = tc::fma2(ww, lo(v[c]), o[i][2 * c]);
              o[i][2 * c + 1] = tc::fma2(ww, hi(v[c]), o[i][2 * c + 1]);
            }
          }
        }
      }
      __syncthreads();                       // this tile's buffers may be filled again
    }

#pragma unroll
    for (int i = 0; i < RPT; ++i) {
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
      const int r = ty * RPT + i;
      if (r >= rows) continue;
      if (it.part >= 0) {
        const int64_t at_part = (int64_t)it.part * a.part_rows + r;
        float* acc = a.part_acc + at_part * D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          *reinterpret_cast<float4*>(acc + 64 * c + 4 * tx) =
              make_float4(o[i][2 * c].x, o[i][2 * c].y, o[i][2 * c + 1].x, o[i][2 * c + 1].y);
        if (tx == 0) {
          a.part_ml[2 * at_part] = m[i];
          a.part_ml[2 * at_part + 1] = l[i];
        }
        continue;
      }
      const int64_t out_row = (int64_t)(it.row0 + (r >> a.log_g)) * a.Hq + it.g * a.G +
                              (r & (a.G - 1));
      const float inv = 1.f / l[i];                 // every row sees its own token: l > 0
      float* dst = static_cast<float*>(a.out) + out_row * D;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        *reinterpret_cast<float4*>(dst + 64 * c + 4 * tx) =
            make_float4(o[i][2 * c].x * inv, o[i][2 * c].y * inv, o[i][2 * c + 1].x * inv,
                        o[i][2 * c + 1].y * inv);
      if (tx == 0 && a.lse != nullptr) a.lse[out_row] = (m[i] + log2f(l[i])) * kLn2;
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
