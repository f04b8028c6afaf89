// Attention of few rows (single tokens in a window, trees) for fp32 caches, on the CUDA cores.
//
// As prefill_simt.cuh, whose items have 128 rows however few are used; here they have 32 (32 / G
// tokens of one KV head). So that a thread's reads of shared memory still feed as many
// multiply-adds (twelve 16-byte reads to 128), a thread keeps 8 x 4 scores, over a quarter of the
// head's columns, and 8 x D/16 of the output, over a quarter of the tile's keys. The quarters of
// the scores meet in shared memory, where eight threads share a row's softmax; those of the output
// meet once, at the item's end.
//
// What bounds it: reads of shared memory and four barriers a tile; an unused group of eight rows
// costs nothing. Measured, 16 sequences in a window of 4000, 32/8 heads of 128: one row to a
// sequence (four with its heads) 262 us, eight 288, where items of 128 rows take 798 and the
// bytes 79; 64 rows to a sequence 543 against 801, 124 rows 1039 against 807.
#pragma once

#include "prefill_simt.cuh"

namespace skv {
namespace {

template <int D> struct SimtFewCfg {
  static constexpr int R = SimtFewShape::rows, KT = SimtFewShape::keys;
  static constexpr int LD = D + 4;                   // padded row, floats
  static constexpr int SLD = KT + 2, PLD = KT + 4;   // of a quarter's scores, of the probabilities
  static constexpr int OFF_RING = R * LD;            // floats
  static constexpr int OFF_PART = OFF_RING + 4 * KT * LD;
  static constexpr int OFF_P = OFF_PART + 4 * R * SLD;
  static constexpr int OFF_ROW = OFF_P + R * PLD;    // per row: what the sums change by, m, l
  static constexpr int OFF_LINE = OFF_ROW + 3 * R;
  static constexpr size_t SMEM = sizeof(float) * (OFF_LINE + R * (kTreeNodes / 32));
  static_assert(4 * R * D <= 4 * KT * LD, "the quarters of the output fit the tiles' buffers");
};

template <int D, Mask M>
__global__ void __launch_bounds__(kThreads, 1)
prefill_simt_few_kernel(const __grid_constant__ kv_cache_desc d,
                        const __grid_constant__ PackedRows pr,
                        const __grid_constant__ PrefillArgs a, const __grid_constant__ DevCtx ctx) {
  using C = SimtFewCfg<D>;
  using Shape = SimtFewShape::With<M>;
  constexpr int LD = C::LD, NC = D / 64, WORDS = kTreeNodes / 32;
  constexpr int R = C::R, KT = C::KT, RPT = 8, KPT = 4;
  extern __shared__ __align__(16) float sm[];
  __shared__ LineScratch scratch;
  float* sq = sm;
  float* ring = sm + C::OFF_RING;            // K, V, K, V; at an item's end the output's quarters
  float* part = sm + C::OFF_PART;            // [4][R][SLD]
  float* sp = sm + C::OFF_P;                 // [R][PLD]
  float* change = sm + C::OFF_ROW;           // [R]
  float* row_m = change + R;
  float* row_l = row_m + R;
  uint32_t* line = reinterpret_cast<uint32_t*>(sm + C::OFF_LINE);
  pdl_trigger();
  pdl_wait();
  finish_empty<float, D>(ctx, d, pr, a);
  const LinePlace at = find_place<Shape>(ctx, d, pr, a, blockIdx.x, &scratch);
  if (at.total == 0) {
    if (threadIdx.x == 0 && a.notes != nullptr) a.notes[blockIdx.x] = BorderNote{0, 0, 0, 0, 0, 0};
    return;
  }
  ItemWalk<Shape> walk(d, pr, a, ctx, at.lo, at.hi, at.b, at.before, blockIdx.x);
  if (threadIdx.x == 0 && a.notes != nullptr) a.notes[blockIdx.x] = walk.border();
  const int tid = threadIdx.x, tx = tid & 15, ty = (tid >> 4) & 3, quarter = tid >> 6;
  const int own_row = tid >> 3, own_key = (tid & 7) * 8;         // of the softmax
  const int Hkv = d.num_kv_heads, PS = d.page_size;
  const float* q = static_cast<const float*>(a.q);
  const float* kp = static_cast<const float*>(d.k_pool);
  const float* vp = static_cast<const float*>(d.v_pool);

  MaskedItem it;
  while (walk.next(&it)) {
    const int32_t* table = d.page_table + (int64_t)it.b * d.page_table_stride;
    const int rows = it.n_tok << a.log_g, keys = it.pos0 + it.n_tok;
    if (M == Mask::kTree && tid < R) {       // row tid's line of ancestors
      const int t0 = it.pos0 - it.past;
      const int32_t* up = a.parents + it.row0 - t0;
      for (int k = 0; k < WORDS; ++k) line[tid * WORDS + (k ^ tid)] = 0;
      for (int v = t0 + min(tid >> a.log_g, it.n_tok - 1); v >= 0;) {
        line[tid * WORDS + (v >> 5 ^ tid)] |= 1u << (v & 31);
        const int next = __ldg(up + v);
        if (next >= v || next < -1) {
          flag(ctx, KV_DEVERR_BAD_SEL);
          break;
        }
        v = next;
      }
    }
    // A thread copies the same columns of every RSTEP-th key, of K and V alike; keys past the
    // item's last are zeros: whatever their slots hold stays out of the sums.
    auto stage_tile = [&](int kt, int buf) {
      constexpr int CPR = D / 4, RSTEP = kThreads / CPR, N = KT / RSTEP;
      const int c = tid % CPR * 4, u0 = kt * KT + tid / CPR;
      float* dst = ring + 2 * buf * KT * LD + tid / CPR * LD + c;
      int P[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        int p = (u0 + i * RSTEP) >> a.page_log;
        if constexpr (M == Mask::kWindow) p += p < a.sink_pages ? 0 : it.skip;
        P[i] = u0 + i * RSTEP < keys ? __ldg(table + p) : 0;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = u0 + i * RSTEP;
        bool have = u < keys;
        if (have && (P[i] < 0 || P[i] >= d.num_phys_pages)) {
          flag(ctx, KV_DEVERR_BAD_PAGE);
          have = false;
        }
        const int64_t from =
            have ? ((((int64_t)P[i] * Hkv + it.g) << a.page_log) + (u & (PS - 1))) * D + c : 0;
        copy16(dst + i * RSTEP * LD, kp + from, have);
        copy16(dst + (KT + i * RSTEP) * LD, vp + from, have);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    stage_rows<D>(sq, R, q, [&](int r) -> const float* {
      return r < rows ? q + (it.row0 + (r >> a.log_g)) * a.q_stride +
                            (int64_t)(it.g * a.G + (r & (a.G - 1))) * D
                      : nullptr;
    });
    stage_tile(it.kt0, 0);
    float m = -INFINITY, l = 0.f;            // of own_row, l over this thread's keys
    const int last = it.pos0 + (own_row >> a.log_g);
    float2 o[RPT][2 * NC];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < 2 * NC; ++j) o[i][j] = make_float2(0.f, 0.f);

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
      const int busy = (rows + RPT - 1) / RPT;           // groups of eight rows in use
      if (ty < busy) {
        float2 s2[RPT][KPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int j = 0; j < KPT; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = quarter * (D / 4); c < (quarter + 1) * (D / 4); c += 4) {
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
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int j = 0; j < KPT; ++j)
            part[(quarter * R + ty * RPT + i) * C::SLD + tx + 16 * j] = s2[i][j].x + s2[i][j].y;
      }
      __syncthreads();
      if (own_row < rows) {
        float s[8], top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float2 x = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x = tc::add2(x, *reinterpret_cast<const float2*>(
                                part + (k * R + own_row) * C::SLD + own_key + e));
          s[e] = x.x * a.scale_log2;
          s[e + 1] = x.y * a.scale_log2;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int u = u0 + own_key + e;
          bool sees = u <= last;
          if (M == Mask::kWindow) sees = sees && (last - u < a.window || u < a.sinks);
          if (M == Mask::kTree && sees && u >= it.past)
            sees = line[own_row * WORDS + ((u - it.past) >> 5 ^ own_row)] >> ((u - it.past) & 31) &
                   1u;
          if (!sees) s[e] = -INFINITY;
          top = fmaxf(top, s[e]);
        }
        const uint32_t eight = 0xffu << (tid & 24);      // a row's lanes
#pragma unroll
        for (int w = 4; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(eight, top, w));
        const float now = fmaxf(m, top);
        const float ref = now == -INFINITY ? 0.f : now;  // no key of this row yet
        const float keep = exp2f(m - ref);
        m = now;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[e] = exp2f(s[e] - ref);
          sum += s[e];
        }
        l = fmaf(l, keep, sum);
        float4* dst = reinterpret_cast<float4*>(sp + own_row * C::PLD + own_key);
        dst[0] = make_float4(s[0], s[1], s[2], s[3]);
        dst[1] = make_float4(s[4], s[5], s[6], s[7]);
        if ((tid & 7) == 0) change[own_row] = keep;
      }
      __syncthreads();
      if (ty < busy) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const float f = ty * RPT + i < rows ? change[ty * RPT + i] : 0.f;
#pragma unroll
          for (int j = 0; j < 2 * NC; ++j) {
            o[i][j].x *= f;
            o[i][j].y *= f;
          }
        }
#pragma unroll 1
        for (int u = quarter * (KT / 4); u < (quarter + 1) * (KT / 4); u += 4) {
          float4 p[RPT];
#pragma unroll
          for (int i = 0; i < RPT; ++i)
            p[i] = *reinterpret_cast<const float4*>(sp + (ty * RPT + i) * C::PLD + u);
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
      }
      __syncthreads();                       // this tile's buffers may be filled again
    }

    if (own_row < rows) {
      const uint32_t eight = 0xffu << (tid & 24);
#pragma unroll
      for (int w = 4; w > 0; w >>= 1) l += __shfl_xor_sync(eight, l, w);
      if ((tid & 7) == 0) {
        row_m[own_row] = m;
        row_l[own_row] = l;
      }
    }
    if (ty * RPT < rows) {
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c)
          *reinterpret_cast<float4*>(ring + (quarter * R + ty * RPT + i) * D + 64 * c + 4 * tx) =
              make_float4(o[i][2 * c].x, o[i][2 * c].y, o[i][2 * c + 1].x, o[i][2 * c + 1].y);
    }
    __syncthreads();
    for (int x = tid; x < rows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), c = x % (D / 4) * 4;
      float4 y = *reinterpret_cast<const float4*>(ring + r * D + c);
#pragma unroll
      for (int k = 1; k < 4; ++k) {
        const float4 z = *reinterpret_cast<const float4*>(ring + (k * R + r) * D + c);
        y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
      }
      if (it.part >= 0) {
        const int64_t at_part = (int64_t)it.part * a.part_rows + r;
        *reinterpret_cast<float4*>(a.part_acc + at_part * D + c) = y;
        if (c == 0) {
          a.part_ml[2 * at_part] = row_m[r];
          a.part_ml[2 * at_part + 1] = row_l[r];
        }
        continue;
      }
      const int64_t out_row = (int64_t)(it.row0 + (r >> a.log_g)) * a.Hq + it.g * a.G +
                              (r & (a.G - 1));
      const float inv = 1.f / row_l[r];      // every row sees its own token: l > 0
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + out_row * D + c) =
          make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      if (c == 0 && a.lse != nullptr) a.lse[out_row] = (row_m[r] + log2f(row_l[r])) * kLn2;
    }
    __syncthreads();                         // the next item's tiles and rows may come
  }
}

template <int D, Mask M>
cudaError_t launch_few_t(const kv_cache_desc& d, const PackedRows& pr, const PrefillArgs& a,
                         DevCtx ctx, cudaStream_t s) {
  auto kern = prefill_simt_few_kernel<D, M>;
  const size_t smem = SimtFewCfg<D>::SMEM;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.NC), dim3(kThreads), smem, s, d, pr, a, ctx);
}

}  // namespace

template <Mask M>
cudaError_t launch_prefill_simt_few(const kv_cache_desc& d, const PackedRows& pr,
                                    const PrefillArgs& a, DevCtx ctx, cudaStream_t s) {
  return d.head_dim == 128 ? launch_few_t<128, M>(d, pr, a, ctx, s)
                           : launch_few_t<64, M>(d, pr, a, ctx, s);
}

}  // namespace skv
