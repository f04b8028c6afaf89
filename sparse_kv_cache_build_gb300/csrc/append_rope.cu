// Packed append with the rotary position applied on the way.
//
// A step's new tokens (whole prompts, chunks of prompts, or one token per sequence) arrive as
// packed rows of queries, keys and values. Token i of sequence b's n_b goes to position
// t = len_b - n_b + i. For each pair j of the first rot_dim columns
//   (u, w) = (a cos x - b sin x, a sin x + b cos x),  x = pos * inv_freq_j,
// with (a, b) = columns (j, j + rot_dim/2), or (2j, 2j + 1) when interleaved. Queries go to
// q_out, keys and values to their slots, and the min/max statistics of every page touched
// follow from the stored keys alone, as kv_append_token keeps them for one token.
//
// Angles: the frequency is held in turns as a 64-bit fraction, so pos * turns modulo 2^64 is
// the fraction of a turn exactly, however far the position. Its leading 32 bits less the nearest
// quarter turn become a float for sincospif, off by 2^-28 of a turn (2.3e-8 rad, below half a
// step of the float sine). A product in 32-bit floats would be off by 2^-24 of the whole angle
// (0.06 rad at position 10^6).
//
// Rounding: the rotation is done in float32 and rounded once to the cache's type; the
// statistics are taken over the rounded keys, as a rebuild from the pool would.
//
// Bound: every row is read once and written once, so the floor is memory. A lane owns 16
// columns of a row as two 16-byte (bf16) chunks that hold eight whole pairs, so no exchange
// between lanes is needed and D/16 lanes cover a row; a warp moves 512/D rows at once. One
// block per (page, KV head) lets the page's statistics be joined inside the block, without
// atomics. Measured, bf16, D = 128: ragged prompts of 64/8 heads in pages of 64 tokens (545 MB)
// 88.2 us, 6.2 TB/s, 91% of the measured copy rate; a prompt of 8192 tokens of 32/8 heads in pages
// of 16 (203 MB) 40.2 us, 5.0 TB/s, as each of the small blocks pays for finding its page. 32
// single tokens take 5 us on the device, three dependent reads long; the call costs the host
// 13 to 15. Bounds of four or five blocks per SM on the registers gave nothing.
#include "packed_rows.cuh"

namespace skv {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr long kManyRows = 8192;       // (token, KV head) pairs

struct RopeArgs {
  const void* q; const void* k; const void* v;      // packed rows
  int64_t q_stride, k_stride, v_stride;             // elements between tokens
  void* q_out; int64_t q_out_stride;
  const int32_t* positions;                         // NULL: the cache position
  const uint64_t* turns;                            // [rot_dim / 2]
  void* stats;
  int Hq, rot;
};

// Sixteen columns of a row as floats: two chunks of eight.
struct Cols { float a[8], b[8]; };

// Rounds to the storage type (to nearest even) and leaves the rounded values in f.
template <typename T> __device__ __forceinline__ void store8(T* p, float* f);
template <> __device__ __forceinline__ void store8<bf16_t>(bf16_t* p, float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ void store8<float>(float* p, float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// The two chunks of lane c of a row and, when they rotate, the first of their eight pairs.
// Half-split pairs join chunk c with chunk c + rot/16; interleaved pairs lie inside chunks
// 2c and 2c + 1; columns from rot on pass through.
template <bool INTER>
__device__ __forceinline__ void lane_chunks(int c, int rot, int* ca, int* cb, bool* turns) {
  *turns = 16 * c < rot;
  *ca = !INTER && *turns ? 8 * c : 16 * c;
  *cb = !INTER && *turns ? 8 * c + rot / 2 : 16 * c + 8;
}

struct Angle { float cos[8], sin[8]; };

__device__ __forceinline__ void angles_at(const uint64_t* f, int pos, Angle* x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t turn = (uint32_t)((f[e] * (uint64_t)(int64_t)pos) >> 32);   // modulo one turn
    // the nearest quarter turn, and what is left of it: at most 2^29 of these units, so the
    // float is off by 2^-28 of a turn (of the whole signed fraction it would be 2^-26)
    const uint32_t quarter = (turn + (1u << 29)) >> 30;
    float s, c;
    sincospif((float)(int32_t)(turn - (quarter << 30)) * 0x1p-31f, &s, &c);
    const float a = quarter & 1u ? s : c, b = quarter & 1u ? c : s;
    x->cos[e] = __uint_as_float(__float_as_uint(a) ^ ((quarter + 1u) & 2u) << 30);
    x->sin[e] = __uint_as_float(__float_as_uint(b) ^ (quarter & 2u) << 30);
  }
}

template <bool INTER>
__device__ __forceinline__ void rotate(Cols* r, const Angle& x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float& a = INTER ? (e < 4 ? r->a[2 * e] : r->b[2 * e - 8]) : r->a[e];
    float& b = INTER ? (e < 4 ? r->a[2 * e + 1] : r->b[2 * e - 7]) : r->b[e];
    const float u = a * x.cos[e] - b * x.sin[e];
    const float w = a * x.sin[e] + b * x.cos[e];
    a = u;
    b = w;
  }
}

// A lane's sixteen columns as they lie in memory: loads of several rows are issued before the
// first is unpacked.
template <typename T> struct Raw {
  static constexpr int N = 8 * sizeof(T) / 16;       // 16-byte loads per chunk
  uint4 a[N], b[N];
};
template <typename T>
__device__ __forceinline__ void load_raw(const void* base, int64_t at, int ca, int cb,
                                         Raw<T>* r) {
  const T* p = static_cast<const T*>(base) + at;
#pragma unroll
  for (int i = 0; i < Raw<T>::N; ++i) {
    r->a[i] = reinterpret_cast<const uint4*>(p + ca)[i];
    r->b[i] = reinterpret_cast<const uint4*>(p + cb)[i];
  }
}
template <typename T> __device__ __forceinline__ void unpack(const Raw<T>& r, Cols* c) {
#pragma unroll
  for (int i = 0; i < Raw<T>::N; ++i) {
    chunk_to_f32<T>(r.a[i], c->a + 8 / Raw<T>::N * i);
    chunk_to_f32<T>(r.b[i], c->b + 8 / Raw<T>::N * i);
  }
}
template <typename T>
__device__ __forceinline__ void load_cols(const void* base, int64_t at, int ca, int cb, Cols* c) {
  Raw<T> r;
  load_raw<T>(base, at, ca, cb, &r);
  unpack<T>(r, c);
}
template <typename T>
__device__ __forceinline__ void store_cols(void* base, int64_t at, int ca, int cb, Cols* r) {
  T* p = static_cast<T*>(base) + at;
  store8<T>(p + ca, r->a);
  store8<T>(p + cb, r->b);
}

template <typename T> __device__ __forceinline__ void store_stat(T* p, float v);
template <> __device__ __forceinline__ void store_stat<bf16_t>(bf16_t* p, float v) {
  p->bits = (uint16_t)(__float_as_uint(v) >> 16);             // exact: v is a bf16 value
}
template <> __device__ __forceinline__ void store_stat<float>(float* p, float v) { *p = v; }

// Folds a key's extremes into a page's: a value replaces the old one only when strictly
// smaller (larger), the rule of the full build.
__device__ __forceinline__ float lower(float a, float b) { return b < a ? b : a; }
__device__ __forceinline__ float upper(float a, float b) { return b > a ? b : a; }

// ------------------------------------------------------------------------------------
// Prompts and chunks: one block per (page touched, KV head).
// ------------------------------------------------------------------------------------
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
append_rope_kernel(kv_cache_desc d, PackedRows pr, RopeArgs a, DevCtx ctx) {
  constexpr int LPR = D / 16;            // lanes per row
  constexpr int RPW = 32 / LPR;          // rows per warp step
  constexpr int HEADS = sizeof(T) == 2 ? 4 : 2;      // query rows in flight per lane
  __shared__ float sh_mn[kRopeWarps][D], sh_mx[kRopeWarps][D];
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0) check_packed_rows(ctx, d, pr);
  // heads vary fastest: blocks that run at the same time read neighbouring columns of the same
  // token rows
  const int PS = d.page_size, Hkv = d.num_kv_heads;
  const int g = blockIdx.x % Hkv, item = blockIdx.x / Hkv;
  int base;
  const int b = find_sequence(pr, d.batch, PS, item, &base);
  const SeqRows sr = seq_rows(ctx, d, pr, b);
  const int start = sr.len - sr.n;
  // item < base only where the offsets fall or do not start at zero: that is nobody's number
  const int page = start / PS + (item - base);
  if (sr.n == 0 || item < base || (int64_t)page * PS >= sr.len) return;
  const int t0 = max(start, page * PS), t1 = min(sr.len - page * PS, PS) + page * PS;
  const int P = d.page_table[(long)b * d.page_table_stride + page];
  const bool mapped = P >= 0 && P < d.num_phys_pages;
  if (!mapped && threadIdx.x == 0) flag(ctx, KV_DEVERR_BAD_PAGE);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane / LPR, c = lane % LPR;
  int ca, cb;
  bool turns;
  lane_chunks<INTER>(c, a.rot, &ca, &cb, &turns);
  uint64_t f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = turns ? a.turns[8 * c + e] : 0;
  const int G = a.Hq / Hkv;
  void* kp = const_cast<void*>(d.k_pool);
  void* vp = const_cast<void*>(d.v_pool);

  Cols mn, mx;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mn.a[e] = mn.b[e] = INFINITY;
    mx.a[e] = mx.b[e] = -INFINITY;
  }
  // Columns of the page's first key that are NaN: the full build begins with that key, so they
  // stay NaN, where those of later keys do not count. (Beginning with the key here instead of
  // with infinities costs 0.9 us of 39 and 87, this mask 0.2.)
  uint32_t nan = 0;
  const int warps = blockDim.x >> 5;
  for (int t = t0 + warp * RPW + r; t < t1; t += warps * RPW) {
    const int64_t row = sr.row0 + (t - start);
    Raw<T> rk, rv, rq[HEADS];
    load_raw<T>(a.k, row * a.k_stride + (int64_t)g * D, ca, cb, &rk);
    load_raw<T>(a.v, row * a.v_stride + (int64_t)g * D, ca, cb, &rv);
    const int64_t q_row = row * a.q_stride + (int64_t)g * G * D;
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
      if (h < G) load_raw<T>(a.q, q_row + h * D, ca, cb, &rq[h]);
    Angle x;
    if (turns) angles_at(f, a.positions != nullptr ? a.positions[row] : t, &x);
    if (mapped) {
      Cols k, v;
      unpack<T>(rk, &k);
      unpack<T>(rv, &v);
      if (turns) rotate<INTER>(&k, x);
      const int64_t slot = (((int64_t)P * Hkv + g) * PS + (t - page * PS)) * D;
      store_cols<T>(kp, slot, ca, cb, &k);
      store_cols<T>(vp, slot, ca, cb, &v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        mn.a[e] = lower(mn.a[e], k.a[e]);
        mn.b[e] = lower(mn.b[e], k.b[e]);
        mx.a[e] = upper(mx.a[e], k.a[e]);
        mx.b[e] = upper(mx.b[e], k.b[e]);
      }
      if (t == page * PS) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          nan |= (isnan(k.a[e]) ? 1u << e : 0u) | (isnan(k.b[e]) ? 256u << e : 0u);
      }
    }
    for (int h0 = 0; h0 < G; h0 += HEADS) {
#pragma unroll
      for (int h = 0; h < HEADS; ++h) {
        if (h0 + h >= G) break;
        Cols q;
        unpack<T>(rq[h], &q);
        if (h0 + HEADS + h < G)
          load_raw<T>(a.q, q_row + (int64_t)(h0 + HEADS + h) * D, ca, cb, &rq[h]);
        if (turns) rotate<INTER>(&q, x);
        store_cols<T>(a.q_out, row * a.q_out_stride + (int64_t)(g * G + h0 + h) * D, ca, cb, &q);
      }
    }
  }
  if (!mapped) return;
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mn.a[e] = lower(mn.a[e], __shfl_xor_sync(0xffffffffu, mn.a[e], o));
      mn.b[e] = lower(mn.b[e], __shfl_xor_sync(0xffffffffu, mn.b[e], o));
      mx.a[e] = upper(mx.a[e], __shfl_xor_sync(0xffffffffu, mx.a[e], o));
      mx.b[e] = upper(mx.b[e], __shfl_xor_sync(0xffffffffu, mx.b[e], o));
    }
  }
  if (r == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sh_mn[warp][ca + e] = mn.a[e];
      sh_mn[warp][cb + e] = mn.b[e];
      sh_mx[warp][ca + e] = mx.a[e];
      sh_mx[warp][cb + e] = mx.b[e];
    }
    if (nan != 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (nan >> e & 1u) sh_mn[warp][ca + e] = sh_mx[warp][ca + e] = NAN;
        if (nan >> e & 256u) sh_mn[warp][cb + e] = sh_mx[warp][cb + e] = NAN;
      }
    }
  }
  __syncthreads();
  T* row = static_cast<T*>(a.stats) + ((int64_t)P * Hkv + g) * 2 * D;
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    float lo = sh_mn[0][i], hi = sh_mx[0][i];
    for (int w = 1; w < warps; ++w) {
      lo = lower(lo, sh_mn[w][i]);
      hi = upper(hi, sh_mx[w][i]);
    }
    if (t0 > page * PS) {                // the page held tokens before this call
      lo = lower(load_elem<T>(row, i), lo);
      hi = upper(load_elem<T>(row, D + i), hi);
    }
    store_stat<T>(row + i, lo);
    store_stat<T>(row + D + i, hi);
  }
}

// ------------------------------------------------------------------------------------
// One token per sequence: D/16 lanes per row, every row of the token side by side, so a call
// is one dependent chain (length, page, row) long.
// ------------------------------------------------------------------------------------
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
append_rope_single_kernel(kv_cache_desc d, RopeArgs a, DevCtx ctx) {
  constexpr int LPR = D / 16;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, PS = d.page_size, Hkv = d.num_kv_heads;
  const int task = blockIdx.y * (kRopeThreads / LPR) + threadIdx.x / LPR;
  const int c = threadIdx.x % LPR;
  if (task >= a.Hq + 2 * Hkv) return;
  // tasks: the query heads, then the keys, then the values
  const bool is_q = task < a.Hq, is_v = task >= a.Hq + Hkv;
  const int head = is_q ? task : (task - a.Hq) % Hkv;
  int ca, cb;
  bool turns;
  lane_chunks<INTER>(c, a.rot, &ca, &cb, &turns);
  Cols x;
  load_cols<T>(is_q ? a.q : is_v ? a.v : a.k,
               b * (is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride) + (int64_t)head * D,
               ca, cb, &x);
  const int len = packed_len(ctx, d, b);
  if (len == 0) return;                                    // nothing to append
  if (turns && !is_v) {
    uint64_t f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = a.turns[8 * c + e];
    Angle y;
    angles_at(f, a.positions != nullptr ? a.positions[b] : len - 1, &y);
    rotate<INTER>(&x, y);
  }
  if (is_q) {
    store_cols<T>(a.q_out, b * a.q_out_stride + (int64_t)head * D, ca, cb, &x);
    return;
  }
  const int page = (len - 1) / PS, slot = (len - 1) % PS;
  const int P = d.page_table[(long)b * d.page_table_stride + page];
  if (P < 0 || P >= d.num_phys_pages) {
    flag(ctx, KV_DEVERR_BAD_PAGE);
    return;
  }
  store_cols<T>(const_cast<void*>(is_v ? d.v_pool : d.k_pool),
                (((int64_t)P * Hkv + head) * PS + slot) * D, ca, cb, &x);
  if (is_v) return;
  const int64_t srow = ((int64_t)P * Hkv + head) * 2 * D;
  Cols mn = x, mx = x;
  if (slot > 0) {
    load_cols<T>(a.stats, srow, ca, cb, &mn);
    load_cols<T>(a.stats, srow + D, ca, cb, &mx);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mn.a[e] = lower(mn.a[e], x.a[e]);
      mn.b[e] = lower(mn.b[e], x.b[e]);
      mx.a[e] = upper(mx.a[e], x.a[e]);
      mx.b[e] = upper(mx.b[e], x.b[e]);
    }
  }
  store_cols<T>(a.stats, srow, ca, cb, &mn);
  store_cols<T>(a.stats, srow + D, ca, cb, &mx);
}

template <typename T, int D, bool INTER>
cudaError_t launch_t(const kv_cache_desc& d, const PackedRows& pr, const RopeArgs& a, DevCtx ctx,
                     cudaStream_t s) {
  if (pr.cu == nullptr) {
    const int rows = a.Hq + 2 * d.num_kv_heads;
    dim3 grid(d.batch, ceil_div(rows, kRopeThreads / (D / 16)));
    return launch_pdl(append_rope_single_kernel<T, D, INTER>, grid, dim3(kRopeThreads), 0, s, d,
                      a, ctx);
  }
  const dim3 grid((unsigned)(page_numbers(pr.total, d.batch, d.page_size) * d.num_kv_heads));
  // With many rows a warp takes four steps of its page, so that finding the page is paid for by
  // more rows (pages of 16 at D = 128 are one warp's: 8192 tokens of 32/8 heads 43.7 us, against
  // 48.1 us with a warp per step). With few, a warp per step makes the call shorter (128 and 512
  // tokens 9.0 us, against 11.0 us); at 1024 tokens the two are equal.
  const int steps = d.page_size * (D / 16) / 32;
  const bool many = (long)pr.total * d.num_kv_heads >= kManyRows;
  const int warps = many ? (steps + 3) / 4 : steps < kRopeWarps ? steps : kRopeWarps;
  return launch_pdl(append_rope_kernel<T, D, INTER>, grid, dim3(32 * warps), 0, s, d, pr, a, ctx);
}

template <typename T, int D>
cudaError_t launch_d(const kv_cache_desc& d, const PackedRows& pr, const RopeArgs& a, bool inter,
                     DevCtx ctx, cudaStream_t s) {
  return inter ? launch_t<T, D, true>(d, pr, a, ctx, s) : launch_t<T, D, false>(d, pr, a, ctx, s);
}

}  // namespace

cudaError_t launch_append_rope(const kv_cache_desc& d, const int32_t* cu, int total,
                               const void* q, int64_t q_stride, int Hq, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride,
                               const int32_t* positions, const uint64_t* turns, int rot,
                               bool interleaved, void* q_out, int64_t q_out_stride, void* stats,
                               DevCtx ctx, cudaStream_t s) {
  const PackedRows pr{cu, total};
  const RopeArgs a{q, k, v, q_stride, k_stride, v_stride, q_out, q_out_stride, positions, turns,
                   stats, Hq, rot};
  if (d.dtype == KV_BF16)
    return d.head_dim == 128 ? launch_d<bf16_t, 128>(d, pr, a, interleaved, ctx, s)
                             : launch_d<bf16_t, 64>(d, pr, a, interleaved, ctx, s);
  return d.head_dim == 128 ? launch_d<float, 128>(d, pr, a, interleaved, ctx, s)
                           : launch_d<float, 64>(d, pr, a, interleaved, ctx, s);
}

}  // namespace skv
