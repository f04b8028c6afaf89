// Kept tokens moved together, in place, and the page statistics of what they leave.
//
// Sequence b's candidates are its last n tokens, from position s = len - n on; the token at
// s + keep[i] moves to s + i, for i = 0 .. cnt - 1 (keep rises, so tokens only move forward). The
// statistics of a page cannot be un-merged, so those of every page from s on are taken anew over
// its tokens, the ones before s too.
//
// In place without a copy: the slot of token i may hold the source of a token j <= i only (keep[j]
// = i means j <= i), so a slot may be written once every source up to it has been read, and what
// later tokens read is never overwritten early. A block owns some 16-byte columns of one KV head's
// keys or values, so blocks need nothing of each other; it walks the tokens in batches, loads the
// next batch, and writes the present one behind a barrier that all its loads are ordered before.
//
// Bound: every moved token is read and written once. A batch costs a block one round of loads, so
// a long list is the columns split further, down to 32 bytes a row (a sector), until there are
// blocks for the whole GPU; a short one, that is a batch at once, is a chain of dependent reads
// (offsets, list, table, token, statistics).
#include "packed_rows.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;              // tokens of a thread in a batch
constexpr int kMinLanes = 2;           // 16-byte columns of a block: at least a sector
constexpr int kBlocksPerSM = 2;

struct CompactArgs {
  const int32_t* cu;                   // [batch + 1], or NULL: every token is a candidate
  const int32_t* keep;                 // [batch][keep_stride]
  const int32_t* keep_cnt;             // [batch]
  int keep_stride;
  int log_lanes;                       // 16-byte columns of a block
  void* stats;                         // or NULL
  int32_t* new_lens;
};

template <typename T> struct Chunk {
  static constexpr int N = 16 / sizeof(T);
  float f[N];
};
template <typename T> __device__ __forceinline__ Chunk<T> unpack(uint4 v) {
  Chunk<T> c;
  chunk_to_f32<T>(v, c.f);
  return c;
}
// The floats hold values of the cache's type exactly.
template <typename T> __device__ __forceinline__ uint4 pack(const Chunk<T>& c) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (__float_as_uint(c.f[2 * i]) >> 16) | (__float_as_uint(c.f[2 * i + 1]) & 0xffff0000u);
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    return make_uint4(__float_as_uint(c.f[0]), __float_as_uint(c.f[1]), __float_as_uint(c.f[2]),
                      __float_as_uint(c.f[3]));
  }
}

// A value replaces the extreme so far only when strictly smaller (larger): the full build's rule.
template <typename T> __device__ __forceinline__ void fold(Chunk<T>* mn, Chunk<T>* mx,
                                                           const Chunk<T>& lo, const Chunk<T>& hi) {
#pragma unroll
  for (int e = 0; e < Chunk<T>::N; ++e) {
    mn->f[e] = lo.f[e] < mn->f[e] ? lo.f[e] : mn->f[e];
    mx->f[e] = hi.f[e] > mx->f[e] ? hi.f[e] : mx->f[e];
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
compact_kernel(const __grid_constant__ kv_cache_desc d, const __grid_constant__ CompactArgs a,
               const __grid_constant__ DevCtx ctx) {
  constexpr int ROW = D * sizeof(T) / 16;            // 16-byte columns of a token
  __shared__ Chunk<T> sh_mn[kThreads], sh_mx[kThreads];
  pdl_trigger();
  pdl_wait();
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int parts = ROW >> a.log_lanes;
  const bool values = (int)blockIdx.x >= parts;
  const int col = (((int)blockIdx.x - (values ? parts : 0)) << a.log_lanes) +
                  (tid & ((1 << a.log_lanes) - 1));
  const int row = tid >> a.log_lanes, rows = kThreads >> a.log_lanes;
  const int PS = d.page_size, Hkv = d.num_kv_heads;
  const bool first_block = blockIdx.x == 0 && g == 0;

  SeqRows s;
  if (a.cu != nullptr) {
    s = seq_rows(ctx, d, PackedRows{a.cu, INT32_MAX}, b);
    if (first_block && b == 0 && tid == 0 && a.cu[0] != 0) flag(ctx, KV_DEVERR_BAD_LEN);
  } else {
    s.row0 = 0;
    s.len = s.n = packed_len(ctx, d, b);
  }
  const int n = s.n, start = s.len - n;
  int cnt = a.keep_cnt[b];
  const bool bad = cnt < 0 || cnt > n || cnt > a.keep_stride;
  if (bad && tid == 0) flag(ctx, KV_DEVERR_BAD_SEL);
  const int fresh = bad ? s.len : start + cnt;
  if (first_block && tid == 0) a.new_lens[b] = fresh;
  if (bad || n == 0) return;

  const int32_t* table = d.page_table + (int64_t)b * d.page_table_stride;
  const int32_t* keep = a.keep + (int64_t)b * a.keep_stride;
  uint4* pool = static_cast<uint4*>(const_cast<void*>(values ? d.v_pool : d.k_pool)) + col;
  // 16-byte index of a token's column, or -1 where its page is unmapped
  auto place = [&](int t) -> int64_t {
    const int P = __ldg(table + t / PS);
    if (P >= 0 && P < d.num_phys_pages) return (((int64_t)P * Hkv + g) * PS + t % PS) * ROW;
    flag(ctx, KV_DEVERR_BAD_PAGE);
    return -1;
  };
  struct Batch {
    int64_t to[kSteps];                              // -1: nothing to move
    uint4 v[kSteps];
  };
  auto load = [&](int i0, Batch* x) {
    int64_t from[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int i = i0 + u * rows + row;
      from[u] = x->to[u] = -1;
      if (i >= cnt) continue;
      const int k = __ldg(keep + i);
      // rising from k >= i on, and inside the candidates
      if (k < i || k >= n || (i > 0 && __ldg(keep + i - 1) >= k)) {
        flag(ctx, KV_DEVERR_BAD_SEL);
        continue;
      }
      if (k == i) continue;
      from[u] = place(start + k);
      x->to[u] = from[u] < 0 ? -1 : place(start + i);
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
      if (x->to[u] >= 0) x->v[u] = __ldcg(pool + from[u]);
  };
  Batch now, next;
  load(0, &now);
  for (int i0 = 0; i0 < cnt; i0 += kSteps * rows) {
    load(i0 + kSteps * rows, &next);
    __syncthreads();                                 // every source up to here has been read
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
      if (now.to[u] >= 0) pool[now.to[u]] = now.v[u];
    now = next;
  }
  if (values || a.stats == nullptr) return;
  __syncthreads();

  // Statistics: `share` threads per page and column take every share-th token, as many as the
  // pages leave free.
  const int p0 = start / PS, pages = fresh > p0 * PS ? (fresh - 1) / PS - p0 + 1 : 0;
  int share = 1;
  while (2 * share * pages <= rows && 2 * share <= PS) share *= 2;
  const int at_once = rows / share, mine = row / share, sub = row % share;
  for (int q = 0; q < pages; q += at_once) {
    const int p = p0 + q + mine;
    const bool have = q + mine < pages;
    const int64_t base = have ? place(p * PS) : -1;
    const int valid = base < 0 ? 0 : min(PS, fresh - p * PS);
    Chunk<T> mn, mx;
#pragma unroll
    for (int e = 0; e < Chunk<T>::N; ++e) {
      mn.f[e] = INFINITY;
      mx.f[e] = -INFINITY;
    }
    // the first key starts the extremes (where it is NaN they stay so), later NaN do not count
    if (sub == 0 && valid > 0) mn = mx = unpack<T>(__ldcg(pool + base));
    for (int t = sub == 0 ? share : sub; t < valid; t += 4 * share) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t + u * share < valid) v[u] = __ldcg(pool + base + (int64_t)(t + u * share) * ROW);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t + u * share < valid) {
          const Chunk<T> c = unpack<T>(v[u]);
          fold(&mn, &mx, c, c);
        }
    }
    if (share > 1) {
      sh_mn[tid] = mn;
      sh_mx[tid] = mx;
      __syncthreads();
      if (sub == 0)
        for (int k = 1; k < share; ++k)
          fold(&mn, &mx, sh_mn[tid + (k << a.log_lanes)], sh_mx[tid + (k << a.log_lanes)]);
      __syncthreads();
    }
    if (sub == 0 && valid > 0) {
      const int P = __ldg(table + p);
      uint4* dst = static_cast<uint4*>(a.stats) + ((int64_t)P * Hkv + g) * 2 * ROW + col;
      dst[0] = pack<T>(mn);
      dst[ROW] = pack<T>(mx);
    }
  }
}

template <typename T, int D>
cudaError_t launch_t(const kv_cache_desc& d, CompactArgs a, int sms, DevCtx ctx, cudaStream_t s) {
  constexpr int ROW = D * sizeof(T) / 16;
  int lanes = ROW;
  // split the columns while a list is more than a batch and blocks are fewer than the GPU takes
  while (lanes > kMinLanes && (long)a.keep_stride * lanes > (long)kSteps * kThreads &&
         2l * d.batch * d.num_kv_heads * (ROW / lanes) < (long)kBlocksPerSM * sms)
    lanes /= 2;
  while (1 << a.log_lanes < lanes) ++a.log_lanes;
  const dim3 grid(2 * ROW / lanes, d.num_kv_heads, d.batch);
  return launch_pdl(compact_kernel<T, D>, grid, dim3(kThreads), 0, s, d, a, ctx);
}

}  // namespace

cudaError_t launch_compact(const kv_cache_desc& d, const int32_t* cu, const int32_t* keep,
                           int keep_stride, const int32_t* keep_cnt, void* stats,
                           int32_t* new_lens, int sms, DevCtx ctx, cudaStream_t s) {
  const CompactArgs a{cu, keep, keep_cnt, keep_stride, 0, stats, new_lens};
  if (d.dtype == KV_BF16)
    return d.head_dim == 128 ? launch_t<bf16_t, 128>(d, a, sms, ctx, s)
                             : launch_t<bf16_t, 64>(d, a, sms, ctx, s);
  return d.head_dim == 128 ? launch_t<float, 128>(d, a, sms, ctx, s)
                           : launch_t<float, 64>(d, a, sms, ctx, s);
}

}  // namespace skv
