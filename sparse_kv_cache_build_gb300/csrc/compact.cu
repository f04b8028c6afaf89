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
// keys or values, so blocks need nothing of each other; it walks the tokens in batches: where they
// come from and go to, worked out once for all columns, then all loads, a barrier, all stores.
//
// Bound: every moved token is read and written once. A batch costs a block one round of reads
// (list, table, token), of which the first two run beside the tokens of the batch before; so a
// long list is the columns split further, down to 32 bytes a row (a sector), as long as the
// blocks find an SM each; a short one, that is a batch at once, is a chain of dependent reads
// (offsets, list, table, token, statistics). Measured: 32 sequences that keep up to 9 of 26
// drafts, 32/8 heads: 8.7 us on the device; one of 32768 tokens that keeps 4600 (39 MB): 18.4 us,
// where columns of 64 bytes take 4 us more, and blocks of half the threads and batch, two to an
// SM, 2 more.
#include "packed_rows.cuh"

namespace skv {
namespace {

constexpr int kFew = 256, kMany = 512; // threads of a block
constexpr int kSteps = 8;              // tokens of a thread in a batch
constexpr int kMinLanes = 2;           // 16-byte columns of a block: at least a sector

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

template <typename T, int D, int NT>
__global__ void __launch_bounds__(NT)
compact_kernel(const __grid_constant__ kv_cache_desc d, const __grid_constant__ CompactArgs a,
               const __grid_constant__ DevCtx ctx) {
  constexpr int ROW = D * sizeof(T) / 16;            // 16-byte columns of a token
  constexpr int BATCH = NT * kSteps / kMinLanes;     // tokens of a batch at most
  // two batches of moves, later the extremes of the pages' parts
  constexpr size_t MOVES = 2 * BATCH * sizeof(uint2), PARTS = 2 * NT * sizeof(Chunk<T>);
  __shared__ __align__(16) uint8_t sh[MOVES > PARTS ? MOVES : PARTS];
  uint2* moves = reinterpret_cast<uint2*>(sh);
  Chunk<T>* sh_mn = reinterpret_cast<Chunk<T>*>(sh);
  Chunk<T>* sh_mx = sh_mn + NT;
  pdl_trigger();
  pdl_wait();
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int parts = ROW >> a.log_lanes;
  const bool values = (int)blockIdx.x >= parts;
  const int col = (((int)blockIdx.x - (values ? parts : 0)) << a.log_lanes) +
                  (tid & ((1 << a.log_lanes) - 1));
  const int row = tid >> a.log_lanes, rows = NT >> a.log_lanes;
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
  // A token's slot in the pool, counted over pages (below 2^32: a slot is 256 bytes of memory and
  // more), or kNone where its page is unmapped.
  constexpr uint32_t kNone = ~0u;
  const int page_log = __ffs(PS) - 1;
  auto slot_at = [&](int P, int t) -> uint32_t {
    if (P >= 0 && P < d.num_phys_pages) return ((uint32_t)P << page_log) + (t & (PS - 1));
    flag(ctx, KV_DEVERR_BAD_PAGE);
    return kNone;
  };
  // where the block's column of a slot lies, in 16 bytes
  auto place = [&](uint32_t slot) {
    return ((((int64_t)(slot >> page_log) * Hkv + g) << page_log) + (slot & (PS - 1))) * ROW;
  };
  const int batch = kSteps * rows;
  // Sources and places of a batch, each level of reads for all of a thread's tokens at once.
  auto find_moves = [&](int i0, uint2* m) {
    constexpr int MINE = kSteps / kMinLanes;
    int k[MINE], before[MINE], from[MINE], to[MINE];
#pragma unroll
    for (int u = 0; u < MINE; ++u) {
      const int x = tid + u * NT, i = i0 + x;
      k[u] = x < batch && i < cnt ? __ldg(keep + i) : i;         // staying where it is: no move
      before[u] = x < batch && i < cnt && i > 0 ? __ldg(keep + i - 1) : -1;
    }
#pragma unroll
    for (int u = 0; u < MINE; ++u) {
      const int i = i0 + tid + u * NT;
      // rising from k >= i on, and inside the candidates
      const bool good = k[u] >= i && k[u] < n && before[u] < k[u];
      if (!good && i < cnt && tid + u * NT < batch) flag(ctx, KV_DEVERR_BAD_SEL);
      if (!good) k[u] = i;
      from[u] = to[u] = -1;
      if (k[u] != i) {
        from[u] = __ldg(table + ((start + k[u]) >> page_log));
        to[u] = __ldg(table + ((start + i) >> page_log));
      }
    }
#pragma unroll
    for (int u = 0; u < MINE; ++u) {
      const int x = tid + u * NT, i = i0 + x;
      if (x >= batch) continue;
      uint2 move = make_uint2(kNone, kNone);
      if (k[u] != i) {
        move.x = slot_at(from[u], start + k[u]);
        move.y = slot_at(to[u], start + i);
        if (move.y == kNone) move.x = kNone;
      }
      m[x] = move;
    }
  };
  find_moves(0, moves);
  for (int i0 = 0, buf = 0; i0 < cnt; i0 += batch, buf ^= 1) {
    __syncthreads();
    const uint2* mine = moves + buf * batch;
    uint2 m[kSteps];
    uint4 v[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      m[u] = mine[u * rows + row];
      if (m[u].x != kNone) v[u] = __ldcg(pool + place(m[u].x));
    }
    if (i0 + batch < cnt) find_moves(i0 + batch, moves + (buf ^ 1) * batch);
    __syncthreads();                                 // every source up to here has been read
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
      if (m[u].x != kNone) pool[place(m[u].y)] = v[u];
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
    const uint32_t page = have ? slot_at(__ldg(table + p), 0) : kNone;
    const int64_t base = place(page);
    const int valid = page == kNone ? 0 : min(PS, fresh - p * PS);
    Chunk<T> mn, mx;
#pragma unroll
    for (int e = 0; e < Chunk<T>::N; ++e) {
      mn.f[e] = INFINITY;
      mx.f[e] = -INFINITY;
    }
    // the first key starts the extremes (where it is NaN they stay so), later NaN do not count
    if (sub == 0 && valid > 0) mn = mx = unpack<T>(__ldcg(pool + base));
    for (int t = sub == 0 ? share : sub; t < valid; t += 8 * share) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (t + u * share < valid) v[u] = __ldcg(pool + base + (int64_t)(t + u * share) * ROW);
#pragma unroll
      for (int u = 0; u < 8; ++u)
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
      uint4* dst = static_cast<uint4*>(a.stats) +
                   ((int64_t)(page >> page_log) * Hkv + g) * 2 * ROW + col;
      dst[0] = pack<T>(mn);
      dst[ROW] = pack<T>(mx);
    }
  }
}

template <typename T, int D>
cudaError_t launch_t(const kv_cache_desc& d, CompactArgs a, int sms, DevCtx ctx, cudaStream_t s) {
  constexpr int ROW = D * sizeof(T) / 16;
  // Lists of more than a batch: larger blocks, one to an SM, and their columns split as long as
  // the blocks find an SM each.
  int lanes = ROW;
  const bool many = (long)a.keep_stride * ROW > (long)kSteps * kFew;
  while (many && lanes > kMinLanes && (long)a.keep_stride * lanes > (long)kSteps * kMany &&
         4l * d.batch * d.num_kv_heads * (ROW / lanes) <= sms)
    lanes /= 2;
  while (1 << a.log_lanes < lanes) ++a.log_lanes;
  const dim3 grid(2 * ROW / lanes, d.num_kv_heads, d.batch);
  return many ? launch_pdl(compact_kernel<T, D, kMany>, grid, dim3(kMany), 0, s, d, a, ctx)
              : launch_pdl(compact_kernel<T, D, kFew>, grid, dim3(kFew), 0, s, d, a, ctx);
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
