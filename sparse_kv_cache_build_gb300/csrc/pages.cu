// Physical pages: copies of whole pages, and the batch's next page table.
//
// kv_copy_pages moves bytes: a block takes 32 KB of a pair's keys, values or statistics, every
// thread with its eight 16-byte loads in flight before the first store. Measured: 2000 pages of
// 262 KB (1065 MB read and written) 157 us, the rate of the measured plain copy; 16 of 64 KB 2 us.
//
// kv_update_pages is two launches. The first builds the new rows from the old ones: a block takes a
// range of an old row's entries, reads each once, and writes it to every new row that continues
// the old one; the page's reference count changes by the rows that kept the entry less one, so
// a row that one row continues costs no atomic. (Counts are sums of whole numbers: the order of
// the atomics does not show.) The second is one cluster of eight blocks. It
//   1. counts the free pages (count zero), each warp its own stretch;
//   2. finds, in every block for itself, the partial pages that rows are about to write to and that
//      others hold too, and adds up the rows' needs;
//   3. tells the blocks each other's free pages, and hands the lowest ones out in the order of the
//      rows: a free page's rank among the free ones says which row and entry it is for.
// A shared page's count never passes zero on the way, so counting and reading it need no order
// but the one barrier. The pool's state is the counts alone: the pages handed out depend on
// nothing else.
//
// Bound: latency. The table is read and written once and the counts once or twice, all of it in
// L2; what shows is the two launches and the second one's chain of dependent reads (parent,
// length, entry, count): 64 rows of 4096 entries over a pool of 65536 10.3 us on the device (15.9
// with the rows dealt out to the blocks and four barriers among them). Rows that share a page
// look for each other among all rows, which for thousands of them is the longest part.
#include <cooperative_groups.h>

#include <atomic>

#include "packed_rows.cuh"

namespace cg = cooperative_groups;

namespace skv {
namespace {

// ------------------------------------------------------------------------------------
// Page copies
// ------------------------------------------------------------------------------------
constexpr int kCopyThreads = 256, kCopySteps = 8;
constexpr int kCopyChunk = kCopyThreads * kCopySteps;      // 16-byte words of a block

struct CopyArgs {
  const int32_t* pairs;        // [n][2]
  int NP;
  int words, stat_words;       // 16-byte words of a page of one pool, and of its statistics
  int chunks, stat_chunks;     // blocks for them
  uint4 *k, *v, *stats;
};

__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(const __grid_constant__ CopyArgs a, const __grid_constant__ DevCtx ctx) {
  pdl_trigger();
  pdl_wait();
  const int per = 2 * a.chunks + a.stat_chunks;
  const int pair = blockIdx.x / per, piece = blockIdx.x % per;
  const int2 p = reinterpret_cast<const int2*>(a.pairs)[pair];
  if (p.x < 0 || p.y < 0) return;                          // no copy
  if (p.x >= a.NP || p.y >= a.NP) {
    if (piece == 0 && threadIdx.x == 0) flag(ctx, KV_DEVERR_BAD_PAGE);
    return;
  }
  const bool stat = piece >= 2 * a.chunks;
  uint4* pool = stat ? a.stats : piece < a.chunks ? a.k : a.v;
  const int words = stat ? a.stat_words : a.words;
  const int chunk = stat ? piece - 2 * a.chunks : piece < a.chunks ? piece : piece - a.chunks;
  const uint4* src = pool + (int64_t)p.x * words;
  uint4* dst = pool + (int64_t)p.y * words;
  const int w0 = chunk * kCopyChunk + threadIdx.x;
  uint4 x[kCopySteps];
#pragma unroll
  for (int i = 0; i < kCopySteps; ++i)
    if (w0 + i * kCopyThreads < words) x[i] = __ldcs(src + w0 + i * kCopyThreads);
#pragma unroll
  for (int i = 0; i < kCopySteps; ++i)
    if (w0 + i * kCopyThreads < words) __stcs(dst + w0 + i * kCopyThreads, x[i]);
}

// ------------------------------------------------------------------------------------
// Page tables
// ------------------------------------------------------------------------------------
constexpr int kRowThreads = 256, kRowEntries = 4 * kRowThreads;
constexpr int kAllocBlocks = 8, kAllocThreads = 1024, kAllocWarps = kAllocThreads / 32;

struct PagesArgs {
  int32_t* refs;
  const int32_t* parents;      // [rows], or NULL: row b continues old row b
  const int32_t* keep_lens;    // [rows], or NULL: all of the old row's tokens
  const int32_t* new_lens;     // [rows]
  int rows;
  int window, sinks;           // window 0: none
  int32_t* table;              // [rows][stride]
  int32_t* copies;             // [rows][2]
  int32_t* free_left;
};

// What becomes of one new row.
struct RowPlan {
  int parent;      // old row, or -1
  int keep, want;  // tokens kept of it, and tokens to have room for
  bool whole;      // the old row's entries stay as they are: its own length says nothing of them
};

// Numbers that do not fit are flagged; the row then keeps what its old row holds.
__device__ __forceinline__ RowPlan row_plan(const DevCtx& c, const kv_cache_desc& d,
                                            const PagesArgs& a, int b) {
  RowPlan r;
  r.parent = a.parents != nullptr ? a.parents[b] : b;
  if (r.parent < -1 || r.parent >= d.batch) {
    flag(c, KV_DEVERR_BAD_SEL);
    r.parent = -1;
  }
  r.whole = false;
  int len = 0;
  if (r.parent >= 0) {
    len = d.seq_lens[r.parent];
    r.whole = len < 0 || len > d.page_table_stride * d.page_size;
  }
  if (r.whole) {
    flag(c, KV_DEVERR_BAD_LEN);
    r.keep = r.want = 0;
    return r;
  }
  r.keep = a.keep_lens != nullptr ? a.keep_lens[b] : len;
  r.want = a.new_lens[b];
  if (r.keep < 0 || r.keep > len || r.want < r.keep ||
      r.want > d.page_table_stride * d.page_size) {
    flag(c, KV_DEVERR_BAD_LEN);
    r.keep = r.want = len;
  }
  return r;
}

// The entries that a row keeps: [0, first) without those that fell out of the window. The next row
// is at position keep and sees the tokens above keep - window.
struct Kept {
  int row, first, dead0, dead1;
  __device__ __forceinline__ bool holds(int p) const {
    return p < first && (p < dead0 || p >= dead1);
  }
};

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
  return tokens / page_size + (tokens % page_size != 0);
}

__global__ void __launch_bounds__(kRowThreads)
fork_rows_kernel(const __grid_constant__ kv_cache_desc d, const __grid_constant__ PagesArgs a,
                 const __grid_constant__ DevCtx ctx) {
  __shared__ Kept list[kRowThreads];
  __shared__ int found;
  pdl_trigger();
  pdl_wait();
  const int old = blockIdx.y, tid = threadIdx.x, stride = d.page_table_stride;
  const bool nobody = old == d.batch;                // the rows that continue no old one
  const int p0 = blockIdx.x * kRowEntries + tid;
  int e[4], kept[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = p0 + i * kRowThreads;
    e[i] = !nobody && p < stride ? d.page_table[(int64_t)old * stride + p] : -1;
    if (e[i] < -1 || e[i] >= d.num_phys_pages) {
      flag(ctx, KV_DEVERR_BAD_PAGE);
      e[i] = -1;
    }
    kept[i] = 0;
  }
  const int b_from = a.parents != nullptr ? 0 : old;
  const int b_to = a.parents != nullptr ? a.rows : old + 1;
  for (int b0 = b_from; b0 < b_to; b0 += kRowThreads) {
    __syncthreads();                                 // the list before has been read
    if (tid == 0) found = 0;
    __syncthreads();
    const int b = b0 + tid;
    if (b < b_to) {
      const int parent = a.parents != nullptr ? a.parents[b] : b;
      const bool mine = nobody ? parent < 0 || parent >= d.batch : parent == old;
      if (mine) {
        const RowPlan r = row_plan(ctx, d, a, b);
        const int PS = d.page_size;
        list[atomicAdd(&found, 1)] =
            Kept{b, r.whole ? stride : pages_of(r.keep, PS), pages_of(a.sinks, PS),
                 a.window > 0 ? max(0, r.keep - a.window + 1) / PS : 0};
      }
    }
    __syncthreads();
    for (int k = 0; k < found; ++k) {
      const Kept x = list[k];
      int32_t* out = a.table + (int64_t)x.row * stride;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = p0 + i * kRowThreads;
        const bool held = x.holds(p) && e[i] >= 0;
        if (p < stride) out[p] = held ? e[i] : -1;
        kept[i] += held;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (e[i] >= 0 && kept[i] != 1) atomicAdd(a.refs + e[i], kept[i] - 1);
}

// Exclusive running sum of `need` over the rows, in place, and their total; by a whole block.
// Sums beyond 32 bits are more than any pool has, and then nothing is handed out.
__device__ __forceinline__ int64_t running_sum(int32_t* need, int rows, int64_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t before = 0;
  for (int b0 = 0; b0 < rows; b0 += kAllocThreads) {
    const int b = b0 + tid, mine = b < rows ? need[b] : 0;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) scratch[warp] = upto;
    __syncthreads();
    int64_t start = before;
    for (int w = 0; w < kAllocWarps; ++w) {
      if (w < warp) start += scratch[w];
      before += scratch[w];
    }
    if (b < rows) need[b] = (int32_t)(start + upto - mine);
    __syncthreads();
  }
  return before;
}

__global__ void __cluster_dims__(kAllocBlocks, 1, 1) __launch_bounds__(kAllocThreads, 1)
alloc_pages_kernel(const __grid_constant__ kv_cache_desc d, const __grid_constant__ PagesArgs a,
                   const __grid_constant__ DevCtx ctx) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t scratch[kAllocWarps];
  __shared__ int warp_free[kAllocWarps], block_free[kAllocBlocks];
  cg::cluster_group cluster = cg::this_cluster();
  // every block must have started before its shared memory is written: half a barrier here, the
  // other half before the first write
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_trigger();
  pdl_wait();
  int32_t* sums = sm;                                // [rows] needs, then a row's first rank
  int32_t* places = sums + a.rows;                   // [rows] its entry, twice, plus 1 for a copy
  int32_t* parts = places + a.rows;                  // [rows] the partial page it writes to, or -1
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster.block_rank(), PS = d.page_size, NP = d.num_phys_pages;
  const int stride = d.page_table_stride;

  // free pages, each warp its own stretch of the counts
  const int warps = kAllocBlocks * kAllocWarps;
  const int64_t each = ((int64_t)NP + warps * 128 - 1) / (warps * 128) * 128;
  const int64_t from = each * (rank * kAllocWarps + warp), to = min((int64_t)NP, from + each);
  auto zeros = [&](int64_t p0) {                     // of the lane's four counts
    uint32_t z = 0;
    const int64_t p = p0 + 4 * lane;
    if (p + 4 <= to) {
      const int4 c = __ldcg(reinterpret_cast<const int4*>(a.refs + p));
      z = (c.x == 0) | (c.y == 0) << 1 | (c.z == 0) << 2 | (c.w == 0) << 3;
    } else {
      for (int i = 0; i < 4; ++i)
        if (p + i < to) z |= (uint32_t)(__ldcg(a.refs + p + i) == 0) << i;
    }
    return z;
  };
  int mine = 0;
#pragma unroll 4
  for (int64_t p = from; p < to; p += 128) mine += __popc(zeros(p));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) warp_free[warp] = mine;

  // Every block works out all rows' needs, so that none has to wait for another's. A row that
  // grows out of a partial page that others hold too gets a fresh one, unless it is the last row
  // of those that alone hold the page.
  for (int b = tid; b < a.rows; b += kAllocThreads) {
    const RowPlan r = row_plan(ctx, d, a, b);
    const int first = pages_of(r.keep, PS);
    const bool writes = r.want > r.keep && r.keep % PS != 0;
    parts[b] = writes ? a.table[(int64_t)b * stride + first - 1] : -1;
    sums[b] = pages_of(r.want, PS) - first;
    places[b] = 2 * first;
  }
  __syncthreads();
  for (int b = tid; b < a.rows; b += kAllocThreads) {
    const int part = parts[b];
    if (part < 0) continue;
    const int holders = __ldcg(a.refs + part);
    if (holders <= 1) continue;
    int writers = 0, last = b;
    for (int k = 0; k < a.rows; ++k)
      if (parts[k] == part) {
        ++writers;
        last = k;
      }
    if (holders > writers || last != b) {
      ++sums[b];
      places[b] -= 1;                                // 2 (first - 1) + 1
    }
  }
  __syncthreads();
  const int64_t total = running_sum(sums, a.rows, scratch);
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (tid < kAllocBlocks) {
    int sum = 0;
    for (int w = 0; w < kAllocWarps; ++w) sum += warp_free[w];
    cluster.map_shared_rank(block_free, tid)[rank] = sum;
  }
  cluster.sync();                                    // counts are known, and have been read
  int64_t at = 0, have = 0;                          // free pages before the warp's, and in all
  for (int r = 0; r < kAllocBlocks; ++r) {
    if (r < rank) at += block_free[r];
    have += block_free[r];
  }
  for (int w = 0; w < warp; ++w) at += warp_free[w];
  const bool enough = total <= have;
  if (rank == 0 && tid == 0) {
    a.free_left[0] = (int32_t)max((int64_t)INT32_MIN, have - total);
    if (!enough) flag(ctx, KV_DEVERR_NO_PAGES);
  }
  for (int b = rank * kAllocThreads + tid; b < a.rows; b += kAllocBlocks * kAllocThreads) {
    const bool fork = enough && (places[b] & 1);
    a.copies[2 * b] = fork ? parts[b] : -1;
    if (!fork) a.copies[2 * b + 1] = -1;             // else by who hands the page out
    else atomicSub(a.refs + parts[b], 1);
  }
  if (!enough) return;
  for (int64_t p0 = from; p0 < to && at < total; p0 += 128) {
    uint32_t z = zeros(p0);
    const int cnt = __popc(z);
    int before = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    const int all = __shfl_sync(0xffffffffu, before, 31);
    int r = (int)at + before - cnt;                  // ranks up to total fit 32 bits here
    for (; z != 0 && r < total; z &= z - 1, ++r) {
      const int page = (int)(p0 + 4 * lane) + __ffs(z) - 1;
      int lo = 0, hi = a.rows;                       // the last row whose pages start at or before r
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= r) lo = mid;
        else hi = mid;
      }
      const int i = r - sums[lo], place = places[lo];
      a.table[(int64_t)lo * stride + (place >> 1) + i] = page;
      a.refs[page] = 1;
      if ((place & 1) && i == 0) a.copies[2 * lo + 1] = page;
    }
    at += all;
  }
}

}  // namespace

cudaError_t launch_copy_pages(const kv_cache_desc& d, const int32_t* pairs, int n, void* stats,
                              DevCtx ctx, cudaStream_t s) {
  const int elem = d.dtype == KV_BF16 ? 2 : 4;
  CopyArgs a{};
  a.pairs = pairs;
  a.NP = d.num_phys_pages;
  a.words = d.num_kv_heads * d.page_size * d.head_dim * elem / 16;
  a.stat_words = d.num_kv_heads * 2 * d.head_dim * elem / 16;
  a.chunks = ceil_div(a.words, kCopyChunk);
  a.stat_chunks = stats != nullptr ? ceil_div(a.stat_words, kCopyChunk) : 0;
  a.k = static_cast<uint4*>(const_cast<void*>(d.k_pool));
  a.v = static_cast<uint4*>(const_cast<void*>(d.v_pool));
  a.stats = static_cast<uint4*>(stats);
  return launch_pdl(copy_pages_kernel, dim3((unsigned)n * (2 * a.chunks + a.stat_chunks)),
                    dim3(kCopyThreads), 0, s, a, ctx);
}

long copy_pages_blocks(const kv_cache_desc& d, long n) {
  const long elem = d.dtype == KV_BF16 ? 2 : 4;
  const long row = (long)d.num_kv_heads * d.head_dim * elem / 16;
  auto chunks = [](long words) { return (words + kCopyChunk - 1) / kCopyChunk; };
  return n * (2 * chunks(row * d.page_size) + chunks(2 * row));
}

cudaError_t launch_update_pages(const kv_cache_desc& d, int32_t* refs, const int32_t* parents,
                                int rows, const int32_t* keep_lens, const int32_t* new_lens,
                                int window, int sinks, int32_t* table, int32_t* copies,
                                int32_t* free_left, DevCtx ctx, cudaStream_t s) {
  const PagesArgs a{refs, parents, keep_lens, new_lens, rows, window, sinks, table, copies,
                    free_left};
  const dim3 grid(ceil_div(d.page_table_stride, kRowEntries), d.batch + (parents != nullptr));
  // The rows' numbers next to the kernel's own memory may pass the 48 KB a launch has by default;
  // raised before anything is launched, so that a call that fails has changed nothing. Set once per
  // device; setting it twice from two threads is harmless.
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(alloc_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kMaxPageRows * 3 * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(1, std::memory_order_release);
  }
  e = launch_pdl(fork_rows_kernel, grid, dim3(kRowThreads), 0, s, d, a, ctx);
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)rows * 3 * sizeof(int32_t);
  return launch_pdl(alloc_pages_kernel, dim3(kAllocBlocks), dim3(kAllocThreads), smem, s, d, a,
                    ctx);
}

}  // namespace skv
