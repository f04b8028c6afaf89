// Packed token rows: how the calls that take the new tokens of a whole batch find the sequence
// a piece of work belongs to, on the device, from offsets the host never reads.
//
// The rows of sequence b are cu_tokens[b] .. cu_tokens[b+1]-1 (one row per sequence when
// cu_tokens is NULL) and hold its last n_b tokens: row i of them is position len_b - n_b + i.
#pragma once

#include "kv_internal.cuh"

namespace skv {

struct PackedRows {
  const int32_t* cu;    // [batch + 1], or NULL: row b is sequence b's one new token
  int32_t total;        // rows in the packed tensors
};

// The new tokens of one sequence; n = 0 when there are none or the offsets are not usable.
struct SeqRows {
  int row0;   // first packed row
  int n;      // rows
  int len;    // sequence length, the new tokens included
};

// Length of sequence b; one that is negative or longer than its page-table row is flagged and 0:
// where its new tokens belong is not known, and clamped they would fall on cached ones.
__device__ __forceinline__ int packed_len(const DevCtx& c, const kv_cache_desc& d, int b) {
  const int len = d.seq_lens[b];
  if (len >= 0 && len <= d.page_table_stride * d.page_size) return len;
  flag(c, KV_DEVERR_BAD_LEN);
  return 0;
}

// Offsets must rise from 0 and stay inside [0, total], and a sequence holds at least its new
// tokens; anything else is flagged and the sequence is left out.
__device__ __forceinline__ SeqRows seq_rows(const DevCtx& c, const kv_cache_desc& d,
                                            const PackedRows& pr, int b) {
  SeqRows s;
  s.len = packed_len(c, d, b);
  if (pr.cu == nullptr) {
    s.row0 = b;
    s.n = s.len > 0 ? 1 : 0;
    return s;
  }
  const int c0 = pr.cu[b], c1 = pr.cu[b + 1];
  s.row0 = c0;
  s.n = c1 - c0;
  if (c0 < 0 || c1 < c0 || c1 > pr.total || s.n > s.len) {
    flag(c, KV_DEVERR_BAD_LEN);
    s.n = 0;
  }
  return s;
}

// Every sequence of the batch, checked by one block, so that bad offsets are flagged even
// where no block's search ends at them.
__device__ __forceinline__ void check_packed_rows(const DevCtx& c, const kv_cache_desc& d,
                                                  const PackedRows& pr) {
  if (pr.cu == nullptr) return;
  for (int b = threadIdx.x; b < d.batch; b += blockDim.x) (void)seq_rows(c, d, pr, b);
  if (threadIdx.x == 0 && pr.cu[0] != 0) flag(c, KV_DEVERR_BAD_LEN);
}

// Pages to append to are numbered over the whole batch without knowing the lengths: sequence b
// owns the numbers from base(b) = floor(cu[b] / PS) + 2 b up to base(b + 1). n new tokens lie in
// at most floor(n / PS) + 2 pages (the first and the last may be partial), so each sequence's
// range holds its pages, and floor(total / PS) + 2 batch numbers hold them all.
//
// The sequence whose range holds `item`, found by one warp, 32 offsets at a time: one round of
// loads for batches up to 32, two up to 1024. Sets *base to the range's first number.
__device__ __forceinline__ int find_sequence(const PackedRows& pr, int batch, int page_size,
                                             int item, int* base) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch, at = 0;
  for (;;) {
    const int step = (hi - lo + 31) >> 5;
    const int b = lo + lane * step;
    const int first = b < hi ? pr.cu[b] / page_size + 2 * b : INT32_MAX;
    int cnt = __popc(__ballot_sync(0xffffffffu, first <= item));
    cnt = cnt < 1 ? 1 : cnt;
    at = __shfl_sync(0xffffffffu, first, cnt - 1);
    lo += (cnt - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) break;
  }
  *base = at;
  return lo;
}

inline long page_numbers(int total, int batch, int page_size) {
  return (long)(total / page_size) + 2l * batch;
}

}  // namespace skv
