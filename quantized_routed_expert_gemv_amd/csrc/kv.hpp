// The paged cache and the batch of sequences, as the kernels see them.
#pragma once
#include "common.hpp"

namespace moe {

struct KvCacheView {
  uint8_t* k;
  uint8_t* v;
  int64_t k_page, k_token, k_head, v_page, v_token, v_head;   // elements
  const float* k_scale;
  const float* v_scale;
  int type, n_pages, page_size, n_heads, D;
  uint32_t page_inv;   // floor((2^32 - 1) / page_size)
};

struct KvBatchView {
  const int32_t* q_start;
  const int32_t* seq_len;
  const int32_t* table;
  int64_t table_stride;
  int n_seq, T, max_pages;
};

struct HeadsView {
  uint8_t* p;
  int64_t token, head;   // elements
};

// pos / page_size and the remainder for 0 <= pos < 2^31. With inv = floor((2^32 - 1) / d) the
// high half of pos * inv is the quotient or one below it.
__device__ __forceinline__ int page_of(uint32_t pos, int page_size, uint32_t inv, int* row) {
  uint32_t q = __umulhi(pos, inv), r = pos - q * (uint32_t)page_size;
  if (r >= (uint32_t)page_size) ++q, r -= (uint32_t)page_size;
  *row = (int)r;
  return (int)q;
}

// x / d for 0 <= x < 2^31, with inv = floor((2^32 - 1) / d).
__device__ __forceinline__ int div_by(int x, int d, uint32_t inv) {
  int rest;
  return page_of((uint32_t)x, d, inv, &rest);
}

// First row of sequence b's new tokens (b = n_seq: the end of the last), within [0, T].
__device__ __forceinline__ int first_row(const KvBatchView& b, int i) {
  return min(max(b.q_start[i], 0), b.T);
}

// The largest i in [0, n) with f(i) <= x, for f that does not fall and f(0) <= x, found by the
// whole wave 64 probes at a time (x is uniform). For any f the answer lies in [0, n).
template <typename F>
__device__ __forceinline__ int wave_find(int n, int64_t x, F f) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, cnt = n;
  while (cnt > 1) {
    const int step = (cnt + kWave - 1) / kWave;
    const int at = lane * step;
    const bool le = at < cnt && f(lo + at) <= x;
    const int k = max(__popcll(__ballot(le)) - 1, 0) * step;
    cnt = min(step, cnt - k);
    lo += k;
  }
  return lo;
}

}  // namespace moe
