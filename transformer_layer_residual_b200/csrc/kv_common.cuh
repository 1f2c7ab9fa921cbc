// The paged key/value cache: parameters and row addressing shared by the
// append, read-back and attention kernels.
//
// A token's keys (or values) of one head are one row: D bf16, or D 4-bit codes
// (two a byte, the lower d in the low nibble) with one (scale, minimum) bf16
// pair; the row stands for minimum + code * scale. Rows of a (page, head) are
// contiguous, heads of a page are contiguous, pages are page_stride bytes apart.
// Every page id read from a block table is checked against the cache before an
// address is formed from it.
#pragma once

#include "common.cuh"

namespace fnl {

enum KvFormat : int { kKvBf16 = 0, kKvInt4 = 1 };

// device status code of a batch description that does not fit its cache: a page
// id outside the cache, a position outside the block table or the rotation
// table, a sequence with more new tokens than max_q or fewer cached than new
constexpr int kStatusBatch = 9;

struct KvParams {
  uint8_t* k;
  uint8_t* v;
  uint32_t* k_scale;        // 4-bit pages: (scale, minimum) bf16 pairs, scale in the low half
  uint32_t* v_scale;
  long long page_stride;    // bytes between pages of k and of v
  long long scale_stride;   // pairs between pages of k_scale and of v_scale
  int num_pages, page_shift, Hkv;
  int B, M, max_q, max_pages;
  const int* cu_q;
  const int* kv_len;
  const int* table;
  int* status;
};

__device__ __forceinline__ void kv_flag(const KvParams& p) { atomicCAS(p.status, 0, kStatusBatch); }

// New tokens [first, first + n) of sequence b in the packed batch and its tokens
// in the cache, held inside the batch and the block table whatever the arrays say.
struct KvSeq {
  int first, n, len;
};
__device__ __forceinline__ KvSeq kv_seq(const KvParams& p, int b) {
  const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
  const int len = p.kv_len[b];
  KvSeq s;
  s.first = min(max(c0, 0), p.M);
  s.n = min(max(c1, s.first), p.M) - s.first;
  const long long room = static_cast<long long>(p.max_pages) << p.page_shift;
  s.len = static_cast<int>(min(static_cast<long long>(max(len, 0)), room));
  // (the length of a sequence without new tokens is not used)
  if (c0 != s.first || c1 - c0 != s.n || (s.n > 0 && (s.n > p.max_q || len != s.len || len < s.n))) kv_flag(p);
  s.n = min(s.n, p.max_q);
  return s;
}

// Index of the row of (token position, head) inside a page set, as (page, row
// in page); -1 when the table has no valid page there. pos >= 0.
__device__ __forceinline__ int kv_page(const KvParams& p, int b, int pos) {
  const int i = pos >> p.page_shift;
  if (i >= p.max_pages) {
    kv_flag(p);
    return -1;
  }
  const int page = __ldg(p.table + static_cast<long long>(b) * p.max_pages + i);
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
    kv_flag(p);
    return -1;
  }
  return page;
}
__device__ __forceinline__ int kv_row_in_page(const KvParams& p, int head, int pos) {
  return (head << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

// Stores of outputs, pages and partial sums. Debug builds (FNL_DEBUG_CHECKS) check each against the `size` bytes
// from `base` on that it may write (of an output, a page, a slot): one outside is skipped and recorded as
// kStatusBounds. Release builds compile the check away.
__device__ __forceinline__ bool kv_in_bounds(const KvParams& p, const void* dst, int bytes, const void* base, long long size) {
#ifdef FNL_DEBUG_CHECKS
  const uint8_t* d = static_cast<const uint8_t*>(dst);
  const uint8_t* b = static_cast<const uint8_t*>(base);
  if (b == nullptr || d < b || d + bytes > b + size) {
    atomicCAS(p.status, 0, kStatusBounds);
    return false;
  }
#endif
  return true;
}
template <typename T>
__device__ __forceinline__ void kv_store(const KvParams& p, void* dst, const T& x, const void* base, long long size) {
  if (kv_in_bounds(p, dst, sizeof(T), base, size)) *static_cast<T*>(dst) = x;
}
// The same past L1: other blocks read it.
template <typename T>
__device__ __forceinline__ void kv_store_cg(const KvParams& p, void* dst, const T& x, const void* base, long long size) {
  if (kv_in_bounds(p, dst, sizeof(T), base, size)) __stcg(static_cast<T*>(dst), x);
}

__device__ __forceinline__ float kv_scale_of(uint32_t pair) { return bf_lo(pair); }
__device__ __forceinline__ float kv_min_of(uint32_t pair) { return bf_hi(pair); }

// Sequence of packed token m: the number of sequences that end at or before m
// (cu_q[i + 1] <= m), counted by all threads of the block at once; p.B when m
// lies behind the last sequence. Every thread of the block calls it.
__device__ __forceinline__ int kv_find_seq(const KvParams& p, int m) {
  int b = 0;
  for (int i = 0; i < p.B; i += blockDim.x) {
    const int j = i + threadIdx.x;
    b += __syncthreads_count(j < p.B && p.cu_q[j + 1] <= m);
  }
  return b;
}

}  // namespace fnl
