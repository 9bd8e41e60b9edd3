// dsa_paged.cuh — what the paged-cache kernels share: the argument block, the
// request a query row belongs to, the slot of a position, and what a NaN or an
// empty row does to a softmax.
#pragma once

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

// Arguments of both attention forms (idx == nullptr: all cached tokens).
struct AttendArgs {
  const void* Q;
  const void* K;
  const void* V;
  const float* K_scale;
  const float* V_scale;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* q_off;
  const int32_t* idx;
  int k;
  int B, total_q, max_q;
  int n_pages, page, max_pages;
  int64_t page_stride;
  int Hq, Hkv, d;
  float scale;
  void* out;
  float* lse;
  int* status;
  // partial results of a split softmax (workspace)
  float* part_o;
  float* part_ml;
};

// The request of one query row: row `row` is query j = row - q0 of its m.
struct RowSeq {
  int b;     // request, -1: the row is padding or its request is not valid
  int len;   // cached tokens, the new ones included
  int pos;   // the row's position, -1 or below: it sees nothing
};

// Row `row` of request lo, if that request keeps the call's rules; else
// reports it.
__device__ __forceinline__ RowSeq row_of(const AttendArgs& a, int lo, int row) {
  RowSeq r;
  r.b = -1;
  r.len = 0;
  r.pos = -1;
  const int q0 = a.q_off[lo], q1 = a.q_off[lo + 1], len = a.lens[lo];
  if (q0 < 0 || row < q0 || row >= q1 || q1 > a.total_q || (a.idx == nullptr && q1 - q0 > a.max_q) || len < 0 ||
      (int64_t)len > (int64_t)a.max_pages * a.page) {
    report_error(a.status, DSA_ERR_INVALID_ARG, 40);
    return r;
  }
  r.b = lo;
  r.len = len;
  r.pos = len - (q1 - q0) + (row - q0);
  return r;
}

// Finds the request whose rows hold `row` (offsets ascend; a request without
// rows is passed over).
__device__ __forceinline__ RowSeq find_row(const AttendArgs& a, int row) {
  if (row < a.q_off[0] || row >= a.q_off[a.B]) return RowSeq{-1, 0, -1};  // in front of the first request, or padding
  int lo = 0, hi = a.B - 1;                            // the last b with q_off[b] <= row
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.q_off[mid] <= row)
      lo = mid;
    else
      hi = mid - 1;
  }
  return row_of(a, lo, row);
}

// The larger of two; NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 1 / sum of a softmax, 0 for a row that sees nothing; a NaN stays one.
__device__ __forceinline__ float inverse(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }

// a / b (a >= 0, b > 0); the 32-bit division is several times shorter.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  return ((a | b) >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// What the debug build checks ahead of an access (in_bounds): a table entry; a
// cache row of d elements, at an element offset in the pool.
__device__ __forceinline__ bool table_ok(const AttendArgs& a, int b, int col) {
  return (unsigned)b < (unsigned)a.B && (unsigned)col < (unsigned)a.max_pages;
}
__device__ __forceinline__ bool cache_ok(const AttendArgs& a, int64_t at) {
  return at >= 0 && at + a.d <= (a.n_pages - 1) * a.page_stride + (int64_t)a.page * a.Hkv * a.d;
}

// Page id of `pos` of request b (0 <= pos < len), -1 if the table names a
// page outside the pool; `off` is the offset within the page.
__device__ __forceinline__ int page_of(const AttendArgs& a, int b, int pos, int& off) {
  const int col = (int)((unsigned)pos / (unsigned)a.page);
  off = pos - col * a.page;
  const int id = in_bounds(table_ok(a, b, col), a.status, 20) ? a.table[(int64_t)b * a.max_pages + col] : -1;
  if ((unsigned)id >= (unsigned)a.n_pages) {
    report_error(a.status, DSA_ERR_INVALID_ARG, 41);
    return -1;
  }
  return id;
}

// The general CUDA-core attention (dsa_attend.cu): `splits` parts a row; a
// block or (without `share`) a warp each.
int launch_attend_general(const AttendArgs& a, int q_dtype, int kv_dtype, int splits, bool share, cudaStream_t st);

// The tensor-core attention (dsa_attend_tc.cu): whether it takes a call, and
// its workspace, for at most `rows` query rows that read the same cache.
bool attend_tc_ok(const AttendArgs& a, int q_dtype, int kv_dtype);
size_t attend_tc_bytes(int sms, int rows, int d);
int run_attend_tc(const AttendArgs& a, int kv_dtype, int rows, int sms, uint8_t* ws, cudaStream_t st);

}  // namespace dsa
