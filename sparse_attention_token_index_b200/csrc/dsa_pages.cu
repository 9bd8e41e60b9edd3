// dsa_pages.cu — page plan (block tables and slot maps from request lengths)
// and the cache write.
//
// Plan.  With P tokens a page, request b holds ceil(len / P) pages and needs
// ceil((len + new) / P).  Two exclusive sums over the requests (new tokens,
// new pages) give q_offsets and each request's first entry of the free list;
// after that every table entry and every token is independent of the others:
// a token finds its request by bisection in q_offsets.  The sums run inside a
// block, so their order is fixed and no atomics are needed.  A decode step is
// all latency: up to 2048 requests, every block forms the sums for itself in
// shared memory and fills its share, one launch in all.  With more, or when
// lens or used is updated in place (a block may read it after another has
// written it), one block forms the sums and a second launch fills.
//
// Cache write.  A row is Hkv * d contiguous elements at its slot: a copy, or
// for e4m3 pages the smallest power of two of lanes that holds a head's d
// elements, sixteen or eight a lane: amax by shuffles, a lane's bytes stored at
// once.  Each row is read and written once, so memory is the floor; the e4m3
// write is held off it by its own instructions (80 % of the issue slots at 44 %
// of the memory's throughput).
#include "dsa_paged.cuh"

namespace dsa {

constexpr int kPlanThreads = 1024;

struct PlanArgs {
  const int32_t* lens;
  const int32_t* new_lens;
  const int32_t* free_pages;
  const int32_t* used;
  int n_free, B, page, n_pages, max_pages, max_tokens;
  int32_t* table;
  int32_t* q_off;
  int64_t* slots;
  int32_t* positions;
  int32_t* lens_out;
  int32_t* used_out;
  int* status;
  int32_t* first;   // [B + 1] new pages handed out before request b (workspace)
  int32_t* state;   // {used at entry} (workspace)
};

// Exclusive sums of two values over the block, and their totals.
__device__ __forceinline__ void block_scan2(int64_t (&v)[2], int64_t (&total)[2], int64_t (*warp_sum)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t inc[2] = {v[0], v[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t u = __shfl_up_sync(0xffffffffu, inc[i], o);
      if (lane >= o) inc[i] += u;
    }
  }
  if (lane == 31) {
    warp_sum[warp][0] = inc[0];
    warp_sum[warp][1] = inc[1];
  }
  __syncthreads();
  int64_t w[2];  // every warp adds up the warps' sums
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = lane < warps ? warp_sum[lane][i] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t u = __shfl_up_sync(0xffffffffu, w[i], o);
      if (lane >= o) w[i] += u;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t before = __shfl_sync(0xffffffffu, w[i], warp > 0 ? warp - 1 : 0);
    v[i] = inc[i] - v[i] + (warp > 0 ? before : 0);
    total[i] = __shfl_sync(0xffffffffu, w[i], 31);
  }
  __syncthreads();
}

// ceil(n / page): both below 2^31, so their sum is an unsigned 32-bit number.
__device__ __forceinline__ int pages_of(int n, int page) {
  return (int)(((unsigned)n + (unsigned)page - 1u) / (unsigned)page);
}

// New tokens and new pages of request b; false if its lengths break a rule.
__device__ __forceinline__ bool plan_request(const PlanArgs& a, int b, int64_t (&v)[2], int& len) {
  const int n = a.lens[b], m = a.new_lens[b];
  len = n;
  if (n < 0 || m < 0 || (int64_t)n + m > (int64_t)a.max_pages * a.page) {
    v[0] = v[1] = 0;
    return false;
  }
  v[0] = m;
  v[1] = pages_of(n + m, a.page) - pages_of(n, a.page);
  return true;
}

// The checks over both sums' totals, by every thread of a block; ok: this
// thread's requests are valid.
__device__ __forceinline__ bool plan_fits(const PlanArgs& a, bool ok, int used, const int64_t (&total)[2], bool report) {
  ok = __syncthreads_and(ok && used >= 0 && used <= a.n_free && total[0] <= a.max_tokens);
  const bool enough = total[1] <= (int64_t)a.n_free - used;
  if (report && threadIdx.x == 0 && !(ok && enough)) report_error(a.status, ok ? DSA_ERR_PAGES : DSA_ERR_INVALID_ARG, 50);
  return ok && enough;
}

// Both sums and the checks, by one block.  Leaves q_off, first, lens_out,
// used_out and the entry state; a step that fails leaves zero sums.
__device__ __forceinline__ void plan_sums(const PlanArgs& a) {
  __shared__ int64_t warp_sum[kPlanThreads / 32][2];
  const int used = a.used[0];
  int64_t total[2] = {0, 0};
  bool ok = true;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {  // totals first: all or nothing
    const int b = b0 + threadIdx.x;
    int64_t v[2] = {0, 0}, t[2];
    int len;
    if (b < a.B) ok = plan_request(a, b, v, len) && ok;
    block_scan2(v, t, warp_sum);
    total[0] += t[0];
    total[1] += t[1];
  }
  ok = plan_fits(a, ok, used, total, true);
  int64_t base[2] = {0, 0};
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int64_t v[2] = {0, 0}, t[2];
    int len = 0;
    if (b < a.B) plan_request(a, b, v, len);
    if (!ok) v[0] = v[1] = 0;
    const int m = (int)v[0];
    block_scan2(v, t, warp_sum);
    if (b < a.B) {
      a.q_off[b] = (int)(base[0] + v[0]);
      a.first[b] = (int)(base[1] + v[1]);
      a.lens_out[b] = len + m;
    }
    base[0] += t[0];
    base[1] += t[1];
  }
  if (threadIdx.x == 0) {
    a.q_off[a.B] = (int)base[0];
    a.first[a.B] = (int)base[1];
    a.state[0] = used;
    a.used_out[0] = used + (int)base[1];
  }
}

// The last b in [0, n) with off[b] <= x (off ascends, off[0] <= x).
__device__ __forceinline__ int bisect(const int32_t* off, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Entry i of the pages handed out this step, -1 if the list names a page
// outside the pool.
__device__ __forceinline__ int fresh_page(const PlanArgs& a, int used, int i) {
  const int id = in_bounds((unsigned)(used + i) < (unsigned)a.n_free, a.status, 31) ? a.free_pages[used + i] : -1;
  if ((unsigned)id < (unsigned)a.n_pages) return id;
  report_error(a.status, DSA_ERR_INVALID_ARG, 51);
  return -1;
}

// Thread t of `step`: table entries t, t + step, ... and its share of the
// tokens.  q_off, first [B + 1] and lens [B] (new tokens included): the sums, in
// global or shared memory.
__device__ __forceinline__ void plan_fill(const PlanArgs& a, const int32_t* q_off, const int32_t* first,
                                          const int32_t* lens, int used, int64_t t, int64_t step) {
  const int n_new = q_off[a.B], n_fresh = first[a.B];
  for (int64_t i = t; i < n_fresh; i += step) {
    const int b = bisect(first, a.B, (int)i);
    const int len = lens[b] - (q_off[b + 1] - q_off[b]);
    const int held = pages_of(len, a.page);
    const int col = held + ((int)i - first[b]);
    if (in_bounds((unsigned)col < (unsigned)a.max_pages, a.status, 32))
      a.table[(int64_t)b * a.max_pages + col] = fresh_page(a, used, (int)i);
  }
  // A warp takes a run of tokens, one a lane and turn (a wider turn is more
  // code, and a step this short waits for its instructions); a lane's next
  // token belongs to the same request or one close behind.
  const int64_t per = (a.max_tokens + step - 1) / step, begin = (t >> 5) * per * 32;
  const int64_t end = min((int64_t)a.max_tokens, begin + per * 32);
  int b = 0, q0 = 0, next = 0, len = 0, held = 0;  // the request, its first token and the one behind its last
#pragma unroll 1
  for (int64_t i = begin + (t & 31); i < end; i += 32) {
    int64_t slot = -1;
    int pos = -1;
    if (i < n_new) {
      if (i >= next) {
        for (int k = 0; k < 3 && next > 0 && i >= next; ++k) next = q_off[++b + 1];
        if (i >= next) {
          b = bisect(q_off, a.B, (int)i);
          next = q_off[b + 1];
        }
        q0 = q_off[b];
        len = lens[b] - (next - q0);
        held = pages_of(len, a.page);
      }
      pos = len + (int)i - q0;
      const int col = (int)((unsigned)pos / (unsigned)a.page);
      // the last page the request held already, or one of this step's
      if (!in_bounds(b < a.B && col < a.max_pages && (col < held || used + first[b] + col - held < a.n_free), a.status, 33)) continue;
      const int id = *(col < held ? a.table + (int64_t)b * a.max_pages + col : a.free_pages + used + first[b] + col - held);
      if ((unsigned)id < (unsigned)a.n_pages)
        slot = (int64_t)id * a.page + (pos - col * a.page);
      else
        report_error(a.status, DSA_ERR_INVALID_ARG, 52);
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
}

constexpr int kOneRequests = 2048, kOneThreads = 512;

// The whole plan in one launch: every block forms the sums of all requests.
__global__ void __launch_bounds__(kOneThreads) page_plan_kernel(const PlanArgs a) {
  constexpr int kEach = kOneRequests / kOneThreads;
  __shared__ int32_t q_off[kOneRequests + 1], first[kOneRequests + 1], lens[kOneRequests];
  __shared__ int64_t warp_sum[kOneThreads / 32][2];
  const int used = a.used[0], each = (a.B + kOneThreads - 1) / kOneThreads, b0 = threadIdx.x * each;
  int64_t sum[2] = {0, 0}, total[2], v[kEach][2];
  int len[kEach];
  bool ok = true;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    v[i][0] = v[i][1] = 0;
    len[i] = 0;
    if (i < each && b0 + i < a.B) ok = plan_request(a, b0 + i, v[i], len[i]) && ok;
    sum[0] += v[i][0];
    sum[1] += v[i][1];
  }
  block_scan2(sum, total, warp_sum);
  ok = plan_fits(a, ok, used, total, blockIdx.x == 0);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (i < each && b0 + i < a.B) {
      q_off[b0 + i] = ok ? (int)sum[0] : 0;
      first[b0 + i] = ok ? (int)sum[1] : 0;
      lens[b0 + i] = len[i] + (ok ? (int)v[i][0] : 0);
    }
    sum[0] += v[i][0];
    sum[1] += v[i][1];
  }
  if (threadIdx.x == 0) {
    q_off[a.B] = ok ? (int)total[0] : 0;
    first[a.B] = ok ? (int)total[1] : 0;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < a.B; b += kOneThreads) {
      a.q_off[b] = q_off[b];
      a.lens_out[b] = lens[b];
    }
    if (threadIdx.x == 0) {
      a.q_off[a.B] = q_off[a.B];
      a.used_out[0] = used + first[a.B];
    }
  }
  plan_fill(a, q_off, first, lens, used, (int64_t)blockIdx.x * kOneThreads + threadIdx.x,
            (int64_t)gridDim.x * kOneThreads);
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_sums_kernel(const PlanArgs a) { plan_sums(a); }

__global__ void __launch_bounds__(256) page_plan_fill_kernel(const PlanArgs a) {
  plan_fill(a, a.q_off, a.first, a.lens_out, a.state[0], (int64_t)blockIdx.x * blockDim.x + threadIdx.x,
            (int64_t)gridDim.x * blockDim.x);
}

int launch_page_plan(const PlanArgs& a, int sms, cudaStream_t st) {
  const NvtxRange nvtx("dsa.page_plan");
  const int64_t items = a.max_tokens;  // a step hands out no more pages than it adds tokens
  if (a.B <= kOneRequests && a.lens_out != a.lens && a.used_out != a.used) {
    // 4 us for 8 requests; 12 us for 1024 with a million tokens in 2 blocks a multiprocessor (1: 14, 4: 16)
    const int64_t blocks = (items + kOneThreads - 1) / kOneThreads, most = (int64_t)sms * 2;
    page_plan_kernel<<<(int)(blocks < 1 ? 1 : (blocks < most ? blocks : most)), kOneThreads, 0, st>>>(a);
  } else {
    const int64_t blocks = (items + 255) / 256, most = (int64_t)sms * 8;
    page_plan_sums_kernel<<<1, kPlanThreads, 0, st>>>(a);
    page_plan_fill_kernel<<<(int)(blocks < 1 ? 1 : (blocks < most ? blocks : most)), 256, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

// ----------------------------------------------------------------------------
// cache write
// ----------------------------------------------------------------------------
struct AppendArgs {
  const void* src[2];  // k, v
  void* pool[2];       // K, V
  float* scale[2];
  const int64_t* slots;
  int T, Hkv, d, n_pages, page, n_src;
  int64_t page_stride;
  int* status;
};

// Element offset of a slot's row in the pool, -1 when the row is skipped.
__device__ __forceinline__ int64_t slot_row(const AppendArgs& a, int64_t slot) {
  if (slot < 0) return -1;
  if (slot >= (int64_t)a.n_pages * a.page) {
    report_error(a.status, DSA_ERR_INVALID_ARG, 60);
    return -1;
  }
  const int64_t id = slot < ((int64_t)1 << 31) ? (unsigned)slot / (unsigned)a.page : slot / a.page;
  const int64_t row = id * a.page_stride + (slot - id * a.page) * a.Hkv * a.d;
  const int64_t end = (a.n_pages - 1) * a.page_stride + (int64_t)a.page * a.Hkv * a.d;
  return in_bounds(row >= 0 && row + (int64_t)a.Hkv * a.d <= end, a.status, 34) ? row : -1;
}

// Same type in source and pool: rows of `units` vectors of type V, a warp
// copies 128 of them.
template <typename V>
__global__ void __launch_bounds__(256) append_copy_kernel(const AppendArgs a, int units, int per_vec) {
  constexpr int kAt = 4;
  const bool second = blockIdx.y != 0;
  const int lane = threadIdx.x & 31, parts = (units + 32 * kAt - 1) / (32 * kAt);
  const int64_t n = (int64_t)a.T * parts, step = (int64_t)gridDim.x * 8;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < n; w += step) {
    const int64_t t = parts == 1 ? w : w / parts;
    const int u0 = (int)(w - t * parts) * 32 * kAt + lane;
    const V* src = static_cast<const V*>(second ? a.src[1] : a.src[0]) + t * units;
    V x[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i)
      if (u0 + 32 * i < units) x[i] = src[u0 + 32 * i];
    const int64_t row = slot_row(a, a.slots[t]);
    if (row < 0) continue;
    V* dst = static_cast<V*>(second ? a.pool[1] : a.pool[0]) + row / per_vec;
#pragma unroll
    for (int i = 0; i < kAt; ++i)
      if (u0 + 32 * i < units) dst[u0 + 32 * i] = x[i];
  }
}

// x / scale, correctly rounded, by a multiplication with the rounded
// reciprocal and one correction of the quotient (Markstein 1990): exact while
// the remainder does not underflow and the divisor's fraction is not all
// ones; `exact` takes the division instead.
__device__ __forceinline__ float divide(float x, float scale, float inv, bool exact) {
  if (exact) return __fdiv_rn(x, scale);
  const float q = x * inv;
  return fmaf(fmaf(-q, scale, x), inv, q);
}

// Scale of a row whose largest magnitude is `top`; NaN where that is infinite
// (by the correction of the quotient) or NaN, so that the row reads back as
// NaN and an overflow is not lost.
__device__ __forceinline__ float row_scale(float top) {
  return max_nan(divide(top, 448.f, 1.f / 448.f, false), 1.17549435e-38f);
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// e4m3 pages, d a multiple of kE (8 or 16) and rows on kE bytes: `lanes` (a
// power of two) a (row, head), kE elements a lane, 16 in flight.  What a row
// costs beside its elements (slot, reductions, scale) is shared by more of
// them with 16 a lane: 32768 rows of 8 heads of 128, K and V, 204 MB, take
// 46 us (31 us at the copy bandwidth), and 74 us with 8 a lane.
template <typename S, int kE>
__global__ void __launch_bounds__(256) append_e4m3_kernel(const AppendArgs a, int lanes) {
  constexpr int kAt = kE == 16 ? 1 : 2;
  const bool second = blockIdx.y != 0;
  const int lane = threadIdx.x & (lanes - 1);
  const S* src = static_cast<const S*>(second ? a.src[1] : a.src[0]);
  uint8_t* pool = static_cast<uint8_t*>(second ? a.pool[1] : a.pool[0]);
  float* scales = second ? a.scale[1] : a.scale[0];
  const int n = a.T * a.Hkv, per_block = 256 / lanes;  // fewer than 2^31 rows (host)
  const bool mine = lane * kE < a.d;
  for (int64_t r0 = (int64_t)blockIdx.x * kAt * per_block; r0 < n; r0 += (int64_t)gridDim.x * kAt * per_block) {
    float x[kAt][kE];
    int64_t slot[kAt];
    int h[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const int64_t r = r0 + i * per_block + threadIdx.x / lanes;
      slot[i] = -1;
      h[i] = 0;
#pragma unroll
      for (int e = 0; e < kE; ++e) x[i][e] = 0.f;
      if (r < n) {
        const int t = (int)((unsigned)r / (unsigned)a.Hkv);
        h[i] = (int)r - t * a.Hkv;
        slot[i] = a.slots[t];
        if (mine) {
#pragma unroll
          for (int e = 0; e < kE; e += 8) load8(src + r * a.d + lane * kE + e, *reinterpret_cast<float(*)[8]>(&x[i][e]));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) top = max_nan(top, fabsf(x[i][e]));
      for (int o = lanes >> 1; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float scale = row_scale(top), inv = __frcp_rn(scale);
      const int64_t row = slot_row(a, slot[i]);
      if (row < 0) continue;
      if (scale < 0x1p-100f || (__float_as_uint(scale) & 0x7fffffu) == 0x7fffffu) {
#pragma unroll
        for (int e = 0; e < kE; ++e) x[i][e] = divide(x[i][e], scale, inv, true);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) x[i][e] = divide(x[i][e], scale, inv, false);
      }
      uint32_t w[kE / 4];
#pragma unroll
      for (int e = 0; e < kE; e += 4)
        w[e >> 2] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[i][e], x[i][e + 1]), __NV_SATFINITE, __NV_E4M3) |
                    (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[i][e + 2], x[i][e + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
      uint8_t* dst = pool + row + (int64_t)h[i] * a.d + lane * kE;
      if constexpr (kE == 16) {
        if (mine) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        if (mine) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      }
      if (lane == 0) scales[slot[i] * a.Hkv + h[i]] = scale;
    }
  }
}

template <typename S>
static void append_e4m3(const AppendArgs& a, int64_t rows, int64_t most, bool wide, cudaStream_t st) {
  const int per = wide ? 16 : 8;
  int lanes = 1;
  while (lanes * per < a.d) lanes *= 2;
  const int64_t at = (wide ? 1 : 2) * (256 / lanes), blocks = (rows + at - 1) / at;
  const dim3 grid((unsigned)(blocks < most ? blocks : most), a.n_src);
  if (wide)
    append_e4m3_kernel<S, 16><<<grid, 256, 0, st>>>(a, lanes);
  else
    append_e4m3_kernel<S, 8><<<grid, 256, 0, st>>>(a, lanes);
}

// e4m3 pages of any d and alignment: one warp a (row, head), lane l holds
// elements l, l + 32, ...
template <typename S>
__global__ void __launch_bounds__(256) append_e4m3_any_kernel(const AppendArgs a) {
  const int which = blockIdx.y, lane = threadIdx.x & 31;
  const S* src = static_cast<const S*>(a.src[which]);
  uint8_t* pool = static_cast<uint8_t*>(a.pool[which]);
  const int64_t n = (int64_t)a.T * a.Hkv, step = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < n; r += step) {
    const int64_t t = r / a.Hkv;
    const int h = (int)(r - t * a.Hkv);
    const int64_t slot = a.slots[t], row = slot_row(a, slot);
    if (row < 0) continue;
    float x[8], top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      x[i] = e < a.d ? (float)src[r * a.d + e] : 0.f;
      top = max_nan(top, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = row_scale(top);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < a.d)
        pool[row + (int64_t)h * a.d + e] = __nv_cvt_float_to_fp8(__fdiv_rn(x[i], scale), __NV_SATFINITE, __NV_E4M3);
    }
    if (lane == 0) a.scale[which][slot * a.Hkv + h] = scale;
  }
}

int launch_page_append(const AppendArgs& a, int src_dtype, int kv_dtype, int sms, cudaStream_t st) {
  const NvtxRange nvtx("dsa.page_append");
  const int64_t most = (int64_t)sms * 16;
  if (kv_dtype == DSA_DTYPE_FP8_E4M3) {
    const int64_t rows = (int64_t)a.T * a.Hkv;
    const uintptr_t pools = reinterpret_cast<uintptr_t>(a.pool[0]) | reinterpret_cast<uintptr_t>(a.pool[1]);
    if (a.d % 8 == 0 && a.page_stride % 8 == 0 && pools % 8 == 0 && rows < ((int64_t)1 << 31)) {
      const bool wide16 = a.d % 16 == 0 && a.page_stride % 16 == 0 && pools % 16 == 0;
      if (src_dtype == DSA_DTYPE_FP32)
        append_e4m3<float>(a, rows, most, wide16, st);
      else
        append_e4m3<__nv_bfloat16>(a, rows, most, wide16, st);
    } else {
      const int64_t blocks = (rows + 7) / 8;
      const dim3 grid((unsigned)(blocks < most ? blocks : most), a.n_src);
      if (src_dtype == DSA_DTYPE_FP32)
        append_e4m3_any_kernel<float><<<grid, 256, 0, st>>>(a);
      else
        append_e4m3_any_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
    }
  } else {
    const int elt = src_dtype == DSA_DTYPE_FP32 ? 4 : 2;
    const int64_t row_bytes = (int64_t)a.Hkv * a.d * elt;
    // 16-byte vectors when every row of the pools starts and ends on 16 bytes
    const uintptr_t pools = reinterpret_cast<uintptr_t>(a.pool[0]) | reinterpret_cast<uintptr_t>(a.pool[1]);
    const bool wide = row_bytes % 16 == 0 && a.page_stride * elt % 16 == 0 && pools % 16 == 0;
    const int vec = wide ? 16 : elt;
    const int units = (int)(row_bytes / vec);
    const int64_t blocks = ((int64_t)a.T * ((units + 127) / 128) + 7) / 8;
    const dim3 grid((unsigned)(blocks < most ? blocks : most), a.n_src);
    if (wide)
      append_copy_kernel<uint4><<<grid, 256, 0, st>>>(a, units, 16 / elt);
    else if (elt == 4)
      append_copy_kernel<uint32_t><<<grid, 256, 0, st>>>(a, units, 1);
    else
      append_copy_kernel<uint16_t><<<grid, 256, 0, st>>>(a, units, 1);
  }
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa

using namespace dsa;

namespace {

// Whether every pointer is a multiple of n bytes (null ones are).
template <typename... P>
bool aligned(uintptr_t n, const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & (n - 1)) == 0;
}

size_t plan_bytes(int B) { return sizeof(WsHeader) + 256 + (((size_t)B + 1) * 4 + 255) / 256 * 256; }

}  // namespace

extern "C" {

int dsa_page_plan_workspace_size(int B, int max_tokens, size_t* bytes) {
  if (!bytes || B < 0 || B > (1 << 20) || max_tokens < 0) return DSA_ERR_INVALID_ARG;
  *bytes = plan_bytes(B);
  return DSA_OK;
}

int dsa_page_plan(const int32_t* lens, const int32_t* new_lens, const int32_t* free_pages, int n_free,
                  const int32_t* used, int B, int page, int n_pages, int max_pages, int max_tokens,
                  int32_t* block_table, int32_t* q_offsets, int64_t* slots, int32_t* positions,
                  int32_t* lens_out, int32_t* used_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || B > (1 << 20) || page < 1 || n_pages < 1 || max_pages < 1 || n_free < 0 || max_tokens < 0)
    return DSA_ERR_INVALID_ARG;
  if ((int64_t)max_pages * page >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
  if (B == 0) return DSA_OK;
  if (!lens || !new_lens || !used || !block_table || !q_offsets || !lens_out || !used_out || !workspace)
    return DSA_ERR_INVALID_ARG;
  if ((n_free > 0 && !free_pages) || (max_tokens > 0 && (!slots || !positions))) return DSA_ERR_INVALID_ARG;
  if (!aligned(16, workspace) || !aligned(8, slots) ||
      !aligned(4, lens, new_lens, free_pages, used, block_table, q_offsets, positions, lens_out, used_out))
    return DSA_ERR_INVALID_ARG;
  if (workspace_bytes < plan_bytes(B)) return DSA_ERR_WORKSPACE;
  int sms = 0;
  const int r = current_device(nullptr, &sms);
  if (r != DSA_OK) return r;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PlanArgs a;
  a.lens = lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.used = used;
  a.n_free = n_free;
  a.B = B;
  a.page = page;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.max_tokens = max_tokens;
  a.table = block_table;
  a.q_off = q_offsets;
  a.slots = slots;
  a.positions = positions;
  a.lens_out = lens_out;
  a.used_out = used_out;
  a.status = reinterpret_cast<int*>(ws);
  a.state = reinterpret_cast<int32_t*>(ws + sizeof(WsHeader));
  a.first = reinterpret_cast<int32_t*>(ws + sizeof(WsHeader) + 256);
  return launch_page_plan(a, sms, static_cast<cudaStream_t>(stream));
}

int dsa_page_append(const void* k, const void* v, const int64_t* slots, int T, int Hkv, int d, int src_dtype,
                    int kv_dtype, void* K, void* V, float* K_scale, float* V_scale, int n_pages, int page,
                    int64_t page_stride, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || Hkv < 1 || d < 1 || n_pages < 1 || page < 1) return DSA_ERR_INVALID_ARG;
  if (d > 256 || Hkv > 1024) return DSA_ERR_UNSUPPORTED;
  if (src_dtype != DSA_DTYPE_BF16 && src_dtype != DSA_DTYPE_FP32) return DSA_ERR_UNSUPPORTED;
  if (kv_dtype != src_dtype && kv_dtype != DSA_DTYPE_FP8_E4M3) return DSA_ERR_UNSUPPORTED;
  if (page_stride < (int64_t)page * Hkv * d) return DSA_ERR_INVALID_ARG;
  if (T == 0) return DSA_OK;
  if (!k || !slots || !K || !workspace || (v == nullptr) != (V == nullptr)) return DSA_ERR_INVALID_ARG;
  const bool scaled = kv_dtype == DSA_DTYPE_FP8_E4M3;
  if (scaled != (K_scale != nullptr) || (scaled && V != nullptr) != (V_scale != nullptr)) return DSA_ERR_INVALID_ARG;
  const uintptr_t elt = kv_dtype == DSA_DTYPE_FP32 ? 4 : (kv_dtype == DSA_DTYPE_BF16 ? 2 : 1);
  if (!aligned(16, k, v, workspace) || !aligned(elt, K, V) || !aligned(8, slots) || !aligned(4, K_scale, V_scale))
    return DSA_ERR_INVALID_ARG;
  if (workspace_bytes < sizeof(WsHeader)) return DSA_ERR_WORKSPACE;
  int sms = 0;
  const int r = current_device(nullptr, &sms);
  if (r != DSA_OK) return r;
  AppendArgs a;
  a.src[0] = k;
  a.src[1] = v;
  a.pool[0] = K;
  a.pool[1] = V;
  a.scale[0] = K_scale;
  a.scale[1] = V_scale;
  a.slots = slots;
  a.T = T;
  a.Hkv = Hkv;
  a.d = d;
  a.n_pages = n_pages;
  a.page = page;
  a.n_src = v ? 2 : 1;
  a.page_stride = page_stride;
  a.status = static_cast<int*>(workspace);
  return launch_page_append(a, src_dtype, kv_dtype, sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
