// dsa_pages.cu — page plan (block tables and slot maps from request lengths)
// and the cache write.
//
// Plan.  With P tokens a page, request b holds ceil(len / P) pages and needs
// ceil((len + new) / P).  Two exclusive sums over the requests (new tokens,
// new pages) give q_offsets and each request's first entry of the free list;
// after that every table entry and every token is independent of the others:
// a token finds its request by bisection in q_offsets.  The sums run in one
// block, so their order is fixed and no atomics are needed.
//
// Cache write.  A row is Hkv * d contiguous elements at its slot: a copy, or
// for e4m3 pages one pass per (row, head) that holds the d elements in
// registers, reduces their amax across the lanes, and stores the bytes and
// the scale.
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
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int64_t before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += warp_sum[w][i];
      all += warp_sum[w][i];
    }
    v[i] = inc[i] - v[i] + before;
    total[i] = all;
  }
  __syncthreads();
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
  v[1] = (n + m + a.page - 1ll) / a.page - (n + a.page - 1ll) / a.page;
  return true;
}

// Both sums and the checks, by one block.  Leaves q_off, first, lens_out,
// used_out and the entry state; a step that fails leaves zero sums.
__device__ __forceinline__ void plan_sums(const PlanArgs& a) {
  __shared__ int64_t warp_sum[kPlanThreads / 32][2];
  const int used = a.used[0];
  int64_t total[2] = {0, 0};
  bool ok = used >= 0 && used <= a.n_free;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {  // totals first: all or nothing
    const int b = b0 + threadIdx.x;
    int64_t v[2] = {0, 0}, t[2];
    int len;
    if (b < a.B) ok = plan_request(a, b, v, len) && ok;
    block_scan2(v, t, warp_sum);
    total[0] += t[0];
    total[1] += t[1];
  }
  ok = __syncthreads_and(ok && total[0] <= a.max_tokens);
  const bool enough = total[1] <= (int64_t)a.n_free - used;
  if (threadIdx.x == 0 && !(ok && enough)) report_error(a.status, ok ? DSA_ERR_PAGES : DSA_ERR_INVALID_ARG, 50);
  ok = ok && enough;
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
  const int id = a.free_pages[used + i];
  if ((unsigned)id < (unsigned)a.n_pages) return id;
  report_error(a.status, DSA_ERR_INVALID_ARG, 51);
  return -1;
}

// Table entries and tokens t, t + step, ...
__device__ __forceinline__ void plan_fill(const PlanArgs& a, int64_t t, int64_t step) {
  const int n_new = a.q_off[a.B], n_fresh = a.first[a.B], used = a.state[0];
  for (int64_t i = t; i < n_fresh; i += step) {
    const int b = bisect(a.first, a.B, (int)i);
    const int m = a.q_off[b + 1] - a.q_off[b], len = a.lens_out[b] - m;
    const int held = (int)((len + a.page - 1ll) / a.page);
    a.table[(int64_t)b * a.max_pages + held + ((int)i - a.first[b])] = fresh_page(a, used, (int)i);
  }
  for (int64_t i = t; i < a.max_tokens; i += step) {
    int64_t slot = -1;
    int pos = -1;
    if (i < n_new) {
      const int b = bisect(a.q_off, a.B, (int)i);
      const int q0 = a.q_off[b], m = a.q_off[b + 1] - q0, len = a.lens_out[b] - m;
      pos = len + (int)i - q0;
      const int held = (int)((len + a.page - 1ll) / a.page), col = pos / a.page;
      int id;
      if (col < held) {  // the last page the request held already
        id = a.table[(int64_t)b * a.max_pages + col];
        if ((unsigned)id >= (unsigned)a.n_pages) {
          report_error(a.status, DSA_ERR_INVALID_ARG, 52);
          id = -1;
        }
      } else {
        id = fresh_page(a, used, a.first[b] + col - held);
      }
      if (id >= 0) slot = (int64_t)id * a.page + (pos - col * a.page);
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_sums_kernel(const PlanArgs a) { plan_sums(a); }

__global__ void __launch_bounds__(256) page_plan_fill_kernel(const PlanArgs a) {
  plan_fill(a, (int64_t)blockIdx.x * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x);
}

int launch_page_plan(const PlanArgs& a, int sms, cudaStream_t st) {
  const NvtxRange nvtx("dsa.page_plan");
  page_plan_sums_kernel<<<1, kPlanThreads, 0, st>>>(a);
  const int64_t items = (int64_t)a.max_tokens > a.B ? a.max_tokens : a.B;
  const int64_t blocks = (items + 255) / 256, most = (int64_t)sms * 8;
  page_plan_fill_kernel<<<(int)(blocks < most ? blocks : most), 256, 0, st>>>(a);
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
  const int64_t id = slot / a.page;
  return id * a.page_stride + (slot - id * a.page) * a.Hkv * a.d;
}

// Same type in source and pool: rows of `units` vectors of type V.
template <typename V>
__global__ void __launch_bounds__(256) append_copy_kernel(const AppendArgs a, int units, int per_vec) {
  const int which = blockIdx.y;
  const V* src = static_cast<const V*>(a.src[which]);
  V* pool = static_cast<V*>(a.pool[which]);
  const int64_t n = (int64_t)a.T * units;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / units;
    const int64_t row = slot_row(a, a.slots[t]);
    if (row >= 0) pool[row / per_vec + (i - t * units)] = src[i];
  }
}

// e4m3 pages: one warp a (row, head), lane l holds elements l, l + 32, ...
template <typename S>
__global__ void __launch_bounds__(256) append_e4m3_kernel(const AppendArgs a) {
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
      top = fmaxf(top, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = fmaxf(__fdiv_rn(top, 448.f), 1.17549435e-38f);
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
    const int64_t rows = (int64_t)a.T * a.Hkv, blocks = (rows + 7) / 8;
    const dim3 grid((unsigned)(blocks < most ? blocks : most), a.n_src);
    if (src_dtype == DSA_DTYPE_FP32)
      append_e4m3_kernel<float><<<grid, 256, 0, st>>>(a);
    else
      append_e4m3_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  } else {
    const int elt = src_dtype == DSA_DTYPE_FP32 ? 4 : 2;
    const int64_t row_bytes = (int64_t)a.Hkv * a.d * elt;
    // 16-byte vectors when every row of the pools starts and ends on 16 bytes
    const uintptr_t pools = reinterpret_cast<uintptr_t>(a.pool[0]) | reinterpret_cast<uintptr_t>(a.pool[1]);
    const bool wide = row_bytes % 16 == 0 && a.page_stride * elt % 16 == 0 && pools % 16 == 0;
    const int vec = wide ? 16 : elt;
    const int units = (int)(row_bytes / vec);
    const int64_t blocks = ((int64_t)a.T * units + 255) / 256;
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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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
  if (!aligned16(k) || !aligned16(v) || reinterpret_cast<uintptr_t>(K) % elt || reinterpret_cast<uintptr_t>(V) % elt)
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
