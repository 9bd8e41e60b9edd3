// dsa_attend.cu — attention over the paged cache: the C entry points and the
// general kernel.
//
// General kernel.  o = sum_s p_s v_s / sum_s p_s with p_s = exp(c q.k_s - m),
// m the running maximum: one pass over the keys, the old sums scaled by
// exp(m_old - m_new) whenever m grows.  A warp takes one (query row, head) and
// steps through its keys 32 at a time (a lane looks up one key's slot); eight
// lanes share a key, an eighth of the head each, so a key costs two wide loads
// a lane and three shuffles, and the warp's four groups of lanes keep a few
// keys each in flight; their sums are joined at the end.  All fp32: it serves
// fp32 queries, where the weights' bf16 rounding of the tensor-core kernel
// would not do, and the head sizes and alignments that kernel has no tiles
// for.  Four warps share a row when rows are few (then also split over blocks,
// whose parts a second kernel joins).  Gathered rows come from L2: 2048 rows of
// 4 heads of 64, 64 entries each, read 268 MB of a 4 MB cache in 28 us.
#include <cmath>

#include "dsa_paged.cuh"

namespace dsa {

constexpr int kGenWarps = 4;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(uint8_t x) { return e4m3_to_f32(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// This lane's eighth of a row: elements e + i of each vector of kE, zero
// behind d.  kVec: rows start on the vectors' alignment and d holds whole ones.
template <typename T, int kD, bool kVec>
__device__ __forceinline__ void load_eighth(const T* row, int sub, int d, float (&x)[kD]) {
  constexpr int kE = 16 / (int)sizeof(T) < kD ? 16 / (int)sizeof(T) : kD;
#pragma unroll
  for (int u = 0; u < kD / kE; ++u) {
    const int e = (u * 8 + sub) * kE;
    if constexpr (kVec) {
      struct alignas(sizeof(T) * kE) Vec { T v[kE]; } v;
      if (e < d) {
        v = *reinterpret_cast<const Vec*>(row + e);
#pragma unroll
        for (int i = 0; i < kE; ++i) x[u * kE + i] = to_f32(v.v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kE; ++i) x[u * kE + i] = 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) x[u * kE + i] = e + i < d ? to_f32(row[e + i]) : 0.f;
    }
  }
}

// The element that x[i] of load_eighth holds.
template <typename T, int kD>
__device__ __forceinline__ int eighth_element(int i, int sub) {
  constexpr int kE = 16 / (int)sizeof(T) < kD ? 16 / (int)sizeof(T) : kD;
  return ((i / kE) * 8 + sub) * kE + i % kE;
}

// kD: elements of the head a lane holds (d <= 8 kD); kShare: warps a row.
template <typename TQ, typename TK, int kD, bool kVec, int kShare>
__global__ void __launch_bounds__(kGenWarps * 32) attend_general_kernel(const AttendArgs a, int splits) {
  constexpr int kKeys = kD <= 16 ? 2 : 1;  // keys in flight in a group of lanes
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane >> 3, sub = lane & 7;
  const int64_t task = kShare == 1 ? (int64_t)blockIdx.x * kGenWarps + warp : blockIdx.x;
  const int split = (int)(task % splits);
  const int64_t rh = task / splits;
  if (rh >= (int64_t)a.total_q * a.Hq) return;  // only with kShare == 1: no barrier below
  const int row = (int)(rh / a.Hq), h = (int)(rh % a.Hq), hk = h / (a.Hq / a.Hkv);
  const RowSeq rs = find_row(a, row);
  if (rs.b < 0) return;  // padding: its outputs stay
  // entries this row scans: list entries, or the tokens up to its position
  const int n = a.idx != nullptr ? a.k : max(0, rs.pos + 1);
  const int chunk = (n + splits - 1) / splits;
  const int n0 = min(n, split * chunk), n1 = min(n, n0 + chunk);
  const TK* K = static_cast<const TK*>(a.K);
  const TK* V = static_cast<const TK*>(a.V);
  float q[kD], o[kD], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kD; ++i) {  // in the keys' order of elements
    const int e = eighth_element<TK, kD>(i, sub);
    q[i] = e < a.d ? to_f32(static_cast<const TQ*>(a.Q)[rh * a.d + e]) * a.scale : 0.f;
    o[i] = 0.f;
  }
  for (int s0 = n0 + (kShare == 1 ? 0 : warp * 32); s0 < n1; s0 += kShare * 32) {
    // this lane's key: element offset of its row, -1 when it is skipped
    int64_t at = -1;
    float ks = 1.f, vs = 1.f;
    if (s0 + lane < n1) {
      const int pos = a.idx != nullptr ? a.idx[(int64_t)row * a.k + s0 + lane] : s0 + lane;
      if (pos >= 0 && pos <= rs.pos) {
        int off;
        const int id = page_of(a, rs.b, pos, off);
        if (id >= 0) {
          at = (int64_t)id * a.page_stride + ((int64_t)off * a.Hkv + hk) * a.d;
          if (!in_bounds(cache_ok(a, at), a.status, 21)) at = -1;
          if (a.K_scale != nullptr) {
            const int64_t sc = ((int64_t)id * a.page + off) * a.Hkv + hk;
            ks = a.K_scale[sc];
            vs = a.V_scale[sc];
          }
        }
      }
    }
    const int cnt = min(32, n1 - s0);
    for (int j0 = 0; j0 < cnt; j0 += 4 * kKeys) {  // key j0 + 4 i + grp
      float s[kKeys], kv[kKeys][kD], w[kKeys];
      int64_t p[kKeys];
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        p[i] = __shfl_sync(0xffffffffu, at, (j0 + 4 * i + grp) & 31);
        if (j0 + 4 * i + grp >= cnt) p[i] = -1;
        if (p[i] >= 0) load_eighth<TK, kD, kVec>(K + p[i], sub, a.d, kv[i]);
      }
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        float dot = 0.f;
        if (p[i] >= 0) {
#pragma unroll
          for (int e = 0; e < kD; ++e) dot = fmaf(q[e], kv[i][e], dot);
          load_eighth<TK, kD, kVec>(V + p[i], sub, a.d, kv[i]);
        }
        s[i] = dot;
      }
#pragma unroll
      for (int x = 4; x > 0; x >>= 1)
#pragma unroll
        for (int i = 0; i < kKeys; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], x);
      float top = m;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        const float k = __shfl_sync(0xffffffffu, ks, (j0 + 4 * i + grp) & 31);
        w[i] = __shfl_sync(0xffffffffu, vs, (j0 + 4 * i + grp) & 31);
        s[i] = p[i] >= 0 ? s[i] * k : -INFINITY;
        top = max_nan(top, s[i]);
      }
      if (top == -INFINITY) continue;  // nothing seen yet (the same in the group's lanes)
      if (!(top <= m)) {  // a larger maximum, or a NaN, which then stays
        const float keep = expf(m - top);
        m = top;
        l *= keep;
#pragma unroll
        for (int e = 0; e < kD; ++e) o[e] *= keep;
      }
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        if (p[i] < 0) continue;
        const float x = expf(s[i] - m), xv = x * w[i];
        l += x;
#pragma unroll
        for (int e = 0; e < kD; ++e) o[e] = fmaf(xv, kv[i][e], o[e]);
      }
    }
  }
  // the groups' sums, joined pairwise
#pragma unroll
  for (int x = 8; x <= 16; x <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, x), l2 = __shfl_xor_sync(0xffffffffu, l, x), top = max_nan(m, m2);
    const float f = m == -INFINITY ? 0.f : expf(m - top), f2 = m2 == -INFINITY ? 0.f : expf(m2 - top);
    m = top;
    l = l * f + l2 * f2;
#pragma unroll
    for (int e = 0; e < kD; ++e) o[e] = o[e] * f + __shfl_xor_sync(0xffffffffu, o[e], x) * f2;
  }
  if constexpr (kShare > 1) {  // the warps' parts, joined in warp order
    __shared__ float so[kShare][kD * 8], sm[kShare], sl[kShare];
    if (grp == 0) {
#pragma unroll
      for (int i = 0; i < kD; ++i) so[warp][i * 8 + sub] = o[i];
    }
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    __syncthreads();
    if (warp > 0) return;
    float top = sm[0];
#pragma unroll
    for (int w = 1; w < kShare; ++w) top = max_nan(top, sm[w]);
    l = 0.f;
#pragma unroll
    for (int i = 0; i < kD; ++i) o[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kShare; ++w) {
      const float f = sm[w] == -INFINITY ? 0.f : expf(sm[w] - top);
      l = fmaf(f, sl[w], l);
#pragma unroll
      for (int i = 0; i < kD; ++i) o[i] = fmaf(f, so[w][i * 8 + sub], o[i]);
    }
    m = top;
  }
  const bool last = splits == 1;
  const float inv = last ? inverse(l) : 1.f;
  if (grp == 0) {
#pragma unroll
    for (int i = 0; i < kD; ++i) {
      const int e = eighth_element<TK, kD>(i, sub);
      if (e >= a.d) continue;
      if (last)
        put(static_cast<TQ*>(a.out) + rh * a.d + e, o[i] * inv);
      else
        a.part_o[task * a.d + e] = o[i];
    }
  }
  if (lane == 0) {
    if (last) {
      if (a.lse != nullptr) a.lse[rh] = l == 0.f ? -INFINITY : m + logf(l);
    } else {
      a.part_ml[2 * task] = m;
      a.part_ml[2 * task + 1] = l;
    }
  }
}

// Joins the `splits` parts of each (row, head): one warp each.
template <typename TQ>
__global__ void __launch_bounds__(128) attend_join_kernel(const AttendArgs a, int splits) {
  const int64_t rh = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (rh >= (int64_t)a.total_q * a.Hq) return;
  if (find_row(a, (int)(rh / a.Hq)).b < 0) return;
  const float* ml = a.part_ml + 2 * rh * splits;
  float top = -INFINITY, sum = 0.f;
  for (int s = 0; s < splits; ++s) top = max_nan(top, ml[2 * s]);
  for (int s = 0; s < splits; ++s)
    if (ml[2 * s] != -INFINITY) sum = fmaf(expf(ml[2 * s] - top), ml[2 * s + 1], sum);
  const float inv = inverse(sum);
  for (int e = lane; e < a.d; e += 32) {
    float x = 0.f;
    for (int s = 0; s < splits; ++s)
      if (ml[2 * s] != -INFINITY) x = fmaf(expf(ml[2 * s] - top), a.part_o[(rh * splits + s) * a.d + e], x);
    put(static_cast<TQ*>(a.out) + rh * a.d + e, x * inv);
  }
  if (lane == 0 && a.lse != nullptr) a.lse[rh] = sum == 0.f ? -INFINITY : top + logf(sum);
}

template <typename TQ, typename TK, int kD>
static void run_general(const AttendArgs& a, int splits, bool share, cudaStream_t st) {
  constexpr int kE = 16 / (int)sizeof(TK) < kD ? 16 / (int)sizeof(TK) : kD;
  constexpr uintptr_t kBytes = kE * sizeof(TK);
  const bool vec = a.d % kE == 0 && a.page_stride % kE == 0 &&
                   (reinterpret_cast<uintptr_t>(a.K) | reinterpret_cast<uintptr_t>(a.V)) % kBytes == 0;
  const int64_t tasks = (int64_t)a.total_q * a.Hq * splits;
  const unsigned grid = (unsigned)(share ? tasks : (tasks + kGenWarps - 1) / kGenWarps);
  if (share && vec)
    attend_general_kernel<TQ, TK, kD, true, kGenWarps><<<grid, kGenWarps * 32, 0, st>>>(a, splits);
  else if (share)
    attend_general_kernel<TQ, TK, kD, false, kGenWarps><<<grid, kGenWarps * 32, 0, st>>>(a, splits);
  else if (vec)
    attend_general_kernel<TQ, TK, kD, true, 1><<<grid, kGenWarps * 32, 0, st>>>(a, splits);
  else
    attend_general_kernel<TQ, TK, kD, false, 1><<<grid, kGenWarps * 32, 0, st>>>(a, splits);
}

template <typename TQ, typename TK>
static int run_general(const AttendArgs& a, int splits, bool share, cudaStream_t st) {
  if (a.d <= 64)
    run_general<TQ, TK, 8>(a, splits, share, st);
  else if (a.d <= 128)
    run_general<TQ, TK, 16>(a, splits, share, st);
  else
    run_general<TQ, TK, 32>(a, splits, share, st);
  if (splits > 1) {
    const int64_t rh = (int64_t)a.total_q * a.Hq;
    attend_join_kernel<TQ><<<(unsigned)((rh + 3) / 4), 128, 0, st>>>(a, splits);
  }
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

int launch_attend_general(const AttendArgs& a, int q_dtype, int kv_dtype, int splits, bool share, cudaStream_t st) {
  const NvtxRange nvtx(a.idx != nullptr ? "dsa.attend_selected" : "dsa.attend_paged");
  if (q_dtype == DSA_DTYPE_FP32) return run_general<float, float>(a, splits, share, st);
  if (kv_dtype == DSA_DTYPE_BF16) return run_general<__nv_bfloat16, __nv_bfloat16>(a, splits, share, st);
  return run_general<__nv_bfloat16, uint8_t>(a, splits, share, st);
}

}  // namespace dsa

using namespace dsa;

namespace {

// Whether every pointer is a multiple of n bytes (null ones are).
template <typename... P>
bool aligned(uintptr_t n, const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & (n - 1)) == 0;
}

// Positions of a request that its table may span.
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 1024;

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// A (row, head) has a warp to itself when that makes 16 warps a
// multiprocessor, and four warps otherwise: 2048 rows of 4 heads, 64 entries
// each, take 28 us so and 65 us with four.
bool general_share(int sms, int total_q, int Hq) { return (int64_t)total_q * Hq < (int64_t)sms * 16; }

// Parts of the keys a (row, head) is split into: enough blocks for eight a
// multiprocessor, at most 64.
int general_splits(int sms, int total_q, int Hq) {
  const int64_t tasks = (int64_t)total_q * Hq, want = (int64_t)sms * 8;
  if (!general_share(sms, total_q, Hq)) return 1;
  const int64_t s = (want + tasks - 1) / tasks;
  return (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
}

struct AttendPlan {
  int splits;
  size_t ml_off, o_off, total;
};

AttendPlan plan_general(int sms, int total_q, int Hq, int d) {
  AttendPlan p;
  p.splits = general_splits(sms, total_q, Hq);
  const size_t parts = p.splits > 1 ? (size_t)total_q * Hq * p.splits : 0;
  p.ml_off = sizeof(WsHeader);
  p.o_off = p.ml_off + round256(parts * 8);
  p.total = p.o_off + round256(parts * d * 4);
  return p;
}

int check_attend(int B, int total_q, int Hq, int Hkv, int d, int q_dtype, int kv_dtype) {
  if (B < 0 || total_q < 0 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0) return DSA_ERR_INVALID_ARG;
  if (Hq > 1024 || Hq / Hkv > 128 || d > 256 || B > (1 << 20)) return DSA_ERR_UNSUPPORTED;
  if ((int64_t)total_q * Hq >= ((int64_t)1 << 30)) return DSA_ERR_UNSUPPORTED;
  const bool f32 = q_dtype == DSA_DTYPE_FP32 && kv_dtype == DSA_DTYPE_FP32;
  const bool b16 = q_dtype == DSA_DTYPE_BF16 && (kv_dtype == DSA_DTYPE_BF16 || kv_dtype == DSA_DTYPE_FP8_E4M3);
  return f32 || b16 ? DSA_OK : DSA_ERR_UNSUPPORTED;
}

// Query rows that read the same cache, at most: the heads of a group, and
// with all cached tokens a request's new queries (max_q; 1 for lists).
int shared_rows(int max_q, int Hq, int Hkv) {
  const int64_t rows = (int64_t)max_q * (Hq / Hkv);
  return rows < 128 ? (int)rows : 128;
}

// Either kernel may take the call (pages are not known yet): the larger need.
size_t attend_need(int sms, int total_q, int max_q, int Hq, int Hkv, int d, int q_dtype) {
  size_t n = plan_general(sms, total_q, Hq, d).total;
  if (q_dtype == DSA_DTYPE_BF16 && d <= 128) {
    const size_t tc = attend_tc_bytes(sms, shared_rows(max_q, Hq, Hkv), d);
    n = tc > n ? tc : n;
  }
  return n;
}

int attend_bytes(int B, int total_q, int max_q, int Hq, int Hkv, int d, int q_dtype, int kv_dtype, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  int r = check_attend(B, total_q, Hq, Hkv, d, q_dtype, kv_dtype);
  if (r != DSA_OK) return r;
  *bytes = sizeof(WsHeader);
  if (B == 0 || total_q == 0) return DSA_OK;
  int sms = 0;
  if ((r = current_device(nullptr, &sms)) != DSA_OK) return r;
  *bytes = attend_need(sms, total_q, max_q, Hq, Hkv, d, q_dtype);
  return DSA_OK;
}

// Both forms; idx == nullptr: all cached tokens.
int attend(AttendArgs& a, const float* softmax_scale, int q_dtype, int kv_dtype, void* workspace,
           size_t workspace_bytes, void* stream) {
  int r = check_attend(a.B, a.total_q, a.Hq, a.Hkv, a.d, q_dtype, kv_dtype);
  if (r != DSA_OK) return r;
  if (a.n_pages < 1 || a.page < 1 || a.max_pages < 1 || a.page_stride < (int64_t)a.page * a.Hkv * a.d)
    return DSA_ERR_INVALID_ARG;
  // the kernels round lengths up to tiles and step past them by a block's keys in 32 bits
  if ((int64_t)a.max_pages * a.page > kMaxTokens) return DSA_ERR_UNSUPPORTED;
  a.scale = softmax_scale != nullptr ? *softmax_scale : 1.f / std::sqrt((float)a.d);
  if (!std::isfinite(a.scale)) return DSA_ERR_INVALID_ARG;
  if (a.B == 0 || a.total_q == 0) return DSA_OK;
  if (!a.Q || !a.K || !a.V || !a.table || !a.lens || !a.q_off || !a.out || !workspace) return DSA_ERR_INVALID_ARG;
  const bool scaled = kv_dtype == DSA_DTYPE_FP8_E4M3;
  if (scaled != (a.K_scale != nullptr) || scaled != (a.V_scale != nullptr)) return DSA_ERR_INVALID_ARG;
  const uintptr_t elt = kv_dtype == DSA_DTYPE_FP32 ? 4 : (kv_dtype == DSA_DTYPE_BF16 ? 2 : 1);
  if (!aligned(16, a.Q, a.out, workspace) || !aligned(elt, a.K, a.V) ||
      !aligned(4, a.table, a.lens, a.q_off, a.idx, a.K_scale, a.V_scale, a.lse))
    return DSA_ERR_INVALID_ARG;
  int sms = 0;
  if ((r = current_device(nullptr, &sms)) != DSA_OK) return r;
  const int max_q = a.idx != nullptr ? 1 : a.max_q;
  if (workspace_bytes < attend_need(sms, a.total_q, max_q, a.Hq, a.Hkv, a.d, q_dtype)) return DSA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.status = reinterpret_cast<int*>(ws);
  if (attend_tc_ok(a, q_dtype, kv_dtype))
    return run_attend_tc(a, kv_dtype, shared_rows(max_q, a.Hq, a.Hkv), sms, ws, static_cast<cudaStream_t>(stream));
  const AttendPlan p = plan_general(sms, a.total_q, a.Hq, a.d);
  a.part_ml = reinterpret_cast<float*>(ws + p.ml_off);
  a.part_o = reinterpret_cast<float*>(ws + p.o_off);
  return launch_attend_general(a, q_dtype, kv_dtype, p.splits, general_share(sms, a.total_q, a.Hq),
                               static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int dsa_attend_paged_workspace_size(int B, int total_q, int max_q, int Hq, int Hkv, int d, int q_dtype,
                                    int kv_dtype, size_t* bytes) {
  if (max_q < 1 || max_q > 65536) return DSA_ERR_INVALID_ARG;
  return attend_bytes(B, total_q, max_q, Hq, Hkv, d, q_dtype, kv_dtype, bytes);
}

int dsa_attend_paged(const void* Q, const void* K, const void* V, const float* K_scale, const float* V_scale,
                     const int32_t* block_table, const int32_t* lens, const int32_t* q_offsets, int B, int total_q,
                     int max_q, int n_pages, int page, int64_t page_stride, int max_pages, int Hq, int Hkv, int d,
                     const float* softmax_scale, int q_dtype, int kv_dtype, void* out, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (max_q < 1 || max_q > 65536) return DSA_ERR_INVALID_ARG;
  AttendArgs a{};
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.K_scale = K_scale;
  a.V_scale = V_scale;
  a.table = block_table;
  a.lens = lens;
  a.q_off = q_offsets;
  a.B = B;
  a.total_q = total_q;
  a.max_q = max_q;
  a.n_pages = n_pages;
  a.page = page;
  a.page_stride = page_stride;
  a.max_pages = max_pages;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.out = out;
  a.lse = lse;
  return attend(a, softmax_scale, q_dtype, kv_dtype, workspace, workspace_bytes, stream);
}

int dsa_attend_selected_workspace_size(int B, int total_q, int k, int Hq, int Hkv, int d, int q_dtype, int kv_dtype,
                                       size_t* bytes) {
  if (k < 1 || k > 65536) return DSA_ERR_INVALID_ARG;
  return attend_bytes(B, total_q, 1, Hq, Hkv, d, q_dtype, kv_dtype, bytes);
}

int dsa_attend_selected(const void* Q, const void* K, const void* V, const float* K_scale, const float* V_scale,
                        const int32_t* block_table, const int32_t* lens, const int32_t* q_offsets,
                        const int32_t* idx, int k, int B, int total_q, int n_pages, int page, int64_t page_stride,
                        int max_pages, int Hq, int Hkv, int d, const float* softmax_scale, int q_dtype, int kv_dtype,
                        void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (k < 1 || k > 65536) return DSA_ERR_INVALID_ARG;
  if (B > 0 && total_q > 0 && !idx) return DSA_ERR_INVALID_ARG;
  AttendArgs a{};
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.K_scale = K_scale;
  a.V_scale = V_scale;
  a.table = block_table;
  a.lens = lens;
  a.q_off = q_offsets;
  a.idx = idx;
  a.k = k;
  a.B = B;
  a.total_q = total_q;
  a.n_pages = n_pages;
  a.page = page;
  a.page_stride = page_stride;
  a.max_pages = max_pages;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.out = out;
  a.lse = lse;
  return attend(a, softmax_scale, q_dtype, kv_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
