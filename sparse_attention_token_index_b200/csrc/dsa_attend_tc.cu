// dsa_attend_tc.cu — attention over the paged cache on the tensor cores.
//
// For one key head and up to N query rows that read the same tokens (the
// heads of the group, times the new queries of a request) and tiles of 128
// tokens:
//     S^T [128 tokens x N rows] = K  Q^T      (A = K tile,   B = Q)
//     P^T = 2^(c S^T - m)                      (m: a reference per row)
//     O^T [d x N rows]         += V^T P^T     (A = V^T tile, B = P)
// with the tokens, never the few query rows, on the 128-lane side of the
// product, so no lane is spent on padding: a softmax thread owns one token
// and N/2 of its rows.  Decoding reads each K and V row once for N rows, 2 N
// flops a byte, and at N <= 128 memory is the bound.
//
// One persistent CTA per SM:
//   * four loader warps turn positions into cache rows (page table, or list
//     entry and page table; a thread looks up one token, a tile ahead) and
//     fetch them by 16-byte asynchronous copies into a ring that K and V tiles
//     share, whatever the page size; a token that no row sees, and the columns
//     behind d, are filled with zeros, so no stale value meets a zero weight.
//     e4m3 rows land in a staging ring of which each thread reads back, once
//     they are there, the bytes it asked for, and writes them as bf16 (exact);
//   * the MMA warp issues S(t+1) before O(t), so that the tensor pipe has
//     work while the softmax of a tile runs;
//   * eight softmax warps: four cover the 128 tokens for the first N/2 rows,
//     four for the rest.
//
// The reference m is not the running maximum but one that no score has
// passed by more than 2^8: as long as that holds no sum needs rescaling, and
// whether it holds is one vote a tile.  When it fails (always in the first
// tile) the rows' true maxima become the new reference and O and the row
// sums are scaled once.  Weights lie in [0, 2^8], and their bf16 rounding
// (2^-8 relative) is the same as for weights in [0, 1]; row sums are fp32
// sums of the unrounded weights.
//
// The work (all tiles of all requests and key heads, end to end) is cut into
// equal runs, one per CTA, wherever the cuts fall: ragged batches and single
// long caches load every SM alike.  A (request, head, row block) that a cut
// divides leaves fp32 parts in the workspace, at most two a CTA, which a
// second kernel joins in tile order.
#include <atomic>

#include "dsa_paged.cuh"

namespace dsa {

constexpr int kTile = 128;           // tokens a tile
constexpr int kSoftWarps = 8;
constexpr int kLoadWarps = 4;
constexpr float kNoMax = -1.7e38f;   // reference of a row that has seen no token
constexpr float kSlack = 8.f;        // log2 of the largest weight

struct TcAttend {
  AttendArgs a;
  int row_stride_page;  // cache rows from one page to the next (page_stride / d)
  int unit_tiles;       // chosen positions: tiles of one (row, head)
  int64_t run;          // chosen positions: tiles of one CTA
  int min_run;          // all tokens: least tiles of one CTA
  struct JoinDesc* desc;
  uint64_t wait_ns;
};

// What the join kernel needs of the unit a CTA's run begins in.
struct JoinDesc {
  int64_t first, last;  // the unit's tiles, counted over all work
  int64_t run;
  int q0, hk, row0, rows;
};

// A unit: the tiles of one (request or row, key head, row block); a segment:
// the part of it in this CTA's run.
struct Seg {
  int b;           // request
  int q0;          // first query row of the unit
  int hk;
  int row0, rows;  // rows row0 .. row0 + rows - 1 of the unit's (query, head) rows, at most N
  int lim0;        // position of the unit's query row 0 (all tokens) / of the row (chosen)
  int end;         // tokens visible to some row of the block (all tokens) / entries (chosen)
  int tile0, tiles;
  int unit_tiles;
  bool valid;
};

__device__ __forceinline__ bool request_ok(const AttendArgs& a, int b, int& q0, int& m, int& len) {
  q0 = a.q_off[b];
  const int q1 = a.q_off[b + 1];
  len = a.lens[b];
  m = q1 - q0;
  return q0 >= 0 && q1 >= q0 && q1 <= a.total_q && m <= a.max_q && len >= 0 &&
         (int64_t)len <= (int64_t)a.max_pages * a.page;
}

// Tiles of row block rb of a request, and the tokens some row of it sees.
template <int N>
__device__ __forceinline__ int block_tiles(int m, int g, int len, int rb, int& end) {
  const int last = min(m * g, (rb + 1) * N) - 1;
  end = max(0, len - m + last / g + 1);
  return max(1, (end + kTile - 1) / kTile);
}

template <int N>
__device__ __forceinline__ int64_t request_tiles(const AttendArgs& a, int b) {
  int q0, m, len;
  if (!request_ok(a, b, q0, m, len)) {
    report_error(a.status, DSA_ERR_INVALID_ARG, 42);
    return 0;
  }
  const int g = a.Hq / a.Hkv, blocks = (m * g + N - 1) / N;
  int64_t sum = 0;
  int end;
  for (int rb = 0; rb < blocks; ++rb) sum += block_tiles<N>(m, g, len, rb, end);
  return sum * a.Hkv;
}

// Steps through the segments of a CTA's run; every role keeps its own.
template <int N, bool kSel>
struct Walk {
  int64_t left;  // tiles still to hand out
  int b, hk, rb, off;
  int q0, m, len, q1;
  int row;

  __device__ __forceinline__ void start(const TcAttend& t, int64_t n, int b_, int64_t off_) {
    left = n;
    if constexpr (kSel) {
      const int64_t u = off_ / t.unit_tiles;
      row = (int)(u / t.a.Hkv);
      hk = (int)(u % t.a.Hkv);
      off = (int)(off_ % t.unit_tiles);
      q0 = q1 = 0;
      b = 0;
    } else {
      b = b_;
      rb = hk = 0;
      if (n > 0) {
        load(t.a);
        int64_t per_head = 0;
        int end;
        const int g = t.a.Hq / t.a.Hkv, blocks = (m * g + N - 1) / N;
        for (int i = 0; i < blocks; ++i) per_head += block_tiles<N>(m, g, len, i, end);
        hk = (int)(off_ / per_head);
        int64_t o = off_ % per_head;
        for (int n_t; o >= (n_t = block_tiles<N>(m, g, len, rb, end)); ++rb) o -= n_t;
        off = (int)o;
      }
    }
  }

  // all tokens: request b, or the next one with rows
  __device__ __forceinline__ void load(const AttendArgs& a) {
    while (b < a.B) {
      if (request_ok(a, b, q0, m, len) && m > 0) return;
      ++b;
    }
  }

  __device__ __forceinline__ bool next(const TcAttend& t, Seg& s) {
    if (left <= 0) return false;
    const AttendArgs& a = t.a;
    const int g = a.Hq / a.Hkv;
    s.valid = true;
    s.hk = hk;
    s.tile0 = off;
    if constexpr (kSel) {
      s.unit_tiles = t.unit_tiles;
      if (row < q0 || row >= q1) {  // another request's row
        const RowSeq r = find_row(a, row);
        b = r.b;
        if (r.b >= 0) {
          q0 = a.q_off[r.b];
          q1 = a.q_off[r.b + 1];
          len = r.len;
        } else {
          q0 = q1 = 0;
        }
      }
      s.valid = b >= 0;
      s.b = b;
      s.q0 = row;
      s.row0 = 0;
      s.rows = g;
      s.lim0 = len - (q1 - q0) + (row - q0);
      s.end = a.k;
    } else {
      s.b = b;
      s.unit_tiles = block_tiles<N>(m, g, len, rb, s.end);
      s.q0 = q0;
      s.row0 = rb * N;
      s.rows = min(N, m * g - rb * N);
      s.lim0 = len - m;
    }
    s.tiles = (int)min((int64_t)(s.unit_tiles - off), left);
    left -= s.tiles;
    off = 0;
    if constexpr (kSel) {
      if (++hk == a.Hkv) {
        hk = 0;
        ++row;
      }
    } else {
      if (++rb == (m * g + N - 1) / N) {
        rb = 0;
        if (++hk == a.Hkv) {
          hk = 0;
          ++b;
          if (left > 0) load(a);
        }
      }
    }
    return true;
  }
};

// ----------------------------------------------------------------------------
// PTX
// ----------------------------------------------------------------------------
// 16 bytes to shared memory; ok == false fills them with zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16u : 0u) : "memory");
}

// The barrier gets this thread's arrival once all its copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Descriptor of an operand whose M (or N) extent is contiguous, in rows (one
// a token, along K) of kRow = 32, 64 or 128 bytes swizzled over that width:
// the stride byte offset leads from one group of 8 rows to the next, the
// leading byte offset from one 128-byte chunk of M to the next.
template <int kRow>
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t smem_addr, uint32_t chunk_bytes) {
  constexpr uint64_t kMode = kRow == 128 ? 2 : (kRow == 64 ? 4 : 6);
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(chunk_bytes >> 4) << 16;
  d |= (uint64_t)((8 * kRow) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= kMode << 61;
  return d;
}

template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[C]) {
  if constexpr (C == 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
  } else if constexpr (C == 16) {
    tmem_ld_32x32b_x16(taddr, v);
  } else {
    static_assert(C == 32, "8, 16 or 32 columns");
    tmem_ld_32x32b_x32(taddr, v);
  }
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool bar_or(int bar, int nthr, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(bar), "r"(nthr)
      : "memory");
  return r != 0;
}

// One value per column (of C <= 32) reduced over the 32 lanes: at each step
// half of the columns go to the partner lane.  Lane l gets column l % C.
template <int C, bool kMax>
__device__ __forceinline__ float warp_columns(float (&v)[C]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = C / 2; w >= 1; w >>= 1) {
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const bool up = (lane & w) != 0;
      const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, w);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  float x = v[0];
#pragma unroll
  for (int w = C; w < 32; w <<= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, x, w);
    x = kMax ? fmaxf(x, got) : x + got;
  }
  return x;
}

// ----------------------------------------------------------------------------
// shared memory
// ----------------------------------------------------------------------------
template <int N, int D, bool kFp8>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kSlotBytes = kTile * D * 2;   // one K or V tile, bf16
  static constexpr int kRawBytes = kTile * D;        // one e4m3 tile
  static constexpr int kQBytes = N * D * 2;
  static constexpr int kQBufs = N <= (kFp8 ? 32 : 64) ? 2 : 1;
  static constexpr int kPBytes = N * kTile * 2;
  static constexpr int kPRow = N >= 64 ? 128 : N * 2;  // bytes of a P row (of its first 64 columns)
  static constexpr int kRaw = kFp8 ? (N >= 128 && D >= 128 ? 3 : 4) : 0;
  static constexpr int kOther = kQBufs * kQBytes + 2 * kPBytes + kRaw * kRawBytes;
  static constexpr int kBudget = 232448 - 1024 - 8192;
  static constexpr int kFit = (kBudget - kOther) / kSlotBytes;
  static constexpr int kSlots = kFit > 8 ? 8 : kFit;
  static constexpr int kWarps = kSoftWarps + 1 + kLoadWarps;
  static constexpr int kCols = N >= 128 ? 512 : (N >= 64 ? 256 : (N >= 32 ? 128 : 64));
  static_assert(kSlots >= 2, "the ring holds a K and a V tile");
};

template <int N, int D, bool kFp8>
struct AttendSmem {
  using C = Cfg<N, D, kFp8>;
  uint8_t ring[C::kSlots][C::kSlotBytes];
  uint8_t q[C::kQBufs][C::kQBytes];
  uint8_t p[2][C::kPBytes];
  uint8_t raw[C::kRaw ? C::kRaw : 1][C::kRaw ? C::kRawBytes : 16];
  uint64_t full[C::kSlots], empty[C::kSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2];
  uint64_t o_full, o_free, drain;
  float red[2][4][N / 2];
  float mref[N], fac[N], lsum[N];
  int lim[N], orow[N];
  int64_t sums[32];
  int64_t begin_off, total;
  int begin_b;
  uint32_t tmem_base;
  int abort_flag;
};

// ----------------------------------------------------------------------------
// the kernel
// ----------------------------------------------------------------------------
template <int N, int D, bool kFp8, bool kSel>
__global__ void __launch_bounds__(Cfg<N, D, kFp8>::kWarps * 32, 1)
    attend_tc_kernel(const __grid_constant__ TcAttend t) {
  using C = Cfg<N, D, kFp8>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto& S = *reinterpret_cast<AttendSmem<N, D, kFp8>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const AttendArgs& a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kMma = kSoftWarps;
  const uint64_t budget = t.wait_ns ? t.wait_ns : kWaitNs;
  volatile int* abort_flag = &S.abort_flag;
  const int g = a.Hq / a.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&S.full[i], kFp8 ? kLoadWarps : kLoadWarps * 32);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], kLoadWarps * 32);
      mbar_init(&S.q_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.s_empty[i], kSoftWarps);
      mbar_init(&S.p_full[i], kSoftWarps);
      mbar_init(&S.p_empty[i], 1);
    }
    mbar_init(&S.o_full, 1);
    mbar_init(&S.o_free, kSoftWarps);
    mbar_init(&S.drain, 1);
    S.abort_flag = 0;
    S.begin_b = 0;
    S.begin_off = 0;
    fence_barrier_init();
  }
  if (warp == kMma) tmem_alloc(&S.tmem_base, C::kCols);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's run of tiles ----
  int64_t begin, run;
  if constexpr (kSel) {
    run = t.run;
    begin = (int64_t)blockIdx.x * run;
    const int64_t total = (int64_t)a.total_q * a.Hkv * t.unit_tiles;
    if (threadIdx.x == 0) S.total = total;
  } else {
    // each thread sums a contiguous share of the requests; a block scan; the
    // thread whose share holds the run's first tile names request and offset
    const int threads = C::kWarps * 32, share = (a.B + threads - 1) / threads;
    const int b0 = min(a.B, (int)threadIdx.x * share), b1 = min(a.B, b0 + share);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += request_tiles<N>(a, b);
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) S.sums[warp] = inc;
    __syncthreads();
    int64_t before = inc - mine, total = 0;
    for (int w = 0; w < C::kWarps; ++w) {
      if (w < warp) before += S.sums[w];
      total += S.sums[w];
    }
    run = (total + gridDim.x - 1) / gridDim.x;
    if (run < t.min_run) run = t.min_run;
    begin = (int64_t)blockIdx.x * run;
    if (begin >= before && begin < before + mine) {
      int64_t at = before;
      int b = b0;
      for (int64_t n; begin >= at + (n = request_tiles<N>(a, b)); ++b) at += n;
      S.begin_b = b;
      S.begin_off = begin - at;
    }
    if (threadIdx.x == 0) S.total = total;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = S.tmem_base;
  const int64_t n_tiles = max((int64_t)0, min(run, S.total - begin));
  Walk<N, kSel> walk;
  walk.start(t, n_tiles, S.begin_b, kSel ? begin : S.begin_off);
  Seg s;

  if (threadIdx.x == 0) {  // the join's description of the unit this run begins in
    JoinDesc d;
    d.rows = 0;
    d.run = run;
    d.first = d.last = begin;
    d.q0 = d.hk = d.row0 = 0;
    if (n_tiles > 0) {
      Walk<N, kSel> w = walk;
      w.next(t, s);
      d.rows = s.valid ? s.rows : 0;
      d.first = begin - s.tile0;
      d.last = d.first + s.unit_tiles;
      d.q0 = s.q0;
      d.hk = s.hk;
      d.row0 = s.row0;
    }
    t.desc[blockIdx.x] = d;
  }

  if (warp > kMma) {
    // ---------------- loaders: positions -> cache rows -> copies ----------------
    const int lw = warp - kMma - 1, tid = lw * 32 + lane;
    constexpr int kElt = kFp8 ? 1 : 2, kUnits = D * kElt / 16;  // 16-byte units of a cache row
    constexpr int kRowsAt = 32 / kUnits;                        // rows a warp copies at a time
    const int unit = lane % kUnits, sub = lane / kUnits;
    const bool unit_ok = unit * 16 < a.d * kElt;
    const int64_t row_bytes = (int64_t)a.d * kElt;
    const uint8_t* pages[2] = {static_cast<const uint8_t*>(a.K) + unit * 16, static_cast<const uint8_t*>(a.V) + unit * 16};
    int fill = 0, qn = 0, ready = 0;  // tiles asked for, queries, e4m3 tiles converted
    bool ok = true;
    auto convert = [&]() {  // e4m3 tile `ready`: this thread's bytes, staged -> ring
      const int r = ready % C::kSlots;
      ok = ok && mbar_wait<true>(&S.empty[r], ((ready / C::kSlots) & 1) ^ 1, abort_flag, a.status, 76, budget);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const uint8_t* src = S.raw[ready % C::kRaw] + tid * 16;
      uint8_t* dst0 = S.ring[r] + (unit >> 2) * kTile * 128;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const uint4 raw = *reinterpret_cast<const uint4*>(src + i * kLoadWarps * 512);
        uint32_t w[8];
        const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __half2_raw h =
              __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(in[e >> 1] >> (16 * (e & 1))), __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
          w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        const int row = lw * 32 + i * kRowsAt + sub, u0 = (unit & 3) * 2, sw = row & 7;
        uint8_t* dst = dst0 + row * 128;
        *reinterpret_cast<uint4*>(dst + ((u0 ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(dst + (((u0 + 1) ^ sw) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.full[r]);
      ++ready;
    };
    while (ok && walk.next(t, s)) {
      if (!s.valid) continue;
      {  // the segment's queries
        const int qb = qn % C::kQBufs;
        if (kFp8 && C::kQBufs == 1) {
          // the only query buffer is free once the last keys, still staged, are multiplied
          asm volatile("cp.async.wait_all;" ::: "memory");
          while (ok && ready < fill) convert();
        }
        if (ok && qn >= C::kQBufs)
          ok = mbar_wait<true>(&S.q_empty[qb], (qn / C::kQBufs - 1) & 1, abort_flag, a.status, 70, budget);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* Q = static_cast<const uint8_t*>(a.Q);
        constexpr int kQUnits = D / 8;
        for (int e = tid; e < N * kQUnits; e += kLoadWarps * 32) {
          const int r = e / kQUnits, u = e % kQUnits, rr = s.row0 + r, j = rr / g;
          const bool in = r < s.rows && u * 8 < a.d;
          const int64_t at = in ? ((int64_t)(s.q0 + j) * a.Hq + s.hk * g + (rr - j * g)) * a.d + u * 8 : 0;
          copy16(smem_u32(S.q[qb]) + (u >> 3) * N * 128 + r * 128 + (((u & 7) ^ (r & 7)) << 4), Q + at * 2, in);
        }
        copies_arrive(&S.q_full[qb]);
        ++qn;
      }
      auto cache_row = [&](int tile) {  // cache row of this thread's token, -1: none
        const int e = tile * kTile + tid;
        int pos = -1;
        if (e < s.end) {
          pos = e;
          if constexpr (kSel) {
            pos = a.idx[(int64_t)s.q0 * a.k + e];
            if (pos > s.lim0) pos = -1;
          }
        }
        if (pos < 0) return -1;
        int off;
        const int id = page_of(a, s.b, pos, off);
        return id >= 0 ? id * t.row_stride_page + off * a.Hkv + s.hk : -1;
      };
      int next = cache_row(s.tile0);
      for (int j = 0; ok && j < s.tiles; ++j) {
        const int row = next;
        if (j + 1 < s.tiles) next = cache_row(s.tile0 + j + 1);  // a tile ahead of its copies
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++fill) {
          uint32_t dst;
          if constexpr (kFp8) {  // this thread has read what the stage held
            dst = smem_u32(S.raw[fill % C::kRaw]) + tid * 16;
          } else {
            const int r = fill % C::kSlots;
            ok = ok && mbar_wait<true>(&S.empty[r], ((fill / C::kSlots) & 1) ^ 1, abort_flag, a.status, 71, budget);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            dst = smem_u32(S.ring[r]) + (unit >> 3) * kTile * 128 + (lw * 32 + sub) * 128;
          }
#pragma unroll
          for (int i = 0; i < kUnits; ++i) {
            const int src = __shfl_sync(0xffffffffu, row, i * kRowsAt + sub);
            const bool in = src >= 0 && unit_ok;
            const uint8_t* from = pages[kv] + (in ? src * row_bytes : -(int64_t)unit * 16);
            if constexpr (kFp8)
              copy16(dst + i * kLoadWarps * 512, from, in);
            else
              copy16(dst + i * kRowsAt * 128 + (((unit & 7) ^ ((i * kRowsAt + sub) & 7)) << 4), from, in);
          }
          if constexpr (kFp8) {
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (fill - ready >= C::kRaw - 1) {
              asm volatile("cp.async.wait_group %0;" ::"n"(C::kRaw > 0 ? C::kRaw - 1 : 0) : "memory");
              convert();
              if (!ok) break;
            }
          } else {
            copies_arrive(&S.full[fill % C::kSlots]);
          }
        }
      }
    }
    // never leave with a copy in flight
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (kFp8)
      while (ok && ready < fill) convert();
  } else if (warp == kMma) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      constexpr uint32_t kIdescS = idesc_bf16_f32(128, N);
      constexpr uint32_t kIdescO = idesc_bf16_f32(D, N) | (1u << 15) | (1u << 16);  // A along M, B along N contiguous
      int n = 0, qn = 0, seg_done = 0;  // tiles issued, segments begun / ended
      bool ok = true, pending = false, pend_first = false, pend_last = false;
      auto values = [&](int i, bool first, bool last) {  // O += V^T P^T of tile i
        const int f = 2 * i + 1, r = f % C::kSlots, pb = i & 1;
        if (!mbar_wait(&S.full[r], (f / C::kSlots) & 1, abort_flag, a.status, 80, budget)) return false;
        if (!mbar_wait(&S.p_full[pb], (i >> 1) & 1, abort_flag, a.status, 81, budget)) return false;
        if (first && seg_done > 0 &&
            !mbar_wait(&S.o_free, (seg_done - 1) & 1, abort_flag, a.status, 82, budget))
          return false;
        fence_async_smem();  // the loaders' copies, before the matrix unit reads them
        tc_fence_after();
        const uint32_t v = smem_u32(S.ring[r]), p = smem_u32(S.p[pb]);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          tc_mma_bf16(tmem_base + 2 * N, mnmajor_desc<128>(v + k * 2048, kTile * 128),
                      mnmajor_desc<C::kPRow>(p + k * 16 * C::kPRow, kTile * 128), kIdescO, !(first && k == 0));
        tc_commit(&S.empty[r]);
        tc_commit(&S.p_empty[pb]);
        if (last) {
          tc_commit(&S.o_full);
          ++seg_done;
        }
        return true;
      };
      while (ok && walk.next(t, s)) {
        if (!s.valid) continue;
        const int qb = qn % C::kQBufs;
        if (!(ok = mbar_wait(&S.q_full[qb], (qn / C::kQBufs) & 1, abort_flag, a.status, 83, budget))) break;
        const uint32_t q = smem_u32(S.q[qb]);
        for (int j = 0; j < s.tiles; ++j, ++n) {
          const int f = 2 * n, r = f % C::kSlots, sb = n & 1;
          if (!(ok = mbar_wait(&S.full[r], (f / C::kSlots) & 1, abort_flag, a.status, 84, budget))) break;
          if (!(ok = mbar_wait(&S.s_empty[sb], ((n >> 1) & 1) ^ 1, abort_flag, a.status, 85, budget))) break;
          fence_async_smem();
          tc_fence_after();
          const uint32_t k = smem_u32(S.ring[r]);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_bf16(tmem_base + sb * N, sw128_kmajor_desc(k + c * kTile * 128 + kk * 32),
                          sw128_kmajor_desc(q + c * N * 128 + kk * 32), kIdescS, (c | kk) != 0);
          tc_commit(&S.empty[r]);
          tc_commit(&S.s_full[sb]);
          if (j == s.tiles - 1) tc_commit(&S.q_empty[qb]);
          if (pending && !(ok = values(n - 1, pend_first, pend_last))) break;
          pending = true;
          pend_first = j == 0;
          pend_last = j == s.tiles - 1;
        }
        ++qn;
      }
      if (ok && pending) values(n - 1, pend_first, pend_last);
      // never leave with an MMA in flight
      tc_commit(&S.drain);
      mbar_wait_drain(&S.drain, 0, a.status, 86);
    }
  } else if (warp < kSoftWarps) {
    // ---------------- softmax ----------------
    constexpr int kC = N / 2, kStep = kC > 32 ? 32 : kC;  // columns of a warp, of one TMEM load
    const int wg = warp >> 2, wq = warp & 3, tid = threadIdx.x & 127, bar = 1 + wg;
    const int key = wq * 32 + lane, c0 = wg * kC;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const float c2 = a.scale * 1.44269504f;  // scores in powers of two
    // this thread's P row: 64 columns a chunk, 16-byte units swizzled over the row's width
    const uint32_t p_off = (uint32_t)((N == 128 ? wg * kTile * 128 : 0) + key * C::kPRow);
    const uint32_t p_unit = N == 128 ? 0 : wg * (kC / 8);
    const uint32_t p_sw = C::kPRow == 128 ? key & 7 : (C::kPRow == 64 ? (key >> 1) & 3 : (key >> 2) & 1);
    int n = 0, seg = 0, first_seg = 1;
    bool ok = true;
    while (walk.next(t, s)) {
      if (!s.valid) {
        first_seg = 0;
        continue;
      }
      if (tid < kC) {
        const int r = c0 + tid, rr = s.row0 + r, j = rr / g;
        S.mref[r] = kNoMax;
        S.lim[r] = kSel ? 0 : s.lim0 + j;
        S.orow[r] = r < s.rows ? (s.q0 + j) * a.Hq + s.hk * g + (rr - j * g) : -1;
      }
      named_bar(bar, 128);
      float l[kC];
#pragma unroll
      for (int i = 0; i < kC; ++i) l[i] = 0.f;
      // what this thread's token of the next tile needs beside its scores
      bool seen_next = true;
      float ks_next = 1.f, vs_next = 1.f;
      auto token = [&](int tile) {
        const int e = tile * kTile + key;
        int pos = e < s.end ? e : -1;
        if constexpr (kSel) {
          if (pos >= 0) {
            pos = a.idx[(int64_t)s.q0 * a.k + e];
            if (pos > s.lim0) pos = -1;
          }
        }
        seen_next = pos >= 0;
        if constexpr (kFp8) {
          ks_next = 0.f;
          vs_next = 0.f;
          if (pos >= 0) {
            int off;
            const int id = page_of(a, s.b, pos, off);
            if (id >= 0) {
              const int64_t at = ((int64_t)id * a.page + off) * a.Hkv + s.hk;
              ks_next = a.K_scale[at];
              vs_next = a.V_scale[at];
            }
          }
        }
      };
      if constexpr (kSel || kFp8) token(s.tile0);
      for (int j = 0; j < s.tiles; ++j, ++n) {
        const int sb = n & 1, tile = s.tile0 + j;
        const float cs = kFp8 ? c2 * ks_next : c2, vs = vs_next;
        const bool seen = seen_next;
        if constexpr (kSel || kFp8)
          if (j + 1 < s.tiles) token(tile + 1);
        const int pos = tile * kTile + key;
        // some row does not see some token of this tile
        const bool masked = kSel || (tile + 1) * kTile > s.lim0 + 1;
        ok = ok && mbar_wait(&S.s_full[sb], (n >> 1) & 1, abort_flag, a.status, 90, budget);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const uint32_t col = tmem_base + lanes + (uint32_t)(sb * N + c0);
        float x[kStep];
        auto scores = [&](int i0) {  // x = log2 weights against the reference
          tmem_ld<kStep>(col + i0, x);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kStep; ++i) {
            float v = x[i];
            if (masked) {
              const bool vis = kSel ? seen : pos <= S.lim[c0 + i0 + i];
              v = vis ? v * cs : -INFINITY;
              x[i] = v - S.mref[c0 + i0 + i];
            } else {
              x[i] = fmaf(v, cs, -S.mref[c0 + i0 + i]);
            }
          }
        };
        float top = -INFINITY;
#pragma unroll
        for (int i0 = 0; i0 < kC; i0 += kStep) {
          scores(i0);
#pragma unroll
          for (int i = 0; i < kStep; ++i) top = fmaxf(top, x[i]);
        }
        if (bar_or(bar, 128, top > kSlack || !ok)) {
          if (bar_or(bar, 128, !ok)) {
            ok = false;
            break;
          }
          // new references: the rows' maxima so far
#pragma unroll
          for (int i0 = 0; i0 < kC; i0 += kStep) {
            if (kC > kStep) scores(i0);
            // back to plain scores: the reference may be far off (none yet)
            tmem_ld<kStep>(col + i0, x);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
              const bool vis = !masked || (kSel ? seen : pos <= S.lim[c0 + i0 + i]);
              x[i] = vis ? x[i] * cs : -INFINITY;
            }
            const float m = warp_columns<kStep, true>(x);
            if (lane < kStep) S.red[wg][wq][i0 + lane] = m;
          }
          named_bar(bar, 128);
          if (tid < kC) {
            const float old = S.mref[c0 + tid];
            float m = old;
#pragma unroll
            for (int w = 0; w < 4; ++w) m = fmaxf(m, S.red[wg][w][tid]);
            S.mref[c0 + tid] = m;
            S.fac[c0 + tid] = ex2(old - m);
          }
          named_bar(bar, 128);
#pragma unroll
          for (int i = 0; i < kC; ++i) l[i] *= S.fac[c0 + i];
          if (j > 0) {  // O holds the tiles before: wait for the last of them, then scale
            ok = ok && mbar_wait(&S.p_empty[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, a.status, 91, budget);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const uint32_t o = tmem_base + lanes + (uint32_t)(2 * N + c0);
#pragma unroll
            for (int i0 = 0; i0 < kC; i0 += 8) {
              float v[8];
              tmem_ld<8>(o + i0, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] *= S.fac[c0 + i0 + i];
              tmem_st8(o + i0, v);
            }
            tmem_st_wait();
          }
          if constexpr (kC == kStep) scores(0);
        }
        // P(n - 2) has been read
        if (n >= 2) ok = ok && mbar_wait(&S.p_empty[sb], ((n >> 1) & 1) ^ 1, abort_flag, a.status, 92, budget);
        ok = __all_sync(0xffffffffu, ok);
        uint8_t* prow = S.p[sb] + p_off;
#pragma unroll
        for (int i0 = 0; i0 < kC; i0 += kStep) {
          if (kC > kStep) scores(i0);
#pragma unroll
          for (int i = 0; i < kStep; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float w0 = ex2(x[i + e]), w1 = ex2(x[i + e + 1]);
              l[i0 + i + e] += w0;
              l[i0 + i + e + 1] += w1;
              const __nv_bfloat162 b = kFp8 ? __floats2bfloat162_rn(w0 * vs, w1 * vs) : __floats2bfloat162_rn(w0, w1);
              w[e >> 1] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(prow + (((p_unit + ((i0 + i) >> 3)) ^ p_sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.s_empty[sb]);
          mbar_arrive(&S.p_full[sb]);
        }
      }
      // ---- the segment's sums ----
      if (bar_or(bar, 128, !ok)) break;
#pragma unroll
      for (int i0 = 0; i0 < kC; i0 += kStep) {
        float v[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i) v[i] = l[i0 + i];
        const float sum = warp_columns<kStep, false>(v);
        if (lane < kStep) S.red[wg][wq][i0 + lane] = sum;
      }
      named_bar(bar, 128);
      const bool whole = s.tiles == s.unit_tiles;
      const int64_t part = 2 * (int64_t)blockIdx.x + (first_seg ? 0 : 1);
      if (tid < kC) {
        const int r = c0 + tid;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += S.red[wg][w][tid];
        if (whole) {
          if (a.lse != nullptr && S.orow[r] >= 0)
            a.lse[S.orow[r]] = sum > 0.f ? (S.mref[r] + log2f(sum)) * 0.693147181f : -INFINITY;
          S.lsum[r] = sum > 0.f ? 1.f / sum : 0.f;
        } else {
          a.part_ml[(part * N + r) * 2] = S.mref[r];
          a.part_ml[(part * N + r) * 2 + 1] = sum;
        }
      }
      named_bar(bar, 128);
      ok = ok && mbar_wait(&S.o_full, seg & 1, abort_flag, a.status, 93, budget);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      // 128 rows of O^T fill the 128 lanes; 64 fill the first 16 lanes of each warp
      const int dv = D == 128 ? wq * 32 + lane : wq * 16 + lane;
      const bool mine = D == 128 || lane < 16;
      const uint32_t o = tmem_base + lanes + (uint32_t)(2 * N + c0);
#pragma unroll
      for (int i0 = 0; i0 < kC; i0 += 8) {
        float v[8];
        tmem_ld<8>(o + i0, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = c0 + i0 + i;
          if (!mine || !ok) continue;
          if (!whole)
            a.part_o[(part * N + r) * D + dv] = v[i];
          else if (S.orow[r] >= 0 && dv < a.d)
            static_cast<__nv_bfloat16*>(a.out)[(int64_t)S.orow[r] * a.d + dv] = __float2bfloat16_rn(v[i] * S.lsum[r]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.o_free);
      named_bar(bar, 128);  // the rows' state is free for the next segment
      ++seg;
      first_seg = 0;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem_base, C::kCols);
}

// ----------------------------------------------------------------------------
// Joins the parts of the units that cuts between CTAs divide.  Block (c, y)
// looks at the cut before CTA c and, if it is the first cut of its unit,
// joins rows 4 y .. 4 y + 3: the warps share the parts, then meet in shared
// memory in a fixed order.
// ----------------------------------------------------------------------------
template <int N, int D>
__global__ void __launch_bounds__(256) attend_tc_join_kernel(const AttendArgs a, const JoinDesc* desc) {
  constexpr int kRows = 4, kPer = D / 32;
  __shared__ float so[8][kRows][D];
  __shared__ float sm[8][kRows], sl[8][kRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const JoinDesc d = desc[c];
  const int r0 = blockIdx.y * kRows;
  if (d.rows <= r0 || d.first >= (int64_t)c * d.run) return;  // no work there, or the cut falls between units
  const int64_t c0 = d.first / d.run, c1 = (d.last - 1) / d.run;
  if (c0 + 1 != c) return;  // an earlier cut of the same unit
  const int parts = (int)(c1 - c0) + 1;
  // parts: the end of run c0 (its only segment, or its last), then the beginnings of the others
  const int64_t slot0 = d.first == c0 * d.run ? 2 * c0 : 2 * c0 + 1;
  float m[kRows], l[kRows], o[kRows][kPer];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    m[r] = kNoMax;
    l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[r][i] = 0.f;
  }
  for (int p = warp; p < parts; p += 8) {
    const int64_t slot = p == 0 ? slot0 : 2 * (c0 + p);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t row = slot * N + r0 + r;
      const float pm = a.part_ml[row * 2], pl = a.part_ml[row * 2 + 1];
      float v[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = a.part_o[row * D + lane + 32 * i];
      const float top = fmaxf(m[r], pm), f = ex2(m[r] - top), pf = ex2(pm - top);
      m[r] = top;
      l[r] = l[r] * f + pl * pf;
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[r][i] = o[r][i] * f + v[i] * pf;
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) so[warp][r][lane + 32 * i] = o[r][i];
    if (lane == 0) {
      sm[warp][r] = m[r];
      sl[warp][r] = l[r];
    }
  }
  __syncthreads();
  const int r = warp;  // one warp a row
  if (r >= kRows || r0 + r >= d.rows) return;
  float top = kNoMax, sum = 0.f;
  for (int w = 0; w < 8; ++w) top = fmaxf(top, sm[w][r]);
  for (int w = 0; w < 8; ++w) sum = fmaf(ex2(sm[w][r] - top), sl[w][r], sum);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int g = a.Hq / a.Hkv, rr = d.row0 + r0 + r, j = rr / g;
  const int64_t orow = (int64_t)(d.q0 + j) * a.Hq + d.hk * g + (rr - j * g);
  for (int e = lane; e < a.d; e += 32) {
    float x = 0.f;
    for (int w = 0; w < 8; ++w) x = fmaf(ex2(sm[w][r] - top), so[w][r][e], x);
    static_cast<__nv_bfloat16*>(a.out)[orow * a.d + e] = __float2bfloat16_rn(x * inv);
  }
  if (lane == 0 && a.lse != nullptr) a.lse[orow] = sum > 0.f ? (top + log2f(sum)) * 0.693147181f : -INFINITY;
}

// ----------------------------------------------------------------------------
// host
// ----------------------------------------------------------------------------
static size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// Rows of a tile: the smallest size that holds the rows sharing a cache
// (heads of a group x new queries), else blocks of 128.
int attend_tc_rows(int rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : 128)); }

size_t attend_tc_bytes(int sms, int rows, int d) {
  const int N = attend_tc_rows(rows);
  d = d > 64 ? 128 : 64;
  return sizeof(WsHeader) + round256((size_t)sms * sizeof(JoinDesc)) + round256((size_t)sms * 2 * N * 8) +
         round256((size_t)sms * 2 * N * d * 4);
}

bool attend_tc_ok(const AttendArgs& a, int q_dtype, int kv_dtype) {
  if (q_dtype != DSA_DTYPE_BF16 || a.d > 128) return false;
  // 16-byte copies; cache rows are 32-bit numbers
  const int elt = kv_dtype == DSA_DTYPE_FP8_E4M3 ? 1 : 2;
  if (a.d * elt % 16 != 0 || a.page_stride % a.d != 0 ||
      ((reinterpret_cast<uintptr_t>(a.K) | reinterpret_cast<uintptr_t>(a.V)) & 15u))
    return false;
  const int64_t per_page = a.page_stride / a.d;
  return per_page < ((int64_t)1 << 31) && per_page * a.n_pages < ((int64_t)1 << 31) - 1;
}

template <int N, int D, bool kFp8, bool kSel>
static int launch_attend_tc(const TcAttend& t, int grid, cudaStream_t st) {
  using C = Cfg<N, D, kFp8>;
  constexpr size_t kSmem = sizeof(AttendSmem<N, D, kFp8>) + 1024;
  static_assert(kSmem <= 232448, "fits the 227 KB opt-in shared memory of one CTA");
  // the shared-memory opt-in is a per-device function attribute: set it once
  // on each device the kernel runs on
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSA_ERR_CUDA;
  const uint64_t bit = uint64_t(1) << dev;
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(attend_tc_kernel<N, D, kFp8, kSel>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kSmem) != cudaSuccess)
      return DSA_ERR_CUDA;
    configured.fetch_or(bit, std::memory_order_release);
  }
  attend_tc_kernel<N, D, kFp8, kSel><<<grid, C::kWarps * 32, kSmem, st>>>(t);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (grid == 1 || (kSel && t.run % t.unit_tiles == 0)) return DSA_OK;  // no unit is divided
  // The join may take its place on the SMs while the last tiles run; it waits
  // for the whole grid before it reads a part.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid - 1, N / 4);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_tc_join_kernel<N, D>, t.a, (const JoinDesc*)t.desc) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

template <int N, int D>
static int launch_attend_tc(const TcAttend& t, bool fp8, int grid, cudaStream_t st) {
  const bool sel = t.a.idx != nullptr;
  if (fp8) return sel ? launch_attend_tc<N, D, true, true>(t, grid, st) : launch_attend_tc<N, D, true, false>(t, grid, st);
  return sel ? launch_attend_tc<N, D, false, true>(t, grid, st) : launch_attend_tc<N, D, false, false>(t, grid, st);
}

template <int N>
static int launch_attend_tc(const TcAttend& t, bool fp8, int grid, cudaStream_t st) {
  return t.a.d > 64 ? launch_attend_tc<N, 128>(t, fp8, grid, st) : launch_attend_tc<N, 64>(t, fp8, grid, st);
}

// rows: the most rows that share a cache; the workspace holds attend_tc_bytes.
int run_attend_tc(const AttendArgs& args, int kv_dtype, int rows, int sms, uint8_t* ws, cudaStream_t st) {
  const NvtxRange nvtx(args.idx != nullptr ? "dsa.attend_selected" : "dsa.attend_paged");
  const int N = attend_tc_rows(rows);
  const bool fp8 = kv_dtype == DSA_DTYPE_FP8_E4M3;
  TcAttend t{};
  t.a = args;
  size_t off = sizeof(WsHeader);
  t.desc = reinterpret_cast<JoinDesc*>(ws + off);
  off += round256((size_t)sms * sizeof(JoinDesc));
  t.a.part_ml = reinterpret_cast<float*>(ws + off);
  off += round256((size_t)sms * 2 * N * 8);
  t.a.part_o = reinterpret_cast<float*>(ws + off);
  t.row_stride_page = (int)(args.page_stride / args.d);
  int grid = sms;
  t.min_run = 2;
  if (args.idx != nullptr) {
    t.unit_tiles = (args.k + kTile - 1) / kTile;
    const int64_t total = (int64_t)args.total_q * args.Hkv * t.unit_tiles;
    t.run = (total + sms - 1) / sms;
    // many units a CTA: whole ones, the few tiles of imbalance cost less than joins
    if (t.run >= 8 * t.unit_tiles) t.run = (t.run + t.unit_tiles - 1) / t.unit_tiles * t.unit_tiles;
    grid = (int)((total + t.run - 1) / t.run);
  }
  if (N == 16) return launch_attend_tc<16>(t, fp8, grid, st);
  if (N == 32) return launch_attend_tc<32>(t, fp8, grid, st);
  if (N == 64) return launch_attend_tc<64>(t, fp8, grid, st);
  return launch_attend_tc<128>(t, fp8, grid, st);
}

}  // namespace dsa
