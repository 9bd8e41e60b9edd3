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
// and N/2 of its rows.  Beyond 64 rows (N = 128) the query rows fill the lanes
// themselves, S = Q K^T and O += P V: a thread owns half a row, whose statistics
// stay in its registers, and the weights are the A operand in tensor memory
// (128 rows over 32 caches of 131072 tokens: 372 us, ten passes in a graph, 901
// with tokens on the lanes).  Decoding reads each K and V row once for N rows,
// 2 N flops a byte.  Few rows are bound by memory (64 ragged caches: 72 % of the
// copy bandwidth); 64 and 128 by the softmax warps as soon as the power cap
// lowers the clock, and e4m3 caches by their conversion.
//
// One persistent CTA per SM:
//   * three lookup warps turn positions into cache rows (page table, or list
//     entry and page table), post them with the tokens' masks and scales a
//     few tiles ahead, and fetch the queries;
//   * sixteen copy warps, eight for K and eight for V, fetch the rows by
//     16-byte asynchronous copies into a ring that K and V tiles share,
//     whatever the page size; a token that no row sees, and the columns
//     behind d, are filled with zeros, so no stale value meets a zero weight.
//     One warp issues such a copy of scattered rows every 60 cycles or so:
//     sixteen reach 17 TB/s from L2 and 7 TB/s from memory in a kernel of
//     such copies alone, eight 14.5 and 5.7, four 8.7 and 3.3.  e4m3 rows come through registers, a tile ahead,
//     and are written as bf16 (exact);
//   * the MMA warp issues S(t+1) before O(t), so that the tensor pipe has
//     work while the softmax of a tile runs;
//   * eight softmax warps: four cover the 128 lanes for the first half of the
//     columns, four for the rest.
//
// The reference m is not the running maximum but one that no score has
// passed by more than 2^16: as long as that holds no sum needs rescaling, and
// whether it holds is one vote a tile, taken behind the exponentials.  When
// it fails (always in the first tile) the rows' true maxima become the new
// reference, and O and the row sums are scaled once.  Weights lie in
// [0, 2^16], where floating point is as exact as in [0, 1]; sums of weights and
// values stay finite for values below 2^112 over the number of tokens.
//
// The matrix unit takes weights in bf16.  One rounding (2^-8 of a weight at
// most) would leave outputs 1.4 times as far off as their own rounding to bf16
// does.  Up to 32 rows each weight goes in as two, its bf16 and the bf16 of what
// that left (2^-16 together): the rests are N more columns of the same product,
// which waits for A's bytes from shared memory and takes no longer for it up
// to 64 columns.  With more rows that costs a quarter of the time (32 caches of
// 131072 tokens, 128 rows each: 473 us for 366), and the weights are rounded
// once.  A row of one token stays exact all the same: with rows on the lanes
// its reference is its score; with 64 rows the output is divided by the sum of
// the rounded weights, and references are whole numbers there, so that weights
// rounded against an old one stay those that the product took.  (e4m3 weights carry V's scales and are always
// split.)  The log-sum-exp comes from the fp32 sum of the weights themselves.
//
// With tokens on the lanes a thread sees many rows, and their references come
// from shared memory, where the copies queue; so the rows share one, in a
// register, while no row's maximum is below it by more than 2^64 (fp32 and
// bf16 hold 2^-126), and have their own beyond that.
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
constexpr int kSoftWarps = 8, kLookWarps = 3, kCopyWarps = 16;
constexpr int kWarps = kSoftWarps + 1 + kLookWarps + kCopyWarps;
constexpr int kLaunchRegs = 72;      // registers a thread at launch: 65536 over 28 warps
constexpr float kNoMax = -1.7e38f;   // reference of a row that has seen no token
constexpr float kSlack = 16.f;       // log2 of the largest weight
constexpr float kSpread = 64.f;      // how far (log2) a shared reference may lie above a row's own maximum

struct TcAttend {
  AttendArgs a;
  int row_stride_page;  // cache rows from one page to the next (page_stride / d)
  int unit_tiles;       // chosen positions: tiles of one (row, head)
  int64_t run;          // chosen positions: tiles of one CTA
  int min_run;          // all tokens: least tiles of one CTA
  struct JoinDesc* desc;
  // failure-path controls (dsa_debug_set_wait; zero in normal calls): the time
  // budget of the waits (0 = the default), and a first tile that CTA 0 never posts
  uint64_t wait_ns;
  int hold_first_tile;
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

// What the debug build checks ahead of an access (in_bounds): a cache row by its number, an output row, a part.
__device__ __forceinline__ bool row_ok(const TcAttend& t, int row) { return cache_ok(t.a, (int64_t)row * t.a.d); }
__device__ __forceinline__ bool out_ok(const AttendArgs& a, int64_t orow) {
  return orow >= 0 && orow < (int64_t)a.total_q * a.Hq;
}
__device__ __forceinline__ bool part_ok(int64_t part, unsigned ctas) { return part >= 0 && part < 2 * (int64_t)ctas; }

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

// Steps through the segments of a CTA's run; every role keeps its own, and
// whole warps step.
template <int N, bool kSel>
struct Walk {
  int64_t left;  // tiles still to hand out
  int b, hk, rb, off;
  int q0, m, len, q1;
  int row;

  __device__ __forceinline__ void start(const TcAttend& t, int64_t n, int b_, int64_t off_) {
    left = n;
    if constexpr (kSel) {
      const int64_t u = div64(off_, t.unit_tiles);
      row = (int)div64(u, t.a.Hkv);
      hk = (int)(u - (int64_t)row * t.a.Hkv);
      off = (int)(off_ - u * t.unit_tiles);
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
        hk = (int)div64(off_, per_head);
        int64_t o = off_ - hk * per_head;
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

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Two fp32 -> two bf16, and the bf16 of what those left of them: the sum of
// both is within 2^-17 of the value.
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x0, x1);
  const float2 h = unpack_bf16(hi), r = add2(make_float2(x0, x1), make_float2(-h.x, -h.y));
  lo = pack_bf16(r.x, r.y);
}

// Four e4m3 bytes -> four bf16, exactly, in the order 0, 2, 1, 3: sign,
// exponent and fraction move to their bf16 places, which reads as the value
// times 2^-120 (the biases differ by 120), subnormals included.
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t w) {
  const __nv_bfloat162 up = __halves2bfloat162(__ushort_as_bfloat16(0x7b80), __ushort_as_bfloat16(0x7b80));  // 2^120
  const uint32_t even = ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u);
  const uint32_t odd = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
  const __nv_bfloat162 e = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&even), up);
  const __nv_bfloat162 o = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&odd), up);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&e), *reinterpret_cast<const uint32_t*>(&o));
}

// Sets the registers of a thread of this warpgroup; the launch's total must
// hold the sum of all shares.
template <int kRegs, bool kMore>
__device__ __forceinline__ void set_regs() {
  if constexpr (kMore)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// True in one lane of a converged warp, always the same one; the compiler
// knows that the branch is uniform, which tcgen05 operands profit from.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// A from tensor memory (lane: row, column: two bf16 along K), B from shared memory.
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
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
constexpr int kEnd = -2;  // in place of the first row: no more tiles
constexpr int kTok = 8;  // tiles whose token masks and scales are kept: more than the ring can run ahead

template <int N, int D, bool kFp8>
struct Cfg {
  static constexpr bool kRows = N == 128;            // query rows, not tokens, on the 128 lanes
  static constexpr int kChunks = D / 64;
  static constexpr int kSlotBytes = kTile * D * 2;   // one K or V tile, bf16
  static constexpr int kQBytes = N * D * 2;
  static constexpr int kQBufs = 2;
  static constexpr bool kSplit = kFp8 || N <= 32;    // weights go in as two bf16
  static constexpr int kPCols = kSplit ? 2 * N : N;
  static constexpr int kPBufs = kSplit && N >= 64 ? 1 : 2;
  static constexpr int kPBytes = kRows ? 0 : kPCols * kTile * 2;
  static constexpr int kPRow = kPCols >= 64 ? 128 : kPCols * 2;  // bytes of a P row (of its first 64 columns)
  static constexpr int kOther = kQBufs * kQBytes + kPBufs * kPBytes + (kFp8 ? kTok * kTile * 8 : 0);
  static constexpr int kBudget = 232448 - 1024 - 10240;
  static constexpr int kFit = (kBudget - kOther) / kSlotBytes;
  static constexpr int kSlots = kFit > 8 ? 8 : kFit;
  // Registers a thread: launched with 72 (28 warps), of which the copy warps
  // give some up, so that the softmax warps hold a row's or token's scores.
  static constexpr int kSoftRegs = kFp8 ? 128 : 144, kMidRegs = 56, kCopyRegs = kFp8 ? 48 : 40;
  static_assert(kSoftWarps % 4 == 0 && (1 + kLookWarps) % 4 == 0 && kCopyWarps % 4 == 0, "roles that share a number of registers fill warpgroups");
  static_assert(256 * kSoftRegs + 128 * kMidRegs + 512 * kCopyRegs <= kWarps * 32 * kLaunchRegs, "the registers of the launch");
  // Tensor memory: two score tiles; with rows on the lanes the weights, two
  // tiles or one and its rests (64 columns each); two output tiles, one where
  // no more fit (tokens on the lanes: the columns of the rests are added when
  // it is stored).
  static constexpr int kSCols = N, kPCol = 2 * N, kOCol = kRows ? 2 * N + 128 : 2 * N, kOCols = kRows ? D : kPCols;
  static constexpr int kOBufs = kRows && D == 128 ? 1 : 2;
  static constexpr int kCols = N >= 64 ? 512 : 8 * N;
  static_assert(kSlots >= 2, "the ring holds a K and a V tile");
};

template <int N, int D, bool kFp8>
struct AttendSmem {
  using C = Cfg<N, D, kFp8>;
  uint8_t ring[C::kSlots][C::kSlotBytes];
  uint8_t q[C::kQBufs][C::kQBytes];
  uint8_t p[C::kPBufs][C::kPBytes ? C::kPBytes : 16];
  float ksc[kTok][kFp8 ? kTile : 4], vsc[kTok][kFp8 ? kTile : 4];
  alignas(16) int rows[kTok][kTile];
  uint32_t seen[kTok][4];
  uint64_t full[C::kSlots], empty[C::kSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], p_empty[2];
  uint64_t o_full[2], o_free[2], tok_full[kTok], tok_empty[kTok], drain;
  float red[2][4][N / 2 > 32 ? 32 : N / 2];
  float sum[2][C::kRows ? N : 1], red2[2][4][N == 64 && C::kSplit == false ? 32 : 1];
  alignas(16) float nref[N];
  float rowmax[N], cref[2];
  int common[2];
  float fac[N], lsum[2][N];
  int lim[N], orow[2][N];
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
__global__ void __launch_bounds__(kWarps * 32, 1)
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
      mbar_init(&S.full[i], kCopyWarps / 2 * (kFp8 ? 1 : 32));
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], kLookWarps * (kFp8 ? 1 : 32));
      mbar_init(&S.q_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], kSoftWarps);
      mbar_init(&S.p_empty[i], 1);
      mbar_init(&S.o_full[i], 1);
      mbar_init(&S.o_free[i], kSoftWarps);
    }
    for (int i = 0; i < kTok; ++i) {
      mbar_init(&S.tok_full[i], 1);
      mbar_init(&S.tok_empty[i], kCopyWarps + (kSel || kFp8 ? kSoftWarps : 0));
    }
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
    const int threads = kWarps * 32, share = (a.B + threads - 1) / threads;
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
    int64_t warps = lane < kWarps ? S.sums[lane] : 0;  // every warp adds up the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, warps, o);
      if (lane >= o) warps += u;
    }
    const int64_t total = __shfl_sync(0xffffffffu, warps, 31);
    const int64_t earlier = __shfl_sync(0xffffffffu, warps, warp > 0 ? warp - 1 : 0);
    const int64_t before = inc - mine + (warp > 0 ? earlier : 0);
    run = div64(total + gridDim.x - 1, gridDim.x);
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
  if (warp >= kSoftWarps + 1 + kLookWarps) {
    // ---------------- copy warps: cache rows -> ring ----------------
    set_regs<C::kCopyRegs, false>();
    const int w = warp - (kSoftWarps + 1 + kLookWarps), kv = w >> 3, row0 = (w & 7) * 16;
    constexpr int kElt = kFp8 ? 1 : 2, kUnits = D * kElt / 16;   // 16-byte units of a cache row
    constexpr int kRowsAt = 32 / kUnits, kTimes = 16 / kRowsAt;  // rows a warp copies at a time, of its 16
    const int unit = lane % kUnits, sub = lane / kUnits;
    const bool unit_ok = unit * 16 < a.d * kElt;
    const uint32_t row_bytes = (uint32_t)(a.d * kElt);
    const uint8_t* pages = static_cast<const uint8_t*>(kv ? a.V : a.K) + unit * 16;
    bool ok = true;
    auto wait_rows = [&](int n) {  // the rows of tile n are there
      ok = ok && mbar_wait<true>(&S.tok_full[n % kTok], (n / kTok) & 1, abort_flag, a.status, 72, budget);
      ok = __all_sync(0xffffffffu, ok);
    };
    auto slot_free = [&](int n) {  // the ring slot of tile n's K or V, once it is free
      const int fill = 2 * n + kv, r = fill % C::kSlots;
      ok = ok && mbar_wait<true>(&S.empty[r], ((fill / C::kSlots) & 1) ^ 1, abort_flag, a.status, 71, budget);
      ok = __all_sync(0xffffffffu, ok);
      return r;
    };
    if constexpr (!kFp8) {
      for (int n = 0;; ++n) {
        wait_rows(n);
        if (!ok || S.rows[n % kTok][0] == kEnd) break;
        const int r = slot_free(n);
        if (!ok) break;
        int rows[kTimes];  // a group of lanes copies consecutive rows: their numbers come in wide loads
#pragma unroll
        for (int i = 0; i < kTimes; i += 4)
          *reinterpret_cast<int4*>(rows + i) = *reinterpret_cast<const int4*>(&S.rows[n % kTok][row0 + sub * kTimes + i]);
        const uint32_t dst = smem_u32(S.ring[r]) + (unit >> 3) * kTile * 128 + (row0 + sub * kTimes) * 128;
#pragma unroll
        for (int i = 0; i < kTimes; ++i) {
          const int row = rows[i];
          const bool in = row >= 0 && unit_ok && in_bounds(row_ok(t, row), a.status, 22);
          copy16(dst + i * 128 + (((unit & 7) ^ ((sub * kTimes + i) & 7)) << 4),
                 in ? pages + (uint64_t)(uint32_t)row * row_bytes : static_cast<const uint8_t*>(a.K), in);
        }
        copies_arrive(&S.full[r]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.tok_empty[n % kTok]);
      }
      // never leave with a copy in flight
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      uint4 raw[kTimes];  // a tile's bytes
      auto load_unit = [&](int i, int row) {
        uint4& v = raw[i];
        v = make_uint4(0, 0, 0, 0);
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
            : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
            : "l"(pages + (uint64_t)(uint32_t)row * row_bytes),
              "r"((uint32_t)(row >= 0 && unit_ok && in_bounds(row_ok(t, row), a.status, 22))));
      };
      // the second 64-element chunk's lanes write their odd unit first, so that no two lanes of a row share banks
      const int flip = (unit >> 2) & 1;
      wait_rows(0);
      bool more = ok && S.rows[0][0] != kEnd;
#pragma unroll
      for (int i = 0; i < kTimes; ++i) load_unit(i, more ? S.rows[0][row0 + sub + i * kRowsAt] : -1);
      for (int n = 0; ok && more; ++n) {
        wait_rows(n + 1);
        const int r = slot_free(n);
        if (!ok) break;
        const int* rows = S.rows[(n + 1) % kTok] + row0 + sub;
        more = S.rows[(n + 1) % kTok][0] != kEnd;
        uint8_t* dst0 = S.ring[r] + (unit >> 2) * kTile * 128;
#pragma unroll
        for (int i = 0; i < kTimes; ++i) {
          const uint2 w0 = e4m3x4_to_bf16(raw[i].x), w1 = e4m3x4_to_bf16(raw[i].y), w2 = e4m3x4_to_bf16(raw[i].z),
                      w3 = e4m3x4_to_bf16(raw[i].w);
          load_unit(i, more ? rows[i * kRowsAt] : -1);  // behind the last tile the entry holds no rows
          const uint4 lo = make_uint4(w0.x, w0.y, w1.x, w1.y), hi = make_uint4(w2.x, w2.y, w3.x, w3.y);
          const int at = row0 + i * kRowsAt + sub, u0 = (unit & 3) * 2, sw = at & 7;
          uint8_t* dst = dst0 + at * 128;
          *reinterpret_cast<uint4*>(dst + (((u0 + flip) ^ sw) << 4)) = flip ? hi : lo;
          *reinterpret_cast<uint4*>(dst + (((u0 + (flip ^ 1)) ^ sw) << 4)) = flip ? lo : hi;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.full[r]);
          mbar_arrive(&S.tok_empty[n % kTok]);
        }
      }
    }
  } else if (warp >= kMma) {
    set_regs<C::kMidRegs, false>();  // the warps of a warpgroup change theirs by one instruction, ahead of their roles
    if (warp > kMma) {
      // ---------------- lookup warps: positions -> cache rows, masks, scales; queries ----------------
      const int lw = warp - kMma - 1;
      Walk<N, kSel> walk;
      walk.start(t, n_tiles, S.begin_b, kSel ? begin : S.begin_off);
      Seg s;
      int n = 0, qn = 0;  // tiles, segments
      bool ok = true;
      auto tile_free = [&]() {
        ok = ok && mbar_wait<true>(&S.tok_empty[n % kTok], ((n / kTok) & 1) ^ 1, abort_flag, a.status, 73, budget);
        ok = __all_sync(0xffffffffu, ok);
      };
      while (ok && walk.next(t, s)) {
        if (!s.valid) continue;
        // the segment's queries, a third each; the first segment's by two warps, as the third looks up its first tile
        const bool split3 = qn > 0;
        const int qb = qn % C::kQBufs;
        if (qn >= C::kQBufs)
          ok = mbar_wait<true>(&S.q_empty[qb], (qn / C::kQBufs - 1) & 1, abort_flag, a.status, 70, budget);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* Q = static_cast<const uint8_t*>(a.Q);
        constexpr int kQUnits = D / 8;
#pragma unroll 2
        for (int e = (split3 ? lw : (lw > 0 ? lw - 1 : N * kQUnits)) * 32 + lane; e < N * kQUnits;
             e += (split3 ? kLookWarps : kLookWarps - 1) * 32) {
          const int r = e / kQUnits, u = e % kQUnits;
          // rows behind the last repeat the first, so that their scores move no reference
          const int rr = s.row0 + (r < s.rows ? r : 0), j = rr / g;
          const bool in = u * 8 < a.d && in_bounds(out_ok(a, (int64_t)(s.q0 + j) * a.Hq + s.hk * g + (rr - j * g)), a.status, 23);
          const int64_t at = in ? ((int64_t)(s.q0 + j) * a.Hq + s.hk * g + (rr - j * g)) * a.d + u * 8 : 0;
          uint8_t* dst = S.q[qb] + (u >> 3) * N * 128 + r * 128 + (((u & 7) ^ (r & 7)) << 4);
          if constexpr (kFp8) {  // in the order of the converted keys: elements 0, 2, 1, 3 of every four
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) v = *reinterpret_cast<const uint4*>(Q + at * 2);
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                           __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
          } else {
            copy16(smem_u32(dst), Q + at * 2, in);
          }
        }
        if constexpr (kFp8) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.q_full[qb]);
        } else {
          copies_arrive(&S.q_full[qb]);
        }
        ++qn;
        for (int j = 0; j < s.tiles; ++j, ++n) {
          if (n % kLookWarps != lw) continue;  // the tiles in turn
          const int tk = n % kTok, e0 = (s.tile0 + j) * kTile + lane;
          int pos[4], id[4], off[4], row[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = e0 + i * 32;
            pos[i] = -1;
            if (e < s.end && in_bounds(!kSel || (e < a.k && s.q0 < a.total_q), a.status, 24)) pos[i] = kSel ? a.idx[(int64_t)s.q0 * a.k + e] : e;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kSel && pos[i] > s.lim0) pos[i] = -1;
            id[i] = -1;
            off[i] = 0;
            if (pos[i] >= 0) {
              const int col = (int)((unsigned)pos[i] / (unsigned)a.page);
              off[i] = pos[i] - col * a.page;
              if (in_bounds(table_ok(a, s.b, col), a.status, 25)) id[i] = a.table[(int64_t)s.b * a.max_pages + col];
            }
          }
          float ks[4], vs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            row[i] = -1;
            ks[i] = vs[i] = 0.f;
            if ((unsigned)id[i] < (unsigned)a.n_pages) {
              row[i] = id[i] * t.row_stride_page + off[i] * a.Hkv + s.hk;
              if constexpr (kFp8) {
                const int64_t at = ((int64_t)id[i] * a.page + off[i]) * a.Hkv + s.hk;
                ks[i] = a.K_scale[at];
                vs[i] = a.V_scale[at];
              }
            } else if (pos[i] >= 0) {
              report_error(a.status, DSA_ERR_INVALID_ARG, 41);
            }
          }
          tile_free();
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            S.rows[tk][i * 32 + lane] = row[i];
            if constexpr (kFp8) {
              S.ksc[tk][i * 32 + lane] = ks[i] * (a.scale * 1.44269504f);
              S.vsc[tk][i * 32 + lane] = vs[i];
            }
            if constexpr (kSel) {
              const uint32_t seen = __ballot_sync(0xffffffffu, row[i] >= 0);
              if (lane == 0) S.seen[tk][i] = seen;
            }
          }
          __syncwarp();
          if (lane == 0 && !(t.hold_first_tile && blockIdx.x == 0 && n == 0)) mbar_arrive(&S.tok_full[tk]);
        }
      }
      if (n % kLookWarps == lw) {  // the end, for the copy warps
        tile_free();
        if (ok) {
          if (lane == 0) {
            S.rows[n % kTok][0] = kEnd;
            mbar_arrive(&S.tok_full[n % kTok]);
          }
          __syncwarp();
        }
      }
      if (lw == 0) {  // what the join needs of the unit this run begins in
        JoinDesc d;
        d.rows = 0;
        d.run = run;
        d.first = d.last = begin;
        d.q0 = d.hk = d.row0 = 0;
        if (n_tiles > 0) {
          walk.start(t, n_tiles, S.begin_b, kSel ? begin : S.begin_off);
          walk.next(t, s);
          d.rows = s.valid ? s.rows : 0;
          d.first = begin - s.tile0;
          d.last = d.first + s.unit_tiles;
          d.q0 = s.q0;
          d.hk = s.hk;
          d.row0 = s.row0;
        }
        if (lane == 0) t.desc[blockIdx.x] = d;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      // ---------------- MMA issuer: the warp waits, one lane issues ----------------
      Walk<N, kSel> walk;
      walk.start(t, n_tiles, S.begin_b, kSel ? begin : S.begin_off);
      Seg s;
      constexpr uint32_t kIdescS = idesc_bf16_f32(128, N);
      constexpr uint32_t kIdescO = C::kRows ? idesc_bf16_f32(128, D) | (1u << 16)                // V along N
                                            : idesc_bf16_f32(D, C::kPCols) | (1u << 15) | (1u << 16);  // V^T along M, P along N
      const bool leader = elect_one();
      const uint64_t kdesc = sw128_kmajor_desc(smem_u32(S.ring[0])), vdesc = mnmajor_desc<128>(smem_u32(S.ring[0]), kTile * 128);
      const uint64_t qdesc = sw128_kmajor_desc(smem_u32(S.q[0])), pdesc = mnmajor_desc<C::kPRow>(smem_u32(S.p[0]), kTile * 128);
      int n = 0, seg = 0;  // tiles, segments
      int slot = 0;        // ring slot of the next K tile
      uint32_t ring_phase = 0;
      bool ok = true, pending = false, pend_first = false, pend_last = false;
      int pend_slot = 0, pend_seg = 0;
      uint32_t pend_phase = 0;
      auto values = [&](int i) {  // the output tile += weights x V of tile i
        const int pb = i & 1, par = pend_seg % C::kOBufs;
        ok = mbar_wait(&S.full[pend_slot], pend_phase, abort_flag, a.status, 80, budget) &&
             mbar_wait(&S.p_full[pb], (i >> 1) & 1, abort_flag, a.status, 81, budget) &&
             (!pend_first || pend_seg < C::kOBufs ||
              mbar_wait(&S.o_free[par], (pend_seg / C::kOBufs - 1) & 1, abort_flag, a.status, 82, budget));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        fence_async_smem();  // the loaders' copies, before the matrix unit reads them
        tc_fence_after();
        if (leader) {
          const uint64_t v = vdesc + (uint64_t)(pend_slot * (C::kSlotBytes >> 4));
          const uint64_t p = pdesc + (uint64_t)(i % C::kPBufs * (C::kPBytes >> 4));
          const uint32_t o = tmem_base + C::kOCol + par * C::kOCols, ps = tmem_base + C::kPCol + (C::kPBufs == 2 ? pb * 64 : 0);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k) {
            const uint64_t vk = v + (uint64_t)(k * (2048 >> 4));
            if constexpr (C::kRows) {
              tc_mma_bf16_ts(o, ps + k * 8, vk, kIdescO, !(pend_first && k == 0));
              if constexpr (C::kSplit) tc_mma_bf16_ts(o, ps + 64 + k * 8, vk, kIdescO, 1);
            } else {
              tc_mma_bf16(o, vk, p + (uint64_t)(k * C::kPRow), kIdescO, !(pend_first && k == 0));
            }
          }
          tc_commit(&S.empty[pend_slot]);
          tc_commit(&S.p_empty[pb]);
          if (pend_last) tc_commit(&S.o_full[par]);
        }
        __syncwarp();
      };
      auto step = [&]() {
        if (++slot == C::kSlots) {
          slot = 0;
          ring_phase ^= 1;
        }
      };
      while (ok && walk.next(t, s)) {
        if (!s.valid) continue;
        const int qb = seg % C::kQBufs;
        ok = mbar_wait(&S.q_full[qb], (seg / C::kQBufs) & 1, abort_flag, a.status, 83, budget);
        ok = __all_sync(0xffffffffu, ok);
        for (int j = 0; ok && j < s.tiles; ++j, ++n) {
          ok = mbar_wait(&S.full[slot], ring_phase, abort_flag, a.status, 84, budget);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          // the score tile is free: the weights of tile n - 2 were waited for below
          fence_async_smem();
          tc_fence_after();
          if (leader) {
            const uint64_t k = kdesc + (uint64_t)(slot * (C::kSlotBytes >> 4));
            const uint64_t q = qdesc + (uint64_t)(qb * (C::kQBytes >> 4));
            const uint32_t d = tmem_base + (n & 1) * C::kSCols;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint64_t ko = k + (uint64_t)((c * kTile * 128 + kk * 32) >> 4);
                const uint64_t qo = q + (uint64_t)((c * N * 128 + kk * 32) >> 4);
                tc_mma_bf16(d, C::kRows ? qo : ko, C::kRows ? ko : qo, kIdescS, (c | kk) != 0);
              }
            tc_commit(&S.empty[slot]);
            tc_commit(&S.s_full[n & 1]);
            if (j == s.tiles - 1) tc_commit(&S.q_empty[qb]);
          }
          __syncwarp();
          step();
          if (pending) values(n - 1);
          pending = true;
          pend_first = j == 0;
          pend_last = j == s.tiles - 1;
          pend_seg = seg;
          pend_slot = slot;
          pend_phase = ring_phase;
          step();
        }
        ++seg;
      }
      if (ok && pending) values(n - 1);
      // never leave with an MMA in flight
      if (leader) {
        tc_commit(&S.drain);
        mbar_wait_drain(&S.drain, 0, a.status, 86);
      }
      __syncwarp();
    }
  } else {
    // ---------------- softmax ----------------
    set_regs<C::kSoftRegs, true>();
    Walk<N, kSel> walk;
    walk.start(t, n_tiles, S.begin_b, kSel ? begin : S.begin_off);
    Seg s;
    const int wg = warp >> 2, wq = warp & 3, tid = threadIdx.x & 127;
    // who shares references: the two warps of 32 rows, or the four of half the rows
    constexpr int kGroup = C::kRows ? 64 : 128;
    const int bar = C::kRows ? 1 + wq : 1 + wg;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const float c2 = a.scale * 1.44269504f;  // scores in powers of two
    int n = 0, seg = 0;
    bool ok = true, first_seg = true;
    // the segment before, whose output tile is stored behind the next one's first tile
    bool pend = false, pend_whole = false;
    int pend_par = 0, pend_phase = 0;
    int64_t pend_part = 0;
    // e4m3: the converted V's columns come in the order 0, 2, 1, 3 of every four
    auto element = [](int c) { return kFp8 ? ((c & ~3) | ((c & 1) << 1) | ((c >> 1) & 1)) : c; };

    if constexpr (C::kRows) {
      // A thread owns one query row and half of the tile's tokens.
      const int r = tid, c0 = wg * 64;
      float pend_inv = 0.f;
      int pend_row = -1;
      auto store_output = [&]() {
        if (!pend) return;
        pend = false;
        ok = ok && mbar_wait(&S.o_full[pend_par], pend_phase, abort_flag, a.status, 93, budget);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        constexpr int kHalf = D / 2;
        const uint32_t o = tmem_base + lanes + (uint32_t)(C::kOCol + pend_par * C::kOCols + wg * kHalf);
#pragma unroll
        for (int i0 = 0; i0 < kHalf; i0 += 32) {
          float v[32];
          tmem_ld<32>(o + i0, v);
          tmem_ld_wait();
          if (!ok) continue;
          const int c = wg * kHalf + i0;
          if (!in_bounds(pend_whole ? pend_row < 0 || out_ok(a, pend_row) : part_ok(pend_part, gridDim.x), a.status, 26)) continue;
          if (!pend_whole) {
            float4* dst = reinterpret_cast<float4*>(a.part_o + (pend_part * N + r) * D + c);
#pragma unroll
            for (int i = 0; i < 32; i += 4) dst[i >> 2] = kFp8 ? make_float4(v[i], v[i + 2], v[i + 1], v[i + 3]) : make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          } else if (pend_row >= 0) {
            uint8_t* dst = static_cast<uint8_t*>(a.out) + ((int64_t)pend_row * a.d + c) * 2;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 8; e += 2)
                w[e >> 1] = pack_bf16(v[element(i + e)] * pend_inv, v[element(i + e + 1)] * pend_inv);
              if (c + i < a.d) *reinterpret_cast<uint4*>(dst + i * 2) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.o_free[pend_par]);
      };
      while (walk.next(t, s)) {
        if (!s.valid) {
          first_seg = false;
          continue;
        }
        const int rr = s.row0 + r, jq = rr / g;
        const int orow = r < s.rows ? (s.q0 + jq) * a.Hq + s.hk * g + (rr - jq * g) : -1;
        const int lim = kSel ? 0x7fffffff : s.lim0 + jq;
        float nref = -kNoMax, l = 0.f;
        for (int j = 0; j < s.tiles; ++j, ++n) {
          const int tile = s.tile0 + j, tk = n % kTok;
          if constexpr (kSel || kFp8) ok = ok && mbar_wait(&S.tok_full[tk], (n / kTok) & 1, abort_flag, a.status, 94, budget);
          ok = ok && mbar_wait(&S.s_full[n & 1], (n >> 1) & 1, abort_flag, a.status, 90, budget);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          const uint32_t col = tmem_base + lanes + (uint32_t)((n & 1) * C::kSCols + c0);
          uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
          bool masked;
          if constexpr (kSel) {
            seen[0] = S.seen[tk][wg * 2];
            seen[1] = S.seen[tk][wg * 2 + 1];
            masked = (seen[0] & seen[1]) != 0xffffffffu;
          } else {
            masked = (tile + 1) * kTile > s.lim0 + 1;  // some row does not see some token of this tile
            if (masked) {
              const int left = lim - tile * kTile - c0 + 1;  // tokens of this half that the row sees
              seen[0] = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1);
              seen[1] = left >= 64 ? 0xffffffffu : (left <= 32 ? 0u : (1u << (left - 32)) - 1);
            }
          }
          float x[64];
          auto scores = [&](float ref) {  // log2 weights against the reference -ref
            tmem_ld<32>(col, *reinterpret_cast<float(*)[32]>(x));
            tmem_ld<32>(col + 32, *reinterpret_cast<float(*)[32]>(x + 32));
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              float4 k = make_float4(c2, c2, c2, c2);
              if constexpr (kFp8) k = *reinterpret_cast<const float4*>(&S.ksc[tk][c0 + i]);
              const float2 u = fma2(make_float2(x[i], x[i + 1]), make_float2(k.x, k.y), make_float2(ref, ref));
              const float2 v = fma2(make_float2(x[i + 2], x[i + 3]), make_float2(k.z, k.w), make_float2(ref, ref));
              x[i] = u.x;
              x[i + 1] = u.y;
              x[i + 2] = v.x;
              x[i + 3] = v.y;
            }
            if (masked) {
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if (!((seen[i >> 5] >> (i & 31)) & 1)) x[i] = -INFINITY;
            }
          };
          auto highest = [&]() {
            float m0 = x[0], m1 = x[1];
#pragma unroll
            for (int i = 2; i < 64; i += 4) {
              m0 = fmaxf(fmaxf(m0, x[i]), x[i + 1]);
              if (i + 3 < 64) m1 = fmaxf(fmaxf(m1, x[i + 2]), x[i + 3]);
            }
            return fmaxf(m0, m1);
          };
          scores(nref);
          if (bar_or(bar, kGroup, highest() > kSlack || !ok)) {
            if (bar_or(bar, kGroup, !ok)) {
              ok = false;
              break;
            }
            // new references: the rows' maxima so far, from the plain scores (the old reference may be far off, or none)
            scores(0.f);
            (&S.red[0][0][0])[wg * 128 + r] = highest();
            named_bar(bar, kGroup);
            const float m = fmaxf(-nref, fmaxf((&S.red[0][0][0])[r], (&S.red[0][0][0])[128 + r]));
            const float fac = ex2(-nref - m);
            nref = -m;
            l *= fac;
            if (j > 0) {  // the output tile holds the tiles before: wait for the last of them, then scale
              ok = ok && mbar_wait(&S.p_empty[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, a.status, 91, budget);
              ok = __all_sync(0xffffffffu, ok);
              tc_fence_after();
              const uint32_t o = tmem_base + lanes + (uint32_t)(C::kOCol + (seg % C::kOBufs) * C::kOCols + wg * (D / 2));
#pragma unroll
              for (int i0 = 0; i0 < D / 2; i0 += 8) {
                float v[8];
                uint32_t w[8];
                tmem_ld<8>(o + i0, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i] * fac);
                tmem_st8(o + i0, w);
              }
              tmem_st_wait();
            }
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] += nref;
          }
          float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const float2 u = make_float2(ex2(x[i]), ex2(x[i + 1]));
            const float2 v = make_float2(ex2(x[i + 2]), ex2(x[i + 3]));
            l2 = add2(l2, add2(u, v));
            float4 vs = make_float4(1.f, 1.f, 1.f, 1.f);
            if constexpr (kFp8) vs = *reinterpret_cast<const float4*>(&S.vsc[tk][c0 + i]);
            x[i] = u.x * vs.x;
            x[i + 1] = u.y * vs.y;
            x[i + 2] = v.x * vs.z;
            x[i + 3] = v.y * vs.w;
          }
          // the weights' tile: two, the scores just read were multiplied after
          // the weights of tile n - 2; one, free once those of tile n - 1 are
          if (C::kPBufs == 1 && n > 0) {
            ok = ok && mbar_wait(&S.p_empty[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, a.status, 92, budget);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
          }
          const uint32_t pcol = tmem_base + lanes + (uint32_t)(C::kPCol + (C::kPBufs == 2 ? (n & 1) * 64 : 0) + wg * 32);
#pragma unroll
          for (int i0 = 0; i0 < 64; i0 += 16) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if constexpr (C::kSplit)
                split_bf16(x[i0 + 2 * i], x[i0 + 2 * i + 1], hi[i], lo[i]);
              else
                hi[i] = pack_bf16(x[i0 + 2 * i], x[i0 + 2 * i + 1]);
            }
            tmem_st8(pcol + (i0 >> 1), hi);
            if constexpr (C::kSplit) tmem_st8(pcol + 64 + (i0 >> 1), lo);
          }
          l += l2.x + l2.y;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&S.p_full[n & 1]);
            if constexpr (kSel || kFp8) mbar_arrive(&S.tok_empty[tk]);
          }
          if (j == 0) store_output();
        }
        // ---- the segment's sums ----
        if (bar_or(bar, kGroup, !ok)) {
          ok = false;
          break;
        }
        S.sum[wg][r] = l;
        named_bar(bar, kGroup);
        const float sum = S.sum[0][r] + S.sum[1][r];
        pend = true;
        pend_whole = s.tiles == s.unit_tiles;
        pend_part = 2 * (int64_t)blockIdx.x + (first_seg ? 0 : 1);
        pend_par = seg % C::kOBufs;
        pend_phase = (seg / C::kOBufs) & 1;
        pend_row = orow;
        pend_inv = inverse(sum);
        if (wg == 0) {
          if (!pend_whole) {
            reinterpret_cast<float4*>(a.part_ml)[pend_part * N + r] = make_float4(-nref, sum, sum, 0.f);
          } else if (a.lse != nullptr && orow >= 0) {
            a.lse[orow] = sum == 0.f ? -INFINITY : (log2f(sum) - nref) * 0.693147181f;
          }
        }
        ++seg;
        first_seg = false;
      }
      if (ok) store_output();
    } else {
      // A thread owns one token and half of the query rows.
      constexpr int kC = N / 2;
      const int key = wq * 32 + lane, c0 = wg * kC;
      // this thread's P row: 16-byte units swizzled over the row's width
      const uint32_t p_off = (uint32_t)(key * C::kPRow), p_unit = wg * (kC / 8);
      // the rests: behind all rows' weights, with 64 rows in the next 64 columns
      constexpr uint32_t kRest = N == 64 ? kTile * 128 : 0, kRestUnit = N == 64 ? 0 : N / 8;
      const uint32_t p_sw = C::kPRow == 128 ? key & 7 : (C::kPRow == 64 ? (key >> 1) & 3 : (key >> 2) & 1);
      // 128 rows of O^T fill the 128 lanes; 64 fill the first 16 lanes of each warp
      const int dv = element(D == 128 ? wq * 32 + lane : wq * 16 + lane);
      const bool dv_ok = (D == 128 || lane < 16);
      auto store_output = [&]() {
        if (!pend) return;
        pend = false;
        ok = ok && mbar_wait(&S.o_full[pend_par], pend_phase, abort_flag, a.status, 93, budget);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const uint32_t o = tmem_base + lanes + (uint32_t)(C::kOCol + pend_par * C::kOCols + c0);
        float v[kC];
        tmem_ld<kC>(o, v);
        if constexpr (C::kSplit) {
          float rest[kC];
          tmem_ld<kC>(o + N, rest);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kC; ++i) v[i] += rest[i];
        } else {
          tmem_ld_wait();
        }
        if (ok && dv_ok && in_bounds(pend_whole || part_ok(pend_part, gridDim.x), a.status, 27)) {
          if (!pend_whole) {
            float* dst = a.part_o + (pend_part * N + c0) * D + dv;
#pragma unroll
            for (int i = 0; i < kC; ++i) dst[i * D] = v[i];
          } else if (dv < a.d) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + dv;
#pragma unroll
            for (int i = 0; i < kC; ++i) {
              const int r = S.orow[pend_par][c0 + i];
              if (r >= 0 && in_bounds(out_ok(a, r), a.status, 28)) out[(int64_t)r * a.d] = __float2bfloat16_rn(v[i] * S.lsum[pend_par][c0 + i]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.o_free[pend_par]);
      };
      while (walk.next(t, s)) {
        if (!s.valid) {
          first_seg = false;
          continue;
        }
        if (tid < kC) {
          const int r = c0 + tid, rr = s.row0 + r, j = rr / g;
          S.nref[r] = -kNoMax;
          S.rowmax[r] = kNoMax;
          S.lim[r] = kSel ? 0 : s.lim0 + (r < s.rows ? j : s.row0 / g);
          S.orow[seg & 1][r] = r < s.rows ? (s.q0 + j) * a.Hq + s.hk * g + (rr - j * g) : -1;
        }
        named_bar(bar, 128);
        constexpr int kL = C::kSplit ? 1 : kC / 2;
        float2 l[kC / 2], lr[kL];  // sums of the weights, and of their bf16
#pragma unroll
        for (int i = 0; i < kC / 2; ++i) l[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kL; ++i) lr[i] = make_float2(0.f, 0.f);
        bool common = true;   // one reference for this half's rows
        float cref = -kNoMax;  // it, negated
        for (int j = 0; j < s.tiles; ++j, ++n) {
          const int tile = s.tile0 + j, tk = n % kTok;
          if constexpr (kSel || kFp8) ok = ok && mbar_wait(&S.tok_full[tk], (n / kTok) & 1, abort_flag, a.status, 94, budget);
          ok = ok && mbar_wait(&S.s_full[n & 1], (n >> 1) & 1, abort_flag, a.status, 90, budget);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          const uint32_t col = tmem_base + lanes + (uint32_t)((n & 1) * C::kSCols + c0);
          const int pos = tile * kTile + key;
          bool masked, seen = true;
          if constexpr (kSel) {
            const uint32_t all = S.seen[tk][wq];
            masked = all != 0xffffffffu;
            seen = (all >> lane) & 1;
          } else {
            masked = (tile + 1) * kTile > s.lim0 + 1;  // some row does not see some token of this tile
          }
          const float cs = kFp8 ? S.ksc[tk][kFp8 ? key : 0] : c2;
          float x[kC];
          auto hide = [&]() {
            if (masked) {
#pragma unroll
              for (int i = 0; i < kC; ++i)
                if (!(kSel ? seen : pos <= S.lim[c0 + i])) x[i] = -INFINITY;
            }
          };
          auto scores = [&]() {  // log2 weights against the references
            tmem_ld<kC>(col, x);
            tmem_ld_wait();
            if (common) {
#pragma unroll
              for (int i = 0; i < kC; i += 2) {
                const float2 u = fma2(make_float2(x[i], x[i + 1]), make_float2(cs, cs), make_float2(cref, cref));
                x[i] = u.x;
                x[i + 1] = u.y;
              }
            } else {
#pragma unroll
              for (int i = 0; i < kC; i += 4) {
                const float4 m = *reinterpret_cast<const float4*>(&S.nref[c0 + i]);
                x[i] = fmaf(x[i], cs, m.x);
                x[i + 1] = fmaf(x[i + 1], cs, m.y);
                x[i + 2] = fmaf(x[i + 2], cs, m.z);
                x[i + 3] = fmaf(x[i + 3], cs, m.w);
              }
            }
            hide();
          };
          uint8_t* prow = S.p[n % C::kPBufs] + p_off;
          const float vs = kFp8 ? S.vsc[tk][kFp8 ? key : 0] : 1.f;
          auto put_weights = [&](auto add) {  // and adds them to the sums
#pragma unroll
            for (int i = 0; i < kC; i += 8) {
              uint32_t hi[4];
              [[maybe_unused]] uint32_t lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float w0 = x[i + 2 * e], w1 = x[i + 2 * e + 1];
                add(l[i / 2 + e], i + 2 * e, make_float2(w0, w1));
                if constexpr (C::kSplit) {
                  split_bf16(kFp8 ? w0 * vs : w0, kFp8 ? w1 * vs : w1, hi[e], lo[e]);
                } else {
                  hi[e] = pack_bf16(w0, w1);
                  add(lr[i / 2 + e], i + 2 * e, unpack_bf16(hi[e]));
                }
              }
              const uint32_t u = p_unit + (i >> 3);
              *reinterpret_cast<uint4*>(prow + ((u ^ p_sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              if constexpr (C::kSplit)
                *reinterpret_cast<uint4*>(prow + kRest + (((u + kRestUnit) ^ p_sw) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          };
          // One pass on the chance that no reference moves.  If one must, what
          // the pass left is either right against the old reference or, where
          // that was none or too far below, dropped.
          scores();
          float top = x[0], top2 = x[1];
#pragma unroll
          for (int i = 2; i < kC; i += 2) {
            top = fmaxf(top, x[i]);
            top2 = fmaxf(top2, x[i + 1]);
          }
          top = fmaxf(top, top2);
#pragma unroll
          for (int i = 0; i < kC; ++i) x[i] = ex2(x[i]);
          // P's buffer: two, the scores just read were multiplied after the
          // weights of tile n - 2; one, free once those of tile n - 1 are
          if (C::kPBufs == 1 && n > 0) {
            ok = ok && mbar_wait(&S.p_empty[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, a.status, 92, budget);
            ok = __all_sync(0xffffffffu, ok);
          }
          put_weights([](float2& u, int, float2 w) { u = add2(u, w); });
          if (bar_or(bar, 128, top > kSlack || !ok)) {
            if (bar_or(bar, 128, !ok)) {
              ok = false;
              break;
            }
            // new references: the rows' maxima so far, from the plain scores (the old reference may be far off, or none)
            tmem_ld<kC>(col, x);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < kC; ++i) x[i] *= cs;
            hide();
            const float m = warp_columns<kC, true>(x);
            if (lane < kC) S.red[wg][wq][lane] = m;
            named_bar(bar, 128);
            if (wq == 0) {
              const int r = c0 + lane % kC;
              const float old = -S.nref[r];
              float tile_max = S.red[wg][0][lane % kC];
#pragma unroll
              for (int w = 1; w < 4; ++w) tile_max = fmaxf(tile_max, S.red[wg][w][lane % kC]);
              const float row_max = fmaxf(S.rowmax[r], tile_max);
              // weights that are rounded once: whole numbers, so that a scaled sum of rounded weights is one of scaled ones
              const float own = fmaxf(old, C::kSplit ? tile_max : ceilf(tile_max));
              float hi = own, lo = row_max <= kNoMax ? INFINITY : row_max;
#pragma unroll
              for (int w = 16; w > 0; w >>= 1) {
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, w));
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, w));
              }
              // one for all while no row's best is too far below it
              const bool one = common && lo >= hi - kSpread;
              const float ref = one ? hi : own;
              __syncwarp();
              if (lane < kC) {
                S.rowmax[r] = row_max;
                S.nref[r] = -ref;
                // a jump that the weights just summed may not have held: 2^-96 of what stood before is nothing beside them
                S.fac[r] = ref - old > 96.f ? 0.f : C::kSplit ? ex2(old - ref) : __uint_as_float((uint32_t)(127 - (int)(ref - old)) << 23);
              }
              if (lane == 0) {
                S.common[wg] = one;
                S.cref[wg] = -hi;
              }
            }
            named_bar(bar, 128);
            common = S.common[wg] != 0;
            cref = S.cref[wg];
            if (j > 0) {  // the output tile holds the tiles before: wait for the last of them, then scale
              ok = ok && mbar_wait(&S.p_empty[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, a.status, 91, budget);
              ok = __all_sync(0xffffffffu, ok);
              tc_fence_after();
              const uint32_t o = tmem_base + lanes + (uint32_t)(C::kOCol + (seg & 1) * C::kOCols + c0);
#pragma unroll
              for (int i0 = 0; i0 < kC; i0 += 8) {
#pragma unroll
                for (int rest = 0; rest < C::kPCols / N; ++rest) {  // the rests' columns too, where there are any
                  float v[8];
                  uint32_t w[8];
                  tmem_ld<8>(o + rest * N + i0, v);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i] * S.fac[c0 + i0 + i]);
                  tmem_st8(o + rest * N + i0, w);
                }
              }
              tmem_st_wait();
            }
            scores();
#pragma unroll
            for (int i = 0; i < kC; ++i) x[i] = ex2(x[i]);
            if (!C::kSplit && j > 0) {
              // what the product takes must be what the sums hold: the bf16 that the first pass left, scaled (exact)
#pragma unroll
              for (int i = 0; i < kC; i += 8) {
                const uint4 w = *reinterpret_cast<const uint4*>(prow + (((p_unit + (i >> 3)) ^ p_sw) << 4));
                const uint32_t old[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 o = unpack_bf16(old[e]);
                  const float f0 = S.fac[c0 + i + 2 * e], f1 = S.fac[c0 + i + 2 * e + 1];
                  x[i + 2 * e] = f0 > 0.f ? o.x * f0 : x[i + 2 * e];
                  x[i + 2 * e + 1] = f1 > 0.f ? o.y * f1 : x[i + 2 * e + 1];
                }
              }
            }
            put_weights([&](float2& u, int c, float2 w) {  // the sums hold this tile already
              const float f0 = S.fac[c0 + c], f1 = S.fac[c0 + c + 1];
              u.x = f0 > 0.f ? u.x * f0 : w.x;
              u.y = f1 > 0.f ? u.y * f1 : w.y;
            });
          }
          fence_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&S.p_full[n & 1]);
            if constexpr (kSel || kFp8) mbar_arrive(&S.tok_empty[tk]);
          }
          if (j == 1) store_output();  // of the segment before: its products are done
        }
        // ---- the segment's sums ----
        if (bar_or(bar, 128, !ok)) {
          ok = false;
          break;
        }
        store_output();  // if this segment had one tile only
        pend = true;
        pend_whole = s.tiles == s.unit_tiles;
        pend_part = 2 * (int64_t)blockIdx.x + (first_seg ? 0 : 1);
        pend_par = seg & 1;
        pend_phase = (seg >> 1) & 1;
        {
          float v[kC];
#pragma unroll
          for (int i = 0; i < kC / 2; ++i) {
            v[2 * i] = l[i].x;
            v[2 * i + 1] = l[i].y;
          }
          const float sum = warp_columns<kC, false>(v);
          if (lane < kC) S.red[wg][wq][lane] = sum;
          if constexpr (!C::kSplit) {
#pragma unroll
            for (int i = 0; i < kC / 2; ++i) {
              v[2 * i] = lr[i].x;
              v[2 * i + 1] = lr[i].y;
            }
            const float rounded = warp_columns<kC, false>(v);
            if (lane < kC) S.red2[wg][wq][lane] = rounded;
          }
        }
        named_bar(bar, 128);
        if (tid < kC) {
          const int r = c0 + tid;
          float sum = 0.f, rounded = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) sum += S.red[wg][w][tid];
          if constexpr (!C::kSplit) {
#pragma unroll
            for (int w = 0; w < 4; ++w) rounded += S.red2[wg][w][tid];
          } else {
            rounded = sum;
          }
          if (!pend_whole) {
            // a row without tokens here says so: it may share a reference far above its own scores elsewhere
            reinterpret_cast<float4*>(a.part_ml)[pend_part * N + r] =
                make_float4(sum == 0.f ? kNoMax : -S.nref[r], sum, rounded, 0.f);
          } else if (a.lse != nullptr && S.orow[pend_par][r] >= 0) {
            a.lse[S.orow[pend_par][r]] = sum == 0.f ? -INFINITY : (log2f(sum) - S.nref[r]) * 0.693147181f;
          }
          S.lsum[pend_par][r] = inverse(rounded);
        }
        named_bar(bar, 128);  // the rows' state is free for the next segment
        ++seg;
        first_seg = false;
      }
      if (ok) store_output();
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
// joins rows 4 y .. 4 y + 3: a warp a row when the parts are few, else the
// warps share the parts of all four and meet in shared memory, in a fixed
// order.  It is all latency, so the loads of four parts are in flight at once.
// ----------------------------------------------------------------------------
template <int D>
struct JoinSum {
  static constexpr int kPer = D / 32;
  float m = kNoMax, l = 0.f, lr = 0.f, o[kPer] = {};
  __device__ __forceinline__ void add(float pm, float pl, float plr, const float (&v)[kPer]) {
    const float top = fmaxf(m, pm), f = ex2(m - top), pf = ex2(pm - top);
    m = top;
    l = l * f + pl * pf;
    lr = lr * f + plr * pf;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + v[i] * pf;
  }
};

template <int N, int D>
__global__ void __launch_bounds__(128) attend_tc_join_kernel(const AttendArgs a, const JoinDesc* desc) {
  constexpr int kRows = 4, kPer = D / 32;
  __shared__ float so[4][kRows][D], sm[4][kRows][3];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const JoinDesc d = desc[c];
  const int r0 = blockIdx.y * kRows;
  if (d.rows <= r0 || d.first >= (int64_t)c * d.run) return;  // no work there, or the cut falls between units
  const int64_t c0 = div64(d.first, d.run), c1 = div64(d.last - 1, d.run);
  if (c0 + 1 != c) return;  // an earlier cut of the same unit
  const int parts = (int)(c1 - c0) + 1;
  // parts: the end of run c0 (its only segment, or its last), then the beginnings of the others
  const int64_t slot0 = d.first == c0 * d.run ? 2 * c0 : 2 * c0 + 1;
  auto load = [&](int p, int r, float4& ml, float (&v)[kPer]) {  // lane l: elements kPer l .. kPer l + kPer - 1
    int64_t at = (p == 0 ? slot0 : 2 * (c0 + p)) * N + r0 + r;
    if (!in_bounds(part_ok(at / N, gridDim.x + 1), a.status, 29)) at = 0;
    ml = reinterpret_cast<const float4*>(a.part_ml)[at];
    if constexpr (kPer == 4) {
      const float4 x = reinterpret_cast<const float4*>(a.part_o + at * D)[lane];
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = reinterpret_cast<const float2*>(a.part_o + at * D)[lane];
      v[0] = x.x, v[1] = x.y;
    }
  };
  JoinSum<D> sum;
  if (parts <= 8) {
    for (int p0 = 0; p0 < parts; p0 += 4) {
      float4 ml[4];
      float v[4][kPer];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p0 + i < parts) load(p0 + i, warp, ml[i], v[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p0 + i < parts) sum.add(ml[i].x, ml[i].y, ml[i].z, v[i]);
    }
  } else {
    JoinSum<D> row[kRows];
    for (int p = warp; p < parts; p += 4) {
      float4 ml[kRows];
      float v[kRows][kPer];
#pragma unroll
      for (int r = 0; r < kRows; ++r) load(p, r, ml[r], v[r]);
#pragma unroll
      for (int r = 0; r < kRows; ++r) row[r].add(ml[r].x, ml[r].y, ml[r].z, v[r]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) so[warp][r][lane * kPer + i] = row[r].o[i];
      if (lane == 0) {
        sm[warp][r][0] = row[r].m;
        sm[warp][r][1] = row[r].l;
        sm[warp][r][2] = row[r].lr;
      }
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float v[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = so[w][warp][lane * kPer + i];
      sum.add(sm[w][warp][0], sm[w][warp][1], sm[w][warp][2], v);
    }
  }
  if (r0 + warp >= d.rows) return;
  const float inv = inverse(sum.lr);
  const int g = a.Hq / a.Hkv, rr = d.row0 + r0 + warp, j = rr / g;
  const int64_t orow = (int64_t)(d.q0 + j) * a.Hq + d.hk * g + (rr - j * g);
  if (!in_bounds(out_ok(a, orow), a.status, 30)) return;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {  // d is even here
    const int e = lane * kPer + i;
    if (e < a.d) *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + orow * a.d + e) = pack_bf16(sum.o[i] * inv, sum.o[i + 1] * inv);
  }
  if (lane == 0 && a.lse != nullptr) a.lse[orow] = sum.l == 0.f ? -INFINITY : (sum.m + log2f(sum.l)) * 0.693147181f;
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
  return sizeof(WsHeader) + round256((size_t)sms * sizeof(JoinDesc)) + round256((size_t)sms * 2 * N * 16) +
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
    // the roles' registers add up to what the launch brings; with fewer their shares would never come
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, attend_tc_kernel<N, D, kFp8, kSel>) != cudaSuccess) return DSA_ERR_CUDA;
    if (attr.numRegs != kLaunchRegs) return DSA_ERR_INTERNAL;
    if (cudaFuncSetAttribute(attend_tc_kernel<N, D, kFp8, kSel>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kSmem) != cudaSuccess)
      return DSA_ERR_CUDA;
    configured.fetch_or(bit, std::memory_order_release);
  }
  attend_tc_kernel<N, D, kFp8, kSel><<<grid, kWarps * 32, kSmem, st>>>(t);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (grid == 1 || (kSel && t.run % t.unit_tiles == 0)) return DSA_OK;  // no unit is divided
  // The join may take its place on the SMs while the last tiles run; it waits
  // for the whole grid before it reads a part.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid - 1, N / 4);
  cfg.blockDim = dim3(128);
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
  off += round256((size_t)sms * 2 * N * 16);
  t.a.part_o = reinterpret_cast<float*>(ws + off);
  t.row_stride_page = (int)(args.page_stride / args.d);
  wait_controls(t.wait_ns, t.hold_first_tile);
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
