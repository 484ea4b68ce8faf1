// mla_fp4_few.cu -- partial MLA decode over the 4-bit cache for requests of at
// most 96 query rows (H * q_len: all heads without drafts, or a tensor-parallel
// share of them with a few).  Same results as mla_tc_fp4.cu, whose clusters pad
// such a request to 256 rows; and, where a work list says so, for larger ones in
// groups of 96 rows, which end sooner when the work is short (mla_plan_sched).
//
// The products are turned round: tokens and value dims are the M side, the query
// rows the N side,
//   S^T[64 tokens, N rows] = K Q^T,   O^T[512 dims, N rows] += V^T P^T,
// so a row costs N = 16, 32, 64 or 96 of the MMA's width, not a padded 128 of
// its height, one CTA holds everything of a (request, part) and a token is
// converted once.  Per page:
//   the raw page   arrives in the converters' registers or by a bulk copy;
//   8 warps        convert it in two halves of the dims into 8-KB boxes (64
//                  tokens x 64 dims f16, 128-byte swizzle) that are the K-major
//                  A of the scores and, read MN-major, the A of the outputs; a
//                  ring of half pages, passed on and freed by halves;
//   1 thread       issues 36 MMAs of M = 64, N, K = 16 for the next page's S^T
//                  and this page's 4 per 128 value dims of O^T (M = 128);
//   4 or 8 warps   softmax: a thread has one token's scores of 8 to 24 rows.  The
//                  running references only change when some score passes the
//                  maximum its row's came from by 2^8: one vote per page; then
//                  the maxima cross the lanes and warps and O^T (lane = dim) is
//                  rescaled in place.  Row sums stay per thread until the end.
// P (f16, row by row over the tokens) and Q (f16, mla_tc_fp4.cu's row scale)
// are the K-major B operands in shared memory.
//
// What bounds it: shared-memory traffic.  A page's boxes are written once (74 KB)
// and read by both products, and an MMA this narrow runs at its operands' bytes,
// 128 a cycle (probe: M = 64 and N = 16, 32, 64, 96: 20, 21, 28, 40 cycles, M =
// 128: 34, 35, 41, 48).  All of it, raw pages included, is 240, 270, 370 and 430
// KB a page for the four widths, 1870 to 3360 cycles; measured at 152 requests,
// one per SM, 1.23, 1.30, 1.86 and 2.61 us a page (2300 to 4900 cycles) and 10 to
// 30 us for the rest of a launch with its merge.  (A profile of N = 96: the tensor
// cores' operand path busy 49% of the time, other shared-memory accesses 36%.)
// 32 ragged requests of 2k to 50k tokens x 16 heads take 86 us (165 MB, 1.9 TB/s),
// x 32 heads 92; 48 ragged x 96 heads 185 (the clusters: 214); 152 x 96 heads x
// 6400 tokens 293 (471).  From 97 rows on O^T and S^T need more than TMEM's 512
// columns.
#include <atomic>
#include <cstring>

#include "mla_combine.cuh"
#include "mla_fp4_decode.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kChunks = MLA_ROW_DIM / 64;  // 9 chunks of 64 dims
constexpr int kBox = kPage * 128;          // 8 KB: 64 tokens x 64 dims f16
constexpr int kHalf = 4 * kBox;            // half of a page's value dims
constexpr int kConvWarps = 8;
// Two softmax groups: 640 threads launch with 96 registers each (61440); the MMA
// warpgroup gives some away.  One-way, 128 x 64 + 256 x 96 + 256 x 112 = 61440.
constexpr int kRegsMma = 64;
constexpr int kRegsSoftmax = 112;

template <int N>
struct Few {
  static constexpr int kGroups = N > 32 ? 2 : 1;      // softmax warpgroups
  static constexpr int kConv0 = 4 * kGroups;          // first converter warp
  static constexpr int kMmaWarp = kConv0 + kConvWarps;
  // Two softmax groups: whole warpgroups, for the split of the registers.
  static constexpr int kThreads = kGroups == 2 ? 640 : 32 * (kMmaWarp + 1);
  static constexpr int kCols1 = N / kGroups;          // rows of a group
  static constexpr int kH = kCols1 / 2;               // rows of a softmax thread
  static constexpr int kLd = N > 16 ? 32 : 16;        // O^T columns read at a time
  // What 227 KB of shared memory and 512 TMEM columns leave room for.  (A ring
  // of three half pages instead of four costs N = 16 and 32 a quarter: 168 and
  // 181 us for 135 and 146 at 152 x 6400 tokens; five, which leave less L1 for
  // the pages on their way, 138 and 142.)
  static constexpr int kHalves = N > 32 ? 3 : 4;      // ring of half pages
  static constexpr int kSBufs = N > 64 ? 1 : 2;       // S^T buffers
  static constexpr int kPBufs = N > 32 ? 1 : 2;       // P buffers
  // How the raw pages arrive: straight to the converters' registers, a page
  // ahead, which saves their way through shared memory but takes as much L1 as
  // a page has bytes, so it loses where the rings leave little of the 256 KB;
  // through one raw buffer; or (0) through the slot that the page's first half
  // is converted into.  At 152 x 6400 tokens, registers against bulk copies: N =
  // 16 135 and 140 us, 32 146 and 150, 64 223 and 199, 96 298 and 286.
  static constexpr bool kDirect = N <= 32;
  static constexpr int kRaw = N > 64 ? 0 : 1;
  // In-slot copies are at most kHalves / 2 pages ahead of the converters.
  static constexpr int kRawFull = kRaw > 0 ? kRaw : 2;
  static_assert(kRaw > 0 || kHalves <= 4, "a raw_full phase per page in the ring");
  static constexpr int kQBox = N * 128;               // N rows x 64 values
  static constexpr uint32_t kColO = kSBufs * N;
  static constexpr uint32_t kIdescS = idesc_f16_f32(64, N, false, false);
  static constexpr uint32_t kIdescO = idesc_f16_f32(128, N, true, false);
  static constexpr uint32_t kCols = N > 32 ? 512 : 256;
  static_assert(kColO + 4 * N <= kCols, "TMEM columns");
  struct __align__(1024) Smem {
    uint8_t v[kHalves][kHalf];
    uint8_t kr[kBox];           // the RoPE key (one: a second has no room)
    uint8_t q[kChunks][kQBox];
    uint8_t pt[kPBufs][kQBox];  // P: rows x 64 tokens
    uint8_t raw[kRaw > 0 && !kDirect ? kRawBytes : 16];
    float sc[N];                // softmax scale (log2) * g * the row's 2^(e - 14)
    float mref[N];              // running references
    int32_t lim[N];             // tokens of the request the row sees
    float wred[4][N];           // per-quadrant maxima, then sums; row 0 passes on
                                // the factors of a rescale and, last, g / l
    uint64_t raw_full[kRawFull];   // a raw page has landed
    uint64_t raw_empty;            // the converter warps have read it
    uint64_t qfull;             // the query rows are written
    uint64_t cfull[kHalves];    // a half page is written (8 warps)
    uint64_t rfull;             // a page's RoPE key is written (8 warps)
    uint64_t vfree[kHalves];    // the outputs' products have read it
    uint64_t sfull[kSBufs];     // the buffer holds a page's scores
    uint64_t sread[kSBufs];     // the softmax warps have them in registers
    uint64_t pready[kPBufs];    // P is written, O^T rescaled
    uint64_t odone[kPBufs];     // a page's outputs are added
    uint64_t drain;
    uint32_t raw_bad[kRawFull];
    uint32_t tmem_base;
    int abort_flag;
    int last;                   // fused combine: the unit's last part
  };
  static_assert(sizeof(Smem) <= 227 * 1024, "shared memory budget");
};

// A unit: a part of a request's pages for one group of at most 96 of its rows.
struct GroupRange : UnitRange {
  int r0;  // the group's first row
};
__device__ __forceinline__ int g_rows(const Fp4Params& p, const GroupRange& w) {
  return min(p.q_len * p.H - w.r0, kFp4FewRows);
}
// Its first row among the partial outputs.
__device__ __forceinline__ int64_t first_row(const Fp4Params& p, const GroupRange& w) {
  const int64_t R = (int64_t)p.q_len * p.H, part = (int64_t)w.split * (p.V / p.B) + w.shard;
  return (part * p.B + w.b) * R + w.r0;
}

template <typename S>
__device__ __forceinline__ void give_up(S& s, const Fp4Params& p) {
  if (p.status) atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
  *const_cast<volatile int*>(&s.abort_flag) = 1;
}

// 32 lanes x N consecutive columns.
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 32) {
    tmem_ld32(taddr, r);
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}
// Whether any of the kThreadsIn softmax threads says so (named barrier 1).
template <int kThreadsIn>
__device__ __forceinline__ bool any_of(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(kThreadsIn)
      : "memory");
  return r != 0;
}

// The query rows, by the softmax and the converter warps while the first page
// arrives: warp k rows k, k + kQWarps, ..., their loads in flight together.
// q 2^(14 - e) as f16 into the K-major operand boxes; rows past R become zeros
// that see nothing.
template <int N>
__device__ __forceinline__ void place_query(typename Few<N>::Smem& s, const Fp4Params& p,
                                            const GroupRange& w, int warp, int lane) {
  constexpr int kWarps = Few<N>::kMmaWarp, kRows = (N + kWarps - 1) / kWarps;
  const int R = g_rows(p, w);
  const float g = p.g[0];
  uint4 x[kRows][3];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int n = warp + kWarps * r;
    const int64_t row = (int64_t)w.b * p.q_len * p.H + w.r0 + n;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int c = lane + 32 * k;  // 16-byte chunk of the row's 72
      x[r][k] = make_uint4(0, 0, 0, 0);
      if (n < R && c < 72) x[r][k] = c < 64 ? p.q_nope[row * 64 + c] : p.q_rope[row * 8 + c - 64];
    }
  }
  float mine = 0.f;  // lane r: 2^(e - 14) of the warp's row r
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int n = warp + kWarps * r;
    uint32_t big2 = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      big2 = __vmaxu2(big2, __vmaxu2(__vmaxu2(x[r][k].x & 0x7FFF7FFFu, x[r][k].y & 0x7FFF7FFFu),
                                     __vmaxu2(x[r][k].z & 0x7FFF7FFFu, x[r][k].w & 0x7FFF7FFFu)));
    const uint32_t big = __reduce_max_sync(kFull, max(big2 & 0xFFFFu, big2 >> 16));
    const int e = max(min((int)(big >> 7), 254) - 127, -100);
    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    const auto conv = [&](uint32_t v) -> uint32_t {
      return pack_f16(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
    };
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int c = lane + 32 * k;
      if (n < N && c < 72)
        *reinterpret_cast<uint4*>(s.q[c >> 3] + (n >> 3) * 1024 + (n & 7) * 128 +
                                  (((c & 7) ^ (n & 7)) << 4)) =
            make_uint4(conv(x[r][k].x), conv(x[r][k].y), conv(x[r][k].z), conv(x[r][k].w));
    }
    if (lane == r) mine = __uint_as_float((uint32_t)(127 + e - 14) << 23);
  }
  const int n = warp + kWarps * lane;
  if (lane < kRows && n < N) {
    const int i = (w.r0 + n) / p.H;
    int64_t lim = 0;
    if (n < R) {
      lim = p.kv_limit ? (int64_t)p.kv_limit[(int64_t)w.v * p.q_len + i] : w.L - p.q_len + 1 + i;
      lim = lim > w.L ? w.L : (lim < 0 ? 0 : lim);
    }
    s.lim[n] = (int32_t)lim;
    s.sc[n] = score_factor(p.scale_log2, g, mine);
    s.mref[n] = -INFINITY;
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&s.qfull));
}

// A position in the ring of half pages and the times it has wrapped round.
template <int K>
struct Ring {
  uint32_t slot = 0, turn = 0;
  __device__ __forceinline__ void next() {
    if (++slot == K) {
      slot = 0;
      ++turn;
    }
  }
};

// One warp: the unit's pages as they are stored, one bulk copy each, into the raw
// ring or, where there is no room for one, into the free half-page slot in which
// the page's first half will be converted.
template <int N>
__device__ __forceinline__ void copy_pages(typename Few<N>::Smem& s, const Fp4Params& p,
                                           const UnitRange& w, int lane) {
  using F = Few<N>;
  bool ok = true;
  int issued = 0;
  int32_t ent = 0;
  Ring<F::kHalves> ring;
  for (int m = 0; m < w.npages && ok; ++m) {
    if (m % 32 == 0) ent = page_entry(p, w, m + lane);
    const int32_t base = checked_base(p, __shfl_sync(kFull, ent, m & 31));
    if (lane == 0) {
      const int f = m % F::kRawFull;
      bool free;
      uint8_t* dst;
      if constexpr (F::kRaw > 0) {
        free = mbar_wait_cta(smem_u32(&s.raw_empty), (m & 1) ^ 1, &s.abort_flag);
        dst = s.raw;
      } else {
        free = ring.turn == 0 || mbar_wait_cta(smem_u32(&s.vfree[ring.slot]), (ring.turn - 1) & 1,
                                           &s.abort_flag);
        dst = s.v[ring.slot];
      }
      if (free) {
        const uint32_t bar = smem_u32(&s.raw_full[f]);
        s.raw_bad[f] = base < 0;
        if (base < 0) {
          if (p.status) atomicOr(p.status, MLA_STATUS_BAD_SLOT);
          mbar_arrive(bar);
        } else {
          mbar_arrive_expect_tx(bar, kRawBytes);
          bulk_load(smem_u32(dst), p.kv + (int64_t)base * kFp4RowBytes, kRawBytes, bar);
        }
        ++issued;
      } else {
        ok = false;
      }
    }
    ring.next();
    ring.next();
    ok = __shfl_sync(kFull, ok, 0);
  }
  if (!ok && lane == 0) {
    give_up(s, p);
    // No copy may still be in flight when the CTA leaves.
    int never = 0;
    for (int i = max(0, issued - F::kRawFull); i < issued; ++i)
      mbar_wait_cta(smem_u32(&s.raw_full[i % F::kRawFull]), (i / F::kRawFull) & 1, &never);
  }
}

// Two E4M3 scales with a NaN (0x7F, 0xFF) replaced by 0.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
  if ((w & 0x7Fu) == 0x7Fu) w &= 0xFF00u;
  if ((w & 0x7F00u) == 0x7F00u) w &= 0x00FFu;
  return w;
}

__device__ __forceinline__ uint4 load_nc(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint16_t load_nc2(const uint8_t* p) {
  uint16_t v;
  asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

// A converter thread's share of a raw page, of which `row` is the warp's first
// token.
struct RawShare {
  uint4 code[4], rope;
  uint32_t scale[4];
  bool bad;

  template <bool kGlobal>
  __device__ __forceinline__ void read(const uint8_t* row, int t4, int v, int rt, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* r = row + (t4 + 4 * (j & 1)) * kFp4RowBytes;
      const uint8_t* c = r + (v + 8 * (j >> 1)) * 16;
      const uint8_t* q = r + kFp4ScaleOff + (v + 8 * (j >> 1)) * 2;
      code[j] = kGlobal ? load_nc(c) : *reinterpret_cast<const uint4*>(c);
      scale[j] = kGlobal ? load_nc2(q) : *reinterpret_cast<const uint16_t*>(q);
    }
    const uint8_t* k = row + rt * kFp4RowBytes + kFp4RopeOff + 16 * (lane & 3);
    rope = kGlobal ? load_nc(k) : *reinterpret_cast<const uint4*>(k);
  }
};

// The converters: warp k has tokens 8 k .. 8 k + 7, in registers from the
// raw page on.  Of the row's 16 vectors of 32 codes a lane has
// vector v = (lane & 1) + 2 (lane / 8) of the four tokens (lane / 2) % 4 + 4 j,
// and v + 8: the eight lanes of a phase of a 16-byte load or store touch
// eight different sixteenths of the banks' 128 bytes.  The scales of tokens past the length or of a bad page count as 0.  A
// NaN scale of a token that only some rows see has to show in those rows' scores
// but must not reach O through a masked p = 0: the boxes, shared by both
// products, hold 0 there and the token's RoPE key, which only the scores read,
// is NaN instead.
template <int N>
__device__ __forceinline__ void convert(typename Few<N>::Smem& s, const Fp4Params& p,
                                        const GroupRange& w, int warp, int lane) {
  using F = Few<N>;
  const int t4 = (lane >> 1) & 3, v = (lane & 1) + 2 * (lane >> 3);
  const int rt = lane >> 2;  // token of the lane's RoPE codes
  const uint32_t at_v = (lane >> 3) * kBox + warp * 1024, ch = 4 * (lane & 1);
  const uint32_t at_r = warp * 1024 + rt * 128;
  bool ok = true;
  // Where the warps meet at a barrier a warp that gave up goes on, waiting for
  // nothing else.
  const auto stop = [&] { return F::kRaw > 0 && !__all_sync(kFull, ok); };
  Ring<F::kHalves> ring;
  RawShare next;
  int32_t ent = 0, ent_next = 0;
  if constexpr (F::kDirect) {
    ent = page_entry(p, w, lane);
    ent_next = page_entry(p, w, 32 + lane);
  }
  const auto load = [&](int m) {
    if (m > 0 && m % 32 == 0) {
      ent = ent_next;
      ent_next = page_entry(p, w, m + 32 + lane);
    }
    const int32_t base = checked_base(p, __shfl_sync(kFull, ent, m & 31));
    next.bad = base < 0;
    if (next.bad) {
      if (warp == 0 && lane == 0 && p.status) atomicOr(p.status, MLA_STATUS_BAD_SLOT);
      return;
    }
    next.read<true>(p.kv + ((int64_t)base + 8 * warp) * kFp4RowBytes, t4, v, rt, lane);
  };
  if constexpr (F::kDirect) load(0);
  place_query<N>(s, p, w, F::kConv0 + warp, lane);
  for (int m = 0; m < w.npages; ++m) {
    RawShare x;
    if constexpr (F::kDirect) {
      x = next;
      if (m + 1 < w.npages) load(m + 1);
    } else {
      const int f = m % F::kRawFull;
      ok = ok && mbar_wait_cta(smem_u32(&s.raw_full[f]), (m / F::kRawFull) & 1, &s.abort_flag);
      if (stop()) break;
      x.bad = s.raw_bad[f] != 0;
      x.read<false>((F::kRaw > 0 ? s.raw : s.v[ring.slot]) + 8 * warp * kFp4RowBytes, t4, v, rt,
                    lane);
      __syncwarp();  // every lane has read the page
      if (F::kRaw > 0 && lane == 0) mbar_arrive(smem_u32(&s.raw_empty));
      // In its slot: every warp has, before it is written over.
      if (F::kRaw == 0) named_bar_sync(3, 32 * kConvWarps);
    }
    const int64_t at = (w.p0 + m) * kPage + 8 * warp;  // the warp's first token
    bool nan = false;  // the token of the lane's RoPE codes has a NaN scale
    if (at + 8 > w.nmin || x.bad) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t4 + 4 * (j & 1);
        const bool live = at + t < w.L && !x.bad;
        const uint32_t f = live ? finite_pair(x.scale[j]) : 0u;
        const uint32_t b = __ballot_sync(kFull, live && f != x.scale[j]);
        if (b & (0x03030303u << (2 * (rt & 3))) && (rt >> 2) == (j & 1)) nan = true;
        x.scale[j] = f;
      }
      if (x.bad) x.rope = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // What lay in this slot before has been read.
      if (ring.turn > 0 && (F::kRaw > 0 || h == 1))
        ok = ok && mbar_wait_cta(smem_u32(&s.vfree[ring.slot]), (ring.turn - 1) & 1, &s.abort_flag);
      if (stop()) break;
      uint8_t* const box = s.v[ring.slot] + at_v;
#pragma unroll
      for (int j = 2 * h; j < 2 * h + 2; ++j) {
        const int t = t4 + 4 * (j & 1);
        const uint32_t sc = e4m3x2_to_f16(x.scale[j]);
        const uint32_t lo = __byte_perm(sc, sc, 0x1010), hi = __byte_perm(sc, sc, 0x3232);
        uint8_t* const b = box + t * 128;
        *reinterpret_cast<uint4*>(b + (((ch + 0) ^ t) << 4)) = scaled8(x.code[j].x, lo);
        *reinterpret_cast<uint4*>(b + (((ch + 1) ^ t) << 4)) = scaled8(x.code[j].y, lo);
        *reinterpret_cast<uint4*>(b + (((ch + 2) ^ t) << 4)) = scaled8(x.code[j].z, hi);
        *reinterpret_cast<uint4*>(b + (((ch + 3) ^ t) << 4)) = scaled8(x.code[j].w, hi);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.cfull[ring.slot]));
      ring.next();
      if (h == 0) {
        // The RoPE key, once the last page's scores have read it.
        if (m > 0)
          ok = ok && mbar_wait_cta(smem_u32(&s.sfull[(m - 1) % F::kSBufs]),
                               ((m - 1) / F::kSBufs) & 1, &s.abort_flag);
        if (stop()) break;
        uint4 r0 = plain8(x.rope.x, x.rope.y);
        if (nan) r0.x = 0x7E007E00u;
        const uint32_t c = 2 * (lane & 3);
        *reinterpret_cast<uint4*>(s.kr + at_r + ((c ^ rt) << 4)) = r0;
        *reinterpret_cast<uint4*>(s.kr + at_r + (((c + 1) ^ rt) << 4)) =
            plain8(x.rope.z, x.rope.w);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.rfull));
      }
    }
    if (stop()) break;
  }
  if (!__all_sync(kFull, ok) && lane == 0) give_up(s, p);
}

// The MMA warp, one lane: every MMA of the unit: of this page's outputs and the
// next page's scores, whichever is ready first (in either fixed order one of
// them holds up the converters).  A ring of three half pages only ever holds
// the first half of the next page before this page's first half is left.
template <int N>
__device__ __forceinline__ void issue_mmas(typename Few<N>::Smem& s, const Fp4Params& p,
                                           const UnitRange& w, uint32_t tmem) {
  using F = Few<N>;
  const uint64_t qd = sdesc_sw128(smem_u32(s.q[0]), 16, 1024);
  const uint64_t pd = sdesc_sw128(smem_u32(s.pt[0]), 16, 1024);
  // K: K-major, 128-byte rows.  V^T: MN-major, the next 64 dims one box on, the
  // next 8 tokens 1 KB on.
  const uint64_t kd = sdesc_sw128(smem_u32(s.v[0]), 16, 1024);
  const uint64_t rd = sdesc_sw128(smem_u32(s.kr), 16, 1024);
  const uint64_t vd = sdesc_sw128(smem_u32(s.v[0]), kBox, 1024);
  bool ok = true;
  Ring<F::kHalves> in, out;  // of the scores and of the outputs
  const auto score_half = [&](int m, int h) {
    const uint32_t sb = m % F::kSBufs, d = tmem + sb * N, slot = in.slot;
    ok = ok && mbar_wait_cta(smem_u32(&s.cfull[slot]), in.turn & 1, &s.abort_flag);
    in.next();
    if (!ok) return;
    fence_proxy_async_smem();
    tc_fence_after();
    const uint64_t k0 = kd + slot * (kHalf >> 4), q0 = qd + h * 4 * (F::kQBox >> 4);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_ss(d, k0 + c * (kBox >> 4) + 2 * k, q0 + c * (F::kQBox >> 4) + 2 * k, F::kIdescS,
               (h | c | k) ? 1u : 0u);
    if (h == 0) {
      ok = ok && mbar_wait_cta(smem_u32(&s.rfull), m & 1, &s.abort_flag);
      if (!ok) return;
      fence_proxy_async_smem();
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_ss(d, rd + 2 * k, qd + 8 * (F::kQBox >> 4) + 2 * k, F::kIdescS, 1u);
    } else {
      mma_commit(smem_u32(&s.sfull[sb]));
    }
  };
  ok = mbar_wait_cta(smem_u32(&s.qfull), 0, &s.abort_flag);
  if (ok) {
    score_half(0, 0);
    score_half(0, 1);
  }
  for (int m = 0; m < w.npages && ok; ++m) {
    const uint32_t pb = m % F::kPBufs;
    const uint32_t pbar = smem_u32(&s.pready[pb]), pph = (m / F::kPBufs) & 1;
    int next = m + 1 < w.npages ? 0 : 2;  // first half of its scores still to issue
    if (next == 0) {
      // With two S^T buffers, that of m + 1 was read before P(m - 1) was ready.
      const uint32_t cbar = smem_u32(&s.cfull[in.slot]), cph = in.turn & 1;
      const uint32_t rbar = smem_u32(&s.sread[0]), rph = m & 1;
      const uint64_t t0 = globaltimer();
      for (uint32_t it = 1; !mbar_test_wait(pbar, pph); ++it) {
        if ((F::kSBufs == 2 || mbar_test_wait(rbar, rph)) && mbar_test_wait(cbar, cph)) {
          score_half(m + 1, next++);
          if (F::kHalves >= 4) score_half(m + 1, next++);
          break;
        }
        if ((it & 63) == 0 && (*const_cast<volatile int*>(&s.abort_flag) ||
                               globaltimer() - t0 > kWaitNs)) {
          ok = false;
          break;
        }
      }
    }
    ok = ok && mbar_wait_cta(pbar, pph, &s.abort_flag);
    if (!ok) break;
    fence_proxy_async_smem();
    tc_fence_after();
    const uint64_t p0 = pd + pb * (F::kQBox >> 4);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t slot = out.slot;
      out.next();
      const uint64_t v0 = vd + slot * (kHalf >> 4);
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(tmem + F::kColO + (uint32_t)(N * (2 * h + b)), v0 + 2 * b * (kBox >> 4) + 128 * k,
                 p0 + 2 * k, F::kIdescO, k ? 1u : (m ? 1u : 0u));
      mma_commit(smem_u32(&s.vfree[slot]));
    }
    mma_commit(smem_u32(&s.odone[pb]));
    while (next < 2 && ok) score_half(m + 1, next++);
  }
  if (!ok) give_up(s, p);
  // No MMA may still run when the accumulators are freed.
  int never = 0;
  mma_commit(smem_u32(&s.drain));
  mbar_wait_cta(smem_u32(&s.drain), 0, &never);
}

// 2 H columns of the 16 TMEM lanes from `taddr` on, the first half of them in
// lanes 0..15, the second half in lanes 16..31.
template <int H>
__device__ __forceinline__ void tmem_ld_halves(uint32_t taddr, uint32_t (&r)[H]) {
  if constexpr (H == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 16;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
#pragma unroll
    for (int k = 0; k < H; k += 8)
      asm volatile(
          "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;"
          : "=r"(r[k]), "=r"(r[k + 1]), "=r"(r[k + 2]), "=r"(r[k + 3]), "=r"(r[k + 4]),
            "=r"(r[k + 5]), "=r"(r[k + 6]), "=r"(r[k + 7])
          : "r"(taddr + k), "n"(H));
  }
}

// Softmax: an accumulator of M = 64 rows lies in the first 16 lanes of every
// TMEM quadrant, so a warp of quadrant `quad` has tokens 16 quad .. + 15 and a
// thread token 16 quad + lane % 16 with kH rows.  At the end, and when O^T is
// rescaled, thread = value dim of a block of 128.
template <int N>
__device__ __forceinline__ void softmax(typename Few<N>::Smem& s, const Fp4Params& p,
                                        const GroupRange& w, uint32_t tmem, int warp, int lane) {
  using F = Few<N>;
  constexpr int H = F::kH, T = 128 * F::kGroups;
  const int quad = warp & 3, group = warp >> 2, dim = quad * 32 + lane;
  const int tok = quad * 16 + (lane & 15), n0 = F::kCols1 * group + H * (lane >> 4);
  const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
  const int R = g_rows(p, w);
  float* const alpha = s.wred[0];
  place_query<N>(s, p, w, warp, lane);
  bool ok = mbar_wait_cta(smem_u32(&s.qfull), 0, &s.abort_flag);
  float l[H];
#pragma unroll
  for (int k = 0; k < H; ++k) l[k] = 0.f;
  uint8_t* const dst0 = s.pt[0] + (n0 >> 3) * 1024 + (tok & 7) * 2;
  for (int m = 0; m < w.npages; ++m) {
    const uint32_t sb = m % F::kSBufs, pb = m % F::kPBufs;
    uint32_t x[H];
    ok = ok && mbar_wait_cta(smem_u32(&s.sfull[sb]), (m / F::kSBufs) & 1, &s.abort_flag);
    tc_fence_after();
    if (__all_sync(kFull, ok)) {
      tmem_ld_halves<H>(trow + sb * N + F::kCols1 * group, x);
      tmem_wait_ld();
    }
    if (F::kSBufs == 1) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.sread[sb]));
    }
    // Scores in units of log2; tokens a row may not see become -inf (a select:
    // garbage or NaN in a masked score never propagates).
    const int64_t t0 = (w.p0 + m) * kPage;
    const bool open = t0 + kPage <= w.nmin;
    float y[H];
    bool over = false;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      if (k % 8 == 0) asm volatile("" ::: "memory");  // no more loads ahead: registers
      y[k] = __uint_as_float(x[k]) * s.sc[n0 + k];
      if (!open && t0 + tok >= s.lim[n0 + k]) y[k] = -INFINITY;
      over |= y[k] > s.mref[n0 + k] + (kLift + kTau);
    }
    if (any_of<T>(over)) {
      // Some row's maximum rises: the page's maxima over its 64 tokens.
#pragma unroll
      for (int k = 0; k < H; ++k) {
        if (k % 8 == 0) asm volatile("" ::: "memory");
        float z = fmaxf(y[k], -INFINITY);  // a NaN counts as none
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) z = fmaxf(z, __shfl_xor_sync(kFull, z, o));
        if ((lane & 15) == 0) s.wred[quad][n0 + k] = z;
      }
      named_bar_sync(2, T);
      if (group == 0 && dim < N) {
        const float mt = fmaxf(fmaxf(s.wred[0][dim], s.wred[1][dim]),
                               fmaxf(s.wred[2][dim], s.wred[3][dim]));
        const float old = s.mref[dim];
        float a = 1.f;
        if (mt > -INFINITY && (old == -INFINITY || mt > old + (kLift + kTau))) {
          const float ref = mt - kLift;
          if (old > -INFINITY) a = ex2(old - ref);  // else O and l are still zero
          s.mref[dim] = ref;
        }
        alpha[dim] = a;
      }
      named_bar_sync(2, T);
      bool scale = false;
#pragma unroll 4
      for (int n = 0; n < N; ++n) scale |= alpha[n] != 1.f;
#pragma unroll
      for (int k = 0; k < H; ++k) l[k] *= alpha[n0 + k];
      if (scale && m > 0) {  // the same in every thread
        ok = ok && mbar_wait_cta(smem_u32(&s.odone[(m - 1) % F::kPBufs]),
                             ((m - 1) / F::kPBufs) & 1, &s.abort_flag);
        tc_fence_after();
        if (__all_sync(kFull, ok)) {
#pragma unroll 1
          for (int b = group; b < 4; b += F::kGroups)
#pragma unroll 1
            for (int c = 0; c < N; c += 16) {
              const uint32_t at = trow + F::kColO + (uint32_t)(N * b + c);
              uint32_t o[16];
              tmem_ld_n<16>(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int n = 0; n < 16; ++n)
                o[n] = __float_as_uint(__uint_as_float(o[n]) * alpha[c + n]);
              tmem_st16(at, o);
            }
          tmem_wait_st();
        }
      }
    }
    // p = 2^(y - m_ref) (0 for a row that has seen nothing yet), f16 (see kLift)
    // at [row][token] once the outputs before have read this buffer.
    if (m >= F::kPBufs)
      ok = ok && mbar_wait_cta(smem_u32(&s.odone[pb]), (m / F::kPBufs - 1) & 1, &s.abort_flag);
    uint8_t* const dst = dst0 + pb * F::kQBox;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      if (k % 8 == 0) asm volatile("" ::: "memory");
      const float ref = s.mref[n0 + k];
      y[k] = ex2(y[k] - (ref == -INFINITY ? 0.f : ref));
      l[k] += y[k];
    }
#pragma unroll
    for (int k = 0; k < H; ++k)
      *reinterpret_cast<__half*>(dst + (k >> 3) * 1024 + (k & 7) * 128 +
                                 (((tok >> 3) ^ (k & 7)) << 4)) = __float2half_rn(y[k]);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.pready[pb]));
  }
  if (!__all_sync(kFull, ok) && lane == 0) give_up(s, p);

  // Row sums over the lanes and warps, LSE, and O_part = g O / l: lane = dim, so
  // every store of a warp is one line of a row.
  named_bar_sync(2, T);
#pragma unroll
  for (int k = 0; k < H; ++k) {
    float z = l[k];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    if ((lane & 15) == 0) s.wred[quad][n0 + k] = z;
  }
  named_bar_sync(2, T);
  const int64_t row0 = first_row(p, w);
  float* const fin = s.wred[0];
  if (group == 0 && dim < N) {
    const float lt = (s.wred[0][dim] + s.wred[1][dim]) + (s.wred[2][dim] + s.wred[3][dim]);
    if (dim < R)
      // no visible token: -inf; a NaN sum (a NaN score seen) stays NaN
      p.LSE_part[row0 + dim] =
          lt == 0.f ? -INFINITY : (s.mref[dim] + log2f(lt)) * 0.69314718055994531f;
    fin[dim] = lt == 0.f ? 0.f : p.g[0] / lt;
  }
  named_bar_sync(2, T);
  const int last = w.npages - 1;
  ok = ok && mbar_wait_cta(smem_u32(&s.odone[last % F::kPBufs]), (last / F::kPBufs) & 1,
                       &s.abort_flag);
  tc_fence_after();
  if (!__all_sync(kFull, ok)) {
    if (lane == 0) give_up(s, p);
    return;
  }
#pragma unroll 1
  for (int b = group; b < 4; b += F::kGroups)
#pragma unroll 1
    for (int c = 0; c < N; c += F::kLd) {
      uint32_t o[F::kLd];
      tmem_ld_n<F::kLd>(trow + F::kColO + (uint32_t)(N * b + c), o);
      tmem_wait_ld();
      const int64_t at = (row0 + c) * MLA_VALUE_DIM + 128 * b + dim;
#pragma unroll
      for (int n = 0; n < F::kLd; ++n) {
        if (c + n >= R) break;
        const float z = __uint_as_float(o[n]) * fin[c + n];
        if (p.o_bf16)
          reinterpret_cast<__nv_bfloat16*>(p.O_part)[at + n * MLA_VALUE_DIM] =
              __float2bfloat16_rn(z);
        else
          p.O_part[at + n * MLA_VALUE_DIM] = z;
      }
    }
}

template <int N>
__global__ void __launch_bounds__(Few<N>::kThreads, 1)
mla_partial_fp4_few_kernel(const Fp4Params p) {
  using F = Few<N>;
  constexpr int kThreads = F::kThreads;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023) {  // no room to round it up
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
    return;
  }
  typename F::Smem& s = *reinterpret_cast<typename F::Smem*>(smem_raw);
  const int warp = __shfl_sync(kFull, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  // The stream's next kernel (the LSE combine) may be scheduled from now on;
  // it waits for this grid's completion before it reads a part.
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int unit = launch_unit(p, blockIdx.x);
  if (unit < 0) {
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, MLA_STATUS_BAD_WORK);
    return;
  }
  GroupRange w;
  // Fewer rows than 96 are one group.
  unit_range(p, N == kFp4FewRows ? unit / p.U : unit, w);
  w.r0 = N == kFp4FewRows ? unit % p.U * kFp4FewRows : 0;
  const int R = p.q_len * p.H;
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    s.last = 0;
    for (int i = 0; i < F::kRawFull; ++i) mbar_init(smem_u32(&s.raw_full[i]), 1);
    mbar_init(smem_u32(&s.raw_empty), kConvWarps);
    for (int i = 0; i < F::kHalves; ++i) {
      mbar_init(smem_u32(&s.cfull[i]), kConvWarps);
      mbar_init(smem_u32(&s.vfree[i]), 1);
    }
    for (int i = 0; i < F::kSBufs; ++i) {
      mbar_init(smem_u32(&s.sfull[i]), 1);
      mbar_init(smem_u32(&s.sread[i]), 4 * F::kGroups);
    }
    for (int i = 0; i < F::kPBufs; ++i) {
      mbar_init(smem_u32(&s.pready[i]), 4 * F::kGroups);
      mbar_init(smem_u32(&s.odone[i]), 1);
    }
    mbar_init(smem_u32(&s.qfull), F::kMmaWarp);
    mbar_init(smem_u32(&s.rfull), kConvWarps);
    mbar_init(smem_u32(&s.drain), 1);
    fence_mbar_init();
    if (p.seq_lens[w.v] > p.r2t_stride && p.status)
      atomicOr(p.status, MLA_STATUS_BAD_LENGTH);
  }
  if (warp == F::kMmaWarp) {
    tmem_alloc(smem_u32(&s.tmem_base), F::kCols);
    tmem_relinquish();
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, s.tmem_base, 0);

  // The end of every role.  Roles that have split the registers never rejoin.
  const auto finish = [&]() {
    if (p.counters) __threadfence();  // this CTA's part before its arrival
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == F::kMmaWarp) tmem_dealloc(tmem, F::kCols);
    if (!p.counters) return;
    // Fused combine: the CTA whose arrival completes its group's count merges the
    // group's rows, every part being in memory by then.  A request has a counter
    // per 128 rows, so group k, which starts at row 96 k, counts at (3 k) / 4, in
    // the high or the low half where groups 4 i and 4 i + 1 share one.
    if (threadIdx.x == 0) {
      const int k = w.r0 / kFp4FewRows, parts = p.num_splits * (p.V / p.B);
      const bool shared = k % 4 == 1 || (k % 4 == 0 && k + 1 < p.U);
      int* c = p.counters + (int64_t)w.b * ((R + 127) / 128) + w.r0 / 128;
      const uint32_t one = k % 4 == 1 ? 1u << 16 : 1u;
      const uint32_t n = (uint32_t)atom_add_acq_rel_gpu(c, (int)one) + one;
      s.last = (!shared ? n : one == 1 ? n & 0xFFFFu : n >> 16) == (uint32_t)parts;
      if (s.last) atomicSub(reinterpret_cast<unsigned*>(c), (uint32_t)parts * one);
    }
    __syncthreads();
    if (!s.last) return;
    __threadfence();
    const int r1 = min(w.r0 + kFp4FewRows, R);
    for (int r = w.r0 + warp; r < r1; r += kThreads / 32)
      combine_row<true>(p.O_part, p.LSE_part, p.num_splits * (p.V / p.B), (int64_t)p.B * R,
                        (int64_t)w.b * R + r, p.out, p.lse_out, lane);
  };

  if (w.npages == 0) {
    // No tokens for this part: O = 0, LSE = -inf.
    const int rows = g_rows(p, w);
    const int64_t row0 = first_row(p, w);
    if ((int)threadIdx.x < rows) p.LSE_part[row0 + threadIdx.x] = -INFINITY;
    const int words = rows * MLA_VALUE_DIM / (p.o_bf16 ? 8 : 4);  // 16-byte words
    uint4* dst = reinterpret_cast<uint4*>(
        reinterpret_cast<uint8_t*>(p.O_part) + row0 * MLA_VALUE_DIM * (p.o_bf16 ? 2 : 4));
    for (int k = threadIdx.x; k < words; k += kThreads) dst[k] = make_uint4(0, 0, 0, 0);
  } else if (warp >= F::kMmaWarp) {
    if constexpr (F::kGroups == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (!F::kDirect && warp == F::kMmaWarp + 1) copy_pages<N>(s, p, w, lane);
    if (warp == F::kMmaWarp && elect_one()) issue_mmas<N>(s, p, w, tmem);
    __syncwarp();
    if constexpr (F::kGroups == 2) return finish();
  } else if (warp >= F::kConv0) {
    convert<N>(s, p, w, warp - F::kConv0, lane);
    if constexpr (F::kGroups == 2) return finish();
  } else {
    if constexpr (F::kGroups == 2)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax<N>(s, p, w, tmem, warp, lane);
    if constexpr (F::kGroups == 2) return finish();
  }
  finish();
}

template <int N>
int launch(const Fp4Params& p, int64_t units, cudaStream_t stream) {
  auto kernel = mla_partial_fp4_few_kernel<N>;
  // The attribute lasts as long as the device's context: set it once.
  static std::atomic<uint64_t> set_on{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(set_on.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(typename Few<N>::Smem));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(fp4 few)");
    set_on.fetch_or(bit);
  }
  kernel<<<(unsigned)units, Few<N>::kThreads, (int)sizeof(typename Few<N>::Smem), stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_partial_fp4_few_kernel");
  return MLA_OK;
}

}  // namespace

int launch_fp4_few(const Fp4Params& p, cudaStream_t stream) {
  const int64_t units = (int64_t)p.V * p.num_splits * p.U;
  const int R = p.q_len * p.H;
  return R <= 16   ? launch<16>(p, units, stream)
         : R <= 32 ? launch<32>(p, units, stream)
         : R <= 64 ? launch<64>(p, units, stream)
                   : launch<96>(p, units, stream);
}

}  // namespace mla
