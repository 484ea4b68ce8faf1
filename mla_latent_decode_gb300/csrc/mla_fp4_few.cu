// mla_fp4_few.cu -- partial MLA decode over the 4-bit cache for requests of at
// most 32 query rows (H * q_len: a tensor-parallel share of the heads without
// or with few drafts).  Same results as mla_tc_fp4.cu, whose clusters pad such
// a request to 256 rows.
//
// With few rows nothing repeats a token's conversion, so the cache's bytes
// bound the work (352 bytes per token against 34 to 70 kFLOP) as long as the
// conversion and the shared-memory traffic keep up.  The products are turned
// round: tokens and value dims are the M side, the query rows the N side,
//   S^T[64 tokens, N rows] = K Q^T,   O^T[512 dims, N rows] += V^T P^T,
// so a row costs N = 16 or 32 of the MMA's width, not a padded 128 of its
// height, and one CTA holds everything of a (request, part).  Per page:
//   warp 0       copies the raw page (one bulk copy; a ring of two);
//   warps 8-15   convert it in two halves of the dims: four threads per token,
//                a block of 16 of every 64 dims each, into 8-KB boxes (64 tokens
//                x 64 dims f16, 128-byte swizzle) that are the K-major A of the
//                scores and, read MN-major, the A of the outputs; two sets of
//                boxes, passed on and freed by halves;
//   warp 1       issues 36 MMAs of M = 64, N, K = 16 for the next page's S^T,
//                then this page's 4 per 128 value dims of O^T (M = 128);
//   warps 4-7    softmax: two threads per token, N / 2 scores each.  The running
//                references only change when some score passes its row's by
//                2^8: one vote per page; then the maxima cross the lanes and
//                warps and O^T (lane = dim) is rescaled in place.  Row sums
//                stay per thread until the end.
// P (f16, row by row over the tokens) and Q (f16, mla_tc_fp4.cu's row scale)
// are the K-major B operands in shared memory.  An MMA of this width costs its
// operand bytes at 128 per cycle (probe: M = 64, N = 16: 23 cycles, M = 128: 39),
// so a page's products take about 1400 cycles.
#include <cstring>

#include "mla_combine.cuh"
#include "mla_fp4_decode.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kChunks = MLA_ROW_DIM / 64;    // 9 chunks of 64 dims
constexpr int kBox = kPage * 128;            // 8 KB: 64 tokens x 64 dims f16
constexpr int kRaw = 2;                      // raw pages in flight

template <int N>
struct Few {
  static constexpr int kQBox = N * 128;               // N rows x 64 values
  static constexpr uint32_t kColO = 2 * N;            // after two S^T buffers
  static constexpr uint32_t kIdescS = idesc_f16_f32(64, N, false, false);
  static constexpr uint32_t kIdescO = idesc_f16_f32(128, N, true, false);
  static constexpr uint32_t kCols = 256;              // 6 N, a power of two
  static_assert(6 * N <= kCols, "TMEM columns");
  struct __align__(1024) Smem {
    uint8_t v[2][kChunks - 1][kBox];
    uint8_t kr[kBox];           // the RoPE key (one set: N = 32 leaves no room)
    uint8_t q[kChunks][kQBox];
    uint8_t pt[2][kQBox];       // P: rows x 64 tokens
    uint8_t raw[kRaw][kRawBytes];
    float sc[N];                // softmax scale (log2) * g * the row's 2^(e - 14)
    float mref[N];              // running references
    float alpha[N];
    float fin[N];               // g / l
    float wred[4][N];           // per-warp maxima, then sums
    int32_t lim[N];             // tokens of the request the row sees
    uint64_t raw_full[kRaw];    // a raw page landed
    uint64_t raw_empty[kRaw];   // the eight converter warps have read it
    uint64_t cfull[2][2];       // half h of box set b is written (8 warps)
    uint64_t sfull[2];          // S^T buffer b holds a page's scores
    uint64_t pready[2];         // P buffer b is written, O^T rescaled (4 warps)
    uint64_t vfree[2][2];       // the outputs' products have read half h of set b
                                // (h = 1: all of it, and P)
    uint64_t drain;
    uint32_t raw_bad[kRaw];
    uint32_t tmem_base;
    int abort_flag;
    int last;                   // fused combine: the unit's last part
  };
  static constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

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
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const uint32_t (&r)[N]) {
  if constexpr (N == 32)
    tmem_st32(taddr, r);
  else
    tmem_st16(taddr, r);
}

// Whether any of the 128 threads of warps 4..7 says so (named barrier 1).
__device__ __forceinline__ bool any_of_128(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// Warp 0: the unit's pages into the raw ring (see copy_pages of
// mla_tc_fp4.cu).
template <int N>
__device__ __forceinline__ void copy_pages(typename Few<N>::Smem& s, const Fp4Params& p,
                                           const UnitRange& w, int lane) {
  bool ok = true;
  int issued = 0;
  int32_t ent = 0;
  for (int m = 0; m < w.npages && ok; ++m) {
    if (m % 32 == 0) ent = page_entry(p, w, m + lane);
    const int32_t base = checked_base(p, __shfl_sync(kFull, ent, m & 31));
    if (lane == 0) {
      const int slot = m % kRaw;
      if (mbar_wait(smem_u32(&s.raw_empty[slot]), ((m / kRaw) & 1) ^ 1, &s.abort_flag)) {
        const uint32_t bar = smem_u32(&s.raw_full[slot]);
        s.raw_bad[slot] = base < 0;
        if (base < 0) {
          if (p.status) atomicOr(p.status, MLA_STATUS_BAD_SLOT);
          mbar_arrive(bar);
        } else {
          mbar_arrive_expect_tx(bar, kRawBytes);
          bulk_load(smem_u32(s.raw[slot]), p.kv + (int64_t)base * kFp4RowBytes, kRawBytes,
                    bar);
        }
        ++issued;
      } else {
        ok = false;
      }
    }
    ok = __shfl_sync(kFull, ok, 0);
  }
  if (!ok && lane == 0) {
    give_up(s, p);
    // No copy may still be in flight when the CTA leaves.
    int never = 0;
    for (int i = max(0, issued - kRaw); i < issued; ++i)
      mbar_wait(smem_u32(&s.raw_full[i % kRaw]), (i / kRaw) & 1, &never);
  }
}

// The query rows, all warps: warp n, n + 16, ... row n.  q 2^(14 - e) as f16
// into the K-major operand boxes; rows past R become zeros that see nothing.
template <int N>
__device__ __forceinline__ void place_query(typename Few<N>::Smem& s, const Fp4Params& p,
                                            const UnitRange& w, int warp, int lane) {
  const int R = p.q_len * p.H;
  for (int n = warp; n < N; n += kThreads / 32) {
    const int64_t row = (int64_t)w.b * R + n;
    uint4 x[3];
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int c = lane + 32 * k;  // 16-byte chunk of the row's 72
      x[k] = make_uint4(0, 0, 0, 0);
      if (n < R && c < 72)
        x[k] = c < 64 ? p.q_nope[row * 64 + c] : p.q_rope[row * 8 + c - 64];
      const uint32_t y[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        big = max(big, max(y[e] & 0x7FFFu, (y[e] >> 16) & 0x7FFFu));
    }
    big = __reduce_max_sync(kFull, big);
    const int e = max(min((int)(big >> 7), 254) - 127, -100);
    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    const auto conv = [&](uint32_t v) -> uint32_t {
      return pack_f16(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
    };
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int c = lane + 32 * k;
      if (c < 72)
        *reinterpret_cast<uint4*>(s.q[c >> 3] + (n >> 3) * 1024 + (n & 7) * 128 +
                                  (((c & 7) ^ (n & 7)) << 4)) =
            make_uint4(conv(x[k].x), conv(x[k].y), conv(x[k].z), conv(x[k].w));
    }
    if (lane == 0) {
      const int i = n / p.H;
      int64_t lim = 0;
      if (n < R) {
        lim = p.kv_limit ? (int64_t)p.kv_limit[(int64_t)w.v * p.q_len + i]
                         : w.L - p.q_len + 1 + i;
        lim = lim > w.L ? w.L : (lim < 0 ? 0 : lim);
      }
      s.lim[n] = (int32_t)lim;
      s.sc[n] = p.scale_log2 * p.g[0] * __uint_as_float((uint32_t)(127 + e - 14) << 23);
      s.mref[n] = -INFINITY;
    }
  }
}

// Warps 8..15: thread = token tid / 4 and block tid % 4 of each 64 dims (the
// 8-byte reads of rows 352 bytes apart and the swizzled 16-byte writes are both
// free of bank conflicts).  The scales of tokens past the length or of a bad
// page count as 0.  A NaN scale of a token that only some rows see has to show
// in those rows' scores but must not reach O through a masked p = 0: the boxes,
// shared by both products, hold 0 there and the token's RoPE key, which only
// the scores read, is NaN instead.
template <int N>
__device__ __forceinline__ void convert(typename Few<N>::Smem& s, const Fp4Params& p,
                                        const UnitRange& w, int tid, int lane) {
  const int t = tid >> 2, part = tid & 3;
  const uint32_t trow = (t >> 3) * 1024 + (t & 7) * 128;
  const uint32_t o0 = trow + (((2 * part) ^ (t & 7)) << 4);
  const uint32_t o1 = trow + (((2 * part + 1) ^ (t & 7)) << 4);
  bool ok = true;
  for (int m = 0; m < w.npages; ++m) {
    const int slot = m % kRaw, set = m & 1;
    const uint8_t* row = s.raw[slot] + t * kFp4RowBytes;
    ok = ok && mbar_wait(smem_u32(&s.raw_full[slot]), (m / kRaw) & 1, &s.abort_flag);
    const int64_t at = (w.p0 + m) * kPage + t;
    const bool bad = s.raw_bad[slot] != 0;
    uint2 code[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      code[c] = *reinterpret_cast<const uint2*>(row + 32 * c + 8 * part);
    const uint4 sa = *reinterpret_cast<const uint4*>(row + kFp4ScaleOff);
    const uint4 sb = *reinterpret_cast<const uint4*>(row + kFp4ScaleOff + 16);
    uint4 rope = *reinterpret_cast<const uint4*>(row + kFp4RopeOff + 16 * part);
    uint32_t sw[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
    bool nan = false;
    if (at >= w.nmin || bad) {
      const bool live = at < w.L && !bad;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t f = live ? finite_scales(sw[c]) : 0u;
        nan |= live && f != sw[c];
        sw[c] = f;
      }
      if (bad) rope = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();  // every lane has read the page
    if (lane == 0) mbar_arrive(smem_u32(&s.raw_empty[slot]));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // The page two back has left this half.
      if (m > 1)
        ok = ok && mbar_wait(smem_u32(&s.vfree[set][h]), ((m >> 1) - 1) & 1, &s.abort_flag);
      // The last page's scores have read the RoPE key.
      if (h == 1 && m > 0)
        ok = ok && mbar_wait(smem_u32(&s.sfull[set ^ 1]), ((m - 1) >> 1) & 1, &s.abort_flag);
      if (!__all_sync(kFull, ok)) break;
#pragma unroll
      for (int c = 4 * h; c < 4 * h + 4; ++c) {
        const uint32_t sc = e4m3x2_to_f16((sw[c] >> (8 * part)) & 0xFFu);
        const uint32_t s2 = __byte_perm(sc, sc, 0x1010);
        *reinterpret_cast<uint4*>(s.v[set][c] + o0) = scaled8(code[c].x, s2);
        *reinterpret_cast<uint4*>(s.v[set][c] + o1) = scaled8(code[c].y, s2);
      }
      if (h == 1) {
        uint4 r0 = plain8(rope.x, rope.y);
        if (nan) r0.x = 0x7E007E00u;
        *reinterpret_cast<uint4*>(s.kr + o0) = r0;
        *reinterpret_cast<uint4*>(s.kr + o1) = plain8(rope.z, rope.w);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.cfull[set][h]));
    }
    if (!__all_sync(kFull, ok)) break;
  }
  if (!__all_sync(kFull, ok) && lane == 0) give_up(s, p);
}

// Warp 1, one lane: every MMA of the unit: of this page's outputs and the next
// page's scores, whichever is ready first (in either fixed order one of them
// holds up the converters: scores first 120 us, as they come 90 us, for 32
// requests x 16 heads, 2k to 60k tokens).
template <int N>
__device__ __forceinline__ void issue_mmas(typename Few<N>::Smem& s, const Fp4Params& p,
                                           const UnitRange& w, uint32_t tmem) {
  using F = Few<N>;
  const uint64_t qd = sdesc_sw128(smem_u32(s.q[0]), 16, 1024);
  const uint64_t pd = sdesc_sw128(smem_u32(s.pt[0]), 16, 1024);
  // K: K-major, 128-byte rows.  V^T: MN-major, the next 64 dims one box on, the
  // next 8 tokens 1 KB on.
  const uint64_t kd = sdesc_sw128(smem_u32(s.v[0][0]), 16, 1024);
  const uint64_t rd = sdesc_sw128(smem_u32(s.kr), 16, 1024);
  const uint64_t vd = sdesc_sw128(smem_u32(s.v[0][0]), kBox, 1024);
  constexpr uint64_t kSet = (kChunks - 1) * (kBox >> 4);
  bool ok = true;
  const auto scores = [&](int m) {
    const uint32_t set = m & 1;
    const uint32_t d = tmem + set * N;
    const uint64_t k0 = kd + set * kSet;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ok = ok && mbar_wait(smem_u32(&s.cfull[set][h]), (m >> 1) & 1, &s.abort_flag);
      if (!ok) return;
      fence_proxy_async_smem();
      tc_fence_after();
#pragma unroll
      for (int c = 4 * h; c < 4 * h + 4 + h; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(d, (c < 8 ? k0 + c * (kBox >> 4) : rd) + 2 * k,
                 qd + c * (F::kQBox >> 4) + 2 * k, F::kIdescS, (c | k) ? 1u : 0u);
    }
    mma_commit(smem_u32(&s.sfull[set]));
  };
  if (w.npages > 0) scores(0);
  for (int m = 0; m < w.npages && ok; ++m) {
    const uint32_t set = m & 1;
    // The buffer of S^T(m + 1) was read before P(m - 1) was ready.
    const uint32_t pbar = smem_u32(&s.pready[set]), pph = (m >> 1) & 1;
    bool next = m + 1 < w.npages;  // its scores are still to issue
    if (next) {
      const uint32_t cbar = smem_u32(&s.cfull[set ^ 1][0]), cph = ((m + 1) >> 1) & 1;
      const uint64_t t0 = globaltimer();
      for (uint32_t it = 1; !mbar_try_wait(pbar, pph); ++it) {
        if (mbar_try_wait(cbar, cph)) {
          scores(m + 1);
          next = false;
          break;
        }
        if ((it & 63) == 0 && (*const_cast<volatile int*>(&s.abort_flag) ||
                               globaltimer() - t0 > kWaitNs)) {
          ok = false;
          break;
        }
      }
    }
    ok = ok && mbar_wait(pbar, pph, &s.abort_flag);
    if (!ok) break;
    fence_proxy_async_smem();
    tc_fence_after();
    const uint64_t v0 = vd + set * kSet, p0 = pd + set * (F::kQBox >> 4);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_ss(tmem + F::kColO + (uint32_t)(N * b), v0 + 2 * b * (kBox >> 4) + 128 * k,
               p0 + 2 * k, F::kIdescO, k ? 1u : (m ? 1u : 0u));
      if (b & 1) mma_commit(smem_u32(&s.vfree[set][b >> 1]));
    }
    if (next) scores(m + 1);
  }
  if (!ok) give_up(s, p);
  // No MMA may still run when the accumulators are freed.
  int never = 0;
  mma_commit(smem_u32(&s.drain));
  mbar_wait(smem_u32(&s.drain), 0, &never);
}

// N columns of the 16 TMEM lanes from `taddr` on, the first half of them in
// lanes 0..15, the second half in lanes 16..31.
template <int N>
__device__ __forceinline__ void tmem_ld_halves(uint32_t taddr, uint32_t (&r)[N / 2]) {
  if constexpr (N == 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 16;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], 8;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7])
        : "r"(taddr));
}

// Warps 4..7: an accumulator of M = 64 rows lies in the first 16 lanes of every
// TMEM quadrant, so warp `quad` has tokens 16 quad .. + 15 and a thread token
// 16 quad + lane % 16 with rows N / 2 (lane / 16) .. .  At the end, and when O^T
// is rescaled, thread = value dim of a block of 128.
template <int N>
__device__ __forceinline__ void softmax(typename Few<N>::Smem& s, const Fp4Params& p,
                                        const UnitRange& w, uint32_t tmem, int warp, int lane) {
  using F = Few<N>;
  constexpr int H = N / 2;
  const int quad = warp & 3, dim = quad * 32 + lane;
  const int tok = quad * 16 + (lane & 15), n0 = H * (lane >> 4);
  const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
  const int R = p.q_len * p.H;
  bool ok = true;
  float l[H], sc[H], m_ref[H];
#pragma unroll
  for (int k = 0; k < H; ++k) {
    l[k] = 0.f;
    sc[k] = s.sc[n0 + k];
    m_ref[k] = -INFINITY;
  }
  uint8_t* const dst0 = s.pt[0] + (tok & 7) * 2;
  for (int m = 0; m < w.npages; ++m) {
    const uint32_t set = m & 1;
    uint32_t x[H];
    ok = ok && mbar_wait(smem_u32(&s.sfull[set]), (m >> 1) & 1, &s.abort_flag);
    tc_fence_after();
    if (__all_sync(kFull, ok)) {
      tmem_ld_halves<N>(trow + set * N, x);
      tmem_wait_ld();
    }
    // Scores in units of log2; tokens a row may not see become -inf (a select:
    // garbage or NaN in a masked score never propagates).
    const int64_t t0 = (w.p0 + m) * kPage;
    const bool open = t0 + kPage <= w.nmin;
    float y[H];
    bool over = false;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      y[k] = __uint_as_float(x[k]) * sc[k];
      if (!open && t0 + tok >= s.lim[n0 + k]) y[k] = -INFINITY;
      over |= y[k] > m_ref[k] + kTau;
    }
    if (any_of_128(over)) {
      // Some row's maximum rises: the page's maxima over its 64 tokens.
#pragma unroll
      for (int k = 0; k < H; ++k) {
        float z = fmaxf(y[k], -INFINITY);  // a NaN counts as none
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) z = fmaxf(z, __shfl_xor_sync(kFull, z, o));
        if ((lane & 15) == 0) s.wred[quad][n0 + k] = z;
      }
      named_bar_sync(2, 128);
      if (dim < N) {
        const float mt = fmaxf(fmaxf(s.wred[0][dim], s.wred[1][dim]),
                               fmaxf(s.wred[2][dim], s.wred[3][dim]));
        const float old = s.mref[dim];
        float a = 1.f;
        if (mt > -INFINITY && (old == -INFINITY || mt > old + kTau)) {
          if (old > -INFINITY) a = ex2(old - mt);  // else O and l are still zero
          s.mref[dim] = mt;
        }
        s.alpha[dim] = a;
      }
      named_bar_sync(2, 128);
      bool scale = false;
#pragma unroll
      for (int n = 0; n < N; ++n) scale |= s.alpha[n] != 1.f;
#pragma unroll
      for (int k = 0; k < H; ++k) {
        l[k] *= s.alpha[n0 + k];
        m_ref[k] = s.mref[n0 + k];
      }
      if (scale && m > 0) {  // the same in every thread
        ok = ok && mbar_wait(smem_u32(&s.vfree[set ^ 1][1]), ((m - 1) >> 1) & 1, &s.abort_flag);
        tc_fence_after();
        if (__all_sync(kFull, ok)) {
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            uint32_t o[N];
            tmem_ld_n<N>(trow + F::kColO + (uint32_t)(N * b), o);
            tmem_wait_ld();
#pragma unroll
            for (int n = 0; n < N; ++n)
              o[n] = __float_as_uint(__uint_as_float(o[n]) * s.alpha[n]);
            tmem_st_n<N>(trow + F::kColO + (uint32_t)(N * b), o);
          }
          tmem_wait_st();
        }
      }
    }
    // p = 2^(y - m_ref) (0 for a row that has seen nothing yet), f16 at
    // [row][token] once the outputs of two pages back have read this buffer.
    if (m > 1) ok = ok && mbar_wait(smem_u32(&s.vfree[set][1]), ((m >> 1) - 1) & 1, &s.abort_flag);
    uint8_t* const dst = dst0 + set * F::kQBox;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const int n = n0 + k;
      const float e = ex2(y[k] - (m_ref[k] == -INFINITY ? 0.f : m_ref[k]));
      l[k] += e;
      *reinterpret_cast<__half*>(dst + (n >> 3) * 1024 + (n & 7) * 128 +
                                 (((tok >> 3) ^ (n & 7)) << 4)) = __float2half_rn(e);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.pready[set]));
  }
  if (!__all_sync(kFull, ok) && lane == 0) give_up(s, p);

  // Row sums over the lanes and warps, LSE, and O_part = g O / l: lane = dim, so
  // every store of a warp is one line of a row.
  named_bar_sync(2, 128);
#pragma unroll
  for (int k = 0; k < H; ++k) {
    float z = l[k];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    if ((lane & 15) == 0) s.wred[quad][n0 + k] = z;
  }
  named_bar_sync(2, 128);
  const int64_t rows = (int64_t)p.B * R;
  const int64_t part = (int64_t)w.split * (p.V / p.B) + w.shard;
  const int64_t row0 = part * rows + (int64_t)w.b * R;
  if (dim < N) {
    const float lt = (s.wred[0][dim] + s.wred[1][dim]) + (s.wred[2][dim] + s.wred[3][dim]);
    if (dim < R)
      // no visible token: -inf; a NaN sum (a NaN score seen) stays NaN
      p.LSE_part[row0 + dim] =
          lt == 0.f ? -INFINITY : (s.mref[dim] + log2f(lt)) * 0.69314718055994531f;
    s.fin[dim] = lt == 0.f ? 0.f : p.g[0] / lt;
  }
  named_bar_sync(2, 128);
  const int last = w.npages - 1;
  ok = ok && mbar_wait(smem_u32(&s.vfree[last & 1][1]), (last >> 1) & 1, &s.abort_flag);
  tc_fence_after();
  if (!__all_sync(kFull, ok)) {
    if (lane == 0) give_up(s, p);
    return;
  }
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    uint32_t o[N];
    tmem_ld_n<N>(trow + F::kColO + (uint32_t)(N * b), o);
    tmem_wait_ld();
    const int64_t at = row0 * MLA_VALUE_DIM + 128 * b + dim;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (n >= R) break;
      const float z = __uint_as_float(o[n]) * s.fin[n];
      if (p.o_bf16)
        reinterpret_cast<__nv_bfloat16*>(p.O_part)[at + n * MLA_VALUE_DIM] =
            __float2bfloat16_rn(z);
      else
        p.O_part[at + n * MLA_VALUE_DIM] = z;
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) mla_partial_fp4_few_kernel(const Fp4Params p) {
  using F = Few<N>;
  extern __shared__ uint8_t smem_raw[];
  typename F::Smem& s = *reinterpret_cast<typename F::Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(kFull, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  // The stream's next kernel (the LSE combine) may be scheduled from now on;
  // it waits for this grid's completion before it reads a part.
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int unit = launch_unit(p, blockIdx.x);
  if (unit < 0) {
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, MLA_STATUS_BAD_WORK);
    return;
  }
  UnitRange w;
  unit_range(p, unit, w);
  const int R = p.q_len * p.H;
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    s.last = 0;
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(smem_u32(&s.raw_full[i]), 1);
      mbar_init(smem_u32(&s.raw_empty[i]), 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.sfull[i]), 1);
      mbar_init(smem_u32(&s.pready[i]), 4);
      for (int h = 0; h < 2; ++h) {
        mbar_init(smem_u32(&s.cfull[i][h]), 8);
        mbar_init(smem_u32(&s.vfree[i][h]), 1);
      }
    }
    mbar_init(smem_u32(&s.drain), 1);
    fence_mbar_init();
    if (p.seq_lens[w.v] > p.r2t_stride && p.status)
      atomicOr(p.status, MLA_STATUS_BAD_LENGTH);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s.tmem_base), F::kCols);
    tmem_relinquish();
  }
  if (w.npages > 0) place_query<N>(s, p, w, warp, lane);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, s.tmem_base, 0);

  if (w.npages > 0) {
    if (warp == 0) {
      copy_pages<N>(s, p, w, lane);
    } else if (warp == 1) {
      if (elect_one()) issue_mmas<N>(s, p, w, tmem);
      __syncwarp();
    } else if (warp >= 8) {
      convert<N>(s, p, w, (int)threadIdx.x - 256, lane);
    } else if (warp >= 4) {
      softmax<N>(s, p, w, tmem, warp, lane);
    }
  } else {
    // No tokens for this part: O = 0, LSE = -inf.
    const int64_t rows = (int64_t)p.B * R;
    const int64_t part = (int64_t)w.split * (p.V / p.B) + w.shard;
    const int64_t row0 = part * rows + (int64_t)w.b * R;
    if ((int)threadIdx.x < R) p.LSE_part[row0 + threadIdx.x] = -INFINITY;
    const int words = R * MLA_VALUE_DIM / (p.o_bf16 ? 8 : 4);  // 16-byte words
    uint4* dst = reinterpret_cast<uint4*>(
        reinterpret_cast<uint8_t*>(p.O_part) + row0 * MLA_VALUE_DIM * (p.o_bf16 ? 2 : 4));
    for (int k = threadIdx.x; k < words; k += kThreads) dst[k] = make_uint4(0, 0, 0, 0);
  }
  if (p.counters) __threadfence();  // this CTA's part before its arrival
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, F::kCols);
  if (!p.counters) return;
  // Fused combine: the part whose arrival completes the request's count merges
  // its rows, every part being in memory by then.
  if (threadIdx.x == 0) {
    int* c = p.counters + w.b;
    s.last = atom_add_acq_rel_gpu(c, 1) == p.num_splits * (p.V / p.B) - 1;
    if (s.last) *c = 0;
  }
  __syncthreads();
  if (!s.last) return;
  __threadfence();
  for (int r = warp; r < R; r += kThreads / 32)
    combine_row<true>(p.O_part, p.LSE_part, p.num_splits * (p.V / p.B), (int64_t)p.B * R,
                      (int64_t)w.b * R + r, p.out, p.lse_out, lane);
}

template <int N>
int launch(const Fp4Params& p, int64_t units, cudaStream_t stream) {
  auto kernel = mla_partial_fp4_few_kernel<N>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Few<N>::kSmemBytes);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(fp4 few)");
  kernel<<<(unsigned)units, kThreads, Few<N>::kSmemBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_partial_fp4_few_kernel");
  return MLA_OK;
}

}  // namespace

int launch_fp4_few(const Fp4Params& p, cudaStream_t stream) {
  const int64_t units = (int64_t)p.V * p.num_splits;
  return p.q_len * p.H <= 16 ? launch<16>(p, units, stream) : launch<32>(p, units, stream);
}

}  // namespace mla
