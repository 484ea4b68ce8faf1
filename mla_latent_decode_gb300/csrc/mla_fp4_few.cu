// mla_fp4_few.cu -- partial MLA decode over the 4-bit cache for requests of at
// most 32 query rows (H * q_len: a tensor-parallel share of the heads without
// or with few drafts).  Same results as mla_tc_fp4.cu, whose clusters pad such
// a request to 256 rows.
//
// With few rows nothing repeats a token's conversion, so the cache's bytes
// bound the work (352 bytes per token against 34 to 70 kFLOP) as long as the
// conversion and the shared-memory traffic keep up.  The products are turned
// round: tokens and value dims are the M side, the query rows the N side,
//   S^T[128 tokens, N rows] = K Q^T,   O^T[512 dims, N rows] += V^T P^T,
// so a row costs N = 16 or 32 of the MMA's width, not a padded 128 of its
// height, and one CTA holds everything of a (request, part):
//   warp 0       raw pages by bulk copy;
//   warps 8-15   convert: thread = token; 128 dims of c_kv at a time go into two
//                16-KB boxes (128 tokens x 64 dims, 128-byte swizzle), which are
//                the K-major A of the scores and the MN-major A of the outputs;
//                the RoPE key goes to TMEM (A of the scores only);
//   warp 1       issues the MMAs of a two-page tile: 36 of M = 128, N, K = 16 for
//                S^T, then 8 per 128 value dims for O^T;
//   warps 4-7    softmax: thread = token, its N scores in registers.  The
//                running references only change when some score passes its
//                row's by 2^8: one vote per tile; then the maxima cross the
//                lanes and warps and O^T (lane = dim) is rescaled in place.
//                Row sums stay per thread until the end.
// P (f16, row by row over the tokens) and Q (f16, mla_tc_fp4.cu's row scale)
// are the K-major B operands in shared memory.
#include <cstring>

#include "mla_combine.cuh"
#include "mla_fp4_decode.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kTileTokens = 128;
constexpr int kChunks = MLA_ROW_DIM / 64;    // 9 chunks of 64 dims
constexpr int kVBox = kTileTokens * 128;     // 16 KB: 128 tokens x 64 dims f16
constexpr int kBatches = 5;                  // per tile: 4 x 128 dims, RoPE
constexpr uint32_t kColS = 32;               // the RoPE key takes TMEM columns [0, 32)

template <int N>
struct Few {
  static constexpr int kQBox = N * 128;               // N rows x 64 values
  static constexpr int kRaw = N == 16 ? 3 : 2;        // raw pages that fit
  static constexpr uint32_t kColO = kColS + N;        // four blocks of N columns
  static constexpr uint32_t kIdescS = idesc_f16_f32(128, N, false, false);
  static constexpr uint32_t kIdescO = idesc_f16_f32(128, N, true, false);
  static_assert(kColO + 4 * N <= 512, "TMEM columns");
  struct __align__(1024) Smem {
    uint8_t v[kChunks - 1][kVBox];
    uint8_t q[kChunks][kQBox];
    uint8_t pt[2][kQBox];       // P: rows x 64 tokens, for either page
    uint8_t raw[kRaw][kRawBytes];
    float sc[N];                // softmax scale (log2) * g * the row's 2^(e - 14)
    float mref[N];              // running references
    float alpha[N];
    float fin[N];               // g / l
    float wred[4][N];           // per-warp maxima, then sums
    int32_t lim[N];             // tokens of the request the row sees
    uint64_t raw_full[kRaw];    // a raw page landed
    uint64_t raw_empty[kRaw];   // its four converter warps are done with it
    uint64_t cfull[kBatches];   // batch i of the tile is converted (4 warps)
    uint64_t sfull;             // S^T is in TMEM (and K has been read)
    uint64_t sread;             // the softmax has read S^T (4 warps)
    uint64_t pready;            // P is written and O^T rescaled (4 warps)
    uint64_t vfree[4];          // the products with value dims 128 b .. have read
                                // their boxes (b = 3: all, and P)
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
  constexpr int kRaw = Few<N>::kRaw;
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

// Warps 8..15: warp % 4 gives the tokens (TMEM lanes) 32 (warp % 4) .. of the
// tile, so warps 2, 3 mod 4 hold the second page; the two sets of four warps
// take alternate batches.  The scales of tokens past the length or of a bad
// page count as 0.  A NaN scale of a token that only some rows see has to show
// in those rows' scores but must not reach O through a masked p = 0: the boxes,
// shared by both products, hold 0 there and the token's RoPE key, which only
// the scores read, is NaN instead.
template <int N>
__device__ __forceinline__ void convert(typename Few<N>::Smem& s, const Fp4Params& p,
                                        const UnitRange& w, uint32_t tmem, int warp,
                                        int lane) {
  constexpr int kRaw = Few<N>::kRaw;
  const int quad = warp & 3, set = (warp >> 2) & 1;
  const int tok = quad * 32 + lane, pg = tok >> 6, tr = tok & 63;
  const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
  const int ntiles = (w.npages + 1) / 2;
  bool ok = true;
  for (int t = 0; t < ntiles; ++t) {
    const int m = 2 * t + pg;
    const bool have = m < w.npages;
    const int slot = m % kRaw;
    const uint8_t* row = s.raw[slot] + tr * kFp4RowBytes;
    uint32_t sw[8] = {};
    bool bad = false, san = false;
    if (have) {
      ok = ok && mbar_wait(smem_u32(&s.raw_full[slot]), (m / kRaw) & 1, &s.abort_flag);
      const int64_t at = (w.p0 + m) * kPage + tr;
      bad = s.raw_bad[slot] != 0;
      san = at >= w.nmin && at < w.L;
      if (!bad && at < w.L) {
        const uint4 a = *reinterpret_cast<const uint4*>(row + kFp4ScaleOff);
        const uint4 b = *reinterpret_cast<const uint4*>(row + kFp4ScaleOff + 16);
        sw[0] = a.x, sw[1] = a.y, sw[2] = a.z, sw[3] = a.w;
        sw[4] = b.x, sw[5] = b.y, sw[6] = b.z, sw[7] = b.w;
      }
    }
    bool nan = false;
    if (san) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t f = finite_scales(sw[k]);
        nan |= f != sw[k];
        sw[k] = f;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatches; ++i) {
      if (((t + i) & 1) != set) continue;
      uint4 code[4];
      if (have) {
        const uint8_t* src = row + (i < 4 ? 64 * i : kFp4RopeOff);
#pragma unroll
        for (int k = 0; k < 4; ++k) code[k] = *reinterpret_cast<const uint4*>(src + 16 * k);
      }
      // The last tile's products have read this batch's boxes (the outputs come
      // after the scores) or its RoPE key (the scores).
      if (t > 0)
        ok = ok && mbar_wait(i < 4 ? smem_u32(&s.vfree[i]) : smem_u32(&s.sfull), (t - 1) & 1,
                             &s.abort_flag);
      if (!__all_sync(kFull, ok)) break;
      if (have && i < 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 32 dims: half a box row
          uint8_t* box = s.v[2 * i + (k >> 1)] + (tok >> 3) * 1024 + (tok & 7) * 128;
          const uint32_t sc =
              e4m3x2_to_f16((sw[2 * i + (k >> 1)] >> (16 * (k & 1))) & 0xFFFFu);
          const uint32_t lo = __byte_perm(sc, sc, 0x1010), hi = __byte_perm(sc, sc, 0x3232);
          const uint32_t cw[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(box + (((4 * (k & 1) + e) ^ (tok & 7)) << 4)) =
                scaled8(cw[e], e < 2 ? lo : hi);
        }
        fence_proxy_async_smem();
      } else if (have) {
        uint32_t h[32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (bad) code[k] = make_uint4(0, 0, 0, 0);
          const uint4 lo = plain8(code[k].x, code[k].y), hi = plain8(code[k].z, code[k].w);
          h[8 * k] = lo.x, h[8 * k + 1] = lo.y, h[8 * k + 2] = lo.z, h[8 * k + 3] = lo.w;
          h[8 * k + 4] = hi.x, h[8 * k + 5] = hi.y, h[8 * k + 6] = hi.z, h[8 * k + 7] = hi.w;
        }
        if (nan) h[0] = 0x7E007E00u;
        tmem_st32(trow, h);
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.cfull[i]));
    }
    if (!__all_sync(kFull, ok)) break;
    if (have && lane == 0) mbar_arrive(smem_u32(&s.raw_empty[slot]));
  }
  if (!__all_sync(kFull, ok) && lane == 0) give_up(s, p);
}

// Warp 1, one lane: every MMA of the unit.
template <int N>
__device__ __forceinline__ void issue_mmas(typename Few<N>::Smem& s, const Fp4Params& p,
                                           const UnitRange& w, uint32_t tmem) {
  using F = Few<N>;
  const uint64_t qd = sdesc_sw128(smem_u32(s.q[0]), 16, 1024);
  const uint64_t pd = sdesc_sw128(smem_u32(s.pt[0]), 16, 1024);
  // K: K-major, 128-byte rows.  V^T: MN-major, the next 64 dims one box on, the
  // next 8 tokens 1 KB on.
  const uint64_t kd = sdesc_sw128(smem_u32(s.v[0]), 16, 1024);
  const uint64_t vd = sdesc_sw128(smem_u32(s.v[0]), kVBox, 1024);
  const int ntiles = (w.npages + 1) / 2;
  bool ok = true;
  for (int t = 0; t < ntiles && ok; ++t) {
    if (t > 0) ok = mbar_wait(smem_u32(&s.sread), (t - 1) & 1, &s.abort_flag);
#pragma unroll
    for (int i = 0; i < kBatches; ++i) {
      ok = ok && mbar_wait(smem_u32(&s.cfull[i]), t & 1, &s.abort_flag);
      if (!ok) break;
      tc_fence_after();
      if (i < 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = 2 * i + (k >> 2);
          mma_ss(tmem + kColS, kd + c * (kVBox >> 4) + 2 * (k & 3),
                 qd + c * (F::kQBox >> 4) + 2 * (k & 3), F::kIdescS, (i | k) ? 1u : 0u);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(tmem + kColS, tmem + 8u * k, qd + 8 * (F::kQBox >> 4) + 2 * k, F::kIdescS, 1u);
      }
    }
    if (!ok) break;
    mma_commit(smem_u32(&s.sfull));
    ok = mbar_wait(smem_u32(&s.pready), t & 1, &s.abort_flag);
    if (!ok) break;
    tc_fence_after();
    const int pages = min(2, w.npages - 2 * t);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t d = tmem + F::kColO + (uint32_t)(N * b);
      for (int g = 0; g < pages; ++g)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(d, vd + 2 * b * (kVBox >> 4) + 512 * g + 128 * k,
                 pd + g * (F::kQBox >> 4) + 2 * k, F::kIdescO, (t | g | k) ? 1u : 0u);
      mma_commit(smem_u32(&s.vfree[b]));
    }
  }
  if (!ok) give_up(s, p);
  // No MMA may still run when the accumulators are freed.
  int never = 0;
  mma_commit(smem_u32(&s.drain));
  mbar_wait(smem_u32(&s.drain), 0, &never);
}

// Warps 4..7: thread = token 32 (warp % 4) + lane of every tile; at the end,
// and when O^T is rescaled, thread = value dim of a block of 128.
template <int N>
__device__ __forceinline__ void softmax(typename Few<N>::Smem& s, const Fp4Params& p,
                                        const UnitRange& w, uint32_t tmem, int warp, int lane) {
  using F = Few<N>;
  const int quad = warp & 3, tok = quad * 32 + lane;
  const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
  const int R = p.q_len * p.H;
  const int ntiles = (w.npages + 1) / 2;
  bool ok = true;
  float l[N];
#pragma unroll
  for (int n = 0; n < N; ++n) l[n] = 0.f;
  for (int t = 0; t < ntiles; ++t) {
    uint32_t x[N];
    ok = ok && mbar_wait(smem_u32(&s.sfull), t & 1, &s.abort_flag);
    tc_fence_after();
    if (__all_sync(kFull, ok)) {
      tmem_ld_n<N>(trow + kColS, x);
      tmem_wait_ld();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.sread));

    // Scores in units of log2; tokens a row may not see become -inf (a select:
    // garbage or NaN in a masked score never propagates).
    const int64_t t0 = (w.p0 + 2 * t) * kPage;
    const bool open = t0 + kTileTokens <= w.nmin && 2 * t + 1 < w.npages;
    const int64_t at = 2 * t + (tok >> 6) < w.npages ? t0 + tok : INT64_MAX;
    float y[N];
    bool over = false;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      y[n] = __uint_as_float(x[n]) * s.sc[n];
      if (!open && at >= s.lim[n]) y[n] = -INFINITY;
      over |= y[n] > s.mref[n] + kTau;
    }
    if (any_of_128(over)) {
      // Some row's maximum rises: the tile's maxima over all 128 tokens, as
      // integers that order like the floats (a NaN counts as none).
      float mine = 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int b = __float_as_int(y[n] == y[n] ? y[n] : -INFINITY);
        const int m = __reduce_max_sync(kFull, b ^ ((b >> 31) & 0x7FFFFFFF));
        if (lane == n) mine = __int_as_float(m ^ ((m >> 31) & 0x7FFFFFFF));
      }
      if (lane < N) s.wred[quad][lane] = mine;
      named_bar_sync(2, 128);
      if (tok < N) {
        const float mt = fmaxf(fmaxf(s.wred[0][tok], s.wred[1][tok]),
                               fmaxf(s.wred[2][tok], s.wred[3][tok]));
        const float old = s.mref[tok];
        float a = 1.f;
        if (mt > -INFINITY && (old == -INFINITY || mt > old + kTau)) {
          if (old > -INFINITY) a = ex2(old - mt);  // else O and l are still zero
          s.mref[tok] = mt;
        }
        s.alpha[tok] = a;
      }
      named_bar_sync(2, 128);
      bool scale = false;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        l[n] *= s.alpha[n];
        scale |= s.alpha[n] != 1.f;
      }
      if (scale && t > 0) {  // the same in every thread
        ok = ok && mbar_wait(smem_u32(&s.vfree[3]), (t - 1) & 1, &s.abort_flag);
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
    // [row][token] once the last tile's products have read P.
    if (t > 0) ok = ok && mbar_wait(smem_u32(&s.vfree[3]), (t - 1) & 1, &s.abort_flag);
    uint8_t* dst = s.pt[tok >> 6] + (tok & 7) * 2;
    const int cc = (tok & 63) >> 3;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float m = s.mref[n];
      const float e = ex2(y[n] - (m == -INFINITY ? 0.f : m));
      l[n] += e;
      *reinterpret_cast<__half*>(dst + (n >> 3) * 1024 + (n & 7) * 128 + ((cc ^ (n & 7)) << 4)) =
          __float2half_rn(e);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.pready));
    if (!__all_sync(kFull, ok) && lane == 0) give_up(s, p);
  }

  // Row sums over the lanes and warps, LSE, and O_part = g O / l: lane = dim, so
  // every store of a warp is one line of a row.
  named_bar_sync(2, 128);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float z = l[n];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    if (lane == 0) s.wred[quad][n] = z;
  }
  named_bar_sync(2, 128);
  const int64_t rows = (int64_t)p.B * R;
  const int64_t part = (int64_t)w.split * (p.V / p.B) + w.shard;
  const int64_t row0 = part * rows + (int64_t)w.b * R;
  if (tok < N) {
    const float lt = (s.wred[0][tok] + s.wred[1][tok]) + (s.wred[2][tok] + s.wred[3][tok]);
    if (tok < R)
      // no visible token: -inf; a NaN sum (a NaN score seen) stays NaN
      p.LSE_part[row0 + tok] =
          lt == 0.f ? -INFINITY : (s.mref[tok] + log2f(lt)) * 0.69314718055994531f;
    s.fin[tok] = lt == 0.f ? 0.f : p.g[0] / lt;
  }
  named_bar_sync(2, 128);
  ok = ok && mbar_wait(smem_u32(&s.vfree[3]), (ntiles - 1) & 1, &s.abort_flag);
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
    const int64_t at = row0 * MLA_VALUE_DIM + 128 * b + tok;
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
    for (int i = 0; i < F::kRaw; ++i) {
      mbar_init(smem_u32(&s.raw_full[i]), 1);
      mbar_init(smem_u32(&s.raw_empty[i]), 4);
    }
    for (int i = 0; i < kBatches; ++i) mbar_init(smem_u32(&s.cfull[i]), 4);
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&s.vfree[i]), 1);
    mbar_init(smem_u32(&s.sfull), 1);
    mbar_init(smem_u32(&s.sread), 4);
    mbar_init(smem_u32(&s.pready), 4);
    mbar_init(smem_u32(&s.drain), 1);
    fence_mbar_init();
    if (p.seq_lens[w.v] > p.r2t_stride && p.status)
      atomicOr(p.status, MLA_STATUS_BAD_LENGTH);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s.tmem_base), 512);
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
      convert<N>(s, p, w, tmem, warp, lane);
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
  if (warp == 1) tmem_dealloc(tmem, 512);
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
