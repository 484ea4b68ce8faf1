// mla_fp4_decode.cuh -- what the decode kernels over the 4-bit cache share:
// launch parameters, a work unit's request and page range, the raw page copies
// and the conversion of codes to f16 operands.
#pragma once

#include <cuda_bf16.h>

#include <cfloat>

#include "mla_fp4.cuh"
#include "mla_internal.h"
#include "ptx_sm103.cuh"

namespace mla {

constexpr int kPage = MLA_PAGE_SIZE;                     // 64 tokens
constexpr int kRawBytes = MLA_PAGE_SIZE * kFp4RowBytes;  // 22528
// A row's running reference is set kLift (log2 units) below the maximum it is
// taken from, and again once some score passes it by kLift + kTau, so a
// probability enters the second product as f16 of at most 2^(kLift + kTau) and
// the tail below the maximum has the rest of f16's range: full precision down to
// 2^-(14 + kLift) of it, nothing lost above 2^-(25 + kLift).  (kTau = 6 and 4, for
// a kLift of 8 and 10, rescale more often: 48 ragged requests x 96 heads 184, 191
// and 243 us, 16 x 5 x 96 x 100k tokens 1115, 1117 and 1341.)
constexpr float kTau = 8.f;
constexpr float kLift = 7.f;
static_assert(kTau + kLift <= 15.f, "2^15 and the rounding of the reference stay under 65504");
constexpr uint32_t kFull = 0xffffffffu;

// Instruction descriptor for kind::f16 with F16 A/B and an FP32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn_major,
                                                     bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
struct Fp4Params {
  const uint4* q_nope;     // bf16 [B, q_len, H, 512] as 16-B chunks
  const uint4* q_rope;     // bf16 [B, q_len, H, 64]
  const uint8_t* kv;
  const float* g;          // the pool's factor
  int64_t num_slots;
  const int32_t* r2t;
  int64_t r2t_stride;
  const int32_t* seq_lens;
  const int32_t* kv_limit;
  const int32_t* split_pages;  // [V, num_splits + 1] page boundaries or NULL
  const int32_t* work;         // unit ids in launch order or NULL
  int B, q_len, H, V, num_splits, U;  // U = row pairs (256 rows) per request
  float scale_log2;        // sm_scale * log2(e)
  float* O_part;
  float* LSE_part;
  int* status;
  int q_box_rows;          // rows of a query TMA box: min(128, B * q_len * H)
  int o_tma;               // O_part rows leave by TMA store (o_map is valid)
  int o_bf16;              // O_part holds bf16 values (else fp32)
  __nv_bfloat16* out;      // fused combine (NULL counters: partials only)
  float* lse_out;
  int* counters;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The factor of a row's raw scores: scale_log2 * g * row, row the power of two
// that its queries were divided by.  Kept a normal number: 0 or an infinity would
// make NaN of a masked column's -inf or of a score of 0, and below 2^-126 every
// score is 0 to the last bit of its exponential anyway.
__device__ __forceinline__ float score_factor(float scale_log2, float g, float row) {
  const float sc = scale_log2 * row * g;
  return sc < FLT_MIN ? FLT_MIN : sc > FLT_MAX ? FLT_MAX : sc;
}

// The kernel for requests of at most kFp4FewRows query rows (mla_fp4_few.cu).
int launch_fp4_few(const Fp4Params& p, cudaStream_t stream);

// A unit's request and its part of the request's pages.
struct UnitRange {
  int v, b, shard, split, npages;
  int64_t L, p0;
  int64_t nmin;  // fewest tokens any query of the request sees
};

// The k-th unit of the launch (split * V + v) * U + u: k itself or, with a
// work list, the list's entry; -1 for an entry outside [0, units).
__device__ __forceinline__ int launch_unit(const Fp4Params& p, int k) {
  if (!p.work) return k;
  const int unit = p.work[k];
  return unit < 0 || (int64_t)unit >= (int64_t)p.V * p.num_splits * p.U ? -1 : unit;
}

// Fills in the range of part sv = split * V + v.
__device__ __forceinline__ void unit_range(const Fp4Params& p, int sv, UnitRange& w) {
  w.v = sv % p.V;
  w.split = sv / p.V;
  w.b = w.v % p.B;
  w.shard = w.v / p.B;
  int64_t L = p.seq_lens[w.v];
  if (L > p.r2t_stride) L = p.r2t_stride;
  if (L < 0) L = 0;
  w.L = L;
  const int64_t P = (L + kPage - 1) / kPage;
  int64_t p1;
  split_page_range(
      p.split_pages ? p.split_pages + (int64_t)w.v * (p.num_splits + 1) : nullptr,
      p.num_splits, w.split, P, w.p0, p1);
  w.npages = (int)(p1 - w.p0);
  // Tokens in [nmin, L) are visible to some query rows of the request and
  // masked for others; tokens at or past L to none.
  int64_t nmin = L - p.q_len + 1;
  if (p.kv_limit) {
    nmin = L;
    for (int i = 0; i < p.q_len; ++i) {
      const int64_t n = p.kv_limit[(int64_t)w.v * p.q_len + i];
      nmin = n < nmin ? n : nmin;
    }
  }
  w.nmin = nmin < 0 ? 0 : (nmin > L ? L : nmin);
}

// The page-table entry of page m of the unit's range as stored (0 past the
// range), and its check: the base slot, or -1 if it lies outside the pool.
// Split so that a load can be put in flight before its value is needed.
__device__ __forceinline__ int32_t page_entry(const Fp4Params& p, const UnitRange& w,
                                              int m) {
  if (m >= w.npages) return 0;
  return p.r2t[(int64_t)w.v * p.r2t_stride + (w.p0 + m) * kPage];
}
__device__ __forceinline__ int32_t checked_base(const Fp4Params& p, int32_t base) {
  if (base < 0 || (base & (kPage - 1)) || (int64_t)base + kPage > p.num_slots)
    return -1;
  return base;
}
// Bulk copy of `bytes` (a multiple of 16) from global memory into this CTA's
// shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// 16 codes (two words) and the f16 pair of their scale (both halves equal) ->
// two 16-byte chunks of operand.
__device__ __forceinline__ uint4 scaled8(uint32_t codes, uint32_t s2) {
  uint32_t h[4];
  e2m1x8_to_f16(codes, h);
  return make_uint4(h2mul(h[0], s2), h2mul(h[1], s2), h2mul(h[2], s2), h2mul(h[3], s2));
}
__device__ __forceinline__ uint4 plain8(uint32_t a, uint32_t b) {
  return make_uint4(e4m3x2_to_f16(a), e4m3x2_to_f16(a >> 16), e4m3x2_to_f16(b),
                    e4m3x2_to_f16(b >> 16));
}

// Block scales with every NaN (0x7F, 0xFF) replaced by 0.
__device__ __forceinline__ uint32_t finite_scales(uint32_t w) {
  uint32_t keep = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (((w >> (8 * k)) & 0x7Fu) != 0x7Fu) keep |= 0xFFu << (8 * k);
  return w & keep;
}

}  // namespace mla
