// mla_append.cu -- appending new tokens to the paged latent pool and reading
// rows back (mla_kv_append, mla_kv_read in include/mla_decode.h).
//
// Append, per token: the latent's RMS norm, the rotation of its RoPE key (and
// of the queries' RoPE parts) by the token's position, and the write of the
// finished row in the pool's format:
//   c = x[:512] * rsqrt(mean(x[:512]^2) + eps) * w
//   (u, v) = (a cos - b sin, a sin + b cos) for each rotation pair (a, b)
// all in fp32 and rounded once, into the stored type.  Both halves of the
// work are streams bound by HBM and, at a decode step's few tokens, by the
// launch; one launch does both, its blocks split by role.  Measured from a CUDA
// graph on a GB300: 2.9 us for one token x 96 heads and for 80, 36.3 for 8191
// (215 MB, 5.9 TB/s, 88% of the copy rate), 7.0 for 16383 bf16 rows (38 MB).
//
// Row blocks: a warp per token.  Lane l holds c_kv elements 16 l .. 16 l + 15,
// one scale block of the 4-bit format, so the block's maximum, scale and codes
// need no exchange; the norm's sum (and E4M3's row maximum) are one warp
// reduction.  Lane l also holds rotation pair l of the 32.
// Query blocks: a thread takes 8 pairs of up to four heads of a token, their
// eight 16-byte loads in flight together, with the token's 16 cosines and sines
// in registers; its neighbours take the other pairs and heads, so a warp's
// accesses are contiguous.  For 8191 tokens x 96 heads, one head per thread and
// a block per token and 64 heads ran 49.3 us, this in blocks of 256 threads
// 39.7, in blocks of 128 36.6.
#include <cuda_bf16.h>

#include <algorithm>

#include "mla_fp4.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHeads = 4;  // query heads of one token a thread rotates
constexpr uint32_t kAll = 0xffffffffu;

struct AppendParams {
  const __nv_bfloat16* rows;
  int64_t row_stride;
  int64_t n;
  const __nv_bfloat16* weight;  // [512] or NULL (no norm)
  float eps;
  const int32_t* slots;
  const int32_t* positions;
  const float* cos_sin;  // [max_pos, 64]: 32 cosines, 32 sines
  int64_t max_pos;
  int interleaved;
  uint8_t* kv;
  float* kv_scale;  // E4M3: written, [num_slots]; FP4: read, [1]
  int64_t num_slots;
  const __nv_bfloat16* q;
  int64_t q_token_stride, q_head_stride;
  __nv_bfloat16* q_out;
  int64_t qo_token_stride, qo_head_stride;
  int H;
  int64_t row_blocks;    // blocks [0, row_blocks) write rows, the rest rotate
  int q_groups;          // ceil(H / kHeads) groups of four threads per token
  int* status;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) {
  return __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                    pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// One token's row.
template <int KIND>
__device__ __forceinline__ void append_row(const AppendParams& p, int64_t r, int lane) {
  const int32_t slot = p.slots[r], pos = p.positions[r];
  const uint4* src =
      reinterpret_cast<const uint4*>(p.rows + r * p.row_stride) + 2 * lane;
  const uint4 a = src[0], b = src[1];
  // the rotation pair of this lane: (2l, 2l + 1) or (l, l + 32)
  const __nv_bfloat16* rp = p.rows + r * p.row_stride + MLA_NOPE_DIM;
  const int i0 = p.interleaved ? 2 * lane : lane;
  const int i1 = p.interleaved ? 2 * lane + 1 : lane + 32;
  const float ra = __bfloat162float(rp[i0]), rb = __bfloat162float(rp[i1]);
  const bool bad_slot = slot < 0 || (int64_t)slot >= p.num_slots;
  const bool bad_pos = pos < 0 || (int64_t)pos >= p.max_pos;
  if (bad_slot || bad_pos) {  // warp-uniform: nothing of this row is written
    if (lane == 0 && p.status)
      atomicOr(p.status, (bad_slot ? MLA_STATUS_BAD_SLOT : 0) |
                             (bad_pos ? MLA_STATUS_BAD_POSITION : 0));
    return;
  }
  const float cs = p.cos_sin[(int64_t)pos * 64 + lane];
  const float sn = p.cos_sin[(int64_t)pos * 64 + 32 + lane];
  float c[2][8];
  unpack8(a, c[0]);
  unpack8(b, c[1]);
  if (p.weight) {
    const uint4* wp = reinterpret_cast<const uint4*>(p.weight) + 2 * lane;
    float w[2][8];
    unpack8(wp[0], w[0]);
    unpack8(wp[1], w[1]);
    float eps = p.eps;
    const auto mean_square = [&]() -> float {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) s = fmaf(c[k / 8][k % 8], c[k / 8][k % 8], s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
      return s * (1.0f / MLA_NOPE_DIM);
    };
    float mean = mean_square();
    if (squares_leave_range(mean, eps)) {  // warp-uniform
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(c[k / 8][k % 8]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      const float f = unit_factor(top);
#pragma unroll
      for (int k = 0; k < 16; ++k) c[k / 8][k % 8] *= f;
      eps = eps * f * f;
      mean = mean_square();
    }
    // rsqrtf (within 2 units in the last place), not 1 / sqrtf: it is also what a
    // reference in PyTorch calls, and where a row's factor is the same bits its
    // values near a code's border fall on the same side.
    const float rs = rsqrtf(mean + eps);
#pragma unroll
    for (int k = 0; k < 16; ++k) c[k / 8][k % 8] = c[k / 8][k % 8] * rs * w[k / 8][k % 8];
  }
  const float u = ra * cs - rb * sn, v = ra * sn + rb * cs;

  if (KIND == MLA_KV_BF16) {
    uint8_t* dst = p.kv + (int64_t)slot * (MLA_ROW_DIM * 2);
    reinterpret_cast<uint4*>(dst)[2 * lane] = pack8(c[0]);
    reinterpret_cast<uint4*>(dst)[2 * lane + 1] = pack8(c[1]);
    __nv_bfloat16* rd = reinterpret_cast<__nv_bfloat16*>(dst) + MLA_NOPE_DIM;
    if (p.interleaved) {
      reinterpret_cast<uint32_t*>(rd)[lane] = pack_bf16(u, v);
    } else {
      rd[i0] = __float2bfloat16_rn(u);
      rd[i1] = __float2bfloat16_rn(v);
    }
    return;
  }
  if (KIND == MLA_KV_FP8_E4M3) {
    // A NaN stays in its code; the scale, which the decode needs finite, is that
    // of the row's other values.
    float amax = fmaxf(fmaxf(0.f, fabsf(u)), fabsf(v));
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(c[k / 8][k % 8]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
    const float scale = __fdiv_rn(amax, 448.0f);
    const Divisor by(scale, amax);
    auto code = [&](float x, float y) -> uint32_t { return e4m3_pair(by(x), by(y)); };
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = code(c[k / 2][(4 * k) % 8], c[k / 2][(4 * k) % 8 + 1]) |
             (code(c[k / 2][(4 * k) % 8 + 2], c[k / 2][(4 * k) % 8 + 3]) << 16);
    uint8_t* dst = p.kv + (int64_t)slot * MLA_ROW_DIM;
    reinterpret_cast<uint4*>(dst)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
    const uint32_t r2 = code(u, v);
    if (p.interleaved) {
      reinterpret_cast<uint16_t*>(dst + MLA_NOPE_DIM)[lane] = (uint16_t)r2;
    } else {
      dst[MLA_NOPE_DIM + i0] = (uint8_t)r2;
      dst[MLA_NOPE_DIM + i1] = (uint8_t)(r2 >> 8);
    }
    if (lane == 0) p.kv_scale[slot] = scale;
    return;
  }
  // FP4: this lane's block of 16 and its scale, NaN if the block holds one (E2M1
  // has none); the pool's factor g is fixed.
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) amax = max_nan(amax, fabsf(c[k / 8][k % 8]));
  const float g = p.kv_scale[0];
  const float f = g > 0x1p+120f ? 0x1p-4f : 1.0f;  // 6 g stays in range
  const uint32_t s8 = e4m3_pair(__fdiv_rn(amax * f, 6.0f * (g * f)), 0.f) & 0xFFu;
  const float step = h2_to_f32(e4m3x2_to_f16(s8)).x * g;
  const Divisor by(step, amax);
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = by(c[k][e]);
    w[k] = e2m1x8(y);
  }
  uint8_t* dst = p.kv + (int64_t)slot * kFp4RowBytes;
  reinterpret_cast<uint2*>(dst)[lane] = make_uint2(w[0], w[1]);
  dst[kFp4ScaleOff + lane] = (uint8_t)s8;
  const uint32_t r2 = e4m3_pair(__fdiv_rn(u, g), __fdiv_rn(v, g));
  if (p.interleaved) {
    reinterpret_cast<uint16_t*>(dst + kFp4RopeOff)[lane] = (uint16_t)r2;
  } else {
    dst[kFp4RopeOff + i0] = (uint8_t)r2;
    dst[kFp4RopeOff + i1] = (uint8_t)(r2 >> 8);
  }
}

// Rotation of query rows: thread (token, group, j) takes pairs 8j .. 8j + 7,
// which are 16-byte chunks 2j, 2j + 1 (interleaved pairs) or j, j + 4 (half-
// split pairs), of heads group, group + q_groups, ...
__device__ __forceinline__ void rotate_queries(const AppendParams& p, int64_t item) {
  const int j = (int)(item & 3);
  item >>= 2;
  const int64_t t = item / p.q_groups;
  if (t >= p.n) return;
  const int h0 = (int)(item % p.q_groups);
  const int32_t pos = p.positions[t];
  const int k0 = p.interleaved ? 2 * j : j, k1 = p.interleaved ? 2 * j + 1 : j + 4;
  const __nv_bfloat16* src = p.q + t * p.q_token_stride;
  uint4 xa[kHeads], xb[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i * p.q_groups;
    if (h < p.H) {
      const uint4* row = reinterpret_cast<const uint4*>(src + h * p.q_head_stride);
      xa[i] = row[k0];
      xb[i] = row[k1];
    }
  }
  if (pos < 0 || (int64_t)pos >= p.max_pos) {
    if (h0 == 0 && j == 0 && p.status) atomicOr(p.status, MLA_STATUS_BAD_POSITION);
    return;
  }
  const float4* tab = reinterpret_cast<const float4*>(p.cos_sin + (int64_t)pos * 64);
  const float4 c0 = tab[2 * j], c1 = tab[2 * j + 1];
  const float4 s0 = tab[8 + 2 * j], s1 = tab[8 + 2 * j + 1];
  const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
  __nv_bfloat16* dst = p.q_out + t * p.qo_token_stride;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i * p.q_groups;
    if (h >= p.H) break;
    float x[8], y[8];
    unpack8(xa[i], x);
    unpack8(xb[i], y);
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = x[2 * e], b = x[2 * e + 1];
        x[2 * e] = a * cs[e] - b * sn[e];
        x[2 * e + 1] = a * sn[e] + b * cs[e];
        const float c = y[2 * e], d = y[2 * e + 1];
        y[2 * e] = c * cs[4 + e] - d * sn[4 + e];
        y[2 * e + 1] = c * sn[4 + e] + d * cs[4 + e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = x[e], b = y[e];
        x[e] = a * cs[e] - b * sn[e];
        y[e] = a * sn[e] + b * cs[e];
      }
    }
    uint4* row = reinterpret_cast<uint4*>(dst + h * p.qo_head_stride);
    row[k0] = pack8(x);
    row[k1] = pack8(y);
  }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads) mla_append_kernel(const AppendParams p) {
  if ((int64_t)blockIdx.x < p.row_blocks) {
    const int64_t r = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (r < p.n) append_row<KIND>(p, r, threadIdx.x % 32);
  } else {
    rotate_queries(p, ((int64_t)blockIdx.x - p.row_blocks) * kThreads + threadIdx.x);
  }
}

// A warp per row: the stored values, rounded once to bf16.  Bound by HBM, or by
// the launch: 1.3 us for one row, 4.3 for 8191 of the 4-bit rows (12 MB), 4.8
// for 16383 bf16 rows (38 MB, most of it in L2 behind the append).
template <int KIND>
__global__ void __launch_bounds__(kThreads)
    mla_read_kernel(const uint8_t* __restrict__ kv, const float* __restrict__ kv_scale,
                    int64_t num_slots, const int32_t* __restrict__ slots, int64_t n,
                    __nv_bfloat16* __restrict__ out, int64_t out_stride, int* status) {
  const int lane = threadIdx.x % 32;
  const int64_t r = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (r >= n) return;
  const int32_t slot = slots[r];
  uint4* dst = reinterpret_cast<uint4*>(out + r * out_stride);
  uint32_t* rdst = reinterpret_cast<uint32_t*>(out + r * out_stride + MLA_NOPE_DIM);
  if (slot < 0 || (int64_t)slot >= num_slots) {
    if (lane == 0 && status) atomicOr(status, MLA_STATUS_BAD_SLOT);
    dst[2 * lane] = dst[2 * lane + 1] = make_uint4(0, 0, 0, 0);
    rdst[lane] = 0;
    return;
  }
  if (KIND == MLA_KV_BF16) {
    const uint4* src =
        reinterpret_cast<const uint4*>(kv + (int64_t)slot * (MLA_ROW_DIM * 2));
    const uint4 a = src[lane], b = src[lane + 32];
    const uint32_t c = reinterpret_cast<const uint32_t*>(src)[MLA_NOPE_DIM / 2 + lane];
    dst[lane] = a;
    dst[lane + 32] = b;
    rdst[lane] = c;
    return;
  }
  uint32_t h[8], rope;  // f16 pairs of this lane's 16 elements, of its RoPE pair
  float f, fr;
  if (KIND == MLA_KV_FP8_E4M3) {
    const uint8_t* src = kv + (int64_t)slot * MLA_ROW_DIM;
    const uint4 a = reinterpret_cast<const uint4*>(src)[lane];
    rope = reinterpret_cast<const uint16_t*>(src + MLA_NOPE_DIM)[lane];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = e4m3x2_to_f16(w[k / 2] >> (16 * (k & 1)));
    f = fr = kv_scale[slot];
  } else {
    const uint8_t* src = kv + (int64_t)slot * kFp4RowBytes;
    const uint2 a = reinterpret_cast<const uint2*>(src)[lane];
    const uint32_t s8 = src[kFp4ScaleOff + lane];
    rope = reinterpret_cast<const uint16_t*>(src + kFp4RopeOff)[lane];
    uint32_t lo[4], hi[4];
    e2m1x8_to_f16(a.x, lo);
    e2m1x8_to_f16(a.y, hi);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = lo[k], h[4 + k] = hi[k];
    fr = kv_scale[0];
    f = h2_to_f32(e4m3x2_to_f16(s8)).x * fr;
  }
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 v = h2_to_f32(h[k]);
    o[k] = pack_bf16(v.x * f, v.y * f);
  }
  dst[2 * lane] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[2 * lane + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  const float2 v = h2_to_f32(e4m3x2_to_f16(rope));
  rdst[lane] = pack_bf16(v.x * fr, v.y * fr);
}

int check_pool(const void* kv, mla_kv_dtype kv_dtype, const float* kv_scale,
               int64_t num_slots, const char* name) {
  if (!kv) return fail(MLA_ERR_INVALID_ARG, "%s: kv_pages is required", name);
  if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3 &&
      kv_dtype != MLA_KV_FP4_E2M1)
    return fail(MLA_ERR_INVALID_ARG, "%s: unknown kv_dtype %d", name, (int)kv_dtype);
  if (kv_dtype != MLA_KV_BF16 && !kv_scale)
    return fail(MLA_ERR_INVALID_ARG, "%s: FP8 and FP4 KV need kv_scale", name);
  if (num_slots < 1 || num_slots > ((int64_t)1 << 31) - 1)
    return fail(MLA_ERR_INVALID_ARG, "%s: num_slots %lld out of range", name,
                (long long)num_slots);
  if (!aligned(kv, 16) || (kv_scale && !aligned(kv_scale, 4)))
    return fail(MLA_ERR_MISALIGNED, "%s: kv_pages needs 16-B alignment, kv_scale 4-B",
                name);
  return MLA_OK;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_kv_append(const void* rows, int64_t row_stride, int64_t n,
                             const void* norm_weight, float eps, const int32_t* slots,
                             const int32_t* positions, const float* cos_sin,
                             int64_t max_pos, int interleaved, void* kv_pages,
                             mla_kv_dtype kv_dtype, float* kv_scale,
                             int64_t num_slots, const void* q, int64_t q_token_stride,
                             int64_t q_head_stride, void* q_out,
                             int64_t qo_token_stride, int64_t qo_head_stride, int H,
                             int* status, mla_stream_t stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "mla_kv_append: n = %lld < 0", (long long)n);
  const int rc = check_pool(kv_pages, kv_dtype, kv_scale, num_slots, "mla_kv_append");
  if (rc != MLA_OK) return rc;
  if (H < 0) return fail(MLA_ERR_INVALID_ARG, "mla_kv_append: H = %d < 0", H);
  if (n == 0) return MLA_OK;  // whose arrays may all be NULL
  if (H > 0 && (!q || !q_out))
    return fail(MLA_ERR_INVALID_ARG, "mla_kv_append: H = %d needs q and q_out", H);
  if (!rows || !slots || !positions || !cos_sin)
    return fail(MLA_ERR_INVALID_ARG,
                "mla_kv_append: rows, slots, positions and cos_sin are required");
  if (max_pos < 1 || row_stride < MLA_ROW_DIM || !(eps >= 0.f) || eps > 1e30f)
    return fail(MLA_ERR_INVALID_ARG, "mla_kv_append: max_pos %lld < 1, row_stride %lld "
                "< 576 or eps %g not a finite number >= 0", (long long)max_pos,
                (long long)row_stride, (double)eps);
  if (H > 0 && ((H > 1 && (q_head_stride < MLA_ROPE_DIM || qo_head_stride < MLA_ROPE_DIM)) ||
                (n > 1 && (q_token_stride < MLA_ROPE_DIM || qo_token_stride < MLA_ROPE_DIM))))
    return fail(MLA_ERR_INVALID_ARG, "mla_kv_append: query strides below 64 elements");
  if (!aligned(rows, 16) || row_stride % 8 || (norm_weight && !aligned(norm_weight, 16)) ||
      !aligned(slots, 4) || !aligned(positions, 4) || !aligned(cos_sin, 16) ||
      (status && !aligned(status, 4)) ||
      (H > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || q_token_stride % 8 ||
                 q_head_stride % 8 || qo_token_stride % 8 || qo_head_stride % 8)))
    return fail(MLA_ERR_MISALIGNED, "mla_kv_append: rows, weights, queries and cos_sin need "
                "16-B alignment (strides a multiple of 8 elements), the other arrays 4-B");
  AppendParams p;
  p.rows = static_cast<const __nv_bfloat16*>(rows);
  p.row_stride = row_stride;
  p.n = n;
  p.weight = static_cast<const __nv_bfloat16*>(norm_weight);
  p.eps = eps;
  p.slots = slots;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_pos = max_pos;
  p.interleaved = interleaved != 0;
  p.kv = static_cast<uint8_t*>(kv_pages);
  p.kv_scale = kv_scale;
  p.num_slots = num_slots;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.qo_token_stride = qo_token_stride;
  p.qo_head_stride = qo_head_stride;
  p.H = H;
  p.status = status;
  p.row_blocks = (n + kWarps - 1) / kWarps;
  p.q_groups = std::max((H + kHeads - 1) / kHeads, 1);
  const int64_t q_blocks = H > 0 ? (n * p.q_groups * 4 + kThreads - 1) / kThreads : 0;
  if (n > 0x7fffffff || p.row_blocks + q_blocks > 0x7fffffff)
    return fail(MLA_ERR_INVALID_ARG, "mla_kv_append: too many rows");
  const unsigned grid = (unsigned)(p.row_blocks + q_blocks);
  const cudaStream_t st = (cudaStream_t)stream;
  if (kv_dtype == MLA_KV_BF16)
    mla_append_kernel<MLA_KV_BF16><<<grid, kThreads, 0, st>>>(p);
  else if (kv_dtype == MLA_KV_FP8_E4M3)
    mla_append_kernel<MLA_KV_FP8_E4M3><<<grid, kThreads, 0, st>>>(p);
  else
    mla_append_kernel<MLA_KV_FP4_E2M1><<<grid, kThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_append_kernel");
  return MLA_OK;
}

extern "C" int mla_kv_read(const void* kv_pages, mla_kv_dtype kv_dtype,
                           const float* kv_scale, int64_t num_slots,
                           const int32_t* slots, int64_t n, void* out,
                           int64_t out_stride, int* status, mla_stream_t stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "mla_kv_read: n = %lld < 0", (long long)n);
  const int rc = check_pool(kv_pages, kv_dtype, kv_scale, num_slots, "mla_kv_read");
  if (rc != MLA_OK) return rc;
  if (n == 0) return MLA_OK;
  if (!slots || !out)
    return fail(MLA_ERR_INVALID_ARG, "mla_kv_read: slots and out are required");
  if (out_stride < MLA_ROW_DIM)
    return fail(MLA_ERR_INVALID_ARG, "mla_kv_read: out_stride %lld < 576",
                (long long)out_stride);
  if (!aligned(slots, 4) || !aligned(out, 16) || out_stride % 8 ||
      (status && !aligned(status, 4)))
    return fail(MLA_ERR_MISALIGNED, "mla_kv_read: out needs 16-B alignment (stride a "
                "multiple of 8 elements), the other arrays 4-B");
  const int64_t blocks = (n + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return fail(MLA_ERR_INVALID_ARG, "mla_kv_read: too many rows");
  const cudaStream_t st = (cudaStream_t)stream;
  const uint8_t* kv = static_cast<const uint8_t*>(kv_pages);
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out);
  if (kv_dtype == MLA_KV_BF16)
    mla_read_kernel<MLA_KV_BF16><<<(unsigned)blocks, kThreads, 0, st>>>(
        kv, kv_scale, num_slots, slots, n, dst, out_stride, status);
  else if (kv_dtype == MLA_KV_FP8_E4M3)
    mla_read_kernel<MLA_KV_FP8_E4M3><<<(unsigned)blocks, kThreads, 0, st>>>(
        kv, kv_scale, num_slots, slots, n, dst, out_stride, status);
  else
    mla_read_kernel<MLA_KV_FP4_E2M1><<<(unsigned)blocks, kThreads, 0, st>>>(
        kv, kv_scale, num_slots, slots, n, dst, out_stride, status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_read_kernel");
  return MLA_OK;
}
