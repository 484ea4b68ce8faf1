// mla_norm.cu -- residual addition and RMS norm, with bf16 and / or E4M3
// output (mla_add_rms_norm in include/mla_decode.h).  Per row of d values:
//   h = x + residual               residual_out = bf16(h)
//   y = h * rsqrt(mean(h^2) + eps) * w
//   out = bf16(y);   out8 = E4M3(y / s), s = max|y| / 448 over the row or over
//   each group of `group` values
// in fp32 throughout, each output rounded once.  y / s is y times the rounded
// reciprocal of s.
//
// A stream bound by HBM (2 + 2 bytes read and 2 + 1 written per value): a
// block per row, the row's h in registers between its one read and the
// writes.  A thread owns V vectors of 8 consecutive values, vector k at
// 8 * (k * threads + thread), so every warp access is contiguous and a group
// of 32, 64 or 128 values lies in 4, 8 or 16 neighbouring lanes: its maximum
// takes 2 to 4 shuffles.  The row's sum (and, with one scale per row, its
// maximum) crosses the warps through shared memory once.  Few rows take a
// thread per vector, the shortest chain; many rows of 257 to 512 vectors two a
// thread (6000 x 3584 29.2 us, with one 30.7; 16383 x 2560 51.0 and 53.1; 6000 x
// 4096 34.0 and 33.4), and of 513 to 1024 vectors four and four blocks per SM,
// whose phases overlap.  Measured on a GB300 at 16383 x 7168, groups of 128 (822
// MB): 153 us, 5.4 TB/s, 80% of the copy rate (three blocks 173, five 172, two
// vectors a thread 185, one 178; a resident grid that loads the next row ahead,
// two blocks of 125 registers, 249); 80 x 7168: 3.0 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "mla_fp4.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kMaxThreads = 1024;
constexpr int kMaxVec = 4;  // vectors of 8 values a thread may own

struct NormParams {
  const __nv_bfloat16* x;
  int64_t x_stride;
  const __nv_bfloat16* res;  // NULL: h = x
  int64_t res_stride;
  __nv_bfloat16* res_out;
  int64_t res_out_stride;
  const __nv_bfloat16* w;
  float eps;
  int d;
  __nv_bfloat16* out;  // NULL: not wanted
  int64_t out_stride;
  uint8_t* out8;  // NULL: not wanted
  int64_t out8_stride;
  float* scales;
  int64_t scales_stride;
  int group;  // 0: one scale per row
  int shift;  // kShift: values from a vector's boundary to row 0
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Pairs of fp32 values, two lanes per instruction: at 16 instructions a value
// the arithmetic, not HBM, bounded this kernel (70% of the issue slots at 16383
// x 7168).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ float2 both(uint64_t x) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(x));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t widen(uint32_t w) {  // two bf16
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t word(const uint4& u, int k) {
  return k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w;
}

// How a row's eight values lie: kAny element by element; kVec on whole vectors;
// kShift on whole vectors but for the row's two ends.
enum Lay { kAny, kVec, kShift };
template <int L>
__device__ __forceinline__ bool whole(int c0, int d) {
  return L == kVec || (L == kShift && c0 >= 0 && c0 + 8 <= d);
}

// Eight bf16 values from column c0 on as packed pairs; columns outside 0 .. d - 1
// read as 0.
template <int L>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* row, int c0, int d) {
  if (whole<L>(c0, d)) return *reinterpret_cast<const uint4*>(row + c0);
  const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = ((unsigned)(c0 + 2 * k) < (unsigned)d ? r[c0 + 2 * k] : 0u) |
           (((unsigned)(c0 + 2 * k + 1) < (unsigned)d ? r[c0 + 2 * k + 1] : 0u) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int L>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c0, int d,
                                       const uint64_t (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = pack_bf16(both(v[k]).x, both(v[k]).y);
  if (whole<L>(c0, d)) {
    *reinterpret_cast<uint4*>(row + c0) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint16_t* r = reinterpret_cast<uint16_t*>(row);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if ((unsigned)(c0 + k) < (unsigned)d) r[c0 + k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
  }
}

// Sum (MAX: maximum, as max_nan) of one value per thread over the block, in
// every thread.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* part) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  const auto reduce = [&](float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float b = __shfl_xor_sync(kAll, a, o);
      a = MAX ? max_nan(a, b) : a + b;
    }
    return a;
  };
  v = reduce(v);
  if (lane == 0) part[warp] = v;
  __syncthreads();
  return reduce(lane < warps ? part[lane] : 0.f);
}

// kVec: d and every stride are multiples of 8 and every pointer is aligned to
// its vector, so whole vectors are in range or out of it.  kShift (one scale per
// row): the arrays' rows are as far from a vector's boundary as each other's, up
// to seven values and changing from row to row, as with an odd d; the vectors
// start on the boundary before the row and the weight, which does not shift with
// it, is read by element (6000 x 7001: 72 us, every array by element 152).
//
// Blocks per SM asked for: four of 256 threads for four vectors (see above), and
// 32 registers for one vector a thread (6000 x 1536: 12.4 us, with 36 14.4).
template <int V, int L, int T>
__global__ void __launch_bounds__(T, T == 256 && V == 4 ? 4 : V == 1 && L == kVec ? 2 : 1)
    mla_norm_kernel(const NormParams p) {
  __shared__ float part[4][32];
  const int64_t r = blockIdx.x;
  const int shift = L == kShift ? (int)((p.shift + r * p.x_stride) & 7) : 0;
  const auto col = [&](int k) {
    return 8 * (k * (int)blockDim.x + (int)threadIdx.x) - shift;
  };
  uint4 x[V], q[V], w[V];  // all loads of the row in flight together
#pragma unroll
  for (int k = 0; k < V; ++k) {
    x[k] = q[k] = w[k] = make_uint4(0, 0, 0, 0);
    if (col(k) < p.d) {
      x[k] = load8<L>(p.x + r * p.x_stride, col(k), p.d);
      if (p.res) q[k] = load8<L>(p.res + r * p.res_stride, col(k), p.d);
      w[k] = load8<L == kVec ? kVec : kAny>(p.w, col(k), p.d);
    }
  }
  uint64_t h[V][4], acc = pair(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[k][e] = add2(widen(word(x[k], e)), widen(word(q[k], e)));
      acc = fma2(h[k][e], h[k][e], acc);
    }
  const float inv_d = 1.0f / (float)p.d;
  const float mean = block_reduce<false>(both(acc).x + both(acc).y, part[0]) * inv_d;
  // every row element has been read: the residual may be updated in place
  const auto store_residual = [&] {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (col(k) < p.d) store8<L>(p.res_out + r * p.res_out_stride, col(k), p.d, h[k]);
  };
  float ms = mean + p.eps;
  const bool far = squares_leave_range(mean, p.eps);  // the same in every thread
  if (far) {
    if (p.res_out) store_residual();  // h as it is; scaled from here on
    float top = 0.f, ss = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top = fmaxf(top, fmaxf(fabsf(both(h[k][e]).x), fabsf(both(h[k][e]).y)));
    const float f = unit_factor(block_reduce<true>(top, part[1]));
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[k][e] = mul2(h[k][e], pair(f, f));
        const float2 v = both(h[k][e]);
        ss = fmaf(v.y, v.y, fmaf(v.x, v.x, ss));
      }
    ms = block_reduce<false>(ss, part[2]) * inv_d + p.eps * f * f;
  }
  if (p.res_out && !far) store_residual();
  const float rs = 1.0f / sqrtf(ms);
  const uint64_t rs2 = pair(rs, rs);
  float amax[V], rowmax = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    amax[k] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[k][e] = mul2(h[k][e], mul2(rs2, widen(word(w[k], e))));
      amax[k] = max_nan(amax[k], max_nan(fabsf(both(h[k][e]).x), fabsf(both(h[k][e]).y)));
    }
    if (p.out && col(k) < p.d) store8<L>(p.out + r * p.out_stride, col(k), p.d, h[k]);
    rowmax = max_nan(rowmax, amax[k]);
  }
  if (!p.out8) return;
  if (p.group == 0) rowmax = block_reduce<true>(rowmax, part[3]);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (p.group == 0) {
      amax[k] = rowmax;
    } else {
      for (int o = p.group / 16; o > 0; o >>= 1)
        amax[k] = max_nan(amax[k], __shfl_xor_sync(kAll, amax[k], o));
    }
    const int c0 = col(k);
    if (c0 >= p.d) continue;
    const float s = __fdiv_rn(amax[k], 448.0f);
    if (p.group ? c0 % p.group == 0 : k == 0 && threadIdx.x == 0)
      p.scales[r * p.scales_stride + (p.group ? c0 / p.group : 0)] = s;
    uint32_t c8[4];
    if (s > 0x1p-90f) {
      const float inv = __frcp_rn(s);
      const uint64_t inv2 = pair(inv, inv);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = both(mul2(h[k][e], inv2));
        c8[e] = e4m3_pair(v.x, v.y);
      }
    } else {  // the reciprocal leaves the range, the group is zero or s is NaN
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = both(h[k][e]);
        c8[e] = s == 0.f ? 0u : e4m3_pair(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s));
      }
    }
    uint8_t* dst = p.out8 + r * p.out8_stride + c0;
    if (whole<L>(c0, p.d)) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(c8[0] | (c8[1] << 16), c8[2] | (c8[3] << 16));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((unsigned)(c0 + e) < (unsigned)p.d) dst[e] = (uint8_t)(c8[e / 2] >> (8 * (e & 1)));
    }
  }
}

template <int L>
void launch(const NormParams& p, int64_t n, int sms, cudaStream_t st) {
  const unsigned grid = (unsigned)n;
  const int vectors = (p.d + (L == kShift ? 7 : 0) + 7) / 8;
  const auto threads = [&](int v) { return ((vectors + v - 1) / v + 31) / 32 * 32; };
  if (n > 2 * sms && vectors > 512 && vectors <= 1024)
    mla_norm_kernel<4, L, 256><<<grid, threads(4), 0, st>>>(p);
  else if (n > 2 * sms && vectors > 256 && vectors <= 512)
    mla_norm_kernel<2, L, 256><<<grid, threads(2), 0, st>>>(p);
  else if (vectors <= 1024)
    mla_norm_kernel<1, L, 1024><<<grid, threads(1), 0, st>>>(p);
  else if (vectors <= 2048)
    mla_norm_kernel<2, L, 1024><<<grid, threads(2), 0, st>>>(p);
  else
    mla_norm_kernel<4, L, 1024><<<grid, threads(4), 0, st>>>(p);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_add_rms_norm(const void* x, int64_t x_stride, const void* residual,
                                int64_t residual_stride, void* residual_out,
                                int64_t residual_out_stride, const void* weight,
                                float eps, int64_t n, int d, void* out,
                                int64_t out_stride, void* out8, int64_t out8_stride,
                                float* scales, int64_t scales_stride, int group,
                                mla_stream_t stream) {
  if (n < 0 || d < 1)
    return fail(MLA_ERR_INVALID_ARG, "mla_add_rms_norm: n = %lld, d = %d", (long long)n, d);
  if (d > 8 * kMaxVec * kMaxThreads)
    return fail(MLA_ERR_UNSUPPORTED, "mla_add_rms_norm: d = %d above %d", d,
                8 * kMaxVec * kMaxThreads);
  if (group != 0 && group != 32 && group != 64 && group != 128)
    return fail(MLA_ERR_INVALID_ARG, "mla_add_rms_norm: group %d: 0, 32, 64 or 128", group);
  if (group && d % group)
    return fail(MLA_ERR_INVALID_ARG, "mla_add_rms_norm: d = %d not a multiple of group %d",
                d, group);
  if (!(eps >= 0.f) || eps > 1e30f)
    return fail(MLA_ERR_INVALID_ARG, "mla_add_rms_norm: eps %g not a finite number >= 0",
                (double)eps);
  if (n == 0) return MLA_OK;
  if (n > 0x7fffffff)
    return fail(MLA_ERR_INVALID_ARG, "mla_add_rms_norm: too many rows");
  if (!x || !weight || (!out && !out8))
    return fail(MLA_ERR_INVALID_ARG, "mla_add_rms_norm: x, weight and one output are required");
  if ((residual == nullptr) != (residual_out == nullptr))
    return fail(MLA_ERR_INVALID_ARG,
                "mla_add_rms_norm: residual and residual_out come together");
  if (out8 && !scales)
    return fail(MLA_ERR_INVALID_ARG, "mla_add_rms_norm: out8 needs scales");
  const int nscales = group ? d / group : 1;
  if (x_stride < d || (residual && (residual_stride < d || residual_out_stride < d)) ||
      (out && out_stride < d) || (out8 && (out8_stride < d || scales_stride < nscales)))
    return fail(MLA_ERR_INVALID_ARG, "mla_add_rms_norm: a row stride is shorter than its row");
  if (!aligned(x, 2) || !aligned(weight, 2) ||
      (residual && (!aligned(residual, 2) || !aligned(residual_out, 2))) ||
      (out && !aligned(out, 2)) || (out8 && !aligned(scales, 4)))
    return fail(MLA_ERR_MISALIGNED,
                "mla_add_rms_norm: bf16 arrays need 2-B alignment, scales 4-B");
  NormParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.x_stride = x_stride;
  p.res = static_cast<const __nv_bfloat16*>(residual);
  p.res_stride = residual_stride;
  p.res_out = static_cast<__nv_bfloat16*>(residual_out);
  p.res_out_stride = residual_out_stride;
  p.w = static_cast<const __nv_bfloat16*>(weight);
  p.eps = eps;
  p.d = d;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_stride = out_stride;
  p.out8 = static_cast<uint8_t*>(out8);
  p.out8_stride = out8_stride;
  p.scales = scales;
  p.scales_stride = scales_stride;
  p.group = group;
  // Whole vectors: every row of every array starts on its vector's boundary.
  const bool vec8 =
      d % 8 == 0 && x_stride % 8 == 0 && aligned(x, 16) && aligned(weight, 16) &&
      (!residual || (residual_stride % 8 == 0 && residual_out_stride % 8 == 0 &&
                     aligned(residual, 16) && aligned(residual_out, 16))) &&
      (!out || (out_stride % 8 == 0 && aligned(out, 16))) &&
      (!out8 || (out8_stride % 8 == 0 && aligned(out8, 8)));
  // Rows that are off that boundary by the same number of values in every array.
  const auto off = [](const void* a, int bytes) {
    return (int)((reinterpret_cast<uintptr_t>(a) / bytes) & 7);
  };
  const auto like_x = [&](const void* a, int64_t stride, int bytes) {
    return !a || (stride % 8 == x_stride % 8 && off(a, bytes) == off(x, 2));
  };
  const bool shifted = group == 0 && d + 7 <= 8 * kMaxVec * kMaxThreads &&
                       like_x(residual, residual_stride, 2) &&
                       like_x(residual_out, residual_out_stride, 2) &&
                       like_x(out, out_stride, 2) && like_x(out8, out8_stride, 1);
  p.shift = off(x, 2);
  static std::atomic<int> sms_of[64];  // asked of each device once
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64) sms = sms_of[dev].load();
  if (e == cudaSuccess && sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64) sms_of[dev].store(sms);
  }
  if (e != cudaSuccess) return cuda_fail(e, "mla_add_rms_norm: device query");
  if (vec8)
    launch<kVec>(p, n, sms, (cudaStream_t)stream);
  else if (shifted)
    launch<kShift>(p, n, sms, (cudaStream_t)stream);
  else
    launch<kAny>(p, n, sms, (cudaStream_t)stream);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_norm_kernel");
  return MLA_OK;
}
