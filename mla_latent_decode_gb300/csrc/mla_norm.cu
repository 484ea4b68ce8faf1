// mla_norm.cu -- residual addition and RMS norm, with bf16 and / or E4M3
// output (mla_add_rms_norm in include/mla_decode.h).  Per row of d values:
//   h = x + residual               residual_out = bf16(h)
//   y = h * rsqrt(mean(h^2) + eps) * w
//   out = bf16(y);   out8 = E4M3(y / s), s = max|y| / 448 over the row or over
//   each group of `group` values
// in fp32 throughout, each output rounded once.
//
// A stream bound by HBM (2 + 2 bytes read and 2 + 1 written per value): a
// block per row, the row's h in registers between its one read and the
// writes.  A thread owns V vectors of 8 consecutive values, vector k at
// 8 * (k * threads + thread), so every warp access is contiguous and a group
// of 32, 64 or 128 values lies in 4, 8 or 16 neighbouring lanes: its maximum
// takes 2 to 4 shuffles.  The row's sum (and, with one scale per row, its
// maximum) crosses the warps through shared memory once.
#include <cuda_bf16.h>

#include <algorithm>

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
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Eight values from column c0 on; columns past d read as 0.
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int c0, int d,
                                      float (&v)[8]) {
  if (VEC) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + c0);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c0 + k < d ? __bfloat162float(row[c0 + k]) : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c0, int d,
                                       const float (&v)[8]) {
  if (VEC) {
    *reinterpret_cast<uint4*>(row + c0) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                   pack_bf16(v[6], v[7]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c0 + k < d) row[c0 + k] = __float2bfloat16_rn(v[k]);
  }
}

// VEC: d and every stride are multiples of 8 and every pointer is aligned to
// its vector, so whole vectors are in range or out of it.
template <int V, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) mla_norm_kernel(const NormParams p) {
  __shared__ float part[2][32];
  const int64_t r = blockIdx.x;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  float h[V][8];
  // The mean is summed, not the sum divided: a row overflows only where its
  // mean square does.
  const float inv_d = 1.0f / (float)p.d;
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c0 = 8 * (k * (int)blockDim.x + (int)threadIdx.x);
    if (c0 < p.d) {
      load8<VEC>(p.x + r * p.x_stride, c0, p.d, h[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = 0.f;
    }
  }
  if (p.res) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c0 = 8 * (k * (int)blockDim.x + (int)threadIdx.x);
      if (c0 < p.d) {
        float q[8];
        load8<VEC>(p.res + r * p.res_stride, c0, p.d, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[k][e] += q[e];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[k][e], h[k][e] * inv_d, ss);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
  if (lane == 0) part[0][warp] = ss;
  __syncthreads();
  // every row element has been read: the residual may be updated in place
  if (p.res_out) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c0 = 8 * (k * (int)blockDim.x + (int)threadIdx.x);
      if (c0 < p.d) store8<VEC>(p.res_out + r * p.res_out_stride, c0, p.d, h[k]);
    }
  }
  ss = lane < warps ? part[0][lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
  const float rs = 1.0f / sqrtf(ss + p.eps);
  float rowmax = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c0 = 8 * (k * (int)blockDim.x + (int)threadIdx.x);
    if (c0 < p.d) {
      float w[8];
      load8<VEC>(p.w, c0, p.d, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[k][e] = h[k][e] * rs * w[e];
        rowmax = fmaxf(rowmax, fabsf(h[k][e]));
      }
      if (p.out) store8<VEC>(p.out + r * p.out_stride, c0, p.d, h[k]);
    }
  }
  if (!p.out8) return;
  if (p.group == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      rowmax = fmaxf(rowmax, __shfl_xor_sync(kAll, rowmax, o));
    if (lane == 0) part[1][warp] = rowmax;
    __syncthreads();
    rowmax = lane < warps ? part[1][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      rowmax = fmaxf(rowmax, __shfl_xor_sync(kAll, rowmax, o));
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c0 = 8 * (k * (int)blockDim.x + (int)threadIdx.x);
    float amax = rowmax;
    if (p.group) {
      amax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(h[k][e]));
      for (int o = p.group / 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
    }
    if (c0 >= p.d) continue;
    const float s = __fdiv_rn(amax, 448.0f);
    if (p.group ? c0 % p.group == 0 : c0 == 0)
      p.scales[r * p.scales_stride + (p.group ? c0 / p.group : 0)] = s;
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      q[e] = s == 0.f ? 0u : e4m3_pair(__fdiv_rn(h[k][2 * e], s), __fdiv_rn(h[k][2 * e + 1], s));
    uint8_t* dst = p.out8 + r * p.out8_stride + c0;
    if (VEC) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c0 + e < p.d) dst[e] = (uint8_t)(q[e / 2] >> (8 * (e & 1)));
    }
  }
}

template <bool VEC>
void launch(const NormParams& p, int64_t n, int vec, int threads, cudaStream_t st) {
  const unsigned grid = (unsigned)n;
  if (vec == 1)
    mla_norm_kernel<1, VEC><<<grid, threads, 0, st>>>(p);
  else if (vec == 2)
    mla_norm_kernel<2, VEC><<<grid, threads, 0, st>>>(p);
  else
    mla_norm_kernel<4, VEC><<<grid, threads, 0, st>>>(p);
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
  if (!aligned(x, 2) || !aligned(weight, 2) || (residual && (!aligned(residual, 2) || !aligned(residual_out, 2))) ||
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
  const int vectors = (d + 7) / 8;
  const int vec = vectors <= kMaxThreads ? 1 : vectors <= 2 * kMaxThreads ? 2 : 4;
  const int threads =
      std::min(kMaxThreads, ((vectors + vec - 1) / vec + 31) / 32 * 32);
  if (vec8)
    launch<true>(p, n, vec, threads, (cudaStream_t)stream);
  else
    launch<false>(p, n, vec, threads, (cudaStream_t)stream);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_norm_kernel");
  return MLA_OK;
}
