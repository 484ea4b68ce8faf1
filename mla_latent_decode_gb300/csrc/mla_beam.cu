// mla_beam.cu -- beam search's selection over all beams and the vocabulary
// (mla_beam_select).
//
//   score(w, t) = c[w] + x[w, t] - ln sum_u exp x[w, u]
//
// and the k largest over (w, t), equal ones by lowest (w, t).  Each logit is
// read once: a thread keeps its 64 bytes of a row in registers, takes their
// maximum and sum of exponentials, and hands on the few that may be among the
// row's k best.  One cluster of 8 CTAs serves a request, each CTA an eighth of
// the vocabulary of all beams; the rows' statistics and the CTAs' k best meet
// through distributed shared memory, so there is one launch, no workspace, and
// no result that depends on an order of arrival.
//
// Which logits of a tile may count: the k-th largest of the warps' largest
// thread maxima is a bound that at least k of the tile's values reach, and few
// more do (about k ln k for values in random order).  Where too many do (masked
// vocabularies, sorted ones) the bound is taken again from all 512 threads'
// maxima with their positions, which no more than k threads' values can reach.
// Exponents are fp32 differences to the thread's own maximum; sums are fp32 per
// thread, warp and CTA (8192 terms deep at 131072 logits, 2^-24 each) and meet
// in fp64, where the scores are formed and compared: two beams' tokens often
// differ by less than fp32 shows of their sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_internal.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kVecs = 4;                    // 16-byte vectors of a row per thread and tile
constexpr int kMaxK = MLA_BEAM_MAX_K, kMaxW = MLA_BEAM_MAX_W;
constexpr int kMaxBound = 5;                // thread maxima per warp in the bound: k / 16 + 1
constexpr int kCap = kMaxK * 32 + kMaxK;    // a tile's values behind the exact bound, and the row's so far
constexpr float kLog2e = 1.44269504088896340736f;

struct BeamParams {
  const void* logits;
  int64_t batch_stride, beam_stride;
  const float* scores;
  const uint8_t* finished;
  int W, V, k, end_token;
  float* out_scores;
  int32_t* parents;
  int32_t* tokens;
  int* status;
};

struct Smem {
  unsigned long long buf[kCap];             // candidates of the row at hand; later: positions
  unsigned long long list[kMaxW * kMaxK];   // each row's best in order; later: their scores
  unsigned long long top[kThreads];         // threads' best (exact bound)
  uint32_t bound[kWarps * kMaxBound];
  float2 warp_stat[kWarps];
  float2 stat[kCluster][kMaxW];             // (max, sum) of every CTA's part of a row
  double lse[kMaxW];
  int num[kMaxW];                           // candidates in a row's list
  double got_score[kCluster * kMaxK];       // in CTA 0: every CTA's best
  long long got_pos[kCluster * kMaxK];
  int got_num[kCluster];
  long long member[kMaxK];
  unsigned long long exact;
  int count[2];
};

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Type;
template <>
struct Type<float> {
  static constexpr int kPer = 4;
  static __device__ __forceinline__ float at(const uint4& v, int j) {
    return __uint_as_float(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w);
  }
  static constexpr uint32_t kNone = 0xff800000u;  // -inf
};
template <>
struct Type<__nv_bfloat16> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ float at(const uint4& v, int j) {
    const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
    return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
  }
  static constexpr uint32_t kNone = 0xff80ff80u;
};
template <>
struct Type<__half> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ float at(const uint4& v, int j) {
    const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return j & 1 ? __high2float(h) : __low2float(h);
  }
  static constexpr uint32_t kNone = 0xfc00fc00u;
};

// Positions [e, e + kPer) of a row, those outside [lo, hi) as -inf.
template <typename T>
__device__ __forceinline__ uint4 load(const T* row, int64_t e, int64_t lo, int64_t hi) {
  constexpr int kPer = Type<T>::kPer;
  if (e >= lo && e + kPer <= hi) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(row + e));
    return v;
  }
  uint32_t w[4] = {Type<T>::kNone, Type<T>::kNone, Type<T>::kNone, Type<T>::kNone};
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (e + j < lo || e + j >= hi) continue;
    if constexpr (sizeof(T) == 4) {
      w[j] = __float_as_uint(row[e + j]);
    } else {
      const uint32_t b = reinterpret_cast<const uint16_t*>(row)[e + j];
      w[j / 2] = j & 1 ? (w[j / 2] & 0xffffu) | b << 16 : (w[j / 2] & 0xffff0000u) | b;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The k best of n keys, in order, to `out`: each key's rank is the number of
// greater ones (keys differ).  All threads; no barrier inside.
__device__ __forceinline__ void best_keys(const unsigned long long* keys, int n, int k,
                                          unsigned long long* out) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long mine = keys[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > mine;
    if (rank < k) out[rank] = mine;
  }
}

// The k best of `lists` sorted lists (list l: num[l] entries at l * pitch) by
// score, equal ones by position; entry e goes to put(rank, e).  Its rank is its
// place in its own list and, by bisection, in every other.
template <typename Put>
__device__ __forceinline__ void merge_lists(const double* score, const long long* pos, const int* num,
                                            int lists, int pitch, int k, Put put) {
  for (int e = threadIdx.x; e < lists * pitch; e += kThreads) {
    const int l = e / pitch, j = e % pitch;
    if (j >= num[l]) continue;
    const double s = score[e];
    const long long at = pos[e];
    int rank = j;
    for (int m = 0; m < lists && rank < k; ++m) {
      if (m == l) continue;
      int lo = 0, hi = num[m];
      while (lo < hi) {
        const int mid = (lo + hi) / 2, f = m * pitch + mid;
        if (score[f] > s || (score[f] == s && pos[f] < at)) lo = mid + 1; else hi = mid;
      }
      rank += lo;
    }
    if (rank < k) put(rank, e);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) __cluster_dims__(kCluster, 1, 1)
    mla_beam_select_kernel(const BeamParams p) {
  constexpr int kPer = Type<T>::kPer, kElems = kVecs * kPer, kTile = kThreads * kElems;
  extern __shared__ __align__(16) uint8_t beam_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(beam_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const int64_t b = blockIdx.x / kCluster;
  const int W = p.W, V = p.V, k = p.k, r = k / 16 + 1;
  const int seg = ((V + kCluster - 1) / kCluster + 63) / 64 * 64;
  const int64_t lo = min((int64_t)V, (int64_t)seg * rank), hi = min((int64_t)V, lo + seg);
  if (tid < 2) sm.count[tid] = 0;
  __syncthreads();

  int turn = 0;  // rows read so far
  for (int w = 0; w < W; ++w) {
    const float c = p.scores[b * W + w];
    const bool done = p.finished && p.finished[b * W + w];
    if (done || !(fabsf(c) < INFINITY)) {  // the same in every thread: nothing of the row counts
      if (tid == 0) {
        sm.num[w] = 0;
        sm.stat[rank][w] = make_float2(-INFINITY, 0.f);
      }
      continue;
    }
    const T* row = static_cast<const T*>(p.logits) + b * p.batch_stride + w * p.beam_stride;
    const int shift = (int)(reinterpret_cast<uintptr_t>(row + lo) / sizeof(T) % kPer);
    int* count = &sm.count[turn & 1];
    int* next_count = &sm.count[++turn & 1];
    float m = -INFINITY, s = 0.f;  // the thread's maximum and sum
    uint32_t bound = 1;            // k values of the row reach it (1: no bound yet)
    int n = 0;
    for (int64_t t0 = lo - shift; t0 < hi; t0 += kTile) {
      uint4 v[kVecs];
#pragma unroll
      for (int u = 0; u < kVecs; ++u) v[u] = load<T>(row, t0 + (int64_t)(u * kThreads + tid) * kPer, lo, hi);
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
#pragma unroll
        for (int j = 0; j < kPer; ++j) mx = fmaxf(mx, Type<T>::at(v[u], j));
      // the bound's thread maxima: r per warp, in order
      const uint32_t mine = mx > -INFINITY ? ordered(mx) : 0;
      uint32_t left = mine;
      for (int j = 0; j < r; ++j) {
        const uint32_t best = __reduce_max_sync(~0u, left);
        const uint32_t who = __ballot_sync(~0u, left == best);
        if (lane == __ffs(who) - 1) left = 0;
        if (lane == 0) sm.bound[warp * r + j] = best;
      }
      if (tid == 0) *next_count = 0;
      // the sum, over differences to the thread's maximum
      if (mx > m) {
        s *= ex2((m - mx) * kLog2e);
        m = mx;
      }
      const float ref = m > -INFINITY ? m : 0.f;
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
#pragma unroll
        for (int j = 0; j < kPer; ++j) s += ex2((Type<T>::at(v[u], j) - ref) * kLog2e);
      __syncthreads();
      {
        uint32_t kth = 0;
        for (int i = lane; i < kWarps * r; i += 32) {
          const uint32_t x = sm.bound[i];
          int above = 0;
          for (int j = 0; j < kWarps * r; ++j) above += sm.bound[j] > x || (sm.bound[j] == x && j < i);
          if (above == k - 1) kth = x;
        }
        bound = max(bound, __reduce_max_sync(~0u, kth));
      }
      const auto key = [&](int u, int j, float x) {
        const int64_t at = t0 + (int64_t)(u * kThreads + tid) * kPer + j;
        return (unsigned long long)ordered(x) << 32 | (uint32_t)~(uint32_t)at;
      };
      if (mine >= bound) {
        const float limit = unordered(bound);
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const float x = Type<T>::at(v[u], j);
            if (bound > 1 ? x >= limit : x > -INFINITY) {
              const int at = atomicAdd(count, 1);
              if (at < kCap) sm.buf[at] = key(u, j, x);
            }
          }
      }
      __syncthreads();
      const int before = n;
      n = *count;
      if (n > kCap) {
        // Too many: the row's best so far stay, the tile's values come again
        // behind the exact bound, at most k threads' values.
        const int stay = min(before, k);
        __syncthreads();
        unsigned long long* mine_row = sm.list + w * k;
        best_keys(sm.buf, before, k, mine_row);
        unsigned long long top = 0;
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const float x = Type<T>::at(v[u], j);
            if (x > -INFINITY) top = max(top, key(u, j, x));
          }
        sm.top[tid] = top;
        if (tid == 0) sm.exact = 1;
        __syncthreads();
        if (tid < stay) sm.buf[tid] = mine_row[tid];
        if (top) {
          int above = 0;
          for (int j = 0; j < kThreads; ++j) above += sm.top[j] > top;
          if (above == k - 1) sm.exact = top;
        }
        if (tid == 0) *count = stay;
        __syncthreads();
        const unsigned long long exact = sm.exact;
        if (top >= exact) {
#pragma unroll
          for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              const float x = Type<T>::at(v[u], j);
              if (x > -INFINITY && key(u, j, x) >= exact) sm.buf[atomicAdd(count, 1)] = key(u, j, x);
            }
        }
        __syncthreads();
        n = *count;
      }
    }
    best_keys(sm.buf, n, k, sm.list + w * k);
    // the row's maximum and sum in this CTA
    const float wm = unordered(__reduce_max_sync(~0u, ordered(m)));
    s *= ex2((wm > -INFINITY ? m - wm : 0.f) * kLog2e);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    if (lane == 0) sm.warp_stat[warp] = make_float2(wm, s);
    __syncthreads();
    if (warp == 0) {
      const float2 x = lane < kWarps ? sm.warp_stat[lane] : make_float2(-INFINITY, 0.f);
      const float cm = unordered(__reduce_max_sync(~0u, ordered(x.x)));
      float sum = x.y * ex2((cm > -INFINITY ? x.x - cm : 0.f) * kLog2e);
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      if (lane == 0) {
        sm.stat[rank][w] = make_float2(cm, sum);
        sm.num[w] = min(n, k);
      }
    }
  }
  __syncthreads();
  // Every CTA gets every CTA's part of the rows' statistics.
  for (int i = tid; i < kCluster * W; i += kThreads) {
    const int to = i / W, w = i % W;
    if (to == (int)rank) continue;
    const float2 x = sm.stat[rank][w];
    const uint32_t at = mapa(smem_u32(&sm.stat[rank][w]), to);
    st_cluster_u32(at, __float_as_uint(x.x));
    st_cluster_u32(at + 4, __float_as_uint(x.y));
  }
  cluster_sync();
  if (tid < W) {
    float m = -INFINITY;
    for (int c = 0; c < kCluster; ++c) m = fmaxf(m, sm.stat[c][tid].x);
    double sum = 0;
    for (int c = 0; c < kCluster; ++c) {
      const float2 x = sm.stat[c][tid];
      sum += m > -INFINITY ? (double)x.y * exp((double)x.x - (double)m) : (double)x.y;
    }
    // an infinite or undefined logit: no continuation of this beam counts
    const double lse = (double)m + log(sum);
    const bool whole = sum > 0 && fabs(lse) < INFINITY;
    sm.lse[tid] = lse;
    if (!whole) sm.num[tid] = 0;
    if (rank == 0) {
      const float c = p.scores[b * W + tid];
      const bool done = p.finished && p.finished[b * W + tid];
      const bool odd = !(c < INFINITY) || (!done && (sum != sum || m == INFINITY));
      if (odd && p.status) atomicOr(p.status, MLA_STATUS_BAD_SCORE);
      if (done && fabsf(c) < INFINITY) sm.num[tid] = -1;  // its end, at its score
    }
  }
  __syncthreads();
  double* score = reinterpret_cast<double*>(sm.list);
  long long* pos = reinterpret_cast<long long*>(sm.buf);
  for (int e = tid; e < W * k; e += kThreads) {
    const int w = e / k, j = e % k;
    const double c = p.scores[b * W + w];
    if (j < sm.num[w]) {
      const unsigned long long key = sm.list[e];
      pos[e] = (long long)w * V + (uint32_t)~(uint32_t)key;
      score[e] = c + ((double)unordered((uint32_t)(key >> 32)) - sm.lse[w]);
    } else if (j == 0 && sm.num[w] < 0) {
      pos[e] = (long long)w * V + p.end_token;
      score[e] = c;
    }
  }
  __syncthreads();
  if (tid < W) sm.num[tid] = abs(sm.num[tid]);
  __syncthreads();
  const uint32_t to_score = mapa(smem_u32(sm.got_score + rank * k), 0);
  const uint32_t to_pos = mapa(smem_u32(sm.got_pos + rank * k), 0);
  merge_lists(score, pos, sm.num, W, k, k, [&](int at, int e) {
    const unsigned long long a = __double_as_longlong(score[e]), q = (unsigned long long)pos[e];
    st_cluster_u32(to_score + 8 * at, (uint32_t)a);
    st_cluster_u32(to_score + 8 * at + 4, (uint32_t)(a >> 32));
    st_cluster_u32(to_pos + 8 * at, (uint32_t)q);
    st_cluster_u32(to_pos + 8 * at + 4, (uint32_t)(q >> 32));
  });
  if (tid == 0) {
    int sum = 0;
    for (int w = 0; w < W; ++w) sum += sm.num[w];
    st_cluster_u32(mapa(smem_u32(sm.got_num + rank), 0), (uint32_t)min(sum, k));
  }
  cluster_sync();
  if (rank != 0) return;
  const auto put = [&](int at, float s, long long q) {
    p.out_scores[b * k + at] = s;
    p.parents[b * k + at] = (int)(b * W + q / V);
    p.tokens[b * k + at] = (int)(q % V);
  };
  int have = 0;
  for (int c = 0; c < kCluster; ++c) have += sm.got_num[c];
  have = min(have, k);
  merge_lists(sm.got_score, sm.got_pos, sm.got_num, kCluster, k, k, [&](int at, int e) {
    put(at, (float)sm.got_score[e], sm.got_pos[e]);
    sm.member[at] = sm.got_pos[e];
  });
  // Fewer than k continuations: the lowest positions that are none, at -inf.
  __syncthreads();
  if (tid < k - have) {
    long long q = tid;
    for (bool moved = true; moved;) {
      int below = 0;
      for (int j = 0; j < have; ++j) below += sm.member[j] <= q;
      moved = tid + below != q;
      q = tid + below;
    }
    put(have + tid, -INFINITY, q);
  }
}

template <typename T>
int launch_beam(const BeamParams& p, int B, cudaStream_t st) {
  const cudaError_t a = cudaFuncSetAttribute(mla_beam_select_kernel<T>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
  if (a != cudaSuccess) return cuda_fail(a, "cudaFuncSetAttribute(mla_beam_select_kernel)");
  mla_beam_select_kernel<T><<<(unsigned)(B * kCluster), kThreads, sizeof(Smem), st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_beam_select_kernel");
  return MLA_OK;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_beam_select(const void* logits, mla_logit_dtype dtype, int64_t batch_stride,
                               int64_t beam_stride, const float* scores, const uint8_t* finished,
                               int B, int W, int V, int end_token, int k, float* out_scores,
                               int32_t* parents, int32_t* tokens, int* status, mla_stream_t stream) {
  if (dtype != MLA_LOGIT_BF16 && dtype != MLA_LOGIT_F16 && dtype != MLA_LOGIT_F32)
    return fail(MLA_ERR_INVALID_ARG, "mla_beam_select: unknown dtype %d", (int)dtype);
  if (B < 0 || W < 1 || V < 1 || k < 1 || (int64_t)k > (int64_t)W * V)
    return fail(MLA_ERR_INVALID_ARG, "mla_beam_select: B=%d < 0, W=%d or V=%d < 1, or k=%d outside "
                "[1, W * V]", B, W, V, k);
  if (W > kMaxW || k > kMaxK)
    return fail(MLA_ERR_UNSUPPORTED, "mla_beam_select: W=%d > %d beams or k=%d > %d", W, kMaxW, k, kMaxK);
  if ((int64_t)B * W > 0x7fffffff || B > 0x7fffffff / kCluster)
    return fail(MLA_ERR_INVALID_ARG, "mla_beam_select: B=%d W=%d: too many rows", B, W);
  if (end_token < 0 || end_token >= V)
    return fail(MLA_ERR_INVALID_ARG, "mla_beam_select: end_token %d outside [0, %d)", end_token, V);
  if ((W > 1 && beam_stride < V) || (B > 1 && batch_stride < V))
    return fail(MLA_ERR_INVALID_ARG, "mla_beam_select: strides %lld, %lld below V=%d", (long long)batch_stride,
                (long long)beam_stride, V);
  if (B == 0) return MLA_OK;
  if (!logits || !scores || !out_scores || !parents || !tokens)
    return fail(MLA_ERR_INVALID_ARG, "mla_beam_select: a required pointer is NULL");
  const void* all[] = {scores, out_scores, parents, tokens, status};
  for (const void* q : all)
    if (q && !aligned(q, 4)) return fail(MLA_ERR_MISALIGNED, "mla_beam_select: arrays need 4-B alignment");
  if (!aligned(logits, dtype == MLA_LOGIT_F32 ? 4 : 2))
    return fail(MLA_ERR_MISALIGNED, "mla_beam_select: logits off their type's alignment");
  const BeamParams p{logits, batch_stride, beam_stride, scores, finished, W, V, k, end_token,
                     out_scores, parents, tokens, status};
  const cudaStream_t st = (cudaStream_t)stream;
  if (dtype == MLA_LOGIT_BF16) return launch_beam<__nv_bfloat16>(p, B, st);
  if (dtype == MLA_LOGIT_F16) return launch_beam<__half>(p, B, st);
  return launch_beam<float>(p, B, st);
}
