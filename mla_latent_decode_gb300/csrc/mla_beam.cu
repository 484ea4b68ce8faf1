// mla_beam.cu -- beam search's selection over all beams and the vocabulary
// (mla_beam_select).
//
//   score(w, t) = c[w] + x[w, t] - ln sum_u exp x[w, u]
//
// and the k largest over (w, t), equal ones by lowest (w, t).  Bound by the logits'
// bytes: each is read once, 64 bytes a lane and tile, the next tile's loads under
// way.  A warp has a part of a row to itself and meets no barrier before its end: it
// keeps the part's maximum and sum of exponentials and its k best, the CTAs of a
// cluster (one request) exchange the rows' statistics and their k best through
// distributed shared memory.  One launch, no workspace, and no result that depends on
// an order of arrival.
//
// Which logits of a tile may count: the k-th largest of the 64 or 128 values that a
// warp's lanes have met as the largest of every second or fourth vector is a bound
// that at least k values of the part reach, and few more do (about k ln k for values
// in random order).  While tiles pass only each lane's largest value of each is kept;
// after 32 of them, or at the part's end, the bound is found and the few lanes' tiles
// that reach it are read again (for k = 16 about 20 times 128 bytes of 128 KB), four
// of them at a time, a vector a lane.  Where
// too many reach it (ties) the best k so far are selected exactly, and later values
// have to exceed the last of them.
//
// Measured: 64 requests x 16 beams x 131072 bf16 logits, a tenth finished (241 MB) 56 us,
// 64% of the copy rate: the 256 CTAs are two on 104 SMs and one on 48, and a tile's
// arithmetic (3.6 instructions a logit) takes as long as its bytes.  Candidates looked
// for tile by tile took 65 us, tiles in registers 165, a CTA a row with its barriers 215.
//
// Exponents are fp32 differences to the lane's own maximum; sums are fp32 over a
// tile (64 terms), compensated over tiles, and meet as pairs of fp32; the scores are
// formed in fp64: two beams' tokens often differ by less than fp32 shows of their sums.
// Scores are compared as ordered integers (fp64 runs at 2 a cycle and SM).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "mla_internal.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;               // (16 of them start later: 16 x 5 x 100003 took 33 us, not 22)
constexpr int kVecs = 8;                    // 16-byte vectors of a row per lane and tile
constexpr int kTops = 4;                    // values a lane gives to the bound: its largest of every fourth vector
constexpr int kStages = 2;                  // tiles of a warp in shared memory
constexpr int kMaxK = MLA_BEAM_MAX_K, kMaxW = MLA_BEAM_MAX_W;
constexpr int kMaxLists = 16;               // parts of rows in a CTA: two for a warp
constexpr int kMaxParts = 512;              // in a cluster
constexpr int kEpoch = 32;                  // tiles whose values are looked for at once
constexpr int kCap = kMaxK + 126;           // candidates of a warp: its best so far, room for a lane's tile
constexpr float kLog2e = 1.44269504088896340736f;
constexpr uint32_t kLeast = 0x00800000u;    // the least finite value's place in the order
typedef unsigned long long u64;

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
  int cluster, parts;  // CTAs of a request, parts of a row
};

// Two CTAs an SM.
struct Smem {
  union {
    uint4 tile[kWarps][kStages][kVecs][32];
    struct {                                // once every CTA has read its logits
      long long pos[kMaxLists * kMaxK];     // w * 2^32 + t of the lists' entries
      u64 got_score[kMaxCluster * kMaxK];   // in CTA 0: every CTA's best
      long long got_pos[kMaxCluster * kMaxK];
    };
  };
  u64 buf[kWarps][kCap + 2];                // candidates of the warps' parts at hand
  uint32_t words[kWarps][64];
  uint16_t tops[kWarps][kEpoch * 32];       // lanes' largest values of the tiles, cut to 16 bits; later: pairs
  u64 list[kMaxLists * kMaxK];              // the parts' best in order; later: their scores
  float2 stat[kMaxParts];                   // (max, sum) of the cluster's parts
  double lse[kMaxW];
  float2 row[kMaxW];                        // (max, sum) of the beams' rows
  int like[kMaxW];                          // the first row with the same values
  int differ[kMaxW];                        // the last round in which a row differed from the one it was compared with
  int num[kMaxLists];                       // entries of a list
  int ends[kMaxW];                          // a finished beam's end counts
  int got_num[kMaxCluster];
  float score[kMaxW], live[kMaxW];          // the beams'; with finished ones at -inf
  long long member[kMaxK];
  uint16_t order[kMaxK];
};
static_assert(sizeof(Smem) <= 113 * 1024, "shared memory of two CTAs an SM");

extern __shared__ __align__(16) uint8_t beam_smem[];
__device__ __forceinline__ Smem& shared() { return *reinterpret_cast<Smem*>(beam_smem); }

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

__device__ __forceinline__ u64 ordered(double x) {
  const u64 u = (u64)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double unordered(u64 u) {
  return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}
__device__ __forceinline__ u64 f2(float a, float b) {
  u64 x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ void f2(u64 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Pairs (hi, lo) of fp32, hi + lo exact to about 2^-45 of it: fp64 arithmetic runs at
// 2 a cycle and SM, and these few sums would take longer than the logits.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two plus(Two a, Two b) {
  const float s = a.hi + b.hi, t = s - a.hi, e = (a.hi - (s - t)) + (b.hi - t) + a.lo + b.lo;
  const float hi = s + e;
  return {hi, s < INFINITY ? e - (hi - s) : 0.f};
}
// e^x for x <= 0 within 2^-24.8 of it (0 from -80 down): 2^n (1 + r + r^2 (1/2 + r/6 + ...)),
// r = x - n ln 2, |r| <= ln 2 / 2, with ln 2 as 355/512 - 2.12194440e-4 (W. J. Cody and W.
// Waite, Software Manual for the Elementary Functions, 1980): n has 7 bits and 355 nine, so
// the first difference is exact.  r is off by 1.07 x 2^-26 (its rounding, and n times that of
// the second part), r^2 (...) by its terms' roundings, 0.8 x 2^-26, the rest of the series
// 2^-32, all of e^r >= 0.707.
__device__ __forceinline__ Two exp_two(float x) {
  if (!(x > -80.f)) return {x == x ? 0.f : x, 0.f};  // (2^-115 of a sum's largest term)
  const float n = rintf(x * kLog2e);
  float r = fmaf(n, -355.f / 512, x);
  r = fmaf(n, 2.12194440e-4f, r);
  float q = 1.f / 40320;
  q = fmaf(q, r, 1.f / 5040);
  q = fmaf(q, r, 1.f / 720);
  q = fmaf(q, r, 1.f / 120);
  q = fmaf(q, r, 1.f / 24);
  q = fmaf(q, r, 1.f / 6);
  q = fmaf(q, r, 0.5f);
  q = q * r * r;
  const float a = 1.f + r, low = (r - (a - 1.f)) + q, scale = __int_as_float((127 + (int)n) << 23);
  const float hi = a + low;
  return {hi * scale, (low - (hi - a)) * scale};
}
// y e^x
__device__ __forceinline__ Two times_exp(float y, float x) {
  const Two e = exp_two(x);
  const float hi = y * e.hi;
  return {hi, fmaf(y, e.hi, -hi) + y * e.lo};
}
// ln of x, 1 <= x <= e^79 (a sum of 2^31 terms at most, the largest 1), within 2^-24.7:
// fp32's l, and a Newton step, l + (x e^-l - 1), which errs as e^-l does.  Both are checked
// against float64 by mla_debug_beam_math (over 2^24 values 1.53 x 2^-26 at most).
__device__ __forceinline__ double log_of(Two x) {
  const float l = logf(x.hi);
  const Two e = exp_two(-l);
  return (double)l + (double)(fmaf(x.hi, e.hi, -1.f) + (x.hi * e.lo + x.lo * e.hi));
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
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ float top(uint32_t a) { return __uint_as_float(a); }
};
template <>
struct Type<__nv_bfloat16> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ float at(const uint4& v, int j) {
    const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
    return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
  }
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  static __device__ __forceinline__ float top(uint32_t a) {
    return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
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
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  static __device__ __forceinline__ float top(uint32_t a) {
    const __half2 h = *reinterpret_cast<const __half2*>(&a);
    return fmaxf(__low2float(h), __high2float(h));
  }
};

// Positions [e, e + kPer) of a row, those outside [lo, hi) as -inf.
template <typename T>
__device__ __noinline__ uint4 load_edge(const T* row, int64_t e, int64_t lo, int64_t hi) {
  constexpr int kPer = Type<T>::kPer;
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

// The k best of a warp's n candidates, in order, to list l, of those with values
// from `limit` on (at least k, or all): they are moved to the front first, then a
// key's rank is the number of greater ones (keys differ).  Returns their number, k at
// most.
__device__ __noinline__ int best_keys(int l, int n, int k, uint32_t limit) {
  Smem& sm = shared();
  const int lane = threadIdx.x & 31;
  u64 *keys = sm.buf[threadIdx.x >> 5], *out = sm.list + l * k;
  __syncwarp();
  int m = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 32) {
    const u64 mine = i0 + lane < n ? keys[i0 + lane] : 0;
    const bool stays = (uint32_t)(mine >> 32) >= limit;
    const uint32_t all = __ballot_sync(~0u, stays);
    if (stays) keys[m + __popc(all & ((1u << lane) - 1))] = mine;
    m += __popc(all);
  }
  if (lane == 0) keys[m] = 0;  // (the buffer has room)
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i < m; i += 64) {  // two a lane at once
    const u64 one = keys[i], two = i + 32 < m ? keys[i + 32] : 0;
    int above = 0, over = 0;
#pragma unroll 4
    for (int j = 0; j < m; j += 2) {
      const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(keys + j);
      above += (x.x > one) + (x.y > one);
      over += (x.x > two) + (x.y > two);
    }
    if (above < k) out[above] = one;
    if (i + 32 < m && over < k) out[over] = two;
  }
  __syncwarp();
  return min(m, k);
}

// Keeps the k best of a warp's n candidates; all later ones have to reach the last
// of them.  Returns their number.
__device__ __noinline__ int select(int l, int n, int k, uint32_t* floor) {
  Smem& sm = shared();
  n = best_keys(l, n, k, *floor);
  for (int i = threadIdx.x & 31; i < n; i += 32) sm.buf[threadIdx.x >> 5][i] = sm.list[l * k + i];
  if (n == k) *floor = max(*floor, (uint32_t)(sm.list[l * k + k - 1] >> 32));
  __syncwarp();
  return n;
}

// The place in the order of the k-th largest of the lanes' kTops values: each is
// compared with all of them, through shared memory.
template <int kTops>
__device__ __forceinline__ uint32_t kth_by_all(const float (&x)[kTops], int k, uint32_t* words) {
  const int lane = threadIdx.x & 31;
  uint32_t mine[kTops];
  int above[kTops];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kTops; ++i) {
    mine[i] = ordered(x[i]);
    above[i] = 0;
    words[32 * i + lane] = mine[i];
  }
  __syncwarp();
#pragma unroll 4
  for (int j = 0; j < 8 * kTops; ++j) {
    const uint4 y = *reinterpret_cast<const uint4*>(words + 4 * j);
#pragma unroll
    for (int i = 0; i < kTops; ++i) above[i] += (y.x > mine[i]) + (y.y > mine[i]) + (y.z > mine[i]) + (y.w > mine[i]);
  }
  // the least value that fewer than k exceed
  uint32_t least = ~0u;
#pragma unroll
  for (int i = 0; i < kTops; ++i) least = min(least, above[i] < k ? mine[i] : ~0u);
  return __reduce_min_sync(~0u, least);
}

// A place in the order that at least k of the lanes' kTops values reach, and no more
// where that many can be told apart (kLeast if fewer are finite): by bisection, ten
// steps of 60 cycles and more (32 where values tie; comparing all 128 takes 4000, all
// 64 1100).
template <int kTops>
__device__ __forceinline__ uint32_t kth_of(const float (&x)[kTops], int k) {
  uint32_t mine[kTops], least = ~0u, most = 0;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kTops; ++i) {
    mine[i] = ordered(x[i]);
    if (mine[i] >= kLeast) least = min(least, mine[i]);
    most = max(most, mine[i]);
    n += __popc(__ballot_sync(~0u, mine[i] >= kLeast));
  }
  if (n < k) return kLeast;
  uint32_t lo = __reduce_min_sync(~0u, least), hi = __reduce_max_sync(~0u, most) + 1;  // hi: none reaches it
#pragma unroll 1
  while (hi - lo > 1 && n != k) {
    const uint32_t mid = lo + (hi - lo) / 2;
    n = 0;
#pragma unroll
    for (int i = 0; i < kTops; ++i) n += __popc(__ballot_sync(~0u, mine[i] >= mid));
    if (n >= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A warp's way through its parts of rows, tile by tile; parts of which nothing
// counts (finished or dead beams) are left out.  Part g is row g / p.parts's; the
// cluster's warps take turns with them.
template <typename T>
struct Walk {
  const T* row;
  int64_t t0, lo, hi;  // the tile's first position, the part
  int g;               // the part; none left: p.W * p.parts
  static constexpr int kTile = 32 * kVecs * Type<T>::kPer;
  __device__ __forceinline__ void enter(const BeamParams& p, const float* score, int64_t b, int64_t len, int from) {
    const int all = p.W * p.parts, step = p.cluster * kWarps;
#pragma unroll 1
    for (g = from; g < all; g += step) {
      const int w = (uint32_t)g / (uint32_t)p.parts;
      row = static_cast<const T*>(p.logits) + b * p.batch_stride + w * p.beam_stride;
      // cut where 16-byte vectors start: only a row's ends have partial ones
      const int shift = (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T) % Type<T>::kPer);
      lo = min((int64_t)p.V, len * (g - w * p.parts));
      hi = min((int64_t)p.V, lo + len);
      if (lo > 0 && lo < p.V) lo -= shift;
      if (hi < p.V) hi -= shift;
      if (!(fabsf(score[w]) < INFINITY) || lo >= hi) continue;
      t0 = lo > 0 ? lo : -shift;
      return;
    }
    g = all;
  }
  __device__ __forceinline__ bool last() const { return t0 + kTile >= hi; }
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

struct Entry {
  u64 score, pos;
  __device__ __forceinline__ bool before(const Entry& o) const {
    return score > o.score || (score == o.score && pos < o.pos);
  }
};

// The k best of sorted lists (list l: num[l] entries at l * k) by score, equal ones by
// position: the i-th of them is entry order[i].  Returns their number.
//
// Few: one after the other by a warp whose lanes hold the lists' heads and the entries
// behind them, about 200 cycles each.  From kTree on: two lists' into the first of
// them, until all are in list 0; k (a power of two from it on) by the greater of one
// list's entries and the other's from its end, which rise and fall, and a warp sorts
// them by halves.  1 x 4 x 32000, k = 8: 11.0 us by heads, 11.5 by pairs; 16 x 5 x
// 100003, k = 10: 20.9 and 21.8; 2 x 7 x 2208, k = 14: 13.8 and 12.9; 23 x 7 x 52472,
// k = 62: 43 and 36 (and 92 with every entry compared with all others).
// A list's own order is that of its row's logits, which stands where two scores agree
// in fp64.
constexpr int kTree = 12;
__device__ __noinline__ int merge_lists(u64* score, long long* pos, int* num, int lists, int k, uint16_t* order) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (k < kTree) {
    static_assert(kMaxLists <= 32 && kMaxCluster <= 32, "a list a lane");
    const int sum = min(__reduce_add_sync(~0u, lane < lists ? num[lane] : 0), k);
    if (warp == 0) {
      int e = lane < lists ? lane * k : 0;
      const int end = lane < lists ? e + num[lane] : 0;
      u64 head = e < end ? score[e] : 0, next = e + 1 < end ? score[e + 1] : 0;  // 0: below every score
#pragma unroll 1
      for (int i = 0; i < sum; ++i) {
        const uint32_t high = __reduce_max_sync(~0u, (uint32_t)(head >> 32));
        bool best = (uint32_t)(head >> 32) == high;
        uint32_t all = __ballot_sync(~0u, best);
        if (all & (all - 1)) {
          const uint32_t low = __reduce_max_sync(~0u, best ? (uint32_t)head : 0);
          best = best && (uint32_t)head == low;
          all = __ballot_sync(~0u, best);
          if (all & (all - 1)) {
            const u64 at = best ? (u64)pos[e] : ~0ull;
            const uint32_t w = __reduce_min_sync(~0u, (uint32_t)(at >> 32));
            best = best && (uint32_t)(at >> 32) == w;
            const uint32_t t = __reduce_min_sync(~0u, best ? (uint32_t)at : ~0u);
            best = best && (uint32_t)at == t;
          }
        }
        if (best) {
          order[i] = (uint16_t)e;
          ++e;
          head = next;
          next = e + 1 < end ? score[e + 1] : 0;
        }
      }
    }
    __syncthreads();
    return sum;
  }
  static_assert(kMaxK <= 64 && kMaxLists <= 2 * kWarps && kMaxCluster <= 2 * kWarps, "two entries a lane, two lists a warp");
  if (threadIdx.x < k) order[threadIdx.x] = (uint16_t)threadIdx.x;
  const int all = 1 << (32 - __clz(k - 1));
#pragma unroll 1
  for (int n = lists; n > 1; n = (n + 1) / 2) {
    const int half = (n + 1) / 2;
    if (warp + half < n && num[warp + half] > 0) {
      const int a = warp, b = warp + half, na = num[a], nb = num[b], sum = min(na + nb, k);
      Entry x[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h, j = all - 1 - i;
        x[h] = {0, ~0ull};  // behind every entry
        if (i < na) x[h] = {score[a * k + i], (u64)pos[a * k + i]};
        if (j >= 0 && j < nb) {
          const Entry y = {score[b * k + j], (u64)pos[b * k + j]};
          if (y.before(x[h])) x[h] = y;
        }
      }
      if (all == 64 && x[1].before(x[0])) {
        const Entry y = x[0];
        x[0] = x[1];
        x[1] = y;
      }
#pragma unroll 1
      for (int d = min(all, 32) / 2; d; d /= 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && all < 64) break;
          const Entry y = {__shfl_xor_sync(~0u, x[h].score, d), __shfl_xor_sync(~0u, x[h].pos, d)};
          if (((lane & d) == 0) != x[h].before(y)) x[h] = y;
        }
      }
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        if (i >= sum) break;
        score[a * k + i] = x[h].score;
        pos[a * k + i] = (long long)x[h].pos;
      }
      if (lane == 0) num[a] = sum;
    }
    __syncthreads();
  }
  return num[0];
}

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(__half x) { return __half2float(x); }

// Part `part` of `parts` of a comparison of two rows, their first elements `from` and
// `at` (not the same) places behind a 16-byte boundary, by a warp: false if it, or
// (*differ >= round) another warp, found a difference.  A vector of x against the two of
// y that hold the same elements, shifted into place; the ends one by one.
template <typename T>
__device__ __forceinline__ bool same_values(const T* x, const T* y, int from, int at, int V, int part, int parts,
                                            volatile int* differ, int round) {
  constexpr int kPer = Type<T>::kPer, kAtOnce = 4;
  const int lane = threadIdx.x & 31;
  const int d = (at - from + kPer) % kPer, bits = d * (int)sizeof(T) % 4 * 8;
  const int64_t begin = (kPer - from) % kPer, head = begin < d ? begin + kPer : begin;  // y's vectors from head - d on
  const int64_t n = max(((int64_t)V - kPer - head + d) / kPer, (int64_t)0);             // vectors whose y lie in the row
  bool equal = true;
  if (part == 0) {
    const int64_t ends = n ? head : V, rest = V - n * kPer;
    for (int64_t i = lane; i < rest; i += 32) {
      const int64_t e = i < ends ? i : i + n * kPer;
      equal = equal && value(x[e]) == value(y[e]);
    }
  }
  bool same = __all_sync(~0u, equal);
#pragma unroll 1
  for (int64_t i0 = (int64_t)part * 32 * kAtOnce; i0 < n && same; i0 += (int64_t)parts * 32 * kAtOnce) {
    uint4 u[kAtOnce], v[kAtOnce][2];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t i = min(i0 + j * 32 + lane, n - 1);
      u[j] = *reinterpret_cast<const uint4*>(x + head + i * kPer);
      v[j][0] = *reinterpret_cast<const uint4*>(y + head - d + i * kPer);
      v[j][1] = *reinterpret_cast<const uint4*>(y + head - d + i * kPer + kPer);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      uint32_t w[8] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w, v[j][1].x, v[j][1].y, v[j][1].z, v[j][1].w};
      const int words = d * (int)sizeof(T) / 4;
#pragma unroll
      for (int k = 0; k < 6; ++k) w[k] = words & 2 ? w[k + 2] : w[k];
#pragma unroll
      for (int k = 0; k < 5; ++k) w[k] = words & 1 ? w[k + 1] : w[k];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], bits);
      if (u[j].x != w[0] || u[j].y != w[1] || u[j].z != w[2] || u[j].w != w[3]) {
        const uint4 z = make_uint4(w[0], w[1], w[2], w[3]);  // 0 and -0 are equal
#pragma unroll
        for (int k = 0; k < kPer; ++k) equal = equal && Type<T>::at(u[j], k) == Type<T>::at(z, k);
      }
    }
    same = __all_sync(~0u, equal && *differ < round);
  }
  return same;
}

// Rows of equal values have equal scores, and the lowest row's tokens go first; but
// where they start at other places modulo 16 bytes their values meet in another order,
// and their sums differ in the last bits.  So rows that start at other places are
// compared, value by value, if their maxima agree and their sums as far as those of
// equal rows do; rows that start at the same place have the same sum if they are equal.
// How far that is, of a sum: a term's exponent is a difference and a product, 2^-24
// of itself each, in hops (to its lane's maximum, to the later ones, to the warp's)
// whose lengths add up to log2 of how often the term goes into the largest one; the
// mean of that over the terms is log2 V, at most 31: 31 x 2^-23 ln 2, or 5.4 x 2^-21.  Every
// hop's exponential errs by 2^-22 and its product by 2^-24, the hops two and one for
// each tile: 0.63 x 2^-21 each; 25 additions of a tile, a part and the lanes by 2^-24: 3.2
// x 2^-21.  That is below (10 + tiles) x 2^-21 for one of the two sums.
//
// All warps of the cluster call it and find the same.  Rounds: every row left is
// compared with the first row it may equal, its values dealt out over all warps,
// which tell each other of a difference.  Measured: 0.3 to 0.6 us where rows start at
// other places and none may be equal (64 x 16 x 32001 bf16 28.0 -> 28.6, 16 x 5 x 100003
// fp32 20.4 -> 20.8), a second reading where all are (64 x 16 x 131071 69 -> 145).
template <typename T>
__device__ __noinline__ int first_equal(const BeamParams& p, int64_t b, uint32_t rank, int tiles) {
  Smem& sm = shared();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = p.W, all = p.cluster * kWarps;
  const T* first = static_cast<const T*>(p.logits) + b * p.batch_stride;
  const int start = (int)(reinterpret_cast<uintptr_t>(first + min(lane, W - 1) * p.beam_stride) / sizeof(T) % Type<T>::kPer);
  const float2 mine = sm.row[min(lane, W - 1)];
  const float near = (float)(2 * (10 + tiles)) * 0x1p-21f * mine.y;
  uint32_t open = 0;  // rows before the lane's that it may equal
#pragma unroll 4
  for (int w = 0; w < W - 1; ++w) {
    const float2 x = sm.row[w];
    open |= (uint32_t)(x.x == mine.x && fabsf(x.y - mine.y) <= near) << w;
  }
  const uint32_t together = __match_any_sync(~0u, start);
  open = lane < W ? open & ~together & ((1u << lane) - 1) : 0;
  int like = lane;
  if (!__any_sync(~0u, open)) return like;
#pragma unroll 1
  for (int round = 1; __any_sync(~0u, open); ++round) {
    const uint32_t rows = __ballot_sync(~0u, open);
    const int pairs = __popc(rows), turns = max(all / pairs, 1);  // warps of a pair
#pragma unroll 1
    for (int t = (int)rank * kWarps + warp; t < pairs * turns; t += all) {
      uint32_t left = rows;
#pragma unroll 1
      for (int i = t % pairs; i; --i) left &= left - 1;
      const int w = __ffs(left) - 1, with = __ffs(__shfl_sync(~0u, open, w)) - 1;
      const bool same = same_values<T>(first + w * p.beam_stride, first + with * p.beam_stride,
                                       __shfl_sync(~0u, start, w), __shfl_sync(~0u, start, with), p.V, t / pairs, turns,
                                       &sm.differ[w], round);
      if (!same && lane < p.cluster) st_cluster_u32(mapa(smem_u32(&sm.differ[w]), lane), (uint32_t)round);
    }
    cluster_sync();
    if (open) {
      // (a row that differed may be told so again by a CTA in the next round)
      if (*reinterpret_cast<volatile int*>(&sm.differ[lane]) >= round) open &= open - 1;
      else like = __ffs(open) - 1, open = 0;
    }
  }
#pragma unroll 1
  for (int w = 1; w < W; ++w) {  // the first of all rows that equal each other
    const int root = __shfl_sync(~0u, like, __shfl_sync(~0u, like, w));
    if (lane == w) like = root;
  }
  return like;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) mla_beam_select_kernel(const __grid_constant__ BeamParams p) {
  Smem& sm = shared();
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const int cluster = p.cluster, parts = p.parts;  // parts of a row in a CTA
  const int64_t b = blockIdx.x / cluster;
  const int W = p.W, V = p.V, k = p.k, all = W * parts, step = cluster * kWarps;
  const int lists = kWarps * ((all + step - 1) / step);  // of this CTA: list l is part own(l)
  const auto own = [&](int l) { return l / kWarps * step + (int)rank * kWarps + l % kWarps; };
  if (tid < W) {
    const float c = p.scores[b * W + tid];
    sm.score[tid] = c;
    sm.live[tid] = p.finished && p.finished[b * W + tid] ? -INFINITY : c;
  }
  cluster_arrive();  // the CTAs have started when they write to each other
  const int64_t len = ((int64_t)(((uint32_t)V + parts - 1) / (uint32_t)parts) + 63) / 64 * 64;
  const int lane = tid & 31;
  if (tid < kMaxW) sm.differ[tid] = 0;
  for (int l = tid; l < lists; l += kThreads) {
    sm.num[l] = 0;
    if (own(l) < all) sm.stat[own(l)] = make_float2(-INFINITY, 0.f);
  }
  __syncthreads();
  constexpr int kPer = Type<T>::kPer;
  Walk<T> at = {}, to = {};  // the tile at hand, the tile to load
  const auto fetch = [&](int stage) {
    if (to.g < all) {
      uint4* dst = &sm.tile[warp][stage][0][lane];
      const int64_t e0 = to.t0 + lane * kPer;
      if (to.t0 >= to.lo && to.t0 + Walk<T>::kTile <= to.hi) {
        const T* src = to.row + e0;
#pragma unroll
        for (int u = 0; u < kVecs; ++u) cp_async16(dst + u * 32, src + u * 32 * kPer);
      } else {
#pragma unroll 1
        for (int u = 0; u < kVecs; ++u) {
          const int64_t e = e0 + u * 32 * kPer;
          if (e >= to.lo && e + kPer <= to.hi) cp_async16(dst + u * 32, to.row + e);
          else if (e + kPer <= to.lo || e >= to.hi) dst[u * 32] = make_uint4(Type<T>::kNone, Type<T>::kNone, Type<T>::kNone, Type<T>::kNone);
          else dst[u * 32] = load_edge<T>(to.row, e, to.lo, to.hi);
        }
      }
      if (to.last()) to.enter(p, sm.live, b, len, to.g + step);
      else to.t0 += Walk<T>::kTile;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  to.enter(p, sm.live, b, len, (int)rank * kWarps + warp);
  at = to;
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  u64* buf = sm.buf[warp];
  float m = -INFINITY, s = 0.f, s_low = 0.f;   // the lane's maximum and sum
  float a[kTops];                              // its largest of every fourth vector
#pragma unroll
  for (int i = 0; i < kTops; ++i) a[i] = -INFINITY;
  uint32_t floor = kLeast, limit = kLeast;     // k values reach the one; from the other on values count
  int n = 0, tiles = 0;                        // candidates, tiles of the epoch
#pragma unroll 1
  for (int stage = 0; at.g < all; stage = stage + 1 < kStages ? stage + 1 : 0) {
    fetch(stage == 0 ? kStages - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    const uint4* tile = &sm.tile[warp][stage][0][lane];
    uint32_t most[kTops];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint4 v = tile[u * 32];
      const uint32_t best = Type<T>::max2(Type<T>::max2(v.x, v.y), Type<T>::max2(v.z, v.w));
      most[u % kTops] = u < kTops ? best : Type<T>::max2(most[u % kTops], best);
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kTops; ++i) {
      const float x = Type<T>::top(most[i]);
      a[i] = fmaxf(a[i], x);
      top = fmaxf(top, x);
    }
    // the sum, over differences to the lane's maximum
    if (top > m) {
      const float f = ex2((m - top) * kLog2e);
      s *= f;
      s_low *= f;
      m = top;
    }
    const float ref = m > -INFINITY ? m : 0.f;
    const u64 minus = f2(-ref, -ref), scale = f2(kLog2e, kLog2e);
    u64 sum[2] = {0, 0};
#pragma unroll 4
    for (int u = 0; u < kVecs; ++u) {
      const uint4 v = tile[u * 32];
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        float x, y;
        f2(mul2(add2(f2(Type<T>::at(v, j), Type<T>::at(v, j + 1)), minus), scale), x, y);
        sum[j / 2 & 1] = add2(sum[j / 2 & 1], f2(ex2(x), ex2(y)));
      }
    }
    float p0, p1, p2, p3;
    f2(sum[0], p0, p1);
    f2(sum[1], p2, p3);
    const float x = (p0 + p1) + (p2 + p3), t = s + x, back = t - s;
    s_low += (s - (t - back)) + (x - back);
    s = t;
    uint16_t* tops = sm.tops[warp];
    const int l = (uint32_t)at.g / (uint32_t)step * kWarps + warp;  // the part's list
    tops[tiles++ * 32 + lane] = (uint16_t)(ordered(top) >> 16);
    if (tiles == kEpoch || at.last()) {
      // the largest of every second vector do for few (10.6 us of one request's
      // beams against 12.5), for k near 64 hardly anything would lie below them
      if (k <= 24) {
        const float two[2] = {fmaxf(a[0], a[2]), fmaxf(a[1], a[3])};
        floor = max(floor, kth_by_all(two, k, sm.words[warp]));
      } else {
        floor = max(floor, kth_of(a, k));
      }
      limit = max(limit, floor);
      // lanes and tiles with a value that reaches it, in place
      int pairs = 0;
#pragma unroll 2
      for (int i = 0; i < tiles; ++i) {
        const bool hit = tops[i * 32 + lane] >= limit >> 16;
        const uint32_t all = __ballot_sync(~0u, hit);
        if (hit) tops[pairs + __popc(all & ((1u << lane) - 1))] = (uint16_t)(i * 32 + lane);
        pairs += __popc(all);
        __syncwarp();
      }
      // their values: the last tile's are at hand, others are read again
      constexpr int kAtOnce = 32 / kVecs, kAhead = 1;  // pairs a step (a vector a lane), steps read ahead
      bool selected = false;
      u64 worst = 0;  // the last of k selected ones
      const auto place = [&](int i) {  // of the lane's vector, from the last tile's first value
        const int pair = tops[min(i + lane / kVecs, pairs - 1)];
        return ((pair >> 5) + 1 - tiles) * Walk<T>::kTile + (lane % kVecs * 32 + (pair & 31)) * kPer;
      };
      const uint4 none = make_uint4(Type<T>::kNone, Type<T>::kNone, Type<T>::kNone, Type<T>::kNone);
      uint4 y[kAhead + 1];
#pragma unroll 1
      for (int i = -kAhead * kAtOnce; i < pairs; i += kAtOnce) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) y[j] = y[j + 1];
        y[kAhead] = none;
        const int ahead = i + kAhead * kAtOnce;
        if (ahead + lane / kVecs < pairs) {
          const int in = place(ahead);
          const int64_t e = at.t0 + in;
          if (in >= 0) y[kAhead] = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(&sm.tile[warp][stage][0][0]) + in);
          else if (e >= at.lo) y[kAhead] = *reinterpret_cast<const uint4*>(at.row + e);
          else if (e + kPer > at.lo) y[kAhead] = load_edge<T>(at.row, e, at.lo, at.hi);
        }
        if (i < 0) continue;
        const float least = unordered(limit);
        const uint32_t where = ~(uint32_t)(at.t0 + place(i));
        uint32_t hits[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) hits[j] = __ballot_sync(~0u, Type<T>::at(y[0], j) >= least);
        const auto key = [&](int j) { return (u64)ordered(Type<T>::at(y[0], j)) << 32 | (where - j); };
        if (worst) {  // (many equal values: 64 x 16 x 131072 zeros took 5.3 ms without)
#pragma unroll
          for (int j = 0; j < kPer; ++j) hits[j] &= __ballot_sync(~0u, key(j) > worst);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if (n + 32 > kCap) {
            // No room for whatever comes: the best so far are selected exactly.
            n = select(l, n, k, &floor);
            limit = max(limit, floor);
            selected = true;
            worst = n == k ? buf[k - 1] : 0;
          }
          if (hits[j] >> lane & 1)
            buf[n + __popc(hits[j] & ((1u << lane) - 1))] = key(j);
          n += __popc(hits[j]);
        }
      }
      __syncwarp();
      if (selected) {  // later tiles' values have to be greater than the last of the best
        n = select(l, n, k, &floor);
        if (n == k) limit = max(limit, floor + 1);
      }
      tiles = 0;
    }
    if (!at.last()) {
      at.t0 += Walk<T>::kTile;
      continue;
    }
    // the part's end
    n = best_keys(l, n, k, floor);
    const float wm = unordered(__reduce_max_sync(~0u, ordered(m)));
    s = (s + s_low) * ex2((wm > -INFINITY ? m - wm : 0.f) * kLog2e);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    if (lane == 0) {
      sm.num[l] = n;
      sm.stat[at.g] = make_float2(wm, s);
    }
    at.enter(p, sm.live, b, len, at.g + step);
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kTops; ++i) a[i] = -INFINITY;
    s = s_low = 0.f;
    floor = limit = kLeast;
    n = 0;
  }
  __syncthreads();
  cluster_wait();
  // Every CTA gets every CTA's part of the rows' statistics.
#pragma unroll 1
  for (int i = tid; i < cluster * lists; i += kThreads) {
    const int to = i / lists, g = own(i % lists);
    if (to == (int)rank || g >= all) continue;
    const float2 x = sm.stat[g];
    const uint32_t at = mapa(smem_u32(&sm.stat[g]), to);
    st_cluster_u32(at, __float_as_uint(x.x));
    st_cluster_u32(at + 4, __float_as_uint(x.y));
  }
  cluster_sync();
  // A row's sum: a quarter warp a row.
#pragma unroll 1
  for (int w0 = 0; w0 < W; w0 += kThreads / 8) {
    const int w = w0 + tid / 8;
    float m = -INFINITY;
    Two sum = {0.f, 0.f};
    if (w < W) {
#pragma unroll 1
      for (int i = tid % 8; i < parts; i += 8) m = fmaxf(m, sm.stat[w * parts + i].x);
    }
#pragma unroll
    for (int d = 4; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    if (w < W) {
#pragma unroll 1
      for (int i = tid % 8; i < parts; i += 8) {
        const float2 x = sm.stat[w * parts + i];
        sum = plus(sum, times_exp(x.y, m > -INFINITY ? x.x - m : 0.f));
      }
    }
#pragma unroll
    for (int d = 4; d; d >>= 1) sum = plus(sum, {__shfl_xor_sync(~0u, sum.hi, d), __shfl_xor_sync(~0u, sum.lo, d)});
    if (w < W && tid % 8 == 0) {
      const float c = sm.score[w];
      const bool done = p.finished && p.finished[b * W + w];
      // an infinite or undefined logit: no continuation of this beam counts
      const bool whole = sum.hi > 0 && sum.hi < INFINITY && fabsf(m) < INFINITY;
      sm.row[w] = make_float2(whole ? m : NAN, sum.hi);
      sm.lse[w] = whole ? (double)m + log_of(sum) : INFINITY;
      sm.ends[w] = done && fabsf(c) < INFINITY;  // its end, at its score
      if (rank == 0 && p.status && (!(c < INFINITY) || (!done && (sum.hi != sum.hi || m == INFINITY))))
        atomicOr(p.status, MLA_STATUS_BAD_SCORE);
    }
  }
  __syncthreads();
  // rows that start at the same place modulo 16 bytes need no comparison
  const int like = p.beam_stride % kPer ? first_equal<T>(p, b, rank, (int)(len / Walk<T>::kTile) + 2) : lane;
  if (warp == 0) sm.like[lane] = like;
  if (tid < lists && own(tid) < all) {
    const int w = own(tid) / parts;
    if (sm.ends[w]) sm.num[tid] = own(tid) % parts == 0;
    else if (!(sm.lse[w] < INFINITY)) sm.num[tid] = 0;
  }
  __syncthreads();
#pragma unroll 1
  for (int e = tid; e < lists * k; e += kThreads) {
    const int l = e / k, w = own(l) / parts;
    if (e % k >= sm.num[l]) continue;
    const double c = sm.score[w];
    const u64 key = sm.list[e];
    const bool end = sm.ends[w];
    sm.pos[e] = (long long)w << 32 | (end ? (uint32_t)p.end_token : (uint32_t)~(uint32_t)key);
    sm.list[e] = ordered(end ? c : c + ((double)unordered((uint32_t)(key >> 32)) - sm.lse[sm.like[w]]));
  }
  __syncthreads();
  const uint32_t to_score = mapa(smem_u32(sm.got_score + rank * k), 0);
  const uint32_t to_pos = mapa(smem_u32(sm.got_pos + rank * k), 0);
  const int sum = merge_lists(sm.list, sm.pos, sm.num, lists, k, sm.order);
  if (tid < sum) {
    const int e = sm.order[tid];
    const u64 a = sm.list[e], q = (u64)sm.pos[e];
    st_cluster_u32(to_score + 8 * tid, (uint32_t)a);
    st_cluster_u32(to_score + 8 * tid + 4, (uint32_t)(a >> 32));
    st_cluster_u32(to_pos + 8 * tid, (uint32_t)q);
    st_cluster_u32(to_pos + 8 * tid + 4, (uint32_t)(q >> 32));
  }
  if (tid == 0) st_cluster_u32(mapa(smem_u32(sm.got_num + rank), 0), (uint32_t)sum);
  cluster_sync();
  if (rank != 0) return;
  const auto put = [&](int at, float s, int w, int t) {
    p.out_scores[b * k + at] = s;
    p.parents[b * k + at] = (int)(b * W + w);
    p.tokens[b * k + at] = t;
  };
  const int have = merge_lists(sm.got_score, sm.got_pos, sm.got_num, cluster, k, sm.order);
  if (tid < have) {
    const int e = sm.order[tid];
    const long long q = sm.got_pos[e];
    put(tid, (float)unordered(sm.got_score[e]), (int)(q >> 32), (int)(uint32_t)q);
    sm.member[tid] = (q >> 32) * V + (uint32_t)q;
  }
  // Fewer than k continuations: the lowest positions that are none, at -inf.
  __syncthreads();
  if (tid < k - have) {
    long long q = tid;
#pragma unroll 1
    for (bool moved = true; moved;) {
      int below = 0;
#pragma unroll 1
      for (int j = 0; j < have; ++j) below += sm.member[j] <= q;
      moved = tid + below != q;
      q = tid + below;
    }
    put(have + tid, -INFINITY, (int)(q / V), (int)(q % V));
  }
}

__global__ void mla_beam_math_kernel(const float* x, const float* y, int64_t n, double* exp_x, double* log_y) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const Two e = exp_two(x[i]);
    exp_x[i] = (double)e.hi + (double)e.lo;
    log_y[i] = log_of({y[i], 0.f});
  }
}

// Clusters of a size that the device holds at once, asked of each device once (fewer
// than its places for CTAs divide into: a GPC's SMs leave a rest).
template <typename T>
int clusters_at_once(cudaLaunchConfig_t cfg, int dev, int* n) {
  static std::atomic<int> known[64][kMaxCluster + 1];
  const int size = (int)cfg.attrs->val.clusterDim.x;
  *n = dev < 64 ? known[dev][size].load() : 0;
  if (*n) return MLA_OK;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(n, mla_beam_select_kernel<T>, &cfg);
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
  if (dev < 64) known[dev][size].store(*n);
  return MLA_OK;
}

// CTAs of a request: as many as all find room at once (two an SM; a second round of
// clusters costs more than it brings: 60 x 8 x 131072 bf16 took 53 us with clusters of
// 5, 37 with 4; 76 requests 60 with 4, 45 with 3), while a warp has about a tile of
// logits.  Parts of a row: the number whose rounds over the cluster's
// warps cost least, a part its tiles and about three more.
template <typename T>
int launch_beam(BeamParams p, int B, cudaStream_t st) {
  auto kernel = mla_beam_select_kernel<T>;
  int dev = 0, sms = 0;
  int rc = device_sms(&dev, &sms);
  static std::atomic<uint64_t> set_on{0};
  if (rc == MLA_OK) rc = allow_shared(kernel, (int)sizeof(Smem), dev, set_on, "cudaFuncSetAttribute(mla_beam_select_kernel)");
  if (rc != MLA_OK) return rc;
  constexpr int kTile = 32 * kVecs * Type<T>::kPer;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(Smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  p.cluster = p.W > kMaxLists ? 2 : 1;
  for (int c = p.cluster + 1; c <= kMaxCluster && (int64_t)B * c <= 2 * sms &&
                              (int64_t)p.W * p.V > (int64_t)(c - 1) * kWarps * kTile / 2; ++c) {
    int at_once = 0;
    cfg.gridDim = dim3((unsigned)c, 1, 1);
    attr[0].val.clusterDim.x = (unsigned)c;
    if ((rc = clusters_at_once<T>(cfg, dev, &at_once)) != MLA_OK) return rc;
    if (B <= at_once) p.cluster = c;
  }
  double least = 0;
  for (int parts = 1; p.W * parts <= std::max(2 * p.cluster * kWarps, p.W) && p.W * parts <= kMaxParts; ++parts) {
    const int rounds = (p.W * parts + p.cluster * kWarps - 1) / (p.cluster * kWarps);
    const double cost = rounds * (double)(p.V / parts / kTile + 4);
    if (parts == 1 || cost < least) least = cost, p.parts = parts;
  }
  cfg.gridDim = dim3((unsigned)(B * p.cluster), 1, 1);
  attr[0].val.clusterDim.x = (unsigned)p.cluster;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
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
  if ((int64_t)B * W > 0x7fffffff || B > 0x7fffffff / kMaxCluster)
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
                     out_scores, parents, tokens, status, 1, 1};
  const cudaStream_t st = (cudaStream_t)stream;
  if (dtype == MLA_LOGIT_BF16) return launch_beam<__nv_bfloat16>(p, B, st);
  if (dtype == MLA_LOGIT_F16) return launch_beam<__half>(p, B, st);
  return launch_beam<float>(p, B, st);
}

extern "C" int mla_debug_beam_math(const float* x, const float* y, int64_t n, double* exp_x, double* log_y,
                                   mla_stream_t stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "mla_debug_beam_math: n = %lld < 0", (long long)n);
  if (n == 0) return MLA_OK;
  if (!x || !y || !exp_x || !log_y) return fail(MLA_ERR_INVALID_ARG, "mla_debug_beam_math: a required pointer is NULL");
  if (!aligned(x, 4) || !aligned(y, 4) || !aligned(exp_x, 8) || !aligned(log_y, 8))
    return fail(MLA_ERR_MISALIGNED, "mla_debug_beam_math: inputs need 4-B alignment, outputs 8-B");
  mla_beam_math_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 1024), 256, 0, (cudaStream_t)stream>>>(x, y, n, exp_x, log_y);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_beam_math_kernel");
  return MLA_OK;
}
