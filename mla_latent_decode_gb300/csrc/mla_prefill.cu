// mla_prefill.cu -- attention within packed prompts before absorption
// (mla_prefill): per head s = scale (q_nope . k_nope + q_rope . k_rope), one
// RoPE key for all heads, and o = softmax(s) v over the keys that a row sees,
// which are always the first ones of its sequence.
//
// A CTA owns 256 query rows of one sequence and head as two tiles of 128 rows.
// Keys come in tiles of 128 tokens: S = Q K^T is 12 tcgen05 MMAs of M = 128,
// N = 128, K = 16 (192 dims), O += P V eight more.  TMEM holds S and O of both
// row tiles (4 x 128 columns); P overwrites its S in bf16 and is the MMA's A
// operand from there.  While the softmax of one row tile runs, the tensor cores
// work for the other: PV_0(j - 1), QK_0(j), PV_1(j - 1), QK_1(j), ...  MMAs of
// one thread execute in order, so "S_g(j) is there" also says that PV_g(j - 1)
// is done: the softmax may rescale O in place then, and S may overwrite P.
//
//   warps 0-3, 4-7   softmax of row tile 0 and 1, one thread per row, then O / l
//   warp 8           TMA: Q (96 KB, stays), K and V through a ring of 8 stages
//                    of 16 KB, K in three (64 dims x 128 tokens each, the third
//                    the RoPE key), V in two (64 tokens x 128 dims)
//   warp 9           MMA issue (one lane)
//   warps 10, 11     clean V: in tiles that hold tokens which some row of the CTA
//                    does not see, values that are not finite become 0 (P is 0
//                    there, and 0 x NaN would reach the row) and are noted per
//                    dim; the rows that do see them get them back at the end
//
// Softmax in base 2 with fp32 statistics; O is rescaled only when a row's
// maximum has risen by more than 2^8, so P stays below 2^8 and its rounding to
// bf16 is 2^-8 of each probability either way.
#include <cuda_bf16.h>

#include <algorithm>

#include "mla_tma.cuh"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kRows = 128;           // rows of a tile (MMA M)
constexpr int kBlock = 2 * kRows;    // rows of a CTA
constexpr int kKeys = 128;           // tokens of a key tile
constexpr int kBox = 128 * 128;      // 16 KB
constexpr int kStages = 8;
constexpr int kThreads = 384;
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpClean = 10;
// 384 threads launch with 168 registers (64512 in all): 256 x 216 + 128 x 72.
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kRise = 8.f;         // log2 of the rise that rescales O
constexpr int kEntry = 8;            // int32 of a work entry

struct PrefillParams {
  const int32_t* cu_q;
  const int32_t* cu_kv;
  const int32_t* prefix;
  int N, H, causal;
  int64_t Tq, Tk;
  float sm_scale, scale2;  // scale2 = sm_scale * log2(e)
  const int32_t* work;
  int num_work, num_parts;
  float* O_part;
  float* LSE_part;
  __nv_bfloat16* out;
  float* lse;
  int* status;
};

struct Ctl {
  uint64_t q[2], full[kStages], empty[kStages];
  uint64_t s[2];      // S of a row tile is in TMEM
  uint64_t p[2];      // its P is, and S has been read
  uint64_t o[2];      // O is complete
  uint64_t raw[2];    // V of a tile to be cleaned has landed (tiles take turns: two may be waiting)
  uint64_t cleaned;   // all of them are
  uint64_t drain;
  int odd[3][kKeys];  // per dim: the first cleaned NaN, +inf, -inf
  uint32_t tmem;
  int abort_flag, any_odd;
};
constexpr int kSmem = 6 * kBox + kStages * kBox + (int)sizeof(Ctl) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory budget");

// What a CTA computes.
struct Unit {
  int seq, h, row0, rows;   // rows: of the block that exist
  int64_t q0, k0;           // first row and key of the sequence
  int lq, lk, prefix;
  int part, parts, slot;
  int n0, n1;               // key tiles of the two row tiles: j0 <= j < n
  int j0, j1;
  int clean0;               // first tile whose V is cleaned
};

// Keys that row i of a sequence sees.
__device__ __forceinline__ int sees(const PrefillParams& p, int lq, int lk, int prefix, int i) {
  if (!p.causal) return lk;
  return min(lk, max(prefix, max(lk - lq + 1 + i, 0)));
}

// The CTA's unit, false if the entry or the lengths are none.
__device__ __forceinline__ bool find_unit(const PrefillParams& p, Unit& u) {
  const int x = blockIdx.x;
  const int32_t* e = p.work + (int64_t)(x / p.H) * kEntry;
  const int g0 = e[5], nb = e[6];
  int bad = 0;
  if (g0 < 0 || nb < 1 || g0 > x / p.H || g0 + nb <= x / p.H || g0 + nb > p.num_work) {
    bad = MLA_STATUS_BAD_WORK;
  } else {
    const int64_t local = x - (int64_t)g0 * p.H;
    u.h = (int)(local / nb);
    e = p.work + (g0 + local % nb) * kEntry;
    u.seq = e[0];
    u.part = e[2];
    u.parts = e[3];
    u.slot = e[4];
    const int64_t row0 = (int64_t)e[1] * kBlock;
    if (u.h >= p.H || u.seq < 0 || u.seq >= p.N || e[1] < 0 || u.parts < 1 ||
        u.parts > MLA_PREFILL_MAX_PARTS || u.part < 0 || u.part >= u.parts ||
        (u.parts > 1 && (u.slot < 0 || u.slot > p.num_parts - u.parts))) {
      bad = MLA_STATUS_BAD_WORK;
    } else {
      u.q0 = p.cu_q[u.seq];
      u.k0 = p.cu_kv[u.seq];
      const int64_t lq = p.cu_q[u.seq + 1] - u.q0, lk = p.cu_kv[u.seq + 1] - u.k0;
      if (u.q0 < 0 || u.k0 < 0 || lq < 0 || lk < 0 || u.q0 + lq > p.Tq || u.k0 + lk > p.Tk) {
        bad = MLA_STATUS_BAD_LENGTH;
      } else if (row0 >= lq) {
        bad = MLA_STATUS_BAD_WORK;
      } else {
        u.lq = (int)lq;
        u.lk = (int)lk;
        u.row0 = (int)row0;
        u.rows = min(kBlock, u.lq - u.row0);
        u.prefix = p.prefix ? p.prefix[u.seq] : 0;
        int n[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int last = min(kRows * (g + 1), u.rows) - 1;
          n[g] = last < kRows * g ? 0
                 : (sees(p, u.lq, u.lk, u.prefix, u.row0 + last) + kKeys - 1) / kKeys;
        }
        const int64_t all = max(n[0], n[1]);
        u.j0 = (int)(all * u.part / u.parts);
        u.j1 = (int)(all * (u.part + 1) / u.parts);
        u.n0 = min(n[0], u.j1);
        u.n1 = min(n[1], u.j1);
        u.clean0 = max(u.j0, sees(p, u.lq, u.lk, u.prefix, u.row0) / kKeys);
        return true;
      }
    }
  }
  if (threadIdx.x == 0 && p.status) atomicOr(p.status, bad);
  return false;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint64_t f2pack(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ void f2unpack(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Ring positions: K(t) at 5 t .. 5 t + 2, V(t) at 5 t + 3, 5 t + 4.
__device__ __forceinline__ void produce(uint8_t* base, Ctl& c, const PrefillParams& p, const Unit& u,
                                        const CUtensorMap* qn, const CUtensorMap* qr,
                                        const CUtensorMap* kn, const CUtensorMap* kr,
                                        const CUtensorMap* v, int lane) {
  const int tiles = u.j1 - u.j0;
  // Q: six boxes, each from its own lane (a thread's loads go one after another)
  const int boxes = u.rows > kRows ? 6 : 3;
  if (lane < 2 && lane * 3 < boxes) mbar_arrive_expect_tx(smem_u32(&c.q[lane]), 3 * kBox);
  __syncwarp();
  if (lane < boxes) {
    const int g = lane / 3, d = lane % 3;
    const int row = (int)(u.q0 + u.row0 + g * kRows);
    const uint32_t dst = smem_u32(base + lane * kBox), bar = smem_u32(&c.q[g]);
    if (d < 2) tma_load_3d(dst, qn, bar, d * 64, u.h, row);
    else tma_load_3d(dst, qr, bar, 0, u.h, row);
  }
  bool ok = true;
  uint32_t pos = 0;
  for (int t = 0; t < tiles && ok; ++t) {
    const int tok = (int)u.k0 + (u.j0 + t) * kKeys;
    for (int i = 0; i < 5; ++i, ++pos) {
      const uint32_t st = pos % kStages, use = pos / kStages;
      if (use > 0 && !mbar_wait_cta(smem_u32(&c.empty[st]), (use - 1) & 1, &c.abort_flag)) {
        ok = false;
        break;
      }
      if (lane == (int)(pos & 3)) {
        const uint32_t dst = smem_u32(base + (6 + st) * kBox), bar = smem_u32(&c.full[st]);
        const int nth = u.j0 + t - u.clean0;
        if (i >= 3 && nth >= 0) {
          // its stage is full once it is clean
          const uint32_t raw = smem_u32(&c.raw[nth & 1]);
          if (i == 3) mbar_arrive_expect_tx(raw, 2 * kBox);
          tma_load_4d(dst, v, raw, 0, tok + (i - 3) * 64, 0, u.h);
          continue;
        }
        mbar_arrive_expect_tx(bar, kBox);
        if (i < 2) tma_load_3d(dst, kn, bar, i * 64, u.h, tok);
        else if (i == 2) tma_load_3d(dst, kr, bar, 0, 0, tok);
        else tma_load_4d(dst, v, bar, 0, tok + (i - 3) * 64, 0, u.h);
      }
    }
    __syncwarp();
  }
  if (!ok && lane == 0) {
    c.abort_flag = 1;
    if (p.status) atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
  }
  // Every load issued has landed before the CTA may exit.
  int never = 0;
  for (int g = 0; g * 3 < boxes; ++g) mbar_wait_cta(smem_u32(&c.q[g]), 0, &never);
  for (uint32_t j = pos > (uint32_t)kStages ? pos - kStages : 0; j < pos; ++j) {
    const int nth = u.j0 + (int)(j / 5) - u.clean0;
    if (j % 5 < 3 || nth < 0) mbar_wait_cta(smem_u32(&c.full[j % kStages]), (j / kStages) & 1, &never);
    else mbar_wait_cta(smem_u32(&c.raw[nth & 1]), nth >> 1 & 1, &never);
  }
}

// a0, a1: key tiles of the two row tiles.
__device__ __forceinline__ void issue_mmas(uint8_t* base, Ctl& c, const PrefillParams& p, int a0, int a1,
                                           uint32_t tmem) {
  constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys, false, false);
  constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, kKeys, false, true);
  const int tiles = max(a0, a1);
  const uint64_t q0 = sdesc_sw128(smem_u32(base), 16, 1024);
  const uint64_t k0 = sdesc_sw128(smem_u32(base + 6 * kBox), 16, 1024);
  // V: MN-major, the next 64 dims 8 KB (LBO) on, the next 8 tokens 1 KB (SBO) on,
  // the next 16 tokens 2 KB; P: 16 tokens in 8 columns
  const uint64_t v0 = sdesc_sw128(smem_u32(base + 6 * kBox), kBox / 2, 1024);
  bool ok = true;
  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && mbar_wait_cta(smem_u32(bar), parity, &c.abort_flag);
    return ok;
  };
  for (int t = 0; t <= tiles && ok; ++t) {
    const uint32_t kpos = 5 * t, vpos = 5 * t - 2;  // vpos: V(t - 1)
#pragma unroll 1
    for (int g = 0; g < 2 && ok; ++g) {
      const uint32_t s = tmem + g * kKeys, o = tmem + (2 + g) * kKeys;
      const int a = g ? a1 : a0;
      if (t > 0 && t - 1 < a) {
        if (!wait(&c.p[g], (t - 1) & 1)) break;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const uint32_t st = (vpos + i) % kStages;
          if (!wait(&c.full[st], (vpos + i) / kStages & 1)) break;
          tc_fence_after();
          const uint64_t b = v0 + st * (kBox >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(o, s + (4 * i + k) * 8, b + 128 * k, idesc_o, (t > 1 || i || k) ? 1u : 0u);
          if (g || t - 1 >= a1) mma_commit(smem_u32(&c.empty[st]));
        }
        if (!ok) break;
        if (t == a) mma_commit(smem_u32(&c.o[g]));
      }
      if (t < a) {
        if (t == 0 && !wait(&c.q[g], 0)) break;
#pragma unroll 1
        for (int i = 0; i < 3; ++i) {
          const uint32_t st = (kpos + i) % kStages;
          if (!wait(&c.full[st], (kpos + i) / kStages & 1)) break;
          tc_fence_after();
          const uint64_t q = q0 + (3 * g + i) * (kBox >> 4), b = k0 + st * (kBox >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ss(s, q + 2 * k, b + 2 * k, idesc_s, (i || k) ? 1u : 0u);
          if (g || t >= a1) mma_commit(smem_u32(&c.empty[st]));
        }
        if (!ok) break;
        mma_commit(smem_u32(&c.s[g]));
      }
    }
  }
  if (!ok) {
    c.abort_flag = 1;
    if (p.status) atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
  }
  // No MMA may still run when the accumulators are freed.
  int never = 0;
  mma_commit(smem_u32(&c.drain));
  mbar_wait_cta(smem_u32(&c.drain), 0, &never);
}

// Tiles from u.clean0 on hold tokens that some row does not see (its own later
// ones, or the next sequence's).  Warp i of the two cleans stage i of a tile's V.
__device__ __forceinline__ void clean_values(uint8_t* base, Ctl& c, const PrefillParams& p, const Unit& u,
                                             int i, int lane) {
  const int from = sees(p, u.lq, u.lk, u.prefix, u.row0);
  for (int j = u.clean0; j < u.j1; ++j) {
    const int nth = j - u.clean0;
    if (!__all_sync(~0u, mbar_wait_cta(smem_u32(&c.raw[nth & 1]), nth >> 1 & 1, &c.abort_flag))) {
      c.abort_flag = 1;
      if (lane == 0 && p.status) atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
      return;
    }
    const uint32_t st = (5 * (j - u.j0) + 3 + i) % kStages;
    uint8_t* box = base + (6 + st) * kBox;
    const int t0 = j * kKeys + i * 64;  // token of the stage's first row
    // 1024 vectors: half (64 dims), row, 16-byte chunk, swizzled by the row
#pragma unroll 4
    for (int x = lane; x < kBox / 16; x += 32) {
      uint4* at = reinterpret_cast<uint4*>(box + x * 16);
      const int half = x >> 9, row = (x >> 3) & 63, chunk = (x & 7) ^ (row & 7);
      uint4 w = *at;
      uint32_t* r = reinterpret_cast<uint32_t*>(&w);
      uint32_t hit = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) hit |= (r[e] & 0x7f807f80u) + 0x00800080u;
      if (!(hit & 0x80008000u) || t0 + row < from) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = r[e / 2] >> (16 * (e & 1)) & 0xffffu;
        if ((b & 0x7f80u) != 0x7f80u) continue;
        r[e / 2] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
        if (t0 + row < u.lk) {
          const int kind = b & 0x7fu ? 0 : b & 0x8000u ? 2 : 1;
          atomicMin(&c.odd[kind][half * 64 + chunk * 8 + e], t0 + row);
          c.any_odd = 1;
        }
      }
      *at = w;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&c.full[st]));
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&c.cleaned));
}

// Softmax of row tile g, one thread per row, then the row's output.
__device__ __forceinline__ void softmax_rows(Ctl& c, const PrefillParams& p, const Unit& u, uint32_t tmem,
                                             int g, int warp, int lane) {
  const int r = (warp & 3) * 32 + lane, i = u.row0 + g * kRows + r;
  const bool exists = g * kRows + r < u.rows;
  const int seen = exists ? sees(p, u.lq, u.lk, u.prefix, i) : 0x7fffffff;  // padding rows: unmasked
  const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t s_at = tmem + quad + g * kKeys, o_at = tmem + quad + (2 + g) * kKeys;
  const uint64_t scale2 = f2pack(p.scale2, p.scale2);
  float ref = -INFINITY, l = 0.f;  // raw scores; sum of 2^((s - ref) scale2)
  bool ok = true;
  const int tiles = (g ? u.n1 : u.n0) - u.j0, seen0 = exists ? seen - u.j0 * kKeys : 0x7fffffff;
  // where the row's output goes: its row of out, or of the part's workspace
  const bool whole = u.parts == 1, cleaned = u.j1 > u.clean0;
  const int64_t row = whole ? (u.q0 + i) * p.H + u.h
                            : ((int64_t)(u.slot + u.part) * p.H + u.h) * kBlock + g * kRows + r;
  for (int t = 0; t < tiles; ++t) {
    if (!(ok = mbar_wait_cta(smem_u32(&c.s[g]), t & 1, &c.abort_flag))) break;
    tc_fence_after();
    float s[kKeys];
#pragma unroll
    for (int b = 0; b < 4; ++b) tmem_ld32(s_at + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * b]));
    tmem_wait_ld();
    const int last = seen0 - t * kKeys;  // columns of this tile that the row sees
    if (__any_sync(~0u, last < kKeys)) {
#pragma unroll
      for (int e = 0; e < kKeys; ++e) s[e] = e < last ? s[e] : -INFINITY;
    }
    float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int e = 4; e < kKeys; e += 8) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        m4[b] = e + 4 + b < kKeys ? max3(m4[b], s[e + b], s[e + 4 + b]) : fmaxf(m4[b], s[e + b]);
    }
    const float m = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
    // A row's first score, or one far above the reference: a new reference.
    const bool rise = (m - ref) * p.scale2 > kRise;  // ref = -inf: true for a finite m
    if (__any_sync(~0u, rise)) {
      float a = 1.f;
      if (rise) {
        a = ref > -INFINITY ? ex2((ref - m) * p.scale2) : 1.f;  // nothing summed so far: O is 0
        l *= a;
        ref = m;
      }
      if (t > 0) {
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          uint32_t o[32];
          tmem_ld32(o_at + 32 * b, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
          tmem_st32(o_at + 32 * b, o);
        }
      }
    }
    const float off = ref > -INFINITY ? -ref * p.scale2 : 0.f;
    const uint64_t off2 = f2pack(off, off);
    uint64_t sum2[2] = {f2pack(l, 0.f), f2pack(0.f, 0.f)};
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t pk[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float ya, yb;
        f2unpack(ffma2(f2pack(s[64 * b + 2 * e], s[64 * b + 2 * e + 1]), scale2, off2), ya, yb);
        const float pa = ex2(ya), pb = ex2(yb);
        sum2[e & 1] = fadd2(sum2[e & 1], f2pack(pa, pb));
        pk[e] = pack_bf16(pa, pb);
      }
      tmem_st32(s_at + 32 * b, pk);
    }
    float x, y, z, w;
    f2unpack(sum2[0], x, y);
    f2unpack(sum2[1], z, w);
    l = (x + y) + (z + w);
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(smem_u32(&c.p[g]));
  }
  if (ok && tiles > 0) ok = mbar_wait_cta(smem_u32(&c.o[g]), 0, &c.abort_flag);
  if (ok && cleaned) ok = mbar_wait_cta(smem_u32(&c.cleaned), 0, &c.abort_flag);
  if (!ok) {
    c.abort_flag = 1;
    if (lane == 0 && p.status) atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
    return;
  }
  tc_fence_after();
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  const float lse = l > 0.f || l != l ? ref * p.sm_scale + logf(l) : -INFINITY;
  const bool odd = *reinterpret_cast<volatile int*>(&c.any_odd) != 0;
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    uint32_t o[32];
    __syncwarp();
    if (tiles > 0) {
      tmem_ld32(o_at + 32 * b, o);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0;
    }
    float f[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) f[e] = l == 0.f ? 0.f : __uint_as_float(o[e]) * inv;
    if (odd) {
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        if (c.odd[0][32 * b + e] < seen) f[e] += NAN;
        if (c.odd[1][32 * b + e] < seen) f[e] += INFINITY;
        if (c.odd[2][32 * b + e] < seen) f[e] -= INFINITY;
      }
    }
    if (exists && whole) {
      uint4* dst = reinterpret_cast<uint4*>(p.out + row * MLA_V_HEAD_DIM + 32 * b);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dst[e] = make_uint4(pack_bf16(f[8 * e], f[8 * e + 1]), pack_bf16(f[8 * e + 2], f[8 * e + 3]),
                            pack_bf16(f[8 * e + 4], f[8 * e + 5]), pack_bf16(f[8 * e + 6], f[8 * e + 7]));
    } else if (exists) {
      float4* dst = reinterpret_cast<float4*>(p.O_part + row * MLA_V_HEAD_DIM + 32 * b);
#pragma unroll
      for (int e = 0; e < 8; ++e) dst[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
    }
  }
  if (exists) {
    if (!whole) p.LSE_part[row] = lse;
    else if (p.lse) p.lse[row] = lse;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap qn, const __grid_constant__ CUtensorMap qr,
                       const __grid_constant__ CUtensorMap kn, const __grid_constant__ CUtensorMap kr,
                       const __grid_constant__ CUtensorMap v, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl& c = *reinterpret_cast<Ctl*>(base + (6 + kStages) * kBox);
  const int warp = __shfl_sync(~0u, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  Unit u;
  if (!find_unit(p, u)) return;  // the whole CTA
  if (threadIdx.x == 0) {
    c.abort_flag = c.any_odd = 0;
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_u32(&c.q[g]), 1);
      mbar_init(smem_u32(&c.s[g]), 1);
      mbar_init(smem_u32(&c.p[g]), kRows);
      mbar_init(smem_u32(&c.o[g]), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&c.full[i]), 1);
      mbar_init(smem_u32(&c.empty[i]), 1);
    }
    mbar_init(smem_u32(&c.raw[0]), 1);
    mbar_init(smem_u32(&c.raw[1]), 1);
    mbar_init(smem_u32(&c.cleaned), 2);
    mbar_init(smem_u32(&c.drain), 1);
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 3 * kKeys; i += kThreads) c.odd[i / kKeys][i % kKeys] = 0x7fffffff;
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&c.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, c.tmem, 0);
  // Roles never rejoin below their register split: each ends with the teardown.
  if (warp >= kWarpTma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kWarpTma) {
      produce(base, c, p, u, &qn, &qr, &kn, &kr, &v, lane);
    } else if (warp == kWarpMma) {
      // uniform values: see elect_one
      const int a0 = __shfl_sync(~0u, u.n0 - u.j0, 0), a1 = __shfl_sync(~0u, u.n1 - u.j0, 0);
      if (elect_one()) issue_mmas(base, c, p, a0, a1, tmem);
    } else {
      clean_values(base, c, p, u, warp - kWarpClean, lane);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(tmem, 512);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax_rows(c, p, u, tmem, warp / 4, warp, lane);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
  }
}

// Merge of a block's parts, a warp per row: weights e^(LSE_s - max), parts in
// order.  Parts without keys (LSE = -inf) weigh nothing; a NaN makes the row NaN.
__global__ void __launch_bounds__(256) mla_prefill_merge_kernel(const PrefillParams p) {
  griddep_wait();
  const int32_t* e = p.work + (int64_t)(blockIdx.x / p.H) * kEntry;
  const int h = blockIdx.x % p.H, seq = e[0], parts = e[3], slot = e[4];
  if (e[2] != 0 || parts < 2 || parts > MLA_PREFILL_MAX_PARTS || slot < 0 ||
      slot > p.num_parts - parts || seq < 0 || seq >= p.N || e[1] < 0)
    return;  // reported by the first launch
  const int64_t q0 = p.cu_q[seq], lq = p.cu_q[seq + 1] - q0, row0 = (int64_t)e[1] * kBlock;
  const int64_t k0 = p.cu_kv[seq], lk = p.cu_kv[seq + 1] - k0;
  if (q0 < 0 || lq < 0 || q0 + lq > p.Tq || k0 < 0 || lk < 0 || k0 + lk > p.Tk) return;
  const int rows = (int)min((int64_t)kBlock, lq - row0), lane = threadIdx.x & 31;
  for (int r = threadIdx.x / 32; r < rows; r += 8) {
    const int64_t at = ((int64_t)slot * p.H + h) * kBlock + r, step = (int64_t)p.H * kBlock;
    const float mine = lane < parts ? p.LSE_part[at + lane * step] : -INFINITY;
    float m = mine;
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    const bool nan = __any_sync(~0u, mine != mine);
    const float w = mine > -INFINITY ? expf(mine - m) : 0.f;
    float sum = w;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < parts; ++s) {
      const float ws = __shfl_sync(~0u, w, s);
      if (ws == 0.f) continue;
      const float4 x = reinterpret_cast<const float4*>(p.O_part + (at + s * step) * MLA_V_HEAD_DIM)[lane];
      o.x += ws * x.x, o.y += ws * x.y, o.z += ws * x.z, o.w += ws * x.w;
    }
    const float inv = nan ? NAN : sum > 0.f ? 1.f / sum : 0.f;
    const int64_t row = (q0 + row0 + r) * p.H + h;
    reinterpret_cast<uint2*>(p.out + row * MLA_V_HEAD_DIM)[lane] =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (lane == 0 && p.lse) p.lse[row] = nan ? NAN : sum > 0.f ? m + logf(sum) : -INFINITY;
  }
}

// Tensor map of [T, H, dims] bf16 in boxes of 64 dims x 128 tokens of a head.
int head_map(CUtensorMap* map, const void* base, int dims, int H, int64_t T, int64_t token_stride,
             int64_t head_stride) {
  const uint64_t d[3] = {(uint64_t)dims, (uint64_t)H, (uint64_t)std::max<int64_t>(T, 1)};
  const uint64_t st[2] = {(uint64_t)(H > 1 ? head_stride : dims) * 2,
                          (uint64_t)(T > 1 ? token_stride : (int64_t)H * dims) * 2};
  const uint32_t box[3] = {64, 1, 128};
  return make_tensor_map_bf16_3d(map, base, d, st, box);
}

// One head's rows of `dims` values at these strides.
bool bad_strides(int64_t T, int H, int dims, int64_t token_stride, int64_t head_stride) {
  return (T > 1 && token_stride < dims) || (H > 1 && head_stride < dims);
}
bool off_vector(const void* base, int64_t T, int H, int64_t token_stride, int64_t head_stride) {
  return !aligned(base, 16) || (T > 1 && token_stride % 8) || (H > 1 && head_stride % 8);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_prefill(const void* q_nope, int64_t qn_token_stride, int64_t qn_head_stride,
                           const void* q_rope, int64_t qr_token_stride, int64_t qr_head_stride,
                           int64_t Tq, const void* k_nope, int64_t kn_token_stride,
                           int64_t kn_head_stride, const void* k_rope, int64_t kr_token_stride,
                           const void* v, int64_t v_token_stride, int64_t v_head_stride, int64_t Tk,
                           int H, const int32_t* cu_q, const int32_t* cu_kv, const int32_t* prefix,
                           int N, int causal, float sm_scale, const int32_t* work, int num_work,
                           int num_parts, float* O_part, float* LSE_part, void* out, float* lse,
                           int* status, mla_stream_t stream) {
  constexpr int kNope = MLA_QK_NOPE_DIM, kRope = MLA_ROPE_DIM, kValue = MLA_V_HEAD_DIM;
  if (Tq < 0 || Tk < 0 || N < 0 || num_work < 0 || num_parts < 0 || H < 1)
    return fail(MLA_ERR_INVALID_ARG, "mla_prefill: Tq=%lld Tk=%lld N=%d num_work=%d num_parts=%d < 0 or H=%d < 1",
                (long long)Tq, (long long)Tk, N, num_work, num_parts, H);
  if (!(sm_scale > 0.f) || sm_scale > 1e30f)
    return fail(MLA_ERR_INVALID_ARG, "mla_prefill: sm_scale %g is not a positive number", (double)sm_scale);
  if (Tq > 0x7fffff00 || Tk > 0x7fffff00 || H > 65535 || (int64_t)num_work * H > 0x7fffffff)
    return fail(MLA_ERR_INVALID_ARG, "mla_prefill: Tq=%lld, Tk=%lld, H=%d or num_work=%d too large",
                (long long)Tq, (long long)Tk, H, num_work);
  if (num_work == 0 || N == 0 || Tq == 0) return MLA_OK;
  if (!q_nope || !q_rope || !out || !cu_q || !cu_kv || !work || (Tk > 0 && (!k_nope || !k_rope || !v)) ||
      (num_parts > 0 && (!O_part || !LSE_part)))
    return fail(MLA_ERR_INVALID_ARG, "mla_prefill: a required pointer is NULL");
  if (bad_strides(Tq, H, kNope, qn_token_stride, qn_head_stride) ||
      bad_strides(Tq, H, kRope, qr_token_stride, qr_head_stride) ||
      bad_strides(Tk, H, kNope, kn_token_stride, kn_head_stride) ||
      bad_strides(Tk, H, kValue, v_token_stride, v_head_stride) ||
      bad_strides(Tk, 1, kRope, kr_token_stride, kRope))
    return fail(MLA_ERR_INVALID_ARG, "mla_prefill: a stride is below its row's length");
  if (off_vector(q_nope, Tq, H, qn_token_stride, qn_head_stride) ||
      off_vector(q_rope, Tq, H, qr_token_stride, qr_head_stride) ||
      (Tk > 0 && (off_vector(k_nope, Tk, H, kn_token_stride, kn_head_stride) ||
                  off_vector(v, Tk, H, v_token_stride, v_head_stride) ||
                  off_vector(k_rope, Tk, 1, kr_token_stride, kRope))) ||
      !aligned(out, 16) || (num_parts > 0 && (!aligned(O_part, 16) || !aligned(LSE_part, 4))) ||
      !aligned(cu_q, 4) || !aligned(cu_kv, 4) || (prefix && !aligned(prefix, 4)) || !aligned(work, 4) ||
      (lse && !aligned(lse, 4)) || (status && !aligned(status, 4)))
    return fail(MLA_ERR_MISALIGNED, "mla_prefill: queries, keys, values, out and O_part need 16-B alignment "
                "(strides a multiple of 8 elements), the other arrays 4-B");
  if (Tk == 0) {  // no keys: the maps are never read through
    k_nope = k_rope = v = out;
    kn_token_stride = kn_head_stride = v_token_stride = v_head_stride = kNope;
    kr_token_stride = kRope;
  }
  CUtensorMap qn, qr, kn, kr, vm;
  int rc = head_map(&qn, q_nope, kNope, H, Tq, qn_token_stride, qn_head_stride);
  if (rc == MLA_OK) rc = head_map(&qr, q_rope, kRope, H, Tq, qr_token_stride, qr_head_stride);
  if (rc == MLA_OK) rc = head_map(&kn, k_nope, kNope, H, Tk, kn_token_stride, kn_head_stride);
  if (rc == MLA_OK) rc = head_map(&kr, k_rope, kRope, 1, Tk, kr_token_stride, kRope);
  if (rc == MLA_OK) {
    // 64 tokens x 128 dims as two halves of 64 dims, one after the other
    const uint64_t d[4] = {64, (uint64_t)std::max<int64_t>(Tk, 1), 2, (uint64_t)H};
    const uint64_t st[3] = {(uint64_t)(Tk > 1 ? v_token_stride : (int64_t)H * kValue) * 2, 128,
                            (uint64_t)(H > 1 ? v_head_stride : kValue) * 2};
    const uint32_t box[4] = {64, 64, 2, 1};
    rc = make_tensor_map_bf16_4d(&vm, v, d, st, box);
  }
  if (rc != MLA_OK) return rc;
  PrefillParams p{cu_q, cu_kv, prefix, N, H, causal != 0, Tq, Tk, sm_scale, sm_scale * kLog2e, work,
                  num_work, num_parts, O_part, LSE_part, static_cast<__nv_bfloat16*>(out), lse, status};
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaFuncSetAttribute(mla_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(mla_prefill_kernel)");
  const unsigned grid = (unsigned)num_work * (unsigned)H;
  mla_prefill_kernel<<<grid, kThreads, kSmem, st>>>(qn, qr, kn, kr, vm, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_prefill_kernel");
  if (num_parts > 0) {
    mla_prefill_merge_kernel<<<grid, 256, 0, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "launch mla_prefill_merge_kernel");
  }
  return MLA_OK;
}
