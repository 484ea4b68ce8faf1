// mla_prefill.cu -- attention within packed prompts before absorption
// (mla_prefill): per head s = scale (q_nope . k_nope + q_rope . k_rope), one
// RoPE key for all heads, and o = softmax(s) v over the keys that a row sees,
// which are always the first ones of its sequence.
//
// Two forms of one kernel.  A work unit is a block of rows of one sequence and head:
// 128 rows on one CTA with one row tile (kCtas = 1; two CTAs share an SM, so that one's
// loads and softmax overlap the other's MMAs), or 512 rows on a pair of CTAs with two
// row tiles each, whose MMAs span both SMs (cta_group::2).  A row tile has 128 rows of
// a CTA; keys come in tiles of 128 tokens: S = Q K^T is 12 MMAs of N = 128, K = 16 (192
// dims), O += P V eight more.  TMEM holds S and O of a row tile (128 columns each); P
// overwrites its S in bf16 and is the MMA's A operand from there.  In a pair, while the
// softmax of one row tile runs, the tensor cores work for the other: PV_0(t - 1),
// QK_0(t), PV_1(t - 1), QK_1(t), ...  MMAs of one thread execute in order, so "S_g(t)
// is there" also says that PV_g(t - 1) is done: the softmax may rescale O in place
// then, and S may overwrite P.
//
// What bounds it (GB300).  Pairs: the tensor cores under the power cap, one prompt of
// 8191 tokens x 96 heads (2.06 TFLOP) in 1172 to 1251 us, 1.65 to 1.75 PFLOP/s, 86 to 92% of
// the measured burst and 96 to 102% of the measured sustained rate, tensor pipe active 78%
// of the cycles; each SM loads and reads half of every K and V tile (40 KB).  On single
// CTAs a row tile's 80 KB of keys and values a tile come in through a ring of 64 KB, so a
// tile waits for loads that are issued as the one before is used up: 64 documents of 33
// to 700 tokens x 96 heads 348 us, 1.62 GB moved, 69% of the copy rate.  A block of 512
// rows of a short sequence would mostly be padding (558 us).
//
//   softmax warps    4 a row tile, one thread per row, then O / l
//   TMA warp         K and V through the ring; on one CTA Q (48 KB) too
//   Q warp           a pair's Q (96 KB a CTA)
//   MMA warp         of a pair's first CTA; runs converged, one lane issues
//   next unit's warp the grid has a CTA (pair) per unit, and running ones take over
//                    those that have not started, in launch order, so the work list is
//                    dealt out as SMs come free and a unit's loads and first MMAs
//                    overlap the end of the one before
//   cleaning warps   clean V: in tiles that hold tokens which some row of the unit
//                    does not see, values that are not finite become 0 (P is 0
//                    there, and 0 x NaN would reach the row) and are noted per
//                    dim; the rows that do see them get them back at the end
//
// Softmax in base 2 with fp32 statistics; O is rescaled only when a row's
// maximum has risen by more than 2^8, so P stays below 2^8 and its rounding to
// bf16 is 2^-8 of each probability either way.  A pair's softmax hands P over in two
// halves, so that PV starts on the first (1414 -> 1298 us); on one CTA, where the
// other CTA fills the gap, the second handshake costs more than it gives (350, 360).
//
// Code size matters as much as any of this: the warps' loops are long and different,
// and at 118 KB of code everything ran at half its speed for want of instructions
// (1414 us and 434 with 66 KB, 1215 and 347 with 55): waits are a few instructions
// each, rare paths loop instead of being unrolled.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "mla_tma.cuh"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kRows = 128;           // rows of a CTA's tile (MMA M per CTA)
constexpr int kSlot = 128;           // rows of a workspace slot, two to a part of the caller's
constexpr int kKeys = 128;           // tokens of a key tile
constexpr int kBox = 128 * 128;      // 16 KB: 64 dims of 128 rows
constexpr int kVBytes = 2 * kBox;    // V of a tile
constexpr int kRaw = 4;              // pieces of V that may wait for cleaning
// The softmax warps take 200 registers a thread, the others 56: as many threads of
// each kind, 128 on average, as the kernels launch with.
constexpr int kRegsSoftmax = 200, kRegsOther = 56;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kRise = 8.f;         // log2 of the rise that rescales O
constexpr int kEntry = 8;            // int32 of a work entry

// A form of the kernel: kCtas CTAs a unit, each with kTiles row tiles.  The ring's
// pieces, each with its barriers: on one CTA a box of 16 KB (64 dims of K or 64
// tokens of V); in a pair a CTA's half of a tile's K (24 KB) or V (16 KB).
template <int kCtas>
struct Form {
  static constexpr int kTiles = kCtas;
  static constexpr int kBlock = kTiles * kRows * kCtas;                   // rows of a unit
  static constexpr int kSoftmax = 4 * kTiles;                             // warps; the others after them
  static constexpr int kTma = kSoftmax, kMma = kTma + 1, kNext = kTma + 2, kClean = kTma + (kCtas == 1 ? 3 : 4);
  static constexpr int kCleaners = kCtas;
  static constexpr int kThreads = 2 * 32 * kSoftmax;
  static constexpr int kK = kCtas == 1 ? 3 : 1, kV = kCtas == 1 ? 2 : 1;  // pieces of a tile
  static constexpr int kTile = kK + kV, kAll = kCtas == 1 ? 4 : 6;
  static constexpr int kHalfBox = kBox / kCtas;                           // 64 dims of a CTA's tokens of K
  static constexpr int kQBytes = 3 * kTiles * kBox, kRing = kCtas == 1 ? 4 * kBox : 15 * kHalfBox;
  static constexpr uint32_t kColumns = 256 * kTiles;                      // tensor memory: S, then O of the row tiles
  static __device__ __forceinline__ uint32_t at(uint32_t piece) {
    return kCtas == 1 ? piece * kBox : (piece >> 1) * (5 * kHalfBox) + (piece & 1) * (3 * kHalfBox);
  }
};
// Where a role stands in the ring.
template <int kCtas>
struct Cursor {
  uint32_t piece, phase;
  __device__ __forceinline__ void next() {
    if (++piece == Form<kCtas>::kAll) piece = 0, phase ^= 1;
  }
  __device__ __forceinline__ void next_tile() {
    piece += Form<kCtas>::kTile;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (piece >= Form<kCtas>::kAll) piece -= Form<kCtas>::kAll, phase ^= 1;
  }
};

// Tensor maps; [1]: boxes of 32 rows, for the ends of sequences (one CTA).
struct PrefillMaps {
  CUtensorMap qn[2], qr[2], kn[2], kr[2], v[2];
};
constexpr int kFew = 32, kFewBytes = kFew * 128;

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
  int ends;                // maps of 32 rows are there
};

// A work unit: `rows` rows from row0 of a sequence (first row q0, first key k0,
// lq rows and lk keys), head h, key tiles j0 <= j < j1 of which the two row
// tiles see those below n0 and n1.
struct Unit {
  int more;                 // 0: no further unit
  int h, row0, rows, q0, k0, lq, lk, prefix;
  int slot;                 // workspace slot of this part, -1: the whole block
  int j0, j1, n0, n1;
  int clean0;               // first tile whose V is cleaned
  int unseen;               // first key that some row does not see
  int end;                  // keys that some row sees
};

// Notes on cleaned values: per kind (NaN, +inf, -inf) and dim the first such token,
// counted from the unit's first unseen one (below the unit's rows).  Kept apart
// from those of earlier units by a tag of the unit's number among the CTA's cleaned
// ones (`nth`, counted alike by the warps that clean and those that read): in a pair
// one that falls, so that one minimum replaces older notes; on one CTA, which has less
// shared memory, all of a dim's in one word under a tag that comes again after 127
// cleaned units, the notes being wiped in between.
template <int kCtas>
struct Notes;
template <>
struct Notes<2> {
  static constexpr int kPastBits = 9;
  uint32_t first[3][kKeys];
  static __device__ __forceinline__ uint32_t tag(uint32_t nth) { return (0x7fffffu - nth) << kPastBits; }
  __device__ __forceinline__ void clear(int dim) { first[0][dim] = first[1][dim] = first[2][dim] = ~0u; }
  __device__ __forceinline__ void add(uint32_t nth, int kind, int dim, uint32_t past, uint32_t rank) {
    atomicMin(&first[kind][dim], tag(nth) | past);
    red_min_cluster_u32(mapa(smem_u32(&first[kind][dim]), rank ^ 1), tag(nth) | past);
  }
  __device__ __forceinline__ bool below(uint32_t nth, int kind, int dim, uint32_t reach) const {
    return first[kind][dim] < tag(nth) + reach;
  }
};
template <>
struct Notes<1> {
  uint32_t word[kKeys];
  static constexpr uint32_t kWipe = 127;
  static __device__ __forceinline__ uint32_t tag(uint32_t nth) { return (nth % kWipe + 1) << 24; }
  __device__ __forceinline__ void clear(int dim) { word[dim] = 0; }
  __device__ __forceinline__ void add(uint32_t nth, int kind, int dim, uint32_t past, uint32_t) {
    uint32_t old = word[dim];
    for (;;) {
      const uint32_t mine = old >> 24 == tag(nth) >> 24 ? old : tag(nth) | 0xffffffu;
      const uint32_t least = min(mine >> (8 * kind) & 0xffu, past);
      const uint32_t next = (mine & ~(0xffu << (8 * kind))) | least << (8 * kind);
      const uint32_t seen = atomicCAS(&word[dim], old, next);
      if (seen == old) return;
      old = seen;
    }
  }
  __device__ __forceinline__ bool below(uint32_t nth, int kind, int dim, uint32_t reach) const {
    return word[dim] >> 24 == tag(nth) >> 24 && (word[dim] >> (8 * kind) & 0xffu) < reach;
  }
};

template <int kCtas>
struct Ctl {
  static constexpr int kTiles = Form<kCtas>::kTiles, kAll = Form<kCtas>::kAll;
  uint64_t q[kTiles], qfree[kTiles];  // Q of a row tile has landed; has been used up
  uint64_t full[kAll], empty[kAll];   // ring
  uint64_t s[kTiles];                 // S of a row tile is in TMEM
  uint64_t p[kTiles][2];              // its P of the tile's first and last 64 keys is, S has been read
                                      // (on one CTA all of it, by [1])
  uint64_t o[kTiles];                 // O is complete
  uint64_t raw[kRaw];                 // V of a tile to be cleaned has landed (tiles take turns)
  uint64_t cleaned;                   // all of a unit's are clean
  uint64_t done;                      // the softmax warps are through with a unit
  uint64_t unit_full[2], unit_empty[2];
  uint64_t answer_full, answer_free;
  uint64_t drain;
  alignas(16) uint32_t answer[4];
  Unit unit[2];
  uint32_t note;                      // where a peer's asynchronous stores go
  uint32_t tmem;
  int abort_flag;
  uint32_t any_odd;                   // the last cleaned unit with notes, counted from 1
  Notes<kCtas> notes;
};
template <int kCtas>
constexpr int kSmem = Form<kCtas>::kQBytes + Form<kCtas>::kRing + (int)sizeof(Ctl<kCtas>);
static_assert(kSmem<1> <= 113 * 1024, "shared memory of two CTAs an SM");
static_assert(kSmem<2> <= 227 * 1024, "shared memory budget");

// Keys that row i of a sequence sees.
__device__ __forceinline__ int sees(const PrefillParams& p, int lq, int lk, int prefix, int i) {
  if (!p.causal) return lk;
  return min(lk, max(prefix, max(lk - lq + 1 + i, 0)));
}

// Unit x of the grid; false if its entry or lengths are none.
template <int kCtas>
__device__ __forceinline__ bool find_unit(const PrefillParams& p, int x, Unit& u) {
  constexpr int kBlock = Form<kCtas>::kBlock, kStride = kEntry * kCtas;
  const int32_t* e = p.work + (int64_t)(x / p.H) * kStride;
  const int g0 = e[5], nb = e[6];
  if (g0 < 0 || nb < 1 || g0 > x / p.H || g0 + nb <= x / p.H || g0 + nb > p.num_work) {
    if (p.status) atomicOr(p.status, MLA_STATUS_BAD_WORK);
    return false;
  }
  const uint32_t local = (uint32_t)(x - (int64_t)g0 * p.H);  // below nb * H <= 2^30
  u.h = (int)(local / (uint32_t)nb);
  e = p.work + (int64_t)(g0 + (int)(local % (uint32_t)nb)) * kStride;
  const int seq = e[0], part = e[2], parts = e[3], slot = e[4];
  const int64_t row0 = (int64_t)e[1] * kBlock;
  if (u.h >= p.H || seq < 0 || seq >= p.N || e[1] < 0 || parts < 1 || parts > MLA_PREFILL_MAX_PARTS ||
      part < 0 || part >= parts || e[7] != kBlock ||
      (parts > 1 && (slot < 0 || slot > 2 * (int64_t)p.num_parts - parts * (kBlock / kSlot)))) {
    if (p.status) atomicOr(p.status, MLA_STATUS_BAD_WORK);
    return false;
  }
  const int64_t q0 = p.cu_q[seq], k0 = p.cu_kv[seq];
  const int64_t lq = p.cu_q[seq + 1] - q0, lk = p.cu_kv[seq + 1] - k0;
  const int prefix = p.prefix ? p.prefix[seq] : 0;
  if (q0 < 0 || k0 < 0 || lq < 0 || lk < 0 || q0 + lq > p.Tq || k0 + lk > p.Tk || row0 >= lq) {
    const bool length = q0 < 0 || k0 < 0 || lq < 0 || lk < 0 || q0 + lq > p.Tq || k0 + lk > p.Tk;
    if (p.status) atomicOr(p.status, length ? MLA_STATUS_BAD_LENGTH : MLA_STATUS_BAD_WORK);
    return false;
  }
  u.more = 1;
  u.row0 = (int)row0;
  u.rows = (int)min((int64_t)kBlock, lq - row0);
  u.q0 = (int)q0, u.k0 = (int)k0, u.lq = (int)lq, u.lk = (int)lk, u.prefix = prefix;
  u.slot = parts > 1 ? slot + part * (kBlock / kSlot) : -1;
  const auto tiles = [&](int first, int end) {
    if (u.rows <= first) return 0;
    return (sees(p, u.lq, u.lk, prefix, u.row0 + min(u.rows, end) - 1) + kKeys - 1) / kKeys;
  };
  constexpr int kTileRows = kBlock / Form<kCtas>::kTiles;
  const int n0 = tiles(0, kTileRows), n1 = Form<kCtas>::kTiles == 1 ? n0 : tiles(kTileRows, kBlock);
  const uint32_t all = (uint32_t)max(n0, n1);  // at most 2^24, parts at most 32
  u.j0 = (int)(all * (uint32_t)part / (uint32_t)parts);
  u.j1 = (int)(all * (uint32_t)(part + 1) / (uint32_t)parts);
  u.n0 = min(n0, u.j1);
  u.n1 = min(n1, u.j1);
  u.unseen = sees(p, u.lq, u.lk, prefix, u.row0);
  u.end = sees(p, u.lq, u.lk, prefix, u.row0 + u.rows - 1);
  u.clean0 = max(u.j0, u.unseen / kKeys);
  return true;
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


// ---- the two forms' instructions
// Waits are inlined (a kernel that rebalances its registers makes no calls), so
// their code is kept short: the kernel's loops have to fit the instruction cache.
// A CTA's own barriers are waited for at CTA scope, also where tensor memory or TMA
// data of the pair is behind them: at cluster scope a wait takes about 170 cycles
// more.  kWide: data that the other CTA's threads have written is behind it.
__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
template <bool kWide = false>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t at = smem_u32(bar);
  uint32_t t0 = 0;
#pragma unroll 1
  while (!(kWide ? mbar_try_wait_suspend(at, parity, kSuspendNs)
                 : mbar_try_wait_suspend_cta(at, parity, kSuspendNs))) {
    if (*abort) return false;
    const uint32_t now = globaltimer_lo() | 1;
    if (t0 == 0) t0 = now;
    if (now - t0 > (uint32_t)kWaitNs) return false;
  }
  return true;
}
// A barrier of the pair's first CTA, which issues the MMAs.
template <int kCtas>
__device__ __forceinline__ uint32_t lead_bar(uint64_t* bar) {
  if constexpr (kCtas == 1) return smem_u32(bar);
  else return mapa(smem_u32(bar), 0);
}
template <int kCtas>
__device__ __forceinline__ void mma_qk(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  constexpr uint32_t idesc = idesc_bf16_f32(kRows * kCtas, kKeys, false, false);
  if constexpr (kCtas == 1) mma_ss(d, a, b, idesc, acc);
  else mma_ss_pair(d, a, b, idesc, acc);
}
template <int kCtas>
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
  constexpr uint32_t idesc = idesc_bf16_f32(kRows * kCtas, kKeys, false, true);
  if constexpr (kCtas == 1) mma_ts(d, a, b, idesc, acc);
  else mma_ts_pair(d, a, b, idesc, acc);
}
// A descriptor some 16-byte units on (the address field never carries out).
__device__ __forceinline__ uint64_t plus(uint64_t desc, uint32_t n) {
  return (desc & 0xffffffff00000000ull) | (uint32_t)((uint32_t)desc + n);
}
// On the barrier of every CTA of the unit.
template <int kCtas>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (kCtas == 1) mma_commit(smem_u32(bar));
  else mma_commit_pair(smem_u32(bar), 3);
}

template <int kCtas>
__device__ __forceinline__ void give_up(Ctl<kCtas>& c, const PrefillParams& p, uint32_t rank) {
  *reinterpret_cast<volatile int*>(&c.abort_flag) = 1;
  if constexpr (kCtas == 2) st_cluster_u32(mapa(smem_u32(&c.abort_flag), rank ^ 1), 1);
  if (p.status) atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
}

// The units of a role, one after another: next() waits for one, release() hands
// its slot back (one lane).
template <int kCtas>
struct Units {
  Ctl<kCtas>& c;
  uint32_t nth = 0;
  __device__ __forceinline__ explicit Units(Ctl<kCtas>& ctl) : c(ctl) {}
  __device__ __forceinline__ const Unit* next(bool& ok) {
    ok = wait_bar(&c.unit_full[nth & 1], nth >> 1 & 1, &c.abort_flag);
    const Unit* u = &c.unit[nth & 1];
    return ok && u->more ? u : nullptr;
  }
  __device__ __forceinline__ void release() {
    mbar_arrive(smem_u32(&c.unit_empty[nth & 1]));
    ++nth;
  }
  __device__ __forceinline__ void skip() { ++nth; }  // for the other lanes
};

// Finds the units and hands them to the CTA's roles: its own first, then those
// it takes over, asked for one unit ahead.
template <int kCtas>
__device__ __forceinline__ void feed(Ctl<kCtas>& c, const PrefillParams& p, uint32_t rank) {
  int x = blockIdx.x / kCtas;
  uint32_t nth = 0, asked = 0;
  bool ok = true;
  while (ok) {
    Unit u;
    u.more = 0;
    const bool found = x >= 0 && find_unit<kCtas>(p, x, u);
    if (found || x < 0) {
      const uint32_t b = nth & 1;
      // (its slot was free before this unit was asked for)
      c.unit[b] = u;
      mbar_arrive(smem_u32(&c.unit_full[b]));
      if (x < 0) return;
      ++nth;
      // one ahead: the unit before this one has ended
      if (nth >= 2 && !(ok = wait_bar(&c.unit_empty[nth & 1], (nth >> 1) - 1 & 1, &c.abort_flag))) break;
    }
    mbar_arrive_expect_tx(smem_u32(&c.answer_full), 16);
    if (rank == 0) {
      // every CTA has armed its barrier and read the answer before
      if (kCtas == 2 && !(ok = wait_bar<true>(&c.answer_free, asked & 1, &c.abort_flag))) break;
      try_cancel<kCtas == 2>(smem_u32(c.answer), smem_u32(&c.answer_full));
    } else {
      mbar_arrive_cluster(mapa(smem_u32(&c.answer_free), 0));
    }
    if (!(ok = wait_bar<kCtas == 2>(&c.answer_full, asked & 1, &c.abort_flag))) break;
    ++asked;
    x = canceled_cta(smem_u32(c.answer));
    // the answer has been read before the next one is written
    fence_proxy_async_smem();
    if (x >= 0) x /= kCtas;
  }
  give_up<kCtas>(c, p, rank);
}

// Where a unit's keys and values go through the ring: on one CTA, box by box.  Q
// comes after the first keys.  At the ends of sequences only what some row needs is
// loaded, in 32 rows: with sequences of a few hundred tokens the rest of a tile,
// the next sequence's, would be a third more traffic (64 documents: 1.49 GB of reads
// for 1.15).  What stays in shared memory there is masked, or cleaned.
__device__ __forceinline__ void produce_one(uint8_t* base, Ctl<1>& c, const PrefillParams& p, const PrefillMaps& m,
                                            int lane) {
  using F = Form<1>;
  const auto v_boxes = [&](int left) { return left > kFew || !p.ends ? 1 : left > 0 ? 2 : 0; };
  const auto v_bytes = [&](int left) { return left > kFew || !p.ends ? kBox : left > 0 ? 2 * kFewBytes : 0; };
  Units<1> units(c);
  bool ok = true;
  uint32_t pos = 0, cleans = 0, uses = 0;
  while (const Unit* u = units.next(ok)) {
    const int h = u->h, k0 = u->k0, j0 = u->j0, j1 = u->j1, clean0 = u->clean0, end = u->end;
    const int row = u->q0 + u->row0, rows = u->rows;
#pragma unroll 1
    for (int j = j0; j < j1 && ok; ++j) {
      const int left = end - j * kKeys;
#pragma unroll 1
      for (int i = 0; i < F::kTile; ++i, ++pos) {
        if (j == j0 && i == F::kK) {
          if (uses > 0 && !(ok = wait_bar(&c.qfree[0], (uses - 1) & 1, &c.abort_flag))) break;
          ++uses;
          const int few = p.ends && rows <= kRows - kFew, n = few ? (rows + kFew - 1) / kFew : 1;
          if (lane == 0) mbar_arrive_expect_tx(smem_u32(&c.q[0]), 3 * (few ? n * kFewBytes : kBox));
          __syncwarp();
          if (lane < 3 * n) {
            const int box = lane % 3, part = lane / 3;
            tma_load_3d(smem_u32(base + box * kBox + part * kFewBytes), box < 2 ? &m.qn[few] : &m.qr[few],
                        smem_u32(&c.q[0]), box < 2 ? box * 64 : 0, h, row + part * kFew);
          }
          __syncwarp();
        }
        const uint32_t piece = pos % F::kAll, use = pos / F::kAll;
        if (use > 0 && !(ok = wait_bar(&c.empty[piece], (use - 1) & 1, &c.abort_flag))) break;
        const uint32_t dst = smem_u32(base + F::kQBytes + F::at(piece));
        uint32_t bar = smem_u32(&c.full[piece]);
        if (i < F::kK) {
          const int few = p.ends && left <= kKeys - kFew, n = few ? (left + kFew - 1) / kFew : 1;
          if (lane == 0) mbar_arrive_expect_tx(bar, few ? n * kFewBytes : kBox);
          __syncwarp();
          if (lane < n)
            tma_load_3d(dst + lane * kFewBytes, i < 2 ? &m.kn[few] : &m.kr[few], bar, i < 2 ? i * 64 : 0,
                        i < 2 ? h : 0, k0 + j * kKeys + lane * kFew);
        } else {
          const int first = (i - F::kK) * 64, n = v_boxes(left - first);
          if (j >= clean0) {
            // its piece is full once it is clean; also one that gets nothing has to be
            // free before it is cleaned
            bar = smem_u32(&c.raw[(cleans + (j - clean0)) % kRaw]);
            if (lane == 0 && n > 0) mbar_arrive_expect_tx(bar, v_bytes(left - first));
            if (lane == 0 && n == 0) mbar_arrive(bar);
          } else if (lane == 0) {
            mbar_arrive_expect_tx(bar, kBox);  // (every row sees all of the tile)
          }
          __syncwarp();
          if (lane < n)
            tma_load_4d(dst + lane * (kBox / 2), &m.v[n == 1 ? 0 : 1], bar, 0, k0 + j * kKeys + first, lane, h);
        }
        __syncwarp();
      }
    }
    if (!ok) break;
    cleans += max(j1 - clean0, 0);
    if (lane == 0) units.release(); else units.skip();
  }
  if (!ok && lane == 0) give_up<1>(c, p, 0);
  // After an abort: every load issued has landed before the CTA may exit (without
  // one, the MMAs have used them all).
  if (!ok) {
    int never = 0;
    if (uses > 0) wait_bar(&c.q[0], (uses - 1) & 1, &never);
    for (uint32_t k = pos > (uint32_t)F::kAll ? pos - F::kAll : 0; k < pos; ++k)
      wait_bar(&c.full[k % F::kAll], (k / F::kAll) & 1, &never);
  }
}

// The same for a pair: a CTA loads its half of a tile's tokens (K) or dims (V); the
// first CTA expects both CTAs' bytes.
__device__ __forceinline__ void produce_pair(uint8_t* base, Ctl<2>& c, const PrefillParams& p, const PrefillMaps& m,
                                             uint32_t rank, int lane) {
  using F = Form<2>;
  Units<2> units(c);
  bool ok = true;
  uint32_t pos = 0, cleans = 0;
  while (const Unit* u = units.next(ok)) {
    const int h = u->h, k0 = u->k0, j0 = u->j0, j1 = u->j1, clean0 = u->clean0;
#pragma unroll 1
    for (int j = j0; j < j1 && ok; ++j) {
      const int tok = k0 + j * kKeys;
#pragma unroll 1
      for (int i = 0; i < F::kTile; ++i, ++pos) {
        const uint32_t piece = pos % F::kAll, use = pos / F::kAll;
        if (use > 0 && !(ok = wait_bar(&c.empty[piece], (use - 1) & 1, &c.abort_flag))) break;
        const uint32_t dst = smem_u32(base + F::kQBytes + F::at(piece)), bar = lead_bar<2>(&c.full[piece]);
        if (i == 0) {
          if (lane == 0 && rank == 0) mbar_arrive_expect_tx(smem_u32(&c.full[piece]), 3 * kBox);
          __syncwarp();
          if (lane < 3)  // a box a lane
            tma_load_3d_pair(dst + lane * F::kHalfBox, lane < 2 ? &m.kn[0] : &m.kr[0], bar, lane < 2 ? lane * 64 : 0,
                             lane < 2 ? h : 0, tok + (int)rank * (kKeys / 2));
        } else if (lane == 0) {
          if (j >= clean0) {
            // its piece is full once it is clean
            const uint32_t raw = smem_u32(&c.raw[(cleans + (j - clean0)) % kRaw]);
            mbar_arrive_expect_tx(raw, kVBytes / 2);
            tma_load_4d(dst, &m.v[0], raw, 0, tok, (int)rank, h);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&c.full[piece]), kVBytes);
            tma_load_4d_pair(dst, &m.v[0], bar, 0, tok, (int)rank, h);
          }
        }
        __syncwarp();
      }
    }
    if (!ok) break;
    cleans += max(j1 - clean0, 0);
    if (lane == 0) units.release(); else units.skip();
  }
  if (!ok && lane == 0) give_up<2>(c, p, rank);
  if (!ok) {
    int never = 0;
    for (uint32_t k = pos > (uint32_t)F::kAll ? pos - F::kAll : 0; rank == 0 && k < pos; ++k)
      wait_bar(&c.full[k % F::kAll], (k / F::kAll) & 1, &never);
  }
}

// A pair's Q has a warp of its own: it waits for the unit before to have used its
// up, which keys and values need not.  Three boxes for each row tile.
__device__ __forceinline__ void load_queries(uint8_t* base, Ctl<2>& c, const PrefillParams& p, const PrefillMaps& m,
                                             uint32_t rank, int lane) {
  Units<2> units(c);
  bool ok = true;
  uint32_t uses[2] = {0, 0};
  while (const Unit* u = units.next(ok)) {
    const int h = u->h, row = u->q0 + u->row0, j0 = u->j0;
    const int n[2] = {u->n0, u->n1};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (n[g] <= j0) continue;
      if (uses[g] > 0) ok = ok && wait_bar(&c.qfree[g], (uses[g] - 1) & 1, &c.abort_flag);
      if (!ok) break;
      ++uses[g];
      if (lane == 0 && rank == 0) mbar_arrive_expect_tx(smem_u32(&c.q[g]), 3 * kBox * 2);
      __syncwarp();
      if (lane < 3)
        tma_load_3d_pair(smem_u32(base + (3 * g + lane) * kBox), lane < 2 ? &m.qn[0] : &m.qr[0], lead_bar<2>(&c.q[g]),
                         lane < 2 ? lane * 64 : 0, h, row + (g * 2 + (int)rank) * kRows);
      __syncwarp();
    }
    if (!ok) break;
    if (lane == 0) units.release(); else units.skip();
  }
  if (!ok && lane == 0) give_up<2>(c, p, rank);
  // After an abort: every load issued has landed before the CTA may exit.
  if (!ok && rank == 0) {
    int never = 0;
    for (int g = 0; g < 2; ++g)
      if (uses[g] > 0) wait_bar(&c.q[g], (uses[g] - 1) & 1, &never);
  }
}

// The whole warp runs the loop, so that what the MMAs take stays in uniform
// registers; one lane issues.
template <int kCtas>
__device__ __forceinline__ void issue_mmas(uint8_t* base, Ctl<kCtas>& c, const PrefillParams& p, uint32_t tmem, int lane) {
  using F = Form<kCtas>;
  const uint64_t qd = sdesc_sw128(smem_u32(base), 16, 1024);
  const uint64_t kd = sdesc_sw128(smem_u32(base + F::kQBytes), 16, 1024);
  // V: MN-major, the next 64 dims 8 KB (LBO) on, the next 8 tokens 1 KB (SBO) on,
  // the next 16 tokens 2 KB; P: 16 tokens in 8 columns
  const uint64_t vd = sdesc_sw128(smem_u32(base + F::kQBytes), kBox / 2, 1024);
  const bool lead = elect_one();
  bool ok = true;
  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && __all_sync(~0u, wait_bar(bar, parity, &c.abort_flag));
    return ok;
  };
  Units<kCtas> units(c);
  Cursor<kCtas> kc{0, 0}, vc{F::kK, 0};         // K(t) and V(t - 1)
  uint32_t ps0 = 0, ps1 = 0, qs0 = 0, qs1 = 0;  // tiles and units of each row tile so far
  while (const Unit* u = units.next(ok)) {
    const int j0 = __shfl_sync(~0u, u->j0, 0), tiles = __shfl_sync(~0u, u->j1, 0) - j0;
    const int a0 = __shfl_sync(~0u, u->n0, 0) - j0, a1 = __shfl_sync(~0u, u->n1, 0) - j0;
    const int clean = kCtas == 1 ? 0x7fffffff : __shfl_sync(~0u, u->clean0, 0) - j0;
#pragma unroll 1
    for (int t = 0; t <= tiles && ok; ++t) {
#pragma unroll 1
      for (int g = 0; g < F::kTiles; ++g) {
        const uint32_t s = tmem + g * kKeys, o = tmem + (F::kTiles + g) * kKeys;
        const int a = g ? a1 : a0;
        if (t > 0 && t - 1 < a) {
          Cursor<kCtas> at = vc;
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // 64 tokens
            if ((F::kV == 2 || i == 0) && (g == 0 || t - 1 >= a0)) {
              if (!wait(&c.full[at.piece], at.phase)) break;
              // cleaned by the other CTA's threads, too
              if (kCtas == 2 && t - 1 >= clean) fence_cluster();
            }
            if ((kCtas == 2 || i == 0) && !wait(&c.p[g][kCtas == 1 ? 1 : i], ((g ? ps1 : ps0) + t - 1) & 1)) break;
            tc_fence_after();
            if (lead) {
              const uint64_t b = plus(vd, (F::at(at.piece) + (F::kV == 1 ? i * F::kHalfBox : 0)) >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_pv<kCtas>(o, s + (4 * i + k) * 8, plus(b, 128 * k), (t > 1 || i || k) ? 1u : 0u);
              if ((F::kV == 2 || i == 1) && (g + 1 == F::kTiles || t - 1 >= a1)) commit<kCtas>(&c.empty[at.piece]);
            }
            if (F::kV == 2) at.next();
          }
          if (!ok) break;
          if (lead && t == a) commit<kCtas>(&c.o[g]);
        }
        if (t < a) {
          if (t == 0 && !wait(&c.q[g], (g ? qs1 : qs0) & 1)) break;
          Cursor<kCtas> at = kc;
#pragma unroll
          for (int i = 0; i < F::kK; ++i, at.next()) {
            if ((g == 0 || t >= a0) && !wait(&c.full[at.piece], at.phase)) break;
            if (lead) {
              const uint64_t q = plus(qd, (3 * g + i) * (kBox >> 4)), b = plus(kd, F::at(at.piece) >> 4);
#pragma unroll
              for (int k = 0; k < 12 / F::kK; ++k)
                mma_qk<kCtas>(s, plus(q, k / 4 * (kBox >> 4) + 2 * (k % 4)),
                              plus(b, k / 4 * (F::kHalfBox >> 4) + 2 * (k % 4)), (i || k) ? 1u : 0u);
              if (g + 1 == F::kTiles || t >= a1) commit<kCtas>(&c.empty[at.piece]);
            }
          }
          if (!ok) break;
          if (lead) {
            commit<kCtas>(&c.s[g]);
            if (t == a - 1) commit<kCtas>(&c.qfree[g]);
          }
        }
      }
      if (t < tiles) kc.next_tile();
      if (t > 0) vc.next_tile();
    }
    if (!ok) break;
    if (a0 > 0) ps0 += a0, ++qs0;
    if (F::kTiles == 2 && a1 > 0) ps1 += a1, ++qs1;
    __syncwarp();
    if (lead) units.release(); else units.skip();
  }
  if (!ok && lead) give_up<kCtas>(c, p, 0);
  // No MMA may still run when the accumulators are freed.
  int never = 0;
  if (lead) commit<kCtas>(&c.drain);
  wait_bar(&c.drain, 0, &never);
}

// Tiles from u.clean0 on hold tokens that some row does not see (its own later
// ones, or the next sequence's).  A warp cleans 16 KB at a time: on one CTA a
// tile's pieces one after the other; a pair's two warps take turns with the tiles.
template <int kCtas>
__device__ __forceinline__ void clean_values(uint8_t* base, Ctl<kCtas>& c, const PrefillParams& p, uint32_t rank, int i,
                                             int lane) {
  using F = Form<kCtas>;
  constexpr int kBatch = 8, kVecs = kBox / 16;  // 16-byte vectors: in flight per lane, of a job
  Units<kCtas> units(c);
  bool ok = true;
  uint32_t at = 0, cleans = 0, turn = 0;  // pieces, cleaned tiles and cleaned units so far
  while (const Unit* u = units.next(ok)) {
    const int j0 = u->j0, j1 = u->j1, clean0 = u->clean0, unseen = u->unseen, lk = u->lk;
    bool read = units.nth == 0;  // the notes on the unit before have been (by both CTAs)
    // `done` is waited for only at a unit that is cleaned: the softmax warps cannot be
    // through with that one, so the phase of the unit before is the last or the present
    // one, and no warp has arrived twice in it.  (They run through units that are not
    // cleaned without these warps; through those without keys not even together.)
    if (kCtas == 1 && j1 > clean0 && turn > 0 && turn % Notes<1>::kWipe == 0) {
      if (!(ok = __all_sync(~0u, read || wait_bar(&c.done, (units.nth - 1) & 1, &c.abort_flag)))) break;
      read = true;
      for (int d = lane; d < kKeys; d += 32) c.notes.clear(d);
      __syncwarp();
    }
#pragma unroll 1
    for (int x = kCtas == 1 ? 2 * clean0 : clean0; x < (kCtas == 1 ? 2 * j1 : j1); ++x) {
      const int j = kCtas == 1 ? x >> 1 : x, half = kCtas == 1 ? x & 1 : 0;
      const uint32_t nth = cleans + (j - clean0);
      if (kCtas == 2 && (nth & 1) != (uint32_t)i) continue;
      if (half == 0 && !(ok = __all_sync(~0u, wait_bar(&c.raw[nth % kRaw], nth / kRaw & 1, &c.abort_flag)))) break;
      const uint32_t piece = (at + F::kTile * (j - j0) + F::kK + half) % F::kAll;
      uint4* box = reinterpret_cast<uint4*>(base + F::kQBytes + F::at(piece));
      const int t0 = j * kKeys + half * 64;  // token of the first row
#pragma unroll 1
      for (int x0 = lane; x0 < kVecs; x0 += 32 * kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) w[b] = box[x0 + 32 * b];
        uint32_t hit = 0;
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          hit |= ((w[b].x & 0x7f807f80u) + 0x00800080u) | ((w[b].y & 0x7f807f80u) + 0x00800080u) |
                 ((w[b].z & 0x7f807f80u) + 0x00800080u) | ((w[b].w & 0x7f807f80u) + 0x00800080u);
        if (!(hit & 0x80008000u)) continue;
        // some value of these is not finite: half (64 dims), row, chunk, swizzled by the row
#pragma unroll 1
        for (int e = 0; e < 8 * kBatch; ++e) {
          const int v = x0 + e / 8 * 32;
          const int dims = kCtas == 1 ? v >> 9 : (int)rank, row = (v >> 3) & (kCtas == 1 ? 63 : 127);
          uint16_t* val = reinterpret_cast<uint16_t*>(box + v) + e % 8;
          const uint32_t bits = *val;
          if ((bits & 0x7f80u) != 0x7f80u || t0 + row < unseen) continue;
          *val = 0;
          const int past = t0 + row - unseen, dim = dims * 64 + ((v & 7) ^ (row & 7)) * 8 + e % 8;
          if (t0 + row < lk && past < F::kBlock) {  // past that no row of the unit sees it
            read = read || wait_bar<kCtas == 2>(&c.done, (units.nth - 1) & 1, &c.abort_flag);
            c.notes.add(turn, bits & 0x7fu ? 0 : bits & 0x8000u ? 2 : 1, dim, past, rank);
            c.any_odd = turn + 1;
            if constexpr (kCtas == 2) st_cluster_u32(mapa(smem_u32(&c.any_odd), rank ^ 1), turn + 1);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (kCtas == 1) mbar_arrive(smem_u32(&c.full[piece]));
        else if (rank == 0) mbar_arrive_expect_tx(smem_u32(&c.full[piece]), 4);
        else st_async_u32(mapa(smem_u32(&c.note), 0), 0, lead_bar<kCtas>(&c.full[piece]));
      }
    }
    if (!ok) break;
    at += F::kTile * (j1 - j0);
    if (j1 > clean0) {
      // not before the softmax warps are through with the unit before, whose phase of
      // `cleaned` they may still have to see
      if (units.nth > 0 &&
          !(ok = __all_sync(~0u, read || wait_bar<kCtas == 2>(&c.done, (units.nth - 1) & 1, &c.abort_flag))))
        break;
      cleans += j1 - clean0;
      ++turn;
      if (lane == 0) {
        mbar_arrive(smem_u32(&c.cleaned));
        if constexpr (kCtas == 2) mbar_arrive_cluster(mapa(smem_u32(&c.cleaned), rank ^ 1));
      }
    }
    __syncwarp();
    if (lane == 0) units.release(); else units.skip();
  }
  if (!ok && lane == 0) give_up<kCtas>(c, p, rank);
}

// Softmax of row tile g, one thread per row, then the row's output.
template <int kCtas>
__device__ __forceinline__ void softmax_rows(Ctl<kCtas>& c, const PrefillParams& p, uint32_t tmem, uint32_t rank, int g,
                                             int warp, int lane) {
  const int r = (warp & 3) * 32 + lane, in_block = (g * kCtas + (int)rank) * kRows + r;
  const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t s_at = tmem + quad + g * kKeys, o_at = tmem + quad + (Form<kCtas>::kTiles + g) * kKeys;
  const uint64_t scale2 = f2pack(p.scale2, p.scale2);
  const uint32_t lead_p = lead_bar<kCtas>(&c.p[g][0]), lead_note = kCtas == 1 ? 0 : mapa(smem_u32(&c.note), 0);
  // half i of a tile's P is in tensor memory
  const auto report = [&](int i) {
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      // a pair's second CTA reports by an asynchronous store, whose completion on
      // the first CTA's barrier is a release at cluster scope (a release arrive
      // costs its round trip); the first CTA's warp 0 arms the barrier for them
      if (kCtas == 1) mbar_arrive(lead_p + 8 * i);
      else if (rank) st_async_u32(lead_note, 0, lead_p + 8 * i);
      else if ((warp & 3) == 0) mbar_arrive_expect_tx(smem_u32(&c.p[g][i]), 16);
      else mbar_arrive(smem_u32(&c.p[g][i]));
    }
  };
  Units<kCtas> units(c);
  bool ok = true;
  uint32_t turns = 0, outs = 0, cleans = 0;  // phases of c.s, c.o and c.cleaned (units cleaned so far)
  while (const Unit* u = units.next(ok)) {
    const int tiles = (g ? u->n1 : u->n0) - u->j0;
    // keys that the row sees, from the unit's first tile on; padding rows: all
    const int seen = in_block < u->rows ? sees(p, u->lq, u->lk, u->prefix, u->row0 + in_block) - u->j0 * kKeys
                                        : 0x7fffffff;
    float ref = -INFINITY, l = 0.f;  // raw scores; sum of 2^((s - ref) scale2)
    for (int t = 0; t < tiles; ++t, ++turns) {
      if (!(ok = wait_bar(&c.s[g], turns & 1, &c.abort_flag))) break;
      tc_fence_after();
      float s[kKeys];
#pragma unroll
      for (int b = 0; b < 4; ++b) tmem_ld32(s_at + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * b]));
      tmem_wait_ld();
      const int last = seen - t * kKeys;  // columns of this tile that the row sees
      if (__any_sync(~0u, last < kKeys)) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int n = last - 32 * b;
          const uint32_t mask = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
#pragma unroll
          for (int e = 0; e < 32; ++e) s[32 * b + e] = mask >> e & 1 ? s[32 * b + e] : -INFINITY;
        }
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
        if (kCtas == 2 || b == 1) report(b);
      }
      float x, y, z, w;
      f2unpack(sum2[0], x, y);
      f2unpack(sum2[1], z, w);
      l = (x + y) + (z + w);
    }
    if (!ok) break;
    if (tiles > 0) {
      if (!(ok = wait_bar(&c.o[g], outs & 1, &c.abort_flag))) break;
      ++outs;
    }
    const bool exists = in_block < u->rows, cleaned = u->j1 > u->clean0, whole = u->slot < 0;
    if (cleaned) {
      if (!(ok = wait_bar<kCtas == 2>(&c.cleaned, cleans & 1, &c.abort_flag))) break;
      ++cleans;
    }
    tc_fence_after();
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const float lse = l > 0.f || l != l ? ref * p.sm_scale + logf(l) : -INFINITY;
    // where the row's output goes: its row of out, or of the part's workspace
    const int64_t row = whole ? ((int64_t)u->q0 + u->row0 + in_block) * p.H + u->h
                              : ((int64_t)(u->slot + in_block / kSlot) * p.H + u->h) * kSlot + in_block % kSlot;
    const int unseen = u->unseen - u->j0 * kKeys;
    // notes of this unit: tokens that the row sees get their values back
    const uint32_t reach = (uint32_t)min(max(seen - unseen, 0), Form<kCtas>::kBlock);
    const uint32_t turn = cleans - 1;
    const bool odd = cleaned && *reinterpret_cast<volatile uint32_t*>(&c.any_odd) == turn + 1;
    __nv_bfloat16* out = p.out + row * MLA_V_HEAD_DIM;
    float* part = p.O_part + row * MLA_V_HEAD_DIM;
    // without a key, or with impossible ones only, 0; in a part these may have left a NaN
    // (0 x inf), which the row's other parts' keys make count
    if (!whole && tiles > 0) l = 1.f;
#pragma unroll 1
    for (int b = 0; b < kKeys; b += 16) {
      uint32_t o[16];
      if (tiles > 0) {
        tmem_ld16(o_at + b, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
      if (exists && whole) {
        uint32_t w[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) w[x] = pack_bf16(__uint_as_float(o[2 * x]), __uint_as_float(o[2 * x + 1]));
        st_global_v8(out + b, w);
      } else if (exists) {
        st_global_v8(part + b, *reinterpret_cast<const uint32_t(*)[8]>(&o[0]));
        st_global_v8(part + b + 8, *reinterpret_cast<const uint32_t(*)[8]>(&o[8]));
      }
      __syncwarp();
    }
    if (odd && exists && l != 0.f) {  // (a row of impossible keys is 0 whatever their values are)
#pragma unroll 1
      for (int e = 0; e < kKeys; ++e) {
        float add = 0.f;
        if (c.notes.below(turn, 0, e, reach)) add = NAN;
        if (c.notes.below(turn, 1, e, reach)) add += INFINITY;
        if (c.notes.below(turn, 2, e, reach)) add -= INFINITY;
        if (add == 0.f) continue;
        if (whole) out[e] = __float2bfloat16(__bfloat162float(out[e]) + add);
        else part[e] += add;
      }
    }
    if (exists) {
      if (!whole) p.LSE_part[row] = lse;
      else if (p.lse) p.lse[row] = lse;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(smem_u32(&c.done));
      if constexpr (kCtas == 2) mbar_arrive_cluster(mapa(smem_u32(&c.done), rank ^ 1));
      units.release();
    } else {
      units.skip();
    }
  }
  if (!ok && lane == 0) give_up<kCtas>(c, p, rank);
}

template <int kCtas>
__global__ void __launch_bounds__(Form<kCtas>::kThreads, kCtas == 1 ? 2 : 1)
    mla_prefill_kernel(const __grid_constant__ PrefillMaps m, const PrefillParams p) {
  extern __shared__ __align__(1024) uint8_t base[];
  using F = Form<kCtas>;
  Ctl<kCtas>& c = *reinterpret_cast<Ctl<kCtas>*>(base + F::kQBytes + F::kRing);
  const int warp = __shfl_sync(~0u, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t rank = kCtas == 1 ? 0 : __shfl_sync(~0u, cluster_ctarank(), 0);
  if (threadIdx.x == 0) {
    c.abort_flag = 0;
    c.any_odd = 0;
    for (int g = 0; g < F::kTiles; ++g) {
      mbar_init(smem_u32(&c.q[g]), 1);
      mbar_init(smem_u32(&c.qfree[g]), 1);
      mbar_init(smem_u32(&c.s[g]), 1);
      for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&c.p[g][i]), 4);
      mbar_init(smem_u32(&c.o[g]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&c.unit_full[i]), 1);
      // TMA (a pair: two warps), MMA, cleaning, softmax
      mbar_init(smem_u32(&c.unit_empty[i]), kCtas + 1 + F::kCleaners + F::kSoftmax);
    }
    for (int i = 0; i < Form<kCtas>::kAll; ++i) {
      mbar_init(smem_u32(&c.full[i]), 1);
      mbar_init(smem_u32(&c.empty[i]), 1);
    }
    for (int i = 0; i < kRaw; ++i) mbar_init(smem_u32(&c.raw[i]), F::kV);
    mbar_init(smem_u32(&c.cleaned), F::kCleaners * kCtas);
    mbar_init(smem_u32(&c.done), F::kSoftmax * kCtas);
    mbar_init(smem_u32(&c.answer_full), 1);
    mbar_init(smem_u32(&c.answer_free), 1);
    mbar_init(smem_u32(&c.drain), 1);
    fence_mbar_init();
    prefetch_tmap(&m.qn[0]);
    prefetch_tmap(&m.qr[0]);
    prefetch_tmap(&m.kn[0]);
    prefetch_tmap(&m.kr[0]);
    prefetch_tmap(&m.v[0]);
  }
  if (threadIdx.x < kKeys) c.notes.clear(threadIdx.x);
  if (warp == F::kMma) {
    if constexpr (kCtas == 1) {
      tmem_alloc(smem_u32(&c.tmem), F::kColumns);
      tmem_relinquish();
    } else {
      tmem_alloc_pair(smem_u32(&c.tmem), F::kColumns);
      tmem_relinquish_pair();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kCtas == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, c.tmem, 0);
  // Roles never rejoin below their register split: each ends with the teardown.
  const auto teardown = [&]() {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (kCtas == 2) cluster_sync();
    tc_fence_after();
    if (warp == F::kMma) {
      if constexpr (kCtas == 1) tmem_dealloc(tmem, F::kColumns);
      else tmem_dealloc_pair(tmem, F::kColumns);
    }
  };
  if (warp >= F::kSoftmax) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == F::kTma) {
      if constexpr (kCtas == 1) produce_one(base, c, p, m, lane);
      else produce_pair(base, c, p, m, rank, lane);
    } else if (warp == F::kMma) {
      if (rank == 0) {
        issue_mmas<kCtas>(base, c, p, tmem, lane);
      } else if (lane == 0) {  // passes the units on
        bool ok;
        Units<kCtas> units(c);
        while (units.next(ok)) units.release();
        int never = 0;
        wait_bar(&c.drain, 0, &never);
      }
    } else if (warp == F::kNext) {
      if (lane == 0) feed<kCtas>(c, p, rank);
    } else if (warp >= F::kClean && warp < F::kClean + F::kCleaners) {
      clean_values<kCtas>(base, c, p, rank, warp - F::kClean, lane);
    } else if constexpr (kCtas == 2) {
      if (warp == F::kNext + 1) load_queries(base, c, p, m, rank, lane);
    }
    teardown();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax_rows<kCtas>(c, p, tmem, rank, warp / 4, warp, lane);
    teardown();
  }
}

// Merge of a block's parts, a warp per row and 16 rows a CTA (a row takes two trips to
// L2 or DRAM, so a warp has few of them): weights e^(LSE_s - max), parts in
// order.  A part that weighs nothing is added all the same, as 0 x inf is NaN where the
// keys are not cut; a NaN makes the row NaN, and a row without a possible key is 0.
constexpr int kMergeRows = 16;
template <int kCtas>
__global__ void __launch_bounds__(256) mla_prefill_merge_kernel(const PrefillParams p) {
  constexpr int kBlock = Form<kCtas>::kBlock, kSlots = kBlock / kSlot;
  const int32_t* e = p.work + (int64_t)(blockIdx.x / p.H) * kEntry * kCtas;
  const int h = blockIdx.x % p.H, seq = e[0], parts = e[3], slot = e[4];
  if (e[2] != 0 || parts < 2 || parts > MLA_PREFILL_MAX_PARTS || slot < 0 ||
      slot > 2 * (int64_t)p.num_parts - parts * kSlots || seq < 0 || seq >= p.N || e[1] < 0 || e[7] != kBlock)
    return;  // reported by the first launch
  const int64_t q0 = p.cu_q[seq], lq = p.cu_q[seq + 1] - q0, row0 = (int64_t)e[1] * kBlock;
  const int64_t k0 = p.cu_kv[seq], lk = p.cu_kv[seq + 1] - k0;
  if (q0 < 0 || lq < 0 || q0 + lq > p.Tq || k0 < 0 || lk < 0 || k0 + lk > p.Tk) return;
  const int rows = (int)min((int64_t)kBlock, lq - row0), lane = threadIdx.x & 31;
  const int r0 = blockIdx.y * kMergeRows;
  for (int r = r0 + threadIdx.x / 32; r < min(rows, r0 + kMergeRows); r += 8) {
    const int64_t at = ((int64_t)(slot + r / kSlot) * p.H + h) * kSlot + r % kSlot;
    const int64_t step = (int64_t)kSlots * p.H * kSlot;
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
      const float4 x = reinterpret_cast<const float4*>(p.O_part + (at + s * step) * MLA_V_HEAD_DIM)[lane];
      o.x += ws * x.x, o.y += ws * x.y, o.z += ws * x.z, o.w += ws * x.w;
    }
    if (sum == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
    const float inv = nan ? NAN : sum > 0.f ? 1.f / sum : 0.f;
    const int64_t row = (q0 + row0 + r) * p.H + h;
    reinterpret_cast<uint2*>(p.out + row * MLA_V_HEAD_DIM)[lane] =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (lane == 0 && p.lse) p.lse[row] = nan ? NAN : sum > 0.f ? m + logf(sum) : -INFINITY;
  }
}

// Tensor map of [T, H, dims] bf16 in boxes of 64 dims x `rows` tokens of a head.
int head_map(CUtensorMap* map, const void* base, int dims, int H, int64_t T, int64_t token_stride,
             int64_t head_stride, int rows) {
  const uint64_t d[3] = {(uint64_t)dims, (uint64_t)H, (uint64_t)std::max<int64_t>(T, 1)};
  const uint64_t st[2] = {(uint64_t)(H > 1 ? head_stride : dims) * 2,
                          (uint64_t)(T > 1 ? token_stride : (int64_t)H * dims) * 2};
  const uint32_t box[3] = {64, 1, (uint32_t)rows};
  return make_tensor_map_bf16_3d(map, base, d, st, box);
}

template <int kCtas>
int launch_prefill(const PrefillMaps& m, const PrefillParams& p, int dev, cudaStream_t st) {
  auto kernel = mla_prefill_kernel<kCtas>;
  static std::atomic<uint64_t> set_on{0};
  const int rc = allow_shared(kernel, kSmem<kCtas>, dev, set_on, "cudaFuncSetAttribute(mla_prefill_kernel)");
  if (rc != MLA_OK) return rc;
  const unsigned units = (unsigned)p.num_work * (unsigned)p.H;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * kCtas, 1, 1);
  cfg.blockDim = dim3(Form<kCtas>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem<kCtas>;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCtas > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, m, p);
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_prefill_kernel");
  if (p.num_parts > 0) {
    mla_prefill_merge_kernel<kCtas><<<dim3(units, Form<kCtas>::kBlock / kMergeRows), 256, 0, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "launch mla_prefill_merge_kernel");
  }
  return MLA_OK;
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
                           int ctas, int num_parts, float* O_part, float* LSE_part, void* out, float* lse,
                           int* status, mla_stream_t stream) {
  constexpr int kNope = MLA_QK_NOPE_DIM, kRope = MLA_ROPE_DIM, kValue = MLA_V_HEAD_DIM;
  if (Tq < 0 || Tk < 0 || N < 0 || num_work < 0 || num_parts < 0 || H < 1)
    return fail(MLA_ERR_INVALID_ARG, "mla_prefill: Tq=%lld Tk=%lld N=%d num_work=%d num_parts=%d < 0 or H=%d < 1",
                (long long)Tq, (long long)Tk, N, num_work, num_parts, H);
  if (!(sm_scale > 0.f) || sm_scale > 1e30f)
    return fail(MLA_ERR_INVALID_ARG, "mla_prefill: sm_scale %g is not a positive number", (double)sm_scale);
  if (ctas != 1 && ctas != 2)
    return fail(MLA_ERR_INVALID_ARG, "mla_prefill: ctas=%d is not 1 or 2", ctas);
  if (Tq > 0x7fffff00 || Tk > 0x7fffff00 || H > 65535 || (int64_t)num_work * H > 1 << 30 ||
      (int64_t)num_work * H * ctas > 0x7fffffff)
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
      !aligned(out, 32) || (num_parts > 0 && (!aligned(O_part, 32) || !aligned(LSE_part, 4))) ||
      !aligned(cu_q, 4) || !aligned(cu_kv, 4) || (prefix && !aligned(prefix, 4)) || !aligned(work, 4) ||
      (lse && !aligned(lse, 4)) || (status && !aligned(status, 4)))
    return fail(MLA_ERR_MISALIGNED, "mla_prefill: queries, keys and values need 16-B alignment (strides a "
                "multiple of 8 elements), out and O_part 32-B, the other arrays 4-B");
  if (Tk == 0) {  // no keys: the maps are never read through
    k_nope = k_rope = v = out;
    kn_token_stride = kn_head_stride = v_token_stride = v_head_stride = kNope;
    kr_token_stride = kRope;
  }
  PrefillMaps m;
  int dev = 0, sms = 0;
  int rc = device_sms(&dev, &sms);
  // boxes of 32 rows pay where there is traffic to save: a few units wait for
  // nothing else, and five more maps take the host 2 us
  const int ends = ctas == 1 && (int64_t)num_work * H >= 2 * sms;
  for (int few = 0; few <= ends && rc == MLA_OK; ++few) {
    const int rows = few ? kFew : kRows, keys = few ? kFew : kKeys / ctas;  // a CTA's tokens of a key tile
    rc = head_map(&m.qn[few], q_nope, kNope, H, Tq, qn_token_stride, qn_head_stride, rows);
    if (rc == MLA_OK) rc = head_map(&m.qr[few], q_rope, kRope, H, Tq, qr_token_stride, qr_head_stride, rows);
    if (rc == MLA_OK) rc = head_map(&m.kn[few], k_nope, kNope, H, Tk, kn_token_stride, kn_head_stride, keys);
    if (rc == MLA_OK) rc = head_map(&m.kr[few], k_rope, kRope, 1, Tk, kr_token_stride, kRope, keys);
    if (rc == MLA_OK) {
      // 64 tokens x 128 dims as two halves of 64 dims, one after the other; in a pair
      // 128 tokens of a CTA's half; few: 32 tokens of a half
      const uint64_t d[4] = {64, (uint64_t)std::max<int64_t>(Tk, 1), 2, (uint64_t)H};
      const uint64_t st[3] = {(uint64_t)(Tk > 1 ? v_token_stride : (int64_t)H * kValue) * 2, 128,
                              (uint64_t)(H > 1 ? v_head_stride : kValue) * 2};
      const uint32_t box[4] = {64, few ? (uint32_t)kFew : 64u * ctas, few || ctas == 2 ? 1u : 2u, 1};
      rc = make_tensor_map_bf16_4d(&m.v[few], v, d, st, box);
    }
  }
  if (rc != MLA_OK) return rc;
  const PrefillParams p{cu_q, cu_kv, prefix, N, H, causal != 0, Tq, Tk, sm_scale, sm_scale * kLog2e, work,
                        num_work, num_parts, O_part, LSE_part, static_cast<__nv_bfloat16*>(out), lse, status, ends};
  const cudaStream_t st = (cudaStream_t)stream;
  return ctas == 1 ? launch_prefill<1>(m, p, dev, st) : launch_prefill<2>(m, p, dev, st);
}
