// mla_tc_fp4.cu -- tensor-core (tcgen05 / TMEM / bulk copy) partial MLA decode
// over the 4-bit latent cache (MLA_KV_FP4_E2M1, mla_fp4.cuh).
//
// Per query row r and visible token t, with c = E2M1 code * E4M3 block scale
// and k = E4M3 RoPE code (both exact in f16) and the pool's factor g:
//   s = sm_scale g (q_nope . c_t + q_rope . k_t),  p = exp(s - m),
//   LSE = m + ln sum p,  O = g (sum p c_t) / sum p.
// The contractions are dense f16 products with M = the request's H * q_len
// rows, so at the framework's 96 x 5 rows the tensor cores bound them (2176
// FLOP per row and token against 352 bytes per token); what the format adds is
// the conversion of each code to f16 in shared memory.
//
// f16, not bf16: an E2M1 x E4M3 product has 6 significant bits and lies in
// [2^-10, 2688], so it is exact, and P keeps 11 bits.  The bf16 queries enter
// as q 2^(14 - e), e the exponent of the row's largest |q|: exact in f16 for
// every element at least 2^-31 of it, off by at most 2^-39 of it below; the
// row's 2^(e - 14) joins the softmax scale in fp32.
//
// Clusters of four CTAs (one per SM) own 256 query rows, as ranks 0, 1 (the S
// pair) and 2, 3 (the O pair), and use CTA-pair MMAs (cta_group::2) that split
// the B operand over the pair: each page is converted once by the S pair (one
// page of every two-page tile per rank) and once by the O pair (half of the
// value dims per rank), not once per 128 rows.
//   S-CTA rank r, row group 2u + r:
//     warp 0       copies raw pages (64 rows x 352 B, contiguous: one bulk
//                  copy) into a ring of three;
//     warps 12-15  convert them, 64 dims at a time, into 8-KB operand boxes (64
//                  tokens x 64 dims f16, K-major, 128-byte swizzle);
//     warp 1       rank 0: issues S[256 rows, 128 tokens] = Q K^T into one of
//                  two TMEM buffers (A = Q_nope from TMEM / Q_rope from shared
//                  memory);
//     warp 2       rank 1: tells rank 0 which boxes are ready;
//     warps 4-11   softmax: warpgroup g takes every second tile, thread = row;
//                  base-2 running statistics with lazy rescaling; P (f16) and
//                  rescale factors travel to the O-CTA by bulk copy (warp 3).
//   O-CTA rank 2 + r, O (128 x 512 fp32) of row group 2u + r in all of TMEM:
//     warps 0, 12-15 as above, over dims [256 n + 128 r, +128), n = 0, 1;
//     warp 1       rank 2: issues O += P V (B = V, MN-major from the same
//                  box layout); rank 3: relays its arrivals to rank 2;
//     warps 4-11   rescale O when a running maximum rose, then the epilogue.
// Two S buffers of N = 128: a probe (unrolled issue, constant descriptors) runs
// M = 128, N = 128, K = 16 f16 MMAs at 64.1 cycles and N = 256 at 128.1, so
// the narrower tile costs nothing and the next tile's products overlap the
// softmax of the last.
// Measured, with the merge: 16 requests x 5 x 96 rows x 100k tokens 1053 us, 1.59
// PFLOP/s of useful products, 84% of the measured bf16 rate (94% of the rows are
// real: 480 of 512); 24 ragged requests of 1k to 200k tokens 612 us, 1.40 PFLOP/s.
#include <cuda_bf16.h>

#include <cstring>

#include "mla_combine.cuh"
#include "mla_fp4_decode.cuh"
#include "mla_tma.cuh"

namespace mla {
namespace {

using namespace ptx;

// Warps 0-3 control, 4-11 softmax (S) or rescale and epilogue (O), 12-15 convert.
constexpr int kThreads = 512;
constexpr int kCtas = 4;             // S pair (ranks 0,1) + O pair (ranks 2,3)
constexpr int kBoxes = 9;            // operand ring: 8-KB boxes
constexpr int kBoxesS = 3;           // S-CTA: a stage is three 64-dim chunks
constexpr int kStagesS = 3;
constexpr int kBoxesO = 4;           // O-CTA: a stage is a page's four boxes
constexpr int kStagesO = 2;
constexpr int kStages = 3;           // barriers of the larger ring
constexpr int kRaw = 3;              // raw page ring
constexpr int kTilePages = 2;        // pages per S tile of the pair, one per S-CTA
constexpr int kChunks = MLA_ROW_DIM / 64;                // 9 boxes per page
static_assert(kBoxesS * kStagesS == kBoxes && kBoxesO * kStagesO <= kBoxes, "ring");
constexpr int kNP = 4;               // P message slots (page index mod 4)
constexpr int kRows = MLA_ROWS_PER_UNIT / 2;  // 128 query rows per CTA
constexpr int kPBytes = kRows * kPage * 2;          // 16384
constexpr int kAlphaOff = kPBytes;                  // float alpha[128]
constexpr int kFlagOff = kPBytes + kRows * 4;       // uint32 flags[4]
constexpr int kPMsgBytes = kFlagOff + 16;           // 16912 = 1057 x 16
constexpr int kPeerFlagOff = kPMsgBytes;            // rank 2: rank 1's flags
constexpr int kPSlotStride = 17408;                 // 17 KB, 1024-aligned
constexpr uint32_t kSCol0 = 256;                    // two S buffers of 128 columns
constexpr int kDequantWarp0 = 12;
constexpr uint32_t kNoteBytes = 4;
constexpr uint16_t kMaskS = 0x3;     // cluster ranks of the S pair
constexpr uint16_t kMaskO = 0xC;     // cluster ranks of the O pair
// Register split of the S-CTAs (setmaxnreg): 512 threads launch with 128 each;
// the control and converter warpgroups give some away so that the softmax can
// hold 128 scores and their p.  One-way: nobody asks for registers back.  Of
// five splits 72/72/184 spills least and is fastest (measured at 16 x 5 x 96 x
// 100k tokens when the kernel took 1140 us: 40/72/200 1175, 56/72/192 1176,
// 80/80/176 1243, 64/96/176 1260).
constexpr int kRegsLaunch = 128;
constexpr int kRegsControl = 72;
constexpr int kRegsConvert = 72;
constexpr int kRegsSoftmax = 184;
static_assert(128 * (kRegsControl + kRegsConvert + 2 * kRegsSoftmax) <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");

constexpr uint32_t kIdescS = idesc_f16_f32(256, 128, false, false);
constexpr uint32_t kIdescO = idesc_f16_f32(256, 256, false, true);

struct __align__(1024) Smem {
  uint8_t ring[kBoxes][kBoxBytes];          // 72 KB of operand boxes
  uint8_t raw[kRaw][kRawBytes];             // 66 KB of pages as stored
  uint8_t qrope[kRows * 128];               // S-CTA: Q_rope rows (f16)
  uint8_t pslot[kNP][kPSlotStride];
  uint32_t note;            // pair leader: where a note lands, of no meaning (relay_made)
  alignas(16) float fin[kRows];
  float mref[kRows];        // S-CTA: every row's running reference
  float xch[2][2][kRows];   // S-CTA: per-warpgroup row values at either end
  uint64_t raw_full[kRaw];  // a raw page landed
  uint64_t raw_empty[kRaw]; // the converters are done with it
  uint64_t full[kStages];    // pair leader: both CTAs' boxes of a stage are written
                             // (its own warps' arrivals, the other CTA's note)
  uint64_t made[kStages];    // pair's other CTA: its boxes of a stage are written
  uint64_t empty[kStages];   // every CTA: its boxes of a stage were consumed
  uint64_t sfull[2];        // S-CTAs: S buffer b holds a tile
  uint64_t sempty[2];       // rank 0: both S-CTAs read buffer b (8 warps)
  uint64_t pmade[kNP];      // S-CTAs: slot k's message is written (4 warps)
  uint64_t pfull[kNP];      // O-CTAs: the P message of slot k landed here
  uint64_t pready[kNP];     // rank 2: rank 3's message of slot k landed
  uint64_t pempty[kNP];     // S-CTAs: slot k consumed by the O pair
  uint64_t drain;           // O-CTAs: all earlier pair MMAs completed
  uint64_t corr_done;       // rank 2: both O-CTAs finished a rescale
  uint64_t fin_full;        // O-CTAs: g/l of every row arrived
  uint64_t epi_go;          // O-CTAs: the epilogue may read O (warps 4-7)
  uint64_t qready;          // rank 0: both S-CTAs' queries are in place
  uint64_t qbar;            // S-CTAs: the query boxes landed
  uint64_t qmoved;          // S-CTAs: the query boxes in the ring are free
  uint32_t raw_bad[kRaw];   // the page lies outside the pool: zeros
  uint32_t tmem_base;
  int abort_flag;
  int ctl_slot;
  int ctl_final;
  int ctl_last;  // fused combine: this cluster wrote the unit's last part
};
constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
static_assert(kPMsgBytes % 16 == 0 && kRawBytes % 1024 == 0, "copy sizes, alignment");
static_assert(kPeerFlagOff + 16 <= kPSlotStride, "P slot layout");

// Three-operand maximum (one ALU instruction on sm_100 and later).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Packed pair arithmetic: two fp32 lanes per instruction.
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

// Arrive on a barrier of the pair leader `lead`: a local arrive when this CTA
// is the leader, otherwise a release at cluster scope, which publishes this
// thread's earlier writes (shared memory, TMEM stores) to the leader.
__device__ __forceinline__ void arrive_leader(uint32_t bar, uint32_t rank,
                                              uint32_t lead) {
  if (rank == lead)
    mbar_arrive(bar);
  else
    mbar_arrive_cluster(mapa(bar, lead));
}

// The same for a signal that only reports completed reads: the thread has its
// scores out of TMEM in registers (tcgen05.wait), so nothing remains to publish
// and the arrive can be relaxed.  A remote release costs the issuing thread hundreds to thousands
// of cycles under load; a relaxed remote arrive a few.
__device__ __forceinline__ void signal_leader(uint32_t bar, uint32_t rank,
                                              uint32_t lead) {
  if (rank == lead) {
    mbar_arrive(bar);
  } else {
    asm volatile(
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
            mapa(bar, lead))
        : "memory");
  }
}

// Record a failed wait: device status and every CTA's abort flag.
__device__ __forceinline__ void signal_abort(Smem& s, const Fp4Params& p,
                                             uint32_t rank) {
  if (p.status) atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
  s.abort_flag = 1;
  for (uint32_t c = 0; c < kCtas; ++c)
    if (c != rank) st_cluster_u32(mapa(smem_u32(&s.abort_flag), c), 1u);
}

// Work of one cluster: unit id (split, virtual request v, row pair u) =
// (split * V + v) * U + u, the cluster's index or, with a work list, the
// list's entry at that index (an entry that names no unit: skip); this
// CTA's row group is 2u + (rank & 1).
struct Work : UnitRange {
  int r_base, nrows;
};

__device__ __forceinline__ Work unit_work(const Fp4Params& p, int unit,
                                          uint32_t rank) {
  Work w;
  unit_range(p, unit / p.U, w);
  w.r_base = (2 * (unit % p.U) + (int)(rank & 1)) * kRows;
  w.nrows = max(0, min(kRows, p.q_len * p.H - w.r_base));
  return w;
}

// S-CTA, warp 0, at kernel entry: initialise the query barriers and put the
// query rows of this CTA's row group in flight (boxes of 64 values x
// q_box_rows rows): Q_nope dims 0..255 into the four P slots, dims 256..511
// into the operand ring (16 KB each), Q_rope into its operand buffer, all on
// qbar.  Lane k issues box k: a thread's TMA loads are processed one after
// another, loads of different threads side by side.
__device__ __forceinline__ uint8_t* query_box(Smem& s, int k) {
  return k < 4 ? s.pslot[k] : s.ring[2 * (k - 4)];
}
static_assert(2 * 4 <= kBoxes, "query boxes in the ring");
__device__ __forceinline__ void issue_query(Smem& s, const CUtensorMap* qn_map,
                                            const CUtensorMap* qr_map,
                                            const Fp4Params& p, int unit,
                                            uint32_t rank, int lane) {
  const int u = unit % p.U;
  const int v = (unit / p.U) % p.V;
  const int b = v % p.B;
  const int qy = b * p.q_len * p.H + (2 * u + (int)(rank & 1)) * kRows;
  const uint32_t qbar = smem_u32(&s.qbar);
  if (lane == 0) {
    mbar_init(qbar, 1);
    mbar_init(smem_u32(&s.qmoved), 1);
    fence_mbar_init();
    prefetch_tmap(qn_map);
    prefetch_tmap(qr_map);
    const uint32_t box = (uint32_t)p.q_box_rows * 128u;
    mbar_arrive_expect_tx(qbar, 9 * box);
  }
  __syncwarp();
  if (lane < 8) {
    tma_load_3d(smem_u32(query_box(s, lane)), qn_map, qbar, 64 * lane, qy, 0);
  } else if (lane == 8) {
    tma_load_3d(smem_u32(s.qrope), qr_map, qbar, 0, qy, 0);
  }
}

// -------------------------------------------------------- raw page copies ---
// Warp 0: pages first, first + step, ... of the unit's range into the raw
// ring.  A page's 64 rows are one contiguous run of the pool, so one bulk copy
// brings it; a page outside the pool is marked instead and converts to zeros.
// Page-table entries are read 32 pages ahead, one per lane.
__device__ __forceinline__ void copy_pages(Smem& s, const Fp4Params& p, const Work& w,
                                           int first, int step, int lane) {
  bool ok = true;
  int slot = 0;
  uint32_t phase = 1;
  int issued = 0;
  int32_t ent = 0;
  for (int m = first, i = 0; m < w.npages && ok; m += step, ++i) {
    if (i % 32 == 0) ent = page_entry(p, w, m + step * lane);
    const int32_t base = checked_base(p, __shfl_sync(kFull, ent, i & 31));
    if (lane == 0) {
      if (mbar_wait(smem_u32(&s.raw_empty[slot]), phase, &s.abort_flag)) {
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
    if (++slot == kRaw) {
      slot = 0;
      phase ^= 1u;
    }
  }
  if (!ok && lane == 0) {
    signal_abort(s, p, 0xFFu);
    // No copy may still be in flight when the CTA leaves (bounded, whatever the
    // abort flag says).
    int never = 0;
    for (int i = max(0, issued - kRaw); i < issued; ++i)
      mbar_wait(smem_u32(&s.raw_full[i % kRaw]), (i / kRaw) & 1, &never);
  }
}

// ------------------------------------------------------------- conversion ---
// Half a token's 64-dim chunk of c_kv (32 codes, scales `two` = 2 bytes) into
// row `t` of a box: chunks 4 h .. 4 h + 3.
__device__ __forceinline__ void convert_half(uint8_t* box, const uint4& c,
                                             uint32_t two, int t, int h) {
  const uint32_t sc = e4m3x2_to_f16(two);
  const uint32_t lo = __byte_perm(sc, sc, 0x1010), hi = __byte_perm(sc, sc, 0x3232);
  *reinterpret_cast<uint4*>(box + box_chunk_offset(t, 4 * h + 0)) = scaled8(c.x, lo);
  *reinterpret_cast<uint4*>(box + box_chunk_offset(t, 4 * h + 1)) = scaled8(c.y, lo);
  *reinterpret_cast<uint4*>(box + box_chunk_offset(t, 4 * h + 2)) = scaled8(c.z, hi);
  *reinterpret_cast<uint4*>(box + box_chunk_offset(t, 4 * h + 3)) = scaled8(c.w, hi);
}

// Half a token's RoPE key (32 codes) into row t of its box.
__device__ __forceinline__ void convert_rope_half(uint8_t* box, const uint4& a, const uint4& b,
                                                  int t, int h) {
  *reinterpret_cast<uint4*>(box + box_chunk_offset(t, 4 * h + 0)) = plain8(a.x, a.y);
  *reinterpret_cast<uint4*>(box + box_chunk_offset(t, 4 * h + 1)) = plain8(a.z, a.w);
  *reinterpret_cast<uint4*>(box + box_chunk_offset(t, 4 * h + 2)) = plain8(b.x, b.y);
  *reinterpret_cast<uint4*>(box + box_chunk_offset(t, 4 * h + 3)) = plain8(b.z, b.w);
}

// A converter warp's arrival for a stage.  One thread of the pair's leader also
// arms full for the other CTA's note.
__device__ __forceinline__ void stage_written(uint64_t* bar, bool arms) {
  if (arms)
    mbar_arrive_expect_tx(smem_u32(bar), kNoteBytes);
  else
    mbar_arrive(smem_u32(bar));
}

// S-CTA, warps 12..15: page 2j + rank of every tile j, chunk by chunk: two
// threads per token, 32 dims each (their 16-byte reads of rows 352 bytes apart
// and their swizzled 16-byte writes are both free of bank conflicts).  The
// leader's own warps arrive on full; the other CTA's arrive on made, which its
// relay passes on.  A tile whose page of this rank does not exist leaves stale
// rows in the columns it feeds, which the softmax masks.
__device__ __forceinline__ void convert_s(Smem& s, const Fp4Params& p, const Work& w,
                                          uint32_t rank, int tid, int lane) {
  const int t = tid >> 1, h = tid & 1;
  uint32_t phase = 1;
  bool ok = mbar_wait(smem_u32(&s.qmoved), 0, &s.abort_flag);
  const int ntiles = (w.npages + kTilePages - 1) / kTilePages;
  uint64_t* const done = rank == 0 ? s.full : s.made;
  int slot = 0;
  uint32_t rphase = 0;
  for (int j = 0; j < ntiles; ++j) {
    const bool have = kTilePages * j + (int)rank < w.npages;
    const uint8_t* row = s.raw[slot] + t * kFp4RowBytes;
    uint4 sa = make_uint4(0, 0, 0, 0), sb = sa;
    uint4 code[kBoxesS + 1];
    bool bad = false;
    // The codes of stage st: loaded before the previous stage's fence, so the
    // loads pass under it (the tile's first stage: under the page's wait).
    const auto load_codes = [&](int st) {
#pragma unroll
      for (int k = 0; k < kBoxesS; ++k) {
        const int c = kBoxesS * st + k;
        if (c < 8) {
          code[k] = *reinterpret_cast<const uint4*>(row + 32 * c + 16 * h);
        } else {
          code[k] = *reinterpret_cast<const uint4*>(row + kFp4RopeOff + 32 * h);
          code[k + 1] = *reinterpret_cast<const uint4*>(row + kFp4RopeOff + 32 * h + 16);
        }
      }
    };
    if (have) {
      ok = ok && mbar_wait(smem_u32(&s.raw_full[slot]), rphase, &s.abort_flag);
      bad = s.raw_bad[slot] != 0;
      load_codes(0);
      sa = *reinterpret_cast<const uint4*>(row + kFp4ScaleOff);
      sb = *reinterpret_cast<const uint4*>(row + kFp4ScaleOff + 16);
      if (bad) sa = sb = make_uint4(0, 0, 0, 0);
    }
    const uint32_t sw[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
    for (int st = 0; st < kStagesS; ++st) {
      ok = ok && mbar_wait(smem_u32(&s.empty[st]), phase, &s.abort_flag);
      if (!__all_sync(kFull, ok)) break;
      if (have) {
#pragma unroll
        for (int k = 0; k < kBoxesS; ++k) {
          const int c = kBoxesS * st + k;
          uint8_t* box = s.ring[c];
          if (c < 8) {
            convert_half(box, code[k], (sw[c] >> (16 * h)) & 0xFFFFu, t, h);
          } else {
            uint4 a = code[k], b = code[k + 1];
            if (bad) a = b = make_uint4(0, 0, 0, 0);
            convert_rope_half(box, a, b, t, h);
          }
        }
        if (st + 1 < kStagesS) load_codes(st + 1);
      }
      __syncwarp();
      if (lane == 0) stage_written(&done[st], rank == 0 && tid == 0);
    }
    phase ^= 1u;
    if (!__all_sync(kFull, ok)) break;
    if (have) {
      if (lane == 0) mbar_arrive(smem_u32(&s.raw_empty[slot]));
      if (++slot == kRaw) {
        slot = 0;
        rphase ^= 1u;
      }
    }
  }
  if (!__all_sync(kFull, ok) && lane == 0) signal_abort(s, p, rank);
}

// O-CTA rank 2 + hh, warps 12..15: dims [256 n + 128 hh, +128) of every page
// (n = 0, 1; box 2n + i of the page's stage = dims 256 n + 128 hh + 64 i).  A
// masked token gets p = 0 exactly, but 0 * NaN would still poison O = P V: the
// only NaN a c_kv value can hold comes from its block scale, so rows at or
// past the length, which can hold anything, and the NaN scales of rows in
// [nmin, L) count as scale 0.  A query that sees such a token has a NaN score
// for it already (the S side converts the scales as they are).
__device__ __forceinline__ void convert_o(Smem& s, const Fp4Params& p, const Work& w,
                                          uint32_t rank, int tid, int lane) {
  const int t = tid >> 1, h = tid & 1, hh = (int)rank - 2;
  uint32_t stage = 0, phase = 1, rphase = 0;
  int slot = 0;
  bool ok = true;
  uint64_t* const done = rank == 2 ? s.full : s.made;
  for (int m = 0; m < w.npages; ++m) {
    ok = ok && mbar_wait(smem_u32(&s.raw_full[slot]), rphase, &s.abort_flag);
    if (!__all_sync(kFull, ok)) break;
    const uint8_t* row = s.raw[slot] + t * kFp4RowBytes;
    uint2 sn[2];
    sn[0] = *reinterpret_cast<const uint2*>(row + kFp4ScaleOff + 8 * hh);
    sn[1] = *reinterpret_cast<const uint2*>(row + kFp4ScaleOff + 16 + 8 * hh);
    const int64_t tok = (w.p0 + m) * kPage + t;
    if (s.raw_bad[slot] || tok >= w.L) {
      sn[0] = sn[1] = make_uint2(0, 0);
    } else if (tok >= w.nmin) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
        sn[n] = make_uint2(finite_scales(sn[n].x), finite_scales(sn[n].y));
    }
    uint4 code[kBoxesO];
#pragma unroll
    for (int k = 0; k < kBoxesO; ++k)
      code[k] = *reinterpret_cast<const uint4*>(row + 128 * (k >> 1) + 64 * hh + 32 * (k & 1) +
                                                16 * h);
    ok = ok && mbar_wait(smem_u32(&s.empty[stage]), phase, &s.abort_flag);
    if (!__all_sync(kFull, ok)) break;
#pragma unroll
    for (int k = 0; k < kBoxesO; ++k)
      convert_half(s.ring[kBoxesO * stage + k], code[k],
                   ((k & 1 ? sn[k >> 1].y : sn[k >> 1].x) >> (16 * h)) & 0xFFFFu, t, h);
    __syncwarp();
    if (lane == 0) {
      stage_written(&done[stage], rank == 2 && tid == 0);
      mbar_arrive(smem_u32(&s.raw_empty[slot]));
    }
    if (++stage == kStagesO) {
      stage = 0;
      phase ^= 1u;
    }
    if (++slot == kRaw) {
      slot = 0;
      rphase ^= 1u;
    }
  }
  if (!__all_sync(kFull, ok) && lane == 0) signal_abort(s, p, rank);
}

// The pair's odd CTA, one thread: passes "stage written" on to the leader, whose
// MMA reads this CTA's boxes too, by a note: an asynchronous store of one word
// into the leader that completes on its full barrier.  The converters' stores
// are ordered before the MMA by made (their release, this thread's acquire), the
// fence to the async proxy, the completion of the note, which is a release at
// cluster scope, and the leader's acquire of it.  A relaxed arrive would order
// nothing; a release arrive does, but holds this thread up for its round trip: at
// 16 x 5 x 96 x 100k tokens the kernel takes 1595 us with that, 1363 with two
// threads taking turns at it, 1113 with the note as a bulk copy (1131 where the
// wait for made may suspend the thread, 1139 where each converter warp sends its
// own, 1480 with stages of one box) and 1053 with the store (ragged 885, 771, 642,
// 648, 658, 827 and 612).
__device__ __forceinline__ void relay_made(Smem& s, const Fp4Params& p, int n, int stages,
                                           uint32_t rank, uint32_t lead) {
  const uint32_t full0 = mapa(smem_u32(&s.full[0]), lead);
  const uint32_t note = mapa(smem_u32(&s.note), lead);
  uint32_t stage = 0, phase = 0;
  for (int i = 0; i < n; ++i) {
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1; !mbar_test_wait(smem_u32(&s.made[stage]), phase); ++it)
      if ((it & 63) == 0 &&
          (*const_cast<volatile int*>(&s.abort_flag) || globaltimer() - t0 > kWaitNs)) {
        signal_abort(s, p, rank);
        return;
      }
    fence_proxy_async_smem();
    st_async_u32(note, 0, full0 + 8u * stage);
    if (++stage == (uint32_t)stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
}

// --------------------------------------------------- S pair: MMA (rank 0) ----
// One thread issues every S-tile MMA of the pair: S[256 rows, 128 tokens] +=
// Q[:, chunk] x K[tokens, chunk]^T, chunks 0..7 with A = Q_nope from TMEM,
// chunk 8 with A = Q_rope from shared memory.
__device__ __forceinline__ void mma_s(Smem& s, const Fp4Params& p, const Work& w,
                                      uint32_t tmem, uint32_t rank) {
  if (!mbar_wait(smem_u32(&s.qready), 0, &s.abort_flag)) {
    signal_abort(s, p, rank);
    return;
  }
  tc_fence_after();
  const uint64_t qr = sdesc_sw128(smem_u32(s.qrope), 16, 1024);
  const uint64_t b0 = sdesc_sw128(smem_u32(s.ring[0]), 16, 1024);
  const int ntiles = (w.npages + kTilePages - 1) / kTilePages;
  for (int j = 0; j < ntiles; ++j) {
    const uint32_t buf = j & 1;
    // both S-CTAs have read the tile before last out of this buffer
    if (!mbar_wait(smem_u32(&s.sempty[buf]), ((j >> 1) & 1) ^ 1u, &s.abort_flag)) {
      signal_abort(s, p, rank);
      return;
    }
    tc_fence_after();
    const uint32_t d = tmem + kSCol0 + 128u * buf;
#pragma unroll 1
    for (int st = 0; st < kStagesS; ++st) {
      if (!mbar_wait(smem_u32(&s.full[st]), j & 1, &s.abort_flag)) {
        signal_abort(s, p, rank);
        return;
      }
      fence_proxy_async_smem();
      tc_fence_after();
      const uint64_t b = b0 + (uint64_t)(kBoxesS * st) * (kBoxBytes >> 4);
      const uint32_t a = tmem + 32u * kBoxesS * st;
#pragma unroll
      for (int k = 0; k < 4 * (kBoxesS - 1); ++k)
        mma_ts_pair(d, a + 8u * k, b + (k >> 2) * (kBoxBytes >> 4) + 2 * (k & 3), kIdescS,
                    (st | k) ? 1u : 0u);
      const uint64_t b2 = b + (kBoxesS - 1) * (kBoxBytes >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (st < kStagesS - 1)
          mma_ts_pair(d, a + 32u * (kBoxesS - 1) + 8u * k, b2 + 2 * k, kIdescS, 1u);
        else
          mma_ss_pair(d, qr + 2 * k, b2 + 2 * k, kIdescS, 1u);
      }
      mma_commit_pair(smem_u32(&s.empty[st]), kMaskS);
    }
    mma_commit_pair(smem_u32(&s.sfull[buf]), kMaskS);
  }
}

// -------------------------------------------- S-CTA: P messages (warp 3) ----
// One thread sends each page's message (P, rescale factors, flags) to the row
// group's O-CTA once the four warps of its warpgroup have written it, so no
// softmax warp spends its time on the copies or on a barrier per page.
__device__ __forceinline__ void ship_pages(Smem& s, const Fp4Params& p, const Work& w,
                                           uint32_t rank) {
  const uint32_t orank = rank + 2;
  const uint32_t peer_pfull0 = mapa(smem_u32(&s.pfull[0]), orank);
  for (int m = 0; m < w.npages; ++m) {
    const int k = m % kNP;
    if (!mbar_wait(smem_u32(&s.pmade[k]), (m / kNP) & 1, &s.abort_flag)) {
      signal_abort(s, p, rank);
      return;
    }
    fence_proxy_async_smem();
    uint8_t* stg = s.pslot[k];
    // The receiver armed pfull[k] with the byte count itself.
    bulk_copy_to_peer(mapa(smem_u32(stg), orank), smem_u32(stg), kPMsgBytes,
                      peer_pfull0 + 8u * k);
    // Rank 2 issues the pair's P x V MMAs and decides on rescales: it gets
    // rank 1's rescale flags too, counted on its own pfull[k].
    if (rank == 1)
      bulk_copy_to_peer(mapa(smem_u32(stg + kPeerFlagOff), 2), smem_u32(stg + kFlagOff), 16,
                        mapa(smem_u32(&s.pfull[k]), 2));
  }
}

// ------------------------------------------------------ S-CTA: the queries ----
// Thread (g, r) of the softmax warpgroups takes dims 256 g .. 256 g + 255 of
// row r (g = 0 also the RoPE part): the row's largest |q| gives the exponent
// e, and q 2^(14 - e) goes to TMEM columns [0, 256) (column c: dims 2c, 2c +
// 1) or back into its place in the RoPE operand, as f16.  Returns 2^(e - 14).
__device__ __forceinline__ float place_query(Smem& s, uint32_t tmem, uint32_t lane_base,
                                             int g, int r, bool row_ok) {
  const auto chunk = [&](const uint8_t* box, int cc) -> uint4 {
    return row_ok ? *reinterpret_cast<const uint4*>(box + (r >> 3) * 1024 +
                                                    box_chunk_offset(r & 7, cc))
                  : make_uint4(0, 0, 0, 0);
  };
  // The exponent fields order like the magnitudes: the largest |q| as bits.
  uint32_t big4[4] = {0, 0, 0, 0};  // two values a word
  const auto take = [&](uint4 v) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) big4[k] = __vmaxu2(big4[k], x[k] & 0x7FFF7FFFu);
  };
#pragma unroll 1
  for (int k = 4 * g; k < 4 * g + 4; ++k)
#pragma unroll
    for (int cc = 0; cc < 8; ++cc) take(chunk(query_box(s, k), cc));
  if (g == 0)
#pragma unroll
    for (int cc = 0; cc < 8; ++cc) take(chunk(s.qrope, cc));
  const uint32_t big2 = __vmaxu2(__vmaxu2(big4[0], big4[1]), __vmaxu2(big4[2], big4[3]));
  uint32_t big = max(big2 & 0xFFFFu, big2 >> 16);
  s.xch[0][g][r] = __uint_as_float(big);
  named_bar_sync(1, 256);
  big = max(big, __float_as_uint(s.xch[0][g ^ 1][r]));
  // A row below 2^-100 keeps its exponent there: 2^(14 - e) stays in fp32.
  const int e = max(min((int)(big >> 7), 254) - 127, -100);
  const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
  const auto conv = [&](uint32_t w) -> uint32_t {
    return pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
  };
#pragma unroll 1
  for (int k = 4 * g; k < 4 * g + 4; ++k) {
    uint32_t o[32];
#pragma unroll
    for (int cc = 0; cc < 8; ++cc) {
      const uint4 v = chunk(query_box(s, k), cc);
      o[4 * cc] = conv(v.x);
      o[4 * cc + 1] = conv(v.y);
      o[4 * cc + 2] = conv(v.z);
      o[4 * cc + 3] = conv(v.w);
    }
    tmem_st32(tmem + lane_base + 32u * k, o);
  }
  if (g == 0) {
#pragma unroll
    for (int cc = 0; cc < 8; ++cc) {
      const uint4 v = chunk(s.qrope, cc);
      *reinterpret_cast<uint4*>(s.qrope + (r >> 3) * 1024 + box_chunk_offset(r & 7, cc)) =
          make_uint4(conv(v.x), conv(v.y), conv(v.z), conv(v.w));
    }
  }
  tmem_wait_st();
  fence_proxy_async_smem();
  tc_fence_before();
  named_bar_sync(1, 256);
  return __uint_as_float((uint32_t)(127 + e - 14) << 23);
}

// ------------------------------------------------------ S-CTA: softmax ----
// What a softmax thread knows of its row, and the query's placement.
struct SoftmaxRow {
  int r;            // row of the group (TMEM lane)
  bool in_range;
  int64_t n, qrow;  // tokens the row sees; its row among the outputs
  float pool, sc;   // g; the score scale in log2 units
  bool ok;          // no wait has given up
};
__device__ __forceinline__ SoftmaxRow softmax_begin(Smem& s, const Fp4Params& p, const Work& w,
                                                    uint32_t tmem, uint32_t rank, int warp,
                                                    int lane) {
  SoftmaxRow t;
  const int quad = warp & 3;
  t.r = quad * 32 + lane;
  t.in_range = t.r < w.nrows;
  const int rr = w.r_base + t.r;
  const int i = t.in_range ? rr / p.H : 0;
  t.n = 0;
  if (t.in_range) {
    t.n = p.kv_limit ? (int64_t)p.kv_limit[(int64_t)w.v * p.q_len + i]
                     : w.L - p.q_len + 1 + i;
    t.n = t.n > w.L ? w.L : (t.n < 0 ? 0 : t.n);
  }
  t.qrow = (int64_t)w.b * p.q_len * p.H + rr;
  t.pool = p.g[0];
  t.ok = mbar_wait(smem_u32(&s.qbar), 0, &s.abort_flag);
  t.sc = score_factor(
      p.scale_log2, t.pool,
      place_query(s, tmem, (uint32_t)(quad * 32) << 16, (warp - 4) >> 2, t.r, t.in_range));
  if (warp == 4 && lane == 0) {
    mbar_arrive(smem_u32(&s.qmoved));
    arrive_leader(smem_u32(&s.qready), rank, 0);
  }
  return t;
}

// Final statistics: both warpgroups' sums, l in units of 2^m_own, in units of
// the last reference; LSE_part, and g / l to the O-CTA.
__device__ __forceinline__ void softmax_end(Smem& s, const Fp4Params& p, const Work& w,
                                            const SoftmaxRow& t, float m_own, float l, bool ok,
                                            uint32_t rank, int warp, int lane) {
  const int g = (warp - 4) >> 2, r = t.r;
  const uint32_t orank = rank + 2;  // the O-CTA of this row group
  s.xch[0][g][r] = m_own;
  s.xch[1][g][r] = l;
  named_bar_sync(1, 256);
  if (g == 0) {
    const float m_ref = s.mref[r];
    const auto part_sum = [&](int k) {  // a sum without a reference is 0 or NaN
      const float m = s.xch[0][k][r], z = s.xch[1][k][r];
      return m == -INFINITY ? z : z * ex2(m - m_ref);
    };
    const float lt = part_sum(0) + part_sum(1);
    if (t.in_range) {
      const int64_t rows = (int64_t)p.B * p.q_len * p.H;
      const int64_t part = (int64_t)w.split * (p.V / p.B) + w.shard;
      // no visible token: -inf; a NaN sum (a NaN score seen) stays NaN
      p.LSE_part[part * rows + t.qrow] =
          lt == 0.f ? -INFINITY : (m_ref + log2f(lt)) * 0.69314718055994531f;
    }
    s.fin[r] = lt == 0.f ? 0.f : t.pool / lt;
    fence_proxy_async_smem();
    named_bar_sync(2, 128);
    if (warp == 4 && lane == 0 && !s.abort_flag)
      bulk_copy_to_peer(mapa(smem_u32(s.fin), orank), smem_u32(s.fin), kRows * 4,
                        mapa(smem_u32(&s.fin_full), orank));
    // Before teardown: every P slot released by the O pair, so no remote
    // arrive can land after this CTA exits.
    for (int m = max(0, w.npages - kNP); m < w.npages && ok; ++m)
      if (!mbar_wait(smem_u32(&s.pempty[m % kNP]), (m / kNP) & 1,
                     &s.abort_flag))
        ok = false;
  }
  if (!__all_sync(kFull, ok) && lane == 0) signal_abort(s, p, rank);
}

// The tile's reference from the last one's and its own maximum; alpha: the
// factor of what O and l hold so far.
__device__ __forceinline__ float next_reference(float m_old, float mt, float& alpha) {
  alpha = 1.f;
  if (!(mt > -INFINITY)) return m_old;
  const float m_new = mt - kLift;
  if (m_old == -INFINITY) return m_new;  // first visible token of this row: O is zero
  if (!(mt > m_old + (kLift + kTau))) return m_old;
  alpha = ex2(m_old - m_new);
  return m_new;
}

// Warps 4..11 of each S-CTA: warpgroup g (warps 4-7, 8-11) takes the tiles j
// with j % 2 = g, which are those of S buffer g, so a tile's chain of loads,
// maximum, exponentials and stores has two tile periods.  Thread = query row r
// (TMEM lane) of this CTA's row group, with the tile's 128 scores in registers:
// the buffer is free for the tile after next as soon as they are loaded (read
// twice instead, the buffer is held through the first page's exponentials:
// 1347 us at 16 x 5 x 96 x 100k tokens).
__device__ __forceinline__ void softmax(Smem& s, const Fp4Params& p, const Work& w,
                                        uint32_t tmem, uint32_t rank, int warp, int lane) {
  const int g = (warp - 4) >> 2, quad = warp & 3;
  const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
  const SoftmaxRow t = softmax_begin(s, p, w, tmem, rank, warp, lane);
  const int r = t.r;
  const int64_t n = t.n;
  const float sc = t.sc;
  bool ok = t.ok;

  // The running reference m of each row passes from tile to tile through
  // mref, from one warpgroup to the other; a warp of each holds the same 32
  // rows, so 64 threads meet per hand-over.
  float m_own = -INFINITY, l = 0.f;  // l: this warpgroup's sum, in units of 2^m_own
  constexpr int kCols = kPage * kTilePages;
  const int ntiles = (w.npages + kTilePages - 1) / kTilePages;
  for (int j = g; j < ntiles; j += 2) {
    const int m0 = j * kTilePages;  // the tile's first page
    const bool two = m0 + 1 < w.npages;
    uint32_t sv[kCols];
    if (ok && !mbar_wait(smem_u32(&s.sfull[g]), (j >> 1) & 1, &s.abort_flag)) ok = false;
    tc_fence_after();
    if (__all_sync(kFull, ok)) {
      const uint32_t col = tmem + lane_base + kSCol0 + 128u * g;
#pragma unroll
      for (int q = 0; q < kCols / 32; ++q)
        tmem_ld32(col + 32u * q, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * q]));
      tmem_wait_ld();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) signal_leader(smem_u32(&s.sempty[g]), rank, 0);
    // Columns this row may not see become -inf (a select: garbage or NaN in a
    // masked column never propagates); only the range's last tiles need it.
    const int64_t nv = n - (w.p0 + m0) * kPage;
    const int most = two ? 2 * kPage : kPage;
    const int nvis = nv <= 0 ? 0 : (nv >= most ? most : (int)nv);
    if (!__all_sync(kFull, nvis == kCols)) {
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        sv[c] = c < nvis ? sv[c] : __float_as_uint(-INFINITY);
    }
    // Row maximum of the raw scores; the scale is positive, so the maximum
    // of the scaled scores is the scaled maximum (rounding is monotone).
    constexpr int kM = kCols / 8;
    float mx[kM];
#pragma unroll
    for (int c = 0; c < kM; ++c) {
      const auto x = [&](int k) { return __uint_as_float(sv[c + kM * k]); };
      mx[c] = fmaxf(max3(x(0), x(1), x(2)), max3(max3(x(3), x(4), x(5)), x(6), x(7)));
    }
#pragma unroll
    for (int c = kM / 2; c > 0; c >>= 1)
#pragma unroll
      for (int k = 0; k < c; ++k) mx[k] = fmaxf(mx[k], mx[k + c]);
    const float mt = mx[0] * sc;
    if (j > 0) named_bar_sync(4 + 2 * quad + g, 64);  // the last tile's reference is in
    const float m_old = j > 0 ? s.mref[r] : -INFINITY;
    float alpha;
    const float m_ref = next_reference(m_old, mt, alpha);
    s.mref[r] = m_ref;
    if (j + 1 < ntiles) named_bar_arrive(4 + 2 * quad + (g ^ 1), 64);
    if (m_own != m_ref) {
      if (m_own != -INFINITY) l *= ex2(m_own - m_ref);
      m_own = m_ref;
    }
    // A row with nothing visible yet keeps m_ref = -inf: shift by 0 instead
    // so every p is ex2(-inf) = 0, not NaN.
    const float shift = m_ref == -INFINITY ? 0.f : m_ref;
    const uint64_t sc2 = f2pack(sc, sc), nshift2 = f2pack(-shift, -shift);
    const bool any = __any_sync(kFull, alpha != 1.f);
#pragma unroll
    for (int q = 0; q < kTilePages; ++q) {
      if (q == 1 && !two) break;
      // p = 2^(x * scale - m_ref): one packed FMA per pair of columns, the
      // row sum of the unrounded p in two packed accumulators.  P is shipped
      // as f16 (see kLift): off by 2^-11 of itself or by 2^-25, whichever is more.
      uint32_t pk[32];
      uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        float ya, yb;
        f2unpack(ffma2(f2pack(__uint_as_float(sv[64 * q + 2 * c]),
                              __uint_as_float(sv[64 * q + 2 * c + 1])),
                       sc2, nshift2),
                 ya, yb);
        const float pa = ex2(ya), pb = ex2(yb);
        if (c & 1) acc1 = fadd2(acc1, f2pack(pa, pb));
        else acc0 = fadd2(acc0, f2pack(pa, pb));
        pk[c] = pack_f16(pa, pb);
      }
      float a0, a1, b0, b1;
      f2unpack(acc0, a0, a1);
      f2unpack(acc1, b0, b1);
      l += (a0 + a1) + (b0 + b1);

      // Write the page's message once its slot is free; warp 3 sends it.
      const int msg = m0 + q;
      const int k = msg % kNP;
      const int u = msg / kNP;  // use index of slot k
      if (u > 0 && ok &&
          !mbar_wait(smem_u32(&s.pempty[k]), (u - 1) & 1, &s.abort_flag))
        ok = false;
      uint8_t* stg = s.pslot[k];
#pragma unroll
      for (int cc = 0; cc < 8; ++cc)
        // K-major, 128-B swizzle: 8-row groups 1024 B apart, 16-B chunk cc
        // of row r at position cc ^ (r % 8) within its 128-B row.
        *reinterpret_cast<uint4*>(stg + (r >> 3) * 1024 + box_chunk_offset(r & 7, cc)) =
            make_uint4(pk[4 * cc], pk[4 * cc + 1], pk[4 * cc + 2], pk[4 * cc + 3]);
      // The tile's rescale travels with its first page only.
      reinterpret_cast<float*>(stg + kAlphaOff)[r] = q == 0 ? alpha : 1.f;
      if (lane == 0)
        reinterpret_cast<uint32_t*>(stg + kFlagOff)[quad] = q == 0 && any ? 1u : 0u;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.pmade[k]));
    }
  }

  softmax_end(s, p, w, t, m_own, l, ok, rank, warp, lane);
}

// --------------------------------------------------- O pair: MMA (rank 2) ----
// One thread issues every P x V MMA of the pair: for each page m (message
// slot k = m mod 4) it needs the P rows of both O-CTAs (its own pfull, which
// also counts rank 1's rescale flags, and rank 3's through pready), then
// O[:, 256n + (0..255)] += P x V for n = 0, 1.
__device__ __forceinline__ void mma_o(Smem& s, const Fp4Params& p,
                                      const Work& w, uint32_t tmem,
                                      uint32_t rank) {
  uint32_t stage = 0, phase = 0, ev = 0;
  bool ok = true;
  const uint32_t drain3 = mapa(smem_u32(&s.drain), 3);
  // Each P message lands by a bulk copy whose bytes complete on pfull[k];
  // the receiving CTA arms the barrier (one arrival + the byte count)
  // itself, so the sender needs no cluster-scope arrive: the first use of
  // each slot is armed at set-up, the next one as soon as a message has been
  // received (here for rank 2, by the relay thread for rank 3).
  for (int m = 0; m < w.npages && ok; ++m) {
    const int k = m % kNP;
    const uint32_t par = (m / kNP) & 1;
    if (!mbar_wait(smem_u32(&s.pfull[k]), par, &s.abort_flag) ||
        !mbar_wait(smem_u32(&s.pready[k]), par, &s.abort_flag)) {
      ok = false;
      break;
    }
    if (m + kNP < w.npages)
      mbar_arrive_expect_tx(smem_u32(&s.pfull[k]), kPMsgBytes + 16);
    const uint32_t* fl =
        reinterpret_cast<const uint32_t*>(s.pslot[k] + kFlagOff);
    const uint32_t* pf =
        reinterpret_cast<const uint32_t*>(s.pslot[k] + kPeerFlagOff);
    if (fl[0] | fl[1] | fl[2] | fl[3] | pf[0] | pf[1] | pf[2] | pf[3]) {
      // Rows of either O-CTA raised their running max: let both CTAs'
      // correction warps rescale once every earlier product has landed.
      s.ctl_slot = k;
      s.ctl_final = 0;
      st_cluster_u32(mapa(smem_u32(&s.ctl_slot), 3), (uint32_t)k);
      st_cluster_u32(mapa(smem_u32(&s.ctl_final), 3), 0u);
      mma_commit_pair(smem_u32(&s.drain), kMaskO);
      mbar_arrive(smem_u32(&s.drain));
      mbar_arrive_cluster(drain3);
      if (!mbar_wait(smem_u32(&s.corr_done), ev & 1, &s.abort_flag)) {
        ok = false;
        break;
      }
      ++ev;
    }
    const uint64_t a = sdesc_sw128(smem_u32(s.pslot[k]), 16, 1024);
    if (!mbar_wait(smem_u32(&s.full[stage]), phase, &s.abort_flag)) {
      ok = false;
      break;
    }
    fence_proxy_async_smem();
    tc_fence_after();
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      // B = V: MN-major, next 64 dims one box (8 KB) on, next 8 tokens 1 KB
      // on; each 16-token K step advances 2048 B (128 descriptor units).
      const uint64_t b =
          sdesc_sw128(smem_u32(s.ring[kBoxesO * stage + 2 * n]), kBoxBytes, 1024);
      const uint32_t d = tmem + 256u * n;
      mma_ss_pair(d, a + 0, b + 0, kIdescO, m > 0 ? 1u : 0u);
      mma_ss_pair(d, a + 2, b + 128, kIdescO, 1u);
      mma_ss_pair(d, a + 4, b + 256, kIdescO, 1u);
      mma_ss_pair(d, a + 6, b + 384, kIdescO, 1u);
    }
    mma_commit_pair(smem_u32(&s.empty[stage]), kMaskO);
    if (++stage == kStagesO) {
      stage = 0;
      phase ^= 1u;
    }
    mma_commit_pair(smem_u32(&s.pempty[k]), kMaskS);  // both S-CTAs
  }
  if (!ok) signal_abort(s, p, rank);
  s.ctl_final = 1;
  st_cluster_u32(mapa(smem_u32(&s.ctl_final), 3), 1u);
  mma_commit_pair(smem_u32(&s.drain), kMaskO);
  mbar_arrive(smem_u32(&s.drain));
  mbar_arrive_cluster(drain3);
}

// --------------------------------------------------- O pair: relay (rank 3) ----
// Tells rank 2 when a P message has landed in rank 3 (bulk-copy bytes can
// only complete on a barrier of the receiving CTA), and re-arms the slot.  The
// arrive is a release: rank 2's MMA reads the message here.  (One thread with
// nothing else to do, four messages ahead: a note costs the same.)
__device__ __forceinline__ void relay_o(Smem& s, const Fp4Params& p,
                                        const Work& w, uint32_t rank) {
  const uint32_t pready0 = mapa(smem_u32(&s.pready[0]), 2);
  for (int m = 0; m < w.npages; ++m) {
    const int k = m % kNP;
    if (!mbar_wait(smem_u32(&s.pfull[k]), (m / kNP) & 1, &s.abort_flag)) {
      signal_abort(s, p, rank);
      return;
    }
    if (m + kNP < w.npages)
      mbar_arrive_expect_tx(smem_u32(&s.pfull[k]), kPMsgBytes);
    mbar_arrive_cluster(pready0 + 8u * k);
  }
}

// ------------------------------------------------ O-CTA: epilogue stores ----
// O_part = O / l for this thread's row r (TMEM lane) over value columns
// [256 half, +256), 32 at a time: the warp stages its 32 rows x 32 values
// in 4 KB of the then idle ring (row r at 128 r bytes, 16-byte chunk e at
// position e ^ (r % 8), so neither the writes nor the reads below conflict)
// and reads them back four rows per instruction, lane l taking chunk l % 8
// of row 4i + l / 8: every store instruction writes four full 128-byte
// lines of O_part.
__device__ __forceinline__ void store_o_rows(Smem& s, const Fp4Params& p,
                                             const CUtensorMap* o_map,
                                             const Work& w, uint32_t tmem,
                                             int warp, int lane, int half) {
  const int quad = warp & 3;
  const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
  const float inv = s.fin[quad * 32 + lane];
  const int64_t rows = (int64_t)p.B * p.q_len * p.H;
  const int64_t part = (int64_t)w.split * (p.V / p.B) + w.shard;
  const int64_t row0 =
      part * rows + (int64_t)w.b * p.q_len * p.H + w.r_base + quad * 32;
  float* const dst0 = p.O_part + row0 * MLA_VALUE_DIM;
  const int nvalid = w.nrows - quad * 32;  // rows of this warp in range
  if (p.o_bf16) {
    // bf16 partial outputs: 64 values (128 bytes) per row of a box, four
    // boxes per warp and half, box k stored by lane k; a partial 32-row
    // block is written by its lanes directly (64 bytes per row and step).
    __nv_bfloat16* const dst_b =
        reinterpret_cast<__nv_bfloat16*>(p.O_part) + row0 * MLA_VALUE_DIM;
    uint8_t* const bufs = &s.ring[0][0] + 16384 * (warp - 4);
    const bool by_tma = p.o_tma && nvalid >= 32;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const int c0 = 256 * half + 64 * k;
      uint32_t va[32], vb[32];
      tmem_ld32(tmem + lane_base + c0, va);
      tmem_ld32(tmem + lane_base + c0 + 32, vb);
      tmem_wait_ld();
      uint4 q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t* v = e < 4 ? va + 8 * e : vb + 8 * (e - 4);
        q[e] = make_uint4(pack_bf16(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv),
                          pack_bf16(__uint_as_float(v[2]) * inv, __uint_as_float(v[3]) * inv),
                          pack_bf16(__uint_as_float(v[4]) * inv, __uint_as_float(v[5]) * inv),
                          pack_bf16(__uint_as_float(v[6]) * inv, __uint_as_float(v[7]) * inv));
      }
      if (by_tma) {
        uint8_t* const box = bufs + k * 4096;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(box + box_chunk_offset(lane, e)) = q[e];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == k) {
          tma_store_3d(o_map, smem_u32(box), c0, (int32_t)row0, 0);
          bulk_commit_group();
        }
      } else if (lane < nvalid) {
        uint4* d = reinterpret_cast<uint4*>(dst_b + (int64_t)lane * MLA_VALUE_DIM + c0);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = q[e];
      }
    }
    if (by_tma) {
      if (lane < 4) bulk_wait_read_all();
      __syncwarp();
    }
    return;
  }
  if (p.o_tma && nvalid >= 32) {
    // Whole 32-row blocks leave by TMA store, 32 values (128 bytes) per
    // box: four boxes of this warp's 16 KB of the idle ring in turn, box i
    // stored by lane i (a thread's TMA operations are processed one after
    // another), which waits for the box's previous store to have read it
    // before the warp refills it.
    uint8_t* const bufs = &s.ring[0][0] + 16384 * (warp - 4);
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      const int c0 = 256 * half + 32 * k;
      const int bi = k & 3;
      uint8_t* const box = bufs + bi * 4096;
      uint32_t v[32];
      tmem_ld32(tmem + lane_base + c0, v);
      if (k >= 4 && lane == bi) bulk_wait_read_all();
      __syncwarp();
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        *reinterpret_cast<float4*>(box + box_chunk_offset(lane, e)) =
            make_float4(__uint_as_float(v[4 * e]) * inv,
                        __uint_as_float(v[4 * e + 1]) * inv,
                        __uint_as_float(v[4 * e + 2]) * inv,
                        __uint_as_float(v[4 * e + 3]) * inv);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == bi) {
        tma_store_2d(o_map, smem_u32(box), c0, (int32_t)row0);
        bulk_commit_group();
      }
    }
    if (lane < 4) bulk_wait_read_all();
    __syncwarp();
    return;
  }
  uint8_t* const buf = &s.ring[0][0] + 16384 * (warp - 4);  // this warp's 16 KB as above
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    const int c0 = 256 * half + 32 * k;
    uint32_t v[32];
    tmem_ld32(tmem + lane_base + c0, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      *reinterpret_cast<float4*>(buf + box_chunk_offset(lane, e)) =
          make_float4(__uint_as_float(v[4 * e]) * inv,
                      __uint_as_float(v[4 * e + 1]) * inv,
                      __uint_as_float(v[4 * e + 2]) * inv,
                      __uint_as_float(v[4 * e + 3]) * inv);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int rr = 4 * i + (lane >> 3), e = lane & 7;
      const float4 f =
          *reinterpret_cast<const float4*>(buf + box_chunk_offset(rr, e));
      if (rr < nvalid)
        *reinterpret_cast<float4*>(dst0 + (int64_t)rr * MLA_VALUE_DIM + c0 +
                                   4 * e) = f;
    }
    __syncwarp();  // every lane read the box before it is refilled
  }
}

// Warps 8..11 of each O-CTA: the second half of the value columns, once
// warps 4..7 have seen the last drain and 1/l.
__device__ __forceinline__ void store_o_upper(Smem& s, const Fp4Params& p,
                                              const CUtensorMap* o_map,
                                              const Work& w, uint32_t tmem,
                                              int warp, int lane) {
  if (!mbar_wait(smem_u32(&s.epi_go), 0, &s.abort_flag)) return;
  tc_fence_after();
  store_o_rows(s, p, o_map, w, tmem, warp, lane, 1);
}

// ---------------------------------------- O-CTA: correction + epilogue ----
// Warps 4..7 of each O-CTA, thread = row r of this CTA's row group.  A
// drain event (every earlier pair MMA complete) either asks for a rescale of
// the rows whose running max rose (factors in the P slot that triggered it)
// or, the last one, for the epilogue: O_part = O / l over the first half of
// the value columns (warps 8..11 take the second, after epi_go).
__device__ __forceinline__ void correct_and_store(Smem& s, const Fp4Params& p,
                                                  const CUtensorMap* o_map,
                                                  const Work& w, uint32_t tmem,
                                                  uint32_t rank, int warp,
                                                  int lane) {
  const int quad = warp & 3;
  const int r = quad * 32 + lane;
  const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
  bool ok = true;
  for (uint32_t ev = 0;; ++ev) {
    if (!mbar_wait(smem_u32(&s.drain), ev & 1, &s.abort_flag)) {
      ok = false;
      break;
    }
    tc_fence_after();
    if (*reinterpret_cast<volatile int*>(&s.ctl_final)) break;
    const int k = *reinterpret_cast<volatile int*>(&s.ctl_slot);
    const float a = reinterpret_cast<const float*>(s.pslot[k] + kAlphaOff)[r];
    if (__any_sync(kFull, a != 1.f)) {
#pragma unroll 1
      for (int c0 = 0; c0 < MLA_VALUE_DIM; c0 += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + lane_base + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          v[e] = __float_as_uint(__uint_as_float(v[e]) * a);
        tmem_st32(tmem + lane_base + c0, v);
      }
      tmem_wait_st();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_leader(smem_u32(&s.corr_done), rank, 2);
  }
  if (ok && !mbar_wait(smem_u32(&s.fin_full), 0, &s.abort_flag)) ok = false;
  if (!__all_sync(kFull, ok)) {
    if (lane == 0) signal_abort(s, p, rank);
    return;
  }
  tc_fence_after();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&s.epi_go));
  store_o_rows(s, p, o_map, w, tmem, warp, lane, 0);
}

// ------------------------------------------------------------- kernel ----
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    mla_partial_fp4_kernel(const __grid_constant__ CUtensorMap qn_map,
                           const __grid_constant__ CUtensorMap qr_map,
                           const __grid_constant__ CUtensorMap o_map,
                           const Fp4Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // Warp-uniform by construction, so that the MMA issue works on uniform
  // registers (see elect_one).
  const int warp = __shfl_sync(kFull, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int unit = launch_unit(p, blockIdx.x / kCtas);
  if (unit < 0) {  // every CTA of the cluster read the same entry
    if (rank == 0 && threadIdx.x == 0 && p.status)
      atomicOr(p.status, MLA_STATUS_BAD_WORK);
    return;
  }
  // The query rows need only the unit id: the S-CTAs put them in flight
  // before anything else, so their load overlaps the rest of the set-up.
  if (rank < 2 && warp == 0) issue_query(s, &qn_map, &qr_map, p, unit, rank, lane);
  const Work w = unit_work(p, unit, rank);

  // The stream's next kernel (the LSE combine) may be scheduled from now
  // on; it waits for this grid's completion before it reads a part.
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    s.ctl_slot = 0;
    s.ctl_final = 0;
    s.ctl_last = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 4);  // 4 local warps; and the other CTA's note
      mbar_init(smem_u32(&s.made[i]), 4);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(smem_u32(&s.raw_full[i]), 1);
      mbar_init(smem_u32(&s.raw_empty[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.sfull[i]), 1);
      mbar_init(smem_u32(&s.sempty[i]), 8);  // a warpgroup of either S-CTA
    }
    for (int i = 0; i < kNP; ++i) {
      mbar_init(smem_u32(&s.pmade[i]), 4);
      mbar_init(smem_u32(&s.pfull[i]), 1);
      mbar_init(smem_u32(&s.pready[i]), 1);
      mbar_init(smem_u32(&s.pempty[i]), 1);
    }
    mbar_init(smem_u32(&s.drain), 2);      // pair commit + rank 2's arrive
    mbar_init(smem_u32(&s.corr_done), 8);  // 4 correction warps x 2 O-CTAs
    mbar_init(smem_u32(&s.fin_full), 1);
    mbar_init(smem_u32(&s.epi_go), 4);
    mbar_init(smem_u32(&s.qready), 2);  // one thread per S-CTA
    if (rank >= 2 && w.npages > 0) {
      mbar_arrive_expect_tx(smem_u32(&s.fin_full), kRows * 4);
      // rank 2 also receives rank 1's 16 flag bytes per message
      for (int k = 0; k < kNP && k < w.npages; ++k)
        mbar_arrive_expect_tx(smem_u32(&s.pfull[k]),
                              kPMsgBytes + (rank == 2 ? 16 : 0));
    }
    fence_mbar_init();
    if (rank >= 2 && p.o_tma) prefetch_tmap(&o_map);
  }
  if (rank == 0 && threadIdx.x == 32 && p.seq_lens[w.v] > p.r2t_stride &&
      p.status)
    atomicOr(p.status, MLA_STATUS_BAD_LENGTH);
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&s.tmem_base), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, s.tmem_base, 0);
  cluster_sync();  // every CTA's barriers exist before any remote operation

  // Fused combine ([K3-MLA], dcp_lse_combine, in the same launch): rank 0
  // counts this cluster's arrival for its (request, row unit) once all four
  // CTAs have written their part; the cluster whose arrival completes the
  // count (shards x splits) resets it and merges the unit's rows, every part
  // being in memory by then.  No cluster waits for another.
  auto fused_arrival = [&]() {
    if (rank == 0 && threadIdx.x == 0) {
      const int unit_u = w.r_base / MLA_ROWS_PER_UNIT;
      int* c = p.counters + (int64_t)w.b * p.U + unit_u;
      const int total = p.num_splits * (p.V / p.B);
      const bool last = atom_add_acq_rel_gpu(c, 1) == total - 1;
      if (last) *c = 0;
      for (uint32_t k = 0; k < kCtas; ++k)
        st_cluster_u32(mapa(smem_u32(&s.ctl_last), k), last ? 1u : 0u);
    }
  };
  auto fused_combine = [&]() {
    if (!*reinterpret_cast<volatile int*>(&s.ctl_last)) return;
    __threadfence();
    const int R = p.q_len * p.H;
    const int r0 = w.r_base / MLA_ROWS_PER_UNIT * MLA_ROWS_PER_UNIT;
    const int n = min(MLA_ROWS_PER_UNIT, R - r0);
    const int64_t rows = (int64_t)p.B * R;
    const int P = p.num_splits * (p.V / p.B);
    constexpr int kWarps = kThreads / 32;
    for (int r = (int)rank * kWarps + warp; r < n; r += kCtas * kWarps)
      combine_row<true>(p.O_part, p.LSE_part, P, rows,
                        (int64_t)w.b * R + r0 + r, p.out, p.lse_out, lane);
  };

  // Teardown, repeated at the end of every S-CTA role: they never rejoin, so no
  // warp ever asks setmaxnreg for registers back.  The pair's TMEM is released
  // only after all four CTAs are done with it.
  auto teardown = [&]() {
    if (p.counters) __threadfence();  // this CTA's part before the arrival
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
    if (p.counters) fused_arrival();
    cluster_sync();
    if (p.counters) fused_combine();
  };

  const bool leads = (rank & 1) == 0;
  if (w.npages > 0 && rank < 2) {
    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
      if (warp == 0) {
        copy_pages(s, p, w, (int)rank, kTilePages, lane);
      } else if (warp == 1) {
        if (leads && elect_one()) mma_s(s, p, w, tmem, rank);
      } else if (warp == 2) {
        if (!leads && lane == 0)
          relay_made(s, p, (w.npages + 1) / kTilePages * kStagesS, kStagesS, rank, 0);
      } else if (lane == 0) {
        ship_pages(s, p, w, rank);
      }
      __syncwarp();
      teardown();
      return;
    }
    if (warp >= kDequantWarp0) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
      convert_s(s, p, w, rank, (warp - kDequantWarp0) * 32 + lane, lane);
      teardown();
      return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax(s, p, w, tmem, rank, warp, lane);
    teardown();
    return;
  }
  if (w.npages > 0) {
    if (warp == 0) {
      copy_pages(s, p, w, 0, 1, lane);
    } else if (warp == 1) {
      if (elect_one()) {
        if (leads)
          mma_o(s, p, w, tmem, rank);
        else
          relay_o(s, p, w, rank);
      }
      __syncwarp();
    } else if (warp == 2) {
      if (lane == 0 && !leads) relay_made(s, p, w.npages, kStagesO, rank, 2);
      __syncwarp();
    } else if (warp >= 4 && warp < 8) {
      correct_and_store(s, p, &o_map, w, tmem, rank, warp, lane);
    } else if (warp >= kDequantWarp0) {
      convert_o(s, p, w, rank, (warp - kDequantWarp0) * 32 + lane, lane);
    } else if (warp >= 8) {
      store_o_upper(s, p, &o_map, w, tmem, warp, lane);
    }
  } else if (rank < 2 && threadIdx.x == 0) {
    // No tokens for this split: the query boxes issued at entry land before
    // the CTA leaves.
    mbar_wait(smem_u32(&s.qbar), 0, &s.abort_flag);
  }
  if (w.npages == 0 && warp >= 4 && warp < 8) {
    // No tokens for this split: O = 0 (O-CTAs), LSE = -inf (S-CTAs).
    const int r = (warp & 3) * 32 + lane;
    if (r < w.nrows) {
      const int64_t rows = (int64_t)p.B * p.q_len * p.H;
      const int64_t part = (int64_t)w.split * (p.V / p.B) + w.shard;
      const int64_t orow =
          part * rows + (int64_t)w.b * p.q_len * p.H + w.r_base + r;
      if (rank < 2) {
        p.LSE_part[orow] = -INFINITY;
      } else if (p.o_bf16) {
        uint4* d = reinterpret_cast<uint4*>(
            reinterpret_cast<__nv_bfloat16*>(p.O_part) + orow * MLA_VALUE_DIM);
        for (int e = 0; e < MLA_VALUE_DIM / 8; ++e) d[e] = make_uint4(0, 0, 0, 0);
      } else {
        float4* d4 = reinterpret_cast<float4*>(p.O_part + orow * MLA_VALUE_DIM);
        for (int e = 0; e < MLA_VALUE_DIM / 4; ++e)
          d4[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  }
  teardown();
}

}  // namespace

int launch_fp4(const DecodeArgs& a) {
  Fp4Params p;
  p.q_nope = static_cast<const uint4*>(a.q_nope);
  p.q_rope = static_cast<const uint4*>(a.q_rope);
  p.kv = static_cast<const uint8_t*>(a.kv);
  p.g = a.kv_scale;
  p.num_slots = a.num_slots;
  p.r2t = a.req_to_token;
  p.r2t_stride = a.r2t_stride;
  p.seq_lens = a.seq_lens;
  p.kv_limit = a.kv_limit;
  p.split_pages = a.split_pages;
  p.work = a.work;
  p.B = a.B;
  p.q_len = a.q_len;
  p.H = a.H;
  p.V = a.B * a.num_shards;
  p.num_splits = a.num_splits;
  p.U = (a.q_len * a.H + MLA_ROWS_PER_UNIT - 1) / MLA_ROWS_PER_UNIT;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.O_part = a.O_part;
  p.LSE_part = a.LSE_part;
  p.status = a.status;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse_out = a.lse_out;
  p.counters = a.counters;
  const int64_t units = (int64_t)p.V * p.num_splits * p.U;
  if (units * kCtas > 0x7fffffff)
    return fail(MLA_ERR_INVALID_ARG, "grid too large");
  p.o_bf16 = a.o_bf16;
  if (few_row_groups(a)) {
    p.U = (a.q_len * a.H + kFp4FewRows - 1) / kFp4FewRows;
    // two groups may count in the halves of one counter
    if (a.counters && p.U > 1 && (int64_t)a.num_splits * a.num_shards > 0xFFFF)
      return fail(MLA_ERR_UNSUPPORTED, "one launch over groups of %d rows: %lld parts above %d",
                  kFp4FewRows, (long long)a.num_splits * a.num_shards, 0xFFFF);
    return launch_fp4_few(p, a.stream);
  }
  CUtensorMap qn_map, qr_map;
  int rc = make_query_maps(&qn_map, &qr_map, a, &p.q_box_rows);
  if (rc != MLA_OK) return rc;
  // The partial outputs leave by TMA store when their rows fit the tensor
  // map's 32-bit coordinates; the fused combine, which reads other
  // clusters' parts in the same launch, keeps the plain stores its fences
  // order.
  CUtensorMap o_map;
  std::memset(&o_map, 0, sizeof(o_map));
  const int64_t o_rows =
      (int64_t)p.num_splits * a.num_shards * a.B * a.q_len * a.H;
  if (p.o_bf16) {
    const uint64_t dims[3] = {(uint64_t)MLA_VALUE_DIM, (uint64_t)o_rows, 1};
    const uint64_t strides[2] = {(uint64_t)MLA_VALUE_DIM * 2,
                                 (uint64_t)o_rows * MLA_VALUE_DIM * 2};
    const uint32_t box[3] = {64, 32, 1};
    p.o_tma = !p.counters && o_rows < 0x7fffffff &&
              make_tensor_map_bf16_3d(&o_map, p.O_part, dims, strides, box) ==
                  MLA_OK;
  } else {
    p.o_tma = !p.counters && o_rows < 0x7fffffff &&
              make_o_part_map(&o_map, p.O_part, o_rows) == MLA_OK;
  }
  cudaError_t e = cudaFuncSetAttribute(
      mla_partial_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(fp4)");
  mla_partial_fp4_kernel<<<(unsigned)(units * kCtas), kThreads, kSmemBytes, a.stream>>>(
      qn_map, qr_map, o_map, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_partial_fp4_kernel");
  return MLA_OK;
}

}  // namespace mla
