// mla_pages.cu -- the page table of a serving step that may branch: rows taken
// over from other rows, shared, shortened, grown, started and ended
// (mla_pages_fork), a pool's live pages moved into its holes
// (mla_pages_compact), and the copy of pages that both ask for (mla_kv_copy).
//
// A page is 64 slots; refs[page] counts the rows that hold it, 0 = free.  Page 0
// is the pool's dummy page: never counted, never given out.  Both bookkeeping
// kernels are one cluster of 8 CTAs: their phases are separated by cluster
// barriers (about 1 us, against 2 us and more for a launch), counts travel
// through distributed shared memory, and every result (which page a row gets,
// where a page moves) is a rank in a fixed order, so it does not depend on
// which CTA was first.  The full pages that rows take over are copied by the rest of
// the grid meanwhile.
//
// Measured: 4 rows forked in 10 us, 256 rows of up to 265 pages in 21 (bound by chains
// of trips to L2: arguments, lengths, table, counts; then the changes of counts, two
// trips each, 10 a thread), a pool of 29 000 pages compacted with 7231 moves and a
// table of 200 rows in 17, and those 326 MB copied in 52, 93% of the copy rate.
#include <algorithm>
#include <atomic>

#include "mla_internal.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kPage = MLA_PAGE_SIZE;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kPerThread = 16;                      // pages a thread looks at in one round
constexpr int kPerCta = kThreads * kPerThread;      // 8192
constexpr int kMaxRows = MLA_FORK_MAX_ROWS;

__host__ __device__ inline int64_t pages_of(int64_t tokens) { return (tokens + kPage - 1) / kPage; }

// Exclusive prefix sum of one int per thread; *total receives the block's sum.
// `scratch`: kWarps ints.
__device__ __forceinline__ int block_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, s, d);
    if (lane >= d) s += o;
  }
  __syncthreads();  // the scratch of an earlier call has been read
  if (lane == 31) scratch[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int x = scratch[w];
    before += w < warp ? x : 0;
    all += x;
  }
  *total = all;
  return before + s - v;
}

// Tell every CTA of the cluster this CTA's two counts: box[2 * rank + {0, 1}].
__device__ __forceinline__ void publish(int* box, uint32_t rank, int a, int b) {
  if (threadIdx.x < kCluster) {
    const uint32_t at = mapa(smem_u32(box + 2 * rank), threadIdx.x);
    st_cluster_u32(at, (uint32_t)a);
    st_cluster_u32(at + 4, (uint32_t)b);
  }
}

// ---------------------------------------------------------------------- fork
struct ForkParams {
  const int32_t* table;
  int64_t stride;
  const int32_t* lens;
  const int32_t* parents;  // NULL: row i goes on as row i
  const int32_t* keep;     // NULL: all of the parent's tokens
  const int32_t* grow;     // NULL: none
  int R;
  int32_t* refs;
  int64_t num_pages;
  int32_t* free_count;
  int32_t* out;
  int64_t out_stride;
  int32_t* lens_out;
  int32_t* copies;  // [3, R]: source page, destination page, tokens
  int* status;
  int vec;          // rows of both tables start on 16-byte boundaries
  int chunks;       // chunks of kChunk entries a row
  int refs_vec;     // refs starts on a 16-byte boundary
};

constexpr int kChunk = 4096;  // entries of one row that a CTA copies at a time (16 KB)

// Row i of the new table: its parent (-1: none) and the tokens taken from it;
// negative tokens: the arguments are no valid row.
__device__ __forceinline__ int taken(const ForkParams& p, int i, int* parent) {
  const int from = p.parents ? p.parents[i] : i;
  *parent = from;
  if (from < -1 || from >= p.R) return -1;
  const int want = p.keep ? p.keep[i] : 0x7fffffff;
  if (from < 0) return 0;
  const int held = p.lens[from];
  if (held < 0 || held > p.stride || want < 0) return -1;
  return min(want, held);
}

// Entries 4 q .. 4 q + 3 of a row's page `at`, cut at the row's end.
__device__ __forceinline__ void write_quad(const ForkParams& p, int row, int64_t at, int page, int q) {
  const int64_t e = at * kPage + 4 * q;
  int32_t* dst = p.out + row * p.out_stride + e;
  const int base = page * kPage + 4 * q;
  if (p.vec && e + 4 <= p.out_stride) {
    *reinterpret_cast<int4*>(dst) = make_int4(base, base + 1, base + 2, base + 3);
  } else {
    for (int j = 0; j < 4 && e + j < p.out_stride; ++j) dst[j] = base + j;
  }
}

// The full pages that a row takes over: entries copied as they are, by every
// CTA past the first cluster.  They depend on nothing that the cluster decides.
__device__ void copy_rows(const ForkParams& p) {
  const int64_t tasks = (int64_t)p.R * p.chunks, step = gridDim.x - kCluster;
  for (int64_t t = blockIdx.x - kCluster; t < tasks; t += step) {
    const int i = (int)(t / p.chunks);
    const int64_t e0 = (t % p.chunks) * kChunk;
    int from;
    const int kept = taken(p, i, &from);
    if (kept < 0 || from < 0) continue;
    const int64_t n = min((int64_t)kept / kPage * kPage, p.out_stride);
    const int64_t e1 = min(e0 + kChunk, n);
    const int32_t* src = p.table + from * p.stride;
    int32_t* dst = p.out + i * p.out_stride;
    if (p.vec) {
      // n is a multiple of 4: pages, or a row's stride, which then is one
      int4 v[kChunk / (4 * kThreads)];
#pragma unroll
      for (int u = 0; u < kChunk / (4 * kThreads); ++u) {
        const int64_t e = e0 + 4 * (threadIdx.x + u * kThreads);
        if (e < e1) v[u] = __ldg(reinterpret_cast<const int4*>(src + e));
      }
#pragma unroll
      for (int u = 0; u < kChunk / (4 * kThreads); ++u) {
        const int64_t e = e0 + 4 * (threadIdx.x + u * kThreads);
        if (e < e1) *reinterpret_cast<int4*>(dst + e) = v[u];
      }
    } else {
      for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) dst[e] = src[e];
    }
  }
}

// What a child asks of its parent, for choosing the heir: most pages taken
// first (a partly taken one counts half), then the lowest row.
__device__ __forceinline__ unsigned long long claim(int kept, int i) {
  return ((unsigned long long)(2u * (kept / kPage) + (kept % kPage != 0) + 1) << 32) |
         (uint32_t)(0x7fffffff - i);
}

__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
    mla_pages_fork_kernel(const ForkParams p) {
  if (blockIdx.x >= kCluster) {
    copy_rows(p);
    return;
  }
  extern __shared__ unsigned long long fork_smem[];
  unsigned long long* best = fork_smem;                      // [R] the heir's claim
  int* kept = reinterpret_cast<int*>(best + p.R);            // [R] tokens taken
  int* from = kept + p.R;                                    // [R] parent
  int* first = from + p.R;                                   // [R + 1] rank of the row's first new page
  int* tail = first + p.R + 1;                               // [R] partly taken page; its sign: copied
  int* held = tail + p.R;                                    // [R] pages of the old row
  uint32_t* ops = reinterpret_cast<uint32_t*>(held + p.R);   // [R + 1] counts to change before the row's
  __shared__ int scratch[kWarps], box[2][2 * kCluster], bad, freed;
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, R = p.R;
  if (tid == 0) bad = freed = 0;
  for (int i = tid; i < R; i += kThreads) best[i] = 0;
  __syncthreads();

  // Every CTA of the cluster works out the same decisions, from arguments and
  // counts that nobody changes before the first cluster barrier.
  for (int i = tid; i < R; i += kThreads) {
    int parent;
    const int k = taken(p, i, &parent);
    const int64_t g = p.grow ? p.grow[i] : 0, old = p.lens[i];
    if (k < 0) {
      atomicOr(&bad, parent < -1 || parent >= R ? MLA_STATUS_BAD_PARENT : MLA_STATUS_BAD_LENGTH);
    } else if (g < 0 || k + g > p.out_stride || old < 0 || old > p.stride) {
      atomicOr(&bad, MLA_STATUS_BAD_LENGTH);
    }
    kept[i] = max(k, 0);
    held[i] = (int)pages_of(max(old, (int64_t)0));
    from[i] = parent;
    if (k >= 0 && parent >= 0) atomicMax(&best[parent], claim(k, i));
  }
  __syncthreads();
  if (bad == 0) {
    for (int i = tid; i < R; i += kThreads) {
      const int k = kept[i], parent = from[i];
      int t = -1;
      if (parent >= 0 && k % kPage) {
        t = p.table[parent * p.stride + k / kPage * kPage] / kPage;
        if (t < 1 || t >= p.num_pages) {
          atomicOr(&bad, MLA_STATUS_BAD_SLOT);
          t = -1;
        } else if (best[parent] != claim(k, i) || p.refs[t] != 1) {
          t = -1 - t;  // somebody else holds it too: copied
        }
      }
      tail[i] = t;  // > 0: the row keeps it, < -1: page -1 - t is copied, -1: none
    }
  }
  __syncthreads();
  // Ranks of the new pages: rows in order, a row's pages in order.
  int64_t total = 0;
  if (bad == 0) {
    int carry = 0;
    for (int i0 = 0; i0 < R; i0 += kThreads) {
      const int i = i0 + tid;
      int need = 0;
      if (i < R)
        need = (int)(pages_of(kept[i] + (int64_t)(p.grow ? p.grow[i] : 0)) - kept[i] / kPage) -
               (tail[i] > 0);
      int sum;
      const int before = block_scan(need, scratch, &sum);
      if (i < R) first[i] = carry + before;
      carry += sum;  // at most R * stride / 64, checked on the host
    }
    if (tid == 0) first[R] = carry;
    total = carry;
    if (tid == 0 && total > *p.free_count) bad = MLA_STATUS_NO_PAGES;
  }
  __syncthreads();
  const int broken = bad;
  // No CTA changes a count before every CTA has read those it decides on.
  cluster_sync();
  if (broken) {
    if (rank == 0) {
      for (int i = tid; i < R; i += kThreads) {
        p.lens_out[i] = 0;
        p.copies[i] = p.copies[R + i] = -1;
        p.copies[2 * R + i] = 0;
      }
      if (tid == 0 && p.status) atomicOr(p.status, broken);
    }
    return;
  }

  const auto row_of = [&](int r) {  // the last row whose first rank is not above r
    int lo = 0, hi = R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= r) lo = mid; else hi = mid;
    }
    return lo;
  };
  // The lowest free pages, in rounds of 8 x 8192 counts.
  int found = 0;
  for (int round = 0; found < total; ++round) {
    const int64_t p0 = ((int64_t)round * kCluster + rank) * kPerCta + tid * kPerThread;
    if ((int64_t)round * kCluster * kPerCta >= p.num_pages) break;  // uniform in the cluster
    uint32_t zero = 0;
    if (p0 + kPerThread <= p.num_pages && p.refs_vec) {
#pragma unroll
      for (int u = 0; u < kPerThread; u += 4) {
        const int4 v = *reinterpret_cast<const int4*>(p.refs + p0 + u);
        zero |= (uint32_t)(v.x == 0) << u | (uint32_t)(v.y == 0) << (u + 1) |
                (uint32_t)(v.z == 0) << (u + 2) | (uint32_t)(v.w == 0) << (u + 3);
      }
    } else {
      for (int u = 0; u < kPerThread; ++u)
        if (p0 + u < p.num_pages) zero |= (uint32_t)(p.refs[p0 + u] == 0) << u;
    }
    if (p0 == 0) zero &= ~1u;  // the dummy page
    int sum;
    int r = block_scan(__popc(zero), scratch, &sum);
    int* b = box[round & 1];
    publish(b, rank, sum, 0);
    cluster_sync();
    int all = 0;
    for (int c = 0; c < kCluster; ++c) {
      if (c < (int)rank) r += b[2 * c];
      all += b[2 * c];
    }
    r += found;
    found += all;
    // Of a new page only the first entry is written here: the lowest pages are mostly
    // one CTA's, and all of them write the rest.
    for (; zero && r < total; zero &= zero - 1, ++r) {
      const int page = (int)(p0 + __ffs(zero) - 1), row = row_of(r), nth = r - first[row];
      p.refs[page] = 1;
      p.out[row * p.out_stride + (kept[row] / kPage + (tail[row] > 0) + (int64_t)nth) * kPage] = page * kPage;
      if (nth == 0 && tail[row] < -1) p.copies[R + row] = page;
    }
  }
  cluster_arrive();
  // A count of free pages above what the pool has: the last rows end with the pages
  // that they hold.
  const int given = (int)min((int64_t)found, total);
  if (given < total && rank == 0 && tid == 0 && p.status) atomicOr(p.status, MLA_STATUS_NO_PAGES);

  // Counts.  Of a parent's pages its heir goes on holding those it takes; the
  // rest lose the parent, and every other child adds its full pages.  A page
  // that gains a holder has one that stays (the heir takes at least as many
  // pages), so a count that reaches 0 is final.  The changes of all rows are dealt
  // out evenly, kOps of a thread under way at once: rows differ in length, and a
  // change takes two trips to L2 (a warp a row took longest with one long row).
  const auto stays = [&](int i) {  // pages of row i that its heir goes on holding
    const unsigned long long b = best[i];
    const int heir = b ? 0x7fffffff - (int)(uint32_t)b : -1;
    return heir < 0 ? 0 : min(held[i], kept[heir] / kPage + (tail[heir] > 0));
  };
  uint32_t changes = 0;
  for (int i0 = 0; i0 < R; i0 += kThreads) {
    const int i = i0 + tid;
    uint32_t mine = 0;
    if (i < R) {
      const int parent = from[i];
      mine = (uint32_t)(held[i] - stays(i));
      if (parent >= 0 && best[parent] != claim(kept[i], i)) mine += (uint32_t)(kept[i] / kPage);
    }
    int sum;
    const int before = block_scan((int)mine, scratch, &sum);
    if (i < R) ops[i] = changes + (uint32_t)before;
    changes += (uint32_t)sum;
  }
  if (tid == 0) ops[R] = changes;
  __syncthreads();
  constexpr int kOps = 8;
  int lost = 0;
  bool bad_slot = false;
  for (int64_t t0 = rank * kThreads + tid; t0 < changes; t0 += (int64_t)kOps * kCluster * kThreads) {
    int page[kOps];
    bool less[kOps];
#pragma unroll
    for (int u = 0; u < kOps; ++u) {
      const int64_t t = t0 + (int64_t)u * kCluster * kThreads;
      page[u] = 0;
      if (t >= changes) continue;
      int lo = 0, hi = R;  // the last row whose changes start at t or before
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (ops[mid] <= (uint32_t)t) lo = mid; else hi = mid;
      }
      const int skip = stays(lo), nth = (int)((uint32_t)t - ops[lo]);
      less[u] = nth < held[lo] - skip;
      const int e = less[u] ? p.table[lo * p.stride + (int64_t)(skip + nth) * kPage]
                            : p.table[from[lo] * p.stride + (int64_t)(nth - (held[lo] - skip)) * kPage];
      page[u] = e / kPage;
      if (e < 0 || page[u] >= p.num_pages) bad_slot = true, page[u] = 0;
    }
#pragma unroll
    for (int u = 0; u < kOps; ++u) {
      if (page[u] <= 0) continue;
      if (less[u]) lost += atomicSub(&p.refs[page[u]], 1) == 1;
      else atomicAdd(&p.refs[page[u]], 1);
    }
  }
  for (int i = rank * kThreads + tid; i < R; i += kCluster * kThreads) {
    int64_t len = kept[i] + (int64_t)(p.grow ? p.grow[i] : 0);
    const int t = tail[i];
    if (first[i + 1] > given) len = min(len, ((int64_t)(kept[i] / kPage) + (t > 0) + max(given - first[i], 0)) * kPage);
    p.lens_out[i] = (int)len;
    const bool copied = t < -1 && first[i] < given;
    p.copies[i] = copied ? -1 - t : -1;
    if (!copied) p.copies[R + i] = -1;
    p.copies[2 * R + i] = copied ? kept[i] % kPage : 0;
  }
  // Entries: kept partly taken pages, then the new ones', 16 threads a page.
  for (int64_t t = rank * kThreads + tid; t < (int64_t)R * 16; t += kCluster * kThreads) {
    const int i = (int)(t / 16);
    if (tail[i] > 0) write_quad(p, i, kept[i] / kPage, tail[i], (int)(t % 16));
  }
  cluster_wait();  // the new pages' first entries; the boxes have been read, too
  for (int64_t t = rank * kThreads + tid; t < (int64_t)given * 16; t += kCluster * kThreads) {
    const int r = (int)(t / 16), row = row_of(r);
    const int64_t at = kept[row] / kPage + (tail[row] > 0) + r - first[row];
    const int page = p.out[row * p.out_stride + at * kPage] / kPage;
    write_quad(p, row, at, page, (int)(t % 16));
  }
  if (bad_slot && p.status) atomicOr(p.status, MLA_STATUS_BAD_SLOT);
  if (lost) atomicAdd(&freed, lost);
  __syncthreads();
  int* b = box[0];
  publish(b, rank, freed, 0);
  cluster_sync();
  if (rank == 0 && tid == 0) {
    int sum = 0;
    for (int c = 0; c < kCluster; ++c) sum += b[2 * c];
    *p.free_count += sum - given;
  }
}

// ------------------------------------------------------------------- compact
struct CompactParams {
  int32_t* refs;
  int64_t num_pages;
  int32_t* src;
  int32_t* dst;
  int max_moves;
  int32_t* count;
  int refs_vec;  // refs starts on a 16-byte boundary
};

struct RenameParams {
  const int32_t* table;
  int64_t stride;
  const int32_t* lens;
  int32_t* out;
  int64_t out_stride;
  int R, chunks, vec;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;
  int* status;
};

// The table's live entries with the moved pages' new numbers, a chunk of a row
// at a time.  The moved pages are the highest live ones, so src is sorted
// (descending) and an entry below its last is not moved; others find their place
// by bisection.
__device__ void rename_rows(const RenameParams& p, int moves, int64_t first, int64_t step) {
  const int lowest = moves ? p.src[moves - 1] : 0x7fffffff;
  const auto renamed = [&](int e) {
    const int page = e / kPage;
    if (page < lowest) return e;
    int lo = 0, hi = moves;  // the first entry not above the page
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.src[mid] > page) lo = mid + 1; else hi = mid;
    }
    return lo < moves && p.src[lo] == page ? p.dst[lo] * kPage + e % kPage : e;
  };
  const bool in_place = p.table == p.out;
  const int64_t tasks = (int64_t)p.R * p.chunks;
  for (int64_t t = first; t < tasks; t += step) {
    const int i = (int)(t / p.chunks);
    const int64_t e0 = (t % p.chunks) * kChunk;
    const int64_t len = p.lens[i], room = min(p.stride, p.out_stride);
    if (len < 0 || len > room) {
      if (e0 == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, MLA_STATUS_BAD_LENGTH);
      continue;
    }
    const int64_t e1 = min(min(e0 + kChunk, pages_of(len) * kPage), room);
    const int32_t* src = p.table + i * p.stride;
    int32_t* dst = p.out + i * p.out_stride;
    if (p.vec) {
      int4 v[kChunk / (4 * kThreads)];
#pragma unroll
      for (int u = 0; u < kChunk / (4 * kThreads); ++u) {
        const int64_t e = e0 + 4 * (threadIdx.x + u * kThreads);
        if (e < e1) v[u] = *reinterpret_cast<const int4*>(src + e);
      }
#pragma unroll
      for (int u = 0; u < kChunk / (4 * kThreads); ++u) {
        const int64_t e = e0 + 4 * (threadIdx.x + u * kThreads);
        if (e >= e1) continue;
        const int x = renamed(v[u].x);  // four entries of one page
        if (in_place && x == v[u].x) continue;
        *reinterpret_cast<int4*>(dst + e) = make_int4(x, v[u].y + (x - v[u].x), v[u].z + (x - v[u].x),
                                                      v[u].w + (x - v[u].x));
      }
    } else {
      for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) {
        const int x = renamed(src[e]);
        if (!in_place || x != src[e]) dst[e] = x;
      }
    }
  }
}

// The k-th lowest hole among pages 1 .. n and the k-th highest live page above
// n, n the number of live pages: after all moves exactly the pages 1 .. n are
// live.  Every thread has a run of pages of its own and looks at it three times
// (from L2 after the first); between them two sums over the block and the cluster.
template <bool kRename>
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
    mla_pages_compact_kernel(const CompactParams p, const RenameParams r) {
  __shared__ int scratch[kWarps], box[2][2 * kCluster];
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x;
  griddep_launch_dependents();
  cluster_arrive();  // the CTAs have started when they write to each other
  const int64_t run = ((p.num_pages + kCluster * kThreads - 1) / (kCluster * kThreads) + 3) / 4 * 4;
  const int64_t a = min(run * (rank * kThreads + tid), p.num_pages), z = min(a + run, p.num_pages);
  // f(page, live) for the thread's pages but the dummy one
  const auto walk = [&](auto f) {
    for (int64_t i = a; i < z; i += 4) {
      int r[4];
      if (p.refs_vec && i + 4 <= z) {
        *reinterpret_cast<int4*>(r) = *reinterpret_cast<const int4*>(p.refs + i);
      } else {
        for (int u = 0; u < 4; ++u) r[u] = i + u < z ? p.refs[i + u] : 0;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u > 0 && i + u < z) f(i + u, r[u] > 0);
    }
  };
  int live = 0;
  walk([&](int64_t, bool is) { live += is; });
  int sum;
  block_scan(live, scratch, &sum);
  cluster_wait();
  publish(box[0], rank, sum, 0);
  cluster_sync();
  int64_t n = 0;
  for (int c = 0; c < kCluster; ++c) n += box[0][2 * c];
  int holes = 0, high = 0;
  walk([&](int64_t i, bool is) {
    holes += i <= n && !is;
    high += i > n && is;
  });
  int my_holes, my_high;
  int hole_at = block_scan(holes, scratch, &my_holes), high_at = block_scan(high, scratch, &my_high);
  publish(box[1], rank, my_holes, my_high);
  cluster_sync();
  int all = 0;
  for (int c = 0; c < kCluster; ++c) {
    if (c < (int)rank) hole_at += box[1][2 * c], high_at += box[1][2 * c + 1];
    all += box[1][2 * c + 1];
  }
  const int moves = min(all, p.max_moves);
  if ((holes && hole_at < moves) || (high && all - high_at - high < moves))
    walk([&](int64_t i, bool is) {
      if (i <= n && !is) {
        if (hole_at < moves) p.dst[hole_at] = (int)i;
        ++hole_at;
      }
      if (i > n && is) {
        const int g = all - 1 - high_at++;
        if (g < moves) p.src[g] = (int)i;
      }
    });
  cluster_sync();
  for (int k = rank * kThreads + tid; k < p.max_moves; k += kCluster * kThreads) {
    if (k < moves) {
      const int s = p.src[k];
      p.refs[p.dst[k]] = p.refs[s];
      p.refs[s] = 0;
    } else {
      p.src[k] = p.dst[k] = -1;
    }
  }
  if (rank == 0 && tid == 0) *p.count = moves;
  if constexpr (kRename) rename_rows(r, moves, rank, kCluster);
}

__global__ void __launch_bounds__(kThreads) mla_pages_rename_kernel(const RenameParams p) {
  griddep_wait();
  rename_rows(p, *p.count, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------------- copy
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;  // 16-byte vectors in flight per thread
constexpr int kSlice = kCopyThreads * kCopyVecs;  // vectors of a block's turn: less than a page's

// All entries' pages as one sequence of 16-byte vectors, so that every turn is
// full whatever a page takes (slices of a page: 326 MB in 4-bit pages took 60 us).
__global__ void __launch_bounds__(kCopyThreads)
    mla_kv_copy_kernel(uint8_t* kv, float* scale, int row_vecs, int64_t num_pages,
                       const int32_t* src, const int32_t* dst, const int32_t* tokens,
                       const int32_t* count, int64_t n, int* status) {
  griddep_wait();
  if (count) n = min(n, (int64_t)max(*count, 0));
  const int vecs = kPage * row_vecs;  // of a page
  uint4* pool = reinterpret_cast<uint4*>(kv);
  for (int64_t t = (int64_t)blockIdx.x * kSlice; t < n * vecs; t += (int64_t)gridDim.x * kSlice) {
    const int64_t entry = t / vecs;
    const int at = (int)(t - entry * vecs) + threadIdx.x;
    uint4 v[kCopyVecs];
    int64_t to[kCopyVecs];
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u) {
      const int past = at + u * kCopyThreads >= vecs, o = at + u * kCopyThreads - past * vecs;
      const int64_t i = entry + past;
      to[u] = -1;
      if (i >= n) continue;
      const int s = src[i], d = dst[i];
      if (s < 0 || d < 0 || s == d) continue;
      if (s >= num_pages || d >= num_pages) {
        if (o == 0 && status) atomicOr(status, MLA_STATUS_BAD_SLOT);
        continue;
      }
      const int live = tokens ? min(max(tokens[i], 0), kPage) : kPage;
      if (o >= live * row_vecs) continue;
      v[u] = pool[(int64_t)s * vecs + o];
      to[u] = (int64_t)d * vecs + o;
      if (scale && o < live) scale[(int64_t)d * kPage + o] = scale[(int64_t)s * kPage + o];
    }
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u)
      if (to[u] >= 0) pool[to[u]] = v[u];
  }
}

// A launch whose first instructions may overlap the end of the kernel before it
// in the stream (which the kernel waits for).
template <class... Args>
cudaError_t launch_after(void (*kernel)(Args...), unsigned grid, unsigned threads, cudaStream_t st,
                         Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_pages_fork(const int32_t* table, int64_t stride, const int32_t* lens,
                              const int32_t* parents, const int32_t* keep, const int32_t* grow,
                              int R, int32_t* refs, int64_t num_pages, int32_t* free_count,
                              int32_t* table_out, int64_t out_stride, int32_t* lens_out,
                              int32_t* copies, int* status, mla_stream_t stream) {
  if (R < 0 || stride < 1 || out_stride < 1 || num_pages < 1)
    return fail(MLA_ERR_INVALID_ARG, "mla_pages_fork: R %d < 0 or strides %lld, %lld or pages %lld < 1",
                R, (long long)stride, (long long)out_stride, (long long)num_pages);
  if (R == 0) return MLA_OK;
  if (R > kMaxRows)
    return fail(MLA_ERR_UNSUPPORTED, "mla_pages_fork: R %d > %d rows", R, kMaxRows);
  if (num_pages > ((int64_t)1 << 31) / kPage || stride > 0x7fffffff || out_stride > 0x7fffffff ||
      R * pages_of(std::max(stride, out_stride)) > 0x3fffffff)
    return fail(MLA_ERR_INVALID_ARG, "mla_pages_fork: more than 2^31 slots or 2^30 table pages");
  if (!table || !lens || !refs || !free_count || !table_out || !lens_out || !copies)
    return fail(MLA_ERR_INVALID_ARG, "mla_pages_fork: a required pointer is NULL");
  if (table_out < table + (R - 1) * stride + stride && table < table_out + (R - 1) * out_stride + out_stride)
    return fail(MLA_ERR_INVALID_ARG, "mla_pages_fork: table_out overlaps table");
  if (lens == lens_out)
    return fail(MLA_ERR_INVALID_ARG, "mla_pages_fork: lens_out is lens");
  const void* all[] = {table, lens, parents, keep, grow, refs, free_count, table_out, lens_out, copies, status};
  for (const void* q : all)
    if (q && !aligned(q, 4)) return fail(MLA_ERR_MISALIGNED, "mla_pages_fork: arrays need 4-B alignment");
  ForkParams p{table, stride, lens, parents, keep, grow, R, refs, num_pages, free_count,
               table_out, out_stride, lens_out, copies, status};
  p.vec = aligned(table, 16) && aligned(table_out, 16) && stride % 4 == 0 && out_stride % 4 == 0;
  p.chunks = (int)((std::min(stride, out_stride) + kChunk - 1) / kChunk);
  p.refs_vec = aligned(refs, 16);
  int dev = 0, sms = 0;
  const int rc = device_sms(&dev, &sms);
  if (rc != MLA_OK) return rc;
  // up to two CTAs per SM for the copies, in whole clusters
  const int64_t tasks = (int64_t)R * p.chunks;
  const int64_t clusters = 1 + std::min<int64_t>((tasks + kCluster - 1) / kCluster, 2 * sms / kCluster);
  const int smem = R * 8 + (6 * R + 2) * 4;
  static_assert(kMaxRows * 32 + 8 <= 200 * 1024, "shared memory budget");
  static std::atomic<uint64_t> set_on{0};
  if (smem > 47 * 1024) {
    const int set = allow_shared(mla_pages_fork_kernel, kMaxRows * 32 + 8, dev, set_on, "cudaFuncSetAttribute(mla_pages_fork_kernel)");
    if (set != MLA_OK) return set;
  }
  mla_pages_fork_kernel<<<(unsigned)(clusters * kCluster), kThreads, smem, (cudaStream_t)stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_pages_fork_kernel");
  return MLA_OK;
}

extern "C" int mla_pages_compact(const int32_t* table, int64_t stride, const int32_t* lens, int R,
                                 int32_t* refs, int64_t num_pages, int32_t* table_out,
                                 int64_t out_stride, int32_t* src, int32_t* dst, int max_moves,
                                 int32_t* count, int* status, mla_stream_t stream) {
  if (R < 0 || stride < 1 || out_stride < 1 || num_pages < 1 || max_moves < 0)
    return fail(MLA_ERR_INVALID_ARG, "mla_pages_compact: R %d or max_moves %d < 0, or strides %lld, "
                "%lld or pages %lld < 1", R, max_moves, (long long)stride, (long long)out_stride,
                (long long)num_pages);
  if (num_pages > ((int64_t)1 << 31) / kPage || stride > 0x7fffffff || out_stride > 0x7fffffff)
    return fail(MLA_ERR_INVALID_ARG, "mla_pages_compact: more than 2^31 slots or table entries a row");
  if (!refs || !count || (R > 0 && (!table || !lens || !table_out)) || (max_moves > 0 && (!src || !dst)))
    return fail(MLA_ERR_INVALID_ARG, "mla_pages_compact: a required pointer is NULL");
  const bool overlap = R > 0 && table_out < table + (R - 1) * stride + stride &&
                       table < table_out + (R - 1) * out_stride + out_stride;
  if (overlap && (table != table_out || stride != out_stride))
    return fail(MLA_ERR_INVALID_ARG, "mla_pages_compact: table_out overlaps table without being it");
  const void* all[] = {table, lens, refs, table_out, src, dst, count, status};
  for (const void* q : all)
    if (q && !aligned(q, 4)) return fail(MLA_ERR_MISALIGNED, "mla_pages_compact: arrays need 4-B alignment");
  const cudaStream_t st = (cudaStream_t)stream;
  const CompactParams c{refs, num_pages, src, dst, max_moves, count, aligned(refs, 16)};
  RenameParams p{table, stride, lens, table_out, out_stride, R, 0, 0, src, dst, count, status};
  p.vec = R > 0 && aligned(table, 16) && aligned(table_out, 16) && stride % 4 == 0 && out_stride % 4 == 0;
  p.chunks = (int)((std::min(stride, out_stride) + kChunk - 1) / kChunk);
  const int64_t tasks = (int64_t)R * p.chunks;
  // a small table is renamed by the same cluster: a launch less
  if (tasks <= 2 * kCluster) mla_pages_compact_kernel<true><<<kCluster, kThreads, 0, st>>>(c, p);
  else mla_pages_compact_kernel<false><<<kCluster, kThreads, 0, st>>>(c, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_pages_compact_kernel");
  if (tasks <= 2 * kCluster) return MLA_OK;
  int dev = 0, sms = 0;
  const int rc = device_sms(&dev, &sms);
  if (rc != MLA_OK) return rc;
  e = launch_after(mla_pages_rename_kernel, (unsigned)std::min<int64_t>(tasks, 4 * sms), kThreads, st, p);
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_pages_rename_kernel");
  return MLA_OK;
}

extern "C" int mla_kv_copy(void* kv_pages, mla_kv_dtype kv_dtype, float* kv_scale, int64_t num_slots,
                           const int32_t* src, const int32_t* dst, const int32_t* tokens,
                           const int32_t* count, int64_t n, int* status, mla_stream_t stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "mla_kv_copy: n = %lld < 0", (long long)n);
  const int row_bytes = kv_dtype == MLA_KV_BF16 ? 2 * MLA_ROW_DIM
                        : kv_dtype == MLA_KV_FP8_E4M3 ? MLA_ROW_DIM
                        : kv_dtype == MLA_KV_FP4_E2M1 ? MLA_FP4_ROW_BYTES : 0;
  if (!row_bytes) return fail(MLA_ERR_INVALID_ARG, "mla_kv_copy: unknown kv_dtype %d", (int)kv_dtype);
  if (num_slots < kPage || num_slots >= (int64_t)1 << 31)
    return fail(MLA_ERR_INVALID_ARG, "mla_kv_copy: num_slots %lld outside [%d, 2^31)",
                (long long)num_slots, kPage);
  if (n == 0) return MLA_OK;
  if (!kv_pages || !src || !dst || (kv_dtype == MLA_KV_FP8_E4M3 && !kv_scale))
    return fail(MLA_ERR_INVALID_ARG, "mla_kv_copy: a required pointer is NULL");
  if (!aligned(kv_pages, 16)) return fail(MLA_ERR_MISALIGNED, "mla_kv_copy: the pool needs 16-B alignment");
  const void* all[] = {kv_scale, src, dst, tokens, count, status};
  for (const void* q : all)
    if (q && !aligned(q, 4)) return fail(MLA_ERR_MISALIGNED, "mla_kv_copy: arrays need 4-B alignment");
  int dev = 0, sms = 0;
  const int rc = device_sms(&dev, &sms);
  if (rc != MLA_OK) return rc;
  static_assert(kSlice <= kPage * MLA_FP4_ROW_BYTES / 16, "a turn touches two pages at most");
  const int row_vecs = row_bytes / 16;
  // a turn's blocks as many as n entries take, up to eight per SM
  const int64_t turns = n > (int64_t)1 << 24 ? (int64_t)1 << 24 : (n * kPage * row_vecs + kSlice - 1) / kSlice;
  const cudaError_t e = launch_after(
      mla_kv_copy_kernel, (unsigned)std::min<int64_t>(turns, 8 * sms), kCopyThreads, (cudaStream_t)stream,
      static_cast<uint8_t*>(kv_pages), kv_dtype == MLA_KV_FP8_E4M3 ? kv_scale : (float*)nullptr, row_vecs,
      num_slots / kPage, src, dst, tokens, count, n, status);
  if (e != cudaSuccess) return cuda_fail(e, "launch mla_kv_copy_kernel");
  return MLA_OK;
}
