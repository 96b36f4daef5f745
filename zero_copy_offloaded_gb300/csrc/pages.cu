// dkv_pages_fork, dkv_pages_compact, dkv_pages_copy: the life of a paged cache's pages on the GPU.
//
// No page carries a count of its holders: the page table says who holds what.  Old sequence s holds the
// ceil(len_s / P) first pages of its row.  A fork lets new sequence b be old sequence src_b: it is every old row's
// fate to go on (some b has src_b = s) or to vanish, and the pages that go back are those that a vanished
// row names and no row that goes on does.  A page that is some row's last, filled in part, is appended to, so one row alone may
// keep it, and none where a row that goes on has it as a full page (a sequence that was cut back shares such a page); the
// others take copies.  Whether a row has the page in full is a mark; who keeps it is found in a table of the
// at most 1024 such pages by page, in shared memory.  A compaction needs the pages that any row names; with L of them the
// i-th page named from L on moves to the i-th page not named below L.  Both are marks of the pool's pages (a byte
// each, plain stores: all writers write 1), a scan over the marks in page order, and a pass over the table.
//
// What bounds them: the table's entries, read once to mark (a scattered byte store each) and once to be
// rewritten, and latency: clearing the marks, marking, counting, what follows from the counts and the rewrite wait for one
// another.  Large tables and pools take a launch of the whole GPU for each, small ones one launch of a cluster with a
// barrier between them.  In a graph: a fork of 512 sequences of up to 32768 rows takes 21.4 us (with a scan by one cluster 46), a
// compaction of their 1 M pages 27 (110); of 64 sequences of up to 4096 rows in a cluster, whose shared memory holds the marks, 10.5
// and 14.9 (with marks in memory 14 and 17).  A copy of 8192 pages of
// 2 x 32 KB and their scales runs at 6.6 TB/s, as fast as a plain copy.
#include <stdio.h>

#include <algorithm>

#include "dkv_internal.cuh"
#include "per_device.h"

namespace dkv {
void set_last_error(dkv_status s, const char* msg);
}

namespace {

using namespace dkv;

constexpr int kThreads = 1024, kWarps = kThreads / 32, kCluster = 8, kSms = 152;
constexpr int kSegment = 256;  // table entries of a warp at a time, eight to a lane
// Table entries plus pages up to which one cluster does everything in one launch.  64 sequences of up to 16384 rows,
// 131000 in all, take 14.3 us to fork and 34 to compact so, 18 and 21.4 in five launches, whose calls take 9 us longer; with half
// of that compactions too are faster in one.
constexpr long long kForkInOne = 1 << 18, kCompactInOne = 1 << 17;

// Each is a launch of its own, or one launch of a cluster runs them all.
enum Phase : int { kAll = -1, kClear = 0, kMark = 1, kCount = 2, kEmit = 3, kWrite = 4 };

struct Row {
  int source;  // old row that this one becomes a copy of; -1: none
  int shared;  // its entries that go on
  int take;    // where the entry behind them, a copy of the source's, comes from, on the stack; -1: there is none
  int pad;
};

struct PageParams {
  const int* table;
  const int* len;
  const int* sources;    // fork
  int* free_pages;
  const int* free_count; // fork
  int* table_out;
  int* len_out;          // fork
  int* free_left;
  int* pairs;            // copies [B][2] or moves [max_moves][2]
  int* report;
  uint8_t* live;         // [num_pages, rounded up to 16]
  uint8_t* tails;        // fork: the same
  uint8_t* dead;         // fork: the same
  Row* rows;             // fork: [B]
  int* old;              // fork in place: [B][max_pages]
  int* rank;             // compact: [num_pages], of pages that move
  int* counts;           // marks that each CTA of the scan has counted [kSms], then pages from which entries move
  int B, max_pages, shift, num_pages, max_moves;
  int mark_shift;        // one launch: log2 of the marks' words of a CTA
};

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ long long pages_of(long long len, int shift) { return (len + (1 << shift) - 1) >> shift; }

// Sum of v over the CTA's threads before this one; `total`: over all.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += o;
  }
  __syncthreads();  // s_warp is free
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  // every warp adds up the warps' sums for itself
  const int w = s_warp[lane];
  total = __reduce_add_sync(~0u, w);
  return x - v + __reduce_add_sync(~0u, lane < warp ? w : 0);
}

// Marks of the pool's pages, bytes of 0 or 1 in words of four: in the workspace, or (one launch) in the cluster's shared
// memory, CTA c the words [c << shift, (c + 1) << shift), where clearing, marking and scanning wait for no memory.
template <bool ONE>
struct Marks {
  uint8_t* global;
  uint32_t shared;  // its address there, the same in every CTA
  int shift;
  __device__ __forceinline__ uint32_t at(int word) const {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(shared + (word & ((1 << shift) - 1)) * 4), "r"(word >> shift));
    return a;
  }
  __device__ __forceinline__ void set(int page) const {
    if constexpr (!ONE) global[page] = 1;
    else asm volatile("st.shared::cluster.u8 [%0], %1;" ::"r"(at(page >> 2) + (page & 3)), "r"(1) : "memory");
  }
  __device__ __forceinline__ bool get(int page) const {
    if constexpr (!ONE) return __ldcg(global + page);
    uint32_t v;
    asm volatile("ld.shared::cluster.u8 %0, [%1];" : "=r"(v) : "r"(at(page >> 2) + (page & 3)) : "memory");
    return v;
  }
  __device__ __forceinline__ uint32_t load(int word) const {
    if constexpr (!ONE) return __ldcg(reinterpret_cast<const uint32_t*>(global) + word);
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at(word)) : "memory");
    return v;
  }
  __device__ __forceinline__ void clear(int num_pages) const {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if constexpr (!ONE) {
      for (int i = blockIdx.x * kThreads + threadIdx.x; i < (num_pages + 15) / 16; i += gridDim.x * kThreads)
        reinterpret_cast<uint4*>(global)[i] = zero;
    } else {
      for (int i = threadIdx.x; i < 1 << shift; i += kThreads)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(shared + i * 4), "r"(0) : "memory");
    }
  }
};

// The marks that each CTA has counted: in the workspace, or in every CTA's shared memory.
template <bool ONE>
struct Counts {
  int* global;
  int* shared;
  __device__ __forceinline__ void put(int own) const {  // the threads together
    if constexpr (!ONE) {
      if (threadIdx.x == 0) global[blockIdx.x] = own;
    } else if (threadIdx.x < kCluster) {
      uint32_t a;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(shared + blockIdx.x)), "r"(threadIdx.x));
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(own) : "memory");
    }
  }
  __device__ __forceinline__ int get(int cta) const { return ONE ? *(volatile int*)(shared + cta) : __ldcg(global + cta); }
};

// The marks that CTAs before `upto` have counted, and those of all; the threads together.
template <bool ONE>
__device__ __forceinline__ int counted(const Counts<ONE>& counts, int upto, int* s_warp, int& total) {
  const int t = threadIdx.x;
  const int v = t < (int)gridDim.x ? counts.get(t) : 0;
  int before;
  block_scan(t < upto ? v : 0, s_warp, before);
  block_scan(v, s_warp, total);
  return before;
}

// f(row, first entry) for each segment of the rows, a warp at a time.
template <typename F>
__device__ __forceinline__ void segments(const PageParams& p, F&& f) {
  const int parts = (p.max_pages + kSegment - 1) / kSegment;
  for (long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); w < (long long)p.B * parts;
       w += (long long)gridDim.x * kWarps) {
    const int b = (int)(w / parts);
    f(b, (int)(w - (long long)b * parts) * kSegment);
  }
}

// Eight entries of a lane, from `first` on, below `end`.
__device__ __forceinline__ void load_segment(const int* row, int first, int end, int (&page)[8]) {
  const int at = first + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < 8; ++i) page[i] = at + 32 * i < end ? __ldcg(row + at + 32 * i) : -1;
}

template <bool ONE>
__device__ __forceinline__ void mark(const PageParams& p, const Marks<ONE>& at, const int (&page)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if ((uint32_t)page[i] < (uint32_t)p.num_pages) at.set(page[i]);
}

// The scan's words of four pages: a CTA has words [cta * per, (cta + 1) * per), a thread n of them from `first` on.
struct Range {
  int per, first, n;
};
__device__ __forceinline__ Range scan_range(const PageParams& p, int cta, bool all) {
  const int words = (p.num_pages + 3) / 4, per = all ? 1 << p.mark_shift : (words + gridDim.x - 1) / gridDim.x;
  const int each = (per + kThreads - 1) / kThreads, at = min((int)threadIdx.x * each, per);
  const int first = (int)min((long long)cta * per + at, (long long)words);
  return {per, first, max(0, min(min(each, per - at), words - first))};
}

// ---- fork -----------------------------------------------------------------------------------

// What every CTA finds out about the batch for itself.
constexpr int kPlaces = 2 * kThreads;
struct Batch {
  int len[kThreads];   // of the old rows, from 0 to what the table holds
  Row rows[kThreads];  // of the new ones
  int goes[kThreads];  // old row s goes on
  // The pages filled in part of rows that go on (outside the pool: num_pages + the row), at the place that their hash gives or the
  // next one free, -1: free; and who keeps each: the lowest new row that is its old self, else 1024 + the lowest.
  int page[kPlaces], keeper[kPlaces];
  int warp[kWarps], counts[kCluster];
  int longest;
  // a source is not there; a length is beyond the table; a row vanishes; one that goes on fills a page in part
  int wrong, far, any, some;

  __device__ __forceinline__ int place_of(int key) {
    int at = (uint32_t)key * 2654435761u >> 21;  // (Knuth, The Art of Computer Programming, volume 3, section 6.4)
    static_assert(kPlaces == 1 << 11, "21 bits of the hash are left out");
    for (;; at = (at + 1) & (kPlaces - 1)) {  // at most 1024 of 2048 places are taken
      const int was = atomicCAS(page + at, -1, key);
      if (was == -1 || was == key) return at;
    }
  }
};

template <bool ALL>
__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const PageParams p, int phase) {
  __shared__ Batch s;
  extern __shared__ uint4 s_marks[];
  // full pages of rows that go on, pages that these fill in part, pages of the others
  const Marks<ALL> live = {p.live, smem_u32(s_marks), p.mark_shift};
  const Marks<ALL> tails = {p.tails, smem_u32(s_marks) + (4 << p.mark_shift), p.mark_shift};
  const Marks<ALL> dead = {p.dead, smem_u32(s_marks) + (8 << p.mark_shift), p.mark_shift};
  const Counts<ALL> counts = {p.counts, s.counts};
  auto load_freed = [&](int word) { return dead.load(word) & ~(live.load(word) | tails.load(word)); };  // held, and not any more
  griddep_wait();
  griddep_launch_dependents();
  const int b = threadIdx.x, lane = b & 31;
  constexpr bool all = ALL;  // phases
  const long long cap = (long long)p.max_pages << p.shift;
  int src = -1, free_count = 0;
  long long len = 0;
  if (phase != kClear && phase != kWrite) {
    src = b < p.B ? p.sources[b] : -1;
    len = b < p.B ? max(p.len[b], 0) : 0;
    free_count = min(max(*p.free_count, 0), p.num_pages);
  }
  if (phase == kClear || all) {
    live.clear(p.num_pages);
    tails.clear(p.num_pages);
    dead.clear(p.num_pages);
    if (!all) return;
  }
  if (phase != kWrite) {
    const int part = (1 << p.shift) - 1;
    s.goes[b] = 0;
    s.len[b] = (int)min(len, cap);
    if (phase == kEmit || all) {
      s.page[b] = s.page[b + kThreads] = -1;
      s.keeper[b] = s.keeper[b + kThreads] = 0x7fffffff;
    }
    if (b == 0) s.longest = s.wrong = s.far = s.any = s.some = 0;
    __syncthreads();
    const bool on = src >= 0 && src < p.B;
    if (on) s.goes[src] = 1;
    if (src >= p.B) s.wrong = 1;
    if (len > cap) s.far = 1;
    const int new_len = on ? s.len[src] : 0, held = (int)pages_of(new_len, p.shift);
    const bool fills = new_len & part;
    if (fills) s.some = 1;
    __syncthreads();
    if (len > 0 && !s.goes[b]) s.any = 1;
    __syncthreads();
    const bool any = s.any, some = s.some;
    int tail = -1;
    if (fills && (phase == kEmit || all)) tail = __ldcg(p.table + (size_t)src * p.max_pages + held - 1);
    if (phase == kMark || all) {
      if (all) cluster_sync();
      segments(p, [&](int r, int first) {
        const int end = (int)pages_of(s.len[r], p.shift), full = s.len[r] >> p.shift;
        if (first >= end) return;
        const bool goes = s.goes[r];
        // in place, a row that another one becomes is read again after it may have been written
        const bool keep = p.old && goes;
        if (!any && !some && !keep) return;
        int page[8];
        load_segment(p.table + (size_t)r * p.max_pages, first, end, page);
        if (any || some) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((uint32_t)page[i] < (uint32_t)p.num_pages)
              (!goes ? dead : first + lane + 32 * i < full ? live : tails).set(page[i]);
        }
        if (keep) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (first + lane + 32 * i < end) p.old[(size_t)r * p.max_pages + first + lane + 32 * i] = page[i];
        }
      });
      if (!all) return;
    }
    // who keeps a page that is filled in part
    const bool in_pool = (uint32_t)tail < (uint32_t)p.num_pages;
    const int rank = src == b ? b : kThreads + b;
    int place = 0;
    if (fills && (phase == kEmit || all)) {
      place = s.place_of(in_pool ? tail : p.num_pages + src);
      atomicMin(&s.keeper[place], rank);
    }
    if (all) cluster_sync();
    const bool whole = in_pool && live.get(tail);  // some row that goes on has it as a full page
    // ---- pages that go back, in page order
    const Range range = scan_range(p, blockIdx.x, all);
    int mine = 0;
    if (any)
      for (int i = 0; i < range.n; ++i) mine += __popc(load_freed(range.first + i));
    int own, freed = 0, at = 0;
    if (any) at = block_scan(mine, s.warp, own);
    if (phase == kCount || all) {
      if (any) counts.put(own);
      if (!all) return;
      cluster_sync();
    }
    if (any) at += counted(counts, blockIdx.x, s.warp, freed);
    if (!all) __syncthreads();
    const bool need = fills && (s.keeper[place] != rank || whole);
    int needed;
    const int k = block_scan(need, s.warp, needed);
    const long long stack = (long long)free_count + freed;
    const bool ok = !s.wrong && !s.far && needed <= stack && stack <= p.num_pages;
    if (ok && mine) {
      int* to = p.free_pages + free_count + at;
      for (int i = 0; i < range.n; ++i) {
        for (uint32_t m = load_freed(range.first + i); m; m &= m - 1)
          *to++ = (range.first + i) * 4 + (__ffs(m) - 1) / 8;
      }
    }
    Row row = {ok ? (on ? src : -1) : b, ok ? held - need : (int)pages_of(s.len[b], p.shift), -1, 0};
    if (ok && need) row.take = (int)(stack - 1 - k);
    s.rows[b] = row;
    // one CTA, where it cannot be the only one to read the inputs, leaves what it writes over them to the next phase
    if (blockIdx.x == gridDim.x - 1) {
      const int length = ok ? new_len : (int)len;
      atomicMax(&s.longest, length);
      if (b < p.B) {
        if (row.take < 0) reinterpret_cast<int2*>(p.pairs)[b] = make_int2(-1, -1);
        p.rows[b] = row;
        p.counts[kSms + 1 + b] = length;
      }
      __syncthreads();
      if (b == 0) {
        p.report[0] = ok ? DKV_OK : s.wrong ? DKV_ERR_INVALID_ARG : DKV_ERR_CAPACITY;
        p.report[1] = ok ? freed : 0;
        p.report[2] = ok ? needed : 0;
        p.report[3] = s.longest;
        p.counts[kSms] = ok ? (int)(stack - needed) : free_count;
      }
    }
    if (!all) return;
    cluster_sync();
  }
  // ---- write the rows
  if (blockIdx.x == 0) {
    if (b < p.B) p.len_out[b] = __ldcg(p.counts + kSms + 1 + b);
    if (b == 0) *p.free_left = __ldcg(p.counts + kSms);
  }
  segments(p, [&](int r, int first) {
    Row row = s.rows[r];
    if (!all) {
      const int4 w = __ldcg(reinterpret_cast<const int4*>(p.rows + r));
      row = {w.x, w.y, w.z, w.w};
    }
    if (row.source < 0 || first >= row.shared + 1 || (p.old && row.source == r && row.take < 0)) return;
    int page[8];
    load_segment((p.old ? p.old : p.table) + (size_t)row.source * p.max_pages, first, row.shared, page);
    int* to = p.table_out + (size_t)r * p.max_pages;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = first + lane + 32 * i;
      if (c < row.shared) {
        to[c] = page[i];
      } else if (c == row.shared && row.take >= 0) {
        const int taken = __ldcg(p.free_pages + row.take);
        const int from = __ldcg((p.old ? p.old : p.table) + (size_t)row.source * p.max_pages + c);
        to[c] = taken;
        reinterpret_cast<int2*>(p.pairs)[r] = make_int2(from, taken);
      }
    }
  });
}

// ---- compaction -----------------------------------------------------------------------------

template <bool ALL>
__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const PageParams p, int phase) {
  __shared__ int s_warp[kWarps], s_longest, s_len[kThreads], s_counts[kCluster];
  extern __shared__ uint4 s_marks[];
  const Marks<ALL> marks = {p.live, smem_u32(s_marks), p.mark_shift};
  const Counts<ALL> counts = {p.counts, s_counts};
  griddep_wait();
  griddep_launch_dependents();
  constexpr bool all = ALL;  // phases
  const int lane = threadIdx.x & 31, t = threadIdx.x;
  const long long cap = (long long)p.max_pages << p.shift;
  const int len = phase != kClear && t < p.B ? max(p.len[t], 0) : 0;
  s_len[t] = (int)min((long long)len, cap);
  __syncthreads();
  auto end_of = [&](int r) { return (int)pages_of(s_len[r], p.shift); };
  if (phase == kClear || all) {
    marks.clear(p.num_pages);
    if (!all) return;
    cluster_sync();
  }
  if (phase == kMark || all) {
    segments(p, [&](int r, int first) {
      const int end = end_of(r);
      if (first >= end) return;
      int page[8];
      load_segment(p.table + (size_t)r * p.max_pages, first, end, page);
      mark(p, marks, page);
    });
    if (!all) return;
    cluster_sync();
  }
  int from = 0;
  if (phase != kWrite) {
    const Range range = scan_range(p, blockIdx.x, all);
    int mine = 0, own;
    for (int i = 0; i < range.n; ++i) mine += __popc(marks.load(range.first + i));
    int before = block_scan(mine, s_warp, own);  // pages named before this thread's
    if (phase == kCount || all) {
      counts.put(own);
      if (!all) return;
      cluster_sync();
    }
    int live;
    before += counted(counts, blockIdx.x, s_warp, live);
    // named pages below `live`, which stay: those of the CTAs before the one that has page `live`, and a part of its own
    const int edge = live / 4 / range.per;
    int ignore, part = 0, low;
    low = counted(counts, edge, s_warp, ignore);
    const Range other = scan_range(p, edge, all);
    for (int i = 0; i < other.n; ++i) {
      const int word = other.first + i, keep = live - word * 4;  // bytes of it below `live`
      part += __popc(marks.load(word) & (keep >= 4 ? ~0u : keep <= 0 ? 0u : (1u << (8 * keep)) - 1));
    }
    block_scan(part, s_warp, part);
    low += part;
    const int moves = live - low;
    if (t == 0) s_longest = 0;
    const bool ok = !__syncthreads_or(len > cap);
    if (ok) {
      for (int i = 0; i < range.n; ++i) {
        const uint32_t word = marks.load(range.first + i);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int named = (word >> (8 * q)) & 1, page = (range.first + i) * 4 + q;
          if (page < live) {
            if (!named) p.pairs[2 * (page - before) + 1] = page;
          } else if (named) {
            p.pairs[2 * (before - low)] = page;
            p.rank[page] = before - low;
          }
          before += named;
        }
      }
    }
    const int rest = ok ? moves : 0, stride = gridDim.x * kThreads;
    for (int i = rest + blockIdx.x * kThreads + t; i < p.max_moves; i += stride)
      reinterpret_cast<int2*>(p.pairs)[i] = make_int2(-1, -1);
    if (ok)
      for (int i = blockIdx.x * kThreads + t; i < p.num_pages - live; i += stride) p.free_pages[i] = p.num_pages - 1 - i;
    if (blockIdx.x == 0) {
      atomicMax(&s_longest, len);
      __syncthreads();
      if (t == 0) {
        if (ok) *p.free_left = p.num_pages - live;
        p.report[0] = ok ? DKV_OK : DKV_ERR_CAPACITY;
        p.report[1] = rest;
        p.report[2] = ok ? live : 0;
        p.report[3] = s_longest;
        p.counts[kSms] = ok ? live : 0x7fffffff;
      }
    }
    from = ok ? live : 0x7fffffff;
    if (!all) return;
    cluster_sync();
  }
  // ---- the tables follow
  // entries from it on have moved
  const int live = phase == kWrite ? __ldcg(p.counts + kSms) : from;
  segments(p, [&](int r, int first) {
    const int end = end_of(r);
    if (first >= end) return;
    int page[8], to[8];
    load_segment(p.table + (size_t)r * p.max_pages, first, end, page);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool moved = page[i] >= live && page[i] < p.num_pages;
      to[i] = moved ? __ldcg(p.rank + page[i]) : -1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (to[i] >= 0) page[i] = __ldcg(p.pairs + 2 * to[i] + 1);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (first + lane + 32 * i < end) p.table_out[(size_t)r * p.max_pages + first + lane + 32 * i] = page[i];
  });
}

// ---- copy -----------------------------------------------------------------------------------

constexpr int kPools = 64;       // of one launch
constexpr int kCopyThreads = 256;
constexpr int kInFlight = 8;     // loads of a lane

struct CopyParams {
  const int2* pairs;
  const uint8_t* src[kPools];
  uint8_t* dst[kPools];
  unsigned long long bytes[kPools];
  int src_pages[kPools], dst_pages[kPools];
  int first[kPools + 1];  // segments before the pool's, of one pair
  int n_pairs, n_pools;
};

// A warp takes a segment of 32 lanes x 8 loads of one page.
template <typename W>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  constexpr int kBytes = 32 * kInFlight * sizeof(W);
  const int lane = threadIdx.x & 31, segs = p.first[p.n_pools];
  for (long long w = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
       w < (long long)p.n_pairs * segs; w += (long long)gridDim.x * (kCopyThreads / 32)) {
    const int i = (int)(w / segs), seg = (int)(w - (long long)i * segs);
    int pool = 0;
    while (seg >= p.first[pool + 1]) ++pool;
    const int2 pair = __ldg(p.pairs + i);
    if ((uint32_t)pair.x >= (uint32_t)p.src_pages[pool] || (uint32_t)pair.y >= (uint32_t)p.dst_pages[pool]) continue;
    const unsigned long long bytes = p.bytes[pool];
    const unsigned long long at = (unsigned long long)(seg - p.first[pool]) * kBytes + lane * sizeof(W);
    const uint8_t* from = p.src[pool] + pair.x * bytes + at;
    uint8_t* to = p.dst[pool] + pair.y * bytes + at;
    const long long room = (long long)(bytes - at);  // may be negative: behind the page
    W x[kInFlight];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k)
      if (k * 32LL * (int)sizeof(W) < room) x[k] = __ldcs(reinterpret_cast<const W*>(from) + k * 32);
#pragma unroll
    for (int k = 0; k < kInFlight; ++k)
      if (k * 32LL * (int)sizeof(W) < room) __stcs(reinterpret_cast<W*>(to) + k * 32, x[k]);
  }
}

// ---- entry points ---------------------------------------------------------------------------

dkv_status refuse(dkv_status s, const char* msg) {
  set_last_error(s, msg);
  return s;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

const char* bad_sizes(int batch, int max_pages, int page_tokens, int num_pages) {
  if (batch <= 0 || batch > DKV_MAX_STEP_BATCH) return "batch outside [1, DKV_MAX_STEP_BATCH]";
  if (page_tokens < 1 || page_tokens > 4096 || (page_tokens & (page_tokens - 1)))
    return "page_tokens must be a power of two in [1, 4096]";
  if (max_pages <= 0 || (long long)max_pages * page_tokens > (1LL << 30))
    return "max_pages must be positive, max_pages * page_tokens at most 2^30";
  if (num_pages <= 0 || (long long)num_pages * page_tokens > (1LL << 30))
    return "num_pages must be positive, num_pages * page_tokens at most 2^30";
  return nullptr;
}

// Workspace: counts, the end of the stack, new lengths | rows | marks | two more, or ranks | the old table.
size_t ws_rows() { return align256((kSms + 1 + DKV_MAX_STEP_BATCH) * sizeof(int)); }
size_t ws_live() { return ws_rows() + align256(DKV_MAX_STEP_BATCH * sizeof(Row)); }
size_t ws_more(int num_pages) { return ws_live() + align256(num_pages); }
size_t ws_old(int num_pages) { return ws_more(num_pages) + align256((size_t)num_pages * 4); }

template <typename K>
cudaError_t launch_one(K* kernel, const PageParams& p, int phase, int grid, cudaStream_t s, int smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  if (phase == kAll) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  } else {  // a phase's CTAs may come to an SM while the last ones of the phase before finish
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = phase == kClear ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, phase);
}

// `one` for up to `most` entries and pages, with so many maps of marks.
template <typename K>
dkv_status launch(K* one, long long most, int maps, K* kernel, PageParams& p, PerDevice& room, cudaStream_t s) {
  cudaError_t e;
  if ((long long)p.B * p.max_pages + p.num_pages <= most) {
    const int words = ((p.num_pages + 3) / 4 + kCluster - 1) / kCluster;
    p.mark_shift = 2;
    while ((1 << p.mark_shift) < words) ++p.mark_shift;
    int device = 0;
    e = cudaGetDevice(&device);
    if (e == cudaSuccess)
      e = room(device, [&] { return cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(maps * most / kCluster)); });
    if (e == cudaSuccess) e = launch_one(one, p, kAll, kCluster, s, maps * (4 << p.mark_shift));
  } else {
    const long long parts = (long long)p.B * ((p.max_pages + kSegment - 1) / kSegment);
    const int grid = (int)std::min<long long>((parts + kWarps - 1) / kWarps, kSms);
    const int scan = std::min((p.num_pages + 4 * kThreads - 1) / (4 * kThreads), kSms);
    e = launch_one(kernel, p, kClear, scan, s);
    if (e == cudaSuccess) e = launch_one(kernel, p, kMark, grid, s);
    if (e == cudaSuccess) e = launch_one(kernel, p, kCount, scan, s);
    if (e == cudaSuccess) e = launch_one(kernel, p, kEmit, scan, s);
    if (e == cudaSuccess) e = launch_one(kernel, p, kWrite, grid, s);
  }
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? DKV_OK : refuse(DKV_ERR_CUDA, cudaGetErrorString(e));
}

void set_workspace(PageParams& p, void* workspace) {
  char* w = static_cast<char*>(workspace);
  p.counts = reinterpret_cast<int*>(w);
  p.rows = reinterpret_cast<Row*>(w + ws_rows());
  p.live = reinterpret_cast<uint8_t*>(w + ws_live());
  p.tails = reinterpret_cast<uint8_t*>(w + ws_more(p.num_pages));  // (the ranks' room holds both: twice num_pages + 15 bytes)
  p.dead = p.tails + ((size_t)p.num_pages + 15) / 16 * 16;
  p.rank = reinterpret_cast<int*>(w + ws_more(p.num_pages));
  p.old = reinterpret_cast<int*>(w + ws_old(p.num_pages));
}

int shift_of(int page_tokens) {
  int s = 0;
  while ((1 << s) < page_tokens) ++s;
  return s;
}

}  // namespace

extern "C" size_t dkv_pages_workspace(int batch, int max_pages, int num_pages) {
  if (bad_sizes(batch, max_pages, 1, num_pages)) return 0;
  return ws_old(num_pages) + align256((size_t)batch * max_pages * 4);
}

extern "C" dkv_status dkv_pages_fork(const int32_t* page_table, const int32_t* kv_len, const int32_t* sources,
                                     int32_t* free_pages, const int32_t* free_count, int batch, int max_pages,
                                     int page_tokens, int num_pages, int32_t* table_out, int32_t* len_out,
                                     int32_t* free_left, int32_t* copies, int32_t* report, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (!page_table || !kv_len || !sources || !free_pages || !free_count || !table_out || !len_out || !free_left ||
      !copies || !report || !workspace)
    return refuse(DKV_ERR_INVALID_ARG, "null pointer argument");
  if (const char* why = bad_sizes(batch, max_pages, page_tokens, num_pages)) return refuse(DKV_ERR_INVALID_ARG, why);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) || (reinterpret_cast<uintptr_t>(copies) & 7))
    return refuse(DKV_ERR_INVALID_ARG, "the workspace must start on a 256-byte boundary, the pairs on 8");
  if (workspace_bytes < dkv_pages_workspace(batch, max_pages, num_pages))
    return refuse(DKV_ERR_INVALID_ARG, "workspace smaller than dkv_pages_workspace says");
  PageParams p = {};
  p.table = page_table; p.len = kv_len; p.sources = sources; p.free_pages = free_pages; p.free_count = free_count;
  p.table_out = table_out; p.len_out = len_out; p.free_left = free_left; p.pairs = copies; p.report = report;
  p.B = batch; p.max_pages = max_pages; p.num_pages = num_pages; p.shift = shift_of(page_tokens);
  set_workspace(p, workspace);
  if (table_out != page_table) p.old = nullptr;
  static PerDevice room;
  return launch(fork_kernel<true>, kForkInOne, 3, fork_kernel<false>, p, room, static_cast<cudaStream_t>(stream));
}

extern "C" dkv_status dkv_pages_compact(const int32_t* page_table, const int32_t* kv_len, int batch, int max_pages,
                                        int page_tokens, int num_pages, int32_t* table_out, int32_t* free_pages,
                                        int32_t* free_left, int32_t* moves, int max_moves, int32_t* report,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  if (!page_table || !kv_len || !table_out || !free_pages || !free_left || !report || !workspace ||
      (!moves && num_pages > 1))
    return refuse(DKV_ERR_INVALID_ARG, "null pointer argument");
  if (const char* why = bad_sizes(batch, max_pages, page_tokens, num_pages)) return refuse(DKV_ERR_INVALID_ARG, why);
  if (max_moves < num_pages / 2) return refuse(DKV_ERR_INVALID_ARG, "max_moves below num_pages / 2");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) || (reinterpret_cast<uintptr_t>(moves) & 7))
    return refuse(DKV_ERR_INVALID_ARG, "the workspace must start on a 256-byte boundary, the pairs on 8");
  if (workspace_bytes < dkv_pages_workspace(batch, max_pages, num_pages))
    return refuse(DKV_ERR_INVALID_ARG, "workspace smaller than dkv_pages_workspace says");
  PageParams p = {};
  p.table = page_table; p.len = kv_len; p.free_pages = free_pages; p.table_out = table_out; p.free_left = free_left;
  p.pairs = moves; p.report = report;
  p.B = batch; p.max_pages = max_pages; p.num_pages = num_pages; p.shift = shift_of(page_tokens);
  p.max_moves = moves ? max_moves : 0;
  set_workspace(p, workspace);
  static PerDevice room;
  return launch(compact_kernel<true>, kCompactInOne, 1, compact_kernel<false>, p, room, static_cast<cudaStream_t>(stream));
}

extern "C" dkv_status dkv_pages_copy(const int32_t* pairs, int n_pairs, const dkv_page_pool_t* pools, int n_pools,
                                     void* stream) {
  if ((!pairs && n_pairs) || !pools) return refuse(DKV_ERR_INVALID_ARG, "null pointer argument");
  if (n_pairs < 0 || n_pairs > (1 << 30)) return refuse(DKV_ERR_INVALID_ARG, "pairs outside [0, 2^30]");
  if (n_pools <= 0 || n_pools > 65536) return refuse(DKV_ERR_INVALID_ARG, "pools outside [1, 65536]");
  if (reinterpret_cast<uintptr_t>(pairs) & 7) return refuse(DKV_ERR_INVALID_ARG, "the pairs must start on an 8-byte boundary");
  for (int i = 0; i < n_pools; ++i) {
    const dkv_page_pool_t& a = pools[i];
    if (!a.src || !a.dst) return refuse(DKV_ERR_INVALID_ARG, "null pool");
    if (a.src_pages <= 0 || a.dst_pages <= 0) return refuse(DKV_ERR_INVALID_ARG, "a pool without pages");
    if (!a.page_bytes || a.page_bytes % 4 || a.page_bytes > (1ull << 30))
      return refuse(DKV_ERR_INVALID_ARG, "page_bytes must be a multiple of 4, at most 2^30");
    if ((reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst)) & 3)
      return refuse(DKV_ERR_INVALID_ARG, "pools must start on 4-byte boundaries");
  }
  if (!n_pairs) return DKV_OK;
  // Pages in words of 16 bytes first, then those that only have words of 4.
  for (int wide = 1; wide >= 0; --wide) {
    CopyParams p;
    p.pairs = reinterpret_cast<const int2*>(pairs);
    p.n_pairs = n_pairs;
    p.n_pools = 0;
    p.first[0] = 0;
    for (int i = 0; i < n_pools; ++i) {
      const dkv_page_pool_t& a = pools[i];
      const bool w16 = !((reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst) | a.page_bytes) & 15);
      if (w16 == (wide == 1)) {
        const int k = p.n_pools++;
        const size_t seg = 32 * kInFlight * (wide ? 16 : 4);
        p.src[k] = static_cast<const uint8_t*>(a.src);
        p.dst[k] = static_cast<uint8_t*>(a.dst);
        p.bytes[k] = a.page_bytes;
        p.src_pages[k] = a.src_pages;
        p.dst_pages[k] = a.dst_pages;
        p.first[k + 1] = p.first[k] + (int)((a.page_bytes + seg - 1) / seg);
      }
      if (p.n_pools == kPools || (i == n_pools - 1 && p.n_pools)) {
        const long long warps = (long long)n_pairs * p.first[p.n_pools];
        const int grid = (int)std::min<long long>((warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32), 8LL * 8 * kSms);
        if (wide) copy_kernel<uint4><<<grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
        else copy_kernel<uint32_t><<<grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return refuse(DKV_ERR_CUDA, cudaGetErrorString(e));
        p.n_pools = 0;
      }
    }
  }
  return DKV_OK;
}
