// dkv_step_plan: lengths and new-token counts of a batch become pages, row
// starts, positions and slots, on the GPU.
//
// For sequence b with len_b cached rows and new_b >= 0 new ones, pages of P rows:
//   held_b = ceil(len_b / P),  need_b = ceil((len_b + new_b) / P) - held_b,
// new_b < 0 releases the sequence (its held_b pages go back, its length is 0).
// Released pages are pushed on the free stack in order of (sequence, page);
// then the k-th page taken, in the same order, is the k-th from the top.  The
// three exclusive scans (need, released, rows) give every sequence its place.
// The new token t of sequence b has position len_b + t and slot
// table[b][pos / P] * P + pos % P.
//
// It moves a few KB to a few hundred KB, so what bounds it is latency, and with many rows their filling
// by eight of the SMs (65536 rows: 11.2 us in a graph, 1024 of as long a batch 5.7).  One launch of one
// cluster of eight CTAs (the largest portable one).  Every CTA scans all sequences, one per thread; a
// cluster barrier then stands between the last read of the inputs and the first write (so
// that lengths and the free count may be updated in place); pages are moved by
// the warps of all CTAs, and behind a second barrier all threads fill the rows.
// In a graph of such launches, a step with one token for each of 64 sequences takes 4.7 us (one
// CTA: 4.9), of 1024 sequences 6.4 us (8.7), with 64 each for 64 sequences 5.9 us (9.7).
#include <stdio.h>

#include "dkv_internal.cuh"

namespace dkv {
void set_last_error(dkv_status s, const char* msg);
}

namespace {

using namespace dkv;

constexpr int kPlanThreads = 1024;

struct PlanParams {
  const int* lengths;
  const int* new_tokens;
  int* table;
  int* free_pages;
  const int* free_count;
  int* row_start;
  int* row_pos;
  int* row_slot;
  int* kv_len;
  int* free_left;
  int* report;
  int B, max_pages, shift, num_pages, max_rows;
};

struct Sums {
  long long need, back, rows;
};

__device__ __forceinline__ Sums add(const Sums& a, const Sums& b) {
  return {a.need + b.need, a.back + b.back, a.rows + b.rows};
}

__device__ __forceinline__ Sums shfl_up(const Sums& v, int d) {
  return {__shfl_up_sync(~0u, v.need, d), __shfl_up_sync(~0u, v.back, d),
          __shfl_up_sync(~0u, v.rows, d)};
}

// Positions and slots of the rows first, first + stride, ...: the sequence of a row is found by
// bisection of the row starts, U rows of a thread at once.
template <int U>
__device__ __forceinline__ void fill_rows(const PlanParams& p, const int* start, const int* kv,
                                          int first, int stride) {
  const int total = start[p.B];
  for (long long r0 = first; r0 < p.max_rows; r0 += (long long)U * stride) {
    int r[U], seq[U] = {}, pos[U], page[U];
#pragma unroll
    for (int i = 0; i < U; ++i) r[i] = (int)min(r0 + (long long)i * stride, (long long)p.max_rows);
    for (int step = 1 << (31 - __clz(p.B)); step; step >>= 1) {  // the last whose start is at most r
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (seq[i] + step < p.B && start[seq[i] + step] <= r[i]) seq[i] += step;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool on = r[i] < total;
      pos[i] = on ? kv[seq[i]] - (start[seq[i] + 1] - r[i]) : 0;
      page[i] = on ? __ldcg(p.table + (size_t)seq[i] * p.max_pages + (pos[i] >> p.shift)) : -1;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (r[i] >= p.max_rows) break;
      p.row_pos[r[i]] = pos[i];
      // no page of the pool (whose slots fit 30 bits; beyond that they would wrap into another page's): padding
      p.row_slot[r[i]] =
          (uint32_t)page[i] < (uint32_t)p.num_pages ? (page[i] << p.shift) + (pos[i] & ((1 << p.shift) - 1)) : -1;
    }
  }
}

// All CTAs of the cluster have come here, and see what the others wrote before.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const PlanParams p) {
  __shared__ int s_start[kPlanThreads + 1], s_kv[kPlanThreads], s_held[kPlanThreads];
  __shared__ int s_need[kPlanThreads + 1], s_back[kPlanThreads + 1];
  __shared__ Sums s_warp[32];
  __shared__ int s_max;
  const int b = threadIdx.x, lane = b & 31, warp = b >> 5, warps = kPlanThreads / 32;
  const int cta = blockIdx.x, ctas = gridDim.x;  // the grid is one cluster
  const long long cap = (long long)p.max_pages << p.shift;
  const int free_count = min(max(*p.free_count, 0), p.num_pages);
  if (b == 0) s_max = 0;
  int len = 0, kv = 0, held = 0;
  Sums own = {0, 0, 0};
  bool bad = false;
  if (b < p.B) {
    len = max(p.lengths[b], 0);
    const int nw = p.new_tokens[b];
    bad = len > cap || (nw > 0 && (long long)len + nw > cap);
    if (!bad) {
      held = (int)(((long long)len + (1 << p.shift) - 1) >> p.shift);
      if (nw < 0) {
        own.back = held;
      } else {
        kv = len + nw;
        own.need = (((long long)kv + (1 << p.shift) - 1) >> p.shift) - held;
        own.rows = nw;
      }
    }
  }
  Sums inc = own;
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shfl_up(inc, d);
    if (lane >= d) inc = add(inc, o);
  }
  if (lane == 31) s_warp[warp] = inc;
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    Sums w = lane < warps ? s_warp[lane] : Sums{0, 0, 0};
    for (int d = 1; d < 32; d <<= 1) {
      const Sums o = shfl_up(w, d);
      if (lane >= d) w = add(w, o);
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  if (warp > 0) inc = add(inc, s_warp[warp - 1]);
  const Sums all = s_warp[warps - 1];
  const long long stack = (long long)free_count + all.back;
  const bool ok = !bad && all.need <= stack && all.rows <= p.max_rows && stack <= p.num_pages;
  if (b < p.B) {
    s_start[b] = ok ? (int)(inc.rows - own.rows) : 0;
    s_kv[b] = ok ? kv : len;
    s_held[b] = held;
    s_need[b] = ok ? (int)(inc.need - own.need) : 0;
    s_back[b] = ok ? (int)(inc.back - own.back) : 0;
    atomicMax(&s_max, ok ? kv : len);
  }
  if (b == 0) {
    s_start[p.B] = ok ? (int)all.rows : 0;
    s_need[p.B] = ok ? (int)all.need : 0;
    s_back[p.B] = ok ? (int)all.back : 0;
  }
  cluster_sync();  // the inputs have been read
  if (cta == 0) {
    for (int i = b; i <= p.B; i += kPlanThreads) {
      p.row_start[i] = s_start[i];
      if (i < p.B) p.kv_len[i] = s_kv[i];
    }
    if (b == 0) {
      *p.free_left = ok ? (int)(stack - all.need) : free_count;
      p.report[0] = ok ? DKV_OK : DKV_ERR_CAPACITY;
      p.report[1] = s_start[p.B];
      p.report[2] = s_need[p.B];
      p.report[3] = s_max;
    }
  }
  // released pages onto the stack: a warp takes up to 256 pages of a sequence, 8 reads to a lane
  // in flight
  if (s_back[p.B] > 0) {
    const int parts = (p.max_pages + 255) / 256;
    for (int w = cta * warps + warp; w < p.B * parts; w += ctas * warps) {
      const int s = w / parts, first = (w - s * parts) * 256;
      const int at = s_back[s], n = s_back[s + 1] - at;
      if (first >= n) continue;
      const int* from = p.table + (size_t)s * p.max_pages + first;
      int page[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (first + i * 32 + lane < n) page[i] = from[i * 32 + lane];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (first + i * 32 + lane < n) p.free_pages[free_count + at + first + i * 32 + lane] = page[i];
    }
    cluster_sync();
  }
  // pages taken, from the top of the stack
  if (s_need[p.B] > 0) {
    for (int k = cta * kPlanThreads + b; k < s_need[p.B]; k += ctas * kPlanThreads) {
      const int page = __ldcg(p.free_pages + stack - 1 - k);
      int s = 0;  // the last sequence whose first page is at most the k-th
      for (int step = 1 << (31 - __clz(p.B)); step; step >>= 1)
        if (s + step < p.B && s_need[s + step] <= k) s += step;
      p.table[(size_t)s * p.max_pages + s_held[s] + k - s_need[s]] = page;
    }
    cluster_sync();
  }
  // Many rows, four of a thread at once, so that their reads do not wait for one another: 65536
  // rows of 512 sequences take 11.6 us so, 13.4 row by row; 1024 rows of as many 7.3 and 6.4.
  const int first = cta * kPlanThreads + b, stride = ctas * kPlanThreads;
  if (p.max_rows > 2 * stride) fill_rows<4>(p, s_start, s_kv, first, stride);
  else fill_rows<1>(p, s_start, s_kv, first, stride);
}

constexpr int kCluster = 8;

dkv_status refuse(dkv_status s, const char* msg) {
  set_last_error(s, msg);
  return s;
}

}  // namespace

extern "C" dkv_status dkv_step_plan(const int32_t* lengths, const int32_t* new_tokens,
                                    int32_t* page_table, int32_t* free_pages,
                                    const int32_t* free_count, int batch, int max_pages,
                                    int page_tokens, int num_pages, int max_rows,
                                    int32_t* row_start, int32_t* row_pos, int32_t* row_slot,
                                    int32_t* kv_len, int32_t* free_left, int32_t* report,
                                    void* stream) {
  if (!lengths || !new_tokens || !page_table || !free_pages || !free_count || !row_start ||
      !row_pos || !row_slot || !kv_len || !free_left || !report)
    return refuse(DKV_ERR_INVALID_ARG, "null pointer argument");
  if (batch <= 0 || batch > DKV_MAX_STEP_BATCH)
    return refuse(DKV_ERR_INVALID_ARG, "batch outside [1, DKV_MAX_STEP_BATCH]");
  if (page_tokens < 1 || page_tokens > 4096 || (page_tokens & (page_tokens - 1)))
    return refuse(DKV_ERR_INVALID_ARG, "page_tokens must be a power of two in [1, 4096]");
  if (max_pages <= 0 || (long long)max_pages * page_tokens > (1LL << 30))
    return refuse(DKV_ERR_INVALID_ARG, "max_pages must be positive, max_pages * page_tokens at most 2^30");
  if (num_pages <= 0 || (long long)num_pages * page_tokens > (1LL << 30))
    return refuse(DKV_ERR_INVALID_ARG, "num_pages must be positive, num_pages * page_tokens at most 2^30");
  if (max_rows <= 0 || max_rows > (1 << 30))
    return refuse(DKV_ERR_INVALID_ARG, "max_rows outside [1, 2^30]");
  PlanParams p;
  p.lengths = lengths; p.new_tokens = new_tokens; p.table = page_table;
  p.free_pages = free_pages; p.free_count = free_count;
  p.row_start = row_start; p.row_pos = row_pos; p.row_slot = row_slot;
  p.kv_len = kv_len; p.free_left = free_left; p.report = report;
  p.B = batch; p.max_pages = max_pages; p.num_pages = num_pages; p.max_rows = max_rows;
  p.shift = 0;
  while ((1 << p.shift) < page_tokens) ++p.shift;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cfg.gridDim.x;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, plan_kernel, p);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? DKV_OK : refuse(DKV_ERR_CUDA, cudaGetErrorString(e));
}
