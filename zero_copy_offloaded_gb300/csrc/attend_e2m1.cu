// dkv_paged_attend: softmax attention of ragged query rows over a paged cache
// held in 4 bits (E2M1 codes, an E4M3 scale per 16 elements).
//
// For query row i of sequence b (n_b rows, len_b cached keys, the rows' own keys
// among them), query head h:
//   s_j = scale * q . k_j   for keys j <= len_b - n_b + i,  o = sum_j softmax(s)_j v_j
// in one pass over the keys with the running maximum and sum of the softmax.
//
// Work: an item is (sequence, KV head, R query rows of that head's group, rows
// counted token-major over the G heads); its keys are cut into tiles of 128.
// All tiles of all items form one line that is dealt to the CTAs in equal
// contiguous ranges, whatever the lengths are, from the lengths on the device
// (no host copy, so a captured graph serves any lengths).  A CTA that holds a whole
// item writes its rows; an item cut between CTAs leaves fp32 partials, which the CTA that
// finishes last joins in CTA order (no CTA waits for another), many pieces in groups first: one
// KV head over 131072 keys takes 19 us so, 98 where one CTA joins its 456 pieces row by row.
//
// Inside a CTA each of 4 warps takes 32 keys of every tile through its own
// cp.async ring, with no barrier between warps until the item ends.  Per 16 keys:
//   S^T[16 keys, 8 rows] = K Q^T  and  O^T[D, 8 rows] += V^T P^T  as m16n8k16 MMAs,
// keys (then dims) in the M = 16 slot, so that a group of up to 8 query heads of a
// single token fills the N = 8 slot.  The contraction order inside an MMA is free:
// each thread uses its codes in the order in which its wide shared-memory load
// brings them, and q, the key order of P and the dims of O follow.  Codes become
// fp16 in registers; code x scale is exact in fp16 (6 significant bits), so the
// MMA operands carry no rounding of the cache.  bf16 queries are brought to fp16's
// range by a power of two per row (exact, undone on the scores; an element below
// 2^-27 of its row's largest may lose bits).  P is rounded to fp16, as the tensor
// operand must be 16 bits: 2^-11 of a weight, and 2^-32 of the row's largest for
// weights below 2^-21 of it (kBias); scores, references, sums and outputs stay in fp32.
//
// Why mma.sync here: tcgen05 takes at least 128 rows (or columns) a tile and its operands from
// shared memory, so the converted keys would be written and read there once more.  Sixteen
// rows of 32/8 heads over 16 x 8192 keys take 111 us in attend_e2m1_tc.cu's kernel, 58 here;
// 32 rows 111 and 84 (heads of 64: 98 and 57); 33 rows and more, for whose outputs there
// are no registers here, go there.
//
// What bounds it: reading 9/16 byte an element, 1152 bytes for 16 keys of a head of 128.  The
// 8 x 32769 keys of 8 heads (302 MB) take 73 us, 4.1 TB/s of 6.8 measured (4 x 131073 keys:
// 126 us, 4.8 TB/s).  With nothing converted or multiplied the same copies take 62 us, and the
// conversion and MMAs on resident data 57 us: the two do not overlap fully with 12 warps on
// an SM.  A sub costs about 260 instructions, 64 of them the conversions of two codes each.
// 168 registers a thread and three CTAs beat 128 and four (75 and 80 us): with fewer the
// compiler computes addresses again and again.  More rows: an MMA m16n8k16 takes 8 cycles of
// a scheduler, 96 of them a warp's 32 keys at 24 rows, a quarter of the time that two
// warps a scheduler need (20 rows over 16 x 8192 keys: 69 us); and a piece has a fixed cost, queries,
// join of the warps and of the CTAs, of about 10000 cycles, near three of its tiles of 128 keys.
#include <float.h>
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>
#include <chrono>
#include <type_traits>

#include "attend_e2m1.cuh"
#include "tc_common.cuh"

namespace dkv {
void set_last_error(dkv_status s, const char* msg);
}

namespace {

using namespace dkv;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 16;                // keys of one MMA, one ring slot
constexpr int kStep = 2 * kSub;         // keys of one warp step
constexpr int kTile = kStep * kWarps;   // keys of one tile
// What an item costs beside its key tiles (its queries, the join of the warps), in tiles: the
// CTAs' ranges are dealt with it.  48 sequences of up to 8193 keys of 32 heads of 64 take 187 us
// with 0, 185 with 1, 150 with 3, 154 with 6.
constexpr int kItemCost = 3;
// Pieces joined at once; beyond that in groups first, of sixteen (one KV head over 131072 keys of 64:
// 16.6 us with 16, 17.6 with 20) or of as many as leave kJoinOnce groups.
constexpr int kJoinOnce = 32, kGroup = 16;
__device__ __forceinline__ int group_size(int pieces) { return max(kGroup, (pieces + kJoinOnce - 1) / kJoinOnce); }
constexpr int kSms = 152, kMaxCtas = 4 * kSms;
// A row's weights are 2^(s - m) with m below its running maximum, so that the largest are 2^kBias to
// 2^(kBias + kLazy): fp16 has room above 1, and a weight keeps all its bits down to 2^-21 of the
// row's largest and counts down to 2^-32 (with m at the maximum itself 2^-14 and 2^-25, where thousands of
// keys beside one that is 17 above them are lost).  A factor of 2 is left below fp16's largest number
// for the rounding of m and of its threshold, at most 2^-2 each for scores up to 2^21.  More bias leaves less
// to kLazy: drafts of 5 with scores of a standard deviation of 4 take 52.4 us with 7 and 8, 54.6 with 10 and 5.
constexpr float kBias = 7.0f;
constexpr float kLazy = 8.0f;    // m moves only when a score passes m + kBias by this
constexpr float kNone = -3e38f;  // m of a row that has seen no key

template <int D, int NT>
struct Cfg {
  static constexpr int R = 8 * NT;                   // query rows per item
  static constexpr int kC = kSub * e2m1::code_bytes(D);
  static constexpr int kS = kSub * e2m1::scale_bytes(D);
  static constexpr int kSlot = 2 * (kC + kS);        // K codes | V codes | K scales | V scales
  static constexpr int kOffScale = 2 * kC;
  static constexpr int kSteps = D == 128 ? 3 : 4;    // steps in a warp's ring
  static constexpr int kRing = 2 * kSteps * kSlot;   // per warp
  static constexpr int kMerge = kWarps * 8 * D * 4;  // one 8-row round of every warp's O
  static constexpr int kOffMerge = kWarps * kRing;
  static constexpr int kOffMl = kOffMerge + kMerge;          // m, l and factor [kWarps][R], m and l [R]
  static constexpr int kQueries = NT > 1 ? NT * (D / 16) * 32 * 8 : 0;  // B fragments of the rows
  static constexpr int kOffQ = kOffMl + (3 * kWarps + 2) * R * 4;       // and their scales, visible keys
  static constexpr int kOffBatch = kOffQ + kQueries + (NT > 1 ? 2 * R * 4 : 0);
  // resident CTAs per SM, by registers: o takes 4 NT D/16 of a thread's.  Eight rows of heads of
  // 64: 48 sequences of up to 8193 keys of 32 heads take 139 us with four, 149 with three; but
  // 16 x 512 keys of 8 heads 11.6 and 10.4, so that the fourth stays out of short ranges.
  static constexpr int kPerSm = NT == 1 && D == 64 ? 4 : NT == 1 || (NT <= 3 && D == 64) ? 3 : 2;
  // subs in flight at once: 20 rows over 16 x 32768 keys of 8 heads of 128 take 214 us with two, 225
  // with one; of 64 141 and 142; four groups of rows have no registers for it
  static constexpr int kBoth = NT == 1 || (NT <= 3 && D == 128) ? 2 : 1;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void cp_async16_u32(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int V>
__device__ __forceinline__ void store_vec(float* to, const float (&x)[V]) {
  if constexpr (V == 4) *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
  else *reinterpret_cast<float2*>(to) = make_float2(x[0], x[1]);
}
template <int V>
__device__ __forceinline__ void load_shared(const float* from, float (&x)[V]) {
  if constexpr (V == 4) {
    const float4 y = *reinterpret_cast<const float4*>(from);
    x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
  } else {
    const float2 y = *reinterpret_cast<const float2*>(from);
    x[0] = y.x; x[1] = y.y;
  }
}
// From L2: another SM wrote it during this kernel.
template <int V>
__device__ __forceinline__ void load_vec(const float* from, float (&x)[V]) {
  if constexpr (V == 4) {
    const float4 y = __ldcg(reinterpret_cast<const float4*>(from));
    x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
  } else {
    const float2 y = __ldcg(reinterpret_cast<const float2*>(from));
    x[0] = y.x; x[1] = y.y;
  }
}

// Whether a sub's keys are all seen by every row of the item.
using Inner = std::false_type;
using Edge = std::true_type;

// Where a CTA is on the line of tiles.
struct Pos {
  int b, h, qt, tile;  // sequence, KV head, query tile, key tile
  int qtiles, tiles;   // of sequence b
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kPerSm) attend_kernel(const AttendParams p) {
  using C = Cfg<D, NT>;
  constexpr int R = C::R, J = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  // MMA row r of a sub is key (r >> 1) for even r, ((r >> 1) ^ 1) + 4 for odd r < 8, and 8 more in
  // the upper half: two rows that one phase of K's 16-byte loads reads have different
  // parity, and so have the keys of neighbouring lanes of V's loads, so that neither meets a
  // bank conflict with K in its natural order.
  const int key_g = g & 1 ? ((g >> 1) ^ 1) + 4 : g >> 1;
  uint8_t* ring = smem + warp * C::kRing;
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  float* s_m = reinterpret_cast<float*>(smem + C::kOffMl);
  float *s_l = s_m + kWarps * R, *s_f = s_l + kWarps * R, *s_top = s_f + kWarps * R, *s_sum = s_top + R;
  uint2* s_q = reinterpret_cast<uint2*>(smem + C::kOffQ);
  float* s_scale = reinterpret_cast<float*>(smem + C::kOffQ + C::kQueries);
  int* s_vis = reinterpret_cast<int*>(s_scale + R);
  __shared__ int s_join[3];
  long long* s_pre = reinterpret_cast<long long*>(smem + C::kOffBatch);  // [B + 1]
  int* s_kv = reinterpret_cast<int*>(s_pre + p.B + 1);                   // [B]
  int* s_row = s_kv + p.B;                                               // [B]
  int* s_n = s_row + p.B;                                                // [B]
  const int G = p.G;

  // the line of tiles: lengths, row counts, and the prefix of tile counts
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    int kv, row, n;
    batch_entry(p, b, kv, row, n);
    s_kv[b] = kv;
    s_row[b] = row;
    s_n[b] = n;
    s_pre[b + 1] = (long long)p.Hkv * ((n * G + R - 1) / R) * (max(1, (kv + kTile - 1) / kTile) + kItemCost);
  }
  if (threadIdx.x == 0) s_pre[0] = 0;
  __syncthreads();
  if (warp == 0) {
    long long carry = 0;
    for (int base = 0; base < p.B; base += 32) {
      long long v = base + lane < p.B ? s_pre[base + lane + 1] : 0;
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(~0u, v, d);
        if (lane >= d) v += o;
      }
      v += carry;
      if (base + lane < p.B) s_pre[base + lane + 1] = v;
      carry = __shfl_sync(~0u, v, 31);
    }
  }
  __syncthreads();
  const long long total = s_pre[p.B];
  // with less work than CTAs the first `total` CTAs take one unit each, so that an
  // item's pieces always lie in consecutive CTAs; a fourth CTA an SM only for long ranges
  long long ctas = min(total, (long long)gridDim.x);
  if (C::kPerSm > 3 && total < 4 * (long long)gridDim.x) ctas = min(ctas, (long long)3 * kSms);
  if ((long long)blockIdx.x >= ctas) return;
  const long long g0 = total * blockIdx.x / ctas, g1 = total * (blockIdx.x + 1) / ctas;
  auto owner = [&](long long at) { return (int)(((at + 1) * ctas - 1) / total); };  // of a unit of the line

  auto enter = [&](Pos& at, int b) {
    at.b = b;
    at.qtiles = (s_n[b] * G + R - 1) / R;
    at.tiles = max(1, (s_kv[b] + kTile - 1) / kTile);
  };
  // The tile after `at`; `left`, the units of the CTA's range from `at` on, goes with it.
  auto next_tile = [&](Pos& at, int& left) {
    --left;
    if (++at.tile < at.tiles) return;
    left -= kItemCost;
    at.tile = 0;
    if (++at.qt < at.qtiles) return;
    at.qt = 0;
    if (++at.h < p.Hkv) return;
    at.h = 0;
    int b = at.b + 1;
    while (b < p.B && s_n[b] == 0) ++b;
    if (b < p.B) enter(at, b);
  };
  Pos cons;
  int left = (int)(g1 - g0);
  {
    int lo = 0, hi = p.B;  // s_pre[lo] <= g0 < s_pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid] <= g0) lo = mid; else hi = mid;
    }
    enter(cons, lo);
    const long long rem = g0 - s_pre[lo];
    const int units = cons.tiles + kItemCost;
    const long long item = rem / units;
    const int in_item = (int)(rem - item * units);  // an item's first units stand for its fixed cost
    cons.tile = max(0, in_item - kItemCost);
    left -= max(0, kItemCost - in_item);
    cons.h = (int)(item / cons.qtiles);
    cons.qt = (int)(item - (long long)cons.h * cons.qtiles);
  }
  if (left <= 0) return;

  // ---- producer side: this warp's next step to fetch -------------------------
  // 16-byte asynchronous copies, a lane's share at fixed places: chunks `lane` and `lane + 32`
  // of a sub's K and V codes, and lanes below 2 kS / 16 one chunk of its scales.  (Bulk copies
  // of whole runs take one instruction sequence per lane that issues one: a warp that
  // issues 8 of them for every step spends a third of its instructions there.)
  Pos prod = cons;
  int to_issue = left;  // units from prod on
  uint32_t have = 0;    // bit 2 * (step in the ring) + sub: the sub holds keys
  constexpr int SCH = C::kS / 16;                    // chunks of one scale block
  constexpr int CPR = e2m1::code_bytes(D) / 16;      // chunks of a key's codes
  const size_t page_stride = (size_t)p.Hkv * p.page_bytes;
  const uint32_t ring_u = smem_u32(ring);
  // V's chunks of keys 2, 3 mod 4 are swapped in pairs (D = 128), which keeps V's loads conflict-free
  const uint32_t dst_k = ring_u + lane * 16;
  const uint32_t dst_v = ring_u + C::kC + (D == 128 ? (lane ^ ((lane / CPR) & 2)) : lane) * 16;
  const uint32_t dst_s = ring_u + C::kOffScale + lane * 16;
  const uint8_t* scale_pool = lane < SCH ? p.k_pool : p.v_pool;
  const size_t scale_off = ((size_t)e2m1::code_bytes(D) << p.page_shift) + (lane & (SCH - 1)) * 16;
  // pool pages of prod's two subs (-1: nothing to fetch)
  auto find_pages = [&](int (&page)[2]) {
    page[0] = page[1] = -1;
    if (to_issue <= 0) return;
    const int t = prod.tile * kTile + warp * kStep, kv = s_kv[prod.b];
    const int* row = p.table + (size_t)prod.b * p.max_pages;
    if (t < kv) page[0] = __ldg(row + (t >> p.page_shift));
    if (t + kSub < kv) page[1] = __ldg(row + ((t + kSub) >> p.page_shift));
  };
  int in = 0;  // the step to issue, in the ring
  auto copy = [&](int h, int tile, const int (&page)[2]) {
    const size_t head = (size_t)h * p.page_bytes;
    const int t = tile * kTile + warp * kStep, mask = (1 << p.page_shift) - 1;
    have &= ~(3u << (2 * in));
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      if ((uint32_t)page[sub] < (uint32_t)p.num_pages) {
        const int row = (t + sub * kSub) & mask;
        const size_t at = (size_t)page[sub] * page_stride + head;
        const size_t codes = at + (size_t)row * e2m1::code_bytes(D) + lane * 16;
        const uint32_t slot = (2 * in + sub) * C::kSlot;
#pragma unroll
        for (int i = 0; i < C::kC / 512; ++i) {
          cp_async16_u32(dst_k + slot + i * 512, p.k_pool + codes + i * 512);
          cp_async16_u32(dst_v + slot + i * 512, p.v_pool + codes + i * 512);
        }
        if (lane < 2 * SCH)
          cp_async16_u32(dst_s + slot, scale_pool + at + scale_off + row * e2m1::scale_bytes(D));
        have |= 1u << (2 * in + sub);
      }
    }
    cp_async_commit();
    in = in + 1 == C::kSteps ? 0 : in + 1;
  };
  int page[2];
  {  // the first steps: every page is looked up before the first one is waited for
    int first[C::kSteps][2], hs[C::kSteps], tiles[C::kSteps];
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) {
      find_pages(first[i]);
      hs[i] = prod.h;
      tiles[i] = prod.tile;
      if (to_issue > 0) next_tile(prod, to_issue);
    }
    find_pages(page);
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) copy(hs[i], tiles[i], first[i]);
  }
  auto issue = [&]() {
    copy(prod.h, prod.tile, page);
    if (to_issue > 0) next_tile(prod, to_issue);
    find_pages(page);
  };

  // ---- consumer side -----------------------------------------------------------
  int ring_at = 0;  // the step to take, in the ring
  while (left > 0) {
    const int b = cons.b, h = cons.h, qt = cons.qt;
    const int kv = s_kv[b], n = s_n[b], row0 = s_row[b];
    const int tile0 = cons.tile;
    const int tile1 = min(cons.tiles, tile0 + left);
    const int last = min((qt + 1) * R, n * G) - 1;  // last packed row of the item
    const int minvis = max(0, kv - n + (qt * R) / G + 1), maxvis = max(0, kv - n + last / G + 1);

    // A piece of a cut item: which CTAs hold it, and the counter of its finished pieces, which
    // stands beside the call's own tag and starts from nothing wherever another tag is found,
    // so that it needs no clearing before the call.  The tag is set here, while nothing waits.
    const bool cut = tile0 > 0 || tile1 < cons.tiles;
    // piece i lies in slot 2 (c0 + i), but the first in slot 2 c0 + 1
    auto slot_of = [&](int c0, int i) { return 2 * (c0 + i) + (i == 0); };
    unsigned long long *counter = nullptr, seen = 0;  // of thread 0
    if (cut && threadIdx.x == 0) {
      const long long first_unit =
          s_pre[b] + ((long long)h * cons.qtiles + qt) * (cons.tiles + kItemCost) + kItemCost;
      const int c0 = owner(first_unit), pieces = owner(first_unit + cons.tiles - 1) - c0 + 1;
      s_join[0] = c0;
      s_join[1] = pieces;
      counter = pieces <= kJoinOnce ? p.done + 2 * kMaxCtas + c0
                                    : p.done + slot_of(c0, ((int)blockIdx.x - c0) / group_size(pieces) * group_size(pieces));
      seen = *reinterpret_cast<volatile unsigned long long*>(counter);
    }

    // Queries as B fragments: eight rows in registers, more in shared memory, where each warp
    // prepares some groups of eight for all.
    constexpr bool QS = C::kQueries > 0;
    uint32_t qf[QS ? 1 : NT][2 * J];
    float sl1[2];  // eight rows: the scales and visible keys of this thread's two score columns
    int vis1[2];
    auto load_q = [&](int nt, uint32_t (&f)[2 * J]) {  // returns what undoes the rows' scaling
      const int pr = qt * R + nt * 8 + g;
      float unscale = 1.0f;
      if (pr <= last) {
        const int t = pr / G;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const T*>(p.q) + (size_t)(row0 + t) * p.q_stride + (size_t)(h * G + pr - t * G) * D +
            c * (D / 4));
#pragma unroll
        for (int i = 0; i < J / 2; ++i) {
          const uint4 w = __ldg(src + i);
          f[4 * i] = w.x; f[4 * i + 1] = w.y; f[4 * i + 2] = w.z; f[4 * i + 3] = w.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2 * J; ++i) f[i] = 0;
      }
      if constexpr (DT<T>::code == DKV_BF16) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * J; ++i) {
          const float2 y = DT<T>::to_f2(f[i]);
          top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
        }
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        // largest element to [2^13, 2^14)
        int e = (int)(__float_as_uint(top) >> 23) - 127;
        e = top > 0.f && top <= FLT_MAX ? max(e, -113) : 13;
        const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
        unscale = __uint_as_float((uint32_t)(127 - 13 + e) << 23);
#pragma unroll
        for (int i = 0; i < 2 * J; ++i) {
          const float2 y = DT<T>::to_f2(f[i]);
          f[i] = tc::pack2<__half>(y.x * up, y.y * up);
        }
      }
      if (p.scale_log2 < 0.f) {  // the scale's sign goes to the queries
#pragma unroll
        for (int i = 0; i < 2 * J; ++i) f[i] ^= 0x80008000u;
      }
      // positive and finite, so that a masked -infinity stays one
      return fminf(fmaxf(fabsf(p.scale_log2) * unscale, 1e-37f), FLT_MAX);
    };
    if constexpr (QS) {
      for (int nt = warp; nt < NT; nt += kWarps) {
        uint32_t f[2 * J];
        const float scale = load_q(nt, f);
#pragma unroll
        for (int j = 0; j < J; ++j) s_q[(nt * J + j) * 32 + lane] = make_uint2(f[2 * j], f[2 * j + 1]);
        if (c == 0) {
          const int pr = qt * R + nt * 8 + g;
          s_scale[nt * 8 + g] = scale;
          s_vis[nt * 8 + g] = pr <= last ? max(0, kv - n + pr / G + 1) : 0;
        }
      }
      __syncthreads();
    }
    if constexpr (!QS) {
      const float scale = load_q(0, qf[0]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        sl1[u] = __shfl_sync(~0u, scale, (2 * c + u) * 4);
        const int pc = qt * R + 2 * c + u;
        vis1[u] = pc <= last ? max(0, kv - n + pc / G + 1) : 0;
      }
    }
    auto scales = [&](int nt) {
      return QS ? *reinterpret_cast<const float2*>(s_scale + nt * 8 + 2 * c) : make_float2(sl1[0], sl1[1]);
    };
    auto visible = [&](int nt) {
      return QS ? *reinterpret_cast<const int2*>(s_vis + nt * 8 + 2 * c) : make_int2(vis1[0], vis1[1]);
    };

    auto tag = [&](unsigned long long* word, unsigned long long was) {
      if ((was ^ p.tag) >> 16) atomicCAS(word, was, p.tag);
    };
    if (cut && threadIdx.x == 0) tag(counter, seen);

    // reference of the weights (base 2, scaled), the raw score that moves it, sum, output
    float m[NT][2], thr[NT][2], l[NT][2], o[NT][J][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNone;
      thr[nt][0] = thr[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < J; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }

    // raw scores of one sub, masked; whether one moves its row's reference
    auto scores = [&](auto edge, const uint8_t* st, int t0, float (&s)[NT][4]) -> bool {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      constexpr int W = D / 32;  // code words of a thread per key
      uint32_t kw[2][W], ks[2][2];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const uint8_t* row = st + (key_g + 8 * rr) * e2m1::code_bytes(D) + c * (D / 8);
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(row);
          kw[rr][0] = w.x; kw[rr][1] = w.y; kw[rr][2] = w.z; kw[rr][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(row);
          kw[rr][0] = w.x; kw[rr][1] = w.y;
        }
        const uint8_t* sp = st + C::kOffScale + (key_g + 8 * rr) * e2m1::scale_bytes(D) + c * (D / 64);
        if constexpr (D == 128) {
          const uint32_t s2 = e2m1::scales_to_h2(*reinterpret_cast<const uint16_t*>(sp));
          ks[rr][0] = __byte_perm(s2, 0, 0x1010);
          ks[rr][1] = __byte_perm(s2, 0, 0x3232);
        } else {
          ks[rr][0] = ks[rr][1] = __byte_perm(e2m1::scales_to_h2(*sp), 0, 0x1010);
        }
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t x[2][4];
        e2m1::codes_to_h2(kw[0][w], x[0]);
        e2m1::codes_to_h2(kw[1][w], x[1]);
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const int j = 2 * w + jj;
          uint32_t a[4];
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            a[rr] = hmul2(x[rr][2 * jj], ks[rr][D == 128 ? w / 2 : 0]);
            a[rr + 2] = hmul2(x[rr][2 * jj + 1], ks[rr][D == 128 ? w / 2 : 0]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (QS) {
              const uint2 q = s_q[(nt * J + j) * 32 + lane];
              mma16816(s[nt], a, q.x, q.y);
            } else {
              mma16816(s[nt], a, qf[nt][2 * j], qf[nt][2 * j + 1]);
            }
          }
        }
      }
      const int tok = t0 + key_g;
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (edge) {
          const int2 vis = visible(nt);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (tok + 8 * (u >> 1) >= (u & 1 ? vis.y : vis.x)) s[nt][u] = -INFINITY;
        }
        up |= fmaxf(s[nt][0], s[nt][2]) > thr[nt][0];
        up |= fmaxf(s[nt][1], s[nt][3]) > thr[nt][1];
      }
      return up;
    };

    // weights of one sub, then o += V^T P^T
    auto values = [&](auto edge, const uint8_t* st, int t0, const float (&s)[NT][4]) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 sl = scales(nt);
        const float p0 = tc::ex2_approx(fmaf(s[nt][0], sl.x, -m[nt][0]));
        const float p1 = tc::ex2_approx(fmaf(s[nt][1], sl.y, -m[nt][1]));
        const float p2 = tc::ex2_approx(fmaf(s[nt][2], sl.x, -m[nt][0]));
        const float p3 = tc::ex2_approx(fmaf(s[nt][3], sl.y, -m[nt][1]));
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        pb[nt][0] = transpose8x8(tc::pack2<__half>(p0, p1));
        pb[nt][1] = transpose8x8(tc::pack2<__half>(p2, p3));
      }
      // keys c, (c^1)+4, c+8, (c^1)+12 of the sub, dims [g * D/8, (g + 1) * D/8)
      constexpr int W = D / 64;
      uint32_t vw[4][W], sb[4];
      const uint8_t* sv = st + C::kOffScale + C::kS + (D == 128 ? g : g >> 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = (k & 1 ? c ^ 1 : c) + 4 * k;
        const uint8_t* row = st + C::kC + t * e2m1::code_bytes(D);
        if constexpr (D == 128) {
          const uint2 w = *reinterpret_cast<const uint2*>(row + ((g >> 1) ^ (t & 2)) * 16 + (g & 1) * 8);
          vw[k][0] = w.x; vw[k][1] = w.y;
        } else {
          vw[k][0] = *reinterpret_cast<const uint32_t*>(row + g * 4);
        }
        sb[k] = sv[t * e2m1::scale_bytes(D)];
      }
      if constexpr (edge) {
#pragma unroll
        for (int k = 0; k < 4; ++k)  // nobody sees this key, or its NaN is dealt out below
          if (t0 + (k & 1 ? c ^ 1 : c) + 4 * k >= maxvis || (sb[k] & 0x7f) == 0x7f) sb[k] = 0;
      }
      const uint32_t vs[2] = {e2m1::scales_to_h2(sb[0] | (sb[1] << 8)),
                              e2m1::scales_to_h2(sb[2] | (sb[3] << 8))};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        // bytes that pair one dim of two keys: even dims, odd dims
        uint32_t ev[2][4], od[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t lo = vw[2 * k][w], hi = vw[2 * k + 1][w];
          e2m1::codes_to_h2((lo & 0x0F0F0F0Fu) | ((hi << 4) & 0xF0F0F0F0u), ev[k]);
          e2m1::codes_to_h2(((lo >> 4) & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u), od[k]);
        }
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          const uint32_t a[4] = {hmul2(ev[0][ii], vs[0]), hmul2(od[0][ii], vs[0]),
                                 hmul2(ev[1][ii], vs[1]), hmul2(od[1][ii], vs[1])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][4 * w + ii], a, pb[nt][0], pb[nt][1]);
        }
      }
      if constexpr (edge) {
        // A NaN block of V reaches the rows that see its key, and no others (a
        // zero weight times NaN would reach them all).
        bool nan = false;  // in this thread's four keys: read again, so that the loop above keeps no flag
#pragma unroll
        for (int k = 0; k < 4; ++k)
          nan |= (reinterpret_cast<const volatile uint8_t*>(sv)[(c + 4 * k) * e2m1::scale_bytes(D)] & 0x7f) == 0x7f;
#pragma unroll 1
        for (int t = __any_sync(~0u, nan) ? 0 : kSub; t < kSub; ++t)
          if ((sv[t * e2m1::scale_bytes(D)] & 0x7f) == 0x7f) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int2 vis = visible(nt);
#pragma unroll
              for (int i = 0; i < J; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  if (t0 + t < (u & 1 ? vis.y : vis.x)) o[nt][i][u] = __int_as_float(0x7fc00000);
            }
          }
      }
    };

    // takes these scores into the references and rescales what was summed under the old ones
    auto raise = [&](const float (&s)[NT][4]) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[2];
        const float2 sl = scales(nt);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float su = u ? sl.y : sl.x;
          float x = fmaxf(s[nt][u], s[nt][u + 2]);
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
          x = fmaxf(fmaf(x, su, -kBias), m[nt][u]);
          f[u] = x == m[nt][u] ? 1.0f : exp2f(m[nt][u] - x);
          m[nt][u] = x;
          if (x != kNone) thr[nt][u] = __fdividef(x + (kBias + kLazy), su);
          l[nt][u] *= f[u];
        }
#pragma unroll
        for (int i = 0; i < J; ++i) {
          o[nt][i][0] *= f[0]; o[nt][i][1] *= f[1];
          o[nt][i][2] *= f[0]; o[nt][i][3] *= f[1];
        }
      }
    };

#pragma unroll 1
    for (int tile = tile0; tile < tile1; ++tile) {
      cp_async_wait_group<C::kSteps - 1>();
      __syncwarp();
      const int t0 = tile * kTile + warp * kStep;
      const uint8_t* st = ring + ring_at * (2 * C::kSlot);
      const uint32_t on = (have >> (2 * ring_at)) & 3;
      if (on == 3 && t0 + kStep <= minvis) {  // every row sees every key
        float s[2][NT][4];
        if constexpr (C::kBoth == 2) {
          const bool a = scores(Inner(), st, t0, s[0]);
          const bool b = scores(Inner(), st + C::kSlot, t0 + kSub, s[1]);
          if (__any_sync(~0u, a | b)) {
            raise(s[0]);
            raise(s[1]);
          }
          values(Inner(), st, t0, s[0]);
          values(Inner(), st + C::kSlot, t0 + kSub, s[1]);
        } else {
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            if (__any_sync(~0u, scores(Inner(), st + k * C::kSlot, t0 + k * kSub, s[0]))) raise(s[0]);
            values(Inner(), st + k * C::kSlot, t0 + k * kSub, s[0]);
          }
        }
      } else {
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          const int ts = t0 + k * kSub;
          if (!((on >> k) & 1) || ts >= maxvis) continue;
          float s[NT][4];
          if (__any_sync(~0u, scores(Edge(), st + k * C::kSlot, ts, s))) raise(s);
          values(Edge(), st + k * C::kSlot, ts, s);
        }
      }
      ring_at = ring_at + 1 == C::kSteps ? 0 : ring_at + 1;
      __syncwarp();
      issue();
    }

    // ---- the piece's end: join the warps --------------------------------------
    // This runs once a piece and mostly waits for its own instructions: loops stay rolled where
    // they can, and the rows of a round are moved to where the one copy of its code takes them.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x = l[nt][u];
        x += __shfl_xor_sync(~0u, x, 4);
        x += __shfl_xor_sync(~0u, x, 8);
        x += __shfl_xor_sync(~0u, x, 16);
        if (lane < 4) {
          s_m[warp * R + nt * 8 + 2 * c + u] = m[nt][u];
          s_l[warp * R + nt * 8 + 2 * c + u] = x;
        }
      }
    __syncthreads();
    if (threadIdx.x < kWarps * R) {  // what a warp's part of a row counts against the CTA's maximum
      const int r = threadIdx.x % R;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w * R + r]);
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) {
        const float mw = s_m[w * R + r], f = mw == top ? 1.0f : exp2f(mw - top);
        sum += s_l[w * R + r] * f;
        if (threadIdx.x == w * R + r) s_f[w * R + r] = f;
      }
      if (threadIdx.x < R) {
        s_top[r] = top;
        s_sum[r] = sum;
      }
    }
    constexpr int V = D / 32;  // outputs of a lane
    const bool starts = tile0 == 0, ends = tile1 == cons.tiles, whole = starts && ends;
    const int slot = 2 * blockIdx.x + (starts ? 1 : 0), rows = last - qt * R + 1, d0 = lane * V;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
      // Eight rows of every warp, a row's pair i of the D/8 dims of thread group g at place
      // J g + (i ^ x), x from the row and g: neither these stores nor the loads below meet a
      // bank conflict (with plain padded rows a round takes 1600 cycles, two thirds of them for conflicts).
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < J; ++i)
          reinterpret_cast<float2*>(merge)[(warp * 8 + 2 * c + u) * (D / 2) + J * g +
                                           (i ^ (D == 128 ? (g >> 1 & 1) | c << 1 : c))] =
              make_float2(o[0][i][u], o[0][i][u + 2]);
      __syncthreads();
#pragma unroll 1
      for (int r = r0 + warp; r < min(rows, r0 + 8); r += kWarps) {
        const int pr = qt * R + r;
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = s_f[w * R + r];
          const int rl = r - r0;
          float x[V];
          load_shared<V>(merge + (w * 8 + rl) * D + g * (2 * J) + (c ^ rl >> 1) * V, x);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(x[e], f, acc[e]);
        }
        if (D == 128 && (lane & 8)) {  // its two pairs lie the other way round
          const float a0 = acc[0], a1 = acc[1];
          acc[0] = acc[V - 2];
          acc[1] = acc[V - 1];
          acc[V - 2] = a0;
          acc[V - 1] = a1;
        }
        if (whole) {
          store_row<T, V>(p, row0 + pr / G, h * G + pr % G, D, d0, acc, s_top[r], s_sum[r], lane == 0);
        } else {
          store_vec<V>(p.part_o + ((size_t)slot * R + r) * D + d0, acc);
          if (lane == 0)
            *reinterpret_cast<float2*>(p.part_ml + ((size_t)slot * R + r) * 2) = make_float2(s_top[r], s_sum[r]);
        }
      }
      if constexpr (NT > 1) {
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt + 1 < NT; ++nt)
#pragma unroll
          for (int i = 0; i < J; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) o[nt][i][u] = o[nt + 1][i][u];
      }
    }
    if (!whole) {
      // ---- the CTA that finishes an item's last open piece joins them all, in CTA order.  An
      // item in many pieces is joined in two levels, first each kGroup consecutive pieces by the
      // CTA that finishes last among them, so that no CTA reads more than a few dozen.
      const int c0 = s_join[0], pieces = s_join[1];
      // this CTA's part is stored: one more of `parts` at a tagged counter; whether it was the last
      auto finish = [&](unsigned long long* word, int parts) {
        __syncthreads();
        if (threadIdx.x == 0) {
          __threadfence();
          const bool final_part = (int)(atomicAdd(word, 1ull) & 0xFFFF) == parts - 1;
          if (final_part) *word = 0;
          __threadfence();
          s_join[2] = final_part;
        }
        __syncthreads();
        return s_join[2] != 0;
      };
      // joins pieces at, at + stride, ...: `count` of them (at most 32), into the outputs or into
      // piece `at`; a warp takes every fourth row, all of them at once, so that their loads
      // are in flight together
      auto join = [&](int at, int stride, int count, bool out) {
        constexpr int RW = R / kWarps;
        auto place = [&](int i, int k) { return (size_t)slot_of(c0, at + i * stride) * R + warp + k * kWarps; };
        const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
        float2 x[RW];
        float f[RW], top[RW], acc[RW][V];
#pragma unroll
        for (int k = 0; k < RW; ++k)
          x[k] = lane < count && warp + k * kWarps < rows ? __ldcg(ml + place(lane, k)) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int k = 0; k < RW; ++k) {
          top[k] = x[k].x;
#pragma unroll
          for (int w = 16; w; w >>= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(~0u, top[k], w));
          f[k] = x[k].x == top[k] ? 1.0f : exp2f(x[k].x - top[k]);
          x[k].y *= f[k];
#pragma unroll
          for (int w = 16; w; w >>= 1) x[k].y += __shfl_xor_sync(~0u, x[k].y, w);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[k][e] = 0.f;
        }
#pragma unroll(16 / RW)
        for (int i = 0; i < count; ++i) {
#pragma unroll
          for (int k = 0; k < RW; ++k) {
            const float fi = __shfl_sync(~0u, f[k], i);
            if (warp + k * kWarps < rows) {
              float v[V];
              load_vec<V>(p.part_o + place(i, k) * D + d0, v);
#pragma unroll
              for (int e = 0; e < V; ++e) acc[k][e] = fmaf(v[e], fi, acc[k][e]);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < RW; ++k) {
          const int r = warp + k * kWarps, pr = qt * R + r;
          if (r >= rows) break;
          if (out) {
            store_row<T, V>(p, row0 + pr / G, h * G + pr % G, D, d0, acc[k], top[k], x[k].y, lane == 0);
          } else {  // the row's loads above are all done: a warp has a row to itself
            __syncwarp();
            store_vec<V>(p.part_o + place(0, k) * D + d0, acc[k]);
            if (lane == 0) *reinterpret_cast<float2*>(p.part_ml + place(0, k) * 2) = make_float2(top[k], x[k].y);
          }
        }
      };
      unsigned long long* whole_item = p.done + 2 * kMaxCtas + c0;
      if (pieces <= kJoinOnce) {
        if (finish(counter, pieces)) join(0, 1, pieces, true);
      } else {
        const int group = group_size(pieces);
        const int first = ((int)blockIdx.x - c0) / group * group, size = min(group, pieces - first);
        if (finish(counter, size)) {
          if (threadIdx.x == 0) tag(whole_item, *reinterpret_cast<volatile unsigned long long*>(whole_item));
          join(first, 1, size, false);
          const int groups = (pieces + group - 1) / group;
          if (finish(whole_item, groups)) join(0, group, groups, true);
        }
      }
    }
    __syncthreads();  // s_m, s_l, merge and s_join are free for the next piece
    left -= tile1 - tile0 - 1;
    cons.tile = tile1 - 1;
    next_tile(cons, left);
  }
}

dkv_status refuse(dkv_status s, const char* msg) {
  set_last_error(s, msg);
  return s;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }


size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Workspace: descriptors or counts | partial (max, sum) | partial o, two slots per CTA.
size_t ws_desc() { return align256(std::max(kMaxCtas * sizeof(AttendDesc), 3 * kMaxCtas * sizeof(unsigned long long))); }

std::atomic<int> g_debug_withhold{0};

// The tag of a call: 48 bits that no earlier call of this process had, scattered so that memory
// left by anything else does not hold one.
unsigned long long next_tag() {
  static std::atomic<unsigned long long> calls{(unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count()};
  unsigned long long z = calls.fetch_add(0x9E3779B97F4A7C15ull) + 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  z = (z ^ (z >> 31)) | 1ull << 63;
  return z & ~0xFFFFull;
}

// Query rows per item: the smallest of 8, 16, 24 and 32 that holds a sequence's rows;
// for more than kTcFrom rows the items of the tcgen05 kernel.
constexpr int kTcFrom = 32;
int rows_per_item(int G, int max_rows) {
  const long long rows = (long long)G * max_rows;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : rows <= kTcFrom ? 32 : kTcRows;
}
int ctas_of(int R) { return R == kTcRows ? kSms : kMaxCtas; }
size_t ws_ml(int R) { return align256((size_t)2 * ctas_of(R) * R * 2 * 4); }
size_t ws_o(int R, int D) { return align256((size_t)2 * ctas_of(R) * R * D * 4); }

template <typename T, int D, int NT>
cudaError_t launch(const AttendParams& p, cudaStream_t s) {
  using C = Cfg<D, NT>;
  const int smem = C::kOffBatch + (p.B + 1) * 8 + 3 * p.B * 4;
  static PerDevice smem_set;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = smem_set(dev, [] {
    return cudaFuncSetAttribute(attend_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::kOffBatch + (DKV_MAX_STEP_BATCH + 1) * 20);
  });
  if (e != cudaSuccess) return e;
  const int fit = 228 * 1024 / (smem + 1024);
  const int grid = kSms * (fit < C::kPerSm ? fit : C::kPerSm);
  attend_kernel<T, D, NT><<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_rows(const AttendParams& p, int R, cudaStream_t s) {
  if (R == kTcRows) return launch_attend_tc<T, D>(p, kSms, s);
  return R == 8    ? launch<T, D, 1>(p, s)
         : R == 16 ? launch<T, D, 2>(p, s)
         : R == 24 ? launch<T, D, 3>(p, s)
                   : launch<T, D, 4>(p, s);
}

}  // namespace

extern "C" size_t dkv_paged_attend_workspace(int batch, int n_q_heads, int n_kv_heads, int head_dim,
                                             int max_rows) {
  if (batch <= 0 || n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads || max_rows <= 0 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  const int R = rows_per_item(n_q_heads / n_kv_heads, max_rows);
  return ws_desc() + ws_ml(R) + ws_o(R, head_dim);
}

extern "C" dkv_status dkv_paged_attend(const dkv_attend_t* a, void* stream) {
  if (!a) return refuse(DKV_ERR_INVALID_ARG, "null description");
  if (!a->q || !a->k_pool || !a->v_pool || !a->page_table || !a->kv_len || !a->out || !a->workspace)
    return refuse(DKV_ERR_INVALID_ARG, "null pointer argument");
  if (a->batch <= 0 || a->batch > DKV_MAX_STEP_BATCH)
    return refuse(DKV_ERR_INVALID_ARG, "batch outside [1, DKV_MAX_STEP_BATCH]");
  if (a->rows <= 0 || a->rows > (1 << 30) || a->max_rows <= 0)
    return refuse(DKV_ERR_INVALID_ARG, "rows outside [1, 2^30] or max_rows not positive");
  if (!a->row_start && (a->rows != a->batch || a->max_rows != 1))
    return refuse(DKV_ERR_INVALID_ARG, "without row_start there is one row per sequence");
  if (a->dtype != DKV_BF16 && a->dtype != DKV_FP16)
    return refuse(DKV_ERR_INVALID_ARG, "dtype is not bf16 (0) or fp16 (1)");
  if (a->head_dim != 64 && a->head_dim != 128)
    return refuse(DKV_ERR_UNSUPPORTED, "head_dim (supported: 64, 128)");
  if (a->n_kv_heads <= 0 || a->n_q_heads <= 0 || a->n_q_heads % a->n_kv_heads || a->n_q_heads > 65536)
    return refuse(DKV_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads");
  if (a->q_stride < (long long)a->n_q_heads * a->head_dim || a->q_stride % 8)
    return refuse(DKV_ERR_INVALID_ARG, "q_stride must hold the heads and be a multiple of 8");
  if (a->page_tokens < e2m1::kMinPageTokens || a->page_tokens > 4096 ||
      (a->page_tokens & (a->page_tokens - 1)))
    return refuse(DKV_ERR_INVALID_ARG, "page_tokens must be a power of two in [16, 4096]");
  if (a->num_pages <= 0 || (long long)a->num_pages * a->page_tokens > (1LL << 30))
    return refuse(DKV_ERR_INVALID_ARG, "num_pages must be positive, num_pages * page_tokens at most 2^30");
  if (a->max_pages <= 0 || (long long)a->max_pages * a->page_tokens > (1LL << 30))
    return refuse(DKV_ERR_INVALID_ARG, "max_pages must be positive, max_pages * page_tokens at most 2^30");
  if (!aligned16(a->q) || !aligned16(a->k_pool) || !aligned16(a->v_pool) || !aligned16(a->out) ||
      (reinterpret_cast<uintptr_t>(a->workspace) & 255))
    return refuse(DKV_ERR_INVALID_ARG, "tensors must start on 16-byte boundaries, the workspace on 256");
  if (!(fabsf(a->scale) <= FLT_MAX) || !(fabsf(a->v_scale) <= FLT_MAX))
    return refuse(DKV_ERR_INVALID_ARG, "scale and v_scale must be finite");
  const int G = a->n_q_heads / a->n_kv_heads, D = a->head_dim;
  if ((long long)a->rows * G > (1LL << 30))
    return refuse(DKV_ERR_INVALID_ARG, "rows times heads per KV head above 2^30");
  const int R = rows_per_item(G, a->max_rows);
  if (a->workspace_bytes < ws_desc() + ws_ml(R) + ws_o(R, D))
    return refuse(DKV_ERR_INVALID_ARG, "workspace smaller than dkv_paged_attend_workspace says");
  AttendParams p;
  char* w = static_cast<char*>(a->workspace);
  p.desc = reinterpret_cast<AttendDesc*>(w);
  p.done = reinterpret_cast<unsigned long long*>(w);
  p.tag = next_tag();
  p.part_ml = reinterpret_cast<float*>(w + ws_desc());
  p.part_o = reinterpret_cast<float*>(w + ws_desc() + ws_ml(R));
  p.q = a->q; p.k_pool = static_cast<const uint8_t*>(a->k_pool); p.v_pool = static_cast<const uint8_t*>(a->v_pool);
  p.table = a->page_table; p.kv_len = a->kv_len; p.row_start = a->row_start;
  p.out = a->out; p.lse = a->lse; p.q_stride = a->q_stride;
  p.B = a->batch; p.N = a->rows; p.Hq = a->n_q_heads; p.Hkv = a->n_kv_heads; p.G = G;
  p.num_pages = a->num_pages; p.max_pages = a->max_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a->page_tokens) ++p.page_shift;
  p.page_bytes = e2m1::page_bytes(D, a->page_tokens);
  p.scale_log2 = (float)(1.4426950408889634 * (double)a->scale);
  p.v_scale = a->v_scale;
  p.debug_withhold = g_debug_withhold;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->dtype == DKV_BF16)
    e = D == 64 ? launch_rows<__nv_bfloat16, 64>(p, R, s) : launch_rows<__nv_bfloat16, 128>(p, R, s);
  else
    e = D == 64 ? launch_rows<__half, 64>(p, R, s) : launch_rows<__half, 128>(p, R, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return refuse(DKV_ERR_CUDA, cudaGetErrorString(e));
  }
  return DKV_OK;
}

extern "C" int dkv_stream_capturing(void* stream) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &status) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return status != cudaStreamCaptureStatusNone;
}

extern "C" dkv_status dkv_paged_attend_debug_withhold(int enable) {
  g_debug_withhold = enable ? 1 : 0;
  return DKV_OK;
}
