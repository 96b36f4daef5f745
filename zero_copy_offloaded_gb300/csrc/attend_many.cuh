// dkv_paged_attend and dkv_block_attend, many rows: the same attention on the 5th-generation tensor cores.
//
// An item is (sequence, KV head, 256 query rows of that head's group, counted
// token-major over the G heads): two tiles of 128 rows whose Q stays in shared memory
// while the keys stream past in tiles of 128.  For each key tile
//   S = Q K^T  (tcgen05, fp32 in TMEM),  P = 2^(s - m) in fp16, written over S,
//   O += P V   (tcgen05, P from TMEM, O in TMEM through the whole item).
// All key tiles of all items form one line that is dealt to the CTAs in equal
// contiguous ranges; an item cut between CTAs leaves fp32 partials that
// attend_tc_join_kernel merges.
//
// Warps (512 threads, one CTA per SM): two softmax groups of four warps, one per Q tile,
// a thread to a row; six warps that turn codes into fp16 tiles (1.64 ms against 1.67 with four);
// one that issues every MMA; one that fetches the codes (bulk copies, a run of 16 keys
// each; of E4M3 a seventh that converts, each with its own loads).  The MMA order per key tile is P.V and the next Q.K^T of tile 0, then of tile 1,
// so one tile's softmax runs under the other tile's MMAs, and a finished Q.K^T also says
// that the P.V before it is finished: O may be rescaled then without a barrier of its own.
//
// A softmax thread takes its row's scores 32 at a time and writes the weights over columns
// that it has read.  The running reference m of a row is 7 (a weight of 2^7) below the maximum of
// the first 32 scores with a visible key; a later 32 whose weights sum to at most 60000 have none
// above that, which fp16 and the fp32 sums hold, so no maximum is taken.  Where they sum to more (or to
// infinity or NaN, as they do at the start) the row takes their maximum, less 7, as m and rescales what
// it has: the tile's earlier weights, l and O.  The largest weight is at least 2^7 throughout, so
// a weight keeps all of fp16's bits down to 2^-21 of the row's largest and counts down to 2^-32.  A lower
// m keeps more and moves more often: with scores of a standard deviation of 1, 2, 4 and 16 the chunk
// below takes 1.54, 1.54, 1.77 and 1.97 ms with 7, 1.54, 1.73, 1.82 and 2.04 with 10, and 1.54, 1.54, 1.59 and
// 1.88 with 0, where weights below 2^-25 are lost.
//
// What bounds it: 4 D flops per (row, key) on the tensor cores.  4096 rows of 32/8 heads of 128
// over 28672 keys and themselves (2.06 TFLOP) take 1.55 ms, 1327 TFLOP/s of 1912 measured.  A key
// tile's MMAs are 2048 cycles; what is left is the softmax's latency (about 2000 cycles for a
// tile's 128 x 128 per group, whose exponentials alone take 1024 of the special-function units),
// which two Q tiles hide only in part, and shared memory's bandwidth, which the MMAs' operands
// (192 KB a key tile) and the converted tiles (64 KB) share.  Tensor memory is full (S and O of two
// tiles), which rules out a third tile and a Q in tensor memory.  Exponentials as degree-4 polynomials
// on the FMA pipe do not help (five of sixteen: 2.20 ms against 1.86).
//
// E4M3: a tile's blocks have scales of their own, and the MMAs see one tile.  So each is split: what the append
// writes are powers of two, and the ratio of a block's scale to that of its piece's first block goes into the converted
// codes (fp16 holds a code times 2^-15 .. 2^7 exactly), while the first block's own multiplies the scores or the outputs.
// A ratio outside, or no power of two, stays with the block: the softmax of a tile that has one multiplies its scores
// by it, or adds log2 of it (V) to them and divides the sum.  With the blocks' scales in the softmax of every tile the
// chunk above takes 2.11 ms, this way 1.63 to 1.66 (1250 TFLOP/s).  The first is what a pool takes whose first block's scale
// lies 2^8 or more below the others' (2.11), or in which one V block of eight has a scale that is no power of two (2.10).
// Codes come from memory into registers: a ring of 8-bit tiles in shared memory leaves its bandwidth short (2.12 ms and more).
// The conversion and its bookkeeping are about a fifth of the instructions.
//
// Every item reads its keys, so a pool is read once for each 256 packed rows.  From HBM that is hidden;
// a pool in host memory crosses the link as often (4096 rows of 32/8 heads over 28672 keys: 10.8 ms, of E4M3 19.1).
#pragma once

#include <float.h>
#include <math.h>

#include <type_traits>

#include "attend.cuh"
#include "tc_common.cuh"

namespace dkv {

namespace {

constexpr int kRows = 128;             // rows of a Q tile, lanes of TMEM
constexpr int kKeys = 128;             // keys of a tile
constexpr int kConvert = 6;            // warps that turn codes into fp16 (E4M3, which needs no loader: one more)
constexpr int kThreads = (10 + kConvert) * 32;
constexpr int kReg = 128 * 128;        // a 128-row x 128-byte swizzled region
constexpr int kRaw = 3;                // E2M1: raw half tiles (K or V codes and scales) in flight
constexpr float kNone = -3e38f;        // m of a row that has seen no key
constexpr float kBias = 7.f;           // m below the maximum that it is taken from
// (32 weights whose maximum gave m sum to 2^12, 2^12.3 with the rounding of m for scores up to 2^21)
constexpr float kSumBound = 60000.f;

constexpr uint32_t kTmS = 0, kTmO = 256;  // S of tile t at 128 t, O at 256 + 128 t

template <Format F, int D>
struct Cfg {
  static constexpr int kCode = F == kE2M1 ? e2m1::code_bytes(D) : D;  // bytes of a key's codes
  static constexpr int DR = D / 64;                 // regions per row
  static constexpr int kTileB = DR * kReg;          // Q, K or V tile as fp16
  static constexpr int kCodes = kKeys * kCode;
  static constexpr int kHalf = kCodes + (F == kE2M1 ? kKeys * e2m1::scale_bytes(D) : 0);
  static constexpr int kOffQ = 0;                   // two Q tiles
  static constexpr int kOffK = 2 * kTileB;          // two K stages
  static constexpr int kOffV = 4 * kTileB;          // two V stages
  static constexpr int kOffRaw = 6 * kTileB;
  static constexpr int kEnd = kOffRaw + (F == kE2M1 ? kRaw * kHalf : 0);
  static constexpr int kSmem = kEnd + 1024;         // room to align the tiles to 1024
};

using Yes = std::true_type;
using No = std::false_type;

template <Format F>
struct Bars {
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_ready[2], s_full[2], p_ready[2], o_full[2], o_free[2];
  uint64_t drain;
  uint32_t tmem;
  volatile int abort;
  long long total, ctas, from, to;  // the line's length and CTAs; this CTA's range of it
  int start[3];      // sequence, KV head, query tile of the CTA's first key tile
  int start_tile;
  uint32_t raw_valid[4];  // bit i: keys 16 i .. of the tile are on a page, by tile & 3
  // by item & 3, for each block of V (E4M3: each dim): item + 1 above the complement of the first key of an
  // edge tile that has a NaN there (the maximum over keys is the first one's)
  static constexpr int kNan = F == kE2M1 ? 8 : 128;
  unsigned long long nan_key[4][kNan];
  uint32_t nan_item[4];   // E4M3: item + 1 of one that has any
  // E4M3.  By item & 3: the powers of two that K's and V's tiles of a piece are converted by.  By tile & 3, for each
  // run of 16 keys: 1 where a scale is left over, 2 where there is no page; what K's codes still have to be multiplied by (the
  // whole scale where it is left over, else the piece's power of two), log2 of what is left of V's and its inverse.  By
  // row: the scale of its scores but for K's.
  float2 ref[4];
  uint2 flags[4];
  float4 block[F == kE2M1 ? 1 : 4][8];
  float sl[F == kE2M1 ? 1 : 2 * kRows];
};

// Where a role is on the line: an item, and the key tiles [tile, end) of it here.
struct Piece {
  int b, h, qt, tile, end, tiles;
  int kv, n, row0, qtiles, last, minvis, maxvis;
};

template <Format F>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Bars<F>* bars) {
  if (mbar_wait_bounded(bar, parity, &bars->abort)) return true;
  bars->abort = 1;
  return false;
}
template <Format F>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Bars<F>* bars) {
  return __all_sync(~0u, wait(bar, parity, bars));
}

// The weights 2^(s sl - m) of 32 scores as fp16 pairs, and their fp32 sum.
__device__ __forceinline__ float weights(const uint32_t (&r)[32], uint32_t (&w)[16], float sl, float m) {
  const unsigned long long sl2 = tc::f2_pack(sl, sl), nm2 = tc::f2_pack(-m, -m);
  unsigned long long acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float p0, p1;
    tc::f2_unpack(tc::f2_fma(tc::f2_pack(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), sl2, nm2),
                  p0, p1);
    p0 = tc::ex2_approx(p0);
    p1 = tc::ex2_approx(p1);
    w[e] = tc::pack2<__half>(p0, p1);
    acc[e & 3] = tc::f2_add(acc[e & 3], tc::f2_pack(p0, p1));
  }
  float s8[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) tc::f2_unpack(acc[q], s8[2 * q], s8[2 * q + 1]);
  return ((s8[0] + s8[1]) + (s8[2] + s8[3])) + ((s8[4] + s8[5]) + (s8[6] + s8[7]));
}

// The same of E4M3's scores, whose two blocks of 16 have scales of their own: weights 2^(s sl + nm), and the blocks' sums.
__device__ __forceinline__ float2 block_weights(const uint32_t (&r)[32], uint32_t (&w)[16], float2 sl, float2 nm) {
  float2 sum;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float slh = h ? sl.y : sl.x, nmh = h ? nm.y : nm.x;
    const unsigned long long sl2 = tc::f2_pack(slh, slh), nm2 = tc::f2_pack(nmh, nmh);
    unsigned long long acc[2] = {0ull, 0ull};
#pragma unroll
    for (int e = 8 * h; e < 8 * h + 8; ++e) {
      float p0, p1;
      tc::f2_unpack(tc::f2_fma(tc::f2_pack(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), sl2, nm2),
                    p0, p1);
      p0 = tc::ex2_approx(p0);
      p1 = tc::ex2_approx(p1);
      w[e] = tc::pack2<__half>(p0, p1);
      acc[e & 1] = tc::f2_add(acc[e & 1], tc::f2_pack(p0, p1));
    }
    float a, b, c, d;
    tc::f2_unpack(acc[0], a, b);
    tc::f2_unpack(acc[1], c, d);
    (h ? sum.y : sum.x) = (a + b) + (c + d);
  }
  return sum;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A load that is issued where it stands.
__device__ __forceinline__ void load_now(uint4& w, const uint8_t* from) {
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(from));
}
__device__ __forceinline__ void load_now(float& x, const float* from) {
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(from));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ int swz(int row, int cc) {
  return (cc / 8) * kReg + row * 128 + (((cc % 8) ^ (row % 8)) * 16);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, int bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Key tiles of query tile qt (256 packed rows): up to the last row's last key.
__device__ __forceinline__ int tiles_of(int kv, int n, int G, int qt) {
  const int last = min((qt + 1) * 2 * kRows, n * G) - 1;
  return max(1, (max(0, kv - n + last / G + 1) + kKeys - 1) / kKeys);
}

__device__ __forceinline__ void enter_item(const AttendParams& p, Piece& c) {
  const int G = p.G;
  c.last = min((c.qt + 1) * 2 * kRows, c.n * G) - 1;
  c.minvis = max(0, c.kv - c.n + c.qt * 2 * kRows / G + 1);
  c.maxvis = max(0, c.kv - c.n + c.last / G + 1);
  c.tiles = max(1, (c.maxvis + kKeys - 1) / kKeys);
}

__device__ __forceinline__ void enter_seq(const AttendParams& p, Piece& c) {
  batch_entry(p, c.b, c.kv, c.row0, c.n);
  c.qtiles = (c.n * p.G + 2 * kRows - 1) / (2 * kRows);
}

// The CTA's next piece, `left` key tiles remaining from it on.
__device__ __forceinline__ void next_piece(const AttendParams& p, Piece& c, int left) {
  if (++c.qt >= c.qtiles) {
    c.qt = 0;
    if (++c.h >= p.Hkv) {
      c.h = 0;
      do {
        ++c.b;
        enter_seq(p, c);
      } while (c.n == 0);
    }
  }
  c.tile = 0;
  enter_item(p, c);
  c.end = min(c.tiles, left);
}

template <Format F, typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_tc_kernel(const AttendParams p) {
  using C = Cfg<F, D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars<F> bars_s;
  Bars<F>* bars = &bars_s;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&bars->raw_full[i], 1);
      mbar_init(&bars->raw_empty[i], kConvert);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->k_full[i], F == kE2M1 ? kConvert : kConvert + 1);
      mbar_init(&bars->k_empty[i], 1);
      mbar_init(&bars->v_full[i], F == kE2M1 ? kConvert : kConvert + 1);
      mbar_init(&bars->v_empty[i], 1);
      mbar_init(&bars->q_ready[i], 4);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_ready[i], 4);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->o_free[i], 4);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    p.desc[blockIdx.x].pieces = 0;
  }
  for (int i = threadIdx.x; i < 4 * Bars<F>::kNan; i += kThreads) bars->nan_key[i / Bars<F>::kNan][i % Bars<F>::kNan] = 0;
  if (threadIdx.x < 4) bars->nan_item[threadIdx.x] = 0;
  if (warp == 8 + kConvert) tc::tmem_alloc(&bars->tmem, 512);
  if (warp == 0) {
    // The length of the line, then the place on it where this CTA begins.
    // Sequence b adds Hkv times the key tiles of its query tiles.
    // key tiles of sequences [base, base + 32), one per lane
    auto lane_tiles = [&](int base) -> long long {
      int kv = 0, row, n = 0;
      if (base + lane < p.B) batch_entry(p, base + lane, kv, row, n);
      const int qtiles = (n * G + 2 * kRows - 1) / (2 * kRows);
      long long w = 0;
      const int seqs = min(32, p.B - base), most = __reduce_max_sync(~0u, qtiles);
      if (most <= 2 * seqs) {
        for (int qt = 0; qt < qtiles; ++qt) w += tiles_of(kv, n, G, qt);
      } else {  // few long ones: the warp together
        for (int i = 0; i < seqs; ++i) {
          const int kvi = __shfl_sync(~0u, kv, i), ni = __shfl_sync(~0u, n, i), qi = __shfl_sync(~0u, qtiles, i);
          long long wi = 0;
          for (int qt = lane; qt < qi; qt += 32) wi += tiles_of(kvi, ni, G, qt);
          for (int d = 16; d; d >>= 1) wi += __shfl_xor_sync(~0u, wi, d);
          if (lane == i) w = wi;
        }
      }
      return w;
    };
    auto scan = [&](long long v) {  // inclusive, over the warp
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(~0u, v, d);
        if (lane >= d) v += o;
      }
      return v;
    };
    long long total = 0, own = 0, sum = 0;
    for (int base = 0; base < p.B; base += 32) {
      own = lane_tiles(base);
      sum = scan(own);
      total += p.Hkv * __shfl_sync(~0u, sum, 31);
    }
    const long long ctas = min(total, (long long)gridDim.x);
    const bool busy = (long long)blockIdx.x < ctas;
    const long long from = busy ? total * blockIdx.x / ctas : 0, to = busy ? total * (blockIdx.x + 1) / ctas : 0;
    if (lane == 0) {
      bars->total = total;
      bars->ctas = ctas;
      bars->from = from;
      bars->to = to;
    }
    if (busy) {
      long long at = from, w = 0;
      int b = 0;
      for (int base = 0;; base += 32) {
        if (p.B > 32) {  // else they are at hand
          own = lane_tiles(base);
          sum = scan(own);
        }
        const long long whole = p.Hkv * __shfl_sync(~0u, sum, 31);
        if (at < whole) {
          const int i = __ffs(__ballot_sync(~0u, at < p.Hkv * sum)) - 1;
          b = base + i;
          w = __shfl_sync(~0u, own, i);
          at -= p.Hkv * (__shfl_sync(~0u, sum, i) - w);
          break;
        }
        at -= whole;
      }
      const int h = (int)(at / w);
      at -= h * w;
      int kv, row, n, qt = 0;
      batch_entry(p, b, kv, row, n);
      const int qtiles = (n * G + 2 * kRows - 1) / (2 * kRows);
      for (int base = 0;; base += 32) {
        const long long own = base + lane < qtiles ? tiles_of(kv, n, G, base + lane) : 0, sum = scan(own);
        const long long whole = __shfl_sync(~0u, sum, 31);
        if (at < whole) {
          const int i = __ffs(__ballot_sync(~0u, at < sum)) - 1;
          qt = base + i;
          at -= __shfl_sync(~0u, sum - own, i);
          break;
        }
        at -= whole;
      }
      if (lane == 0) {
        bars->start[0] = b;
        bars->start[1] = h;
        bars->start[2] = qt;
        bars->start_tile = (int)at;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  griddep_launch_dependents();
  const uint32_t tmem = bars->tmem;
  int left = (int)(bars->to - bars->from);  // key tiles of this CTA from the current piece on
  // Each warp's place on the line, in shared memory (its fields are read once an item or a tile:
  // the registers are the softmax's), moved by one lane.
  __shared__ Piece s_piece[kThreads / 32];
  Piece& c = s_piece[warp];
  if (left > 0 && lane == 0) {
    c.b = bars->start[0];
    c.h = bars->start[1];
    c.qt = bars->start[2];
    enter_seq(p, c);
    enter_item(p, c);
    c.tile = bars->start_tile;
    c.end = min(c.tiles, c.tile + left);
  }
  __syncwarp();
  auto advance = [&]() {  // to the next piece; false behind the last
    left -= c.end - c.tile;
    if (left <= 0) return false;
    __syncwarp();
    if (lane == 0) next_piece(p, c, left);
    __syncwarp();
    return true;
  };

  if (left > 0) {
    if (warp < 8) {
      // ================================================================ softmax
      const int t = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
      const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
      const uint32_t ts = tmem + kTmS + 128 * t + lane_off, to = tmem + kTmO + 128 * t + lane_off;
      uint8_t* qs = smem + C::kOffQ + t * C::kTileB;
      uint32_t tiles_done = 0, items_done = 0;  // of this Q tile
      uint32_t items = 0, all_tiles = 0;        // of the CTA
      bool dead = false;
      // Q of piece c's rows of this warp into shared memory, as fp16: D/8 lanes read a row, so
      // that a load covers whole lines; returns the scale of the scores of this thread's row
      auto load_q = [&]() {
        constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes per row, rows per load
        constexpr int STEP = 8;                     // loads in flight
        const int l = lane % LPR, sub = lane / LPR, base = c.qt * 2 * kRows + t * kRows + quarter * 32;
        const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // the scale's sign goes to q
        float unscale = 1.0f;
        int pr = base + sub, tok = pr / G, g = pr - tok * G;  // of the next load
        const T* q = static_cast<const T*>(p.q) + (size_t)c.row0 * p.q_stride + (size_t)c.h * G * D + l * 8;
#pragma unroll 1
        for (int i0 = 0; i0 < 32 / RPI; i0 += STEP) {
          uint4 w[STEP];
#pragma unroll
          for (int i = 0; i < STEP; ++i) {
            w[i] = make_uint4(0, 0, 0, 0);
            if (pr <= c.last) w[i] = __ldg(reinterpret_cast<const uint4*>(q + tok * p.q_stride + g * D));
            pr += RPI;
            g += RPI;
            while (g >= G) {
              g -= G;
              ++tok;
            }
          }
#pragma unroll
          for (int i = 0; i < STEP; ++i) {
            uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            if constexpr (DT<T>::code == DKV_BF16) {
              // the largest magnitude, as bits of two bf16 side by side
              uint32_t top2 = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) top2 = max_u16x2(top2, u[k] & 0x7FFF7FFFu);
#pragma unroll
              for (int d = 1; d < LPR; d <<= 1) top2 = max_u16x2(top2, __shfl_xor_sync(~0u, top2, d));
              const uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
              int e = (int)(top >> 7) - 127;  // the largest goes to [2^13, 2^14)
              e = top > 0 && top < 0x7F80u ? max(e, -113) : 13;
              const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
              // to the thread whose row this is
              const int back = __shfl_sync(~0u, e, (lane % RPI) * LPR);
              if (lane / RPI == i0 + i) unscale = __uint_as_float((uint32_t)(127 - 13 + back) << 23);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = DT<T>::to_f2(u[k]);
                u[k] = tc::pack2<__half>(f.x * up, f.y * up);
              }
            }
            *reinterpret_cast<uint4*>(qs + swz(quarter * 32 + (i0 + i) * RPI + sub, l)) =
                make_uint4(u[0] ^ sign, u[1] ^ sign, u[2] ^ sign, u[3] ^ sign);
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_ready[t]);
        // positive and finite, so that a masked -infinity stays one; E4M3's is so once it has K's scale
        return fminf(fmaxf(fabsf(p.scale_log2) * unscale, F == kE2M1 ? 1e-37f : 0.f), FLT_MAX);
      };
      auto positive = [](float x) {  // (a NaN stays one)
        float r;
        asm("max.NaN.f32 %0, %1, %2;\n\tmin.NaN.f32 %0, %0, %3;" : "=&f"(r) : "f"(x), "f"(1e-37f), "f"(FLT_MAX));
        return r;
      };
      auto active = [&]() { return c.last >= c.qt * 2 * kRows + t * kRows; };
      bool go = true;
      float sl = 1.f;
      if (active()) sl = load_q();
      while (go) {
        // what the epilogue needs of this piece
        const int pr = c.qt * 2 * kRows + t * kRows + row;
        const bool on = active(), mine = pr <= c.last;
        const int vis = mine ? max(0, c.kv - c.n + pr / G + 1) : 0;
        const bool starts = c.tile == 0, ends = c.end == c.tiles;
        const int h = c.h, row0 = c.row0, first = c.qt * 2 * kRows, last = c.last, b_tiles = c.tiles;
        const long long at = bars->to - left - c.tile;  // where the item begins on the line
        float m = mine ? kNone : 0.f, l = 0.f;
        if (on) {
          const int tile0 = c.tile, tile1 = c.end, minvis = c.minvis;
#pragma unroll 1
          for (int tile = tile0; tile < tile1; ++tile, ++tiles_done) {
            if (!dead && !warp_wait(&bars->s_full[t], tiles_done & 1, bars)) dead = true;
            if (dead) {
              l = __int_as_float(0x7fc00000);
              continue;
            }
            tc::fence_after_sync();
            const int k0 = tile * kKeys;
            uint32_t valid = 0xFFu;
            bool slow = false;  // E4M3: blocks have scales of their own left
            const uint32_t place = (all_tiles + tile - tile0) & 3;
            if constexpr (F == kE2M1) {
              valid = bars->raw_valid[place];
            } else {
              const uint2 f = bars->flags[place];
              if (f.x | f.y) {
                slow = (f.x | f.y) & 0x01010101u;
                // bit 1 of four bytes side by side
                valid ^= (f.x >> 1 & 0x01010101u) * 0x10204080u >> 28 | ((f.y >> 1 & 0x01010101u) * 0x10204080u >> 28) << 4;
              }
              if (tile == tile0) {
                bars->sl[t * kRows + row] = sl;  // this thread alone reads it
                sl = positive(sl * bars->ref[items & 3].x);
              }
            }
            const bool edge = k0 + kKeys > minvis || valid != 0xFFu;
            const int nvis = vis - k0;  // keys [0, nvis) of the tile are seen, where on a page
            auto chunk = [&](auto scaled, int pc, uint32_t (&r)[32]) {
              // the scales that are left to the chunk's two blocks, neutral where the row sees none of one
              float2 bsl, blv, brv;
              if constexpr (scaled) {
                const float4 b0 = bars->block[place][2 * pc], b1 = bars->block[place][2 * pc + 1];
                const bool see0 = nvis - pc * 32 > 0, see1 = nvis - pc * 32 > 16;
                // (not from `sl`, which is held inside fp32's range, and a ratio, which can leave it)
                const float raw = bars->sl[t * kRows + row];
                bsl = make_float2(see0 ? positive(raw * b0.x) : 1.f, see1 ? positive(raw * b1.x) : 1.f);
                blv = make_float2(see0 ? b0.y : 0.f, see1 ? b1.y : 0.f);
                brv = make_float2(see0 ? b0.z : 1.f, see1 ? b1.z : 1.f);
              }
              if (edge) {
                const int n = nvis - pc * 32;
                uint32_t see = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
                if (!((valid >> (2 * pc)) & 1)) see &= 0xFFFF0000u;
                if (!((valid >> (2 * pc)) & 2)) see &= 0x0000FFFFu;
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!((see >> k) & 1)) r[k] = 0xFF800000u;  // -infinity
              }
              uint32_t w[16];
              float sum;
#pragma unroll 1
              for (int again = 0;; ++again) {
                float part = 0.f;
                if constexpr (scaled) {
                  const float2 two = block_weights(r, w, bsl, make_float2(blv.x - m, blv.y - m));
                  sum = two.x + two.y;
                  part = fmaf(two.x, brv.x, two.y * brv.y);
                } else {
                  sum = weights(r, w, sl, m);
                }
                const bool raise = m == kNone || !(sum <= kSumBound);
                if (again) {  // above its own maximum: an infinity or a NaN is among the scores
                  if (!(sum <= kSumBound)) sum = __int_as_float(0x7fc00000);
                  else if (scaled) sum = part;
                  break;
                }
                if (!__any_sync(~0u, raise)) {
                  if (scaled) sum = part;
                  break;
                }
                float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 32; ++k) {  // scaled: a block to two of them
                  const int at = scaled ? (k >> 4) * 2 + (k & 1) : k & 3;
                  x[at] = fmaxf(x[at], __uint_as_float(r[k]));
                }
                float top;
                if constexpr (scaled)
                  top = fmaxf(fmaf(fmaxf(x[0], x[1]), bsl.x, blv.x - kBias), fmaf(fmaxf(x[2], x[3]), bsl.y, blv.y - kBias));
                else top = fmaf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), sl, -kBias);
                const float nm = raise ? fmaxf(m, top) : m;
                const float f = nm == m ? 1.0f : exp2f(m - nm);
                m = nm;
                l *= f;
                tc::tmem_wait_st();
#pragma unroll 1
                for (int q = 0; q < pc; ++q) {  // this tile's weights so far
                  uint32_t v[16];
                  tc::tmem_ld16(ts + q * 16, v);
                  tc::tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&v[e]));
                    v[e] = tc::pack2<__half>(y.x * f, y.y * f);
                  }
                  tc::tmem_st16(ts + q * 16, v);
                }
                if (tile != tile0) {  // O of the tiles before: their P.V finished before this S
#pragma unroll 1
                  for (int q = 0; q < D / 16; ++q) {
                    uint32_t v[16];
                    tc::tmem_ld16(to + q * 16, v);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                    tc::tmem_st16(to + q * 16, v);
                  }
                }
              }
              l += sum;
              tc::tmem_st16(ts + pc * 16, w);
            };
            auto all = [&](auto scaled) {
#pragma unroll 1
              for (int pc = 0; pc < kKeys / 32; ++pc) {
                uint32_t ra[32];
                tc::tmem_ld32(ts + pc * 32, ra);
                tc::tmem_wait_ld();
                chunk(scaled, pc, ra);
              }
            };
            if constexpr (F == kE4M3) {
              if (slow) all(Yes());
              else all(No());
            } else {
              all(No());
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_ready[t]);
          }
        }
        const uint32_t item = items++;
        all_tiles += c.end - c.tile;
        // Q of the next piece: every Q.K^T of this one has completed
        go = advance();
        float next_sl = 1.f;
        if (go && active()) next_sl = load_q();
        // ---- epilogue of the piece that just ended
        if (on) {
          const uint32_t slot = 2 * blockIdx.x + (starts ? 1 : 0);
          if (!dead && !warp_wait(&bars->o_full[t], items_done & 1, bars)) dead = true;
          ++items_done;
          tc::fence_after_sync();
          const bool whole = starts && ends;
          const float bad = __int_as_float(0x7fc00000);
          if (m == kNone && l == l) l = 0.f;  // no key of the piece is seen
          if (dead) l = bad;  // the wait for O may be the one that gave up: no lse beside outputs that are NaN
          const float vs = F == kE4M3 ? bars->ref[item & 3].y : p.v_scale;
          const float inv = dead ? bad : whole ? (l == 0.f ? 0.f : vs / l) : 1.0f;
          const int tok = pr / G;
          const size_t orow = (size_t)(row0 + tok) * p.Hq + h * G + (pr - tok * G);
          T* out = static_cast<T*>(p.out) + orow * D;
          // partials: [slot][D / 4][256 rows][4], so that a warp's rows lie side by side
          const bool any_nan = F == kE2M1 || bars->nan_item[item & 3] == item + 1;
          float4* po = reinterpret_cast<float4*>(p.part_o) + (size_t)slot * (D / 4) * kTcRows + t * kRows + row;
#pragma unroll 1
          for (int pc = 0; pc < D / 32; ++pc) {
            uint32_t r[32];
            if (!dead) {
              tc::tmem_ld32(to + pc * 32, r);
              tc::tmem_wait_ld();
            }
            float v[32];
            bool poison = false;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              // a row that saw no key of the piece holds what P = 0 gave, 0
              v[k] = dead ? bad : __uint_as_float(r[k]) * inv;
              if (any_nan && (F == kE4M3 || k % 16 == 0)) {
                const unsigned long long tag = bars->nan_key[item & 3][F == kE4M3 ? pc * 32 + k : pc * 2 + k / 16];
                poison = (uint32_t)(tag >> 32) == item + 1 && (int)~(uint32_t)tag < vis;
              }
              if (poison) v[k] = bad;
            }
            if (mine && whole) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = tc::pack2<T>(v[8 * k + 2 * e], v[8 * k + 2 * e + 1]);
                *reinterpret_cast<uint4*>(out + pc * 32 + 8 * k) = make_uint4(u[0], u[1], u[2], u[3]);
              }
            } else if (mine) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                po[(size_t)(pc * 8 + k) * kTcRows] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
            __syncwarp();
          }
          if (mine) {
            if (whole) {
              if (p.lse) p.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            } else {
              float2* ml = reinterpret_cast<float2*>(p.part_ml) + (size_t)slot * 2 * kRows + t * kRows + row;
              // E4M3: pieces have V scales of their own, which join the exponents: times O they could pass fp32
              *ml = F == kE4M3 ? make_float2(m + e4m3::log2_of(vs), l * (1.0f / vs)) : make_float2(m, l);
            }
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->o_free[t]);
          if (!ends && threadIdx.x == 0) {
            AttendDesc d;
            auto holder = [&](long long tile) { return (int)(((tile + 1) * bars->ctas - 1) / bars->total); };
            d.begin = holder(at);
            d.pieces = holder(at + b_tiles - 1) - d.begin + 1;
            d.row0 = row0; d.first = first; d.last = last; d.head0 = h * G;
            p.desc[blockIdx.x] = d;
          }
        }
        sl = next_sl;
      }
    } else if (F == kE4M3 && warp != 8 + kConvert) {
      // ================================================== E4M3: codes to fp16 tiles
      // Seven warps deal out a tile's groups of 512 bytes (4 keys of 128, 8 of 64).  Codes come from memory straight
      // into registers (staged in shared memory they would take another eighth of its bandwidth), V's while K's are
      // converted, the next tile's K's while V's are, and that tile's pages before.  Lane i looks after the place
      // and the scales of the warp's i-th group.  The loads are volatile: the compiler would move them to where
      // their values are needed.
      constexpr int kWarps = kConvert + 1, kRowsOf = 512 / D, kGroups = kKeys / kRowsOf, kIter = (kGroups + kWarps - 1) / kWarps;
      constexpr int PPR = D / 16;            // 16-byte pieces of a row
      constexpr uint32_t kNowhere = ~0u;
      const int cw = warp < 8 + kConvert ? warp - 8 : kConvert, mask = (1 << p.page_shift) - 1;
      auto group = [&](int i) { return i * kWarps + cw; };
      const bool mine = lane < kIter && group(lane) < kGroups;
      const int run = mine ? group(lane) * kRowsOf / 16 : 0;           // of this lane's group, in the tile
      const bool speaks = mine && group(lane) * kRowsOf % 16 == 0;      // for its run
      uint4 wk[kIter], wv[kIter];
      uint32_t at[kIter];        // the groups' runs of 16 keys in a pool
      float ks = 1.f, vs = 1.f;  // of the run's block
      float kref = 1.f, vref = 1.f, kback = 1.f, vback = 1.f;  // the piece's powers of two, and their inverses
      auto lookup = [&](int tile, int first) {  // the page of keys tile * 128 + first ..
        const int key = tile * kKeys + first;
        return key < c.kv ? __ldg(p.table + (size_t)c.b * p.max_pages + (key >> p.page_shift)) : -1;
      };
      // a run of 16 keys in a pool, of less than 4 TB (and its block's scale)
      auto place = [&](int tile, int first, int head, int page) {
        return (uint32_t)page < (uint32_t)p.num_pages
                   ? (((uint32_t)page * p.Hkv + head) << (p.page_shift - 4)) + (((tile * kKeys + first) & mask) >> 4) : kNowhere;
      };
      auto fetch = [&](const uint8_t* pool, uint4 (&w)[kIter]) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          w[i] = make_uint4(0, 0, 0, 0);
          if (at[i] != kNowhere)
            load_now(w[i], pool + (size_t)at[i] * (16 * D) + (group(i) * 512 & (16 * D - 1)) + lane * 16);
        }
      };
      auto fetch_keys = [&](uint32_t mine_at) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          at[i] = __shfl_sync(~0u, mine_at, i);
          if (group(i) >= kGroups) at[i] = kNowhere;
        }
        fetch(p.k_pool, wk);
      };
      auto fetch_scales = [&](uint32_t at, float& k, float& v) {
        k = v = 1.f;
        if (at != kNowhere) {
          load_now(k, p.k_scales + at);
          load_now(v, p.v_scales + at);
        }
      };
      int tile = c.tile, minvis = c.minvis, maxvis = c.maxvis;
      uint32_t item = 0;
      const int part = lane % PPR;
      // The pieces of a row's upper half write their words in the other order, so that the
      // eight lanes of one phase of a store hit eight different bank groups.
      const bool flip = PPR == 8 && part >= 4;
      const int to = swz(cw * kRowsOf + lane / PPR, part * 2 + flip);  // of the first word of group 0
      auto convert = [&](uint8_t* dst, uint4 (&w)[kIter], bool value, uint32_t factor) {
        if ((tile + 1) * kKeys > minvis) {
          // a key that nobody sees must weigh nothing; a NaN of V in a tile that some rows see in part is
          // dealt out by the epilogue
#pragma unroll
          for (int i = 0; i < kIter; ++i) {
            const int key = tile * kKeys + group(i) * kRowsOf + lane / PPR;
            if (key >= maxvis) {
              w[i] = make_uint4(0, 0, 0, 0);
            } else if (value) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t& wq = q == 0 ? w[i].x : q == 1 ? w[i].y : q == 2 ? w[i].z : w[i].w;
                const uint32_t nan = __vcmpeq4(wq & 0x7f7f7f7fu, 0x7f7f7f7fu);
                wq &= ~nan;
#pragma unroll 1
                for (int e = 0; nan && e < 4; ++e)
                  if ((nan >> (8 * e)) & 1) {
                    atomicMax(&bars->nan_key[item & 3][part * 16 + q * 4 + e],
                              ((unsigned long long)(item + 1) << 32) | ~(uint32_t)key);
                    bars->nan_item[item & 3] = item + 1;
                  }
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          if (group(i) >= kGroups) break;
          const uint32_t f = __shfl_sync(~0u, factor, i);
          const uint32_t x[4] = {flip ? w[i].z : w[i].x, flip ? w[i].w : w[i].y, flip ? w[i].x : w[i].z, flip ? w[i].y : w[i].w};
          // groups of four rows: every other of a warp's is four rows further in the swizzle
          uint8_t* row = dst + (D == 128 && (i & 1) ? to ^ 64 : to) + i * (kWarps * kRowsOf * 128);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint4*>(k ? dst + ((D == 128 && (i & 1) ? to ^ 64 : to) ^ 16) + i * (kWarps * kRowsOf * 128) : row) =
                make_uint4(hmul2(e4m3::lo_to_h2(x[2 * k]), f), hmul2(e4m3::hi_to_h2(x[2 * k]), f),
                           hmul2(e4m3::lo_to_h2(x[2 * k + 1]), f), hmul2(e4m3::hi_to_h2(x[2 * k + 1]), f));
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
      };
      // The factor that codes are multiplied by, as an fp16 pair, and what is left of the scale: all of scale / ref
      // where that is a power of two from 2^-15 to 2^7, which fp16 takes exactly (codes are multiples of 2^-9 up to 448).
      auto split = [](float ratio, float& rest) {
        const uint32_t bits = __float_as_uint(ratio);
        const int up = (int)(bits >> 23) - 127;
        const bool taken = !(bits & 0x807fffffu) && up >= -15 && up <= 7;
        rest = taken ? 1.f : ratio;
        return !taken ? 0x3c003c00u : up < -14 ? 0x02000200u : (uint32_t)(up + 15) * 0x04000400u;
      };
      uint32_t lead = place(tile, 0, c.h, lookup(tile, 0));  // the piece's first block
      uint32_t here = place(tile, run * 16, c.h, lookup(tile, run * 16));
      bool opens = true;  // the piece
      fetch_keys(here);
      fetch_scales(here, ks, vs);
#pragma unroll 1
      for (uint32_t j = 0;; ++j) {
        const uint32_t st = j & 1, parity = ((j >> 1) & 1) ^ 1;
        fetch(p.v_pool, wv);
        const bool opened = opens;
        if (opens) {
          float k, v;
          fetch_scales(lead, k, v);
          auto ref = [](float s, float& back) {  // its power of two, 1 for what is not positive and normal
            const uint32_t bits = __float_as_uint(s) - (1u << 23) < 0x7f000000u ? __float_as_uint(s) & 0x7f800000u : 127u << 23;
            back = __uint_as_float((254u << 23) - bits);
            return __uint_as_float(bits);
          };
          kref = ref(k, kback);
          vref = ref(v, vback);
        }
        // the tile after this one
        bool more = true;
        int next = tile + 1;
        opens = next >= c.end;
        int page = -1, first_page = -1;
        if (opens) {
          more = advance();
          next = c.tile;
          if (more) first_page = lookup(next, 0);
        }
        if (more) page = lookup(next, run * 16);
        float rest_k, rest_v;
        const bool held = here != kNowhere;
        const uint32_t fk = split(held ? ks * kback : 1.f, rest_k), fv = split(held ? vs * vback : 1.f, rest_v);
        if (!warp_wait(&bars->k_empty[st], parity, bars)) break;
        // the softmax has done with tile j - 3
        if (opened && lane == 0) bars->ref[item & 3] = make_float2(kref, vref);
        if (speaks) {
          const bool left_over = rest_k != 1.f || rest_v != 1.f;
          bars->block[j & 3][run] = left_over ? make_float4(rest_k != 1.f ? ks : kref, e4m3::log2_of(rest_v), __fdividef(1.0f, rest_v), 0.f)
                                              : make_float4(kref, 0.f, 1.f, 0.f);
          reinterpret_cast<uint8_t*>(&bars->flags[j & 3])[run] = left_over | (held ? 0 : 2);
        }
        convert(smem + C::kOffK + st * C::kTileB, wk, false, fk);
        if (lane == 0) mbar_arrive(&bars->k_full[st]);
        if (more) {
          here = place(next, run * 16, c.h, page);
          if (opens) lead = place(next, 0, c.h, first_page);
          fetch_keys(here);
          fetch_scales(here, ks, vs);
        }
        if (!warp_wait(&bars->v_empty[st], parity, bars)) break;
        convert(smem + C::kOffV + st * C::kTileB, wv, true, fv);
        if (lane == 0) mbar_arrive(&bars->v_full[st]);
        if (!more) break;
        if (opens) {
          ++item;
          minvis = c.minvis;
          maxvis = c.maxvis;
        }
        tile = next;
      }
    } else if (F == kE2M1 && warp < 8 + kConvert) {
      // ================================================== codes to fp16 tiles
      const int tid = threadIdx.x - 256;
      uint32_t half = 0, tiles = 0, items = 0;  // half tiles, tiles and items so far
      bool go = true;
      while (go && !bars->abort) {
        for (int tile = c.tile; tile < c.end && !bars->abort; ++tile, ++tiles) {
          const bool edge = (tile + 1) * kKeys > c.minvis;
          for (int kv = 0; kv < 2; ++kv, ++half) {
            const uint32_t rs = half % kRaw, st = tiles & 1;
            if (!warp_wait(&bars->raw_full[rs], (half / kRaw) & 1, bars)) break;
            if (!warp_wait(kv ? &bars->v_empty[st] : &bars->k_empty[st], ((tiles >> 1) & 1) ^ 1, bars)) break;
            const uint32_t valid = bars->raw_valid[tiles & 3];
            const uint8_t* raw = smem + C::kOffRaw + rs * C::kHalf;
            uint8_t* dst = smem + (kv ? C::kOffV : C::kOffK) + st * C::kTileB;
            constexpr int PPR = D / 32;  // 16-byte pieces of a row's codes: 32 elements each
#pragma unroll
            for (int i = 0; i < (kKeys * PPR + kConvert * 32 - 1) / (kConvert * 32); ++i) {
              const int ch = i * kConvert * 32 + tid, r = ch / PPR, part = ch % PPR;
              if (kKeys * PPR % (kConvert * 32) && ch >= kKeys * PPR) break;
              const uint4 w4 = *reinterpret_cast<const uint4*>(raw + ch * 16);
              uint32_t sb = *reinterpret_cast<const uint16_t*>(raw + C::kCodes + r * e2m1::scale_bytes(D) + part * 2);
              const bool ok = (valid >> (r >> 4)) & 1;
              if (edge || !ok) {
                // a key that nobody sees, or one without a page, must weigh nothing; a NaN of V
                // in a tile that some rows see in part is dealt out by the epilogue
                if (!ok || tile * kKeys + r >= c.maxvis) {
                  sb = 0;
                } else if (kv) {
#pragma unroll
                  for (int u = 0; u < 2; ++u)
                    if (((sb >> (8 * u)) & 0x7f) == 0x7f) {
                      sb &= ~(0xffu << (8 * u));
                      atomicMax(&bars->nan_key[items & 3][part * 2 + u],
                                ((unsigned long long)(items + 1) << 32) | ~(uint32_t)(tile * kKeys + r));
                    }
                }
              }
              const uint32_t s2 = e2m1::scales_to_h2(sb);
              const uint32_t sc[2] = {__byte_perm(s2, 0, 0x1010), __byte_perm(s2, 0, 0x3232)};
              // The pieces of a row's upper half write their words in another order, so that the
              // eight lanes of one phase of a store hit eight different bank groups.
              const bool flip = PPR == 4 && part >= 2;
              const uint32_t w[4] = {flip ? w4.z : w4.x, flip ? w4.w : w4.y, flip ? w4.x : w4.z, flip ? w4.y : w4.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t x[4];
                e2m1::codes_to_h2(w[k], x);
                const uint32_t sk = flip ? sc[1 - k / 2] : sc[k / 2];
                const __half2 s = *reinterpret_cast<const __half2*>(&sk);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x[e]), s);
                  x[e] = *reinterpret_cast<const uint32_t*>(&y);
                }
                *reinterpret_cast<uint4*>(dst + swz(r, part * 4 + (flip ? k ^ 2 : k))) =
                    make_uint4(x[0], x[1], x[2], x[3]);
              }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bars->raw_empty[rs]);
              mbar_arrive(kv ? &bars->v_full[st] : &bars->k_full[st]);
            }
          }
        }
        ++items;
        go = advance();
      }
    } else {
     if (warp == 8 + kConvert) {
      // ==================================================================== MMA
      {
        const uint32_t one = tc::elect_one();
        const uint32_t idesc_s = tc::idesc_f16(false, 128, kKeys, false, false);
        const uint32_t idesc_o = tc::idesc_f16(false, 128, D, false, true);
        const uint32_t base = smem_u32(smem);
        uint32_t np[2] = {0, 0}, nq[2] = {0, 0}, no[2] = {0, 0};  // phases waited for, per Q tile
        // Descriptors differ in their address field alone (16-byte units, low word): one add each.
        const uint64_t d0 = tc::sdesc_sw128(base, 16, 1024), dv0 = tc::sdesc_sw128(base + C::kOffV, kReg, 1024);
        auto qk = [&](int t, uint32_t st) {
          const uint64_t dq = d0 + ((C::kOffQ + t * C::kTileB) >> 4), dk = d0 + ((C::kOffK + st * C::kTileB) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = ((kk / 4) * kReg + (kk % 4) * 32) >> 4;
            tc::mma_ss_one(tmem + kTmS + 128 * t, dq + at, dk + at, idesc_s, kk != 0, one);
          }
          if (one) tc::mma_commit(&bars->s_full[t]);
        };
        auto pv = [&](int t, uint32_t st, bool fresh) {
          const uint64_t dv = dv0 + ((st * C::kTileB) >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            tc::mma_ts_one(tmem + kTmO + 128 * t, tmem + kTmS + 128 * t + kk * 8, dv + (kk * 2048 >> 4), idesc_o,
                           !(fresh && kk == 0), one);
        };
        // the piece of the current tile (cur) and of the next one (c runs one tile ahead)
        uint32_t j = 0;  // tile
        bool two = c.last >= c.qt * 2 * kRows + kRows, fresh = true, ok = true;
        int at = c.tile, end = c.end;
        ok = warp_wait(&bars->k_full[0], 0, bars);
        for (int t = 0; ok && t < 1 + two; ++t) {
          ok = warp_wait(&bars->q_ready[t], nq[t]++ & 1, bars);
          tc::fence_after_sync();
          if (ok) qk(t, 0);
        }
        if (ok) if (one) tc::mma_commit(&bars->k_empty[0]);
        while (ok) {
          const bool final_tile = at + 1 == end;  // of the piece
          bool more = true, next_two = two;
          if (final_tile) {
            more = advance();
            if (more) next_two = c.last >= c.qt * 2 * kRows + kRows;
          }
          const uint32_t st = j & 1, sn = (j + 1) & 1;
          ok = warp_wait(&bars->v_full[st], (j >> 1) & 1, bars);
          if (ok && more) ok = warp_wait(&bars->k_full[sn], ((j + 1) >> 1) & 1, bars);
          for (int t = 0; ok && t < 2; ++t) {
            if (t == 0 || two) {
              ok = warp_wait(&bars->p_ready[t], np[t]++ & 1, bars);
              // O of both tiles has been read out: neither group is more than an item behind.  (In a piece of
              // one key tile the second Q tile waits for the first's read-out of the same piece.)
              for (int u = 0; u < 2 && ok && fresh; ++u)
                if (no[u] > 0 && (u != 1 || t == 1 || !two)) ok = warp_wait(&bars->o_free[u], (no[u] - 1) & 1, bars);
              if (!ok) break;
              tc::fence_after_sync();
              pv(t, st, fresh);
              if (final_tile) {
                if (one && !p.debug_withhold) tc::mma_commit(&bars->o_full[t]);
                ++no[t];
              }
            }
            if (more && (t == 0 || next_two)) {
              if (final_tile) {
                ok = warp_wait(&bars->q_ready[t], nq[t]++ & 1, bars);
                if (!ok) break;
                tc::fence_after_sync();
              }
              qk(t, sn);
            }
          }
          if (!ok || !more) break;
          if (one) tc::mma_commit(&bars->v_empty[st]);
          if (one) tc::mma_commit(&bars->k_empty[sn]);
          ++j;
          fresh = final_tile;
          if (final_tile) {
            two = next_two;
            at = c.tile;
            end = c.end;
          } else {
            ++at;
          }
        }
        // nothing may be in flight when TMEM and shared memory go
        if (one) tc::mma_commit(&bars->drain);
        mbar_wait_drain(&bars->drain, 0);
      }
     } else if (F == kE2M1 && warp == 9 + kConvert) {
      // ================================================================= loader
      uint32_t half = 0, tiles = 0;
      const int sub = (lane >> 1) & 7, scales = lane & 1;
      const int bytes = 16 * (scales ? e2m1::scale_bytes(D) : e2m1::code_bytes(D));
      const int row_bytes = scales ? e2m1::scale_bytes(D) : e2m1::code_bytes(D);
      const size_t off = scales ? (size_t)e2m1::code_bytes(D) << p.page_shift : 0;
      const int dst = (scales ? C::kCodes : 0) + sub * bytes;
      auto find = [&](int b, int kv, int tile) {
        const int t = tile * kKeys + sub * 16;
        return lane < 16 && t < kv ? __ldg(p.table + (size_t)b * p.max_pages + (t >> p.page_shift)) : -1;
      };
      int page = find(c.b, c.kv, c.tile);
      bool go = true;
      while (go && !bars->abort) {
        for (int tile = c.tile; tile < c.end && !bars->abort; ++tile, ++tiles) {
          const bool ok = page >= 0 && page < p.num_pages;
          const uint32_t runs = __ballot_sync(~0u, ok && !scales);
          uint32_t valid = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) valid |= ((runs >> (2 * i)) & 1) << i;
          const size_t src = ((size_t)page * p.Hkv + c.h) * p.page_bytes + off +
                             (size_t)((tile * kKeys + sub * 16) & ((1 << p.page_shift) - 1)) * row_bytes;
          const int next = tile + 1 < c.end ? find(c.b, c.kv, tile + 1) : -1;
          for (int kv = 0; kv < 2; ++kv, ++half) {
            const uint32_t rs = half % kRaw;
            if (!warp_wait(&bars->raw_empty[rs], ((half / kRaw) & 1) ^ 1, bars)) break;
            if (lane == 0) {
              if (kv == 0) bars->raw_valid[tiles & 3] = valid;
              tc::mbar_expect_tx(&bars->raw_full[rs],
                                 __popc(valid) * 16 * (e2m1::code_bytes(D) + e2m1::scale_bytes(D)));
            }
            __syncwarp();
            if (ok)
              bulk_load(smem + C::kOffRaw + rs * C::kHalf + dst, (kv ? p.v_pool : p.k_pool) + src, bytes,
                        &bars->raw_full[rs]);
          }
          page = next;
        }
        go = advance();
        if (go) page = find(c.b, c.kv, c.tile);
      }
      if (bars->abort)
        for (int i = 0; i < kRaw; ++i) {
          mbar_wait_drain(&bars->raw_full[i], 0);
          mbar_wait_drain(&bars->raw_full[i], 1);
        }
     }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 8 + kConvert) tc::tmem_dealloc(tmem, 512);
}

// Joins the partials of each cut item.  An item in few pieces: block (c, y) takes 32 rows, a row
// to a lane, of the item that CTA c began, and each of its eight warps D / 8 outputs.  An item
// in more pieces than 32-output parts of a row: the blocks of the CTAs that it fills take a part
// each, their warps every eighth piece, and the eight meet in shared memory.  (One block a CTA's
// rows for all pieces: 82 us instead of 44 for 16 rows of one KV head over 131072 keys.)
template <typename T, int D>
__global__ void __launch_bounds__(256) attend_tc_join_kernel(const AttendParams p) {
  __shared__ float4 s_acc[8][8][32];  // [warp][four outputs][row]
  __shared__ float2 s_ml[8][32];
  griddep_wait();
  const AttendDesc d = p.desc[blockIdx.x];
  constexpr int kParts = D / 32;
  const int rank = (int)blockIdx.x - d.begin;  // among the CTAs that hold the item
  const bool many = d.pieces > kParts;
  if (d.pieces < 2 || rank >= (many ? kParts : 1) || d.first + (int)blockIdx.y * 32 > d.last) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y * 32 + lane, pr = d.first + r;
  // piece i lies in slot 2 (c + i), but the first in slot 2 c + 1
  auto slot = [&](int i) { return (size_t)(2 * (d.begin + i) + (i == 0)); };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  const float4* po = reinterpret_cast<const float4*>(p.part_o);
  float top = -INFINITY, sum = 0.f;
  auto add = [](float4& a, const float4& v, float f) {
    a.x = fmaf(v.x, f, a.x);
    a.y = fmaf(v.y, f, a.y);
    a.z = fmaf(v.z, f, a.z);
    a.w = fmaf(v.w, f, a.w);
  };
  auto store = [&]<int W>(const float4 (&a)[W], int q) {
    if (pr > d.last) return;
    float o[4 * W];
#pragma unroll
    for (int k = 0; k < W; ++k) o[4 * k] = a[k].x, o[4 * k + 1] = a[k].y, o[4 * k + 2] = a[k].z, o[4 * k + 3] = a[k].w;
    store_row<T, 4 * W>(p, d.row0 + pr / p.G, d.head0 + pr % p.G, D, 4 * q, o, top, sum, q == 0);
  };
  if (!many) {
    constexpr int W = D / 32;  // its outputs in fours
    float4 a[W] = {};
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      if (i < d.pieces) top = fmaxf(top, ml[slot(i) * kTcRows + r].x);
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      if (i >= d.pieces) break;
      const float2 x = ml[slot(i) * kTcRows + r];
      const float f = x.x == top ? 1.0f : exp2f(x.x - top);
      sum = fmaf(x.y, f, sum);
#pragma unroll
      for (int k = 0; k < W; ++k) add(a[k], po[(slot(i) * (D / 4) + warp * W + k) * kTcRows + r], f);
    }
    store(a, warp * W);
    return;
  }
  const int q0 = rank * 8;
  float t = -INFINITY, l = 0.f;
  for (int i = warp; i < d.pieces; i += 8) t = fmaxf(t, ml[slot(i) * kTcRows + r].x);
  {
    float4 a[8] = {};
    for (int i = warp; i < d.pieces; i += 8) {
      const float2 x = ml[slot(i) * kTcRows + r];
      const float f = x.x == t ? 1.0f : exp2f(x.x - t);
      l = fmaf(x.y, f, l);
#pragma unroll
      for (int q = 0; q < 8; ++q) add(a[q], po[(slot(i) * (D / 4) + q0 + q) * kTcRows + r], f);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) s_acc[warp][q][lane] = a[q];
    s_ml[warp][lane] = make_float2(t, l);
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = fmaxf(top, s_ml[w][lane].x);
  float4 a[1] = {};
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float2 x = s_ml[w][lane];
    const float f = x.x == top ? 1.0f : exp2f(x.x - top);
    sum = fmaf(x.y, f, sum);
    add(a[0], s_acc[w][warp][lane], f);
  }
  store(a, q0 + warp);
}

}  // namespace

template <Format F, typename T, int D>
cudaError_t launch_attend_many(const AttendParams& p, int grid, cudaStream_t s) {
  auto k = attend_tc_kernel<F, T, D>;
  static PerDevice smem_set;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = smem_set(dev, [k] { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<F, D>::kSmem); });
  if (e != cudaSuccess) return e;
  k<<<grid, kThreads, Cfg<F, D>::kSmem, s>>>(p);
  const cudaError_t l = cudaGetLastError();
  if (l != cudaSuccess) return l;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, kTcRows / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_tc_join_kernel<T, D>, p);
}

}  // namespace dkv
