// The 4-bit paged attention for many query rows, on the 5th-generation tensor cores.
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
// each).  The MMA order per key tile is P.V and the next Q.K^T of tile 0, then of tile 1,
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
// Every item reads its keys, so a pool is read once for each 256 packed rows.  From HBM that is hidden;
// a pool in host memory crosses the link as often (4096 rows of 32/8 heads over 28672 keys: 10.8 ms).
#include <float.h>
#include <math.h>

#include <type_traits>

#include "attend_e2m1.cuh"
#include "tc_common.cuh"

namespace dkv {

namespace {

constexpr int kRows = 128;             // rows of a Q tile, lanes of TMEM
constexpr int kKeys = 128;             // keys of a tile
constexpr int kConvert = 6;            // warps that turn codes into fp16
constexpr int kThreads = (10 + kConvert) * 32;
constexpr int kReg = 128 * 128;        // a 128-row x 128-byte swizzled region
constexpr int kRaw = 3;                // raw half tiles (K or V codes and scales) in flight
constexpr float kNone = -3e38f;        // m of a row that has seen no key
constexpr float kBias = 7.f;           // m below the maximum that it is taken from
// (32 weights whose maximum gave m sum to 2^12, 2^12.3 with the rounding of m for scores up to 2^21)
constexpr float kSumBound = 60000.f;

constexpr uint32_t kTmS = 0, kTmO = 256;  // S of tile t at 128 t, O at 256 + 128 t

template <int D>
struct Cfg {
  static constexpr int DR = D / 64;                 // regions per row
  static constexpr int kTileB = DR * kReg;          // Q, K or V tile as fp16
  static constexpr int kCodes = kKeys * e2m1::code_bytes(D);
  static constexpr int kHalf = kCodes + kKeys * e2m1::scale_bytes(D);
  static constexpr int kOffQ = 0;                   // two Q tiles
  static constexpr int kOffK = 2 * kTileB;          // two K stages
  static constexpr int kOffV = 4 * kTileB;          // two V stages
  static constexpr int kOffRaw = 6 * kTileB;
  static constexpr int kEnd = kOffRaw + kRaw * kHalf;
  static constexpr int kSmem = kEnd + 1024;         // room to align the tiles to 1024
};

using Yes = std::true_type;
using No = std::false_type;

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
  // by item & 3, for each block of V: item + 1 above the complement of the first key of an
  // edge tile that has a NaN there (the maximum over keys is the first one's)
  unsigned long long nan_key[4][8];
};

// Where a role is on the line: an item, and the key tiles [tile, end) of it here.
struct Piece {
  int b, h, qt, tile, end, tiles;
  int kv, n, row0, qtiles, last, minvis, maxvis;
};

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Bars* bars) {
  if (mbar_wait_bounded(bar, parity, &bars->abort)) return true;
  bars->abort = 1;
  return false;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Bars* bars) {
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

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_tc_kernel(const AttendParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars_s;
  Bars* bars = &bars_s;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&bars->raw_full[i], 1);
      mbar_init(&bars->raw_empty[i], kConvert);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->k_full[i], kConvert);
      mbar_init(&bars->k_empty[i], 1);
      mbar_init(&bars->v_full[i], kConvert);
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
  if (threadIdx.x < 32) bars->nan_key[threadIdx.x / 8][threadIdx.x % 8] = 0;
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
        return fminf(fmaxf(fabsf(p.scale_log2) * unscale, 1e-37f), FLT_MAX);
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
            const uint32_t valid = bars->raw_valid[(all_tiles + tile - tile0) & 3];
            const bool edge = k0 + kKeys > minvis || valid != 0xFFu;
            const int nvis = vis - k0;  // keys [0, nvis) of the tile are seen, where on a page
            auto chunk = [&](int pc, uint32_t (&r)[32]) {
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
                sum = weights(r, w, sl, m);
                const bool raise = m == kNone || !(sum <= kSumBound);
                if (again) {  // above its own maximum: an infinity or a NaN is among the scores
                  if (!(sum <= kSumBound)) sum = __int_as_float(0x7fc00000);
                  break;
                }
                if (!__any_sync(~0u, raise)) break;
                float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k & 3] = fmaxf(x[k & 3], __uint_as_float(r[k]));
                const float nm = raise ? fmaxf(m, fmaf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), sl, -kBias)) : m;
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
#pragma unroll 1
            for (int pc = 0; pc < kKeys / 32; ++pc) {
              uint32_t ra[32];
              tc::tmem_ld32(ts + pc * 32, ra);
              tc::tmem_wait_ld();
              chunk(pc, ra);
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
          const float inv = dead ? bad : whole ? (l == 0.f ? 0.f : p.v_scale / l) : 1.0f;
          const int tok = pr / G;
          const size_t orow = (size_t)(row0 + tok) * p.Hq + h * G + (pr - tok * G);
          T* out = static_cast<T*>(p.out) + orow * D;
          // partials: [slot][D / 4][256 rows][4], so that a warp's rows lie side by side
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
              if (k % 16 == 0) {
                const unsigned long long tag = bars->nan_key[item & 3][pc * 2 + k / 16];
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
              *ml = make_float2(m, l);
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
    } else if (warp < 8 + kConvert) {
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
     } else if (warp == 9 + kConvert) {
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

template <typename T, int D>
cudaError_t launch_attend_tc(const AttendParams& p, int grid, cudaStream_t s) {
  auto k = attend_tc_kernel<T, D>;
  static PerDevice smem_set;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = smem_set(dev, [k] { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem); });
  if (e != cudaSuccess) return e;
  k<<<grid, kThreads, Cfg<D>::kSmem, s>>>(p);
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
template cudaError_t launch_attend_tc<__nv_bfloat16, 64>(const AttendParams&, int, cudaStream_t);
template cudaError_t launch_attend_tc<__nv_bfloat16, 128>(const AttendParams&, int, cudaStream_t);
template cudaError_t launch_attend_tc<__half, 64>(const AttendParams&, int, cudaStream_t);
template cudaError_t launch_attend_tc<__half, 128>(const AttendParams&, int, cudaStream_t);

}  // namespace dkv
