// dkv_block_append: per-head RMS norm of queries and keys, rotation to their positions, and the append of keys and
// values to a paged cache of E4M3 codes with one scale for each block of 16 tokens of a head.
//
// Norm and rotation are dkv_qkv_append's, operation by operation.  For the rows y that a call writes to one block:
//   need = the smallest power of two with max|y| <= 448 need,  s = max(need, the block's scale so far)
// where a block whose first row is among them has none so far.  Where s is above it the rows already there
// are brought to the new scale, code <- e4m3(code * old / s); new rows are e4m3(y / s).  Scales are powers of two so that
// the quotients are exact: a code rounds once, and again only in E4M3's subnormals when its block's scale grows.
//
// One to four warps take the rows of one block and head together (16 at most, all loads in flight, their fp32 values in
// registers until the largest of them is known), so that the scale needs no second pass and no atomics; blocks that a
// call gives few rows go to a warp of several heads.  The rows of a block lie within 16 consecutive rows of the call; a
// warp looks at 16 tokens and takes the blocks whose rows begin there.
//
// What bounds it: 23 KB a row of 32/8 heads of 128, 4096 of them 14 us at the measured copy rate; they take 26.8, of which
// queries alone 17.5, keys and values alone 17.1.  Neither memory nor a pipe is full: the warps wait for chains of fp32 (the keys'
// exact sums of squares, the values that have to live until the block's largest is known) and for instructions, of
// which the unrolled rows have many.  Sums, norms and rotations take two elements an instruction where they can.
#include "append.cuh"
#include "append_geometry.h"
#include "e4m3.cuh"

namespace {

using namespace dkv;

constexpr int kThreads = kAppendThreads, kWarps = kThreads / 32;
static_assert(kWarps == kAppendWarps && kLook == kWarps * e4m3::kBlock && kIterQ == kAppendIterQ, "append_geometry.h");

// Blocks that a call gives at most kShort rows go to warps that take one block of several heads (append_tokens), the others to
// warps that take all of a block's rows (append_blocks).  Which is which is seen on the device, so both are launched.
// 64 sequences' five rows each: 7.8 us with 6, 16.8 with 4; 512 single rows 9.1 us so, 55 by block; one sequence's 1024
// rows 10.3 us by block, 27 by token.  Four rows of 1024 sequences, 39.8 us for 14 us of memory traffic: append_few goes over the
// rows of a block twice, norm and rotation included, with one of them in flight.
constexpr int kShort = 6;

struct BlockParams {
  AppendParams a;
  float* k_scales;
  float* v_scales;
  AppendGeometry g;
};

// The block of a slot; -1: padding.
__device__ __forceinline__ int block_of(const AppendParams& p, int slot) {
  return slot < 0 || slot >= p.slots ? -1 : slot / e4m3::kBlock;
}

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}
// NaN for what is not finite (an infinity too: E4M3 has none), and the largest size of what is.
template <int N>
__device__ __forceinline__ float odd_values(float (&x)[N]) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (fabsf(x[e]) <= FLT_MAX) top = fmaxf(top, fabsf(x[e]));
    else x[e] = __int_as_float(0x7fc00000);
  }
  return top;
}

// A lane's codes of a row, and what they stand for.
template <typename T, int D, bool PAIRED>
__device__ __forceinline__ void store_row(uint8_t* to, T* out, uint2 c, float s, int off0, int off1, int l) {
  if constexpr (PAIRED) {
    *reinterpret_cast<uint32_t*>(to + off0) = c.x;
    *reinterpret_cast<uint32_t*>(to + off1) = c.y;
  } else {
    *reinterpret_cast<uint2*>(to + l * 8) = c;
  }
  if (!out) return;
  const uint32_t h2[4] = {e4m3::lo_to_h2(c.x), e4m3::hi_to_h2(c.x), e4m3::lo_to_h2(c.y), e4m3::hi_to_h2(c.y)};
  float y[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2[e]));
    y[2 * e] = __fmul_rn(f.x, s);
    y[2 * e + 1] = __fmul_rn(f.y, s);
  }
  *reinterpret_cast<uint2*>(out + off0) = pack4<T>(y);
  *reinterpret_cast<uint2*>(out + off1) = pack4<T>(y + 4);
}

// Warps that share a run.
template <int D>
constexpr int kShare = append_share(D);

// The rows t0 .. t0 + 15 of heads h0 .. h1 - 1 that lie in block `block` of the pool, row t0 among them.  The warps that
// share it come here together; `turn` alternates between the heads that they take.  (Loading the next head's rows
// meanwhile costs registers that are not there: 4096 rows 33 us.)
template <typename T, int D, bool INTER, int KIND>
__device__ __forceinline__ void append_run(const BlockParams& bp, int h0, int h1, int t0, int block, uint32_t* s_top, int& turn) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, SH = kShare<D>, ITER = e4m3::kBlock / RPW / SH;
  constexpr bool PAIRED = KIND == kKey && !INTER;  // a lane holds both partners of its pairs
  const AppendParams& p = bp.a;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR, part = (threadIdx.x >> 5) % SH;
  const float nan = __int_as_float(0x7fc00000);
  const int half = p.rot / 2;
  const bool in_rot = KIND == kKey && p.pos && l * 8 < p.rot;
  const int off0 = PAIRED && in_rot ? 4 * l : 8 * l, off1 = PAIRED && in_rot ? half + 4 * l : 8 * l + 4;
  auto row_of = [&](int i) { return (i * SH + part) * RPW + sub; };
  // lane r: slot and position of row t0 + r; bit r: it lies in the block
  const bool in = lane < e4m3::kBlock && t0 + lane < p.N;
  const int slot_l = in ? __ldg(p.slot + t0 + lane) : -1, pos_l = KIND == kKey && p.pos && in ? __ldg(p.pos + t0 + lane) : 0;
  const uint32_t members = __ballot_sync(~0u, in && block_of(p, slot_l) == block);
  if (__popc(members) <= kShort) return;
  auto member = [&](int i) { return (members >> row_of(i)) & 1; };
  // the block's rows that this run writes
  const uint32_t rows = __reduce_or_sync(~0u, (members >> lane) & 1 ? 1u << (slot_l & (e4m3::kBlock - 1)) : 0u);
  const int per_page = 1 << (p.page_shift - 4), page = block >> (p.page_shift - 4);
  const size_t first_head = (size_t)page * p.Hkv + h0;
  float* scale = (KIND == kKey ? bp.k_scales : bp.v_scales) + first_head * per_page + (block & (per_page - 1));
  uint8_t* codes = (KIND == kKey ? p.k_pool : p.v_pool) +
                   ((first_head << p.page_shift) + (block & (per_page - 1)) * e4m3::kBlock) * D;
  T* out = static_cast<T*>(KIND == kKey ? p.k_out : p.v_out);
  if (out) out += ((size_t)t0 * p.Hkv + h0) * D;
  const long long stride = KIND == kKey ? p.ks : p.vs;
  const T* src = static_cast<const T*>(KIND == kKey ? p.k : p.v) + (size_t)t0 * stride + (size_t)h0 * D + row_of(0) * stride;
  uint2 w[ITER][2];
  float old;
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const T* row = src + i * (SH * RPW) * stride;
      w[i][0] = w[i][1] = make_uint2(0, 0);
      if (member(i)) {
        if constexpr (PAIRED) {
          w[i][0] = *reinterpret_cast<const uint2*>(row + off0);
          w[i][1] = *reinterpret_cast<const uint2*>(row + off1);
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(row + l * 8);
          w[i][0] = make_uint2(u.x, u.y);
          w[i][1] = make_uint2(u.z, u.w);
        }
      }
    }
    old = *scale;
  };

  const T* gam = static_cast<const T*>(KIND == kKey ? p.k_gamma : nullptr);
  float g[8];
  if (KIND == kKey && gam) {
    unpack4<T>(__ldg(reinterpret_cast<const uint2*>(gam + off0)), g);
    unpack4<T>(__ldg(reinterpret_cast<const uint2*>(gam + off1)), g + 4);
  }
  // the cosines and sines of a lane's four pairs, a row ahead; whether the row is outside their table
  float4 ahead[2];
  bool ahead_far = false;
  auto angles = [&](int i) {
    const int pos = __shfl_sync(~0u, pos_l, row_of(i));
    ahead_far = (pos < 0 || pos >= p.max_pos) && member(i);
    ahead[0] = make_float4(1.f, 1.f, 1.f, 1.f);
    ahead[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (member(i) && !ahead_far && in_rot) {
      const float* from = p.cos_sin + (size_t)pos * p.rot + 4 * l;
      ahead[0] = __ldg(reinterpret_cast<const float4*>(from));
      ahead[1] = __ldg(reinterpret_cast<const float4*>(from + half));
    }
  };
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    load();
    if (KIND == kKey && p.pos) angles(0);
    float x[ITER][8], most = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      unpack4<T>(w[i][0], x[i]);
      unpack4<T>(w[i][1], x[i] + 4);
    }
    const float had = (rows & 1) || !(old > 0.f && old <= FLT_MAX) ? 0.f : old;  // a fresh block has no scale
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (KIND == kKey) {
        const float c[4] = {ahead[0].x, ahead[0].y, ahead[0].z, ahead[0].w};
        const float s[4] = {ahead[1].x, ahead[1].y, ahead[1].z, ahead[1].w};
        const bool far = ahead_far;
        if (p.pos && i + 1 < ITER) angles(i + 1);
        if (gam) norm_row<LPR, kExactPairs>(x[i], g, p.eps);
        if (in_rot) rotate<INTER>(x[i], c, s);
        if (far) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][e] = nan;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) most = max_abs(most, x[i][e], x[i][e + 1]);
    }
    if (__any_sync(~0u, !(most <= FLT_MAX))) {
      most = 0.f;
#pragma unroll
      for (int i = 0; i < ITER; ++i) most = fmaxf(most, odd_values(x[i]));
    }
    uint32_t top = __float_as_uint(most);
    top = __reduce_max_sync(~0u, top);
    if constexpr (SH > 1) {  // of all of them, who also have read `old` behind this
      const int team = threadIdx.x / (32 * SH);
      uint32_t* mine = s_top + SH * (team * 2 + turn);
      if (lane == 0) mine[part] = top;
      named_bar_sync(1 + team, 32 * SH);
#pragma unroll
      for (int i = 0; i < SH; ++i) top = max(top, mine[i]);
    }
    const float need = e4m3::scale_for(top), s = fmaxf(need, had);
    if (s > had && had > 0.f) {  // the rows already there, to the new scale
      const float f = __fdiv_rn(had, s);
#pragma unroll
      for (int i = 0; i < D / 32 / SH; ++i) {
        const int piece = (i * SH + part) * 32 + lane;
        if ((rows >> (piece * 16 / D)) & 1) continue;
        uint4* to = reinterpret_cast<uint4*>(codes) + piece;
        const uint4 v = *to;
        uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t a2 = e4m3::lo_to_h2(u[q]), b2 = e4m3::hi_to_h2(u[q]);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&a2));
          const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&b2));
          u[q] = e4m3::to_codes(__fmul_rn(a.x, f), __fmul_rn(a.y, f), __fmul_rn(b.x, f), __fmul_rn(b.y, f));
        }
        *to = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
    if (lane == 0 && part == 0 && s != had) *scale = s;
    // a power of two, but for a scale that something else has written
    float inv = __frcp_rn(s);
    if (__float_as_uint(s) & 0x7fffffu) {
      inv = 1.f;
#pragma unroll
      for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = __fdiv_rn(x[i][e], s);
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int slot = __shfl_sync(~0u, slot_l, row_of(i));
      if (!member(i)) continue;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(x[i][e], inv);
      const uint2 c = make_uint2(e4m3::to_codes(y[0], y[1], y[2], y[3]), e4m3::to_codes(y[4], y[5], y[6], y[7]));
      store_row<T, D, PAIRED>(codes + (slot & (e4m3::kBlock - 1)) * D,
                              out ? out + (size_t)row_of(i) * p.Hkv * D : nullptr, c, s, off0, off1, l);
    }
    scale += per_page;
    src += D;
    codes += (size_t)D << p.page_shift;
    if (out) out += D;
    turn ^= 1;
  }
}

// The rows of the block that begins at token t, where they are kShort at most, of as many heads from h0 on (below h1) as a warp has
// groups of D / 8 lanes, one to a group: it goes over the rows twice (once for one row).
template <typename T, int D, bool INTER, int KIND>
__device__ __forceinline__ void append_few(const BlockParams& bp, int t, int h0, int h1) {
  constexpr int LPR = D / 8;
  constexpr bool PAIRED = KIND == kKey && !INTER;
  const AppendParams& p = bp.a;
  const int lane = threadIdx.x & 31, l = lane % LPR, h = h0 + lane / LPR;
  const bool active = h < h1;
  const float nan = __int_as_float(0x7fc00000);
  const int half = p.rot / 2;
  const bool in_rot = KIND == kKey && p.pos && l * 8 < p.rot;
  const int off0 = PAIRED && in_rot ? 4 * l : 8 * l, off1 = PAIRED && in_rot ? half + 4 * l : 8 * l + 4;
  const T* gam = static_cast<const T*>(KIND == kKey ? p.k_gamma : nullptr);
  const long long stride = KIND == kKey ? p.ks : p.vs;
  const int per_page = 1 << (p.page_shift - 4);
  T* out = static_cast<T*>(KIND == kKey ? p.k_out : p.v_out);
  float g[8];
  if (KIND == kKey && gam) {
    unpack4<T>(__ldg(reinterpret_cast<const uint2*>(gam + off0)), g);
    unpack4<T>(__ldg(reinterpret_cast<const uint2*>(gam + off1)), g + 4);
  }
  // lane i: slot and position of token t + i, from 16 on of token t - 31 + i
  const int token = lane < e4m3::kBlock ? t + lane : t - 31 + lane;
  const bool in = token >= 0 && token < p.N && lane < 31;
  const int slot_l = in ? __ldg(p.slot + token) : -1, pos_l = KIND == kKey && p.pos && in ? __ldg(p.pos + token) : 0;
  const T* src = static_cast<const T*>(KIND == kKey ? p.k : p.v) + (size_t)t * stride + (size_t)h * D;
  uint2 w[2];
  auto load = [&](int r) {
    w[0] = w[1] = make_uint2(0, 0);
    if (!active) return;
    const T* row = src + (size_t)r * stride;
    if constexpr (PAIRED) {
      w[0] = *reinterpret_cast<const uint2*>(row + off0);
      w[1] = *reinterpret_cast<const uint2*>(row + off1);
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(row + l * 8);
      w[0] = make_uint2(v.x, v.y);
      w[1] = make_uint2(v.z, v.w);
    }
  };
  load(0);
  const int block = block_of(p, __shfl_sync(~0u, slot_l, 0));
  const uint32_t same = __ballot_sync(~0u, in && block_of(p, slot_l) == block);
  // padding, or the block's rows began before, or there are too many
  if (block < 0 || same >> e4m3::kBlock || __popc(same) > kShort) return;
  const uint32_t rows = __reduce_or_sync(~0u, (same >> lane) & 1 ? 1u << (slot_l & (e4m3::kBlock - 1)) : 0u);
  const int page = block >> (p.page_shift - 4);
  const size_t head = (size_t)page * p.Hkv + (active ? h : 0);
  float* scale = (KIND == kKey ? bp.k_scales : bp.v_scales) + head * per_page + (block & (per_page - 1));
  uint8_t* codes = (KIND == kKey ? p.k_pool : p.v_pool) +
                   ((head << p.page_shift) + (block & (per_page - 1)) * e4m3::kBlock) * D;
  float old = *scale;
  if ((rows & 1) || !(old > 0.f && old <= FLT_MAX)) old = 0.f;
  float x[8];
  // Row r from w, and the row after it on its way into w.
  auto row = [&](int r, int next) {
    unpack4<T>(w[0], x);
    unpack4<T>(w[1], x + 4);
    const int pos = __shfl_sync(~0u, pos_l, r);
    const bool far = KIND == kKey && p.pos && (pos < 0 || pos >= p.max_pos);
    float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in_rot && !far) {
      const float* from = p.cos_sin + (size_t)pos * p.rot + 4 * l;
      c4 = __ldg(reinterpret_cast<const float4*>(from));
      s4 = __ldg(reinterpret_cast<const float4*>(from + half));
    }
    if (next >= 0) load(next);
    if constexpr (KIND == kKey) {
      if (gam) norm_row<LPR, kExactPairs>(x, g, p.eps);
      if (in_rot) {
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
        rotate<INTER>(x, c, s);
      }
    }
    if (far) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = nan;
    }
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) most = max_abs(most, x[e], x[e + 1]);
    if (!(most <= FLT_MAX)) most = odd_values(x);
    return __float_as_uint(most);
  };
  auto next_row = [&](int r) { return __ffs(same >> r >> 1) + r; };          // r: none (31 - clz below: -1)
  auto previous_row = [&](int r) { return 31 - __clz(same & ((1u << r) - 1)); };
  const int last = 31 - __clz(same);
  uint32_t top = 0;
#pragma unroll 1
  for (int r = 0;; r = next_row(r)) {
    top = max(top, row(r, r < last ? next_row(r) : previous_row(r)));
    if (r == last) break;
  }
#pragma unroll
  for (int d = 1; d < LPR; d <<= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
  const float s = fmaxf(e4m3::scale_for(top), old);
  if (active && s > old && old > 0.f) {  // the rows already there, to the new scale
    const float f = __fdiv_rn(old, s);
#pragma unroll 1
    for (int piece = l; piece < D; piece += LPR) {
      if ((rows >> (piece * 16 / D)) & 1) continue;
      uint32_t u4[4];
      uint4* to = reinterpret_cast<uint4*>(codes) + piece;
      *reinterpret_cast<uint4*>(u4) = *to;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t a2 = e4m3::lo_to_h2(u4[q]), b2 = e4m3::hi_to_h2(u4[q]);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&a2));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&b2));
        u4[q] = e4m3::to_codes(__fmul_rn(a.x, f), __fmul_rn(a.y, f), __fmul_rn(b.x, f), __fmul_rn(b.y, f));
      }
      *to = *reinterpret_cast<const uint4*>(u4);
    }
  }
  if (active && l == 0 && s != old) *scale = s;
  const bool exact = !(__float_as_uint(s) & 0x7fffffu);
  const float inv = __frcp_rn(s);
#pragma unroll 1
  for (int r = last; r >= 0; r = previous_row(r)) {  // the last row is at hand
    if (r < last) row(r, previous_row(r));
    const int slot = __shfl_sync(~0u, slot_l, r);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(x[e], inv);
    if (!exact) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __fdiv_rn(x[e], s);
    }
    const uint2 c = make_uint2(e4m3::to_codes(y[0], y[1], y[2], y[3]), e4m3::to_codes(y[4], y[5], y[6], y[7]));
    if (!active) continue;
    store_row<T, D, PAIRED>(codes + (slot & (e4m3::kBlock - 1)) * D, out ? out + ((size_t)(t + r) * p.Hkv + h) * D : nullptr,
                            c, s, off0, off1, l);
  }
}

template <typename T, int D, bool INTER, int KIND>
__device__ __forceinline__ void append_blocks(const BlockParams& bp, int cta, uint32_t* s_top) {
  constexpr int kTeams = kWarps / kShare<D>;
  const AppendParams& p = bp.a;
  const int lane = threadIdx.x & 31;
  const int groups = (p.Hkv + bp.g.heads - 1) / bp.g.heads, units = (p.N + kUnit - 1) / kUnit * groups;
  int turn = 0;
  for (int u = cta * kTeams + (threadIdx.x >> 5) / kShare<D>; u < units; u += bp.g.block_ctas * kTeams) {
    const int chunk = u / groups, h = (u - chunk * groups) * bp.g.heads, first = chunk * kUnit;
    // lane i: the block of token first - 16 + i
    const int token = first - kUnit + lane;
    const int mine = token >= 0 && token < p.N ? block_of(p, __ldg(p.slot + token)) : -1;
    const uint32_t same = __match_any_sync(~0u, mine), before = ((1u << lane) - 1) & ~((1u << lane >> 15) - 1);
    uint32_t heads = __ballot_sync(~0u, mine >= 0 && !(same & before)) >> kUnit;
    const int end = min(h + bp.g.heads, p.Hkv);
    while (heads) {
      const int at = __ffs(heads) - 1;
      heads &= heads - 1;
      append_run<T, D, INTER, KIND>(bp, h, end, first + at, __shfl_sync(~0u, mine, kUnit + at), s_top, turn);
    }
  }
}

// All such blocks.  Short calls, where most are: a warp takes a token.  Long ones: the warps of a CTA look for them among kLook
// tokens, 16 each, and share what they find, with other CTAs that look at the same.
template <typename T, int D, bool INTER, int KIND>
__device__ __forceinline__ void append_tokens(const BlockParams& bp, int cta, uint32_t* s_todo) {
  constexpr int RPW = 256 / D;
  const AppendParams& p = bp.a;
  const int groups = (p.Hkv + RPW - 1) / RPW, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!bp.g.span) {
    for (int u = cta * kWarps + warp; u < p.N * groups; u += bp.g.token_ctas * kWarps) {
      const int t = u / groups;
      append_few<T, D, INTER, KIND>(bp, t, (u - t * groups) * RPW, p.Hkv);
    }
    return;
  }
  const int spans = (groups + bp.g.span - 1) / bp.g.span, units = (p.N + kLook - 1) / kLook * spans * bp.g.parts;
  for (int u = cta; u < units; u += bp.g.token_ctas) {
    const int part = u % bp.g.parts, look = u / bp.g.parts / spans, from = (u / bp.g.parts - look * spans) * bp.g.span;
    const int first = look * kLook, n = min(bp.g.span, groups - from);
    // lane i: the blocks of tokens at - 16 + i and at + i
    const int at = first + warp * e4m3::kBlock, token = at + lane;
    const int old = token >= e4m3::kBlock && token - e4m3::kBlock < p.N ? block_of(p, __ldg(p.slot + token - e4m3::kBlock)) : -1;
    const int now = token < p.N ? block_of(p, __ldg(p.slot + token)) : -1;
    const uint32_t same = __match_any_sync(~0u, old), before = ((1u << lane) - 1) & ~((1u << lane >> 15) - 1);
    const uint32_t starts = __ballot_sync(~0u, old >= 0 && !(same & before)) >> e4m3::kBlock;
    const uint32_t rows = __match_any_sync(~0u, now) & 0xffffu << lane;
    const uint32_t todo = __ballot_sync(~0u, lane < e4m3::kBlock && (starts >> lane & 1) && __popc(rows) <= kShort);
    if (lane == 0) s_todo[warp] = todo;
    __syncthreads();
    int turn = part * kWarps + warp;
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t found = s_todo[w];
      const int items = __popc(found) * n;
      for (; turn < items; turn += kWarps * bp.g.parts) {
        uint32_t rest = found;
        for (int k = turn / n; k; --k) rest &= rest - 1;
        append_few<T, D, INTER, KIND>(bp, first + w * e4m3::kBlock + __ffs(rest) - 1, (from + turn % n) * RPW, p.Hkv);
      }
      turn -= items;
    }
    __syncthreads();
  }
}

// Keys first (they take longest), then values, then queries.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) append_block_kernel(const __grid_constant__ BlockParams p) {
  __shared__ uint32_t s_top[2 * kWarps];  // by team and turn, of its warps; or what they found
  const int kv_ctas = p.g.block_ctas + p.g.token_ctas;
  int cta = blockIdx.x;
  if (cta < kv_ctas) {
    if (cta < p.g.block_ctas) append_blocks<T, D, INTER, kKey>(p, cta, s_top);
    else append_tokens<T, D, INTER, kKey>(p, cta - p.g.block_ctas, s_top);
  } else if ((cta -= kv_ctas) < kv_ctas) {
    if (cta < p.g.block_ctas) append_blocks<T, D, INTER, kValue>(p, cta, s_top);
    else append_tokens<T, D, INTER, kValue>(p, cta - p.g.block_ctas, s_top);
  } else {
    constexpr int GROUPQ = kIterQ * 32 / (D / 8);
    cta -= kv_ctas;
    const int j = cta % p.a.q_items, per = p.g.q_ctas / p.a.q_items;
    append_rows<T, D, INTER, kQuery>(p.a, j * GROUPQ, min(GROUPQ, p.a.Hq - j * GROUPQ),
                                     cta / p.a.q_items * kWarps + (threadIdx.x >> 5), per * kWarps);
  }
}

dkv_status refuse(dkv_status s, const char* msg) {
  set_last_error(s, msg);
  return s;
}

template <typename T, int D>
void launch(BlockParams& p, cudaStream_t s) {
  p.g = append_geometry(p.a.N, p.a.q ? p.a.Hq : 0, p.a.Hkv, D);
  p.a.q_items = p.g.q_items;
  if (p.a.inter) append_block_kernel<T, D, true><<<p.g.grid, kThreads, 0, s>>>(p);
  else append_block_kernel<T, D, false><<<p.g.grid, kThreads, 0, s>>>(p);
}

}  // namespace

extern "C" dkv_status dkv_block_append(const dkv_block_append_t* b, void* stream) {
  if (!b) return refuse(DKV_ERR_INVALID_ARG, "null description");
  if (!b->k || !b->k_pool || !b->k_scales || !b->v_scales)
    return refuse(DKV_ERR_INVALID_ARG, "keys, values, pools and their scales come together");
  if ((reinterpret_cast<uintptr_t>(b->k_scales) | reinterpret_cast<uintptr_t>(b->v_scales)) & 3)
    return refuse(DKV_ERR_INVALID_ARG, "scales must start on 4-byte boundaries");
  dkv_append_t a = {};
  a.q = b->q; a.k = b->k; a.v = b->v;
  a.q_stride = b->q_stride; a.k_stride = b->k_stride; a.v_stride = b->v_stride;
  a.q_gamma = b->q_gamma; a.k_gamma = b->k_gamma; a.cos_sin = b->cos_sin;
  a.positions = b->positions; a.slots = b->slots;
  a.k_pool = b->k_pool; a.v_pool = b->v_pool; a.q_out = b->q_out; a.k_out = b->k_out; a.v_out = b->v_out;
  a.rows = b->rows; a.n_q_heads = b->n_q_heads; a.n_kv_heads = b->n_kv_heads; a.head_dim = b->head_dim;
  a.dtype = b->dtype; a.rotary_dim = b->rotary_dim; a.max_positions = b->max_positions;
  a.interleaved = b->interleaved; a.page_tokens = b->page_tokens; a.num_pages = b->num_pages;
  a.eps = b->eps; a.k_scale = a.v_scale = 1.0f;
  const dkv_status st = check_append(&a);
  if (st != DKV_OK) return st;
  BlockParams p;
  fill_append(&a, p.a);
  p.k_scales = b->k_scales;
  p.v_scales = b->v_scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.dtype == DKV_BF16) {
    if (a.head_dim == 64) launch<__nv_bfloat16, 64>(p, s); else launch<__nv_bfloat16, 128>(p, s);
  } else {
    if (a.head_dim == 64) launch<__half, 64>(p, s); else launch<__half, 128>(p, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DKV_OK : refuse(DKV_ERR_CUDA, cudaGetErrorString(e));
}
