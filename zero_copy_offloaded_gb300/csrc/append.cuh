// What the appends share: norm, rotation and E2M1 quantisation of head rows, and the checks of their arguments.
#pragma once

#include <float.h>
#include <stdio.h>

#include "e2m1.cuh"
#include "tc_common.cuh"

namespace dkv {

void set_last_error(dkv_status s, const char* msg);

struct AppendParams {
  const void* q;
  const void* k;
  const void* v;
  long long qs, ks, vs;  // token strides (elements)
  const int* pos;        // null: no rotation
  const int* slot;       // null: no append
  const float* cos_sin;  // [max_pos, rot]
  const void* q_gamma;
  const void* k_gamma;
  uint8_t* k_pool;
  uint8_t* v_pool;
  void* q_out;
  void* k_out;
  void* v_out;
  long long slots;       // rows of the pool
  int N, Hq, Hkv, rot, max_pos, inter;
  int page_shift;
  int q_items, kv_items;  // head groups of queries, of keys and of values
  float eps, k_scale, v_scale;
};

constexpr int kAppendThreads = 256;
// Rows of each lane group for one token, loaded at once: a query row is the lighter work.
constexpr int kIterQ = 8, kIterKV = 4;

// s + b with its rounding error added to e, for any order of magnitudes (Knuth, The Art of Computer
// Programming, volume 2, section 4.2.2).
__device__ __forceinline__ void two_sum(float& s, float& e, float b) {
  const float t = __fadd_rn(s, b);
  const float z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(b, z)));
  s = t;
}

// fp32(1 / sqrt((hi + lo) / D + eps)): one Newton step on rsqrt with the residual
// 1 - m y^2 in two words.  Returns 0 where the mean lies outside fp32's safe range.
template <int D>
__device__ __forceinline__ float inv_rms(float hi, float lo, float eps) {
  float s = hi * (1.0f / D), e = lo * (1.0f / D);  // exact: D is a power of two
  two_sum(s, e, eps);
  const float m = __fadd_rn(s, e);
  const float ml = __fadd_rn(__fsub_rn(s, m), e);
  if (!(m > 1e-30f && m < 1e30f)) return 0.f;
  const float y = rsqrtf(m);
  const float p = __fmul_rn(y, y), pe = __fmaf_rn(y, y, -p);
  float t = __fmaf_rn(-m, p, 1.0f);
  t = __fmaf_rn(-m, pe, t);
  t = __fmaf_rn(-ml, p, t);
  return __fmaf_rn(y, __fmaf_rn(0.375f * t, t, 0.5f * t), y);
}

// The same in fp64, for rows whose squares leave fp32's range.
template <int LPR>
__device__ __noinline__ float inv_rms_wide(float a, float b, float c, float d, float e, float f, float g,
                                           float h, float eps) {
  double sum = (double)a * a + (double)b * b + (double)c * c + (double)d * d + (double)e * e +
               (double)f * f + (double)g * g + (double)h * h;
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) sum += __shfl_xor_sync(~0u, sum, m);
  return (float)(1.0 / sqrt(sum / (8 * LPR) + (double)eps));
}

template <typename T>
__device__ __forceinline__ void unpack4(const uint2& w, float* x) {
  const float2 a = DT<T>::to_f2(w.x), b = DT<T>::to_f2(w.y);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

template <typename T>
__device__ __forceinline__ uint2 pack4(const float* x) {
  return make_uint2(tc::pack2<T>(x[0], x[1]), tc::pack2<T>(x[2], x[3]));
}

// Two fp32 operations an instruction: a - b, and two_sum, of which b may be a product that is exact in fp32.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 f2_sub(f32x2 a, f32x2 b) { return tc::f2_fma(b, tc::f2_pack(-1.f, -1.f), a); }
__device__ __forceinline__ void two_sum2(f32x2& s, f32x2& e, f32x2 b) {
  const f32x2 t = tc::f2_add(s, b), z = f2_sub(t, s);
  e = tc::f2_add(e, tc::f2_add(f2_sub(s, f2_sub(t, z)), f2_sub(b, z)));
  s = t;
}

// How a row's squares are added up: in fp32, in two words, in two words for each half of the elements.
enum Sum : int { kPlain, kExact, kExactPairs };

// x (8 elements of a row held by LPR lanes) times the row's 1 / rms and the norm weights.
template <int LPR, Sum SUM>
__device__ __forceinline__ void norm_row(float (&x)[8], const float (&g)[8], float eps) {
  constexpr bool EXACT = SUM != kPlain;
  float hi = 0.f, lo = 0.f;
  if constexpr (EXACT) {
    if constexpr (SUM == kExactPairs) {
      f32x2 s, e;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 v = tc::f2_pack(x[2 * i], x[2 * i + 1]), sq = tc::f2_mul(v, v);
        if (i) {
          two_sum2(s, e, sq);
        } else {
          s = sq;
          e = 0;
        }
      }
      float oh, ol;
      tc::f2_unpack(s, hi, oh);
      tc::f2_unpack(e, lo, ol);
      two_sum(hi, lo, oh);
      lo = __fadd_rn(lo, ol);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) two_sum(hi, lo, __fmul_rn(x[e], x[e]));
    }
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1) {
      const float oh = __shfl_xor_sync(~0u, hi, d), ol = __shfl_xor_sync(~0u, lo, d);
      two_sum(hi, lo, oh);
      lo = __fadd_rn(lo, ol);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) hi = fmaf(x[e], x[e], hi);
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1) hi += __shfl_xor_sync(~0u, hi, d);
  }
  float r;
  if constexpr (EXACT) {
    r = inv_rms<8 * LPR>(hi, lo, eps);
  } else {
    const float m = fmaf(hi, 1.0f / (8 * LPR), eps);
    r = m > 1e-30f && m < 1e30f ? rsqrtf(m) : 0.f;
  }
  if (__any_sync(~0u, r == 0.f)) {
    const float wide = inv_rms_wide<LPR>(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], eps);
    if (r == 0.f) r = wide;
  }
  const f32x2 r2 = tc::f2_pack(r, r);
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    tc::f2_unpack(tc::f2_mul(tc::f2_mul(tc::f2_pack(x[e], x[e + 1]), r2), tc::f2_pack(g[e], g[e + 1])), x[e], x[e + 1]);
}

// (a, b) <- (a c - b s, b c + a s) of four pairs: elements e and 4 + e, or (INTER) 2 e and 2 e + 1.  The products take two
// elements an instruction; an add.rn.f32x2 of them becomes an FMA, whose product is not rounded (a quarter of the sums
// differ), so that the sums take one.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&x)[8], const float* c, const float* s) {
  if constexpr (INTER) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float &a = x[2 * e], &b = x[2 * e + 1];
      const float ra = __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
      b = __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]));
      a = ra;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const f32x2 a = tc::f2_pack(x[e], x[e + 1]), b = tc::f2_pack(x[4 + e], x[5 + e]);
      const f32x2 c2 = tc::f2_pack(c[e], c[e + 1]), s2 = tc::f2_pack(s[e], s[e + 1]);
      float u[2], v[2];
      tc::f2_unpack(tc::f2_mul(a, c2), u[0], u[1]);
      tc::f2_unpack(tc::f2_mul(b, s2), v[0], v[1]);
      x[e] = __fsub_rn(u[0], v[0]);
      x[e + 1] = __fsub_rn(u[1], v[1]);
      tc::f2_unpack(tc::f2_mul(b, c2), u[0], u[1]);
      tc::f2_unpack(tc::f2_mul(a, s2), v[0], v[1]);
      x[4 + e] = __fadd_rn(u[0], v[0]);
      x[5 + e] = __fadd_rn(u[1], v[1]);
    }
  }
}

// y / s for s whose correctly rounded reciprocal is r: the quotient's residual is exact in one fused
// multiply-add, and a second one corrects it (Markstein, Computation of elementary functions on the IBM RISC
// System/6000 processor, 1990).  For the divisors here, E4M3 numbers (four bits) and 6, the result is
// the correctly rounded quotient for every significand of y.
__device__ __forceinline__ float divide(float y, float s, float r) {
  const float q = __fmul_rn(y, r);
  return __fmaf_rn(__fmaf_rn(-q, s, y), r, q);
}

// Quantises the 8 elements x of a lane (a block is two neighbouring lanes): the codes and, on
// the even lane, the scale byte.  Leaves the block's scale in `sf`.
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t& sb, float& sf) {
  uint32_t top = 0;  // as bits, NaN above infinity above every number
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(~0u, top, 1));
  sb = top >= 0x7f800000u  // a NaN scale: the block reads back as NaN
           ? 0x7fu
           : __nv_cvt_float_to_fp8(divide(__uint_as_float(top), 6.0f, 1.0f / 6.0f), __NV_SATFINITE, __NV_E4M3);
  const uint32_t sh = e2m1::scales_to_h2(sb);
  sf = __low2float(*reinterpret_cast<const __half2*>(&sh));
  const bool some = sf > 0.f;
  const float r = __frcp_rn(some ? sf : 1.0f);
  uint32_t code = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    code |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(divide(x[2 * e], sf, r), divide(x[2 * e + 1], sf, r)),
                                               __NV_E2M1, cudaRoundNearest)
            << (8 * e);
  return some ? code : 0;
}

constexpr int kQuery = 0, kKey = 1, kValue = 2;

// The rows of `heads` heads from h0 on, for tokens first, first + step, ...  A row takes D/8 lanes,
// 8 elements each.  Query rows need no blocks, so a lane holds both partners of its pairs
// (two runs of 4 elements); key and value rows keep 8 neighbouring elements on a lane, and
// keys exchange their partners.
template <typename T, int D, bool INTER, int KIND>
__device__ __forceinline__ void append_rows(const AppendParams& p, int h0, int heads, int first, int step) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  constexpr bool PAIRED = KIND == kQuery && !INTER;
  constexpr int ITER = KIND == kQuery ? kIterQ : kIterKV;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const float nan = __int_as_float(0x7fc00000);
  const int half = p.rot / 2;
  const bool in_rot = KIND != kValue && p.pos && l * 8 < p.rot;
  const int off0 = PAIRED && in_rot ? 4 * l : 8 * l, off1 = PAIRED && in_rot ? half + 4 * l : 8 * l + 4;
  const T* base = static_cast<const T*>(KIND == kQuery ? p.q : KIND == kKey ? p.k : p.v) + (size_t)(h0 + sub) * D;
  const long long stride = KIND == kQuery ? p.qs : KIND == kKey ? p.ks : p.vs;
  const int H = KIND == kQuery ? p.Hq : p.Hkv;
  T* out = static_cast<T*>(KIND == kQuery ? p.q_out : KIND == kKey ? p.k_out : p.v_out);
  const T* gam = static_cast<const T*>(KIND == kQuery ? p.q_gamma : KIND == kKey ? p.k_gamma : nullptr);
  const bool norm = KIND != kValue && gam != nullptr;
  float g[8];
  if (norm) {
    unpack4<T>(__ldg(reinterpret_cast<const uint2*>(gam + off0)), g);
    unpack4<T>(__ldg(reinterpret_cast<const uint2*>(gam + off1)), g + 4);
  }
  // half pairs of keys: -1 the lane holds the first of its pairs, 1 the second
  const int side = KIND == kKey && !INTER && in_rot ? (l * 8 < half ? -1 : 1) : 0;
  const int partner = lane - side * (p.rot / 16);
  const size_t page_bytes = e2m1::page_bytes(D, 1 << p.page_shift);
  const float mul = KIND == kKey ? p.k_scale : p.v_scale;
  uint8_t* pool = (KIND == kKey ? p.k_pool : p.v_pool) + (KIND == kQuery ? 0 : (size_t)(h0 + sub) * page_bytes);

#pragma unroll 1
  for (int tok = first; tok < p.N; tok += step) {
    const T* src = base + (size_t)tok * stride;
    auto load = [&](int h, uint2& a, uint2& b) {  // head h0 + h + sub
      if (h + sub < heads) {
        if constexpr (PAIRED) {
          a = *reinterpret_cast<const uint2*>(src + h * D + off0);
          b = *reinterpret_cast<const uint2*>(src + h * D + off1);
        } else {
          const uint4 w = *reinterpret_cast<const uint4*>(src + h * D + l * 8);
          a = make_uint2(w.x, w.y);
          b = make_uint2(w.z, w.w);
        }
      }
    };
    uint2 w[ITER][2] = {};
#pragma unroll
    for (int i = 0; i < ITER; ++i) load(i * RPW, w[i][0], w[i][1]);
    const int slot = p.slot ? __ldg(p.slot + tok) : 0;
    if (p.slot && (slot < 0 || slot >= p.slots)) continue;  // padding: nothing of it is written
    bool far = false, turn = false;
    float c[8], s[8];
    if (KIND != kValue && p.pos) {
      const int pos = __ldg(p.pos + tok);
      far = pos < 0 || pos >= p.max_pos;
      turn = !far && in_rot;
      if (turn) {
        // 4 pairs of a lane's own, or the 8 pairs that its elements are one side of
        const float* at = p.cos_sin + (size_t)pos * p.rot + (KIND == kKey && !INTER ? 8 * l - (side > 0 ? half : 0) : 4 * l);
#pragma unroll
        for (int i = 0; i < (KIND == kKey && !INTER ? 2 : 1); ++i) {
          const float4 a = __ldg(reinterpret_cast<const float4*>(at + 4 * i));
          const float4 b = __ldg(reinterpret_cast<const float4*>(at + half + 4 * i));
          c[4 * i] = a.x; c[4 * i + 1] = a.y; c[4 * i + 2] = a.z; c[4 * i + 3] = a.w;
          s[4 * i] = b.x; s[4 * i + 1] = b.y; s[4 * i + 2] = b.z; s[4 * i + 3] = b.w;
        }
        if (side < 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = -s[e];
        }
      }
    }
    uint8_t* codes = nullptr;
    uint8_t* scale = nullptr;
    if (KIND != kQuery && p.slot) {
      const int row = slot & ((1 << p.page_shift) - 1);
      uint8_t* page = pool + (size_t)(slot >> p.page_shift) * p.Hkv * page_bytes;
      codes = page + row * e2m1::code_bytes(D) + l * 4;
      scale = page + ((size_t)e2m1::code_bytes(D) << p.page_shift) + row * e2m1::scale_bytes(D) + l / 2;
    }
    T* to = out ? out + ((size_t)tok * H + h0 + sub) * D : nullptr;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int h = i * RPW;
      if (h >= heads) break;
      float x[8];
      unpack4<T>(w[i][0], x);
      unpack4<T>(w[i][1], x + 4);
      if (norm) norm_row<LPR, KIND == kKey ? kExact : kPlain>(x, g, p.eps);
      if constexpr (KIND == kKey && !INTER) {
        if (p.pos) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float o = __shfl_sync(~0u, x[e], partner);
            // the first of a pair: x c - o s, the second: x c + o s (the sign is in s)
            if (turn) x[e] = __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(o, s[e]));
          }
        }
      } else if constexpr (KIND != kValue) {
        if (turn) rotate<INTER>(x, c, s);
      }
      if (KIND != kValue && far) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = nan;
      }
      const bool write = h + sub < heads;
      if (KIND != kQuery && p.slot) {
        if (mul != 1.0f) {  // (a reciprocal would round twice, and move codes next to a border)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(x[e], mul);
        }
        uint32_t sb;
        float sf;
        const uint32_t code = quantise(x, sb, sf);
        if (write) {
          *reinterpret_cast<uint32_t*>(codes + (size_t)h * page_bytes) = code;
          if (!(l & 1)) scale[(size_t)h * page_bytes] = (uint8_t)sb;
        }
        if (to) {  // what the cache now holds
          uint32_t y[4];
          e2m1::codes_to_h2(code, y);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y[e]));
            x[2 * e] = __fmul_rn(__fmul_rn(f.x, sf), mul);
            x[2 * e + 1] = __fmul_rn(__fmul_rn(f.y, sf), mul);
          }
        }
      }
      if (to && write) {
        const uint2 a = pack4<T>(x), b = pack4<T>(x + 4);
        if constexpr (PAIRED) {
          *reinterpret_cast<uint2*>(to + h * D + off0) = a;
          *reinterpret_cast<uint2*>(to + h * D + off1) = b;
        } else {
          *reinterpret_cast<uint4*>(to + h * D + l * 8) = make_uint4(a.x, a.y, b.x, b.y);
        }
      }
    }
  }
}

// append_e2m1.cu: what either append refuses, and its arguments as the kernels take them.
dkv_status check_append(const dkv_append_t* a);
void fill_append(const dkv_append_t* a, AppendParams& p);

}  // namespace dkv
