// dkv_qkv_append: per-head RMS norm of queries and keys, rotation to their
// positions, and the append of keys and values to a paged E2M1 cache, in one
// pass over the projection's output.
//
// For a row x of one head (D elements), with the norm weights g:
//   r = 1 / sqrt(sum x^2 / D + eps),  y_i = (x_i r) g_i
//   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)   for each rotated pair (a, b)
// and, for keys and values, blocks of 16: scale = e4m3(max|y| / 6), code = e2m1(y / scale).
//
// Arithmetic is fp32 and every step above rounds once, with no contracted
// multiply-adds, so the result does not depend on the launch: a code next to a
// rounding border is the same code everywhere.  The one sum, sum x^2 of a key
// row, is carried in two fp32 words (squares of 16-bit values are exact in
// fp32 or nearly so, and each addition keeps its error), which makes r the
// correctly rounded one up to 2^-20 of the rows; query rows, which are only
// rounded to 16 bits, use a plain fp32 sum.
//
// What bounds it: each byte once through memory, 26 KB a row of 32/8 heads of 128.  4096 such rows
// take 29 us (3.7 TB/s of 6.8 measured), 16384 rows of 32/32 fp16 heads of 64, rotated in half
// and without norms, 86 us (5.1 TB/s).  In the first neither memory nor a pipe is full: its warps wait for
// their own chains of scalar fp32 (norms, exact sums, quantisation; about 60 % of the issue slots), and queries
// alone (15 us) and keys and values alone (14) add up.  A pool in host memory takes 53 us for them: the codes
// cross the link in stores of 4 bytes a lane, the scales of 1.
#include <float.h>
#include <stdio.h>

#include "e2m1.cuh"
#include "tc_common.cuh"

namespace dkv {
void set_last_error(dkv_status s, const char* msg);
}

namespace {

using namespace dkv;

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

constexpr int kThreads = 256;
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

// x (8 elements of a row held by LPR lanes) times the row's 1 / rms and the norm weights.
template <int LPR, bool EXACT>
__device__ __forceinline__ void norm_row(float (&x)[8], const float (&g)[8], float eps) {
  float hi = 0.f, lo = 0.f;
  if constexpr (EXACT) {
#pragma unroll
    for (int e = 0; e < 8; ++e) two_sum(hi, lo, __fmul_rn(x[e], x[e]));
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
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], r), g[e]);
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
      if (norm) norm_row<LPR, KIND == kKey>(x, g, p.eps);
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
        if (turn) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float &a = INTER ? x[2 * e] : x[e], &b = INTER ? x[2 * e + 1] : x[4 + e];
            const float ra = __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
            b = __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]));
            a = ra;
          }
        }
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

// blockIdx.y: a group of head rows of one kind, keys first (they take longest), then
// values, then queries; a warp takes one token of it at a time.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const AppendParams p) {
  constexpr int GROUP = kIterKV * 32 / (D / 8), GROUPQ = kIterQ * 32 / (D / 8);
  const int first = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), step = gridDim.x * (kThreads / 32);
  int j = blockIdx.y;
  if (j < p.kv_items) {
    append_rows<T, D, INTER, kKey>(p, j * GROUP, min(GROUP, p.Hkv - j * GROUP), first, step);
  } else if ((j -= p.kv_items) < p.kv_items) {
    append_rows<T, D, INTER, kValue>(p, j * GROUP, min(GROUP, p.Hkv - j * GROUP), first, step);
  } else {
    j -= p.kv_items;
    append_rows<T, D, INTER, kQuery>(p, j * GROUPQ, min(GROUPQ, p.Hq - j * GROUPQ), first, step);
  }
}

dkv_status refuse(dkv_status s, const char* msg) {
  set_last_error(s, msg);
  return s;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, int D>
void launch(AppendParams& p, cudaStream_t s) {
  constexpr int GROUP = kIterKV * 32 / (D / 8), GROUPQ = kIterQ * 32 / (D / 8);
  p.q_items = p.q ? (p.Hq + GROUPQ - 1) / GROUPQ : 0;
  p.kv_items = p.k ? (p.Hkv + GROUP - 1) / GROUP : 0;
  // a token per warp up to eight waves of CTAs, so that the kinds' unequal times even out
  const long long y = p.q_items + 2LL * p.kv_items, want = (p.N + kThreads / 32 - 1) / (kThreads / 32);
  const long long most = (8 * 3 * 152 + y - 1) / y;
  const dim3 grid((unsigned)(want < most ? want : most), (unsigned)y);
  if (p.inter) append_kernel<T, D, true><<<grid, kThreads, 0, s>>>(p);
  else append_kernel<T, D, false><<<grid, kThreads, 0, s>>>(p);
}

}  // namespace

extern "C" dkv_status dkv_qkv_append(const dkv_append_t* a, void* stream) {
  if (!a) return refuse(DKV_ERR_INVALID_ARG, "null description");
  if (!a->q && !a->k) return refuse(DKV_ERR_INVALID_ARG, "neither queries nor keys");
  if (!a->k != !a->v) return refuse(DKV_ERR_INVALID_ARG, "keys and values come together");
  if (a->q && !a->q_out) return refuse(DKV_ERR_INVALID_ARG, "null q_out");
  if (a->rows <= 0 || a->rows > (1 << 30)) return refuse(DKV_ERR_INVALID_ARG, "rows outside [1, 2^30]");
  if (a->dtype != DKV_BF16 && a->dtype != DKV_FP16)
    return refuse(DKV_ERR_INVALID_ARG, "dtype is not bf16 (0) or fp16 (1)");
  if (a->head_dim != 64 && a->head_dim != 128)
    return refuse(DKV_ERR_UNSUPPORTED, "head_dim (supported: 64, 128)");
  const int D = a->head_dim;
  if ((a->q && (a->n_q_heads <= 0 || a->n_q_heads > 65536)) ||
      (a->k && (a->n_kv_heads <= 0 || a->n_kv_heads > 65536)))
    return refuse(DKV_ERR_INVALID_ARG, "head counts outside [1, 65536]");
  if ((a->q && (a->q_stride < (long long)a->n_q_heads * D || a->q_stride % 8)) ||
      (a->k && (a->k_stride < (long long)a->n_kv_heads * D || a->k_stride % 8 ||
                a->v_stride < (long long)a->n_kv_heads * D || a->v_stride % 8)))
    return refuse(DKV_ERR_INVALID_ARG, "a token stride must hold the heads and be a multiple of 8");
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->q_out) ||
      !aligned16(a->k_out) || !aligned16(a->v_out) || !aligned16(a->q_gamma) ||
      !aligned16(a->k_gamma) || !aligned16(a->cos_sin) || !aligned16(a->k_pool) ||
      !aligned16(a->v_pool))
    return refuse(DKV_ERR_INVALID_ARG, "tensors must start on 16-byte boundaries");
  if ((a->k_pool != nullptr) != (a->slots != nullptr) || !a->k_pool != !a->v_pool)
    return refuse(DKV_ERR_INVALID_ARG, "both pools and the slots come together");
  if (a->k_pool && !a->k) return refuse(DKV_ERR_INVALID_ARG, "pools without keys");
  if (a->k && !a->k_pool && (!a->k_out || !a->v_out))
    return refuse(DKV_ERR_INVALID_ARG, "keys go to the pools or to k_out and v_out");
  if (a->k_pool) {
    if (a->page_tokens < e2m1::kMinPageTokens || a->page_tokens > 4096 ||
        (a->page_tokens & (a->page_tokens - 1)))
      return refuse(DKV_ERR_INVALID_ARG, "page_tokens must be a power of two in [16, 4096]");
    if (a->num_pages <= 0 || (long long)a->num_pages * a->page_tokens > (1LL << 30))
      return refuse(DKV_ERR_INVALID_ARG, "num_pages must be positive, num_pages * page_tokens at most 2^30");
    if (!(a->k_scale > 0.f && a->k_scale <= FLT_MAX && a->v_scale > 0.f && a->v_scale <= FLT_MAX) ||
        1.0f / a->k_scale > FLT_MAX || 1.0f / a->v_scale > FLT_MAX)
      return refuse(DKV_ERR_INVALID_ARG, "k_scale and v_scale must be positive, finite and have a finite inverse");
  }
  if (a->cos_sin) {
    if (!a->positions) return refuse(DKV_ERR_INVALID_ARG, "a rotation needs positions");
    if (a->rotary_dim <= 0 || a->rotary_dim > D || a->rotary_dim % 16)
      return refuse(DKV_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16, at most head_dim");
    if (a->max_positions <= 0) return refuse(DKV_ERR_INVALID_ARG, "max_positions must be positive");
  }
  if (!(a->eps >= 0.f && a->eps <= FLT_MAX)) return refuse(DKV_ERR_INVALID_ARG, "eps must be finite and not negative");
  AppendParams p;
  p.q = a->q; p.k = a->k; p.v = a->v;
  p.qs = a->q_stride; p.ks = a->k_stride; p.vs = a->v_stride;
  p.pos = a->cos_sin ? a->positions : nullptr;
  p.slot = a->slots;
  p.cos_sin = a->cos_sin;
  p.q_gamma = a->q_gamma; p.k_gamma = a->k_gamma;
  p.k_pool = static_cast<uint8_t*>(a->k_pool); p.v_pool = static_cast<uint8_t*>(a->v_pool);
  p.q_out = a->q_out; p.k_out = a->k_out; p.v_out = a->v_out;
  p.slots = (long long)a->num_pages * a->page_tokens;
  p.N = a->rows; p.Hq = a->n_q_heads; p.Hkv = a->n_kv_heads;
  p.rot = a->cos_sin ? a->rotary_dim : 16; p.max_pos = a->max_positions; p.inter = a->interleaved;
  p.page_shift = 0;
  while (a->k_pool && (1 << p.page_shift) < a->page_tokens) ++p.page_shift;
  p.eps = a->eps; p.k_scale = a->k_scale; p.v_scale = a->v_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->dtype == DKV_BF16) {
    if (D == 64) launch<__nv_bfloat16, 64>(p, s); else launch<__nv_bfloat16, 128>(p, s);
  } else {
    if (D == 64) launch<__half, 64>(p, s); else launch<__half, 128>(p, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DKV_OK : refuse(DKV_ERR_CUDA, cudaGetErrorString(e));
}
