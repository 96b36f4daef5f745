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
#include <float.h>
#include <stdio.h>

#include "e2m1.cuh"

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
  int q_items, kv_items;  // items (of kHeads heads) per token
  float eps, k_scale, v_scale, k_inv, v_inv;
};

constexpr int kThreads = 256;
constexpr int kIter = 4;  // rows of each lane group in flight

// s + e of a and b with the rounding error kept (any order of magnitudes).
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
__device__ __noinline__ float inv_rms_wide(const float (&x)[8], float eps) {
  double sum = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum = fma((double)x[e], (double)x[e], sum);
#pragma unroll
  for (int d = 1; d < LPR; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
  return (float)(1.0 / sqrt(sum / (8 * LPR) + (double)eps));
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = DT<T>::to_f2(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const T a = DT<T>::from_f(x[2 * i]), b = DT<T>::from_f(x[2 * i + 1]);
    u[i] = (uint32_t)(*reinterpret_cast<const uint16_t*>(&a)) |
           ((uint32_t)(*reinterpret_cast<const uint16_t*>(&b)) << 16);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// A warp takes one item: up to kIter * (32 / (D/8)) heads of one kind of one
// token, D/8 lanes to a head row, 8 elements (16 bytes) to a lane.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, HEADS = kIter * RPW;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const int per_tok = p.q_items + 2 * p.kv_items;
  const long long items = (long long)p.N * per_tok;
  const long long step = (long long)gridDim.x * (kThreads / 32);
  for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < items;
       it += step) {
    const int tok = (int)(it / per_tok);
    int j = (int)(it - (long long)tok * per_tok);
    int kind = 0;  // 0 query, 1 key, 2 value
    if (j >= p.q_items) {
      j -= p.q_items;
      kind = 1;
      if (j >= p.kv_items) {
        j -= p.kv_items;
        kind = 2;
      }
    }
    const int heads = kind == 0 ? p.Hq : p.Hkv, h0 = j * HEADS;
    const int slot = p.slot ? p.slot[tok] : -1;
    const int pos = p.pos ? p.pos[tok] : 0;
    const bool skip = p.slot && (slot < 0 || slot >= p.slots);  // padding: nothing of it is written
    if (skip) continue;
    const T* src = kind == 0   ? static_cast<const T*>(p.q) + (size_t)tok * p.qs
                   : kind == 1 ? static_cast<const T*>(p.k) + (size_t)tok * p.ks
                               : static_cast<const T*>(p.v) + (size_t)tok * p.vs;
    uint4 w[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int h = h0 + i * RPW + sub;
      w[i] = h < heads ? *reinterpret_cast<const uint4*>(src + (size_t)h * D + l * 8)
                       : make_uint4(0, 0, 0, 0);
    }
    // this lane's cosines and sines; `side`: 0 not rotated, -1 first of its pairs, 1 second
    float c[8], s[8];
    int side = 0;
    const bool turn = kind < 2 && p.cos_sin != nullptr;
    const bool far = turn && (pos < 0 || pos >= p.max_pos);
    if (turn && l * 8 < p.rot && !far) {
      const float* row = p.cos_sin + (size_t)pos * p.rot;
      const int half = p.rot / 2;
      if (p.inter) {
        side = 2;
        const float4 a = *reinterpret_cast<const float4*>(row + l * 4);
        const float4 b = *reinterpret_cast<const float4*>(row + half + l * 4);
        c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
        s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
      } else {
        side = l * 8 < half ? -1 : 1;
        const float* at = row + (side < 0 ? l * 8 : l * 8 - half);
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) {
          const float4 a = *reinterpret_cast<const float4*>(at + 4 * q4);
          const float4 b = *reinterpret_cast<const float4*>(at + half + 4 * q4);
          c[4 * q4] = a.x; c[4 * q4 + 1] = a.y; c[4 * q4 + 2] = a.z; c[4 * q4 + 3] = a.w;
          s[4 * q4] = b.x; s[4 * q4 + 1] = b.y; s[4 * q4 + 2] = b.z; s[4 * q4 + 3] = b.w;
        }
      }
    }
    const int partner = side < 0 ? lane + p.rot / 16 : side == 1 ? lane - p.rot / 16 : lane;
    const T* gam = static_cast<const T*>(kind == 0 ? p.q_gamma : kind == 1 ? p.k_gamma : nullptr);
    float g[8];
    if (gam) unpack8<T>(*reinterpret_cast<const uint4*>(gam + l * 8), g);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int h = h0 + i * RPW + sub;
      float x[8];
      unpack8<T>(w[i], x);
      if (gam) {
        float hi = 0.f, lo = 0.f;
        if (kind == 1) {
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
        float r = inv_rms<D>(hi, lo, p.eps);
        if (__any_sync(~0u, r == 0.f)) {
          const float wide = inv_rms_wide<LPR>(x, p.eps);
          if (r == 0.f) r = wide;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], r), g[e]);
      }
      if (turn) {
        if (p.inter) {
          if (side) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = x[2 * e], b = x[2 * e + 1];
              x[2 * e] = __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
              x[2 * e + 1] = __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]));
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float o = __shfl_sync(~0u, x[e], partner);
            if (side < 0) x[e] = __fsub_rn(__fmul_rn(x[e], c[e]), __fmul_rn(o, s[e]));
            if (side > 0) x[e] = __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(o, s[e]));
          }
        }
        if (far) {  // no such row in the table
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __int_as_float(0x7fc00000);
        }
      }
      if (kind == 0) {
        if (h < heads)
          *reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + ((size_t)tok * p.Hq + h) * D + l * 8) =
              pack8<T>(x);
        continue;
      }
      T* out = static_cast<T*>(kind == 1 ? p.k_out : p.v_out);
      if (p.slot) {
        const float inv = kind == 1 ? p.k_inv : p.v_inv;
        uint32_t top = 0;  // as bits, NaN above infinity above every number
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = __fmul_rn(x[e], inv);
          top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
        }
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        const float amax = __uint_as_float(top);
        const uint32_t sb = top >= 0x7f800000u
                                ? 0x7fu  // a NaN scale: the block reads back as NaN
                                : __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.0f), __NV_SATFINITE, __NV_E4M3);
        const __half_raw sh = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)sb, __NV_E4M3);
        const float sf = __half2float(*reinterpret_cast<const __half*>(&sh));
        uint32_t code = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 t = sf > 0.f ? make_float2(__fdiv_rn(x[2 * e], sf), __fdiv_rn(x[2 * e + 1], sf))
                                    : make_float2(0.f, 0.f);
          code |= (uint32_t)__nv_cvt_float2_to_fp4x2(t, __NV_E2M1, cudaRoundNearest) << (8 * e);
        }
        if (h < heads) {
          uint8_t* page = (kind == 1 ? p.k_pool : p.v_pool) +
                          ((size_t)(slot >> p.page_shift) * p.Hkv + h) *
                              e2m1::page_bytes(D, 1 << p.page_shift);
          const int row = slot & ((1 << p.page_shift) - 1);
          *reinterpret_cast<uint32_t*>(page + (size_t)row * e2m1::code_bytes(D) + l * 4) = code;
          if (!(l & 1))
            page[((size_t)e2m1::code_bytes(D) << p.page_shift) + row * e2m1::scale_bytes(D) + l / 2] =
                (uint8_t)sb;
        }
        if (out) {  // what the cache now holds
          const float mul = kind == 1 ? p.k_scale : p.v_scale;
          uint32_t hh[4];
          e2m1::codes_to_h2(code, hh);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh[e]));
            x[2 * e] = __fmul_rn(__fmul_rn(f.x, sf), mul);
            x[2 * e + 1] = __fmul_rn(__fmul_rn(f.y, sf), mul);
          }
        }
      }
      if (out && h < heads)
        *reinterpret_cast<uint4*>(out + ((size_t)tok * p.Hkv + h) * D + l * 8) = pack8<T>(x);
    }
  }
}

dkv_status refuse(dkv_status s, const char* msg) {
  set_last_error(s, msg);
  return s;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, int D>
void launch(AppendParams& p, cudaStream_t s) {
  constexpr int HEADS = kIter * 32 / (D / 8);
  p.q_items = p.q ? (p.Hq + HEADS - 1) / HEADS : 0;
  p.kv_items = p.k ? (p.Hkv + HEADS - 1) / HEADS : 0;
  const long long items = (long long)p.N * (p.q_items + 2 * p.kv_items);
  const long long blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
  append_kernel<T, D><<<(unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), kThreads, 0, s>>>(p);
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
  p.k_inv = a->k_pool ? 1.0f / a->k_scale : 1.0f;
  p.v_inv = a->k_pool ? 1.0f / a->v_scale : 1.0f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->dtype == DKV_BF16) {
    if (D == 64) launch<__nv_bfloat16, 64>(p, s); else launch<__nv_bfloat16, 128>(p, s);
  } else {
    if (D == 64) launch<__half, 64>(p, s); else launch<__half, 128>(p, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DKV_OK : refuse(DKV_ERR_CUDA, cudaGetErrorString(e));
}
