// dkv_block_append: per-head RMS norm of queries and keys, rotation to their positions, and the append of keys and
// values to a paged cache of E4M3 codes with one scale for each block of 16 tokens of a head.
//
// Norm and rotation are dkv_qkv_append's, operation by operation.  For the rows y that a call writes to one block:
//   need = the smallest power of two with max|y| <= 448 need,  s = max(need, the block's scale so far)
// where a block whose first row is among them has none so far.  Where s is above it the rows already there
// are brought to the new scale, code <- e4m3(code * old / s); new rows are e4m3(y / s).  Scales are powers of two so that
// the quotients are exact: a code rounds once, and again only in E4M3's subnormals when its block's scale grows.
//
// A warp takes the rows of one block and head together (16 at most, all loads in flight, their fp32 values in
// registers until the largest of them is known), so that the scale needs no second pass and no atomics.  The rows of a
// block are consecutive rows of the call; a warp looks at one token, or at 16 of a long call, and takes the blocks
// that begin there.
#include "append.cuh"
#include "e4m3.cuh"

namespace {

using namespace dkv;

constexpr int kThreads = kAppendThreads, kWarps = kThreads / 32;

struct BlockParams {
  AppendParams a;
  float* k_scales;
  float* v_scales;
  long long kv_units;   // warps' units of keys, and of values: (tokens, KV head)
  int kv_ctas, q_ctas;  // CTAs of each kind; keys first, then values, then queries
  int per_unit;         // tokens of a unit
};

// One run: rows t0 .. t0 + n - 1 of head h, all in block `block` of the pool.
template <typename T, int D, bool INTER, int KIND>
__device__ __forceinline__ void append_run(const BlockParams& bp, int h, int t0, int n, int block) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, ITER = e4m3::kBlock / RPW;
  const AppendParams& p = bp.a;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const float nan = __int_as_float(0x7fc00000);
  const T* src = static_cast<const T*>(KIND == kKey ? p.k : p.v) + (size_t)h * D + l * 8;
  const long long stride = KIND == kKey ? p.ks : p.vs;
  uint4 w[ITER];
  int slot[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int r = i * RPW + sub;
    w[i] = make_uint4(0, 0, 0, 0);
    slot[i] = -1;
    if (r < n) {
      w[i] = *reinterpret_cast<const uint4*>(src + (size_t)(t0 + r) * stride);
      slot[i] = __ldg(p.slot + t0 + r);
    }
  }
  const int per_page = 1 << (p.page_shift - 4), page = block >> (p.page_shift - 4);
  float* scale = (KIND == kKey ? bp.k_scales : bp.v_scales) + ((size_t)page * p.Hkv + h) * per_page + (block & (per_page - 1));
  uint8_t* codes = (KIND == kKey ? p.k_pool : p.v_pool) +
                   ((((size_t)page * p.Hkv + h) << p.page_shift) + (block & (per_page - 1)) * e4m3::kBlock) * D;
  float old = *scale;
  bool fresh = false;
#pragma unroll
  for (int i = 0; i < ITER; ++i) fresh |= slot[i] >= 0 && !(slot[i] & (e4m3::kBlock - 1));
  if (__any_sync(~0u, fresh) || !(old > 0.f && old <= FLT_MAX)) old = 0.f;

  const int half = p.rot / 2;
  const bool in_rot = KIND == kKey && p.pos && l * 8 < p.rot;
  const int side = KIND == kKey && !INTER && in_rot ? (l * 8 < half ? -1 : 1) : 0;
  const int partner = lane - side * (p.rot / 16);
  const T* gam = static_cast<const T*>(KIND == kKey ? p.k_gamma : nullptr);
  float g[8];
  if (KIND == kKey && gam) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(gam + l * 8));
    unpack4<T>(make_uint2(u.x, u.y), g);
    unpack4<T>(make_uint2(u.z, u.w), g + 4);
  }
  float x[ITER][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    unpack4<T>(make_uint2(w[i].x, w[i].y), x[i]);
    unpack4<T>(make_uint2(w[i].z, w[i].w), x[i] + 4);
    if (KIND == kKey && i * RPW < n) {  // norm and rotation; the warp together
      if (gam) norm_row<LPR, true>(x[i], g, p.eps);
      if (p.pos) {
        const int pos = slot[i] >= 0 ? __ldg(p.pos + t0 + i * RPW + sub) : 0;
        const bool far = pos < 0 || pos >= p.max_pos, turn = !far && in_rot;
        float c[8], s[8];
        if (turn) {
          const float* at = p.cos_sin + (size_t)pos * p.rot + (INTER ? 4 * l : 8 * l - (side > 0 ? half : 0));
#pragma unroll
          for (int j = 0; j < (INTER ? 1 : 2); ++j) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(at + 4 * j));
            const float4 b = __ldg(reinterpret_cast<const float4*>(at + half + 4 * j));
            c[4 * j] = a.x; c[4 * j + 1] = a.y; c[4 * j + 2] = a.z; c[4 * j + 3] = a.w;
            s[4 * j] = b.x; s[4 * j + 1] = b.y; s[4 * j + 2] = b.z; s[4 * j + 3] = b.w;
          }
        }
        if constexpr (INTER) {
          if (turn) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float &a = x[i][2 * e], &b = x[i][2 * e + 1];
              const float ra = __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
              b = __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]));
              a = ra;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float o = __shfl_sync(~0u, x[i][e], partner);
            // the first of a pair: x c - o s, the second: x c + o s
            if (turn) x[i][e] = __fadd_rn(__fmul_rn(x[i][e], c[e]), __fmul_rn(o, side < 0 ? -s[e] : s[e]));
          }
        }
        if (far) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][e] = nan;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t m = __float_as_uint(x[i][e]) & 0x7fffffffu;
      if (m >= 0x7f800000u) x[i][e] = nan;  // an infinity too: E4M3 has none
      else top = max(top, m);
    }
  }
  top = __reduce_max_sync(~0u, top);
  const float need = e4m3::scale_for(top), s = fmaxf(need, old);
  if (s > old && old > 0.f) {  // the rows already there, to the new scale
    const float f = __fdiv_rn(old, s);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint4* at = reinterpret_cast<uint4*>(codes) + i * 32 + lane;
      const uint4 v = *at;
      uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t a2 = e4m3::lo_to_h2(u[q]), b2 = e4m3::hi_to_h2(u[q]);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&a2));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&b2));
        u[q] = e4m3::to_codes(__fmul_rn(a.x, f), __fmul_rn(a.y, f), __fmul_rn(b.x, f), __fmul_rn(b.y, f));
      }
      *at = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __syncwarp();
  }
  if (lane == 0 && s != old) *scale = s;
  // a power of two, but for a scale that something else has written
  const bool exact = !(__float_as_uint(s) & 0x7fffffu);
  const float inv = __frcp_rn(s);
  T* out = static_cast<T*>(KIND == kKey ? p.k_out : p.v_out);
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    if (slot[i] < 0) continue;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = exact ? __fmul_rn(x[i][e], inv) : __fdiv_rn(x[i][e], s);
    const uint2 c = make_uint2(e4m3::to_codes(y[0], y[1], y[2], y[3]), e4m3::to_codes(y[4], y[5], y[6], y[7]));
    *reinterpret_cast<uint2*>(codes + (slot[i] & (e4m3::kBlock - 1)) * D + l * 8) = c;
    if (out) {  // what the cache now holds
      const uint32_t h2[4] = {e4m3::lo_to_h2(c.x), e4m3::hi_to_h2(c.x), e4m3::lo_to_h2(c.y), e4m3::hi_to_h2(c.y)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2[e]));
        y[2 * e] = __fmul_rn(f.x, s);
        y[2 * e + 1] = __fmul_rn(f.y, s);
      }
      const uint2 a = pack4<T>(y), b = pack4<T>(y + 4);
      *reinterpret_cast<uint4*>(out + ((size_t)(t0 + i * RPW + sub) * p.Hkv + h) * D + l * 8) =
          make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

template <typename T, int D, bool INTER, int KIND>
__device__ __forceinline__ void append_blocks(const BlockParams& bp, int cta) {
  const AppendParams& p = bp.a;
  const int lane = threadIdx.x & 31;
  for (long long u = (long long)cta * kWarps + (threadIdx.x >> 5); u < bp.kv_units; u += (long long)bp.kv_ctas * kWarps) {
    const long long chunk = u / p.Hkv;
    const int h = (int)(u - chunk * p.Hkv), first = (int)(chunk * bp.per_unit);
    auto block_of = [&](int t) {  // -1: padding, or outside the call
      if (t < 0 || t >= p.N) return -1;
      const int slot = __ldg(p.slot + t);
      return slot < 0 || slot >= p.slots ? -1 : slot / e4m3::kBlock;
    };
    // lane i: the block of token first + i; a block that begins inside the unit may end behind it
    const int mine = block_of(first + lane), last = __shfl_up_sync(~0u, mine, 1);
    const int before = lane ? last : block_of(first - 1);
    uint32_t heads = __ballot_sync(~0u, lane < bp.per_unit && mine >= 0 && mine != before);
    while (heads) {
      const int at = __ffs(heads) - 1;
      heads &= heads - 1;
      const int block = __shfl_sync(~0u, mine, at);
      const uint32_t same = __ballot_sync(~0u, mine == block) >> at;
      // at most 16 rows, all within the 32 that the lanes have seen
      const int n = min(e4m3::kBlock, ~same ? __ffs(~same) - 1 : 32);
      append_run<T, D, INTER, KIND>(bp, h, first + at, n, block);
    }
  }
}

// Keys first (they take longest), then values, then queries.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) append_block_kernel(const __grid_constant__ BlockParams p) {
  int cta = blockIdx.x;
  if (cta < p.kv_ctas) {
    append_blocks<T, D, INTER, kKey>(p, cta);
  } else if ((cta -= p.kv_ctas) < p.kv_ctas) {
    append_blocks<T, D, INTER, kValue>(p, cta);
  } else {
    constexpr int GROUPQ = kIterQ * 32 / (D / 8);
    cta -= p.kv_ctas;
    const int j = cta % p.a.q_items, per = p.q_ctas / p.a.q_items;
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
  constexpr int GROUPQ = kIterQ * 32 / (D / 8);
  constexpr long long kMost = 16 * 2 * 152;  // CTAs of a kind
  p.a.q_items = p.a.q ? (p.a.Hq + GROUPQ - 1) / GROUPQ : 0;
  // Long calls look at 16 tokens a warp.
  p.per_unit = p.a.N >= 2048 ? 16 : 1;
  p.kv_units = (p.a.N + (long long)p.per_unit - 1) / p.per_unit * p.a.Hkv;
  const long long kv = (p.kv_units + kWarps - 1) / kWarps, tokens = (p.a.N + kWarps - 1) / kWarps;
  p.kv_ctas = (int)(kv < kMost ? kv : kMost);
  const long long per = p.a.q_items ? (kMost + p.a.q_items - 1) / p.a.q_items : 0;
  p.q_ctas = (int)(tokens < per ? tokens : per) * p.a.q_items;
  const int grid = 2 * p.kv_ctas + p.q_ctas;
  if (p.a.inter) append_block_kernel<T, D, true><<<grid, kThreads, 0, s>>>(p);
  else append_block_kernel<T, D, false><<<grid, kThreads, 0, s>>>(p);
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
