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
// take 26.8 us in a graph (4.0 TB/s of 6.7 measured; 28.8 a call), 16384 rows of 32/32 fp16 heads of 64, rotated in half
// and without norms, 85.4 us (87.3).  In the first neither memory nor a pipe is full: its warps wait for
// their own chains of fp32 (norms, exact sums, quantisation; about 60 % of the issue slots; products two elements an
// instruction where they can), and queries alone (17.7 us) and keys and values alone (10.8) add up.  A pool in host
// memory takes 51 us for them: the codes cross the link in stores of 4 bytes a lane, the scales of 1.
#include "append.cuh"

namespace {

using namespace dkv;

constexpr int kThreads = kAppendThreads;

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

dkv_status dkv::check_append(const dkv_append_t* a) {
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
  return DKV_OK;
}

void dkv::fill_append(const dkv_append_t* a, AppendParams& p) {
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
}

extern "C" dkv_status dkv_qkv_append(const dkv_append_t* a, void* stream) {
  const dkv_status st = check_append(a);
  if (st != DKV_OK) return st;
  AppendParams p;
  fill_append(a, p);
  const int D = a->head_dim;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->dtype == DKV_BF16) {
    if (D == 64) launch<__nv_bfloat16, 64>(p, s); else launch<__nv_bfloat16, 128>(p, s);
  } else {
    if (D == 64) launch<__half, 64>(p, s); else launch<__half, 128>(p, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DKV_OK : refuse(DKV_ERR_CUDA, cudaGetErrorString(e));
}
