// dkv_paged_attend and dkv_block_attend: the checks of their arguments, workspaces, and the choice of a kernel.
#include <float.h>
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>
#include <chrono>

#include "attend.cuh"

namespace dkv {
void set_last_error(dkv_status s, const char* msg);
}

namespace {

using namespace dkv;

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

template <Format F, typename T, int D>
cudaError_t launch_rows(const AttendParams& p, int R, cudaStream_t s) {
  return R == kTcRows ? launch_attend_many<F, T, D>(p, kSms, s) : launch_attend_few<F, T, D>(p, R, s);
}

template <Format F>
cudaError_t launch(const AttendParams& p, int dtype, int D, int R, cudaStream_t s) {
  if (dtype == DKV_BF16)
    return D == 64 ? launch_rows<F, __nv_bfloat16, 64>(p, R, s) : launch_rows<F, __nv_bfloat16, 128>(p, R, s);
  return D == 64 ? launch_rows<F, __half, 64>(p, R, s) : launch_rows<F, __half, 128>(p, R, s);
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

// Either call, of a cache of this format; the scales of an E4M3 pool beside it.
static dkv_status attend(const dkv_attend_t* a, Format format, const float* k_scales, const float* v_scales,
                         void* stream) {
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
  if (format == kE4M3 && (long long)a->num_pages * a->page_tokens / e4m3::kBlock * a->n_kv_heads >= 0xFFFFFFFFLL)
    return refuse(DKV_ERR_INVALID_ARG, "a pool has fewer than 2^32 - 1 blocks");
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
  p.page_bytes = format == kE2M1 ? e2m1::page_bytes(D, a->page_tokens) : (size_t)D * a->page_tokens;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.scale_log2 = (float)(1.4426950408889634 * (double)a->scale);
  p.v_scale = a->v_scale;
  p.debug_withhold = g_debug_withhold;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = format == kE2M1 ? launch<kE2M1>(p, a->dtype, D, R, s) : launch<kE4M3>(p, a->dtype, D, R, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return refuse(DKV_ERR_CUDA, cudaGetErrorString(e));
  }
  return DKV_OK;
}

extern "C" dkv_status dkv_paged_attend(const dkv_attend_t* a, void* stream) {
  return attend(a, kE2M1, nullptr, nullptr, stream);
}

extern "C" dkv_status dkv_block_attend(const dkv_block_attend_t* b, void* stream) {
  if (!b) return refuse(DKV_ERR_INVALID_ARG, "null description");
  if (!b->k_scales || !b->v_scales) return refuse(DKV_ERR_INVALID_ARG, "null pointer argument");
  if ((reinterpret_cast<uintptr_t>(b->k_scales) | reinterpret_cast<uintptr_t>(b->v_scales)) & 3)
    return refuse(DKV_ERR_INVALID_ARG, "scales must start on 4-byte boundaries");
  dkv_attend_t a = {};
  a.q = b->q; a.q_stride = b->q_stride; a.k_pool = b->k_pool; a.v_pool = b->v_pool;
  a.page_table = b->page_table; a.kv_len = b->kv_len; a.row_start = b->row_start; a.out = b->out; a.lse = b->lse;
  a.workspace = b->workspace; a.workspace_bytes = b->workspace_bytes;
  a.batch = b->batch; a.rows = b->rows; a.max_rows = b->max_rows;
  a.n_q_heads = b->n_q_heads; a.n_kv_heads = b->n_kv_heads; a.head_dim = b->head_dim; a.dtype = b->dtype;
  a.page_tokens = b->page_tokens; a.num_pages = b->num_pages; a.max_pages = b->max_pages;
  a.scale = b->scale; a.v_scale = 1.0f;
  return attend(&a, kE4M3, b->k_scales, b->v_scales, stream);
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
