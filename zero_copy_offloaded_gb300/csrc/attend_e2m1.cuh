// What the kernels of the 4-bit paged attention share.
#pragma once

#include <math.h>

#include "e2m1.cuh"
#include "per_device.h"

namespace dkv {

// The item that a CTA left unfinished: one that it began, or one that fills it.
struct AttendDesc {
  int pieces;           // how many CTAs hold it; 0: there is none
  int begin;            // the first of them
  int row0;             // first query row of the sequence
  int first, last;      // packed rows (token-major over the group's heads) of the item
  int head0;            // first query head of the group
  int pad[2];
};

struct AttendParams {
  const void* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const int* table;      // [B][max_pages]
  const int* kv_len;     // [B]
  const int* row_start;  // [B + 1], or null: row b is sequence b's only one
  void* out;
  float* lse;
  AttendDesc* desc;             // many rows: by CTA
  unsigned long long* done;     // few rows: finished pieces, by slot of a group's first one and by the
                                // CTA that began the item
  unsigned long long tag;       // the call's own, in the upper 48 bits
  float* part_ml;
  float* part_o;
  long long q_stride;
  size_t page_bytes;
  int B, N, Hq, Hkv, G;
  int num_pages, max_pages, page_shift;
  float scale_log2, v_scale;
  int debug_withhold;    // test hook: the many-row kernel never signals that an item's outputs are done
};

// Sequence b's cached keys, first row and rows, held inside what the buffers have.
__device__ __forceinline__ void batch_entry(const AttendParams& p, int b, int& kv, int& row, int& n) {
  kv = min(max(p.kv_len[b], 0), p.max_pages << p.page_shift);
  if (p.row_start) {
    row = min(max(p.row_start[b], 0), p.N);
    n = min(max(p.row_start[b + 1], row), p.N) - row;
  } else {
    row = b;
    n = 1;
  }
}

// attend_e2m1_tc.cu: items of kTcRows query rows, one CTA on each of `grid` SMs, and their join.
constexpr int kTcRows = 256;
template <typename T, int D>
cudaError_t launch_attend_tc(const AttendParams& p, int grid, cudaStream_t s);

// Rows are normalised and rounded once; a row that saw no key is zero, its lse -infinity.
// A NaN sum or output stays NaN.
template <typename T, int V>
__device__ __forceinline__ void store_row(const AttendParams& p, int row, int head, int D, int d0,
                                          const float (&acc)[V], float top, float sum, bool lead) {
  const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
  T* o = static_cast<T*>(p.out) + ((size_t)row * p.Hq + head) * D + d0;
  uint32_t w[V / 2];  // V: 2, 4, 8 or 16
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const T a = DT<T>::from_f(acc[2 * i] * inv), b = DT<T>::from_f(acc[2 * i + 1] * inv);
    w[i] = (uint32_t)(*reinterpret_cast<const uint16_t*>(&a)) |
           ((uint32_t)(*reinterpret_cast<const uint16_t*>(&b)) << 16);
  }
  if constexpr (V == 2) *reinterpret_cast<uint32_t*>(o) = w[0];
  else if constexpr (V == 4) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
  else
#pragma unroll
    for (int i = 0; i < V / 8; ++i)
      reinterpret_cast<uint4*>(o)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  if (lead && p.lse)
    p.lse[(size_t)row * p.Hq + head] =
        sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace dkv
