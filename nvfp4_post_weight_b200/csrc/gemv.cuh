// What the two kernels of the products with solved NVFP4 weights share
// (gemv.cu: any sizes; gemv_fp4.cu: the block-scaled tensor-core path).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "nvfp4_format.cuh"

namespace nvfp4 {

// One call: Y = X Q^T, or silu(X Q0^T) * (X Q1^T) for two matrices, of one
// matrix (offsets null) or of experts over sorted rows.
struct Product {
  const void* X;
  const int* rows;      // X row of each sorted row, or null
  const int* offsets;   // n_experts + 1 row offsets, or null
  const uint8_t* codes[2];
  const uint8_t* scales[2];
  const float* sg[2];
  void* Y;
  int64_t n_x, n_rows, n_experts, d_out, d_in;
  int64_t row0;         // the sorted row that rows, Y and (without rows) X begin with
  int nb;               // blocks of 16 per weight row
  int n_w;              // matrices
  int x_bf16, y_bf16;   // else fp32
};

// gemv_fp4.cu
bool product_fp4_shape(int64_t n_rows, int64_t d_in);
size_t product_fp4_ws_bytes(int64_t n_rows, int64_t d_in);
bool product_fp4_supported(const Product& p);
nvfp4_status launch_product_fp4(const Product& p, void* ws, cudaStream_t st);

// Passes over expert e's rows, `tokens` at a time (offsets are cut to the call's
// n_rows from row0 on), and its first row, from row0, and their number.
__device__ __forceinline__ int expert_passes(const Product& p, int e, int tokens, int* r0, int* n) {
  const int first = (int)p.row0, end = (int)(p.row0 + p.n_rows);
  *r0 = min(max(__ldg(p.offsets + e), first), end) - first;
  *n = max(min(max(__ldg(p.offsets + e + 1), first), end) - first - *r0, 0);
  return (*n + tokens - 1) / tokens;
}

// The slot-th pass of all experts' (of the one matrix's): expert, first sorted
// row, number of rows; false when there are fewer, their number then in *t0.
// Warp-wide; four experts a lane and step.
__device__ __forceinline__ bool find_pass(const Product& p, int tokens, int slot, int* e, int* t0,
                                          int* n) {
  if (!p.offsets) {
    const int count = (int)((p.n_rows + tokens - 1) / tokens);
    *e = 0;
    if (slot >= count) {
      *t0 = count;
      return false;
    }
    *t0 = slot * tokens;
    *n = min((int)p.n_rows - *t0, tokens);
    return true;
  }
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int e0 = 0; e0 < p.n_experts; e0 += 128) {
    int passes[4], r0[4], rows[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      passes[i] = 0;
      const int x = e0 + 4 * lane + i;
      if (x < p.n_experts) passes[i] = expert_passes(p, x, tokens, &r0[i], &rows[i]);
      mine += passes[i];
    }
    int upto = mine;   // inclusive scan over the lanes
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + upto > slot);
    if (hit) {
      int left = slot - before - (upto - mine), fe = 0, ft = 0, fn = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (left >= 0 && left < passes[i]) {
          fe = e0 + 4 * lane + i;
          ft = r0[i] + left * tokens;
          fn = min(rows[i] - left * tokens, tokens);
        }
        left -= passes[i];
      }
      const int src = __ffs(hit) - 1;
      *e = __shfl_sync(0xffffffffu, fe, src);
      *t0 = __shfl_sync(0xffffffffu, ft, src);
      *n = __shfl_sync(0xffffffffu, fn, src);
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  *t0 = before;
  return false;
}

// Number of passes.  Warp-wide.
__device__ __forceinline__ int count_passes(const Product& p, int tokens) {
  int e, count, n;
  find_pass(p, tokens, 0x7FFFFFFF, &e, &count, &n);
  return count;
}

// Output element (row, o) from the product(s) v.
template <int NW>
__device__ __forceinline__ void write_product(const Product& p, const float* v, int64_t row,
                                              int64_t o) {
  float y = v[0];
  if constexpr (NW == 2) y = v[0] / (1.f + expf(-v[0])) * v[1];
  const int64_t at = row * p.d_out + o;
  if (p.y_bf16)
    static_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(y);
  else
    static_cast<float*>(p.Y)[at] = y;
}

}  // namespace nvfp4
