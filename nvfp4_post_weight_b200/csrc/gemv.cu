// Products of a few tokens with NVFP4 weights as the solve leaves them:
// Y = X Q^T, Q = e2m1(code) * e4m3(scale) * s_g, one matrix or one matrix per
// expert over rows sorted by expert, and the gated pair silu(X Qg^T) * X Qu^T.
#include <cuda_bf16.h>

#include "common.cuh"
#include "nvfp4_format.cuh"

namespace nvfp4 {
namespace {

constexpr int kTok = 8;   // tokens per pass over a weight row

struct ProductArgs {
  const void* X;
  const int* rows;      // X row of each sorted row, or null
  const int* offsets;   // n_experts + 1 row offsets, or null (one matrix)
  const uint8_t* codes[2];
  const uint8_t* scales[2];
  const float* sg[2];
  void* Y;
  int64_t n_x, n_rows, d_out, d_in;
};

template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 2)
    return __bfloat162float(*p);
  else
    return *p;
}

// One warp per output column and matrix, one lane per block of 16 weights.
template <typename TX, typename TY, bool kGlu>
__global__ void __launch_bounds__(256) product_kernel(ProductArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t o = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (o >= a.d_out) return;
  const int64_t e = blockIdx.y;
  int64_t r0 = 0, r1 = a.n_rows;
  if (a.offsets) {
    r0 = min((int64_t)max(a.offsets[e], 0), a.n_rows);
    r1 = min((int64_t)max(a.offsets[e + 1], 0), a.n_rows);
  }
  const int64_t nb = a.d_in / kBlock;
  const int64_t wrow = (e * a.d_out + o) * nb;
  for (int64_t t0 = r0; t0 < r1; t0 += kTok) {
    float acc[kGlu ? 2 : 1][kTok] = {};
    int64_t xr[kTok];
    for (int t = 0; t < kTok; ++t) {
      xr[t] = t0 + t < r1 ? (a.rows ? a.rows[t0 + t] : t0 + t) : -1;
      if (xr[t] >= a.n_x) xr[t] = -1;
    }
    for (int64_t b = lane; b < nb; b += 32) {
      for (int m = 0; m < (kGlu ? 2 : 1); ++m) {
        const uint2 c = reinterpret_cast<const uint2*>(a.codes[m])[wrow + b];
        const uint64_t p = ((uint64_t)c.y << 32) | c.x;
        const float sb = (float)e4m3_value(a.scales[m][wrow + b] & 0x7F);
        for (int j = 0; j < kBlock; ++j) {
          const float w = e2m1_value((uint32_t)(p >> (4 * j)) & 0xF) * sb;
          for (int t = 0; t < kTok; ++t)
            if (xr[t] >= 0)
              acc[m][t] = fmaf(load1(static_cast<const TX*>(a.X) + xr[t] * a.d_in + b * kBlock + j),
                               w, acc[m][t]);
        }
      }
    }
    for (int t = 0; t < kTok; ++t) {
      float v[2];
      for (int m = 0; m < (kGlu ? 2 : 1); ++m) {
        float s = acc[m][t];
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        v[m] = s * a.sg[m][e];
      }
      if (lane == 0 && t0 + t < r1) {
        const float y = kGlu ? v[0] / (1.f + expf(-v[0])) * v[1] : v[0];
        static_cast<TY*>(a.Y)[(t0 + t) * a.d_out + o] = (TY)y;
      }
    }
  }
}

template <typename TX, typename TY>
void launch_typed(const ProductArgs& a, dim3 grid, bool glu, cudaStream_t st) {
  if (glu)
    product_kernel<TX, TY, true><<<grid, 256, 0, st>>>(a);
  else
    product_kernel<TX, TY, false><<<grid, 256, 0, st>>>(a);
}

nvfp4_status launch_product(const ProductArgs& a, nvfp4_dtype xt, nvfp4_dtype yt, int64_t n_experts,
                            bool glu, cudaStream_t st) {
  if (a.n_rows == 0 || a.d_out == 0 || n_experts == 0) return NVFP4_OK;
  ProfileScope ps(kPhaseProduct, st);
  const dim3 grid((unsigned)((a.d_out + 7) / 8), (unsigned)n_experts);
  if (xt == NVFP4_BF16 && yt == NVFP4_BF16)
    launch_typed<__nv_bfloat16, __nv_bfloat16>(a, grid, glu, st);
  else if (xt == NVFP4_BF16)
    launch_typed<__nv_bfloat16, float>(a, grid, glu, st);
  else if (yt == NVFP4_BF16)
    launch_typed<float, __nv_bfloat16>(a, grid, glu, st);
  else
    launch_typed<float, float>(a, grid, glu, st);
  NVFP4_LAUNCH_CHECK();
  count_launches(1);
  return NVFP4_OK;
}

constexpr int64_t kMaxDim = 1 << 17, kMaxRows = 1 << 22;

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_io(nvfp4_dtype t) { return t == NVFP4_BF16 || t == NVFP4_F32; }

struct Matrix {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* sg;
};

// The checks that every product shares, then its launch.  offsets null: one
// matrix, n_x == n_rows.
nvfp4_status product(const void* X, nvfp4_dtype xt, int64_t n_x, const int* rows,
                     const int* offsets, int64_t n_experts, int64_t n_rows, const Matrix* w,
                     int n_w, int64_t d_out, int64_t d_in, void* Y, nvfp4_dtype yt,
                     nvfp4_stream_t stream) {
  if (n_x < 0 || n_rows < 0 || n_experts < 0 || d_out < 0 || d_in < 0) return NVFP4_ERR_INVALID_ARG;
  if (!is_io(xt) || !is_io(yt)) return NVFP4_ERR_INVALID_ARG;
  if (d_in % kBlock || d_in > kMaxDim || d_out > kMaxRows || n_rows > kMaxRows || n_x > kMaxRows ||
      n_experts > NVFP4_MAX_EXPERTS)
    return NVFP4_ERR_SHAPE;
  ProductArgs a{};
  for (int m = 0; m < n_w; ++m) {
    if (n_rows > 0 && d_out > 0 && n_experts > 0 &&
        (!w[m].sg || (d_in > 0 && (!w[m].codes || !w[m].scales))))
      return NVFP4_ERR_INVALID_ARG;
    if (!is_aligned(w[m].codes, 8) || !is_aligned(w[m].sg, 4)) return NVFP4_ERR_INVALID_ARG;
    a.codes[m] = w[m].codes;
    a.scales[m] = w[m].scales;
    a.sg[m] = w[m].sg;
  }
  if (n_rows > 0 && d_out > 0 && n_experts > 0 && (!Y || (n_x > 0 && d_in > 0 && !X)))
    return NVFP4_ERR_INVALID_ARG;
  if (!is_aligned(X, 16) || !is_aligned(Y, yt == NVFP4_BF16 ? 2 : 4) || !is_aligned(rows, 4) ||
      !is_aligned(offsets, 4))
    return NVFP4_ERR_INVALID_ARG;
  a.X = X;
  a.rows = rows;
  a.offsets = offsets;
  a.Y = Y;
  a.n_x = n_x;
  a.n_rows = n_rows;
  a.d_out = d_out;
  a.d_in = d_in;
  return launch_product(a, xt, yt, n_experts, n_w == 2, as_cuda(stream));
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status nvfp4_gemv(const void* X, nvfp4_dtype x_dtype, int64_t n_tok, const uint8_t* codes,
                        const uint8_t* scales, const float* global_scale, int64_t d_out,
                        int64_t d_in, void* Y, nvfp4_dtype y_dtype, nvfp4_stream_t stream) {
  const Matrix w[1] = {{codes, scales, global_scale}};
  return product(X, x_dtype, n_tok, nullptr, nullptr, 1, n_tok, w, 1, d_out, d_in, Y, y_dtype,
                 stream);
}

nvfp4_status nvfp4_gemv_swiglu(const void* X, nvfp4_dtype x_dtype, int64_t n_tok,
                               const uint8_t* gate_codes, const uint8_t* gate_scales,
                               const float* gate_global_scale, const uint8_t* up_codes,
                               const uint8_t* up_scales, const float* up_global_scale,
                               int64_t d_out, int64_t d_in, void* Y, nvfp4_dtype y_dtype,
                               nvfp4_stream_t stream) {
  const Matrix w[2] = {{gate_codes, gate_scales, gate_global_scale},
                       {up_codes, up_scales, up_global_scale}};
  return product(X, x_dtype, n_tok, nullptr, nullptr, 1, n_tok, w, 2, d_out, d_in, Y, y_dtype,
                 stream);
}

nvfp4_status nvfp4_gemv_experts(const void* X, nvfp4_dtype x_dtype, int64_t n_x, const int32_t* rows,
                                const int32_t* offsets, int64_t n_experts, int64_t n_rows,
                                const uint8_t* codes, const uint8_t* scales,
                                const float* global_scales, int64_t d_out, int64_t d_in, void* Y,
                                nvfp4_dtype y_dtype, nvfp4_stream_t stream) {
  if (n_experts > 0 && n_rows > 0 && !offsets) return NVFP4_ERR_INVALID_ARG;
  if (!rows && n_x != n_rows) return NVFP4_ERR_INVALID_ARG;
  const Matrix w[1] = {{codes, scales, global_scales}};
  return product(X, x_dtype, n_x, rows, offsets, n_experts, n_rows, w, 1, d_out, d_in, Y, y_dtype,
                 stream);
}

nvfp4_status nvfp4_gemv_swiglu_experts(
    const void* X, nvfp4_dtype x_dtype, int64_t n_x, const int32_t* rows, const int32_t* offsets,
    int64_t n_experts, int64_t n_rows, const uint8_t* gate_codes, const uint8_t* gate_scales,
    const float* gate_global_scales, const uint8_t* up_codes, const uint8_t* up_scales,
    const float* up_global_scales, int64_t d_out, int64_t d_in, void* Y, nvfp4_dtype y_dtype,
    nvfp4_stream_t stream) {
  if (n_experts > 0 && n_rows > 0 && !offsets) return NVFP4_ERR_INVALID_ARG;
  if (!rows && n_x != n_rows) return NVFP4_ERR_INVALID_ARG;
  const Matrix w[2] = {{gate_codes, gate_scales, gate_global_scales},
                       {up_codes, up_scales, up_global_scales}};
  return product(X, x_dtype, n_x, rows, offsets, n_experts, n_rows, w, 2, d_out, d_in, Y, y_dtype,
                 stream);
}

}  // extern "C"
