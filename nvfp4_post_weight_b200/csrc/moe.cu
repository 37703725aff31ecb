// Tokens sorted by expert and back: a stable counting sort of the routing
// slots, the gather of token rows into expert order, the weighted sum of the
// experts' rows per token, and its gradient.
//
// A slot s = t * top_k + j is token t's j-th choice; `position` holds each
// slot's row in expert order, or -1 for a slot without an expert.  Every
// kernel but the sort goes by slots, so that a token's row is read once and
// every sorted row is read or written by one warp: no atomics, and the result
// does not depend on the order of the CTAs.
#include <cuda_bf16.h>

#include "common.cuh"

namespace nvfp4 {
namespace {

// ---- the sort ----------------------------------------------------------------
constexpr int kSortWarps = 16;
constexpr int kSortChunk = 4096;    // slots per CTA; at least NVFP4_MAX_EXPERTS
constexpr int kSortMaxChunks = 512; // longer inputs take longer chunks
static_assert(kSortChunk >= NVFP4_MAX_EXPERTS, "a chunk's counts lie in its own positions");

// Expert of slot s, or n_experts for a slot without one.
__device__ __forceinline__ int slot_expert(const void* ids, int wide, int64_t s, int n_experts) {
  if (wide) {
    const int64_t v = static_cast<const int64_t*>(ids)[s];
    return v < 0 || v >= n_experts ? n_experts : (int)v;
  }
  const int v = static_cast<const int32_t*>(ids)[s];
  return v < 0 || v >= n_experts ? n_experts : v;
}

// Counts of one warp's slots [s0, s1) per expert into cnt (shared, zeroed);
// kWrite: cnt holds the row where the warp's first slot of each expert goes,
// and every slot's position and its row's token are written instead.
template <bool kWrite>
__device__ __forceinline__ void warp_slots(const void* ids, int wide, int64_t s0, int64_t s1,
                                           int n_experts, int top_k, int* cnt, int32_t* rows,
                                           int32_t* position) {
  const int lane = threadIdx.x & 31;
  for (int64_t b = s0; b < s1; b += 32) {
    const int64_t s = b + lane;
    const int e = s < s1 ? slot_expert(ids, wide, s, n_experts) : n_experts;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int before = __popc(same & ((1u << lane) - 1));
    int base = 0;
    if (e < n_experts) base = cnt[e];
    __syncwarp();
    if (e < n_experts && before == 0) cnt[e] = base + __popc(same);
    __syncwarp();
    if (kWrite && s < s1) {
      if (e < n_experts) {
        position[s] = base + before;
        rows[base + before] = (int32_t)(s / top_k);
      } else {
        position[s] = -1;
      }
    }
  }
}

// Slots [s0, s1) of one CTA, shared out over its warps in order.
__device__ __forceinline__ void warp_range(int64_t s0, int64_t s1, int64_t* w0, int64_t* w1) {
  const int64_t per = ((s1 - s0 + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int w = threadIdx.x >> 5;
  *w0 = min(s0 + w * per, s1);
  *w1 = min(*w0 + per, s1);
}

__device__ __forceinline__ void chunk_range(int64_t n, int64_t chunk, int n_chunks, int c,
                                            int64_t* s0, int64_t* s1) {
  *s0 = c * chunk;
  *s1 = c + 1 == n_chunks ? n : *s0 + chunk;   // the last chunk takes the remainder
}

// Inclusive scan of v over the CTA's kSortWarps * 32 threads.
__device__ __forceinline__ int cta_scan(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  if (w == 0) {
    int t = lane < kSortWarps ? warp_sums[lane] : 0;
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += u;
    }
    if (lane < kSortWarps) warp_sums[lane] = t;
  }
  __syncthreads();
  if (w > 0) v += warp_sums[w - 1];
  __syncthreads();
  return v;
}

// Turns the warps' counts cnt[w][e] into each warp's first row of each expert
// given the CTA's first row of it (first[e]).
__device__ __forceinline__ void counts_to_rows(int* cnt, int n_experts, const int* first) {
  for (int e = threadIdx.x; e < n_experts; e += blockDim.x) {
    int r = first[e];
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w * n_experts + e];
      cnt[w * n_experts + e] = r;
      r += c;
    }
  }
}

// Offsets of the experts from their totals (tot, shared; replaced by each
// expert's first row); every thread of the CTA takes two neighbours.
__device__ __forceinline__ void scan_totals(int* tot, int n_experts, int* warp_sums,
                                            int32_t* offsets) {
  const int e = 2 * threadIdx.x;
  const int a = e < n_experts ? tot[e] : 0, b = e + 1 < n_experts ? tot[e + 1] : 0;
  const int end = cta_scan(a + b, warp_sums);
  if (e < n_experts) {
    tot[e] = end - a - b;
    offsets[e + 1] = end - b;
  }
  if (e + 1 < n_experts) {
    tot[e + 1] = end - b;
    offsets[e + 2] = end;
  }
  if (threadIdx.x == 0) offsets[0] = 0;
  __syncthreads();
}

// All slots in one CTA.
__global__ void __launch_bounds__(kSortWarps * 32)
    sort_small_kernel(const void* ids, int wide, int64_t n, int n_experts, int top_k,
                      int32_t* offsets, int32_t* rows, int32_t* position) {
  extern __shared__ int cnt[];   // kSortWarps x n_experts counts, then n_experts totals
  __shared__ int warp_sums[32];
  int* tot = cnt + kSortWarps * n_experts;
  for (int i = threadIdx.x; i < kSortWarps * n_experts; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  int64_t w0, w1;
  warp_range(0, n, &w0, &w1);
  int* mine = cnt + (threadIdx.x >> 5) * n_experts;
  warp_slots<false>(ids, wide, w0, w1, n_experts, top_k, mine, nullptr, nullptr);
  __syncthreads();
  for (int e = threadIdx.x; e < n_experts; e += blockDim.x) {
    int s = 0;
    for (int w = 0; w < kSortWarps; ++w) s += cnt[w * n_experts + e];
    tot[e] = s;
  }
  __syncthreads();
  scan_totals(tot, n_experts, warp_sums, offsets);
  counts_to_rows(cnt, n_experts, tot);
  __syncthreads();
  warp_slots<true>(ids, wide, w0, w1, n_experts, top_k, mine, rows, position);
  // the rows behind the last expert's (the CTA's own write, read after a barrier)
  const int64_t kept = n_experts > 0 ? offsets[n_experts] : 0;
  for (int64_t r = kept + threadIdx.x; r < n; r += blockDim.x) rows[r] = -1;
}

// Long inputs: the chunks' counts, kept in the first n_experts positions of
// each chunk until its own CTA of the last kernel replaces them.
__global__ void __launch_bounds__(kSortWarps * 32)
    sort_count_kernel(const void* ids, int wide, int64_t n, int64_t chunk, int n_experts,
                      int32_t* position) {
  extern __shared__ int cnt[];
  for (int i = threadIdx.x; i < kSortWarps * n_experts; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  int64_t s0, s1, w0, w1;
  chunk_range(n, chunk, gridDim.x, blockIdx.x, &s0, &s1);
  warp_range(s0, s1, &w0, &w1);
  warp_slots<false>(ids, wide, w0, w1, n_experts, 1, cnt + (threadIdx.x >> 5) * n_experts, nullptr,
                    nullptr);
  __syncthreads();
  for (int e = threadIdx.x; e < n_experts; e += blockDim.x) {
    int s = 0;
    for (int w = 0; w < kSortWarps; ++w) s += cnt[w * n_experts + e];
    position[s0 + e] = s;
  }
}

// One CTA: chunk counts -> each chunk's first row of each expert, and offsets.
__global__ void __launch_bounds__(kSortWarps * 32)
    sort_scan_kernel(int64_t chunk, int n_chunks, int n_experts, int32_t* offsets,
                     int32_t* position) {
  extern __shared__ int tot[];
  __shared__ int warp_sums[32];
  pdl_wait();
  for (int e = threadIdx.x; e < n_experts; e += blockDim.x) {
    int s = 0;
#pragma unroll 8
    for (int c = 0; c < n_chunks; ++c) s += position[c * chunk + e];
    tot[e] = s;
  }
  __syncthreads();
  scan_totals(tot, n_experts, warp_sums, offsets);
  for (int e = threadIdx.x; e < n_experts; e += blockDim.x) {
    int r = tot[e];
#pragma unroll 8
    for (int c = 0; c < n_chunks; ++c) {
      const int v = position[c * chunk + e];
      position[c * chunk + e] = r;
      r += v;
    }
  }
}

__global__ void __launch_bounds__(kSortWarps * 32)
    sort_place_kernel(const void* ids, int wide, int64_t n, int64_t chunk, int n_experts, int top_k,
                      const int32_t* offsets, int32_t* rows, int32_t* position) {
  extern __shared__ int cnt[];
  int* first = cnt + kSortWarps * n_experts;
  for (int i = threadIdx.x; i < kSortWarps * n_experts; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  int64_t s0, s1, w0, w1;
  chunk_range(n, chunk, gridDim.x, blockIdx.x, &s0, &s1);
  warp_range(s0, s1, &w0, &w1);
  int* mine = cnt + (threadIdx.x >> 5) * n_experts;
  warp_slots<false>(ids, wide, w0, w1, n_experts, top_k, mine, nullptr, nullptr);
  pdl_wait();
  for (int e = threadIdx.x; e < n_experts; e += blockDim.x) first[e] = position[s0 + e];
  __syncthreads();   // every thread has its counts: the positions may be written
  counts_to_rows(cnt, n_experts, first);
  __syncthreads();
  warp_slots<true>(ids, wide, w0, w1, n_experts, top_k, mine, rows, position);
  const int64_t kept = offsets[n_experts];
  for (int64_t r = kept + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < n;
       r += (int64_t)gridDim.x * blockDim.x)
    rows[r] = -1;
}

// ---- rows there and back -------------------------------------------------------
// V elements of T at p (V * sizeof(T) bytes, aligned to that), as floats.
template <typename T, int V>
struct Vec {
  alignas(sizeof(T) * V) T v[V];
};

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Token blockIdx.x's row to the sorted rows of its slots: one read, top_k writes.
template <typename T>   // T: the bytes one thread moves
__global__ void __launch_bounds__(256)
    gather_kernel(const T* __restrict__ X, const int32_t* __restrict__ position, int top_k,
                  int64_t n_slots, int64_t cols, T* __restrict__ Xs) {
  const int64_t t = blockIdx.x;
  for (int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; c < cols;
       c += (int64_t)gridDim.y * blockDim.x) {
    const T v = X[t * cols + c];
    for (int j = 0; j < top_k; ++j) {
      const int64_t p = position[t * top_k + j];
      if (p >= 0 && p < n_slots) Xs[p * cols + c] = v;
    }
  }
}

// Y[t] = sum_j w[t, j] Ys[position[t, j]] in fp32, j ascending; one rounding.
template <typename TS, typename TY, int V>
__global__ void __launch_bounds__(256)
    combine_kernel(const TS* __restrict__ Ys, const int32_t* __restrict__ position,
                   const float* __restrict__ weights, int top_k, int64_t n_slots, int64_t d,
                   TY* __restrict__ Y) {
  const int64_t t = blockIdx.x;
  for (int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V; c < d;
       c += (int64_t)gridDim.y * blockDim.x * V) {
    float acc[V] = {};
#pragma unroll 4
    for (int j = 0; j < top_k; ++j) {
      const int64_t p = position[t * top_k + j];
      if (p < 0 || p >= n_slots) continue;
      const float w = weights ? weights[t * top_k + j] : 1.f;
      const Vec<TS, V> y = *reinterpret_cast<const Vec<TS, V>*>(Ys + p * d + c);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(w, as_f32(y.v[i]), acc[i]);
    }
    Vec<TY, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.v[i] = (TY)acc[i];
    *reinterpret_cast<Vec<TY, V>*>(Y + t * d + c) = o;
  }
}

// One warp per slot: dYs[p] = w dY[t], dw = <dY[t], Ys[p]> (fp32).
template <typename T, int V>
__global__ void __launch_bounds__(256)
    combine_backward_kernel(const T* __restrict__ dY, const T* __restrict__ Ys,
                            const int32_t* __restrict__ position,
                            const float* __restrict__ weights, int top_k, int64_t n_slots,
                            int64_t d, T* __restrict__ dYs, float* __restrict__ dweights) {
  const int lane = threadIdx.x & 31;
  const int64_t s = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (s >= n_slots) return;
  const int64_t p = position[s];
  float dot = 0.f;
  if (p >= 0 && p < n_slots) {
    const float w = weights[s];
    const int64_t t = s / top_k;
#pragma unroll 4
    for (int64_t c = (int64_t)lane * V; c < d; c += 32 * V) {
      const Vec<T, V> g = *reinterpret_cast<const Vec<T, V>*>(dY + t * d + c);
      const Vec<T, V> y = *reinterpret_cast<const Vec<T, V>*>(Ys + p * d + c);
      Vec<T, V> o;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float gi = as_f32(g.v[i]);
        dot = fmaf(gi, as_f32(y.v[i]), dot);
        o.v[i] = (T)(w * gi);
      }
      *reinterpret_cast<Vec<T, V>*>(dYs + p * d + c) = o;
    }
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  }
  if (lane == 0) dweights[s] = dot;
}

constexpr int64_t kMaxDim = 1 << 17, kMaxTokens = 1 << 26, kMaxSlots = 1 << 30;

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_io(nvfp4_dtype t) { return t == NVFP4_BF16 || t == NVFP4_F32; }
size_t io_size(nvfp4_dtype t) { return t == NVFP4_BF16 ? 2 : 4; }

nvfp4_status check_slots(int64_t n_tok, int64_t top_k) {
  if (n_tok < 0 || top_k < 1) return NVFP4_ERR_INVALID_ARG;
  if (n_tok > kMaxTokens || top_k > NVFP4_MAX_EXPERTS || n_tok * top_k > kMaxSlots)
    return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

// CTAs along the columns: one per 256 threads' worth, at most 8 (a token's CTAs
// all read its positions).
unsigned col_blocks(int64_t items) {
  const int64_t b = (items + 255) / 256;
  return (unsigned)(b < 1 ? 1 : b > 8 ? 8 : b);
}

template <typename TS, typename TY, int V>
void launch_combine(const void* Ys, const int32_t* pos, const float* w, int64_t n_tok, int top_k,
                    int64_t d, void* Y, cudaStream_t st) {
  const dim3 grid((unsigned)n_tok, col_blocks((d + V - 1) / V));
  combine_kernel<TS, TY, V><<<grid, 256, 0, st>>>(static_cast<const TS*>(Ys), pos, w, top_k,
                                                  n_tok * top_k, d, static_cast<TY*>(Y));
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status nvfp4_moe_sort(const void* expert_ids, int id_bytes, int64_t n_tok, int64_t top_k,
                            int64_t n_experts, int32_t* offsets, int32_t* rows, int32_t* position,
                            nvfp4_stream_t stream) {
  if (n_experts < 0 || !offsets || (id_bytes != 4 && id_bytes != 8)) return NVFP4_ERR_INVALID_ARG;
  if (nvfp4_status s = check_slots(n_tok, top_k)) return s;
  if (n_experts > NVFP4_MAX_EXPERTS) return NVFP4_ERR_SHAPE;
  const int64_t n = n_tok * top_k;
  if (n > 0 && (!expert_ids || !rows || !position)) return NVFP4_ERR_INVALID_ARG;
  if (!is_aligned(expert_ids, id_bytes) || !is_aligned(offsets, 4) || !is_aligned(rows, 4) ||
      !is_aligned(position, 4))
    return NVFP4_ERR_INVALID_ARG;
  cudaStream_t st = as_cuda(stream);
  ProfileScope ps(kPhaseRoute, st);
  const int E = (int)n_experts, wide = id_bytes == 8, k = (int)top_k;
  const size_t smem = sizeof(int) * (kSortWarps + 1) * (size_t)E;
  const dim3 block(kSortWarps * 32);
  static_assert(sizeof(int) * (kSortWarps + 1) * NVFP4_MAX_EXPERTS <= 227 * 1024, "shared memory");
  if (smem > 48 * 1024) {
    // (per device and kernel; setting it again is harmless)
    NVFP4_CUDA_TRY(cudaFuncSetAttribute(sort_small_kernel,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    NVFP4_CUDA_TRY(cudaFuncSetAttribute(sort_count_kernel,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    NVFP4_CUDA_TRY(cudaFuncSetAttribute(sort_place_kernel,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  }
  if (n < 2 * kSortChunk || E == 0) {
    sort_small_kernel<<<1, block, smem, st>>>(expert_ids, wide, n, E, k, offsets, rows, position);
    NVFP4_LAUNCH_CHECK();
    count_launches(1);
    return NVFP4_OK;
  }
  int64_t chunk = (n + kSortMaxChunks - 1) / kSortMaxChunks;
  if (chunk < kSortChunk) chunk = kSortChunk;
  const int n_chunks = (int)(n / chunk);
  sort_count_kernel<<<n_chunks, block, smem, st>>>(expert_ids, wide, n, chunk, E, position);
  NVFP4_LAUNCH_CHECK();
  NVFP4_CUDA_TRY(launch_chained(sort_scan_kernel, dim3(1), block, sizeof(int) * E, st, chunk,
                                n_chunks, E, offsets, position));
  NVFP4_CUDA_TRY(launch_chained(sort_place_kernel, dim3(n_chunks), block, smem, st, expert_ids, wide,
                                n, chunk, E, k, (const int32_t*)offsets, rows, position));
  count_launches(3);
  return NVFP4_OK;
}

nvfp4_status nvfp4_moe_gather(const void* X, nvfp4_dtype dtype, const int32_t* position,
                              int64_t n_tok, int64_t top_k, int64_t d, void* Xs,
                              nvfp4_stream_t stream) {
  if (d < 0 || !is_io(dtype)) return NVFP4_ERR_INVALID_ARG;
  if (nvfp4_status s = check_slots(n_tok, top_k)) return s;
  if (d > kMaxDim) return NVFP4_ERR_SHAPE;
  if (n_tok == 0 || d == 0) return NVFP4_OK;
  const size_t size = io_size(dtype), row = size * d;
  if (!X || !position || !Xs || !is_aligned(X, size) || !is_aligned(Xs, size) ||
      !is_aligned(position, 4))
    return NVFP4_ERR_INVALID_ARG;
  cudaStream_t st = as_cuda(stream);
  ProfileScope ps(kPhaseRoute, st);
  const uintptr_t all = reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(Xs) | row;
  const int64_t n = n_tok * top_k;
  // the widest access that the rows' length and the bases allow
  if (all % 16 == 0)
    gather_kernel<uint4><<<dim3((unsigned)n_tok, col_blocks(row / 16)), 256, 0, st>>>(
        static_cast<const uint4*>(X), position, (int)top_k, n, row / 16, static_cast<uint4*>(Xs));
  else if (all % 4 == 0)
    gather_kernel<uint32_t><<<dim3((unsigned)n_tok, col_blocks(row / 4)), 256, 0, st>>>(
        static_cast<const uint32_t*>(X), position, (int)top_k, n, row / 4,
        static_cast<uint32_t*>(Xs));
  else
    gather_kernel<uint16_t><<<dim3((unsigned)n_tok, col_blocks(row / 2)), 256, 0, st>>>(
        static_cast<const uint16_t*>(X), position, (int)top_k, n, row / 2,
        static_cast<uint16_t*>(Xs));
  NVFP4_LAUNCH_CHECK();
  count_launches(1);
  return NVFP4_OK;
}

nvfp4_status nvfp4_moe_combine(const void* Ys, nvfp4_dtype s_dtype, const int32_t* position,
                               const float* weights, int64_t n_tok, int64_t top_k, int64_t d,
                               void* Y, nvfp4_dtype y_dtype, nvfp4_stream_t stream) {
  if (d < 0 || !is_io(s_dtype) || !is_io(y_dtype)) return NVFP4_ERR_INVALID_ARG;
  if (nvfp4_status s = check_slots(n_tok, top_k)) return s;
  if (d > kMaxDim) return NVFP4_ERR_SHAPE;
  if (n_tok == 0 || d == 0) return NVFP4_OK;
  const size_t ss = io_size(s_dtype), ys = io_size(y_dtype);
  if (!Ys || !position || !Y || !is_aligned(Ys, ss) || !is_aligned(Y, ys) ||
      !is_aligned(position, 4) || !is_aligned(weights, 4))
    return NVFP4_ERR_INVALID_ARG;
  cudaStream_t st = as_cuda(stream);
  ProfileScope ps(kPhaseRoute, st);
  // 8 (bf16) or 4 columns a thread where every row of both sides starts aligned for it
  const bool vec = d % 8 == 0 && is_aligned(Ys, 16) && is_aligned(Y, 16);
  const int k = (int)top_k;
#define NVFP4_COMBINE(TS, TY, V)                                                            \
  (vec ? launch_combine<TS, TY, V>(Ys, position, weights, n_tok, k, d, Y, st)               \
       : launch_combine<TS, TY, 1>(Ys, position, weights, n_tok, k, d, Y, st))
  if (s_dtype == NVFP4_BF16 && y_dtype == NVFP4_BF16)
    NVFP4_COMBINE(__nv_bfloat16, __nv_bfloat16, 8);
  else if (s_dtype == NVFP4_BF16)
    NVFP4_COMBINE(__nv_bfloat16, float, 4);
  else if (y_dtype == NVFP4_BF16)
    NVFP4_COMBINE(float, __nv_bfloat16, 4);
  else
    NVFP4_COMBINE(float, float, 4);
#undef NVFP4_COMBINE
  NVFP4_LAUNCH_CHECK();
  count_launches(1);
  return NVFP4_OK;
}

nvfp4_status nvfp4_moe_combine_backward(const void* dY, const void* Ys, nvfp4_dtype dtype,
                                        const int32_t* position, const float* weights,
                                        int64_t n_tok, int64_t top_k, int64_t d, void* dYs,
                                        float* dweights, nvfp4_stream_t stream) {
  if (d < 0 || !is_io(dtype)) return NVFP4_ERR_INVALID_ARG;
  if (nvfp4_status s = check_slots(n_tok, top_k)) return s;
  if (d > kMaxDim) return NVFP4_ERR_SHAPE;
  if (n_tok == 0) return NVFP4_OK;
  const size_t size = io_size(dtype);
  if (!position || !weights || !dweights || (d > 0 && (!dY || !Ys || !dYs)) ||
      !is_aligned(dY, size) || !is_aligned(Ys, size) || !is_aligned(dYs, size) ||
      !is_aligned(position, 4) || !is_aligned(weights, 4) || !is_aligned(dweights, 4))
    return NVFP4_ERR_INVALID_ARG;
  cudaStream_t st = as_cuda(stream);
  ProfileScope ps(kPhaseRoute, st);
  const int64_t n = n_tok * top_k;
  const unsigned grid = (unsigned)((n + 7) / 8);
  const bool vec = (size * d) % 16 == 0 && is_aligned(dY, 16) && is_aligned(Ys, 16) &&
                   is_aligned(dYs, 16);
#define NVFP4_BACKWARD(T, V)                                                                     \
  combine_backward_kernel<T, V><<<grid, 256, 0, st>>>(                                           \
      static_cast<const T*>(dY), static_cast<const T*>(Ys), position, weights, (int)top_k, n, d, \
      static_cast<T*>(dYs), dweights)
  if (dtype == NVFP4_BF16) {
    if (vec)
      NVFP4_BACKWARD(__nv_bfloat16, 8);
    else
      NVFP4_BACKWARD(__nv_bfloat16, 1);
  } else {
    if (vec)
      NVFP4_BACKWARD(float, 4);
    else
      NVFP4_BACKWARD(float, 1);
  }
#undef NVFP4_BACKWARD
  NVFP4_LAUNCH_CHECK();
  count_launches(1);
  return NVFP4_OK;
}

}  // extern "C"
