// Tokens sorted by expert and back: a stable counting sort of the routing
// slots, the gather of token rows into expert order, the weighted sum of the
// experts' rows per token, and its gradient.
//
// A slot s = t * top_k + j is token t's j-th choice; `position` holds each
// slot's row in expert order, or -1 for a slot without an expert.  Every
// kernel but the sort goes by slots, so that a token's row is read once and
// every sorted row is read or written by one warp or one column's thread: no
// global atomics, and the result does not depend on the order of the CTAs.
//
// All of it is bound by DRAM bytes where there are many tokens (8192 x 8 slots, 3%
// of them empty, rows of 4096 bf16: the sort 8 us, the gather 99 us and the weighted
// sum 88 us for 587 MB each, its gradient 170 us for 1.11 GB: 5.9 to 6.7 TB/s), by
// launches and one or two memory latencies where there are few (64 x 8: the sort 3
// us, the gather 2.4, the sum 2.4).
#include <cuda_bf16.h>

#include "common.cuh"

namespace nvfp4 {
namespace {

NVFP4_CHECK_WORD(g_check);

// ---- the sort ----------------------------------------------------------------
// Placing a warp's 32 slots in order takes about 60 cycles of its SM (the warp's
// match and the counters), counting them by shared atomics less.  Up to 4096 slots
// one CTA does both in one launch (512 slots: 3 us); longer inputs go over as
// many CTAs as have 1024 slots, in three launches (65536 slots: 8 us; one CTA
// took 125 us).
constexpr int kSortWarps = 32;
constexpr int kSortOneCta = 4096;   // slots that one CTA sorts by itself
constexpr int kSortChunk = 1024;    // least slots per CTA beyond; at least NVFP4_MAX_EXPERTS
constexpr int kSortMaxChunks = 128;
static_assert(kSortChunk >= NVFP4_MAX_EXPERTS, "a chunk's counts lie in its own positions");
static_assert(kSortWarps * 32 >= NVFP4_MAX_EXPERTS, "a thread per expert");

// Expert of slot s, or n_experts for a slot without one.
__device__ __forceinline__ int slot_expert(const void* ids, int wide, int64_t s, int n_experts) {
  if (wide) {
    const int64_t v = static_cast<const int64_t*>(ids)[s];
    return v < 0 || v >= n_experts ? n_experts : (int)v;
  }
  const int v = static_cast<const int32_t*>(ids)[s];
  return v < 0 || v >= n_experts ? n_experts : v;
}

// Adds one warp's slots [s0, s1) per expert to cnt (shared).
__device__ __forceinline__ void count_slots(const void* ids, int wide, int64_t s0, int64_t s1,
                                            int n_experts, int* cnt) {
#pragma unroll 4
  for (int64_t s = s0 + (threadIdx.x & 31); s < s1; s += 32) {
    const int e = slot_expert(ids, wide, s, n_experts);
    if (e < n_experts) atomicAdd(cnt + e, 1);
  }
}

// Gives one warp's slots [s0, s1) their rows in order: next (shared) holds the
// row where the warp's next slot of each expert goes.
__device__ __forceinline__ void place_slots(const void* ids, int wide, int64_t s0, int64_t s1,
                                            int64_t n, int n_experts, int top_k, int* next,
                                            int32_t* rows, int32_t* position) {
  const int lane = threadIdx.x & 31;
  for (int64_t b = s0; b < s1; b += 32) {
    const int64_t s = b + lane;
    const int e = s < s1 ? slot_expert(ids, wide, s, n_experts) : n_experts;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int before = __popc(same & ((1u << lane) - 1));
    int r = -1;
    if (e < n_experts) r = next[e] + before;
    __syncwarp();
    if (e < n_experts && before == 0) next[e] = r + __popc(same);
    __syncwarp();
    if (s < s1 && NVFP4_DCHECK(s >= 0 && s < n && r < n, &g_check)) {
      position[s] = r;
      if (r >= 0) rows[r] = (int32_t)(s / top_k);
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
    int t = warp_sums[lane];
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += u;
    }
    warp_sums[lane] = t;
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
// expert's first row).
__device__ __forceinline__ void scan_totals(int* tot, int n_experts, int* warp_sums,
                                            int32_t* offsets) {
  const int e = threadIdx.x, n = e < n_experts ? tot[e] : 0;
  const int end = cta_scan(n, warp_sums);
  if (e < n_experts) {
    tot[e] = end - n;
    offsets[e + 1] = end;
  }
  if (e == 0) offsets[0] = 0;
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
  count_slots(ids, wide, w0, w1, n_experts, mine);
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
  place_slots(ids, wide, w0, w1, n, n_experts, top_k, mine, rows, position);
  // the rows behind the last expert's (the CTA's own write, read after a barrier)
  const int64_t kept = n_experts > 0 ? offsets[n_experts] : 0;
  if (!NVFP4_DCHECK(kept >= 0 && kept <= n, &g_check)) return;
  for (int64_t r = kept + threadIdx.x; r < n; r += blockDim.x) rows[r] = -1;
}

// Long inputs: the chunks' counts, kept in the first n_experts positions of
// each chunk until its own CTA of the last kernel replaces them.
__global__ void __launch_bounds__(kSortWarps * 32)
    sort_count_kernel(const void* ids, int wide, int64_t n, int64_t chunk, int n_experts,
                      int32_t* position) {
  extern __shared__ int cnt[];   // n_experts
  for (int i = threadIdx.x; i < n_experts; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  int64_t s0, s1, w0, w1;
  chunk_range(n, chunk, gridDim.x, blockIdx.x, &s0, &s1);
  warp_range(s0, s1, &w0, &w1);
  count_slots(ids, wide, w0, w1, n_experts, cnt);
  __syncthreads();
  for (int e = threadIdx.x; e < n_experts; e += blockDim.x)
    if (NVFP4_DCHECK(s0 + e < s1 && s1 <= n, &g_check)) position[s0 + e] = cnt[e];
}

// One CTA: chunk counts -> each chunk's first row of each expert, and offsets.
// parts threads share an expert's chunks.
__global__ void __launch_bounds__(kSortWarps * 32)
    sort_scan_kernel(int64_t chunk, int n_chunks, int n_experts, int parts, int32_t* offsets,
                     int32_t* position) {
  extern __shared__ int sums[];   // parts x n_experts, then n_experts totals
  __shared__ int warp_sums[32];
  int* tot = sums + parts * n_experts;
  pdl_wait();
  const int e = threadIdx.x % n_experts, part = threadIdx.x / n_experts;
  const int per = (n_chunks + parts - 1) / parts;
  const int c0 = min(part * per, n_chunks);
  int c1 = part < parts ? min(c0 + per, n_chunks) : c0;
  if (!NVFP4_DCHECK(n_experts <= chunk && c1 <= n_chunks, &g_check)) c1 = c0;
  int s = 0;
#pragma unroll 8
  for (int c = c0; c < c1; ++c) s += position[c * chunk + e];
  if (part < parts) sums[threadIdx.x] = s;
  __syncthreads();
  if (part == 0) {
    int t = 0;
    for (int p = 0; p < parts; ++p) t += sums[p * n_experts + e];
    tot[e] = t;
  }
  __syncthreads();
  scan_totals(tot, n_experts, warp_sums, offsets);
  int r = tot[e];
  for (int p = 0; p < part && p < parts; ++p) r += sums[p * n_experts + e];
#pragma unroll 8
  for (int c = c0; c < c1; ++c) {
    const int v = position[c * chunk + e];
    position[c * chunk + e] = r;
    r += v;
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
  count_slots(ids, wide, w0, w1, n_experts, mine);
  pdl_wait();
  for (int e = threadIdx.x; e < n_experts; e += blockDim.x)
    if (NVFP4_DCHECK(s0 + e < s1 && s1 <= n, &g_check)) first[e] = position[s0 + e];
  __syncthreads();   // every thread has its counts: the positions may be written
  counts_to_rows(cnt, n_experts, first);
  __syncthreads();
  place_slots(ids, wide, w0, w1, n, n_experts, top_k, mine, rows, position);
  const int64_t kept = offsets[n_experts];
  if (!NVFP4_DCHECK(kept >= 0 && kept <= n, &g_check)) return;
  for (int64_t r = kept + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < n;
       r += (int64_t)gridDim.x * blockDim.x)
    rows[r] = -1;
}

// ---- rows there and back -------------------------------------------------------
// V elements of a row: consecutive ones in one access where every row starts on
// its boundary (kVec), else V elements one thread of 256 (32) apart, so that a
// warp's accesses stay whole and V of them are in flight either way.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};
template <typename T, int V, bool kVec, int kApart>
__device__ __forceinline__ void load_row(const T* row, int64_t c, int64_t d, T* v) {
  if (kVec) {
    *reinterpret_cast<Vec<T, V>*>(v) = *reinterpret_cast<const Vec<T, V>*>(row + c);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i * kApart < d) v[i] = row[c + i * kApart];
  }
}
template <typename T, int V, bool kVec, int kApart>
__device__ __forceinline__ void store_row(T* row, int64_t c, int64_t d, const T* v) {
  if (kVec) {
    *reinterpret_cast<Vec<T, V>*>(row + c) = *reinterpret_cast<const Vec<T, V>*>(v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i * kApart < d) row[c + i * kApart] = v[i];
  }
}
// First of the V columns of thread t of `threads` in block b of V * threads.
template <int V, bool kVec>
__device__ __forceinline__ int64_t first_column(int64_t b, int t, int threads) {
  return b * V * threads + (kVec ? t * V : t);
}

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// V elements of a row, held until they are used.  Of one access: as 32-bit words (as
// arrays of bf16 they do not stay in registers: 8192 x 8 rows of 4096 took 108 us to
// add up, 88 us so).
template <typename T, int V, bool kVec>
struct alignas(sizeof(T) * V) Held {
  uint32_t w[V * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T* row, int64_t c, int64_t) {
    *this = *reinterpret_cast<const Held*>(row + c);
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};
template <typename T, int V>
struct Held<T, V, false> {
  T v[V];
  __device__ __forceinline__ void load(const T* row, int64_t c, int64_t d) {
    load_row<T, V, false, 256>(row, c, d, v);
  }
  __device__ __forceinline__ float operator[](int i) const { return as_f32(v[i]); }
};

// Token blockIdx.x's row to the sorted rows of its slots: one read, top_k writes.
template <typename T, int V, bool kVec>
__global__ void __launch_bounds__(256)
    gather_kernel(const T* __restrict__ X, const int32_t* __restrict__ position, int top_k,
                  int64_t n_slots, int64_t d, T* __restrict__ Xs) {
  const int64_t t = blockIdx.x;
  for (int64_t b = blockIdx.y; b * V * 256 < d; b += gridDim.y) {
    const int64_t c = first_column<V, kVec>(b, threadIdx.x, 256);
    if (c >= d) break;
    alignas(16) T v[V];
    if (!NVFP4_DCHECK((t + 1) * top_k <= n_slots && (!kVec || c + V <= d), &g_check)) break;
    load_row<T, V, kVec, 256>(X + t * d, c, d, v);
    for (int j = 0; j < top_k; ++j) {
      const int64_t p = position[t * top_k + j];
      if (p >= 0 && p < n_slots && NVFP4_DCHECK(!kVec || c + V <= d, &g_check))
        store_row<T, V, kVec, 256>(Xs + p * d, c, d, v);
    }
  }
}

// Y[t] = sum_j w[t, j] Ys[position[t, j]] in fp32, j ascending; one rounding.
template <typename TS, typename TY, int V, bool kVec>
__global__ void __launch_bounds__(256)
    combine_kernel(const TS* __restrict__ Ys, const int32_t* __restrict__ position,
                   const float* __restrict__ weights, int top_k, int64_t n_slots, int64_t d,
                   TY* __restrict__ Y) {
  constexpr int kAhead = sizeof(TS) == 4 ? 8 : 4;   // 32 registers of rows
  const int64_t t = blockIdx.x;
  for (int64_t b = blockIdx.y; b * V * 256 < d; b += gridDim.y) {
    const int64_t c = first_column<V, kVec>(b, threadIdx.x, 256);
    if (c >= d) break;
    float acc[V] = {};
    for (int j0 = 0; j0 < top_k; j0 += kAhead) {
      int64_t p[kAhead];
      Held<TS, V, kVec> y[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        p[j] = j0 + j < top_k ? position[t * top_k + j0 + j] : -1;
        if (p[j] >= n_slots) p[j] = -1;
        if (kVec) y[j] = {};   // (else the loads wait for the positions: 92 us)
        if (!NVFP4_DCHECK(!kVec || c + V <= d, &g_check)) p[j] = -1;
        if (p[j] >= 0) y[j].load(Ys + p[j] * d, c, d);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (p[j] < 0) continue;
        const float w = weights ? weights[t * top_k + j0 + j] : 1.f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(w, y[j][i], acc[i]);
      }
    }
    alignas(16) TY o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = (TY)acc[i];
    if (NVFP4_DCHECK((t + 1) * top_k <= n_slots && (!kVec || c + V <= d), &g_check))
      store_row<TY, V, kVec, 256>(Y + t * d, c, d, o);
  }
}

// One warp per slot: dYs[p] = w dY[t], dw = <dY[t], Ys[p]> (fp32).
template <typename T, int V, bool kVec>
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
    // (columns of one step lie in each row V at a time, or 32 apart)
#pragma unroll 4
    for (int64_t c = kVec ? lane * V : lane; c < d; c += 32 * V) {
      alignas(16) T g[V], y[V], o[V];
      if (!NVFP4_DCHECK(!kVec || c + V <= d, &g_check)) break;
      load_row<T, V, kVec, 32>(dY + t * d, c, d, g);
      load_row<T, V, kVec, 32>(Ys + p * d, c, d, y);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool in = kVec || c + i * 32 < d;
        const float gi = in ? as_f32(g[i]) : 0.f;
        if (in) dot = fmaf(gi, as_f32(y[i]), dot);
        o[i] = (T)(w * gi);
      }
      store_row<T, V, kVec, 32>(dYs + p * d, c, d, o);
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
unsigned col_blocks(int64_t d, int V) {
  const int64_t b = (d + 256 * V - 1) / (256 * V);
  return (unsigned)(b > 8 ? 8 : b);
}

template <typename TS, typename TY, int V>
void launch_combine(bool vec, const void* Ys, const int32_t* pos, const float* w, int64_t n_tok,
                    int top_k, int64_t d, void* Y, cudaStream_t st) {
  const dim3 grid((unsigned)n_tok, col_blocks(d, V));
  auto kernel = vec ? combine_kernel<TS, TY, V, true> : combine_kernel<TS, TY, V, false>;
  kernel<<<grid, 256, 0, st>>>(static_cast<const TS*>(Ys), pos, w, top_k, n_tok * top_k, d,
                               static_cast<TY*>(Y));
}

template <typename T, int V>
void launch_gather(bool vec, const void* X, const int32_t* pos, int64_t n_tok, int top_k, int64_t d,
                   void* Xs, cudaStream_t st) {
  const dim3 grid((unsigned)n_tok, col_blocks(d, V));
  auto kernel = vec ? gather_kernel<T, V, true> : gather_kernel<T, V, false>;
  kernel<<<grid, 256, 0, st>>>(static_cast<const T*>(X), pos, top_k, n_tok * top_k, d,
                               static_cast<T*>(Xs));
}

template <typename T, int V>
void launch_backward(bool vec, const void* dY, const void* Ys, const int32_t* pos, const float* w,
                     int64_t n_tok, int top_k, int64_t d, void* dYs, float* dw, cudaStream_t st) {
  const int64_t n = n_tok * top_k;
  auto kernel = vec ? combine_backward_kernel<T, V, true> : combine_backward_kernel<T, V, false>;
  kernel<<<(unsigned)((n + 7) / 8), 256, 0, st>>>(static_cast<const T*>(dY),
                                                  static_cast<const T*>(Ys), pos, w, top_k, n, d,
                                                  static_cast<T*>(dYs), dw);
}

}  // namespace

int route_take_status(cudaStream_t st) { return NVFP4_TAKE_WORD(g_check, st); }

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
  // The limit is state of the kernel on this device that every thread's calls share, so
  // it is always the largest call's, whatever this one needs: a call's own size could
  // undercut another thread's between its setting and its launch.  (Static shared
  // memory counts towards the 48 KB that need no setting: 372 experts are above it.)
  constexpr int kMostSmem = sizeof(int) * (kSortWarps + 1) * NVFP4_MAX_EXPERTS;
  static_assert(kMostSmem + 1024 <= 227 * 1024, "shared memory");
  if (smem > 32 * 1024) {
    NVFP4_CUDA_TRY(cudaFuncSetAttribute(sort_small_kernel,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem));
    NVFP4_CUDA_TRY(cudaFuncSetAttribute(sort_place_kernel,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem));
  }
  if (n <= kSortOneCta || E == 0) {
    sort_small_kernel<<<1, block, smem, st>>>(expert_ids, wide, n, E, k, offsets, rows, position);
    NVFP4_LAUNCH_CHECK();
    count_launches(1);
    return NVFP4_OK;
  }
  int64_t chunk = (n + kSortMaxChunks - 1) / kSortMaxChunks;
  if (chunk < kSortChunk) chunk = kSortChunk;
  const int n_chunks = (int)(n / chunk);
  sort_count_kernel<<<n_chunks, block, sizeof(int) * E, st>>>(expert_ids, wide, n, chunk, E, position);
  NVFP4_LAUNCH_CHECK();
  const int parts = kSortWarps * 32 / E;
  NVFP4_CUDA_TRY(launch_chained(sort_scan_kernel, dim3(1), block, sizeof(int) * (parts + 1) * E, st,
                                chunk, n_chunks, E, parts, offsets, position));
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
  const bool vec = row % 16 == 0 && is_aligned(X, 16) && is_aligned(Xs, 16);
  if (dtype == NVFP4_BF16)
    launch_gather<__nv_bfloat16, 8>(vec, X, position, n_tok, (int)top_k, d, Xs, st);
  else
    launch_gather<float, 4>(vec, X, position, n_tok, (int)top_k, d, Xs, st);
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
  const bool vec = d % 8 == 0 && is_aligned(Ys, 16) && is_aligned(Y, 16);
  const int k = (int)top_k;
  if (s_dtype == NVFP4_BF16 && y_dtype == NVFP4_BF16)
    launch_combine<__nv_bfloat16, __nv_bfloat16, 8>(vec, Ys, position, weights, n_tok, k, d, Y, st);
  else if (s_dtype == NVFP4_BF16)
    launch_combine<__nv_bfloat16, float, 4>(vec, Ys, position, weights, n_tok, k, d, Y, st);
  else if (y_dtype == NVFP4_BF16)
    launch_combine<float, __nv_bfloat16, 4>(vec, Ys, position, weights, n_tok, k, d, Y, st);
  else
    launch_combine<float, float, 4>(vec, Ys, position, weights, n_tok, k, d, Y, st);
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
  const bool vec = (size * d) % 16 == 0 && is_aligned(dY, 16) && is_aligned(Ys, 16) &&
                   is_aligned(dYs, 16);
  const int k = (int)top_k;
  if (dtype == NVFP4_BF16)
    launch_backward<__nv_bfloat16, 8>(vec, dY, Ys, position, weights, n_tok, k, d, dYs, dweights, st);
  else
    launch_backward<float, 4>(vec, dY, Ys, position, weights, n_tok, k, d, dYs, dweights, st);
  NVFP4_LAUNCH_CHECK();
  count_launches(1);
  return NVFP4_OK;
}

}  // extern "C"
