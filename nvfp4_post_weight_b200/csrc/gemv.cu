// Products of a few tokens with NVFP4 weights as the solve leaves them:
// Y = X Q^T, Q = e2m1(code) * e4m3(scale) * s_g, one matrix or one matrix per
// expert over rows sorted by expert, and the gated pair silu(X Qg^T) * X Qu^T.
//
// The product e2m1 * e4m3 has at most six significant bits and is exact in
// bf16, so a bf16 matrix instruction multiplies it with bf16 tokens exactly and
// sums in fp32; fp32 tokens are cut into three bf16 pieces (exact: 8 bits
// each), which take three instructions.  With few tokens the 9/16 byte per
// weight bounds the product, and the decoding of the codes comes next: about
// two integer instructions per weight.
//
// A warp takes 16 output columns (rows of Q; of both matrices for the pair)
// over one slice of K, as the 16-row operand of mma.m16n8k16 with the tokens as
// its 8 columns.  K is taken in chunks of 128: lane (g, t) holds the 32
// weights 32 t .. 32 t + 31 of rows g and g + 8, one 16-byte load each, in
// whatever order decoding leaves them, and the tokens in shared memory follow
// that order (any order of K gives the same sum).  Eight warps with a tile
// each share the tokens' slice; the slices of K are the CTAs of a cluster,
// which add up their sums through distributed shared memory in a fixed order:
// no workspace, no atomics, the same bits every time.
//
// This kernel takes what the FP4 path (gemv_fp4.cu) does not: fp32 tokens, rows
// that are not whole panels of 256 columns, other alignments, and sizes that are
// over before that path's chain of stages is.  What bounds it there is latency
// (1024 x 8192, one token: 4.7 MB in 6.2 us, of which a launch, a DRAM access, the
// staging of the tokens and the join take five); with more weights the issue of
// some 3.7 instructions per weight (the 28672 x 8192 pair: 86 us).  fp16 operands
// by the e2m1 conversion instruction needed 2.5 per weight and took longer (94
// us: the conversion is issued at a fraction of the rate), as did a persistent
// form with the codes copied to shared memory (77 us for the pair, but 708 us
// where this takes 305: 64 tokens' rows through 128 experts' pairs).
#include <cooperative_groups.h>
#include <math.h>

#include "gemv.cuh"

namespace nvfp4 {
namespace {

namespace cg = cooperative_groups;

NVFP4_CHECK_WORD(g_check);
#ifdef NVFP4_DEBUG
// Debug build: `bytes` at p lie in the launch's dynamic shared memory, which begins at base.
__device__ __forceinline__ bool in_smem(const void* base, const void* p, int64_t bytes) {
  uint32_t size;
  asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(size));
  const int64_t at = static_cast<const char*>(p) - static_cast<const char*>(base);
  return at >= 0 && at + bytes <= (int64_t)size;
}
#endif

constexpr int kWarps = 8;
constexpr int kRowsCta = 16 * kWarps;
constexpr int kChunk = 128;                   // K per step: 64 bytes of codes a row
constexpr int kXSmem = 64 * 1024;             // tokens' share of shared memory

struct Args {
  Product p;
  int slice;            // chunks of K per CTA of the cluster
  int stage;            // chunks of tokens in shared memory at a time
  int* status;          // the call's status word, or null: cleared (no wait here can run out)
};

// Eight codes (one word) as four bf16 pairs: elements (0,4), (1,5), (2,6),
// (3,7).  A nibble s e e m times 0x1040 puts e e m at bits 6..8, the end of
// the exponent and the top of the mantissa, and s at the sign: the bf16 (for
// e e = 0 subnormal, with the right value) e2m1 * 2^-126.  Times the scale
// e4m3 * 2^118 that is e2m1 * e4m3 * 2^-8, exact.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a),
                             *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t* o) {
  constexpr uint32_t kMask = 0x81C081C0u;
  const uint32_t v = w >> 8;
  o[0] = mul_bf16x2(((w & 0x000F000Fu) * 0x1040u) & kMask, scale);
  o[1] = mul_bf16x2(((w & 0x00F000F0u) * 0x0104u) & kMask, scale);
  o[2] = mul_bf16x2(((v & 0x000F000Fu) * 0x1040u) & kMask, scale);
  o[3] = mul_bf16x2(((v & 0x00F000F0u) * 0x0104u) & kMask, scale);
}

// A scale code as a pair of bf16 e4m3 * 2^118: the code's seven bits at the
// top of the fp32 mantissa are e4m3 * 2^-120 (subnormal codes included).
__device__ __forceinline__ uint32_t scale_pair(uint32_t code) {
  const float f = __uint_as_float((code & 0x7Fu) << 20) * 0x1p120f * 0x1p118f;
  return __byte_perm(__float_as_uint(f), 0, 0x3232);
}

__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One lane's codes and scales of one row in one chunk: 32 weights, 2 scales.
struct Piece {
  uint32_t c[4];
  uint32_t s;
};

// block: the first of the lane's two blocks in the row; nb: blocks of the row;
// blocks past the end are zero.  kWide: rows and bases allow 16-byte code and
// 2-byte scale loads (then nb is even).
template <bool kWide>
__device__ __forceinline__ Piece load_piece(const uint8_t* codes, const uint8_t* scales, int block,
                                            int nb) {
  Piece p = {{0, 0, 0, 0}, 0};
  if (kWide) {
    if (block < nb) {
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(p.c[0]), "=r"(p.c[1]), "=r"(p.c[2]), "=r"(p.c[3])
                   : "l"(codes + 8 * block));
      p.s = __ldg(reinterpret_cast<const uint16_t*>(scales + block));
    }
  } else {
    if (block < nb) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(codes) + block);
      p.c[0] = v.x;
      p.c[1] = v.y;
      p.s = __ldg(scales + block);
    }
    if (block + 1 < nb) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(codes) + block + 1);
      p.c[2] = v.x;
      p.c[3] = v.y;
      p.s |= (uint32_t)__ldg(scales + block + 1) << 8;
    }
  }
  return p;
}

// The tokens t0 .. t0 + n - 1 over chunks [c0, c1) in shared memory, in the
// order that decode8 gives: per chunk and token 256 bytes, 16-byte unit
// 4 i + t (XOR 4 for odd tokens: eight lanes then read all 32 banks) holds
// elements 32 t + 8 i .. + 7 as the pairs (0,4), (1,5), (2,6), (3,7).  fp32
// tokens take three planes.  Columns past d_in are zeros.
template <typename TX>
__device__ __forceinline__ void stage_tokens(const Product& a, int64_t t0, int n, int c0,
                                             int c1, uint4* xs, int plane) {
  const TX* X = static_cast<const TX*>(a.X);
  const int units = (c1 - c0) * 16;
  for (int i = threadIdx.x; i < n * units; i += blockDim.x) {
    const int tok = i / units, u = i - tok * units;
    const int64_t r = a.rows ? __ldg(a.rows + t0 + tok) : t0 + tok;
    const int64_t k = (int64_t)c0 * kChunk + u * 8;
    const int at = ((u >> 4) * n + tok) * 16 +
                   ((((u & 3) << 2) | ((u >> 2) & 3)) ^ ((tok & 1) << 2));
    const bool ok = k < a.d_in && r >= 0 && r < a.n_x;   // (d_in is a multiple of 8)
    if (!NVFP4_DCHECK(at < plane && t0 + tok < a.n_rows &&
                          in_smem(xs, xs + (sizeof(TX) == 2 ? 0 : 2) * plane + at, 16),
                      &g_check))
      continue;
    if constexpr (sizeof(TX) == 2) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (ok) v = __ldg(reinterpret_cast<const uint4*>(X + r * a.d_in + k));
      xs[at] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                          __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
    } else {
      float f[8] = {};
      if (ok) {
        const float4 lo = __ldg(reinterpret_cast<const float4*>(X + r * a.d_in + k));
        const float4 hi = __ldg(reinterpret_cast<const float4*>(X + r * a.d_in + k) + 1);
        f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w;
        f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        // the upper halves are the next eight bits; an infinity leaves nothing
        xs[p * plane + at] = make_uint4(
            __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[4]), 0x7632),
            __byte_perm(__float_as_uint(f[1]), __float_as_uint(f[5]), 0x7632),
            __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[6]), 0x7632),
            __byte_perm(__float_as_uint(f[3]), __float_as_uint(f[7]), 0x7632));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float top = __uint_as_float(__float_as_uint(f[j]) & 0xFFFF0000u);
          f[j] = f[j] == top ? 0.f : f[j] - top;
        }
      }
    }
  }
}

// NW matrices (2: the gated pair), NT * 8 tokens per pass, kWide as in
// load_piece.  Grid: (cluster ranks fastest: slices of K) x tiles of 128
// columns, and experts.
template <typename TX, int NW, int NT, bool kWide>
__global__ void __launch_bounds__(256, NT * NW > 4 ? 1 : 2) product_kernel(const Args args) {
  constexpr int kPlanes = sizeof(TX) == 2 ? 1 : 3, kAcc = kPlanes == 1 ? 2 : 3;
  constexpr int kDepth = NW == 1 && kPlanes == 1 ? 4 : 2;   // chunks loaded ahead
  extern __shared__ uint4 smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;

  const Product& a = args.p;
  if (args.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *args.status = 0;
  int e, first, count;
  if (!find_pass(a, (int)a.n_rows, blockIdx.y, &e, &first, &count))
    return;   // (the whole cluster: it shares blockIdx.y)
  const int64_t r0 = first, r1 = first + count;
  const int64_t o0 = (int64_t)(blockIdx.x / S) * kRowsCta;
  const int64_t row = o0 + warp * 16;
  const int nb = a.nb;
  const int n_chunks = (nb + 7) / 8;
  const int c_begin = min(rank * args.slice, n_chunks), c_end = min(c_begin + args.slice, n_chunks);

  // this lane's two rows of each matrix; rows past d_out read the last one
  const uint8_t *codes[NW][2], *scales[NW][2];
#pragma unroll
  for (int m = 0; m < NW; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int64_t r = (int64_t)e * a.d_out + min(row + g + 8 * h, a.d_out - 1);
      if (!NVFP4_DCHECK(r >= 0 && r < a.n_experts * a.d_out, &g_check)) r = 0;
      codes[m][h] = a.codes[m] + r * nb * 8;
      scales[m][h] = a.scales[m] + r * nb;
    }

  uint4* xs = smem;
  const int max_tok = (int)min(r1 - r0, (int64_t)(8 * NT));
  float* part = reinterpret_cast<float*>(smem + (size_t)kPlanes * args.stage * max_tok * 16);

  for (int64_t t0 = r0; t0 < r1; t0 += 8 * NT) {
    const int n = (int)min(r1 - t0, (int64_t)(8 * NT));
    const int plane = args.stage * n * 16;
    Piece q[kDepth][NW][2];
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int m = 0; m < NW; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          q[d][m][h] = load_piece<kWide>(codes[m][h], scales[m][h],
                                         c_begin + d < c_end ? (c_begin + d) * 8 + 2 * t : nb, nb);
    float tot[NW][NT][4] = {};
    for (int c0 = c_begin; c0 < c_end; c0 += args.stage) {
      const int c1 = min(c0 + args.stage, c_end);
      if (c0 > c_begin) __syncthreads();   // the previous tokens are used up
      stage_tokens<TX>(a, t0, n, c0, c1, xs, plane);
      __syncthreads();
      for (int cb = c0; cb < c1; cb += kDepth) {   // (stage is a multiple of kDepth)
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int c = cb + d;
          if (c >= c1) break;
          float acc[NW][NT][kAcc][4] = {};
          uint32_t sc[NW][2][2];
#pragma unroll
          for (int m = 0; m < NW; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              sc[m][h][0] = scale_pair(q[d][m][h].s);
              sc[m][h][1] = scale_pair(q[d][m][h].s >> 8);
            }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t A[NW][2][4];
#pragma unroll
            for (int m = 0; m < NW; ++m) {
              uint32_t p[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) decode8(q[d][m][h].c[w], sc[m][h][w >> 1], p[h]);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                A[m][j][0] = p[0][2 * j];
                A[m][j][1] = p[1][2 * j];
                A[m][j][2] = p[0][2 * j + 1];
                A[m][j][3] = p[1][2 * j + 1];
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int tok = 8 * nt + g;
#pragma unroll
              for (int pl = 0; pl < kPlanes; ++pl) {
                uint4 b = make_uint4(0, 0, 0, 0);
                if (tok < n && NVFP4_DCHECK(((c - c0) * n + tok) * 16 + 16 <= plane, &g_check))
                  b = xs[pl * plane + ((c - c0) * n + tok) * 16 + ((4 * w + t) ^ ((tok & 1) << 2))];
#pragma unroll
                for (int m = 0; m < NW; ++m) {
                  float* sum = acc[m][nt][pl == 0 ? w >> 1 : 2];
                  mma(sum, A[m][0], b.x, b.y);
                  mma(sum, A[m][1], b.z, b.w);
                }
              }
            }
          }
          // The matrix unit does not round its sums to nearest: it makes chains of
          // four (and one of the fp32 tokens' lesser pieces), which fp32 additions
          // join, so that its error neither shows nor grows with K.
#pragma unroll
          for (int m = 0; m < NW; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float sum = acc[m][nt][0][i] + acc[m][nt][1][i];
                if (kAcc == 3) sum += acc[m][nt][kAcc - 1][i];
                tot[m][nt][i] += sum;
              }
          const int next = c + kDepth;
#pragma unroll
          for (int m = 0; m < NW; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              q[d][m][h] = load_piece<kWide>(codes[m][h], scales[m][h],
                                             next < c_end ? next * 8 + 2 * t : nb, nb);
        }
      }
    }
    // sums of this slice: part[matrix][token][column]
#pragma unroll
    for (int m = 0; m < NW; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 8 * nt + 2 * t + (i & 1);
          float* at = part + (m * max_tok + tok) * kRowsCta + warp * 16 + g + 8 * (i >> 1);
          if (tok < n && NVFP4_DCHECK(in_smem(smem, at, 4), &g_check)) *at = tot[m][nt][i];
        }
    cluster.sync();
    // each CTA joins and writes its share of the columns
    const int share = kRowsCta / S;
    for (int i = threadIdx.x; i < n * share; i += blockDim.x) {
      const int tok = i / share, col = rank * share + i - tok * share;
      if (o0 + col < a.d_out &&
          NVFP4_DCHECK(col < kRowsCta && t0 + tok < a.n_rows && n <= max_tok, &g_check)) {
        float v[NW];
#pragma unroll
        for (int m = 0; m < NW; ++m) {
          float s = 0.f;
          for (int c = 0; c < S; ++c)
            s += cluster.map_shared_rank(part, c)[(m * max_tok + tok) * kRowsCta + col];
          v[m] = s * (0x1p8f * __ldg(a.sg[m] + e));
        }
        write_product<NW>(a, v, t0 + tok, o0 + col);
      }
    }
    cluster.sync();   // the sums are read: part may be rewritten, the CTA may end
  }
}

// Chunks of tokens that are staged at a time, and the shared memory of a launch: the
// staged planes of tok tokens and the sums of n_w matrices.
constexpr int64_t stage_chunks(int planes, int64_t tok) {
  const int64_t stage = kXSmem / (planes * tok * 256) / 4 * 4;
  return stage < 4 ? 4 : stage;
}
constexpr int64_t smem_bytes(int planes, int n_w, int64_t tok, int64_t stage) {
  return stage * planes * tok * 256 + (int64_t)sizeof(float) * n_w * tok * kRowsCta;
}
// The most that any call of one instantiation takes.
constexpr int most_smem(int planes, int n_w, int nt) {
  int64_t most = 0;
  for (int64_t tok = 1; tok <= 8 * nt; ++tok) {
    const int64_t bytes = smem_bytes(planes, n_w, tok, stage_chunks(planes, tok));
    if (bytes > most) most = bytes;
  }
  return (int)most;
}

template <typename TX, int NW, int NT, bool kWide>
nvfp4_status launch_kernel(const Args& a, dim3 grid, int S, size_t smem, cudaStream_t st) {
  auto kernel = product_kernel<TX, NW, NT, kWide>;
  // (always the largest call's: the limit is state of the kernel on this device that
  // other threads' calls of other sizes share)
  constexpr int kMostSmem = most_smem(sizeof(TX) == 2 ? 1 : 3, NW, NT);
  static_assert(kMostSmem <= 226 * 1024, "shared memory");
  if (smem > 48 * 1024)
    NVFP4_CUDA_TRY(
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem));
  if (S > 8)
    NVFP4_CUDA_TRY(
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  NVFP4_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, a));
  return NVFP4_OK;
}

// How the general kernel divides its work.  The size of the workspace goes by it too,
// so that it depends on sizes alone: no addresses, and a B200's SMs whether a device
// is there or not (one with other SMs gets the same, right division).
constexpr int kSms = 148;
struct Division {
  int64_t tiles, slots;   // of output columns; experts that may have rows
  int n_chunks, slices;   // of K
  int nt;                 // eights of tokens per pass: the rows of one expert on average
  int64_t wave;           // CTAs that run at a time
};

// Slices of K, each of two chunks at least: as many as leave the CTAs one wave; beyond
// it to four where the wave would be less than two thirds full.  8192 x 8192, one
// token: 4 slices 15.2 us, 8 (1.7 waves) 18.1; 12288 x 8192: 4 slices (1.3 waves) 23.5,
// 2 (0.65) 26.1.  (5, 6 and 7 slices, whose clusters fill the SMs unevenly, take
// longer than 4 and 8.)  Sixteen, a cluster that needs leave and joins more slowly,
// where that still leaves an SM to each CTA and three chunks a slice: 1024 x 8192, one
// token 6.5 to 6.2 us, 512 x 8192 6.5 to 5.1, 256 x 16384 9.2 to 6.6; but 1000 x 4112, 5
// fp32 tokens (33 chunks) 8.0 to 8.4.
Division divide(int64_t n_rows, int64_t d_out, int64_t d_in, int64_t n_experts, int n_w) {
  Division v;
  v.tiles = (d_out + kRowsCta - 1) / kRowsCta;
  v.slots = n_experts == 0 ? 1 : n_experts < n_rows ? n_experts : n_rows;
  v.n_chunks = (int)((d_in + kChunk - 1) / kChunk);
  const int64_t mean = (n_rows + v.slots - 1) / v.slots, work = v.tiles * v.slots;
  v.nt = mean <= 8 ? 1 : mean <= 16 ? 2 : 4;
  v.wave = (v.nt * n_w > 4 ? 1 : 2) * kSms;   // (the kernel's launch bounds)
  v.slices = 1;
  while (v.slices < 8 && v.n_chunks >= 4 * v.slices &&
         (2 * v.slices * work <= v.wave || (v.slices < 4 && 3 * v.slices * work < 2 * v.wave)))
    v.slices *= 2;
  if (v.slices == 8 && 16 * work <= kSms && v.n_chunks >= 48 && v.wave > kSms) v.slices = 16;
  return v;
}

nvfp4_status launch_general(const Product& p, int* status, cudaStream_t st) {
  Args a{};
  a.p = p;
  a.status = status;
  const bool glu = p.n_w == 2;
  const Division v = divide(p.n_rows, p.d_out, p.d_in, p.offsets ? p.n_experts : 0, p.n_w);
  const int64_t tiles = v.tiles, slots = v.slots;
  const int n_chunks = v.n_chunks, S = v.slices, nt = v.nt;
  a.slice = (n_chunks + S - 1) / S;
  const int64_t tok = p.n_rows < 8 * nt ? p.n_rows : 8 * nt;
  const int planes = p.x_bf16 ? 1 : 3;
  int64_t stage = stage_chunks(planes, tok);
  if (stage > a.slice) stage = (a.slice + 3) / 4 * 4;
  a.stage = (int)stage;
  const size_t smem = smem_bytes(planes, p.n_w, tok, stage);
  bool wide = p.d_in % 32 == 0;
  for (int m = 0; m < p.n_w; ++m)
    wide = wide && (reinterpret_cast<uintptr_t>(p.codes[m]) & 15) == 0 &&
           (reinterpret_cast<uintptr_t>(p.scales[m]) & 1) == 0;
  const dim3 grid((unsigned)(tiles * S), (unsigned)slots);
  nvfp4_status s = NVFP4_ERR_INVALID_ARG;
#define NVFP4_PRODUCT_W(TX, NW, NT)                                \
  s = wide ? launch_kernel<TX, NW, NT, true>(a, grid, S, smem, st) \
           : launch_kernel<TX, NW, NT, false>(a, grid, S, smem, st)
#define NVFP4_PRODUCT(TX, NW)       \
  if (nt == 1) {                    \
    NVFP4_PRODUCT_W(TX, NW, 1);     \
  } else if (nt == 2) {             \
    NVFP4_PRODUCT_W(TX, NW, 2);     \
  } else {                          \
    NVFP4_PRODUCT_W(TX, NW, 4);     \
  }
  if (p.x_bf16 && glu) {
    NVFP4_PRODUCT(__nv_bfloat16, 2)
  } else if (p.x_bf16) {
    NVFP4_PRODUCT(__nv_bfloat16, 1)
  } else if (glu) {
    NVFP4_PRODUCT(float, 2)
  } else {
    NVFP4_PRODUCT(float, 1)
  }
#undef NVFP4_PRODUCT
#undef NVFP4_PRODUCT_W
  if (s == NVFP4_OK) count_launches(1);
  return s;
}

// Whether the FP4 path is the faster one.  It starts with a launch of its own and walks
// all of K, or half, one stage after another, however few rows a CTA has; the general
// kernel slices K further, but decodes, and once for every 32 tokens.  So for one matrix
// or pair both are estimated, in columns of K that the general kernel decodes: its
// CTA's slice with some 300 for each start and pass, times what more tokens cost it,
// less where its CTAs do not fill the SMs, against 1100 and a sixth of K or, from 32
// tokens on, four tenths (its further passes lie beside one another).  Measured, us,
// FP4 / general, one token and 32: 1024 x 8192: 14.7 / 6.2 and 24.6 / 13.6; 8192 x 2048:
// 8.9 / 6.8 and 15.3 / 14.2; 8192 x 8192: 16.7 / 15.4 and 26.9 / 35.1; 4096 x 28672:
// 26.0 / 23.3; 5120 x 12288: 18.0 / 20.7 and 31.4 / 48.1; 10240 x 8192: 17.5 / 23.3 and
// 30.7 / 56.0; the pair of 4096 x 8192: 17.6 / 15.6 and 22.8 / 33.4.  33, 65, 256 and 2048
// tokens: 1024 x 8192: 21.0 / 20.4, 22.2 / 30.6, 44 / 87 and 166 / 699; 1024 x 1024: 11.8 /
// 11.9, 12.7 / 18.4, 21 / 51 and 48 / 388; 4096 x 4096: 17.7 / 21.8, 18.4 / 32.7, 49 / 88 and
// 217 / 686; the pair of 8192 x 8192: 32 / 101, 61 / 161, 151 / 487 and 1394 / 4650.
// By expert it also has to find its rows.  The general kernel's CTAs are one per tile,
// slice and expert, and decode a small expert in no time: 512 of 128 x 1024 (64 KB), 2 and
// 16 rows each 50 / 23 and 163 / 49; 256 pairs of 256 x 512 (128 KB) 29 / 21 and 77 / 49; 64
// pairs of 256 x 1024 (256 KB), 8 and 32 rows 22 / 25 and 42 / 39.  With larger ones the bytes
// of the experts' codes decide, the more rows they have the sooner: 8 pairs of 768 x 2048
// (13 MB), 4, 8 and 16 rows each 14.7 / 11.8, 15.5 / 19.8 and 16.7 / 25.7; 8 of 4096 x 1536 (25
// MB), 1, 2 and 8 rows 15.9 / 14.3, 14.3 / 14.6 and 18.0 / 26.6; 16 of 2048 x 1024 (17 MB), 4 and
// 8 rows 13.9 / 12.9 and 16.7 / 21.6; 8 pairs of 1536 x 4096 (50 MB), one row 19.9 / 25.7; 128
// pairs of 768 x 2048 (200 MB), 1 and 64 rows 52 / 73 and 271 / 528.  And few experts of many
// rows leave SMs to the passes: one of 1024 x 1024, 256 and 1024 rows 21 / 51 and 53 / 196; 8 of
// 64 x 256, 256 rows each 36 / 75 (but 64 pairs of 64 x 512, 256 rows each 254 / 108).
// n_experts 0: one matrix or pair.
bool fp4_path(int64_t n_rows, int64_t d_out, int64_t d_in, int64_t n_experts, int n_w,
              nvfp4_dtype xt) {
  if (xt != NVFP4_BF16 || !product_fp4_shape(n_rows, d_in)) return false;
  const Division v = divide(n_rows, d_out, d_in, n_experts, n_w);
  const int64_t ctas = v.tiles * v.slices * v.slots;
  if (n_experts > 0) {
    const double rows = (double)n_rows / (double)v.slots;
    if (rows >= 128. && 2 * ctas < kSms) return true;
    const double each = (double)n_w * (double)d_out * (double)d_in / 2;
    const double bytes = each * (double)v.slots;
    return each >= 300e3 && (bytes * cbrt(rows) >= 40e6 || (rows >= 6. && bytes >= 12e6));
  }
  const double waves = (double)((ctas + v.wave - 1) / v.wave);
  const double passes = v.nt == 4 ? (double)((n_rows + 31) / 32) : 1.;
  const double decode = v.nt == 1 ? 1. : v.nt == 2 ? 1.5 : 2.6 * passes;
  double general = waves * ((double)d_in / v.slices * n_w * decode + 300. * passes);
  if (ctas < kSms) general *= 0.5 + 0.5 * (double)ctas / kSms;
  const double more = n_rows <= 8 ? 0. : (double)((n_rows < 32 ? n_rows : 32) - 8);
  return general >= 1100. + (0.17 + 0.01 * more) * (double)d_in;
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
                     int n_w, int64_t d_out, int64_t d_in, void* Y, nvfp4_dtype yt, void* ws,
                     size_t ws_bytes, nvfp4_stream_t stream) {
  if (n_x < 0 || n_rows < 0 || n_experts < 0 || d_out < 0 || d_in < 0) return NVFP4_ERR_INVALID_ARG;
  if (!is_io(xt) || !is_io(yt)) return NVFP4_ERR_INVALID_ARG;
  if (d_in % kBlock || d_in > kMaxDim || d_out > kMaxRows || n_rows > kMaxRows || n_x > kMaxRows ||
      n_experts > NVFP4_MAX_EXPERTS)
    return NVFP4_ERR_SHAPE;
  const bool any = n_rows > 0 && d_out > 0 && n_experts > 0;
  Product p{};
  for (int m = 0; m < n_w; ++m) {
    if (any && (!w[m].sg || (d_in > 0 && (!w[m].codes || !w[m].scales))))
      return NVFP4_ERR_INVALID_ARG;
    if (!is_aligned(w[m].codes, 8) || !is_aligned(w[m].sg, 4)) return NVFP4_ERR_INVALID_ARG;
    p.codes[m] = w[m].codes;
    p.scales[m] = w[m].scales;
    p.sg[m] = w[m].sg;
  }
  if (any && (!Y || (n_x > 0 && d_in > 0 && !X))) return NVFP4_ERR_INVALID_ARG;
  if (!is_aligned(X, 16) || !is_aligned(Y, yt == NVFP4_BF16 ? 2 : 4) || !is_aligned(rows, 4) ||
      !is_aligned(offsets, 4))
    return NVFP4_ERR_INVALID_ARG;
  const bool fp4 = any && fp4_path(n_rows, d_out, d_in, offsets ? n_experts : 0, n_w, xt);
  const size_t need = fp4 ? product_fp4_ws_bytes(n_rows, d_in) : 0;
  if (need && (!ws || !is_aligned(ws, 256) || ws_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (!any) return NVFP4_OK;
  p.X = X;
  p.rows = rows;
  p.offsets = offsets;
  p.Y = Y;
  p.n_x = n_x;
  p.n_rows = n_rows;
  p.n_experts = n_experts;
  p.d_out = d_out;
  p.d_in = d_in;
  p.nb = (int)(d_in / kBlock);
  p.n_w = n_w;
  p.x_bf16 = xt == NVFP4_BF16;
  p.y_bf16 = yt == NVFP4_BF16;
  cudaStream_t st = as_cuda(stream);
  ProfileScope ps(kPhaseProduct, st);
  if (fp4 && product_fp4_supported(p)) return launch_product_fp4(p, ws, st);
  return launch_general(p, need ? static_cast<int*>(ws) : nullptr, st);
}

}  // namespace

int product_general_take_status(cudaStream_t st) { return NVFP4_TAKE_WORD(g_check, st); }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_gemv_workspace_size(int64_t n_rows, int64_t d_out, int64_t d_in, int64_t n_experts,
                                 int pair, nvfp4_dtype x_dtype) {
  if (n_rows < 0 || d_out < 0 || n_experts < 0 || d_out > kMaxRows || d_in > kMaxDim ||
      n_experts > NVFP4_MAX_EXPERTS ||
      !fp4_path(n_rows, d_out, d_in, n_experts, pair ? 2 : 1, x_dtype))
    return 0;
  return product_fp4_ws_bytes(n_rows, d_in);
}

nvfp4_status nvfp4_product_status(nvfp4_stream_t stream) {
  cudaStream_t st = as_cuda(stream);
  const int words[3] = {product_fp4_take_status(st), product_general_take_status(st),
                        route_take_status(st)};
  for (int w : words)
    if (w != 0) return static_cast<nvfp4_status>(w);
  return NVFP4_OK;
}

nvfp4_status nvfp4_gemv(const void* X, nvfp4_dtype x_dtype, int64_t n_tok, const uint8_t* codes,
                        const uint8_t* scales, const float* global_scale, int64_t d_out,
                        int64_t d_in, void* Y, nvfp4_dtype y_dtype, void* ws, size_t ws_bytes,
                        nvfp4_stream_t stream) {
  const Matrix w[1] = {{codes, scales, global_scale}};
  return product(X, x_dtype, n_tok, nullptr, nullptr, 1, n_tok, w, 1, d_out, d_in, Y, y_dtype, ws,
                 ws_bytes, stream);
}

nvfp4_status nvfp4_gemv_swiglu(const void* X, nvfp4_dtype x_dtype, int64_t n_tok,
                               const uint8_t* gate_codes, const uint8_t* gate_scales,
                               const float* gate_global_scale, const uint8_t* up_codes,
                               const uint8_t* up_scales, const float* up_global_scale,
                               int64_t d_out, int64_t d_in, void* Y, nvfp4_dtype y_dtype, void* ws,
                               size_t ws_bytes, nvfp4_stream_t stream) {
  const Matrix w[2] = {{gate_codes, gate_scales, gate_global_scale},
                       {up_codes, up_scales, up_global_scale}};
  return product(X, x_dtype, n_tok, nullptr, nullptr, 1, n_tok, w, 2, d_out, d_in, Y, y_dtype, ws,
                 ws_bytes, stream);
}

nvfp4_status nvfp4_gemv_experts(const void* X, nvfp4_dtype x_dtype, int64_t n_x, const int32_t* rows,
                                const int32_t* offsets, int64_t n_experts, int64_t n_rows,
                                const uint8_t* codes, const uint8_t* scales,
                                const float* global_scales, int64_t d_out, int64_t d_in, void* Y,
                                nvfp4_dtype y_dtype, void* ws, size_t ws_bytes,
                                nvfp4_stream_t stream) {
  if (n_experts > 0 && n_rows > 0 && !offsets) return NVFP4_ERR_INVALID_ARG;
  if (!rows && n_rows > 0 && n_x != n_rows) return NVFP4_ERR_INVALID_ARG;
  const Matrix w[1] = {{codes, scales, global_scales}};
  return product(X, x_dtype, n_x, rows, offsets, n_experts, n_rows, w, 1, d_out, d_in, Y, y_dtype,
                 ws, ws_bytes, stream);
}

nvfp4_status nvfp4_gemv_swiglu_experts(
    const void* X, nvfp4_dtype x_dtype, int64_t n_x, const int32_t* rows, const int32_t* offsets,
    int64_t n_experts, int64_t n_rows, const uint8_t* gate_codes, const uint8_t* gate_scales,
    const float* gate_global_scales, const uint8_t* up_codes, const uint8_t* up_scales,
    const float* up_global_scales, int64_t d_out, int64_t d_in, void* Y, nvfp4_dtype y_dtype,
    void* ws, size_t ws_bytes, nvfp4_stream_t stream) {
  if (n_experts > 0 && n_rows > 0 && !offsets) return NVFP4_ERR_INVALID_ARG;
  if (!rows && n_rows > 0 && n_x != n_rows) return NVFP4_ERR_INVALID_ARG;
  const Matrix w[2] = {{gate_codes, gate_scales, gate_global_scales},
                       {up_codes, up_scales, up_global_scales}};
  return product(X, x_dtype, n_x, rows, offsets, n_experts, n_rows, w, 2, d_out, d_in, Y, y_dtype,
                 ws, ws_bytes, stream);
}

}  // extern "C"
