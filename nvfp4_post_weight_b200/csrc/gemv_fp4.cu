// Products of a few bf16 tokens with NVFP4 weights on the block-scaled FP4 tensor
// cores: the codes and the block scales go to the matrix unit as they are
// (tcgen05.mma kind::mxf4nvf4, 16-element blocks with E4M3 scales), and the
// tokens are taken apart into FP4 digits instead.
//
// Digits: a 16-element block of a token is a fixed-point integer
// v = rn(x 2^(27 - eb)), |v| <= 2^28, eb the exponent of the block's largest
// entry, written with eight digits of base 13, each one of 0, +-1, +-2, +-3, +-4,
// +-6, +-8: one of them for every remainder, and half of each an E2M1 value.  The
// block's power of two 2^(eb - E) (E: the token's largest exponent) is its E4M3
// scale.  Each token is eight columns of the product, and
// x . q = 2^(E - 34) sum_p 13^p D_p.  The products are exact; a column is summed
// in fp32 by the matrix unit.  An entry is kept to 2^-28 of the largest of its
// block, or to 2^-45 of the token's largest (blocks more than 17 octaves below
// it), and bf16 entries within 2^-20 of their block's largest are exact: an output
// whose weight at a block's outlier is zero keeps the others' bits.  What is left out
// of a block is added by the warps that write the outputs where it may be more than
// 2^-20 of the token's typical magnitude: of 2^m, m the mean exponent of the largest of
// every eight entries, all zeros aside.  (That takes an outlier some 2^9 above the
// others which has entries 2^-20 of itself in its block: one in ten of 8191 tokens of
// N(0, 1) beside 2^13, all beside 2^20.)  Digits -4 .. 3 of base 8, 22 bits, left 4e-5
// of relative error beside one entry of 10^4 among 8191 of N(0, 1), 3e-3 beside 10^6,
// where now 9e-8 and 2e-7 are left.  (The unit's own sums: over K = 28672 of positive
// products 6e-8 off, 3e-7 at most, to neither side.)  fp32 tokens would lose bits of
// every entry; they take the other kernel.
//
// Nothing is decoded: one warp has the weights copied, one the digits, one issues
// the matrix instructions (an N <= 64 takes 45 cycles, N = 128 64), three groups
// of four warps bring the block scales to tensor memory (and read the sums).  One
// CTA per SM streams rows of its own, equal to eight rows over all SMs, as tiles
// of up to 128 rows (an M = 128 instruction may have rows that are not there: rows
// do not mix), 256 or 512 columns of K a stage.  Where few rows have many columns, two
// CTAs share the columns: the second's sums go to the first's shared memory.
//
// What bounds it: one token's DRAM bytes (the 28672 x 8192 pair, 264 MB in 50.2 us, 82%
// of the copy rate); with more tokens the traffic from L2 to the SMs, where
// every CTA reads all digits, four bytes an entry, beside its rows (the pair with
// 32 tokens, two passes, 0.95 GB in 94 us); with few rows an SM the chain of
// stages (some 0.25 us per 256 columns).  Loading scales through registers instead
// of TMA took 58 us for the one-token pair, copies of scales by tcgen05.cp from
// the issuing thread 95 us, a single warp lane's non-uniform loop 68 us.
#include <cuda_bf16.h>
#include <string.h>

#include "gemv.cuh"
#include "sm100.cuh"

namespace nvfp4 {
namespace {

using namespace sm100;

constexpr int kPanelK = 256;                      // columns of K in a 128-byte row of codes
constexpr int kMaxPanels = 2;                     // panels per stage
constexpr int kMaxStages = 12;
constexpr int kGroups = 3;                        // groups of four warps that move scales
// Warps by role: the groups, with one matrix four more that read its sums, one each
// for the codes' copies, the matrix instructions and the digits' copies.  With two
// matrices the groups read the sums too, a third of the tokens each: their
// accumulator mostly has no second one beside it, so that reading it has to be
// quick (64 tokens' rows through 128 experts' pairs: 146 us, 165 us with warps of
// their own); with one matrix and few columns of K the scales of the next tile then
// waited for them (the down projections: 100 us, 84 us so).
template <int NW>
struct Roles {
  static constexpr bool kOwnSums = NW == 1;
  static constexpr int kSumWarp = 4 * kGroups, kCodeWarp = kSumWarp + (kOwnSums ? 4 : 0),
                       kMmaWarp = kCodeWarp + 1, kDigitWarp = kMmaWarp + 1,
                       kThreads = (kDigitWarp + 1) * 32;
};
// Sorted rows that are taken apart at a time: more go in as many equal parts as it
// takes, one after another in one workspace (four bytes an entry).
constexpr int64_t kMaxRows = 2048;
constexpr int kTile = 128;
constexpr int kSplitCols = 6144;                  // least columns of K that are shared out
constexpr int kUnit = 8;                          // output columns that are shared out together
constexpr int kSmem = 225 * 1024;
constexpr int kTmemCols = 512;                    // sums, then buffers of a stage's scales
constexpr int kNonFinite = 0x7FFFFFFF;            // in place of a token's exponent
constexpr int kLeftOut = 1 << 20;                 // added to one that has blocks to complete

struct Fp4Args {
  // codes and scales of each matrix in boxes of tile and of 32 rows by one stage
  CUtensorMap codes[2][2], scales[2][2];
  Product p;
  const uint8_t* digits;    // per panel and sorted row: 8 x 128 bytes, 128-byte swizzle
  const uint8_t* sf;        // per panel and sorted row: 16 scale codes
  const int* expo;          // per sorted row: E or kNonFinite
  const uint16_t* blocks;   // per sorted row and panel: a bit per block to be completed
  int* status;
  int panels;               // per stage
  int n_stages;             // of K
  int tokens;               // per pass
  int tile;                 // output columns per accumulator, at most kTile
  int ring;                 // stages of shared memory
  int stage_bytes;
  int d_bufs;               // accumulators
  int sf_bufs;              // buffers of scales in tensor memory (at most ring)
  int split;                // CTAs (one or two) that share a tile's columns of K
  int part_bytes;           // of shared memory for the other CTA's sums
};

// ---- the tokens' digits --------------------------------------------------------
// CTA (r, part): sorted row r (zeros if it points outside X), 4096 columns.
constexpr int kDigitThreads = 512, kDigitCols = kDigitThreads * 8;

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(h[j] << 16);
    f[2 * j + 1] = __uint_as_float(h[j] & 0xFFFF0000u);
  }
}

// Exponent of a magnitude's bits (subnormals as the least normal one).
__device__ __forceinline__ int exponent(uint32_t bits) {
  return max((int)(bits >> 23), 1) - 127;
}

// Row of X of sorted row r, or -1.
__device__ __forceinline__ int64_t x_row(const Product& p, int64_t r) {
  if (!p.rows) return r;
  const int64_t x = __ldg(p.rows + r);
  return x < p.n_x ? x : -1;
}

// Half a digit as E2M1 code by the remainder that it leaves: 0, 1, 2, 3, 4, -8, 6, -6,
// 8, -4, -3, -2, -1.
constexpr uint64_t kDigitCodes = 0x9ABC6D5E43210ull;
// The eighth digit is what seven leave of |v| <= 2^28: at most 2^28 / 13^7 + 8 / 12 < 5.
// Five are added for it at the start: codes of -4 .. 4 for 1 .. 9.
constexpr int kBias = 5 * 62748517;   // 5 * 13^7
constexpr uint64_t kTopCodes = 0x432109ABC0ull;
// u / 13 for u < 2^30: 13 * 330382100 = 2^32 + 4.
__device__ __forceinline__ uint32_t div13(uint32_t u) { return __umulhi(u, 330382100u); }

// f 2^e, |e| <= 252, in two steps that stay in fp32's range.
__device__ __forceinline__ float scaled(float f, int e) {
  return f * __uint_as_float((uint32_t)(e / 2 + 127) << 23) *
         __uint_as_float((uint32_t)(e - e / 2 + 127) << 23);
}

// Entries of a row of block masks: one per panel, and zeros up to whole 16-byte words.
__host__ __device__ constexpr int mask_stride(int n_panels) { return (n_panels + 7) / 8 * 8; }

// Magnitude bits (of fp32) of the largest of eight entries, compared two at a time.
__device__ __forceinline__ uint32_t largest(const uint4& v) {
  constexpr uint32_t kBits = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & kBits, v.y & kBits), __vmaxu2(v.z & kBits, v.w & kBits));
  return max(m << 16, m & 0xFFFF0000u);
}

__global__ void __launch_bounds__(kDigitThreads)
    digits_kernel(const Product p, uint8_t* __restrict__ digits, uint8_t* __restrict__ sf,
                  int* __restrict__ expo, uint16_t* __restrict__ blocks, int* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kWarps = kDigitThreads / 32;
  __shared__ uint32_t warp_max[kWarps];
  __shared__ int warp_sum[kWarps], warp_count[kWarps];
  const int64_t r = blockIdx.x;
  const int d_in = (int)p.d_in;
  const int64_t row = x_row(p, r);
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.X) + row * d_in;
  if (p.row0 + r == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  // the row's largest magnitude (bits order like values; not finite: above all), and the
  // exponents of the largest of every eight entries that are not all zero, summed, and
  // their number
  uint32_t big = 0;
  int sum = 0, count = 0;
  if (row >= 0)
#pragma unroll 4
    for (int k = threadIdx.x * 8; k < d_in; k += kDigitThreads * 8) {
      const uint32_t most = largest(__ldg(reinterpret_cast<const uint4*>(x + k)));
      big = max(big, most);
      if (most) sum += exponent(most), ++count;
    }
  big = __reduce_max_sync(0xffffffffu, big);
  sum = __reduce_add_sync(0xffffffffu, sum);
  count = __reduce_add_sync(0xffffffffu, count);
  if ((threadIdx.x & 31) == 0) {
    warp_max[threadIdx.x >> 5] = big;
    warp_sum[threadIdx.x >> 5] = sum;
    warp_count[threadIdx.x >> 5] = count;
  }
  __syncthreads();
  const int w = threadIdx.x & (kWarps - 1);   // (sums of all warps, twice: 32 lanes)
  big = __reduce_max_sync(0xffffffffu, warp_max[w]);
  sum = __reduce_add_sync(0xffffffffu, warp_sum[w]);
  count = __reduce_add_sync(0xffffffffu, warp_count[w]);
  const bool finite = big < 0x7F800000u;
  const int E = exponent(big);
  if (blockIdx.y == 0 && threadIdx.x == 0) expo[r] = finite ? E : kNonFinite;
  const int k = blockIdx.y * kDigitCols + threadIdx.x * 8;
  // (warp-uniform: whole panels)
  const bool in = k < d_in && NVFP4_DCHECK(k + 8 <= d_in && r < p.n_rows, status);
  uint4 entries = make_uint4(0, 0, 0, 0);
  if (in && row >= 0 && finite) entries = __ldg(reinterpret_cast<const uint4*>(x + k));
  float f[8];
  unpack8(entries, f);
  uint32_t most = largest(entries);
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));   // a block is two lanes' entries
  const int below = min(E - exponent(most), 17);
  const int up = 27 - (E - below);
  uint32_t u[8];   // what is left of each entry, made positive for the first seven digits
  bool whole = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float at = scaled(f[j], up);
    u[j] = (uint32_t)(__float2int_rn(at) + kBias);
    // (eight bits from 2^7 on are whole; below, what an integer's addition rounds away)
    const float rest = at - (__fadd_rn(at, 0x1.8p23f) - 0x1.8p23f);
    whole = whole && (fabsf(at) >= 128.f || (rest == 0.f && (at != 0.f || f[j] == 0.f)));
  }
  // half a unit of v is 2^(E - below - 28): above 2^(sum / count - 20)?
  const unsigned open = __ballot_sync(0xffffffffu, !whole && (E - below - 8) * count > sum);
  if ((threadIdx.x & 31) == 0 && k / kPanelK < mask_stride(d_in / kPanelK)) {
    uint32_t bits = 0;   // a block's two lanes to one bit
    for (int b = 0; open && b < 16; ++b) bits |= (uint32_t)((open >> (2 * b) & 3u) != 0) << b;
    blocks[r * mask_stride(d_in / kPanelK) + k / kPanelK] = (uint16_t)bits;
  }
  if (in) {
    const int panel = k / kPanelK, byte = (k % kPanelK) / 2;
    const int64_t at = panel * p.n_rows + r;
    uint8_t* out = digits + at * 1024;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t word = 0;   // E2M1 codes, first element lowest
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t code;
        if (p < 7) {
          const uint32_t q = div13(u[j]);
          code = (uint32_t)(kDigitCodes >> 4 * (u[j] - 13 * q)) & 0xFu;
          u[j] = q + (code >> 3);   // a digit below zero borrowed 13
        } else {
          code = (uint32_t)(kTopCodes >> 4 * u[j]) & 0xFu;
        }
        word |= code << (4 * j);
      }
      *reinterpret_cast<uint32_t*>(out + p * 128 + ((((byte >> 4) ^ p) & 7) << 4) + (byte & 15)) =
          word;
    }
    if ((threadIdx.x & 1) == 0) {
      // 2^(8 - below) in E4M3: normal down to 2^-6, then 2^-7, 2^-8, 2^-9
      const int code = below <= 14 ? (15 - below) << 3 : 4 >> (below - 15);
      sf[at * 16 + (k % kPanelK) / 16] = (uint8_t)code;
    }
  }
}

// ---- the product -----------------------------------------------------------------
struct Shared {
  uint64_t weights[kMaxStages];   // codes and scales of a stage have landed
  uint64_t tokens[kMaxStages];    // its digits have
  uint64_t scaled[kMaxStages];    // its scales are in tensor memory
  uint64_t empty[kMaxStages];     // its matrix instructions are done
  uint64_t d_full[2], d_empty[2]; // an accumulator is complete, has been read
  uint64_t part_full, part_free;  // the other CTA's sums are here, have been read
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

// The first timeout of any call since the host last asked: kept beside the calls' own
// words, which go with their workspaces.
__device__ int g_product_status;

__device__ __forceinline__ void give_up(Shared* sh, int* status) {
  atomicExch(&sh->abort, 1);
  atomicCAS(&g_product_status, 0, (int)NVFP4_ERR_TIMEOUT);
  pdl_wait();   // (the kernel before this one clears the word)
  atomicCAS(status, 0, (int)NVFP4_ERR_TIMEOUT);
}
__device__ __forceinline__ bool aborted(Shared* sh) {
  return *reinterpret_cast<volatile int*>(&sh->abort) != 0;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// The pipeline waits of sm100.cuh with the limit read once; given up too when
// another role has.  Warp-wide (so that what follows stays warp-uniform and the
// matrix instructions' operands in uniform registers).
template <typename Wait>
__device__ __forceinline__ bool wait_by(Wait look, unsigned long long limit, Shared* sh) {
  bool ok = look(limit <= 1);
  if (!__all_sync(0xffffffffu, ok)) {
    const uint64_t t0 = globaltimer();
    while (!ok && limit > 1 && !aborted(sh) && globaltimer() - t0 <= limit)
      for (int i = 0; i < 16 && !ok; ++i) ok = look(false);
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, unsigned long long limit,
                                     Shared* sh) {
  return wait_by([&](bool once) { return once ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity); },
                 limit, sh);
}
// The same for a barrier that the cluster's other CTA arrives at.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity,
                                             unsigned long long limit, Shared* sh) {
  return wait_by(
      [&](bool) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        return ok != 0;
      },
      limit, sh);
}
// This CTA's place in its cluster; the address of `p` in CTA `rank` of it.
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// 16 (4) consecutive columns of this thread's TMEM lane (warp-wide).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint4* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z),
      "r"(v[1].w), "r"(v[2].x), "r"(v[2].y), "r"(v[2].z), "r"(v[2].w), "r"(v[3].x), "r"(v[3].y),
      "r"(v[3].z), "r"(v[3].w)
      : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint4& v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void mma_nvfp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8_twice(uint32_t ta, uint32_t tb, float (*v)[8]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i >> 3][i & 7] = __uint_as_float(r[i]);
}

// What one CTA works through: pieces of (expert, pass over its tokens), each a
// range of output columns.
struct Piece {
  int e, t0, n;             // expert, its first sorted row and their number in this pass
  int64_t row0, row1;       // output columns
};
struct Pieces {
  int64_t u, u_end, units;
  __device__ __forceinline__ void init(const Fp4Args& a, int split) {
    units = (a.p.d_out + kUnit - 1) / kUnit;
    const int passes = count_passes(a.p, a.tokens), ctas = gridDim.x / split,
              b = blockIdx.x / split;
    const int per = passes ? ctas / passes : 0;   // CTAs per pass
    if (per * passes * 16 >= ctas * 15) {
      // few passes: a whole number of CTAs each, so that no CTA has two pieces
      u = b < per * passes ? b / per * units + units * (b % per) / per : 0;
      u_end = b < per * passes ? b / per * units + units * (b % per + 1) / per : 0;
    } else {
      const int64_t all = passes * units;
      u = all * b / ctas;
      u_end = all * (b + 1) / ctas;
    }
  }
  // Warp-wide.  (The debug build leaves out a piece that is not inside the call's
  // arrays, in every role alike.)
  __device__ __forceinline__ bool next(const Fp4Args& a, Piece* q) {
    while (u < u_end) {
      const int64_t slot = u / units, ub = u - slot * units;
      const int64_t ue = min(units, u_end - slot * units);
      u = slot * units + ue;
      const bool found = find_pass(a.p, a.tokens, (int)slot, &q->e, &q->t0, &q->n);
      q->row0 = ub * kUnit;
      q->row1 = min(ue * kUnit, a.p.d_out);
      if (NVFP4_DCHECK(found && q->e >= 0 && q->e < a.p.n_experts && q->n > 0 &&
                           q->n <= a.tokens && q->t0 >= 0 && q->t0 + q->n <= a.p.n_rows &&
                           q->row0 < q->row1,
                       a.status))
        return true;
    }
    return false;
  }
};

// One product x . q where digits do not do, sorted row r, column o of matrix w of expert
// e.  A token with a NaN or an infinity: by plain sums.  One with blocks to complete:
// the digits' product and what they leave out of those.  Warp-wide, each lane its own
// column: the lanes have an entry of the block each and hand it round.  (Some 3.5 us for
// a token with one block: round trips to memory one after another.  A call of its own, so
// that the loops that have no such token keep their registers.)
__device__ __noinline__ float special_product(const Fp4Args& a, int w, int e, int64_t r, int64_t o,
                                              int E, double digits) {
  const Product& p = a.p;
  const int lane = threadIdx.x & 31, n_panels = p.nb / 16;
  const int64_t block = (e * p.d_out + o) * p.nb;
  const uint2* codes = reinterpret_cast<const uint2*>(p.codes[w]) + block;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.X) + x_row(p, r) * p.d_in;
  const uint16_t* masks = a.blocks + r * mask_stride(n_panels);
  const bool plain = E == kNonFinite - kLeftOut;
  float sum = 0.f;
  for (int first = 0; first < n_panels; first += 32) {
    uint32_t mine = 0;   // the blocks of panel first + lane
    if (first + lane < n_panels) mine = plain ? 0xFFFFu : __ldca(masks + first + lane);
    for (unsigned some = __ballot_sync(~0u, mine != 0); some; some &= some - 1) {
      const int at = __ffs(some) - 1;
      for (uint32_t bits = __shfl_sync(~0u, mine, at); bits; bits &= bits - 1) {
        const int b = (first + at) * 16 + __ffs(bits) - 1;
        const uint2 c = codes[b];
        const float scale = (float)e4m3_value(p.scales[w][block + b] & 0x7F);
        float f = lane < kBlock ? __bfloat162float(x[b * kBlock + lane]) : 0.f;
        if (!plain) {
          const uint32_t most = __reduce_max_sync(~0u, __float_as_uint(f) & 0x7FFFFFFFu);
          const int up = 27 - max(exponent(most), E - 17);
          f -= scaled(rintf(scaled(f, up)), -up);
        }
#pragma unroll
        for (int j = 0; j < kBlock; ++j)
          sum = fmaf(__shfl_sync(~0u, f, j),
                     e2m1_value((j < 8 ? c.x : c.y) >> (4 * (j & 7)) & 0xF) * scale, sum);
      }
    }
  }
  const double sg = p.sg[w][e];
  return plain ? sum * (float)sg : (float)(digits + (double)sum * sg);
}

template <int NW, int kSplit>
__global__ void __launch_bounds__(Roles<NW>::kThreads, 1)
    product_fp4_kernel(const __grid_constant__ Fp4Args a) {
  extern __shared__ uint8_t smem_raw[];
  // the other CTA's sums, the stages
  float* part = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~uintptr_t(1023));
  uint8_t* stages = reinterpret_cast<uint8_t*>(part) + a.part_bytes;
  __shared__ Shared shared;
  Shared* sh = &shared;
  constexpr int kSumWarp = Roles<NW>::kSumWarp, kCodeWarp = Roles<NW>::kCodeWarp,
                kMmaWarp = Roles<NW>::kMmaWarp, kDigitWarp = Roles<NW>::kDigitWarp;
  constexpr bool kOwnSums = Roles<NW>::kOwnSums;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.panels, S = a.ring;
  const int rank = kSplit > 1 ? cluster_rank() : 0;
  const int k0 = a.n_stages * rank / kSplit, k1 = a.n_stages * (rank + 1) / kSplit;
  const int columns = (a.tokens + 1) / 2 * 16;   // of an accumulator, per matrix
  const int blocks = columns > 128 ? 2 : 1;      // 128-row groups of the digits' scales
  const int sf_cols = (NW + blocks) * 16 * P;    // TMEM columns of a stage's scales
  // a stage: codes (matrix, panel, row), digits (panel, token), scales of the
  // codes (matrix, row, panel), scales of the digits (panel, token).  (A matrix
  // instruction reads 128 rows of codes, also where a tile has fewer: what
  // follows them in shared memory, which only rows that are not written see.)
  const int panel_bytes = a.tile * 128;
  const int b_at = NW * P * panel_bytes, sfa_at = b_at + P * columns * 128;
  const int sfb_at = sfa_at + NW * a.tile * 16 * P;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh->weights[s], 1);
      mbar_init(&sh->tokens[s], 1);
      mbar_init(&sh->scaled[s], 4);
      mbar_init(&sh->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->d_full[i], 1);
      mbar_init(&sh->d_empty[i], kOwnSums ? 4 : 4 * kGroups);
    }
    mbar_init(&sh->drain, 1);
    mbar_init(&sh->part_full, kOwnSums ? 4 : 4 * kGroups);
    mbar_init(&sh->part_free, kOwnSums ? 4 : 4 * kGroups);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sh->tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  if (kSplit > 1) cluster_sync();   // (the other CTA's barriers are there)
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  const unsigned long long limit = __ldg(&g_wait_limit_ns);

  Pieces pieces;
  pieces.init(a, kSplit);
#ifdef NVFP4_DEBUG
  // what the launch laid out fits: the other CTA's sums and the ring (with the rows behind
  // a short tile) into shared memory, sums and scales into tensor memory
  uint32_t smem_size;
  asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(smem_size));
  const int64_t end = stages + (int64_t)S * a.stage_bytes + (kTile - a.tile) * (128 + 16 * P) - smem_raw;
  if (!NVFP4_DCHECK(end <= (int64_t)smem_size && S <= kMaxStages && a.sf_bufs <= S &&
                        a.tile <= kTile && sfb_at + ((P - 1) * a.tokens + 16 * blocks) * 16 <= a.stage_bytes &&
                        a.d_bufs * NW * columns + a.sf_bufs * sf_cols <= kTmemCols &&
                        (kSplit == 1 || a.tokens * NW * kTile * 4 <= a.part_bytes),
                    a.status))
    pieces.u = pieces.u_end;
#endif
  Piece q;
  int s = 0;          // slot of shared memory and its phase
  uint32_t ph = 0;
  auto step = [&] {
    if (++s == S) s = 0, ph ^= 1;
  };
  int issued = 0;     // stages that a copying role has issued
  // The sums of tile no. g at output columns row ..: thread = column (TMEM lane),
  // tokens first, first + apart, ...  Warp-wide.  Each lane keeps the exponent of one
  // of the pass' tokens (32 at most): fetched when its token's turn comes, they took
  // the down projections of 64 tokens 18 us longer.  Two sums a round trip to tensor
  // memory instead of one: 88 to 84 us.
  int exponent = 0;
  bool any_special = false;
  float sg[NW];
  auto enter_pass = [&](const Piece& q) {
    // (ordinary loads: the kernel before this one, which this one may have started beside,
    // wrote them, and the read-only path wants data that nobody writes meanwhile)
    exponent = 0;
    if (lane < q.n) {
      exponent = __ldca(a.expo + q.t0 + lane);
      const int words = mask_stride(a.p.nb / 16) / 8;
      const uint4* masks = reinterpret_cast<const uint4*>(a.blocks) + (int64_t)(q.t0 + lane) * words;
      uint32_t left = 0;
#pragma unroll 4
      for (int i = 0; i < words; ++i) {
        const uint4 m = __ldca(masks + i);
        left |= m.x | m.y | m.z | m.w;
      }
      if (left) exponent += kLeftOut;
    }
    any_special = __any_sync(~0u, exponent >= kLeftOut / 2);
#pragma unroll
    for (int w = 0; w < NW; ++w) sg[w] = __ldg(a.p.sg[w] + q.e);
  };
  auto read_sums = [&](const Piece& q, int64_t row, int g, int first, int apart) {
    const int buf = a.d_bufs == 2 ? g & 1 : 0, use = a.d_bufs == 2 ? g >> 1 : g;
    if (!wait(&sh->d_full[buf], use & 1, limit, sh)) return false;
    if (rank > 0 && g > 0 && !wait_cluster(&sh->part_free, (g - 1) & 1, limit, sh)) return false;
    if (rank == 0 && kSplit > 1 && !wait_cluster(&sh->part_full, g & 1, limit, sh)) return false;
    tc_fence_after();
    const uint32_t to = rank > 0 ? cluster_addr(part, 0) : 0;
    const int col = threadIdx.x & (kTile - 1);
    const int64_t o = row + col, o_end = min(row + a.tile, q.row1);
    const uint32_t d = tmem + ((uint32_t)((warp & 3) * 32) << 16) + buf * NW * columns;
    // sum_p 13^p D_p, four digits exactly for a single product before the one rounding
    // that joins them
    auto join = [&](const float* c) {
      float high = c[7], low = c[3];
#pragma unroll
      for (int p = 2; p >= 0; --p) {
        high = fmaf(high, 13.f, c[p + 4]);
        low = fmaf(low, 13.f, c[p]);
      }
      return fmaf(high, 28561.f, low);
    };
    auto value = [&](float sum, int E, int w) {
      // (what a token of the second loop gives here, its E not being one, is written over)
      const double power = __hiloint2double((int)((uint32_t)(E - 34 + 1023) << 20), 0);
      return (double)sum * (power * (double)sg[w]);
    };
    // two sums at a time: both matrices' of a token, or one matrix' of two tokens
    constexpr int kTokens = 2 / NW;
    for (int i0 = first; i0 < q.n; i0 += apart * kTokens) {
      float c[2][8], v[2];
      const int second = min(i0 + apart, q.n - 1);
      tmem_ld8_twice(d + 8 * i0, NW == 2 ? d + columns + 8 * i0 : d + 8 * second, c);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int w = k * (NW - 1), i = NW == 2 || k == 0 ? i0 : second;
        const int E = __shfl_sync(~0u, exponent, i);
        float sum = join(c[k]);
        const int at = (i * NW + w) * kTile + col;
        if (rank > 0) {
          cluster_store(to + 4 * at, sum);
          continue;
        }
        if (kSplit > 1) sum += part[at];
        if (o < o_end) v[k] = (float)value(sum, E, w);
      }
      if (rank == 0 && o < o_end) {
        write_product<NW>(a.p, v, q.t0 + i0, o);
        if (NW == 1 && i0 + apart < q.n) write_product<NW>(a.p, v + 1, q.t0 + second, o);
      }
    }
    // once more for tokens that digits alone do not stand for (kept apart: with the call in
    // the loop above its registers spill)
    if (rank == 0 && any_special)
      for (int i = first; i < q.n; i += apart) {
        const int E = __shfl_sync(~0u, exponent, i);
        if (E < kLeftOut / 2) continue;
        float c[2][8], v[2];
        tmem_ld8_twice(d + 8 * i, d + (NW - 1) * columns + 8 * i, c);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          float sum = join(c[w]);
          if (kSplit > 1) sum += part[(i * NW + w) * kTile + col];
          v[w] = special_product(a, w, q.e, q.t0 + i, min(o, o_end - 1), E - kLeftOut,
                                 value(sum, E - kLeftOut, w));
        }
        if (o < o_end) write_product<NW>(a.p, v, q.t0 + i, o);
        __syncwarp();
      }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sh->d_empty[buf]);
      if (kSplit > 1)
        cluster_arrive(rank ? cluster_addr(&sh->part_full, 0) : cluster_addr(&sh->part_free, 1));
    }
    __syncwarp();
    return true;
  };

  if (warp == kCodeWarp) {
    // ---------------------------------------------------------------- codes and their scales
    bool ok = true;
    while (ok && pieces.next(a, &q)) {
      for (int64_t row = q.row0; ok && row < q.row1; row += a.tile) {
        // a tile is one box (rows past the piece's end are not used); of experts a
        // part of a tile takes boxes of 32 rows and one panel
        const int valid = (int)min(q.row1 - row, (int64_t)a.tile);
        const int part = a.p.offsets && valid <= a.tile - 32 ? 1 : 0;
        const int step_rows = part ? 32 : a.tile, boxes = (valid + step_rows - 1) / step_rows;
        const int ops = part ? P : 1;
        const uint32_t bytes = (uint32_t)(NW * boxes * step_rows * (128 + 16) * P);
        const int y = (int)(q.e * a.p.d_out + row);
        for (int st = k0; st < k1; ++st) {
          ok = wait(&sh->empty[s], ph ^ 1, limit, sh);
          if (!ok) break;
          uint8_t* stage = stages + s * a.stage_bytes;
          uint64_t* bar = &sh->weights[s];
          if (elect()) {
            mbar_arrive_expect_tx(bar, bytes);
            for (int b = 0; b < boxes; ++b) {
              const int off = b * step_rows;
#pragma unroll
              for (int m = 0; m < NW; ++m) {
                for (int p = 0; p < ops; ++p)
                  tma_load_3d(stage + (m * P + p) * panel_bytes + off * 128, &a.codes[m][part], bar,
                              0, y + off, st * P + p);
                tma_load_2d(stage + sfa_at + (m * a.tile + off) * 16 * P, &a.scales[m][part], bar,
                            st * 16 * P, y + off);
              }
            }
          }
          __syncwarp();
          ++issued;
          step();
        }
      }
    }
    if (!ok) give_up(sh, a.status);
  } else if (warp == kDigitWarp) {
    // ---------------------------------------------------------------- digits
    pdl_wait();
    bool ok = true;
    while (ok && pieces.next(a, &q)) {
      const uint32_t bytes = (uint32_t)(q.n * (1024 + 16) * P);
      const int64_t next_d = a.p.n_rows * 1024, next_s = a.p.n_rows * 16;
      for (int64_t row = q.row0; ok && row < q.row1; row += a.tile) {
        const uint8_t* d = a.digits + (int64_t)q.t0 * 1024 + k0 * P * next_d;
        const uint8_t* f = a.sf + (int64_t)q.t0 * 16 + k0 * P * next_s;
        for (int st = k0; st < k1; ++st) {
          ok = wait(&sh->empty[s], ph ^ 1, limit, sh);
          if (!ok) break;
          uint8_t* stage = stages + s * a.stage_bytes;
          uint64_t* bar = &sh->tokens[s];
          if (elect()) {
            mbar_arrive_expect_tx(bar, bytes);
            for (int p = 0; p < P; ++p) {
              bulk_load(stage + b_at + p * columns * 128, d + p * next_d, q.n * 1024, bar);
              bulk_load(stage + sfb_at + p * a.tokens * 16, f + p * next_s, q.n * 16, bar);
            }
          }
          __syncwarp();
          d += P * next_d;
          f += P * next_s;
          ++issued;
          step();
        }
      }
    }
    if (!ok) give_up(sh, a.status);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- matrix instructions
    int g = 0, sf = 0;   // accumulators so far, buffer of scales
    bool ok = true;
    while (ok && pieces.next(a, &q)) {
      // E2M1 x E2M1, E4M3 scales, M = 128
      const int cols = (q.n + 1) / 2 * 16;
      const uint32_t idesc = (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) | (1u << 27);
      for (int64_t row = q.row0; ok && row < q.row1; row += a.tile, ++g) {
        const int buf = a.d_bufs == 2 ? g & 1 : 0, use = a.d_bufs == 2 ? g >> 1 : g;
        ok = wait(&sh->d_empty[buf], (use & 1) ^ 1, limit, sh);
        tc_fence_after();
        const uint32_t d = tmem + buf * NW * columns;
        bool ready = false;
        for (int st = k0; ok && st < k1; ++st) {
          // (the group that wrote the scales has waited for the stage's copies)
          ok = ready || wait(&sh->scaled[s], ph, limit, sh);
          if (!ok) break;
          tc_fence_after();
          // the next stage is looked at now: behind this one's instructions the look
          // would queue for their issue
          const int s1 = s + 1 == S ? 0 : s + 1;
          ready = st + 1 < k1 && limit > 1 && mbar_test_wait(&sh->scaled[s1], s1 == 0 ? ph ^ 1 : ph);
          ready = __all_sync(0xffffffffu, ready);
          const uint32_t stage = smem_u32(stages) + s * a.stage_bytes;
          uint64_t da = smem_desc_sw128(stage, 16, 1024);
          uint64_t db = smem_desc_sw128(stage + b_at, 16, 1024);
          uint32_t sfa = tmem + a.d_bufs * NW * columns + sf * sf_cols;
          uint32_t sfb = sfa + NW * P * 16;
          if (++sf == a.sf_bufs) sf = 0;
          if (elect()) {
            for (int p = 0; p < P; ++p) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int m = 0; m < NW; ++m)
                  mma_nvfp4(d + m * columns, da + (m * P * panel_bytes + 32 * k) / 16,
                            db + 32 * k / 16, idesc, sfa + (m * P * 4 + k) * 4, sfb + k * blocks * 4,
                            (uint32_t)((st - k0) | p | k));
              da += panel_bytes / 16;
              db += columns * 128 / 16;
              sfa += 16;
              sfb += blocks * 16;
            }
            mma_commit(&sh->empty[s]);
          }
          __syncwarp();
          step();
        }
        if (ok && elect()) mma_commit(&sh->d_full[buf]);
        __syncwarp();
      }
    }
    if (!ok) give_up(sh, a.status);
    // every instruction above completes before TMEM is released
    if (elect()) mma_commit(&sh->drain);
    __syncwarp();
    mbar_wait_drain(&sh->drain, 0);
  } else if (warp < kSumWarp) {
    // ---------------------------------------------------------------- scales
    // Groups of four warps, one warp per quarter of TMEM's lanes: lane l of each
    // quarter gets, per 64 columns of K, the words of rows l, l + 32, l + 64 and
    // l + 96.  A group takes the stages of its slots (a stage takes a group some
    // 700 cycles, the matrix instructions 400; a slot's stages all fall to one
    // group, which so sees each phase of its barriers).
    const int group = warp >> 2;
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    if (!kOwnSums) pdl_wait();   // (for the tokens' exponents)
    int g = 0;                          // accumulators so far
    int stage_no = 0, sf = 0, os = 0;   // stages so far, buffer of scales, slot of its last stage
    uint32_t oph = 0;
    auto get = [&](const uint8_t* p, int bytes_apart, uint4* v) {
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = *reinterpret_cast<const uint4*>(p + j * bytes_apart);
        x[j].x &= 0x7F7F7F7Fu, x[j].y &= 0x7F7F7F7Fu, x[j].z &= 0x7F7F7F7Fu, x[j].w &= 0x7F7F7F7Fu;
      }
      v[0] = make_uint4(x[0].x, x[1].x, x[2].x, x[3].x);
      v[1] = make_uint4(x[0].y, x[1].y, x[2].y, x[3].y);
      v[2] = make_uint4(x[0].z, x[1].z, x[2].z, x[3].z);
      v[3] = make_uint4(x[0].w, x[1].w, x[2].w, x[3].w);
    };
    bool ok = true;
    while (ok && pieces.next(a, &q)) {
      if (!kOwnSums) enter_pass(q);
      for (int64_t row = q.row0; ok && row < q.row1; row += a.tile, ++g) {
        for (int st = k0; st < k1; ++st) {
          const int slot = s, buf = sf, no = stage_no, free_slot = os;
          const uint32_t phase = ph, free_phase = oph;
          step();
          ++stage_no;
          if (++sf == a.sf_bufs) sf = 0;
          if (no >= a.sf_bufs && ++os == S) os = 0, oph ^= 1;
          if (slot % kGroups != group) continue;
          // the buffer in TMEM is free when the instructions that read it last are
          // done (where there are as many buffers as slots, the copies waited for it)
          ok = wait(&sh->weights[slot], phase, limit, sh) && wait(&sh->tokens[slot], phase, limit, sh);
          if (a.sf_bufs < S && no >= a.sf_bufs)
            ok = ok && wait(&sh->empty[free_slot], free_phase, limit, sh);
          if (!ok) break;
          const uint8_t* stage = stages + slot * a.stage_bytes;
          const uint32_t sfa = quarter + tmem + a.d_bufs * NW * columns + buf * sf_cols;
          const uint32_t sfb = sfa + NW * P * 16;
          uint4 v[4];
          for (int p = 0; p < P; ++p) {
#pragma unroll
            for (int m = 0; m < NW; ++m) {
              get(stage + sfa_at + ((m * a.tile + lane) * P + p) * 16, 32 * 16 * P, v);
              tmem_st16(sfa + (m * P + p) * 16, v);
            }
            for (int b = 0; b < blocks; ++b) {   // a token has eight columns
              get(stage + sfb_at + (p * a.tokens + b * 16 + (lane >> 3)) * 16, 4 * 16, v);
#pragma unroll
              for (int k = 0; k < 4; ++k) tmem_st4(sfb + ((p * 4 + k) * blocks + b) * 4, v[k]);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->scaled[slot]);
        }
        if (!kOwnSums && ok) ok = read_sums(q, row, g, group, kGroups);
      }
    }
    if (!ok) give_up(sh, a.status);
  } else {
    // ---------------------------------------------------------------- sums
    pdl_wait();   // (for the tokens' exponents)
    int g = 0;
    bool ok = true;
    while (ok && pieces.next(a, &q)) {
      enter_pass(q);
      for (int64_t row = q.row0; ok && row < q.row1; row += a.tile, ++g)
        ok = read_sums(q, row, g, 0, 1);
    }
    if (!ok) give_up(sh, a.status);
  }
  __syncthreads();
  // Some role gave up, maybe one that the copying roles never waited for (a CTA of no
  // more stages than the ring has slots finds them all free): the copies that nobody
  // has waited for land before the CTA exits.
  if (aborted(sh) && (warp == kCodeWarp || warp == kDigitWarp)) {
    uint64_t* bars = warp == kCodeWarp ? sh->weights : sh->tokens;
    for (int k = 0; k < S && k < issued; ++k) {
      if (--s < 0) s = S - 1, ph ^= 1;
      mbar_wait_drain(&bars[s], ph);
    }
  }
#ifdef NVFP4_DEBUG
  // no copy is in flight, whichever way the roles ended (the first use of a slot has
  // phase 0, its i-th i & 1)
  if (warp == kCodeWarp || warp == kDigitWarp)
    for (int k = max(issued - S, 0); k < issued; ++k)
      if (!mbar_test_wait(warp == kCodeWarp ? &sh->weights[k % S] : &sh->tokens[k % S], k / S & 1))
        atomicExch(a.status, (int)NVFP4_ERR_BOUNDS);
#endif
  if (kSplit > 1) cluster_sync();   // (no CTA ends while the other may still write to it)
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

int panels_of(int64_t d_in) { return (int)(d_in / kPanelK); }

}  // namespace

bool product_fp4_shape(int64_t n_rows, int64_t d_in) {
  return d_in % kPanelK == 0 && d_in > 0 && n_rows > 0;
}

int product_fp4_take_status(cudaStream_t st) { return take_status_word(g_product_status, st); }

size_t product_fp4_ws_bytes(int64_t n_rows, int64_t d_in) {
  const size_t rows = n_rows < kMaxRows ? n_rows : kMaxRows, n = panels_of(d_in);
  return kWsHeader + align256(rows * sizeof(int)) + align256(rows * mask_stride(n) * 2) +
         align256(rows * n * 16) + rows * n * 1024;
}

bool product_fp4_supported(const Product& p) {
  bool ok = product_fp4_shape(p.n_rows, p.d_in) && p.n_experts * p.d_out < (int64_t(1) << 31);
  for (int m = 0; m < p.n_w; ++m)
    ok = ok && (reinterpret_cast<uintptr_t>(p.codes[m]) & 15) == 0 &&
         (reinterpret_cast<uintptr_t>(p.scales[m]) & 15) == 0;
  return ok;
}

static nvfp4_status launch_part(const Product& p, void* ws, cudaStream_t st) {
  Fp4Args a;
  memset(&a, 0, sizeof(a));
  a.p = p;
  const int n_panels = panels_of(p.d_in);
  char* w = static_cast<char*>(ws);
  const size_t rows = p.n_rows;
  a.status = reinterpret_cast<int*>(w);
  w += kWsHeader;
  int* expo = reinterpret_cast<int*>(w);
  w += align256(rows * sizeof(int));
  uint16_t* blocks = reinterpret_cast<uint16_t*>(w);
  w += align256(rows * mask_stride(n_panels) * 2);
  uint8_t* sf = reinterpret_cast<uint8_t*>(w);
  w += align256(rows * n_panels * 16);
  uint8_t* digits = reinterpret_cast<uint8_t*>(w);
  a.expo = expo;
  a.blocks = blocks;
  a.sf = sf;
  a.digits = digits;
  const dim3 grid((unsigned)p.n_rows, (unsigned)((p.d_in + kDigitCols - 1) / kDigitCols));
  digits_kernel<<<grid, kDigitThreads, 0, st>>>(p, digits, sf, expo, blocks, a.status);
  NVFP4_LAUNCH_CHECK();
  // tokens per pass: what the accumulators hold, in equal passes; for experts
  // 16, so that an expert's rows of a small batch take one pass
  const int most = p.n_w == 2 ? 24 : 32;
  if (p.offsets) {
    a.tokens = p.n_rows < 16 ? (int)p.n_rows : 16;
  } else {
    const int64_t passes = (p.n_rows + most - 1) / most;
    a.tokens = (int)((p.n_rows + passes - 1) / passes);
  }
  const int columns = (a.tokens + 1) / 2 * 16;
  const int64_t units = (p.d_out + kUnit - 1) / kUnit;
  const int64_t slots = p.offsets ? (p.n_experts < p.n_rows ? p.n_experts : p.n_rows)
                                  : (p.n_rows + a.tokens - 1) / a.tokens;
  // one CTA per SM, or pairs of CTAs with half of K each: where the double share of
  // rows is still one tile, the pair reads half the digits and is done with its chain
  // of stages in half the time, for some 1.7 us of starting and joining (8192 x 28672,
  // 8 tokens: 39.1 to 34.8 us, 32: 67 to 53; 6144 x 8192, 8: 18.1 to 17.2; but 8192 x
  // 2048, 8: 10.4 to 12.0, and 9472 x 8192, whose tile would be full, 18.1 to 19.3)
  int64_t ctas = units * slots < num_sms() ? units * slots : num_sms();
  int64_t share = (units * slots + ctas - 1) / ctas * kUnit;   // the largest of a CTA
  a.split = 2 * share < kTile && p.d_in >= kSplitCols ? 2 : 1;
  if (a.split == 2) {
    ctas = units * slots < num_sms() / 2 ? units * slots : num_sms() / 2;
    share = (units * slots + ctas - 1) / ctas * kUnit;
  }
  // equal tiles for it (experts': in steps of 32, see the copies)
  const int64_t tiles = (share + kTile - 1) / kTile, grain = p.offsets ? 32 : kUnit;
  a.tile = (int)(((share + tiles - 1) / tiles + grain - 1) / grain * grain);
  a.part_bytes = a.split > 1 ? (a.tokens * p.n_w * kTile * 4 + 1023) / 1024 * 1024 : 0;
  // panels per stage: two (a stage costs each role a few hundred cycles whatever its
  // size) where that leaves a ring of three stages, or four for two matrices
  for (a.panels = kMaxPanels; a.panels >= 1; a.panels /= 2) {
    // (the digits' scales are read for whole groups of 16 tokens)
    a.stage_bytes = (a.panels * (p.n_w * a.tile * (128 + 16) + columns * 128 + a.tokens * 16) +
                     32 * 16 + 1023) / 1024 * 1024;
    // (rows that a tile lacks are read behind the last stage too)
    const int behind = (kTile - a.tile) * (128 + 16 * a.panels);
    a.ring = (kSmem - 1024 - behind - a.part_bytes) / a.stage_bytes;
    const int sf_cols = (p.n_w + (columns > 128 ? 2 : 1)) * 16 * a.panels;
    a.d_bufs = 2 * p.n_w * columns + 2 * sf_cols <= kTmemCols ? 2 : 1;
    a.sf_bufs = (kTmemCols - a.d_bufs * p.n_w * columns) / sf_cols;
    if (a.panels == 1 || (n_panels % a.panels == 0 && a.ring >= p.n_w + 2 && a.sf_bufs >= 3)) break;
  }
  if (a.ring > kMaxStages) a.ring = kMaxStages;
  if (a.sf_bufs > a.ring) a.sf_bufs = a.ring;
  if (a.ring < 2 || a.sf_bufs < 1) return NVFP4_ERR_UNSUPPORTED;   // (three stages fit at least)
  a.n_stages = n_panels / a.panels;
  const uint64_t rows_w = (uint64_t)(p.n_experts * p.d_out), pitch = (uint64_t)p.d_in / 2;
  for (int m = 0; m < p.n_w; ++m)
    for (int b = 0; b < 2; ++b) {
      const uint32_t box_rows = b == 0 ? a.tile : 32;
      const uint64_t dc[3] = {128, rows_w, (uint64_t)n_panels}, sc[2] = {pitch, 128};
      const uint32_t bc[3] = {128, box_rows, b == 0 ? (uint32_t)a.panels : 1u};
      const uint64_t ds[2] = {(uint64_t)p.nb, rows_w}, ss[1] = {(uint64_t)p.nb};
      const uint32_t bs[2] = {16u * a.panels, box_rows};
      if (!encode_tmap_nd(&a.codes[m][b], p.codes[m], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dc, sc, bc,
                          CU_TENSOR_MAP_SWIZZLE_128B) ||
          !encode_tmap_2d(&a.scales[m][b], p.scales[m], CU_TENSOR_MAP_DATA_TYPE_UINT8, ds, ss, bs,
                          CU_TENSOR_MAP_SWIZZLE_NONE))
        return NVFP4_ERR_CUDA;
    }
  auto kernel = a.split == 2 ? (p.n_w == 2 ? product_fp4_kernel<2, 2> : product_fp4_kernel<1, 2>)
                             : (p.n_w == 2 ? product_fp4_kernel<2, 1> : product_fp4_kernel<1, 1>);
  const int threads = p.n_w == 2 ? Roles<2>::kThreads : Roles<1>::kThreads;
  NVFP4_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas * a.split));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  NVFP4_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, a));
  count_launches(2);
  return NVFP4_OK;
}

nvfp4_status launch_product_fp4(const Product& p, void* ws, cudaStream_t st) {
  const int64_t parts = (p.n_rows + kMaxRows - 1) / kMaxRows;
  const int64_t rows = (p.n_rows + parts - 1) / parts;
  for (int64_t r = 0; r < p.n_rows; r += rows) {
    Product q = p;
    q.row0 = r;
    q.n_rows = p.n_rows - r < rows ? p.n_rows - r : rows;
    if (p.rows)
      q.rows = p.rows + r;
    else
      q.X = static_cast<const char*>(p.X) + r * p.d_in * (int64_t)sizeof(__nv_bfloat16);
    q.Y = static_cast<char*>(p.Y) + r * p.d_out * (p.y_bf16 ? 2 : 4);
    if (nvfp4_status s = launch_part(q, ws, st)) return s;
  }
  return NVFP4_OK;
}

}  // namespace nvfp4
