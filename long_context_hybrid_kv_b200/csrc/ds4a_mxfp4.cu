// Microscaled 4-bit quantisation and product of the grouped output projection
// (layout in ds4a_mxfp4.cuh).
//
//   D[m][n] = sum_k (a[m][k] 2^sa[m][k/32]) (b[n][k] 2^sb[n][k/32])
//
// The tensor core takes the scales itself: tcgen05.mma kind::mxf4 multiplies
// E2M1 operands from shared memory (two values a byte, K-major, 128-byte
// swizzle) by E8M0 scales from tensor memory, one for 32 values of K, and adds
// in float32.  Every operand value is exact, so the only rounding before the
// output is the accumulation's.
//
// Tile 128 rows x 256 outputs, K in steps of 256 (128 bytes of codes a row; 2
// KiB + 1 KiB of scales), four stages of 51 KiB.  An MMA is 128 x 256 x 64; a
// step is four of them after six copies of 512 bytes of scales into tensor
// memory, which keep their order with the MMAs.  Two accumulators of 256
// columns and the scales' 24 do not fit the 512 columns, so the accumulators
// overlap in 32 columns, which an epilogue reads first: the next tile waits
// for those, not for the rest.
//
// Thread block (192 threads, one per SM, persistent over work units):
//   warp 0     lane 0: TMA (codes) and bulk copies (scales)
//   warp 1     TMEM allocation; issues scale copies and MMAs
//   warps 2-5  epilogue: a thread a row, 32 outputs at a time, which are just
//              one block of a next product's operand
#include <cuda.h>
#include <cudaTypedefs.h>

#include "ds4a_mxfp4.cuh"
#include "ds4a_tc.cuh"

namespace ds4a {
namespace {

using namespace tc;

// 32 values -> 16 bytes of codes, and the scale's code
__device__ __forceinline__ int mx_block(const float (&v)[32], uint4* codes) {
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) amax = fmaxf(amax, fabsf(v[k]));
  const int code = mx_scale_code<true>(amax);
  const float inv = mx_inv_scale(code);
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    w[q] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[q] |= to_e2m1x2(v[8 * q + 2 * k] * inv, v[8 * q + 2 * k + 1] * inv) << (8 * k);
  }
  *codes = make_uint4(w[0], w[1], w[2], w[3]);
  return code;
}

// the same for 32 bf16 values: the largest magnitude as 16-bit integers, two at
// a time (positive floats order like their bits)
__device__ __forceinline__ int mx_block_words(const uint4 (&u)[4], uint4* codes) {
  unsigned int m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    m = __vmaxu2(m, u[q].x & 0x7FFF7FFFu);
    m = __vmaxu2(m, u[q].y & 0x7FFF7FFFu);
    m = __vmaxu2(m, u[q].z & 0x7FFF7FFFu);
    m = __vmaxu2(m, u[q].w & 0x7FFF7FFFu);
  }
  m = max(m & 0xFFFFu, m >> 16);
  const int code = mx_scale_code<true>(__uint_as_float(m << 16));
  const float inv = mx_inv_scale(code);
  const float2 inv2 = make_float2(inv, inv);
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const unsigned int x[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
    w[q] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = mul_f2(bf2x2_to_f2(x[k]), inv2);
      w[q] |= to_e2m1x2(f.x, f.y) << (8 * k);
    }
  }
  *codes = make_uint4(w[0], w[1], w[2], w[3]);
  return code;
}

// A thread a 32-value block.  64 bytes in, 16.5 out: bound by HBM (16384 x
// 32768 values in 223 us, 6.1 TB/s).  kEarly: the next kernel may start while
// this one runs.  Only for a next kernel that waits before it reads the result:
// the products load their weights before they wait, so a matrix that may become
// a weight is quantised without it, and the next kernel starts when it is done.
template <bool kEarly>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(int n_rows, int rows_pad, int K, const uint16_t* in,
                                                             int64_t in_stride, uint8_t* codes, uint8_t* scales) {
  if (kEarly) pdl_trigger();
  pdl_wait();
  const int kb = K / kMxBlock;
  const int64_t n = (int64_t)rows_pad * kb;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / kb;
    const int blk = (int)(i - row * kb);
    int code = 0;
    uint4 c = make_uint4(0, 0, 0, 0);
    if (row < n_rows) {
      uint4 u[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) u[q] = reinterpret_cast<const uint4*>(in + row * in_stride + blk * kMxBlock)[q];
      code = mx_block_words(u, &c);
    }
    if (row < n_rows) *reinterpret_cast<uint4*>(codes + row * (K / 2) + blk * 16) = c;
    scales[mxfp4_scale_at(row, blk, K)] = (uint8_t)code;
  }
}

constexpr int kBM = 128, kBN = 256, kBK = 256;
constexpr int kStages = 4;
constexpr int kThreads = 192;
constexpr uint32_t kStageA = kBM * kBK / 2;        // 16 KiB
constexpr uint32_t kStageB = kBN * kBK / 2;        // 32 KiB
constexpr uint32_t kOffSA = kStageA + kStageB;     // 2 blocks of 512 bytes
constexpr uint32_t kOffSB = kOffSA + 1024;         // 2 row ranges x 2 blocks
constexpr uint32_t kStageBytes = kOffSB + 2048;    // 51 KiB
constexpr uint32_t kOffBar = kStages * kStageBytes;
constexpr uint32_t kOffMisc = kOffBar + 256;
constexpr uint32_t kSmemBytes = kOffMisc + 64 + 1024;
static_assert(kStageBytes % 1024 == 0 && kSmemBytes <= 232448, "shared memory");
constexpr int kBand = 8;  // row tiles per raster band
// tensor memory columns
constexpr uint32_t kAcc1 = 224;   // the second accumulator: columns 224 .. 479
constexpr uint32_t kColSA = 480;  // 2 x 4
constexpr uint32_t kColSB = 488;  // 2 x 8

enum Bar { kFull = 0, kEmpty = kFull + kStages, kAccFull0 = kEmpty + kStages, kAccFull1, kAccEmpty0, kAccEmpty1, kShared0,
           kShared1, kDrain, kNumBars };

struct GemmParams {
  int M, N, k_steps;    // rows, outputs, K / 256
  int n_per_group;
  int64_t a_blocks, b_blocks;  // 128-value blocks of a row of A, of B
  int a_group_blocks;   // of a group's slice of A
  int m_tiles, n_tiles, ksplit, steps_per_split, n_units;
  const uint8_t *a_scales, *b_scales;
  uint16_t* y;
  uint8_t *q_codes, *q_scales;
  float* part;
  unsigned int* err;
};

struct Unit {
  int m0, n0, k0, k1, ks, a_blk;  // a_blk: first 128-value block of the group's slice of A
};
__device__ __forceinline__ Unit make_unit(const GemmParams& p, int u) {
  Unit w;
  w.ks = u % p.ksplit;
  const int v = u / p.ksplit;
  const int band = v / (kBand * p.n_tiles);
  const int bm = min(kBand, p.m_tiles - band * kBand);
  const int in_band = v - band * kBand * p.n_tiles;
  const int nt = in_band / bm;
  w.m0 = (band * kBand + in_band % bm) * kBM;
  w.n0 = nt * kBN;
  w.k0 = w.ks * p.steps_per_split;
  w.k1 = min(p.k_steps, w.k0 + p.steps_per_split);
  w.a_blk = w.n0 / p.n_per_group * p.a_group_blocks;
  return w;
}

// Instruction descriptor of kind::mxf4: E2M1 A and B, E8M0 scales, N >> 3 at
// bit 17, M >> 7 at bit 27; the scales' place in their 4-byte columns (0 or 2,
// for two scales an MMA) at bits 4 (B) and 29 (A).
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27) | (sf << 29);
}
__device__ __forceinline__ void mma_mxf4_elect(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                               uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %6, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// 512 bytes of scales (32 rows of 16 bytes) -> 4 columns, in all four lane quarters
__device__ __forceinline__ void scales_to_tmem_elect(uint32_t dst, uint64_t desc) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n @q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(dst),
      "l"(desc)
      : "memory");
}
__device__ __forceinline__ void commit_elect(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
// no swizzle: 8 rows of 16 bytes a core matrix, 128 bytes to the next 8 rows
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(16u >> 4) << 16) | ((uint64_t)(128u >> 4) << 32) | (1ull << 46);
}

enum Out { kOutBf16 = 0, kOutMx = 1, kOutPart = 2 };

template <int kOut>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                      const __grid_constant__ GemmParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + kOffBar + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned int* err = p.err;

  pdl_trigger();
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kFull + s), 1);
      mbar_init(bar(kEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kAccFull0 + i), 1);
      mbar_init(bar(kAccEmpty0 + i), 128);
      mbar_init(bar(kShared0 + i), 128);
    }
    mbar_init(bar(kDrain), 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // =================== copies ===================
    if (lane == 0) {
      uint32_t kt = 0;
      bool waited = false;
      for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
        const Unit w = make_unit(p, u);
        for (int k = w.k0; k < w.k1; ++k, ++kt) {
          const uint32_t s = kt % kStages, dst = sbase + s * kStageBytes, full = bar(kFull + s);
          if (kt >= (uint32_t)kStages && !mbar_wait(bar(kEmpty + s), (kt / kStages - 1) & 1u, abort_flag, err)) break;
          mbar_expect_tx(full, kStageBytes);
          // the weights are an input (their quantiser lets no kernel start
          // before it is done): the first stages' come while the kernel
          // before this one ends
          tma_load_2d(dst + kStageA, &bmap, k * (kBK / 2), w.n0, full);
          const uint8_t* sb = p.b_scales + ((int64_t)(w.n0 / 128) * p.b_blocks + 2 * k) * 512;
          bulk_g2s(dst + kOffSB, sb, 1024, full);
          bulk_g2s(dst + kOffSB + 1024, sb + p.b_blocks * 512, 1024, full);
          if (!waited && (kt + 1 == (uint32_t)kStages || (k + 1 == w.k1 && u + (int)gridDim.x >= p.n_units))) {
            // everything that is left of these stages: A
            pdl_wait();
            waited = true;
            uint32_t j = 0;
            for (int u2 = blockIdx.x; j <= kt; u2 += gridDim.x) {
              const Unit v = make_unit(p, u2);
              for (int k2 = v.k0; k2 < v.k1 && j <= kt; ++k2, ++j) {
                const uint32_t d2 = sbase + j * kStageBytes, f2 = bar(kFull + j);
                tma_load_2d(d2, &amap, (v.a_blk + 2 * k2) * 64, v.m0, f2);
                bulk_g2s(d2 + kOffSA, p.a_scales + ((int64_t)(v.m0 / 128) * p.a_blocks + v.a_blk + 2 * k2) * 512, 1024, f2);
              }
            }
          } else if (waited) {
            tma_load_2d(dst, &amap, (w.a_blk + 2 * k) * 64, w.m0, full);
            bulk_g2s(dst + kOffSA, p.a_scales + ((int64_t)(w.m0 / 128) * p.a_blocks + w.a_blk + 2 * k) * 512, 1024, full);
          }
        }
      }
      if (!waited) pdl_wait();
      // no copy into this block's shared memory is left in flight at exit
      for (uint32_t j = kt > (uint32_t)kStages ? kt - kStages : 0; j < kt; ++j)
        mbar_drain(bar(kFull + j % kStages), (j / kStages) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // =================== scale copies and MMAs ===================
    pdl_wait();
    uint32_t kt = 0, at = 0;
    for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
      const Unit w = make_unit(p, u);
      if (w.k1 <= w.k0) continue;
      const uint32_t ab = at & 1u, acc = tmem + ab * kAcc1;
      // this accumulator is free, and the other's epilogue has read the
      // columns that the two share
      if (at >= 2) mbar_wait(bar(kAccEmpty0 + ab), ((at >> 1) - 1) & 1u, abort_flag, err);
      if (at >= 1) mbar_wait(bar(kShared0 + (ab ^ 1u)), ((at - 1) >> 1) & 1u, abort_flag, err);
      __syncwarp();
      tc_fence_after();
      for (int k = w.k0; k < w.k1; ++k, ++kt) {
        const uint32_t s = kt % kStages, st = sbase + s * kStageBytes;
        mbar_wait(bar(kFull + s), (kt / kStages) & 1u, abort_flag, err);
        __syncwarp();
        tc_fence_after();
        const uint64_t sa = sdesc_scales(st + kOffSA), sb = sdesc_scales(st + kOffSB);
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
          scales_to_tmem_elect(tmem + kColSA + 4 * i, sa + ((512u * i) >> 4));
          scales_to_tmem_elect(tmem + kColSB + 8 * i, sb + ((512u * i) >> 4));
          scales_to_tmem_elect(tmem + kColSB + 8 * i + 4, sb + ((1024u + 512u * i) >> 4));
        }
        const uint64_t da = sdesc_sw128(st, 16, 1024), db = sdesc_sw128(st + kStageA, 16, 1024);
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          mma_mxf4_elect(acc, da + ((32u * i) >> 4), db + ((32u * i) >> 4), idesc_mxf4(kBM, kBN, 2 * (i & 1)),
                         tmem + kColSA + 4 * (i >> 1), tmem + kColSB + 8 * (i >> 1), k > w.k0 || i > 0 ? 1u : 0u);
        commit_elect(bar(kEmpty + s));
      }
      commit_elect(bar(kAccFull0 + ab));
      ++at;
    }
    commit_elect(bar(kDrain));
    mbar_wait(bar(kDrain), 0, abort_flag, err);
    __syncwarp();
  } else {
    // =================== epilogue ===================
    pdl_wait();
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the tile
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    uint32_t at = 0;
    for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
      const Unit w = make_unit(p, u);
      const int row = w.m0 + r;
      const bool live = row < p.M;
      if (w.k1 <= w.k0) continue;  // (only the last split, whose partial sums then are not added)
      const uint32_t ab = at & 1u;
      mbar_wait(bar(kAccFull0 + ab), (at >> 1) & 1u, abort_flag, err);
      __syncwarp();
      tc_fence_after();
      uint32_t sc = 0;  // scale codes of four blocks
#pragma unroll 1
      for (int i = 0; i < kBN / 32; ++i) {
        // the shared columns first: they are the last of the first
        // accumulator and the first of the second
        const int c = ab == 0 ? (i + 7) & 7 : i;
        float v[32];
        tmem_ld32(t_lane + ab * kAcc1 + (uint32_t)(c * 32), v);
        tmem_ld_wait();
        if (i == 0) {
          tc_fence_before();
          mbar_arrive(bar(kShared0 + ab));
        }
        const int col = w.n0 + c * 32;
        if (kOut == kOutBf16) {
          if (live) {
            uint4* dst = reinterpret_cast<uint4*>(p.y + (int64_t)row * p.N + col);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              dst[q] = make_uint4(f2_to_bf2x2(v[8 * q], v[8 * q + 1]), f2_to_bf2x2(v[8 * q + 2], v[8 * q + 3]),
                                  f2_to_bf2x2(v[8 * q + 4], v[8 * q + 5]), f2_to_bf2x2(v[8 * q + 6], v[8 * q + 7]));
          }
        } else if (kOut == kOutMx) {
          uint4 codes;
          const int code = mx_block(v, &codes);
          if (live) *reinterpret_cast<uint4*>(p.q_codes + (int64_t)row * (p.N / 2) + col / 2) = codes;
          // (padding rows are sums of zeros: their scales are written too)
          p.q_scales[mxfp4_scale_at(row, col / 32, p.N)] = (uint8_t)(live ? code : 0);
          (void)sc;
        } else if (live) {
          float4* dst = reinterpret_cast<float4*>(p.part + ((int64_t)w.ks * p.M + row) * p.N + col);
#pragma unroll
          for (int q = 0; q < 8; ++q) dst[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      }
      tc_fence_before();
      mbar_arrive(bar(kAccEmpty0 + ab));
      ++at;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Split K: the partial sums in split order -> bf16, or quantised again; a
// thread a 32-value block.
template <bool kMx>
__global__ void __launch_bounds__(128) mxfp4_finish_kernel(const GemmParams p) {
  pdl_trigger();
  pdl_wait();
  const int kb = p.N / 32;
  const int64_t n = (int64_t)(kMx ? p.m_tiles * kBM : p.M) * kb;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int row = (int)(i / kb), blk = (int)(i - (int64_t)row * kb);
    float v[32];
#pragma unroll
    for (int q = 0; q < 32; ++q) v[q] = 0.f;
    if (row < p.M)
      for (int s = 0; s < p.ksplit; ++s) {
        const float4* src = reinterpret_cast<const float4*>(p.part + ((int64_t)s * p.M + row) * p.N + blk * 32);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 x = src[q];
          v[4 * q] += x.x;
          v[4 * q + 1] += x.y;
          v[4 * q + 2] += x.z;
          v[4 * q + 3] += x.w;
        }
      }
    if (kMx) {
      uint4 codes;
      const int code = mx_block(v, &codes);
      if (row < p.M) *reinterpret_cast<uint4*>(p.q_codes + (int64_t)row * (p.N / 2) + blk * 16) = codes;
      p.q_scales[mxfp4_scale_at(row, blk, p.N)] = (uint8_t)(row < p.M ? code : 0);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(p.y + (int64_t)row * p.N + blk * 32);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        dst[q] = make_uint4(f2_to_bf2x2(v[8 * q], v[8 * q + 1]), f2_to_bf2x2(v[8 * q + 2], v[8 * q + 3]),
                            f2_to_bf2x2(v[8 * q + 4], v[8 * q + 5]), f2_to_bf2x2(v[8 * q + 6], v[8 * q + 7]));
    }
  }
}

// ---------------------------------------------------------------------------
// Up to 128 rows (a decode batch): the weights stream past once, and what
// counts is the chain of latencies.  K is split over a cluster of up to four
// blocks (a cluster of eight waited for room: 23 us instead of 15 for the
// second product), tiles are 256 or 128 outputs wide, whichever fills the SMs
// better, and a block's ring holds half of its loads or all of them, the
// weights' out before the kernel ahead has ended.  The first product quantises
// its rows of o straight into the operand (a 32-value block is one 16-byte
// piece of the swizzled row), four warps a stage and two blocks a thread at a
// time (four took 2 us longer for 77 rows: at a first pass instructions cost
// more than waiting), so no kernel does it before.  The blocks of a cluster leave their float sums in shared memory and
// each adds a share of the columns, in the order of the splits, and finishes
// it: two launches in all instead of five.  64 heads x 512 -> 8 x 1024 -> 4096,
// both products: 16.0 us for one row, 17.5 for 16, 23.4 for 77, 27.7 for 128;
// the weights alone take 5.5 us.
// ---------------------------------------------------------------------------
constexpr int kQuantWarps = 16;  // that quantise; the first four of them read the sums
constexpr int kSmallThreads = 64 + 32 * kQuantWarps;
template <int kN>
struct Small {  // a tile kN outputs wide
  static constexpr int kRing = kN == 256 ? 4 : 6;
  static constexpr uint32_t kB = kN * kBK / 2, kSA = kStageA + kB, kSB = kSA + 1024, kStage = kSB + kN * 8;
  static constexpr uint32_t kBar = kRing * kStage, kMisc = kBar + 256, kBytes = kMisc + 64 + 1024;
  static constexpr uint32_t kPitch = kN * 4 + 16;  // bytes of a row of sums: rows fall into different banks
  static_assert(kStage % 1024 == 0 && kBytes <= 232448 && 128 * kPitch <= kBar, "shared memory");
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// kQuant: A is quantised from o (bf16 [M][o_cols]) here; kMx: the result goes
// out quantised, else as bf16
template <int kN, bool kQuant, bool kMx>
__global__ void __launch_bounds__(kSmallThreads, 1)
    mxfp4_small_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                       const __grid_constant__ GemmParams p, const uint16_t* __restrict__ o, int64_t o_cols) {
  using S = Small<kN>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  auto full = [&](int j) { return sbase + S::kBar + 8u * (uint32_t)(j % S::kRing); };
  auto empty = [&](int j) { return sbase + S::kBar + 64u + 8u * (uint32_t)(j % S::kRing); };
  const uint32_t acc_full = sbase + S::kBar + 128u;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned int* err = p.err;
  // the blocks of a cluster are the splits of one tile
  const int split = blockIdx.x % p.ksplit, n0 = blockIdx.x / p.ksplit * kN;
  const int k0 = split * p.steps_per_split, steps = max(0, min(p.k_steps, k0 + p.steps_per_split) - k0);
  const int a_blk = n0 / p.n_per_group * p.a_group_blocks;

  pdl_trigger();
  if (tid == 0) {
    *abort_flag = 0;
    for (int j = 0; j < S::kRing; ++j) {
      mbar_init(full(j), kQuant ? 8 * kQuantWarps + 1 : 1);
      mbar_init(empty(j), 1);
    }
    mbar_init(acc_full, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      auto load_b = [&](int j) {
        const uint32_t dst = sbase + (j % S::kRing) * S::kStage;
        mbar_expect_tx(full(j), S::kB + kN * 8u + (kQuant ? 0u : kStageA + 1024u));
        tma_load_2d(dst + kStageA, &bmap, (k0 + j) * (kBK / 2), n0, full(j));
        const uint8_t* sb = p.b_scales + ((int64_t)(n0 / 128) * p.b_blocks + 2 * (k0 + j)) * 512;
        bulk_g2s(dst + S::kSB, sb, 1024, full(j));
        if (kN == 256) bulk_g2s(dst + S::kSB + 1024, sb + p.b_blocks * 512, 1024, full(j));
      };
      auto load_a = [&](int j) {
        if (kQuant) return;
        const uint32_t dst = sbase + (j % S::kRing) * S::kStage;
        tma_load_2d(dst, &amap, (a_blk + 2 * (k0 + j)) * 64, 0, full(j));
        bulk_g2s(dst + S::kSA, p.a_scales + ((int64_t)a_blk + 2 * (k0 + j)) * 512, 1024, full(j));
      };
      const int first = min(steps, S::kRing);
      for (int j = 0; j < first; ++j) load_b(j);
      pdl_wait();
      for (int j = 0; j < first; ++j) load_a(j);
      int sent = first;
      for (; sent < steps; ++sent) {
        if (!mbar_wait(empty(sent), (sent / S::kRing - 1) & 1u, abort_flag, err)) break;
        load_b(sent);
        load_a(sent);
      }
      for (int j = max(0, sent - S::kRing); j < sent; ++j) mbar_drain(full(j), (j / S::kRing) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    for (int j = 0; j < steps; ++j) {
      const uint32_t st = sbase + (j % S::kRing) * S::kStage;
      mbar_wait(full(j), (j / S::kRing) & 1u, abort_flag, err);
      __syncwarp();
      tc_fence_after();
      const uint64_t sa = sdesc_scales(st + S::kSA), sb = sdesc_scales(st + S::kSB);
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        scales_to_tmem_elect(tmem + kColSA + 4 * i, sa + ((512u * i) >> 4));
        scales_to_tmem_elect(tmem + kColSB + 8 * i, sb + ((512u * i) >> 4));
        if (kN == 256) scales_to_tmem_elect(tmem + kColSB + 8 * i + 4, sb + ((1024u + 512u * i) >> 4));
      }
      const uint64_t da = sdesc_sw128(st, 16, 1024), db = sdesc_sw128(st + kStageA, 16, 1024);
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
        mma_mxf4_elect(tmem, da + ((32u * i) >> 4), db + ((32u * i) >> 4), idesc_mxf4(kBM, kN, 2 * (i & 1)),
                       tmem + kColSA + 4 * (i >> 1), tmem + kColSB + 8 * (i >> 1), j > 0 || i > 0 ? 1u : 0u);
      commit_elect(empty(j));
    }
    commit_elect(acc_full);
    mbar_wait(acc_full, 0, abort_flag, err);  // every MMA has finished before the block exits
    __syncwarp();
  } else {
    pdl_wait();
    if (kQuant) {
      // warps 2 + q, 6 + q, ... quantise the steps q, q + 4, ...  (Rows behind the
      // last are left as they are: whatever lies there only reaches rows of
      // the sums that are not looked at.)
      const int t = (warp - 2) / 4 * 32 + lane;
      constexpr int kT = 8 * kQuantWarps;
      for (int j = (warp - 2) & 3; j < steps; j += 4) {
        if (j >= S::kRing) mbar_wait(empty(j), (j / S::kRing - 1) & 1u, abort_flag, err);
        unsigned char* st = smem + (j % S::kRing) * S::kStage;
        const uint16_t* src = o + ((int64_t)a_blk + 2 * (k0 + j)) * 128;
        for (int i0 = t; i0 < p.M * 8; i0 += 2 * kT) {
          uint4 u[2][4];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int i = min(i0 + kT * q, p.M * 8 - 1);
#pragma unroll
            for (int c = 0; c < 4; ++c) u[q][c] = reinterpret_cast<const uint4*>(src + (i >> 3) * o_cols + (i & 7) * 32)[c];
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int i = i0 + kT * q, row = i >> 3, blk = i & 7;
            if (i >= p.M * 8) break;
            uint4 codes;
            const int code = mx_block_words(u[q], &codes);
            *reinterpret_cast<uint4*>(st + sw128((uint32_t)row, (uint32_t)blk)) = codes;
            st[S::kSA + (blk >> 2) * 512 + (row & 31) * 16 + (row >> 5) * 4 + (blk & 3)] = (unsigned char)code;
          }
        }
        fence_async_smem();
        mbar_arrive(full(j));
      }
    }
    if (warp < 6) {
      // the sums of this split into shared memory (the ring has been read)
      const int quarter = warp & 3, r = quarter * 32 + lane;
      mbar_wait(acc_full, 0, abort_flag, err);
      __syncwarp();
      tc_fence_after();
      if (quarter * 32 < p.M) {
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < kN / 32; c += 2) {
          float v[32], x[32];
          tmem_ld32(t_lane + (uint32_t)(c * 32), v);
          tmem_ld32(t_lane + (uint32_t)(c * 32 + 32), x);
          tmem_ld_wait();
          if (r < p.M) {
            float4* dst = reinterpret_cast<float4*>(smem + r * S::kPitch + c * 128);
#pragma unroll
            for (int q = 0; q < 8; ++q) dst[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
#pragma unroll
            for (int q = 0; q < 8; ++q) dst[8 + q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  pdl_wait();
  if (p.ksplit > 1) cluster_sync();
  // this block's columns of the tile: eight threads a 32-column block
  const int cols = kN / p.ksplit, c_base = split * cols, per = cols / 4, sh = __ffs(per) - 1;  // threads a row (ksplit 1, 2 or 4)
  const int used = (p.k_steps + p.steps_per_split - 1) / p.steps_per_split;  // splits with steps
  // (of the operand's padding rows neither codes nor scales are written: they
  // only reach padding rows of the next sums)
#pragma unroll 1
  for (int i = tid; i < p.M * per; i += kSmallThreads) {
    const int row = i >> sh, c = c_base + (i & (per - 1)) * 4, col = n0 + c;
    const uint32_t at = (uint32_t)row * S::kPitch + (uint32_t)c * 4u;
    float4 y[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      y[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < used) y[s] = p.ksplit > 1 ? ld_cluster4(sbase + at, (uint32_t)s) : *reinterpret_cast<const float4*>(smem + at);
    }
    float4 x = y[0];
#pragma unroll
    for (int s = 1; s < 4; ++s) {
      x.x += y[s].x;
      x.y += y[s].y;
      x.z += y[s].z;
      x.w += y[s].w;
    }
    if (!kMx) {
      *reinterpret_cast<uint2*>(p.y + (int64_t)row * p.N + col) = make_uint2(f2_to_bf2x2(x.x, x.y), f2_to_bf2x2(x.z, x.w));
    } else {
      // (M per is a multiple of eight: all threads of a block are here)
      const unsigned int eight = 0xFFu << (lane & 24);
      float amax = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
      for (int q = 1; q < 8; q <<= 1) amax = fmaxf(amax, __shfl_xor_sync(eight, amax, q));
      const int code = mx_scale_code<true>(amax);
      const float inv = mx_inv_scale(code);
      const uint32_t two = to_e2m1x2(x.x * inv, x.y * inv) | (to_e2m1x2(x.z * inv, x.w * inv) << 8);
      *reinterpret_cast<uint16_t*>(p.q_codes + (int64_t)row * (p.N / 2) + col / 2) = (uint16_t)two;
      if ((tid & 7) == 0) p.q_scales[mxfp4_scale_at(row, col / 32, p.N)] = (uint8_t)code;
    }
  }
  if (p.ksplit > 1) cluster_sync();  // no block leaves while another may still read its sums
}

// codes as rows of bytes, boxes of 128 bytes x box_rows
bool encode_codes(CUtensorMap* map, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = get_encode();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kOut>
cudaError_t launch_gemm_kernel(const CUtensorMap& amap, const CUtensorMap& bmap, const GemmParams& p, cudaStream_t s) {
  static std::atomic<int> cache[kMaxDevices];
  const cudaError_t e = ensure_smem(mxfp4_gemm_kernel<kOut>, (int)kSmemBytes, cache);
  if (e != cudaSuccess) return e;
  TraceScope tr("mxfp4_gemm", s);
  return launch_pdl(mxfp4_gemm_kernel<kOut>, dim3(min(p.n_units, 148)), dim3(kThreads), kSmemBytes, s, amap, bmap, p);
}

}  // namespace

cudaError_t launch_quantize_mxfp4(int n_rows, int K, const uint16_t* in, int64_t in_stride, uint8_t* codes,
                                  uint8_t* scales, bool early, cudaStream_t s) {
  const int pad = (n_rows + 127) / 128 * 128;
  const int64_t blocks = ((int64_t)pad * (K / kMxBlock) + 255) / 256;
  const int grid = (int)(blocks < 148 * 8 ? blocks : 148 * 8);
  TraceScope tr("quantize_mxfp4", s);
  return launch_pdl(early ? quantize_mxfp4_kernel<true> : quantize_mxfp4_kernel<false>, dim3(grid), dim3(256), 0, s,
                    n_rows, pad, K, in, in_stride, codes, scales);
}

// Few rows cannot fill the SMs with tiles; K is then split until they do, as
// long as a split keeps four steps or more (a full ring of loads).
int mxfp4_ksplit(int M, int N, int K) {
  const int tiles = (M + kBM - 1) / kBM * (N / kBN), steps = K / kBK;
  int ks = 1;
  while (ks * 2 * tiles <= 148 && steps / (ks * 2) >= 4) ks *= 2;
  return ks;
}

bool mxfp4_small(int M) { return M <= kBM; }

template <int kN, bool kQuant, bool kMx>
static cudaError_t launch_small_kernel(const CUtensorMap& amap, const CUtensorMap& bmap, const GemmParams& p,
                                       const uint16_t* o, int64_t o_cols, cudaStream_t s) {
  static std::atomic<int> cache[kMaxDevices];
  const cudaError_t e = ensure_smem(mxfp4_small_kernel<kN, kQuant, kMx>, (int)Small<kN>::kBytes, cache);
  if (e != cudaSuccess) return e;
  TraceScope tr("mxfp4_small", s);
  return launch_pdl_cluster(mxfp4_small_kernel<kN, kQuant, kMx>, dim3(p.N / kN * p.ksplit), dim3(kSmallThreads),
                            Small<kN>::kBytes, s, p.ksplit, amap, bmap, p, o, o_cols);
}

// The tile and the split of K (1, 2 or 4) that use most SMs, the wider tile
// if both use as many: it quantises, or loads, A half as often.
static cudaError_t launch_small(const Mxfp4Product& q, GemmParams p, cudaStream_t s) {
  int best = 0, wide = 1;
  p.ksplit = 1;
  for (int w = 1; w >= 0; --w)
    for (int ks = 1; ks <= 4; ks *= 2) {
      const int blocks = q.N / (w ? 256 : 128) * ks;
      if (ks > p.k_steps || (blocks > 148 && best > 0) || blocks <= best) continue;
      best = blocks;
      wide = w;
      p.ksplit = ks;
    }
  p.steps_per_split = (p.k_steps + p.ksplit - 1) / p.ksplit;
  CUtensorMap amap, bmap;
  memset(&amap, 0, sizeof(amap));
  if (!q.o && !encode_codes(&amap, q.a_codes, (uint64_t)q.a_cols / 2, (uint64_t)q.M, kBM)) return cudaErrorInvalidValue;
  if (!encode_codes(&bmap, q.b_codes, (uint64_t)q.K / 2, (uint64_t)q.N, wide ? 256 : 128)) return cudaErrorInvalidValue;
#define DS4A_SMALL(n, quant, mx) launch_small_kernel<n, quant, mx>(amap, bmap, p, q.o, q.a_cols, s)
  if (wide) {
    if (q.o) return q.y ? DS4A_SMALL(256, true, false) : DS4A_SMALL(256, true, true);
    return q.y ? DS4A_SMALL(256, false, false) : DS4A_SMALL(256, false, true);
  }
  if (q.o) return q.y ? DS4A_SMALL(128, true, false) : DS4A_SMALL(128, true, true);
  return q.y ? DS4A_SMALL(128, false, false) : DS4A_SMALL(128, false, true);
#undef DS4A_SMALL
}

cudaError_t launch_mxfp4_product(const Mxfp4Product& q, cudaStream_t s) {
  GemmParams p;
  p.M = q.M; p.N = q.N; p.k_steps = q.K / kBK; p.n_per_group = q.n_per_group;
  p.a_blocks = q.a_cols / 128; p.b_blocks = q.K / 128;
  p.a_group_blocks = q.n_per_group < q.N ? q.K / 128 : 0;
  p.a_scales = q.a_scales; p.b_scales = q.b_scales;
  p.y = q.y; p.q_codes = q.q_codes; p.q_scales = q.q_scales; p.part = q.part; p.err = q.err;
  p.m_tiles = (q.M + kBM - 1) / kBM; p.n_tiles = q.N / kBN;
  if (mxfp4_small(q.M)) return launch_small(q, p, s);
  CUtensorMap amap, bmap;
  if (!encode_codes(&amap, q.a_codes, (uint64_t)q.a_cols / 2, (uint64_t)q.M, kBM)) return cudaErrorInvalidValue;
  if (!encode_codes(&bmap, q.b_codes, (uint64_t)q.K / 2, (uint64_t)q.N, kBN)) return cudaErrorInvalidValue;
  p.ksplit = mxfp4_ksplit(q.M, q.N, q.K);
  p.steps_per_split = (p.k_steps + p.ksplit - 1) / p.ksplit;
  p.ksplit = (p.k_steps + p.steps_per_split - 1) / p.steps_per_split;  // no empty split
  p.n_units = p.m_tiles * p.n_tiles * p.ksplit;
  if (p.ksplit == 1)
    return q.y ? launch_gemm_kernel<kOutBf16>(amap, bmap, p, s) : launch_gemm_kernel<kOutMx>(amap, bmap, p, s);
  const cudaError_t e = launch_gemm_kernel<kOutPart>(amap, bmap, p, s);
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)(q.y ? q.M : p.m_tiles * kBM) * (q.N / 32), blocks = (n + 127) / 128;
  const int grid = (int)(blocks < 148 * 8 ? blocks : 148 * 8);
  TraceScope tr("mxfp4_finish", s);
  return q.y ? launch_pdl(mxfp4_finish_kernel<false>, dim3(grid), dim3(128), 0, s, p)
             : launch_pdl(mxfp4_finish_kernel<true>, dim3(grid), dim3(128), 0, s, p);
}

}  // namespace ds4a
