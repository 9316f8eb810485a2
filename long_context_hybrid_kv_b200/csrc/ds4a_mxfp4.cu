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

// A thread a 32-value block.  64 bytes in, 16.5 out: bound by HBM.
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(int n_rows, int rows_pad, int K, const uint16_t* in,
                                                             int64_t in_stride, uint8_t* codes, uint8_t* scales) {
  pdl_trigger();
  const int kb = K / kMxBlock;
  const int64_t n = (int64_t)rows_pad * kb;
  bool waited = false;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / kb;
    const int blk = (int)(i - row * kb);
    int code = 0;
    uint4 c = make_uint4(0, 0, 0, 0);
    if (row < n_rows) {
      const uint4* p = reinterpret_cast<const uint4*>(in + row * in_stride + blk * kMxBlock);
      uint4 u[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) u[q] = p[q];
      float v[32];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const unsigned int x[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = bf2x2_to_f2(x[k]);
          v[8 * q + 2 * k] = f.x;
          v[8 * q + 2 * k + 1] = f.y;
        }
      }
      code = mx_block(v, &c);
    }
    if (!waited) pdl_wait();  // (the rows are an input; what is written may still be read)
    waited = true;
    if (row < n_rows) *reinterpret_cast<uint4*>(codes + row * (K / 2) + blk * 16) = c;
    scales[mxfp4_scale_at(row, blk, K)] = (uint8_t)code;
  }
  if (!waited) pdl_wait();
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
          // the weights are an input: the first stages' come while the
          // kernel before this one ends
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
                                  uint8_t* scales, cudaStream_t s) {
  const int pad = (n_rows + 127) / 128 * 128;
  const int64_t blocks = ((int64_t)pad * (K / kMxBlock) + 255) / 256;
  const int grid = (int)(blocks < 148 * 8 ? blocks : 148 * 8);
  TraceScope tr("quantize_mxfp4", s);
  return launch_pdl(quantize_mxfp4_kernel, dim3(grid), dim3(256), 0, s, n_rows, pad, K, in, in_stride, codes, scales);
}

// Few rows cannot fill the SMs with tiles; K is then split until they do, as
// long as a split keeps four steps or more (a full ring of loads).
int mxfp4_ksplit(int M, int N, int K) {
  const int tiles = (M + kBM - 1) / kBM * (N / kBN), steps = K / kBK;
  int ks = 1;
  while (ks * 2 * tiles <= 148 && steps / (ks * 2) >= 4) ks *= 2;
  return ks;
}

cudaError_t launch_mxfp4_product(const Mxfp4Product& q, cudaStream_t s) {
  CUtensorMap amap, bmap;
  if (!encode_codes(&amap, q.a_codes, (uint64_t)q.a_cols / 2, (uint64_t)q.M, kBM)) return cudaErrorInvalidValue;
  if (!encode_codes(&bmap, q.b_codes, (uint64_t)q.K / 2, (uint64_t)q.N, kBN)) return cudaErrorInvalidValue;
  GemmParams p;
  p.M = q.M; p.N = q.N; p.k_steps = q.K / kBK; p.n_per_group = q.n_per_group;
  p.a_blocks = q.a_cols / 128; p.b_blocks = q.K / 128;
  p.a_group_blocks = q.n_per_group < q.N ? q.K / 128 : 0;
  p.m_tiles = (q.M + kBM - 1) / kBM; p.n_tiles = q.N / kBN;
  p.ksplit = mxfp4_ksplit(q.M, q.N, q.K);
  p.steps_per_split = (p.k_steps + p.ksplit - 1) / p.ksplit;
  p.ksplit = (p.k_steps + p.steps_per_split - 1) / p.steps_per_split;  // no empty split
  p.n_units = p.m_tiles * p.n_tiles * p.ksplit;
  p.a_scales = q.a_scales; p.b_scales = q.b_scales;
  p.y = q.y; p.q_codes = q.q_codes; p.q_scales = q.q_scales; p.part = q.part; p.err = q.err;
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
