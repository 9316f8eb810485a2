// Microscaled 4-bit quantisation and product of the grouped output projection
// (layout in ds4a_mxfp4.cuh).
#include "ds4a_mxfp4.cuh"

namespace ds4a {
namespace {

// A thread a 32-value block: its largest magnitude, the smallest power-of-two
// scale that keeps it within 6, 16 bytes of codes.
template <bool kF32>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(int n_rows, int rows_pad, int K, const void* in, int64_t in_stride,
                                                             uint8_t* codes, uint8_t* scales) {
  pdl_trigger();
  pdl_wait();
  const int kb = K / kMxBlock;
  const int64_t n = (int64_t)rows_pad * kb;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / kb;
    const int blk = (int)(i % kb);
    uint8_t* sc = scales + mxfp4_scale_at(row, blk, K);
    if (row >= n_rows) {
      *sc = 0;
      continue;
    }
    float v[32];
    if (kF32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(in) + row * in_stride + blk * kMxBlock);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 f = p[q];
        v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
      }
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(in) + row * in_stride + blk * kMxBlock);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 u = p[q];
        const unsigned int x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = bf2x2_to_f2(x[k]);
          v[8 * q + 2 * k] = f.x;
          v[8 * q + 2 * k + 1] = f.y;
        }
      }
    }
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
    *reinterpret_cast<uint4*>(codes + row * (K / 2) + blk * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    *sc = (uint8_t)code;
  }
}

// The product on CUDA cores: 64 x 64 outputs a block, 4 x 4 a thread, one
// 32-value block of K a step; float32 sums.
__global__ void __launch_bounds__(256) mxfp4_product_kernel(const Mxfp4Product p) {
  __shared__ float as[32][68], bs[32][68];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64, tid = threadIdx.x;
  const int a_off = n0 / p.n_per_group * p.K;  // first A column of the group
  pdl_trigger();
  pdl_wait();
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += 32) {
    __syncthreads();
    const int r = tid >> 2, q = tid & 3;  // row, 8 values
    {
      uint32_t w = 0;
      float s = 0.f;
      if (m0 + r < p.M) {
        w = *reinterpret_cast<const uint32_t*>(p.a_codes + (int64_t)(m0 + r) * (p.a_cols / 2) + (a_off + k0) / 2 + 4 * q);
        s = mx_scale(p.a_scales[mxfp4_scale_at(m0 + r, (a_off + k0) / 32, p.a_cols)]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = e2m1x2_to_f2(w >> (8 * i));
        as[8 * q + 2 * i][r] = f.x * s;
        as[8 * q + 2 * i + 1][r] = f.y * s;
      }
      w = *reinterpret_cast<const uint32_t*>(p.b_codes + (int64_t)(n0 + r) * (p.K / 2) + k0 / 2 + 4 * q);
      s = mx_scale(p.b_scales[mxfp4_scale_at(n0 + r, k0 / 32, p.K)]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = e2m1x2_to_f2(w >> (8 * i));
        bs[8 * q + 2 * i][r] = f.x * s;
        bs[8 * q + 2 * i + 1][r] = f.y * s;
      }
    }
    __syncthreads();
    const int tm = (tid >> 4) * 4, tn = (tid & 15) * 4;
#pragma unroll
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][tm + i], bs[k][tn + j], acc[i][j]);
  }
  const int tm = (tid >> 4) * 4, tn = (tid & 15) * 4;
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + tm + i;
    if (m >= p.M) break;
    for (int j = 0; j < 4; ++j) {
      if (p.y) p.y[(int64_t)m * p.N + n0 + tn + j] = f2bf(acc[i][j]);
      else p.mid[(int64_t)m * p.N + n0 + tn + j] = acc[i][j];
    }
  }
}

}  // namespace

cudaError_t launch_quantize_mxfp4(int n_rows, int K, const void* in, bool f32, int64_t in_stride, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t s) {
  const int pad = (n_rows + 127) / 128 * 128;
  const int64_t blocks = ((int64_t)pad * (K / kMxBlock) + 255) / 256;
  const int grid = (int)(blocks < 148 * 8 ? blocks : 148 * 8);
  TraceScope tr("quantize_mxfp4", s);
  return f32 ? launch_pdl(quantize_mxfp4_kernel<true>, dim3(grid), dim3(256), 0, s, n_rows, pad, K, in, in_stride, codes, scales)
             : launch_pdl(quantize_mxfp4_kernel<false>, dim3(grid), dim3(256), 0, s, n_rows, pad, K, in, in_stride, codes, scales);
}

cudaError_t launch_mxfp4_product(const Mxfp4Product& p, cudaStream_t s) {
  TraceScope tr("mxfp4_product", s);
  return launch_pdl(mxfp4_product_kernel, dim3(p.N / 64, (p.M + 63) / 64), dim3(256), 0, s, p);
}

}  // namespace ds4a
