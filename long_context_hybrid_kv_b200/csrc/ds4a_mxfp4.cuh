// Microscaled 4-bit (E2M1 elements, one E8M0 scale per 32 values along K)
// matrices for products: the layout of their scales, and the launchers.
//
// codes   [rows][K / 2] bytes, element 2i in the low nibble
// scales  blocks of 128 rows x 4 scales (128 values of K), 512 bytes each:
//         row r, scale j of a block at (r % 32) * 16 + (r / 32) * 4 + j; the
//         K / 128 blocks of a row range lie side by side.  This is the order
//         in which the tensor core's scale memory takes them (32 lanes of 16
//         bytes), so a product copies whole blocks and rearranges nothing.
#pragma once

#include "ds4a_internal.cuh"
#include "ds4a_mx.cuh"

namespace ds4a {

__host__ __device__ constexpr int64_t mxfp4_scale_bytes(int64_t rows, int64_t K) {
  return (rows + 127) / 128 * (K / 128) * 512;
}
__host__ __device__ constexpr int64_t mxfp4_scale_at(int64_t row, int64_t block, int64_t K) {
  return ((row / 128) * (K / 128) + block / 4) * 512 + (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4;
}

// bf16 rows -> codes and scales; padding rows of the last block of 128 get
// zero scales.  early: the next kernel of the stream may start before they are
// written (it has to wait before it reads them, as the products do for A, but
// not for their weights)
cudaError_t launch_quantize_mxfp4(int n_rows, int K, const uint16_t* in, int64_t in_stride, uint8_t* codes,
                                  uint8_t* scales, bool early, cudaStream_t s);

// One grouped product: outputs n of group j = n / n_per_group take the
// columns j * K .. (j + 1) * K of A's a_cols.  The result goes out as bf16
// (y), or quantised again (q_codes, q_scales) for a next product over N.
// part: float [mxfp4_ksplit][M][N] when the K axis is split.  o: A as bf16 [M]
// [a_cols] instead of codes and scales, where mxfp4_small(M).
struct Mxfp4Product {
  int M, N, K, n_per_group, a_cols;
  const uint16_t* o;
  const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
  uint16_t* y;
  uint8_t *q_codes, *q_scales;
  float* part;
  unsigned int* err;
};
int mxfp4_ksplit(int M, int N, int K);
bool mxfp4_small(int M);
cudaError_t launch_mxfp4_product(const Mxfp4Product& p, cudaStream_t s);

}  // namespace ds4a
