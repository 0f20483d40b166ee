// Microscaled 4-bit operands (MXFP4) and the gradient clip: format, tables
// and launchers (host declarations, device format helpers).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace psgd {

// ---- element types of the tensors that callers hand over (PSGD_DTYPE_*)
constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;
__host__ __device__ constexpr int dtype_bytes(int d) { return d == kF32 ? 4 : 2; }

// ---- operand format: `rows` x `cols` values in blocks of 32 along a row
// codes:  16 bytes per block, row after row (the last block padded with zero
//         codes); element 2j in the low nibble of byte j.
// scales: tiles of 32 rows x 256 columns, 256 bytes each, row tile by row
//         tile: the byte of row i, block b is at
//         ((i/32) * nch + b/8) * 256 + mx_scale_in_tile(i%32, b%8), so that
//         lane (i%16) + 16 * ((b%8)/2) of a wavefront finds the scales of its
//         two matrix-core steps for rows i%16 and 16 + i%16 in one dword and
//         a wavefront loads a tile with one 256-byte access.  Blocks past the
//         last column have scale 0 (2^-127): the product of two such blocks
//         is at most 32 * 36 * 2^-254, below 2^-243, and vanishes in fp32,
//         whatever their codes.
constexpr int kMxBlock = 32;
__host__ __device__ constexpr int mx_scale_in_tile(int row, int blk) {
  return (blk >> 1) * 64 + (row & 15) * 4 + (row >> 4) * 2 + (blk & 1);
}
__host__ __device__ inline int64_t mx_blocks(int64_t cols) { return (cols + 31) >> 5; }
__host__ __device__ inline int64_t mx_pitch(int64_t cols) { return mx_blocks(cols) * 16; }
__host__ __device__ inline int64_t mx_chunks(int64_t cols) { return (cols + 255) >> 8; }
__host__ __device__ inline int64_t mx_scale_bytes(int64_t rows, int64_t cols) {
  return ((rows + 31) >> 5) * mx_chunks(cols) * 256;
}

struct MxOperand {
  const uint8_t* codes;
  const uint8_t* scales;
};

struct MxQuantArgs {
  const void* x;
  int dtype;
  int64_t rows, cols, ld;
  const uint8_t* rand;  // rows x cols bytes, or null: nearest
  uint8_t* row_codes;   // blocks along the columns' axis of x (null: not wanted)
  uint8_t* row_scales;
  uint8_t* col_codes;   // the operand of x^T: blocks along the rows' axis (null: not wanted)
  uint8_t* col_scales;
  void* values;         // rows x cols values of the row operand, x's type (null: not wanted)
  int64_t ldv;
};
hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t s);
// Two matrices, in one launch where both want both operands in the same way.
hipError_t launch_mx_quantize_pair(const MxQuantArgs& a, const MxQuantArgs& b, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                                int dtype, int64_t ld, hipStream_t s);

struct MxProductArgs {
  int64_t m, n, k;
  MxOperand a, b;  // m x k and n x k
  void* c;         // m x n, row stride ldc
  int dtype;
  int64_t ldc;
  bool accumulate;
};
hipError_t launch_mx_product(const MxProductArgs& p, hipStream_t s);
// y = Q(x) B^T in one launch, for so few activations that every workgroup
// quantises them by itself (mx_linear_fuses); p.a is not read.
bool mx_linear_fuses(int64_t m, int64_t n, int64_t k, int x_dtype);
hipError_t launch_mx_linear_fused(const MxProductArgs& p, const void* x, int x_dtype, int64_t ldx, hipStream_t s);

}  // namespace psgd
