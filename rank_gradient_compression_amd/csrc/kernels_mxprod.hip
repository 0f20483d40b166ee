// Products of microscaled 4-bit operands, C = A B^T (gfx950, wave64).
//
// C[i][j] = sum over blocks b of 2^(ea[i][b] + eb[j][b]) * sum over the
// block's 32 codes of a * b: what v_mfma_scale_f32_32x32x64_f8f6f4 computes
// for 32 rows of A, 32 rows of B and two blocks, with fp32 accumulators (the
// products of two E2M1 values are exact).  A lane holds 32 consecutive codes
// of one row: row lane % 32, and of the 8 blocks of a 256-column chunk the
// blocks 4 * (lane / 32) + s in step s = 0..3.  The order of the summed axis
// is free as long as both operands use the same, and this one makes a lane's
// four scales one dword of the operand's scale tiles.

#include <hip/hip_runtime.h>

#include "psgd_mx_device.h"

namespace psgd {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ v8i mx_regs(uint4 q) {
  return v8i{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
}

// One matrix-core step: 32 x 32 outputs, 64 columns; S selects the scale byte.
template <int S>
__device__ __forceinline__ v16f mx_mfma(uint4 a, uint4 b, v16f c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_regs(a), mx_regs(b), c, 4, 4, S, (int)sa, S, (int)sb);
}

template <int DT>
__device__ __forceinline__ void store_c(void* c, int64_t i, float v, bool acc) {
  auto* p = static_cast<typename Elem<DT>::type*>(c) + i;
  *p = Elem<DT>::down(acc ? v + Elem<DT>::up(*p) : v);
}

// Any sizes: one wavefront = one 32 x 32 tile of C, operands straight from
// memory (a lane reads 64 consecutive bytes of its row per chunk).  Row and
// block indexes past the end are clamped into the operand: such rows are not
// stored, and such blocks have scale 0 in both operands.
template <int DT>
__global__ __launch_bounds__(256) void k_mx_prod_tile(MxProductArgs p, int ntn) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t tm = (int64_t)(blockIdx.x / ntn) * 2 + (wave >> 1), tn = (int64_t)(blockIdx.x % ntn) * 2 + (wave & 1);
  if (tm * 32 >= p.m || tn * 32 >= p.n) return;
  const int64_t nch = mx_chunks(p.k), nblk = mx_blocks(p.k), pitch = nblk * 16;
  const int r = lane & 31, g = lane >> 5;
  const uint8_t* ar = p.a.codes + min(tm * 32 + r, p.m - 1) * pitch;
  const uint8_t* br = p.b.codes + min(tn * 32 + r, p.n - 1) * pitch;
  const uint32_t* as = reinterpret_cast<const uint32_t*>(p.a.scales) + tm * nch * 64 + lane;
  const uint32_t* bs = reinterpret_cast<const uint32_t*>(p.b.scales) + tn * nch * 64 + lane;
  v16f acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int64_t ch = 0; ch < nch; ++ch) {
    uint4 a[4], b[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t blk = min(ch * 8 + 4 * g + s, nblk - 1);
      a[s] = *reinterpret_cast<const uint4*>(ar + blk * 16);
      b[s] = *reinterpret_cast<const uint4*>(br + blk * 16);
    }
    const uint32_t sa = as[ch * 64], sb = bs[ch * 64];
    acc = mx_mfma<0>(a[0], b[0], acc, sa, sb);
    acc = mx_mfma<1>(a[1], b[1], acc, sa, sb);
    acc = mx_mfma<2>(a[2], b[2], acc, sa, sb);
    acc = mx_mfma<3>(a[3], b[3], acc, sa, sb);
  }
  const int64_t col = tn * 32 + r;
  if (col >= p.n) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t row = tm * 32 + g * 4 + (i >> 2) * 8 + (i & 3);
    if (row < p.m) store_c<DT>(p.c, row * p.ldc + col, acc[i], p.accumulate);
  }
}

// An empty sum: C = 0, or C unchanged.
template <int DT>
__global__ __launch_bounds__(256) void k_mx_prod_zero(MxProductArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < p.m * p.n) store_c<DT>(p.c, i / p.n * p.ldc + i % p.n, 0.f, false);
}

size_t mx_product_workspace(int64_t, int64_t, int64_t) { return 0; }

template <int DT>
static void product_dt(const MxProductArgs& p, hipStream_t s) {
  if (p.k == 0) {
    if (!p.accumulate)
      hipLaunchKernelGGL((k_mx_prod_zero<DT>), dim3((unsigned)((p.m * p.n + 255) / 256)), dim3(256), 0, s, p);
    return;
  }
  const int ntn = (int)((p.n + 63) / 64);
  hipLaunchKernelGGL((k_mx_prod_tile<DT>), dim3((unsigned)(((p.m + 63) / 64) * ntn)), dim3(256), 0, s, p, ntn);
}

hipError_t launch_mx_product(const MxProductArgs& p, void*, hipStream_t s) {
  if (p.m == 0 || p.n == 0) return hipSuccess;
  if (p.dtype == kF32)
    product_dt<kF32>(p, s);
  else if (p.dtype == kBF16)
    product_dt<kBF16>(p, s);
  else
    product_dt<kF16>(p, s);
  return hipGetLastError();
}

}  // namespace psgd
