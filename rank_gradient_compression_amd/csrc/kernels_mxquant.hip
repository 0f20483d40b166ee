// Quantisation to microscaled 4-bit operands and back (gfx950, wave64).
//
// A block of 32 values shares one power of two 2^k, k the smallest integer
// with max|x| <= 6 * 2^k (the factor payload's rule with E2M1's largest value
// 6: nothing saturates, so no value of a block is biased towards zero); each
// value becomes an E2M1 code of x * 2^-k.  All arithmetic is exact (scaling by
// powers of two, then one rounding), so codes do not depend on how the work
// is split.  Bound: HBM, one read of x and one write of codes, scales and
// values.

#include <hip/hip_runtime.h>

#include "psgd_mx_device.h"

namespace psgd {

// N consecutive elements from p, `n` of them valid (the rest become zero), with
// accesses of VB bytes where all N are valid.
template <int DT, int N, int VB>
__device__ __forceinline__ void load_elems(const typename Elem<DT>::type* p, int n, typename Elem<DT>::type (&v)[N]) {
  using T = typename Elem<DT>::type;
  constexpr int E = VB / (int)sizeof(T);
  static_assert(E >= 1 && N % E == 0, "access width");
  if (n >= N) {
#pragma unroll
    for (int i = 0; i < N; i += E) __builtin_memcpy(&v[i], __builtin_assume_aligned(p + i, VB), VB);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? p[i] : (T)0;
  }
}

template <int DT, int N, int VB>
__device__ __forceinline__ void store_elems(typename Elem<DT>::type* p, int n, const typename Elem<DT>::type (&v)[N]) {
  using T = typename Elem<DT>::type;
  constexpr int E = VB / (int)sizeof(T);
  if (n >= N) {
#pragma unroll
    for (int i = 0; i < N; i += E) __builtin_memcpy(__builtin_assume_aligned(p + i, VB), &v[i], VB);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = v[i];
  }
}

// Largest magnitude (bit pattern) over groups of L consecutive lanes.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t a) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o));
  return a;
}

// Row operand.  One workgroup = 32 rows x 256 columns (one tile of scales);
// every thread takes 16 bytes of a row at a time, so 4 (16-bit types) or 8
// (fp32) neighbouring lanes share a block and agree on its exponent by lane
// exchanges; scales are gathered in LDS and leave as one 256-byte tile.
template <int DT, int VB, bool RAND, bool VALUES>
__global__ __launch_bounds__(256) void k_mx_quant_rows(MxQuantArgs a, int nch) {
  using T = typename Elem<DT>::type;
  constexpr int E = 16 / (int)sizeof(T);   // elements per thread and row
  constexpr int L = kMxBlock / E;          // lanes per block
  constexpr int TPR = 256 / E;             // threads per row of the tile
  constexpr int RPP = 256 / TPR;           // rows per sweep of the workgroup
  constexpr int SWEEPS = 32 / RPP;
  __shared__ uint32_t tile[64];
  const int rt = blockIdx.x / nch, ch = blockIdx.x % nch;
  const int64_t row0 = (int64_t)rt * 32;
  const int col = ch * 256 + (int)(threadIdx.x % TPR) * E;
  const int nvalid = (int)min((int64_t)E, max((int64_t)0, a.cols - col));
  const int nrows = (int)min((int64_t)32, a.rows - row0);
  const int64_t nblk = mx_blocks(a.cols);
  const T* x = static_cast<const T*>(a.x);
  T v[SWEEPS][E];
#pragma unroll
  for (int s = 0; s < SWEEPS; ++s) {
    const int r = s * RPP + (int)threadIdx.x / TPR;
    load_elems<DT, E, VB>(x + (row0 + min(r, nrows - 1)) * a.ld + col, nvalid, v[s]);
  }
  uint8_t* tb = reinterpret_cast<uint8_t*>(tile);
#pragma unroll
  for (int s = 0; s < SWEEPS; ++s) {
    const int r = s * RPP + (int)threadIdx.x / TPR;
    const int64_t row = row0 + r;
    const bool live = r < nrows;
    float f[E];
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      f[i] = Elem<DT>::up(v[s][i]);
      am = max(am, __float_as_uint(f[i]) & 0x7fffffffu);
    }
    am = group_max<L>(am);
    const uint32_t sb = mx_scale_byte(am);
    const float inv = sb == 255u ? 0.f : mx_inv_scale(sb);
    uint8_t rnd[E];
    if constexpr (RAND) {
      const uint8_t* rp = a.rand + (row0 + min(r, nrows - 1)) * a.cols + col;
#pragma unroll
      for (int i = 0; i < E; ++i) rnd[i] = i < nvalid ? rp[i] : 0;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      float t = f[i] * inv;
      if (sb == 255u) t = 0.f;  // 0 * NaN
      if constexpr (RAND) t = mx_stochastic(t, rnd[i]);
      f[i] = t;
    }
    uint32_t code;
    if constexpr (E == 8)
      code = mx_encode8(f);
    else
      code = mx_encode4(f);
    const int blk = col >> 5;
    if ((threadIdx.x % L) == 0) tb[((blk & 7) >> 2) * 128 + r * 4 + (blk & 3)] = (uint8_t)sb;
    if (live && blk < nblk) {
      if (a.row_codes) {
        uint8_t* cp = a.row_codes + row * (nblk * 16) + (col >> 1);
        if constexpr (E == 8)
          *reinterpret_cast<uint32_t*>(cp) = code;
        else
          *reinterpret_cast<uint16_t*>(cp) = (uint16_t)code;
      }
      if constexpr (VALUES) {
        const int k = (int)sb - 127;
        T o[E];
        float2 d[E / 2];
        d[0] = mx_decode2<0>(code, k);
        d[1] = mx_decode2<1>(code, k);
        if constexpr (E == 8) {
          d[2] = mx_decode2<2>(code, k);
          d[3] = mx_decode2<3>(code, k);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float q = sb == 255u ? __uint_as_float(0x7fc00000u) : (i & 1) ? d[i / 2].y : d[i / 2].x;
          o[i] = Elem<DT>::down(q);
        }
        store_elems<DT, E, VB>(static_cast<T*>(a.values) + row * a.ldv + col, nvalid, o);
      }
    }
  }
  if (!a.row_scales) return;
  __syncthreads();
  if (threadIdx.x < 64)
    reinterpret_cast<uint32_t*>(a.row_scales)[((int64_t)rt * nch + ch) * 64 + threadIdx.x] = tile[threadIdx.x];
}

// Column operand (the operand of x^T, blocks along x's rows), with the row
// operand of the same reading of x where it is wanted.  One workgroup = 128 x
// 128 values held in LDS: four blocks per column give 64 contiguous bytes of
// codes per column and per row.  In LDS each group of 32 rows is shifted by
// 64 bytes against the one above (16 columns of two 2-byte values), so that
// the four blocks of a column that neighbouring lanes read fall into distinct
// banks.
template <int DT, int VB, bool RAND, bool ROWS>
__global__ __launch_bounds__(256) void k_mx_quant_cols(MxQuantArgs a, int nct) {
  using T = typename Elem<DT>::type;
  constexpr int E = 16 / (int)sizeof(T);
  constexpr int L = kMxBlock / E;
  constexpr int TPR = 128 / E;
  constexpr int RPP = 256 / TPR;
  constexpr int SWEEPS = 128 / RPP;
  constexpr int P = 128 + 16 / (int)sizeof(T);             // row pitch in LDS, elements
  constexpr int SKEW = 64 * (DT == kF32 ? 2 : 1) / (int)sizeof(T);  // shift per 32 rows
  constexpr int RP = 132;
  __shared__ __align__(16) T tile[128 * P + 4 * SKEW];
  __shared__ __align__(16) uint8_t rtile[RAND ? 128 * RP : 16];
  __shared__ uint32_t stile[ROWS ? 128 : 1];
  const int rt = blockIdx.x / nct, ct = blockIdx.x % nct;
  const int64_t row0 = (int64_t)rt * 128;
  const int64_t col0 = (int64_t)ct * 128;
  const int c = (int)(threadIdx.x % TPR) * E;
  const int64_t col = col0 + c;
  const int nvalid = (int)min((int64_t)E, max((int64_t)0, a.cols - col));
  const int nrows = (int)min((int64_t)128, max((int64_t)0, a.rows - row0));
  const T* x = static_cast<const T*>(a.x);
  const int64_t nblk_r = mx_blocks(a.cols), nblk_c = mx_blocks(a.rows);
#pragma unroll
  for (int s0 = 0; s0 < SWEEPS; s0 += 4) {
    T v[4][E];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int r = (s0 + s) * RPP + (int)threadIdx.x / TPR;
      load_elems<DT, E, VB>(x + (row0 + max(0, min(r, nrows - 1))) * a.ld + col, r < nrows ? nvalid : 0, v[s]);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int r = (s0 + s) * RPP + (int)threadIdx.x / TPR;
      __builtin_memcpy(__builtin_assume_aligned(&tile[r * P + (r >> 5) * SKEW + c], 16), v[s], 16);
      uint8_t rnd[E];
      if constexpr (RAND) {
        const uint8_t* rp = a.rand + (row0 + max(0, min(r, nrows - 1))) * a.cols + col;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          rnd[i] = i < nvalid && r < nrows ? rp[i] : 0;
          rtile[r * RP + c + i] = rnd[i];
        }
      }
      if constexpr (ROWS) {
        float f[E];
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          f[i] = Elem<DT>::up(v[s][i]);
          am = max(am, __float_as_uint(f[i]) & 0x7fffffffu);
        }
        am = group_max<L>(am);
        const uint32_t sb = mx_scale_byte(am);
        const float inv = sb == 255u ? 0.f : mx_inv_scale(sb);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          float t = f[i] * inv;
          if (sb == 255u) t = 0.f;
          if constexpr (RAND) t = mx_stochastic(t, rnd[i]);
          f[i] = t;
        }
        const int64_t blk = col >> 5;
        if ((threadIdx.x % L) == 0) reinterpret_cast<uint8_t*>(stile)[r * 4 + (c >> 5)] = (uint8_t)sb;
        if (r < nrows && blk < nblk_r) {
          uint8_t* cp = a.row_codes + (row0 + r) * (nblk_r * 16) + (col >> 1);
          if constexpr (E == 8)
            *reinterpret_cast<uint32_t*>(cp) = mx_encode8(f);
          else
            *reinterpret_cast<uint16_t*>(cp) = (uint16_t)mx_encode4(f);
        }
      }
    }
  }
  __syncthreads();
  if constexpr (ROWS) {
    // rows row0 .. row0+127 are four row tiles; these columns are half a chunk
    if (threadIdx.x < 128) {
      const int64_t tr = row0 / 32 + threadIdx.x / 32;
      if (tr < (a.rows + 31) / 32)
        reinterpret_cast<uint32_t*>(a.row_scales)[(tr * mx_chunks(a.cols) + ct / 2) * 64 + (ct & 1) * 32 +
                                                  threadIdx.x % 32] = stile[threadIdx.x];
    }
  }
  const int rb = threadIdx.x & 3, cp = threadIdx.x >> 2;  // block of 32 rows, pair of columns
  const int64_t B = row0 / 32 + rb;
  float f[2][32];
  uint32_t am[2] = {0, 0};
  const T* base = &tile[rb * 32 * P + rb * SKEW + cp * 2];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    T v[2];
    __builtin_memcpy(v, __builtin_assume_aligned(base + i * P, 2 * sizeof(T)), 2 * sizeof(T));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f[j][i] = Elem<DT>::up(v[j]);
      am[j] = max(am[j], __float_as_uint(f[j][i]) & 0x7fffffffu);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t sb = mx_scale_byte(am[j]);
    const float inv = sb == 255u ? 0.f : mx_inv_scale(sb);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float t = f[j][i] * inv;
      if (sb == 255u) t = 0.f;
      if constexpr (RAND) t = mx_stochastic(t, rtile[(rb * 32 + i) * RP + cp * 2 + j]);
      f[j][i] = t;
    }
    uint4 q;
    q.x = mx_encode8(&f[j][0]);
    q.y = mx_encode8(&f[j][8]);
    q.z = mx_encode8(&f[j][16]);
    q.w = mx_encode8(&f[j][24]);
    uint32_t s4 = sb << (8 * rb);  // the four scales of a column, from its four lanes
    s4 |= (uint32_t)__shfl_xor((int)s4, 1);
    s4 |= (uint32_t)__shfl_xor((int)s4, 2);
    const int64_t cc = col0 + cp * 2 + j;
    if (cc < a.cols) {
      if (B < nblk_c) *reinterpret_cast<uint4*>(a.col_codes + (cc * nblk_c + B) * 16) = q;
      if (rb == 0)
        reinterpret_cast<uint32_t*>(a.col_scales)[((cc / 32) * mx_chunks(a.rows) + rt / 2) * 64 + (rt & 1) * 32 +
                                                  cc % 32] = s4;
    }
  }
}

// Codes back to values: one thread = 8 codes (4 bytes) of a row.
template <int DT, int VB>
__global__ __launch_bounds__(256) void k_mx_dequant(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                    int64_t rows, int64_t cols, typename Elem<DT>::type* __restrict__ out,
                                                    int64_t ld, int nch) {
  using T = typename Elem<DT>::type;
  const int rt = blockIdx.x / nch, ch = blockIdx.x % nch;
  const int64_t row0 = (int64_t)rt * 32;
  const int c = (int)(threadIdx.x % 32) * 8;
  const int64_t col = (int64_t)ch * 256 + c;
  const int nvalid = (int)min((int64_t)8, max((int64_t)0, cols - col));
  const int nrows = (int)min((int64_t)32, rows - row0);
  const int64_t nblk = mx_blocks(cols);
  if (nvalid == 0) return;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int r = s * 8 + (int)threadIdx.x / 32;
    if (r >= nrows) break;
    const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + (row0 + r) * (nblk * 16) + (col >> 1));
    const int b = c >> 5;
    const uint32_t sb = scales[((int64_t)rt * nch + ch) * 256 + (b >> 2) * 128 + r * 4 + (b & 3)];
    const int k = (int)sb - 127;
    const float2 d[4] = {mx_decode2<0>(q, k), mx_decode2<1>(q, k), mx_decode2<2>(q, k), mx_decode2<3>(q, k)};
    T o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = Elem<DT>::down(sb == 255u ? __uint_as_float(0x7fc00000u) : (i & 1) ? d[i / 2].y : d[i / 2].x);
    store_elems<DT, 8, VB>(out + (row0 + r) * ld + col, nvalid, o);
  }
}

// Widest access (16 bytes down to one element) that a base address and a row
// stride in bytes allow for every row.
static int access_bytes(const void* p, int64_t stride_bytes, int elem) {
  const uint64_t m = (uint64_t)(uintptr_t)p | (uint64_t)stride_bytes;
  for (int vb = 16; vb > elem; vb >>= 1)
    if ((m & (uint64_t)(vb - 1)) == 0) return vb;
  return elem;
}

template <int DT, int VB>
static void quant_rows(const MxQuantArgs& a, hipStream_t s) {
  const int nch = (int)mx_chunks(a.cols);
  const dim3 g((unsigned)(((a.rows + 31) / 32) * nch)), b(256);
  if (a.rand && a.values)
    hipLaunchKernelGGL((k_mx_quant_rows<DT, VB, true, true>), g, b, 0, s, a, nch);
  else if (a.rand)
    hipLaunchKernelGGL((k_mx_quant_rows<DT, VB, true, false>), g, b, 0, s, a, nch);
  else if (a.values)
    hipLaunchKernelGGL((k_mx_quant_rows<DT, VB, false, true>), g, b, 0, s, a, nch);
  else
    hipLaunchKernelGGL((k_mx_quant_rows<DT, VB, false, false>), g, b, 0, s, a, nch);
}

template <int DT, int VB>
static void quant_cols(const MxQuantArgs& a, hipStream_t s) {
  // whole chunks of 256 both ways, so that the scales past the end are written
  const int nct = 2 * (int)mx_chunks(a.cols);
  const dim3 g((unsigned)(2 * mx_chunks(a.rows) * nct)), b(256);
  const bool rows = a.row_codes != nullptr;
  if (a.rand && rows)
    hipLaunchKernelGGL((k_mx_quant_cols<DT, VB, true, true>), g, b, 0, s, a, nct);
  else if (a.rand)
    hipLaunchKernelGGL((k_mx_quant_cols<DT, VB, true, false>), g, b, 0, s, a, nct);
  else if (rows)
    hipLaunchKernelGGL((k_mx_quant_cols<DT, VB, false, true>), g, b, 0, s, a, nct);
  else
    hipLaunchKernelGGL((k_mx_quant_cols<DT, VB, false, false>), g, b, 0, s, a, nct);
}

template <int DT, int VB>
static void quant_vb(const MxQuantArgs& a, hipStream_t s) {
  if (a.col_codes) {
    MxQuantArgs c = a;
    if (a.values) c.row_codes = c.row_scales = nullptr;  // the row operand comes with its values below
    quant_cols<DT, VB>(c, s);
    if (!a.values) return;
  }
  quant_rows<DT, VB>(a, s);
}

template <int DT>
static void quant_dt(const MxQuantArgs& a, hipStream_t s) {
  constexpr int eb = dtype_bytes(DT);
  int vb = access_bytes(a.x, a.ld * eb, eb);
  if (a.values) vb = min(vb, access_bytes(a.values, a.ldv * eb, eb));
  if (vb == 16)
    quant_vb<DT, 16>(a, s);
  else if (vb == 8)
    quant_vb<DT, 8>(a, s);
  else if (vb == 4)
    quant_vb<DT, 4>(a, s);
  else
    quant_vb<DT, eb>(a, s);
}

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t s) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  if (a.dtype == kF32)
    quant_dt<kF32>(a, s);
  else if (a.dtype == kBF16)
    quant_dt<kBF16>(a, s);
  else
    quant_dt<kF16>(a, s);
  return hipGetLastError();
}

template <int DT>
static void dequant_dt(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out, int64_t ld,
                       hipStream_t s) {
  constexpr int eb = dtype_bytes(DT);
  using T = typename Elem<DT>::type;
  const int nch = (int)mx_chunks(cols);
  const dim3 g((unsigned)(((rows + 31) / 32) * nch)), b(256);
  T* o = static_cast<T*>(out);
  const int vb = access_bytes(out, ld * eb, eb);
  if (vb == 16)
    hipLaunchKernelGGL((k_mx_dequant<DT, 16>), g, b, 0, s, codes, scales, rows, cols, o, ld, nch);
  else if (vb == 8)
    hipLaunchKernelGGL((k_mx_dequant<DT, 8>), g, b, 0, s, codes, scales, rows, cols, o, ld, nch);
  else
    hipLaunchKernelGGL((k_mx_dequant<DT, eb>), g, b, 0, s, codes, scales, rows, cols, o, ld, nch);
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                                int dtype, int64_t ld, hipStream_t s) {
  if (rows == 0 || cols == 0) return hipSuccess;
  if (dtype == kF32)
    dequant_dt<kF32>(codes, scales, rows, cols, out, ld, s);
  else if (dtype == kBF16)
    dequant_dt<kBF16>(codes, scales, rows, cols, out, ld, s);
  else
    dequant_dt<kF16>(codes, scales, rows, cols, out, ld, s);
  return hipGetLastError();
}

}  // namespace psgd
