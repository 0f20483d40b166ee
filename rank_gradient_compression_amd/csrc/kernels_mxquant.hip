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

// How a run of elements that may cross the row's end is read.  FULL: all of it
// is inside the row.  EDGE: the row is at least as long as the run, which is
// read from an earlier column if need be, inside the row, and shifted down
// (what is shifted out may be another tile's, which writes it in place).
// NARROW: element by element, at columns clamped into the row (a branch around
// a load would make the compiler wait for it before it issues the next).
// Whatever the row's alignment: the hardware takes 16-byte accesses at any
// element's address, and on rows of 650 floats they beat pairs of 8-byte ones.
enum Reach { FULL, EDGE, NARROW };

// w shifted down by `bytes` (any number up from 0; zeros come in).
template <int N>
__device__ __forceinline__ void shift_down(uint32_t (&w)[N], uint32_t bytes) {
  const uint32_t words = bytes / 4;
#pragma unroll
  for (int h = N / 2; h > 0; h /= 2) {
    const uint32_t on = words & h ? ~0u : 0u;  // (a mask: the choice of an array's element would put it into memory)
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = (i + h < N ? w[i + h < N ? i + h : 0] & on : 0u) | (w[i] & ~on);
  }
  const uint32_t any = bytes < 4 * N ? ~0u : 0u;
#pragma unroll
  for (int i = 0; i < N; ++i)
    w[i] = __builtin_amdgcn_alignbyte(i + 1 < N ? w[i + 1 < N ? i + 1 : 0] : 0u, w[i], bytes & 3) & any;
}

// N words of consecutive elements of a row from column `col` on; zero past
// `cols`.
template <int DT, Reach R, int N>
__device__ __forceinline__ void load_elems(const typename Elem<DT>::type* row, int64_t col, int64_t cols,
                                           uint32_t (&w)[N]) {
  using T = typename Elem<DT>::type;
  constexpr int E = N * kPerWord<DT>;
  if (R == FULL) {
    __builtin_memcpy(w, row + col, sizeof w);
  } else if (R == EDGE) {
    __builtin_memcpy(w, row + min(col, cols - E), sizeof w);
  } else {
    T v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = row[min(col + i, cols - 1)];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = col + i < cols ? v[i] : (T)0;
    __builtin_memcpy(w, v, sizeof w);
  }
}

// What is left to do once the words are there (apart from the loads, so that
// all loads of a thread are issued first).
template <int BYTES, Reach R, int N>
__device__ __forceinline__ void settle(int64_t col, int64_t cols, uint32_t (&w)[N]) {
  constexpr int E = N * 4 / BYTES;
  if (R == EDGE) shift_down(w, (uint32_t)max((int64_t)0, col - (cols - E)) * BYTES);
}

template <int DT, bool WHOLE, int N>
__device__ __forceinline__ void store_elems(typename Elem<DT>::type* p, int n, const typename Elem<DT>::type (&v)[N]) {
  if (WHOLE || n >= N) {
    __builtin_memcpy(p, v, sizeof v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = v[i];
  }
}

// N words of random bytes of a row, clamped into it as above.
template <Reach R, int N>
__device__ __forceinline__ void load_bytes(const uint8_t* row, int64_t col, int64_t cols, uint32_t (&w)[N]) {
  if (R == FULL) {
    __builtin_memcpy(w, row + col, sizeof w);
  } else if (R == EDGE) {
    __builtin_memcpy(w, row + min(col, cols - 4 * N), sizeof w);
  } else {
    uint8_t v[4 * N];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) v[i] = row[min(col + i, cols - 1)];
    __builtin_memcpy(w, v, sizeof w);
  }
}

// Largest of a value over groups of L consecutive lanes, by lane exchanges of
// the vector unit: within pairs, within quads, quads of eight mirrored.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t a) {
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xf, 0xf, true));
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xf, 0xf, true));
  if (L == 8) a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x141, 0xf, 0xf, true));
  return a;
}

// Row operand.  One workgroup = 32 rows x 256 columns (one tile of scales);
// every thread takes 8 values of a row at a time, so 4 neighbouring lanes share
// a block and agree on its exponent by lane exchanges; scales are gathered in
// LDS and leave as one 256-byte tile.
template <int DT, bool RAND, bool VALUES, Reach R>
__device__ __forceinline__ void quant_rows_tile(const MxQuantArgs& a, int nch, uint32_t (&tile)[64]) {
  using T = typename Elem<DT>::type;
  constexpr int W = 8 / kPerWord<DT>;  // words of 8 values
  const int rt = blockIdx.x / nch, ch = blockIdx.x % nch;
  const int64_t row0 = (int64_t)rt * 32;
  const int64_t col = (int64_t)ch * 256 + (int)(threadIdx.x % 32) * 8;
  const int nvalid = (int)min((int64_t)8, max((int64_t)0, a.cols - col));
  const int nrows = (int)min((int64_t)32, a.rows - row0);
  const int64_t nblk = mx_blocks(a.cols);
  const T* x = static_cast<const T*>(a.x);
  uint8_t* tb = reinterpret_cast<uint8_t*>(tile);
  auto load = [&](int s, uint32_t(&v)[W], uint32_t(&rnd)[2]) {
    const int64_t row = row0 + min(s * 8 + (int)threadIdx.x / 32, nrows - 1);
    load_elems<DT, R>(x + row * a.ld, col, a.cols, v);
    if constexpr (RAND) load_bytes<R>(a.rand + row * a.cols, col, a.cols, rnd);
  };
  auto quantise = [&](int s, uint32_t(&v)[W], uint32_t(&rnd)[2]) {
    const int r = s * 8 + (int)threadIdx.x / 32;
    settle<sizeof(T), R>(col, a.cols, v);
    if constexpr (RAND) {
      settle<1, R>(col, a.cols, rnd);
      rnd[0] = ~rnd[0], rnd[1] = ~rnd[1];
    }
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) am = mx_max_words<DT>(am, v[i]);
    const uint32_t sb = mx_scale_byte(group_max<4>(mx_max_bits<DT>(am)));
    const uint32_t code = mx_encode8<DT, RAND>(v, sb, rnd);
    const int blk = (int)(col >> 5);
    // (a row past the last holds the last one's values, which in place another wavefront may have rounded already)
    if ((threadIdx.x & 3) == 0) tb[mx_scale_in_tile(r, blk & 7)] = r < nrows ? (uint8_t)sb : 0;
    if (r < nrows && (R == FULL || blk < nblk)) {
      if (a.row_codes) *reinterpret_cast<uint32_t*>(a.row_codes + (row0 + r) * (nblk * 16) + (col >> 1)) = code;
      if constexpr (VALUES) {
        const int k = (int)sb - 127;
        const float2 d[4] = {mx_decode2<0>(code, k), mx_decode2<1>(code, k), mx_decode2<2>(code, k),
                             mx_decode2<3>(code, k)};
        T o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = Elem<DT>::down(sb == 255u ? __uint_as_float(0x7fc00000u) : (i & 1) ? d[i / 2].y : d[i / 2].x);
        store_elems<DT, R == FULL>(static_cast<T*>(a.values) + (row0 + r) * a.ldv + col, nvalid, o);
      }
    }
  };
  if constexpr (R == NARROW) {  // (one row at a time: the addresses of all would take the other tiles' registers)
#pragma unroll 1
    for (int s = 0; s < 4; ++s) {
      uint32_t v[W], rnd[2];
      load(s, v, rnd);
      quantise(s, v, rnd);
    }
  } else {
    uint32_t v[4][W], rnd[4][2];
#pragma unroll
    for (int s = 0; s < 4; ++s) load(s, v[s], rnd[s]);
#pragma unroll
    for (int s = 0; s < 4; ++s) quantise(s, v[s], rnd[s]);
  }
  if (!a.row_scales) return;
  __syncthreads();
  if (threadIdx.x < 64)
    reinterpret_cast<uint32_t*>(a.row_scales)[((int64_t)rt * nch + ch) * 64 + threadIdx.x] = tile[threadIdx.x];
}

template <int DT, bool RAND, bool VALUES>
__global__ __launch_bounds__(256) void k_mx_quant_rows(MxQuantArgs a, int nch) {
  __shared__ uint32_t tile[64];
  if ((int64_t)(blockIdx.x % nch) * 256 + 256 <= a.cols)
    quant_rows_tile<DT, RAND, VALUES, FULL>(a, nch, tile);
  else if (a.cols >= 8)
    quant_rows_tile<DT, RAND, VALUES, EDGE>(a, nch, tile);
  else
    quant_rows_tile<DT, RAND, VALUES, NARROW>(a, nch, tile);
}

// Column operand (the operand of x^T, blocks along x's rows), with the row
// operand of the same reading of x where it is wanted.  One workgroup = 128 x
// 128 values held in LDS: four blocks per column give 64 contiguous bytes of
// codes per column and per row.  In LDS each group of 32 rows is shifted by
// 64 bytes against the one above, so that reading the values down the columns,
// where neighbouring lanes take the four blocks of a column, the 64 lanes'
// words fall into 64 banks.  The other accesses do meet: the random bytes, whose
// tile has no such shift (blocks two apart share banks), 16-byte stores and the
// reads along the rows; over all LDS instructions 2.4 conflict cycles each are
// counted, 3.0 with random bytes.
template <int DT>
constexpr int kColPitch = 128 + 16 / dtype_bytes(DT);  // row pitch in LDS, elements
template <int DT>
constexpr int kColSkew = 64 / dtype_bytes(DT);  // shift per 32 rows, elements
constexpr int kColRandPitch = 132;

// The tile into LDS, and its random bytes' complements: all of a thread's
// 16-byte loads under way at once, or a quarter of them where a narrow matrix
// is read element by element (the addresses would take the registers that keep
// further workgroups resident).
template <int DT, bool RAND, Reach R>
__device__ __forceinline__ void cols_tile_load(const MxQuantArgs& a, int64_t row0, int64_t col0,
                                               typename Elem<DT>::type* tile, uint8_t* rtile) {
  using T = typename Elem<DT>::type;
  constexpr int E = 4 * kPerWord<DT>, TPR = 128 / E, RPP = 256 / TPR, SWEEPS = 128 / RPP;  // 16 bytes per thread and row
  constexpr int GROUP = R == NARROW ? SWEEPS / 4 : SWEEPS;
  const T* x = static_cast<const T*>(a.x);
  const int c = (int)(threadIdx.x % TPR) * E, r0 = (int)threadIdx.x / TPR;
#pragma unroll 1
  for (int s0 = 0; s0 < SWEEPS; s0 += GROUP) {
    uint32_t v[GROUP][4], rnd[GROUP][E / 4];
#pragma unroll
    for (int s = 0; s < GROUP; ++s) {
      const int64_t row = min(row0 + (s0 + s) * RPP + r0, a.rows - 1);
      load_elems<DT, R>(x + row * a.ld, col0 + c, a.cols, v[s]);
      if constexpr (RAND) load_bytes<R>(a.rand + row * a.cols, col0 + c, a.cols, rnd[s]);
    }
#pragma unroll
    for (int s = 0; s < GROUP; ++s) {
      const int r = (s0 + s) * RPP + r0;
      settle<sizeof(T), R>(col0 + c, a.cols, v[s]);
      if constexpr (RAND) {
        settle<1, R>(col0 + c, a.cols, rnd[s]);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) rnd[s][i] = ~rnd[s][i];
      }
      uint4 q = make_uint4(v[s][0], v[s][1], v[s][2], v[s][3]);
      if (row0 + r >= a.rows) q = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(&tile[r * kColPitch<DT> + (r >> 5) * kColSkew<DT> + c]) = q;
      if constexpr (RAND) __builtin_memcpy(__builtin_assume_aligned(&rtile[r * kColRandPitch + c], 4), rnd[s], E);
    }
  }
}

// A block of 32 values to 16 bytes of codes.
template <int DT, bool RAND>
__device__ __forceinline__ uint4 encode_block(const uint32_t (&w)[32 / kPerWord<DT>], uint32_t sb,
                                              const uint32_t (&rnd)[8]) {
  constexpr int W = 8 / kPerWord<DT>;
  return make_uint4(mx_encode8<DT, RAND>(w, sb, rnd), mx_encode8<DT, RAND>(w + W, sb, rnd + 2),
                    mx_encode8<DT, RAND>(w + 2 * W, sb, rnd + 4), mx_encode8<DT, RAND>(w + 3 * W, sb, rnd + 6));
}

// Up to two matrices of one launch: a small layer's training pass is bound by
// its launches (700 x 650 and 2600 x 650 in fp32: 8.3 us together, 5.6 and 6.7
// one by one, and 2.6 us of the host for each launch).
struct MxQuantJobs {
  MxQuantArgs job[2];
  int tiles[2], nct[2];  // tiles of 128 x 128, and how many of them side by side
};

// (The instructions of a small call come from memory too: the parts are
// loops, and the kinds of tiles share all but their loads.)
template <int DT, bool RAND, bool ROWS>
__global__ __launch_bounds__(256) void k_mx_quant_cols(MxQuantJobs jobs) {
  const int which = (int)blockIdx.x >= jobs.tiles[0];
  const MxQuantArgs& a = jobs.job[which];
  const int nct = jobs.nct[which];
  using T = typename Elem<DT>::type;
  constexpr int P = kColPitch<DT>, SKEW = kColSkew<DT>, RP = kColRandPitch, PW = kPerWord<DT>;
  __shared__ __align__(16) T tile[128 * P + 4 * SKEW];
  __shared__ __align__(16) uint8_t rtile[RAND ? 128 * RP : 16];
  __shared__ uint32_t stile[ROWS ? 128 : 1], ctile[128];  // four tiles' half chunks
  // (a tile writes half lines of codes; neighbouring tiles on one XCD fill them up in its L2)
  const int t0 = xcd_position(blockIdx.x - which * jobs.tiles[0], jobs.tiles[which]), rt = t0 / nct, ct = t0 % nct;
  const int64_t row0 = (int64_t)rt * 128, col0 = (int64_t)ct * 128;
  const int64_t nblk_r = mx_blocks(a.cols), nblk_c = mx_blocks(a.rows);
  if (col0 + 128 <= a.cols)
    cols_tile_load<DT, RAND, FULL>(a, row0, col0, tile, rtile);
  else if (a.cols >= 8)
    cols_tile_load<DT, RAND, EDGE>(a, row0, col0, tile, rtile);
  else
    cols_tile_load<DT, RAND, NARROW>(a, row0, col0, tile, rtile);
  __syncthreads();
  if constexpr (ROWS) {
    // A thread takes blocks of 32 columns of a row: 512 blocks in the tile, the
    // four of a row in neighbouring lanes (64 contiguous bytes of codes).
#pragma unroll 1
    for (int i = threadIdx.x; i < 512; i += 256) {
      const int r = i >> 2, b = i & 3;
      const T* src = &tile[r * P + (r >> 5) * SKEW + b * 32];
      uint32_t w[32 / PW], rnd[8], am = 0;
      __builtin_memcpy(w, __builtin_assume_aligned(src, 16), sizeof w);
      if constexpr (RAND) __builtin_memcpy(rnd, __builtin_assume_aligned(&rtile[r * RP + b * 32], 4), 32);
#pragma unroll
      for (int j = 0; j < 32 / PW; ++j) am = mx_max_words<DT>(am, w[j]);
      const uint32_t sb = mx_scale_byte(mx_max_bits<DT>(am));
      const uint4 q = encode_block<DT, RAND>(w, sb, rnd);
      reinterpret_cast<uint8_t*>(stile)[r / 32 * 128 + mx_scale_in_tile(r % 32, b)] = (uint8_t)sb;
      if (row0 + r < a.rows && ct * 4 + b < nblk_r)
        *reinterpret_cast<uint4*>(a.row_codes + ((row0 + r) * nblk_r + ct * 4 + b) * 16) = q;
    }
  }
  // A thread takes blocks of 32 rows of a column, or of a pair of columns of a
  // 16-bit type (one word of each row); the four blocks of a column sit in
  // neighbouring lanes.
#pragma unroll 1
  for (int i = threadIdx.x; i < 512 / PW; i += 256) {
    const int b = i & 3, c = (i >> 2) * PW;
    const T* src = &tile[b * (32 * P + SKEW) + c];
    uint32_t w[32], am = 0;
    uint16_t rnd[RAND ? 32 : 1];  // PW random bytes of each row
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      __builtin_memcpy(&w[j], __builtin_assume_aligned(src + j * P, 4), 4);
      if constexpr (RAND && PW == 1) rnd[j] = rtile[(b * 32 + j) * RP + c];
      if constexpr (RAND && PW == 2) __builtin_memcpy(&rnd[j], __builtin_assume_aligned(&rtile[(b * 32 + j) * RP + c], 2), 2);
      am = mx_max_words<DT>(am, w[j]);
    }
#pragma unroll
    for (int h = 0; h < PW; ++h) {  // column c + h
      const uint32_t sb = mx_scale_byte(PW == 1 ? am : mx_half_max_bits<DT>(h ? am >> 16 : am & 0xffffu));
      uint4 q;
      if constexpr (RAND) {
        uint32_t code[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          code[j] = h ? mx_stochastic8_column<DT, 1>(w + 8 * j, sb, rnd + 8 * j)
                      : mx_stochastic8_column<DT, 0>(w + 8 * j, sb, rnd + 8 * j);
        q = make_uint4(code[0], code[1], code[2], code[3]);
      } else {
        uint32_t u[32 / PW];
#pragma unroll
        for (int j = 0; j < 32 / PW; ++j)
          u[j] = PW == 1 ? w[j] : __builtin_amdgcn_perm(w[PW * j + PW - 1], w[PW * j], h ? 0x07060302u : 0x05040100u);
        q = make_uint4(mx_nearest8<DT>(u, sb), mx_nearest8<DT>(u + 8 / PW, sb), mx_nearest8<DT>(u + 16 / PW, sb),
                       mx_nearest8<DT>(u + 24 / PW, sb));
      }
      reinterpret_cast<uint8_t*>(ctile)[c / 32 * 128 + mx_scale_in_tile(c % 32 + h, b)] = (uint8_t)sb;
      if (col0 + c + h < a.cols && rt * 4 + b < nblk_c)
        *reinterpret_cast<uint4*>(a.col_codes + ((col0 + c + h) * nblk_c + rt * 4 + b) * 16) = q;
    }
  }
  __syncthreads();
  // 128 rows (columns) are four tiles of scales, 128 columns (rows) half a chunk
  const int t = threadIdx.x % 128 / 32, at = threadIdx.x % 32;
  if (threadIdx.x < 128) {
    if (col0 / 32 + t < (a.cols + 31) / 32)
      reinterpret_cast<uint32_t*>(a.col_scales)[((col0 / 32 + t) * mx_chunks(a.rows) + rt / 2) * 64 + (rt & 1) * 32 + at] =
          ctile[threadIdx.x];
  } else if constexpr (ROWS) {
    if (row0 / 32 + t < (a.rows + 31) / 32)
      reinterpret_cast<uint32_t*>(a.row_scales)[((row0 / 32 + t) * mx_chunks(a.cols) + ct / 2) * 64 + (ct & 1) * 32 + at] =
          stile[threadIdx.x - 128];
  }
}

// Codes back to values: one thread = 8 codes (4 bytes) of a row.  The bytes
// would take 60 us for 32000 x 4096 to bf16; it takes 128 (2.6 TB/s).
template <int DT>
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
    const uint32_t sb = scales[((int64_t)rt * nch + ch) * 256 + mx_scale_in_tile(r, b)];
    const int k = (int)sb - 127;
    const float2 d[4] = {mx_decode2<0>(q, k), mx_decode2<1>(q, k), mx_decode2<2>(q, k), mx_decode2<3>(q, k)};
    T o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = Elem<DT>::down(sb == 255u ? __uint_as_float(0x7fc00000u) : (i & 1) ? d[i / 2].y : d[i / 2].x);
    store_elems<DT, false>(out + (row0 + r) * ld + col, nvalid, o);
  }
}

template <int DT>
static void quant_rows(const MxQuantArgs& a, hipStream_t s) {
  const int nch = (int)mx_chunks(a.cols);
  const dim3 g((unsigned)(((a.rows + 31) / 32) * nch)), b(256);
  if (a.rand && a.values)
    hipLaunchKernelGGL((k_mx_quant_rows<DT, true, true>), g, b, 0, s, a, nch);
  else if (a.rand)
    hipLaunchKernelGGL((k_mx_quant_rows<DT, true, false>), g, b, 0, s, a, nch);
  else if (a.values)
    hipLaunchKernelGGL((k_mx_quant_rows<DT, false, true>), g, b, 0, s, a, nch);
  else
    hipLaunchKernelGGL((k_mx_quant_rows<DT, false, false>), g, b, 0, s, a, nch);
}

// b: a second matrix that wants the same operands with the same rounding.
template <int DT>
static void quant_cols(const MxQuantArgs& a, const MxQuantArgs* b, hipStream_t s) {
  MxQuantJobs j{{a, b ? *b : MxQuantArgs{}}, {0, 0}, {0, 0}};
  for (int i = 0; i < (b ? 2 : 1); ++i) {
    // whole chunks of 256 both ways, so that the scales past the end are written
    j.nct[i] = 2 * (int)mx_chunks(j.job[i].cols);
    j.tiles[i] = (int)(2 * mx_chunks(j.job[i].rows)) * j.nct[i];
  }
  const dim3 g((unsigned)(j.tiles[0] + j.tiles[1])), blk(256);
  const bool rows = a.row_codes != nullptr;
  if (a.rand && rows)
    hipLaunchKernelGGL((k_mx_quant_cols<DT, true, true>), g, blk, 0, s, j);
  else if (a.rand)
    hipLaunchKernelGGL((k_mx_quant_cols<DT, true, false>), g, blk, 0, s, j);
  else if (rows)
    hipLaunchKernelGGL((k_mx_quant_cols<DT, false, true>), g, blk, 0, s, j);
  else
    hipLaunchKernelGGL((k_mx_quant_cols<DT, false, false>), g, blk, 0, s, j);
}

template <int DT>
static void quantize(const MxQuantArgs& a, hipStream_t s) {
  if (a.col_codes) {
    MxQuantArgs c = a;
    if (a.values) c.row_codes = c.row_scales = nullptr;  // the row operand comes with its values below
    quant_cols<DT>(c, nullptr, s);
    if (!a.values) return;
  }
  quant_rows<DT>(a, s);
}

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t s) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  if (a.dtype == kF32)
    quantize<kF32>(a, s);
  else if (a.dtype == kBF16)
    quantize<kBF16>(a, s);
  else
    quantize<kF16>(a, s);
  return hipGetLastError();
}

hipError_t launch_mx_quantize_pair(const MxQuantArgs& a, const MxQuantArgs& b, hipStream_t s) {
  auto both = [](const MxQuantArgs& q) {
    return q.rows && q.cols && q.row_codes && q.col_codes && !q.rand && !q.values;
  };
  if (a.dtype == b.dtype && both(a) && both(b)) {
    if (a.dtype == kF32)
      quant_cols<kF32>(a, &b, s);
    else if (a.dtype == kBF16)
      quant_cols<kBF16>(a, &b, s);
    else
      quant_cols<kF16>(a, &b, s);
    return hipGetLastError();
  }
  if (hipError_t e = launch_mx_quantize(a, s); e != hipSuccess) return e;
  return launch_mx_quantize(b, s);
}

template <int DT>
static void dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out, int64_t ld,
                       hipStream_t s) {
  const int nch = (int)mx_chunks(cols);
  hipLaunchKernelGGL((k_mx_dequant<DT>), dim3((unsigned)(((rows + 31) / 32) * nch)), dim3(256), 0, s, codes, scales,
                     rows, cols, static_cast<typename Elem<DT>::type*>(out), ld, nch);
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                                int dtype, int64_t ld, hipStream_t s) {
  if (rows == 0 || cols == 0) return hipSuccess;
  if (dtype == kF32)
    dequantize<kF32>(codes, scales, rows, cols, out, ld, s);
  else if (dtype == kBF16)
    dequantize<kBF16>(codes, scales, rows, cols, out, ld, s);
  else
    dequantize<kF16>(codes, scales, rows, cols, out, ld, s);
  return hipGetLastError();
}

}  // namespace psgd
