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

// Large products: a workgroup computes a BM x BN tile of C with four
// wavefronts (2 x 2), each TM x TN tiles of 32 x 32 in accumulators.  Per
// chunk of 256 columns a row is 128 bytes of codes; both operands' chunks go
// from memory straight into LDS (16 bytes per lane, no registers), two
// stages, so the next chunk arrives while the matrix cores work on this one.
// The hardware writes LDS in lane order; each lane therefore *fetches* the
// block that belongs there: block b of row r sits at slot b ^ (r % 8), which
// spreads the 16-byte reads of 8 neighbouring rows over all banks.  Scales
// come from memory into registers a chunk ahead, 256 contiguous bytes per
// 32 rows.  Buffer descriptors end with the tile's last row: rows past it read
// as zero, without a fault.
constexpr int kChunkBytes = 128;

// Workgroup to tile: consecutive workgroups go to the eight XCDs in turn, each
// with an L2 of its own, so XCD x gets the x-th eighth of the tiles, and these
// are walked in groups of 8 tile rows: the 32 tiles that an XCD's compute
// units work on at a time form an 8 x 4 block that shares its operands in L2.
__device__ __forceinline__ void tile_of_block(int b, int ntm, int ntn, int* tm, int* tn) {
  const int total = ntm * ntn, q = total / 8, rem = total % 8, x = b % 8;
  const int t = x * q + min(x, rem) + b / 8;
  const int first = t / (8 * ntn) * 8, rows = min(8, ntm - first), in = t % (8 * ntn);
  *tm = first + in % rows;
  *tn = in / rows;
}

template <int ROWS>
__device__ __forceinline__ void fetch_chunk(__amdgpu_buffer_rsrc_t rs, uint8_t* lds, uint32_t lane_off, uint32_t lane_off1, uint32_t pitch,
                                            uint32_t chunk_off, int wave) {
#pragma unroll
  for (int j = 0; j < ROWS / 32; ++j) {
    const int row = wave * (ROWS / 4) + j * 8;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rs, (__attribute__((address_space(3))) void*)(lds + row * kChunkBytes), 16,
        (int)((j & 1 ? lane_off1 : lane_off) + (uint32_t)row * pitch + chunk_off), 0, 0, 0);
  }
}

// Operand registers of one matrix-core step.
template <int TM, int TN>
struct Frags {
  uint4 a[TM], b[TN];
  __device__ __forceinline__ void read(const uint8_t* la, const uint8_t* lb) {
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const uint4*>(la + i * 32 * kChunkBytes);
#pragma unroll
    for (int j = 0; j < TN; ++j) b[j] = *reinterpret_cast<const uint4*>(lb + j * 32 * kChunkBytes);
  }
};

template <int S, int TM, int TN>
__device__ __forceinline__ void mx_step(const Frags<TM, TN>& f, const uint32_t (&sa)[TM], const uint32_t (&sb)[TN],
                                        v16f (&acc)[TM][TN]) {
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = mx_mfma<S>(f.a[i], f.b[j], acc[i][j], sa[i], sb[j]);
}

// Issue order of one step: the reads of the next step's operands, one behind
// each of the first products, which hide them.
template <int TM, int TN>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < TM + TN; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix-core product
  }
  __builtin_amdgcn_sched_group_barrier(0x008, TM * TN - TM - TN, 0);
  __builtin_amdgcn_sched_barrier(0);
}

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// E values as one 16-byte vector of the result's type.
template <int DT>
__device__ __forceinline__ v4u pack16(const float* v) {
  if constexpr (DT == kF32) {
    return v4u{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  } else {
    v4u q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = Elem<DT>::down2(v[2 * i], v[2 * i + 1]);
    return q;
  }
}
template <int DT>
__device__ __forceinline__ void add16(float* v, v4u q) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kF32) {
      v[i] += __uint_as_float(q[i]);
    } else {
      v[2 * i] += Elem<DT>::up((uint16_t)q[i]);
      v[2 * i + 1] += Elem<DT>::up((uint16_t)(q[i] >> 16));
    }
  }
}

// Accumulators to C.  A lane holds column lane % 32 and rows 4 * (lane / 32)
// + 8 j + 0..3 of a 32 x 32 tile.  Each wavefront passes 32 rows at a time
// through LDS of its own and stores 16 bytes per lane, whole rows of its
// TN * 32 columns: eight times fewer instructions than storing 16-bit results
// from the accumulators' layout, and the instruction count is what this part
// costs.  The row pitch of 8 floats beyond a multiple of 16 puts the two rows
// that a write covers into opposite banks.  Rows past the end of C lie outside
// the buffer descriptor, columns past it get an offset outside it.
template <int DT, int TM, int TN, bool ACC>
__device__ __forceinline__ void mx_store(const MxProductArgs& p, float* lds, int64_t row0, int64_t col0, int lane,
                                         const v16f (&acc)[TM][TN]) {
  using T = typename Elem<DT>::type;
  constexpr int E = 16 / (int)sizeof(T);
  constexpr int COLS = TN * 32, PITCH = COLS + 8, LPR = COLS / E, RPI = 64 / LPR;
  const int64_t rl = p.m - row0, cl = p.n - col0;  // rows and columns of C from here on
  if (rl <= 0 || cl <= 0) return;
  const uint32_t cols = (uint32_t)min((int64_t)COLS, cl), ldb = (uint32_t)(p.ldc * sizeof(T));
  T* base = static_cast<T*>(p.c) + row0 * p.ldc + col0;
  const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
      base, 0, (int)(((uint32_t)min((int64_t)(TM * 32), rl) - 1) * ldb + cols * (uint32_t)sizeof(T)), 0x00020000);
  const bool wide = ((((uint32_t)(uintptr_t)base | ldb | cols * (uint32_t)sizeof(T))) & 15) == 0;
  float* wr = lds + (lane >> 5) * 4 * PITCH + (lane & 31);
  const uint32_t c = (lane % LPR) * E;
  const float* rd = lds + (lane / LPR) * PITCH + c;
  const uint32_t off = c < cols ? (lane / LPR) * ldb + c * (uint32_t)sizeof(T) : 0x80000000u;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) wr[((e >> 2) * 8 + (e & 3)) * PITCH + j * 32] = acc[i][j][e];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (wide) {
#pragma unroll
      for (int k = 0; k < 32; k += RPI) {
        const uint32_t o = off + (uint32_t)(i * 32 + k) * ldb;
        float v[E];
        __builtin_memcpy(v, __builtin_assume_aligned(rd + k * PITCH, 16), sizeof v);
        if constexpr (ACC) add16<DT>(v, __builtin_amdgcn_raw_buffer_load_b128(rc, (int)o, 0, 0));
        __builtin_amdgcn_raw_buffer_store_b128(pack16<DT>(v), rc, (int)o, 0, 0);
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < 32; ++k) {
#pragma unroll
        for (uint32_t x = lane; x < COLS; x += 64) {
          const uint32_t o = x < cols ? (uint32_t)(i * 32 + k) * ldb + x * (uint32_t)sizeof(T) : 0x80000000u;
          float v = lds[k * PITCH + x];
          if constexpr (sizeof(T) == 4) {
            if constexpr (ACC) v += __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rc, (int)o, 0, 0));
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rc, (int)o, 0, 0);
          } else {
            if constexpr (ACC) v += Elem<DT>::up(__builtin_amdgcn_raw_buffer_load_b16(rc, (int)o, 0, 0));
            __builtin_amdgcn_raw_buffer_store_b16(Elem<DT>::down(v), rc, (int)o, 0, 0);
          }
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <int DT, int TM, int TN, int OCC>
__global__ __launch_bounds__(256, OCC) void k_mx_prod_lds(MxProductArgs p, int ntm, int ntn) {
  constexpr int BM = 64 * TM, BN = 64 * TN;
  __shared__ __align__(16) uint8_t a0[BM * kChunkBytes], b0[BN * kChunkBytes], a1[BM * kChunkBytes],
      b1[BN * kChunkBytes];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave >> 1, wn = wave & 1;
  int tm, tn;
  tile_of_block(blockIdx.x, ntm, ntn, &tm, &tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const uint32_t nch = (uint32_t)mx_chunks(p.k), pitch = (uint32_t)mx_pitch(p.k);
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.a.codes + m0 * pitch), 0, (int)((uint32_t)min((int64_t)BM, p.m - m0) * pitch), 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.b.codes + n0 * pitch), 0, (int)((uint32_t)min((int64_t)BN, p.n - n0) * pitch), 0x00020000);
  // (r / 2) % 8 of this lane's row in an even and in an odd group of 8 rows
  const uint32_t lane_off = (lane >> 3) * pitch + (((lane & 7) ^ (lane >> 4)) << 4);
  const uint32_t lane_off1 = (lane >> 3) * pitch + (((lane & 7) ^ (4 + (lane >> 4))) << 4);
  const int r = lane & 31, g = lane >> 5;
  uint32_t off[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) off[s] = r * kChunkBytes + (((4 * g + s) ^ ((r >> 1) & 7)) << 4);
  // a wavefront's scale tiles; past the last tile of rows the last one again
  const uint32_t rtm = (uint32_t)((p.m + 31) / 32 - 1 - m0 / 32), rtn = (uint32_t)((p.n + 31) / 32 - 1 - n0 / 32);
  const __amdgpu_buffer_rsrc_t rsa = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.a.scales + m0 / 32 * nch * 256), 0, (int)((min(rtm, 2u * TM - 1) + 1) * nch * 256), 0x00020000);
  const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.b.scales + n0 / 32 * nch * 256), 0, (int)((min(rtn, 2u * TN - 1) + 1) * nch * 256), 0x00020000);
  uint32_t as[TM], bs[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) as[i] = min((uint32_t)(wm * TM + i), rtm) * nch * 256;
#pragma unroll
  for (int j = 0; j < TN; ++j) bs[j] = min((uint32_t)(wn * TN + j), rtn) * nch * 256;
  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  uint32_t sa[TM], sb[TN], ta[TM], tb[TN];
  auto scales = [&](uint32_t ch, uint32_t(&xa)[TM], uint32_t(&xb)[TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i) xa[i] = __builtin_amdgcn_raw_buffer_load_b32(rsa, lane * 4, (int)(as[i] + ch * 256), 0);
#pragma unroll
    for (int j = 0; j < TN; ++j) xb[j] = __builtin_amdgcn_raw_buffer_load_b32(rsb, lane * 4, (int)(bs[j] + ch * 256), 0);
  };
  const int la = wm * TM * 32 * kChunkBytes, lb = wn * TN * 32 * kChunkBytes;
  Frags<TM, TN> f0, f1;
  // One chunk, entered with its step 0 in f0: the operands of each step are
  // read while the matrix cores work on the step before.  The barrier stands
  // before the last step, whose products cover it and the first reads of the
  // next chunk; behind it every wavefront is done with this chunk's stage.
  auto chunk = [&](const uint8_t* ca, const uint8_t* cb, const uint8_t* na, const uint8_t* nb,
                   const uint32_t(&xa)[TM], const uint32_t(&xb)[TN]) {
    f1.read(ca + la + off[1], cb + lb + off[1]);
    mx_step<0>(f0, xa, xb, acc);
    interleave<TM, TN>();
    f0.read(ca + la + off[2], cb + lb + off[2]);
    mx_step<1>(f1, xa, xb, acc);
    interleave<TM, TN>();
    f1.read(ca + la + off[3], cb + lb + off[3]);
    mx_step<2>(f0, xa, xb, acc);
    interleave<TM, TN>();
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    f0.read(na + la + off[0], nb + lb + off[0]);
    mx_step<3>(f1, xa, xb, acc);
    interleave<TM, TN>();
  };
  scales(0, sa, sb);
  auto fetch = [&](uint32_t ch, uint8_t* da, uint8_t* db) {
    // no chunk past the last: an offset beyond the descriptor reads nothing
    const uint32_t o = ch < nch ? ch * kChunkBytes : 0x80000000u;
    fetch_chunk<BM>(ra, da, lane_off, lane_off1, pitch, o, wave);
    fetch_chunk<BN>(rb, db, lane_off, lane_off1, pitch, o, wave);
  };
  fetch(0, a0, b0);
  __syncthreads();
  f0.read(a0 + la + off[0], b0 + lb + off[0]);
  // (an odd last chunk is paired with one of zero codes)
  for (uint32_t ch = 0; ch < nch; ch += 2) {
    scales(min(ch + 1, nch - 1), ta, tb);
    fetch(ch + 1, a1, b1);
    chunk(a0, b0, a1, b1, sa, sb);
    scales(min(ch + 2, nch - 1), sa, sb);
    fetch(ch + 2, a0, b0);
    chunk(a1, b1, a0, b0, ta, tb);
  }
  // (every wavefront is behind its last barrier: the stages are free)
  float* ep = reinterpret_cast<float*>(wave == 0 ? a0 : wave == 1 ? b0 : wave == 2 ? a1 : b1);
  if (p.accumulate)
    mx_store<DT, TM, TN, true>(p, ep, m0 + wm * TM * 32, n0 + wn * TN * 32, lane, acc);
  else
    mx_store<DT, TM, TN, false>(p, ep, m0 + wm * TM * 32, n0 + wn * TN * 32, lane, acc);
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
  if (p.m >= 256 && p.n >= 256 && mx_pitch(p.k) * 256 <= INT32_MAX && p.ldc * 4 * 128 <= INT32_MAX) {
    const int ntm = (int)((p.m + 255) / 256), nt = (int)((p.n + 255) / 256);
    hipLaunchKernelGGL((k_mx_prod_lds<DT, 4, 4, 1>), dim3((unsigned)(ntm * nt)), dim3(256), 0, s, p, ntm, nt);
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
