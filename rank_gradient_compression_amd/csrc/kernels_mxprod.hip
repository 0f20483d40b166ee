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

#include <algorithm>
#include <type_traits>

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

template <int ROWS, int WAVES>
__device__ __forceinline__ void fetch_chunk(__amdgpu_buffer_rsrc_t rs, uint8_t* lds, uint32_t lane_off, uint32_t lane_off1, uint32_t pitch,
                                            uint32_t chunk_off, int wave) {
#pragma unroll
  for (int j = 0; j < ROWS / 8 / WAVES; ++j) {
    const int row = wave * (ROWS / WAVES) + j * 8;
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
template <int DT, int RE, int TM, int TN, bool ACC>
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
  for (int i = 0; i < TM * (32 / RE); ++i) {  // RE rows: registers e0 .. e0 + RE / 2 of row tile i * RE / 32
    const int e0 = i * (RE / 2) % 16;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < RE / 2; ++e)
        wr[((e >> 2) * 8 + (e & 3)) * PITCH + j * 32] = acc[i * RE / 32][j][e0 + e];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (wide) {
#pragma unroll
      for (int k = 0; k < RE; k += RPI) {
        const uint32_t o = off + (uint32_t)(i * RE + k) * ldb;
        float v[E];
        __builtin_memcpy(v, __builtin_assume_aligned(rd + k * PITCH, 16), sizeof v);
        if constexpr (ACC) add16<DT>(v, __builtin_amdgcn_raw_buffer_load_b128(rc, (int)o, 0, 0));
        __builtin_amdgcn_raw_buffer_store_b128(pack16<DT>(v), rc, (int)o, 0, 0);
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < RE; ++k) {
#pragma unroll
        for (uint32_t x = lane; x < COLS; x += 64) {
          const uint32_t o = x < cols ? (uint32_t)(i * RE + k) * ldb + x * (uint32_t)sizeof(T) : 0x80000000u;
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

// Rows of results that a wavefront passes through LDS at a time: 32, or 16
// where the stages have no room for 32 of each wavefront (rows of TN * 32 + 8
// floats, as many wavefronts to a stage array as fit).
template <int WAVES, int TN, int SA, int SB>
constexpr int mx_epilogue_rows() {
  constexpr int need = 32 * (TN * 32 + 8) * 4;
  return 2 * (SA / need + SB / need) >= WAVES ? 32 : 16;
}
template <int WAVES, int TN, int SA, int SB>
__device__ __forceinline__ float* mx_epilogue_lds(int wave, uint8_t* a0, uint8_t* b0, uint8_t* a1, uint8_t* b1) {
  constexpr int NEED = mx_epilogue_rows<WAVES, TN, SA, SB>() * (TN * 32 + 8) * 4, NA = SA / NEED, NB = SB / NEED;
  static_assert(2 * (NA + NB) >= WAVES, "stages too small for the results");
  if (wave < NA) return reinterpret_cast<float*>(a0 + wave * NEED);
  if (wave < NA + NB) return reinterpret_cast<float*>(b0 + (wave - NA) * NEED);
  if (wave < 2 * NA + NB) return reinterpret_cast<float*>(a1 + (wave - NA - NB) * NEED);
  return reinterpret_cast<float*>(b1 + (wave - 2 * NA - NB) * NEED);
}

template <int DT, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_mx_prod_lds(MxProductArgs p, int ntm, int ntn) {
  constexpr int WAVES = WM * WN, BM = WM * 32 * TM, BN = WN * 32 * TN;
  __shared__ __align__(16) uint8_t a0[BM * kChunkBytes], b0[BN * kChunkBytes], a1[BM * kChunkBytes],
      b1[BN * kChunkBytes];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN;
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
      const_cast<uint8_t*>(p.a.scales + m0 / 32 * nch * 256), 0, (int)((min(rtm, (uint32_t)(WM * TM - 1)) + 1) * nch * 256), 0x00020000);
  const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.b.scales + n0 / 32 * nch * 256), 0, (int)((min(rtn, (uint32_t)(WN * TN - 1)) + 1) * nch * 256), 0x00020000);
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
    fetch_chunk<BM, WAVES>(ra, da, lane_off, lane_off1, pitch, o, wave);
    fetch_chunk<BN, WAVES>(rb, db, lane_off, lane_off1, pitch, o, wave);
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
  constexpr int RE = mx_epilogue_rows<WAVES, TN, sizeof a0, sizeof b0>();
  float* ep = mx_epilogue_lds<WAVES, TN, sizeof a0, sizeof b0>(wave, a0, b0, a1, b1);
  if (p.accumulate)
    mx_store<DT, RE, TM, TN, true>(p, ep, m0 + wm * TM * 32, n0 + wn * TN * 32, lane, acc);
  else
    mx_store<DT, RE, TM, TN, false>(p, ep, m0 + wm * TM * 32, n0 + wn * TN * 32, lane, acc);
}

// Few rows on one side (up to 128): the product is a stream of the other
// operand, "wide" here, and what counts is how many of its bytes are under
// way.  One workgroup = MT * 32 rows of the narrow operand (all of them) times
// NT * 32 rows of the wide one; its wavefronts take the summed axis' chunks in
// turn (neighbouring wavefronts read neighbouring 128 bytes of a row) and their
// partial tiles are added through LDS in wavefront order.  Each wavefront
// stages its chunks in LDS of its own, two ahead, straight from memory in
// whole 128-byte rows: reading the matrix cores' layout (16 bytes of each of
// 32 rows per access) from memory instead kept the cache's address lookup
// busy and took 12 us where this takes 8 (24 x 4096 x 11008).
// The narrow operand comes from memory (XDT < 0), or, for a few thousand
// values, straight from the activations of type XDT, which every workgroup
// quantises into LDS by itself: one launch instead of two, and the first
// loads of the wide operand are already on their way meanwhile.
// With MT = NT = 2 the same kernel serves small products of any shape.
struct MxSkinnyArgs {
  int64_t narrow, wide, k;  // rows of the two operands, summed axis
  MxOperand x, w;           // narrow (XDT < 0) and wide operand
  const void* act;          // narrow x k activations, row stride ld (XDT >= 0)
  int64_t ld;
  void* c;
  int64_t ldc;
  int dtype;
  bool accumulate;
};

// Waits until at most N of this wavefront's memory accesses are under way.
template <int N>
__device__ __forceinline__ void wait_memory() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x0f70 | (N >> 4) << 14);
  __builtin_amdgcn_sched_barrier(0);
}

// One operand's part of a wavefront's chunk: T tiles of 32 rows.
template <int T>
struct MxTiles {
  __amdgpu_buffer_rsrc_t codes, scales;
  uint32_t pitch, nch, so[T];
  __device__ __forceinline__ MxTiles(const MxOperand& o, int64_t t0, int64_t rows, int64_t k) {
    pitch = (uint32_t)mx_pitch(k);
    nch = (uint32_t)mx_chunks(k);
    const uint32_t left = (uint32_t)min((int64_t)(T * 32), rows - t0 * 32), tiles = (left + 31) / 32;
    codes = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(o.codes + t0 * 32 * pitch), 0, (int)(left * pitch),
                                              0x00020000);
    scales = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(o.scales + t0 * nch * 256), 0,
                                               (int)(tiles * nch * 256), 0x00020000);
#pragma unroll
    for (int t = 0; t < T; ++t) so[t] = min((uint32_t)t, tiles - 1) * nch * 256;
  }
  // Chunk ch to LDS (T * 4 KB) and its scales to s; past the last chunk,
  // nothing (zero codes).
  __device__ __forceinline__ void fetch(uint32_t ch, uint8_t* lds, uint32_t (&s)[T], uint32_t off0, uint32_t off1,
                                        int lane) const {
    const uint32_t o = ch < nch ? ch * kChunkBytes : 0x80000000u, sc = min(ch, nch - 1) * 256;
#pragma unroll
    for (int t = 0; t < T; ++t) s[t] = __builtin_amdgcn_raw_buffer_load_b32(scales, lane * 4, (int)(so[t] + sc), 0);
#pragma unroll
    for (int j = 0; j < T * 4; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(codes, (__attribute__((address_space(3))) void*)(lds + j * 1024), 16,
                                               (int)((j & 1 ? off1 : off0) + j * 8 * pitch + o), 0, 0, 0);
  }
};

// One block of 32 activations (n of them valid) to codes and scale byte.
template <int DT>
__device__ __forceinline__ uint32_t mx_quant_block(const typename Elem<DT>::type* p, int n, uint4* q) {
  using T = typename Elem<DT>::type;
  T v[32];
  if (n >= 32 && ((uintptr_t)p & 15) == 0) {
#pragma unroll
    for (int i = 0; i < 32; i += 16 / (int)sizeof(T))
      __builtin_memcpy(&v[i], __builtin_assume_aligned(p + i, 16), 16);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i < n ? p[i] : (T)0;
  }
  float f[32];
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    f[i] = Elem<DT>::up(v[i]);
    am = max(am, __float_as_uint(f[i]) & 0x7fffffffu);
  }
  const uint32_t sb = mx_scale_byte(am);
  const float inv = sb == 255u ? 0.f : mx_inv_scale(sb);
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = sb == 255u ? 0.f : f[i] * inv;
  q->x = mx_encode8(f);
  q->y = mx_encode8(f + 8);
  q->z = mx_encode8(f + 16);
  q->w = mx_encode8(f + 24);
  return sb;
}

// Activations that a workgroup quantises by itself: at most this many blocks,
// four for each thread of a workgroup of 256.  (Every workgroup repeats the
// work; from here on a launch of its own is cheaper.)
constexpr int kFusedBlocks = 1024;

template <int WAVES, int MT, int NT, bool SWAP, int XDT>
__global__ __launch_bounds__(WAVES * 64, 1) void k_mx_prod_skinny(MxSkinnyArgs p, int nwt) {
  constexpr int XT = XDT >= 0 ? 0 : MT, XT1 = XT > 0 ? XT : 1;  // tiles of the narrow operand that are staged
  constexpr int STAGE = (XT + NT) * 4096, LOADS = 5 * (XT + NT);
  constexpr int RED = WAVES * MT * NT * 4096;
  static_assert(RED <= 2 * WAVES * STAGE, "no room for the partial tiles");
  __shared__ __align__(16) uint8_t st0[WAVES * STAGE], st1[WAVES * STAGE];
  __shared__ __align__(16) uint8_t xc[XDT >= 0 ? kFusedBlocks * 16 : 16], xs[XDT >= 0 ? kFusedBlocks : 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  const int64_t x0 = (int64_t)(blockIdx.x / nwt) * MT, w0 = (int64_t)(blockIdx.x % nwt) * NT;  // first tiles of 32
  const MxTiles<NT> w(p.w, w0, p.wide, p.k);
  const MxTiles<XT1> x(XT > 0 ? p.x : p.w, XT > 0 ? x0 : w0, XT > 0 ? p.narrow : p.wide, p.k);
  const uint32_t nch = w.nch, pitch = w.pitch;
  // (the slots of the large products' tiles)
  const uint32_t off0 = (lane >> 3) * pitch + (((lane & 7) ^ (lane >> 4)) << 4);
  const uint32_t off1 = (lane >> 3) * pitch + (((lane & 7) ^ (4 + (lane >> 4))) << 4);
  uint32_t off[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) off[s] = r * kChunkBytes + (((4 * g + s) ^ ((r >> 1) & 7)) << 4);
  uint8_t *const m0 = st0 + wave * STAGE, *const m1 = st1 + wave * STAGE;
  uint32_t sw0[NT], sw1[NT], sx0[XT1], sx1[XT1];
  auto fetch = [&](uint32_t ch, uint8_t* m, uint32_t(&sw)[NT], uint32_t(&sx)[XT1]) {
    w.fetch(ch, m, sw, off0, off1, lane);
    if constexpr (XT > 0) x.fetch(ch, m + NT * 4096, sx, off0, off1, lane);
  };
  uint32_t ch = wave;
  // (the order of the loads is what wait_memory counts on)
  fetch(ch, m0, sw0, sx0);
  __builtin_amdgcn_sched_barrier(0);
  fetch(ch + WAVES, m1, sw1, sx1);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (XDT >= 0) {
    constexpr int XD = XDT < 0 ? 0 : XDT;
    const auto* act = static_cast<const typename Elem<XD>::type*>(p.act);
    const int rows = (int)p.narrow, nblk = (int)mx_blocks(p.k), per = (int)nch * 8;
    // (blocks past the last get zero codes and scale 0; scales as in an operand's tiles: chunk, half, row, byte)
    for (int i = threadIdx.x; i < rows * per; i += WAVES * 64) {
      const int row = i / per, b = i % per;
      uint4 q = make_uint4(0, 0, 0, 0);
      uint32_t sb = 0;
      if (b < nblk) sb = mx_quant_block<XD>(act + row * p.ld + b * 32, (int)min((int64_t)32, p.k - b * 32), &q);
      reinterpret_cast<uint4*>(xc)[i] = q;
      xs[((b >> 2) * rows + row) * 4 + (b & 3)] = (uint8_t)sb;
    }
    // (a barrier that waits for LDS alone: the stages stay under way)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  }
  v16f acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[t][u][e] = 0.f;
  auto chunk = [&](uint32_t at, const uint8_t* m, const uint32_t(&sw)[NT], const uint32_t(&sx)[XT1]) {
    const int xrow = XDT >= 0 ? min(r, (int)p.narrow - 1) : 0;
    uint32_t fx = 0;
    if constexpr (XDT >= 0) fx = reinterpret_cast<const uint32_t*>(xs)[(min(at, nch - 1) * 2 + g) * (int)p.narrow + xrow];
    auto step = [&](auto S) {
      constexpr int s = decltype(S)::value;
      uint4 a[MT], b[NT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if constexpr (XDT >= 0)
          a[t] = reinterpret_cast<const uint4*>(xc)[xrow * (int)nch * 8 + min(at, nch - 1) * 8 + 4 * g + s];
        else
          a[t] = *reinterpret_cast<const uint4*>(m + (NT + t) * 4096 + off[s]);
      }
#pragma unroll
      for (int u = 0; u < NT; ++u) b[u] = *reinterpret_cast<const uint4*>(m + u * 4096 + off[s]);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          const uint32_t ss = XDT >= 0 ? fx : sx[XDT >= 0 ? 0 : t];
          acc[t][u] = SWAP ? mx_mfma<s>(b[u], a[t], acc[t][u], sw[u], ss) : mx_mfma<s>(a[t], b[u], acc[t][u], ss, sw[u]);
        }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  };
  // (a wavefront without a chunk adds one of zero codes)
  do {
    wait_memory<LOADS>();
    chunk(ch, m0, sw0, sx0);
    __builtin_amdgcn_sched_barrier(0);
    fetch(ch + 2 * WAVES, m0, sw0, sx0);
    wait_memory<LOADS>();
    chunk(ch + WAVES, m1, sw1, sx1);
    __builtin_amdgcn_sched_barrier(0);
    fetch(ch + 3 * WAVES, m1, sw1, sx1);
    ch += 2 * WAVES;
  } while (ch < nch);
  __syncthreads();  // (waits for the last fetches, of nothing, as well)
  // the partial tiles: the first WAVES * STAGE bytes in st0, the rest in st1
  constexpr int UNITS = MT * NT * 16;  // 256-byte registers of a wavefront
  constexpr int SPLIT = WAVES * STAGE / 256;
  auto at = [&](int i) { return reinterpret_cast<float*>(i < SPLIT ? st0 + i * 256 : st1 + (i - SPLIT) * 256) + lane; };
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) *at(wave * UNITS + (t * NT + u) * 16 + e) = acc[t][u][e];
  __syncthreads();
  // Register e of tile (t, u): lane % 32 is the column of C, 4 * (lane / 32) +
  // e / 4 * 8 + e % 4 its row; the wavefronts share the registers.
  const int64_t rows = SWAP ? p.wide : p.narrow, cols = SWAP ? p.narrow : p.wide;
  for (int o = wave; o < UNITS; o += WAVES) {
    const int e = o % 16, u = o / 16 % NT, t = o / 16 / NT;
    const int64_t tx = (x0 + t) * 32, tw = (w0 + u) * 32;
    const int64_t row0 = (SWAP ? tw : tx) + (e >> 2) * 8 + (e & 3), col = (SWAP ? tx : tw) + r;
    if (row0 >= rows) continue;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < WAVES; ++k) v += *at(k * UNITS + o);
    const int64_t row = row0 + g * 4;
    if (row >= rows || col >= cols) continue;
    const int64_t ci = row * p.ldc + col;
    if (p.dtype == kF32)
      store_c<kF32>(p.c, ci, v, p.accumulate);
    else if (p.dtype == kBF16)
      store_c<kBF16>(p.c, ci, v, p.accumulate);
    else
      store_c<kF16>(p.c, ci, v, p.accumulate);
  }
}

// Eight wavefronts to a workgroup where all tiles fit on the compute units
// together (their stages take 128 KB of LDS), four (two workgroups to a
// compute unit) where they do not, or where there is nothing to share.
template <int MT, int NT, bool SWAP, int XDT>
static void skinny(const MxSkinnyArgs& p, hipStream_t s) {
  const int64_t nwt = (p.wide + NT * 32 - 1) / (NT * 32), tiles = nwt * ((p.narrow + MT * 32 - 1) / (MT * 32));
  if constexpr (MT == 1 && NT == 1) {
    if (tiles <= 256 && mx_chunks(p.k) > 4) {
      hipLaunchKernelGGL((k_mx_prod_skinny<8, MT, NT, SWAP, XDT>), dim3((unsigned)tiles), dim3(512), 0, s, p, (int)nwt);
      return;
    }
  }
  hipLaunchKernelGGL((k_mx_prod_skinny<4, MT, NT, SWAP, XDT>), dim3((unsigned)tiles), dim3(256), 0, s, p, (int)nwt);
}

// SWAP: the narrow side is C's columns.
template <bool SWAP>
static void product_skinny(const MxSkinnyArgs& p, hipStream_t s) {
  if (p.narrow <= 32)
    skinny<1, 1, SWAP, -1>(p, s);
  else if (p.narrow <= 64)
    skinny<2, 1, SWAP, -1>(p, s);
  else
    skinny<4, 1, SWAP, -1>(p, s);
}

bool mx_linear_fuses(int64_t m, int64_t k) { return m <= 32 && k > 0 && m * mx_chunks(k) * 8 <= kFusedBlocks; }

hipError_t launch_mx_linear_fused(const MxProductArgs& p, const void* x, int x_dtype, int64_t ldx, hipStream_t s) {
  MxSkinnyArgs a{p.m, p.n, p.k, {nullptr, nullptr}, p.b, x, ldx, p.c, p.ldc, p.dtype, false};
  if (x_dtype == kF32)
    skinny<1, 1, false, kF32>(a, s);
  else if (x_dtype == kBF16)
    skinny<1, 1, false, kBF16>(a, s);
  else
    skinny<1, 1, false, kF16>(a, s);
  return hipGetLastError();
}

// An empty sum: C = 0, or C unchanged.
template <int DT>
__global__ __launch_bounds__(256) void k_mx_prod_zero(MxProductArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < p.m * p.n) store_c<DT>(p.c, i / p.n * p.ldc + i % p.n, 0.f, false);
}

size_t mx_product_workspace(int64_t, int64_t, int64_t) { return 0; }

template <int DT, int WM, int WN, int TM, int TN>
static void product_lds(const MxProductArgs& p, hipStream_t s) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  const int ntm = (int)((p.m + BM - 1) / BM), ntn = (int)((p.n + BN - 1) / BN);
  hipLaunchKernelGGL((k_mx_prod_lds<DT, WM, WN, TM, TN>), dim3((unsigned)(ntm * ntn)), dim3(64 * WM * WN), 0, s, p, ntm,
                     ntn);
}

template <int DT>
static void product_dt(const MxProductArgs& p, hipStream_t s) {
  if (p.k == 0) {
    if (!p.accumulate)
      hipLaunchKernelGGL((k_mx_prod_zero<DT>), dim3((unsigned)((p.m * p.n + 255) / 256)), dim3(256), 0, s, p);
    return;
  }
  const MxSkinnyArgs ab{p.m, p.n, p.k, p.a, p.b, nullptr, 0, p.c, p.ldc, p.dtype, p.accumulate};
  const MxSkinnyArgs ba{p.n, p.m, p.k, p.b, p.a, nullptr, 0, p.c, p.ldc, p.dtype, p.accumulate};
  const bool fits = mx_pitch(p.k) * 256 <= INT32_MAX && p.ldc * 4 * 128 <= INT32_MAX;  // 32-bit offsets in a tile
  if (fits && (p.m <= 128 || p.n <= 128)) {
    if (p.m <= p.n)
      product_skinny<false>(ab, s);
    else
      product_skinny<true>(ba, s);
    return;
  }
  // Tiles as large as still give each of the 256 compute units one: a larger
  // tile reads its operands fewer times, but an idle compute unit costs more
  // (2048 x 4096 x 11008: 128 tiles of 256 x 256 70 us, 256 of 128 x 256 54;
  // 2048 x 11008 x 4096: 344 of 256 x 256 58 us, 688 of 128 x 256 72).  A
  // single chunk is a write of C and hardly a product: small workgroups that
  // store from the accumulators (11008 x 4096 x 64: 33 us against 41).
  auto tiles = [&](int64_t bm, int64_t bn) { return ((p.m + bm - 1) / bm) * ((p.n + bn - 1) / bn); };
  if (fits && p.k > 256) {
    if (tiles(64, 64) <= 256)
      skinny<2, 2, false, -1>(ab, s);
    else if (tiles(128, 128) <= 256)
      product_lds<DT, 2, 2, 2, 2>(p, s);
    else if (tiles(128, 256) <= 256)
      product_lds<DT, 2, 2, 2, 4>(p, s);
    else
      product_lds<DT, 2, 4, 4, 2>(p, s);
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
