// Products of microscaled 4-bit operands, C = A B^T (gfx950, wave64).
//
// C[i][j] = sum over blocks b of 2^(ea[i][b] + eb[j][b]) * sum over the
// block's 32 codes of a * b: what v_mfma_scale_f32_16x16x128_f8f6f4 computes
// for 16 rows of A, 16 rows of B and four blocks, with fp32 accumulators (the
// products of two E2M1 values are exact).  A lane holds 32 consecutive codes
// of one row: row lane % 16 and, of the 8 blocks of a 256-column chunk, block
// 2 * (lane / 16) + s in step s = 0, 1.  The order of the summed axis is free
// as long as both operands use the same, and this one makes a lane's scales
// for two tiles of 16 rows and both steps one dword of the operand's scale
// tiles.  (On random codes, where the power limit sets the clock, this shape
// runs at 7.3 PFLOP/s out of registers, the 32 x 32 x 64 one at 6.6.)
// The rows of B are the instruction's first operand: a lane then ends up with
// four neighbouring columns of C, columns 4 * (lane / 16) + 0..3 of row
// lane % 16 of a 16 x 16 tile.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "psgd_mx_device.h"

namespace psgd {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v8i mx_regs(uint4 q) {
  return v8i{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
}

// One matrix-core step: 16 x 16 outputs, 128 columns; BF and BS select the
// scale bytes of the two operands.
template <int BF, int BS>
__device__ __forceinline__ v4f mx_mfma(uint4 f, uint4 s, v4f c, uint32_t sf, uint32_t ss) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_regs(f), mx_regs(s), c, 4, 4, BF, (int)sf, BS, (int)ss);
}

// The same with the byte (half of the 32 rows, step) as run-time constants
// that unrolling folds.
__device__ __forceinline__ v4f mx_mfma_at(int s, int hf, int hs, uint4 f, uint4 q, v4f c, uint32_t sf, uint32_t ss) {
  switch (s * 4 + hf * 2 + hs) {
    case 0: return mx_mfma<0, 0>(f, q, c, sf, ss);
    case 1: return mx_mfma<0, 2>(f, q, c, sf, ss);
    case 2: return mx_mfma<2, 0>(f, q, c, sf, ss);
    case 3: return mx_mfma<2, 2>(f, q, c, sf, ss);
    case 4: return mx_mfma<1, 1>(f, q, c, sf, ss);
    case 5: return mx_mfma<1, 3>(f, q, c, sf, ss);
    case 6: return mx_mfma<3, 1>(f, q, c, sf, ss);
    default: return mx_mfma<3, 3>(f, q, c, sf, ss);
  }
}

// Up to four neighbouring results of one row (any alignment to the type).
template <int DT>
__device__ __forceinline__ void store4(void* c, int64_t i, v4f v, int64_t n, bool acc) {
  using T = typename Elem<DT>::type;
  T* p = static_cast<T*>(c) + i;
  T o[4];
  if (n >= 4) {
    if (acc) __builtin_memcpy(o, p, sizeof o);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = Elem<DT>::down(acc ? v[e] + Elem<DT>::up(o[e]) : v[e]);
    __builtin_memcpy(p, o, sizeof o);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) p[e] = Elem<DT>::down(acc ? v[e] + Elem<DT>::up(p[e]) : v[e]);
  }
}

// The walk of the large products: groups of 8 tile rows, so that the 32 tiles
// that an XCD's compute units work on at a time form an 8 x 4 block that
// shares its operands in L2.
__device__ __forceinline__ void tile_of_block(int b, int ntm, int ntn, int* tm, int* tn) {
  const int t = xcd_position(b, ntm * ntn);
  const int first = t / (8 * ntn) * 8, rows = min(8, ntm - first), in = t % (8 * ntn);
  *tm = first + in % rows;
  *tn = in / rows;
}

template <int DT>
__device__ __forceinline__ void store1(void* c, int64_t i, float v, bool acc) {
  auto* p = static_cast<typename Elem<DT>::type*>(c) + i;
  *p = Elem<DT>::down(acc ? v + Elem<DT>::up(*p) : v);
}

// Any sizes, and the choice for sums of one chunk, which are a write of C and
// hardly a product: one wavefront = one 32 x 32 tile of C, operands straight
// from memory.  Row and block indexes past the end are clamped into the
// operand: such rows are not stored, and such blocks have scale 0 in both
// operands.  Here A's rows are the first operand, so that a register is 16
// columns of four rows; two neighbouring tiles exchange quarters of the
// lanes, and every store is 128 bytes of fp32 in two rows (11008 x 4096 x 64:
// 33 us; with 64 bytes in 16 rows, from the other operand order, 56).
template <int DT>
__global__ __launch_bounds__(256) void k_mx_prod_tile(MxProductArgs p, int ntn) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = xcd_position(blockIdx.x, gridDim.x);  // (lines that two neighbouring tiles write meet in one L2)
  const int64_t tm = (int64_t)(t / ntn) * 2 + (wave >> 1), tn = (int64_t)(t % ntn) * 2 + (wave & 1);
  if (tm * 32 >= p.m || tn * 32 >= p.n) return;
  const int64_t nch = mx_chunks(p.k), nblk = mx_blocks(p.k), pitch = nblk * 16;
  const int r = lane & 15, g = lane >> 4;
  const uint8_t *ar[2], *br[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    ar[h] = p.a.codes + min(tm * 32 + 16 * h + r, p.m - 1) * pitch;
    br[h] = p.b.codes + min(tn * 32 + 16 * h + r, p.n - 1) * pitch;
  }
  const uint32_t* as = reinterpret_cast<const uint32_t*>(p.a.scales) + tm * nch * 64 + lane;
  const uint32_t* bs = reinterpret_cast<const uint32_t*>(p.b.scales) + tn * nch * 64 + lane;
  v4f acc[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i / 2][i % 2] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int64_t ch = 0; ch < nch; ++ch) {
    uint4 a[2][2], b[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t blk = min(ch * 8 + 2 * g + s, nblk - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[s][h] = *reinterpret_cast<const uint4*>(ar[h] + blk * 16);
        b[s][h] = *reinterpret_cast<const uint4*>(br[h] + blk * 16);
      }
    }
    const uint32_t sa = as[ch * 64], sb = bs[ch * 64];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mx_mfma_at(s, i, j, a[s][i], b[s][j], acc[i][j], sa, sb);
  }
  const int64_t row0 = tm * 32 + 8 * (g >> 1), col = tn * 32 + 16 * (g & 1) + r;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i][0][e]), __float_as_uint(acc[i][1][e]),
                                                      false, false);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = row0 + 16 * i + 4 * h + e;
        if (row < p.m && col < p.n) store1<DT>(p.c, row * p.ldc + col, __uint_as_float(x[h]), p.accumulate);
      }
    }
}

// Large products: a workgroup computes a BM x BN tile of C with WM x WN
// wavefronts, each TM x TN tiles of 32 x 32 in accumulators.  Per chunk of 256
// columns a row is 128 bytes of codes; both operands' chunks go from memory
// straight into LDS (16 bytes per lane, no registers), two stages, so the next
// chunk arrives while the matrix cores work on this one.  The hardware writes
// LDS in lane order; each lane therefore *fetches* the block that belongs
// there: block b of row r sits at slot b ^ mx_slot_key(r).  Scales come from
// memory into registers a chunk ahead, 256 contiguous bytes per 32 rows.
// Buffer descriptors end with the tile's last row: rows past it read as zero,
// without a fault.
constexpr int kChunkBytes = 128;

// Two rows of 128 bytes cover the 64 banks.  A 16-byte read goes through them
// in groups of lanes that take rows 0-3 and 12-15 of one block and rows 4-11
// of the block two further: with key (r / 2) % 8 both halves meet (counted:
// 3.7 conflict cycles a read), (r / 2 + 6) % 8 keeps them apart (0.1), and
// eight neighbouring rows stay apart too.
__device__ __forceinline__ int mx_slot_key(int row) { return ((row >> 1) + 6) & 7; }

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

// Accumulators to C.  Each wavefront passes RE rows at a time through LDS of
// its own and stores 16 bytes per lane, whole rows of its TN * 32 columns:
// straight from the accumulators 16-bit results would leave in 32-byte pieces,
// and the number of instructions is what this part costs.  The row pitch of 4
// floats beyond a multiple of 32 spreads the 16 rows that a write covers over
// all banks.  Rows past the end of C lie outside the buffer descriptor,
// columns past it get an offset outside it.  What C held is read RE rows at a
// time, before they pass through LDS (11008 x 4096 x 2048 fp32, added to C: 131
// -> 117 us; 4096 x 4096 x 2048, where the cache holds C, 35 -> 38).
template <int DT, int RE, int TM, int TN, bool ACC>
__device__ __forceinline__ void mx_store(const MxProductArgs& p, float* lds, int64_t row0, int64_t col0, int lane,
                                         const v4f (&acc)[2 * TM][2 * TN]) {
  using T = typename Elem<DT>::type;
  constexpr int E = 16 / (int)sizeof(T);
  constexpr int COLS = TN * 32, PITCH = COLS + 4, LPR = COLS / E, RPI = 64 / LPR;
  const int64_t rl = p.m - row0, cl = p.n - col0;  // rows and columns of C from here on
  if (rl <= 0 || cl <= 0) return;
  const uint32_t cols = (uint32_t)min((int64_t)COLS, cl), ldb = (uint32_t)(p.ldc * sizeof(T));
  T* base = static_cast<T*>(p.c) + row0 * p.ldc + col0;
  const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
      base, 0, (int)(((uint32_t)min((int64_t)(TM * 32), rl) - 1) * ldb + cols * (uint32_t)sizeof(T)), 0x00020000);
  const bool wide = ((((uint32_t)(uintptr_t)base | ldb | cols * (uint32_t)sizeof(T))) & 15) == 0;
  float* wr = lds + (lane & 15) * PITCH + (lane >> 4) * 4;
  const uint32_t c = (lane % LPR) * E;
  const float* rd = lds + (lane / LPR) * PITCH + c;
  const uint32_t off = c < cols ? (lane / LPR) * ldb + c * (uint32_t)sizeof(T) : 0x80000000u;
  constexpr int LOADS = RE / RPI;
#pragma unroll
  for (int i = 0; i < TM * 32 / RE; ++i) {
    v4u old[LOADS];
    if (ACC && wide)
#pragma unroll
      for (int k = 0; k < LOADS; ++k)
        old[k] = __builtin_amdgcn_raw_buffer_load_b128(rc, (int)(off + (uint32_t)(i * RE + k * RPI) * ldb), 0, 0);
#pragma unroll
    for (int h = 0; h < RE / 16; ++h)
#pragma unroll
      for (int j = 0; j < 2 * TN; ++j)
        *reinterpret_cast<v4f*>(wr + h * 16 * PITCH + j * 16) = acc[i * (RE / 16) + h][j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (wide) {
#pragma unroll
      for (int k = 0; k < LOADS; ++k) {
        float v[E];
        __builtin_memcpy(v, __builtin_assume_aligned(rd + k * RPI * PITCH, 16), sizeof v);
        if constexpr (ACC) add16<DT>(v, old[k]);
        __builtin_amdgcn_raw_buffer_store_b128(pack16<DT>(v), rc, (int)(off + (uint32_t)(i * RE + k * RPI) * ldb), 0, 0);
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
// where the stages have no room for 32 of each wavefront (rows of TN * 32 + 4
// floats, as many wavefronts to a stage array as fit).
template <int WAVES, int TN, int SA, int SB>
constexpr int mx_epilogue_rows() {
  constexpr int need = 32 * (TN * 32 + 4) * 4;
  return 2 * (SA / need + SB / need) >= WAVES ? 32 : 16;
}
template <int WAVES, int TN, int SA, int SB>
__device__ __forceinline__ float* mx_epilogue_lds(int wave, uint8_t* a0, uint8_t* b0, uint8_t* a1, uint8_t* b1) {
  constexpr int NEED = mx_epilogue_rows<WAVES, TN, SA, SB>() * (TN * 32 + 4) * 4, NA = SA / NEED, NB = SB / NEED;
  static_assert(2 * (NA + NB) >= WAVES, "stages too small for the results");
  if (wave < NA) return reinterpret_cast<float*>(a0 + wave * NEED);
  if (wave < NA + NB) return reinterpret_cast<float*>(b0 + (wave - NA) * NEED);
  if (wave < 2 * NA + NB) return reinterpret_cast<float*>(a1 + (wave - NA - NB) * NEED);
  return reinterpret_cast<float*>(b1 + (wave - 2 * NA - NB) * NEED);
}

template <int DT, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_mx_prod_lds(MxProductArgs p, int ntm, int ntn) {
  constexpr int WAVES = WM * WN, BM = WM * 32 * TM, BN = WN * 32 * TN;
  // Groups of products: one tile of 16 rows of A times all of the wavefront's
  // B; a chunk is two steps of HA groups.  A's operands are read DEPTH groups
  // ahead, B's one step ahead.
  constexpr int HA = 2 * TM, HB = 2 * TN, GROUPS = 2 * HA, DEPTH = 4;
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
  // One of the PA + PB loads of 8 rows of a wavefront's share of a chunk: the
  // slots of its blocks depend on whether the group of 8 rows is an even or an
  // odd one of the tile.
  constexpr int PA = BM / 8 / WAVES, PB = BN / 8 / WAVES;
  const int swap_a = PA & wave & 1, swap_b = PB & wave & 1;  // the wavefront's first group is an odd one
  auto lane_off = [&](int odd) { return (lane >> 3) * pitch + (((lane & 7) ^ mx_slot_key(8 * odd + (lane >> 3))) << 4); };
  const uint32_t lane_a[2] = {lane_off(swap_a), lane_off(1 - swap_a)};
  const uint32_t lane_b[2] = {lane_off(swap_b), lane_off(1 - swap_b)};
  const int r = lane & 15, g = lane >> 4;
  uint32_t off[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) off[s] = r * kChunkBytes + (((2 * g + s) ^ mx_slot_key(r)) << 4);
  // a wavefront's scale tiles; past the last tile of rows the last one again
  const uint32_t rtm = (uint32_t)((p.m + 31) / 32 - 1 - m0 / 32), rtn = (uint32_t)((p.n + 31) / 32 - 1 - n0 / 32);
  const __amdgpu_buffer_rsrc_t rsa =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.a.scales + m0 / 32 * nch * 256), 0,
                                        (int)((min(rtm, (uint32_t)(WM * TM - 1)) + 1) * nch * 256), 0x00020000);
  const __amdgpu_buffer_rsrc_t rsb =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.b.scales + n0 / 32 * nch * 256), 0,
                                        (int)((min(rtn, (uint32_t)(WN * TN - 1)) + 1) * nch * 256), 0x00020000);
  uint32_t as[TM], bs[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) as[i] = min((uint32_t)(wm * TM + i), rtm) * nch * 256;
#pragma unroll
  for (int j = 0; j < TN; ++j) bs[j] = min((uint32_t)(wn * TN + j), rtn) * nch * 256;
  v4f acc[HA][HB];
#pragma unroll
  for (int i = 0; i < HA; ++i)
#pragma unroll
    for (int j = 0; j < HB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  uint32_t sa[TM], sb[TN], ta[TM], tb[TN];
  const int la = wm * TM * 32 * kChunkBytes, lb = wn * TN * 32 * kChunkBytes;
  // One of those loads, and one of the wavefront's TM + TN scale tiles.  No
  // chunk past the last: an offset beyond the descriptor reads nothing.
  auto load_rows = [&](int j, uint32_t ch, uint8_t* da, uint8_t* db) {
    const bool isa = j < PA;
    const int i = isa ? j : j - PA, row = wave * (isa ? BM / WAVES : BN / WAVES) + i * 8;
    const uint32_t o = ch < nch ? ch * kChunkBytes : 0x80000000u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        isa ? ra : rb, (__attribute__((address_space(3))) void*)((isa ? da : db) + row * kChunkBytes), 16,
        (int)((isa ? lane_a : lane_b)[i & 1] + (uint32_t)row * pitch + o), 0, 0, 0);
  };
  auto load_scale = [&](int j, uint32_t ch, uint32_t(&xa)[TM], uint32_t(&xb)[TN]) {
    const uint32_t o = min(ch, nch - 1) * 256;
    if (j < TM)
      xa[j < TM ? j : 0] = __builtin_amdgcn_raw_buffer_load_b32(rsa, lane * 4, (int)(as[j < TM ? j : 0] + o), 0);
    else
      xb[j < TM ? 0 : j - TM] =
          __builtin_amdgcn_raw_buffer_load_b32(rsb, lane * 4, (int)(bs[j < TM ? 0 : j - TM] + o), 0);
  };
  auto read_a = [&](const uint8_t* m, int q) {  // group q of a chunk
    return *reinterpret_cast<const uint4*>(m + la + off[q / HA] + q % HA * 16 * kChunkBytes);
  };
  auto read_b = [&](const uint8_t* m, int s, int j) {
    return *reinterpret_cast<const uint4*>(m + lb + off[s] + j * 16 * kChunkBytes);
  };
  uint4 qa[DEPTH], qb[HB];  // entering a chunk: A's first DEPTH groups, B's step 0
  // The barrier stands DEPTH groups before the chunk's end: their operands are
  // in registers, so their products cover it and the first reads of the next
  // chunk, and behind it every wavefront is done with this chunk's stage.
  // From there on the loads of the chunk after the next go into that stage,
  // two to a group of a 128 x 128 tile, one to a group of the larger ones, so
  // that the last of them has three quarters of a chunk to arrive (2048 x 4096
  // x 11008: 55 us with the loads in the next chunk's first groups, 52 so);
  // all at once they hold up the products behind them.
  constexpr int PER_GROUP = (PA + PB) * 2 / GROUPS;
  static_assert(PA + PB <= PER_GROUP * GROUPS && TM + TN <= GROUPS - DEPTH, "loads between two barriers");
  auto chunk = [&](uint32_t next, uint8_t* ca, uint8_t* cb, uint8_t* na, uint8_t* nb,
                   const uint32_t(&xa)[TM], const uint32_t(&xb)[TN], uint32_t(&ya)[TM], uint32_t(&yb)[TN]) {
    uint4 a[GROUPS + DEPTH], b[3][HB];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) a[d] = qa[d];
#pragma unroll
    for (int j = 0; j < HB; ++j) b[0][j] = qb[j];
#pragma unroll
    for (int q = 0; q < GROUPS; ++q) {
      const int s = q / HA, i = q % HA;
      int reads = 1;
      if (q == GROUPS - DEPTH) {
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
      }
      const bool behind = q >= GROUPS - DEPTH;
      const int load = (behind ? q - (GROUPS - DEPTH) : q + DEPTH) * PER_GROUP;
#pragma unroll
      for (int j = load; j < load + PER_GROUP; ++j)
        if (j < PA + PB) load_rows(j, behind ? next + 1 : next, behind ? ca : na, behind ? cb : nb);
      if (q < TM + TN) load_scale(q, next, ya, yb);
      // B's next operands first: the first groups of step 0 read step 1's, the
      // first groups behind the barrier the next chunk's
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        if (q == j * (HA / 2) / HB) b[1][j] = read_b(cb, 1, j), ++reads;
        if (q == GROUPS - DEPTH + j * 2 / HB) b[2][j] = read_b(nb, 0, j), ++reads;
      }
      a[q + DEPTH] = q + DEPTH < GROUPS ? read_a(ca, q + DEPTH) : read_a(na, q + DEPTH - GROUPS);
#pragma unroll
      for (int j = 0; j < HB; ++j) acc[i][j] = mx_mfma_at(s, j & 1, i & 1, b[s][j], a[q], acc[i][j], xb[j / 2], xa[i / 2]);
      if (reads == 1)
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS reads
      else if (reads <= 3)
        __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
      else
        __builtin_amdgcn_sched_group_barrier(0x100, 5, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, HB, 0);  // products
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) qa[d] = a[GROUPS + d];
#pragma unroll
    for (int j = 0; j < HB; ++j) qb[j] = b[2][j];
  };
#pragma unroll
  for (int j = 0; j < TM + TN; ++j) load_scale(j, 0, sa, sb);
#pragma unroll
  for (int j = 0; j < PA + PB; ++j) load_rows(j, 0, a0, b0);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < min(PA + PB, DEPTH * PER_GROUP); ++j) load_rows(j, 1, a1, b1);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) qa[d] = read_a(a0, d);
#pragma unroll
  for (int j = 0; j < HB; ++j) qb[j] = read_b(b0, 0, j);
  // (an odd last chunk is paired with one of zero codes)
  for (uint32_t ch = 0; ch < nch; ch += 2) {
    chunk(ch + 1, a0, b0, a1, b1, sa, sb, ta, tb);
    chunk(ch + 2, a1, b1, a0, b0, ta, tb, sa, sb);
  }
  __syncthreads();  // (the last loads, of no chunk, write zeros into a stage)
  constexpr int RE = mx_epilogue_rows<WAVES, TN, sizeof a0, sizeof b0>();
  float* ep = mx_epilogue_lds<WAVES, TN, sizeof a0, sizeof b0>(wave, a0, b0, a1, b1);
  if (p.accumulate)
    mx_store<DT, RE, TM, TN, true>(p, ep, m0 + wm * TM * 32, n0 + wn * TN * 32, lane, acc);
  else
    mx_store<DT, RE, TM, TN, false>(p, ep, m0 + wm * TM * 32, n0 + wn * TN * 32, lane, acc);
}

// Few rows on one side (up to 128): the product is a stream of the other
// operand, "wide" here, and what counts is how many of its bytes are under
// way.  One workgroup = MT * 16 rows of the narrow operand (all of them) times
// NT * 32 rows of the wide one; its wavefronts take the summed axis' chunks in
// turn (neighbouring wavefronts read neighbouring 128 bytes of a row) and their
// partial tiles are added through LDS in wavefront order.  Each wavefront
// stages its chunks in LDS of its own, two ahead, straight from memory in
// whole 128-byte rows: reading the matrix cores' layout (16 bytes of each of
// many rows per access) from memory instead kept the cache's address lookup
// busy and took 12 us where this takes 7.5 (24 x 4096 x 11008).
// The narrow operand comes from memory (XDT < 0), or, where it is small enough,
// straight from the activations of type XDT, which every workgroup
// quantises into LDS by itself: one launch instead of two, with the first
// loads of the wide operand asked for before those of the activations.
// With 64 x 64 tiles the same kernel serves small products of any shape.
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

// One operand's part of a wavefront's chunk: R rows (a multiple of 16).
template <int R>
struct MxRows {
  static constexpr int T = (R + 31) / 32, kLoads = R / 8 + T, kBytes = R * kChunkBytes;
  __amdgpu_buffer_rsrc_t codes, scales;
  uint32_t pitch, nch, so[T];
  __device__ __forceinline__ MxRows(const MxOperand& o, int64_t row0, int64_t rows, int64_t k) {
    pitch = (uint32_t)mx_pitch(k);
    nch = (uint32_t)mx_chunks(k);
    const uint32_t left = (uint32_t)min((int64_t)R, rows - row0), tiles = (left + 31) / 32;
    codes = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(o.codes + row0 * pitch), 0, (int)(left * pitch),
                                              0x00020000);
    scales = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(o.scales + row0 / 32 * nch * 256), 0,
                                               (int)(tiles * nch * 256), 0x00020000);
#pragma unroll
    for (int t = 0; t < T; ++t) so[t] = min((uint32_t)t, tiles - 1) * nch * 256;
  }
  // Chunk ch to LDS and its scales to s; past the last chunk, nothing (zero
  // codes).
  __device__ __forceinline__ void fetch(uint32_t ch, uint8_t* lds, uint32_t (&s)[T], uint32_t off0, uint32_t off1,
                                        int lane) const {
    const uint32_t o = ch < nch ? ch * kChunkBytes : 0x80000000u, sc = min(ch, nch - 1) * 256;
#pragma unroll
    for (int t = 0; t < T; ++t) s[t] = __builtin_amdgcn_raw_buffer_load_b32(scales, lane * 4, (int)(so[t] + sc), 0);
#pragma unroll
    for (int j = 0; j < R / 8; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(codes, (__attribute__((address_space(3))) void*)(lds + j * 1024), 16,
                                               (int)((j & 1 ? off1 : off0) + j * 8 * pitch + o), 0, 0, 0);
  }
};

// One block of 32 activations (n of them valid) to codes and scale byte.
template <int DT>
__device__ __forceinline__ uint32_t mx_quant_block(const typename Elem<DT>::type* p, int n, uint4* q) {
  using T = typename Elem<DT>::type;
  constexpr int W = 32 / kPerWord<DT>;
  uint32_t w[W], am = 0;
  if (n >= 32) {
    __builtin_memcpy(w, p, sizeof w);
  } else {
    T v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i < n ? p[i] : (T)0;
    __builtin_memcpy(w, v, sizeof w);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) am = mx_max_words<DT>(am, w[i]);
  const uint32_t sb = mx_scale_byte(mx_max_bits<DT>(am));
  *q = make_uint4(mx_nearest8<DT>(w, sb), mx_nearest8<DT>(w + W / 4, sb), mx_nearest8<DT>(w + W / 2, sb),
                  mx_nearest8<DT>(w + 3 * W / 4, sb));
  return sb;
}

// The operand of the activations that a workgroup quantises by itself: codes
// and scales, in dynamic LDS (18 bytes per block).
extern __shared__ __align__(16) uint8_t psgd_mx_act[];

template <int WAVES, int MT, int NT, bool SWAP, int XDT>
__global__ __launch_bounds__(WAVES * 64, 1) void k_mx_prod_skinny(MxSkinnyArgs p, int nwt) {
  using WR = MxRows<NT * 32>;
  using XR = MxRows<MT * 16>;
  constexpr bool STAGED = XDT < 0;  // the narrow operand is staged like the wide one
  constexpr int STAGE = WR::kBytes + (STAGED ? XR::kBytes : 0), LOADS = WR::kLoads + (STAGED ? XR::kLoads : 0);
  constexpr int TILES = MT * 2 * NT;  // 16 x 16 tiles of a wavefront, 1 KB each
  static_assert(TILES * 1024 <= 2 * STAGE, "no room for the partial tiles");
  __shared__ __align__(16) uint8_t st0[WAVES * STAGE], st1[WAVES * STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t x0 = (int64_t)(blockIdx.x / nwt) * (MT * 16), w0 = (int64_t)(blockIdx.x % nwt) * (NT * 32);  // first rows
  const WR w(p.w, w0, p.wide, p.k);
  const XR x(STAGED ? p.x : p.w, STAGED ? x0 : w0, STAGED ? p.narrow : p.wide, p.k);
  const uint32_t nch = w.nch, pitch = w.pitch;
  // (the slots of the large products' tiles)
  const uint32_t off0 = (lane >> 3) * pitch + (((lane & 7) ^ mx_slot_key(lane >> 3)) << 4);
  const uint32_t off1 = (lane >> 3) * pitch + (((lane & 7) ^ mx_slot_key(8 + (lane >> 3))) << 4);
  uint32_t off[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) off[s] = r * kChunkBytes + (((2 * g + s) ^ mx_slot_key(r)) << 4);
  uint8_t *const m0 = st0 + wave * STAGE, *const m1 = st1 + wave * STAGE;
  uint32_t sw0[WR::T], sw1[WR::T], sx0[XR::T], sx1[XR::T];
  auto fetch = [&](uint32_t ch, uint8_t* m, uint32_t(&sw)[WR::T], uint32_t(&sx)[XR::T]) {
    w.fetch(ch, m, sw, off0, off1, lane);
    if constexpr (STAGED) x.fetch(ch, m + WR::kBytes, sx, off0, off1, lane);
  };
  uint32_t ch = wave;
  // (the order of the loads is what wait_memory counts on)
  fetch(ch, m0, sw0, sx0);
  __builtin_amdgcn_sched_barrier(0);
  fetch(ch + WAVES, m1, sw1, sx1);
  __builtin_amdgcn_sched_barrier(0);
  const int xrows = STAGED ? 0 : (int)p.narrow, xr16 = min(xrows, 16), xper = (int)nch * 8;
  uint8_t *const xc = psgd_mx_act, *const xs = xc + xrows * xper * 16;
  if constexpr (!STAGED) {
    constexpr int XD = XDT < 0 ? 0 : XDT;
    const auto* act = static_cast<const typename Elem<XD>::type*>(p.act);
    const int nblk = (int)mx_blocks(p.k);
    // (blocks past the last get zero codes and scale 0; scales in the dwords of
    // an operand's tiles, for the rows there are: chunk, pair of blocks, row % 16)
    for (int i = threadIdx.x; i < xrows * xper; i += WAVES * 64) {
      const int row = i / xper, b = i % xper;
      uint4 q = make_uint4(0, 0, 0, 0);
      uint32_t sb = 0;
      if (b < nblk) sb = mx_quant_block<XD>(act + row * p.ld + b * 32, (int)min((int64_t)32, p.k - b * 32), &q);
      reinterpret_cast<uint4*>(xc)[i] = q;
      xs[((b >> 1) * xr16 + (row & 15)) * 4 + (row >> 4) * 2 + (b & 1)] = (uint8_t)sb;
    }
    // (A barrier for LDS alone.  The stages were asked for first and loads come
    // back in order, so a wavefront that has its activations has its stages too.)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  }
  v4f acc[MT][2 * NT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < 2 * NT; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
  auto chunk = [&](uint32_t at, const uint8_t* m, const uint32_t(&sw)[WR::T], const uint32_t(&sx)[XR::T]) {
    const int xch = (int)min(at, nch - 1);
    uint32_t fx = 0;
    if constexpr (!STAGED) fx = reinterpret_cast<const uint32_t*>(xs)[(xch * 4 + g) * xr16 + min(r, xr16 - 1)];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint4 a[MT], b[2 * NT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if constexpr (STAGED)
          a[t] = *reinterpret_cast<const uint4*>(m + WR::kBytes + t * 16 * kChunkBytes + off[s]);
        else
          a[t] = reinterpret_cast<const uint4*>(xc)[min(t * 16 + r, xrows - 1) * xper + xch * 8 + 2 * g + s];
      }
#pragma unroll
      for (int u = 0; u < 2 * NT; ++u) b[u] = *reinterpret_cast<const uint4*>(m + u * 16 * kChunkBytes + off[s]);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < 2 * NT; ++u) {
          const uint32_t ss = STAGED ? sx[t / 2] : fx;
          acc[t][u] = SWAP ? mx_mfma_at(s, t & 1, u & 1, a[t], b[u], acc[t][u], ss, sw[u / 2])
                           : mx_mfma_at(s, u & 1, t & 1, b[u], a[t], acc[t][u], sw[u / 2], ss);
        }
    }
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
  // the partial tiles: as many as fit in st0, the rest in st1
  constexpr int SPLIT = WAVES * STAGE / 1024;
  auto at = [&](int i) {
    return reinterpret_cast<v4f*>(i < SPLIT ? st0 + i * 1024 : st1 + (i - SPLIT) * 1024) + lane;
  };
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < 2 * NT; ++u) *at(wave * TILES + t * 2 * NT + u) = acc[t][u];
  __syncthreads();
  // the wavefronts share the tiles; a lane has four columns of a row of C
  const int64_t rows = SWAP ? p.wide : p.narrow, cols = SWAP ? p.narrow : p.wide;
  for (int o = wave; o < TILES; o += WAVES) {
    const int64_t tx = x0 + o / (2 * NT) * 16, tw = w0 + o % (2 * NT) * 16;
    const int64_t row0 = SWAP ? tw : tx, col = (SWAP ? tx : tw) + 4 * g;
    if (row0 >= rows) continue;
    v4f v = *at(o);
#pragma unroll
    for (int k = 1; k < WAVES; ++k) v += *at(k * TILES + o);
    const int64_t row = row0 + r;
    if (row >= rows || col >= cols) continue;
    const int64_t ci = row * p.ldc + col;
    if (p.dtype == kF32)
      store4<kF32>(p.c, ci, v, cols - col, p.accumulate);
    else if (p.dtype == kBF16)
      store4<kBF16>(p.c, ci, v, cols - col, p.accumulate);
    else
      store4<kF16>(p.c, ci, v, cols - col, p.accumulate);
  }
}

// Eight wavefronts to a workgroup where all tiles fit on the compute units
// together (their stages take most of the LDS), four (two workgroups to a
// compute unit) where they do not, or where there is nothing to share.
template <int MT, int NT, bool SWAP, int XDT>
static void skinny(const MxSkinnyArgs& p, hipStream_t s) {
  const int64_t nwt = (p.wide + NT * 32 - 1) / (NT * 32), tiles = nwt * ((p.narrow + MT * 16 - 1) / (MT * 16));
  const uint32_t lds = XDT < 0 ? 0 : (uint32_t)(p.narrow * mx_chunks(p.k) * 8 * 18);
  if constexpr (MT <= 2 && NT == 1) {
    if (tiles <= 256 && mx_chunks(p.k) > 4) {
      hipLaunchKernelGGL((k_mx_prod_skinny<8, MT, NT, SWAP, XDT>), dim3((unsigned)tiles), dim3(512), lds, s, p,
                         (int)nwt);
      return;
    }
  }
  hipLaunchKernelGGL((k_mx_prod_skinny<4, MT, NT, SWAP, XDT>), dim3((unsigned)tiles), dim3(256), lds, s, p, (int)nwt);
}

// SWAP: the narrow side is C's columns.
template <bool SWAP>
static void product_skinny(const MxSkinnyArgs& p, hipStream_t s) {
  if (p.narrow <= 16)
    skinny<1, 1, SWAP, -1>(p, s);
  else if (p.narrow <= 32)
    skinny<2, 1, SWAP, -1>(p, s);
  else if (p.narrow <= 64)
    skinny<4, 1, SWAP, -1>(p, s);
  else
    skinny<8, 1, SWAP, -1>(p, s);
}

// Every workgroup (32 rows of the weights) repeats the activations' work, and
// those of one compute unit share it.  What that may cost is what a launch of
// its own takes, about 4 us, and an fp32 block costs three of 16 bits: 3584
// blocks is where that is reached (LDS would take more: beside the stages' 64 KB
// there is room for 5461 blocks of 18 bytes.  Two launches take 10.1 us.
// 4096 rows of weights, bf16: 16 x 4096 6.6, 24 x 4096 7.9, 8 x 11008 10.1;
// fp32: 8 x 4096 7.8, 12 x 4096 9.6, 4 x 11008 11.8.  11008 rows, bf16: 8 x 4096
// 8.3, 12 x 4096 9.6, 16 x 4096 10.5; fp32: 4 x 4096 9.1, 8 x 4096 12.4).
bool mx_linear_fuses(int64_t m, int64_t n, int64_t k, int x_dtype) {
  const int64_t blocks = m * mx_chunks(k) * 8, per_cu = (n + 32 * 256 - 1) / (32 * 256);
  return m <= 32 && k > 0 && blocks * (x_dtype == kF32 ? 3 : 1) * per_cu <= 3584;
}

template <int MT>
static void linear_fused(const MxSkinnyArgs& a, int x_dtype, hipStream_t s) {
  if (x_dtype == kF32)
    skinny<MT, 1, false, kF32>(a, s);
  else if (x_dtype == kBF16)
    skinny<MT, 1, false, kBF16>(a, s);
  else
    skinny<MT, 1, false, kF16>(a, s);
}

hipError_t launch_mx_linear_fused(const MxProductArgs& p, const void* x, int x_dtype, int64_t ldx, hipStream_t s) {
  const MxSkinnyArgs a{p.m, p.n, p.k, {nullptr, nullptr}, p.b, x, ldx, p.c, p.ldc, p.dtype, false};
  if (p.m <= 16)
    linear_fused<1>(a, x_dtype, s);
  else
    linear_fused<2>(a, x_dtype, s);
  return hipGetLastError();
}

// An empty sum: C = 0.
template <int DT>
__global__ __launch_bounds__(256) void k_mx_prod_zero(MxProductArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < p.m * p.n) static_cast<typename Elem<DT>::type*>(p.c)[i / p.n * p.ldc + i % p.n] = Elem<DT>::down(0.f);
}


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
  // Large tiles read their operands fewer times, but 256 compute units work on
  // one each at a time, so what counts is the rounds.  192 rows instead of 256
  // where their rounds, 3/4 as long, end sooner (2048 x 11008 x 4096,
  // bf16: 344 tiles of 256 x 256, two rounds, 65 us; 473 of 192 x 256, two
  // shorter ones, 54; 1376 of 128 x 128 59).  Where large tiles occupy at most
  // half of the compute units, 128 x 128, two to a compute unit (2048 x 4096 x
  // 11008: 128 tiles of 256 x 256 70 us, 176 of 192 x 256 61, 512 of 128 x 128
  // 52); where even 64 x 64 tiles are few, such tiles whose wavefronts share
  // the summed axis.  A single chunk is a write of C and hardly a product:
  // small workgroups.
  auto tiles = [&](int64_t bm, int64_t bn) { return ((p.m + bm - 1) / bm) * ((p.n + bn - 1) / bn); };
  auto rounds = [&](int64_t bm) { return (tiles(bm, 256) + 255) / 256; };
  if (fits && p.k > 256) {
    if (tiles(64, 64) <= 256)
      skinny<4, 2, false, -1>(ab, s);
    else if (tiles(256, 256) <= 128)
      product_lds<DT, 2, 2, 2, 2>(p, s);
    else if (3 * rounds(192) < 4 * rounds(256))
      product_lds<DT, 2, 4, 3, 2>(p, s);
    else
      product_lds<DT, 2, 4, 4, 2>(p, s);
    return;
  }
  const int ntn = (int)((p.n + 63) / 64);
  hipLaunchKernelGGL((k_mx_prod_tile<DT>), dim3((unsigned)(((p.m + 63) / 64) * ntn)), dim3(256), 0, s, p, ntn);
}

hipError_t launch_mx_product(const MxProductArgs& p, hipStream_t s) {
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
