// Products of 16-bit matrices on the matrix cores (gfx950): the tile loop that
// the vocabulary cross entropy and the orthogonalised step share, each with
// epilogues of its own.
//
// A workgroup computes a BM x BN tile of C = A B^T with WM x WN wavefronts, each
// TM x TN tiles of 32 x 32 in accumulators, in chunks along the summed axis: 64
// values of 16-bit matrices.  An fp32 matrix is held as two fp16 pieces, hi + lo (22
// bits of a value down to 2^-16 of the largest of the scale they share; an error of
// 2^-38 of that largest, half of fp16's smallest step, below): 32 upper pieces
// followed by the same values' lower ones (a line of 128 bytes); of such matrices a
// chunk is 32 values, both pieces of both operands, and a product
// hi lo + hi hi + lo hi.  (As three products one after the other every piece is read
// one and a half times as often, and LDS reads are what the smaller tiles wait for.)
//
// Each operand's tile goes from memory straight into LDS (16 bytes per lane, no
// registers), two stages, so the next chunk arrives while the matrix cores work
// on this one.  Operands come in two orders:
//   K-contiguous  rows of the tile's axis, the summed axis along a row: 128
//                 bytes of every row (and piece: 64) per chunk;
//   K-strided     rows of the summed axis, the tile's axis along a row: 64 rows
//                 (or 32 of each piece) of the tile's width per chunk, which the
//                 transposing LDS read hands to the matrix cores in their own
//                 order.  So no operand is ever transposed in memory.
// The hardware writes LDS in lane order; each lane therefore *fetches* the 16
// bytes that belong at its place.  Buffer descriptors end with the operand:
// rows past it read as zero, without a fault.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "psgd_mx_device.h"

namespace psgd {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

template <bool PAIR>
constexpr int kMmaK = PAIR ? 32 : 64;      // values of the summed axis in a chunk
constexpr int kMmaBytes = 128;             // bytes of a tile's row in a chunk
constexpr uint32_t kMmaOff = 0x80000000u;  // an offset that no descriptor reaches

// One operand: `len` (K-contiguous) or k (K-strided) rows, 16-byte aligned, the
// row stride a multiple of 8.  K-contiguous rows are zero from k on to the next
// multiple of 8.
struct MmaSide {
  const uint16_t* p;
  int64_t ld;   // row stride (in pieces where there are two)
  int64_t len;  // size of the tile's axis
};

// Where value c of a row of pairs has its upper piece (its lower one: kMmaLow on).
constexpr int kMmaLow = 32;
__host__ __device__ constexpr int64_t mma_piece(int64_t c) { return c / 32 * 64 + c % 32; }

template <int DT>
__device__ __forceinline__ v4f mma16(uint4 a, uint4 b, v4f c) {
  if constexpr (DT == kBF16) {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  } else {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
}

// The place of a 16-byte block in a row of 128 bytes of a K-contiguous tile:
// block ^ key (what a 16-byte read's groups of lanes need to miss each other,
// see the 4-bit products).
__device__ __forceinline__ int mma_key(int row) { return ((row >> 1) + 6) & 7; }
// K-strided: units of 32 bytes, that is 16 values of a row, move by unit ^ key.
// A transposing read takes rows 16 g + 8 s + 0..3 (or 4..7) of one unit for the
// lanes' groups g: four neighbouring rows and two neighbouring g stay apart.
template <int UNITS>
__device__ __forceinline__ int mma_tunit(int unit, int k) {
  static_assert((UNITS & (UNITS - 1)) == 0, "keys of whole powers of two");
  return unit ^ (((k & 3) | (k >> 2 & 4)) & (UNITS - 1));
}

// One operand's side of the tile loop: R rows of the tile's axis, W wavefronts
// that load it.  The 16-byte blocks that a wavefront reads in its two steps
// alternate (MmaRead), so pieces do: block 2 b of a K-contiguous row is block b
// of the upper piece's values and block 2 b + 1 of the lower one's, and 8 rows of
// a K-strided tile are of the upper piece, the next 8 of the lower one.
template <bool PAIR, bool KC, int R, int W>
struct MmaLoad {
  static constexpr int kLoads = R / 8 / W, kBytes = R * kMmaBytes, K = kMmaK<PAIR>;
  static_assert(R % (8 * W) == 0, "whole loads");
  static constexpr int kSlots = R / 8;  // K-strided: 16-byte slots of a row
  const uint16_t* p;  // the tile's first value
  int64_t ld;
  uint32_t rows, left, off[kLoads], slot[2];
  __amdgpu_buffer_rsrc_t r;  // of the present chunk
  __device__ __forceinline__ MmaLoad(const MmaSide& s, int64_t r0, int wave, int lane) {
    ld = s.ld;
    rows = (uint32_t)min((int64_t)R, s.len - r0);
    p = s.p + (KC ? r0 * s.ld : PAIR ? mma_piece(r0) : r0);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      if constexpr (KC) {
        const int row = (wave * kLoads + j) * 8 + (lane >> 3), b = (lane & 7) ^ mma_key(row);
        off[j] = (uint32_t)(row * s.ld * 2) + (PAIR ? (b >> 1) * 16 + (b & 1) * (kMmaLow * 2) : b * 16);
      } else {
        const int at = (wave * kLoads + j) * 64 + lane, row = at / kSlots, b = at % kSlots;
        const int c = mma_tunit<kSlots / 2>(b >> 1, row) * 2 + (b & 1);  // the block of 8 columns
        off[j] = PAIR ? (uint32_t)(((row >> 4) * 8 + (row & 7)) * s.ld * 2) + (c >> 2) * 128 + (c & 3) * 16 +
                            (row >> 3 & 1) * (kMmaLow * 2)
                      : (uint32_t)(row * s.ld * 2) + c * 16;
      }
    }
    if constexpr (KC) {  // first values of the blocks of even and odd groups of 8 rows
      slot[0] = (((lane & 7) ^ mma_key(lane >> 3)) >> (PAIR ? 1 : 0)) * 8;
      slot[1] = (((lane & 7) ^ mma_key(8 + (lane >> 3))) >> (PAIR ? 1 : 0)) * 8;
    }
  }
  // To a chunk of which `left` values are left (0: a chunk of zeros).  Without
  // branches, which would cut the loop into pieces that the compiler schedules
  // one by one.  (Rows of pairs are whole lines.)
  __device__ __forceinline__ void seek(uint32_t chunk, uint32_t left_) {
    left = left_;
    const uint16_t* at = p + (int64_t)chunk * (KC ? 64 : K * ld);
    const uint32_t some = min(left, 1u), pitch = (uint32_t)ld * 2;
    uint32_t n;
    if constexpr (KC)
      n = (rows - 1) * pitch + (PAIR ? kMmaBytes : left * 2);
    else
      n = (min(left, (uint32_t)K) - some) * pitch + (PAIR ? (rows + 31) / 32 * 128 : rows * 2);
    r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(at), 0, (int)(((n + 15) & ~15u) * some), 0x00020000);
  }
  // Load j of that chunk.
  __device__ __forceinline__ void load(int j, uint8_t* lds, int wave) const {
    uint32_t o = off[j];
    if constexpr (KC) o = slot[(wave * kLoads + j) & 1] < left ? o : kMmaOff;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)(lds + (wave * kLoads + j) * 1024), 16, (int)o, 0, 0, 0);
  }
};

// What a wavefront reads of an operand's tile: its tile of 16 rows number i,
// step s of a chunk; lane group g gets blocks 2 g + s: values (2 g + s) * 8 .. + 7
// of the summed axis, or values 8 g .. + 7 of the upper (s = 0) or lower piece.
template <bool KC, int R>
struct MmaRead {
  static constexpr int kReads = KC ? 1 : 2;  // LDS reads an operand takes
  uint32_t off[2];
  int base;  // first tile of 16 rows
  __device__ __forceinline__ MmaRead(int first, int lane) {
    const int r = lane & 15, g = lane >> 4;
    base = first;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if constexpr (KC)
        off[s] = r * kMmaBytes + (((2 * g + s) ^ mma_key(r)) << 4);
      else
        off[s] = ((2 * g + s) * 8 + (r >> 2)) * (R * 2) + (r & 3) * 8;
    }
  }
  __device__ __forceinline__ uint4 operator()(const uint8_t* m, int s, int i) const {
    if constexpr (KC) {
      return *reinterpret_cast<const uint4*>(m + off[s] + (base + i) * 16 * kMmaBytes);
    } else {
      // (rows 4 apart have the same key)
      typedef short v4s __attribute__((ext_vector_type(4)));
      const uint8_t* q = m + off[s] + (mma_tunit<R / 16>(base + i, (threadIdx.x & 15) >> 2 | (threadIdx.x & 16)) << 5);
      typedef __attribute__((address_space(3))) v4s* lds4;
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(__attribute__((address_space(3))) void*)(q));
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(__attribute__((address_space(3))) void*)(q + 4 * R * 2));
      const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
      return make_uint4(x.x, x.y, y.x, y.y);
    }
  }
};

template <int N>
__device__ __forceinline__ void sched_lds_reads() {
  __builtin_amdgcn_sched_group_barrier(0x100, N, 0);
}

// The loop: accumulators of chunks c0 .. c1 - 1.
//
// Groups of products: one tile of 16 rows of A times all of the wavefront's B;
// a chunk is two steps of HA groups, of pieces the upper one of A (times both of
// B) and the lower one (times the upper one).  A's operands are read DEPTH
// groups ahead, B's one step (of pieces: a chunk) ahead.  The barrier stands
// DEPTH groups before the chunk's end: their operands are in registers, so their
// products cover it and the first reads of the next chunk, and behind it every
// wavefront is done with this chunk's stage.  From there on the loads of the
// chunk after the next go into that stage, spread over the groups.
template <int DT, bool PAIR, bool AKC, bool BKC, int WM, int WN, int TM, int TN>
struct MmaTile {
  static constexpr int WAVES = WM * WN, BM = WM * 32 * TM, BN = WN * 32 * TN;
  static constexpr int HA = 2 * TM, HB = 2 * TN, GROUPS = 2 * HA, DEPTH = HA >= 8 ? 4 : 2;
  using LA = MmaLoad<PAIR, AKC, BM, WAVES>;
  using LB = MmaLoad<PAIR, BKC, BN, WAVES>;
  static constexpr int PA = LA::kLoads, PB = LB::kLoads, K = kMmaK<PAIR>;
  static constexpr int PER_GROUP = (PA + PB + GROUPS * 3 / 4 - 1) / (GROUPS * 3 / 4);
  static_assert(PA + PB <= PER_GROUP * GROUPS, "loads between two barriers");
  typedef v4f Acc[HA][HB];

  static __device__ __forceinline__ void run(const MmaSide& sa, const MmaSide& sb, int64_t k, uint32_t c0, uint32_t c1,
                                             int64_t m0, int64_t n0, uint8_t* a0, uint8_t* b0, uint8_t* a1,
                                             uint8_t* b1, Acc& acc) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    LA la(sa, m0, wave, lane);
    LB lb(sb, n0, wave, lane);
    const MmaRead<AKC, BM> ra(wave / WN * HA, lane);
    const MmaRead<BKC, BN> rb(wave % WN * HB, lane);
    uint32_t at = c0;  // the next chunk to load
    auto seek = [&] {
      const uint32_t c = min(at, c1 - 1), left = ((uint32_t)k - c * K) * min(c1 - min(at, c1), 1u);
      la.seek(c, left);
      lb.seek(c, left);
    };
    auto step = [&] {
      ++at;
      seek();
    };
    seek();
    auto load = [&](int j, uint8_t* da, uint8_t* db) {
      if (j < PA)
        la.load(j < PA ? j : 0, da, wave);
      else
        lb.load(j < PA ? 0 : j - PA, db, wave);
    };
#pragma unroll
    for (int i = 0; i < HA; ++i)
#pragma unroll
      for (int j = 0; j < HB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    // entering a chunk: A's first DEPTH groups, B's step 0 (of pieces: both)
    constexpr int NB = PAIR ? 2 : 1;
    uint4 qa[DEPTH], qb[NB][HB];
    auto chunk = [&](uint8_t* ca, uint8_t* cb, uint8_t* na, uint8_t* nb) {
      uint4 a[GROUPS + DEPTH], b[2 + NB][HB];
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) a[d] = qa[d];
#pragma unroll
      for (int s = 0; s < NB; ++s)
#pragma unroll
        for (int j = 0; j < HB; ++j) b[s][j] = qb[s][j];
#pragma unroll
      for (int q = 0; q < GROUPS; ++q) {
        const int s = q / HA, i = q % HA;
        int nb_reads = 0;
        if (q == GROUPS - DEPTH) {
          __syncthreads();
          step();
          __builtin_amdgcn_sched_barrier(0);
        }
        const bool behind = q >= GROUPS - DEPTH;
        const int first = (behind ? q - (GROUPS - DEPTH) : q + DEPTH) * PER_GROUP;
#pragma unroll
        for (int j = first; j < first + PER_GROUP; ++j)
          if (j < PA + PB) load(j, behind ? ca : na, behind ? cb : nb);
#pragma unroll
        for (int j = 0; j < HB; ++j) {
          if (!PAIR && q == j * (HA / 2) / HB) b[1][j] = rb(cb, 1, j), ++nb_reads;
          if (q == GROUPS - DEPTH + j * (PAIR ? DEPTH : DEPTH / 2) / HB) {
#pragma unroll
            for (int n = 0; n < NB; ++n) b[2 + n][j] = rb(nb, n, j), ++nb_reads;
          }
        }
        a[q + DEPTH] = q + DEPTH < GROUPS ? ra(ca, (q + DEPTH) / HA, (q + DEPTH) % HA) : ra(na, 0, q + DEPTH - GROUPS);
        if constexpr (PAIR) {
          if (s == 0) {
#pragma unroll
            for (int j = 0; j < HB; ++j) acc[i][j] = mma16<DT>(b[1][j], a[q], acc[i][j]);
          }
#pragma unroll
          for (int j = 0; j < HB; ++j) acc[i][j] = mma16<DT>(b[0][j], a[q], acc[i][j]);
        } else {
#pragma unroll
          for (int j = 0; j < HB; ++j) acc[i][j] = mma16<DT>(b[s][j], a[q], acc[i][j]);
        }
        constexpr int RA = MmaRead<AKC, BM>::kReads, RB = MmaRead<BKC, BN>::kReads;
        if (nb_reads == 0)
          sched_lds_reads<RA>();
        else if (nb_reads == 1)
          sched_lds_reads<RA + RB>();
        else if (nb_reads == 2)
          sched_lds_reads<RA + 2 * RB>();
        else
          sched_lds_reads<RA + 4 * RB>();
        if (PAIR && s == 0)
          __builtin_amdgcn_sched_group_barrier(0x008, 2 * HB, 0);  // products
        else
          __builtin_amdgcn_sched_group_barrier(0x008, HB, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) qa[d] = a[GROUPS + d];
#pragma unroll
      for (int s = 0; s < NB; ++s)
#pragma unroll
        for (int j = 0; j < HB; ++j) qb[s][j] = b[2 + s][j];
    };
#pragma unroll
    for (int j = 0; j < PA + PB; ++j) load(j, a0, b0);
    step();
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PA + PB; ++j)
      if (j < DEPTH * PER_GROUP) load(j, a1, b1);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) qa[d] = ra(a0, 0, d);
#pragma unroll
    for (int s = 0; s < NB; ++s)
#pragma unroll
      for (int j = 0; j < HB; ++j) qb[s][j] = rb(b0, s, j);
    // (an odd last chunk is paired with one of zeros)
    for (uint32_t c = c0; c < c1; c += 2) {
      chunk(a0, b0, a1, b1);
      chunk(a1, b1, a0, b0);
    }
    __syncthreads();  // (the last loads, of no chunk, write zeros into a stage)
  }
};

// Accumulators to memory: C = alpha * 2^(exponent + the row's) * sum (+ add) (+ C).
// Each wavefront passes 32 rows at a time through LDS of its own and stores 16 bytes per lane, whole
// rows of its TN * 32 columns; the row pitch of 4 floats beyond a multiple of 32
// spreads the 16 rows that a write covers over all banks.
struct MmaOut {
  void* c;
  int64_t ldc, m, n;
  const float* add;  // m x n fp32, row stride n, or null
  bool accumulate;
  const int* row;  // m exponents, or null
};

// v times a power of two that need be no fp32 number, behind one rounding.
__device__ __forceinline__ float mma_scaled(float v, float alpha, int exponent) {
  return __builtin_amdgcn_ldexpf(v * alpha, exponent);
}

template <class Tile>
__device__ __forceinline__ float* mma_epilogue_lds(int wave, uint8_t* a0, uint8_t* b0, uint8_t* a1, uint8_t* b1) {
  constexpr int NEED = 32 * (Tile::HB * 16 + 4) * 4, NA = Tile::BM * kMmaBytes / NEED, NB = Tile::BN * kMmaBytes / NEED;
  static_assert(2 * (NA + NB) >= Tile::WAVES, "stages too small for the results");
  if (wave < NA) return reinterpret_cast<float*>(a0 + wave * NEED);
  if (wave < NA + NB) return reinterpret_cast<float*>(b0 + (wave - NA) * NEED);
  if (wave < 2 * NA + NB) return reinterpret_cast<float*>(a1 + (wave - NA - NB) * NEED);
  return reinterpret_cast<float*>(b1 + (wave - 2 * NA - NB) * NEED);
}

// N neighbouring values of the caller's memory, n of them there: as one vector,
// as pairs where a row starts on a pair only, or one by one.
template <int DT, int N>
__device__ __forceinline__ void load_run(const typename Elem<DT>::type* at, float (&v)[N], int n) {
  using T = typename Elem<DT>::type;
  T o[N];
  if (N > 2 && n >= N && ((uintptr_t)at & 15) == 0) {
    __builtin_memcpy(o, __builtin_assume_aligned(at, 16), sizeof o);
  } else if (N > 1 && n >= N && ((uintptr_t)at & (2 * sizeof(T) - 1)) == 0) {
#pragma unroll
    for (int e = 0; e + 1 < N; e += 2) __builtin_memcpy(o + e, __builtin_assume_aligned(at + e, 2 * sizeof(T)), 2 * sizeof(T));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = e < n ? at[e] : (T)0;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = Elem<DT>::up(o[e]);
}
template <int DT, int N>
__device__ __forceinline__ void store_run(typename Elem<DT>::type* at, const float (&v)[N], int n) {
  using T = typename Elem<DT>::type;
  T o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = Elem<DT>::down(v[e]);
  if (N > 2 && n >= N && ((uintptr_t)at & 15) == 0) {
    __builtin_memcpy(__builtin_assume_aligned(at, 16), o, sizeof o);
  } else if (N > 1 && n >= N && ((uintptr_t)at & (2 * sizeof(T) - 1)) == 0) {
#pragma unroll
    for (int e = 0; e + 1 < N; e += 2) __builtin_memcpy(__builtin_assume_aligned(at + e, 2 * sizeof(T)), o + e, 2 * sizeof(T));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < n) at[e] = o[e];
  }
}

// 32 rows of C from LDS, E neighbouring values a lane: as many as the address and
// the row stride allow to be one access, so that lanes write without gaps.
template <int DT, int E, int COLS>
__device__ __forceinline__ void mma_store_rows(const MmaOut& p, int exponent, const float* lds, int64_t row0, int64_t col0) {
  using T = typename Elem<DT>::type;
  constexpr int PITCH = COLS + 4, LPR = COLS / E, RPI = 64 / LPR;
  const int lane = threadIdx.x & 63, c = lane % LPR * E;
  const int n = (int)min((int64_t)E, p.n - col0 - c);
#pragma unroll 4
  for (int k = 0; k < 32 / RPI; ++k) {
    const int in = k * RPI + lane / LPR;
    const int64_t row = row0 + in;
    if (row >= p.m || n <= 0) continue;
    float v[E], w[E];
    __builtin_memcpy(v, __builtin_assume_aligned(lds + in * PITCH + c, E >= 4 ? 16 : 4 * E), sizeof v);
    const int x = exponent + (p.row ? p.row[row] : 0);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = __builtin_amdgcn_ldexpf(v[e], x);
    if (p.add) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += e < n ? p.add[row * p.n + col0 + c + e] : 0.f;
    }
    T* const at = static_cast<T*>(p.c) + row * p.ldc + col0 + c;
    if (p.accumulate) {
      load_run<DT, E>(at, w, n);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += w[e];
    }
    if (n < E) {
      store_run<DT, E>(at, v, n);
    } else {
      T o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = Elem<DT>::down(v[e]);
      __builtin_memcpy(__builtin_assume_aligned(at, E * sizeof(T)), o, sizeof o);
    }
  }
}

// (exponent: of what is in LDS, which may be taken times it here or before)
template <int DT, int COLS>
__device__ __forceinline__ void mma_store_any(const MmaOut& p, int exponent, const float* lds, int64_t row0, int64_t col0) {
  using T = typename Elem<DT>::type;
  const uintptr_t step = (uintptr_t)(static_cast<T*>(p.c) + row0 * p.ldc + col0) | (uintptr_t)(p.ldc * (int64_t)sizeof(T));
  if ((step & 15) == 0)
    mma_store_rows<DT, 16 / (int)sizeof(T), COLS>(p, exponent, lds, row0, col0);
  else if ((step & (2 * sizeof(T) - 1)) == 0)
    mma_store_rows<DT, 2, COLS>(p, exponent, lds, row0, col0);
  else
    mma_store_rows<DT, 1, COLS>(p, exponent, lds, row0, col0);
}

template <int DT, int HA, int HB>
__device__ __forceinline__ void mma_store(const MmaOut& p, float alpha, int exponent, float* lds, int64_t row0, int64_t col0,
                                          const v4f (&acc)[HA][HB]) {
  using T = typename Elem<DT>::type;
  const int lane = threadIdx.x & 63;
  constexpr int E = 16 / (int)sizeof(T);
  constexpr int COLS = HB * 16, PITCH = COLS + 4, LPR = COLS / E, RPI = 64 / LPR;
  if (row0 >= p.m || col0 >= p.n) return;
  T* const base = static_cast<T*>(p.c) + row0 * p.ldc + col0;
  const uintptr_t step = (uintptr_t)base | (uintptr_t)(p.ldc * (int64_t)sizeof(T));
  const bool whole = (step & 15) == 0 && p.n - col0 >= COLS && p.m - row0 >= HA * 16 && !p.add && !p.accumulate && !p.row;
  float* const wr = lds + (lane & 15) * PITCH + (lane >> 4) * 4;
#pragma unroll
  for (int i = 0; i < HA / 2; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        v4f v = acc[i * 2 + h][j];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= alpha;
        *reinterpret_cast<v4f*>(wr + h * 16 * PITCH + j * 16) = v;
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (whole) {
#pragma unroll
      for (int k = 0; k < 32 / RPI; ++k) {
        const int row = k * RPI + lane / LPR;
        float v[E];
        __builtin_memcpy(v, __builtin_assume_aligned(lds + row * PITCH + lane % LPR * E, 16), sizeof v);
        T o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = Elem<DT>::down(__builtin_amdgcn_ldexpf(v[e], exponent));
        __builtin_memcpy(__builtin_assume_aligned(base + (i * 32 + row) * p.ldc + lane % LPR * E, 16), o, sizeof o);
      }
    } else {
      mma_store_any<DT, COLS>(p, exponent, lds, row0 + i * 32, col0);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Largest value and sum over the four groups of 16 lanes, in all of them.
__device__ __forceinline__ float groups_max(float v) {
  const uint32_t a = __float_as_uint(v);
  const auto x = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const uint32_t b = __float_as_uint(fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])));
  const auto y = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
__device__ __forceinline__ float groups_sum(float v) {
  const uint32_t a = __float_as_uint(v);
  const auto x = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const uint32_t b = __float_as_uint(__uint_as_float(x[0]) + __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}

// The walk over the tiles: groups of 8 tile rows, so that the 32 tiles that an
// XCD's compute units work on at a time form an 8 x 4 block that shares its
// operands in L2.
__device__ __forceinline__ void mma_tile_of_block(int b, int ntm, int ntn, int* tm, int* tn) {
  const int t = xcd_position(b, ntm * ntn);
  const int first = t / (8 * ntn) * 8, rows = min(8, ntm - first), in = t % (8 * ntn);
  *tm = first + in % rows;
  *tn = in / rows;
}

}  // namespace psgd
