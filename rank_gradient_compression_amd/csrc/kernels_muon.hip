// Orthogonalised updates of a list of matrices (gfx950).
//
//   m <- mu m + g,  u = g + mu m (Nesterov) or m,  X = u / (||u|| + eps)
//   steps times:  A = X X^T,  B = b A + c A^2,  X <- a X + B X
//   p <- decay p - step X
//
// with the shorter side's Gram matrix: A = X^T X and X <- a X + X B where there
// are more rows than columns.  A and B are symmetric: only their tiles on and
// above the diagonal are computed, and each is stored a second time across it.
//
// Every launch takes all matrices of a group, whatever their sizes and which way
// round they are: a list of many small matrices costs as many launches as one.
// No matrix is transposed in memory; the tile loop reads its operands in either
// order (psgd_mma_device.h).
//
// Precision.  X is kept as two fp16 pieces (22 bits) times a power of two.
// Where results have 16 bits' worth to give (bfloat16), the products take X's
// upper piece and A and B as one fp16 piece, while a X, the part that carries
// the small singular values from step to step, is formed from both pieces: with
// X itself in 16 bits, what rounding adds under large singular values grows by a
// a step with the small ones (512 x 512, rank 16 over noise of 1/20: 6e-3 off
// with fp16 X, 5e-2 with bfloat16, 1.5e-4 so; Gaussian: 1.5e-3).  Over gradients'
// spectra that is 1.77e-3 where bfloat16's own rounding is 1.66e-3.  Other results,
// and thin matrices' (kMuonThin), take two pieces of everything, three products for
// one.  In the last two steps, where singular values are near 1 and B near b + c, the
// identity's part of a X that cancels against B's goes into B instead, whose
// roundings are then of what is left: X <- (a + b + c) X + (B - (b + c) I) X
// (Gaussian: 1.7e-3 -> 1.0e-3; from the first step on it would cost the small singular
// values what the two pieces gave them).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "psgd_mma_device.h"
#include "psgd_muon.h"

namespace psgd {

constexpr int kSumGroups = 1024;  // workgroups of one matrix's norm, at most
constexpr int kSumChunk = 4096;   // values of a workgroup at a time

__host__ __device__ inline int64_t muon_ld(int64_t c) { return (c + 63) / 64 * 64; }

__device__ __forceinline__ float muon_load(const void* p, int dtype, int64_t i) {
  if (dtype == kF32) return static_cast<const float*>(p)[i];
  if (dtype == kBF16) return Elem<kBF16>::up(static_cast<const uint16_t*>(p)[i]);
  return Elem<kF16>::up(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void muon_save(void* p, int dtype, int64_t i, float v) {
  if (dtype == kF32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == kBF16)
    static_cast<uint16_t*>(p)[i] = Elem<kBF16>::down(v);
  else
    static_cast<uint16_t*>(p)[i] = Elem<kF16>::down(v);
}
// Four neighbouring values.
__device__ __forceinline__ float4 muon_load4(const void* p, int dtype, int64_t i) {
  if (dtype == kF32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  const uint16_t h[4] = {(uint16_t)w.x, (uint16_t)(w.x >> 16), (uint16_t)w.y, (uint16_t)(w.y >> 16)};
  if (dtype == kBF16)
    return make_float4(Elem<kBF16>::up(h[0]), Elem<kBF16>::up(h[1]), Elem<kBF16>::up(h[2]), Elem<kBF16>::up(h[3]));
  return make_float4(Elem<kF16>::up(h[0]), Elem<kF16>::up(h[1]), Elem<kF16>::up(h[2]), Elem<kF16>::up(h[3]));
}
__device__ __forceinline__ float2 muon_load2(const void* p, int dtype, int64_t i) {
  if (dtype == kF32) return *reinterpret_cast<const float2*>(static_cast<const float*>(p) + i);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + i);
  if (dtype == kBF16) return make_float2(Elem<kBF16>::up((uint16_t)w), Elem<kBF16>::up((uint16_t)(w >> 16)));
  return make_float2(Elem<kF16>::up((uint16_t)w), Elem<kF16>::up((uint16_t)(w >> 16)));
}
__device__ __forceinline__ bool aligned2(const void* p, int dtype) {
  return ((uintptr_t)p & (dtype == kF32 ? 7 : 3)) == 0;
}
__device__ __forceinline__ bool aligned4(const void* p, int dtype) {
  return ((uintptr_t)p & (dtype == kF32 ? 15 : 7)) == 0;
}

// The tables, from the arguments of one launch (5 us).
__global__ __launch_bounds__(256) void k_muon_table(MuonTable p, MuonTable* t) {
  const uint32_t* from = reinterpret_cast<const uint32_t*>(&p);
  uint32_t* to = reinterpret_cast<uint32_t*>(t);
  for (int i = threadIdx.x; i < (int)(sizeof p / 4); i += 256) to[i] = from[i];
}

__device__ __forceinline__ uint16_t* muon_at(const MuonArgs& p, uint32_t place) {
  return reinterpret_cast<uint16_t*>(p.ws + (size_t)place * 256);
}
__device__ __forceinline__ uint16_t* muon_x(const MuonArgs& p, const MuonMat& t, bool next) {
  return muon_at(p, p.odd != next ? t.x1 : t.x0);
}

// The last matrix whose range starts at t or before: every lane looks at one.
__device__ __forceinline__ int muon_find(const int32_t (&starts)[kMuonGroup], int t) {
  const int lane = threadIdx.x & 63;
  return __popcll(__ballot(starts[min(lane, kMuonGroup - 1)] <= t && lane < kMuonGroup)) - 1;
}

__device__ __forceinline__ float muon_momentum(float mu, float m, float g) { return fmaf(mu, m, g); }
__device__ __forceinline__ float muon_update(const MuonArgs& p, bool has, float g, float m) {
  return !has ? g : p.nesterov ? fmaf(p.mu, m, g) : m;
}

// New momentum and the sum of squares of u, in fp64 and a fixed order.  Bound by
// HBM: 202 million bf16 gradients with momentum 382 us, 2.0 GB, 5.3 TB/s; six of
// 2600 x 650 fp32 31 us, 122 MB, 3.9 TB/s.
__global__ __launch_bounds__(256) void k_muon_norm(MuonArgs p) {
  const int i = muon_find(p.table->first[kNorm], blockIdx.x);
  const int sum0 = p.table->first[kNorm][i], nsums = p.table->chunks[kNorm][i];
  const MuonMat t = p.table->mat[i];
  const int64_t n = (int64_t)t.r * t.c;
  const bool has = t.mom != nullptr;
  const bool wide = (t.ldg == t.c || t.r == 1) && aligned4(t.grad, t.gdt) && (!has || aligned4(t.mom, kF32));
  double s = 0.0;
  for (int64_t e0 = (int64_t)(blockIdx.x - sum0) * kSumChunk; e0 < n; e0 += (int64_t)nsums * kSumChunk) {
    if (wide && e0 + kSumChunk <= n) {
      float4 g[4], m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) g[k] = muon_load4(t.grad, t.gdt, e0 + (k * 256 + threadIdx.x) * 4);
      if (has) {
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = *reinterpret_cast<const float4*>(t.mom + e0 + (k * 256 + threadIdx.x) * 4);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float gv[4] = {g[k].x, g[k].y, g[k].z, g[k].w}, mv[4] = {m[k].x, m[k].y, m[k].z, m[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (has) mv[e] = muon_momentum(p.mu, mv[e], gv[e]);
          const double u = muon_update(p, has, gv[e], mv[e]);
          s = fma(u, u, s);
        }
        if (has)
          *reinterpret_cast<float4*>(t.mom + e0 + (k * 256 + threadIdx.x) * 4) = make_float4(mv[0], mv[1], mv[2], mv[3]);
      }
    } else {
      const int64_t end = min(n, e0 + kSumChunk);
      for (int64_t e = e0 + threadIdx.x; e < end; e += 256) {
        const float g = muon_load(t.grad, t.gdt, e / t.c * t.ldg + e % t.c);
        float m = 0.f;
        if (has) t.mom[e] = m = muon_momentum(p.mu, t.mom[e], g);
        const double u = muon_update(p, has, g, m);
        s = fma(u, u, s);
      }
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  __shared__ double part[4];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) p.sums[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

__device__ __forceinline__ void muon_pieces(const float (&v)[8], uint4* hi, uint4* lo) {
  uint16_t h[8], l[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h[e] = Elem<kF16>::down(v[e]);
    const float r = v[e] - Elem<kF16>::up(h[e]);
    l[e] = Elem<kF16>::down(r == r ? r : 0.f);  // (infinite and NaN values stay so in the upper piece)
  }
  __builtin_memcpy(hi, h, sizeof h);
  __builtin_memcpy(lo, l, sizeof l);
}

// The first X, zeros behind a row's end: eight values a thread at a time.  Bound
// by HBM: 202 million values 390 us, 2.0 GB, 5.2 TB/s.
//
// Rounds of 2048 values of a workgroup of the first X and of new weights.  Each adds
// up the matrix's sums of squares: where they are many, four rounds share that (a
// 4096 x 4096 matrix 21 us, with one round 28), else more workgroups are worth more
// (six of 2600 x 650 30 us, with four rounds 34).
__host__ __device__ constexpr int muon_rounds(int64_t sums) { return sums >= 1024 ? 4 : 1; }
__global__ __launch_bounds__(256) void k_muon_start(MuonArgs p) {
  const int i = muon_find(p.table->first[kStart], blockIdx.x);
  const int sum0 = p.table->first[kNorm][i], nsums = p.table->chunks[kNorm][i];
  const MuonMat t = p.table->mat[i];
  __shared__ double part[4];
  {
    double s = 0.0;
    for (int k = threadIdx.x; k < nsums; k += 256) s += p.sums[sum0 + k];
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  }
  __syncthreads();
  const double norm = sqrt(part[0] + part[1] + part[2] + part[3]);
  // (a double: 1 over the norm of tiny gradients is no fp32 number)
  const double under = norm + (double)p.eps, inv = under == 0.0 ? 0.0 : (double)p.sx / under;  // (0 stays 0 without eps)
  const int64_t ld = muon_ld(t.c), per = ld / 8;
  const int rounds = muon_rounds(nsums);
  const int64_t first = (int64_t)(blockIdx.x - p.table->first[kStart][i]) * (256 * rounds) + threadIdx.x;
  const bool has = t.mom != nullptr;
  const bool whole4 = t.c % 4 == 0 && t.ldg % 4 == 0 && aligned4(t.grad, t.gdt) && (!has || aligned4(t.mom, kF32));
  const bool whole2 = t.c % 2 == 0 && t.ldg % 2 == 0 && aligned2(t.grad, t.gdt) && (!has || aligned2(t.mom, kF32));
#pragma unroll 1
  for (int round = 0; round < rounds; ++round) {
    const int64_t at = first + round * 256;
    if (at >= t.r * per) return;
    const int64_t row = at / per, col = at % per * 8, ge = row * t.ldg + col, me = row * t.c + col;
    float v[8];
    if (whole4 && col + 8 <= t.c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 g = muon_load4(t.grad, t.gdt, ge + 4 * h);
        const float4 m = has ? *reinterpret_cast<const float4*>(t.mom + me + 4 * h) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[4 * h] = muon_update(p, has, g.x, m.x), v[4 * h + 1] = muon_update(p, has, g.y, m.y);
        v[4 * h + 2] = muon_update(p, has, g.z, m.z), v[4 * h + 3] = muon_update(p, has, g.w, m.w);
      }
    } else if (whole2 && col + 8 <= t.c) {
      float2 g[4], m[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        g[h] = muon_load2(t.grad, t.gdt, ge + 2 * h);
        m[h] = has ? *reinterpret_cast<const float2*>(t.mom + me + 2 * h) : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h)
        v[2 * h] = muon_update(p, has, g[h].x, m[h].x), v[2 * h + 1] = muon_update(p, has, g[h].y, m[h].y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = col + e < t.c ? muon_update(p, has, muon_load(t.grad, t.gdt, ge + e), has ? t.mom[me + e] : 0.f) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = col + e < t.c ? (float)((double)v[e] * inv) : 0.f;
    uint4 hi, lo;
    muon_pieces(v, &hi, &lo);
    // (where products take both pieces, they alternate; else the lower ones follow
    // behind a row's upper ones)
    uint16_t* const x = muon_at(p, t.x0) + row * 2 * ld + (t.pieces == 2 ? mma_piece(col) : col);
    *reinterpret_cast<uint4*>(x) = hi;
    *reinterpret_cast<uint4*>(x + (t.pieces == 2 ? kMmaLow : ld)) = lo;
  }
}

// The last X to the caller's tensors where their rows are no whole vectors (else
// the last product does it): two values a thread, pairs where they are aligned to
// one.
template <int DT>
__device__ __forceinline__ void muon_pair(void* p, int64_t i, int n, bool read, float decay, float f, const float* v) {
  using T = typename Elem<DT>::type;
  T* const at = static_cast<T*>(p) + i;
  T w[2] = {0, 0};
  const bool pair = n == 2 && ((uintptr_t)at & (2 * sizeof(T) - 1)) == 0;
  if (read) {
    if (pair) {
      __builtin_memcpy(w, __builtin_assume_aligned(at, 2 * sizeof(T)), sizeof w);
    } else {
      w[0] = at[0];
      w[1] = at[n - 1];
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) w[e] = Elem<DT>::down(read ? fmaf(decay, Elem<DT>::up(w[e]), f * v[e]) : f * v[e]);
  if (pair) {
    __builtin_memcpy(__builtin_assume_aligned(at, 2 * sizeof(T)), w, sizeof w);
  } else {
    at[0] = w[0];
    if (n == 2) at[1] = w[1];
  }
}
__device__ __forceinline__ void muon_pair_any(void* p, int dtype, int64_t i, int n, bool read, float decay, float f,
                                              const float* v) {
  if (dtype == kF32)
    muon_pair<kF32>(p, i, n, read, decay, f, v);
  else if (dtype == kBF16)
    muon_pair<kBF16>(p, i, n, read, decay, f, v);
  else
    muon_pair<kF16>(p, i, n, read, decay, f, v);
}
// New weights and updates from the last X, where rows are no whole vectors (else
// the last product writes them): six of 2600 x 650 fp32 30 us, 122 MB, 4.0 TB/s.
__global__ __launch_bounds__(256) void k_muon_apply(MuonArgs p) {
  const int i = muon_find(p.table->first[kStart], blockIdx.x);
  const MuonMat t = p.table->mat[i];
  const int64_t ld = muon_ld(t.c), per = ld / 2;
  const int rounds = muon_rounds(p.table->chunks[kNorm][i]);
  const int64_t base = (int64_t)(blockIdx.x - p.table->first[kStart][i]) * (1024 * rounds);
  const uint16_t* const x = muon_x(p, t, false);
  const int64_t low = t.pieces == 2 ? kMmaLow : ld;
#pragma unroll 4
  for (int q = 0; q < 4 * rounds; ++q) {
    const int64_t at = base + q * 256 + threadIdx.x, row = at / per, col = at % per * 2;
    if (row >= t.r || col >= t.c) continue;
    const uint16_t* y = x + row * 2 * ld + (t.pieces == 2 ? mma_piece(col) : col);
    const uint32_t hi = *reinterpret_cast<const uint32_t*>(y), lo = *reinterpret_cast<const uint32_t*>(y + low);
    const float v[2] = {(Elem<kF16>::up((uint16_t)hi) + Elem<kF16>::up((uint16_t)lo)) / p.sx,
                        (Elem<kF16>::up((uint16_t)(hi >> 16)) + Elem<kF16>::up((uint16_t)(lo >> 16))) / p.sx};
    const int n = (int)min((int64_t)2, t.c - col);
    if (t.upd) muon_pair_any(t.upd, t.udt, row * t.ldu + col, n, false, 0.f, 1.f, v);
    if (t.param) muon_pair_any(t.param, t.pdt, row * t.ldp + col, n, true, p.decay, -t.step, v);
  }
}

// ------------------------------------------------------- matrices in one piece
// Where every matrix of a call, or of a group, is so small, a workgroup takes one whole: X (the
// shorter side down), A and B in LDS in fp32, products on the fp32 matrix
// instruction.  One launch for everything instead of eighteen: a 64 x 27 matrix 15
// us, 100 by those.  Bound by the chain of the steps' products and barriers.
constexpr int kTinyShort = 64, kTinyLong = 256;
constexpr int kTinyX = kTinyLong + 4, kTinyA = kTinyShort + 4;  // row pitches: 16 rows' values meet in no bank

// Products of 16 x 16 tiles of lists a and b (their rows r0 + 0..15, summed along
// the rows' 4 n values; b_down: b's tile is of columns, summed down them).
template <bool B_DOWN>
__device__ __forceinline__ v4f tiny_tile(const float* a, int pa, const float* b, int pb, int n, int lane) {
  const int r = lane & 15, g = lane >> 4;
  v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < n; ++s)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r * pa + 4 * s + g], B_DOWN ? b[(4 * s + g) * pb + r] : b[r * pb + 4 * s + g],
                                               acc, 0, 0, 0);
  return acc;
}

__global__ __launch_bounds__(512) void k_muon_tiny(MuonTiny p) {
  __shared__ float x[kTinyShort * kTinyX], a[kTinyShort * kTinyA], b[kTinyShort * kTinyA];
  __shared__ double part[8];
  const MuonMat t = p.mat[blockIdx.x];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const bool tall = t.r > t.c, has = t.mom != nullptr;
  const int k = min(t.r, t.c), l = max(t.r, t.c), kt = (k + 15) / 16, lt = (l + 15) / 16, n = t.r * t.c;
  for (int i = threadIdx.x; i < kt * 16 * kTinyX; i += 512) x[i] = 0.f;
  __syncthreads();
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 512) {
    const int row = i / t.c, col = i % t.c;
    const float v = muon_load(t.grad, t.gdt, row * t.ldg + col);
    float m = 0.f;
    if (has) t.mom[i] = m = muon_momentum(p.mu, t.mom[i], v);
    const float u = !has ? v : p.nesterov ? fmaf(p.mu, m, v) : m;
    x[tall ? col * kTinyX + row : row * kTinyX + col] = u;
    s = fma((double)u, (double)u, s);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0) part[wave] = s;
  __syncthreads();
  s = 0.0;
  for (int i = 0; i < 8; ++i) s += part[i];
  const double under = sqrt(s) + (double)p.eps, inv = under == 0.0 ? 0.0 : 1.0 / under;
  for (int i = threadIdx.x; i < kt * 16 * lt * 16; i += 512) {
    float& v = x[i / (lt * 16) * kTinyX + i % (lt * 16)];
    v = (float)((double)v * inv);
  }
  __syncthreads();
  for (int step = 0; step < p.steps; ++step) {
    // (the product's lanes: column r, rows 4 g .. + 3; A and B are symmetric)
    for (int i = wave; i < kt * kt; i += 8) {
      const int m = i / kt * 16, c = i % kt * 16;
      const v4f v = tiny_tile<false>(x + m * kTinyX, kTinyX, x + c * kTinyX, kTinyX, lt * 4, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) a[(m + 4 * g + e) * kTinyA + c + r] = v[e];
    }
    __syncthreads();
    for (int i = wave; i < kt * kt; i += 8) {
      const int m = i / kt * 16, c = i % kt * 16;
      const v4f v = tiny_tile<false>(a + m * kTinyA, kTinyA, a + c * kTinyA, kTinyA, kt * 4, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = (m + 4 * g + e) * kTinyA + c + r;
        b[at] = fmaf(p.c, v[e], p.b * a[at]);
      }
    }
    __syncthreads();
    constexpr int MOST = (kTinyShort / 16) * (kTinyLong / 16) / 8;
    v4f next[MOST];
#pragma unroll
    for (int q = 0; q < MOST; ++q) {
      const int i = wave + 8 * q, m = i / lt * 16, c = i % lt * 16;
      if (i >= kt * lt) continue;
      next[q] = tiny_tile<true>(b + m * kTinyA, kTinyA, x + c, kTinyX, kt * 4, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) next[q][e] = fmaf(p.a, x[(m + 4 * g + e) * kTinyX + c + r], next[q][e]);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < MOST; ++q) {
      const int i = wave + 8 * q, m = i / lt * 16, c = i % lt * 16;
      if (i >= kt * lt) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[(m + 4 * g + e) * kTinyX + c + r] = next[q][e];
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += 512) {
    const int row = i / t.c, col = i % t.c;
    const float v = x[tall ? col * kTinyX + row : row * kTinyX + col];
    if (t.upd) muon_save(t.upd, t.udt, row * t.ldu + col, v);
    if (t.param) {
      const int64_t at = row * t.ldp + col;
      muon_save(t.param, t.pdt, at, fmaf(p.decay, muon_load(t.param, t.pdt, at), -t.step * v));
    }
  }
}

// ---------------------------------------------------------------- products
// Tile t of those on and above the diagonal of n x n: groups of 8 tile rows,
// column by column, so that neighbours share their operands in L2.
__device__ __forceinline__ void muon_sym_tile(int t, int n, int* tm, int* tn) {
  for (int g = 0;; g += 8) {
    const int h = min(8, n - g), cols = n - g;  // the diagonal crosses the first h columns
    int c = 0;
    for (; c < h && t >= c + 1; ++c) t -= c + 1;
    if (c < h) {
      *tm = g + t;
      *tn = g + c;
      return;
    }
    if (t < h * (cols - h)) {
      *tm = g + t % h;
      *tn = g + h + t / h;
      return;
    }
    t -= h * (cols - h);
  }
}

__device__ __forceinline__ void muon_add(float (&v)[8], float f, uint4 q) {  // v += f * eight halves
  uint16_t h[8];
  __builtin_memcpy(h, &q, sizeof h);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fmaf(f, Elem<kF16>::up(h[e]), v[e]);
}

// w <- decay w + f v for eight values of a type (w0; of fp32, w0 and w1).
__device__ __forceinline__ void muon_eight(int dtype, float decay, float f, const float (&v)[8], uint4& w0, uint4& w1) {
  if (dtype == kF32) {
    float a[4], b[4];
    __builtin_memcpy(a, &w0, sizeof a);
    __builtin_memcpy(b, &w1, sizeof b);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = fmaf(decay, a[e], f * v[e]), b[e] = fmaf(decay, b[e], f * v[4 + e]);
    __builtin_memcpy(&w0, a, sizeof a);
    __builtin_memcpy(&w1, b, sizeof b);
  } else {
    uint16_t h[8];
    __builtin_memcpy(h, &w0, sizeof h);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float n = fmaf(decay, dtype == kBF16 ? Elem<kBF16>::up(h[e]) : Elem<kF16>::up(h[e]), f * v[e]);
      h[e] = dtype == kBF16 ? Elem<kBF16>::down(n) : Elem<kF16>::down(n);
    }
    __builtin_memcpy(&w0, h, sizeof h);
  }
}

// Results of 32 rows of one wavefront's columns from their sums, through LDS of
// its own: eight neighbouring columns a lane, and, across the diagonal, 32
// neighbouring rows.  What they are added to (A, or X) is asked for a piece
// ahead.
template <int OP, bool PAIR, int HB>
struct MuonResults {
  static constexpr int COLS = HB * 16, PITCH = COLS + 4, LPR = COLS / 8, RPI = 64 / LPR, Q = 32 / RPI;
  static constexpr bool SYM = OP == kGram || OP == kPoly;
  static_assert(COLS == 64, "a column a lane");
  const MuonArgs& p;
  const MuonMat& t;
  int lane;
  bool mirror;
  int64_t k, rows, ld, pitch, low;  // (zeros behind a row's end as well)
  static constexpr bool TWO = !SYM || PAIR;
  __device__ __forceinline__ static int64_t place(int64_t c) { return PAIR ? mma_piece(c) : c; }
  struct Old {
    uint4 hi[Q], lo[Q];
  };

  __device__ __forceinline__ MuonResults(const MuonArgs& args, const MuonMat& mat, bool across)
      : p(args), t(mat), lane(threadIdx.x & 63), mirror(SYM && across), k(min(mat.r, mat.c)) {
    rows = SYM ? k : mat.r;
    ld = muon_ld(SYM ? k : mat.c);
    pitch = TWO ? 2 * ld : ld;
    low = PAIR ? kMmaLow : ld;
  }
  __device__ __forceinline__ void ask(int64_t row0, int64_t col0, Old& o) const {
    if constexpr (OP != kGram) {
      const uint16_t* at = (OP == kPoly ? muon_at(p, t.a) : muon_x(p, t, false)) +
                           place(min(col0 + lane % LPR * 8, ld - 8));
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const uint16_t* x = at + min(row0 + q * RPI + lane / LPR, rows - 1) * pitch;
        o.hi[q] = *reinterpret_cast<const uint4*>(x);
        if (TWO) o.lo[q] = *reinterpret_cast<const uint4*>(x + low);
      }
    }
  }
  __device__ __forceinline__ static void meet() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __device__ __forceinline__ void put(float* lds, int64_t row0, int64_t col0, const v4f (&acc)[2][HB],
                                      const Old& o) const {
    if (row0 >= rows || col0 >= ld) return;
    const int64_t col = col0 + lane % LPR * 8;
    float* const wr = lds + (lane & 15) * PITCH + (lane >> 4) * 4;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int j = 0; j < HB; ++j) *reinterpret_cast<v4f*>(wr + q * 16 * PITCH + j * 16) = acc[q][j];
    meet();
    const float f = OP == kGram ? p.sa / (p.sx * p.sx) : OP == kPoly ? p.c * (p.sb / (p.sa * p.sa))
                                                       : OP == kUpdate ? 1.f / p.sb : 1.f / (p.sb * p.sx);
    const float g = OP == kPoly ? p.b * (p.sb / p.sa) : OP == kUpdate ? p.own : p.own / p.sx;
    const bool diagonal = OP == kPoly && p.rest != 0.f && row0 < col0 + COLS && col0 < row0 + 32;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int in = q * RPI + lane / LPR;
      const int64_t row = row0 + in;
      float* const at = lds + in * PITCH + lane % LPR * 8;
      float v[8];
      __builtin_memcpy(v, __builtin_assume_aligned(at, 16), sizeof v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= f;
      if constexpr (OP != kGram) {
        muon_add(v, g, o.hi[q]);
        if (TWO) muon_add(v, g, o.lo[q]);
      }
      if (diagonal) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += row == col + e && row < k ? p.rest * p.sb : 0.f;
      }
      if (OP == kLast || mirror) __builtin_memcpy(__builtin_assume_aligned(at, 16), v, sizeof v);
      if constexpr (OP != kLast) {
        if (row < rows && col < ld) {
          uint16_t* out = (OP == kUpdate ? muon_x(p, t, true) : muon_at(p, OP == kGram ? t.a : t.b)) + row * pitch + place(col);
          uint4 h, l;
          muon_pieces(v, &h, &l);
          *reinterpret_cast<uint4*>(out) = h;
          if (TWO) *reinterpret_cast<uint4*>(out + low) = l;
        }
      }
    }
    meet();
    if constexpr (OP == kLast) {  // (only where the caller's rows are whole vectors)
      const bool there = col < t.c;
      if (t.param) {
        const int64_t eb = dtype_bytes(t.pdt);
        uint8_t* const at = static_cast<uint8_t*>(t.param) + min(col, (int64_t)t.c - 8) * eb;
        uint4 w[2 * Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const uint8_t* x = at + min(row0 + q * RPI + lane / LPR, rows - 1) * t.ldp * eb;
          w[2 * q] = *reinterpret_cast<const uint4*>(x);
          if (eb == 4) w[2 * q + 1] = *reinterpret_cast<const uint4*>(x + 16);
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int64_t row = row0 + q * RPI + lane / LPR;
          float v[8];
          __builtin_memcpy(v, __builtin_assume_aligned(lds + (q * RPI + lane / LPR) * PITCH + lane % LPR * 8, 16), sizeof v);
          muon_eight(t.pdt, p.decay, -t.step, v, w[2 * q], w[2 * q + 1]);
          if (row >= rows || !there) continue;
          uint8_t* out = at + row * t.ldp * eb;
          *reinterpret_cast<uint4*>(out) = w[2 * q];
          if (eb == 4) *reinterpret_cast<uint4*>(out + 16) = w[2 * q + 1];
        }
      }
      if (t.upd) {
        const int64_t eb = dtype_bytes(t.udt);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int64_t row = row0 + q * RPI + lane / LPR;
          float v[8];
          uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
          __builtin_memcpy(v, __builtin_assume_aligned(lds + (q * RPI + lane / LPR) * PITCH + lane % LPR * 8, 16), sizeof v);
          muon_eight(t.udt, 0.f, 1.f, v, w0, w1);
          if (row >= rows || !there) continue;
          uint8_t* out = static_cast<uint8_t*>(t.upd) + (row * t.ldu + col) * eb;
          *reinterpret_cast<uint4*>(out) = w0;
          if (eb == 4) *reinterpret_cast<uint4*>(out + 16) = w1;
        }
      }
      meet();
    }
    if (mirror) {
      const int64_t mrow = col0 + lane;
      if (mrow < k) {
        uint16_t* const out = muon_at(p, OP == kGram ? t.a : t.b) + mrow * pitch;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = row0 + q * 8 + e < k ? lds[(q * 8 + e) * PITCH + lane] : 0.f;
          uint4 h, l;
          muon_pieces(v, &h, &l);
          *reinterpret_cast<uint4*>(out + place(row0 + q * 8)) = h;
          if (TWO) *reinterpret_cast<uint4*>(out + place(row0 + q * 8) + low) = l;
        }
      }
      meet();
    }
  }
};

struct MuonTile {
  int tm, tn;
};
template <int OP, int BM, int BN>
__device__ __forceinline__ MuonTile muon_tile(const MuonMat& t, int at) {  // tile `at` of the matrix
  MuonTile r;
  if constexpr (OP == kUpdate || OP == kLast) {
    const int ntm = (t.r + BM - 1) / BM, ntn = (t.c + BN - 1) / BN;
    const int first = at / (8 * ntn) * 8, rows = min(8, ntm - first), in = at % (8 * ntn);
    r.tm = first + in % rows;
    r.tn = in / rows;
  } else {
    muon_sym_tile(at, (min(t.r, t.c) + BM - 1) / BM, &r.tm, &r.tn);
  }
  return r;
}

// First chunk of a share.
__device__ __forceinline__ int muon_share(const MuonShares& s, int w) {
  return s.chunk0 + (int)((int64_t)s.chunks * w / s.shares);
}

// One of a step's three products over all matrices of a group.  The matrix cores
// bound it where there are rounds of tiles: a 7B-shaped layer's seven matrices, bf16,
// 784 + 474 + 1503 us for A, B and X, cores 55 - 57 % busy.  The rest goes to X's
// tiles: their old pieces are read and the new ones written (4 + 4 bytes a value, 25 -
// 30 us for a round of 256 tiles) after the sums, on a compute unit that holds one
// workgroup, so nothing runs under them.  4096 x 4096: 100 + 101 + 126 us, 136
// tiles, then 256, one round each.  Small matrices are start, end and latency: six of
// 2600 x 650 fp32 40 + 23 + 59 us, and A^2's 21 chunks a tile are 7 us of products; tiles of
// 64 x 64, where all fit one round, shorten that (27 us in tiles of 128 x 128; over
// ResNet18's convolutions 15 for 21).  (With the loads of two chunks under way, three
// stages and one workgroup a compute unit, tiles of 128 x 128 took 41 + 24 us.)
template <int OP, bool PAIR, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_muon_product(MuonArgs p) {
  using Wide = MmaTile<kF16, PAIR, true, OP == kGram || OP == kPoly, WM, WN, TM, TN>;
  using Tall = MmaTile<kF16, PAIR, OP != kGram, OP != kGram, WM, WN, TM, TN>;
  constexpr int HA = Wide::HA, HB = Wide::HB, BM = Wide::BM, BN = Wide::BN;
  __shared__ __align__(16) uint8_t a0[BM * kMmaBytes], b0[BN * kMmaBytes], a1[BM * kMmaBytes], b1[BN * kMmaBytes];
  constexpr bool kOwn = TM * TN == 2;  // (a stage is too small for results)
  __shared__ __align__(16) float own[kOwn ? WM * WN * 32 * 68 : 4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  constexpr int KIND = OP == kLast ? kUpdate : OP;
  const MuonTable& tab = *p.table;
  // Whole tiles in blocks of 32 to an XCD (workgroups go to the eight XCDs in
  // turn), shares in eighths; a share's chunks are those of tiles in a row.
  int b = blockIdx.x, c, end;
  const bool share = b >= p.sh.whole;
  if (!share) {
    const int x = b % 8, j = b / 8;
    if (b < p.sh.whole / 256 * 256) b = (j / 32 * 8 + x) * 32 + j % 32;
    const int i = muon_find(tab.first[KIND], b), n = tab.chunks[KIND][i];
    c = tab.chunk0[KIND][i] + (b - tab.first[KIND][i]) * n;
    end = c + n;
  } else {
    b = xcd_position(b - p.sh.whole, p.sh.shares);
    c = muon_share(p.sh, b);
    end = muon_share(p.sh, b + 1);
  }
  for (int slot = 0; c < end; slot = 1) {
    const int i = muon_find(tab.chunk0[KIND], c), chunk0 = tab.chunk0[KIND][i], chunks = tab.chunks[KIND][i];
    const MuonMat t = tab.mat[i];
    const int c0 = (c - chunk0) % chunks, c1 = min(chunks, c0 + end - c);
    const MuonTile at = muon_tile<OP, BM, BN>(t, (c - chunk0) / chunks);
    const int64_t m0 = (int64_t)at.tm * BM, n0 = (int64_t)at.tn * BN;
    const int64_t k = min(t.r, t.c), ldk = muon_ld(k), ld = muon_ld(t.c);
    const bool tall = t.r > t.c;
    const MmaSide x{muon_x(p, t, false), 2 * ld, OP == kGram ? k : tall ? t.r : t.c};
    const MmaSide s{muon_at(p, OP == kPoly ? t.a : t.b), PAIR ? 2 * ldk : ldk, k};
    const int64_t sum = OP == kGram ? max(t.r, t.c) : k;
    typename Wide::Acc acc;
    if constexpr (OP == kPoly) {
      Wide::run(s, s, sum, c0, c1, m0, n0, a0, b0, a1, b1, acc);
    } else {
      if (tall)
        Tall::run(x, OP == kGram ? x : s, sum, c0, c1, m0, n0, a0, b0, a1, b1, acc);
      else
        Wide::run(OP == kGram ? x : s, x, sum, c0, c1, m0, n0, a0, b0, a1, b1, acc);
    }
    if (c1 - c0 == chunks) {
      float* lds;
      if constexpr (kOwn)
        lds = own + wave * (32 * 68);
      else
        lds = mma_epilogue_lds<Wide>(wave, a0, b0, a1, b1);
      const MuonResults<OP, PAIR, HB> res(p, t, at.tn != at.tm);
      const int64_t row0 = m0 + wave / WN * TM * 32, col0 = n0 + wave % WN * TN * 32;
      typename MuonResults<OP, PAIR, HB>::Old old[2];
      res.ask(row0, col0, old[0]);
#pragma unroll
      for (int h = 0; h < HA / 2; ++h) {
        v4f piece[2][HB];
#pragma unroll
        for (int j = 0; j < HB; ++j) piece[0][j] = acc[2 * h][j], piece[1][j] = acc[2 * h + 1][j];
        if (h + 1 < HA / 2) res.ask(row0 + (h + 1) * 32, col0, old[(h + 1) & 1]);
        res.put(lds, row0 + h * 32, col0, piece, old[h & 1]);
      }
    } else {
      v4f* const part = reinterpret_cast<v4f*>(p.parts) + (int64_t)(2 * b + slot) * (BM * BN / 4) +
                        wave * (HA * HB * 64) + lane;
#pragma unroll
      for (int h = 0; h < HA * HB; ++h) part[h * 64] = acc[h / HB][h % HB];
    }
    c += c1 - c0;
    if (share) __syncthreads();  // (the next tile's loads go where results passed)
  }
}

// Tiles of several shares: their sums added in order.  One wavefront takes 32
// rows of what one wavefront of the product had.  A launch and a chain of loads: 12 -
// 15 us.  A of six 2600 x 650 matrices takes 39 + 12 us so; its 126 tiles of 82 chunks
// as a workgroup each, on half of the compute units, come to 74 by the costs below.
template <int OP, bool PAIR, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(64) void k_muon_join(MuonArgs p) {
  constexpr int HB = 2 * TN, HA = 2 * TM, BM = WM * TM * 32, BN = WN * TN * 32, PIECES = WM * WN * TM;
  __shared__ __align__(16) float lds[32 * (HB * 16 + 4)];
  constexpr int KIND = OP == kLast ? kUpdate : OP;
  const MuonTable& tab = *p.table;
  const int tile = p.sh.whole + blockIdx.x / PIECES, wave = blockIdx.x % PIECES / TM, h = blockIdx.x % TM;
  const int mat = muon_find(tab.first[KIND], tile), in = tile - tab.first[KIND][mat], chunks = tab.chunks[KIND][mat];
  const MuonMat t = tab.mat[mat];
  const MuonTile at = muon_tile<OP, BM, BN>(t, in);
  const int c0 = tab.chunk0[KIND][mat] + in * chunks, c1 = c0 + chunks;
  int w = (int)((int64_t)(c0 - p.sh.chunk0) * p.sh.shares / p.sh.chunks);  // (rounded down, so it may be one share early)
  while (w + 1 < p.sh.shares && muon_share(p.sh, w + 1) <= c0) ++w;
  if (muon_share(p.sh, w + 1) >= c1) return;  // one share did it all
  const MuonResults<OP, PAIR, HB> res(p, t, at.tn != at.tm);
  const int64_t row0 = (int64_t)at.tm * BM + wave / WN * TM * 32 + h * 32, col0 = (int64_t)at.tn * BN + wave % WN * TN * 32;
  typename MuonResults<OP, PAIR, HB>::Old old;
  res.ask(row0, col0, old);
  v4f acc[2][HB];
#pragma unroll
  for (int i = 0; i < 2 * HB; ++i) acc[i / HB][i % HB] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int c = c0; c < c1; ++w) {
    const int slot = c == muon_share(p.sh, w) ? 0 : 1;
    const v4f* part = reinterpret_cast<const v4f*>(p.parts) + (int64_t)(2 * w + slot) * (BM * BN / 4) +
                      wave * (HA * HB * 64) + h * 2 * HB * 64 + (threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < 2 * HB; ++i) acc[i / HB][i % HB] += part[i * 64];
    c = muon_share(p.sh, w + 1);
  }
  res.put(lds, row0, col0, acc, old);
}

// ---------------------------------------------------------------- the host
static int64_t cdiv(int64_t v, int64_t by) { return (v + by - 1) / by; }
static size_t up256(size_t b) { return (b + 255) / 256 * 256; }

bool muon_scales(const MuonOpts& o, float* sx, float* sa, float* sb) {
  // The largest singular value after each step, and of B, from the largest
  // before it: the polynomials on a grid, with a little room for rounding.
  double top = 1.0, xmax = 1.0, bmax = 0.0;
  for (int s = 0; s < o.steps; ++s) {
    double next = 0.0;
    const double rest = muon_late(o, s) ? -(double)o.b - o.c : 0.0;
    for (int i = 0; i <= 512; ++i) {
      const double x = top * i / 512.0, y = x * x, q = (o.b + o.c * y) * y;
      next = std::max(next, std::abs(x * (o.a + q)));
      bmax = std::max(bmax, std::abs(q + rest));
    }
    top = next * 1.02 + 1e-3;
    if (!(top < 16.0) || !(bmax < 4096.0)) return false;
    xmax = std::max(xmax, top);
  }
  auto fit = [](double m) { return std::ldexp(1.0f, 14 - (int)std::ceil(std::log2(std::max(m, 1e-3)))); };
  *sx = fit(xmax);
  *sa = fit(xmax * xmax);
  *sb = fit(bmax);
  return true;
}

// A group: matrices that a launch takes together.  One that would hold more than
// this many values ends (the workspace holds one group's X, A and B at a time).
constexpr int64_t kGroupValues = int64_t(1) << 28;

// The tiles that a launch may be made of, and what they cost as measured
// (us): a chunk of a tile on a card full of such tiles, and what a tile takes
// besides (first loads, results: of A and B, of X).  The small ones are for one round
// of a few.
struct MuonShape {
  int bm, bn, slots;  // slots: workgroups that the card holds
  double chunk, tile, update;
  double lone;  // a chunk where a compute unit has one such tile only
};
constexpr MuonShape kShapes[] = {{256, 256, 256, 1.40, 10.0, 30.0, 1.40},
                                 {128, 128, 512, 1.02, 8.0, 14.0, 0.80},
                                 {64, 64, 768, 0.42, 6.0, 9.0, 0.38}};
constexpr double kJoin = 10.0;  // a joining launch
// Bytes that parts move in a us: as many as the last level of cache keeps beside the
// operands, or more.
constexpr double kPartsKept = 64.0e6, kKeptRate = 12.0e6, kPartsRate = 4.0e6;

struct MuonLaunch {
  int shape;
  MuonShares sh;
};
struct MuonGroup {
  int first, n, pieces;
  std::vector<int> order;  // longest sums first
  MuonLaunch gram, poly, full;
  size_t sums_off, parts_off, mats_off, bytes;
};

static int64_t norm_groups(const MuonTensor& t) { return std::min<int64_t>(kSumGroups, cdiv(t.r * t.c, kSumChunk)); }
static int64_t start_groups(const MuonTensor& t) { return cdiv(t.r * (muon_ld(t.c) / 8), 256 * muon_rounds(norm_groups(t))); }
static int64_t op_tiles(const MuonTensor& t, int op, const MuonShape& s) {
  if (op == kUpdate) return cdiv(t.r, s.bm) * cdiv(t.c, s.bn);
  const int64_t m = cdiv(std::min(t.r, t.c), s.bm);
  return m * (m + 1) / 2;  // on and above the diagonal
}
static int64_t op_chunks(const MuonTensor& t, int op) {
  return cdiv(op == kGram ? std::max(t.r, t.c) : std::min(t.r, t.c), t.pieces == 2 ? kMmaK<true> : kMmaK<false>);
}

// The shape and the division that take least time by those figures.
static MuonLaunch plan_launch(const std::vector<MuonTensor>& t, const MuonGroup& g, int op) {
  MuonLaunch best{};
  double least = 0.0;
  const double per = g.pieces == 2 ? 1.5 : 1.0;  // (three products of 32 for two of 64)
  for (int shape = 0; shape < 3; ++shape) {
    const MuonShape& s = kShapes[shape];
    const double tile = op == kUpdate ? s.update : s.tile;
    int64_t tiles = 0, chunks = 0, longest = 0;
    for (int i : g.order) {
      const int64_t n = op_tiles(t[i], op, s), q = op_chunks(t[i], op);
      tiles += n;
      chunks += n * q;
      longest = std::max(longest, q);
    }
    if (s.bm == 64 && tiles > s.slots) continue;  // (in shares they lost: ResNet18's convolutions' A 48 us for 41)
    auto split = [&](int64_t whole) {  // the first `whole` tiles as they are, the rest shared
      MuonShares h{};
      h.tiles = (int32_t)tiles;
      h.whole = (int32_t)whole;
      int64_t at = 0, c = 0;
      for (int i : g.order) {
        const int64_t n = op_tiles(t[i], op, s), q = op_chunks(t[i], op), in = std::min(n, whole - at);
        c += in * q;
        at += in;
      }
      h.chunk0 = (int32_t)c;
      h.chunks = (int32_t)(chunks - c);
      h.shares = h.chunks ? (int32_t)std::max<int64_t>(1, std::min<int64_t>(s.slots, h.chunks / 6)) : 0;
      return h;
    };
    auto consider = [&](int64_t whole) {
      const MuonShares h = split(whole);
      // (whole tiles: the average load, and at least the longest tile)
      double us = 0.0;
      if (whole) {
        const double rounds = (double)cdiv(whole, s.slots);
        us += std::max((double)h.chunk0 / (double)whole * rounds, (double)longest) * (whole <= 256 ? s.lone : s.chunk) * per +
              rounds * tile;
      }
      if (h.chunks) {
        const double parts = h.shares > 1 ? std::min<double>(2.0 * h.shares, 2.0 * (double)(tiles - whole) + h.shares) : 0.0;
        us += (double)h.chunks / h.shares * s.chunk * per + tile;
        const double bytes = parts * s.bm * s.bn * sizeof(float);
        if (h.shares > 1) us += kJoin + 2.0 * bytes / (bytes <= kPartsKept ? kKeptRate : kPartsRate);
      }
      if (least == 0.0 || us < least) least = us, best = {shape, h};
    };
    consider(tiles);
    if (s.bm > 64 && tiles % s.slots) consider(tiles / s.slots * s.slots);
  }
  return best;
}

static MuonGroup make_group(const std::vector<MuonTensor>& t, int first) {
  MuonGroup g{};
  g.first = first;
  g.pieces = t[(size_t)first].pieces;
  int64_t values = 0, sums = 0;
  size_t mats = 0;
  for (int i = first; i < (int)t.size() && g.n < kMuonGroup; ++i) {
    const int64_t r = t[i].r, c = t[i].c, k = std::min(r, c);
    if (g.n && (values + r * c > kGroupValues || t[i].pieces != g.pieces)) break;
    values += r * c;
    ++g.n;
    g.order.push_back(i);
    sums += norm_groups(t[i]);
    mats += 2 * up256((size_t)r * muon_ld(c) * 4) + 2 * up256((size_t)k * muon_ld(k) * 2 * t[i].pieces);
  }
  std::stable_sort(g.order.begin(), g.order.end(), [&](int x, int y) {
    return std::min(t[x].r, t[x].c) > std::min(t[y].r, t[y].c);
  });
  g.gram = plan_launch(t, g, kGram);
  g.poly = plan_launch(t, g, kPoly);
  g.full = plan_launch(t, g, kUpdate);
  size_t parts = 0;
  for (const MuonLaunch* l : {&g.gram, &g.poly, &g.full})
    parts = std::max(parts, (size_t)2 * l->sh.shares * kShapes[l->shape].bm * kShapes[l->shape].bn * sizeof(float));
  g.sums_off = up256(sizeof(MuonTable));
  g.parts_off = g.sums_off + up256((size_t)sums * sizeof(double));
  g.mats_off = g.parts_off + up256(parts);
  g.bytes = g.mats_off + mats;
  return g;
}

static bool tiny(const MuonTensor& x) {
  return std::min(x.r, x.c) <= kTinyShort && std::max(x.r, x.c) <= kTinyLong;
}
static bool all_tiny(const std::vector<MuonTensor>& t) { return std::all_of(t.begin(), t.end(), tiny); }
static bool all_tiny(const std::vector<MuonTensor>& t, const MuonGroup& g) {
  return std::all_of(g.order.begin(), g.order.end(), [&](int i) { return tiny(t[(size_t)i]); });
}

size_t muon_workspace(const std::vector<MuonTensor>& t) {
  size_t bytes = 256;
  if (all_tiny(t)) return bytes;
  for (int i = 0; i < (int)t.size();) {
    const MuonGroup g = make_group(t, i);
    if (!all_tiny(t, g)) bytes = std::max(bytes, g.bytes);
    i += g.n;
  }
  return bytes;
}

template <int OP, bool PAIR, int WM, int WN, int TM, int TN>
static void product(const MuonArgs& p, hipStream_t s) {
  hipLaunchKernelGGL((k_muon_product<OP, PAIR, WM, WN, TM, TN>), dim3((unsigned)(p.sh.whole + p.sh.shares)),
                     dim3(64 * WM * WN), 0, s, p);
  if constexpr (TM * TN > 2) {
    if (p.sh.shares > 1)
      hipLaunchKernelGGL((k_muon_join<OP, PAIR, WM, WN, TM, TN>), dim3((unsigned)((p.sh.tiles - p.sh.whole) * WM * WN * TM)),
                         dim3(64), 0, s, p);
  }
}
template <int OP, bool PAIR>
static void product_in(const MuonArgs& p, int shape, hipStream_t s) {
  if (shape == 0)
    product<OP, PAIR, 2, 4, 4, 2>(p, s);
  else if (shape == 1)
    product<OP, PAIR, 2, 2, 2, 2>(p, s);
  else
    product<OP, PAIR, 2, 1, 1, 2>(p, s);
}
template <int OP>
static void product_of(MuonArgs& p, const MuonGroup& g, const MuonLaunch& l, hipStream_t s) {
  p.sh = l.sh;
  if (g.pieces == 2)
    product_in<OP, true>(p, l.shape, s);
  else
    product_in<OP, false>(p, l.shape, s);
}

// What a matrix's entry says of the caller's tensors.
static void describe(const MuonTensor& x, MuonMat* q) {
  q->grad = x.grad, q->mom = x.mom, q->param = x.param, q->upd = x.upd;
  q->ldg = x.ldg, q->ldp = x.ldp, q->ldu = x.ldu, q->r = (int32_t)x.r, q->c = (int32_t)x.c, q->step = x.step;
  q->gdt = (uint8_t)x.gdt, q->pdt = (uint8_t)x.pdt, q->udt = (uint8_t)x.udt, q->pieces = (uint8_t)x.pieces;
}

// The caller's rows are whole vectors of eight values throughout a group.
static bool whole_vectors(const std::vector<MuonTensor>& t, const MuonGroup& g) {
  return std::all_of(g.order.begin(), g.order.end(), [&](int i) {
    const MuonTensor& x = t[(size_t)i];
    auto fits = [&](const void* p, int64_t ld) { return !p || (((uintptr_t)p & 15) == 0 && ld % 8 == 0); };
    return x.c % 8 == 0 && fits(x.param, x.ldp) && fits(x.upd, x.ldu);
  });
}

// `n` matrices from `first` on, a workgroup each.
static void launch_tiny(const std::vector<MuonTensor>& t, size_t first, size_t n, const MuonOpts& o, hipStream_t s) {
  MuonTiny p{};
  p.n = (int32_t)n;
  for (int i = 0; i < p.n; ++i) describe(t[first + (size_t)i], &p.mat[i]);
  p.mu = o.mu, p.decay = o.decay, p.a = o.a, p.b = o.b, p.c = o.c, p.eps = o.eps, p.steps = o.steps;
  p.nesterov = o.nesterov;
  hipLaunchKernelGGL(k_muon_tiny, dim3((unsigned)p.n), dim3(512), 0, s, p);
}

hipError_t launch_muon(const std::vector<MuonTensor>& t, const MuonOpts& o, void* workspace, hipStream_t s) {
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  if (all_tiny(t)) {
    for (size_t first = 0; first < t.size(); first += kMuonGroup)
      launch_tiny(t, first, std::min<size_t>(kMuonGroup, t.size() - first), o, s);
    return hipGetLastError();
  }
  for (int first = 0; first < (int)t.size();) {
    const MuonGroup g = make_group(t, first);
    if (all_tiny(t, g)) {
      launch_tiny(t, (size_t)first, (size_t)g.n, o, s);
      first += g.n;
      continue;
    }
    MuonTable* const table = reinterpret_cast<MuonTable*>(ws);
    MuonTable m{};
    for (int k = 0; k < kMuonKinds; ++k)
      for (int i = 0; i < kMuonGroup; ++i) m.first[k][i] = m.chunk0[k][i] = INT32_MAX, m.chunks[k][i] = 1;
    size_t at = g.mats_off / 256;
    auto take = [&](size_t bytes) {
      const size_t was = at;
      at += up256(bytes) / 256;
      return (uint32_t)was;
    };
    int64_t next[kMuonKinds] = {}, chunk[kMuonKinds] = {};
    for (int i = 0; i < g.n; ++i) {
      const MuonTensor& x = t[(size_t)g.order[(size_t)i]];
      const int64_t k = std::min(x.r, x.c);
      const size_t xb = (size_t)x.r * muon_ld(x.c) * 4, kb = (size_t)k * muon_ld(k) * 2 * x.pieces;
      MuonMat& q = m.mat[i];
      describe(x, &q);
      q.x0 = take(xb), q.x1 = take(xb), q.a = take(kb), q.b = take(kb);
      for (int kind = 0; kind < kMuonKinds; ++kind) {
        const MuonLaunch* l = kind == kGram ? &g.gram : kind == kPoly ? &g.poly : &g.full;
        const int64_t n = kind == kNorm ? norm_groups(x) : kind == kStart ? start_groups(x) : op_tiles(x, kind, kShapes[l->shape]);
        const int64_t c = kind == kNorm ? n : kind == kStart ? 1 : op_chunks(x, kind);
        m.first[kind][i] = (int32_t)next[kind];
        m.chunk0[kind][i] = (int32_t)chunk[kind];
        m.chunks[kind][i] = (int32_t)c;
        next[kind] += n;
        chunk[kind] += n * c;
      }
    }
    hipLaunchKernelGGL(k_muon_table, dim3(1), dim3(256), 0, s, m, table);
    MuonArgs p{};
    p.table = table;
    p.ws = ws;
    p.nesterov = o.nesterov, p.mu = o.mu, p.decay = o.decay, p.a = o.a, p.b = o.b, p.c = o.c, p.eps = o.eps;
    muon_scales(o, &p.sx, &p.sa, &p.sb);
    p.sums = reinterpret_cast<double*>(ws + g.sums_off);
    p.parts = reinterpret_cast<float*>(ws + g.parts_off);
    hipLaunchKernelGGL(k_muon_norm, dim3((unsigned)next[kNorm]), dim3(256), 0, s, p);
    hipLaunchKernelGGL(k_muon_start, dim3((unsigned)next[kStart]), dim3(256), 0, s, p);
    for (int step = 0; step < o.steps; ++step) {
      p.own = muon_late(o, step) ? o.a + o.b + o.c : o.a;
      p.rest = o.a - p.own;
      product_of<kGram>(p, g, g.gram, s);
      product_of<kPoly>(p, g, g.poly, s);
      if (step + 1 < o.steps || !whole_vectors(t, g))
        product_of<kUpdate>(p, g, g.full, s);
      else
        product_of<kLast>(p, g, g.full, s);
      p.odd = !p.odd;
    }
    if (!whole_vectors(t, g)) hipLaunchKernelGGL(k_muon_apply, dim3((unsigned)next[kStart]), dim3(256), 0, s, p);
    first += g.n;
  }
  return hipGetLastError();
}

}  // namespace psgd
