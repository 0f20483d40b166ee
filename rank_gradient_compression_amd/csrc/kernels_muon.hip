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
// with fp16 X, 5e-2 with bfloat16, 1.5e-4 so; Gaussian: 1.5e-3).  Other results
// take two pieces of everything, three products for one.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "psgd_mma_device.h"
#include "psgd_muon.h"

namespace psgd {

constexpr int kSumGroups = 256;   // workgroups of one matrix's norm, at most
constexpr int kSumChunk = 8192;   // values of a workgroup at a time

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
__device__ __forceinline__ bool aligned4(const void* p, int dtype) {
  return ((uintptr_t)p & (dtype == kF32 ? 15 : 7)) == 0;
}

// The matrix whose range, from first(mat) on, holds workgroup or tile t.
template <typename F>
__device__ __forceinline__ int muon_find(const MuonArgs& p, int t, F first) {
  int i = 0;
  while (i + 1 < p.n && t >= first(p.mat[i + 1])) ++i;
  return i;
}

__device__ __forceinline__ float muon_momentum(float mu, float m, float g) { return fmaf(mu, m, g); }
__device__ __forceinline__ float muon_update(const MuonArgs& p, bool has, float g, float m) {
  return !has ? g : p.nesterov ? fmaf(p.mu, m, g) : m;
}

// New momentum and the sum of squares of u, in fp64 and a fixed order.
__global__ __launch_bounds__(256) void k_muon_norm(MuonArgs p) {
  const int i = muon_find(p, blockIdx.x, [](const MuonMat& m) { return m.sum0; });
  const MuonMat& t = p.mat[i];
  const int64_t n = (int64_t)t.r * t.c;
  const bool has = t.mom != nullptr;
  const bool wide = (t.ldg == t.c || t.r == 1) && aligned4(t.grad, t.gdt) && (!has || aligned4(t.mom, kF32));
  double s = 0.0;
  for (int64_t e0 = (int64_t)(blockIdx.x - t.sum0) * kSumChunk; e0 < n; e0 += (int64_t)t.nsums * kSumChunk) {
    if (wide && e0 + kSumChunk <= n) {
      float4 g[8], m[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = muon_load4(t.grad, t.gdt, e0 + (k * 256 + threadIdx.x) * 4);
      if (has) {
#pragma unroll
        for (int k = 0; k < 8; ++k) m[k] = *reinterpret_cast<const float4*>(t.mom + e0 + (k * 256 + threadIdx.x) * 4);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
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
__device__ __forceinline__ void muon_add(float (&v)[8], float f, const uint16_t* p) {  // v += f * p[0..7]
  uint16_t h[8];
  __builtin_memcpy(h, __builtin_assume_aligned(p, 16), sizeof h);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fmaf(f, Elem<kF16>::up(h[e]), v[e]);
}

// The first X, zeros behind a row's end: eight values a thread.
__global__ __launch_bounds__(256) void k_muon_start(MuonArgs p) {
  const int i = muon_find(p, blockIdx.x, [](const MuonMat& m) { return m.start0; });
  const MuonMat& t = p.mat[i];
  __shared__ double part[4];
  {
    double s = 0.0;
    for (int k = threadIdx.x; k < t.nsums; k += 256) s += p.sums[t.sum0 + k];
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  }
  __syncthreads();
  const double norm = sqrt(part[0] + part[1] + part[2] + part[3]);
  // (a double: 1 over the norm of tiny gradients is no fp32 number)
  const double inv = (double)p.sx / (norm + (double)p.eps);
  const int64_t ld = muon_ld(t.c), per = ld / 8, at = (int64_t)(blockIdx.x - t.start0) * 256 + threadIdx.x;
  if (at >= t.r * per) return;
  const int64_t row = at / per, col = at % per * 8;
  const bool has = t.mom != nullptr;
  float v[8];
  const int64_t ge = row * t.ldg + col, me = row * t.c + col;
  const bool wide = col + 8 <= t.c && t.c % 4 == 0 && t.ldg % 4 == 0 && aligned4(t.grad, t.gdt) &&
                    (!has || aligned4(t.mom, kF32));
  if (wide) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 g = muon_load4(t.grad, t.gdt, ge + 4 * h);
      const float4 m = has ? *reinterpret_cast<const float4*>(t.mom + me + 4 * h) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[4 * h] = muon_update(p, has, g.x, m.x), v[4 * h + 1] = muon_update(p, has, g.y, m.y);
      v[4 * h + 2] = muon_update(p, has, g.z, m.z), v[4 * h + 3] = muon_update(p, has, g.w, m.w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = col + e < t.c ? muon_update(p, has, muon_load(t.grad, t.gdt, ge + e), has ? t.mom[me + e] : 0.f) : 0.f;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = col + e < t.c ? (float)((double)v[e] * inv) : 0.f;
  uint4 hi, lo;
  muon_pieces(v, &hi, &lo);
  *reinterpret_cast<uint4*>(t.x0 + row * ld + col) = hi;
  *reinterpret_cast<uint4*>(t.x0 + t.r * ld + row * ld + col) = lo;
}

// ---------------------------------------------------------------- products
enum { kGram, kPoly, kUpdate };

// Tile number t of the upper triangle of nt x nt tiles, row by row.
__device__ __forceinline__ void muon_sym_tile(int t, int nt, int* tm, int* tn) {
  int m = 0;
  while (t >= nt - m) t -= nt - m, ++m;
  *tm = m;
  *tn = m + t;
}

// Eight finished values of row `row` from column `col` on.  acc: the product's.
template <int OP>
__device__ __forceinline__ void muon_finish(const MuonArgs& p, const MuonMat& t, int64_t row, int64_t col,
                                            float (&v)[8]) {
  const int64_t k = min(t.r, t.c), ldk = muon_ld(k), ld = muon_ld(t.c);
  if constexpr (OP == kGram) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= p.sa / (p.sx * p.sx);
  } else if constexpr (OP == kPoly) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= p.c * (p.sb / (p.sa * p.sa));
    const float f = p.b * (p.sb / p.sa);
    muon_add(v, f, t.a + row * ldk + col);
    if (t.pieces == 2) muon_add(v, f, t.a + k * ldk + row * ldk + col);
  } else {
    const float s = p.last ? 1.f / p.sx : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= s / p.sb;
    muon_add(v, p.a * s, t.x0 + row * ld + col);
    muon_add(v, p.a * s, t.x0 + t.r * ld + row * ld + col);
  }
  if (OP == kUpdate && p.last) {
    for (int e = 0; e < 8; ++e) {
      if (col + e >= t.c) break;
      if (t.upd) muon_save(t.upd, t.udt, row * t.ldu + col + e, v[e]);
      if (t.param) {
        const int64_t i = row * t.ldp + col + e;
        muon_save(t.param, t.pdt, i, fmaf(p.decay, muon_load(t.param, t.pdt, i), -t.step * v[e]));
      }
    }
    return;
  }
  uint16_t* out = OP == kGram ? t.a + row * ldk + col : OP == kPoly ? t.b + row * ldk + col : t.x1 + row * ld + col;
  uint4 hi, lo;
  muon_pieces(v, &hi, &lo);
  *reinterpret_cast<uint4*>(out) = hi;
  if (OP == kUpdate)
    *reinterpret_cast<uint4*>(out + t.r * ld) = lo;
  else if (t.pieces == 2)
    *reinterpret_cast<uint4*>(out + k * ldk) = lo;
}

// 32 values of column `row` of the tile, that is of row `row` across the
// diagonal, from its column `col` on.
template <int OP>
__device__ __forceinline__ void muon_mirror(const MuonMat& t, int64_t row, int64_t col, const float (&v)[32]) {
  const int64_t k = min(t.r, t.c), ldk = muon_ld(k);
  uint16_t* out = (OP == kGram ? t.a : t.b) + row * ldk + col;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v[q * 8 + e];
    uint4 hi, lo;
    muon_pieces(x, &hi, &lo);
    *reinterpret_cast<uint4*>(out + q * 8) = hi;
    if (t.pieces == 2) *reinterpret_cast<uint4*>(out + k * ldk + q * 8) = lo;
  }
}

// A launch's tiles (blockIdx.x) times the pieces of the summed axis
// (blockIdx.y).  PHASE 0: sums and results; 1: sums of one piece to memory, in
// the lanes' own order; 2: those added in order, and results.
template <int OP, int PHASE, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_muon_product(MuonArgs p) {
  using Wide = MmaTile<kF16, true, OP != kUpdate, WM, WN, TM, TN>;
  using Tall = MmaTile<kF16, OP != kGram, OP != kGram, WM, WN, TM, TN>;
  constexpr int HA = Wide::HA, HB = Wide::HB, BM = Wide::BM, BN = Wide::BN;
  __shared__ __align__(16) uint8_t a0[BM * kMmaBytes], b0[BN * kMmaBytes], a1[BM * kMmaBytes], b1[BN * kMmaBytes];
  const int tile = xcd_position(blockIdx.x, gridDim.x);
  const int i = muon_find(p, tile, [](const MuonMat& m) { return OP == kUpdate ? m.full0 : m.sym0; });
  const MuonMat& t = p.mat[i];
  const int64_t k = min(t.r, t.c), ldk = muon_ld(k), ld = muon_ld(t.c);
  const bool tall = t.r > t.c;
  int tm, tn;
  if constexpr (OP == kUpdate) {
    const int ntm = (t.r + BM - 1) / BM, ntn = (t.c + BN - 1) / BN, at = tile - t.full0;
    const int first = at / (8 * ntn) * 8, rows = min(8, ntm - first), in = at % (8 * ntn);
    tm = first + in % rows;
    tn = in / rows;
  } else {
    muon_sym_tile(tile - t.sym0, (int)((k + BM - 1) / BM), &tm, &tn);
  }
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  typename Wide::Acc acc;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  v4f* const part = reinterpret_cast<v4f*>(p.partial) + (int64_t)tile * (BM * BN / 4) + wave * (HA * HB * 64) + lane;
  const int64_t piece = (int64_t)p.tiles * (BM * BN / 4);
  if constexpr (PHASE < 2) {
    const MmaSide x{t.x0, t.r * ld, ld, OP == kGram ? k : tall ? t.r : t.c};
    const MmaSide s{OP == kPoly ? t.a : t.b, k * ldk, ldk, k};
    const int64_t sum = OP == kGram ? max(t.r, t.c) : k;
    const uint32_t terms = t.pieces == 2 ? 3 : 1, total = (uint32_t)((sum + kMmaK - 1) / kMmaK) * terms;
    const uint32_t c0 = (uint32_t)((uint64_t)total * blockIdx.y / gridDim.y);
    const uint32_t c1 = (uint32_t)((uint64_t)total * (blockIdx.y + 1) / gridDim.y);
    if constexpr (OP == kPoly) {
      Wide::run(s, s, sum, terms, c0, c1, m0, n0, a0, b0, a1, b1, acc);
    } else {
      if (tall)
        Tall::run(x, OP == kGram ? x : s, sum, terms, c0, c1, m0, n0, a0, b0, a1, b1, acc);
      else
        Wide::run(OP == kGram ? x : s, x, sum, terms, c0, c1, m0, n0, a0, b0, a1, b1, acc);
    }
  }
  if constexpr (PHASE == 1) {
#pragma unroll
    for (int h = 0; h < HA * HB; ++h) part[blockIdx.y * piece + h * 64] = acc[h / HB][h % HB];
    return;
  }
  if constexpr (PHASE == 2) {
#pragma unroll
    for (int h = 0; h < HA * HB; ++h) {
      v4f v = part[h * 64];
      for (int q = 1; q < p.splits; ++q) v += part[q * piece + h * 64];
      acc[h / HB][h % HB] = v;
    }
  }
  // Results, 32 rows of the wavefront's at a time, through LDS of its own: eight
  // neighbouring columns a lane, and, across the diagonal, 32 neighbouring rows.
  constexpr int COLS = HB * 16, PITCH = COLS + 4;
  float* const lds = mma_epilogue_lds<Wide>(wave, a0, b0, a1, b1);
  float* const wr = lds + (lane & 15) * PITCH + (lane >> 4) * 4;
  const int64_t row0 = m0 + wave / WN * TM * 32, col0 = n0 + wave % WN * TN * 32;
  const int64_t rows = OP == kUpdate ? t.r : k, cols = OP == kUpdate ? ld : ldk;  // (zeros behind the row's end as well)
  const bool mirror = OP != kUpdate && tm != tn;
#pragma unroll
  for (int h = 0; h < HA / 2; ++h) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int j = 0; j < HB; ++j) *reinterpret_cast<v4f*>(wr + q * 16 * PITCH + j * 16) = acc[h * 2 + q][j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int LPR = COLS / 8, RPI = 64 / LPR;
#pragma unroll 1
    for (int q = 0; q < 32 / RPI; ++q) {
      const int in = q * RPI + lane / LPR;
      const int64_t row = row0 + h * 32 + in, col = col0 + lane % LPR * 8;
      if (row >= rows || col >= cols) continue;
      float* const at = lds + in * PITCH + lane % LPR * 8;
      float v[8];
      __builtin_memcpy(v, __builtin_assume_aligned(at, 16), sizeof v);
      muon_finish<OP>(p, t, row, col, v);
      if (mirror) __builtin_memcpy(__builtin_assume_aligned(at, 16), v, sizeof v);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (mirror) {
      const int64_t row = col0 + lane, col = row0 + h * 32;
      if (row < k && col < ldk) {
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = row0 + h * 32 + e < k ? lds[e * PITCH + lane] : 0.f;
        muon_mirror<OP>(t, row, col, v);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
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
    for (int i = 0; i <= 512; ++i) {
      const double x = top * i / 512.0, y = x * x, q = (o.b + o.c * y) * y;
      next = std::max(next, std::abs(x * (o.a + q)));
      bmax = std::max(bmax, std::abs(q));
    }
    top = next * 1.02 + 1e-3;
    if (!(top < 16.0) || !(bmax < 4096.0)) return false;
    xmax = std::max(xmax, top);
    if (s > 64) break;  // (bounded so far; what a step maps into itself stays there)
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

struct MuonGroup {
  int first, n;
  bool large;               // 256 x 256 tiles
  int64_t sums, starts, sym, full;
  int gram_splits, poly_splits, full_splits;
  size_t sums_off, partial_off, mats_off, bytes;
};

static int64_t sym_tiles(int64_t k, int64_t b) { return cdiv(k, b) * (cdiv(k, b) + 1) / 2; }

// Pieces of the summed axis (of `chunks` chunks in the longest sum) for a
// launch of so few tiles that most compute units would have none.
static int splits_for(int64_t tiles, int64_t chunks, bool large) {
  const int64_t slots = large ? 256 : 512;
  return (int)std::max<int64_t>(1, std::min<int64_t>({slots / tiles, chunks / 8, 16}));
}

static MuonGroup make_group(const std::vector<MuonTensor>& t, int first) {
  MuonGroup g{};
  g.first = first;
  int64_t values = 0, sym256 = 0;
  for (int i = first; i < (int)t.size() && g.n < kMuonGroup; ++i) {
    const int64_t n = t[i].r * t[i].c;
    if (g.n && values + n > kGroupValues) break;
    values += n;
    ++g.n;
    sym256 += sym_tiles(std::min(t[i].r, t[i].c), 256);
  }
  g.large = sym256 >= 128;
  const int64_t b = g.large ? 256 : 128;
  int64_t gram = 0, poly = 0;
  size_t mats = 0;
  for (int i = first; i < first + g.n; ++i) {
    const int64_t r = t[i].r, c = t[i].c, k = std::min(r, c), terms = t[i].pieces == 2 ? 3 : 1;
    g.sums += std::min<int64_t>(kSumGroups, cdiv(r * c, kSumChunk));
    g.starts += cdiv(r * (muon_ld(c) / 8), 256);
    g.sym += sym_tiles(k, b);
    g.full += cdiv(r, b) * cdiv(c, b);
    gram = std::max(gram, cdiv(std::max(r, c), kMmaK) * terms);
    poly = std::max(poly, cdiv(k, kMmaK) * terms);
    mats += 2 * up256((size_t)r * muon_ld(c) * 4) + 2 * up256((size_t)k * muon_ld(k) * 2 * t[i].pieces);
  }
  g.gram_splits = splits_for(g.sym, gram, g.large);
  g.poly_splits = splits_for(g.sym, poly, g.large);
  g.full_splits = splits_for(g.full, poly, g.large);
  const int64_t tiles = std::max({g.gram_splits > 1 ? g.gram_splits * g.sym : 0, g.poly_splits > 1 ? g.poly_splits * g.sym : 0,
                                  g.full_splits > 1 ? g.full_splits * g.full : 0});
  g.sums_off = 0;
  g.partial_off = up256((size_t)g.sums * sizeof(double));
  g.mats_off = g.partial_off + up256((size_t)tiles * b * b * sizeof(float));
  g.bytes = g.mats_off + mats;
  return g;
}

size_t muon_workspace(const std::vector<MuonTensor>& t) {
  size_t bytes = 256;
  for (int i = 0; i < (int)t.size();) {
    const MuonGroup g = make_group(t, i);
    bytes = std::max(bytes, g.bytes);
    i += g.n;
  }
  return bytes;
}

template <int OP, int WM, int WN, int TM, int TN>
static void product(MuonArgs p, int64_t tiles, int splits, hipStream_t s) {
  const dim3 b(64 * WM * WN);
  p.splits = splits;
  p.tiles = (int32_t)tiles;
  if (splits == 1) {
    hipLaunchKernelGGL((k_muon_product<OP, 0, WM, WN, TM, TN>), dim3((unsigned)tiles), b, 0, s, p);
  } else {
    hipLaunchKernelGGL((k_muon_product<OP, 1, WM, WN, TM, TN>), dim3((unsigned)tiles, (unsigned)splits), b, 0, s, p);
    hipLaunchKernelGGL((k_muon_product<OP, 2, WM, WN, TM, TN>), dim3((unsigned)tiles), b, 0, s, p);
  }
}
template <int OP>
static void product_of(const MuonArgs& p, bool large, int64_t tiles, int splits, hipStream_t s) {
  if (large)
    product<OP, 2, 4, 4, 2>(p, tiles, splits, s);
  else
    product<OP, 2, 2, 2, 2>(p, tiles, splits, s);
}

hipError_t launch_muon(const std::vector<MuonTensor>& t, const MuonOpts& o, void* workspace, hipStream_t s) {
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  for (int first = 0; first < (int)t.size();) {
    const MuonGroup g = make_group(t, first);
    MuonArgs p{};
    p.n = g.n;
    p.nesterov = o.nesterov, p.mu = o.mu, p.decay = o.decay, p.a = o.a, p.b = o.b, p.c = o.c, p.eps = o.eps;
    muon_scales(o, &p.sx, &p.sa, &p.sb);
    p.sums = reinterpret_cast<double*>(ws + g.sums_off);
    p.partial = reinterpret_cast<float*>(ws + g.partial_off);
    uint8_t* at = ws + g.mats_off;
    auto take = [&](size_t bytes) {
      uint16_t* const q = reinterpret_cast<uint16_t*>(at);
      at += up256(bytes);
      return q;
    };
    const int64_t b = g.large ? 256 : 128;
    int32_t sum0 = 0, start0 = 0, sym0 = 0, full0 = 0;
    for (int i = 0; i < g.n; ++i) {
      const MuonTensor& x = t[(size_t)(first + i)];
      const int64_t k = std::min(x.r, x.c);
      const size_t xb = (size_t)x.r * muon_ld(x.c) * 4, kb = (size_t)k * muon_ld(k) * 2 * x.pieces;
      MuonMat& m = p.mat[i];
      m.grad = x.grad, m.mom = x.mom, m.param = x.param, m.upd = x.upd;
      m.x0 = take(xb), m.x1 = take(xb), m.a = take(kb), m.b = take(kb);
      m.ldg = x.ldg, m.ldp = x.ldp, m.ldu = x.ldu, m.r = (int32_t)x.r, m.c = (int32_t)x.c, m.step = x.step;
      m.gdt = (uint8_t)x.gdt, m.pdt = (uint8_t)x.pdt, m.udt = (uint8_t)x.udt, m.pieces = (uint8_t)x.pieces;
      m.sum0 = sum0, m.nsums = (int32_t)std::min<int64_t>(kSumGroups, cdiv(x.r * x.c, kSumChunk));
      m.start0 = start0, m.sym0 = sym0, m.full0 = full0;
      sum0 += m.nsums;
      start0 += (int32_t)cdiv(x.r * (muon_ld(x.c) / 8), 256);
      sym0 += (int32_t)sym_tiles(k, b);
      full0 += (int32_t)(cdiv(x.r, b) * cdiv(x.c, b));
    }
    hipLaunchKernelGGL(k_muon_norm, dim3((unsigned)g.sums), dim3(256), 0, s, p);
    hipLaunchKernelGGL(k_muon_start, dim3((unsigned)g.starts), dim3(256), 0, s, p);
    for (int step = 0; step < o.steps; ++step) {
      p.last = step + 1 == o.steps;
      product_of<kGram>(p, g.large, g.sym, g.gram_splits, s);
      product_of<kPoly>(p, g.large, g.sym, g.poly_splits, s);
      product_of<kUpdate>(p, g.large, g.full, g.full_splits, s);
      for (int i = 0; i < g.n; ++i) std::swap(p.mat[i].x0, p.mat[i].x1);
    }
    first += g.n;
  }
  return hipGetLastError();
}

}  // namespace psgd
