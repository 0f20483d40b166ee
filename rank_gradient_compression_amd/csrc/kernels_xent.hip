// Softmax cross entropy over a large vocabulary from hidden states and output
// weights, without keeping the logits, and its gradients (gfx950).
//
//   l = x w^T + b,  lse_t = log sum_v exp l_tv,  loss_t = lse_t - l_{t, y_t}
//   G_tv = u_t (exp(l_tv - lse_t) - [v = y_t])
//   dx = s G w,  dw = s G^T x,  db = s sum_t G_t
//
// The vocabulary is taken in pieces: a tile of the product x w^T ends with its
// rows' maximum m and sum of exp(l - m) over each segment of columns, and the
// logits are gone.  Training keeps E = exp(l - m), at most 1, for a block of tokens
// whatever the batch, from which one pass over the block makes G once the rows' sums
// are known.  That is three products of T x V x D in all; forming the logits again
// for the gradients instead of keeping E would be a fourth (a third more of the
// time), the pass over E and G is 4 bytes a value (4% of it at D = 4096: 0.12 of 2.6
// ms at 4096 x 32000 x 4096 bf16, the products 0.93, 0.83 and 0.89 ms).
//
// Digits.  Sums, maxima and products are fp32.  E is fp32 for fp32 tensors and few
// tokens, else held times 2^15 in fp16: a relative error of 2^-11 down to 2^-29 of its
// segment's largest (20 nats below), 2^-40 of that largest under it, and nothing of
// what is below 2^-40 (28 nats; held as it is, 17).  G is rounded once to the type
// that the products take (of few tokens it has two pieces of it): with more it would
// be a second product for dx and for dw each, and what one leaves is 1.05 to 1.25
// times the gradients' own rounding.  The target's entry, which would cancel, is
// formed from the loss, exp(-loss) - 1.  A row's largest logit M and its S = sum
// exp(l - M) are kept apart for loss = log S - (l_y - M) and p = exp(l - M) / S: lse,
// rounded at its full size, would leave that in both (an entry of -0.0106 was 0.4%
// off with logits around 1000).
//
// Tokens' weights.  A row of G is held times a power of two that brings its own
// weight u_t to 2^13 .. 2^14, so that a token of small weight keeps its digits in
// dx; the copy of x that dw's product takes carries the other powers of two,
// relative to the largest weight's.
//
// fp32 tensors are split into two fp16 pieces (psgd_mma_device.h) under a power of
// two that brings the largest finite value to 2^13 .. 2^14: of its row for x in the
// logits, which take it back row by row, so that no token's digits depend on what
// another one, or a row of padding, holds; of the whole matrix for w, and of all
// rows that count for x in dw, whose sum runs over them.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "psgd_mma_device.h"
#include "psgd_xent.h"

namespace psgd {

// scalars that the device works out for itself
// (kE*: exponents.  A product's factor, scale over the operands' powers of two, may be
// no fp32 number where the result is one: it is kept as kS times 2 to kEdx, kEdw or
// kEdb.)
enum { kSx, kSw, kEw, kEg, kS, kEdx, kEdw, kEdb, kScalars };

constexpr int64_t kFewTokens = 32;  // of few tokens: a stream of the weights, one block
constexpr int kMaxGroups = 1024;    // workgroups that look for a tensor's largest value
constexpr int64_t kBlockBytes = int64_t(1) << 30;  // of E (and G) at a time, or of segments' sums without gradients
constexpr int64_t kBlockTokens = int64_t(1) << 23;  // (a launch holds 2^32 threads)
constexpr int kGradRows = 16;       // tokens of a workgroup of the pass over E, at most
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHeld = 32768.f;  // what E is held times in fp16

__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  if (dtype == kF32) return static_cast<const float*>(p)[i];
  if (dtype == kBF16) return Elem<kBF16>::up(static_cast<const uint16_t*>(p)[i]);
  return Elem<kF16>::up(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float v) {
  if (dtype == kF32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == kBF16)
    static_cast<uint16_t*>(p)[i] = Elem<kBF16>::down(v);
  else
    static_cast<uint16_t*>(p)[i] = Elem<kF16>::down(v);
}
__device__ __forceinline__ bool ignored(int64_t y, int64_t ignore) { return y < 0 || y == ignore; }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// ------------------------------------------------------------ preparations
// 2^e that brings m to 2^13 .. 2^14, e within what fp32 can hold and invert.
__device__ __forceinline__ int fit_exponent(float m) {
  if (!(m > 0.f)) return 0;
  int e;
  (void)frexpf(m, &e);  // m = f 2^e, f in [1/2, 1)
  return min(max(14 - e, -126), 126);
}

// A token that the gradients see.
__device__ __forceinline__ bool counted(const XentArgs& a, int64_t t) {
  const int64_t y = a.targets[t];
  return !ignored(y, a.ignore) && y < a.v && !(a.weights && a.weights[t] == 0.f);
}

// A word that a bias of minus infinity takes out (fp32).
__device__ __forceinline__ bool word_out(const void* bias, int64_t v) {
  return bias && static_cast<const float*>(bias)[v] == -__builtin_inff();
}

// Largest finite magnitude of the rows of w that a bias leaves in and of the rows of
// x that count, one partial maximum per workgroup: the first `kMaxGroups` take x, the
// others w; and the exponent of every row of x.  A row of x is a workgroup's where
// each can have one, else a wavefront's; rows of w without gaps are read as one, with
// the biases of the two rows that four values may lie in.  Bound by HBM's latency and
// reads (33278 x 650: 24 us, 3.7 TB/s; 28 with a bias).
__global__ __launch_bounds__(256) void k_xent_max(XentArgs a, bool train, float* out, int* rows_x) {
  const int b = blockIdx.x % kMaxGroups, wave = threadIdx.x >> 6;
  __shared__ float part[4];
  float m = 0.f;
  auto larger = [](float& to, float v) {
    v = fabsf(v);
    to = v < __builtin_inff() ? fmaxf(to, v) : to;
  };
  auto larger4 = [&](float& to, const float4& v) { larger(to, v.x), larger(to, v.y), larger(to, v.z), larger(to, v.w); };
  if (blockIdx.x < kMaxGroups) {
    const float* p = static_cast<const float*>(a.x);
    const bool whole = a.t <= kMaxGroups, vec = a.d % 4 == 0 && a.ldx % 4 == 0 && ((uintptr_t)p & 15) == 0;
    const int64_t lane = whole ? threadIdx.x : threadIdx.x & 63, lanes = whole ? 256 : 64;
    for (int64_t row = whole ? b : (int64_t)b * 4 + wave; row < a.t; row += whole ? kMaxGroups : kMaxGroups * 4) {
      const float* q = p + row * a.ldx;
      float r = 0.f;
      if (vec) {
#pragma unroll 8
        for (int64_t i = lane; i < a.d / 4; i += lanes) larger4(r, reinterpret_cast<const float4*>(q)[i]);
      } else {
#pragma unroll 8
        for (int64_t i = lane; i < a.d; i += lanes) larger(r, q[i]);
      }
      r = wave_max(r);
      if (whole) {  // (one row at most: the barrier is every thread's)
        if ((threadIdx.x & 63) == 0) part[wave] = r;
        __syncthreads();
        r = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
        __syncthreads();
      }
      if (lane == 0) rows_x[row] = fit_exponent(r);
      if (train && counted(a, row)) m = fmaxf(m, r);
    }
  } else {
    const float* p = static_cast<const float*>(a.w);
    if (a.ldw == a.d && a.d >= 4 && ((uintptr_t)p & 15) == 0) {
      const int64_t n = a.v * a.d, n4 = n / 4, i0 = (int64_t)b * 256 + threadIdx.x;
      const float4* q = reinterpret_cast<const float4*>(p);
      if (a.bias) {
        constexpr int64_t step = kMaxGroups * 256 * 4;
        const int64_t rows = step / a.d, cols = step % a.d;
        int64_t row = i0 * 4 / a.d, col = i0 * 4 % a.d;
#pragma unroll 8
        for (int64_t i = i0; i < n4; i += kMaxGroups * 256) {
          const float4 v = q[i];
          const bool out = word_out(a.bias, row), next = word_out(a.bias, min(row + 1, a.v - 1));
          larger(m, out ? 0.f : v.x), larger(m, (col + 1 < a.d ? out : next) ? 0.f : v.y);
          larger(m, (col + 2 < a.d ? out : next) ? 0.f : v.z), larger(m, (col + 3 < a.d ? out : next) ? 0.f : v.w);
          row += rows, col += cols;
          if (col >= a.d) col -= a.d, ++row;
        }
      } else {
#pragma unroll 8
        for (int64_t i = i0; i < n4; i += kMaxGroups * 256) larger4(m, q[i]);
      }
      if (b == 0 && threadIdx.x < n - n4 * 4 && !word_out(a.bias, a.v - 1)) larger(m, p[n4 * 4 + threadIdx.x]);
    } else {
      for (int64_t row = (int64_t)b * 4 + wave; row < a.v; row += kMaxGroups * 4) {
        if (word_out(a.bias, row)) continue;
        const float* q = p + row * a.ldw;
#pragma unroll 8
        for (int64_t i = threadIdx.x & 63; i < a.d; i += 64) larger(m, q[i]);
      }
    }
  }
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) part[wave] = m;
  __syncthreads();
  if (threadIdx.x == 0) out[blockIdx.x] = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
}

// Exponent of a token's weight; `most` (the largest weight's, the smallest
// exponent) for one that has none.  The two may be 240 apart, so a power of two
// between them is no fp32 number: what goes by both takes the difference.
__device__ __forceinline__ int weight_exponent(float u, int most) {
  u = fabsf(u);
  return u > 0.f && u < __builtin_inff() ? max(fit_exponent(u), most) : most;
}

// The scalars, by one workgroup.
__device__ void xent_scalars(const XentArgs& a, bool train, bool split, const float* partmax, float* sc) {
  float u = 0.f, mx = 0.f, mw = 0.f;
  double n = 0.0;
  if (train)
    for (int64_t t = threadIdx.x; t < a.t; t += 256) {
      if (ignored(a.targets[t], a.ignore)) continue;
      n += 1.0;
      const float v = a.weights ? fabsf(a.weights[t]) : 1.f;
      u = v < __builtin_inff() ? fmaxf(u, v) : u;
    }
  if (split)
    for (int i = threadIdx.x; i < kMaxGroups; i += 256) {
      mx = fmaxf(mx, partmax[i]);
      mw = fmaxf(mw, partmax[kMaxGroups + i]);
    }
  u = wave_max(u), mx = wave_max(mx), mw = wave_max(mw);
#pragma unroll
  for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o);
  __shared__ float pu[4], px[4], pw[4];
  __shared__ double pn[4];
  if ((threadIdx.x & 63) == 0) {
    const int w = threadIdx.x >> 6;
    pu[w] = u, px[w] = mx, pw[w] = mw, pn[w] = n;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 4; ++w) u = fmaxf(u, pu[w]), mx = fmaxf(mx, px[w]), mw = fmaxf(mw, pw[w]), n += pn[w];
  const int ex = split ? fit_exponent(mx) : 0, ew = split ? fit_exponent(mw) : 0, eg = fit_exponent(u);
  const double s = a.mean ? (double)a.scale / fmax(n, 1.0) : (double)a.scale;
  sc[kSx] = ldexpf(1.f, ex);
  sc[kSw] = ldexpf(1.f, ew);
  sc[kEw] = (float)ew;
  int es;
  sc[kS] = (float)frexp(s, &es);
  sc[kEg] = (float)eg;
  sc[kEdx] = (float)(es - eg - ew);
  sc[kEdw] = (float)(es - eg - ex);
  sc[kEdb] = (float)(es - eg);
}

__global__ __launch_bounds__(256) void k_xent_prep(XentArgs a, bool train, bool split, const float* partmax, float* sc) {
  xent_scalars(a, train, split, partmax, sc);
}

// Rows to operands: 16-bit values, or two pieces of fp32 ones, zeros behind the
// row's end.  One thread = 8 values.  fp32 rows of x have a power of two each; those
// of w that a bias takes out are zeros, so that they may hold any finite values.
// clean: a second copy, the one that dw's product takes, under one power of two, with
// rows of tokens that do not count zero (their G is zero, and zero times what such a
// row may hold need not be) and the others times their weight's power of two, whose
// exponent goes to `factors` as well.  Bound by HBM: 33278 x 650 fp16 18 us, 92 MB read
// and written, 5.1 TB/s; fp32 31 us, 176 MB, 5.7 TB/s.
struct XentPack {
  const void* x;
  int64_t ld, rows, d, dp;
  const void* bias;      // of w's rows where they are fp32, or null
  const float* scale;    // of the whole matrix
  const int* exponents;  // of every row in `out`, or null: the matrix's
  uint16_t *out, *clean;
  const int64_t* targets;
  int64_t ignore, v;
  const float* weights;
  const float* sc;
  int* factors;

  XentPack rows_from(int64_t at, int64_t n, int dtype) const {  // `n` of the rows, from `at` on
    XentPack p = *this;
    const int64_t pitch = dp * (dtype == kF32 ? 2 : 1);
    p.x = static_cast<const uint8_t*>(x) + at * ld * dtype_bytes(dtype);
    p.rows = n;
    if (bias) p.bias = static_cast<const float*>(bias) + at;
    if (exponents) p.exponents = exponents + at;
    if (out) p.out = out + at * pitch;
    if (clean) p.clean = clean + at * pitch;
    if (targets) p.targets = targets + at;
    if (weights) p.weights = weights + at;
    if (factors) p.factors = factors + at;
    return p;
  }
};
template <int DT>
__global__ __launch_bounds__(256) void k_xent_pack(XentPack w, XentPack x, unsigned first) {
  using T = typename Elem<DT>::type;
  const bool second = blockIdx.x >= first;
  const XentPack p = second ? x : w;
  const int64_t i = (int64_t)(blockIdx.x - (second ? first : 0)) * 256 + threadIdx.x, per = p.dp / 8;
  if (i >= p.rows * per) return;
  const int64_t row = i / per, c = i % per * 8;
  const T* q = static_cast<const T*>(p.x) + row * p.ld + c;
  T v[8];
  if (c + 8 <= p.d) {
    __builtin_memcpy(v, q, sizeof v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < p.d ? q[e] : (T)0;
  }
  const int64_t at = DT == kF32 ? row * 2 * p.dp + mma_piece(c) : row * p.dp + c;
  auto put = [&](uint16_t* to, float f, float scale) {
    uint16_t hi[8], lo[8];
    if constexpr (DT == kF32) {
      const float s = scale * f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = v[e] * s;
        const _Float16 h = (_Float16)z;
        hi[e] = __builtin_bit_cast(uint16_t, h);
        const float r = z - (float)h;
        lo[e] = Elem<kF16>::down(r == r ? r : 0.f);  // (infinite and NaN values stay so in hi)
      }
    } else {
      __builtin_memcpy(hi, v, sizeof hi);
      if (f != 1.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) hi[e] = Elem<DT>::down(Elem<DT>::up(hi[e]) * f);
      }
    }
    if (f == 0.f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) hi[e] = lo[e] = 0;
    }
    __builtin_memcpy(to + at, hi, sizeof hi);
    if constexpr (DT == kF32) __builtin_memcpy(to + kMmaLow + at, lo, sizeof lo);
  };
  if (p.out) {
    const float scale = DT != kF32 ? 1.f : p.exponents ? ldexpf(1.f, p.exponents[row]) : *p.scale;
    put(p.out, DT == kF32 && word_out(p.bias, row) ? 0.f : 1.f, scale);
  }
  if (!p.factors) return;
  float f = 1.f;
  if (p.weights) {
    const int most = (int)p.sc[kEg], less = most - weight_exponent(p.weights[row], most);
    f = ldexpf(1.f, less);  // (0 where that is no fp32 number: the row vanishes beside the largest weight's)
    if (c == 0) p.factors[row] = less;
    if (p.weights[row] == 0.f) f = 0.f;
  }
  if (!p.clean) return;
  const int64_t y = p.targets[row];
  put(p.clean, ignored(y, p.ignore) || y >= p.v ? 0.f : f, DT != kF32 ? 1.f : *p.scale);
}

// ------------------------------------------------------------------ logits
struct XentTile {
  MmaSide x, w;
  int64_t t, v, d;  // tokens of the block
  const float* sc;
  const int* exponents;  // of the rows of x as pairs
  const void* bias;
  int bias_dtype;
  const int64_t* targets;
  float2* stats;  // t x nseg: maximum and sum
  int64_t nseg;
  float* target;  // t: the target's logit
  void* e;        // t x vp
  int64_t vp;
};

// Exponent that the sums of a row of pairs are to be taken times.
template <bool PAIR>
__device__ __forceinline__ int xent_shift(const XentTile& p, int64_t row) {
  return PAIR && row < p.t ? -(p.exponents[row] + (int)p.sc[kEw]) : 0;
}

// A row's logits of one segment: lane group g has columns col0 + 16 j + 4 g + e.
// They become E, and the segment's maximum and sum are written.
template <bool PAIR, int HB>
__device__ __forceinline__ void xent_row(const XentTile& p, int64_t row, int64_t col0, int g, const v4f (&acc)[HB],
                                         const v4f (&bias)[HB], int shift, int64_t y, float (&ex)[HB * 4]) {
  float l[HB * 4], m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < HB * 4; ++i)
    l[i] = (PAIR ? __builtin_amdgcn_ldexpf(acc[i / 4][i % 4], shift) : acc[i / 4][i % 4]) + bias[i / 4][i % 4];
  if (col0 + HB * 16 > p.v) {
#pragma unroll
    for (int i = 0; i < HB * 4; ++i) l[i] = col0 + i / 4 * 16 + 4 * g + i % 4 < p.v ? l[i] : -__builtin_inff();
  }
#pragma unroll
  for (int i = 0; i < HB * 4; ++i) m = fmaxf(m, l[i]);
  m = groups_max(m);
  const float ref = m == -__builtin_inff() ? 0.f : m;  // (a segment of masked words: sums of zero)
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < HB * 4; ++i) {
    // (the difference first: times log2 e each, m's rounding would be left of a
    // segment of large logits, and a finite mask's is anything, infinity included)
    ex[i] = __builtin_amdgcn_exp2f((l[i] - ref) * kLog2e);
    sum += ex[i];
  }
  sum = groups_sum(sum);
  if (row >= p.t) return;
  if (g == 0) p.stats[row * p.nseg + col0 / (HB * 16)] = make_float2(m, sum);
  const int64_t at = y - col0 - 4 * g;  // the target among this lane's columns
  if (at >= 0 && at < HB * 16 && at % 16 < 4 && y < p.v) {
#pragma unroll
    for (int i = 0; i < HB * 4; ++i)
      if (at == i / 4 * 16 + i % 4) p.target[row] = l[i];
  }
}

__device__ __forceinline__ uint32_t two_halves(float v, float w) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef _Float16 v2h __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{v, w}), v2h));
}

__device__ __forceinline__ uint32_t held_halves(float v, float w) { return two_halves(v * kHeld, w * kHeld); }

template <int HB>
__device__ __forceinline__ void xent_bias(const XentTile& p, int64_t col0, int g, v4f (&bias)[HB]) {
#pragma unroll
  for (int i = 0; i < HB * 4; ++i) {
    const int64_t col = col0 + i / 4 * 16 + 4 * g + i % 4;
    bias[i / 4][i % 4] = p.bias && col < p.v ? load_any(p.bias, p.bias_dtype, col) : 0.f;
  }
}

// x w^T in the tile loop, then every wavefront's segments.  The matrix cores bound
// it, and what power leaves of their clock: 4096 x 32000 x 4096 bf16 0.87 - 0.93 ms,
// 1.15 - 1.24 PFLOP/s, matrix cores 64 % busy (counted), E included; without E and
// with 2048 tokens 0.44 - 0.46 ms.  700 x 33278 x 650 fp32, three products: 114 us, 0.80
// PFLOP/s; 390 tiles on 256 compute units leave a quarter of two rounds idle.
template <int DT, bool PAIR, int KEEP, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_xent_logits(XentTile p, int ntm, int ntn) {
  using Tile = MmaTile<DT, PAIR, true, true, WM, WN, TM, TN>;
  __shared__ __align__(16) uint8_t a0[Tile::BM * kMmaBytes], b0[Tile::BN * kMmaBytes], a1[Tile::BM * kMmaBytes],
      b1[Tile::BN * kMmaBytes];
  int tm, tn;
  mma_tile_of_block(blockIdx.x, ntm, ntn, &tm, &tn);
  typename Tile::Acc acc;
  Tile::run(p.x, p.w, p.d, 0, (uint32_t)((p.d + Tile::K - 1) / Tile::K), (int64_t)tm * Tile::BM, (int64_t)tn * Tile::BN, a0, b0, a1, b1, acc);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t row0 = (int64_t)tm * Tile::BM + wave / WN * TM * 32 + r;
  const int64_t col0 = (int64_t)tn * Tile::BN + wave % WN * TN * 32;
  if (col0 >= p.v) return;
  v4f bias[Tile::HB];
  xent_bias<Tile::HB>(p, col0, g, bias);
  // E goes out in whole rows of the wavefront's 64 columns, 32 rows at a time
  // through LDS of its own (straight from the lanes' four columns it left in
  // 32-byte pieces and took 20 us a round of tiles more).
  constexpr int COLS = Tile::HB * 16, PITCH = COLS * (KEEP == 2 ? 4 : 2) + 16;
  uint8_t* const lds = reinterpret_cast<uint8_t*>(mma_epilogue_lds<Tile>(__builtin_amdgcn_readfirstlane(wave), a0, b0, a1, b1));
  int64_t ys[Tile::HA];
#pragma unroll
  for (int i = 0; i < Tile::HA; ++i) ys[i] = row0 + i * 16 < p.t ? p.targets[row0 + i * 16] : -1;
#pragma unroll
  for (int i = 0; i < Tile::HA; ++i) {
    float ex[Tile::HB * 4];
    xent_row<PAIR, Tile::HB>(p, row0 + i * 16, col0, g, acc[i], bias, xent_shift<PAIR>(p, row0 + i * 16), ys[i], ex);
    if constexpr (KEEP > 0) {
      uint8_t* const wr = lds + (i % 2 * 16 + r) * PITCH + 4 * g * (KEEP == 2 ? 4 : 2);
#pragma unroll
      for (int j = 0; j < Tile::HB; ++j) {
        if constexpr (KEEP == 2)
          *reinterpret_cast<float4*>(wr + j * 64) = make_float4(ex[4 * j], ex[4 * j + 1], ex[4 * j + 2], ex[4 * j + 3]);
        else
          *reinterpret_cast<uint2*>(wr + j * 32) = make_uint2(held_halves(ex[4 * j], ex[4 * j + 1]),
                                                              held_halves(ex[4 * j + 2], ex[4 * j + 3]));
      }
      if (i % 2 == 0) continue;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      constexpr int LPR = KEEP == 2 ? 16 : 8, RPI = 64 / LPR;
      const int64_t first = row0 - r + (i - 1) * 16;
      uint8_t* const out = static_cast<uint8_t*>(p.e) + (first * p.vp + col0) * (KEEP == 2 ? 4 : 2) + lane % LPR * 16;
#pragma unroll
      for (int q = 0; q < 32 / RPI; ++q) {
        const int in = q * RPI + lane / LPR;
        const uint4 x = *reinterpret_cast<const uint4*>(lds + in * PITCH + lane % LPR * 16);
        if (first + in < p.t) *reinterpret_cast<uint4*>(out + in * p.vp * (KEEP == 2 ? 4 : 2)) = x;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// Few tokens: a stream of the weights, and what counts is how many of its bytes
// are under way.  A workgroup takes all tokens (MT * 16) and 32 words; its
// wavefronts take the chunks in turn, each staging its own weights in LDS, two
// chunks ahead, in whole 128-byte rows, and its blocks of x, which every workgroup
// reads from L2, in registers (staged in LDS as well they left room for one
// workgroup to a compute unit: 50 us for the 47 below).  The wavefronts' partial
// tiles are added in their order.  32000 x 4096 bf16 weights (262 MB): 1 token 47 us,
// 5.5 TB/s, 24 tokens 54 - 57; 33278 x 650 from the last level of cache, where the
// copy has just gone: 16 us.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x0f70 | (N >> 4) << 14);
  __builtin_amdgcn_sched_barrier(0);
}

template <int DT, bool PAIR, bool KEEP, int MT, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 1) void k_xent_logits_few(XentTile p) {
  constexpr int HB = 2;
  using LW = MmaLoad<PAIR, true, 32, 1>;
  constexpr int STAGE = LW::kBytes, LOADS = LW::kLoads + 2 * MT, TILES = MT * HB;
  static_assert(TILES * 1024 <= 2 * STAGE, "no room for the partial tiles");
  __shared__ __align__(16) uint8_t st0[WAVES * STAGE], st1[WAVES * STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t col0 = (int64_t)xcd_position(blockIdx.x, gridDim.x) * 32;
  LW lw(p.w, col0, 0, lane);
  const MmaRead<true, 32> rw(0, lane);
  const uint32_t total = (uint32_t)((p.d + LW::K - 1) / LW::K);
  // A lane's blocks of x, as the products take them, two of a chunk for each 16 rows,
  // go to registers; rows past the last and blocks past a row's end read as zero.
  typedef v4u Rows[MT][2];
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(p.x.p), 0, (int)(((p.t - 1) * p.x.ld + (PAIR ? 2 * LW::K * total : (p.d + 7) / 8 * 8)) * 2), 0x00020000);
  uint32_t xo[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xo[i] = i * 16 + r < p.t ? (uint32_t)((i * 16 + r) * p.x.ld * 2) + g * (PAIR ? 16 : 32) : kMmaOff;
  uint8_t *const m0 = st0 + wave * STAGE, *const m1 = st1 + wave * STAGE;
  auto fetch = [&](uint32_t c, uint8_t* m, Rows& x) {
    const uint32_t at = min(c, total - 1), left = c < total ? (uint32_t)p.d - at * LW::K : 0;
    lw.seek(at, left);
#pragma unroll
    for (int j = 0; j < LW::kLoads; ++j) lw.load(j, m, 0);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        x[i][h] = __builtin_amdgcn_raw_buffer_load_b128(
            rx, (PAIR ? g * 8u : (2 * g + h) * 8u) < left ? (int)(xo[i] + at * kMmaBytes) : (int)kMmaOff,
            h * (PAIR ? kMmaLow * 2 : 16), 0);
  };
  v4f acc[MT][HB];
#pragma unroll
  for (int i = 0; i < TILES; ++i) acc[i / HB][i % HB] = v4f{0.f, 0.f, 0.f, 0.f};
  auto chunk = [&](const uint8_t* m, const Rows& x) {
    uint4 b[2][HB];
#pragma unroll
    for (int j = 0; j < 2 * HB; ++j) b[j / HB][j % HB] = rw(m, j / HB, j % HB);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const uint4 a0 = __builtin_bit_cast(uint4, x[i][0]), a1 = __builtin_bit_cast(uint4, x[i][1]);
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        if constexpr (PAIR) {
          acc[i][j] = mma16<DT>(b[1][j], a0, acc[i][j]);
          acc[i][j] = mma16<DT>(b[0][j], a1, acc[i][j]);
          acc[i][j] = mma16<DT>(b[0][j], a0, acc[i][j]);
        } else {
          acc[i][j] = mma16<DT>(b[0][j], a0, acc[i][j]);
          acc[i][j] = mma16<DT>(b[1][j], a1, acc[i][j]);
        }
      }
    }
  };
  uint32_t c = wave;
  Rows x0, x1;
  fetch(c, m0, x0);
  __builtin_amdgcn_sched_barrier(0);
  fetch(c + WAVES, m1, x1);
  // (a wavefront without a chunk adds one of zeros)
  do {
    wait_loads<LOADS>();
    chunk(m0, x0);
    __builtin_amdgcn_sched_barrier(0);
    fetch(c + 2 * WAVES, m0, x0);
    wait_loads<LOADS>();
    chunk(m1, x1);
    __builtin_amdgcn_sched_barrier(0);
    fetch(c + 3 * WAVES, m1, x1);
    c += 2 * WAVES;
  } while (c < total);
  __syncthreads();  // (waits for the last fetches, of nothing, as well)
  constexpr int SPLIT = WAVES * STAGE / 1024;  // partial tiles in st0, the rest in st1
  auto at = [&](int i) {
    return reinterpret_cast<v4f*>(i < SPLIT ? st0 + i * 1024 : st1 + (i - SPLIT) * 1024) + lane;
  };
#pragma unroll
  for (int i = 0; i < TILES; ++i) *at(wave * TILES + i) = acc[i / HB][i % HB];
  __syncthreads();
  for (int i = wave; i < MT; i += WAVES) {
    if (i * 16 >= p.t) break;
    v4f v[HB], bias[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      v[j] = *at(i * HB + j);
#pragma unroll
      for (int k = 1; k < WAVES; ++k) v[j] += *at(k * TILES + i * HB + j);
    }
    xent_bias<HB>(p, col0, g, bias);
    const int64_t row = i * 16 + r;
    float ex[HB * 4];
    xent_row<PAIR, HB>(p, row, col0, g, v, bias, xent_shift<PAIR>(p, row), row < p.t ? p.targets[row] : -1, ex);
    if (row >= p.t) continue;
    if constexpr (KEEP) {
      float* e = static_cast<float*>(p.e) + row * p.vp + col0 + 4 * g;
#pragma unroll
      for (int j = 0; j < HB; ++j)
        *reinterpret_cast<float4*>(e + j * 16) = make_float4(ex[4 * j], ex[4 * j + 1], ex[4 * j + 2], ex[4 * j + 3]);
    }
  }
}

// One workgroup per token: the sum over the segments, in a fixed order.  One
// more, where wanted, works out the scalars, which the gradients need.  A launch's
// time (5 us) up to some hundred tokens, 11 us for 4096 of 500 segments.
struct XentSums {
  const float2* stats;
  int64_t t, nseg;
  const int64_t* targets;
  const float* target;
  float *loss, *lse, *sc;
  float2* sums;  // largest logit and 1 over the sum of exponentials below it, for the gradient
};
__global__ __launch_bounds__(256) void k_xent_lse(XentArgs a, XentSums p) {
  const int64_t row = blockIdx.x;
  if (row == p.t) return xent_scalars(a, true, false, nullptr, p.sc);
  const float2* s = p.stats + row * p.nseg;
  float m = -__builtin_inff(), sum = 0.f;
  for (int64_t i = threadIdx.x; i < p.nseg; i += 256) {
    const float2 x = s[i];
    const float n = fmaxf(m, x.x), ref = n == -__builtin_inff() ? 0.f : n;
    sum = sum * __builtin_amdgcn_exp2f((m - ref) * kLog2e) + x.y * __builtin_amdgcn_exp2f((x.x - ref) * kLog2e);
    m = n;
  }
  __shared__ float tops[4], sums[4];
  const int wave = threadIdx.x >> 6;
  float top = wave_max(m);
  if ((threadIdx.x & 63) == 0) tops[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const float ref = top == -__builtin_inff() ? 0.f : top;
  sum = wave_sum(sum * __builtin_amdgcn_exp2f((m - ref) * kLog2e));
  if ((threadIdx.x & 63) == 0) sums[wave] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  // (the loss from differences to the largest logit: lse is rounded at its full
  // size, which would stay in the loss and in the target's entry of G)
  const float s1 = sums[0] + sums[1] + sums[2] + sums[3], l = logf(s1);
  p.lse[row] = ref + l;
  if (p.sums) p.sums[row] = make_float2(ref, 1.f / s1);
  const int64_t y = p.targets[row];
  p.loss[row] = ignored(y, a.ignore) ? 0.f : y < a.v ? l - (p.target[row] - ref) : __builtin_nanf("");
}

// ------------------------------------------------------------- the gradient
struct XentGrad {
  int64_t t, v, vp, nseg;
  int seg_shift, rows;  // rows: tokens of a workgroup
  const float2 *stats, *sums;
  const float *loss, *weights, *sc;
  const int* factors;  // exponents
  const int64_t* targets;
  int64_t ignore;
  void* e;       // fp16 (G in its place) or fp32
  uint16_t* g;   // G, or its two pieces; of few tokens' the lower ones kFewTokens rows on
  float* db;     // partial sums, or null
};

// E to G, eight columns a thread, `rows` tokens a workgroup one after the other, the
// next reading under way while one is worked on (two at a time: with four the
// registers cost 4096 x 32000 8 us).  A workgroup's columns' sums go to its row of
// db.  Bound by HBM: 4096 x 32000 in 16 bits 115 us, 4.6 TB/s; 700 x 33278 from fp32 to
// two pieces 46 us, 4.1 TB/s.
template <int DT, bool FEW>  // of G: kF16 and kBF16 in E's place, kF32 as two pieces; FEW: two pieces of a 16-bit type
__global__ __launch_bounds__(256) void k_xent_grad(XentGrad p) {
  const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 8, t0 = (int64_t)blockIdx.x * p.rows;
  if (c >= p.vp) return;
  const int most = (int)p.sc[kEg];
  const float gs = ldexpf(1.f, most);
  const int64_t seg = min(c >> p.seg_shift, p.nseg - 1);
  const int n = (int)min((int64_t)p.rows, p.t - t0);
  float sums[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[e] = 0.f;
#pragma unroll 2
  for (int i = 0; i < n; ++i) {
    const int64_t row = t0 + i, at = row * p.vp + c, y = p.targets[row];
    const bool off = ignored(y, p.ignore) || y >= p.v || (p.weights && p.weights[row] == 0.f);
    float v[8];
    if constexpr (DT == kF32 || FEW) {
      __builtin_memcpy(v, static_cast<const float*>(p.e) + at, sizeof v);
    } else {
      uint16_t h[8];
      __builtin_memcpy(h, static_cast<const uint16_t*>(p.e) + at, sizeof h);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = Elem<kF16>::up(h[e]);
    }
    // (a row's own power of two: the largest weight's less the row's exponent)
    const int less = p.weights ? p.factors[row] : 0;
    const float back = ldexpf(1.f, less), u = p.weights ? ldexpf(p.weights[row], most - less) : gs;
    const float2 sum = p.sums[row];
    const float f = u * (__builtin_amdgcn_exp2f((p.stats[row * p.nseg + seg].x - sum.x) * kLog2e) * sum.y) *
                    (DT == kF32 || FEW ? 1.f : 1.f / kHeld);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = off || c + e >= p.v ? 0.f : v[e] * f;
    if (!off && y >= c && y < c + 8) {
      const float z = u * expm1f(-p.loss[row]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (y == c + e) v[e] = z;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[e] = fmaf(v[e], back, sums[e]);
    uint16_t h[8];
    if constexpr (DT == kF32 || FEW) {
      constexpr int T = DT == kF32 ? kF16 : DT;
      uint16_t lo[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[e] = Elem<T>::down(v[e]);
        const float r = v[e] - Elem<T>::up(h[e]);
        lo[e] = Elem<T>::down(r == r ? r : 0.f);
      }
      uint16_t* const g = FEW ? p.g + at : p.g + row * 2 * p.vp + mma_piece(c);
      __builtin_memcpy(g, h, sizeof h);
      __builtin_memcpy(g + (FEW ? kFewTokens * p.vp : kMmaLow), lo, sizeof lo);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = Elem<DT>::down(v[e]);
      __builtin_memcpy(p.g + at, h, sizeof h);
    }
  }
  if (p.db) {
    float* d = p.db + (int64_t)blockIdx.x * p.vp + c;
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = sums[e];
  }
}

// db = (add +) the scale times the partial sums in order.  Blocks of tokens before the last
// add up in `sum`, fp32: one rounding to db's type, and no partial sum in it.
__global__ __launch_bounds__(256) void k_xent_db(const float* part, int64_t rows, int64_t vp, int64_t v, const float* sc,
                                                 float* sum, bool first, bool last, void* db, int dtype, bool add) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= v) return;
  float s = 0.f;
#pragma unroll 8
  for (int64_t i = 0; i < rows; ++i) s += part[i * vp + c];
  if (!first) s += sum[c];
  if (!last) {
    sum[c] = s;
    return;
  }
  s = ldexpf(s * sc[kS], (int)sc[kEdb]);
  if (add) s += load_any(db, dtype, c);
  store_any(db, dtype, c, s);
}

struct XentProduct {
  MmaSide a, b;
  int64_t k;
  const float* sc;  // the scalars, or null: the sums as they are
  int exponent;     // which of them the result is 2 to the power of
  MmaOut out;
  int64_t split_stride;  // elements between the results of two pieces of the summed axis
  int pieces;            // of them
  int64_t low;           // elements from a's rows to their lower pieces, kFewTokens rows on, 0: none
};

// dx (G's rows K-contiguous) and dw (K-strided).  4096 x 32000 x 4096 bf16: dx 0.78 -
// 0.83 ms, 1.3 - 1.4 PFLOP/s, matrix cores 71 % busy; dw 0.83 - 0.89 ms, 66 %: its
// 32000 x 4096 results are more to write, and every operand comes through the
// transposing read.  dx of few tokens: pieces of the vocabulary, so that there are
// workgroups enough (20 x 33278 x 650: 15 us, and 5 for their sum).
template <int DT, bool PAIR, int ODT, bool AKC, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_xent_product(XentProduct p, int ntm, int ntn) {
  using Tile = MmaTile<DT, PAIR, AKC, false, WM, WN, TM, TN>;
  __shared__ __align__(16) uint8_t a0[Tile::BM * kMmaBytes], b0[Tile::BN * kMmaBytes], a1[Tile::BM * kMmaBytes],
      b1[Tile::BN * kMmaBytes];
  // (the tiles of one piece of the summed axis share their operands: neighbours in
  // the walk, which an XCD takes an eighth of)
  int tm, tn, piece = 0;
  if (p.pieces == 1) {
    mma_tile_of_block(blockIdx.x, ntm, ntn, &tm, &tn);
  } else {
    const int t = xcd_position(blockIdx.x, gridDim.x), in = t % (ntm * ntn);
    piece = t / (ntm * ntn);
    tm = in % ntm;
    tn = in / ntm;
  }
  const int64_t m0 = (int64_t)tm * Tile::BM, n0 = (int64_t)tn * Tile::BN;
  const uint32_t total = (uint32_t)((p.k + Tile::K - 1) / Tile::K);
  const uint32_t c0 = (uint32_t)((uint64_t)total * piece / p.pieces);
  const uint32_t c1 = (uint32_t)((uint64_t)total * (piece + 1) / p.pieces);
  typename Tile::Acc acc;
  Tile::run(p.a, p.b, p.k, c0, c1, m0, n0, a0, b0, a1, b1, acc);
  if (AKC && !PAIR && p.low) {  // (few tokens: rows 32 on are the lower pieces of the first ones)
    static_assert(Tile::HA >= 4 && kFewTokens == 32, "both pieces' rows in one wavefront");
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < Tile::HB; ++j) acc[i][j] += acc[i + 2][j];
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* lds = mma_epilogue_lds<Tile>(wave, a0, b0, a1, b1);
  p.out.c = static_cast<typename Elem<ODT>::type*>(p.out.c) + piece * p.split_stride;
  mma_store<ODT>(p.out, p.sc ? p.sc[kS] : 1.f, p.sc ? (int)p.sc[p.exponent] : 0, lds, m0 + wave / WN * TM * 32, n0 + wave % WN * TN * 32, acc);
}

// Four neighbouring values of each of a lane's eight rows of an operand of at most
// 32, by tile.
template <bool PAIR>
__device__ __forceinline__ void outer_read(const MmaSide& s, int64_t k, int64_t first, int piece, uint4 (&v)[4]) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t c = first + 4 * r;  // (rows are padded to 64 values)
  const uint16_t* q = s.p + (PAIR ? mma_piece(c) + piece * kMmaLow : c);
  uint2 x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = *reinterpret_cast<const uint2*>(q + min((int64_t)8 * g + e, k - 1) * s.ld);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 8 * g + e < k ? x[e] : make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = __builtin_amdgcn_perm(i < 2 ? x[2 * e + 1].x : x[2 * e + 1].y, i < 2 ? x[2 * e].x : x[2 * e].y,
                                   i % 2 ? 0x07060302u : 0x05040100u);
    v[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// dw of at most 32 tokens: one step of the matrix cores and a write of the result.
// A wavefront takes 64 x 64 of it.  The summed axis is the operands' rows, so a
// lane reads four neighbouring values of each of its eight rows, one for each of
// its four tiles: tile i has rows 4 r + i of the 64, and lane (r, g) ends up with
// columns 16 g .. + 15 of rows 4 r .. + 3.
template <int DT, bool PAIR, int ODT>
__global__ __launch_bounds__(256) void k_xent_outer(XentProduct p, int ntn) {
  __shared__ __align__(16) float lds[4][32 * 68];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int t = xcd_position(blockIdx.x, gridDim.x);
  const int64_t m0 = (int64_t)(t / ntn) * 128 + wave / 2 * 64, n0 = (int64_t)(t % ntn) * 128 + wave % 2 * 64;
  if (m0 >= p.out.m || n0 >= p.out.n) return;
  constexpr int N = PAIR ? 2 : 1;
  uint4 a[2][4], b[N][4];
#pragma unroll
  for (int n = 0; n < N; ++n) outer_read<PAIR>(p.a, p.k, m0, n, a[n]), outer_read<PAIR>(p.b, p.k, n0, n, b[n]);
  const bool low = !PAIR && p.low != 0;
  if (low) outer_read<false>(MmaSide{p.a.p + p.low, p.a.ld, p.a.len}, p.k, m0, 0, a[1]);
  const float alpha = p.sc[kS];
  const int exponent = (int)p.sc[p.exponent];
  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
      if constexpr (PAIR) {
        acc[i][j] = mma16<DT>(b[N - 1][j], a[0][i], acc[i][j]);
        acc[i][j] = mma16<DT>(b[0][j], a[1][i], acc[i][j]);
      }
      if (low) acc[i][j] = mma16<DT>(b[0][j], a[1][i], acc[i][j]);
      acc[i][j] = mma16<DT>(b[0][j], a[0][i], acc[i][j]);
    }
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // 32 rows, half of the lanes', at a time
    if (r / 8 == h) {
      float* const wr = lds[wave] + 4 * (r % 8) * 68 + 16 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<v4f*>(wr + i * 68 + 4 * e) =
              v4f{mma_scaled(acc[i][0][e], alpha, exponent), mma_scaled(acc[i][1][e], alpha, exponent),
                  mma_scaled(acc[i][2][e], alpha, exponent), mma_scaled(acc[i][3][e], alpha, exponent)};
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    mma_store_any<ODT, 64>(p.out, 0, lds[wave], m0 + h * 32, n0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// The same for rows that are no whole vectors but follow each other without a gap:
// a workgroup takes 32 whole rows, which lie in one piece that starts on a vector,
// puts them together in LDS as they lie in memory and writes that.  A lane reads two
// neighbouring values of G's rows here: tile i has rows 2 r + i of the 32.  33278 x
// 650 fp16 (43 MB written, 2.8 TB/s): 16 us, by the rows' own 4-byte stores 27.
constexpr int kOuterThreads = 512;  // (15.8 us at 33278 x 650 fp16 of 20 tokens; 256 take 17.8, 1024 17.5)
template <int DT, bool PAIR, int ODT>
__global__ __launch_bounds__(kOuterThreads) void k_xent_outer_rows(XentProduct p) {
  using T = typename Elem<ODT>::type;
  extern __shared__ __align__(16) uint8_t rows_lds[];
  T* const lds = reinterpret_cast<T*>(rows_lds);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)xcd_position(blockIdx.x, gridDim.x) * 32;
  const int n = (int)p.out.n;
  constexpr int N = PAIR ? 2 : 1;
  const float alpha = p.sc[kS];
  const int exponent = (int)p.sc[p.exponent];
  const bool low = !PAIR && p.low != 0;
  uint4 a[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!PAIR && h == 1 && !low) break;
    const int64_t c = m0 + 2 * r;  // (rows are padded to 64 values)
    const uint16_t* q = p.a.p + (PAIR ? mma_piece(c) + h * kMmaLow : c + h * p.low);
    uint32_t x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = *reinterpret_cast<const uint32_t*>(q + min((int64_t)8 * g + e, p.k - 1) * p.a.ld);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 8 * g + e < p.k ? x[e] : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __builtin_amdgcn_perm(x[2 * e + 1], x[2 * e], i ? 0x07060302u : 0x05040100u);
      a[h][i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  for (int n0 = wave * 64; n0 < n; n0 += kOuterThreads) {
    uint4 b[N][4];
#pragma unroll
    for (int h = 0; h < N; ++h) outer_read<PAIR>(p.b, p.k, n0, h, b[h]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v4f acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
        if constexpr (PAIR) {
          acc[j] = mma16<DT>(b[N - 1][j], a[0][i], acc[j]);
          acc[j] = mma16<DT>(b[0][j], a[1][i], acc[j]);
        }
        if (low) acc[j] = mma16<DT>(b[0][j], a[1][i], acc[j]);
        acc[j] = mma16<DT>(b[0][j], a[0][i], acc[j]);
      }
      const int row = 2 * r + i;
      T* const to = lds + row * n;
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // columns 16 g + 2 e and the next
        const int col = n0 + 16 * g + 2 * e;
        const float u = mma_scaled(acc[e % 2 * 2][e / 2], alpha, exponent);
        const float v = mma_scaled(acc[e % 2 * 2 + 1][e / 2], alpha, exponent);
        if constexpr (sizeof(T) == 2) {
          if (n % 2 == 0) {
            const uint32_t both = (uint32_t)Elem<ODT>::down(u) | (uint32_t)Elem<ODT>::down(v) << 16;
            if (col < n) *reinterpret_cast<uint32_t*>(to + col) = both;
            continue;
          }
        }
        if (col < n) to[col] = Elem<ODT>::down(u);
        if (col + 1 < n) to[col + 1] = Elem<ODT>::down(v);
      }
    }
  }
  __syncthreads();
  const int values = (int)min((int64_t)32, p.out.m - m0) * n, whole = values / (16 / (int)sizeof(T));
  T* const out = static_cast<T*>(p.out.c) + m0 * n;
  for (int i = threadIdx.x; i < whole; i += kOuterThreads)
    reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(lds)[i];
  for (int i = whole * (16 / (int)sizeof(T)) + threadIdx.x; i < values; i += kOuterThreads) out[i] = lds[i];
}

// dx = the scale times the pieces' sums in order.
__global__ __launch_bounds__(256) void k_xent_dx(const float* part, int64_t pieces, int64_t t, int64_t d,
                                                 const float* sc, const int* factors, void* dx, int dtype,
                                                 int64_t lddx) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= t * d) return;
  float s = 0.f;
#pragma unroll 8
  for (int64_t k = 0; k < pieces; ++k) s += part[k * t * d + i];
  store_any(dx, dtype, i / d * lddx + i % d, mma_scaled(s, sc[kS], (int)sc[kEdx] + (factors ? factors[i / d] : 0)));
}

// Gradients of a loss over no word or no token.
__global__ __launch_bounds__(256) void k_xent_zero(void* p, int dtype, int64_t rows, int64_t cols, int64_t ld) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * cols; i += (int64_t)gridDim.x * 256)
    store_any(p, dtype, i / cols * ld + i % cols, 0.f);
}

// The sum of the losses, or their mean over the tokens that are not ignored, in fp64
// and a fixed order.  One workgroup up to 65536 tokens (6 us at 4096 and 20000); of
// more (1 Mi: 360 us by one) each of `kTotalGroups` leaves its part and a second
// launch adds those up: 11 us, 16 Mi tokens 33 us, 6 TB/s.
constexpr int kTotalThreads = 1024, kTotalGroups = 256;
constexpr int64_t kTotalAlone = 65536;
__device__ __forceinline__ bool total_of_threads(double& s, double& n) {  // in thread 0, which it is true for
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o), n += __shfl_xor(n, o);
  __shared__ double ps[kTotalThreads / 64], pn[kTotalThreads / 64];
  if ((threadIdx.x & 63) == 0) ps[threadIdx.x >> 6] = s, pn[threadIdx.x >> 6] = n;
  __syncthreads();
  if (threadIdx.x != 0) return false;
  for (int i = 1; i < (int)blockDim.x / 64; ++i) s += ps[i], n += pn[i];
  return true;
}
__global__ __launch_bounds__(kTotalThreads) void k_xent_total(const float* loss, const int64_t* targets, int64_t t,
                                                              int64_t ignore, bool mean, double2* parts, float* total) {
  double s = 0.0, n = 0.0;
#pragma unroll 8
  for (int64_t i = (int64_t)blockIdx.x * kTotalThreads + threadIdx.x; i < t; i += (int64_t)gridDim.x * kTotalThreads) {
    s += loss[i];
    n += mean && !ignored(targets[i], ignore) ? 1.0 : 0.0;
  }
  if (!total_of_threads(s, n)) return;
  if (gridDim.x > 1)
    parts[blockIdx.x] = make_double2(s, n);
  else
    *total = (float)(mean ? s / fmax(n, 1.0) : s);
}
__global__ __launch_bounds__(kTotalGroups) void k_xent_total_join(const double2* parts, bool mean, float* total) {
  double s = parts[threadIdx.x].x, n = parts[threadIdx.x].y;
  if (total_of_threads(s, n)) *total = (float)(mean ? s / fmax(n, 1.0) : s);
}

// Gradients times the incoming value, which only the device knows: one product in
// fp32 and one rounding, 16 bytes a thread where both addresses allow it.  Bound by
// HBM: 32000 x 4096 bf16 98 us, 5.3 TB/s.
template <int DT>
__global__ __launch_bounds__(256) void k_xent_scale(const void* from, void* to, int64_t n, const float* factor) {
  using T = typename Elem<DT>::type;
  constexpr int N = 16 / (int)sizeof(T);
  const float f = *factor;
  const T* const in = static_cast<const T*>(from);
  T* const out = static_cast<T*>(to);
  const int64_t stride = (int64_t)gridDim.x * 256, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t whole = (((uintptr_t)from | (uintptr_t)to) & 15) == 0 ? n / N : 0;
#pragma unroll 4
  for (int64_t i = first; i < whole; i += stride) {
    T v[N];
    __builtin_memcpy(v, __builtin_assume_aligned(in + i * N, 16), sizeof v);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = Elem<DT>::down(Elem<DT>::up(v[e]) * f);
    __builtin_memcpy(__builtin_assume_aligned(out + i * N, 16), v, sizeof v);
  }
  for (int64_t i = whole * N + first; i < n; i += stride) out[i] = Elem<DT>::down(Elem<DT>::up(in[i]) * f);
}

// ---------------------------------------------------------------- the host
static int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
static int64_t cdiv(int64_t v, int64_t by) { return (v + by - 1) / by; }
static unsigned grid(int64_t n) { return (unsigned)cdiv(n, 256); }

// An operand that the tile loop can read where it is.
static bool readable(const void* p, int64_t ld, int64_t d, int dtype) {
  return dtype != kF32 && ((uintptr_t)p & 15) == 0 && ld % 8 == 0 && d % 8 == 0;
}

// Of few tokens of a 16-bit type G has two pieces, from an E in fp32: single
// entries of G (the target's) dominate a sum over few, whose rounding to the type
// made the gradients of one or two tokens up to 1.7 times as inexact as their own
// rounding does (over many tokens 1.05 to 1.25 times, which two pieces would cost a
// second product each for).  Here they cost no more than the second piece's rows, in
// tiles that are mostly empty: 20 x 33278 x 650 fp16 81 us a call, 80 with one.
static bool few_pieces(const XentArgs& a) { return a.dtype != kF32 && a.t <= kFewTokens; }

// Tokens of a workgroup of the pass over E: fewer where that leaves too few of them.
static int64_t grad_rows(int64_t tokens, int64_t vp) {
  return std::min<int64_t>(kGradRows, std::max<int64_t>(1, tokens * cdiv(vp, 2048) / 1024));
}

// (train: with gradients, one at least)
XentLayout xent_layout(const XentArgs& a, bool train) {
  XentLayout l{};
  const bool f32 = a.dtype == kF32;
  l.parts = f32 ? 2 : 1;
  l.pack_x = !readable(a.x, a.ldx, a.d, a.dtype);
  l.pack_w = !readable(a.w, a.ldw, a.d, a.dtype);
  l.dp = up(a.d, 64);
  l.vp = up(a.v, 64);
  l.seg_shift = a.t <= kFewTokens ? 5 : 6;
  l.nseg = cdiv(a.v, int64_t(1) << l.seg_shift);
  // (a block's rows are a multiple of the tiles', and few tokens are one block; its
  // size bounds the workspace and every launch of a workgroup a token)
  const int64_t held = train ? l.vp * (f32 ? 8 : 2) : l.nseg * (int64_t)sizeof(float2);
  l.block = std::min({std::max<int64_t>(1, a.t), kBlockTokens, std::max<int64_t>(256, kBlockBytes / held / 256 * 256)});
  const int64_t tiles = cdiv(l.block, 128) * cdiv(a.d, 128), chunks = cdiv(a.v, f32 ? kMmaK<true> : kMmaK<false>);
  l.dx_splits = std::max<int64_t>(1, std::min<int64_t>({512 / std::max<int64_t>(1, tiles), chunks / 8, 128}));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += (bytes + 255) / 256 * 256;
    return was;
  };
  l.scalars = take(kScalars * sizeof(float));
  l.partmax = take(f32 ? 2 * kMaxGroups * sizeof(float) : 0);
  l.xrow = take(f32 ? (size_t)a.t * sizeof(int) : 0);
  l.rows = take(train && a.weights ? (size_t)a.t * sizeof(int) : 0);
  // x as the logits' operand, then (for dw) with rows of tokens that do not count zero
  l.x = take((size_t)((l.pack_x ? 1 : 0) + (train && a.dw ? 1 : 0)) * l.parts * a.t * l.dp * 2);
  l.w = take(l.pack_w ? (size_t)l.parts * a.v * l.dp * 2 : 0);
  l.stats = take((size_t)l.block * l.nseg * sizeof(float2));
  l.target = take((size_t)l.block * sizeof(float));
  const bool few = few_pieces(a);
  if (train) {
    l.sums = take((size_t)l.block * sizeof(float2));
    l.e = take((size_t)l.block * l.vp * (f32 || few ? 4 : 2));
    l.g = f32 ? take((size_t)l.block * l.vp * 4) : few ? take((size_t)2 * kFewTokens * l.vp * 2) : l.e;
    l.db = take(a.dbias ? (size_t)cdiv(l.block, grad_rows(l.block, l.vp)) * l.vp * sizeof(float) : 0);
    l.dbs = take(a.dbias && l.block < a.t ? (size_t)a.v * sizeof(float) : 0);
    l.dxp = take(a.dx && l.dx_splits > 1 ? (size_t)l.dx_splits * l.block * a.d * sizeof(float) : 0);
    l.dwp = take(a.dw && a.dw_dtype != kF32 && l.block < a.t ? (size_t)a.v * a.d * sizeof(float) : 0);
  }
  l.bytes = std::max<size_t>(at, 256);
  return l;
}

// The weights' operand and the hidden states' in one launch; rows 0: none of it.
static void pack(const XentPack& w, const XentPack& x, int dtype, hipStream_t s) {
  // (a launch holds 2^32 threads: larger operands in pieces, one after the other)
  constexpr int64_t most = int64_t(1) << 31;
  if (w.rows * (w.dp / 8) + x.rows * (x.dp / 8) > most) {
    if (w.rows && x.rows) {
      pack(w, XentPack{}, dtype, s);
      pack(XentPack{}, x, dtype, s);
    } else {
      const XentPack& p = w.rows ? w : x;
      const int64_t half = p.rows / 2;
      for (int64_t at : {int64_t(0), half}) {
        const XentPack q = p.rows_from(at, at ? p.rows - half : half, dtype);
        pack(w.rows ? q : XentPack{}, w.rows ? XentPack{} : q, dtype, s);
      }
    }
    return;
  }
  const unsigned first = grid(w.rows * w.dp / 8), all = first + grid(x.rows * x.dp / 8);
  if (all == 0) return;
  if (dtype == kF32)
    hipLaunchKernelGGL((k_xent_pack<kF32>), dim3(all), dim3(256), 0, s, w, x, first);
  else if (dtype == kBF16)
    hipLaunchKernelGGL((k_xent_pack<kBF16>), dim3(all), dim3(256), 0, s, w, x, first);
  else
    hipLaunchKernelGGL((k_xent_pack<kF16>), dim3(all), dim3(256), 0, s, w, x, first);
}

template <int DT, bool PAIR, bool TRAIN>
static void logits(const XentTile& p, int64_t tokens, hipStream_t s) {
  if (tokens <= kFewTokens) {
    // (four wavefronts, five workgroups to a compute unit, where eight would have
    // hardly a chunk each)
    const dim3 g((unsigned)cdiv(p.v, 32));
    const bool brief = p.d <= 16 * kMmaK<PAIR>;
    if (p.t <= 16 && brief)
      hipLaunchKernelGGL((k_xent_logits_few<DT, PAIR, TRAIN, 1, 4>), g, dim3(256), 0, s, p);
    else if (p.t <= 16)
      hipLaunchKernelGGL((k_xent_logits_few<DT, PAIR, TRAIN, 1, 8>), g, dim3(512), 0, s, p);
    else if (brief)
      hipLaunchKernelGGL((k_xent_logits_few<DT, PAIR, TRAIN, 2, 4>), g, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((k_xent_logits_few<DT, PAIR, TRAIN, 2, 8>), g, dim3(512), 0, s, p);
    return;
  }
  constexpr int KEEP = !TRAIN ? 0 : PAIR ? 2 : 1;
  if (cdiv(p.t, 256) * cdiv(p.v, 256) >= 256) {
    const int ntm = (int)cdiv(p.t, 256), ntn = (int)cdiv(p.v, 256);
    hipLaunchKernelGGL((k_xent_logits<DT, PAIR, KEEP, 2, 4, 4, 2>), dim3(ntm * ntn), dim3(512), 0, s, p, ntm, ntn);
  } else {
    const int ntm = (int)cdiv(p.t, 128), ntn = (int)cdiv(p.v, 128);
    hipLaunchKernelGGL((k_xent_logits<DT, PAIR, KEEP, 2, 2, 2, 2>), dim3(ntm * ntn), dim3(256), 0, s, p, ntm, ntn);
  }
}

template <int DT, bool PAIR, int ODT, bool AKC>
static void product_to(XentProduct p, int64_t pieces, hipStream_t s) {
  p.pieces = (int)pieces;
  if (!AKC && p.k <= 32) {
    const int64_t es = sizeof(typename Elem<ODT>::type), rows = 32 * p.out.n * es;
    if (!p.out.add && !p.out.accumulate && !p.out.row && p.out.ldc == p.out.n && ((uintptr_t)p.out.c & 15) == 0 &&
        p.out.n * es % 16 != 0 && rows <= 64 * 1024) {
      hipLaunchKernelGGL((k_xent_outer_rows<DT, PAIR, ODT>), dim3((unsigned)cdiv(p.out.m, 32)), dim3(kOuterThreads), (size_t)rows, s, p);
      return;
    }
    const int64_t ntm = cdiv(p.out.m, 128), ntn = cdiv(p.out.n, 128);
    hipLaunchKernelGGL((k_xent_outer<DT, PAIR, ODT>), dim3((unsigned)(ntm * ntn)), dim3(256), 0, s, p, (int)ntn);
    return;
  }
  if (pieces == 1 && cdiv(p.out.m, 256) * cdiv(p.out.n, 256) >= 192) {
    const int ntm = (int)cdiv(p.out.m, 256), ntn = (int)cdiv(p.out.n, 256);
    hipLaunchKernelGGL((k_xent_product<DT, PAIR, ODT, AKC, 2, 4, 4, 2>), dim3(ntm * ntn), dim3(512), 0, s, p, ntm, ntn);
  } else {
    const int ntm = (int)cdiv(p.out.m, 128), ntn = (int)cdiv(p.out.n, 128);
    hipLaunchKernelGGL((k_xent_product<DT, PAIR, ODT, AKC, 2, 2, 2, 2>), dim3((unsigned)(ntm * ntn * pieces)), dim3(256), 0, s,
                       p, ntm, ntn);
  }
}
template <int DT, bool PAIR, bool AKC>
static void product(const XentProduct& p, int odt, int64_t pieces, hipStream_t s) {
  if (odt == kF32)
    product_to<DT, PAIR, kF32, AKC>(p, pieces, s);
  else if (odt == kBF16)
    product_to<DT, PAIR, kBF16, AKC>(p, pieces, s);
  else
    product_to<DT, PAIR, kF16, AKC>(p, pieces, s);
}

// DT: what the products take; PAIR: two pieces of it for a value.
template <int DT, bool PAIR>
static void block(const XentArgs& a, const XentLayout& l, bool train, uint8_t* ws, int64_t t0, hipStream_t s) {
  constexpr int PIECES = PAIR ? 2 : 1;
  const int64_t n = std::min(l.block, a.t - t0), pitch = PIECES * l.dp;
  const float* sc = reinterpret_cast<const float*>(ws + l.scalars);
  uint16_t* const px = reinterpret_cast<uint16_t*>(ws + l.x);
  float2* const stats = reinterpret_cast<float2*>(ws + l.stats);
  float* const target = reinterpret_cast<float*>(ws + l.target);
  XentTile p{};
  p.x = l.pack_x ? MmaSide{px + t0 * pitch, pitch, n}
                 : MmaSide{static_cast<const uint16_t*>(a.x) + t0 * a.ldx, a.ldx, n};
  p.w = l.pack_w ? MmaSide{reinterpret_cast<uint16_t*>(ws + l.w), pitch, a.v}
                 : MmaSide{static_cast<const uint16_t*>(a.w), a.ldw, a.v};
  p.t = n, p.v = a.v, p.d = a.d, p.sc = sc, p.exponents = reinterpret_cast<const int*>(ws + l.xrow) + t0, p.bias = a.bias, p.bias_dtype = a.dtype;
  p.targets = a.targets + t0, p.stats = stats, p.nseg = l.nseg, p.target = target, p.e = ws + l.e, p.vp = l.vp;
  if (train)
    logits<DT, PAIR, true>(p, a.t, s);
  else
    logits<DT, PAIR, false>(p, a.t, s);
  const bool scalars = train && !PAIR && !a.weights && t0 == 0;
  float2* const sums = train ? reinterpret_cast<float2*>(ws + l.sums) : nullptr;
  hipLaunchKernelGGL(k_xent_lse, dim3((unsigned)n + (scalars ? 1 : 0)), dim3(256), 0, s, a,
                     XentSums{stats, n, l.nseg, a.targets + t0, target, a.loss + t0, a.lse + t0,
                              reinterpret_cast<float*>(ws + l.scalars), sums});
  if (!train) return;
  uint16_t* const g = reinterpret_cast<uint16_t*>(ws + l.g);
  float* const db = reinterpret_cast<float*>(ws + l.db);
  const int rows = (int)grad_rows(l.block, l.vp);
  const int64_t parts = cdiv(n, rows);
  const int* const factors = a.weights ? reinterpret_cast<int*>(ws + l.rows) + t0 : nullptr;
  const XentGrad q{n,       a.v, l.vp,           l.nseg,   l.seg_shift, rows, stats, sums, a.loss + t0,
                   a.weights ? a.weights + t0 : nullptr, sc, factors, a.targets + t0, a.ignore, ws + l.e, g,
                   a.dbias ? db : nullptr};
  const bool few = few_pieces(a);
  const int64_t low = few ? kFewTokens * l.vp : 0;
  const dim3 gg((unsigned)parts, (unsigned)cdiv(l.vp, 2048));
  if (few)
    hipLaunchKernelGGL((k_xent_grad<DT, !PAIR>), gg, dim3(256), 0, s, q);
  else
    hipLaunchKernelGGL((k_xent_grad<PAIR ? kF32 : DT, false>), gg, dim3(256), 0, s, q);
  if (a.dbias)
    hipLaunchKernelGGL(k_xent_db, dim3(grid(a.v)), dim3(256), 0, s, db, parts, l.vp, a.v, sc,
                       reinterpret_cast<float*>(ws + l.dbs), t0 == 0, t0 + n == a.t, a.dbias, a.dtype, a.accumulate);
  if (a.dx) {
    XentProduct d{};
    d.a = MmaSide{g, PIECES * l.vp, few ? 2 * kFewTokens : n};  // (rows in between are anything, and so are their sums)
    d.low = low;
    d.b = p.w;
    d.b.len = a.d;
    d.k = a.v;
    const int eb = dtype_bytes(a.dtype);
    uint8_t* const dx = static_cast<uint8_t*>(a.dx) + t0 * a.lddx * eb;
    if (l.dx_splits > 1) {
      float* const part = reinterpret_cast<float*>(ws + l.dxp);
      d.out = MmaOut{part, a.d, n, a.d, nullptr, false, nullptr};
      d.split_stride = n * a.d;
      product<DT, PAIR, true>(d, kF32, l.dx_splits, s);
      hipLaunchKernelGGL(k_xent_dx, dim3(grid(n * a.d)), dim3(256), 0, s, part, l.dx_splits, n, a.d, sc,
                         factors, dx, a.dtype, a.lddx);
    } else {
      d.sc = sc, d.exponent = kEdx;
      d.out = MmaOut{dx, a.lddx, n, a.d, nullptr, false, factors};
      product<DT, PAIR, true>(d, a.dtype, 1, s);
    }
  }
  if (a.dw) {
    XentProduct d{};
    d.a = MmaSide{g, PIECES * l.vp, a.v};
    d.b = MmaSide{px + (l.pack_x ? a.t * pitch : 0) + t0 * pitch, pitch, a.d};
    d.k = n, d.sc = sc, d.exponent = kEdw, d.low = low;
    // Blocks before the last add up in fp32: in dw itself, or in memory of
    // their own where dw has fewer bits.
    const bool last = t0 + n == a.t, wide = a.dw_dtype == kF32;
    float* const sum = reinterpret_cast<float*>(ws + l.dwp);
    if (wide)
      d.out = MmaOut{a.dw, a.lddw, a.v, a.d, nullptr, a.accumulate || t0 > 0, nullptr};
    else if (!last)
      d.out = MmaOut{sum, a.d, a.v, a.d, nullptr, t0 > 0, nullptr};
    else
      d.out = MmaOut{a.dw, a.lddw, a.v, a.d, t0 > 0 ? sum : nullptr, a.accumulate, nullptr};
    product<DT, PAIR, false>(d, wide || !last ? kF32 : a.dw_dtype, 1, s);
  }
}

hipError_t launch_xent(const XentArgs& a, const XentLayout& l, bool train, void* workspace, hipStream_t s) {
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  float* const sc = reinterpret_cast<float*>(ws + l.scalars);
  float* const partmax = reinterpret_cast<float*>(ws + l.partmax);
  int* const xrow = reinterpret_cast<int*>(ws + l.xrow);
  const bool f32 = a.dtype == kF32;
  if (a.t == 0) {
    if (train && !a.accumulate) {
      if (a.dw && a.v && a.d)
        hipLaunchKernelGGL(k_xent_zero, dim3(std::min(grid(a.v * a.d), 1u << 16)), dim3(256), 0, s, a.dw, a.dw_dtype, a.v, a.d, a.lddw);
      if (a.dbias)
        hipLaunchKernelGGL(k_xent_zero, dim3(grid(a.v)), dim3(256), 0, s, a.dbias, a.dtype, int64_t(1), a.v, a.v);
    }
    return hipGetLastError();
  }
  if (f32) hipLaunchKernelGGL(k_xent_max, dim3(2 * kMaxGroups), dim3(256), 0, s, a, train, partmax, xrow);
  if (f32 || (train && a.weights))
    hipLaunchKernelGGL(k_xent_prep, dim3(1), dim3(256), 0, s, a, train, f32, partmax, sc);
  XentPack w{}, x{};
  if (l.pack_w) w = XentPack{a.w, a.ldw, a.v, a.d, l.dp, f32 ? a.bias : nullptr, sc + kSw, nullptr, reinterpret_cast<uint16_t*>(ws + l.w)};
  if (l.pack_x || (train && (a.dw || a.weights))) {
    uint16_t* const px = reinterpret_cast<uint16_t*>(ws + l.x);
    x = XentPack{a.x,       a.ldx,    a.t,       a.d, l.dp, nullptr, sc + kSx, xrow, l.pack_x ? px : nullptr,
                 train && a.dw ? px + (l.pack_x ? l.parts * a.t * l.dp : 0) : nullptr,
                 a.targets, a.ignore, a.v, a.weights, sc, train ? reinterpret_cast<int*>(ws + l.rows) : nullptr};
  }
  pack(w, x, a.dtype, s);
  for (int64_t t0 = 0; t0 < a.t; t0 += l.block) {
    if (a.dtype == kBF16)
      block<kBF16, false>(a, l, train, ws, t0, s);
    else if (a.dtype == kF16)
      block<kF16, false>(a, l, train, ws, t0, s);
    else
      block<kF16, true>(a, l, train, ws, t0, s);
  }
  return hipGetLastError();
}

hipError_t launch_xent_total(const float* loss, const int64_t* targets, int64_t t, int64_t ignore, bool mean,
                             float* total, void* ws, hipStream_t s) {
  static_assert(kTotalGroups * sizeof(double2) == kXentTotalBytes, "the parts");
  double2* const parts = static_cast<double2*>(ws);
  const unsigned groups = t <= kTotalAlone ? 1 : kTotalGroups;
  hipLaunchKernelGGL(k_xent_total, dim3(groups), dim3(kTotalThreads), 0, s, loss, targets, t, ignore, mean, parts, total);
  if (groups > 1) hipLaunchKernelGGL(k_xent_total_join, dim3(1), dim3(kTotalGroups), 0, s, parts, mean, total);
  return hipGetLastError();
}

hipError_t launch_xent_scale(const void* in, int dtype, int64_t n, const float* factor, void* out, hipStream_t s) {
  if (n == 0) return hipSuccess;
  const dim3 g((unsigned)std::min<int64_t>(cdiv(n, 256 * 8), 4096));
  if (dtype == kF32)
    hipLaunchKernelGGL((k_xent_scale<kF32>), g, dim3(256), 0, s, in, out, n, factor);
  else if (dtype == kBF16)
    hipLaunchKernelGGL((k_xent_scale<kBF16>), g, dim3(256), 0, s, in, out, n, factor);
  else
    hipLaunchKernelGGL((k_xent_scale<kF16>), g, dim3(256), 0, s, in, out, n, factor);
  return hipGetLastError();
}

}  // namespace psgd
