// Global gradient norm over many tensors, and clipping (gfx950, wave64).
//
//   n_t = || scale * g_t ||,  N = sqrt(sum n_t^2),  c = min(1, max_norm / (N + 1e-6)),
//   out_t = scale * c * g_t
//
// Sums of squares; their sum in one fixed order, by a workgroup of its own or,
// for short lists, by every workgroup of the next launch; the scaled write.
// Squares are summed in fp64: an fp32 square overflows from 1.8e19 on, and the
// one conversion per element is hidden behind the reads.
// Bound: HBM, the gradients read twice (the second reading from the last level
// of cache as far as it holds them) and written once.  Sums are made in a
// fixed order without atomics, so a repeated call agrees bit for bit.

#include <hip/hip_runtime.h>

#include "psgd_clip.h"
#include "psgd_mx_device.h"

namespace psgd {

__global__ __launch_bounds__(256) void k_clip_bind(ClipTensor* tensors, ClipPointers p, int first, int n) {
  const int i = threadIdx.x;
  if (i >= n) return;
  tensors[first + i].in = p.in[i];
  tensors[first + i].out = p.out[i];
}

// E consecutive elements from p, as one access.
template <int DT, int E, bool NT>
__device__ __forceinline__ void load_group(const typename Elem<DT>::type* p, typename Elem<DT>::type (&v)[E]) {
  using T = typename Elem<DT>::type;
  typedef uint32_t vec __attribute__((ext_vector_type(E * sizeof(T) / 4)));
  const vec* q = reinterpret_cast<const vec*>(p);
  const vec x = NT ? __builtin_nontemporal_load(q) : *q;
  __builtin_memcpy(v, &x, sizeof x);
}

// Calls f(i, values, valid) for the groups of E consecutive elements that this
// thread takes of the elements [e0, e1), e1 - e0 <= kClipChunk: all loads
// first.  Groups that do not start on E elements' bytes are read one element
// at a time.
template <int DT, int E, bool NT, typename F>
__device__ __forceinline__ void walk(const void* base, int64_t e0, int64_t e1, F f) {
  using T = typename Elem<DT>::type;
  constexpr int UNROLL = kClipChunk / 256 / E;
  const T* g = static_cast<const T*>(base) + e0;
  const int n = (int)(e1 - e0);
  if (((uintptr_t)g & (E * sizeof(T) - 1)) == 0 && n == kClipChunk) {
    T v[UNROLL][E];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) load_group<DT, E, NT>(g + (u * 256 + (int)threadIdx.x) * E, v[u]);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      float x[E];
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = Elem<DT>::up(v[u][j]);
      f(e0 + (u * 256 + (int)threadIdx.x) * E, x, E);
    }
  } else {
    for (int i = (int)threadIdx.x * E; i < n; i += 256 * E) {
      float x[E];
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = i + j < n ? Elem<DT>::up(g[i + j]) : 0.f;
      f(e0 + i, x, min(E, n - i));
    }
  }
}

template <int DT, bool NT>
__device__ __forceinline__ double chunk_squares(const ClipTensor& t, int first) {
  constexpr int E = 16 / dtype_bytes(DT);
  double s0 = 0, s1 = 0;
  for (int64_t e0 = (int64_t)first * kClipChunk; e0 < t.numel; e0 += (int64_t)t.nsums * kClipChunk)
    walk<DT, E, NT>(t.in, e0, min(t.numel, e0 + kClipChunk), [&](int64_t, const float(&x)[E], int) {
#pragma unroll
      for (int j = 0; j < E; j += 2) {
        s0 = fma((double)x[j], (double)x[j], s0);
        s1 = fma((double)x[j + 1], (double)x[j + 1], s1);
      }
    });
  return s0 + s1;
}

// Workgroup i of a tensor takes the chunks i, i + nsums, ...: the workgroups
// that run together read one moving front of the tensor.
template <bool NT>
__global__ __launch_bounds__(256) void k_clip_sums(ClipArgs a) {
  const ClipTensor t = a.tensors[a.sum_map[blockIdx.x]];
  const int first = (int)blockIdx.x - t.first_sum;
  double s = !t.in                 ? __longlong_as_double(0x7ff8000000000000)  // never bound
             : t.in_dtype == kF32  ? chunk_squares<kF32, NT>(t, first)
             : t.in_dtype == kBF16 ? chunk_squares<kBF16, NT>(t, first)
                                   : chunk_squares<kF16, NT>(t, first);
  __shared__ double w[4];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.sums[blockIdx.x] = (w[0] + w[1]) + (w[2] + w[3]);
}

// Sum of all n sums, by 256 threads in one order whoever asks: every 256th by
// one thread, then the lanes', then the four wavefronts'.  Known to all 256
// threads behind the next barrier, in w.
template <typename Load>
__device__ __forceinline__ void total_of_sums(int n, Load load, double (&w)[4]) {
  double s = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += 256) s += load(i);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
}

__device__ __forceinline__ float2 norm_and_coefficient(const ClipArgs& a, const double (&w)[4]) {
  const double norm = sqrt((w[0] + w[1]) + (w[2] + w[3])) * fabs((double)a.scale);
  const double c = (double)a.max_norm / (norm + 1e-6);
  // (an infinite max_norm clips nothing, an infinite norm included: the quotient is NaN there)
  return make_float2((float)norm, norm != norm ? (float)norm : c < 1.0 ? (float)c : 1.f);
}

// The norms of tensors first, first + step, ... below end, by one wavefront:
// where their sums are is read for 64 tensors at a time.
template <typename Load>
__device__ __forceinline__ void tensor_norms(const ClipArgs& a, int first, int step, int end, Load load) {
  const int lane = threadIdx.x & 63;
  for (int t0 = first; t0 < end; t0 += 64 * step) {
    const int mine = t0 + lane * step;
    const int f_mine = mine < end ? a.tensors[mine].first_sum : 0, n_mine = mine < end ? a.tensors[mine].nsums : 0;
    for (int k = 0; k < 64 && t0 + k * step < end; ++k) {
      const int f = __builtin_amdgcn_readlane(f_mine, k), n = __builtin_amdgcn_readlane(n_mine, k);
      double s = 0;
#pragma unroll 8
      for (int i = lane; i < n; i += 64) s += load(f + i);
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
      if (lane == 0) a.stats[2 + t0 + k * step] = (float)(sqrt(s) * fabs((double)a.scale));
    }
  }
}

// One workgroup: all sums into LDS at once (in one wait for memory), then four
// wavefronts add them all, and all add each tensor's.  Sums beyond LDS (lists
// of more than a thousand tensors) are read where they are.
__global__ __launch_bounds__(1024) void k_clip_final(ClipArgs a) {
  __shared__ double part[4];
  constexpr int N = 2;
  __shared__ double lds[N * 1024];
  double v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = i * 1024 + (int)threadIdx.x;
    v[i] = at < a.nsums ? a.sums[at] : 0.0;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) lds[i * 1024 + threadIdx.x] = v[i];
  __syncthreads();
  auto sums = [&](auto load) {
    if (threadIdx.x < 256) total_of_sums(a.nsums, load, part);
    tensor_norms(a, __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64), 16, a.ntensors, load);
  };
  if (a.nsums <= N * 1024)
    sums([&](int i) { return lds[i]; });
  else
    sums([&](int i) { return a.sums[i]; });
  __syncthreads();
  if (threadIdx.x == 0) {
    const float2 r = norm_and_coefficient(a, part);
    a.stats[0] = r.x;
    a.stats[1] = r.y;
  }
}

// One chunk, from type IN to type OUT, in groups of 16 bytes of the wider
// one, so that the loads and the stores of a wavefront are contiguous.  Stores
// are nontemporal where in and out together would not stay in the last level
// of cache: they leave the gradients there from the norm's pass to this one,
// and no dirty lines for the next call's norm to push out (fp32, 64 Mi values:
// 155 -> 128 us, with a reader of the outputs behind it 228 -> 216; 32 Mi: 80
// -> 68, 110 -> 113; 8 Mi: 21.3 and 21.4, 31.5 and 34, stored as usual).
// Loads are nontemporal beyond a gibibyte of gradients (300 Mi: 638 -> 600 us).
template <int IN, int OUT, bool NTL, bool NTS>
__device__ __forceinline__ void scale_chunk(const ClipTensor& t, int64_t e0, float c) {
  constexpr int E = 16 / (dtype_bytes(IN) > dtype_bytes(OUT) ? dtype_bytes(IN) : dtype_bytes(OUT));
  using T = typename Elem<OUT>::type;
  typedef uint32_t vec __attribute__((ext_vector_type(E * sizeof(T) / 4)));
  walk<IN, E, NTL>(t.in, e0, min(t.numel, e0 + kClipChunk), [&](int64_t i, const float(&x)[E], int n) {
    T* o = static_cast<T*>(t.out) + i;
    T v[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = Elem<OUT>::down(x[j] * c);
    if (n == E && ((uintptr_t)o & (sizeof(vec) - 1)) == 0) {
      vec q;
      __builtin_memcpy(&q, v, sizeof q);
      if (NTS)
        __builtin_nontemporal_store(q, reinterpret_cast<vec*>(o));
      else
        *reinterpret_cast<vec*>(o) = q;
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (j < n) o[j] = v[j];
    }
  });
}

// Workgroups run through the chunks from the last to the first: the norm's
// pass has read the last ones last, and the cache still holds them.
// INLINE: every workgroup adds the sums by itself, and further ones write the
// norms, kClipStatsTensors tensors each, instead of a launch in between (fp32,
// two lists in turn: 2 Mi values 13.5 against 15.8 us, 32 Mi 69.4 and 71.5, 64
// Mi 130 and 132; but 667e6 bf16 values, 81 thousand workgroups, 905 and 876).
template <bool NTL, bool NTS, bool INLINE>
__global__ __launch_bounds__(256) void k_clip_apply(ClipArgs a) {
  float coefficient;
  if constexpr (INLINE) {
    __shared__ double part[4];
    auto load = [&](int i) { return a.sums[i]; };
    total_of_sums(a.nsums, load, part);
    __syncthreads();
    const float2 r = norm_and_coefficient(a, part);
    coefficient = r.y;
    const int extra = (int)blockIdx.x - a.nchunks;
    if (extra >= 0) {
      const int first = extra * kClipStatsTensors;
      tensor_norms(a, first + __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64), 4,
                   min(a.ntensors, first + kClipStatsTensors), load);
      if (extra == 0 && threadIdx.x == 0) {
        a.stats[0] = r.x;
        a.stats[1] = r.y;
      }
      return;
    }
  } else {
    coefficient = a.stats[1];
  }
  const int chunk = a.nchunks - 1 - (int)blockIdx.x;
  const ClipTensor t = a.tensors[a.chunk_map[chunk]];
  if (!t.in || !t.out) return;  // bound without outputs, or never
  const int64_t e0 = (int64_t)(chunk - t.first_chunk) * kClipChunk;
  const float c = coefficient * a.scale;
  switch (t.in_dtype * 3 + t.out_dtype) {
    case kF32 * 3 + kF32: return scale_chunk<kF32, kF32, NTL, NTS>(t, e0, c);
    case kF32 * 3 + kBF16: return scale_chunk<kF32, kBF16, NTL, NTS>(t, e0, c);
    case kF32 * 3 + kF16: return scale_chunk<kF32, kF16, NTL, NTS>(t, e0, c);
    case kBF16 * 3 + kF32: return scale_chunk<kBF16, kF32, NTL, NTS>(t, e0, c);
    case kBF16 * 3 + kBF16: return scale_chunk<kBF16, kBF16, NTL, NTS>(t, e0, c);
    case kBF16 * 3 + kF16: return scale_chunk<kBF16, kF16, NTL, NTS>(t, e0, c);
    case kF16 * 3 + kF32: return scale_chunk<kF16, kF32, NTL, NTS>(t, e0, c);
    case kF16 * 3 + kBF16: return scale_chunk<kF16, kBF16, NTL, NTS>(t, e0, c);
    default: return scale_chunk<kF16, kF16, NTL, NTS>(t, e0, c);
  }
}

hipError_t launch_clip_bind(ClipTensor* tensors, const ClipPointers& p, int first, int n, hipStream_t s) {
  hipLaunchKernelGGL(k_clip_bind, dim3(1), dim3(256), 0, s, tensors, p, first, n);
  return hipGetLastError();
}

static hipError_t launch_clip_sums(const ClipArgs& a, hipStream_t s) {
  if (a.nsums == 0) return hipSuccess;
  if (a.stream_in)
    hipLaunchKernelGGL(k_clip_sums<true>, dim3((unsigned)a.nsums), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(k_clip_sums<false>, dim3((unsigned)a.nsums), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_clip_norm(const ClipArgs& a, hipStream_t s) {
  if (hipError_t e = launch_clip_sums(a, s); e != hipSuccess) return e;
  hipLaunchKernelGGL(k_clip_final, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_clip_apply(const ClipArgs& a, hipStream_t s) {
  if (a.nchunks == 0) return launch_clip_norm(a, s);
  const dim3 b(256);
  if (a.nsums <= kClipInlineSums && a.nchunks <= kClipInlineChunks) {  // (far below the streaming loads' size)
    if (hipError_t e = launch_clip_sums(a, s); e != hipSuccess) return e;
    const dim3 g((unsigned)(a.nchunks + (a.ntensors - 1) / kClipStatsTensors + 1));
    if (a.stream_out)
      hipLaunchKernelGGL((k_clip_apply<false, true, true>), g, b, 0, s, a);
    else
      hipLaunchKernelGGL((k_clip_apply<false, false, true>), g, b, 0, s, a);
    return hipGetLastError();
  }
  if (hipError_t e = launch_clip_norm(a, s); e != hipSuccess) return e;
  const dim3 g((unsigned)a.nchunks);
  if (a.stream_in)
    hipLaunchKernelGGL((k_clip_apply<true, true, false>), g, b, 0, s, a);
  else if (a.stream_out)
    hipLaunchKernelGGL((k_clip_apply<false, true, false>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((k_clip_apply<false, false, false>), g, b, 0, s, a);
  return hipGetLastError();
}

}  // namespace psgd
