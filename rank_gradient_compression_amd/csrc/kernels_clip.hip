// Global gradient norm over many tensors, and clipping (gfx950, wave64).
//
//   n_t = || scale * g_t ||,  N = sqrt(sum n_t^2),  c = min(1, max_norm / (N + 1e-6)),
//   out_t = scale * c * g_t
//
// Three launches: sums of squares per tile, their fixed-order sum (one
// workgroup), the scaled write.  Squares are summed in fp64: an fp32 square
// overflows from 1.8e19 on, and the one conversion per element is hidden
// behind the reads.  Bound: HBM, the gradients read twice (once if the last
// level of cache holds them) and written once.  Sums are made in a fixed
// order without atomics, so a repeated call agrees bit for bit.

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

// Calls f(i, values, valid) for every group of E consecutive elements of the
// tile [e0, e1) that this thread takes; 16-byte loads where the address allows.
template <int DT, int E, int UNROLL, typename F>
__device__ __forceinline__ void walk(const void* base, int64_t e0, int64_t e1, F f) {
  using T = typename Elem<DT>::type;
  const T* g = static_cast<const T*>(base);
  const bool wide = ((uintptr_t)(g + e0) & (E * sizeof(T) - 1)) == 0;
  for (int64_t i0 = e0; i0 < e1; i0 += 256 * E * UNROLL) {
    T v[UNROLL][E];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t i = i0 + (u * 256 + (int)threadIdx.x) * E;
      if (wide && i + E <= e1) {
        __builtin_memcpy(v[u], __builtin_assume_aligned(g + i, E * sizeof(T)), E * sizeof(T));
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) v[u][j] = i + j < e1 ? g[i + j] : (T)0;
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t i = i0 + (u * 256 + (int)threadIdx.x) * E;
      float x[E];
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = Elem<DT>::up(v[u][j]);
      if (i < e1) f(i, x, (int)min((int64_t)E, e1 - i));
    }
  }
}

__device__ __forceinline__ double block_sum(double s) {
  __shared__ double w[4];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  return (w[0] + w[1]) + (w[2] + w[3]);
}

__global__ __launch_bounds__(256) void k_clip_sums(ClipArgs a) {
  const int tile = blockIdx.x;
  const ClipTensor t = a.tensors[a.map[tile]];
  const int64_t e0 = (int64_t)(tile - t.first_tile) * a.tile, e1 = min(t.numel, e0 + a.tile);
  double s = 0;
  auto add = [&](int64_t, auto& x, int) {
    for (float v : x) s = fma((double)v, (double)v, s);
  };
  if (t.in_dtype == kF32)
    walk<kF32, 4, 4>(t.in, e0, e1, add);
  else if (t.in_dtype == kBF16)
    walk<kBF16, 8, 4>(t.in, e0, e1, add);
  else
    walk<kF16, 8, 4>(t.in, e0, e1, add);
  s = block_sum(s);
  if (threadIdx.x == 0) a.sums[tile] = s;
}

// One workgroup: wavefront w sums the tiles of tensors w, w + 16, ... and
// the tensors' sums are added in order.
__global__ __launch_bounds__(1024) void k_clip_final(ClipArgs a) {
  __shared__ double part[16];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  double tot = 0;
  for (int t = w; t < a.ntensors; t += 16) {
    const int f = a.tensors[t].first_tile, n = a.tensors[t].ntiles;
    double s = 0;
    for (int i = lane; i < n; i += 64) s += a.sums[f + i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    tot += s;
    if (lane == 0) a.stats[2 + t] = (float)(sqrt(s) * fabs((double)a.scale));
  }
  if (lane == 0) part[w] = tot;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0;
    for (int i = 0; i < 16; ++i) s += part[i];
    const double norm = sqrt(s) * fabs((double)a.scale);
    const double c = (double)a.max_norm / (norm + 1e-6);
    a.stats[0] = (float)norm;
    a.stats[1] = c < 1.0 || c != c ? (float)c : 1.f;  // NaN stays NaN
  }
}

template <int DT, int E>
__device__ __forceinline__ void store_group(void* base, int64_t i, const float (&x)[E], float c, int n) {
  using T = typename Elem<DT>::type;
  T* o = static_cast<T*>(base) + i;
  T v[E];
#pragma unroll
  for (int j = 0; j < E; ++j) v[j] = Elem<DT>::down(x[j] * c);
  if (n == E && ((uintptr_t)o & (E * sizeof(T) - 1)) == 0) {
    __builtin_memcpy(__builtin_assume_aligned(o, E * sizeof(T)), v, E * sizeof(T));
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < n) o[j] = v[j];
  }
}

__global__ __launch_bounds__(256) void k_clip_apply(ClipArgs a) {
  const int tile = blockIdx.x;
  const ClipTensor t = a.tensors[a.map[tile]];
  const int64_t e0 = (int64_t)(tile - t.first_tile) * a.tile, e1 = min(t.numel, e0 + a.tile);
  const float c = a.stats[1] * a.scale;
  auto put = [&](int64_t i, auto& x, int n) {
    if (t.out_dtype == kF32)
      store_group<kF32>(t.out, i, x, c, n);
    else if (t.out_dtype == kBF16)
      store_group<kBF16>(t.out, i, x, c, n);
    else
      store_group<kF16>(t.out, i, x, c, n);
  };
  if (t.in_dtype == kF32)
    walk<kF32, 4, 4>(t.in, e0, e1, put);
  else if (t.in_dtype == kBF16)
    walk<kBF16, 8, 4>(t.in, e0, e1, put);
  else
    walk<kF16, 8, 4>(t.in, e0, e1, put);
}

hipError_t launch_clip_bind(ClipTensor* tensors, const ClipPointers& p, int first, int n, hipStream_t s) {
  hipLaunchKernelGGL(k_clip_bind, dim3(1), dim3(256), 0, s, tensors, p, first, n);
  return hipGetLastError();
}

hipError_t launch_clip_norm(const ClipArgs& a, hipStream_t s) {
  if (a.ntiles > 0) {
    hipLaunchKernelGGL(k_clip_sums, dim3((unsigned)a.ntiles), dim3(256), 0, s, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_clip_final, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_clip_apply(const ClipArgs& a, hipStream_t s) {
  if (a.ntiles == 0) return hipSuccess;
  hipLaunchKernelGGL(k_clip_apply, dim3((unsigned)a.ntiles), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace psgd
