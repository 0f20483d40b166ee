// Global gradient norm and clipping over a list of tensors: host object,
// device tables and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <vector>

#include "../../include/psgd.h"

namespace psgd {

// Elements that a workgroup handles at a time: 32 of each of its 256 threads.
constexpr int kClipChunk = 8192;
// Workgroups of the norm's pass over the whole list (and one more per tensor
// at most): nearly four on each compute unit, each with 32 KB under way, are
// enough for the memory, and their sums few (667e6 bf16 values: 876 us with the
// writing pass, 885 with 4096 workgroups).
constexpr int kClipSumGroups = 960;

// Gradients and outputs of more bytes than this do not stay side by side in the
// 256 MB last level of cache.
constexpr int64_t kClipCacheBytes = int64_t(192) << 20;

// Up to this many sums of squares, and workgroups that read them all, the
// writing pass adds them by itself.
constexpr int kClipInlineSums = 2048;
constexpr int kClipInlineChunks = 8192;
constexpr int kClipStatsTensors = 8;  // tensors whose norms one of its workgroups then writes

struct ClipTensor {
  const void* in;
  void* out;
  int64_t numel;
  int32_t in_dtype, out_dtype;
  int32_t first_sum, nsums;  // its workgroups of the norm's pass (each takes every nsums-th chunk)
  int32_t first_chunk;       // its workgroups of the writing pass, one per chunk
  int32_t pad;
};

// Workspace: [tensors][norm workgroup -> tensor][writing workgroup -> tensor][sums of squares, fp64].
struct ClipLayout {
  size_t sum_map_off, chunk_map_off, sums_off, bytes;
};

constexpr int kClipBindPairs = 240;  // pointer pairs one launch carries in its arguments
struct ClipPointers {
  const void* in[kClipBindPairs];
  void* out[kClipBindPairs];
};

struct ClipArgs {
  const ClipTensor* tensors;
  const int32_t *sum_map, *chunk_map;
  double* sums;
  int32_t ntensors, nsums, nchunks;
  bool stream_in, stream_out;  // more bytes than the caches keep: streaming loads, streaming stores
  float scale, max_norm;
  float* stats;
};

hipError_t launch_clip_bind(ClipTensor* tensors, const ClipPointers& p, int first, int n, hipStream_t s);
hipError_t launch_clip_norm(const ClipArgs& a, hipStream_t s);
// The norm, and the clipped gradients.
hipError_t launch_clip_apply(const ClipArgs& a, hipStream_t s);

}  // namespace psgd

struct psgd_clip {
  std::vector<psgd::ClipTensor> tensors;
  std::vector<int32_t> sum_map, chunk_map;
  std::vector<uint8_t> tables;  // tensors and maps, as uploaded
  psgd::ClipLayout lay{};
  bool stream_in = false, stream_out = false;  // stream_in implies stream_out
};
