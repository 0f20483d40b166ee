// Global gradient norm and clipping over a list of tensors: host object,
// device tables and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <vector>

#include "../../include/psgd.h"

namespace psgd {

struct ClipTensor {
  const void* in;
  void* out;
  int64_t numel;
  int32_t in_dtype, out_dtype;
  int32_t first_tile, ntiles;
};

// Workspace: [tensors][tile map][tile sums of squares, fp64].
struct ClipLayout {
  size_t map_off, sums_off, bytes;
};

constexpr int kClipBindPairs = 240;  // pointer pairs one launch carries in its arguments
struct ClipPointers {
  const void* in[kClipBindPairs];
  void* out[kClipBindPairs];
};

struct ClipArgs {
  const ClipTensor* tensors;
  const int32_t* map;  // tile -> tensor
  double* sums;
  int32_t ntensors, ntiles;
  int32_t tile;  // elements of a tile
  float scale, max_norm;
  float* stats;
};

hipError_t launch_clip_bind(ClipTensor* tensors, const ClipPointers& p, int first, int n, hipStream_t s);
hipError_t launch_clip_norm(const ClipArgs& a, hipStream_t s);
hipError_t launch_clip_apply(const ClipArgs& a, hipStream_t s);

}  // namespace psgd

struct psgd_clip {
  std::vector<psgd::ClipTensor> tensors;
  std::vector<int32_t> map;
  std::vector<uint8_t> tables;  // tensors + map, as uploaded
  psgd::ClipLayout lay{};
  int32_t tile = 0;
};
