// Softmax cross entropy over a large vocabulary: arguments and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "psgd_mx.h"

namespace psgd {

// One call: T tokens, V words, D values a token.
struct XentArgs {
  int64_t t, v, d;
  int dtype;  // of x, w, bias, dx, dbias
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const void* bias;  // V, or null
  const int64_t* targets;
  int64_t ignore;
  const float* weights;  // a token's weight in the gradients, or null: ones
  float scale;
  bool mean;  // scale over the number of tokens that are not ignored
  float *loss, *lse;
  void* dx;  // null: not wanted
  int64_t lddx;
  void* dw;
  int dw_dtype;
  int64_t lddw;
  void* dbias;
  bool accumulate;  // dw and dbias are added to
};

// Where a call keeps what in its workspace (bytes from its start; 0 bytes of
// what it does not need), and how it splits its work.
struct XentLayout {
  bool pack_x, pack_w;
  int parts;                 // pieces of a value: 2 fp16 ones for fp32, else 1
  int64_t dp;                // row stride of packed operands
  int64_t vp;                // row stride of the probabilities
  int64_t block;             // tokens whose probabilities are held at a time
  int seg_shift;             // columns that share a maximum: 32 (few tokens) or 64
  int64_t nseg;
  int64_t dx_splits;         // pieces of the vocabulary that dx is summed in
  size_t scalars, partmax, xrow, rows, x, w, stats, target, sums, e, g, db, dbs, dxp, dwp, bytes;
};
XentLayout xent_layout(const XentArgs& a, bool train);
hipError_t launch_xent(const XentArgs& a, const XentLayout& l, bool train, void* ws, hipStream_t s);
constexpr size_t kXentTotalBytes = 4096;  // of its workspace
hipError_t launch_xent_total(const float* loss, const int64_t* targets, int64_t t, int64_t ignore, bool mean,
                             float* total, void* ws, hipStream_t s);
hipError_t launch_xent_scale(const void* in, int dtype, int64_t n, const float* factor, void* out, hipStream_t s);

}  // namespace psgd
