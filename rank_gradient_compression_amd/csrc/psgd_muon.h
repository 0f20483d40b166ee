// Orthogonalised updates by Newton-Schulz products: tables and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <vector>

#include "psgd_mx.h"

namespace psgd {

// One matrix of a group, as the kernels' arguments carry it.
struct MuonMat {
  const void* grad;
  float* mom;   // r x c, or null
  void* param;  // or null
  void* upd;    // or null
  uint16_t *x0, *x1;  // X before and after a step: two fp16 planes of r x ldx
  uint16_t *a, *b;    // A and B: `pieces` fp16 planes of k x ldk, k = min(r, c)
  int64_t ldg, ldp, ldu;
  int32_t r, c;
  float step;              // lr times the matrix's own scale
  int32_t sum0, nsums;     // its workgroups of the norm
  int32_t start0;          // its first workgroup of the first X
  int32_t sym0, full0;     // its first tile of k x k (on and above the diagonal), of r x c
  uint8_t gdt, pdt, udt, pieces;
};
static_assert(sizeof(MuonMat) == 128, "what the kernels' arguments hold");
constexpr int kMuonGroup = 28;  // matrices of a launch (its arguments hold 4 KB)

struct MuonArgs {
  MuonMat mat[kMuonGroup];
  int32_t n;
  bool nesterov, last;
  float mu, decay;   // momentum; what a step leaves of a weight
  float a, b, c, eps;
  float sx, sa, sb;  // powers of two that X, A and B are held times
  double* sums;      // the norm's partial sums of squares
  float* partial;    // tiles' partial sums, where the summed axis is split
  int32_t splits, tiles;  // pieces of the summed axis, tiles of a launch
};

// What the caller gives for one matrix (sizes checked).
struct MuonTensor {
  const void* grad;
  float* mom;
  void *param, *upd;
  int64_t ldg, ldp, ldu, r, c;
  float step;
  int gdt, pdt, udt, pieces;
};
struct MuonOpts {
  float mu, decay, a, b, c, eps;
  int steps;
  bool nesterov;
};
// Powers of two that keep X, A and B within fp16 whatever the matrix; false
// where the polynomial lets singular values grow beyond that.
bool muon_scales(const MuonOpts& o, float* sx, float* sa, float* sb);
size_t muon_workspace(const std::vector<MuonTensor>& t);
hipError_t launch_muon(const std::vector<MuonTensor>& t, const MuonOpts& o, void* ws, hipStream_t s);

}  // namespace psgd
