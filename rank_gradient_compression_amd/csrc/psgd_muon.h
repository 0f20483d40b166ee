// Orthogonalised updates by Newton-Schulz products: tables and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <vector>

#include "psgd_mx.h"

namespace psgd {

// The kernels of a step, each with ranges of its own over a group's matrices.
enum { kNorm, kStart, kGram, kPoly, kUpdate, kMuonKinds, kLast = kMuonKinds };

// Matrices whose shorter side is at most this take two pieces for bfloat16 results
// too: the roundings of one, which many singular values share out, fall on few (one
// piece left 17 x 650 1.8 times as far off as bfloat16's own rounding does, 33 x 650
// 1.4, 48 x 650 1.3, 97 x 650 1.25 times).  64 of 16 x 4096 take 745 us so, with one
// piece 629; 48 x 2600 149, with one 166.
constexpr int kMuonThin = 48;
// Operations of a list's matrices of one piece, up to which they take two beside
// others of two: with two of 27 x 512, three of 1152 x 256 (4.5e9) 225 us so, in
// groups of their own 281; two of 1024 x 1024 (43e9) 388 and 389, four 469 and 435.
constexpr double kMuonJoined = 40e9;
constexpr int kMuonGroup = 27;  // matrices of a group (what the arguments of one launch hold)

// One matrix of a group.
struct MuonMat {
  const void* grad;
  float* mom;   // r x c, or null
  void* param;  // or null
  void* upd;    // or null
  // Places in the workspace, in 256 bytes: X before and after every other step
  // (r rows of two fp16 pieces), A and B (min(r, c) rows of `pieces` fp16 pieces).
  uint32_t x0, x1, a, b;
  int64_t ldg, ldp, ldu;
  int32_t r, c;
  float step;  // lr times the matrix's own scale
  uint8_t gdt, pdt, udt, pieces;
};

// A group's tables, in the workspace: the kernels of a step read them from
// there.  (In every launch's own arguments, which lie in host memory, a search
// over 20 matrices took longer than a small matrix's product.)
struct MuonTable {
  int32_t first[kMuonKinds][kMuonGroup];   // a matrix's first workgroup or tile; past the last matrix INT32_MAX
  int32_t chunk0[kMuonKinds][kMuonGroup];  // its first chunk, alike
  int32_t chunks[kMuonKinds][kMuonGroup];  // chunks of one of its tiles; workgroups of its norm
  MuonMat mat[kMuonGroup];
};
static_assert(sizeof(MuonTable) <= 4080, "what a kernel's arguments hold beside the address");

// How a launch of products is divided.  The first `whole` tiles are a workgroup
// each.  The chunks of the others, from `chunk0` on, are divided evenly among
// `shares` workgroups; a tile that several of them work on is put together by a
// second launch, from the parts that each left in memory (its first and its last
// tile can be such).
struct MuonShares {
  int32_t tiles, whole, shares;
  int32_t chunk0, chunks;
};

struct MuonArgs {
  const MuonTable* table;
  uint8_t* ws;
  bool nesterov, odd;  // odd: X is in x1
  float mu, decay;     // momentum; what a step leaves of a weight
  float a, b, c, eps;
  float own, rest;     // X <- own X + B X, B = b A + c A^2 + rest I: own + rest = a
  float sx, sa, sb;    // powers of two that X, A and B are held times
  double* sums;        // the norm's partial sums of squares
  float* parts;        // tiles' sums of one share
  MuonShares sh;
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
// Steps from which on X's own part is as small as it gets (k_muon_product).
inline bool muon_late(const MuonOpts& o, int step) { return step >= 3 && step + 2 >= o.steps; }
struct MuonTiny {  // matrices that a workgroup each takes whole
  MuonMat mat[kMuonGroup];
  float mu, decay, a, b, c, eps;
  int32_t n, steps;
  bool nesterov;
};
static_assert(sizeof(MuonTiny) <= 4096, "what a kernel's arguments hold");
size_t muon_workspace(const std::vector<MuonTensor>& t);
hipError_t launch_muon(const std::vector<MuonTensor>& t, const MuonOpts& o, void* ws, hipStream_t s);

}  // namespace psgd
