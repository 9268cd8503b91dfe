// xent_args.hpp -- kernel arguments of the cross entropy over a product.
#pragma once

#include <float.h>

#include "host.hpp"
#include "product_args.hpp"

namespace sg {

constexpr float kLog2e = 1.44269502f;

// What a row's powers of two are relative to, from its largest logit: finite, so that
// a row of infinities subtracts no infinity from itself.
__device__ __forceinline__ float xent_reference(float m) {
  return fminf(fmaxf(m * kLog2e, -FLT_MAX), FLT_MAX);
}

// A token's target, or -1 where it has none.
struct Targets {
  const void* ids;
  int wide;        // int64, else int32
  int V;

  __device__ __forceinline__ int of(int64_t t) const {
    const int64_t id = wide ? static_cast<const int64_t*>(ids)[t]
                            : (int64_t)static_cast<const int32_t*>(ids)[t];
    return id >= 0 && id < V ? (int)id : -1;
  }
};

// What the gradient needs of a row: one load (workspaces are aligned to 4 bytes).  An
// infinite lse leaves no rest, so that exp(z - lse) is 0 at every finite z.
struct XentRow {
  int target;
  float ref, rest;   // lse times log2 e, rounded, and what that left
  float grad;        // dloss
};
__device__ __forceinline__ XentRow xent_row(int target, float lse, float dloss) {
  const float ref = lse * kLog2e;
  return {target, ref, fabsf(ref) < INFINITY ? fmaf(lse, kLog2e, -ref) : 0.0f, dloss};
}

// The rows with a target, one after another ("kept" rows), made on the device.
// Token t is row place[t], or -1.
struct XentRows {
  int32_t* offsets;   // 0 and how many: one group of kRowGroups
  int32_t* place;
  int32_t* target;    // forward: of each kept row
  XentRow* row;       // backward
  float* X;           // the rows, T x H
};

struct XentProductArgs : ProductArgs {
  // Forward.
  Targets targets;
  const int32_t* target;  // of each row; null: row r is token r, see targets
  float* max;             // [strip][row]: a row's largest logit in a strip of columns
  float* sum;             // and the sum of exp(logit) over its exp, both as powers of two
  float* hit;             // [row]: the target's logit
  int ld_strip;           // rows
  int turn;               // tiles begin at slabs of their own
  // Backward.
  const XentRow* row;
  int column0;            // the first column's number in the vocabulary
};

// Few rows: from a product's planes (product_planes.hpp).
struct XentPlanesArgs {
  const float* planes;    // [plane][rows][N]
  float* dZ;              // backward: may be the first plane; leading dimension N
  Targets targets;        // forward: row r is token r
  float* max;             // [strip of 256 columns][row]
  float* sum;
  float* hit;
  const int32_t* offsets;   // backward: how many rows
  const XentRow* row;       // null: row r is token r, see targets and
  const float* lse;
  const float* dloss;
  int rows, N, count, column0;
};

// Few rows (kernel_xent_few.hpp).  In rows without a target P and Q do not
// count, whatever they hold.
struct XentFewArgs {
  Targets targets;
  const float* B;         // as it is stored, rows x cols
  const float* P;         // T x rows
  const float* Q;         // T x cols
  float* D;               // rows x cols: P'Q; null: not wanted
  float* planes;          // parts of P·B or Q·B', T x cols or rows; null: not wanted
  int T, rows, cols, ldb, ldp, ldq, ldd;
  int part;               // rows of B of a workgroup
  int blocks;             // workgroups that take the same rows
};

struct XentFewSumArgs {
  Targets targets;
  const float* planes;    // [plane][T][H]
  float* dX;              // 0 in rows without a target
  int64_t lddx;
  int T, H, count;
};

struct XentPlaceArgs {
  Targets targets;
  XentRows rows;
  const float* lse;      // null: forward
  const float* dloss;
  int64_t T, chunk;      // tokens of a workgroup
  const float* X;        // xent_gather_kernel copies its rows too
  int64_t ldx;
  int H;
};

struct XentLossArgs {
  Targets targets;
  const int32_t* place;   // null: token t is row t
  const float* max;
  const float* sum;
  const float* hit;
  float* loss;
  float* lse;             // null: not wanted
  int64_t T;
  int strips, ld_strip;
};

// A tile of the product with either epilogue.
struct XentVariant {
  host::TileCost cost;
  int strip;                            // columns of a wave
  void (*stats)(XentProductArgs);
  void (*grad)(XentProductArgs);
};

constexpr int kXentVariants = 7;
const XentVariant* xent_variants_ff();   // B is V x H
const XentVariant* xent_variants_fs();   // B is H x V

}  // namespace sg
