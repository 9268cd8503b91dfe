// product_args.hpp -- kernel arguments of the epilogue products: dense ones,
// products over groups of rows, and products that sum over a group's rows.
#pragma once

#include "common.hpp"

namespace sg {

constexpr int kMaxGroups = 1024;

enum ProductMode {
  kDense = 0,      // C = op(A)·op(B)
  kRowGroups = 1,  // rows offsets[g] .. offsets[g+1]-1 of A and C with B_g
  kSumGroups = 2   // C_g = the sum over k = offsets[g] .. offsets[g+1]-1
};

struct ProductArgs {
  const float* A;
  const float* B;
  float* C;
  int M, N, K;                         // kSumGroups: K is unused
  int lda, ldb, ldc;
  // Epilogue.
  const float* bias;
  const float* residual;
  float* preact;
  int64_t ld_bias;                     // group to group
  int ldr, ldp, act;
  // Groups.
  int mode, groups, rows;              // rows: what offsets are clamped to
  const int32_t* offsets;
  int64_t stride_b, stride_c;          // group to group, floats
  // Tiles and splits, as in GemmArgs.
  int tiles_m, tiles_n, group_m;
  int splits, k_split;
  float* W;
};

// Group g's range, clamped to 0 .. rows and not negative: bad offsets give
// wrong sums but no access outside the operands.
__device__ __forceinline__ void group_range(const int32_t* offsets, int g, int rows, int& begin,
                                            int& end) {
  begin = min(max(offsets[g], 0), rows);
  end = min(max(offsets[g + 1], begin), rows);
}

// Inclusive sum over the lanes of a wave, by row shifts and row broadcasts.
__device__ __forceinline__ int scan64(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31
  return v;
}

}  // namespace sg
