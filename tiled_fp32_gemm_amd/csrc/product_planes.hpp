// product_planes.hpp -- a product left as the partial sums of its split, for kernels
// that add them up as they read them (linear.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace sg {
namespace host {

struct PlanesPlan {
  bool possible;
  bool rows;        // by rows (kernel_rows.hpp), all in one reading of B
  int count;        // planes of M x N floats; 1: the product itself
  double seconds;   // estimated
};

// A·op(B), A of M x K stored M x K, op(B) of K x N; `room`: bytes for the planes, at
// least one.  grouped: of one group of rows (kRowGroups).
PlanesPlan plan_planes(bool grouped, bool trans_b, int64_t M, int64_t N, int64_t K, int64_t room);

// Launches it: `count` planes one after another from `planes` on.  offsets: null, or
// the group's, on the device.
int launch_planes(bool trans_b, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                  const float* B, int64_t ldb, const int32_t* offsets, float* planes,
                  int64_t room, hipStream_t stream, int& count);

}  // namespace host
}  // namespace sg
