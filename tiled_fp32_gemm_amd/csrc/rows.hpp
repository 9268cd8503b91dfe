// rows.hpp -- four floats of a row at any 4-byte alignment.
//
// These are global accesses: unlike the buffer form, their 16-byte kind takes
// any 4-byte aligned address.
#pragma once

#include "common.hpp"

namespace sg {

// Four floats at any 4-byte aligned address.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// Up to n (1..4) floats at p, zeros past them; and the same stored.
__device__ __forceinline__ f32x4 load_upto(const float* p, int n) {
  if (n >= 4) return *reinterpret_cast<const f32x4u*>(p);
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  v[0] = p[0];
  if (n > 1) v[1] = p[1];
  if (n > 2) v[2] = p[2];
  return v;
}
// load_upto for data that is read once.
__device__ __forceinline__ f32x4 load_upto_once(const float* p, int n) {
  if (n >= 4) return __builtin_nontemporal_load(reinterpret_cast<const f32x4u*>(p));
  return load_upto(p, n);
}
__device__ __forceinline__ void store_upto(float* p, int n, f32x4 v) {
  if (n >= 4) {
    *reinterpret_cast<f32x4u*>(p) = v;
    return;
  }
  p[0] = v[0];
  if (n > 1) p[1] = v[1];
  if (n > 2) p[2] = v[2];
}

// store_upto for data that is not read back soon.
__device__ __forceinline__ void store_upto_once(float* p, int n, f32x4 v) {
  if (n >= 4) __builtin_nontemporal_store(f32x4u(v), reinterpret_cast<f32x4u*>(p));
  else store_upto(p, n, v);
}

}  // namespace sg
