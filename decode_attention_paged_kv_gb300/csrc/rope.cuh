// rope.cuh -- rows of new tokens taken 16 channels a thread, and their rotation by the
// position's angles.
#pragma once

#include <stdint.h>

#include "dkv_device.cuh"

namespace dkv {

// The 16 channels of a thread: 8 from c1 on and 8 from c2 on.
struct Chunks {
  int c1, c2;
};
template <bool IL>
__device__ __forceinline__ Chunks chunks_of(int j, int r, bool rotated) {
  if (!IL && rotated) return {8 * j, r / 2 + 8 * j};
  return {16 * j, 16 * j + 8};
}

struct Raw {
  uint4 u, w;
};
__device__ __forceinline__ Raw load_raw(const uint16_t* row, Chunks c) {
  return {*reinterpret_cast<const uint4*>(row + c.c1), *reinterpret_cast<const uint4*>(row + c.c2)};
}
template <bool F16>
__device__ __forceinline__ void widen(const Raw& r, float (&x)[16]) {
  const uint32_t v[8] = {r.u.x, r.u.y, r.u.z, r.u.w, r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = lo16<F16>(v[i]);
    x[2 * i + 1] = hi16<F16>(v[i]);
  }
}

template <bool F16>
__device__ __forceinline__ void store16(uint16_t* row, Chunks c, const float (&x)[16]) {
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = pack2<F16>(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(row + c.c1) = make_uint4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<uint4*>(row + c.c2) = make_uint4(v[4], v[5], v[6], v[7]);
}

// cos and sin of the 8 pairs of slot j at position pos.
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ Angles angles_of(const float* cos, const float* sin, int r, int pos,
                                            int j) {
  Angles t;
  const int64_t at = static_cast<int64_t>(pos) * (r / 2) + 8 * j;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(cos + at + i));
    const float4 w = __ldg(reinterpret_cast<const float4*>(sin + at + i));
    t.c[i] = u.x, t.c[i + 1] = u.y, t.c[i + 2] = u.z, t.c[i + 3] = u.w;
    t.s[i] = w.x, t.s[i + 1] = w.y, t.s[i + 2] = w.z, t.s[i + 3] = w.w;
  }
  return t;
}
// Rotate a slot's 8 pairs.  (Intrinsics: no contraction into fused
// multiply-adds, so a step has one result whatever the compiler.)
template <bool IL>
__device__ __forceinline__ void rotate16(const Angles& t, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& p = x[IL ? 2 * i : i];
    float& q = x[IL ? 2 * i + 1 : 8 + i];
    const float u = p, w = q;
    p = __fsub_rn(__fmul_rn(u, t.c[i]), __fmul_rn(w, t.s[i]));
    q = __fadd_rn(__fmul_rn(w, t.c[i]), __fmul_rn(u, t.s[i]));
  }
}

}  // namespace dkv
