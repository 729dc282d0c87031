// What the kernels that put new tokens into the cache's pages have in common: a token's place, its rotary phase, and
// 16-byte vectors of either type.
#pragma once

#include "serve.cuh"

namespace dcp {

struct Where {
  int64_t off;   // element offset of the token's row in head 0 of the pool, -1: not stored
  int32_t phase;
  int32_t seq;   // -1: no sequence owns the row
};

// Elements of a 16-byte vector in fp32 and back (bf16: round to nearest even, once).
template <typename T>
struct Elems;
template <>
struct Elems<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& x, float (&y)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = bf16lo(w[i]);
      y[2 * i + 1] = bf16hi(w[i]);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&y)[8]) {
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                      pack_bf16x2(y[6], y[7]));
  }
  static __device__ __forceinline__ float one(const uint4* row, int d) {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[d]);
  }
};
template <>
struct Elems<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4& x, float (&y)[4]) {
    y[0] = __uint_as_float(x.x), y[1] = __uint_as_float(x.y), y[2] = __uint_as_float(x.z), y[3] = __uint_as_float(x.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&y)[4]) {
    return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
  }
  static __device__ __forceinline__ float one(const uint4* row, int d) {
    return reinterpret_cast<const float*>(row)[d];
  }
};

enum Pairs {
  kInterleaved,  // pair (2p, 2p + 1): inside a vector
  kHalfVec,      // pair (p, p + half), half a whole number of vectors: a unit is the two vectors of its pairs
  kHalfAny,      // any other half: partners are read from a copy of the rows in shared memory
};

#ifdef __CUDACC__

// (cos, sin) of the phase in turns, an integer product modulo 2^64, times the amplitude.
__device__ __forceinline__ float2 turn_at(int32_t phase, uint64_t turns, float amplitude) {
  const uint64_t turn = (uint64_t)(int64_t)phase * turns;
  // the fraction of a turn, 32 bits: what fp32 holds of it, and the rest as a first-order correction
  const int32_t fraction = (int32_t)(turn >> 32);
  const float most = (float)fraction;
  const float rest = (float)((int64_t)fraction - (int64_t)most) * (float)(3.14159265358979323846 * 0x1p-31);
  float s, c;
  sincospif(most * 0x1p-31f, &s, &c);
  return make_float2(fmaf(-s, rest, c) * amplitude, fmaf(c, rest, s) * amplitude);
}

#endif

}  // namespace dcp
