// rows.cuh -- 16-byte pieces of bf16 and fp32 rows as fp32 values, shared by
// the row kernels of a training step (train_rows.cu, swiglu_ckpt.cu, route_bwd.cu).
#pragma once

#include "common.cuh"

namespace moe {

// Element type of a row: kN values per 16 bytes.
struct RowBf16 {
  static constexpr int kN = 8;
  __device__ static void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

struct RowF32 {
  static constexpr int kN = 4;
  __device__ static void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Eight e4m3 codes (ascending bytes) as fp32 values, scaled.
__device__ __forceinline__ void e4m3x8(const uint2& q, float s, float (&f)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * j)), __NV_E4M3);
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[4 * i + 2 * j] = v.x * s;
      f[4 * i + 2 * j + 1] = v.y * s;
    }
  }
}

// The sorted row of pair i, or -1: a dropped pair, or an entry outside [0, P)
// (reported, and treated as dropped).
__device__ __forceinline__ int pair_row(const int32_t* __restrict__ inv, long long i, int P, int* status) {
  const int p = __ldg(inv + i);
  if (p < 0) return -1;
  if (p >= P) {
    flag_status(status, MOE_DEV_BAD_INDEX);
    return -1;
  }
  return p;
}

}  // namespace moe
