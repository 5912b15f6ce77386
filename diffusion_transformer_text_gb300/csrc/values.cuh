// Groups of 8 consecutive values of a tensor, loaded to and stored from fp32 registers.
#pragma once
#include "ptx.cuh"

namespace qi {

// 8 values of a 16-bit type from 16 bytes
template <typename T>
__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]);
template <>
__device__ __forceinline__ void unpack8<__half>(uint4 w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(uint4 w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&v)[8]) {
  unpack8<T>(*reinterpret_cast<const uint4*>(src), v);
}
template <>
__device__ __forceinline__ void load8(const float* src, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ uint4 pack8(const __half*, const float (&v)[8]) {
  return make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack8(const __nv_bfloat16*, const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(dst) = pack8(dst, v);
}

// 8 values in 16-byte pieces: one of a 16-bit type, two of fp32
template <typename T>
__device__ __forceinline__ void from_pieces(const uint4 (&u)[1], float (&v)[8]) {
  unpack8<T>(u[0], v);
}
template <typename T>
__device__ __forceinline__ void from_pieces(const uint4 (&u)[2], float (&v)[8]) {
  v[0] = __uint_as_float(u[0].x), v[1] = __uint_as_float(u[0].y), v[2] = __uint_as_float(u[0].z);
  v[3] = __uint_as_float(u[0].w), v[4] = __uint_as_float(u[1].x), v[5] = __uint_as_float(u[1].y);
  v[6] = __uint_as_float(u[1].z), v[7] = __uint_as_float(u[1].w);
}

}  // namespace qi
