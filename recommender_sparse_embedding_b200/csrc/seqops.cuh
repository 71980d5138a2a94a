// seqops.cuh -- shared by the sequence operators (embed.cu, norm.cu, attend*.cu):
// element types, vector loads and stores with conversion, the status word.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace recis {

// device status word of the sequence operators on the current device (NULL:
// its address could not be had)
int* sequence_status();

constexpr int64_t align256(int64_t b) { return (b + 255) & ~(int64_t)255; }
inline bool float_type(int t) { return t == RECIS_F32 || t == RECIS_BF16 || t == RECIS_F16; }
inline int type_bytes(int t) { return t == RECIS_F32 ? 4 : 2; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// two fp32 values packed to 16 bits each (lo in the low half)
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// V consecutive elements at p as they lie in memory: V = 8 (16- or 32-byte
// loads; p aligned to 16 bytes) or V = 1.
template <typename T, int V>
struct RawVec;
template <typename T>
struct RawVec<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = to_f32(v); }
};
template <>
struct RawVec<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};
template <typename T>
struct RawVec16 {
  uint4 a;
  __device__ __forceinline__ void load(const T* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    const float2 x = unpack2<T>(a.x), y = unpack2<T>(a.y), z = unpack2<T>(a.z), w = unpack2<T>(a.w);
    f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
    f[4] = z.x; f[5] = z.y; f[6] = w.x; f[7] = w.y;
  }
};
template <>
struct RawVec<__nv_bfloat16, 8> : RawVec16<__nv_bfloat16> {};
template <>
struct RawVec<__half, 8> : RawVec16<__half> {};

template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[1]) { *p = from_f32<T>(f[0]); }
__device__ __forceinline__ void store_vec(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                                            pack2<T>(f[6], f[7]));
}

// f(T{}) with the element type of a type code
template <typename F>
auto with_type(int t, F&& f) {
  switch (t) {
    case RECIS_BF16: return f(__nv_bfloat16());
    case RECIS_F16: return f(__half());
    default: return f(float());
  }
}

// rows of `stride` elements of type t from p: every row start aligned to 16 bytes
inline bool rows_aligned16(const void* p, int64_t stride, int t) {
  return !misaligned(p, 16) && (stride * type_bytes(t)) % 16 == 0;
}

}  // namespace recis
