// Rows of the caller's tensors as the cache's and the rotary kernels take them: eight
// values of a lane, loaded, looked at and stored.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"

namespace tld {

// The largest of three magnitudes; NaN if one is.
__device__ __forceinline__ float largest(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// The larger magnitudes of two bf16 pairs (with some sign); NaN if either is.
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// Two fp32 numbers handled by one instruction.
struct Two {
  uint64_t w;
  __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit Two(float a) : Two(a, a) {}
  __device__ __forceinline__ float2 get() const {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(w));
    return y;
  }
};
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a.w) : "l"(b.w), "l"(c.w));
  return a;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.w) : "l"(b.w));
  return a;
}

// Eight values of the caller's type as they are loaded, their fp32 values, and
// the largest magnitude among them and those of four neighbouring lanes (NaN if
// one of them is).
template <class T>
struct Eight;
template <>
struct Eight<float> {
  float4 u, w;
  __device__ __forceinline__ void load(const float* p) {
    u = reinterpret_cast<const float4*>(p)[0], w = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    u = make_float4(x[0], x[1], x[2], x[3]), w = make_float4(x[4], x[5], x[6], x[7]);
  }
  // the largest magnitude of this lane's eight alone
  __device__ __forceinline__ float top_here() const {
    return largest(largest(largest(u.x, u.y, u.z), u.w, w.x), largest(w.y, w.z, w.w), 0.f);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
  }
  __device__ __forceinline__ float top() const {
    float y = largest(largest(largest(u.x, u.y, u.z), u.w, w.x), w.y, w.z);
    y = largest(y, w.w, __shfl_xor_sync(0xffffffffu, largest(y, w.w, 0.f), 1));
    return largest(y, __shfl_xor_sync(0xffffffffu, y, 2), 0.f);
  }
};
template <>
struct Eight<uint16_t> {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float top_here() const {
    const uint32_t y = larger2(larger2(u.x, u.y), larger2(u.z, u.w));
    return largest(bf16lo(y), bf16hi(y), 0.f);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = bf16lo(u.x), x[1] = bf16hi(u.x), x[2] = bf16lo(u.y), x[3] = bf16hi(u.y);
    x[4] = bf16lo(u.z), x[5] = bf16hi(u.z), x[6] = bf16lo(u.w), x[7] = bf16hi(u.w);
  }
  __device__ __forceinline__ float top() const {
    uint32_t y = larger2(larger2(u.x, u.y), larger2(u.z, u.w));
    y = larger2(y, __shfl_xor_sync(0xffffffffu, y, 1));
    y = larger2(y, __shfl_xor_sync(0xffffffffu, y, 2));
    return largest(bf16lo(y), bf16hi(y), 0.f);
  }
};
// wide: p is a multiple of 32 bytes, which one store then writes whole; two
// stores of half a sector each take longer (8185 rows of 32 heads of 128 read
// from 4-bit pages: 81 us, against 51).
__device__ __forceinline__ void store8(float* p, const float (&x)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}
__device__ __forceinline__ uint32_t pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8], bool) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pair(x[0], x[1]), pair(x[2], x[3]), pair(x[4], x[5]), pair(x[6], x[7]));
}

// One value of the caller's type, as fp32 and from it.
__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ void put(float& to, float x) { to = x; }
__device__ __forceinline__ void put(uint16_t& to, float x) { to = f32_to_bf16_bits(x); }

constexpr int kSms = 152;  // of a GB300

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer

}  // namespace tld
