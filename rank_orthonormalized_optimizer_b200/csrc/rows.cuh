// Device helpers of the row operators: 8 consecutive elements of a row as fp32, and the
// 8-bit form of a block of 32 features.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dion {

// The kernels before this one on the stream have ended and their writes are visible; and: the
// next kernel's CTAs may be set up now (operator.h, launch_after).
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// Raw bits of 8 consecutive elements (16 bytes for the 2-byte types, 32 for fp32, moved at
// once: in two 16-byte halves each access of a warp would touch half of every sector); the
// pointer is aligned to them.  Loaded past L1, where the gains of a norm stay instead.
template <typename T> struct Raw8 { uint4 a; };
template <> struct Raw8<float> { uint4 a, b; };

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void ld_stream32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p) : "memory");
}
__device__ __forceinline__ void st_vec32(void* p, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
__device__ __forceinline__ void st_vec(void* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

template <typename T> __device__ __forceinline__ Raw8<T> load_raw(const T* p) { return {ld_stream(p)}; }
template <> __device__ __forceinline__ Raw8<float> load_raw<float>(const float* p) {
  Raw8<float> r;
  ld_stream32(p, r.a, r.b);
  return r;
}
template <typename T> __device__ __forceinline__ Raw8<T> zero_raw() { return {make_uint4(0, 0, 0, 0)}; }
template <> __device__ __forceinline__ Raw8<float> zero_raw<float>() {
  return {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
}

__device__ __forceinline__ void unpack(const Raw8<float>& r, float* v) {
  v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
  v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
  v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
  v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
}
__device__ __forceinline__ void unpack(const Raw8<__nv_bfloat16>& r, float* v) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw8<__half>& r, float* v) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void store8(float* p, const float* v) {
  st_vec32(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])),
           make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
}
__device__ __forceinline__ uint4 pack8(const float* v, __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack8(const float* v, __half) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) { st_vec(p, pack8(v, __nv_bfloat16())); }
__device__ __forceinline__ void store8(__half* p, const float* v) { st_vec(p, pack8(v, __half())); }

// ---- 8-bit form: a block of 32 features x_i is e4m3(x_i 2^-e) and the byte e + 127, e the
// smallest exponent with max|x_i| <= 448 2^e (448 = 1.75 2^8 is e4m3's largest value), kept in
// [-117, 119]: then e4m3's smallest step 2^-9 2^e is a normal bf16 number and 448 2^e is finite,
// and every value is exact in bf16.  Rounding is to nearest even: half a step of 3 fraction
// bits, 2^-4 relative, which is what 8 bits cost.  Magnitudes above 448 2^119 (2.98e38, the top
// quarter of fp32's last binade) are cut to it.
// A block that holds an infinity or a NaN is marked 255: all of it reads as NaN.
constexpr uint32_t kInfBits = 0x7f800000u;

// max over the block of the magnitudes' bits (they order as the values do, NaN on top)
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// the same over 8 values as they are stored: 16-bit magnitudes order by their bits, too
__device__ __forceinline__ uint32_t abs_bits8(const Raw8<float>& r) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, w[i] & 0x7fffffffu);
  return top;
}
template <typename T>
__device__ __forceinline__ uint32_t abs_bits8(const Raw8<T>& r) {
  constexpr uint32_t M = 0x7fff7fffu;
  const uint32_t two = __vmaxu2(__vmaxu2(r.a.x & M, r.a.y & M), __vmaxu2(r.a.z & M, r.a.w & M));
  const uint16_t one = (uint16_t)max(two & 0xffffu, two >> 16);
  return __float_as_uint(to_float(*reinterpret_cast<const T*>(&one)));
}

__device__ __forceinline__ int act_exponent(uint32_t top) {
  const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -117), 119);
}
// 2^-e for e in [-117, 119]
__device__ __forceinline__ float act_unscale(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// two values to two e4m3 bytes (lo in bits 0..7)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^(E - 127) of a scale byte; 255 is NaN
__device__ __forceinline__ float act_scale(uint32_t E) {
  return __uint_as_float(E == 255u ? 0x7fc00000u : E == 0u ? 0x00400000u : E << 23);
}
// e4m3 pair to fp32 (exact)
__device__ __forceinline__ float2 e4m3x2_float(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace dion
