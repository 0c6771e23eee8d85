// e4m3 codes with power-of-two scales, and 16-byte accesses of the three
// element types.
//
// A block of values x shares the scale 2^e, e the smallest integer with
// max|x| * 2^-e <= 448 (the largest e4m3 value), held as the byte e + 127
// (hardware UE8M0).  Multiplying by 2^-e is exact, so a code is one
// round-to-nearest-even of its value: the same bits in any wider arithmetic.
// A power of two costs no precision against an arbitrary scale: e4m3 is a
// floating type, so only the position of its 18 binades shifts, by less than 1.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace dllm {

constexpr int kScaleNan = 255;   // scale byte of a block that held a NaN or an infinity

// Scale byte of a block from the bits of its largest |x| (a float's bits
// without the sign: as integers they order like the values, NaN on top).
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return kScaleNan;
  if (amax_bits == 0) return 127;
  const int k = (int)(amax_bits >> 23);             // biased exponent, 0 for a subnormal
  // 448 = 1.75 * 2^8: values up to 1.75 * 2^k fit with e = k - 8
  const int e = k - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  // below 2^-127 (a subnormal block, or one under 2^-118): the byte's floor
  return e < 0 ? 0 : e;
}

// 2^-(byte - 127) and 2^(byte - 127).  Bytes of finite blocks are 0..247, so
// the inverse is a normal float.
__device__ __forceinline__ float scale_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }
__device__ __forceinline__ float scale_value(int byte) {
  return byte == kScaleNan ? __uint_as_float(0x7fffffffu)
                           : byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)byte << 23);
}

// Two floats to two e4m3 codes (a in the low byte), and back.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t cvt_f16x2_e4m3x2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The same on packed halves: a in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t cvt_e4m3x2_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t sub_mul16_f16x2(uint32_t a, uint32_t b) {
  const __half2 d = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b)),
                            __floats2half2_rn(16.0f, 16.0f));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Eight codes (one 8-byte word) of eight values times 2^-e.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = cvt_e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}
__device__ __forceinline__ void decode8(uint2 c, float scale, float (&x)[8]) {
  const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = f16x2_to_f32(cvt_f16x2_e4m3x2((uint16_t)w[i]));
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
}

// ------------------------------------------------------------ element types
// Raw8<E>: the 16-byte words of 8 elements as loaded, so that several loads can
// be in flight before the first is unpacked.
template <typename E>
struct Raw8 {
  static constexpr int W = (int)sizeof(typename E::T) / 2;
  uint4 w[W];
  __device__ __forceinline__ void load(const typename E::T* p) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const { E::load8(reinterpret_cast<const typename E::T*>(w), x); }
  __device__ __forceinline__ void from(const float (&x)[8]) { E::store8(reinterpret_cast<typename E::T*>(w), x); }

  // The same shared out over the L lanes of a row of 8 L elements: lane l's word i is
  // the row's word i L + l, so that a warp's access is contiguous (two words a
  // lane side by side made every access of float32 rows use half its sectors).
  // The 8 / W elements of a word keep their codes together.
  template <int L>
  __device__ __forceinline__ void load(const typename E::T* row, int l) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint4*>(row)[i * L + l];
  }
  template <int L>
  __device__ __forceinline__ void store(typename E::T* row, int l) const {
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint4*>(row)[i * L + l] = w[i];
  }
  template <int L>
  static __device__ __forceinline__ void store_codes(uint8_t* row, int l, uint2 c) {
    if constexpr (W == 1) {
      reinterpret_cast<uint2*>(row)[l] = c;
    } else {
      reinterpret_cast<uint32_t*>(row)[l] = c.x;
      reinterpret_cast<uint32_t*>(row)[L + l] = c.y;
    }
  }
  template <int L>
  static __device__ __forceinline__ uint2 load_codes(const uint8_t* row, int l) {
    if constexpr (W == 1) return reinterpret_cast<const uint2*>(row)[l];
    return make_uint2(reinterpret_cast<const uint32_t*>(row)[l], reinterpret_cast<const uint32_t*>(row)[L + l]);
  }
};

struct ElemF32 {
  using T = float;
  static __device__ __forceinline__ float get(const T* p) { return *p; }
  static __device__ __forceinline__ void put(T* p, float v) { *p = v; }
  static __device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  static __device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
};
struct ElemBf16 {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(const T* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void put(T* p, float v) { *p = __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
struct ElemF16 {
  using T = __half;
  static __device__ __forceinline__ float get(const T* p) { return __half2float(*p); }
  static __device__ __forceinline__ void put(T* p, float v) { *p = __float2half_rn(v); }
  static __device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = f16x2_to_f32(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ uint32_t abs_bits8(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  return m;
}

}  // namespace dllm
