// packed.cuh -- float32 pairs: one instruction works on two values.
#pragma once

#include <stdint.h>

namespace rwkv7 {

// two float32 values in a register pair, and the packed operations on them (one instruction each)
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 make2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split2(f32x2 x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return fma2(b, make2(-1.f, -1.f), a); }
// rounded to nearest-even bf16, the first value in the low half
__device__ __forceinline__ uint32_t pack2(f32x2 x) {
  float a, b;
  split2(x, a, b);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// two bf16 in a word, the first in the low half, as a pair
__device__ __forceinline__ f32x2 unpack2(uint32_t u) {
  return make2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

}  // namespace rwkv7
