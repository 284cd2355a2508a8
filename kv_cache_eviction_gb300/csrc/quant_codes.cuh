// Numbers of the 8-bit cache: codes, and the scale of a block of 16 rows of one head.
//
// A value is code * scale, with scale a power of two 2^t:  t is the smallest, from kLeast on, with
//   largest finite |x| of the block <= kMost 2^t,        kMost = 448 (e4m3) or 127 (int8).
// A power of two costs at most one bit of the code's range.  What it buys: x / 2^t and code * 2^t
// are exact, so a value is rounded once, by its code alone, and a block that moves to a larger
// scale rounds again only what falls below the code's last place (in e4m3 what is subnormal there).
// kLeast keeps scales and their reciprocals normal floats with room for the attention's factors:
// in blocks of that scale, values below 2^-106 (1.2e-32; int8 2^-97, 6e-30) become zero.
//
// Infinities become the code's largest number and do not count for the scale; a NaN is a NaN in
// e4m3 and zero in int8.
#pragma once

#include <cuda_fp16.h>

#include "kv_internal.cuh"

namespace kv {
namespace quant {

constexpr int kBlock = 16;     // rows
constexpr int kLeast = -96;

// Formats: pack4 takes any float, pack4_held only what is within the code's range (after a
// scale_for of a maximum that is finite).
struct E4M3 {
  // 448 = 0.875 * 2^9: a mantissa past 0.875 (1.75 as 1.m) needs a step more
  static constexpr int kTopExp = 9;
  static constexpr uint32_t kTopMant = 0x600000u;
  // two codes, x in the low byte
  static __device__ __forceinline__ uint32_t pack2(float x, float y) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
    return r;
  }
  static __device__ __forceinline__ uint32_t pack4(float x, float y, float z, float w) {
    return pack2(x, y) | pack2(z, w) << 16;
  }
  static __device__ __forceinline__ uint32_t pack4_held(float x, float y, float z, float w,
                                                        float by) {
    return pack4(x * by, y * by, z * by, w * by);
  }
  // the numbers of a word's codes 0, 1 and 2, 3
  static __device__ __forceinline__ void halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
  // of codes 0, 2 and 1, 3
  static __device__ __forceinline__ void columns(uint32_t w, uint32_t& even, uint32_t& odd) {
    halves(__byte_perm(w, 0u, 0x3120), even, odd);
  }
};

struct Int8 {
  // 127 = 0.9921875 * 2^7
  static constexpr int kTopExp = 7;
  static constexpr uint32_t kTopMant = 0x7E0000u;
  static __device__ __forceinline__ uint32_t pack4(float x, float y, float z, float w) {
    const int a = max(__float2int_rn(x), -127), b = max(__float2int_rn(y), -127);
    const int c = max(__float2int_rn(z), -127), d = max(__float2int_rn(w), -127);
    uint32_t hi, r;
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(hi) : "r"(d), "r"(c), "r"(0));
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(b), "r"(a), "r"(hi));
    return r;
  }
  // x times `by` in the last places of 1.5 * 2^23, rounded there: its low byte is the code
  static __device__ __forceinline__ uint32_t pack4_held(float x, float y, float z, float w,
                                                        float by) {
    constexpr float kBase = 12582912.f;
    const uint32_t a = __float_as_uint(fmaf(x, by, kBase)), b = __float_as_uint(fmaf(y, by, kBase));
    const uint32_t c = __float_as_uint(fmaf(z, by, kBase)), d = __float_as_uint(fmaf(w, by, kBase));
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  }
  // code + 128 in the last places of 1024 (fp16 has ten of them, so 1024 + n is 0x6400 + n for n below
  // 1024): less 1152 it is the code, exactly
  static __device__ __forceinline__ uint32_t less(uint32_t x) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x64806480u));
    return r;
  }
  static __device__ __forceinline__ void halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    lo = less(__byte_perm(w, 0x64646464u, 0x4140));
    hi = less(__byte_perm(w, 0x64646464u, 0x4342));
  }
  static __device__ __forceinline__ void columns(uint32_t w, uint32_t& even, uint32_t& odd) {
    w ^= 0x80808080u;
    even = less(__byte_perm(w, 0x64646464u, 0x4240));
    odd = less(__byte_perm(w, 0x64646464u, 0x4341));
  }
};

__device__ __forceinline__ float2 floats_of(uint32_t h2) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

// The scale of a block whose largest finite magnitude has the bits `top`.
template <typename F>
__device__ __forceinline__ float scale_for(uint32_t top) {
  int t = (int)(top >> 23) - 126 - F::kTopExp + ((top & 0x7FFFFFu) > F::kTopMant ? 1 : 0);
  t = t < kLeast ? kLeast : t;
  return __uint_as_float((uint32_t)(t + 127) << 23);
}

// The scale of a block after it got rows of that maximum: `old`, that of the rows held (0 where there
// are none), or what the new rows need where that is more.  An old one that is no finite number does not
// count, as the values it stands for do not; times old / the new one they are then coded as what they
// are, NaN and infinities.
template <typename F>
__device__ __forceinline__ float scale_after(uint32_t top, float old) {
  const float need = scale_for<F>(top);
  return need < old && old < INFINITY ? old : need;
}

// 16 codes of a piece at another scale: rounded times `by`.
template <typename F>
__device__ __forceinline__ uint4 again(uint4 c, float by) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    F::halves(w[i], lo, hi);
    const float2 a = floats_of(lo), b = floats_of(hi);
    w[i] = F::pack4(a.x * by, a.y * by, b.x * by, b.y * by);
  }
  return c;
}

// 16 bytes of a row: kN elements.
template <typename T>
struct Piece {
  static constexpr int kN = 16 / (int)sizeof(T);
  uint4 w;
  __device__ __forceinline__ uint32_t word(int i) const {
    return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
  }
  __device__ __forceinline__ float at(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(word(i));
    return __uint_as_float(i & 1 ? word(i / 2) & 0xFFFF0000u : word(i / 2) << 16);
  }
  // The largest of m and the magnitudes' bits, infinities and NaN among them: kInf and more.  (Of
  // bf16, two magnitudes side by side in m; see whole().)
  __device__ __forceinline__ uint32_t top(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = sizeof(T) == 4 ? max(m, word(i) & 0x7FFFFFFFu) : __vmaxu2(m, word(i) & 0x7FFF7FFFu);
    return m;
  }
  static __device__ __forceinline__ uint32_t whole(uint32_t m) {
    return sizeof(T) == 4 ? m : max(m << 16, m & 0xFFFF0000u);
  }
  // The same without infinities and NaN.
  __device__ __forceinline__ uint32_t finite_top(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t u = __float_as_uint(at(i)) & 0x7FFFFFFFu;
      m = u < 0x7F800000u && u > m ? u : m;
    }
    return m;
  }
  // Four codes from element i on, x times `inv`.  held: every element is finite and in range.
  template <typename F>
  __device__ __forceinline__ uint32_t codes(int i, float inv, bool held) const {
    if (held) return F::pack4_held(at(i), at(i + 1), at(i + 2), at(i + 3), inv);
    return F::pack4(at(i) * inv, at(i + 1) * inv, at(i + 2) * inv, at(i + 3) * inv);
  }
};
constexpr uint32_t kInf = 0x7F800000u;

}  // namespace quant
}  // namespace kv
