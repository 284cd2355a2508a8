// One warp's online softmax over tiles of 32 K and V rows of 8-bit codes (paged_mma.cuh has the idea
// and the tile's layout): the warp matrix instructions in fp16.
//
// fp16 holds every code exactly, and the block's scales are factors of a tile's sums: of the scores
// (after the product with q) and of the outputs (when a tile's sums, which start from zero, are added
// to o).  So the codes cost their conversion and nothing else.
//   q is taken times a power of two that brings its largest element to 2^13..2^14, which fp16 holds to
//     2^-24, 2^-37 of it; bf16's 8 bits are then exact, and fp32's are held as two fp16 (22 bits), the
//     lower 2^11 times larger.
//   p, at most 1, is taken 2^14 times as large and held as two fp16 in the same way.
//
// K's words hold four columns of a row, 16 p + 4 c + 0..3 for lane c of 4: they are taken as columns
// 2 c, 2 c + 1 and 2 c + 8, 2 c + 9 of the instruction, and q's likewise.  V's transposed load moves pairs
// of columns, so a word has two rows of two columns: even and odd columns are products of their own, and
// a lane ends with the outputs of four neighbouring columns.
#pragma once

#include "paged_mma.cuh"
#include "quant_codes.cuh"

namespace kv {
namespace qmma {

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with sums that start from zero.
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t f16x2_of(float x, float y) {   // x in the low half
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x, y = hi + 2^-11 lo, both pairs of fp16
__device__ __forceinline__ void f16_split(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = f16x2_of(x, y);
  const float2 h = quant::floats_of(hi);
  lo = f16x2_of((x - h.x) * 2048.f, (y - h.y) * 2048.f);
}

template <typename T, typename F, int H>
struct Tile : pmma::State<H * 8, 1> {
  static constexpr int RT = 32;
  static constexpr int NT = H * 8;
  static constexpr int D = H * 64;     // columns held (d rounded up; the rest is zero)
  static constexpr bool kWords = sizeof(T) == 2;
  static constexpr int NQ = H * (kWords ? 8 : 16);   // 32-bit words of q per lane, as loaded
  static constexpr int NF = H * 8;                   // and as pairs of fp16
  uint32_t qh[NF], ql[kWords ? 1 : NF];
  float unit;        // what a score of qh, ql and codes counts for

  static constexpr int kWide = 4, kGroups = NT / 2;
  __device__ __forceinline__ void group(int t, float by, float (&x)[4]) const {
    x[0] = this->o[2 * t][0] * by;
    x[1] = this->o[2 * t + 1][0] * by;
    x[2] = this->o[2 * t][1] * by;
    x[3] = this->o[2 * t + 1][1] * by;
  }

  static __device__ __forceinline__ void load_q(const T* src, int G, int d, uint32_t (&w)[NQ]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int p = 0; p < H * 4; ++p) {
      const bool in = g < G && 16 * p < d;
      const T* at = src + g * d + 16 * p + 4 * c;
      if (kWords) {
        const uint2 x = in ? *reinterpret_cast<const uint2*>(at) : make_uint2(0u, 0u);
        w[2 * p] = x.x;
        w[2 * p + 1] = x.y;
      } else {
        const uint4 x = in ? *reinterpret_cast<const uint4*>(at) : make_uint4(0u, 0u, 0u, 0u);
        w[(4 * p) % NQ] = x.x;
        w[(4 * p + 1) % NQ] = x.y;
        w[(4 * p + 2) % NQ] = x.z;
        w[(4 * p + 3) % NQ] = x.w;
      }
    }
  }
  __device__ __forceinline__ void set_q(const uint32_t (&w)[NQ], const pmma::Scale& sc) {
    auto at = [&](int i) {
      if (!kWords) return __uint_as_float(w[i % NQ]);
      return __uint_as_float(i & 1 ? w[i / 2 % NQ] & 0xFFFF0000u : w[i / 2 % NQ] << 16);
    };
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * NF; ++i) top = fmaxf(top, fabsf(at(i)));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^13 <= top * by < 2^14; by within 2^-114..2^120
    int e = (int)(__float_as_uint(top) >> 23);
    e = e < 20 ? 20 : e;
    const float by = __uint_as_float((uint32_t)(267 - e) << 23) * (sc.flip ? -1.f : 1.f);
    unit = __uint_as_float((uint32_t)(e - 13) << 23);
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const float x = at(2 * i) * by, y = at(2 * i + 1) * by;
      if (kWords) qh[i] = f16x2_of(x, y);
      else f16_split(x, y, qh[i], ql[i % (kWords ? 1 : NF)]);
    }
  }

  // One tile at shared address st (128-byte aligned); bit r of `mask`: row r counts (others hold
  // zeros).  scales: of K's and V's codes in the first block, and in the second.
  __device__ __forceinline__ void tile(uint32_t st, uint32_t mask, float c2, const float4& scales) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    const uint32_t ka = st + (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4);
    const uint32_t va = st + (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4) +
                        (H == 2 ? RT * 128 : 0);
    float z[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // eight rows
      float s[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = 0.f;
      uint32_t b[H][4];
#pragma unroll
      for (int kk = 0; kk < H; ++kk) pmma::ldsm4(b[kk], (ka ^ (kk * 64)) + j * 1024);
#pragma unroll
      for (int kk = 0; kk < H; ++kk)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int i = 2 * (4 * kk + m);
          uint32_t lo, hi;
          F::halves(b[kk][m], lo, hi);
          mma_f16(s[m & 1], qh[i], kWords ? 0u : ql[i % (kWords ? 1 : NF)], qh[i + 1],
                  kWords ? 0u : ql[(i + 1) % (kWords ? 1 : NF)], lo, hi);
        }
      const float by = (j < 2 ? scales.x : scales.z) * unit;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = s[0][e] + s[1][e];
        if (!kWords) x = fmaf(s[0][2 + e] + s[1][2 + e], 0x1p-11f, x);
        z[j][e] = x * by;
      }
    }
    if (mask != 0xFFFFFFFFu) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!(mask >> (8 * j + 2 * c + e) & 1)) z[j][e] = -INFINITY;
    }
    float top = fmaxf(z[0][0], z[0][1]);
#pragma unroll
    for (int j = 1; j < 4; ++j) top = fmaxf(top, fmaxf(z[j][0], z[j][1]));
    this->raise(top, c2);
    const float base = this->base();
    uint32_t hi[4], lo[4];
    float ps = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float p0 = ptx::ex2((z[j][0] - base) * c2), p1 = ptx::ex2((z[j][1] - base) * c2);
      ps += p0 + p1;
      f16_split(p0 * 16384.f, p1 * 16384.f, hi[j], lo[j]);
    }
    this->add_l(ps);
#pragma unroll
    for (int b = 0; b < 2; ++b) {   // blocks
      const float vs = b == 0 ? scales.y : scales.w;
      const float2 f1 = make_float2(vs * 0x1p-14f, vs * 0x1p-14f);
      const float2 f2 = make_float2(vs * 0x1p-25f, vs * 0x1p-25f);
      // V: rows 0..7 and 8..15 of two pieces at a time
      uint32_t v[H * 2][4];
#pragma unroll
      for (int t = 0; t < H * 2; ++t)
        pmma::ldsm4_t(v[t], (va ^ ((2 * t + (H == 1 ? 4 : 0)) * 16)) + b * 2048);
#pragma unroll
      for (int p = 0; p < H * 4; ++p) {
        uint32_t e0, o0, e1, o1;
        F::columns(v[p / 2][p % 2 * 2], e0, o0);
        F::columns(v[p / 2][p % 2 * 2 + 1], e1, o1);
        float d[2][4];
        mma_f16_new(d[0], hi[2 * b], lo[2 * b], hi[2 * b + 1], lo[2 * b + 1], e0, e1);
        mma_f16_new(d[1], hi[2 * b], lo[2 * b], hi[2 * b + 1], lo[2 * b + 1], o0, o1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float(&o)[2] = this->o[2 * p + x];
          const float2 y = ptx::ffma2(make_float2(d[x][0], d[x][1]), f1,
                                      ptx::ffma2(make_float2(d[x][2], d[x][3]), f2,
                                                 make_float2(o[0], o[1])));
          o[0] = y.x;
          o[1] = y.y;
        }
      }
    }
  }
};

}  // namespace qmma
}  // namespace kv
