// One warp's online softmax over tiles of 32 K and V rows of 8-bit codes, for up to 8 query rows,
// on the warp matrix instructions in fp16 (paged_mma.cuh has the sums and the tile's layout).
//
// fp16 holds every code exactly, and the block's scales are factors of a tile's sums: of the scores
// (after the product with q) and of the outputs (when a tile's sums, which start from zero, are
// added to o).  So the codes cost their conversion and nothing else.
//   q is taken times a power of two that brings its largest element to 2^13..2^14, which fp16 holds
//     to 2^-24, 2^-37 of it; bf16's 8 bits are then exact, and fp32's are held as two fp16 (22 bits).
//   p, at most 1, is taken 2^14 times as large and held as two fp16 as well: 22 bits, or 2^-39.
//
// m16n8k16's larger side is the codes': scores are K q^T (16 rows, 8 queries), outputs V^T p^T (16
// columns, 8 queries).  With the queries on that side half of its rows stood empty (or held the
// lower parts), and its four registers had to be put together for every product: 770 instructions a
// tile, and 322 us on 2.1 GB. K's words hold four columns of a row, 16 p + 4 c + 0..3 for lane c of
// 4: they are taken as columns 2 c, 2 c + 1 and 2 c + 8, 2 c + 9 of the instruction, and q's
// likewise.  V's transposed load moves pairs of columns, so a word has two rows of two columns:
// rows 0..7 of V^T's 16 are the even ones of a piece, 8..15 the odd ones.  A lane (4 g + c) has the
// scores of rows g and g + 8 for queries 2 c and 2 c + 1; as right operand the second product wants
// rows 2 c and 2 c + 1 for query g: a transposition of 8 by 8, movmatrix.
#pragma once

#include "paged_mma.cuh"
#include "quant_codes.cuh"

namespace kv {
namespace qmma {

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with sums that start from zero.
__device__ __forceinline__ void mma_f16_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// An 8 by 8 matrix of 16-bit elements, transposed: lane 4 g + c gives row g, columns 2 c and 2 c +
// 1.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of(float x, float y) {   // x in the low half
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x, y = hi + lo, both pairs of fp16
__device__ __forceinline__ void f16_split(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = f16x2_of(x, y);
  const float2 h = quant::floats_of(hi);
  lo = f16x2_of(x - h.x, y - h.y);
}

// NP: pieces of 16 columns, even.
template <typename T, typename F, int NP>
struct Tile {
  static constexpr int RT = 32;
  static constexpr int H = NP <= 4 ? 1 : 2;   // 64-byte parts of a row in a stage
  static constexpr int D = NP * 16;           // columns held (d rounded up; the rest is zero)
  static constexpr bool kWords = sizeof(T) == 2;
  static constexpr int NQ = NP * (kWords ? 2 : 4);   // 32-bit words of q per lane, as loaded
  static constexpr int NL = kWords ? 1 : 2 * NP;     // words of its lower part
  uint32_t qh[2 * NP], ql[NL];
  // of queries 2 c and 2 c + 1: what a score of qh, ql and codes counts for, running maximum, this
  // lane's share of the sum, and what its rounding has added
  float unit[2], m[2], l[2], lc[2];
  float o[NP][4];   // columns 16 p + 2 g (both queries), and 16 p + 2 g + 1

  // A lane's outputs: kQ queries, and for each kPairs pairs of neighbouring columns.
  static constexpr int kQ = 2, kPairs = NP;
  static __device__ __forceinline__ int query(int e) { return 2 * (threadIdx.x & 3) + e; }
  static __device__ __forceinline__ int column(int t) {
    return 16 * t + 2 * ((threadIdx.x & 31) >> 2);
  }
  static __device__ __forceinline__ bool owns_sums() { return (threadIdx.x & 31) < 4; }
  __device__ __forceinline__ float2 pair(int t, int e) const {
    return make_float2(o[t][e], o[t][2 + e]);
  }
  __device__ __forceinline__ float max_of(int e) const { return m[e]; }
  __device__ __forceinline__ float sum_of(int e) const { return l[e]; }

  // q of query lane / 4: columns 16 p + 4 c + 0..3 (zero past d and for queries from G on).
  static __device__ __forceinline__ void load_q(const T* src, int G, int d, uint32_t (&w)[NQ]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
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
    for (int i = 0; i < 4 * NP; ++i) top = fmaxf(top, fabsf(at(i)));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^13 <= top * by < 2^14, by between 2^-115 and 2^120
    int e = (int)(__float_as_uint(top) >> 23);
    e = e < 20 ? 20 : e;
    const float by = __uint_as_float((uint32_t)(267 - e) << 23) * (sc.flip ? -1.f : 1.f);
    const float one = __uint_as_float((uint32_t)(e - 13) << 23);
#pragma unroll
    for (int x = 0; x < 2; ++x) unit[x] = __shfl_sync(0xffffffffu, one, 4 * query(x));
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
      const float x = at(2 * i) * by, y = at(2 * i + 1) * by;
      if (kWords) qh[i] = f16x2_of(x, y);
      else f16_split(x, y, qh[i], ql[i % NL]);
    }
  }
  __device__ __forceinline__ void begin() {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = -INFINITY;
      l[e] = lc[e] = 0.f;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) o[p][0] = o[p][1] = o[p][2] = o[p][3] = 0.f;
  }
  // After the last tile: the sums whole in every lane of a query.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int s = 4; s < 32; s <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], s);
  }

  // One tile at shared address st (128-byte aligned); bit r of `mask`: row r counts (others hold
  // zeros).  scales: of K's and V's codes in the first block, and in the second.
  __device__ __forceinline__ void tile(uint32_t st, uint32_t mask, float c2, const float4& scales) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    // K and V: rows 0..7 and 8..15 of a block, of two pieces at a time
    const uint32_t ka = st + (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
    const uint32_t va = H == 2 ? ka + RT * 128 : ka ^ 64u;
    float z[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      // (u: the lower part of q.  The instruction cuts its sums off towards zero, so the fewer in
      // a chain the better: over 500 drawn shapes fp32 outputs were 2.2e-7 off in the mean, 3.1e-7
      // with both parts in one chain and 5.0e-7 in plain float32; a sum in float after every
      // product changes nothing more.)
      float s[2][4], u[2][4];
#pragma unroll
      for (int p = 0; p < NP; p += 2) {
        uint32_t w[4];
        pmma::ldsm4(w, (ka ^ (p * 16)) + b * 2048);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t a[4];
          F::halves(w[2 * x], a[0], a[2]);
          F::halves(w[2 * x + 1], a[1], a[3]);
          if (p == 0) mma_f16_new(s[x], a, qh[2 * x], qh[2 * x + 1]);
          else mma_f16(s[x], a, qh[2 * (p + x)], qh[2 * (p + x) + 1]);
          if (!kWords) {
            if (p == 0) mma_f16_new(u[x], a, ql[2 * (p + x) % NL], ql[(2 * (p + x) + 1) % NL]);
            else mma_f16(u[x], a, ql[2 * (p + x) % NL], ql[(2 * (p + x) + 1) % NL]);
          }
        }
      }
      const float ks = b == 0 ? scales.x : scales.z;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float low = kWords ? 0.f : u[0][i] + u[1][i];
        z[b][i] = ((s[0][i] + s[1][i]) + low) * (ks * unit[i & 1]);
      }
    }
    if (mask != 0xFFFFFFFFu) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(mask >> (16 * b + 8 * (i >> 1) + g) & 1)) z[b][i] = -INFINITY;
    }
    float mt[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mt[e] = fmaxf(fmaxf(z[0][e], z[0][2 + e]), fmaxf(z[1][e], z[1][2 + e]));
#pragma unroll
      for (int s = 4; s < 32; s <<= 1) mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], s));
    }
    if (__any_sync(0xffffffffu, mt[0] > m[0] || mt[1] > m[1])) {
      float a[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(m[e], mt[e]);
        a[e] = mn > m[e] ? ptx::ex2((m[e] - mn) * c2) : 1.f;   // 0 while m is -inf
        m[e] = mn;
        l[e] *= a[e];
        lc[e] *= a[e];
      }
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[p][i] *= a[i & 1];
    }
    uint32_t hi[2][2], lo[2][2];
    float ps[2] = {0.f, 0.f};
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float base = m[e] == -INFINITY ? 0.f : m[e];
          p[e] = ptx::ex2((z[b][2 * r + e] - base) * c2);
          ps[e] += p[e];
        }
        f16_split(p[0] * 16384.f, p[1] * 16384.f, hi[b][r], lo[b][r]);
        hi[b][r] = transposed(hi[b][r]);
        lo[b][r] = transposed(lo[b][r]);
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {   // (a compensated sum, as paged_mma.cuh's)
      const float x = ps[e] - lc[e], s = l[e] + x;
      lc[e] = (s - l[e]) - x;
      l[e] = s;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float vs = (b == 0 ? scales.y : scales.w) * 0x1p-14f;
      const float2 f = make_float2(vs, vs);
#pragma unroll
      for (int p = 0; p < NP; p += 2) {
        uint32_t w[4];
        pmma::ldsm4_t(w, (va ^ (p * 16)) + b * 2048);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t a[4];
          F::columns(w[2 * x], a[0], a[1]);
          F::columns(w[2 * x + 1], a[2], a[3]);
          float d[4];
          mma_f16_new(d, a, hi[b][0], hi[b][1]);
          mma_f16(d, a, lo[b][0], lo[b][1]);
          float(&y)[4] = o[p + x];
          const float2 u = ptx::ffma2(make_float2(d[0], d[1]), f, make_float2(y[0], y[1]));
          const float2 v = ptx::ffma2(make_float2(d[2], d[3]), f, make_float2(y[2], y[3]));
          y[0] = u.x;
          y[1] = u.y;
          y[2] = v.x;
          y[3] = v.y;
        }
      }
    }
  }
};

}  // namespace qmma
}  // namespace kv
