// One warp's online softmax over tiles of K and V rows in shared memory, on the warp matrix
// instructions, for up to 8 query rows:  (m, l, o) := running maximum, sum and output of
//   p_r = exp2(c2 (q . k_r - m)),  l = sum p_r,  o = sum p_r v_r,   c2 > 0.
//
// A tile is RT rows of K and V of H half segments (64 bytes) each, in segments of [RT][128 bytes]
// with the 16-byte pieces of row r permuted by r & 7, so that every access below touches 8
// different pieces of the 32 banks: K's whole segments, V's, and for odd H one that holds the
// rest of K's row, then of V's.
//
// m16n8k16 (bf16) and m16n8k8 (tf32) have 16 rows where a KV head has at most 8 queries.  The
// other 8 rows carry what is lost by holding the left operand in few bits: rows 0..7 hold the
// high parts, rows 8..15 the rest, and their sums are added at the end, in the same lane.
//   bf16: q and k are bf16, their products are exact.  p is held as two bf16 (16 bits).
//   fp32: q and p are held as two tf32 (22 bits), and so are k and v, at one instruction each.
// The sums are fp32.  Against one bf16 p this costs no instruction, and the error of p (2^-16)
// stays far under that of the bf16 output.
//
// The score fragment of lane (4 g + c) holds query g and rows 2c, 2c + 1 of each 8; as left
// operand of the second product the same lane holds the same rows (for tf32, whose lane holds
// columns c and c + 4, the rows of each 8 are taken in the order 0, 2, 4, 6, 1, 3, 5, 7), so p
// never leaves its lane.
//
// The scale is no factor of its own: p = exp2((s - m) c2), maxima are of q . k.  (As
// exp2(fma(s, c2, -m c2)), an addition less a score, the rounding of m c2 moves every exponent,
// beyond float's range for |m c2| past 2^31: finite scores gave zeros and NaN.)  A negative scale is
// taken into q's sign, and a zero one is the smallest positive number, so that masked scores
// (-inf) give zeros (Scale).
#pragma once

#include "kv_internal.cuh"
#include "tc_ptx.cuh"

namespace kv {
namespace pmma {

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32_1688(float (&d)[4], uint32_t a0, uint32_t a1,
                                              uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with sums that start from zero.
__device__ __forceinline__ void mma_bf16_16816_new(float (&d)[4], uint32_t a0, uint32_t a1,
                                                   uint32_t a2, uint32_t a3, uint32_t b0,
                                                   uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_tf32_1688_new(float (&d)[4], uint32_t a0, uint32_t a1,
                                                  uint32_t a2, uint32_t a3, uint32_t b0,
                                                  uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float lds_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// x = hi + lo to 22 bits, both tf32 (11 significant bits, the low 13 of the word zero): hi is x
// to the nearest (halves away from zero), x - hi is exact and at most 2^-11 of x's power of two,
// so what lo's truncation drops is below 2^-22 of x.  (Adding half a step to the word rounds as
// cvt.rna.tf32 does, in fewer instructions: 31 % of the kernel at d = 128; a NaN stays one in lo.)
__device__ __forceinline__ void tf32_split(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xFFFFE000u;
}
__device__ __forceinline__ uint32_t bf16x2_of(float x, float y) {   // x in the low half
  const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Byte offset of 16-byte piece c of K's (V's) row r within a tile of RT rows.
template <int RT, int H>
__device__ __forceinline__ uint32_t k_piece(int r, int c) {
  const int seg = c >> 3;
  return (uint32_t)((seg < H / 2 ? seg : H / 2 * 2) * (RT * 128) + r * 128 + (((c ^ r) & 7) << 4));
}
template <int RT, int H>
__device__ __forceinline__ uint32_t v_piece(int r, int c) {
  const int seg = c >> 3;
  return seg < H / 2 ? k_piece<RT, H>(r, c) + H / 2 * (RT * 128) : k_piece<RT, H>(r, c) ^ 64u;
}

struct Scale {
  float c2;        // > 0
  uint32_t flip;   // sign bits of q to flip (bf16: of both halves)
};

template <typename T, int H>
struct Tile;

// What both types share: lane (4 g + c)'s running state for query g, and its part of o:
// columns 8 t + 2 c and + 1 for every t < NT.
//
// The matrix instruction cuts its sums off instead of rounding them, always towards zero: with o as
// its accumulator over all tiles of a warp, outputs of positive values shrank by 2^-25 to 2^-23 a
// tile (fp32: 1e-5 to 4.5e-5 after 446 tiles, where plain float sums are 1e-7 off).  So it adds up
// kHold tiles at most, and their sums are added to o rounded to the nearest (4e-7).  bf16 takes a
// tile: 607 us on 4.2 GB, 606 with o as accumulator.  fp32, bound by instructions, takes four up to
// d = 96 and one above, where registers are short.  64 sequences of 4000 rows, o as accumulator /
// four / one, us: d = 64 162 / 163 / 162, 72 210 / 209 / 227, 96 245 / 254 / 259, 128 315 / 324 / 317.
template <int NT, int kHold>
struct State {
  float m, l, lc;    // l: this lane's share of the sum; lc: what its rounding has added
  float o[NT][2];
  // sums of the last `held` tiles: [0..1] high rows, [2..3] low rows
  float acc[kHold > 1 ? NT : 1][4];
  int held;
  // A lane's outputs: kQ queries, and for each kPairs pairs of neighbouring columns.
  static constexpr int kQ = 1, kPairs = NT;
  static __device__ __forceinline__ int query(int) { return (threadIdx.x & 31) >> 2; }
  static __device__ __forceinline__ int column(int t) { return 8 * t + 2 * (threadIdx.x & 3); }
  static __device__ __forceinline__ bool owns_sums() { return (threadIdx.x & 3) == 0; }
  __device__ __forceinline__ float2 pair(int t, int) const { return make_float2(o[t][0], o[t][1]); }
  __device__ __forceinline__ float max_of(int) const { return m; }
  __device__ __forceinline__ float sum_of(int) const { return l; }
  __device__ __forceinline__ void begin() {
    m = -INFINITY;
    l = lc = 0.f;
    held = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      o[t][0] = o[t][1] = 0.f;
      if (kHold > 1) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
    }
  }
  // l gains x, a tile's weights (one value a tile and a lane, so a compensated sum is cheap; equal
  // weights round to the same side tile after tile, 4e-6 after 446 tiles).
  __device__ __forceinline__ void add_l(float x) {
    x -= lc;
    const float s = l + x;
    lc = (s - l) - x;
    l = s;
  }
  // Sums of columns 8 t.. (high rows, low rows) to o.
  __device__ __forceinline__ void add(int t, const float (&d)[4]) {
    const float2 s = ptx::fadd2(make_float2(o[t][0], o[t][1]),
                                ptx::fadd2(make_float2(d[0], d[1]), make_float2(d[2], d[3])));
    o[t][0] = s.x;
    o[t][1] = s.y;
  }
  // After a tile in acc.
  __device__ __forceinline__ void tile_done() {
    if (++held < kHold) return;
    held = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      add(t, acc[t]);
      acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
    }
  }
  // New maximum of this lane's query from the tile's scores; o and l follow.
  __device__ __forceinline__ void raise(float mt, float c2) {
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
    if (__any_sync(0xffffffffu, mt > m)) {
      const float mn = fmaxf(m, mt);
      const float a = mn > m ? ptx::ex2((m - mn) * c2) : 1.f;   // 0 while m is -inf
      m = mn;
      l *= a;
      lc *= a;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          o[t][e] *= a;
          if (kHold > 1) {
            acc[t][e] *= a;
            acc[t][2 + e] *= a;
          }
        }
    }
  }
  __device__ __forceinline__ float base() const { return m == -INFINITY ? 0.f : m; }
  // After the last tile: l whole in every lane of the query.
  __device__ __forceinline__ void finish() {
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (kHold > 1) {
#pragma unroll
      for (int t = 0; t < NT; ++t) add(t, acc[t]);
    }
  }
};

template <int H>
struct Tile<__nv_bfloat16, H> : State<H * 4, 1> {
  static constexpr int RT = 16;
  static constexpr int NT = H * 4;
  static constexpr int D = H * 32;     // columns held (d rounded up; the rest is zero)
  static constexpr int NQ = H * 4;     // 32-bit words of q per lane
  uint32_t q[NQ];

  // Words of q for query g = lane / 4 (zero past d and for g >= G).
  static __device__ __forceinline__ void load_q(const __nv_bfloat16* src, int G, int d,
                                                uint32_t (&w)[NQ]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int x = 8 * i + 2 * c;
      w[i] = g < G && x < d ? *reinterpret_cast<const uint32_t*>(src + g * d + x) : 0u;
    }
  }
  __device__ __forceinline__ void set_q(const uint32_t (&w)[NQ], const Scale& sc) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) q[i] = w[i] ^ sc.flip;
  }

  // One tile at shared address st (128-byte aligned); bit r of `mask`: row r counts
  // (others hold zeros: 0 * NaN is NaN).
  // A piece's address is its row's with piece bits under xor (r & 7) * 16, so the pieces of a
  // lane's row are one address xor a constant.
  __device__ __forceinline__ void tile(uint32_t st, uint32_t mask, float c2) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    // scores: two sums per 8 rows (even and odd k-steps), short chains
    float s[2][2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][0][e] = s[j][1][e] = 0.f;
    const uint32_t ka = st + (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4);
    // (all loads first: their latency once, not once a step)
    uint32_t b[H][2][4];
#pragma unroll
    for (int kk = 0; kk < H; ++kk)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        ldsm4(b[kk][j], (ka ^ ((kk & 1) * 64)) + (kk < H / 2 * 2 ? kk >> 1 : kk) * (RT * 128) +
                            j * 1024);
#pragma unroll
    for (int kk = 0; kk < H; ++kk)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma_bf16_16816(s[j][0], q[4 * kk], 0u, q[4 * kk + 1], 0u, b[kk][j][0], b[kk][j][1]);
        mma_bf16_16816(s[j][1], q[4 * kk + 2], 0u, q[4 * kk + 3], 0u, b[kk][j][2], b[kk][j][3]);
      }
    // V too, while the softmax is worked out
    const uint32_t va = st + (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
    uint32_t v[NT / 2][4];
#pragma unroll
    for (int t = 0; t < NT; t += 2) {
      const bool rest = (t >> 3) >= H / 2;   // behind K's
      ldsm4_t(v[t / 2], (va ^ ((rest ? t & 2 | 4 : t & 6) * 16)) +
                            (rest ? H / 2 * 2 : H / 2 + (t >> 3)) * (RT * 128));
    }
    float z[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) z[j][e] = s[j][0][e] + s[j][1][e];
    if (mask != 0xFFFFu) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!(mask >> (8 * j + 2 * c + e) & 1)) z[j][e] = -INFINITY;
    }
    this->raise(fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[1][0], z[1][1])), c2);
    const float base = this->base();
    uint32_t hi[2], lo[2];
    float ps[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float p0 = ptx::ex2((z[j][0] - base) * c2), p1 = ptx::ex2((z[j][1] - base) * c2);
      ps[j] = p0 + p1;
      hi[j] = bf16x2_of(p0, p1);
      lo[j] = bf16x2_of(p0 - __uint_as_float(hi[j] << 16),
                        p1 - __uint_as_float(hi[j] & 0xFFFF0000u));
    }
    this->add_l(ps[0] + ps[1]);
#pragma unroll
    for (int t = 0; t < NT; t += 2) {
      float d[2][4];
      mma_bf16_16816_new(d[0], hi[0], lo[0], hi[1], lo[1], v[t / 2][0], v[t / 2][1]);
      mma_bf16_16816_new(d[1], hi[0], lo[0], hi[1], lo[1], v[t / 2][2], v[t / 2][3]);
      this->add(t, d[0]);
      this->add(t + 1, d[1]);
    }
  }
};

template <int H>
struct Tile<float, H> : State<H * 2, (H > 6 ? 1 : 4)> {
  static constexpr int kHold = H > 6 ? 1 : 4;
  // 16 rows where two stages of them fit a warp's ring: fewer instructions a row (64 ragged
  // sequences, d = 72: 111 us against 127 with 8)
  static constexpr int RT = H > 5 ? 8 : 16;
  static constexpr int NT = H * 2;
  static constexpr int D = H * 16;
  static constexpr int NQ = H * 4;
  uint32_t qh[NQ], ql[NQ];

  static __device__ __forceinline__ void load_q(const float* src, int G, int d,
                                                uint32_t (&w)[NQ]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int x = 4 * i + c;
      w[i] = g < G && x < d ? __float_as_uint(src[g * d + x]) : 0u;
    }
  }
  __device__ __forceinline__ void set_q(const uint32_t (&w)[NQ], const Scale& sc) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) tf32_split(__uint_as_float(w[i] ^ sc.flip), qh[i], ql[i]);
  }

  __device__ __forceinline__ void tile(uint32_t st, uint32_t mask, float c2) {
    constexpr int NB = RT / 8;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // scores: the high and the low parts of k, even and odd k-steps in sums of their own
    float z[NB][2], mt = -INFINITY;
    const uint32_t ka = st + g * 128 + (g << 4) + 4 * c;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i >> 2][i & 3] = 0.f;
      // (all loads first: their latency once, not once a step)
      float x[2 * NT];
#pragma unroll
      for (int k = 0; k < 2 * NT; ++k)
        x[k] = lds_f((ka ^ ((k & 7) << 4)) + (k < H / 2 * 8 ? k >> 3 : H / 2 * 2) * (RT * 128) +
                     j * 1024);
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        uint32_t h0, l0, h1, l1;
        tf32_split(x[2 * k], h0, l0);
        tf32_split(x[2 * k + 1], h1, l1);
        mma_tf32_1688(s[k & 1], qh[2 * k], ql[2 * k], qh[2 * k + 1], ql[2 * k + 1], h0, h1);
        mma_tf32_1688(s[2 + (k & 1)], qh[2 * k], ql[2 * k], qh[2 * k + 1], ql[2 * k + 1], l0, l1);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        z[j][e] = ((s[0][e] + s[1][e]) + (s[0][2 + e] + s[1][2 + e])) +
                  ((s[2][e] + s[3][e]) + (s[2][2 + e] + s[3][2 + e]));
        if (mask != (1u << RT) - 1u && !(mask >> (8 * j + 2 * c + e) & 1)) z[j][e] = -INFINITY;
        mt = fmaxf(mt, z[j][e]);
      }
    }
    this->raise(mt, c2);
    const float base = this->base();
    // rows 2 c and 2 c + 1 of each 8, pieces under xor their row
    const uint32_t v0 = st + 2 * c * 128 + (((g >> 2) ^ (2 * c)) << 4) + 4 * (g & 3);
    const uint32_t v1 = v0 + 128 - (((g >> 2) ^ (2 * c)) << 4) + (((g >> 2) ^ (2 * c + 1)) << 4);
    uint32_t h0[NB], l0[NB], h1[NB], l1[NB];
    float ps = 0.f;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const float p0 = ptx::ex2((z[j][0] - base) * c2), p1 = ptx::ex2((z[j][1] - base) * c2);
      ps += p0 + p1;
      tf32_split(p0, h0[j], l0[j]);
      tf32_split(p1, h1[j], l1[j]);
    }
    this->add_l(ps);
    float x[NB][2 * NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const bool rest = (t >> 2) >= H / 2;   // behind K's
        const uint32_t at = (rest ? H / 2 * 2 : H / 2 + (t >> 2)) * (RT * 128) + j * 1024;
        const uint32_t flip = (rest ? 2 * t & 3 | 4 : 2 * t & 7) << 4;
        x[j][2 * t] = lds_f((v0 ^ flip) + at);
        x[j][2 * t + 1] = lds_f((v1 ^ flip) + at);
      }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float fresh[4];
      float(&d)[4] = kHold > 1 ? this->acc[kHold > 1 ? t : 0] : fresh;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        uint32_t vh0, vl0, vh1, vl1;
        tf32_split(x[j][2 * t], vh0, vl0);
        tf32_split(x[j][2 * t + 1], vh1, vl1);
        if (kHold == 1 && j == 0) mma_tf32_1688_new(d, h0[j], l0[j], h1[j], l1[j], vh0, vh1);
        else mma_tf32_1688(d, h0[j], l0[j], h1[j], l1[j], vh0, vh1);
        mma_tf32_1688(d, h0[j], l0[j], h1[j], l1[j], vl0, vl1);
      }
      if (kHold == 1) this->add(t, d);
    }
    if (kHold > 1) this->tile_done();
  }
};

}  // namespace pmma
}  // namespace kv
