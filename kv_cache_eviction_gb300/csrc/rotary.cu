// Rotary positions: the pairs (a, b) of a head's first `rot` columns turned by position *
// frequency,
//   (a, b) -> m (a cos t - b sin t, a sin t + b cos t),
// pairs (x_i, x_{i + rot/2}) or (x_2i, x_2i+1).  A copy with a few operations: bound by reading and
// writing every row once.
//
// Angles are counted in turns, as 64-bit fractions of one: frequency / 2 pi is cut to 2^-62 of a
// turn once (in integers: 64-bit floats are slow here), and position * frequency is an integer
// product whose whole turns fall off at the top. So a position of 2^31 has the angle of a small
// one, to 2^-30 of a turn.  The fraction is cut to its nearest quarter turn before it becomes a
// float, which then has it to 2^-27 of a turn.
//
// A warp takes a row: a lane's pairs are the same ones in every head, so their sines and cosines
// are worked out once a row, shared by the lanes of the heads that it turns at a time.  Rows of
// small calls are split by heads.  On GB300: 131072 rows of 32 + 8 heads of 128 bf16 (2.7 GB read
// and written) 412 us, 6.5 TB/s or 0.96 of the measured copy rate; 20011 fp32 rows of 8 heads of
// 80, 24 columns of them turned, 21.5 us (24.4 with the other columns copied one after the other);
// 64 rows 2.6 us (3.7 with every lane working out all of its pairs' sines); 65536 fp32 rows of 32 + 8
// heads of 128 397 us, 6.8 TB/s.  What the small and the fp32 calls gained by the shared sines and the
// pieces copied four at a time cost the 131072 rows 1 % (408 us before).  bf16's `half` kernel of 8 pairs
// a lane spills one register at its 72.
#include "kv_internal.cuh"
#include "tc_ptx.cuh"

namespace kv {
namespace {

// Small CTAs, and more of them than are resident, even out what the SMs get through.  131072 rows /
// 20011 fp32 rows, us: 128 CTAs of two warps 412 / 21.5, 64 of four 413 / 23.0, 16 of four 447 /
// 22.8, 8 of eight 442 / 21.4.  (Heads loaded ahead of the one that is turned: 447 / 24.0.  One
// head at a time instead of four unrolled: 462 / 22.4.)
constexpr int kThreads = 64;
constexpr int kGrid = 128;      // CTAs of an SM, at most
constexpr uint64_t kInvTwoPi = 0x28be60db9391054aull;       // 2^64 / 2 pi,
constexpr uint64_t kInvTwoPiNext = 0x7f09d5f47d4d3770ull;   // and the 64 bits behind it

struct RotaryArgs {
  const void *q, *k;
  void *q_out, *k_out;
  const int32_t* pos;
  const double* freq;
  const int64_t* n_rows;
  int64_t rows, q_stride, k_stride, qo_stride, ko_stride;   // elements
  int hq, hkv, d, rot, lph_shift, parts;
  bool q_copy, k_copy;     // columns behind rot are copied (not in place)
  bool back;
  float magnitude;
};

// V elements as one load.
template <typename T, int V>
struct Vec {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if (kWords == 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x; w[1] = x.y; w[kWords > 2 ? 2 : 0] = x.z; w[kWords > 2 ? 3 : 0] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if (kWords == 4)
      *reinterpret_cast<uint4*>(p) =
          make_uint4(w[0], w[1], w[kWords > 2 ? 2 : 0], w[kWords > 2 ? 3 : 0]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ float get(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(w[i % kWords]);
    const uint32_t x = w[i / 2 % kWords];
    return __uint_as_float(i & 1 ? x & 0xFFFF0000u : x << 16);
  }
  // elements i and i + 1 (i even)
  __device__ __forceinline__ void set2(int i, float x, float y) {
    if (sizeof(T) == 4) {
      w[i % kWords] = __float_as_uint(x);
      w[(i + 1) % kWords] = __float_as_uint(y);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
      w[i / 2 % kWords] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
};

// frequency / 2 pi as a fraction of a turn, to 2^-62 of one: the double's 53 bits times 1 / 2 pi, whole
// turns dropped.  The first 64 bits of 1 / 2 pi leave 2^-64 of the frequency, so frequencies from 2 on
// take the next 64 too.  (Without, the angle at position 2^31 was 6e-8 turns off for a frequency of
// 1000, and had nothing to do with the position for 2^33.  For every frequency: calls of 64 rows 4.06
// us, 3.85 without, 3.92 so.)  Zero for what is no number below 2^52.
__device__ __forceinline__ uint64_t fraction(double frequency) {
  const uint64_t bits = (uint64_t)__double_as_longlong(frequency);
  const int e = (int)(bits >> 52) & 0x7FF, sh = 1075 - e;   // frequency = m 2^-sh
  if (e == 0 || sh <= 0 || sh >= 128) return 0;
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | 1ull << 52;
  uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  if (e > 1023) {
    const uint64_t next = __umul64hi(m, kInvTwoPiNext);
    lo += next;
    hi += lo < next ? 1 : 0;
  }
  const uint64_t r = sh < 64 ? lo >> sh | hi << (64 - sh) : hi >> (sh - 64);
  return bits >> 63 ? 0ull - r : r;
}
// Position * fraction in turns, modulo one, to 2^-32 (pos >= 0).
__device__ __forceinline__ uint32_t turns(uint32_t pos, uint64_t f) {
  return pos * (uint32_t)(f >> 32) + __umulhi(pos, (uint32_t)f);
}
__device__ __forceinline__ void sincos_turns(uint32_t t, float& s, float& c) {
  // quarters, and the rest from -1/8 to 1/8 of a turn
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const int32_t rest = (int32_t)(t - (quarter << 30));
  float sr, cr;
  sincospif((float)rest * 0x1p-31f, &sr, &cr);
  const bool swap = quarter & 1;
  s = swap ? cr : sr;
  c = swap ? sr : cr;
  if (quarter & 2) s = -s;
  if ((quarter + 1) & 2) c = -c;
}

// V: pairs of a lane.  kOwn: those whose sines it works out; the lanes that have the same pairs of
// other heads give it the rest.
template <typename T, int V, bool kHalf, int kOwn>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  const int lane = threadIdx.x & 31;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();   // nothing of the call before is read or written until it ends
  int64_t rows = a.rows;
  if (a.n_rows != nullptr) rows = min(rows, *a.n_rows);
  const int half = a.rot / 2, chunk = lane & ((1 << a.lph_shift) - 1);
  const int sub = lane >> a.lph_shift, heads_at_once = 32 >> a.lph_shift;
  const int heads = a.hq + a.hkv, i0 = chunk * V;   // the lane's pairs
  const bool turns_any = i0 < half;
  uint64_t f[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
    f[i] = turns_any ? fraction(a.freq[i0 + (sub & (V / kOwn - 1)) * kOwn + i]) : 0ull;
  // columns of the two loads
  const int c0 = kHalf ? i0 : 2 * i0, c1 = kHalf ? i0 + half : 2 * i0 + V;
  const int64_t items = rows * a.parts;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  int64_t it = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  auto row_of = [&](int64_t x) { return a.parts == 1 ? x : x / a.parts; };
  int32_t next = it < items ? a.pos[row_of(it)] : -1;   // (under way beside a row's work)
  for (; it < items; it += step) {
    const int64_t row = row_of(it);
    const int part = (int)(it - row * a.parts);
    const int32_t pos = next;
    next = it + step < items ? a.pos[row_of(it + step)] : -1;
    if (pos < 0) continue;
    const T* q = (const T*)a.q + row * a.q_stride;
    const T* k = (const T*)a.k + row * a.k_stride;
    T* qo = (T*)a.q_out + row * a.qo_stride;
    T* ko = (T*)a.k_out + row * a.ko_stride;
    auto from = [&](int h) { return h < a.hq ? q + h * a.d : k + (h - a.hq) * a.d; };
    auto to = [&](int h) { return h < a.hq ? qo + h * a.d : ko + (h - a.hq) * a.d; };
    int h = part * heads_at_once + sub;
    float s[V], c[V];
    {
      float so[kOwn], co[kOwn];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        sincos_turns(turns((uint32_t)pos, f[i]), so[i], co[i]);
        so[i] *= a.back ? -a.magnitude : a.magnitude;
        co[i] *= a.magnitude;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int src = (i / kOwn << a.lph_shift) + chunk;
        s[i] = kOwn == V ? so[i % kOwn] : __shfl_sync(0xffffffffu, so[i % kOwn], src);
        c[i] = kOwn == V ? co[i % kOwn] : __shfl_sync(0xffffffffu, co[i % kOwn], src);
      }
    }
#pragma unroll 4
    for (; h < heads; h += a.parts * heads_at_once) {
      if (!turns_any) continue;
      Vec<T, V> x, y, u, w;
      x.load(from(h) + c0);
      y.load(from(h) + c1);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        if (kHalf) {
          const float a0 = x.get(i), b0 = y.get(i), a1 = x.get(i + 1), b1 = y.get(i + 1);
          u.set2(i, a0 * c[i] - b0 * s[i], a1 * c[i + 1] - b1 * s[i + 1]);
          w.set2(i, a0 * s[i] + b0 * c[i], a1 * s[i + 1] + b1 * c[i + 1]);
        } else {
          const int j = i / 2, m = V / 2 + j;
          const float a0 = x.get(i), b0 = x.get(i + 1), a1 = y.get(i), b1 = y.get(i + 1);
          u.set2(i, a0 * c[j] - b0 * s[j], a0 * s[j] + b0 * c[j]);
          w.set2(i, a1 * c[m] - b1 * s[m], a1 * s[m] + b1 * c[m]);
        }
      }
      u.store(to(h) + c0);
      w.store(to(h) + c1);
    }
    // the columns that stay: four pieces of 16 bytes of a lane at a time
    constexpr int kE = 16 / (int)sizeof(T);
    const int first = a.q_copy ? 0 : a.hq, last = a.k_copy ? heads : a.hq;   // heads with such
    if (first >= last) continue;
    const int per = (a.d - a.rot) / kE, all = (last - first) * per;
    for (int p0 = part * 128 + lane; p0 < all; p0 += a.parts * 128) {
      uint4 z[4];
      int at[4], head[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = p0 + 32 * j, n = p / per;
        head[j] = p < all ? first + n : -1;
        at[j] = a.rot + (p - n * per) * kE;
        if (p < all) z[j] = *reinterpret_cast<const uint4*>(from(head[j]) + at[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (head[j] >= 0) *reinterpret_cast<uint4*>(to(head[j]) + at[j]) = z[j];
    }
  }
}

template <typename T, int V, bool kHalf, int kOwn>
cudaError_t launch_own(const RotaryArgs& a, cudaStream_t st) {
  int64_t grid = cdiv(a.rows * a.parts, kThreads / 32);
  const int64_t most = (int64_t)num_sms() * kGrid;
  if (grid > most) grid = most;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;   // (calls of 64 rows one after the other 2.6 us, 4.2 without)
  const cudaError_t e = cudaLaunchKernelEx(&cfg, rotary_kernel<T, V, kHalf, kOwn>, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}
template <typename T, int V, bool kHalf>
cudaError_t launch(RotaryArgs& a, cudaStream_t st) {
  const int chunks = (a.rot / 2 + V - 1) / V;
  a.lph_shift = 0;
  while ((1 << a.lph_shift) < chunks) ++a.lph_shift;
  const int at_once = 32 >> a.lph_shift;
  const int passes = (a.hq + a.hkv + at_once - 1) / at_once;
  // parts of a row: until every SM has 32 warps
  const int64_t want = (int64_t)num_sms() * 32;
  a.parts = 1;
  if (a.rows < want) {
    const int64_t p = want / a.rows;
    a.parts = (int)(p < passes ? p : passes);
  }
  // the sines of V pairs shared by the lanes of `at_once` heads
  if (V <= at_once) return launch_own<T, V, kHalf, 1>(a, st);
  if (V == 2 * at_once) return launch_own<T, V, kHalf, 2>(a, st);
  return launch_own<T, V, kHalf, 4>(a, st);
}
}  // namespace

cudaError_t launch_rotary(const RotaryShape& s, bool back, const void* q, int64_t q_stride,
                          const void* k, int64_t k_stride, const int32_t* pos, const double* freq,
                          int64_t rows, const int64_t* n_rows, void* q_out, int64_t qo_stride,
                          void* k_out, int64_t ko_stride, cudaStream_t st) {
  RotaryArgs a{q, k, q_out, k_out, pos, freq, n_rows, rows, q_stride, k_stride, qo_stride,
               ko_stride, s.hq, s.hkv, s.d, s.rot, 0, 1, q != q_out && s.rot < s.d,
               k != k_out && s.rot < s.d, back, s.magnitude};
  const bool half = s.layout == KV_ROTARY_HALF;
  if (s.dtype == KV_F32)
    return half ? launch<float, 4, true>(a, st) : launch<float, 4, false>(a, st);
  // bf16: 16 bytes a load where both of a lane's loads begin at multiples of them
  if (s.rot % 16 == 0)
    return half ? launch<__nv_bfloat16, 8, true>(a, st) : launch<__nv_bfloat16, 8, false>(a, st);
  return half ? launch<__nv_bfloat16, 4, true>(a, st) : launch<__nv_bfloat16, 4, false>(a, st);
}

}  // namespace kv
