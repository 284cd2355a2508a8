// Attention of one new token per sequence over the paged cache:
//   z_r = scale * q . k_r,  p = softmax(z) over the rows of the table,  o = sum_r p_r v_r.
//
// The step reads every K and V row once and little else (4 d G flops for 2 d elements): it is
// bound by that stream, or by latency when the cache is small.  So the rows are split evenly,
// whatever the lengths.  On GB300 (32 query heads over 8, bf16, d = 128; devices differ by 1 %):
// 128 ragged sequences of 8000 rows, 4.2 GB, 606 us (6.87 TB/s, 1.01 of the measured copy rate); 64 of
// 2000 rows 85 us (6.0 TB/s); one of 131000 rows 85 us (6.3 TB/s); 256 heads of 128 rows 11.0 us;
// one sequence of 500 rows 8.3 us.  fp32, 64 of 4000 rows: d = 128 317 us (6.6 TB/s), 96 254 us
// (6.1), 72 209 us (5.6), 64 163 us (6.4).
//
//   1. Every CTA reads the tables' lengths.  In tiles of RT rows, the units (table, head) laid
//      one after the other are one range [0, total): CTA c takes [total c / Ne, total (c + 1) /
//      Ne) and each of its warps an equal part of that.  A CTA boundary that falls inside a
//      short unit moves to the nearer end of it, so only long units cross CTAs.
//   2. A warp walks its tiles 32 at a time: lane i works out tile i (its table by a search
//      over 32 tables' running sums, then the page number).  Tiles are copied 16 bytes a lane
//      (cp.async), swizzled, into the warp's own ring of stages; the warp runs the online
//      softmax of paged_mma.cuh over them.  No CTA barrier in the loop.  (TMA boxes of 16 rows
//      by 128 bytes, four a tile, cost the issuing warp 430 cycles a tile of about 1100, and
//      618 us where these copies take 603.)
//   3. A unit held by one warp is written out by it.  The parts of a unit split between warps
//      are merged in shared memory; of one that crosses CTAs, each CTA leaves one part in the
//      workspace, and the last of them to finish (a ticket) merges those in order, so the
//      result does not depend on which that is.
//
// The new token's row comes from k_new / v_new: it is copied beside the stage that holds its
// place, put there when the stage has landed, and stored to its slot.
// Rows past a table's last one, and rows of pages outside the pool, are masked: their scores
// are -inf and their values zeros.  No CTA waits for another.
//
// The kernel is written for two kinds of pool (Rows and Codes below): rows of q's type, and rows of
// 8-bit codes with a scale for each block of 16 rows of a head, two of which are a tile.  Codes, the
// same GB300 and heads (e4m3, bf16 q unless stated): 128 ragged sequences of 8000 rows, 2.1 GB, 317 us
// (6.6 TB/s, 0.97 of the copy rate; int8 333 us, fp32 q 324 us); 64 of 2000 rows 55 us (4.7 TB/s);
// one of 131000 rows 49 us (5.4 TB/s; int8, fp32 q 56 us); 256 heads of 128 rows 9.3 us; one
// sequence of 500 rows 8.3 us.  Tiles of one block took 434 us on the 2.1 GB: what a tile costs
// beside its products is then spent every 16 rows, and two warps a scheduler hide little of it.
#pragma once

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "paged_mma.cuh"
#include "quant_mma.cuh"

namespace kv {
namespace {   // (each file that includes this has its own instances)

// Eight warps per SM and rings of 128 KB (144 where a row has three or six half segments, 160 where
// it has five), full of copies in flight: enough for the memory, and the SMs share it evenly.  With
// 24 KB a warp (192 KB per SM) some SMs finish a fifth before others: 622 us against 603 on the
// 4.2 GB cache.  Six warps per SM 610.
//
// They are two CTAs of four warps or one of eight.  Two even out ragged calls better; one makes
// half as many parts of a unit to be merged through the workspace, which counts where few units
// are cut many times.  CTAs of 4 / 8 warps, us, ragged lengths:
//   units                8           16          32          40          64          128
//   500 rows         8.2 / 8.8   9.8 / 10.5  10.7 / 11.0  11.1 / 11.3  11.6 / 11.7  13.2 / 13.6
//   2000            13.3 / 9.4  13.0 / 12.1  16.9 / 15.3  18.2 / 17.8  21.0 / 21.0  27.6 / 28.1
//   8000            15.5 / 13.9 23.2 / 21.5  31.2 / 30.5  35.1 / 35.1  48.4 / 48.8  75.5 / 76.2
// fp32, d = 72, 3000 rows: 10 units 15.6 / 14.7, 16 17.0 / 16.6, 38 24.8 / 25.4, 64 32.3 / 33.8.
constexpr int kSmWarps = 8;
// CTAs of eight warps: at most this many units, a quarter of the SMs (from there on the two are level,
// or four warps are ahead), and tiles for every CTA of four, as far as the host knows them from the
// tables' columns.  With fewer tiles neither is ahead throughout: of 8 to 32 units of equal lengths,
// four warps by 2 to 14 % at 500 to 700 rows, eight by 10 to 40 % at 300 rows and for 8 units of 1400 or
// 2000; of ragged ones, eight by 3 to 10 % from 700 rows.  Where the tables have columns for 131072
// rows and few are held: 8 units of 500 rows 8.4 / 8.5, of 2000 12.6 / 9.5, 40 units of 500 11.3 / 11.4.
// (Tiles of 16 rows.  Of codes, in tiles of 32 and so from half as many on: 8 units of 500 rows 8.3 / 8.9,
// 2000 11.7 / 11.3, 4000 15.0 / 9.6, 16000 17.8 / 16.1; 32 ragged units of 8000 24.3 / 22.3.)
constexpr int kLongUnits = 38;
constexpr int kMaxCtas = 320;
constexpr int kMaxCtasOfCodes = 480;
constexpr int kRingBytes = 20 * 1024;   // of a warp, at most (and four tiles)
// Tiles per CTA at least: a small call runs on as few CTAs as that allows.  One tile a warp: one
// sequence of 500 rows 8.2 us; with two 8.9, with four 11.2.
constexpr int kMinTiles = 4;
// A boundary inside a unit of at most this many tiles moves to the unit's nearer end: a part in
// the workspace and a ticket cost 2 us, the tiles less than that.  16 / 24 / 32 / 48 tiles: 256 heads
// of 128 rows 11.2 / 10.9 / 10.6 / 10.6 us; units of 500 rows (32 tiles), 8 of them 8.2 / 8.2 / 11.2 /
// 11.2, 16 9.8 / 9.8 / 11.4 / 11.4, 64 11.6 / 11.7 / 11.7 / 13.2, 128 13.2 / 13.2 / 13.1 / 15.2;
// units of 2000 rows level.  Those are tiles of 16 rows.  Of 32, 8 / 12 / 15 / 20 tiles: units of 500 rows
// (16 tiles), 8 of them 8.3 / 8.3 / 8.3 / 10.2 us; 64 ragged ones 10.5 / 10.5 / 10.5 / 10.7; 256 heads of
// 128 rows, all of at most 10 tiles, 11.8 / 9.4 / 9.4 / 9.4, two of them of 13 and 14 11.7 with 12, 11.0
// with 15 and 20.  Few units of 13 to 15 tiles pay for that: 8 of 384 / 416 / 448 / 480 / 500 rows 8.9 /
// 9.3 / 9.3 / 9.3 / 8.5 us with 15, 8.9 / 8.8 / 8.9 / 9.0 / 8.5 with 12; 32 of them 9.2 / 9.9 / 10.1 /
// 10.2 / 9.1 and 9.2 / 9.7 / 9.7 / 10.1 / 9.0.  (The rule knows a unit's length, not how many there are.)
template <int RT>
constexpr int kSnapTiles = RT == 32 ? 15 : 24;
// Part of a unit in the workspace: max[8], sum[8], then o[G][D].
constexpr int kPartHead = 16;
constexpr int kPartFloats = kPartHead + 8 * 128;

struct PagedArgs {
  const void *q, *kn, *vn;
  const int64_t *cu, *slots;
  int64_t slot_cap;
  void *kp, *vp;
  const int32_t *table, *lens;
  float *ks, *vs;   // scales of the blocks (pools of codes)
  void* out;
  WsHeader* hdr;
  uint32_t* tick;   // [k]: parts done of the unit that crosses CTA k's end
  float* part;      // two parts a CTA
  int U, Hp, G, d, shift, max_pages;
  int64_t num_pages, page_stride;
  pmma::Scale scale;
};

// Pools of rows of T.  H: 64-byte parts of a row.  Stages as wide as d needs: fp32 d = 72 in 5 instead
// of 6 parts took 8 % less time, bf16 d = 96 in 3 instead of 4 2 %.
template <typename T_, int H_>
struct Rows {
  using T = T_;
  using E = T_;                            // element of the pool
  using F = void;
  using Tl = pmma::Tile<T_, H_>;
  static constexpr int H = H_, kMaxStages = 4;
  static constexpr int kNewRow = H_ * 64;  // bytes of a new row beside a stage
  static constexpr int kWarps = kSmWarps;  // of an SM, in CTAs of four
  static constexpr bool kCodes = false;
};
// Pools of codes of the format F, for q, new rows and outputs of T, in NP pieces of 16 columns.  Up
// to 64 columns a tile is half as many bytes for two thirds of the instructions, and twelve warps an
// SM fit (64 ragged sequences of 4000 rows of 64: 58 us, with eight 66; 128 of 8000 183 and 214;
// 256 heads of 128 rows 8.3 and 7.8).
template <typename T_, typename F_, int NP>
struct Codes {
  using T = T_;
  using E = unsigned char;
  using F = F_;
  using Tl = qmma::Tile<T_, F_, NP>;
  static constexpr int kWarps = NP <= 4 ? 12 : kSmWarps;
  static constexpr int H = Tl::H, kMaxStages = NP <= 4 ? 3 : 4;
  static constexpr int kNewRow = NP * 16 * (int)sizeof(T_);
  static constexpr bool kCodes = true;
};
template <typename P_>
struct Cfg {
  using P = P_;
  using Tl = typename P::Tl;
  static constexpr int RT = Tl::RT, H = P::H;
  static constexpr int kRow = H * 64;                      // bytes of a row in a stage
  static constexpr int kStage = RT * 2 * kRow;             // of a tile, K and V
  static constexpr int kStages =
      kRingBytes / kStage < P::kMaxStages ? kRingBytes / kStage : P::kMaxStages;
  static_assert(kStages >= 2, "ring");
  static constexpr int kNewRow = P::kNewRow;
  // beside a stage: its new row of K and of V, and the block's scales
  static constexpr int kBeside = 2 * kNewRow + (P::kCodes ? 16 : 0);
  static constexpr int kSide = kStages * kBeside;          // of a warp
  // a copy instruction of a warp: kRows rows of kLanes 16-byte pieces
  static constexpr int kLanes = H <= 1 ? 4 : H <= 2 ? 8 : H <= 4 ? 16 : 32;
  static constexpr int kRows = 32 / kLanes;
};

template <typename C, int kPWarps>
struct PagedSmem {
  unsigned char ring[kPWarps][C::kStages * C::kStage];
  unsigned char side[kPWarps][C::kSide];
  float4 part4[kPWarps][2][2 * C::Tl::D];    // outputs of the warps' parts a and b (see below),
                                             // [query][column]
  uint32_t strip[kPWarps * 32];              // tiles before thread t's tables
  int32_t lens[kPWarps * 32];                // rows per table, where a thread has one table
  uint32_t wsum[kPWarps];
  uint32_t bnd[2];                           // the CTA's first tile and its end
  // the parts warp w leaves: of a unit that began before its tiles (a), of one that goes on
  // after them (b); unit or -1, and whether the unit of part a goes on as well
  float ml[kPWarps][2][16];                  // max[8], sum[8]
  int32_t a_unit[kPWarps], b_unit[kPWarps], a_open[kPWarps];
  int32_t some[kPWarps];                     // warp w has tiles
  uint2 ends[kPWarps][2];                    // first tile and end of the units of warp w's
                                             // first and last tiles
  int32_t won[2];                            // this CTA's part of a crossing unit was the last
};

// 32 tables in a warp: lane i holds table w0 + i's rows and the end of its tiles (all heads).
// (Tile numbers are 32 bits: the host refuses shapes that could hold 2^31 tiles.)
struct Window {
  int w0, len;
  uint32_t end;
};

template <int RT>
__device__ __forceinline__ int tiles_of(int len) { return (int)(((uint32_t)len + RT - 1) / RT); }

__device__ __forceinline__ int clamp_len(int len, int most) {
  return len < 0 ? 0 : len > most ? most : len;
}

__device__ __forceinline__ uint32_t warp_incl_scan(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// `base`: the tiles before table w0; `lens`: the lengths, cut to the table.
template <int RT, typename Lens>
__device__ __forceinline__ void load_window(Window& w, int w0, uint32_t base, const PagedArgs& a,
                                            Lens lens) {
  const int lane = threadIdx.x & 31;
  w.w0 = w0;
  w.len = w0 + lane < a.U ? lens(w0 + lane) : 0;
  w.end = base + warp_incl_scan((uint32_t)tiles_of<RT>(w.len) * a.Hp);
}
__device__ __forceinline__ uint32_t window_end(const Window& w) {
  return __shfl_sync(0xffffffffu, w.end, 31);
}
// Moves the window to the one that holds tile x (x < total, and not before the window).
template <int RT, typename Lens>
__device__ __forceinline__ void seek(Window& w, uint32_t x, const PagedArgs& a, Lens lens) {
#pragma unroll 1
  for (;;) {
    const uint32_t e = window_end(w);
    if (x < e || w.w0 + 32 >= a.U) return;
    load_window<RT>(w, w.w0 + 32, e, a, lens);
  }
}

// What a lane knows of one tile.
struct Desc {
  int32_t unit;
  int64_t at;            // element of the pool where the tile's first row begins; in pages of half
                         // a tile, of its first half
  int64_t at2;           // of its second half
  uint32_t word;         // see Word
  int64_t slot;          // where the new row (the unit's last) goes, or -1
  int64_t scale, scale2; // the blocks' scales (pools of codes)
};
constexpr uint32_t kFirst = 1u << 16, kLast = 1u << 17;
// A tile's rows in a word: kFirst / kLast: the unit's first / last tile.  Tiles of up to 16 rows: bits
// 0..15 rows that count, 24..27 the last row.  Of 32: bits 0..5 the number of rows, 18 and 19 halves
// that do not count.
template <int RT>
struct Word {
  static constexpr uint32_t kAll = RT == 32 ? ~0u : (1u << (RT & 31)) - 1u;
  static __device__ __forceinline__ uint32_t of(int n) {
    return RT == 32 ? (uint32_t)n : ((1u << n) - 1u) | (uint32_t)(n - 1) << 24;
  }
  static __device__ __forceinline__ uint32_t without(uint32_t w, bool lo, bool hi) {
    if (RT == 32) return w | (lo ? 1u << 18 : 0u) | (hi ? 1u << 19 : 0u);
    constexpr uint32_t low = (1u << (RT / 2)) - 1u;
    return w & ~((lo ? low : 0u) | (hi ? kAll & ~low : 0u));
  }
  static __device__ __forceinline__ bool whole(uint32_t w) {
    return RT == 32 ? (w & 0xC003Fu) == 32u : (w & kAll) == kAll;
  }
  static __device__ __forceinline__ uint32_t rows(uint32_t w) {
    if (RT != 32) return w & kAll;
    const uint32_t n = w & 63u, m = n == 32 ? ~0u : (1u << n) - 1u;
    return m & ~((w >> 18 & 1 ? 0xFFFFu : 0u) | (w >> 19 & 1 ? 0xFFFF0000u : 0u));
  }
  static __device__ __forceinline__ int last(uint32_t w) {
    return RT == 32 ? (int)(w & 63u) - 1 : (int)(w >> 24 & 15);
  }
};

template <typename T>
__device__ __forceinline__ void store2(T* p, float x, float y);
template <>
__device__ __forceinline__ void store2<float>(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}
template <>
__device__ __forceinline__ void store2<__nv_bfloat16>(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ void store4(float* p, const float4& v) {
  *reinterpret_cast<float4*>(p) = v;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& v) {
  uint2 w;
  w.x = pmma::bf16x2_of(v.x, v.y);
  w.y = pmma::bf16x2_of(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = w;
}
// 16 bytes from global to shared memory; `bytes` of them are read, the rest is zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {   // all groups but the last N
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The line-th 128 bytes of a tensor of `bytes`, if it has them, into L2.
__device__ __forceinline__ void prefetch_line(const void* p, int64_t line, int64_t bytes) {
  if (line * 128 < bytes)
    asm volatile("prefetch.global.L2 [%0];" ::"l"((const char*)p + line * 128));
}
__device__ __forceinline__ uint32_t atomic_add_acq_rel(uint32_t* p, uint32_t x) {
  uint32_t r;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(x) : "memory");
  return r;
}
// Merge of up to kB parts (max of q . k, sum, 4 outputs each; max -inf: none) into (M, L, acc).
// (A part whose every score is a NaN has max -inf too, and a sum and outputs of NaN: with factors
// of 0, not left out, they stay.)
template <int kB>
__device__ __forceinline__ void merge_parts(const float (&m)[kB], const float (&l)[kB],
                                            const float4 (&o)[kB], float c2, float& M, float& L,
                                            float4& acc) {
  float mn = M;
#pragma unroll
  for (int b = 0; b < kB; ++b) mn = fmaxf(mn, m[b]);
  const float base = mn == -INFINITY ? 0.f : mn;
  const float f = ptx::ex2((M - base) * c2);   // 0 while M is -inf
  M = mn;
  L *= f;
  acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    const float w = ptx::ex2((m[b] - base) * c2);
    L = fmaf(l[b], w, L);
    acc.x = fmaf(o[b].x, w, acc.x);
    acc.y = fmaf(o[b].y, w, acc.y);
    acc.z = fmaf(o[b].z, w, acc.z);
    acc.w = fmaf(o[b].w, w, acc.w);
  }
}

// A new row beside a stage (K's at `fresh`, V's kNewRow behind it), as row r of a block (quant_codes.cuh
// has the numbers): in the stage, where the block's rows begin `above` rows down, and in the pools at
// `at`.  scale: the block's, K's and V's; returned as they are afterwards.  K by the warp's first half, V
// by the other.
template <typename C>
__device__ __forceinline__ float2 put_rows(unsigned char* stage, int above,
                                           const unsigned char* fresh, const PagedArgs& a,
                                           int64_t at, int64_t scale_at, float2 scale, int r) {
  using T = typename C::P::T;
  using F = typename C::P::F;
  const int lane = threadIdx.x & 31, part = lane & 15, pieces = a.d / 16;
  const bool v = lane >= 16;
  unsigned char* pool = (unsigned char*)(v ? a.vp : a.kp) + at;
  auto place = [&](int row, int p) {
    return reinterpret_cast<uint4*>(stage + (v ? pmma::v_piece<C::RT, C::H>(above + row, p)
                                               : pmma::k_piece<C::RT, C::H>(above + row, p)));
  };
  // (16 elements of a lane: what makes a piece of codes)
  constexpr int kLoads = (int)sizeof(T);
  quant::Piece<T> x[kLoads];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    x[i].w = make_uint4(0u, 0u, 0u, 0u);
    if (part < pieces)
      x[i].w = reinterpret_cast<const uint4*>(fresh + (v ? C::kNewRow : 0))[part * kLoads + i];
    top = x[i].finite_top(top);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  top = __shfl_sync(0xffffffffu, top, lane & 16);
  const float old = r == 0 ? 0.f : v ? scale.y : scale.x;   // (a block that is begun anew has none)
  const float now = quant::scale_after<F>(top, old), inv = 1.f / now;
  if (now != old) {   // (raised, or in the place of a NaN or an infinity)
    for (int i = part; i < r * pieces; i += 16) {
      const int row = i / pieces;
      uint4* from = place(row, i - row * pieces);
      const uint4 c = quant::again<F>(*from, old * inv);
      *from = c;
      reinterpret_cast<uint4*>(pool)[i] = c;
    }
    if (part == 0) (v ? a.vs : a.ks)[scale_at] = now;
  }
  if (part < pieces) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = x[4 * i / quant::Piece<T>::kN].template codes<F>(4 * i % quant::Piece<T>::kN, inv, false);
    const uint4 c = make_uint4(w[0], w[1], w[2], w[3]);
    *place(r, part) = c;
    reinterpret_cast<uint4*>(pool + r * a.d)[part] = c;
  }
  return make_float2(__shfl_sync(0xffffffffu, now, 0), __shfl_sync(0xffffffffu, now, 16));
}

// kPWarps: warps of a CTA.
template <typename P, int kPWarps>
__global__ void __launch_bounds__(kPWarps * 32, P::kWarps / kPWarps)
paged_decode_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int kPThreads = kPWarps * 32;
  using C = Cfg<P>;
  using Tl = typename C::Tl;
  using T = typename P::T;
  using E = typename P::E;
  constexpr int RT = C::RT, S = C::kStages, D = Tl::D, H = P::H;
  constexpr int VE = 16 / (int)sizeof(E);   // elements of a piece of the pool
  constexpr int VN = 16 / (int)sizeof(T);   // and of a new row
  static_assert(!P::kCodes || RT == 2 * quant::kBlock, "a tile is two blocks");
  using W = Word<RT>;
  extern __shared__ unsigned char dsm_raw[];
  PagedSmem<C, kPWarps>& sm = *reinterpret_cast<PagedSmem<C, kPWarps>*>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int N = (int)gridDim.x, c = (int)blockIdx.x;
  const int page = 1 << a.shift, d = a.d, G = a.G;
  const int most = a.max_pages << a.shift;
  // a programmatic dependent launch: nothing of the call before is read or written until it ends
  ptx::griddep_launch_dependents();
  if constexpr (P::kCodes) {
    // (what the chain of loads below begins with, into L2 while the call before ends: no reading)
    const int64_t line = (int64_t)c * kPThreads + tid;
    prefetch_line(a.lens, line, (int64_t)a.U * 4);
    prefetch_line(a.table, line, (int64_t)a.U * a.max_pages * 4);
    prefetch_line(a.q, line, (int64_t)a.U * a.Hp * G * d * (int)sizeof(T));
    if (a.kn != nullptr) {
      prefetch_line(a.kn, line, (int64_t)a.U * a.Hp * d * (int)sizeof(T));
      prefetch_line(a.vn, line, (int64_t)a.U * a.Hp * d * (int)sizeof(T));
    }
  }
  ptx::griddep_wait();

  // ---- 1. tiles of all tables.  Up to 32 tables fit a warp's window: every warp finds its
  // tiles by itself.  More: each thread sums a strip of K tables, the CTA their prefix.
  const bool few = a.U <= 32;
  const int K = few ? 1 : (a.U + kPThreads - 1) / kPThreads;
  Window w;
  uint32_t total;
  {
    uint32_t sum = 0;
    for (int i = 0; i < K; ++i) {
      const int u = (few ? lane : tid) * K + i;
      int len = 1;
      if (u < a.U) {
        const int raw = a.lens[u];
        len = clamp_len(raw, most);
        if (raw != len && c == 0) raise_dev(a.hdr, DEV_PAGE_TABLE, (unsigned)u);
        sum += tiles_of<RT>(len);
        if (K == 1 && !few) sm.lens[u] = len;
      } else if (few) {
        len = 0;
      }
      if (few) {
        w.w0 = 0;
        w.len = len;
      }
      // tables with no rows: zeros, table u by CTA u % N
      uint32_t todo = __ballot_sync(0xffffffffu, u < a.U && len == 0);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const int ut = ((few ? 0 : warp * 32) + src) * K + i;
        if (ut % N != c || (few && warp != (src & (kPWarps - 1)))) continue;
        T* dst = (T*)a.out + (int64_t)ut * a.Hp * G * d;
        const int n16 = a.Hp * G * d * (int)sizeof(T) / 16;
        for (int x = lane; x < n16; x += 32)
          reinterpret_cast<uint4*>(dst)[x] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (few) {
      w.end = warp_incl_scan(sum * a.Hp);
      total = window_end(w);
    } else {
      const uint32_t incl = warp_incl_scan(sum);
      if (lane == 31) sm.wsum[warp] = incl;
      __syncthreads();
      uint32_t before = 0;
      total = 0;
#pragma unroll
      for (int k = 0; k < kPWarps; ++k) {
        if (k == warp) before = total;
        total += sm.wsum[k];
      }
      sm.strip[tid] = before + incl - sum;
      total *= a.Hp;
      __syncthreads();
    }
  }
  if (total == 0) return;
  const uint32_t want = (total + kMinTiles - 1) / kMinTiles;
  uint32_t Ne = want > (uint32_t)N ? N : want;   // CTAs that take tiles
  // One sequence: as many to each head, so that no CTA has parts of two (of 2000 rows 11.7 us with 126
  // CTAs for 8 heads).  Good for short ones, and for long ones as long as what it takes off is little.
  // With / without, us, one query a head: 2000 rows of 8 / 40 / 64 / 96 / 112 heads 9.7 / 11.3 / 13.7 /
  // 15.3 / 19.1 and 10.7 / 12.5 / 14.4 / 16.3 / 17.6; 32000 rows 18.1 / 59.0 / 94.9 / 124.6 / 180.5 and
  // 17.9 / 59.5 / 84.0 / 124.6 / 143.6 (64 heads leave 256 of 304 CTAs, 112 leave 224).
  if (P::kCodes && a.U == 1 && Ne > (uint32_t)a.Hp) Ne -= Ne % a.Hp;
  if (c >= (int)Ne) return;

  auto rows_of = [&](int u) { return K == 1 ? sm.lens[u] : clamp_len(a.lens[u], most); };
  // the window of tables that holds tile x
  auto find = [&](uint32_t x) {
    if (few) return;
    // the strip: the last one that starts at or before x, by 32nds, then among one's strips
    constexpr int kPer = kPThreads / 32;
    const int hi = __popc(__ballot_sync(0xffffffffu, sm.strip[lane * kPer] * a.Hp <= x)) - 1;
    const uint32_t at = sm.strip[hi * kPer + lane % kPer] * a.Hp;
    const int st = hi * kPer + __popc(__ballot_sync(0xffffffffu, lane < kPer && at <= x)) - 1;
    load_window<RT>(w, st * K, sm.strip[st] * a.Hp, a, rows_of);
    seek<RT>(w, x, a, rows_of);
  };
  // CTA k's first tile, moved to the nearer end of a short unit it falls in
  auto bound = [&](uint32_t k) -> uint32_t {
    const uint32_t x = total / Ne * k + total % Ne * k / Ne;
    if (x == 0 || x >= total) return x;
    find(x);
    const int j = __popc(__ballot_sync(0xffffffffu, w.end <= x));
    const uint32_t nt = tiles_of<RT>(__shfl_sync(0xffffffffu, w.len, j));
    const uint32_t tb = __shfl_sync(0xffffffffu, w.end, j) - nt * a.Hp;
    const uint32_t lo = tb + (x - tb) / nt * nt;
    if (nt > kSnapTiles<RT>) return x;
    return x - lo <= lo + nt - x ? lo : lo + nt;
  };
  // the CTA that holds tile x of a unit that crosses CTAs
  auto cta_of = [&](uint32_t x) {
    if (P::kCodes && total < 1u << 23)   // (a quarter of the instructions; Ne < 2^9)
      return (int)(((x + 1) * Ne + total - 1) / total) - 1;
    return (int)((((uint64_t)x + 1) * Ne + total - 1) / total) - 1;
  };
  // the CTA's ends: with few tables every warp finds both, else two warps find one each
  uint32_t b0 = 0, b1 = 0;
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    if (!few && warp != e) continue;
    b1 = bound(c + e);
    if (e == 0) b0 = b1;
    if (!few && lane == 0) sm.bnd[e] = b1;
  }
  if (!few) {
    __syncthreads();
    b0 = sm.bnd[0];
    b1 = sm.bnd[1];
  }
  const uint32_t span = b1 - b0;
  if (span == 0) return;   // uniform in the CTA
  // (rounded up: warp 0 has the CTA's first tile)
  const uint32_t xs = b0 + (uint32_t)(((uint64_t)span * warp + kPWarps - 1) / kPWarps);
  const uint32_t xe = b0 + (uint32_t)(((uint64_t)span * (warp + 1) + kPWarps - 1) / kPWarps);
  const int count = (int)(xe - xs);

  // ---- 2. this warp's tiles
  unsigned char* ring = sm.ring[warp];
  unsigned char* side = sm.side[warp];
  const uint32_t ring_u = ptx::smem_u32(ring), side_u = ptx::smem_u32(side);
  const int pieces = d / VE;   // 16-byte pieces of a row
  const int new_pieces = d / VN;
  const bool has_new = a.kn != nullptr;
  const T* qp = (const T*)a.q;
  Tl att;
  // cur holds tiles cur0..cur0 + 31, nxt the 32 behind them
  Desc cur, nxt;
  int cur0 = 0;
  // loads on nxt's account that have not been looked at: its pages, and cu of the last tile's
  // table and the next
  int32_t p_page = 0, p_page2 = 0, p_row = 0;   // p_row: head * page + row within the page
  int64_t p_c0 = 0, p_c1 = 0;
  bool ready = true;     // there are none

  // lane i's tile x0 + i (nothing past xe)
  auto describe = [&](uint32_t x0) {
    const uint32_t x = x0 + lane;
    bool open = x < xe;
    nxt.unit = -1;
    nxt.word = 0;
    p_page = p_page2 = 0;
    p_c0 = p_c1 = 0;
#pragma unroll 1
    for (;;) {
      const uint32_t wend = window_end(w);
      // tables whose tiles end at or before x
      int j = 0;
#pragma unroll
      for (int step = 16; step > 0; step >>= 1)
        if (__shfl_sync(0xffffffffu, w.end, j + step - 1) <= x) j += step;
      const int len = __shfl_sync(0xffffffffu, w.len, j & 31);
      const uint32_t e = __shfl_sync(0xffffffffu, w.end, j & 31);
      if (open && x < wend) {
        open = false;
        const int u = w.w0 + j;
        const uint32_t nt = tiles_of<RT>(len);
        const uint32_t y = x - (e - nt * a.Hp);
        const int h = (int)(y / nt), tt = (int)(y - h * nt);
        const int r0 = tt * RT, nv = len - r0 < RT ? len - r0 : RT;
        const int32_t* entry = a.table + (int64_t)u * a.max_pages + (r0 >> a.shift);
        p_page = entry[0];
        if (page < RT && nv > page) p_page2 = entry[1];
        nxt.word = W::of(nv);
        if (tt == 0) nxt.word |= kFirst;
        if (tt == (int)nt - 1) {
          nxt.word |= kLast;
          if (has_new) {
            p_c0 = a.cu[u];
            p_c1 = a.cu[u + 1];
          }
        }
        nxt.unit = u * a.Hp + h;
        p_row = h * page + (r0 & (page - 1));
        // the units of the warp's first and last tiles, for the merges
        const uint32_t first = x - tt;
        if (x == xs) sm.ends[warp][0] = make_uint2(first, first + nt);
        if (x == xe - 1) sm.ends[warp][1] = make_uint2(first, first + nt);
      }
      if (!__any_sync(0xffffffffu, open) || w.w0 + 32 >= a.U) break;
      load_window<RT>(w, w.w0 + 32, wend, a, rows_of);
    }
    ready = false;
  };
  // What describe() asked for, once it is there.  Rows of pages outside the pool do not count.
  // The slot of a unit's new row is only asked for here.
  auto settle = [&]() {
    if (ready) return;
    ready = true;
    const bool bad = p_page < 0 || p_page >= a.num_pages;
    const bool bad2 = p_page2 < 0 || p_page2 >= a.num_pages;
    nxt.at = (bad ? 0 : p_page) * a.page_stride + p_row * (int64_t)d;
    if (P::kCodes) {
      const int64_t blocks = (int64_t)a.Hp << (a.shift - 4);   // of a page
      nxt.scale = (bad ? 0 : p_page * blocks) + (p_row >> 4);
      nxt.scale2 = page < RT ? (bad2 ? 0 : p_page2 * blocks) + (p_row >> 4) : nxt.scale + 1;
      // (no row's place; a second page's at2 is one of page 0's.  What keeps a new row out of a page
      // outside the pool is its row in the mask, which does not count.)
      if (bad) nxt.at = -1;
    }
    nxt.at2 = (bad2 ? 0 : p_page2) * a.page_stride + p_row * (int64_t)d;
    if (bad || bad2) nxt.word = W::without(nxt.word, bad, page < RT ? bad2 : bad);
    if (bad || bad2) raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)nxt.unit);
    nxt.slot = -1;
    if (p_c1 > p_c0 && p_c1 > 0 && p_c1 <= a.slot_cap) nxt.slot = a.slots[p_c1 - 1];
  };
  // Lane src's tile of t into stage s: rows `i kRows + lr`, piece `pc` of each is this lane's.
  // (A piece's address is xor its row's low bits, and kRows divides 8: one address per lane for K
  // and one for V, xor and plus constants.)
  const int pc = lane % C::kLanes, lr = lane / C::kLanes;
  const uint32_t to = ring_u + pmma::k_piece<RT, H>(lr, pc);
  const uint32_t to_v = ring_u + pmma::v_piece<RT, H>(lr, pc);
  const int64_t from = (int64_t)lr * d + pc * VE;
  auto issue = [&](const Desc& t, int src, int s) {
    const int64_t at = __shfl_sync(0xffffffffu, (long long)t.at, src) + from;
    const uint32_t word = __shfl_sync(0xffffffffu, t.word, src);
    const uint32_t dst = to + s * C::kStage, dst_v = to_v + s * C::kStage;
    const E* ks = (const E*)a.kp + at;
    const E* vs = (const E*)a.vp + at;
    // in pages of half a tile: from a row of the first half to one of the second
    int64_t skip = 0;
    if (page < RT)
      skip = __shfl_sync(0xffffffffu, (long long)(t.at2 - t.at), src) - RT / 2 * (int64_t)d;
    if (pc < pieces) {
      // (without odd half segments V's stage is K's with an offset)
      auto copy = [&](int i, const E* k, const E* v, int bytes) {
        const uint32_t flip = ((i * C::kRows) & 7) << 4, row = i * C::kRows * 128;
        const uint32_t x = (dst ^ flip) + row;
        cp_async16(x, k, bytes);
        cp_async16(H % 2 == 0 ? x + C::kStage / 2 : (dst_v ^ flip) + row, v, bytes);
      };
      if (P::kCodes && d == D && W::whole(word)) {
        // rows that fill their pieces: the strides are constants (int8 on the 2.1 GB 333 us, 338 without)
        const E *k2 = ks + skip, *v2 = vs + skip;
#pragma unroll
        for (int i = 0; i < RT / C::kRows; ++i) {
          const bool second = i * C::kRows >= RT / 2;
          copy(i, (second ? k2 : ks) + i * C::kRows * D, (second ? v2 : vs) + i * C::kRows * D, 16);
        }
      } else if (W::whole(word)) {
#pragma unroll
        for (int i = 0; i < RT / C::kRows; ++i) {
          const int64_t o = i * C::kRows * d + (i * C::kRows >= RT / 2 ? skip : (int64_t)0);
          copy(i, ks + o, vs + o, 16);
        }
      } else {
        // rows that do not count are not read: zeros
        const uint32_t mask = W::rows(word);
#pragma unroll
        for (int i = 0; i < RT / C::kRows; ++i) {
          const int r = i * C::kRows + lr, n = mask >> r & 1 ? 16 : 0;
          const int64_t o = n == 0 ? -at : i * C::kRows * d + (r >= RT / 2 ? skip : (int64_t)0);
          copy(i, ks + o, vs + o, n);
        }
      }
    }
    const uint32_t beside = side_u + s * C::kBeside;
    if (has_new && (word & kLast)) {
      const int64_t u = __shfl_sync(0xffffffffu, t.unit, src);
      for (int p = lane; p < new_pieces; p += 32) {
        cp_async16(beside + p * 16, (const T*)a.kn + u * d + p * VN);
        cp_async16(beside + C::kNewRow + p * 16, (const T*)a.vn + u * d + p * VN);
      }
    }
    if (P::kCodes && lane == src) {
      // (a second block that has no rows: its scales are in the pool, or page 0's, and not used)
      cp_async4(beside + 2 * C::kNewRow, a.ks + t.scale);
      cp_async4(beside + 2 * C::kNewRow + 4, a.vs + t.scale);
      cp_async4(beside + 2 * C::kNewRow + 8, a.ks + t.scale2);
      cp_async4(beside + 2 * C::kNewRow + 12, a.vs + t.scale2);
    }
  };
  int32_t unit_a = -1, unit_b = -1;
  bool open_a = false;
  if (count > 0) {
    find(xs);
    describe(xs);
    settle();
    cur = nxt;
  }
  if (pieces < H * 4) {   // columns past d: zeros, for good
    for (int i = lane; i < S * C::kStage / 16; i += 32)
      reinterpret_cast<uint4*>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < S; ++i) {   // one group of copies a tile, empty past the last
    if (i < count) issue(cur, i, i);
    cp_async_commit();
  }
  if (count > 32) describe(xs + 32);
  bool whole = false;    // the warp has the unit from its first tile on
  int s = 0;             // stage of tile i
  uint32_t firsts = 0, lasts = 0, cuts = 0;   // cur's tiles: units' first, last; not all rows
  for (int i = 0; i < count; ++i) {
    if (i - cur0 == 32) {
      settle();
      cur = nxt;
      cur0 += 32;
      if (count - cur0 > 32) describe(xs + cur0 + 32);
    }
    const int src = i - cur0;
    if (src == 0) {
      firsts = __ballot_sync(0xffffffffu, cur.word & kFirst);
      lasts = __ballot_sync(0xffffffffu, cur.word & kLast);
      cuts = __ballot_sync(0xffffffffu, !W::whole(cur.word));
    }
    const bool last = lasts >> src & 1;
    if (i == 0 || (firsts >> src & 1)) {
      const int32_t unit = __shfl_sync(0xffffffffu, cur.unit, src);
      uint32_t qw[Tl::NQ];
      Tl::load_q(qp + (int64_t)unit * G * d, G, d, qw);
      att.set_q(qw, a.scale);
      att.begin();
      whole = firsts >> src & 1;
    }
    cp_async_wait<S - 1>();
    __syncwarp();
    {
      unsigned char* beside = side + s * C::kBeside;
      float4 scales = make_float4(1.f, 1.f, 1.f, 1.f);   // K's and V's of the first block, the second
      if (P::kCodes) scales = *reinterpret_cast<const float4*>(beside + 2 * C::kNewRow);
      uint32_t mask = W::kAll;
      if ((cuts >> src & 1) || (has_new && last)) {
        mask = __shfl_sync(0xffffffffu, cur.word, src);
        const int r = W::last(mask);   // the unit's last row, if this is its last tile
        mask = W::rows(mask);
        unsigned char* st = ring + s * C::kStage;
        if (has_new && last) {
          const int64_t slot = __shfl_sync(0xffffffffu, (long long)cur.slot, src);
          const int32_t unit = __shfl_sync(0xffffffffu, cur.unit, src);
          const bool in_pool = slot >= 0 && slot < (a.num_pages << a.shift);
          if (slot != -1 && !in_pool && lane == 0) raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)unit);
          const int64_t at = (slot >> a.shift) * a.page_stride +
                             (((int64_t)(unit % a.Hp) << a.shift) + (slot & (page - 1))) * d;
          if constexpr (P::kCodes) {
            // (only in its own block, whose scale and rows are at hand)
            const bool hi = r >= quant::kBlock;
            const int rb = r & (quant::kBlock - 1), above = hi ? quant::kBlock : 0;
            const int64_t block_at =
                hi && page >= RT
                    ? __shfl_sync(0xffffffffu, (long long)cur.at, src) + quant::kBlock * d
                    : __shfl_sync(0xffffffffu, (long long)(hi ? cur.at2 : cur.at), src);
            const int64_t sc =
                __shfl_sync(0xffffffffu, (long long)(hi ? cur.scale2 : cur.scale), src);
            if (in_pool && (mask >> r & 1) && at == block_at + rb * d) {
              const float2 now =
                  put_rows<C>(st, above, beside, a, block_at, sc,
                              hi ? make_float2(scales.z, scales.w) : make_float2(scales.x, scales.y),
                              rb);
              (hi ? scales.z : scales.x) = now.x;
              (hi ? scales.w : scales.y) = now.y;
            } else if (in_pool && lane == 0) {
              raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)unit);
            }
          } else if (in_pool) {
            // the new row, to its place in the tile and to its slot
            mask |= 1u << r;
            for (int p = lane; p < pieces; p += 32) {
              const uint4 kx = *reinterpret_cast<const uint4*>(beside + p * 16);
              const uint4 vx = *reinterpret_cast<const uint4*>(beside + C::kNewRow + p * 16);
              *reinterpret_cast<uint4*>(st + pmma::k_piece<RT, H>(r, p)) = kx;
              *reinterpret_cast<uint4*>(st + pmma::v_piece<RT, H>(r, p)) = vx;
              *reinterpret_cast<uint4*>((T*)a.kp + at + p * (16 / (int)sizeof(T))) = kx;
              *reinterpret_cast<uint4*>((T*)a.vp + at + p * (16 / (int)sizeof(T))) = vx;
            }
          }
        }
        if (P::kCodes) {   // blocks of no rows: what was copied is no scale
          if ((mask & 0xFFFFu) == 0) scales.x = scales.y = 1.f;
          if (mask >> 16 == 0) scales.z = scales.w = 1.f;
        }
        __syncwarp();
      }
      if constexpr (P::kCodes) att.tile(ring_u + s * C::kStage, mask, a.scale.c2, scales);
      else att.tile(ring_u + s * C::kStage, mask, a.scale.c2);
      __syncwarp();   // every lane is done with stage s
      const int n = src + S;
      if (i + S < count) {
        if (n >= 32) settle();
        issue(n < 32 ? cur : nxt, n & 31, s);
      }
      cp_async_commit();
    }
    // ---- the end of a unit, or of the warp's tiles
    if (last || i == count - 1) {
      const int32_t unit = __shfl_sync(0xffffffffu, cur.unit, src);
      att.finish();
      if (whole && last) {
#pragma unroll
        for (int e = 0; e < Tl::kQ; ++e) {
          const int g = Tl::query(e);
          if (g >= G) continue;
          const float l = att.sum_of(e), inv = l != 0.f ? 1.f / l : 0.f;
          T* dst = (T*)a.out + ((int64_t)unit * G + g) * d;
#pragma unroll
          for (int t = 0; t < Tl::kPairs; ++t) {
            const float2 x = att.pair(t, e);
            if (Tl::column(t) < d) store2(dst + Tl::column(t), x.x * inv, x.y * inv);
          }
        }
      } else {
        // a part of the unit
        if (whole) {
          unit_b = unit;
        } else {
          unit_a = unit;
          open_a = !last;
        }
        float* dst = reinterpret_cast<float*>(sm.part4[warp][whole]);
#pragma unroll
        for (int e = 0; e < Tl::kQ; ++e) {
          const int g = Tl::query(e);
          if (Tl::owns_sums()) {
            sm.ml[warp][whole][g] = att.max_of(e);
            sm.ml[warp][whole][8 + g] = att.sum_of(e);
          }
#pragma unroll
          for (int t = 0; t < Tl::kPairs; ++t)
            *reinterpret_cast<float2*>(dst + g * D + Tl::column(t)) = att.pair(t, e);
        }
      }
    }
    if (++s == S) s = 0;
  }

  // ---- 3. what the warps leave
  if (lane == 0) {
    sm.a_unit[warp] = unit_a;
    sm.a_open[warp] = open_a ? 1 : 0;
    sm.b_unit[warp] = unit_b;
    sm.some[warp] = count > 0 ? 1 : 0;
  }
  __syncthreads();
  // Heads: lane 0 stands for the unit of warp 0's part a, lane i > 0 for that of warp
  // i - 1's part b.  A head's unit goes on in the parts a of the warps behind it, up to
  // the first warp with tiles whose part a (if any) ends there; if there is none it crosses
  // the CTA's end.
  int32_t unit = -1;
  uint32_t part_a, stops;
  {
    const bool in = lane < kPWarps;
    const int32_t ua = in ? sm.a_unit[lane] : -1, ub = in ? sm.b_unit[lane] : -1;
    part_a = __ballot_sync(0xffffffffu, ua >= 0);
    stops = __ballot_sync(0xffffffffu, in && sm.some[lane] && !sm.a_open[lane]);
    const int32_t before = __shfl_up_sync(0xffffffffu, ub, 1);
    unit = lane == 0 ? ua : lane <= kPWarps ? before : -1;
  }
  const uint32_t after = ~0u << (lane == 0 ? 1 : lane & 15), stop = stops & after;
  uint32_t members = part_a & after & (stop ? (stop ^ (stop - 1)) : ~0u);
  if (lane == 0 && (stops & 1)) members = 0;
  const uint32_t heads = __ballot_sync(0xffffffffu, unit >= 0);
  const uint32_t cross = __ballot_sync(0xffffffffu, unit >= 0 && (lane == 0 || stop == 0));

  const int nsl = G * (D / 4);   // 4-float slices of a part's output
  for (uint32_t todo = heads; todo; todo &= todo - 1) {
    const int i = __ffs(todo) - 1;
    const int32_t un = __shfl_sync(0xffffffffu, unit, i);
    uint32_t mem = __shfl_sync(0xffffffffu, members, i);
    for (int idx = tid; idx < nsl; idx += kPThreads) {
      const int g = idx / (D / 4), col = (idx - g * (D / 4)) * 4;
      float m[kPWarps], l[kPWarps];
      float4 o[kPWarps];
#pragma unroll
      for (int k = 0; k < kPWarps; ++k) {
        // warp k's part: b where the unit begins with it, else a
        const bool b = i == k + 1, in = b || (mem >> k & 1) || (i == 0 && k == 0);
        m[k] = in ? sm.ml[k][b][g] : -INFINITY;
        l[k] = in ? sm.ml[k][b][8 + g] : 0.f;
        o[k] = in ? sm.part4[k][b][(g * D + col) / 4]
                  : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float M = -INFINITY, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      merge_parts<kPWarps>(m, l, o, a.scale.c2, M, L, acc);
      if (cross >> i & 1) {
        float* Q = a.part + (int64_t)(2 * c + (i == 0 ? 0 : 1)) * kPartFloats;
        if (col == 0) {
          Q[g] = M;
          Q[8 + g] = L;
        }
        *reinterpret_cast<float4*>(Q + kPartHead + g * D + col) = acc;
      } else if (col < d) {
        const float inv = L != 0.f ? 1.f / L : 0.f;
        store4((T*)a.out + ((int64_t)un * G + g) * d + col,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      }
    }
  }

  if (cross == 0) return;   // uniform in the CTA

  // units that cross CTAs (at most the one that began before this CTA and the one that goes on
  // after it): the last of a unit's CTAs to get here merges its parts
  const int i1 = 31 - __clz((int)cross);   // the second's head, if it is not 0
  const int32_t units[2] = {cross & 1 ? __shfl_sync(0xffffffffu, unit, 0) : -1,
                            i1 > 0 ? __shfl_sync(0xffffffffu, unit, i1) : -1};
  int first[2], parts[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const uint2 ends = y == 0 ? sm.ends[0][0] : sm.ends[i1 > 0 ? i1 - 1 : 0][1];
    first[y] = units[y] >= 0 ? cta_of(ends.x) : 0;
    parts[y] = units[y] >= 0 ? cta_of(ends.y - 1) - first[y] + 1 : 0;
  }
  __syncthreads();   // the CTA's parts are written
  if constexpr (P::kCodes) {
    // (a thread for each: the release of the CTA's parts and the acquiring of the others' in one)
    if (tid < 2) {
      const int32_t un = tid == 0 ? units[0] : units[1];
      const int at = tid == 0 ? first[0] : first[1], of = tid == 0 ? parts[0] : parts[1];
      sm.won[tid] = un >= 0 && atomic_add_acq_rel(&a.tick[at], 1u) == (uint32_t)of - 1;
      if (sm.won[tid]) a.tick[at] = 0u;
    }
    __syncthreads();
    const int n0 = sm.won[0] ? parts[0] : 0, n1 = sm.won[1] ? parts[1] : 0;
    if (n0 + n1 == 0) return;
    // The parts come through the rings, which are free now: many at a time, of both units at once, with
    // little code.  (Few CTAs get here, so its instructions are not at hand; one unit after the other,
    // 8 ragged sequences of 2000 rows took 18.8 us.)
    const int part4s = (kPartHead + G * D) / 4;   // 16-byte pieces of a part
    // The parts of a unit are summed `half` at a time, whether the CTA has one unit or two: what it
    // has depends on which CTA was the last, and the sums shall not.
    const int half = kPWarps * S * C::kStage / 32 / part4s;   // half of what the rings hold
    const int room = n0 > 0 && n1 > 0 ? half : 2 * half;
    constexpr int kSlices = (8 * (D / 4) + kPThreads - 1) / kPThreads;   // of a thread, at most
    const uint32_t to = ptx::smem_u32(sm.ring);
    const float* ring_f = reinterpret_cast<const float*>(sm.ring);
    float M[2][kSlices], L[2][kSlices];
    float4 acc[2][kSlices];
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int j = 0; j < kSlices; ++j) {
        M[y][j] = -INFINITY;
        L[y][j] = 0.f;
        acc[y][j] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll 1
    for (int k0 = 0; k0 < max(n0, n1); k0 += room) {
      // parts k0.. of the first unit at the ring's beginning, of the second behind them
      const int c0 = max(min(room, n0 - k0), 0), c1 = max(min(room, n1 - k0), 0);
#pragma unroll 1
      for (int k = warp; k < c0 + c1; k += kPWarps) {
        const int y = k >= c0, of = k0 + (y ? k - c0 : k);
        // (the unit is the second of its first CTA)
        const int slot = 2 * ((y ? first[1] : first[0]) + of) + (of == 0 ? 1 : 0);
        const float* W = a.part + (int64_t)slot * kPartFloats + lane * 4;
        const uint32_t dst = to + (k * part4s + lane) * 16;
#pragma unroll 4
        for (int i = 0; i < part4s - lane; i += 32) cp_async16(dst + i * 16, W + i * 4);
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncthreads();
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int n = y ? c1 : c0;
        const float* in = ring_f + (y ? c0 * part4s * 4 : 0);
        if (n == 0) continue;
#pragma unroll
        for (int j = 0; j < kSlices; ++j) {
          const int idx = tid + j * kPThreads, g = idx / (D / 4);
          if (idx >= nsl) continue;
#pragma unroll 1
          for (int from = 0; from < n; from += half) {
            const float* at = in + from * part4s * 4;
            const int count = min(half, n - from);
            float mn = M[y][j];
#pragma unroll 4
            for (int k = 0; k < count; ++k) mn = fmaxf(mn, at[k * part4s * 4 + g]);
            const float base = mn == -INFINITY ? 0.f : mn;
            const float f = ptx::ex2((M[y][j] - base) * a.scale.c2);   // 0 while M is -inf
            float4 o = acc[y][j];
            float l = L[y][j] * f;
            o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll 4
            for (int k = 0; k < count; ++k) {
              const float* W = at + k * part4s * 4;
              const float w = ptx::ex2((W[g] - base) * a.scale.c2);
              const float4 x = *reinterpret_cast<const float4*>(W + kPartHead + idx * 4);
              l = fmaf(W[8 + g], w, l);
              o.x = fmaf(x.x, w, o.x);
              o.y = fmaf(x.y, w, o.y);
              o.z = fmaf(x.z, w, o.z);
              o.w = fmaf(x.w, w, o.w);
            }
            M[y][j] = mn;
            L[y][j] = l;
            acc[y][j] = o;
          }
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if ((y ? n1 : n0) == 0) continue;
#pragma unroll
      for (int j = 0; j < kSlices; ++j) {
        const int idx = tid + j * kPThreads, g = idx / (D / 4), col = (idx - g * (D / 4)) * 4;
        if (idx >= nsl || col >= d) continue;
        const float inv = L[y][j] != 0.f ? 1.f / L[y][j] : 0.f;
        store4((T*)a.out + ((int64_t)units[y] * G + g) * d + col,
               make_float4(acc[y][j].x * inv, acc[y][j].y * inv, acc[y][j].z * inv,
                           acc[y][j].w * inv));
      }
    }
    return;
  }
  if (tid == 0) {
    __threadfence();
    uint32_t drawn[2] = {0, 0};
#pragma unroll
    for (int y = 0; y < 2; ++y)
      if (units[y] >= 0) drawn[y] = atomicAdd(&a.tick[first[y]], 1u);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      sm.won[y] = units[y] >= 0 && drawn[y] == (uint32_t)parts[y] - 1;
      if (sm.won[y]) atomicExch(&a.tick[first[y]], 0u);
    }
    __threadfence();
  }
  __syncthreads();
  // groups of threads take the parts in turn, and their sums are added in order
  const int groups = nsl < kPThreads ? kPThreads / nsl : 1;
#pragma unroll 1
  for (int y = 0; y < 2; ++y) {
    if (!sm.won[y]) continue;
#pragma unroll 1
    for (int sl = 0; sl < nsl; sl += kPThreads) {
      const int grp = nsl < kPThreads ? tid / nsl : 0, idx = sl + tid - grp * nsl;
      const int g = idx / (D / 4), col = (idx - g * (D / 4)) * 4;
      const bool in_part = grp < groups && idx < nsl;
      float M = -INFINITY, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      // a round of loads: as many parts as there are, or 16
      auto take = [&](int k0, auto parts_at_once) {
        constexpr int kB = decltype(parts_at_once)::value;
        float m[kB], l[kB];
        float4 o[kB];
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const int k = k0 + b * groups;
          // (the unit is the second of its first CTA)
          const float* W = a.part + (int64_t)(2 * (first[y] + k) + (k == 0 ? 1 : 0)) * kPartFloats;
          const bool in = k < parts[y];
          m[b] = in ? __ldcg(W + g) : -INFINITY;
          l[b] = in ? __ldcg(W + 8 + g) : 0.f;
          o[b] = in ? __ldcg(reinterpret_cast<const float4*>(W + kPartHead + g * D + col))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        merge_parts<kB>(m, l, o, a.scale.c2, M, L, acc);
      };
      if (in_part && parts[y] <= 8 * groups) {
        take(grp, std::integral_constant<int, 8>());
      } else if (in_part) {
#pragma unroll 1
        for (int k0 = grp; k0 < parts[y]; k0 += 16 * groups)
          take(k0, std::integral_constant<int, 16>());
      }
      if (groups > 1) {
        // (where the warp's parts were)
        sm.part4[warp][0][2 * lane] = acc;
        sm.part4[warp][0][2 * lane + 1] = make_float4(M, L, 0.f, 0.f);
        __syncthreads();
        for (int k = 1; grp == 0 && k < groups; ++k) {
          const int t = tid + k * nsl;
          const float4* p = sm.part4[t >> 5][0] + 2 * (t & 31);
          const float m[1] = {p[1].x}, l[1] = {p[1].y};
          const float4 o[1] = {p[0]};
          merge_parts<1>(m, l, o, a.scale.c2, M, L, acc);
        }
        __syncthreads();
      }
      if (in_part && grp == 0 && col < d) {
        const float inv = L != 0.f ? 1.f / L : 0.f;
        store4((T*)a.out + ((int64_t)units[y] * G + g) * d + col,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      }
    }
  }
}

// ------------------------------------- host side ----------------------------------------

constexpr size_t kTickBytes = 2048;
static_assert(kMaxCtasOfCodes * sizeof(uint32_t) <= kTickBytes, "tickets");

template <typename P, int kPWarps>
cudaError_t launch_w(const PagedShape& s, const PagedArgs& a, int64_t tiles, cudaStream_t st) {
  using C = Cfg<P>;
  constexpr int per_sm = P::kWarps / kPWarps;
  constexpr size_t smem = sizeof(PagedSmem<C, kPWarps>) + 1024;
  static_assert(per_sm * (smem + 1024) <= 228 * 1024 && smem <= 227 * 1024, "CTAs per SM");
  static std::atomic<int> slot[kMaxDevices];
  const int ok = per_device(slot, []() {
    return cudaFuncSetAttribute(paged_decode_kernel<P, kPWarps>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem) == cudaSuccess ? 1 : 0;
  });
  if (!ok) return cudaErrorInvalidConfiguration;
  // no more CTAs than the tables could ever fill
  int64_t grid = cdiv(tiles, kMinTiles);
  if (grid > per_sm * num_sms()) grid = per_sm * num_sms();
  constexpr int64_t most = P::kCodes ? kMaxCtasOfCodes : kMaxCtas;
  if (grid > most) grid = most;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kPWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  // A programmatic dependent launch costs the host 0.8 us: worth it where the call fills the SMs
  // (256 heads of 128 rows 10.9 us against 11.4), not where the host is the slower side (one
  // sequence of 500 rows: 8.1 us on the device either way, 9.2 against 10.0 us from Python).
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  // Codes: quant_decode_attn's call costs the host 3 us (csrc/binding.cpp), so always: 8.7 us a call of
  // 500 rows from Python, 10.3 without.
  cfg.numAttrs = P::kCodes || grid >= per_sm * num_sms() ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<P, kPWarps>, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <typename P>
cudaError_t launch_t(const PagedShape& s, const PagedArgs& a, cudaStream_t st) {
  const int64_t units = (int64_t)s.seqs * s.Hkv;
  // tiles that the tables could hold
  const int64_t tiles = units * cdiv((int64_t)s.max_pages * s.page, Cfg<P>::RT);
  constexpr int64_t least = 2 * kMinTiles * 16 / (Cfg<P>::RT < 16 ? 16 : Cfg<P>::RT);   // an SM
  const bool few_long = units <= kLongUnits && tiles >= least * num_sms();
  return few_long ? launch_w<P, 8>(s, a, tiles, st) : launch_w<P, 4>(s, a, tiles, st);
}

size_t ws_bytes(int ctas) {
  return kWsHeader + kTickBytes + (size_t)2 * ctas * kPartFloats * sizeof(float);
}

PagedArgs args(const PagedShape& s, const void* q, const void* kn, const void* vn,
               const int64_t* cu, const int64_t* slots, int64_t slot_capacity, void* kp, void* vp,
               float* ks, float* vs, const int32_t* table, const int32_t* lens, float scale,
               void* out, char* ws) {
  int shift = 0;
  while ((1 << shift) < s.page) ++shift;
  const float c2 = fabsf(scale) * 1.4426950408889634f;   // times log2 e
  const uint32_t flip = scale >= 0.f ? 0u : s.dtype == KV_BF16 ? 0x80008000u : 0x80000000u;
  return PagedArgs{q, kn, vn, cu, slots, slot_capacity, kp, vp, table, lens, ks, vs, out,
                   reinterpret_cast<WsHeader*>(ws), reinterpret_cast<uint32_t*>(ws + kWsHeader),
                   reinterpret_cast<float*>(ws + kWsHeader + kTickBytes),
                   (int)s.U(), s.Hp(),
                   s.G(), s.d, shift, s.max_pages, s.num_pages, s.page_stride,
                   pmma::Scale{c2 > FLT_MIN ? c2 : FLT_MIN, flip}};
}

}  // namespace
}  // namespace kv
