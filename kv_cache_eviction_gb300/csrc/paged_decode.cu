// Attention of one new token per sequence over the paged cache:
//   z_r = scale * q . k_r,  p = softmax(z) over the rows of the table,  o = sum_r p_r v_r.
//
// The step reads every K and V row once and little else: it is bound by that stream, or by
// latency when the cache is small.  So the rows are split evenly, whatever the lengths, and
// every SM keeps close to 200 KB of loads in flight.
//
//   1. Every CTA (one per SM, 8 warps) reads the tables' lengths.  In tiles of RT rows, the
//      units (table, head) laid one after the other are one range [0, total): CTA c takes
//      [total c / Ne, total (c + 1) / Ne) and a warp an eighth of that.  A CTA boundary inside a
//      short unit moves to the nearer end of it, so only long units cross CTAs.
//   2. A warp walks its tiles 32 at a time: lane i works out tile i (its table by a search
//      over 32 tables' running sums, then the page number) and later issues its TMA boxes.
//      K and V tiles land, swizzled, in the warp's own ring of stages; the warp runs the
//      online softmax of paged_mma.cuh over them.  No CTA barrier in the loop.
//   3. A unit held by one warp is written out by it.  The parts of a unit split between warps
//      are merged in shared memory; of one that crosses CTAs, each CTA leaves one part in the
//      workspace, and the last of them to finish (a ticket) merges those in order, so the
//      result does not depend on which that is.
//
// The new token's row comes from k_new / v_new: it is copied beside the stage that holds its
// place, put there when the stage has landed, and stored to its slot.
// Rows past a table's last one, and rows of pages outside the pool, are masked: their scores
// are -inf and their values zeros.  No CTA waits for another.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "paged_mma.cuh"

namespace kv {
namespace {

constexpr int kPWarps = 8;
constexpr int kPThreads = kPWarps * 32;
constexpr int kMaxCtas = 160;
constexpr int kRingBytes = 24 * 1024;   // of a warp
constexpr int kSideBytes = 3 * 1024;    // of a warp: the new rows of its stages
constexpr int kMaxStages = 6;
// Tiles per CTA at least: a small call runs on as few CTAs as that allows.
constexpr int kMinTiles = 16;
// A CTA boundary inside a unit of at most this many tiles moves to the unit's nearer end.
constexpr int kSnapTiles = 16;
// Part of a unit in the workspace or in shared memory: max[8], sum[8], then o[G][D].
constexpr int kPartHead = 16;
constexpr int kPartFloats = kPartHead + 8 * 128;

struct PagedArgs {
  const void *q, *kn, *vn;
  const int64_t *cu, *slots;
  int64_t slot_cap;
  void *kp, *vp;
  const int32_t *table, *lens;
  void* out;
  WsHeader* hdr;
  uint32_t* tick;
  float* part;
  int U, Hp, G, d, shift, max_pages;
  int64_t num_pages, page_stride;
  float c2;   // softmax scale * log2 e
};

template <typename T, int NSEG>
struct Cfg {
  using Tl = pmma::Tile<T, NSEG>;
  static constexpr int RT = Tl::RT;
  static constexpr int kRow = NSEG * 128;                  // bytes of a row in a stage
  static constexpr int kHalf = RT * kRow;                  // K, then V
  static constexpr int kStages = kRingBytes / (2 * kHalf);
  static_assert(kStages >= 3 && kStages <= kMaxStages, "ring");
  static_assert(kStages * 2 * kRow <= kSideBytes, "new rows");
};

struct PagedSmem {
  unsigned char ring[kPWarps][kRingBytes];   // after the stream: the parts of the units
  unsigned char side[kPWarps][kSideBytes];
  uint32_t strip[kPThreads];                 // tiles before thread t's tables
  uint32_t wsum[kPWarps];
  uint32_t bnd[2];                           // the CTA's first tile and its end
  uint64_t full[kPWarps][kMaxStages];
  // the parts warp w leaves: of a unit that began before its tiles (a), of one that goes on
  // after them (b); unit or -1, and whether the unit of part a goes on as well
  int32_t a_unit[kPWarps], b_unit[kPWarps], a_open[kPWarps];
  int32_t some[kPWarps];                     // warp w has tiles
  uint32_t start[kPWarps + 1], end[kPWarps + 1];   // units of warp 0's part a, of warps' parts b
  int32_t win[2];
};
static_assert(2 * kPWarps * kPartFloats * 4 <= kPWarps * kRingBytes, "parts fit the rings");

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
// `base`: the tiles before table w0.
template <int RT>
__device__ __forceinline__ void load_window(Window& w, int w0, uint32_t base, const PagedArgs& a) {
  const int lane = threadIdx.x & 31;
  w.w0 = w0;
  w.len = w0 + lane < a.U ? clamp_len(a.lens[w0 + lane], a.max_pages << a.shift) : 0;
  w.end = base + warp_incl_scan((uint32_t)tiles_of<RT>(w.len) * a.Hp);
}
__device__ __forceinline__ uint32_t window_end(const Window& w) {
  return __shfl_sync(0xffffffffu, w.end, 31);
}
// Moves the window to the one that holds tile x (x < total, and not before the window).
template <int RT>
__device__ __forceinline__ void seek(Window& w, uint32_t x, const PagedArgs& a) {
  for (;;) {
    const uint32_t e = window_end(w);
    if (x < e || w.w0 + 32 >= a.U) return;
    load_window<RT>(w, w.w0 + 32, e, a);
  }
}

// What a lane knows of one tile.
struct Desc {
  int32_t unit;
  int32_t page, page2;   // page2: of the tile's second 8 rows, when a page holds 8
  int32_t row;           // row of the pool's page: head * page + first row within the page
  int32_t tt, nt;        // the tile within its unit, and the unit's tiles
  uint32_t mask;         // rows that count; kFirst / kLast: the unit's first / last tile
  int64_t slot;          // where the new row (the unit's last) goes, or -1
};
constexpr uint32_t kFirst = 1u << 16, kLast = 1u << 17;

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
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Running merge of parts: (M, L, acc) with one part's (m, l, o).
__device__ __forceinline__ void merge_part(float m, float l, const float4& o, float& M, float& L,
                                           float4& acc) {
  if (m == -INFINITY) return;
  const float mn = fmaxf(M, m);
  const float f = ptx::ex2(M - mn), w = ptx::ex2(m - mn);   // f is 0 while M is -inf
  M = mn;
  L = fmaf(L, f, l * w);
  acc.x = fmaf(acc.x, f, o.x * w);
  acc.y = fmaf(acc.y, f, o.y * w);
  acc.z = fmaf(acc.z, f, o.z * w);
  acc.w = fmaf(acc.w, f, o.w * w);
}

template <typename T, int NSEG>
__global__ void __launch_bounds__(kPThreads, 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const PagedArgs a) {
  using C = Cfg<T, NSEG>;
  using Tl = typename C::Tl;
  constexpr int RT = C::RT, S = C::kStages, NT = Tl::NT, D = Tl::D;
  constexpr int kSegElems = 128 / (int)sizeof(T);
  extern __shared__ unsigned char dsm_raw[];
  PagedSmem& sm = *reinterpret_cast<PagedSmem*>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int N = (int)gridDim.x, c = (int)blockIdx.x;
  const int page = 1 << a.shift, d = a.d, G = a.G;
  const int most = a.max_pages << a.shift;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) ptx::mbar_init(&sm.full[warp][s], 1);
    ptx::fence_mbar_init();
    if (warp == 0) {
      ptx::tma_prefetch_desc(&kmap);
      ptx::tma_prefetch_desc(&vmap);
    }
  }

  // a programmatic dependent launch: nothing of the call before is read or written until it ends
  ptx::griddep_launch_dependents();
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
  const uint32_t want = (total + kMinTiles - 1) / kMinTiles;
  const uint32_t Ne = want > (uint32_t)N ? N : want;   // CTAs that take tiles
  if (c >= (int)Ne) return;

  // the window of tables that holds tile x
  auto find = [&](uint32_t x) {
    if (few) return;
    int lo = 0, hi = kPThreads;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sm.strip[mid] * a.Hp <= x) lo = mid;
      else hi = mid;
    }
    load_window<RT>(w, lo * K, sm.strip[lo] * a.Hp, a);
    seek<RT>(w, x, a);
  };
  // CTA k's first tile: total k / Ne, moved to the nearer end of a short unit it falls in
  auto bound = [&](uint32_t k) -> uint32_t {
    const uint32_t x = total / Ne * k + total % Ne * k / Ne;
    if (x == 0 || x >= total) return x;
    find(x);
    const int j = __popc(__ballot_sync(0xffffffffu, w.end <= x));
    const uint32_t nt = tiles_of<RT>(__shfl_sync(0xffffffffu, w.len, j));
    const uint32_t tb = __shfl_sync(0xffffffffu, w.end, j) - nt * a.Hp;
    const uint32_t lo = tb + (x - tb) / nt * nt;
    if (nt > kSnapTiles) return x;
    return x - lo <= lo + nt - x ? lo : lo + nt;
  };
  uint32_t b0, b1;
  if (few) {
    b0 = bound(c);
    b1 = bound(c + 1);
  } else {
    if (warp < 2) {
      const uint32_t b = bound(c + warp);
      if (lane == 0) sm.bnd[warp] = b;
    }
    __syncthreads();
    b0 = sm.bnd[0];
    b1 = sm.bnd[1];
  }
  const uint32_t span = b1 - b0;
  if (span == 0) return;   // uniform in the CTA
  // (rounded up: warp 0 has the CTA's first tile)
  const uint32_t xs = b0 + (uint32_t)(((uint64_t)span * warp + kPWarps - 1) / kPWarps);
  const uint32_t xe = b0 + (uint32_t)(((uint64_t)span * (warp + 1) + kPWarps - 1) / kPWarps);

  // ---- 2. this warp's tiles
  unsigned char* ring = sm.ring[warp];
  unsigned char* side = sm.side[warp];
  uint64_t* full = sm.full[warp];
  const uint32_t ring_u = ptx::smem_u32(ring), side_u = ptx::smem_u32(side);
  const int pieces = d * (int)sizeof(T) / 16;   // 16-byte pieces of a row
  const bool has_new = a.kn != nullptr;
  const T* qp = (const T*)a.q;

  Tl att;
  float am = -INFINITY, al = 0.f, ao[NT][2];   // part a
  int32_t unit_a = -1, unit_b = -1;
  bool open_a = false;
  uint32_t start_a = 0, end_a = 0, start_b = 0, end_b = 0;
  int issued = 0, consumed = 0;   // stage uses
  bool ok = true;
  if (xs < xe) {
    find(xs);
    // lane i's tile x0 + i (nothing past xe)
    auto describe = [&](uint32_t x0) -> Desc {
      Desc t{-1, 0, 0, 0, 0, 0, 0u, -1};
      const uint32_t x = x0 + lane;
      bool open = x < xe;
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
          const uint32_t nt = tiles_of<RT>(len);
          const uint32_t y = x - (e - nt * a.Hp);
          const int h = (int)(y / nt), tt = (int)(y - h * nt);
          const int u = w.w0 + j;
          const int r0 = tt * RT, nv = len - r0 < RT ? len - r0 : RT;
          const int32_t* entry = a.table + (int64_t)u * a.max_pages + (r0 >> a.shift);
          t.unit = u * a.Hp + h;
          t.row = h * page + (r0 & (page - 1));
          t.tt = tt;
          t.nt = nt;
          t.mask = (1u << nv) - 1u;
          if (tt == 0) t.mask |= kFirst;
          if (tt == (int)nt - 1) t.mask |= kLast;
          t.page = entry[0];
          if (page < RT && nv > page) t.page2 = entry[1];
        }
        if (!__any_sync(0xffffffffu, open) || w.w0 + 32 >= a.U) break;
        load_window<RT>(w, w.w0 + 32, wend, a);
      }
      return t;
    };
    // pages outside the pool: their rows do not count (page 0 is read in their place)
    auto check_pages = [&](Desc& t) {
      bool bad = t.page < 0 || t.page >= a.num_pages;
      if (bad) {
        t.page = 0;
        t.mask &= page < RT ? ~0xFFu : ~0xFFFFu;
      }
      if (t.page2 < 0 || t.page2 >= a.num_pages) {
        t.page2 = 0;
        t.mask &= ~0xFF00u;
        bad = true;
      }
      if (bad) raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)t.unit);
    };
    // where the new row of a unit's last tile goes
    auto look_up_slot = [&](Desc& t) {
      if (!has_new || !(t.mask & kLast)) return;
      const int u = t.unit / a.Hp;
      const int64_t c0 = a.cu[u], c1 = a.cu[u + 1];
      if (c1 > c0 && c1 > 0 && c1 <= a.slot_cap) t.slot = a.slots[c1 - 1];
      if (t.slot < -1 || t.slot >= (a.num_pages << a.shift)) {
        t.slot = -1;
        raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)t.unit);
      }
    };
    const int count = (int)(xe - xs);
    Desc cur = describe(xs), nxt{-1, 0, 0, 0, 0, 0, 0u, -1};
    check_pages(cur);
    int cur0 = 0;   // index of cur's lane 0

    // tile i (of this warp) into the ring: the lane that knows it issues
    auto issue = [&](int i) {
      const int src = i - cur0;   // 0..63
      const Desc& t = src < 32 ? cur : nxt;
      const int s = issued % S;
      if (lane == (src & 31)) {
        ptx::mbar_arrive_expect_tx(&full[s], 2u * C::kHalf);
        unsigned char* st = ring + s * 2 * C::kHalf;
#pragma unroll
        for (int g = 0; g < NSEG; ++g) {
          if (page >= RT) {
            ptx::tma_load_3d(st + g * RT * 128, &kmap, &full[s], g * kSegElems, t.row, t.page);
            ptx::tma_load_3d(st + C::kHalf + g * RT * 128, &vmap, &full[s], g * kSegElems, t.row,
                             t.page);
          } else {
            ptx::tma_load_3d(st + g * RT * 128, &kmap, &full[s], g * kSegElems, t.row, t.page);
            ptx::tma_load_3d(st + g * RT * 128 + 1024, &kmap, &full[s], g * kSegElems, t.row,
                             t.page2);
            ptx::tma_load_3d(st + C::kHalf + g * RT * 128, &vmap, &full[s], g * kSegElems, t.row,
                             t.page);
            ptx::tma_load_3d(st + C::kHalf + g * RT * 128 + 1024, &vmap, &full[s],
                             g * kSegElems, t.row, t.page2);
          }
        }
      }
      const uint32_t flags = __shfl_sync(0xffffffffu, src < 32 ? cur.mask : nxt.mask, src & 31);
      if (has_new && (flags & kLast)) {
        const int64_t u = __shfl_sync(0xffffffffu, src < 32 ? cur.unit : nxt.unit, src & 31);
        for (int p = lane; p < pieces; p += 32) {
          cp_async16(side_u + s * 2 * C::kRow + p * 16, (const T*)a.kn + u * d + p * kSegElems / 8);
          cp_async16(side_u + s * 2 * C::kRow + C::kRow + p * 16,
                     (const T*)a.vn + u * d + p * kSegElems / 8);
        }
      }
      ++issued;
    };
    __syncwarp();   // the barriers are initialised
    int next = 0;
    for (; next < S && next < count; ++next) issue(next);
    // (with the first copies under way)
    look_up_slot(cur);
    if (count > 32) {
      nxt = describe(xs + 32);
      check_pages(nxt);
      look_up_slot(nxt);
    }

    uint32_t qw[Tl::NQ];
    int32_t q_unit = -1;   // unit whose q words qw holds
    bool whole = false;    // the warp has the unit from its first tile on
    for (int i = 0; i < count; ++i) {
      if (i - cur0 == 32) {
        cur = nxt;
        cur0 += 32;
        if (count - cur0 > 32) {
          nxt = describe(xs + cur0 + 32);
          check_pages(nxt);
          look_up_slot(nxt);
        }
      }
      const int src = i - cur0;
      uint32_t mask = __shfl_sync(0xffffffffu, cur.mask, src);
      const int32_t unit = __shfl_sync(0xffffffffu, cur.unit, src);
      if (i == 0 || (mask & kFirst)) {
        if (q_unit != unit) Tl::load_q(qp + (int64_t)unit * G * d, G, d, qw);
        att.set_q(qw);
        att.begin();
        whole = (mask & kFirst) != 0;
        // the next unit's q, while this one streams
        q_unit = -1;
        if (unit + 1 < a.U * a.Hp && i + 1 < count) {
          q_unit = unit + 1;
          Tl::load_q(qp + (int64_t)q_unit * G * d, G, d, qw);
        }
      }
      const int s = consumed % S;
      if (ok) {
        const bool landed = ptx::mbar_wait(&full[s], (uint32_t)((consumed / S) & 1));
        if (__any_sync(0xffffffffu, !landed)) {
          ok = false;
          if (lane == 0) raise_dev(a.hdr, DEV_WAIT_TIMEOUT, 0x800u + (unsigned)s);
        }
      }
      if (ok) {
        const uint32_t ks = ring_u + s * 2 * C::kHalf, vs = ks + C::kHalf;
        if (has_new && (mask & kLast)) {
          const int64_t slot = __shfl_sync(0xffffffffu, (long long)cur.slot, src);
          cp_async_wait_all();
          __syncwarp();
          if (slot >= 0) {
            // to its place in the tile, the unit's last row, and to its slot
            const int u = unit / a.Hp;
            const int r = (clamp_len(a.lens[u], most) - 1) & (RT - 1);
            mask |= 1u << r;
            const int64_t at = (slot >> a.shift) * a.page_stride +
                               (((int64_t)(unit % a.Hp) << a.shift) + (slot & (page - 1))) * d;
            for (int p = lane; p < pieces; p += 32) {
              const uint4 kx = *reinterpret_cast<const uint4*>(side + s * 2 * C::kRow + p * 16);
              const uint4 vx =
                  *reinterpret_cast<const uint4*>(side + s * 2 * C::kRow + C::kRow + p * 16);
              unsigned char* st = ring + s * 2 * C::kHalf + pmma::piece<RT>(r, p);
              *reinterpret_cast<uint4*>(st) = kx;
              *reinterpret_cast<uint4*>(st + C::kHalf) = vx;
              *reinterpret_cast<uint4*>((T*)a.kp + at + p * (16 / (int)sizeof(T))) = kx;
              *reinterpret_cast<uint4*>((T*)a.vp + at + p * (16 / (int)sizeof(T))) = vx;
            }
            ptx::fence_proxy_async_smem();   // before the stage is refilled
            __syncwarp();
          }
        }
        att.tile(ks, vs, mask & 0xFFFFu, a.c2);
        __syncwarp();   // every lane is done with stage s
        ++consumed;
        if (next < count) {
          issue(next);
          ++next;
        }
      }
      // ---- the end of a unit, or of the warp's tiles
      if ((mask & kLast) || i == count - 1) {
        att.finish();
        const uint32_t start = xs + i - __shfl_sync(0xffffffffu, cur.tt, src);
        const uint32_t end = start + __shfl_sync(0xffffffffu, cur.nt, src);
        if (whole && (mask & kLast)) {
          const int g = lane >> 2, col = 2 * (lane & 3);
          if (g < G) {
            const float inv = att.l > 0.f ? 1.f / att.l : 0.f;
            T* dst = (T*)a.out + ((int64_t)unit * G + g) * d + col;
#pragma unroll
            for (int t = 0; t < NT; ++t)
              if (8 * t < d) store2(dst + 8 * t, att.o[t][0] * inv, att.o[t][1] * inv);
          }
        } else if (!whole) {
          am = att.m;
          al = att.l;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            ao[t][0] = att.o[t][0];
            ao[t][1] = att.o[t][1];
          }
          unit_a = unit;
          open_a = (mask & kLast) == 0;
          start_a = start;
          end_a = end;
        } else {
          unit_b = unit;
          start_b = start;
          end_b = end;
        }
      }
    }
    if (!ok && lane == 0)   // a wait gave up: let what is in flight land before the memory is reused
      for (int i = consumed; i < issued; ++i)
        (void)ptx::mbar_wait(&full[i % S], (uint32_t)((i / S) & 1), 20000000ull);
  }
  if (lane == 0) {
    sm.a_unit[warp] = unit_a;
    sm.a_open[warp] = open_a ? 1 : 0;
    sm.b_unit[warp] = unit_b;
    sm.some[warp] = xs < xe ? 1 : 0;
    sm.start[1 + warp] = start_b;
    sm.end[1 + warp] = end_b;
    if (warp == 0) {
      sm.start[0] = start_a;
      sm.end[0] = end_a;
    }
  }
  __syncthreads();   // every ring is idle: its memory holds the parts now

  // ---- 3. merges
  float* wp = reinterpret_cast<float*>(&sm.ring[0][0]);   // part a of warp w: 2 w, part b: 2 w + 1
  const int g4 = lane >> 2, c4 = lane & 3;
  if (unit_a >= 0) {
    float* P = wp + (2 * warp) * kPartFloats;
    if (c4 == 0) {
      P[g4] = am;
      P[8 + g4] = al;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<float2*>(P + kPartHead + g4 * D + 8 * t + 2 * c4) =
          make_float2(ao[t][0], ao[t][1]);
  }
  if (unit_b >= 0) {
    float* P = wp + (2 * warp + 1) * kPartFloats;
    if (c4 == 0) {
      P[g4] = att.m;
      P[8 + g4] = att.l;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<float2*>(P + kPartHead + g4 * D + 8 * t + 2 * c4) =
          make_float2(att.o[t][0], att.o[t][1]);
  }
  __syncthreads();
  const int nsl = G * (D / 4);   // 16-byte slices of a part's output
  int cross_a = -1, cross_b = -1;   // units that began before this CTA / go on after it: the
                                    // candidate (0: warp 0's part a, 1 + w: warp w's part b)
  for (int cand = 0; cand <= kPWarps; ++cand) {
    const int32_t unit = cand == 0 ? sm.a_unit[0] : sm.b_unit[cand - 1];
    if (unit < 0) continue;
    const int first = cand == 0 ? 0 : 2 * cand - 1;
    uint32_t members = 0;   // warps whose part a goes on with the unit
    bool open = cand == 0 ? sm.a_open[0] != 0 : true;
    for (int k = cand == 0 ? 1 : cand; k < kPWarps && open; ++k) {
      if (!sm.some[k]) continue;
      if (sm.a_unit[k] != unit) break;
      members |= 1u << k;
      open = sm.a_open[k] != 0;
    }
    const bool crosses = cand == 0 || open;
    if (cand == 0) cross_a = 0;
    else if (open) cross_b = cand;
    for (int idx = tid; idx < nsl; idx += kPThreads) {
      const int g = idx / (D / 4), col = (idx - g * (D / 4)) * 4;
      const float* P = wp + first * kPartFloats;
      float M = -INFINITY, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      merge_part(P[g], P[8 + g], *reinterpret_cast<const float4*>(P + kPartHead + g * D + col), M,
                 L, acc);
      for (uint32_t m = members; m; m &= m - 1) {
        P = wp + 2 * (__ffs(m) - 1) * kPartFloats;
        merge_part(P[g], P[8 + g], *reinterpret_cast<const float4*>(P + kPartHead + g * D + col),
                   M, L, acc);
      }
      if (crosses) {
        float* Q = a.part + (int64_t)(cand == 0 ? 2 * c : 2 * c + 1) * kPartFloats;
        if (col == 0) {
          Q[g] = M;
          Q[8 + g] = L;
        }
        *reinterpret_cast<float4*>(Q + kPartHead + g * D + col) = acc;
      } else if (col < d) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        store4((T*)a.out + ((int64_t)unit * G + g) * d + col,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      }
    }
  }
  if (cross_a < 0 && cross_b < 0) return;   // uniform in the CTA

  // units that cross CTAs: the CTA that holds tile x, and the last of a unit's CTAs merges
  auto cta_of = [&](uint32_t x) {
    return (int)((((uint64_t)x + 1) * Ne + total - 1) / total) - 1;
  };
  __threadfence();
  __syncthreads();
  if (tid < 2) {
    const int cand = tid == 0 ? cross_a : cross_b;
    int won = -1;
    if (cand >= 0) {
      const int ca = cta_of(sm.start[cand]), cb = cta_of(sm.end[cand] - 1);
      const uint32_t old = atomicAdd(&a.tick[ca], 1u);
      if (old == (uint32_t)(cb - ca)) {
        atomicExch(&a.tick[ca], 0u);
        won = cand;
      }
    }
    sm.win[tid] = won;
  }
  __syncthreads();
  __threadfence();
  for (int y = 0; y < 2; ++y) {
    const int cand = sm.win[y];
    if (cand < 0) continue;
    const int32_t unit = cand == 0 ? sm.a_unit[0] : sm.b_unit[cand - 1];
    const int ca = cta_of(sm.start[cand]), cb = cta_of(sm.end[cand] - 1);
    for (int idx = tid; idx < nsl; idx += kPThreads) {
      const int g = idx / (D / 4), col = (idx - g * (D / 4)) * 4;
      float M = -INFINITY, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kB = 8;   // parts per round of loads
      for (int c0 = ca; c0 <= cb; c0 += kB) {
        float m[kB], l[kB];
        float4 o[kB];
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          m[b] = -INFINITY;
          l[b] = 0.f;
          o[b] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c0 + b <= cb) {
            const int k = c0 + b;
            const float* P = a.part + (int64_t)(k == ca ? 2 * k + 1 : 2 * k) * kPartFloats;
            m[b] = __ldcg(P + g);
            l[b] = __ldcg(P + 8 + g);
            o[b] = __ldcg(reinterpret_cast<const float4*>(P + kPartHead + g * D + col));
          }
        }
#pragma unroll
        for (int b = 0; b < kB; ++b) merge_part(m[b], l[b], o[b], M, L, acc);
      }
      if (col < d) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        store4((T*)a.out + ((int64_t)unit * G + g) * d + col,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      }
    }
  }
}

// ------------------------------------- host side ----------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 paged_encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// The pool as [num_pages][Hp * page rows][d], in boxes of 128 bytes of `rows` rows of one page,
// swizzled; columns past d read as zero.
bool pool_map(CUtensorMap* map, const void* base, const PagedShape& s, int rows) {
  auto fn = paged_encode_fn();
  if (fn == nullptr) return false;
  const uint64_t e = (uint64_t)s.esize();
  const cuuint64_t dims[3] = {(cuuint64_t)s.d, (cuuint64_t)s.Hp() * s.page,
                              (cuuint64_t)s.num_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)s.d * e, (cuuint64_t)s.page_stride * e};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / e), (cuuint32_t)rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map,
            s.dtype == KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
            3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kTickBytes = 1024;
static_assert(kMaxCtas * sizeof(uint32_t) <= kTickBytes, "tickets");

template <typename T, int NSEG>
cudaError_t launch_t(const PagedShape& s, const PagedArgs& a, cudaStream_t st) {
  using C = Cfg<T, NSEG>;
  constexpr size_t smem = sizeof(PagedSmem) + 1024;
  static_assert(smem <= 227 * 1024, "one CTA per SM");
  static std::atomic<int> slot[kMaxDevices];
  const int ok = per_device(slot, []() {
    return cudaFuncSetAttribute(paged_decode_kernel<T, NSEG>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem) == cudaSuccess ? 1 : 0;
  });
  if (!ok) return cudaErrorInvalidConfiguration;
  CUtensorMap km, vm;
  const int rows = s.page < C::RT ? s.page : C::RT;
  if (!pool_map(&km, a.kp, s, rows) || !pool_map(&vm, a.vp, s, rows))
    return cudaErrorInvalidValue;
  // no more CTAs than the tables could ever fill
  const int64_t tiles = (int64_t)s.seqs * s.Hkv * cdiv((int64_t)s.max_pages * s.page, C::RT);
  int64_t grid = cdiv(tiles, kMinTiles);
  if (grid > num_sms()) grid = num_sms();
  if (grid > kMaxCtas) grid = kMaxCtas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<T, NSEG>, km, vm, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}
}  // namespace

size_t paged_decode_ws_bytes(const PagedShape&) {
  return kWsHeader + kTickBytes + (size_t)2 * kMaxCtas * kPartFloats * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedShape& s, const void* q, const void* kn, const void* vn,
                                const int64_t* cu, const int64_t* slots, int64_t slot_capacity,
                                void* kp, void* vp, const int32_t* table, const int32_t* lens,
                                float scale, void* out, char* ws, cudaStream_t st) {
  int shift = 0;
  while ((1 << shift) < s.page) ++shift;
  const PagedArgs a{q, kn, vn, cu, slots, slot_capacity, kp, vp, table, lens, out,
                    reinterpret_cast<WsHeader*>(ws), reinterpret_cast<uint32_t*>(ws + kWsHeader),
                    reinterpret_cast<float*>(ws + kWsHeader + kTickBytes), (int)s.U(), s.Hp(),
                    s.G(), s.d, shift, s.max_pages, s.num_pages, s.page_stride,
                    scale * 1.4426950408889634f};
  if (s.dtype == KV_BF16)
    return s.d <= 64 ? launch_t<__nv_bfloat16, 1>(s, a, st) : launch_t<__nv_bfloat16, 2>(s, a, st);
  switch ((s.d + 31) / 32) {
    case 1: return launch_t<float, 1>(s, a, st);
    case 2: return launch_t<float, 2>(s, a, st);
    case 3: return launch_t<float, 3>(s, a, st);
    default: return launch_t<float, 4>(s, a, st);
  }
}

}  // namespace kv
