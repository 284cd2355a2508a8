// Block tables, slot map and free ring of the paged cache, from the rows each table holds and
// the rows it gains or loses.
//
// With P(x) = ceil(x / page), new = max(len + add, 0), a table needs (P(new) - P(len))+ pages
// and returns (P(len) - P(new))+.  Three exclusive prefix sums over the tables -- rows added,
// pages needed, pages returned -- give every row its place in the slot map and every page its
// place in the ring.  The ring is a queue: pages are taken from its head and returned to its
// tail.  What a call takes, [head, head + need), and what it returns to, [tail, tail + back),
// are different entries as long as the ring has room for what comes back, so no CTA depends on
// another's pages, and which page goes where is the same in every run.
//
// One launch.  Every CTA forms the prefix sums of all tables (a table costs 8 bytes of L2
// reads).  The thread that has a table's sums at hand gives it its slots if it gains few rows,
// so a decode step, one CTA, ends there.  Tables that gain many (prompts) are cut by slots: a
// warp takes runs of 128, finds the table of each in shared memory, and the lane of a page's
// first row writes the block table entry; pages returned are cut likewise.  Where the lengths or
// the ring's state are updated in place, the last CTA to finish writes them.
//
// Bound by latency: lengths, ring or block table, slots are dependent loads and a store.  On
// GB300: one token for 8 tables 3.3 us, for 1024 tables 5.7 us (both one CTA), prompts of 460K
// rows over 96 tables 8.8 us (3.65 MB of slots; 16.3 us with runs of 256, on a quarter of the
// SMs).
#include "kv_internal.cuh"
#include "tc_ptx.cuh"

namespace kv {
namespace {

constexpr int kMThreads = 1024;   // most threads of a CTA
constexpr int kOwnRows = 4;       // a table that gains at most these is one thread's work
constexpr int kRun = 128;         // slots (or pages) of a warp at a time

struct MapArgs {
  const int32_t* lens;
  const int32_t* add;
  int32_t* ring;
  const int64_t* state;
  int64_t slot_cap;
  int32_t* table;
  int32_t* lens_out;
  int64_t* state_out;
  int64_t* cu;
  int64_t* slots;
  WsHeader* hdr;
  uint32_t* done;
  int U, max_pages, shift;   // page = 1 << shift
  int in_place;              // lens_out is lens, or state_out is state
  int64_t num_pages;
};

// What one table asks for.
struct Ask {
  int len, now;    // rows held and rows asked for
  int gain;        // rows to give slots to
  int need, back;  // pages to take / to return
  bool bad;        // a length outside the table: nothing is done
};
__device__ __forceinline__ int pages_of(int x, int shift) {
  return (int)(((int64_t)x + (1 << shift) - 1) >> shift);
}
__device__ __forceinline__ Ask ask_of(int len, int add, int max_pages, int shift) {
  Ask a;
  const int64_t most = (int64_t)max_pages << shift;
  const int64_t now = (int64_t)len + add;
  a.len = len;
  a.gain = add > 0 ? add : 0;
  a.bad = len < 0 || len > most || now > most;
  a.now = a.bad ? len : (int)(now > 0 ? now : 0);
  const int d = a.bad ? 0 : pages_of(a.now, shift) - pages_of(len, shift);
  a.need = d > 0 ? d : 0;
  a.back = d < 0 ? -d : 0;
  return a;
}
__device__ __forceinline__ int32_t sat(int64_t x) { return x > INT32_MAX ? INT32_MAX : (int32_t)x; }

// Largest u in [0, U) with pre[u] <= x (pre[0] = 0).
__device__ __forceinline__ int table_of(const int32_t* pre, int U, int32_t x) {
  int lo = 0, hi = U;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kMThreads) page_map_kernel(const MapArgs a) {
  // exclusive prefixes, held to int32: slot_cap and num_pages are within it, and a prefix past
  // either only has to stay past it
  extern __shared__ int32_t pre_sm[];
  int32_t* cuS = pre_sm;                 // [U + 1] rows added
  int32_t* needS = cuS + a.U + 1;        // [U + 1] pages taken
  int32_t* backS = needS + a.U + 1;      // [U + 1] pages returned
  __shared__ int64_t wsum[3][kMThreads / 32];
  __shared__ int32_t wtaken[kMThreads / 32];
  __shared__ uint32_t last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nthreads = blockDim.x, nwarps = nthreads >> 5;
  const bool alone = gridDim.x == 1;
  ptx::griddep_launch_dependents();
  const int64_t head = a.state[0], tail = a.state[1];
  const bool ring_ok = head >= 0 && tail >= head && tail < ((int64_t)1 << 62) &&
                       tail - head <= a.num_pages;
  const int64_t avail = ring_ok ? tail - head : 0;
  // place i of the ring from its head, 0 <= i < num_pages
  const uint32_t n = (uint32_t)a.num_pages;
  const uint32_t head0 = ring_ok ? (uint32_t)((uint64_t)head % n) : 0u;
  auto ring_at = [&](uint32_t i) {
    const uint32_t x = head0 + i;   // < 2^32
    return x >= n ? x - n : x;
  };
  const int page = 1 << a.shift;
  // the slot of row `row` of table u, whose first page taken is place `first` of the ring
  auto slot_of = [&](int u, const Ask& k, int64_t first, int row) -> int64_t {
    const int col = row >> a.shift, held = pages_of(k.len, a.shift);
    int32_t* entry = a.table + (int64_t)u * a.max_pages + col;
    int32_t p;
    if (col < held) {
      p = *entry;
    } else {
      p = a.ring[ring_at((uint32_t)(first + col - held))];
      if ((row & (page - 1)) == 0) *entry = p;
    }
    if (p >= 0 && p < a.num_pages) return ((int64_t)p << a.shift) + (row & (page - 1));
    raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)u);
    return -1;
  };

  // ---- prefix sums; the tables that gain few rows
  int64_t carry[3] = {0, 0, 0};
  bool more = false;   // rows left for the cut by slots
  int taken = 0;       // pages taken: the tables that take some are the first that need any
  for (int u0 = 0; u0 < a.U; u0 += nthreads) {
    const int u = u0 + tid;
    Ask k{};
    if (u < a.U) k = ask_of(a.lens[u], a.add[u], a.max_pages, a.shift);
    int64_t x[3] = {k.gain, k.need, k.back};
#pragma unroll
    for (int j = 0; j < 3; ++j) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, (long long)x[j], o);
        if (lane >= o) x[j] += y;
      }
      if (lane == 31) wsum[j][warp] = x[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      int64_t t = lane < nwarps ? wsum[j][lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, (long long)t, o);
        if (lane >= o) t += y;
      }
      const int64_t before = __shfl_sync(0xffffffffu, (long long)t, warp > 0 ? warp - 1 : 0);
      x[j] += carry[j] + (warp > 0 ? before : 0);
      carry[j] += __shfl_sync(0xffffffffu, (long long)t, 31);
    }
    if (u < a.U) {
      const int64_t cu = x[0] - k.gain, first = x[1] - k.need;
      cuS[u] = sat(cu);
      needS[u] = sat(first);
      backS[u] = sat(x[2] - k.back);
      const bool own = k.gain <= kOwnRows;
      more = more || !own;
      const bool fits = !k.bad && x[0] <= a.slot_cap && (k.need == 0 || x[1] <= avail);
      if (blockIdx.x == 0) {
        a.cu[u] = cu;
        if (u == a.U - 1) a.cu[a.U] = x[0];
        if (k.bad) raise_dev(a.hdr, DEV_PAGE_TABLE, (unsigned)u);
        else if (k.need > 0 && x[1] > avail) raise_dev(a.hdr, DEV_NO_PAGES, (unsigned)u);
        if (k.gain > 0 && x[0] > a.slot_cap) raise_dev(a.hdr, DEV_SLOT_CAPACITY, (unsigned)u);
        if (own && k.gain > 0) {
          for (int i = 0; i < k.gain && cu + i < a.slot_cap; ++i)
            a.slots[cu + i] = fits ? slot_of(u, k, first, k.len + i) : -1;
          // (the length is read again only by other CTAs)
          if (alone) a.lens_out[u] = fits ? k.now : k.len;
          if (fits && k.need > 0) taken = (int)x[1];
        }
      }
    }
    __syncthreads();   // the warp sums are reused
  }
  if (tid == 0) {
    cuS[a.U] = sat(carry[0]);
    needS[a.U] = sat(carry[1]);
    backS[a.U] = sat(carry[2]);
  }
  more = __syncthreads_or(more);
  const bool back_ok = ring_ok && tail + carry[2] <= head + a.num_pages;
  if (blockIdx.x == 0 && tid == 0 && (!ring_ok || !back_ok)) raise_dev(a.hdr, DEV_FREE_RING, 0);

  // whether table u's rows are given to it (gain > 0) or taken from it (gain == 0)
  auto served = [&](int u, const Ask& k) -> bool {
    if (k.bad) return false;
    if (k.gain == 0) return k.now == k.len || back_ok;
    if (cuS[u + 1] > a.slot_cap) return false;
    return k.need == 0 || (int64_t)needS[u] + k.need <= avail;
  };
  const int64_t run0 = ((int64_t)blockIdx.x * nwarps + warp) * kRun;
  const int64_t run_step = (int64_t)gridDim.x * nwarps * kRun;

  // ---- the tables that gain many rows, by slots
  if (more) {
    const int64_t nslots = cuS[a.U] < a.slot_cap ? cuS[a.U] : a.slot_cap;
    for (int64_t b = run0; b < nslots; b += run_step) {
      int u = table_of(cuS, a.U, (int32_t)b);
#pragma unroll 4
      for (int j = 0; j < kRun / 32; ++j) {
        const int64_t i = b + j * 32 + lane;
        if (i >= nslots) break;
        if (cuS[u + 1] <= i) u = table_of(cuS, a.U, (int32_t)i);
        const Ask k = ask_of(a.lens[u], a.add[u], a.max_pages, a.shift);
        if (k.gain > kOwnRows)
          a.slots[i] = served(u, k) ? slot_of(u, k, needS[u], k.len + (int)(i - cuS[u])) : -1;
      }
    }
  }
  // ---- pages returned
  if (back_ok && carry[2] > 0) {
    const uint32_t tail0 = (uint32_t)((uint64_t)tail % n);
    for (int64_t b = run0; b < backS[a.U]; b += run_step) {
      for (int j = 0; j < kRun / 32; ++j) {
        const int64_t i = b + j * 32 + lane;
        if (i >= backS[a.U]) break;
        const int u = table_of(backS, a.U, (int32_t)i);
        const Ask k = ask_of(a.lens[u], a.add[u], a.max_pages, a.shift);
        const int col = pages_of(k.now, a.shift) + (int)(i - backS[u]);
        const int32_t p = a.table[(int64_t)u * a.max_pages + col];
        if (p < 0 || p >= a.num_pages) raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)u);
        const uint32_t at = tail0 + (uint32_t)i;
        a.ring[at >= n ? at - n : at] = p;
      }
    }
  }

  // ---- lengths and the ring's state; in place, once every CTA has read the old ones
  if (!a.in_place && blockIdx.x != 0) return;
  __syncthreads();
  if (!alone && a.in_place) {
    if (tid == 0) {
      __threadfence();
      last = atomicAdd(a.done, 1u) == gridDim.x - 1;
      if (last) atomicExch(a.done, 0u);
    }
    __syncthreads();
    if (!last) return;
  }
  for (int u = tid; u < a.U; u += nthreads) {
    const Ask k = ask_of(a.lens[u], a.add[u], a.max_pages, a.shift);
    if (alone && k.gain > 0 && k.gain <= kOwnRows) continue;   // done
    const bool ok = served(u, k);
    a.lens_out[u] = ok ? k.now : k.len;
    if (ok && k.need > 0) taken = max(taken, needS[u] + k.need);
  }
  // (the largest; needS is non-decreasing over the tables)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
  if (lane == 0) wtaken[warp] = taken;
  __syncthreads();
  if (tid == 0) {
    int t = 0;
    for (int w = 0; w < nwarps; ++w) t = max(t, wtaken[w]);
    a.state_out[0] = head + t;
    a.state_out[1] = tail + (back_ok ? carry[2] : 0);
  }
}
}  // namespace

cudaError_t launch_page_map(const PagedShape& s, const int32_t* lens, const int32_t* add,
                            int32_t* ring, const int64_t* state, int64_t slot_capacity,
                            int32_t* table, int32_t* lens_out, int64_t* state_out, int64_t* cu,
                            int64_t* slots, char* ws, cudaStream_t st) {
  const int U = (int)s.U();
  const size_t smem = (size_t)(U + 1) * 3 * sizeof(int32_t);
  static std::atomic<int> slot[kMaxDevices];
  const int ok = per_device(slot, []() {
    const int most = (KV_PAGE_MAP_MAX_TABLES + 1) * 3 * (int)sizeof(int32_t);
    return cudaFuncSetAttribute(page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                most) == cudaSuccess ? 1 : 0;
  });
  if (!ok) return cudaErrorInvalidConfiguration;
  int shift = 0;
  while ((1 << shift) < s.page) ++shift;
  // a CTA for every run of slots of its warps; small calls are one small CTA
  const int threads = U <= 256 && slot_capacity <= 4096 ? 256 : U <= 512 ? 512 : kMThreads;
  int64_t grid = cdiv(slot_capacity, (int64_t)(threads / 32) * kRun);
  if (slot_capacity <= (int64_t)kOwnRows * U || grid < 1) grid = 1;
  if (grid > 2 * num_sms()) grid = 2 * num_sms();
  MapArgs a{lens, add, ring, state, slot_capacity, table, lens_out, state_out, cu, slots,
            reinterpret_cast<WsHeader*>(ws), reinterpret_cast<uint32_t*>(ws + kWsHeader), U,
            s.max_pages, shift, lens_out == lens || state_out == state, s.num_pages};
  // (as a programmatic dependent launch 3.1 us on the device against 3.35, 8.4 from Python
  // against 7.7; its dependents may be one)
  page_map_kernel<<<(unsigned)grid, (unsigned)threads, smem, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace kv
