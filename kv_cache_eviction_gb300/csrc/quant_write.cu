// Rows of K and V stored in 8 bits at their slots, with a scale for each block of 16 slots and head
// (quant_codes.cuh).  Bound by reading the rows and writing the codes once.
//
// A run of rows whose slots follow each other within one block is a unit: a warp loads a head's
// rows of it, finds their largest magnitude, and writes the codes from its registers.  Rows of the
// block below the run were held before: where the scale grows, their codes are rounded to it. The
// slots of a warp's next rows are under way while it works (a chain of slots, rows, codes
// otherwise).  On GB300: 131072 rows of 8 heads of 128 bf16 (806 MB read and written) 120 us, 6.7
// TB/s or 0.99 of the measured copy rate (134 us without, 32 bytes a lane and two divisions a
// piece); 100003 fp32 rows of one head of 64 15.8 us (21.9), 4.1 TB/s: 3.4 runs a warp; 64 rows 2.3
// us.
#include "quant_codes.cuh"
#include "tc_ptx.cuh"

namespace kv {
namespace {

using quant::Piece;
constexpr int kThreads = 128;
// CTAs of an SM by a lane's pieces, for both types.  131072 bf16 rows of 128 (8 pieces), us: 4 CTAs
// 133, 5 124, 6 120, 7 134, 8 (the registers then spill) 140; 100003 fp32 rows of 64 (8 pieces): 16.9,
// 15.1, 15.8, 15.6, 15.5.  So fp32 would be 4 % better off with 5: its kernel spills 60 bytes with 6.
// fp32 rows of 128 (16 pieces, 159 registers, 3 CTAs): 131072 of 8 heads 209 us, 6.4 TB/s.
constexpr int resident(int pieces) { return pieces <= 4 ? 8 : pieces <= 8 ? 6 : 3; }

struct QWriteArgs {
  const uint4* src[2];     // k, v
  unsigned char* pool[2];
  float* scale[2];
  const int64_t* slots;
  const int64_t* n_rows;
  WsHeader* hdr;
  int64_t rows, src_vec, page_stride, num_slots;   // src_vec: 16-byte pieces from row to row
  int Hp, d, shift, window_shift, pieces;          // pieces: of a head's row
};

// KP: pieces of a lane, for 16 rows of a head of up to 2 KP pieces.
template <typename T, typename F, int KP>
__global__ void __launch_bounds__(kThreads, resident(KP))
quant_write_kernel(const __grid_constant__ QWriteArgs a) {
  constexpr int kN = Piece<T>::kN;
  constexpr int kLanes = 2 * KP, kStep = 32 / kLanes;   // lanes of a row, rows at a time
  const int lane = threadIdx.x & 31, lr = lane / kLanes, lp = lane % kLanes;
  const int page = 1 << a.shift, window = 1 << a.window_shift, pairs = a.Hp * 2;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();   // nothing of the call before is read or written until it ends
  int64_t rows = a.rows;
  if (a.n_rows != nullptr) rows = min(rows, *a.n_rows);
  // a warp's items: windows of rows, and of each the pairs (head, K or V)
  const int warps = (int)gridDim.x * (kThreads / 32);
  const int me = (int)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int win_step = warps / pairs, pair_step = warps - win_step * pairs;
  int64_t win = me / pairs;
  int pair = me - (int)win * pairs;
  // lane i: the slot of row i0 + i, for the window and the 15 rows behind it; lane 31: that of the
  // row before.  (-1 outside the rows)
  auto load_slot = [&](int64_t i0) {
    const int64_t row = lane == 31 ? i0 - 1 : i0 + lane;
    const bool in = row >= 0 && row < rows && (lane == 31 || lane < window + 15);
    return in ? a.slots[row] : (int64_t)-1;
  };
  int64_t next = load_slot(win << a.window_shift);
  while ((win << a.window_shift) < rows) {
    const int t = pair & 1, h = pair >> 1;
    const int64_t i0 = win << a.window_shift, slot = next;
    win += win_step;
    pair += pair_step;
    if (pair >= pairs) {
      pair -= pairs;
      ++win;
    }
    next = load_slot(win << a.window_shift);   // (its latency beside this item's work)
    const bool ok = slot >= 0 && slot < a.num_slots;
    const int64_t before = __shfl_sync(0xffffffffu, (long long)slot, (lane + 31) & 31);
    const bool goes_on = ok && lane < 31 && (slot & (quant::kBlock - 1)) != 0 && before == slot - 1;
    // a neighbour of its own block that it does not follow: refused, and so is what goes on from it
    const bool astray = ok && !goes_on && before >= 0 && ((before ^ slot) >> 4) == 0;
    if ((astray || (!ok && slot != -1)) && lane < window && h == 0 && t == 0)
      raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)(i0 + lane));
    const uint32_t more = __ballot_sync(0xffffffffu, goes_on);
    uint32_t starts = __ballot_sync(0xffffffffu, ok && !goes_on && !astray && lane < window);
    for (; starts; starts &= starts - 1) {
      const int s = __ffs(starts) - 1;
      const int n = __ffs(~(more >> s >> 1));   // rows of the run (at most 16, within lanes 0..30)
      const int64_t slot0 = __shfl_sync(0xffffffffu, (long long)slot, s);
      const bool mine = lp < a.pieces;
      Piece<T> x[KP];
      const uint4* src = a.src[t] + (i0 + s + lr) * a.src_vec + h * a.pieces + lp;
#pragma unroll
      for (int j = 0; j < KP; ++j) {
        x[j].w = make_uint4(0u, 0u, 0u, 0u);
        if (mine && lr + j * kStep < n) x[j].w = src[j * kStep * a.src_vec];
      }
      const int first = (int)(slot0 & (quant::kBlock - 1));
      const int64_t pg = slot0 >> a.shift;
      const int r = (int)(slot0 & (page - 1));
      float* sc = a.scale[t] + (pg * a.Hp + h) * (page / quant::kBlock) + r / quant::kBlock;
      const float old = first > 0 ? *sc : 0.f;
      unsigned char* dst = a.pool[t] + pg * a.page_stride + ((int64_t)h * page + r) * a.d;
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < KP; ++j) top = x[j].top(top);
      top = __reduce_max_sync(0xffffffffu, Piece<T>::whole(top));
      const bool finite = top < quant::kInf;
      if (!finite) {
        top = 0;
#pragma unroll
        for (int j = 0; j < KP; ++j) top = x[j].finite_top(top);
        top = __reduce_max_sync(0xffffffffu, top);
      }
      const float now = quant::scale_after<F>(top, old), inv = 1.f / now;
      if (now != old) {   // (raised, or in the place of a NaN or an infinity)
        // (the run's rows are contiguous in the pool, and so are those before it)
        for (int p = lane; p < first * (a.d / 16); p += 32) {
          uint4* at = reinterpret_cast<uint4*>(dst - first * a.d) + p;
          *at = quant::again<F>(*at, old * inv);
        }
        if (lane == 0) *sc = now;
      }
      dst += lr * a.d + lp * kN;
      auto put = [&](bool held) {
#pragma unroll
        for (int j = 0; j < KP; ++j) {
          if (!mine || lr + j * kStep >= n) continue;
          unsigned char* at = dst + j * kStep * a.d;
          if (kN == 8)
            *reinterpret_cast<uint2*>(at) = make_uint2(x[j].template codes<F>(0, inv, held),
                                                       x[j].template codes<F>(4 % kN, inv, held));
          else
            *reinterpret_cast<uint32_t*>(at) = x[j].template codes<F>(0, inv, held);
        }
      };
      if (finite) put(true);
      else put(false);
    }
  }
}

template <typename T, typename F, int KP>
cudaError_t launch_kp(const PagedShape& s, QWriteArgs& a, cudaStream_t st) {
  // rows of a window: 16, or fewer where that leaves warps without work
  const int64_t want = (int64_t)num_sms() * 32;
  a.window_shift = 4;
  while (a.window_shift > 0 && (cdiv(a.rows, (int64_t)1 << a.window_shift) * s.Hp() * 2 < want))
    --a.window_shift;
  const int64_t items = cdiv(a.rows, (int64_t)1 << a.window_shift) * s.Hp() * 2;
  int64_t grid = cdiv(items, kThreads / 32);
  const int64_t most = (int64_t)num_sms() * resident(KP);
  if (grid > most) grid = most;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;   // (calls of 64 rows one after the other 3.2 us, 4.2 without)
  const cudaError_t e = cudaLaunchKernelEx(&cfg, quant_write_kernel<T, F, KP>, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <typename T, typename F>
cudaError_t launch(const PagedShape& s, QWriteArgs& a, cudaStream_t st) {
  constexpr int kMost = 16 * 128 / 32 / Piece<T>::kN;   // at d = 128
  if (s.d <= 32) return launch_kp<T, F, kMost / 4>(s, a, st);
  return s.d <= 64 ? launch_kp<T, F, kMost / 2>(s, a, st) : launch_kp<T, F, kMost>(s, a, st);
}
}  // namespace

cudaError_t launch_quant_write(const PagedShape& s, int format, const void* k, const void* v,
                               int64_t src_stride, const int64_t* slots, int64_t rows,
                               const int64_t* n_rows, void* kp, void* vp, float* ks, float* vs,
                               WsHeader* hdr, cudaStream_t st) {
  int shift = 0;
  while ((1 << shift) < s.page) ++shift;
  QWriteArgs a{{(const uint4*)k, (const uint4*)v}, {(unsigned char*)kp, (unsigned char*)vp},
               {ks, vs}, slots, n_rows, hdr, rows, src_stride * s.esize() / 16, s.page_stride,
               s.num_pages << shift, s.Hp(), s.d, shift, 0, s.d * s.esize() / 16};
  if (s.dtype == KV_BF16)
    return format == KV_E4M3 ? launch<__nv_bfloat16, quant::E4M3>(s, a, st)
                             : launch<__nv_bfloat16, quant::Int8>(s, a, st);
  return format == KV_E4M3 ? launch<float, quant::E4M3>(s, a, st)
                           : launch<float, quant::Int8>(s, a, st);
}

}  // namespace kv
