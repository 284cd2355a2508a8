// Rows of K and V stored in 8 bits at their slots, with a scale for each block of 16 slots and
// head (quant_codes.cuh).  Bound by reading the rows and writing the codes once.
//
// A run of rows whose slots follow each other within one block is a unit: a warp loads a head's
// rows of it, finds their largest magnitude, and writes the codes from its registers.  Rows of
// the block below the run were held before: where the scale grows, their codes are rounded to it.
#include "quant_codes.cuh"
#include "tc_ptx.cuh"

namespace kv {
namespace {

using quant::Piece;
constexpr int kThreads = 256;

struct QWriteArgs {
  const uint4* src[2];     // k, v
  unsigned char* pool[2];
  float* scale[2];
  const int64_t* slots;
  const int64_t* n_rows;
  WsHeader* hdr;
  int64_t rows, src_vec, page_stride, num_slots;   // src_vec: 16-byte pieces from row to row
  int Hp, d, shift, window_shift;
};

template <typename T, typename F>
__global__ void __launch_bounds__(kThreads) quant_write_kernel(const __grid_constant__ QWriteArgs a) {
  constexpr int kPer = Piece<T>::kLoads;
  constexpr int kPieces = quant::kBlock * 8 / 32;    // of a lane: a block of rows of up to 128
  const int lane = threadIdx.x & 31;
  const int page = 1 << a.shift, dv = a.d / 16, window = 1 << a.window_shift;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();   // nothing of the call before is read or written until it ends
  int64_t rows = a.rows;
  if (a.n_rows != nullptr) rows = min(rows, *a.n_rows);
  const int64_t items = cdiv(rows, window) * a.Hp * 2;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t it = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < items;
       it += step) {
    const int t = (int)(it & 1);
    const int64_t win = (it >> 1) / a.Hp;
    const int h = (int)((it >> 1) - win * a.Hp);
    const int64_t i0 = win << a.window_shift;
    // lane i: the slot of row i0 + i, for the window and the 15 rows behind it; lane 31: that of
    // the row before
    const int64_t row = lane == 31 ? i0 - 1 : i0 + lane;
    int64_t slot = -1;
    if (row >= 0 && row < rows && (lane == 31 || lane < window + 15)) slot = a.slots[row];
    const bool ok = slot >= 0 && slot < a.num_slots;
    if (!ok && slot != -1 && lane < window && h == 0 && t == 0)
      raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)row);
    int64_t before = __shfl_sync(0xffffffffu, (long long)slot, (lane + 31) & 31);
    const bool goes_on = ok && lane < 31 && (slot & (quant::kBlock - 1)) != 0 && before == slot - 1;
    const uint32_t more = __ballot_sync(0xffffffffu, goes_on);
    uint32_t starts = __ballot_sync(0xffffffffu, ok && !goes_on && lane < window);
    for (; starts; starts &= starts - 1) {
      const int s = __ffs(starts) - 1;
      const int n = __ffs(~(more >> s >> 1));   // rows of the run (at most 16, within lanes 0..30)
      const int64_t slot0 = __shfl_sync(0xffffffffu, (long long)slot, s);
      const int first = (int)(slot0 & (quant::kBlock - 1));
      const int64_t pg = slot0 >> a.shift;
      const int r = (int)(slot0 & (page - 1));
      unsigned char* dst = a.pool[t] + pg * a.page_stride + ((int64_t)h * page + r) * a.d;
      float* sc = a.scale[t] + (pg * a.Hp + h) * (page / quant::kBlock) + r / quant::kBlock;
      const float old = first > 0 ? *sc : 0.f;
      const uint4* src = a.src[t] + (i0 + s) * a.src_vec + h * (dv * kPer);
      Piece<T> x[kPieces];
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int p = lane + 32 * j, pr = p / dv;
        if (pr < n) {
          const uint4* from = src + pr * a.src_vec + (p - pr * dv) * kPer;
#pragma unroll
          for (int k = 0; k < kPer; ++k) x[j].w[k] = from[k];
        }
      }
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if ((lane + 32 * j) / dv < n) top = x[j].top(top);
      top = __reduce_max_sync(0xffffffffu, top);
      const float now = fmaxf(quant::scale_for<F>(top), old), inv = 1.f / now;
      if (now > old) {
        // (the run's rows are contiguous in the pool, and so are those before it)
        for (int p = lane; p < first * dv; p += 32) {
          uint4* at = reinterpret_cast<uint4*>(dst - first * a.d) + p;
          *at = quant::again<F>(*at, old * inv);
        }
        if (lane == 0) *sc = now;
      }
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int p = lane + 32 * j;
        if (p / dv < n) reinterpret_cast<uint4*>(dst)[p] = quant::encode<F>(x[j], inv);
      }
    }
  }
}

template <typename T, typename F>
cudaError_t launch(const PagedShape& s, QWriteArgs& a, cudaStream_t st) {
  // rows of a window: 16, or fewer where that leaves warps without work
  const int64_t want = (int64_t)num_sms() * 32;
  a.window_shift = 4;
  while (a.window_shift > 0 && (cdiv(a.rows, (int64_t)1 << a.window_shift) * s.Hp() * 2 < want))
    --a.window_shift;
  const int64_t items = cdiv(a.rows, (int64_t)1 << a.window_shift) * s.Hp() * 2;
  int64_t grid = cdiv(items, kThreads / 32);
  const bool full = grid >= (int64_t)num_sms() * 4;
  if (grid > (int64_t)num_sms() * 8) grid = (int64_t)num_sms() * 8;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = full ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, quant_write_kernel<T, F>, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
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
               s.num_pages << shift, s.Hp(), s.d, shift, 0};
  if (s.dtype == KV_BF16)
    return format == KV_E4M3 ? launch<__nv_bfloat16, quant::E4M3>(s, a, st)
                             : launch<__nv_bfloat16, quant::Int8>(s, a, st);
  return format == KV_E4M3 ? launch<float, quant::E4M3>(s, a, st)
                           : launch<float, quant::Int8>(s, a, st);
}

}  // namespace kv
