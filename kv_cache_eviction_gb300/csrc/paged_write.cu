// Rows of K and V stored at their slots of the page pool: pool[slot / page][h][slot % page] =
// row i's head h.  A copy: bound by reading and writing every row once.
//
// A thread moves one 16-byte piece of a row of K and the same piece of V.
#include "kv_internal.cuh"

namespace kv {
namespace {

constexpr int kWThreads = 256;

__global__ void __launch_bounds__(kWThreads)
paged_write_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v, int64_t src_vec,
                   const int64_t* __restrict__ slots, int64_t rows,
                   const int64_t* __restrict__ n_rows, uint4* __restrict__ kp,
                   uint4* __restrict__ vp, int hp, int dvec, int shift, int64_t page_vec,
                   int64_t num_pages, WsHeader* hdr) {
  if (n_rows != nullptr) {
    const int64_t n = *n_rows;
    rows = n < rows ? n : rows;
  }
  const int per_row = hp * dvec;
  const int64_t total = rows * per_row;
  const int64_t step = (int64_t)gridDim.x * kWThreads;
  for (int64_t i = (int64_t)blockIdx.x * kWThreads + threadIdx.x; i < total; i += step) {
    const int64_t row = i / per_row;
    const int x = (int)(i - row * per_row);
    const int64_t slot = slots[row];
    if (slot < 0 || slot >= (num_pages << shift)) {
      if (slot != -1) raise_dev(hdr, DEV_PAGE_ID, (unsigned)row);
      continue;
    }
    const int h = x / dvec, c = x - h * dvec;
    const int64_t page = slot >> shift, r = slot & ((1 << shift) - 1);
    const int64_t dst = page * page_vec + (((int64_t)h << shift) + r) * dvec + c;
    kp[dst] = k[row * src_vec + x];
    vp[dst] = v[row * src_vec + x];
  }
}
}  // namespace

cudaError_t launch_paged_write(const PagedShape& s, const void* k, const void* v,
                               int64_t src_stride, const int64_t* slots, int64_t rows,
                               const int64_t* n_rows, void* kp, void* vp, WsHeader* hdr,
                               cudaStream_t st) {
  const int ve = 16 / s.esize();
  int shift = 0;
  while ((1 << shift) < s.page) ++shift;
  const int64_t total = rows * s.Hp() * (s.d / ve);
  int64_t grid = cdiv(total, kWThreads);
  if (grid > (int64_t)num_sms() * 8) grid = (int64_t)num_sms() * 8;
  paged_write_kernel<<<(unsigned)grid, kWThreads, 0, st>>>(
      (const uint4*)k, (const uint4*)v, src_stride / ve, slots, rows, n_rows, (uint4*)kp,
      (uint4*)vp, s.Hp(), s.d / ve, shift, s.page_stride / ve, s.num_pages, hdr);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace kv
