// Rows of K and V stored at their slots of the page pool: pool[slot / page][h][slot % page] =
// row i's head h.  A copy: bound by reading and writing every row once (latency, for a few rows).
//
// A warp moves groups of rows, 128 16-byte pieces of K and of V at a time: rows of up to 64
// pieces share a group, each padded to a power of two pieces so that a lane finds its row by a
// shift; longer rows take several groups.  The eight loads of a lane do not wait for the slots,
// only its stores do.  On GB300: 131072 rows of 8 heads of 128 bf16 (1.07 GB read and written)
// 161 us, 6.67 TB/s or 0.98 of the measured copy rate (172 us with one piece a thread and its
// divisions); 100003 rows of one head of 64 fp32 16.7 us, 6.2 TB/s; 64 rows 2.3 us.
#include "kv_internal.cuh"
#include "tc_ptx.cuh"

namespace kv {
namespace {

constexpr int kWThreads = 256;
constexpr int kWPieces = 4;   // pieces of K (and of V) of a lane at a time

struct WriteArgs {
  const uint4 *k, *v;
  const int64_t* slots;
  const int64_t* n_rows;
  uint4 *kp, *vp;
  WsHeader* hdr;
  int64_t rows, src_vec, page_vec, num_slots;   // *_vec: 16-byte pieces
  int per_row, pad_shift;   // pieces of a row, and log2 of its padded pieces (7: whole groups)
  int dvec, div_dvec;       // pieces of a head's row; x / dvec = x * div_dvec >> 20
  int page_shift;
};

__global__ void __launch_bounds__(kWThreads) paged_write_kernel(const WriteArgs a) {
  const int lane = threadIdx.x & 31;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();   // nothing of the call before is read or written until it ends
  int64_t rows = a.rows;
  if (a.n_rows != nullptr) rows = min(rows, *a.n_rows);
  const int in_group = 128 >> a.pad_shift;   // rows
  const int64_t warp = (int64_t)blockIdx.x * (kWThreads / 32) + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * (kWThreads / 32) * in_group;
  const int heads_apart = ((1 << a.page_shift) - 1) * a.dvec;   // extra pieces from head to head
  for (int64_t row0 = warp * in_group; row0 < rows; row0 += step) {
    for (int x0 = 0; x0 < a.per_row; x0 += 128) {
      uint4 kx[kWPieces], vx[kWPieces];
      int64_t slot[kWPieces];
#pragma unroll
      for (int j = 0; j < kWPieces; ++j) {
        const int i = lane + 32 * j;
        const int64_t row = row0 + (i >> a.pad_shift);
        const int x = x0 + (i & ((1 << a.pad_shift) - 1));
        slot[j] = -1;
        if (x < a.per_row && row < rows) {
          slot[j] = a.slots[row];
          kx[j] = a.k[row * a.src_vec + x];
          vx[j] = a.v[row * a.src_vec + x];
        }
      }
#pragma unroll
      for (int j = 0; j < kWPieces; ++j) {
        const int i = lane + 32 * j;
        const int x = x0 + (i & ((1 << a.pad_shift) - 1));
        if (slot[j] >= 0 && slot[j] < a.num_slots) {
          const int64_t page = slot[j] >> a.page_shift;
          const int r = (int)(slot[j] & ((1 << a.page_shift) - 1));
          const int h = x * a.div_dvec >> 20;
          const int64_t dst = page * a.page_vec + r * a.dvec + x + h * heads_apart;
          a.kp[dst] = kx[j];
          a.vp[dst] = vx[j];
        } else if (slot[j] != -1) {
          raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)(row0 + (i >> a.pad_shift)));
        }
      }
    }
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
  const int dvec = s.d / ve, per_row = s.Hp() * dvec;
  int pad = 0;
  while (pad < 7 && (1 << pad) < per_row) ++pad;
  // x / dvec by a product: x < 256 * 32, and the product is too large by less than dvec / 2^20
  // a unit, so the quotient is exact (8192 * 32 < 2^20)
  const int div = ((1 << 20) + dvec - 1) / dvec;
  const WriteArgs a{(const uint4*)k, (const uint4*)v, slots, n_rows, (uint4*)kp, (uint4*)vp, hdr,
                    rows, src_stride / ve, s.page_stride / ve, s.num_pages << shift, per_row, pad,
                    dvec, div, shift};
  int64_t grid = cdiv(rows, (int64_t)(128 >> pad) * (kWThreads / 32));
  if (grid > (int64_t)num_sms() * 8) grid = (int64_t)num_sms() * 8;
  // A programmatic dependent launch costs the host 0.7 us: worth it where the call fills the SMs
  // (100003 rows of one head 16.7 us against 17.2), not where the host is the slower side (64 rows:
  // 1.9 us on the device against 2.1, 9.0 from Python against 8.3).
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kWThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = grid == (int64_t)num_sms() * 8 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_write_kernel, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace kv
