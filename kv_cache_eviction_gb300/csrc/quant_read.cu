// Rows of the 8-bit cache as the values they stand for: code * scale, which bf16 and fp32 hold
// exactly.  Bound by reading the codes and writing the rows once.  A lane writes 16 bytes of K's
// rows and of V's at a time, its neighbours those beside them.  On GB300: 131072 rows of 8 heads of
// 128 bf16 from int8 (806 MB) 121.6 us, 6.6 TB/s or 0.98 of the measured copy rate (141 us with 16
// codes a lane, whose stores fill half sectors), into fp32 rows (1.3 GB) 202 us; 513 rows 2.4 us.
#include "quant_codes.cuh"
#include "tc_ptx.cuh"

namespace kv {
namespace {

constexpr int kThreads = 128;
constexpr int kPieces = 4;   // 16-byte pieces of K's rows (and of V's) of a lane at a time

struct QReadArgs {
  const unsigned char *kp, *vp;
  const float *ks, *vs;
  const int64_t* slots;
  const int64_t* n_rows;
  uint4 *k, *v;
  WsHeader* hdr;
  int64_t rows, dst_vec, page_stride, num_slots;   // dst_vec: 16-byte pieces from row to row
  int per_row, pad_shift;    // pieces of a row, and log2 of its padded pieces (a group's, at most)
  int Hp, d, shift;
  int dvec, div_dvec;        // pieces of a head's row; x / dvec = x * div_dvec >> 20
};

// kN codes: those of 16 bytes of a row.
template <typename T>
struct Code;
template <>
struct Code<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void load(const unsigned char* p) {
    w = *reinterpret_cast<const uint2*>(p);
  }
  template <typename F>
  __device__ __forceinline__ uint4 row(float s) const {
    auto two = [&](uint32_t h) {
      const float2 x = quant::floats_of(h);
      const __nv_bfloat162 y = __floats2bfloat162_rn(x.x * s, x.y * s);
      return *reinterpret_cast<const uint32_t*>(&y);
    };
    uint32_t a, b, c, d;
    F::halves(w.x, a, b);
    F::halves(w.y, c, d);
    return make_uint4(two(a), two(b), two(c), two(d));
  }
};
template <>
struct Code<float> {
  uint32_t w;
  __device__ __forceinline__ void load(const unsigned char* p) {
    w = *reinterpret_cast<const uint32_t*>(p);
  }
  template <typename F>
  __device__ __forceinline__ uint4 row(float s) const {
    uint32_t a, b;
    F::halves(w, a, b);
    const float2 x = quant::floats_of(a), y = quant::floats_of(b);
    return make_uint4(__float_as_uint(x.x * s), __float_as_uint(x.y * s), __float_as_uint(y.x * s),
                      __float_as_uint(y.y * s));
  }
};

template <typename T, typename F>
__global__ void __launch_bounds__(kThreads, 8)
quant_read_kernel(const __grid_constant__ QReadArgs a) {
  constexpr int kN = 16 / (int)sizeof(T);   // codes of a piece
  const int lane = threadIdx.x & 31, page = 1 << a.shift;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();   // nothing of the call before is read or written until it ends
  int64_t rows = a.rows;
  if (a.n_rows != nullptr) rows = min(rows, *a.n_rows);
  constexpr int kGroup = 32 * kPieces;            // pieces at a time
  const int in_group = kGroup >> a.pad_shift;     // rows, at most 32
  const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32) * in_group;
  // lane i: the slot of the group's row i, -1 outside the rows
  auto load_slot = [&](int64_t row0) {
    return lane < in_group && row0 + lane < rows ? a.slots[row0 + lane] : (int64_t)-1;
  };
  int64_t next = load_slot(warp * in_group);
  for (int64_t row0 = warp * in_group; row0 < rows; row0 += step) {
    int64_t slot = next;
    next = load_slot(row0 + step);   // (its latency beside this group's)
    if (slot < 0 || slot >= a.num_slots) {
      if (slot != -1) raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)(row0 + lane));
      slot = -1;
    }
    for (int x0 = 0; x0 < a.per_row; x0 += kGroup) {
      Code<T> kc[kPieces], vc[kPieces];
      float ks[kPieces], vs[kPieces];
      bool in[kPieces];
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int i = lane + 32 * j;
        const int x = x0 + (i & ((1 << a.pad_shift) - 1));
        const int64_t s = __shfl_sync(0xffffffffu, (long long)slot, i >> a.pad_shift);
        in[j] = x < a.per_row && s >= 0;
        if (in[j]) {
          const int64_t pg = s >> a.shift;
          const int r = (int)(s & (page - 1)), h = x * a.div_dvec >> 20;
          const int64_t at =
              pg * a.page_stride + ((int64_t)h * page + r) * a.d + (x - h * a.dvec) * kN;
          const int64_t sc = (pg * a.Hp + h) * (page / quant::kBlock) + r / quant::kBlock;
          kc[j].load(a.kp + at);
          vc[j].load(a.vp + at);
          ks[j] = a.ks[sc];
          vs[j] = a.vs[sc];
        }
      }
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        if (!in[j]) continue;
        const int i = lane + 32 * j;
        const int64_t row = row0 + (i >> a.pad_shift);
        const int x = x0 + (i & ((1 << a.pad_shift) - 1));
        a.k[row * a.dst_vec + x] = kc[j].template row<F>(ks[j]);
        a.v[row * a.dst_vec + x] = vc[j].template row<F>(vs[j]);
      }
    }
  }
}

template <typename T, typename F>
cudaError_t launch(const QReadArgs& a, cudaStream_t st) {
  int64_t grid = cdiv(a.rows, (int64_t)(32 * kPieces >> a.pad_shift) * (kThreads / 32));
  // (many small CTAs even out what the SMs get through: 131072 rows 121.6 us; 122.9 with 32 of
  // twice the threads, 130.6 with 8, 126.2 without a limit)
  const int64_t most = (int64_t)num_sms() * 64;
  if (grid > most) grid = most;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;   // (calls of 513 rows one after the other 3.0 us, 4.2 without)
  const cudaError_t e = cudaLaunchKernelEx(&cfg, quant_read_kernel<T, F>, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}
}  // namespace

cudaError_t launch_quant_read(const PagedShape& s, int format, const void* kp, const void* vp,
                              const float* ks, const float* vs, const int64_t* slots, int64_t rows,
                              const int64_t* n_rows, void* k, void* v, int64_t dst_stride,
                              WsHeader* hdr, cudaStream_t st) {
  int shift = 0;
  while ((1 << shift) < s.page) ++shift;
  const int dvec = s.d * s.esize() / 16, per_row = s.Hp() * dvec;
  int pad = 0;   // a group has at most 32 rows
  while ((32 * kPieces >> pad) > 32 || ((32 * kPieces >> pad) > 1 && (1 << pad) < per_row)) ++pad;
  // x / dvec by a product: x < 256 * 32, and the product is too large by less than dvec / 2^20 a
  // unit, so the quotient is exact (8192 * 32 < 2^20)
  const int div = ((1 << 20) + dvec - 1) / dvec;
  const QReadArgs a{(const unsigned char*)kp, (const unsigned char*)vp, ks, vs, slots, n_rows,
                    (uint4*)k, (uint4*)v, hdr, rows, dst_stride * s.esize() / 16, s.page_stride,
                    s.num_pages << shift, per_row, pad, s.Hp(), s.d, shift, dvec,
                    div};
  if (s.dtype == KV_BF16)
    return format == KV_E4M3 ? launch<__nv_bfloat16, quant::E4M3>(a, st)
                             : launch<__nv_bfloat16, quant::Int8>(a, st);
  return format == KV_E4M3 ? launch<float, quant::E4M3>(a, st)
                           : launch<float, quant::Int8>(a, st);
}

}  // namespace kv
