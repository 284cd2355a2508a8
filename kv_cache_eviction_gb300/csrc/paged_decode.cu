// Attention of one new token per sequence over the paged cache:
//   z_r = scale * q . k_r,  p = softmax(z) over the rows of the table,  o = sum_r p_r v_r.
//
// One CTA per (sequence, KV head); its warps take the rows in turn, each with a running maximum,
// sum and output per query head (online softmax), merged in shared memory at the end.
#include "kv_internal.cuh"

namespace kv {
namespace {

constexpr int kPWarps = 8;
constexpr int kPThreads = kPWarps * 32;
constexpr int kMaxG = 8;
constexpr int kLaneVals = 4;   // d <= 128 over 32 lanes

struct PagedArgs {
  const void *q, *kn, *vn;
  const int64_t *cu, *slots;
  int64_t slot_cap;
  void *kp, *vp;
  const int32_t *table, *lens;
  void* out;
  WsHeader* hdr;
  int Hkv, G, d, tables, shift, max_pages;
  int64_t num_pages, page_stride;
  float c2;   // softmax scale * log2 e
};

template <typename T>
__global__ void __launch_bounds__(kPThreads) paged_decode_kernel(const PagedArgs a) {
  __shared__ float sm[kPWarps][kMaxG], sl[kPWarps][kMaxG];
  __shared__ float so[kPWarps][kMaxG][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = blockIdx.x;                 // sequence * Hkv + KV head
  const int64_t seq = unit / a.Hkv;
  const int g0 = (int)(unit - seq * a.Hkv);
  const int64_t u = a.tables == 1 ? seq : unit;    // its block table
  const int hp = a.tables == 1 ? g0 : 0;           // its head within a page
  const int d = a.d, G = a.G, page = 1 << a.shift;

  int64_t len = a.lens[u];
  const int64_t most = (int64_t)a.max_pages << a.shift;
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) raise_dev(a.hdr, DEV_PAGE_TABLE, (unsigned)u);
    len = len < 0 ? 0 : most;
  }
  int64_t slot = -1;   // of the new row
  if (a.kn != nullptr && len > 0) {
    const int64_t c0 = a.cu[u], c1 = a.cu[u + 1];
    if (c1 > c0 && c1 > 0 && c1 <= a.slot_cap) slot = a.slots[c1 - 1];
    if (slot < -1 || slot >= (a.num_pages << a.shift)) {
      if (threadIdx.x == 0) raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)u);
      slot = -1;
    }
  }
  const T* q = (const T*)a.q + unit * G * d;
  float qf[kMaxG][kLaneVals], o[kMaxG][kLaneVals], m[kMaxG], l[kMaxG];
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < kLaneVals; ++e) {
      const int x = lane + 32 * e;
      qf[g][e] = g < G && x < d ? to_f(q[g * d + x]) * a.c2 : 0.f;
      o[g][e] = 0.f;
    }
  }
  for (int64_t r = warp; r < len; r += kPWarps) {
    const T *kr, *vr;
    if (r == len - 1 && slot >= 0) {
      kr = (const T*)a.kn + unit * d;
      vr = (const T*)a.vn + unit * d;
      const int64_t at = (slot >> a.shift) * a.page_stride +
                         (((int64_t)hp << a.shift) + (slot & (page - 1))) * d;
      for (int x = lane; x < d; x += 32) {
        ((T*)a.kp)[at + x] = kr[x];
        ((T*)a.vp)[at + x] = vr[x];
      }
    } else {
      const int32_t p = a.table[u * a.max_pages + (r >> a.shift)];
      if (p < 0 || p >= a.num_pages) {
        if (lane == 0) raise_dev(a.hdr, DEV_PAGE_ID, (unsigned)u);
        continue;
      }
      const int64_t at = p * a.page_stride + (((int64_t)hp << a.shift) + (r & (page - 1))) * d;
      kr = (const T*)a.kp + at;
      vr = (const T*)a.vp + at;
    }
    float kf[kLaneVals], vf[kLaneVals];
#pragma unroll
    for (int e = 0; e < kLaneVals; ++e) {
      const int x = lane + 32 * e;
      kf[e] = x < d ? to_f(kr[x]) : 0.f;
      vf[e] = x < d ? to_f(vr[x]) : 0.f;
    }
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
      if (g < G) {
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < kLaneVals; ++e) z = fmaf(qf[g][e], kf[e], z);
        z = warp_sum(z);
        const float mn = fmaxf(m[g], z);
        const float w = exp2f(m[g] - mn), p = exp2f(z - mn);
        m[g] = mn;
        l[g] = fmaf(l[g], w, p);
#pragma unroll
        for (int e = 0; e < kLaneVals; ++e) o[g][e] = fmaf(o[g][e], w, p * vf[e]);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    if (lane == 0) {
      sm[warp][g] = m[g];
      sl[warp][g] = l[g];
    }
#pragma unroll
    for (int e = 0; e < kLaneVals; ++e) so[warp][g][lane + 32 * e] = o[g][e];
  }
  __syncthreads();
  T* out = (T*)a.out + unit * G * d;
  for (int i = threadIdx.x; i < G * d; i += kPThreads) {
    const int g = i / d, x = i - g * d;
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int w = 0; w < kPWarps; ++w) M = fmaxf(M, sm[w][g]);
    for (int w = 0; w < kPWarps; ++w) {
      if (sl[w][g] > 0.f) {
        const float f = exp2f(sm[w][g] - M);
        L = fmaf(sl[w][g], f, L);
        acc = fmaf(so[w][g][x], f, acc);
      }
    }
    out[i] = from_f<T>(L > 0.f ? acc / L : 0.f);
  }
}
}  // namespace

size_t paged_decode_ws_bytes(const PagedShape& s) { return kWsHeader; }

cudaError_t launch_paged_decode(const PagedShape& s, const void* q, const void* kn, const void* vn,
                                const int64_t* cu, const int64_t* slots, int64_t slot_capacity,
                                void* kp, void* vp, const int32_t* table, const int32_t* lens,
                                float scale, void* out, char* ws, cudaStream_t st) {
  int shift = 0;
  while ((1 << shift) < s.page) ++shift;
  PagedArgs a{q, kn, vn, cu, slots, slot_capacity, kp, vp, table, lens, out,
              reinterpret_cast<WsHeader*>(ws), s.Hkv, s.G(), s.d, s.tables, shift, s.max_pages,
              s.num_pages, s.page_stride, scale * 1.4426950408889634f};
  const unsigned grid = (unsigned)((int64_t)s.seqs * s.Hkv);
  if (s.dtype == KV_BF16) paged_decode_kernel<__nv_bfloat16><<<grid, kPThreads, 0, st>>>(a);
  else paged_decode_kernel<float><<<grid, kPThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace kv
