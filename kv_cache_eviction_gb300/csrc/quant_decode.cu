// quant_decode_attn: attention over pages of 8-bit codes.
#include "paged_decode.cuh"

namespace kv {
namespace {
template <typename T, typename F>
cudaError_t by_width(const PagedShape& s, const PagedArgs& a, cudaStream_t st) {
  if (s.d <= 64)
    return s.d <= 32 ? launch_t<Codes<T, F, 2>>(s, a, st) : launch_t<Codes<T, F, 4>>(s, a, st);
  return s.d <= 96 ? launch_t<Codes<T, F, 6>>(s, a, st) : launch_t<Codes<T, F, 8>>(s, a, st);
}
}  // namespace

size_t quant_decode_ws_bytes(const PagedShape&) { return ws_bytes(kMaxCtasOfCodes); }

cudaError_t launch_quant_decode(const PagedShape& s, int format, const void* q, const void* kn,
                                const void* vn, const int64_t* cu, const int64_t* slots,
                                int64_t slot_capacity, void* kp, void* vp, float* ks, float* vs,
                                const int32_t* table, const int32_t* lens, float scale, void* out,
                                char* ws, cudaStream_t st) {
  const PagedArgs a = args(s, q, kn, vn, cu, slots, slot_capacity, kp, vp, ks, vs, table, lens,
                           scale, out, ws);
  if (s.dtype == KV_BF16)
    return format == KV_E4M3 ? by_width<__nv_bfloat16, quant::E4M3>(s, a, st)
                             : by_width<__nv_bfloat16, quant::Int8>(s, a, st);
  return format == KV_E4M3 ? by_width<float, quant::E4M3>(s, a, st)
                           : by_width<float, quant::Int8>(s, a, st);
}

}  // namespace kv
