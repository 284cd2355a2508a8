// paged_decode_attn: attention over pages of bf16 or fp32 rows.
#include "paged_decode.cuh"

namespace kv {

size_t paged_decode_ws_bytes(const PagedShape&) { return ws_bytes(kMaxCtas); }

cudaError_t launch_paged_decode(const PagedShape& s, const void* q, const void* kn, const void* vn,
                                const int64_t* cu, const int64_t* slots, int64_t slot_capacity,
                                void* kp, void* vp, const int32_t* table, const int32_t* lens,
                                float scale, void* out, char* ws, cudaStream_t st) {
  const PagedArgs a = args(s, q, kn, vn, cu, slots, slot_capacity, kp, vp, nullptr, nullptr, table,
                           lens, scale, out, ws);
  if (s.dtype == KV_BF16) {
    if (s.d <= 64) return launch_t<Rows<__nv_bfloat16, 2>>(s, a, st);
    return s.d <= 96 ? launch_t<Rows<__nv_bfloat16, 3>>(s, a, st)
                     : launch_t<Rows<__nv_bfloat16, 4>>(s, a, st);
  }
  if (s.d <= 32) return launch_t<Rows<float, 2>>(s, a, st);
  if (s.d <= 64) return launch_t<Rows<float, 4>>(s, a, st);
  if (s.d <= 80) return launch_t<Rows<float, 5>>(s, a, st);
  return s.d <= 96 ? launch_t<Rows<float, 6>>(s, a, st) : launch_t<Rows<float, 8>>(s, a, st);
}

}  // namespace kv
