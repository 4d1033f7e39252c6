// Attention of one new token of each sequence over the paged cache (pq_attn_decode).
//
// One wave per (row, query head): D / 64 channels per lane, the keys one by one with a running maximum and sum.
#include <algorithm>

#include "pq_attn.h"

namespace pq {

struct DecodeArgs {
  CacheArgs c;
  const uint16_t* q;
  int64_t ldq, hsq;
  const int32_t* lens;
  int B, Hq;
  float scale_log2;
  uint16_t* o;
  int out_type;
};

template <int D, bool kBf16, bool kQuant>
__global__ __launch_bounds__(64) void attn_decode_kernel(DecodeArgs a) {
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq, h = hq / (a.Hq / a.c.Hkv);
  float q[D / 64], k[D / 64], v[D / 64];
  lane_values<D, kBf16>(a.q + b * a.ldq + hq * a.hsq, q);
  RowState<D> r;
  const int64_t len = std::min<int64_t>(a.lens[b], static_cast<int64_t>(a.c.width) << a.c.page_shift);
  bool any = false;
  for (int64_t j = 0; j < len; ++j) {
    const int64_t row = cache_row(a.c, b, h, j);
    if (row < 0) continue;
    any = true;
    if constexpr (kQuant) {
      lane_values<D>(static_cast<const uint8_t*>(a.c.k) + row * D, a.c.ks[row], k);
      lane_values<D>(static_cast<const uint8_t*>(a.c.v) + row * D, a.c.vs[row], v);
    } else {
      lane_values<D, kBf16>(static_cast<const uint16_t*>(a.c.k) + row * D, k);
      lane_values<D, kBf16>(static_cast<const uint16_t*>(a.c.v) + row * D, v);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) s += q[i] * k[i];
    r.add(lanes_sum(s), a.scale_log2, v);
  }
  store_row<D>(a.o + (static_cast<int64_t>(b) * a.Hq + hq) * D, r, any, a.out_type);
}

template <int D>
static hipError_t decode_launch(const DecodeArgs& a, int type, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B * a.Hq)), block(64);
  if (a.c.ks)
    return type == PQ_BF16 ? launch_kernel((attn_decode_kernel<D, true, true>), grid, block, 0, s, a)
                           : launch_kernel((attn_decode_kernel<D, false, true>), grid, block, 0, s, a);
  return type == PQ_BF16 ? launch_kernel((attn_decode_kernel<D, true, false>), grid, block, 0, s, a)
                         : launch_kernel((attn_decode_kernel<D, false, false>), grid, block, 0, s, a);
}
}  // namespace pq

extern "C" {

size_t pq_attn_decode_workspace_bytes(int B, int Hq, int Hkv, int D) { return 0; }

int pq_attn_decode(const uint16_t* q_d, int64_t ldq, int64_t hsq, int type, const void* kc_d, const void* vc_d, const float* ks_d, const float* vs_d,
                   int64_t pages, int page, const int32_t* table_d, int width, const int32_t* lens_d, int B, int Hq, int Hkv, int D, float scale,
                   uint16_t* o_d, int out_type, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_attn_decode";
  if (B < 0 || width < 0) return set_error(PQ_ERR_SHAPE, "%s: B=%d, width=%d: negative", what, B, width);
  int rc = check_attention(what, type, out_type, Hq, Hkv, D, scale);
  if (rc == PQ_OK) rc = check_cache(what, kc_d, vc_d, ks_d, vs_d, pages, page, Hkv, D);
  if (rc == PQ_OK) rc = check_heads(what, "q", q_d, ldq, hsq, B, Hq, D);
  if (rc != PQ_OK) return rc;
  if (static_cast<int64_t>(B) * Hq * 64 > 0xFFFFFFFFll) return set_error(PQ_ERR_SHAPE, "%s: B=%d sequences too many for one call", what, B);
  if (B == 0) return PQ_OK;
  if (!o_d || !lens_d || (width && !table_d)) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (!aligned(o_d, 16) || !aligned(lens_d, 4) || !aligned(table_d, 4)) return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  DecodeArgs a{{kc_d, vc_d, ks_d, vs_d, table_d, pages, width, Hkv, __builtin_ctz(page)}, q_d, ldq, hsq, lens_d, B, Hq,
               scale * 1.44269504088896340736f, o_d, out_type};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return launch_status(what, D == 64 ? decode_launch<64>(a, type, s) : D == 128 ? decode_launch<128>(a, type, s) : decode_launch<256>(a, type, s));
}

}  // extern "C"
