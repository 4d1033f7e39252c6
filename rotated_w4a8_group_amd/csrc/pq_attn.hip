// Attention of one new token of each sequence over the paged cache (pq_attn_decode) and over packed prompts
// (pq_attn_prefill).
//
// One wave per (row, query head): D / 64 channels per lane, the keys one by one with a running maximum and sum.
#include <algorithm>

#include "pq_attn.h"

namespace pq {

// Sum over the wave, the same value in every lane.
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m);
  return v;
}

// The D / 64 values of this lane in a 16-bit row.
template <int D, bool kBf16>
__device__ __forceinline__ void lane_values(const uint16_t* row, float (&v)[D / 64]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const uint32_t w = row[lane * (D / 64) + i];
    v[i] = kBf16 ? bf16_to_f32(w) : f16_to_f32(w);
  }
}
template <int D>
__device__ __forceinline__ void lane_values(const uint8_t* row, float s, float (&v)[D / 64]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) v[i] = s * __builtin_amdgcn_cvt_f32_fp8(row[lane * (D / 64) + i], 0);
}

// Running softmax of one query row: the largest score so far, the sum of exp2(c (score - largest)) and the weighted values.
template <int D>
struct RowState {
  float m = -__builtin_inff(), l = 0.0f, o[D / 64] = {};
  __device__ __forceinline__ void add(float s, float c, const float (&v)[D / 64]) {
    const float n = s > m ? s : m;   // a NaN score leaves m and makes the sum NaN
    const float f = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(c * (m - n));
    const float p = s == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(c * (s - n));
    m = n;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) o[i] = o[i] * f + p * v[i];
  }
};

template <int D>
__device__ __forceinline__ void store_row(uint16_t* out, const RowState<D>& r, bool any, int out_type) {
  const int lane = threadIdx.x & 63;
  const float inv = any ? 1.0f / r.l : 0.0f;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const float v = any ? r.o[i] * inv : 0.0f;
    out[lane * (D / 64) + i] = static_cast<uint16_t>(out_type == PQ_BF16 ? pack2<true>(v, v) : pack2<false>(v, v));
  }
}

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

struct PrefillArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t ldq, hsq, ldk, hsk, ldv, hsv;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk, Hq, Hkv, causal;
  float scale_log2;
  uint16_t* o;
  int out_type;
};

template <int D, bool kBf16>
__global__ __launch_bounds__(64) void attn_prefill_kernel(PrefillArgs a) {
  const int64_t t = blockIdx.x / a.Hq;
  const int hq = blockIdx.x % a.Hq, h = hq / (a.Hq / a.Hkv);
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_q[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int q0 = std::max(a.cu_q[lo], 0), q1 = std::min(a.cu_q[lo + 1], a.Tq);
  if (t < q0 || t >= q1) return;
  const int k0 = std::min(std::max(a.cu_k[lo], 0), a.Tk), nk = std::min(std::max(a.cu_k[lo + 1], k0), a.Tk) - k0;
  const int keys = a.causal ? std::max<int64_t>(0, std::min<int64_t>(nk, t - q1 + nk + 1)) : nk;
  float q[D / 64], k[D / 64], v[D / 64];
  lane_values<D, kBf16>(a.q + t * a.ldq + hq * a.hsq, q);
  RowState<D> r;
  for (int j = 0; j < keys; ++j) {
    lane_values<D, kBf16>(a.k + static_cast<int64_t>(k0 + j) * a.ldk + h * a.hsk, k);
    lane_values<D, kBf16>(a.v + static_cast<int64_t>(k0 + j) * a.ldv + h * a.hsv, v);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) s += q[i] * k[i];
    r.add(lanes_sum(s), a.scale_log2, v);
  }
  store_row<D>(a.o + (t * a.Hq + hq) * D, r, keys > 0, a.out_type);
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
template <int D>
static hipError_t prefill_launch(const PrefillArgs& a, int type, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.Tq * a.Hq)), block(64);
  return type == PQ_BF16 ? launch_kernel((attn_prefill_kernel<D, true>), grid, block, 0, s, a)
                         : launch_kernel((attn_prefill_kernel<D, false>), grid, block, 0, s, a);
}

static int check_attention(const char* what, int type, int out_type, int Hq, int Hkv, int D, float scale) {
  if ((type != PQ_F16 && type != PQ_BF16) || (out_type != PQ_F16 && out_type != PQ_BF16))
    return set_error(PQ_ERR_SHAPE, "%s: types (%d, out %d): f16 or bf16", what, type, out_type);
  if (D != 64 && D != 128 && D != 256) return set_error(PQ_ERR_SHAPE, "%s: head size D=%d must be 64, 128 or 256", what, D);
  if (Hkv <= 0 || Hkv > kAttnMaxHeads || Hq <= 0 || Hq > kAttnMaxHeads || Hq % Hkv)
    return set_error(PQ_ERR_SHAPE, "%s: Hq=%d must be a multiple of Hkv=%d, both in 1..%d", what, Hq, Hkv, kAttnMaxHeads);
  if (!(scale > 0.0f) || !(scale < __builtin_inff())) return set_error(PQ_ERR_SHAPE, "%s: scale must be positive and finite", what);
  return PQ_OK;
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

size_t pq_attn_prefill_workspace_bytes(int B, int Tq, int Tk, int Hq, int Hkv, int D) { return 0; }

int pq_attn_prefill(const uint16_t* q_d, int64_t ldq, int64_t hsq, const uint16_t* k_d, int64_t ldk, int64_t hsk, const uint16_t* v_d, int64_t ldv,
                    int64_t hsv, int type, const int32_t* cu_q_d, const int32_t* cu_k_d, int B, int Tq, int Tk, int Hq, int Hkv, int D, float scale,
                    int causal, uint16_t* o_d, int out_type, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_attn_prefill";
  if (B < 0 || Tq < 0 || Tk < 0) return set_error(PQ_ERR_SHAPE, "%s: B=%d, Tq=%d, Tk=%d: negative", what, B, Tq, Tk);
  int rc = check_attention(what, type, out_type, Hq, Hkv, D, scale);
  if (rc == PQ_OK) rc = check_heads(what, "q", q_d, ldq, hsq, Tq, Hq, D);
  if (rc == PQ_OK) rc = check_heads(what, "k", k_d, ldk, hsk, Tk, Hkv, D);
  if (rc == PQ_OK) rc = check_heads(what, "v", v_d, ldv, hsv, Tk, Hkv, D);
  if (rc != PQ_OK) return rc;
  if (static_cast<int64_t>(Tq) * Hq * 64 > 0xFFFFFFFFll) return set_error(PQ_ERR_SHAPE, "%s: Tq=%d rows too many for one call", what, Tq);
  if (Tq == 0 || B == 0) return PQ_OK;
  if (!o_d || !cu_q_d || !cu_k_d) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (!aligned(o_d, 16) || !aligned(cu_q_d, 4) || !aligned(cu_k_d, 4)) return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  PrefillArgs a{q_d, k_d, v_d, ldq, hsq, ldk, hsk, ldv, hsv, cu_q_d, cu_k_d, B, Tq, Tk, Hq, Hkv, causal, scale * 1.44269504088896340736f, o_d, out_type};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return launch_status(what, D == 64 ? prefill_launch<64>(a, type, s) : D == 128 ? prefill_launch<128>(a, type, s) : prefill_launch<256>(a, type, s));
}

}  // extern "C"
