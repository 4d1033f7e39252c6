// Helpers shared by the key-value cache and the attention kernels (gfx950).
#pragma once

#include "pq_device.h"
#include "pq_internal.h"

namespace pq {

constexpr int kAttnMaxHeads = 1 << 16;
constexpr int64_t kAttnMaxStride = (1ll << 31) - 8;

typedef uint32_t attn_u32x4 __attribute__((ext_vector_type(4)));

// 8 values of a 16-bit type from 16 loaded bytes.
template <bool kBf16>
__device__ __forceinline__ void unpack16x8(const attn_u32x4& q, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = q[i];
    v[2 * i] = kBf16 ? __builtin_bit_cast(float, w << 16) : f16_to_f32(w);
    v[2 * i + 1] = kBf16 ? __builtin_bit_cast(float, w & 0xFFFF0000u) : f16_to_f32(w >> 16);
  }
}

// Two values, or 8, rounded (to nearest even) to a 16-bit type.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return kBf16 ? bf16x2_rn(a, b) : f16x2_rn(a, b);
}
template <bool kBf16>
__device__ __forceinline__ attn_u32x4 pack16x8(const float (&v)[8]) {
  return attn_u32x4{pack2<kBf16>(v[0], v[1]), pack2<kBf16>(v[2], v[3]), pack2<kBf16>(v[4], v[5]), pack2<kBf16>(v[6], v[7])};
}

// 8 e4m3 codes as the values they stand for.
__device__ __forceinline__ void decode8(const uint2& c, float (&v)[8]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const pq_f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), true);
    v[4 * i] = lo.x;
    v[4 * i + 1] = lo.y;
    v[4 * i + 2] = hi.x;
    v[4 * i + 3] = hi.y;
  }
}

// A paged cache and the pages of its sequences.
struct CacheArgs {
  const void* k;
  const void* v;
  const float* ks;          // null: 16-bit rows
  const float* vs;
  const int32_t* table;     // [B][width]
  int64_t pages;
  int width, Hkv, page_shift;
};

// Row of position pos of sequence b and head h in the cache, or -1 where the table has no page of the cache for it.
__device__ __forceinline__ int64_t cache_row(const CacheArgs& c, int b, int h, int64_t pos) {
  const int64_t at = pos >> c.page_shift;
  if (at >= c.width) return -1;
  const int64_t page = c.table[static_cast<int64_t>(b) * c.width + at];
  if (page < 0 || page >= c.pages) return -1;
  return ((page * c.Hkv + h) << c.page_shift) + (pos & ((1ll << c.page_shift) - 1));
}

// Checks shared by the entry points: PQ_OK, or an error code with its message.
int check_cache(const char* what, const void* kc, const void* vc, const float* ks, const float* vs, int64_t pages, int page, int Hkv, int D);
int check_heads(const char* what, const char* name, const void* p, int64_t ld, int64_t hs, int T, int H, int D);

}  // namespace pq
