// Helpers shared by the key-value cache and the attention kernels (gfx950).
#pragma once

#include "pq_gemm_device.h"
#include "pq_internal.h"

namespace pq {

constexpr int kAttnMaxHeads = 1 << 16;
constexpr float kAttnMaxScale = 0x1p64f;
constexpr int64_t kAttnMaxStride = 1ll << 24;   // elements: 64 rows stay within 32-bit offsets

typedef uint32_t attn_u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

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
// sum + the two values of a word
template <bool kBf16>
__device__ __forceinline__ float add_pair(uint32_t w, float sum) {
  if constexpr (kBf16) return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(pq_bf16x2, w), pq_bf16x2{1.0f, 1.0f}, sum, false);
  else return __builtin_amdgcn_fdot2(__builtin_bit_cast(pq_f16x2, w), pq_f16x2{1.0f, 1.0f}, sum, false);
}
template <bool kBf16>
__device__ __forceinline__ attn_u32x4 pack16x8(const float (&v)[8]) {
  return attn_u32x4{pack2<kBf16>(v[0], v[1]), pack2<kBf16>(v[2], v[3]), pack2<kBf16>(v[4], v[5]), pack2<kBf16>(v[6], v[7])};
}

// Four values rounded to the type of an output.
__device__ __forceinline__ uint2 pack4(int type, float x, float y, float z, float w) {
  return type == PQ_BF16 ? make_uint2(pack2<true>(x, y), pack2<true>(z, w)) : make_uint2(pack2<false>(x, y), pack2<false>(z, w));
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

// A direct load of 16 bytes a lane (LDS address uniform, lane i lands 16 i bytes in) of data that is read once: it does not stay
// in the caches.
__device__ __forceinline__ void lds_dma16_nt(const void* sbase, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(voff), "s"(sbase), "{m0}"(lds) : "memory");
}

// The same number, where the compiler may not know it: what an address takes from it is computed where it is used, a few vector
// instructions, and not kept in a register for the whole loop.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int lanes_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // within 16 lanes: 1, 2, 4, 8 back
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // the last lane of 16 to the next 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // that of 32 to the upper 32
  return v;
}
__device__ __forceinline__ int lanes_total(int v) { return __builtin_amdgcn_readlane(lanes_scan(v), 63); }

// 4 keys of one channel a lane: lane l gives the address of key l % 16 / 4 and channels 4 (l % 4) .. + 3 of its 16 lanes' 4 x 16 block
// and gets channel l % 16 of the 4 keys.
__device__ __forceinline__ uint2 lds_read_transposed(const uint8_t* p) {
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uintptr_t)lds_addr(p)));
}

// A value of this lane and of the same lane of the other half of the wave, the lower half's first.
struct Halves { float lo, hi; };
__device__ __forceinline__ Halves both_halves(float v) {
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  const uint32_t lo = r[0], hi = r[1];
  return {__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}
__device__ __forceinline__ float both_halves_max(float v) { const Halves x = both_halves(v); return __builtin_fmaxf(x.lo, x.hi); }
__device__ __forceinline__ float both_halves_sum(float v) { const Halves x = both_halves(v); return x.lo + x.hi; }

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

// Running softmax of one query row: the largest score so far, the sum of exp2(c (score - largest)) and the mean of the values so
// far under these weights - a mean, as the weighted sum of finite values may pass binary32 where their mean does not.
template <int D>
struct RowState {
  float m = -__builtin_inff(), l = 0.0f, o[D / 64] = {};
  __device__ __forceinline__ void add(float s, float c, const float (&v)[D / 64]) {
    const float n = s > m ? s : m;   // a NaN score leaves m and makes the sum NaN
    const float f = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(c * (m - n));
    const float p = s == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(c * (s - n));
    m = n;
    l = l * f + p;
    if (l == 0.0f) return;           // scores of -inf alone so far
    const float w = p / l, rest = 1.0f - w;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) o[i] = o[i] * rest + v[i] * w;
  }
};

template <int D>
__device__ __forceinline__ void store_row(uint16_t* out, const RowState<D>& r, bool any, int out_type) {
  const int lane = threadIdx.x & 63;
  const float none = r.l > 0.0f ? 0.0f : __builtin_nanf("");   // no weight at all, or NaN
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const float v = any ? r.o[i] + none : 0.0f;
    out[lane * (D / 64) + i] = static_cast<uint16_t>(out_type == PQ_BF16 ? pack2<true>(v, v) : pack2<false>(v, v));
  }
}

// Bytes that T rows of H heads reach over from their first element on.
inline int64_t heads_span(int64_t ld, int64_t hs, int64_t T, int64_t H, int64_t D) { return T <= 0 ? 0 : 2 * ((T - 1) * ld + (H - 1) * hs + D); }
// Whether two ranges of bytes have one in common; an output shares none with an input.
inline bool ranges_meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && p < q + static_cast<uintptr_t>(nb) && q < p + static_cast<uintptr_t>(na);
}
inline int overlap(const char* what) { return set_error(PQ_ERR_SHAPE, "%s: an output overlaps an input or another output", what); }

// Checks shared by the entry points: PQ_OK, or an error code with its message.
int check_cache(const char* what, const void* kc, const void* vc, const float* ks, const float* vs, int64_t pages, int page, int Hkv, int D);
int64_t cache_bytes(const float* scales, int64_t pages, int page, int Hkv, int D);
int64_t scale_bytes(const float* scales, int64_t pages, int page, int Hkv);
int check_heads(const char* what, const char* name, const void* p, int64_t ld, int64_t hs, int T);
inline int check_attention(const char* what, int type, int out_type, int Hq, int Hkv, int D, float scale) {
  if ((type != PQ_F16 && type != PQ_BF16) || (out_type != PQ_F16 && out_type != PQ_BF16))
    return set_error(PQ_ERR_SHAPE, "%s: types (%d, out %d): f16 or bf16", what, type, out_type);
  if (D != 64 && D != 128 && D != 256) return set_error(PQ_ERR_SHAPE, "%s: head size D=%d must be 64, 128 or 256", what, D);
  if (Hkv <= 0 || Hkv > kAttnMaxHeads || Hq <= 0 || Hq > kAttnMaxHeads || Hq % Hkv)
    return set_error(PQ_ERR_SHAPE, "%s: Hq=%d must be a multiple of Hkv=%d, both in 1..%d", what, Hq, Hkv, kAttnMaxHeads);
  if (!(scale > 0.0f) || !(scale <= kAttnMaxScale)) return set_error(PQ_ERR_SHAPE, "%s: scale must be positive, at most 2^64", what);
  return PQ_OK;
}

}  // namespace pq
