// Device helpers of the kernels that read the packed weights (the GEMMs and the 16-bit products).
// The packed image and SZ words are described in pq_gemm.hip.
#pragma once

#include <algorithm>

#include "pq_device.h"

namespace pq {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v8i unpack_codes(const u32x4& w) {
  v8i b;
  b[0] = static_cast<int>(w.x & 0x0F0F0F0Fu);
  b[1] = static_cast<int>((w.x >> 4) & 0x0F0F0F0Fu);
  b[2] = static_cast<int>(w.y & 0x0F0F0F0Fu);
  b[3] = static_cast<int>((w.y >> 4) & 0x0F0F0F0Fu);
  b[4] = static_cast<int>(w.z & 0x0F0F0F0Fu);
  b[5] = static_cast<int>((w.z >> 4) & 0x0F0F0F0Fu);
  b[6] = static_cast<int>(w.w & 0x0F0F0F0Fu);
  b[7] = static_cast<int>((w.w >> 4) & 0x0F0F0F0Fu);
  return b;
}

// {512*sc, zero-point factor} from one SZ word (sc in the low half, zsc in the high half). The
// product is fed the raw int4 code c (factor 8*sc + zsc = sc * zp, zsc = sc * (zp - 8)) or the
// signed int5 code c - 16 (factor zsc = sc * (zp - 16)).
template <bool kW5 = false>
__device__ __forceinline__ float2 sz_factors(uint32_t w) {
  const float sc = f16_to_f32(w), zsc = f16_to_f32(w >> 16);
  if constexpr (kW5) return make_float2(sc * 512.0f, zsc);
  else return make_float2(sc * 512.0f, __builtin_fmaf(sc, 8.0f, zsc));
}

// Direct global -> LDS loads (64 lanes x 4 or 16 bytes to M0 + lane * size; inactive lanes write
// nothing)
// Issued as inline asm so the compiler does not see the LDS write: it would otherwise wait for
// every outstanding request before each LDS read. Completion is tracked explicitly with
// s_waitcnt vmcnt before the workgroup barrier (vmcnt completes in order, so the compiler's
// own waits on its loads stay correct).
// The compiler's hazard checks do not look inside inline asm, so each helper carries the wait
// states its operands may need: a vector memory instruction that reads an SGPR written by a VALU
// instruction (the compiler reloads spilled SGPRs with v_readlane) needs 5, and one that reads M0
// right after an SALU write of M0 needs 1.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ void lds_dma16(const void* g, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void lds_dma4(const void* g, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(g), "{m0}"(lds) : "memory");
}

__device__ __forceinline__ void lds_dma16_on(const void* g, uint32_t lds, bool on) {
  if (on) lds_dma16(g, lds);
}
__device__ __forceinline__ void lds_dma4_on(const void* g, uint32_t lds, bool on) {
  if (on) lds_dma4(g, lds);
}
// scalar base + per-lane 32-bit offset: the per-group address arithmetic stays on the SALU
__device__ __forceinline__ void lds_dma16_s(const void* sbase, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(sbase), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void lds_dma4_s(const void* sbase, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(sbase), "{m0}"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------------------------------
// The column ranges of the kernels that give every CU the same share of the weights (decode, below
// 17 rows): 4-column quarters, dealt out evenly inside each partition.
struct DecodeMap {
  int wg0[4];   // first range of partition q; wg0[3] = number of ranges (the grid)
  int c0[3];    // first column of partition q
  int nq[3];    // quarters (4 columns) of partition q
  int xcd;      // 1: range r = (b % 8) * (grid / 8) + b / 8 for workgroup b
};

// Deals the N/4 column quarters out to ranges: about one range per CU (at most maxq quarters
// each, more ranges in rounds when N is that large), split over the partitions in proportion to
// their quarters, each partition's quarters split evenly over its ranges.
inline void decode_map(int N, int pb1, int pb2, int cus, int maxq, DecodeMap* map) {
  const int cb[4] = {0, pb1 < N ? pb1 : N, pb2 < N ? pb2 : N, N};
  const int64_t Q = N / 4;
  const int64_t tq = std::max<int64_t>(1, std::min<int64_t>(maxq, (Q + cus - 1) / cus));
  int wg = 0;
  for (int q = 0; q < 3; ++q) {
    const int nq = (cb[q + 1] - cb[q]) / 4;
    map->wg0[q] = wg;
    map->c0[q] = cb[q];
    map->nq[q] = nq;
    if (nq > 0) wg += static_cast<int>((nq + tq - 1) / tq);
  }
  map->wg0[3] = wg;
  map->xcd = (wg % 8) == 0;
}

}  // namespace pq
