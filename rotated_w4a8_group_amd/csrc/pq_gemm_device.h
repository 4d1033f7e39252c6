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

__device__ __forceinline__ v4f mfma_fp8(const v8i& a, const v8i& b) {
  const v4f zero = {0.f, 0.f, 0.f, 0.f};
  // format 0 = OCP e4m3 for both operands; scale operands 0 select the unscaled instruction
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

typedef int v4i __attribute__((ext_vector_type(4)));

// Integer-code product of one 128-group: two 16x16x64 int8 matrix-core steps over the same
// 32-byte fragments as the fp8 step (each step pairs the same byte positions of A and B, so the
// two halves together cover every k of the group once); exact in int32, returned as float.
__device__ __forceinline__ v4f mfma_i8(const v8i& a, const v8i& b) {
  v4i c = {0, 0, 0, 0};
  c = __builtin_amdgcn_mfma_i32_16x16x64_i8(v4i{a[0], a[1], a[2], a[3]}, v4i{b[0], b[1], b[2], b[3]}, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_i32_16x16x64_i8(v4i{a[4], a[5], a[6], a[7]}, v4i{b[4], b[5], b[6], b[7]}, c, 0, 0, 0);
  return v4f{static_cast<float>(c[0]), static_cast<float>(c[1]), static_cast<float>(c[2]), static_cast<float>(c[3])};
}

// The group product for either activation code domain: e4m3 codes times the raw weight codes as
// e4m3 values c * 2^-9, or int8 codes times the raw codes as integers.
template <bool kI8>
__device__ __forceinline__ v4f group_product(const v8i& a, const v8i& b) {
  if constexpr (kI8) return mfma_i8(a, b);
  else return mfma_fp8(a, b);
}

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

// int5 weights: the codes' fifth bits ride in a plane beside the nibble image, and the matrix
// core takes c - 16 as the e4m3 value (c - 16) * 2^-9, exact for every code. With the fifth bit
// set that is the low nibble's own byte (as in the int4 path); without it the value is negative
// with magnitude 16 - l, whose e4m3 byte is 0x80 | (16 - l) = 0x90 - l (16 * 2^-9 = 2^-5 is the
// byte 0x10). Bit 8b + j of a lane's plane word belongs to byte b of operand dword j; v_perm
// takes each byte from the nibble value (selector 4 + b) or its negative (selector b).
template <int J>
__device__ __forceinline__ int w5_dword(uint32_t L, uint32_t H) {
  const uint32_t hb = (J >= 2 ? (H >> (J - 2)) : (H << (2 - J))) & 0x04040404u;
  return static_cast<int>(__builtin_amdgcn_perm(L, 0x90909090u - L, 0x03020100u | hb));
}

__device__ __forceinline__ v8i unpack_codes5(const u32x4& w, uint32_t H) {
  v8i b;
  b[0] = w5_dword<0>(w.x & 0x0F0F0F0Fu, H);
  b[1] = w5_dword<1>((w.x >> 4) & 0x0F0F0F0Fu, H);
  b[2] = w5_dword<2>(w.y & 0x0F0F0F0Fu, H);
  b[3] = w5_dword<3>((w.y >> 4) & 0x0F0F0F0Fu, H);
  b[4] = w5_dword<4>(w.z & 0x0F0F0F0Fu, H);
  b[5] = w5_dword<5>((w.z >> 4) & 0x0F0F0F0Fu, H);
  b[6] = w5_dword<6>(w.w & 0x0F0F0F0Fu, H);
  b[7] = w5_dword<7>((w.w >> 4) & 0x0F0F0F0Fu, H);
  return b;
}

// The weight operand of one fragment: int4 nibbles, or nibbles plus the fifth-bit word.
template <bool kW5>
__device__ __forceinline__ v8i weight_operand(const u32x4& w, uint32_t H) {
  if constexpr (kW5) return unpack_codes5(w, H);
  else return unpack_codes(w);
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
// A wave-uniform address in scalar registers, where the compiler computed it on the vector ALU.
__device__ __forceinline__ const void* scalar_addr(const void* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a)), hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
  return reinterpret_cast<const void*>(static_cast<uint64_t>(hi) << 32 | lo);
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Every LDS read issued so far has returned: before a direct load is issued into memory that they read.
__device__ __forceinline__ void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

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
