// W4A8 group GEMM for gfx950: weight packing, the decode kernel (M <= 16) and the prefill
// kernel, all on the fp8 matrix cores (v_mfma_f32_16x16x128_f8f6f4).
//
// Method ("ParoQuant (PARO) W4A8 on gfx1201 — engineering log", section "Design" items 1, 2
// and 4): per 128-group g the weight value is sc * (c - zp) with (c - zp) = (c - 8) - d,
// d = zp - 8, so
//     y[m,n] = sum_g asg[m,g] * ( sc * sum_k D(a_k) (c_k - 8) - fl16(sc*d) * rs[m,g] ),
// with rs the code-domain row-sum the prologue emits and SZ = {sc, fl16(sc*d)} interleaved.
//
// gfx950 operand choice (this library's, not the page's): the matrix core takes the raw
// 4-bit code c as an OCP e4m3 byte. Codes 0x00..0x0F are exactly c * 2^-9 (subnormals, then
// the first normal binade), and the MFMA handles e4m3 subnormals exactly, so unpacking a
// nibble is a mask — no lookup table. The MFMA then returns T = 2^-9 * sum_k D(a_k) c_k and
//     sc * sum_k D(a_k)(c_k - 8) - zsc * rs = (512 sc) * T - (8 sc + zsc) * rs,
// both factors exact in fp32 (512 sc is a power-of-two scaling, 8 sc + zsc needs < 24 bits).
//
// Packed weight image (pq_pack_weights): the codes below, then the zero-point epilogue operand,
// then the prefill fold's fp32 column factors 512 sc [G][N].
// Packed code layout, tile-major so that one column tile's whole K extent
// is one contiguous run: for 16-column tile t and group g, 1 KiB at ((t * G + g) * 1024): lane l (column 16t + l%16, k = 128g + 32*(l/16) + 0..31) owns 16 bytes
// = 4 words; byte b of word q holds code(k0 + 8q + b) in its low nibble and code(k0 + 8q + 4 + b)
// in its high nibble. (w & 0x0F0F0F0F) and ((w >> 4) & 0x0F0F0F0F) are then the lane's B
// operand registers 2q and 2q+1, matching the A operand's 32 consecutive k bytes.
#include <mutex>

#include "pq_device.h"
#include "pq_gemm_device.h"
#include "pq_internal.h"
#include "pq_prefill.h"

namespace pq {

// column n -> nibble position inside its AWQ word (inverse of the order 0,2,4,6,1,3,5,7)
__device__ __forceinline__ int awq_shift(int n) {
  const int c = n & 7;
  return 4 * ((c >> 1) + ((c & 1) << 2));
}

// ---------------------------------------------------------------------------------------
// packing
__global__ void pack_weights_kernel(const int32_t* __restrict__ qweight, int K, int N,
                                    uint32_t* __restrict__ wpk) {
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t total = static_cast<int64_t>(K) * N / 8;
  if (idx >= total) return;
  const int q = static_cast<int>(idx & 3);
  const int l = static_cast<int>((idx >> 2) & 63);
  const int64_t rest = idx >> 8;
  const int G = K >> 7;
  const int t = static_cast<int>(rest / G);
  const int g = static_cast<int>(rest % G);
  const int n = 16 * t + (l & 15);
  const int k0 = 128 * g + 32 * (l >> 4) + 8 * q;
  const int shift = awq_shift(n);
  const int64_t N8 = N / 8;
  uint32_t w = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t lo = (static_cast<uint32_t>(qweight[(k0 + b) * N8 + n / 8]) >> shift) & 0xFu;
    const uint32_t hi = (static_cast<uint32_t>(qweight[(k0 + 4 + b) * N8 + n / 8]) >> shift) & 0xFu;
    w |= (lo | (hi << 4)) << (8 * b);
  }
  wpk[idx] = w;
}

__global__ void pack_sz_kernel(const int32_t* __restrict__ qzeros, const uint16_t* __restrict__ scales,
                               int G, int N, uint32_t* __restrict__ sz) {
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= static_cast<int64_t>(G) * N) return;
  const int g = static_cast<int>(idx / N), n = static_cast<int>(idx % N);
  const uint32_t zp = (static_cast<uint32_t>(qzeros[static_cast<int64_t>(g) * (N / 8) + n / 8]) >> awq_shift(n)) & 0xFu;
  const uint16_t sc = scales[idx];
  // sc * (zp - 8) is exact in fp32 (11 x 4 significand bits); one rounding to f16
  const _Float16 zsc = static_cast<_Float16>(f16_to_f32(sc) * static_cast<float>(static_cast<int>(zp) - 8));
  sz[idx] = static_cast<uint32_t>(sc) | (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, zsc)) << 16);
}

// int5 fifth-bit plane image: per (16-column tile t, group g) 64 lanes x 4 B; bit 8b + j of lane
// l's word is the fifth bit of the code at k = 128g + 32(l/16) + 4j + b, column 16t + l%16 (the
// k of byte b of dword j of the lane's weight operand). One thread per word.
__global__ void pack_hi_kernel(const int32_t* __restrict__ qweight_hi, int K, int N, uint32_t* __restrict__ hi) {
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int G = K >> 7;
  if (idx >= static_cast<int64_t>(N / 16) * G * 64) return;
  const int l = static_cast<int>(idx & 63);
  const int64_t rest = idx >> 6;
  const int t = static_cast<int>(rest / G), g = static_cast<int>(rest % G);
  const int n = 16 * t + (l & 15);
  const int k0 = 128 * g + 32 * (l >> 4);
  const int64_t N32 = N / 32;
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t bit = (static_cast<uint32_t>(qweight_hi[static_cast<int64_t>(k0 + 4 * j + b) * N32 + n / 32]) >> (n & 31)) & 1u;
      word |= bit << (8 * b + j);
    }
  hi[idx] = word;
}

// SZ words of int5 weights: {sc, fl16(sc * (zp - 16))}, zp = low nibble + 16 * fifth bit; the
// product sc * (zp - 16) is exact in fp32 (11 x 5 significand bits), rounded once to f16.
__global__ void pack_sz5_kernel(const int32_t* __restrict__ qzeros, const int32_t* __restrict__ qzeros_hi,
                                const uint16_t* __restrict__ scales, int G, int N, uint32_t* __restrict__ sz) {
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= static_cast<int64_t>(G) * N) return;
  const int g = static_cast<int>(idx / N), n = static_cast<int>(idx % N);
  const uint32_t lo = (static_cast<uint32_t>(qzeros[static_cast<int64_t>(g) * (N / 8) + n / 8]) >> awq_shift(n)) & 0xFu;
  const uint32_t h5 = (static_cast<uint32_t>(qzeros_hi[static_cast<int64_t>(g) * (N / 32) + n / 32]) >> (n & 31)) & 1u;
  const int zp = static_cast<int>(lo + 16 * h5);
  const uint16_t sc = scales[idx];
  const _Float16 zsc = static_cast<_Float16>(f16_to_f32(sc) * static_cast<float>(zp - 16));
  sz[idx] = static_cast<uint32_t>(sc) | (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, zsc)) << 16);
}

// Column factors of the prefill kernel's fold, fp32 [G][N]: 512 sc from the SZ words (exact: a
// power-of-two scaling of an f16 value), so the group loop reads them with no conversion.
__global__ void pack_s9_kernel(const uint32_t* __restrict__ sz, int64_t gn, float* __restrict__ s9) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < gn) s9[i] = f16_to_f32(sz[i]) * 512.0f;
}

// ---------------------------------------------------------------------------------------
// zero-point epilogue operand (load time). The prefill kernel moves the zero-point term
//   Z[m, n] = sum_g (asg * rs)[m, g] * (8 sc + zsc)[g, n]
// out of its group loop ("zero-point epilogue" of the page) and computes it once per tile as
// a bf16 matrix-core product with split operands: ar = a1 + a2 and zz = z1 + z2 (each piece the
// bf16 rounding of what is left), Z ~= a1 z1 + a1 z2 + a2 z1 (relative error ~2^-16).
// K' = 3G is laid out as [a1 | a1 | a2] x [z1 ; z2 ; z1], padded with zeros to whole chunks of 32.
// Layout per 16-column tile t and chunk c (zpe_chunks): 1 KiB, lane l (column 16t + l%16) holds
// the 8 bf16 at k' = 32c + 8(l/16) + 0..7 — the bf16 16x16x32 B operand.

template <bool kW5>
__global__ void pack_zpe_kernel(const uint32_t* __restrict__ sz, int G, int N, u32x4* __restrict__ zpe) {
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int KC = zpe_chunks(G);
  if (idx >= static_cast<int64_t>(N / 16) * KC * 64) return;
  const int l = static_cast<int>(idx & 63);
  const int c = static_cast<int>((idx >> 6) % KC);
  const int t = static_cast<int>((idx >> 6) / KC);
  const int n = 16 * t + (l & 15);
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int kp = 32 * c + 8 * (l >> 4) + e;
    uint32_t v = 0;
    if (kp < 3 * G) {
      const int piece = kp / G, g = kp % G;
      const float2 f = sz_factors<kW5>(sz[static_cast<size_t>(g) * N + n]);
      const uint32_t z1 = f32_to_bf16(f.y);
      v = (piece == 1) ? f32_to_bf16(f.y - bf16_to_f32(z1)) : z1;
    }
    h[e] = v;
  }
  zpe[idx] = u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
}

// Activation side of the zero-point epilogue, built per GEMM call into the workspace:
// for partition p, 16-row tile mt and chunk c, 1 KiB where lane l (row 16mt + l%16) holds the
// 8 bf16 at k' = 32c + 8(l/16) + 0..7 of -[a1 | a1 | a2], ar = asg * rs = a1 + a2 (bf16 pieces).
// kTok: per-token scales, the operand is the plain row-sum (the row scale comes in the epilogue)
// and no transposed copy is written.
template <bool kTok>
__global__ void zpe_act_kernel(const float* __restrict__ ASG, const float* __restrict__ RS, int M, int G,
                               int P, u32x4* __restrict__ zpa, float* __restrict__ asgt) {
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int KC = zpe_chunks(G), MT = (M + 15) / 16;
  if (idx >= static_cast<int64_t>(P) * MT * KC * 64) return;
  const int l = static_cast<int>(idx & 63);
  int64_t rest = idx >> 6;
  const int c = static_cast<int>(rest % KC);
  rest /= KC;
  const int mt = static_cast<int>(rest % MT);
  const int p = static_cast<int>(rest / MT);
  const int row = 16 * mt + (l & 15);
  // every load first (clamped to valid memory), then the arithmetic, then the stores: a store
  // between loads would make each load wait for the previous store
  const size_t rbase = (static_cast<size_t>(p) * M + min(row, M - 1)) * G;
  float av[8], rv[8];
  int piece[8], gg[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int kp = 32 * c + 8 * (l >> 4) + e;
    piece[e] = (kp < 3 * G && row < M) ? kp / G : -1;
    gg[e] = kp < 3 * G ? kp % G : 0;
    av[e] = kTok ? 1.0f : ASG[rbase + gg[e]];
    rv[e] = RS[rbase + gg[e]];
  }
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // ar = fl32(asg rs) and a2 = bf16(ar - a1) round separately, as where the prologue writes
    // these operands: the multiply must not fuse into the subtraction
#pragma clang fp contract(off)
    uint32_t v = 0;
    if (piece[e] >= 0) {
      const float ar = kTok ? rv[e] : av[e] * rv[e];
      const uint32_t a1 = f32_to_bf16(ar);
      v = ((piece[e] == 2) ? f32_to_bf16(ar - bf16_to_f32(a1)) : a1) ^ 0x8000u;   // negated
    }
    h[e] = v;
  }
  if (!kTok) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (piece[e] == 0) asgt[(static_cast<size_t>(p) * G + gg[e]) * M + row] = av[e];   // [P][G][M] copy
  }
  zpa[idx] = u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
}

int zero_point_operands(const float* asg, const float* rs, int M, int G, int P, void* ws, int ws_parts, void* stream) {
  const int64_t zt = static_cast<int64_t>(P) * ((M + 15) / 16) * zpe_chunks(G) * 64;
  float* asgt = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + zpe_act_bytes(M, G, ws_parts));
  return launch_kernel(zpe_act_kernel<false>, dim3(static_cast<unsigned>((zt + 255) / 256)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), asg, rs, M, G, P, static_cast<u32x4*>(ws), asgt);
}

// Per-token scales broadcast to every group, [P][M][G], for the decode kernel.
__global__ void tok_expand_kernel(const float* __restrict__ AS, int PM, int G, float* __restrict__ asg) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < static_cast<int64_t>(PM) * G) asg[i] = AS[i / G];
}

size_t zpe_act_bytes(int M, int G, int P) {
  return static_cast<size_t>(P) * ((M + 15) / 16) * zpe_chunks(G) * 1024;
}

// The group scales transposed to [P][G][M] (f32), so that a tile's scales of one group are
// contiguous for the direct loads.
size_t asgt_bytes(int M, int G, int P) {
  return (static_cast<size_t>(P) * G * M * 4 + 255) / 256 * 256;
}

// ---------------------------------------------------------------------------------------
// decode: M <= 16, a stream of the packed weights. A CU's memory pipeline delivers a bounded
// rate, so the kernel time is set by the CU with the most bytes. The columns are therefore dealt
// out in quarters of a tile (4 columns): one 8-wave workgroup per CU (its ring fills the LDS), each
// taking a contiguous column range of the same number of quarters (gate_up N = 17408 on 256 CUs:
// exactly 68 columns each; ranges differ by at most one quarter in general), inside one
// partition. A range starts and ends anywhere on a 4-column line, so the tiles at its two ends are
// loaded with the lanes of the other columns masked off (each lane owns one column of a tile
// block) and their products for those columns are dropped. Consecutive ranges go to the same
// XCD (workgroups are dispatched to the XCDs round-robin), so a cache line shared by two
// neighbouring ranges is fetched once into that XCD's L2.
// The 8 waves of a workgroup split the groups; each streams its groups through a private LDS ring
// of D slots with direct LDS loads: a slot holds one group's tile blocks, the activation rows, the
// SZ words and the rows' asg/rs values. Group g+D-1 is requested before group g is computed and an
// explicit vmcnt wait covers exactly group g, so D-1 groups stay in flight. The loads are
// invisible to the compiler, which therefore never inserts waits of its own on them (register
// rings lose their depth to such waits when the allocator copies an in-flight register). The
// waves' partial sums meet in LDS at the end.
constexpr int kDecWaves = 8;
constexpr int kDecMaxNT = 6;                       // tile blocks one range touches
constexpr int kDecMaxQ = 4 * (kDecMaxNT - 1);      // quarters per range at most (80 columns)
constexpr int kDecRingBytes = 20480;               // per wave
constexpr int kDecLds = kDecWaves * kDecRingBytes; // 160 KiB: one workgroup per CU
// MA = activation rows held in a slot (8 when M <= 8, else 16)
template <int NT, int MA, bool kW5>
struct DecodeSlot {
  static constexpr int kSzWords = 16 * NT;
  static constexpr int kSzLoads = (kSzWords + 63) / 64;         // 64 SZ words per load
  static constexpr int kOffA = NT * 1024;                       // [MA rows][128 B]
  static constexpr int kOffSz = kOffA + MA * 128;               // [16 NT] words
  static constexpr int kOffSc = kOffSz + (kSzWords * 4 + 15) / 16 * 16;   // [16] asg, [16] rs
  static constexpr int kOffH = kOffSc + 128;                    // int5: [NT][64 lanes] fifth-bit words
  static constexpr int kBytes = kOffH + (kW5 ? NT * 256 : 0);
  static constexpr int kDepth = kDecRingBytes / kBytes > 16 ? 16 : kDecRingBytes / kBytes;
  static constexpr int kLoads = NT + MA / 8 + kSzLoads + 2 + (kW5 ? NT : 0);   // loads per group
  static_assert(kDepth >= 2 && (kDepth - 1) * kLoads <= 63, "decode ring does not fit vmcnt");
};

// MR = activation rows held per lane that can be live (1 when M == 1, else 4)
template <int NT, int MR, int MA, bool kI8, bool kW5>
__device__ __forceinline__ void decode_body(
    const uint8_t* __restrict__ A, const float* __restrict__ asgp, const float* __restrict__ rsp,
    int M, int K, const u32x4* __restrict__ wpk, const uint32_t* __restrict__ hi,
    const uint32_t* __restrict__ sz, int N, int p, int c0, int c1, uint16_t* __restrict__ y, int64_t ldy,
    uint8_t* smem) {
  using S = DecodeSlot<NT, MA, kW5>;
  constexpr int D = S::kDepth;
  const int G = K >> 7;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform: scalar loop bounds
  const int col = lane & 15, kq = lane >> 4;
  const int tfirst = c0 >> 4, n0 = 16 * tfirst;
  const int g0 = (G * wave) / kDecWaves, g1 = (G * (wave + 1)) / kDecWaves;

  // Sources: a scalar base per group plus a fixed per-lane offset. Weight tile t: every lane owns
  // column n0 + 16t + lane % 16; lanes whose column is outside [c0, c1) load nothing (each tile
  // keeps at least 4 columns, so every load has live lanes in every wave and is counted by
  // vmcnt). Activation rows: lane l loads 16 bytes of row l / 8 (rows past M repeat row M - 1).
  const uint8_t* wbase = reinterpret_cast<const uint8_t*>(wpk) + static_cast<size_t>(tfirst) * G * 1024;
  const uint32_t woff = 16 * lane;
  bool won[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = n0 + 16 * t + col;
    won[t] = n >= c0 && n < c1;
  }
  const uint8_t* hbase = reinterpret_cast<const uint8_t*>(hi) + static_cast<size_t>(tfirst) * G * 256;
  const uint8_t* abase = A + static_cast<size_t>(p) * M * K;
  const int ar0 = min(lane >> 3, M - 1), ar1 = min((lane >> 3) + 8, M - 1);
  const uint32_t aoff0 = static_cast<uint32_t>(ar0 * K + 16 * (lane & 7));
  const uint32_t aoff1 = static_cast<uint32_t>(ar1 * K + 16 * (lane & 7));
  const uint8_t* zbase = reinterpret_cast<const uint8_t*>(sz + n0);
  const uint32_t zoff = 4 * lane;
  const int srow = lane & 15;
  const bool as_on = lane < 16 && srow < M, rs_on = lane >= 16 && lane < 32 && srow < M;
  const uint32_t soff = static_cast<uint32_t>(4 * (srow < M ? srow : 0) * G);

  uint8_t* ringp = smem + wave * kDecRingBytes;
  const uint32_t ring = lds_addr(ringp);
  auto issue = [&](int g, int slot) {
    const uint32_t sb = ring + slot * S::kBytes;
    const uint8_t* wg = wbase + static_cast<size_t>(g) * 1024;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (won[t]) lds_dma16_s(wg + static_cast<size_t>(t) * G * 1024, woff, sb + t * 1024);
    if constexpr (kW5) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (won[t]) lds_dma4_s(hbase + (static_cast<size_t>(t) * G + g) * 256, 4 * lane, sb + S::kOffH + t * 256);
    }
    lds_dma16_s(abase + 128 * g, aoff0, sb + S::kOffA);
    if constexpr (MA == 16) lds_dma16_s(abase + 128 * g, aoff1, sb + S::kOffA + 1024);
    const uint8_t* zg = zbase + static_cast<size_t>(g) * N * 4;
#pragma unroll
    for (int j = 0; j < S::kSzLoads; ++j)
      if (lane + 64 * j < S::kSzWords) lds_dma4_s(zg + 256 * j, zoff, sb + S::kOffSz + j * 256);
    if (as_on) lds_dma4_s(asgp + g, soff, sb + S::kOffSc);
    if (rs_on) lds_dma4_s(rsp + g, soff, sb + S::kOffSc);
  };
  const int ng = g1 - g0;
  for (int i = 0; i < D - 1 && i < ng; ++i) issue(g0 + i, i);

  v4f acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
  // MFMA A operand: lane l takes row l % 16 (folded onto the MA rows held), k 32 (l / 16) .. + 31
  const int arow = (lane & 15) & (MA - 1);
  int slot = 0;
  for (int g = g0; g < g1; ++g) {
    if (g + D - 1 < g1) {
      issue(g + D - 1, slot == 0 ? D - 1 : slot - 1);
      wait_vm<(D - 1) * S::kLoads>();   // group g has landed; D-1 groups remain in flight
    } else {
      wait_vm<0>();
    }
    const uint8_t* sp = ringp + slot * S::kBytes;
    const u32x4 a0 = *reinterpret_cast<const u32x4*>(sp + S::kOffA + arow * 128 + 32 * kq);
    const u32x4 a1 = *reinterpret_cast<const u32x4*>(sp + S::kOffA + arow * 128 + 32 * kq + 16);
    const v8i av = v8i{(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
    const v4f as = *reinterpret_cast<const v4f*>(sp + S::kOffSc + 16 * kq);
    const v4f rs = *reinterpret_cast<const v4f*>(sp + S::kOffSc + 64 + 16 * kq);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const u32x4 bw = *reinterpret_cast<const u32x4*>(sp + t * 1024 + 16 * lane);
      float2 f = sz_factors<kW5>(*reinterpret_cast<const uint32_t*>(sp + S::kOffSz + 4 * (16 * t + col)));
      if constexpr (kI8) f.x *= 0x1p-9f;   // integer products carry no 2^-9
      const uint32_t hw = kW5 ? *reinterpret_cast<const uint32_t*>(sp + S::kOffH + t * 256 + 4 * lane) : 0u;
      const v4f T = group_product<kI8>(av, weight_operand<kW5>(bw, hw));
#pragma unroll
      for (int i = 0; i < MR; ++i) acc[t][i] += as[i] * (f.x * T[i] - f.y * rs[i]);
    }
    slot = slot + 1 == D ? 0 : slot + 1;
  }

  __syncthreads();   // every ring has drained: the reduction reuses that LDS
  float* sred = reinterpret_cast<float*>(smem);   // [waves][16 rows][16 NT]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < MR; ++i) sred[(wave * 16 + 4 * kq + i) * 16 * NT + 16 * t + col] = acc[t][i];
  __syncthreads();
  // bf16 pairs of columns (c0, c1 and ldy even: 4-byte stores)
  const int half = (c1 - c0) >> 1, pairs = M * half;
  for (int idx = tid; idx < pairs; idx += 64 * kDecWaves) {
    const int m = idx / half, c = c0 - n0 + 2 * (idx % half);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWaves; ++w) {
      s0 += sred[(w * 16 + m) * 16 * NT + c];
      s1 += sred[(w * 16 + m) * 16 * NT + c + 1];
    }
    *reinterpret_cast<uint32_t*>(y + static_cast<size_t>(m) * ldy + n0 + c) = bf16x2_rn(s0, s1);
  }
}

template <bool kI8, bool kW5>
__global__ __launch_bounds__(64 * kDecWaves, 1) void gemm_decode_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ ASG, const float* __restrict__ RS,
    int M, int K, const u32x4* __restrict__ wpk, const uint32_t* __restrict__ hi,
    const uint32_t* __restrict__ sz, int N, DecodeMap map, uint16_t* __restrict__ y, int64_t ldy) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kDecLds];
  const int b = blockIdx.x, W = map.wg0[3];
  const int r = map.xcd ? (b % 8) * (W / 8) + b / 8 : b;
  const int q = (r >= map.wg0[1]) + (r >= map.wg0[2]);          // partition
  const int nwq = map.wg0[q + 1] - map.wg0[q], rq = r - map.wg0[q];
  const int base = map.nq[q] / nwq, extra = map.nq[q] % nwq;
  const int cnt = base + (rq < extra);
  const int c0 = map.c0[q] + 4 * (rq * base + (rq < extra ? rq : extra));
  const int c1 = c0 + 4 * cnt;
  const int nt = ((c1 - 1) >> 4) - (c0 >> 4) + 1;
  const size_t MG = static_cast<size_t>(M) * (K >> 7);
  const float* asgp = ASG + q * MG;
  const float* rsp = RS + q * MG;
#define PQ_DECODE_CASE(n)                                                                                           \
  case n:                                                                                                           \
    if (M == 1) decode_body<n, 1, 8, kI8, kW5>(A, asgp, rsp, M, K, wpk, hi, sz, N, q, c0, c1, y, ldy, smem);         \
    else if (M <= 8) decode_body<n, 4, 8, kI8, kW5>(A, asgp, rsp, M, K, wpk, hi, sz, N, q, c0, c1, y, ldy, smem);    \
    else decode_body<n, 4, 16, kI8, kW5>(A, asgp, rsp, M, K, wpk, hi, sz, N, q, c0, c1, y, ldy, smem);               \
    break;
  switch (nt) {
    PQ_DECODE_CASE(1) PQ_DECODE_CASE(2) PQ_DECODE_CASE(3)
    PQ_DECODE_CASE(4) PQ_DECODE_CASE(5) PQ_DECODE_CASE(6)
    default: break;
  }
#undef PQ_DECODE_CASE
}

template <bool kTok, bool kI8, bool kW5>
__global__ __launch_bounds__(512, 1) void gemm_prefill_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ ASGT, int M, int K,
    const u32x4* __restrict__ wpk, const uint32_t* __restrict__ hi, const u32x4* __restrict__ zpe,
    const u32x4* __restrict__ zpa, const float* __restrict__ s9img, int N, int pb1, int pb2,
    uint16_t* __restrict__ y, int64_t ldy, PrefillMap map, bool vec16) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kPfLds];
  const int b = blockIdx.x;
  const int bm = map.shape == kPfWide ? 256 : 128, bn = map.shape == kPfNarrow ? 128 : 256;
  const bool piece = b >= map.full;
  const int big = piece ? map.full + (b - map.full) / map.split : b;
  const int r = piece ? (b - map.full) % map.split : 0;
  const int t = xcd_tile(big, map.ntiles);
  int trow, tcol;
  tile_rc(t, map.tiles_m, map.tiles_n, trow, tcol);
  int m0 = trow * bm, n0 = tcol * bn;
  const int split = piece ? map.split : 1;
  // piece r of a whole tile: split 2 -> 2 row halves; 4 -> 2 x 2 quarters; 8 -> 4 row x 2 column
  if (split == 2) m0 += (bm / 2) * r;
  else if (split == 4) { m0 += 128 * (r & 1); n0 += 128 * (r >> 1); }
  else if (split == 8) { m0 += 64 * (r & 3); n0 += 128 * (r >> 2); }
  if (m0 >= M || n0 >= N) return;   // a piece wholly past the matrix
  const int p = (n0 >= pb1) + (n0 >= pb2);
  if constexpr (kW5) {
    if (map.shape == kPfWide) {
      // the fifth-bit planes make a 256x256 stage 54 KiB: a ring of two (one group loaded ahead)
      if (split == 1) prefill_tile<256, 256, 2, 4, kTok, kI8, true, 2>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
      else if (split == 2) prefill_tile<128, 256, 2, 4, kTok, kI8, true>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
      else if (split == 4) prefill_tile<128, 128, 2, 4, kTok, kI8, true>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
      else prefill_tile<64, 128, 2, 4, kTok, kI8, true>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
      return;
    }
    if (split == 1) prefill_tile<128, 128, 2, 4, kTok, kI8, true>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
    else prefill_tile<64, 128, 2, 4, kTok, kI8, true>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
  } else if (map.shape == kPfWide) {
    if (split == 1) prefill_tile<256, 256, 2, 4, kTok, kI8, false>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
    else if (split == 2) prefill_tile<128, 256, 2, 4, kTok, kI8, false>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
    else if (split == 4) prefill_tile<128, 128, 2, 4, kTok, kI8, false>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
    else prefill_tile<64, 128, 2, 4, kTok, kI8, false>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
  } else {
    if (split == 1) prefill_tile<128, 128, 2, 4, kTok, kI8, false>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
    else prefill_tile<64, 128, 2, 4, kTok, kI8, false>(A, ASGT, M, K, wpk, hi, zpe, zpa, s9img, N, p, m0, n0, y, ldy, vec16, smem);
  }
}

}  // namespace pq

extern "C" {

size_t pq_packed_weight_bytes(int K, int N) {
  if (K <= 0 || N <= 0 || K % PQ_GROUP || N % 16) return 0;
  const size_t codes = static_cast<size_t>(K) * static_cast<size_t>(N) / 2;
  const size_t zpe = static_cast<size_t>(N / 16) * pq::zpe_chunks(K / PQ_GROUP) * 1024;
  return codes + zpe + static_cast<size_t>(K / PQ_GROUP) * N * 4;
}

int pq_pack_weights(const int32_t* qweight_d, const int32_t* qzeros_d, const uint16_t* scales_d,
                    int K, int N, void* wpk_d, uint16_t* sz_d, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  if (K <= 0 || K % PQ_GROUP || K > (1 << 24)) return set_error(PQ_ERR_SHAPE, "pq_pack_weights: K=%d must be a positive multiple of 128", K);
  if (N <= 0 || N % 16 || N > (1 << 24)) return set_error(PQ_ERR_SHAPE, "pq_pack_weights: N=%d must be a positive multiple of 16", N);
  if (!qweight_d || !qzeros_d || !scales_d || !wpk_d || !sz_d) return set_error(PQ_ERR_NULL, "pq_pack_weights: NULL pointer");
  if (!aligned(qweight_d, 4) || !aligned(qzeros_d, 4) || !aligned(scales_d, 2) || !aligned(wpk_d, 16) || !aligned(sz_d, 4))
    return set_error(PQ_ERR_ALIGN, "pq_pack_weights: misaligned pointer");
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int G = K / PQ_GROUP;
  const int64_t words = static_cast<int64_t>(K) * N / 8;
  hipError_t launched = launch_kernel(pack_weights_kernel, dim3(static_cast<unsigned>((words + 255) / 256)), dim3(256), 0, s,
                                      qweight_d, K, N, static_cast<uint32_t*>(wpk_d));
  const int64_t gn = static_cast<int64_t>(G) * N;
  if (launched == hipSuccess)
    launched = launch_kernel(pack_sz_kernel, dim3(static_cast<unsigned>((gn + 255) / 256)), dim3(256), 0, s,
                             qzeros_d, scales_d, G, N, reinterpret_cast<uint32_t*>(sz_d));
  const int64_t zl = static_cast<int64_t>(N / 16) * zpe_chunks(G) * 64;
  u32x4* zpe = reinterpret_cast<u32x4*>(static_cast<uint8_t*>(wpk_d) + static_cast<size_t>(K) * N / 2);
  auto zk = pack_zpe_kernel<false>;
  if (launched == hipSuccess)
    launched = launch_kernel(zk, dim3(static_cast<unsigned>((zl + 255) / 256)), dim3(256), 0, s,
                             reinterpret_cast<const uint32_t*>(sz_d), G, N, zpe);
  float* s9 = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(zpe) + static_cast<size_t>(N / 16) * zpe_chunks(G) * 1024);
  if (launched == hipSuccess)
    launched = launch_kernel(pack_s9_kernel, dim3(static_cast<unsigned>((gn + 255) / 256)), dim3(256), 0, s,
                             reinterpret_cast<const uint32_t*>(sz_d), gn, s9);
  return launch_status("pq_pack_weights", launched);
}

size_t pq_packed_weight5_bytes(int K, int N) {
  if (K <= 0 || N <= 0 || K % PQ_GROUP || N % 32) return 0;
  const size_t kn = static_cast<size_t>(K) * static_cast<size_t>(N);
  const size_t zpe = static_cast<size_t>(N / 16) * pq::zpe_chunks(K / PQ_GROUP) * 1024;
  return kn / 2 + kn / 8 + zpe + static_cast<size_t>(K / PQ_GROUP) * N * 4;
}

int pq_pack_weights5(const int32_t* qweight_d, const int32_t* qweight_hi_d, const int32_t* qzeros_d,
                     const int32_t* qzeros_hi_d, const uint16_t* scales_d, int K, int N, void* wpk_d,
                     uint16_t* sz_d, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  if (K <= 0 || K % PQ_GROUP || K > (1 << 24)) return set_error(PQ_ERR_SHAPE, "pq_pack_weights5: K=%d must be a positive multiple of 128", K);
  if (N <= 0 || N % 32 || N > (1 << 24)) return set_error(PQ_ERR_SHAPE, "pq_pack_weights5: N=%d must be a positive multiple of 32", N);
  if (!qweight_d || !qweight_hi_d || !qzeros_d || !qzeros_hi_d || !scales_d || !wpk_d || !sz_d)
    return set_error(PQ_ERR_NULL, "pq_pack_weights5: NULL pointer");
  if (!aligned(qweight_d, 4) || !aligned(qweight_hi_d, 4) || !aligned(qzeros_d, 4) || !aligned(qzeros_hi_d, 4) ||
      !aligned(scales_d, 2) || !aligned(wpk_d, 16) || !aligned(sz_d, 4))
    return set_error(PQ_ERR_ALIGN, "pq_pack_weights5: misaligned pointer");
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int G = K / PQ_GROUP;
  const int64_t words = static_cast<int64_t>(K) * N / 8;
  uint8_t* wb = static_cast<uint8_t*>(wpk_d);
  hipError_t launched = launch_kernel(pack_weights_kernel, dim3(static_cast<unsigned>((words + 255) / 256)), dim3(256), 0, s,
                                      qweight_d, K, N, reinterpret_cast<uint32_t*>(wb));
  const int64_t hw = static_cast<int64_t>(N / 16) * G * 64;
  if (launched == hipSuccess)
    launched = launch_kernel(pack_hi_kernel, dim3(static_cast<unsigned>((hw + 255) / 256)), dim3(256), 0, s,
                             qweight_hi_d, K, N, reinterpret_cast<uint32_t*>(wb + static_cast<size_t>(K) * N / 2));
  const int64_t gn = static_cast<int64_t>(G) * N;
  if (launched == hipSuccess)
    launched = launch_kernel(pack_sz5_kernel, dim3(static_cast<unsigned>((gn + 255) / 256)), dim3(256), 0, s,
                             qzeros_d, qzeros_hi_d, scales_d, G, N, reinterpret_cast<uint32_t*>(sz_d));
  const int64_t zl = static_cast<int64_t>(N / 16) * zpe_chunks(G) * 64;
  u32x4* zpe = reinterpret_cast<u32x4*>(wb + static_cast<size_t>(K) * N / 2 + static_cast<size_t>(K) * N / 8);
  auto zk = pack_zpe_kernel<true>;
  if (launched == hipSuccess)
    launched = launch_kernel(zk, dim3(static_cast<unsigned>((zl + 255) / 256)), dim3(256), 0, s,
                             reinterpret_cast<const uint32_t*>(sz_d), G, N, zpe);
  float* s9 = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(zpe) + static_cast<size_t>(N / 16) * zpe_chunks(G) * 1024);
  if (launched == hipSuccess)
    launched = launch_kernel(pack_s9_kernel, dim3(static_cast<unsigned>((gn + 255) / 256)), dim3(256), 0, s,
                             reinterpret_cast<const uint32_t*>(sz_d), gn, s9);
  return launch_status("pq_pack_weights5", launched);
}

size_t pq_gemm_workspace_bytes(int M, int N, int K) {
  (void)N;
  if (M <= 16 || K <= 0 || K % PQ_GROUP) return 0;     // the decode kernel needs none
  return pq::zpe_act_bytes(M, K / PQ_GROUP, PQ_MAX_PARTITIONS) + pq::asgt_bytes(M, K / PQ_GROUP, PQ_MAX_PARTITIONS);
}

size_t pq_gemm_tok_workspace_bytes(int M, int N, int K) {
  (void)N;
  if (M <= 0 || K <= 0 || K % PQ_GROUP) return 0;
  const int G = K / PQ_GROUP;
  if (M <= 16) return (static_cast<size_t>(PQ_MAX_PARTITIONS) * M * G * 4 + 255) / 256 * 256;   // scales per group
  return pq::zpe_act_bytes(M, G, PQ_MAX_PARTITIONS);
}

}  // extern "C"

namespace pq {

// The GEMM behind pq_gemm (kTok = false: a_scale = ASG [P, M, G]), pq_gemm_tok (kTok = true:
// a_scale = AS [P, M]), pq_gemm_i8 (kI8) and pq_gemm5 (kW5: int5 packed weights); validation is
// the caller's.
// ws_parts: the partition count the workspace layout is sized for (the transposed scales follow
// the zero-point operand of that many partitions).
// prepared: the workspace already holds those operands (pq_rotate_quant_for_gemm wrote them).
template <bool kTok, bool kI8, bool kW5 = false>
static int gemm_launch(const char* what, const uint8_t* a_d, const float* a_scale, const float* rs_d, int M, int K,
                       int P, const void* wpk_d, const uint16_t* sz_d, int N, int pb1, int pb2, uint16_t* y_d,
                       int64_t ldy, void* ws_d, hipStream_t s, int ws_parts = PQ_MAX_PARTITIONS,
                       bool prepared = false) {
  const int G = K / PQ_GROUP;
  const u32x4* wpk = static_cast<const u32x4*>(wpk_d);
  const uint32_t* sz = reinterpret_cast<const uint32_t*>(sz_d);
  // packed image: codes (K N / 2 bytes), [int5: fifth-bit planes (K N / 8)], zero-point operand
  const uint8_t* wb = static_cast<const uint8_t*>(wpk_d);
  const uint32_t* hi = kW5 ? reinterpret_cast<const uint32_t*>(wb + static_cast<size_t>(K) * N / 2) : nullptr;
  const u32x4* zpe = reinterpret_cast<const u32x4*>(wb + static_cast<size_t>(K) * N / 2 + (kW5 ? static_cast<size_t>(K) * N / 8 : 0));
  const float* s9img = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(zpe) +
                                                      static_cast<size_t>(N / 16) * zpe_chunks(G) * 1024);
  hipError_t launched = hipSuccess;
  if (M <= 16) {
    const float* asg = a_scale;
    if (kTok) {
      // the decode kernel folds per group: give every group the token's scale
      float* ex = static_cast<float*>(ws_d);
      const int64_t n = static_cast<int64_t>(P) * M * G;
      launched = launch_kernel(tok_expand_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s,
                               a_scale, P * M, G, ex);
      asg = ex;
    }
    DecodeMap map;
    decode_map(N, pb1, pb2, cu_count(), kDecMaxQ, &map);
    auto dec = gemm_decode_kernel<kI8, kW5>;
    if (launched == hipSuccess)
      launched = launch_kernel(dec, dim3(map.wg0[3]), dim3(64 * kDecWaves), 0, s,
                               a_d, asg, rs_d, M, K, wpk, hi, sz, N, map, y_d, ldy);
    return launch_status(what, launched);
  }
  // 256x256 tiles (one workgroup per CU) unless a partition boundary is not on
  // a 256-column line
  const bool on256 = (pb1 >= N || pb1 % 256 == 0) && (pb2 >= N || pb2 % 256 == 0);
  const int shape = !on256 ? kPfNarrow : kPfWide;
  const int64_t tiles = static_cast<int64_t>((M + 127) / 128) * ((N + 127) / 128);
  if (tiles * 8 > 0x7FFFFFFF) return set_error(PQ_ERR_SHAPE, "%s: problem too large", what);
  // the prefill kernel addresses a partition's activations with 32-bit lane offsets
  if (static_cast<int64_t>(M) * K > 0x7FFFFFFF || static_cast<int64_t>(M) * (K / PQ_GROUP) * 4 > 0x7FFFFFFF)
    return set_error(PQ_ERR_SHAPE, "%s: M * K too large for one call (split the rows)", what);
  const PrefillMap map = prefill_map(M, N, shape, cu_count());
  const int64_t grid = static_cast<int64_t>(map.full) + static_cast<int64_t>(map.ntiles - map.full) * map.split;
  u32x4* zpa = static_cast<u32x4*>(ws_d);
  float* asgt = kTok ? nullptr
                     : reinterpret_cast<float*>(static_cast<uint8_t*>(ws_d) + zpe_act_bytes(M, G, ws_parts));
  if (!prepared) {
    const int64_t zt = static_cast<int64_t>(P) * ((M + 15) / 16) * zpe_chunks(G) * 64;
    launched = launch_kernel(zpe_act_kernel<kTok>, dim3(static_cast<unsigned>((zt + 255) / 256)), dim3(256), 0, s,
                             a_scale, rs_d, M, G, P, zpa, asgt);
  }
  // 16-byte output stores need a 16-byte aligned y and a row pitch of 8 elements
  const bool vec16 = aligned(y_d, 16) && ldy % 8 == 0;
  auto prefill = gemm_prefill_kernel<kTok, kI8, kW5>;
  if (launched == hipSuccess)
    launched = launch_kernel(prefill, dim3(static_cast<unsigned>(grid)), dim3(64 * kPfWaves), 0, s,
                             a_d, kTok ? a_scale : asgt, M, K, wpk, hi, zpe, zpa, s9img, N, pb1, pb2, y_d, ldy, map, vec16);
  return launch_status(what, launched);
}

// Shared validation of pq_gemm / pq_gemm_tok; returns PQ_OK to go on, 1 for the M == 0 no-op.
static int gemm_check(const char* what, const uint8_t* a_d, const float* scale_d, const float* rs_d, int M, int K,
                      int P, const void* wpk_d, const uint16_t* sz_d, int N, int pb1, int pb2, uint16_t* y_d,
                      int64_t ldy, void* ws_d, size_t ws_bytes, size_t ws_need) {
  if (M < 0) return set_error(PQ_ERR_SHAPE, "%s: M=%d < 0", what, M);
  if (K <= 0 || K % PQ_GROUP || K > (1 << 24)) return set_error(PQ_ERR_SHAPE, "%s: K=%d must be a positive multiple of 128", what, K);
  if (N <= 0 || N % 16 || N > (1 << 24)) return set_error(PQ_ERR_SHAPE, "%s: N=%d must be a positive multiple of 16", what, N);
  if (ldy < N || (ldy & 1)) return set_error(PQ_ERR_SHAPE, "%s: ldy=%lld must be even and >= N=%d", what, static_cast<long long>(ldy), N);
  const int perr = check_partitions(P, pb1, pb2, N);
  if (perr != PQ_OK) return perr;
  if (ws_bytes < ws_need) return set_error(PQ_ERR_WORKSPACE, "%s: workspace too small", what);
  if (M == 0) return 1;
  if (!a_d || !scale_d || !rs_d || !wpk_d || !sz_d || !y_d) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (ws_need && !ws_d) return set_error(PQ_ERR_NULL, "%s: NULL workspace", what);
  if (!aligned(a_d, 16) || !aligned(scale_d, 4) || !aligned(rs_d, 4) || !aligned(wpk_d, 16) || !aligned(sz_d, 4) ||
      !aligned(y_d, 4) || !aligned(ws_d, 16))
    return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  return PQ_OK;
}

}  // namespace pq

extern "C" {

int pq_gemm(const uint8_t* a_d, const float* asg_d, const float* rs_d, int M, int K, int P,
            const void* wpk_d, const uint16_t* sz_d, int N, int pb1, int pb2, uint16_t* y_d,
            int64_t ldy, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const int rc = gemm_check("pq_gemm", a_d, asg_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy, ws_d, ws_bytes,
                            pq_gemm_workspace_bytes(M, N, K));
  if (rc != PQ_OK) return rc == 1 ? PQ_OK : rc;
  return gemm_launch<false, false>("pq_gemm", a_d, asg_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy, ws_d,
                            reinterpret_cast<hipStream_t>(stream));
}

int pq_gemm_prepared(const uint8_t* a_d, const float* asg_d, const float* rs_d, int M, int K, int P,
                     const void* wpk_d, const uint16_t* sz_d, int N, int pb1, int pb2, uint16_t* y_d,
                     int64_t ldy, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const int rc = gemm_check("pq_gemm_prepared", a_d, asg_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy, ws_d,
                            ws_bytes, pq_gemm_workspace_bytes(M, N, K));
  if (rc != PQ_OK) return rc == 1 ? PQ_OK : rc;
  return gemm_launch<false, false>("pq_gemm_prepared", a_d, asg_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy,
                                   ws_d, reinterpret_cast<hipStream_t>(stream), PQ_MAX_PARTITIONS, true);
}

int pq_gemm_tok(const uint8_t* a_d, const float* as_d, const float* rs_d, int M, int K, int P,
                const void* wpk_d, const uint16_t* sz_d, int N, int pb1, int pb2, uint16_t* y_d,
                int64_t ldy, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const int rc = gemm_check("pq_gemm_tok", a_d, as_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy, ws_d,
                            ws_bytes, pq_gemm_tok_workspace_bytes(M, N, K));
  if (rc != PQ_OK) return rc == 1 ? PQ_OK : rc;
  return gemm_launch<true, false>("pq_gemm_tok", a_d, as_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy, ws_d,
                           reinterpret_cast<hipStream_t>(stream));
}

int pq_gemm5(const uint8_t* a_d, const float* asg_d, const float* rs_d, int M, int K, int P,
             const void* wpk5_d, const uint16_t* sz_d, int N, int pb1, int pb2, uint16_t* y_d,
             int64_t ldy, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  if (N % 32) return set_error(PQ_ERR_SHAPE, "pq_gemm5: N=%d must be a multiple of 32", N);
  const int rc = gemm_check("pq_gemm5", a_d, asg_d, rs_d, M, K, P, wpk5_d, sz_d, N, pb1, pb2, y_d, ldy, ws_d, ws_bytes,
                            pq_gemm_workspace_bytes(M, N, K));
  if (rc != PQ_OK) return rc == 1 ? PQ_OK : rc;
  return gemm_launch<false, false, true>("pq_gemm5", a_d, asg_d, rs_d, M, K, P, wpk5_d, sz_d, N, pb1, pb2, y_d, ldy,
                                         ws_d, reinterpret_cast<hipStream_t>(stream));
}

int pq_gemm_i8(const int8_t* a_d, const float* asg_d, const float* rs_d, int M, int K, int P,
               const void* wpk_d, const uint16_t* sz_d, int N, int pb1, int pb2, uint16_t* y_d,
               int64_t ldy, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const uint8_t* a8 = reinterpret_cast<const uint8_t*>(a_d);
  const int rc = gemm_check("pq_gemm_i8", a8, asg_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy, ws_d, ws_bytes,
                            pq_gemm_workspace_bytes(M, N, K));
  if (rc != PQ_OK) return rc == 1 ? PQ_OK : rc;
  return gemm_launch<false, true>("pq_gemm_i8", a8, asg_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy, ws_d,
                                  reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------------------
// pq_gemm_noalloc: pq_gemm for callers that cannot allocate. The prefill kernel's scratch (the
// zero-point operand and the transposed group scales, sized for the call's own P) lives in this
// file-scope device array instead of a caller workspace. The host side never uses the array's
// name as an address: each device's copy is looked up once with hipGetSymbolAddress and that
// pointer is what the kernels get. Every call on a device shares its copy, so calls that overlap
// on one device (several streams, or threads) race on it.
namespace pq {

constexpr size_t kScratchBytes = size_t(16) << 20;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
static std::mutex g_scratch_mu;
static void* g_scratch_ptr[kMaxDevices] = {};

// The current device's copy of `scratch` (looked up on its first use). Returns PQ_OK or an error.
static int scratch_for_current_device(const char* what, void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return set_error(PQ_ERR_DEVICE, "%s: hipGetDevice failed: %s", what, hipGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return set_error(PQ_ERR_DEVICE, "%s: device %d out of range", what, dev);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || !p)
      return set_error(PQ_ERR_DEVICE, "%s: hipGetSymbolAddress(scratch) failed: %s", what, hipGetErrorString(e));
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return PQ_OK;
}

// Scratch bytes pq_gemm_noalloc needs (0 at M <= 16, where the decode kernel uses none).
static size_t noalloc_bytes(int M, int K, int P) {
  if (M <= 16) return 0;
  const int G = K / PQ_GROUP;
  return zpe_act_bytes(M, G, P) + asgt_bytes(M, G, P);
}

}  // namespace pq

extern "C" {

size_t pq_gemm_noalloc_max_scratch_bytes(void) { return pq::kScratchBytes; }

int pq_gemm_noalloc(const uint8_t* a_d, const float* asg_d, const float* rs_d, int M, int K, int P,
                    const void* wpk_d, const uint16_t* sz_d, int N, int pb1, int pb2, uint16_t* y_d,
                    int64_t ldy, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  // the same checks as pq_gemm, with the library's own scratch standing in for the workspace
  const int rc = gemm_check("pq_gemm_noalloc", a_d, asg_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy,
                            nullptr, 0, 0);
  if (rc != PQ_OK) return rc == 1 ? PQ_OK : rc;
  const size_t need = noalloc_bytes(M, K, P);
  if (need > kScratchBytes)
    return set_error(PQ_ERR_SHAPE, "pq_gemm_noalloc: M=%d K=%d P=%d needs %zu scratch bytes, more than the %zu the "
                     "library holds (use pq_gemm with a workspace)", M, K, P, need, kScratchBytes);
  void* ws = nullptr;
  if (need) {
    const int src = scratch_for_current_device("pq_gemm_noalloc", &ws);
    if (src != PQ_OK) return src;
  }
  return gemm_launch<false, false>("pq_gemm_noalloc", a_d, asg_d, rs_d, M, K, P, wpk_d, sz_d, N, pb1, pb2, y_d, ldy,
                                   ws, reinterpret_cast<hipStream_t>(stream), P);
}

}  // extern "C"
