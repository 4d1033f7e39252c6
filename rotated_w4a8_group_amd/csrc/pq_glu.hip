// The gated feed-forward pair (pq_gemm_glu): h = act(x Wg) * (x Wu) in one launch, for the merged
// projection gate | up that pq_pack_weights lays out (N = 2 F columns), from the prologue's e4m3 codes.
// The products, the fold and the zero point are the GEMM's (pq_gemm.hip); what is new is that one
// workgroup takes the gate and the up columns of the same outputs, so that both sums meet in binary32
// registers and neither projection is written to memory, read back or rounded in between. The weights
// need no layout of their own: a column strip is addressed where it lies.
//
// M <= 16, layers of at most one such range per CU: the weight stream bounds it. One 8-wave workgroup per CU takes a
// contiguous range of output columns (an even number, so that every CU streams the same bytes to within 2 of about 34
// columns) and both projections' tiles of that range; the waves split the groups and stream them through private LDS
// rings, as the decode GEMM does, one group ahead of the one that is computed (as many as the ring holds: K=5120,
// F=4352 7.9 against 7.4 us at M=1, 9.1 against 8.5 at M=7 with two rotations; nor do narrow layers, whose slots are
// small, gain by more: K=10112, F=64 7.25 us with one group ahead, 7.65 with three).
// Up to about 128 rows of a wide layer, more of a narrow one, and M <= 16 of a wider one: the same for blocks of rows, both operands
// streamed.
// Above: the prefill tile with its column strips alternating gate and up (pq_prefill.h); the matrix
// cores and the fold bound it, as they do the GEMM.
#include "pq_device.h"
#include "pq_gemm_device.h"
#include "pq_internal.h"
#include "pq_prefill.h"

namespace pq {

// ---------------------------------------------------------------------------------------
// M <= 16
constexpr int kGdWaves = 8;
constexpr int kGdRingBytes = 20480;                  // per wave
constexpr int kGdLds = kGdWaves * kGdRingBytes;

// NT tiles of each projection, MA activation rows held (8 when M <= 8, else 16) of PA partitions
template <int NT, int MA, int PA>
struct GluSlot {
  static constexpr int kOffA = 2 * NT * 1024;                   // [PA][MA rows][128 B]
  static constexpr int kOffSz = kOffA + PA * MA * 128;          // [gate, up][16 NT] words
  static constexpr int kOffSc = kOffSz + 2 * NT * 64;           // [PA][16 asg, 16 rs]
  static constexpr int kBytes = kOffSc + PA * 128;
  static constexpr int kDepth = 2;
  static constexpr int kLoads = 2 * NT + PA * (MA / 8) + 2 + 2 * PA;
  static_assert(kDepth * kBytes <= kGdRingBytes && (kDepth - 1) * kLoads <= 63, "ring");
};

// The most tiles of a projection that a range may touch for its slot to fit the ring twice, and the most
// columns that touch no more wherever an even start lies.
constexpr int glu_max_tiles(int MA, int PA) { return MA * PA == 8 ? 4 : MA * PA == 16 ? 3 : 2; }
constexpr int glu_max_columns(int MA, int PA) { return 16 * (glu_max_tiles(MA, PA) - 1) + 2; }

template <int NT, int MR, int MA, int PA>
__device__ __forceinline__ void glu_decode_body(
    const uint8_t* __restrict__ A, const float* __restrict__ ASG, const float* __restrict__ RS, int M, int K,
    const u32x4* __restrict__ wpk, const uint32_t* __restrict__ sz, int F, int c0, int c1, int act,
    uint16_t* __restrict__ h, int64_t ldh, bool out_bf16, uint8_t* smem) {
  using S = GluSlot<NT, MA, PA>;
  constexpr int D = S::kDepth;
  const int G = K >> 7;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int tfirst = c0 >> 4, n0 = 16 * tfirst;
  const int g0 = (G * wave) / kGdWaves, g1 = (G * (wave + 1)) / kGdWaves;

  // Sources as in the decode GEMM: a scalar base per group and a fixed lane offset; lanes of columns
  // outside [c0, c1) load no codes (every tile keeps at least 2 columns, so every load is issued).
  const uint8_t* wbase = reinterpret_cast<const uint8_t*>(wpk) + static_cast<size_t>(tfirst) * G * 1024;
  const size_t up = static_cast<size_t>(F / 16) * G * 1024;     // from a gate tile to its up tile
  bool won[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = n0 + 16 * t + col;
    won[t] = n >= c0 && n < c1;
  }
  const int ar0 = min(lane >> 3, M - 1), ar1 = min((lane >> 3) + 8, M - 1);
  const uint32_t aoff0 = static_cast<uint32_t>(ar0 * K + 16 * (lane & 7));
  const uint32_t aoff1 = static_cast<uint32_t>(ar1 * K + 16 * (lane & 7));
  const size_t MG = static_cast<size_t>(M) * G;
  const int srow = lane & 15;
  const bool as_on = lane < 16 && srow < M, rs_on = lane >= 16 && lane < 32 && srow < M;
  const uint32_t soff = static_cast<uint32_t>(4 * (srow < M ? srow : 0) * G);

  uint8_t* ringp = smem + wave * kGdRingBytes;
  const uint32_t ring = lds_addr(ringp);
  auto issue = [&](int g, int slot) {
    const uint32_t sb = ring + slot * S::kBytes;
    const uint8_t* wg = wbase + static_cast<size_t>(g) * 1024;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (won[t]) {
        lds_dma16_s(wg + static_cast<size_t>(t) * G * 1024, 16 * lane, sb + t * 1024);
        lds_dma16_s(wg + up + static_cast<size_t>(t) * G * 1024, 16 * lane, sb + (NT + t) * 1024);
      }
    const uint32_t* zg = sz + static_cast<size_t>(g) * 2 * F + n0;
    if (lane < 16 * NT) {
      lds_dma4_s(zg, 4 * lane, sb + S::kOffSz);
      lds_dma4_s(zg + F, 4 * lane, sb + S::kOffSz + NT * 64);
    }
#pragma unroll
    for (int p = 0; p < PA; ++p) {
      const uint8_t* ag = A + static_cast<size_t>(p) * M * K + 128 * static_cast<size_t>(g);
      lds_dma16_s(ag, aoff0, sb + S::kOffA + p * MA * 128);
      if constexpr (MA == 16) lds_dma16_s(ag, aoff1, sb + S::kOffA + p * MA * 128 + 1024);
      if (as_on) lds_dma4_s(ASG + p * MG + g, soff, sb + S::kOffSc + p * 128);
      if (rs_on) lds_dma4_s(RS + p * MG + g, soff, sb + S::kOffSc + p * 128);
    }
  };
  const int ng = g1 - g0;
  for (int i = 0; i < D - 1 && i < ng; ++i) issue(g0 + i, i);

  v4f acc[2][NT];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[s][t] = v4f{0.f, 0.f, 0.f, 0.f};
  const int arow = (lane & 15) & (MA - 1);
  int slot = 0;
  for (int g = g0; g < g1; ++g) {
    if (g + D - 1 < g1) {
      wait_lds_reads();   // group g - 1's, from the slot that is filled now
      issue(g + D - 1, slot == 0 ? D - 1 : slot - 1);
      wait_vm<(D - 1) * S::kLoads>();   // group g has landed; D - 1 groups remain in flight
    } else {
      wait_vm<0>();
    }
    const uint8_t* sp = ringp + slot * S::kBytes;
    v8i av[PA];
    v4f as[PA], rs[PA];
#pragma unroll
    for (int p = 0; p < PA; ++p) {
      const uint8_t* ap = sp + S::kOffA + p * MA * 128 + arow * 128 + 32 * kq;
      const u32x4 a0 = *reinterpret_cast<const u32x4*>(ap);
      const u32x4 a1 = *reinterpret_cast<const u32x4*>(ap + 16);
      av[p] = v8i{(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
      as[p] = *reinterpret_cast<const v4f*>(sp + S::kOffSc + p * 128 + 16 * kq);
      rs[p] = *reinterpret_cast<const v4f*>(sp + S::kOffSc + p * 128 + 64 + 16 * kq);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int p = PA == 1 ? 0 : s;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const u32x4 bw = *reinterpret_cast<const u32x4*>(sp + (s * NT + t) * 1024 + 16 * lane);
        const float2 f = sz_factors<false>(*reinterpret_cast<const uint32_t*>(sp + S::kOffSz + s * NT * 64 + 4 * (16 * t + col)));
        const v4f T = mfma_fp8(av[p], unpack_codes(bw));
#pragma unroll
        for (int i = 0; i < MR; ++i) acc[s][t][i] += as[p][i] * (f.x * T[i] - f.y * rs[p][i]);
      }
    }
    slot = slot + 1 == D ? 0 : slot + 1;
  }

  __syncthreads();   // every ring has drained: the reduction reuses that LDS
  constexpr int W = 16 * NT, R = 2 * W + 4;   // the 4 extra words put every fourth row a quarter of the banks further
  float* sred = reinterpret_cast<float*>(smem);   // [waves][16 rows][gate, up][16 NT], rows padded
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < MR; ++i) sred[(wave * 16 + 4 * kq + i) * R + s * W + 16 * t + col] = acc[s][t][i];
  __syncthreads();
  const int half = (c1 - c0) >> 1, pairs = M * half;   // c0, c1 and ldh even: 4-byte stores
  for (int idx = tid; idx < pairs; idx += 64 * kGdWaves) {
    const int m = idx / half, c = c0 - n0 + 2 * (idx % half);
    float v[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int w = 0; w < kGdWaves; ++w)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const float2 q = *reinterpret_cast<const float2*>(sred + (w * 16 + m) * R + s * W + c);
        v[s][0] += q.x;
        v[s][1] += q.y;
      }
    const float h0 = glu_value(v[0][0], v[1][0], act), h1 = glu_value(v[0][1], v[1][1], act);
    *reinterpret_cast<uint32_t*>(h + static_cast<size_t>(m) * ldh + n0 + c) = out_bf16 ? bf16x2_rn(h0, h1) : f16x2_rn(h0, h1);
  }
}

// F / 2 column pairs dealt out evenly over gridDim.x ranges; consecutive ranges go to one XCD, so that a line
// shared by neighbours is fetched once into its L2.
template <int MR, int MA, int PA>
__global__ __launch_bounds__(64 * kGdWaves, 1) void glu_decode_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ ASG, const float* __restrict__ RS, int M, int K,
    const u32x4* __restrict__ wpk, const uint32_t* __restrict__ sz, int F, int act, uint16_t* __restrict__ h, int64_t ldh,
    int out_bf16) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kGdLds];
  const int b = blockIdx.x, W = gridDim.x;
  const int r = W % 8 == 0 ? (b % 8) * (W / 8) + b / 8 : b;
  const int base = (F / 2) / W, extra = (F / 2) % W;
  const int c0 = 2 * (r * base + min(r, extra)), c1 = c0 + 2 * (base + (r < extra));
  const int nt = ((c1 - 1) >> 4) - (c0 >> 4) + 1;
  constexpr int kMax = glu_max_tiles(MA, PA);
  if (nt == 1) glu_decode_body<1, MR, MA, PA>(A, ASG, RS, M, K, wpk, sz, F, c0, c1, act, h, ldh, out_bf16 != 0, smem);
  else if (nt == 2) glu_decode_body<2, MR, MA, PA>(A, ASG, RS, M, K, wpk, sz, F, c0, c1, act, h, ldh, out_bf16 != 0, smem);
  if constexpr (kMax >= 3)
    if (nt == 3) glu_decode_body<3, MR, MA, PA>(A, ASG, RS, M, K, wpk, sz, F, c0, c1, act, h, ldh, out_bf16 != 0, smem);
  if constexpr (kMax >= 4)
    if (nt == 4) glu_decode_body<4, MR, MA, PA>(A, ASG, RS, M, K, wpk, sz, F, c0, c1, act, h, ldh, out_bf16 != 0, smem);
}

// ---------------------------------------------------------------------------------------
// From 17 rows on, while the weights or the launch are still most of the work: the same streaming scheme for
// blocks of 16 MF rows. The W waves of a workgroup split the groups; a wave's LDS slot holds one group's tiles of
// both projections, the block's activation rows (16-byte chunks swizzled as in the prefill tile), SZ words
// and the rows' scales and sums, so the zero point is folded in the loop and no pass runs before. Where only one
// slot fits, a wave loads a group, waits for it and computes it: the other waves of its SIMD compute meanwhile. (Four waves
// with two slots each, which load one group ahead, take 21.9 us where eight with one take 19.4, at M=64, K=5120,
// F=8704: a wave is held up while its loads are accepted, and then its SIMD is idle.) The sums meet in LDS in
// an order that the shape fixes.
constexpr int kGmColumns = 50;    // a range's columns at most: 4 tiles from any even start

template <int NT, int MF, int PA, int W>
struct GluMidSlot {
  static constexpr int kOffA = 2 * NT * 1024;                   // [PA][16 MF rows][8 chunks of 16 B]
  static constexpr int kOffSz = kOffA + PA * MF * 2048;         // [gate, up][16 NT] words
  static constexpr int kOffSc = kOffSz + 2 * NT * 64;           // [PA][16 MF asg, 16 MF rs]
  static constexpr int kBytes = kOffSc + PA * MF * 128;
  static constexpr int kRed = (W / 2) * 16 * MF * (2 * 16 * NT + 4) * 4;   // the sums of half the waves reuse the slots
  // Two slots, one group ahead, where they fit: M=17, K=5120, F=2048 6.7 against 7.3 us, M=18, K=7808, F=720 8.6 / 9.2,
  // M=33, K=10240, F=1024 13.7 / 14.4, M=40, K=5120, F=2048 9.4 / 9.2.
  static constexpr int kDepth = 2 * W * kBytes <= (W == 8 ? 163840 : 81920) ? 2 : 1;
  static constexpr int kLoads = 2 * NT + PA * 2 * MF + 2 + 2 * PA;
  static constexpr int kLds = kDepth * W * kBytes > kRed ? kDepth * W * kBytes : kRed;
  static_assert(kLds <= 163840, "LDS");
};

template <int NT, int MF, int PA, int W>
__device__ __forceinline__ void glu_mid_body(
    const uint8_t* __restrict__ A, const float* __restrict__ ASG, const float* __restrict__ RS, int M, int K,
    const u32x4* __restrict__ wpk, const uint32_t* __restrict__ sz, int F, int m0, int c0, int c1, int act,
    uint16_t* __restrict__ h, int64_t ldh, bool out_bf16, uint8_t* smem) {
  using S = GluMidSlot<NT, MF, PA, W>;
  const int G = K >> 7;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int tfirst = c0 >> 4, n0 = 16 * tfirst;
  const int g0 = (G * wave) / W, g1 = (G * (wave + 1)) / W;

  const uint8_t* wbase = reinterpret_cast<const uint8_t*>(wpk) + static_cast<size_t>(tfirst) * G * 1024;
  const size_t up = static_cast<size_t>(F / 16) * G * 1024;
  bool won[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = n0 + 16 * t + col;
    won[t] = n >= c0 && n < c1;
  }
  // lane l of activation load j: row 8 j + l / 8 of the block (rows past M repeat row M - 1)
  uint32_t aoff[2 * MF];
#pragma unroll
  for (int j = 0; j < 2 * MF; ++j) {
    const int r = 8 * j + (lane >> 3);
    aoff[j] = static_cast<uint32_t>(min(m0 + r, M - 1) * K + 16 * ((lane & 7) ^ (r & 7) ^ ((r >> 3) & 1)));
  }
  const size_t MG = static_cast<size_t>(M) * G;
  const uint32_t soff = static_cast<uint32_t>(min(m0 + lane, M - 1) * 4 * G);

  constexpr int D = S::kDepth;
  const uint8_t* ringp = smem + wave * D * S::kBytes;
  const uint32_t ring = lds_addr(ringp);
  auto issue = [&](int g, int slot) {
    const uint32_t sb = ring + slot * S::kBytes;
    const uint8_t* wg = wbase + static_cast<size_t>(g) * 1024;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (won[t]) {
        lds_dma16_s(scalar_addr(wg + static_cast<size_t>(t) * G * 1024), 16 * lane, sb + t * 1024);
        lds_dma16_s(scalar_addr(wg + up + static_cast<size_t>(t) * G * 1024), 16 * lane, sb + (NT + t) * 1024);
      }
    const uint32_t* zg = sz + static_cast<size_t>(g) * 2 * F + n0;
    if (lane < 16 * NT) {
      lds_dma4_s(scalar_addr(zg), 4 * lane, sb + S::kOffSz);
      lds_dma4_s(scalar_addr(zg + F), 4 * lane, sb + S::kOffSz + NT * 64);
    }
#pragma unroll
    for (int p = 0; p < PA; ++p) {
      const uint8_t* ag = A + static_cast<size_t>(p) * M * K + 128 * static_cast<size_t>(g);
#pragma unroll
      for (int j = 0; j < 2 * MF; ++j) lds_dma16_s(scalar_addr(ag), aoff[j], sb + S::kOffA + (p * 2 * MF + j) * 1024);
      if (lane < 16 * MF) {
        lds_dma4_s(scalar_addr(ASG + p * MG + g), soff, sb + S::kOffSc + p * MF * 128);
        lds_dma4_s(scalar_addr(RS + p * MG + g), soff, sb + S::kOffSc + p * MF * 128 + MF * 64);
      }
    }
  };
  v4f acc[2][NT][MF];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int f = 0; f < MF; ++f) acc[s][t][f] = v4f{0.f, 0.f, 0.f, 0.f};
  const int sw = (col & 7) ^ (col >> 3);
  const int aread0 = col * 128 + 16 * ((2 * kq) ^ sw), aread1 = col * 128 + 16 * ((2 * kq + 1) ^ sw);
  if (D == 2 && g0 < g1) issue(g0, 0);
  int slot = 0;
  for (int g = g0; g < g1; ++g) {
    if (D == 1) {
      wait_lds_reads();   // the last group's, from the slot that is filled now
      issue(g, 0);
      wait_vm<0>();
    } else if (g + 1 < g1) {
      wait_lds_reads();
      issue(g + 1, slot ^ 1);
      wait_vm<S::kLoads>();
    } else {
      wait_vm<0>();
    }
    const uint8_t* sp = ringp + slot * S::kBytes;
    if (D == 2) slot ^= 1;
    v8i bw[2][NT];
    float2 fz[2][NT];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        bw[s][t] = unpack_codes(*reinterpret_cast<const u32x4*>(sp + (s * NT + t) * 1024 + 16 * lane));
        fz[s][t] = sz_factors<false>(*reinterpret_cast<const uint32_t*>(sp + S::kOffSz + s * NT * 64 + 4 * (16 * t + col)));
      }
#pragma unroll
    for (int p = 0; p < PA; ++p) {
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const uint8_t* ap = sp + S::kOffA + (p * MF + f) * 2048;
        const u32x4 a0 = *reinterpret_cast<const u32x4*>(ap + aread0);
        const u32x4 a1 = *reinterpret_cast<const u32x4*>(ap + aread1);
        const v8i av = v8i{(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
        const v4f as = *reinterpret_cast<const v4f*>(sp + S::kOffSc + p * MF * 128 + 64 * f + 16 * kq);
        const v4f rs = *reinterpret_cast<const v4f*>(sp + S::kOffSc + p * MF * 128 + MF * 64 + 64 * f + 16 * kq);
#pragma unroll
        for (int s = PA == 1 ? 0 : p; s < (PA == 1 ? 2 : p + 1); ++s)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const v4f T = mfma_fp8(av, bw[s][t]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[s][t][f][i] += as[i] * (fz[s][t].x * T[i] - fz[s][t].y * rs[i]);
          }
      }
    }
  }

  __syncthreads();   // every slot is free: the sums reuse that LDS
  constexpr int C = 16 * NT, R = 2 * C + 4;   // a row's sums; the 4 extra words put every fourth row a quarter of the banks further
  float* sred = reinterpret_cast<float*>(smem);
  // the upper half of the waves hand their sums to the lower half, which add them in registers
  if (wave >= W / 2) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int f = 0; f < MF; ++f)
          *reinterpret_cast<v4f*>(sred + ((((wave - W / 2) * 2 + s) * NT + t) * MF + f) * 256 + 4 * lane) = acc[s][t][f];
  }
  __syncthreads();
  if (wave < W / 2) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int f = 0; f < MF; ++f)
          acc[s][t][f] += *reinterpret_cast<const v4f*>(sred + (((wave * 2 + s) * NT + t) * MF + f) * 256 + 4 * lane);
  }
  __syncthreads();
  if (wave < W / 2) {   // [W / 2 waves][16 MF rows][gate, up][16 NT]
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int f = 0; f < MF; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i) sred[(wave * 16 * MF + 16 * f + 4 * kq + i) * R + s * C + 16 * t + col] = acc[s][t][f][i];
  }
  __syncthreads();
  const int half = (c1 - c0) >> 1, pairs = min(16 * MF, M - m0) * half;
  for (int idx = tid; idx < pairs; idx += 64 * W) {
    const int m = idx / half, c = c0 - n0 + 2 * (idx % half);
    float v[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int w = 0; w < W / 2; ++w)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const float2 q = *reinterpret_cast<const float2*>(sred + (w * 16 * MF + m) * R + s * C + c);
        v[s][0] += q.x;
        v[s][1] += q.y;
      }
    const float h0 = glu_value(v[0][0], v[1][0], act), h1 = glu_value(v[0][1], v[1][1], act);
    *reinterpret_cast<uint32_t*>(h + static_cast<size_t>(m0 + m) * ldh + n0 + c) = out_bf16 ? bf16x2_rn(h0, h1) : f16x2_rn(h0, h1);
  }
}

// LDS for ranges of at most nt tiles: a range that touches fewer may take more (two slots of less).
template <int MF, int PA, int W>
static int glu_mid_lds(int nt) {
  const int each[4] = {GluMidSlot<1, MF, PA, W>::kLds, GluMidSlot<2, MF, PA, W>::kLds, GluMidSlot<3, MF, PA, W>::kLds, GluMidSlot<4, MF, PA, W>::kLds};
  return *std::max_element(each, each + nt);
}

// Workgroup b: of row block and column range, one is b / fast, the other (rows_fast: the block) b % fast; `fast` is how many
// there are of the latter. Consecutive b run on one XCD. The columns are dealt out `gran` at a time.
template <int MF, int PA, int W>
__global__ __launch_bounds__(64 * W, 2) void glu_mid_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ ASG, const float* __restrict__ RS, int M, int K,
    const u32x4* __restrict__ wpk, const uint32_t* __restrict__ sz, int F, int ranges, int gran, int fast, int rows_fast, int act, uint16_t* __restrict__ h,
    int64_t ldh, int out_bf16) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int b = xcd_tile(blockIdx.x, gridDim.x);
  // uniform, but the divisions run on the vector ALU: back to scalar registers, which the loads' bases need
  const int q = __builtin_amdgcn_readfirstlane(b / fast), rest = b - q * fast;
  const int block = rows_fast ? rest : q, r = rows_fast ? q : rest, m0 = 16 * MF * block;
  const int units = F / gran, base = __builtin_amdgcn_readfirstlane(units / ranges), extra = units - base * ranges;
  const int c0 = gran * (r * base + min(r, extra)), c1 = c0 + gran * (base + (r < extra));
  const int nt = ((c1 - 1) >> 4) - (c0 >> 4) + 1;
  if (nt == 1) glu_mid_body<1, MF, PA, W>(A, ASG, RS, M, K, wpk, sz, F, m0, c0, c1, act, h, ldh, out_bf16 != 0, smem);
  else if (nt == 2) glu_mid_body<2, MF, PA, W>(A, ASG, RS, M, K, wpk, sz, F, m0, c0, c1, act, h, ldh, out_bf16 != 0, smem);
  else if (nt == 3) glu_mid_body<3, MF, PA, W>(A, ASG, RS, M, K, wpk, sz, F, m0, c0, c1, act, h, ldh, out_bf16 != 0, smem);
  else glu_mid_body<4, MF, PA, W>(A, ASG, RS, M, K, wpk, sz, F, m0, c0, c1, act, h, ldh, out_bf16 != 0, smem);
}

// How the rows and columns are cut: blocks of 16 MF rows times column ranges. It serves while blocks of the most rows a slot
// holds (64, or 32 with two rotations) times ranges of kGmColumns are at most two per CU; where they are at most one, and K has
// more than 4 groups (of fewer, half of eight waves would get none), one 8-wave workgroup per CU, else two of 4 waves. Among the
// block heights the one whose workgroups issue and compute least per group and CU: loads (2 MF P of activations, 2 nt of
// weights, 2 + 2 P of scales) and 2 nt MF products; two 4-wave workgroups side by side count as 1.6. The tallest blocks throughout
// were slower wherever F is small: M=297, K=5504, F=208 12.6 against 6.6 us, M=68, K=8448, F=544 15.9 / 10.5, M=32, K=10240,
// F=1024 12.4 / 8.4; M=18, K=7808, F=720 is one of the few the rule costs something, 8.4 / 9.3.
// K=5120, F=8704: 12.8 to 13.2 us at M=17..32, 18.8 at 64, 29.3 at 128 (the tiles below take 50 at M=129..256, this kernel 58).
struct GluMidPlan {
  int MF, blocks, ranges;
  int gran, nt;    // columns are dealt out gran at a time; tiles of a projection that a range may touch
  bool eight;      // one 8-wave workgroup per CU, else two 4-wave workgroups
  bool rows_fast;  // consecutive workgroups take the blocks of one range, else the ranges of one block
};
static bool glu_mid_plan(int M, int F, int P, int G, int cus, GluMidPlan* best) {
  const int64_t least = (F + kGmColumns - 1) / kGmColumns;
  const int most_mf = P == 1 ? 4 : 2;
  if ((M + 16 * most_mf - 1) / (16 * most_mf) * least > 2 * static_cast<int64_t>(cus)) return false;
  int64_t cost = -1;
  for (int MF = most_mf; MF >= 1; --MF) {
    GluMidPlan p{};
    p.MF = MF;
    p.blocks = (M + 16 * MF - 1) / (16 * MF);
    const int64_t work = p.blocks * least;
    if (work > 2 * static_cast<int64_t>(cus)) break;
    p.eight = work <= cus && G > 4;
    p.ranges = static_cast<int>(std::min<int64_t>(F / 2, std::max<int64_t>(least, (p.eight ? cus : 2 * cus) / p.blocks)));
    const int widest = 2 * ((F / 2 + p.ranges - 1) / p.ranges), pairs_nt = (widest + 14 + 15) / 16, tiles_nt = (F / 16 + p.ranges - 1) / p.ranges;
    // Columns are dealt out in pairs, so that every CU streams as many, or, from three row blocks on (the weights come
    // from the L2 then), in whole tiles where that leaves a range fewer tiles to compute and to sum: M=301, K=1024,
    // F=1424 6.8 against 7.9 us, M=192, K=4096, F=2048 13.6 / 15.5; with fewer blocks no faster, or 4 % slower.
    p.gran = p.blocks > 2 && tiles_nt < pairs_nt && F / 16 >= p.ranges ? 16 : 2;
    p.nt = p.gran == 16 ? tiles_nt : pairs_nt;
    const int64_t per_cu = p.eight ? 10 : 8 * ((static_cast<int64_t>(p.blocks) * p.ranges + cus - 1) / cus);
    const int64_t c = per_cu * (2 * MF * P + 2 * p.nt + 2 + 2 * P + 2 * p.nt * MF);
    if (cost < 0 || c <= cost) { cost = c; *best = p; }
  }
  // What an XCD's consecutive workgroups share: the weights of a range, or the rows of a block where those are more bytes
  // (M=90, K=4096, F=4096, two rotations 13.8 against 16.4 us, M=192, K=4096, F=2048 10.6 / 12.4; M=844, K=6912, F=32 7.3 / 6.5).
  best->rows_fast = F > static_cast<int64_t>(M) * P;
  return cost >= 0;
}

// ---------------------------------------------------------------------------------------
// Prompts
template <int PA>
__global__ __launch_bounds__(512, 1) void glu_prefill_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ ASGT, int M, int K, const u32x4* __restrict__ wpk,
    const u32x4* __restrict__ zpe, const u32x4* __restrict__ zpa, const float* __restrict__ s9img, int F, int act,
    uint16_t* __restrict__ h, int64_t ldh, int out_bf16, PrefillMap map, bool vec16) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kPfLds];
  const int b = blockIdx.x;
  const int bm = PA == 1 ? 256 : 128;
  const bool piece = b >= map.full;
  const int big = piece ? map.full + (b - map.full) / map.split : b;
  const int r = piece ? (b - map.full) % map.split : 0;
  const int t = xcd_tile(big, map.ntiles);
  int trow, tcol;
  tile_rc(t, map.tiles_m, map.tiles_n, trow, tcol);
  int m0 = trow * bm, n0 = tcol * 256;   // n0: gate and up columns together, twice the output column
  const int split = piece ? map.split : 1;
  if (split == 2) m0 += (bm / 2) * r;
  else if (split == 4) { m0 += 128 * (r & 1); n0 += 128 * (r >> 1); }
  else if (split == 8) { m0 += 64 * (r & 3); n0 += 128 * (r >> 2); }
  if (m0 >= M || n0 >= 2 * F) return;   // a piece wholly past the matrix
#define PQ_GLU_TILE(TM, TN)                                                                                          \
  prefill_tile<TM, TN, 2, 4, false, false, false, kPfStages, PA>(A, ASGT, M, K, wpk, nullptr, zpe, zpa, s9img, 2 * F, 0, m0, \
                                                                 n0, h, ldh, vec16, smem, act, out_bf16 != 0)
  if constexpr (PA == 1) {
    if (split == 1) PQ_GLU_TILE(256, 256);
    else if (split == 2) PQ_GLU_TILE(128, 256);
    else if (split == 4) PQ_GLU_TILE(128, 128);
    else PQ_GLU_TILE(64, 128);
  } else {
    if (split == 1) PQ_GLU_TILE(128, 256);
    else PQ_GLU_TILE(64, 256);
  }
#undef PQ_GLU_TILE
}

// 128 x 128 tiles (64 output columns), two workgroups per CU, one rotation: for grids of up to about two such tiles per
// CU, where 256 x 256 tiles would leave many CUs without work, and for very short rows (pq_gemm_glu says when).
using GluSmallTile = PfTile<128, 128, 2, 4, false, false, kPfStages, 1>;
__global__ __launch_bounds__(512, 4) void glu_small_tile_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ ASGT, int M, int K, const u32x4* __restrict__ wpk,
    const u32x4* __restrict__ zpe, const u32x4* __restrict__ zpa, const float* __restrict__ s9img, int F, int act,
    uint16_t* __restrict__ h, int64_t ldh, int out_bf16, int tiles_m, int tiles_n, bool vec16) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kPfStages * GluSmallTile::kStage];
  static_assert(2 * sizeof(smem) <= 163840 && sizeof(smem) >= 128 * GluSmallTile::kOutStride * 2, "two workgroups' LDS");
  int trow, tcol;
  tile_rc(xcd_tile(blockIdx.x, gridDim.x), tiles_m, tiles_n, trow, tcol);
  prefill_tile<128, 128, 2, 4, false, false, false, kPfStages, 1>(A, ASGT, M, K, wpk, nullptr, zpe, zpa, s9img, 2 * F, 0, 128 * trow,
                                                                  128 * tcol, h, ldh, vec16, smem, act, out_bf16 != 0);
}

}  // namespace pq

extern "C" {

int pq_gemm_glu(const uint8_t* a_d, const float* asg_d, const float* rs_d, int M, int K, int P, const void* wpk_d,
                const uint16_t* sz_d, int F, int act, uint16_t* h_d, int64_t ldh, int h_type, void* ws_d,
                size_t ws_bytes, int prepared, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_gemm_glu";
  if (M < 0) return set_error(PQ_ERR_SHAPE, "%s: M=%d < 0", what, M);
  if (K <= 0 || K % PQ_GROUP || K > (1 << 24)) return set_error(PQ_ERR_SHAPE, "%s: K=%d must be a positive multiple of 128", what, K);
  if (F <= 0 || F % 16 || F > (1 << 23)) return set_error(PQ_ERR_SHAPE, "%s: F=%d must be a positive multiple of 16", what, F);
  if (ldh < F || (ldh & 1)) return set_error(PQ_ERR_SHAPE, "%s: ldh=%lld must be even and >= F=%d", what, static_cast<long long>(ldh), F);
  if (act != PQ_ACT_SILU && act != PQ_ACT_GELU) return set_error(PQ_ERR_SHAPE, "%s: act=%d", what, act);
  if (h_type != PQ_F16 && h_type != PQ_BF16) return set_error(PQ_ERR_SHAPE, "%s: h_type=%d must be f16 or bf16", what, h_type);
  if (P != 1 && P != 2) return set_error(PQ_ERR_PARTITION, "%s: P=%d must be 1 or 2 (the gate's rotation and the up projection's)", what, P);
  const size_t need = pq_gemm_workspace_bytes(M, 2 * F, K);
  if (ws_bytes < need) return set_error(PQ_ERR_WORKSPACE, "%s: workspace too small", what);
  if (M == 0) return PQ_OK;
  if (!a_d || !asg_d || !rs_d || !wpk_d || !sz_d || !h_d) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (need && !ws_d) return set_error(PQ_ERR_NULL, "%s: NULL workspace", what);
  if (!aligned(a_d, 16) || !aligned(asg_d, 4) || !aligned(rs_d, 4) || !aligned(wpk_d, 16) || !aligned(sz_d, 4) ||
      !aligned(h_d, 4) || !aligned(ws_d, 16))
    return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  // lane offsets into a partition's codes and scales are 32-bit
  if (static_cast<int64_t>(M) * K > 0x7FFFFFFF) return set_error(PQ_ERR_SHAPE, "%s: M * K too large for one call (split the rows)", what);
  const int G = K / PQ_GROUP, cus = cu_count();
  const u32x4* wpk = static_cast<const u32x4*>(wpk_d);
  const size_t N = 2 * static_cast<size_t>(F);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int out_bf16 = h_type == PQ_BF16;
  hipError_t launched = hipSuccess;
  GluMidPlan plan;
  const bool mid = glu_mid_plan(M, F, P, G, cus, &plan);
  const int MA = M <= 8 ? 8 : 16, most = glu_max_columns(MA, P);
  // the fewest whole rounds of one range per CU whose ranges are short enough
  const int64_t rounds = (static_cast<int64_t>(F) + static_cast<int64_t>(cus) * most - 1) / (static_cast<int64_t>(cus) * most);
  // Layers too wide for one round go to the row blocks, whose ranges are longer, while those fit: K=5120: M=9, F=9216 13.1 us here,
  // 11.5 there, M=16, F=8704 with two rotations 17.2 / 13.6; M=12, K=2048, F=19984 14.8 / 11.1. One round: M=16, F=8704 11.7 in
  // either, M=8, F=1424 6.7 here, 7.4 there.
  if (M <= 16 && (rounds == 1 || !mid)) {
    const int64_t ranges = std::min<int64_t>(F / 2, rounds * cus);
#define PQ_GLU_DECODE(MR, MA, PA)                                                                                                 \
  launched = launch_kernel((glu_decode_kernel<MR, MA, PA>), dim3(static_cast<unsigned>(ranges)), dim3(64 * kGdWaves), 0, s, a_d, \
                           asg_d, rs_d, M, K, wpk, reinterpret_cast<const uint32_t*>(sz_d), F, act, h_d, ldh, out_bf16)
    if (P == 1) {
      if (M == 1) PQ_GLU_DECODE(1, 8, 1);
      else if (M <= 8) PQ_GLU_DECODE(4, 8, 1);
      else PQ_GLU_DECODE(4, 16, 1);
    } else {
      if (M == 1) PQ_GLU_DECODE(1, 8, 2);
      else if (M <= 8) PQ_GLU_DECODE(4, 8, 2);
      else PQ_GLU_DECODE(4, 16, 2);
    }
#undef PQ_GLU_DECODE
    return launch_status(what, launched);
  }
  if (mid) {
#define PQ_GLU_MID(MF, PA, W)                                                                                                  \
  do {                                                                                                                         \
    const int lds = glu_mid_lds<MF, PA, W>(plan.nt);                                                                           \
    launched = launch_kernel((glu_mid_kernel<MF, PA, W>), dim3(static_cast<unsigned>(plan.blocks) * plan.ranges), dim3(64 * W), lds, s, \
                             a_d, asg_d, rs_d, M, K, wpk, reinterpret_cast<const uint32_t*>(sz_d), F, plan.ranges, plan.gran,  \
                             plan.rows_fast ? plan.blocks : plan.ranges, plan.rows_fast ? 1 : 0, act, h_d, ldh, out_bf16);     \
  } while (0)
#define PQ_GLU_MID_WAVES(MF, PA)          \
  do {                                    \
    if (plan.eight) PQ_GLU_MID(MF, PA, 8); \
    else PQ_GLU_MID(MF, PA, 4);           \
  } while (0)
    if (P == 2 && plan.MF == 1) PQ_GLU_MID_WAVES(1, 2);
    else if (P == 2) PQ_GLU_MID_WAVES(2, 2);
    else if (plan.MF == 1) PQ_GLU_MID_WAVES(1, 1);
    else if (plan.MF == 2) PQ_GLU_MID_WAVES(2, 1);
    else if (plan.MF == 3) PQ_GLU_MID_WAVES(3, 1);
    else PQ_GLU_MID_WAVES(4, 1);
#undef PQ_GLU_MID_WAVES
#undef PQ_GLU_MID
    return launch_status(what, launched);
  }
  // Less than a round of 256 x 256 tiles, that the map takes whole or in halves: 128 x 128 tiles, two at a time on a CU, up
  // to 2.25 per CU. K=5120, F=8704: M=256 52.9 against 53.4 us, M=300 51.9 / 81.1, M=384 51.6 / 81, M=512 76.0 / 81.5,
  // M=768 (3.2 per CU) 96.4 / 82.1; K=2048, F=4096: M=512 19.8 / 20.7. Also for one or two groups, where a tile is mostly its
  // beginning and its end, which two workgroups overlap: M=1200, K=256, F=4640 16.9 against 18.8 us, M=2048, K=256, F=8704 32.2 /
  // 33.4; at eight groups 58.1 / 56.1.
  const int rows128 = (M + 127) / 128, cols128 = (2 * F + 127) / 128;
  const int64_t small = static_cast<int64_t>(rows128) * cols128;
  if (small * 8 > 0x7FFFFFFF) return set_error(PQ_ERR_SHAPE, "%s: problem too large", what);
  const PrefillMap map = prefill_map(M, 2 * F, P == 1 ? kPfWide : kPfPair, cus);
  const bool small_tiles = P == 1 && (G <= 2 || (map.full == 0 && map.split < 4 && 4 * small <= 9 * static_cast<int64_t>(cus)));
  const int64_t grid = small_tiles ? small : static_cast<int64_t>(map.full) + static_cast<int64_t>(map.ntiles - map.full) * map.split;
  if (grid * 64 * kPfWaves > 0xFFFFFFFFll)   // the runtime counts a launch's threads in 32 bits
    return set_error(PQ_ERR_SHAPE, "%s: M=%d rows too many for one call (split the rows)", what, M);
  const uint8_t* wb = static_cast<const uint8_t*>(wpk_d);
  const u32x4* zpe = reinterpret_cast<const u32x4*>(wb + static_cast<size_t>(K) * N / 2);
  const float* s9img = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(zpe) + (N / 16) * zpe_chunks(G) * 1024);
  const float* asgt = reinterpret_cast<const float*>(static_cast<const uint8_t*>(ws_d) + zpe_act_bytes(M, G, PQ_MAX_PARTITIONS));
  const bool vec16 = aligned(h_d, 16) && ldh % 8 == 0;
  if (!prepared) {
    const int rc = launch_status(what, zero_point_operands(asg_d, rs_d, M, G, P, ws_d, PQ_MAX_PARTITIONS, s));
    if (rc != PQ_OK) return rc;
  }
  if (small_tiles) {
    launched = launch_kernel(glu_small_tile_kernel, dim3(static_cast<unsigned>(grid)), dim3(64 * kPfWaves), 0, s, a_d, asgt, M, K, wpk, zpe,
                             static_cast<const u32x4*>(ws_d), s9img, F, act, h_d, ldh, out_bf16, rows128, cols128, vec16);
    return launch_status(what, launched);
  }
  auto kern = P == 1 ? glu_prefill_kernel<1> : glu_prefill_kernel<2>;
  launched = launch_kernel(kern, dim3(static_cast<unsigned>(grid)), dim3(64 * kPfWaves), 0, s, a_d, asgt, M, K, wpk, zpe,
                           static_cast<const u32x4*>(ws_d), s9img, F, act, h_d, ldh, out_bf16, map, vec16);
  return launch_status(what, launched);
}

}  // extern "C"
