// The prefill tile of the packed-weight GEMMs (M > 16), its grid and its output stores.
#pragma once

#include "pq_device.h"
#include "pq_gemm_device.h"
#include "pq_internal.h"

namespace pq {

// ---------------------------------------------------------------------------------------
// prefill (M > 16). One 512-thread workgroup (8 waves) per output tile of TM x TN; the waves
// form a WM x WN grid of (TM/WM) x (TN/WN) blocks; one 128-group per k-step. Operands move
// global -> LDS by direct LDS loads through a ring of S stages (S - 1 groups ahead: 3 stages, or 2
// for int5 256x256 tiles whose stage does not fit three times in LDS). The activation slab
// arrives as whole 128-byte rows (8 rows per load, fully used cache lines) with the 16-byte chunk
// index XOR-swizzled by (row%8) ^ ((row/8)%2): each 16-lane quarter of a fragment read then
// covers the 64 LDS banks once (measured on gfx950: (row/2)%8 and row%8 read ~40% slower); the
// weight image is already in fragment order (each lane reads 16 contiguous bytes). Per group and
// wave the products T = MFMA(codes_g, A_g) are folded as acc += (asg * 512 sc) * T (2 VALU per output),
// each row fragment's products issued before the previous fragment's fold. The zero-point term is
// subtracted as a bf16 matrix-core product (pack_zpe_kernel / zpe_act_kernel operands) in KC more
// k-steps of the same ring, their loads issued while the last groups compute; the bf16 tile is then
// staged in LDS and written as whole rows.
//
// Tiles (PrefillMap): whole rounds of 256x256 tiles, one workgroup per CU, numbered in bands of
// 4 row tiles (tile_rc) so that the tiles an XCD runs at once share their activation and weight
// codes in its L2; the tiles of the last, partial round are cut into 2, 4 or 8 pieces (128x256,
// 128x128, 64x128) so that round costs a fraction of a full one instead of a full round at low
// occupancy. Partition boundaries that are not multiples of 256 switch the whole launch to
// 128x128 tiles (pieces 64x128).
constexpr int kPfStages = 3;
constexpr int kPfWaves = 8;
constexpr int kPfLds = kPfStages * 51200;   // the 256x256 ring (the largest)

// kGlu: 0 for a plain product. 1 or 2: the gated pair of pq_gemm_glu with that many partitions. The
// weights are then gate | up, N = 2 F columns; the tile's TN columns are TN/2 of each, interleaved by
// 16-column strips (even strips gate, odd strips up, pf_strip), so that a lane holds the gate and up
// values of the same output in neighbouring fragments and the epilogue writes act(gate) * up. With two
// partitions the stage holds both partitions' activation rows and scales.
template <int TM, int TN, int WM, int WN, bool kTok = false, bool kW5 = false, int S = kPfStages, int kGlu = 0>
struct PfTile {
  static constexpr int PA = kGlu == 2 ? 2 : 1;                 // activation partitions in a stage
  static constexpr int MF = TM / WM / 16, NF = TN / WN / 16;   // fragments per wave
  static constexpr int kOffA = 0;                              // [TM rows][8 chunks][16 B], chunks swizzled
  static constexpr int kOffB = PA * TM * 128;                       // [TN/16 tiles][64 lanes][16 B]
  static constexpr int kOffAsg = kOffB + TN * 64;              // [TM] f32
  static constexpr int kOffS9 = kOffAsg + PA * TM * 4;              // [TN] f32 column factors 512 sc
  static constexpr int kOffH = kOffS9 + TN * 4;                // int5: [TN/16 tiles][64 lanes] u32
  static constexpr int kStage = (kOffH + (kW5 ? TN * 16 : 0) + 255) / 256 * 256;
  static constexpr int nA = PA * TM / 8, nB = TN / 16, nAs = kTok ? 0 : PA * TM / 64, nS9 = TN / 64;
  static constexpr int nH = kW5 ? TN / 16 : 0;
  static constexpr int nD = nA + nB + nAs + nS9 + nH;          // direct loads per group
  static constexpr int kPerWave = (nD + 3) / 4;                 // loads per wave of the issuing half
  static constexpr int kOutCols = kGlu ? TN / 2 : TN;
  static constexpr int kOutStride = kOutCols + 8;              // 16-bit values per staged output row
  static_assert(WM * WN == kPfWaves && MF >= 1 && NF >= 1 && TM % 64 == 0 && TN % 64 == 0, "tile");
  static_assert(S >= 2 && S * kStage <= kPfLds && TM * kOutStride * 2 <= kPfLds, "LDS");
  static_assert(kPerWave <= 31, "vmcnt");
};

// The 16-column strip of the weights that strip j of a gated tile reads, h0 its first output column: past
// F the last one, whose results are never stored.
__device__ __forceinline__ int pf_strip(int h0, int j, int F) {
  return min(h0 / 16 + (j >> 1), F / 16 - 1) + (j & 1 ? F / 16 : 0);
}

// act(g) * u for silu and gelu (tanh form): both are g * sigmoid(t), t = g or 2 sqrt(2/pi) (g + 0.044715 g^3).
// exp and the reciprocal by the hardware's instructions, 1 ulp (2 u, u = 2^-24) each. The exponent is off by the product's and
// the constant's rounding, and for gelu by its polynomial's 4: 2 |t| u of the result for silu, 6 |t| u for gelu, so with the other
// steps' 8 u at most 2^-14.9 wherever sigmoid is a normal number (t > -87.3), below the half step of f16 (2^-11) and bf16 (2^-8) that
// the one rounding then takes; below that t the result is 0.
__device__ __forceinline__ float glu_value(float g, float u, int act) {
  const float t = act == PQ_ACT_GELU ? g * __builtin_fmaf(0.0713548162726f * g, g, 1.59576912161f) : g;
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504089f * t)) * u;
}

template <int N>
__device__ __forceinline__ void wait_vm_lgkm_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Writes an LDS-staged bf16 tile [TM rows][STRIDE] to y (rows < M, columns < N): 16-byte stores
// of 8 columns when y and ldy allow it (vec16), else 4-byte stores of 2 columns. Uses all threads
// of the workgroup.
template <int TM, int TN, int STRIDE>
__device__ __forceinline__ void store_tile_rows(const uint16_t* ot, uint16_t* __restrict__ y, int64_t ldy,
                                                int m0, int n0, int M, int N, bool vec16) {
  const int nthr = blockDim.x;
  if (vec16) {
    constexpr int CH = TN / 8;
    for (int c = threadIdx.x; c < TM * CH; c += nthr) {
      const int r = c / CH, ch = c % CH;
      const int m = m0 + r, n = n0 + 8 * ch;
      if (m < M && n < N)
        *reinterpret_cast<u32x4*>(y + static_cast<size_t>(m) * ldy + n) =
            *reinterpret_cast<const u32x4*>(ot + r * STRIDE + 8 * ch);
    }
  } else {
    constexpr int CH = TN / 2;
    for (int c = threadIdx.x; c < TM * CH; c += nthr) {
      const int r = c / CH, ch = c % CH;
      const int m = m0 + r, n = n0 + 2 * ch;
      if (m < M && n < N)
        *reinterpret_cast<uint32_t*>(y + static_cast<size_t>(m) * ldy + n) =
            *reinterpret_cast<const uint32_t*>(ot + r * STRIDE + 2 * ch);
    }
  }
}

// Workgroups are dispatched to the 8 XCDs round-robin; give each XCD a contiguous range of
// tile numbers.
__device__ __forceinline__ int xcd_tile(int bid, int ntiles) {
  const int q = ntiles / 8;
  return bid < 8 * q ? (bid % 8) * q + bid / 8 : bid;
}

// Tile number -> (row tile, column tile), in bands of kPfBand row tiles: within a band the
// columns in order, within a column the band's rows (a last, shorter band takes the remaining
// rows). An XCD's contiguous range of numbers then covers a few row tiles by many columns, so
// the tiles it runs at once share both operands in its L2: 32 tiles as 4 rows x 8 columns need
// 128 KiB of activation codes and 128 KiB of weight codes per group step (256x256 tiles),
// where a column of 32 row tiles needs 1 MiB of activation codes.
constexpr int kPfBand = 4;
__device__ __forceinline__ void tile_rc(int t, int tiles_m, int tiles_n, int& row, int& col) {
  const int bands = tiles_m / kPfBand, band_tiles = kPfBand * tiles_n;
  const int band = t / band_tiles;
  if (band < bands) {
    const int rem = t - band * band_tiles;
    col = rem / kPfBand;
    row = band * kPfBand + rem % kPfBand;
  } else {
    const int last = tiles_m - bands * kPfBand, rem = t - bands * band_tiles;
    col = rem / last;
    row = bands * kPfBand + rem % last;
  }
}

template <int TM, int TN, int WM, int WN, bool kTok, bool kI8, bool kW5, int S = kPfStages, int kGlu = 0>
__device__ __forceinline__ void prefill_tile(
    const uint8_t* __restrict__ A, const float* __restrict__ ASGT, int M, int K,
    const u32x4* __restrict__ wpk, const uint32_t* __restrict__ hi, const u32x4* __restrict__ zpe,
    const u32x4* __restrict__ zpa, const float* __restrict__ s9img, int N, int p, int m0, int n0,
    uint16_t* __restrict__ y, int64_t ldy, bool vec16, uint8_t* smem, int act = 0, bool out_bf16 = true) {
  using TL = PfTile<TM, TN, WM, WN, kTok, kW5, S, kGlu>;
  constexpr int PA = TL::PA;
  const int F = N / 2, h0 = n0 / 2;   // gated pair: N = 2 F, the tile's first output column
  static_assert(S == 2 || S == 3, "the wait counts below cover rings of 2 and 3 stages");
  constexpr int D = S - 1;   // groups loaded ahead
  constexpr int MF = TL::MF, NF = TL::NF, PW = TL::kPerWave;
  const int G = K >> 7;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform: load table stays scalar
  const int wm = wave / WN, wn = wave % WN;
  const int kq = lane >> 4;
  const int last_tile = N / 16 - 1;
  const float* asgp = ASGT + static_cast<size_t>(p) * G * M;   // [G][M] for this partition

  // The direct loads of a group are issued by one half of the workgroup, waves 0-3 for even
  // groups and waves 4-7 for odd ones (one wave per SIMD each), so that on every SIMD one wave
  // computes while its partner is held up issuing loads. This wave's share: entry
  // d = (wave % 4) + 4 i of the tile's list (A half-fragments, weight tiles, asg rows, SZ
  // columns), taken modulo the list length so every wave of a half issues PW loads (a repeated
  // entry writes the same bytes again). Each entry is a scalar
  // base (advanced per group on the scalar unit) plus a fixed 32-bit lane offset. Rows past M
  // and column tiles past N are clamped to valid memory; their results are never stored.
  const uint8_t* sbase[PW];
  uint32_t voff[PW];
  size_t step[PW];
  uint32_t dst[PW];
  bool wide[PW];
  const uint8_t* Ap = A + static_cast<size_t>(p) * M * K;
#pragma unroll
  for (int i = 0; i < PW; ++i) {
    const int d = ((wave & 3) + 4 * i) % TL::nD;
    if (d < TL::nA) {
      const int r = 8 * (PA == 1 ? d : d % (TM / 8)) + (lane >> 3);   // tile row; lane%8 = chunk slot
      const int row = min(m0 + r, M - 1);
      sbase[i] = PA == 1 || d < TM / 8 ? Ap : Ap + static_cast<size_t>(M) * K;
      voff[i] = static_cast<uint32_t>(row * K + 16 * ((lane & 7) ^ (r & 7) ^ ((r >> 3) & 1)));
      step[i] = 128; dst[i] = TL::kOffA + d * 1024; wide[i] = true;
    } else if (d < TL::nA + TL::nB) {
      const int j = d - TL::nA;
      const int tt = kGlu ? pf_strip(h0, j, F) : min(n0 / 16 + j, last_tile);
      sbase[i] = reinterpret_cast<const uint8_t*>(wpk) + static_cast<size_t>(tt) * G * 1024;
      voff[i] = 16 * lane;
      step[i] = 1024; dst[i] = TL::kOffB + j * 1024; wide[i] = true;
    } else if (d < TL::nA + TL::nB + TL::nAs) {
      const int j = d - TL::nA - TL::nB;
      sbase[i] = reinterpret_cast<const uint8_t*>(PA == 1 || j < TM / 64 ? asgp : asgp + static_cast<size_t>(G) * M);
      voff[i] = static_cast<uint32_t>(min(m0 + 64 * (PA == 1 ? j : j % (TM / 64)) + lane, M - 1) * 4);
      step[i] = static_cast<size_t>(M) * 4; dst[i] = TL::kOffAsg + j * 256; wide[i] = false;
    } else if (d < TL::nA + TL::nB + TL::nAs + TL::nS9) {
      const int j = d - TL::nA - TL::nB - TL::nAs;
      sbase[i] = reinterpret_cast<const uint8_t*>(s9img);
      voff[i] = kGlu ? static_cast<uint32_t>((16 * pf_strip(h0, 4 * j + (lane >> 4), F) + (lane & 15)) * 4)
                     : static_cast<uint32_t>(min(n0 + 64 * j + lane, N - 1) * 4);
      step[i] = static_cast<size_t>(N) * 4; dst[i] = TL::kOffS9 + j * 256; wide[i] = false;
    } else {
      const int j = d - TL::nA - TL::nB - TL::nAs - TL::nS9;   // int5 fifth-bit words of tile j
      const int tt = min(n0 / 16 + j, last_tile);
      sbase[i] = reinterpret_cast<const uint8_t*>(hi) + static_cast<size_t>(tt) * G * 256;
      voff[i] = 4 * lane;
      step[i] = 256; dst[i] = TL::kOffH + j * 256; wide[i] = false;
    }
  }
  const uint32_t lds0 = lds_addr(smem);
  auto issue = [&](int stage, int g) {
    const uint32_t st = lds0 + stage * TL::kStage;
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      if (wide[i]) lds_dma16_s(sbase[i] + g * step[i], voff[i], st + dst[i]);
      else lds_dma4_s(sbase[i] + g * step[i], voff[i], st + dst[i]);
    }
  };
  // Zero-point epilogue operands (pack_zpe_kernel / zpe_act_kernel): for chunk c of KC, the tile's
  // TM/16 activation-side and TN/16 weight-side fragments, 1 KiB each, go to a stage at
  // f * 1024 (f = fragment) like one more group; this half's share: fragments (wave % 4) + 4 i.
  // The source of each is computed on the scalar unit when it is issued.
  constexpr int ZA = PA * TM / 16, NZ = ZA + TN / 16, PWZ = (NZ + 3) / 4;
  static_assert(PWZ <= PW && NZ * 1024 <= TL::kStage, "zero-point chunks ride the group ring");
  const int KC = zpe_chunks(G), MT = (M + 15) / 16;
  auto zissue = [&](int stage, int c) {
    const uint32_t st = lds0 + stage * TL::kStage;
#pragma unroll
    for (int i = 0; i < PWZ; ++i) {
      const int f = (wave & 3) + 4 * i;
      if (f < NZ) {
        const int fa = PA == 1 ? f : f % (TM / 16), fp = PA == 1 ? p : f / (TM / 16);
        const uint8_t* src = (f < ZA)
            ? reinterpret_cast<const uint8_t*>(zpa) + ((static_cast<size_t>(fp) * MT + min(m0 / 16 + fa, MT - 1)) * KC + c) * 1024
            : reinterpret_cast<const uint8_t*>(zpe) + (static_cast<size_t>(kGlu ? pf_strip(h0, f - ZA, F) : min(n0 / 16 + f - ZA, last_tile)) * KC + c) * 1024;
        lds_dma16_s(src, 16 * lane, st + f * 1024);
      }
    }
  };
  // k-steps 0 .. G-1 are the groups, G .. G+KC-1 the zero-point chunks
  const int GT = G + KC;
  auto issue_step = [&](int stage, int j) {
    if (j < G) issue(stage, j);
    else zissue(stage, j - G);
  };

  v4f acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // Group j's loads go into stage j % S and are issued during group j - D (D = S - 1 groups
  // ahead; the first D groups before the loop) by half (j - D) % 2.
  const int half = wave >> 2;
  for (int j = 0; j < D && j < GT; ++j)
    if (((j - D) & 1) == half) issue_step(j % S, j);
  // Step g was loaded by half (g - D) % 2, whose only outstanding loads are step g's: it waits
  // for all of them. With D = 2 the other half's outstanding loads (at most PW, step g+1) need
  // not land; with D = 1 it has none. The barrier then makes step g visible to every wave and
  // guarantees that no wave still reads stage (g + D) % S, the one step g - 1 used.
  // (__syncthreads would also drain the step g+1 loads.) A zero-point chunk step has at most
  // PWZ <= PW loads per wave, so the same waits hold.
  auto step_begin = [&](int g) {
    if (((g - D) & 1) == half) wait_vm_lgkm_barrier<0>();
    else wait_vm_lgkm_barrier<D >= 2 ? PW : 0>();
    if (g + D < GT && (g & 1) == half) issue_step((g + D) % S, g + D);
  };
  for (int g = 0; g < G; ++g) {
    step_begin(g);
    const uint8_t* st = smem + (g % S) * TL::kStage;

    // Products are taken as (weights) x (activations)^T, so a lane's 4 results are one output row
    // (the fragment row lane % 16) and 4 consecutive columns (4 (lane / 16) .. + 3): the row scale
    // is one value per lane, the column factors a float4.
    u32x4 braw[NF];
    uint32_t hw[NF];
    v8i bf[NF];
    float4 s9[NF];
#pragma unroll
    for (int nf = 0; nf < NF; ++nf) {
      hw[nf] = kW5 ? *reinterpret_cast<const uint32_t*>(st + TL::kOffH + (wn * NF + nf) * 256 + lane * 4) : 0u;
      braw[nf] = *reinterpret_cast<const u32x4*>(st + TL::kOffB + (wn * NF + nf) * 1024 + lane * 16);
      s9[nf] = *reinterpret_cast<const float4*>(st + TL::kOffS9 + (wn * NF * 16 + 16 * nf + 4 * kq) * 4);
    }
    // fragment lane l: row l%16 of the 16-row block, k chunks 2(l/16) and 2(l/16)+1, swizzled
    const int arow = lane & 15, ac0 = 2 * (lane >> 4), asw = (arow & 7) ^ (arow >> 3);
    const int aoff0 = arow * 128 + 16 * (ac0 ^ asw), aoff1 = arow * 128 + 16 * ((ac0 + 1) ^ asw);
    auto load_a = [&](int mf, v8i& a, float& as, int pa) {
      const uint8_t* ap = st + TL::kOffA + (wm * MF + mf + pa * (TM / 16)) * 2048;
      const u32x4 a0 = *reinterpret_cast<const u32x4*>(ap + aoff0);
      const u32x4 a1 = *reinterpret_cast<const u32x4*>(ap + aoff1);
      a = v8i{(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
      if constexpr (!kTok) as = *reinterpret_cast<const float*>(st + TL::kOffAsg + (wm * MF * 16 + 16 * mf + arow + pa * TM) * 4);
    };
    // Row fragment mf's products are interleaved one for one with the folds of fragment mf-1
    // (acc += f T, f = asg * 512 sc: 8 VALU per product), so the matrix core and the vector ALU
    // work side by side; fragment mf+1's operands are read from LDS while mf computes, and the
    // weight codes are unpacked beside fragment 0's products.
    v4f Tb[2][NF];
    // The up projection's rows, where it has its own, are objects apart (au, asu): an array over the partitions made the compiler
    // split the plain product's paired scale reads and schedule its tiles otherwise (down, M=64 81.4 against 79.9 us, K=4096,
    // N=8192, M=64 25.5 / 25.0).
    v8i a[2], au[2];
    float asb[2] = {0.f, 0.f}, asu[2] = {0.f, 0.f};
    load_a(0, a[0], asb[0], 0);
    if constexpr (PA == 2) load_a(0, au[0], asu[0], 1);
#pragma unroll
    for (int mf = 0; mf <= MF; ++mf) {
      // fragment mf-1's row scale is taken before the prefetch reuses its slot
      const int pm = mf - 1;
      float as = 0.f, as_up = 0.f;
      if constexpr (!kTok) as = kI8 ? asb[pm & 1] * 0x1p-9f : asb[pm & 1];   // integer products carry no 2^-9
      if (mf + 1 < MF) load_a(mf + 1, a[(mf + 1) & 1], asb[(mf + 1) & 1], 0);
      if constexpr (PA == 2) {
        as_up = asu[pm & 1];
        if (mf + 1 < MF) load_a(mf + 1, au[(mf + 1) & 1], asu[(mf + 1) & 1], 1);
      }
#pragma unroll
      for (int nf = 0; nf < NF; ++nf) {
        if (mf == 0) bf[nf] = weight_operand<kW5>(braw[nf], hw[nf]);
        const bool up = PA == 2 && (nf & 1);   // gated pair of two partitions: odd strips are the up projection
        if (mf < MF) Tb[mf & 1][nf] = group_product<kI8>(bf[nf], up ? au[mf & 1] : a[mf & 1]);
        if (mf > 0) {
          const v4f& T = Tb[pm & 1][nf];
          if constexpr (kTok) {
            // per-token scales: the row scale is applied once in the epilogue
            acc[pm][nf][0] = __builtin_fmaf(s9[nf].x, T[0], acc[pm][nf][0]);
            acc[pm][nf][1] = __builtin_fmaf(s9[nf].y, T[1], acc[pm][nf][1]);
            acc[pm][nf][2] = __builtin_fmaf(s9[nf].z, T[2], acc[pm][nf][2]);
            acc[pm][nf][3] = __builtin_fmaf(s9[nf].w, T[3], acc[pm][nf][3]);
          } else {
            // the four factors first, in registers of their own (the empty asm keeps the compiler
            // from pairing each multiply with its dependent FMA through one temporary)
            const float f = up ? as_up : as;
            const float f0 = f * s9[nf].x, f1 = f * s9[nf].y, f2 = f * s9[nf].z, f3 = f * s9[nf].w;
            asm volatile("" ::"v"(f0), "v"(f1), "v"(f2), "v"(f3));
            acc[pm][nf][0] = __builtin_fmaf(f0, T[0], acc[pm][nf][0]);
            acc[pm][nf][1] = __builtin_fmaf(f1, T[1], acc[pm][nf][1]);
            acc[pm][nf][2] = __builtin_fmaf(f2, T[2], acc[pm][nf][2]);
            acc[pm][nf][3] = __builtin_fmaf(f3, T[3], acc[pm][nf][3]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // zero-point chunk c = g - G: acc += (-[a1|a1|a2]) x [z1;z2;z1] over its 32 k' (bf16 pieces of
  // asg*rs and of the zero-point factor, relative error ~2^-16), weights as the first operand
  for (int g = G; g < GT; ++g) {
    step_begin(g);
    const uint8_t* st = smem + (g % S) * TL::kStage;
    u32x4 zb[NF];
#pragma unroll
    for (int nf = 0; nf < NF; ++nf)
      zb[nf] = *reinterpret_cast<const u32x4*>(st + (ZA + wn * NF + nf) * 1024 + lane * 16);
#pragma unroll
    for (int mf = 0; mf < MF; ++mf) {
      u32x4 za[PA];
#pragma unroll
      for (int pa = 0; pa < PA; ++pa) za[pa] = *reinterpret_cast<const u32x4*>(st + (wm * MF + mf + pa * (TM / 16)) * 1024 + lane * 16);
#pragma unroll
      for (int nf = 0; nf < NF; ++nf)
        acc[mf][nf] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, zb[nf]),
                                                               __builtin_bit_cast(bf16x8, za[PA == 1 ? 0 : nf & 1]), acc[mf][nf], 0, 0, 0);
    }
  }

  // ---- bf16 tile through LDS (the ring is idle now), then whole rows with wide stores
  __syncthreads();   // every wave has finished reading the ring
  // (per-token path: each row's token scale is applied here; ASGT holds AS [P][M] in that mode and
  // the lane's row is lane % 16 of the fragment)
  uint16_t* ot = reinterpret_cast<uint16_t*>(smem);
#pragma unroll
  for (int mf = 0; mf < MF; ++mf) {
    float a = 1.0f;
    if constexpr (kTok) a = ASGT[static_cast<size_t>(p) * M + min(m0 + wm * MF * 16 + 16 * mf + (lane & 15), M - 1)];
    if constexpr (kGlu != 0) {
#pragma unroll
      for (int nf = 0; nf < NF; nf += 2) {
        float h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = glu_value(acc[mf][nf][i], acc[mf][nf + 1][i], act);
        *reinterpret_cast<uint2*>(ot + (wm * MF * 16 + 16 * mf + (lane & 15)) * TL::kOutStride + wn * NF * 8 + 8 * nf + 4 * kq) =
            out_bf16 ? make_uint2(bf16x2_rn(h[0], h[1]), bf16x2_rn(h[2], h[3])) : make_uint2(f16x2_rn(h[0], h[1]), f16x2_rn(h[2], h[3]));
      }
      continue;
    }
#pragma unroll
    for (int nf = 0; nf < NF; ++nf) {
      v4f v = acc[mf][nf];
      if constexpr (kTok) v *= a;
      *reinterpret_cast<uint2*>(ot + (wm * MF * 16 + 16 * mf + (lane & 15)) * TL::kOutStride + wn * NF * 16 + 16 * nf + 4 * kq) =
          make_uint2(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]));
    }
  }
  __syncthreads();
  store_tile_rows<TM, TL::kOutCols, TL::kOutStride>(ot, y, ldy, m0, kGlu ? h0 : n0, M, kGlu ? F : N, vec16);
}

// Tile shapes of the prefill grid: 256x256 (pieces 128x256, 128x128, 64x128), or 128x128 (pieces
// 64x128) when a partition boundary is not on a 256-column line. int5 whole 256x256 tiles run a
// ring of two stages: the fifth-bit planes make a stage 54 KiB, and three do not fit in LDS.
// The gated pair of two partitions: 128x256 tiles, whose stage holds two sets of activation rows (pieces 64x256).
enum PfShape : int { kPfWide = 0, kPfNarrow = 1, kPfPair = 2 };
struct PrefillMap {
  int tiles_m;   // whole tiles per tile column
  int tiles_n;   // whole tiles per tile row
  int ntiles;    // whole tiles
  int full;      // workgroups that run whole tiles (whole rounds); the rest run pieces
  int split;     // pieces per remaining tile: 1, 2, 4 or 8 (wide) / 1 or 2 (narrow)
  int shape;     // PfShape
};

// Whole rounds of tiles (one workgroup per CU), then the remaining tiles in pieces.
inline PrefillMap prefill_map(int M, int N, int shape, int cus) {
  PrefillMap m{};
  const int bm = shape == kPfWide ? 256 : 128, bn = shape == kPfNarrow ? 128 : 256;
  m.shape = shape;
  m.tiles_m = (M + bm - 1) / bm;
  m.tiles_n = (N + bn - 1) / bn;
  const int64_t nt = static_cast<int64_t>(m.tiles_m) * m.tiles_n;
  m.ntiles = static_cast<int>(nt);
  const int64_t full = (nt / cus) * cus, rem = nt - full;
  m.full = static_cast<int>(full);
  m.split = 1;
  if (rem > 0) {
    static const int cands[3][3] = {{8, 4, 2}, {2, 0, 0}, {2, 0, 0}};
    for (int i = 0; i < 3 && cands[shape][i]; ++i)
      if (rem * cands[shape][i] <= cus) { m.split = cands[shape][i]; break; }
  }
  return m;
}

}  // namespace pq
