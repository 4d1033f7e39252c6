// Products of few 16-bit rows (M <= 16, f16 or bf16) with the packed 4-bit weights of pq_pack_weights
// (pq_matvec), for layers whose activations are not to be quantised:
//   y[m,n] = sum_g ( sc[g,n] * sum_{k in g} x[m,k] c[k,n]  -  (8 sc + zsc)[g,n] * sum_{k in g} x[m,k] )
// which is sum_k x W with W = sc (c - 8) - zsc, the weights the GEMMs multiply.
//
// The weight stream is what bounds it, so the kernel streams as the W4A8 decode kernel does: one
// 8-wave workgroup per CU on a range of whole 4-column quarters, the waves splitting the groups, each
// with a private LDS ring that direct global -> LDS loads fill; one group is computed while the
// next is in flight; partial sums meet in LDS in a fixed order. One group ahead is the best depth
// everywhere: K=5120, N=17408, M=1 takes 11.6 / 10.7 / 11.9 us a launch with none, one and two groups
// ahead, K=5120, N=8192 6.7 / 6.0 / 6.4 us, K=17408, N=5120 14.7 / 12.2 / 12.3 us (weights in the last
// level cache; each further group adds about 0.35 us, the time the CU's load path takes to accept it).
// Two workgroups per CU on half the columns each: 10.9 and 18.1 us for the first and last.
//
// A group's codes become 16-bit matrix operands without a table: a nibble is the OCP e4m3 byte of
// c * 2^-9, and one convert instruction turns two such bytes times 2^9 into two f16 or bf16 values,
// exact for 0..15. Word q of a lane's fragment holds the codes of k = 32 (lane / 16) + 8 q .. + 7, so a
// 16x16x32 step q takes them as they come and x's 16-byte chunk 4 (lane / 16) + q beside them. The
// group's sums of x come from the matrix core too: the same steps against a fragment of ones give
// each lane the sums of exactly the rows whose products it holds, in binary32.
#include "pq_device.h"
#include "pq_gemm_device.h"
#include "pq_internal.h"

namespace pq {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kMvWaves = 8;
constexpr int kMvRingBytes = 20480;                  // per wave: the rings fill the LDS
constexpr int kMvLds = kMvWaves * kMvRingBytes;

// Rows of x held in a ring slot, the most tiles that a range may touch (whose slots fit the ring twice, or, above 8 rows, 5
// tiles twice and 6 to 8 once) and the longest range that touches no more wherever it starts. Wide layers so take one round
// where 20 quarters (17 above 8 rows) took a second of the few ranges left over: M=1, K=5120, N=20496 16.6 -> 12.5 us, M=16,
// N=18432 20.0 -> 12.4, M=6, K=256, three partitions of 22336 columns 7.1 -> 4.5.
constexpr int mv_rows(int M) { return M == 1 ? 1 : M <= 4 ? 4 : M <= 8 ? 8 : 16; }
constexpr int mv_max_tiles(int MX) { return MX == 1 ? 9 : MX == 4 ? 8 : MX == 8 ? 7 : 8; }
constexpr int mv_max_quarters(int M) { return 4 * mv_max_tiles(mv_rows(M)) - 3; }

template <int NT, int MX>
struct MatvecSlot {
  static constexpr int kSzWords = 16 * NT;
  static constexpr int kSzLoads = (kSzWords + 63) / 64;
  static constexpr int kOffX = NT * 1024;                       // [MX rows][16 chunks of 16 B], chunks XORed with the row
  static constexpr int kOffSz = kOffX + MX * 256;
  static constexpr int kBytes = kOffSz + (kSzWords * 4 + 15) / 16 * 16;
  static constexpr int kXLoads = (MX + 3) / 4;                  // 4 rows of 256 B per load
  static constexpr int kLoads = NT + kXLoads + kSzLoads;
  static constexpr int kDepth = 2 * kBytes <= kMvRingBytes ? 2 : 1;
  static_assert(kDepth * kBytes <= kMvRingBytes && (kDepth - 1) * kLoads <= 63, "ring");
};

// Two codes (e4m3 bytes of c * 2^-9, the low or high half of w) as 16-bit values.
template <bool kBf16, bool HI>
__device__ __forceinline__ uint32_t codes16(uint32_t w) {
  if constexpr (kBf16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, HI));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 512.0f, HI));
}

template <bool kBf16>
__device__ __forceinline__ v4f mfma16(const u32x4& a, const u32x4& b, const v4f& c) {
  if constexpr (kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// MR: rows per lane that can be live (1 when M == 1, else 4)
template <int NT, int MR, int MX, bool kBf16>
__device__ __forceinline__ void matvec_body(
    const uint16_t* __restrict__ x, int64_t ldx, int M, int K, const u32x4* __restrict__ wpk,
    const uint32_t* __restrict__ sz, int N, int c0, int c1, uint16_t* __restrict__ y, int64_t ldy, bool out_bf16,
    uint8_t* smem) {
  using S = MatvecSlot<NT, MX>;
  constexpr int D = S::kDepth;
  const int G = K >> 7;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int tfirst = c0 >> 4, n0 = 16 * tfirst;
  const int g0 = (G * wave) / kMvWaves, g1 = (G * (wave + 1)) / kMvWaves;

  // Sources: a scalar base per group plus a fixed per-lane offset. Lanes whose column is outside
  // [c0, c1) load no codes (every tile of the range keeps at least 4 columns, so each load is issued).
  // Lane l of x's load j takes row 4 j + l / 16 (rows past M repeat row M - 1) and the chunk
  // (l % 16) ^ row, so that the 16 lanes of a fragment read find their rows in different banks.
  const uint8_t* wbase = reinterpret_cast<const uint8_t*>(wpk) + static_cast<size_t>(tfirst) * G * 1024;
  bool won[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = n0 + 16 * t + col;
    won[t] = n >= c0 && n < c1;
  }
  const uint8_t* xbase = reinterpret_cast<const uint8_t*>(x);
  uint32_t xoff[S::kXLoads];
#pragma unroll
  for (int j = 0; j < S::kXLoads; ++j) {
    const int r = 4 * j + (lane >> 4);
    xoff[j] = static_cast<uint32_t>(min(r, M - 1) * 2 * ldx + 16 * ((lane & 15) ^ (r & 15)));
  }
  const uint8_t* zbase = reinterpret_cast<const uint8_t*>(sz + n0);

  uint8_t* ringp = smem + wave * kMvRingBytes;
  const uint32_t ring = lds_addr(ringp);
  auto issue = [&](int g, int slot) {
    const uint32_t sb = ring + slot * S::kBytes;
    const uint8_t* wg = wbase + static_cast<size_t>(g) * 1024;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (won[t]) lds_dma16_s(wg + static_cast<size_t>(t) * G * 1024, 16 * lane, sb + t * 1024);
#pragma unroll
    for (int j = 0; j < S::kXLoads; ++j)
      if (lane + 64 * j < 16 * MX) lds_dma16_s(xbase + 256 * static_cast<size_t>(g), xoff[j], sb + S::kOffX + j * 1024);
    const uint8_t* zg = zbase + static_cast<size_t>(g) * N * 4;
#pragma unroll
    for (int j = 0; j < S::kSzLoads; ++j)
      if (lane + 64 * j < S::kSzWords) lds_dma4_s(zg + 256 * j, 4 * lane, sb + S::kOffSz + j * 256);
  };
  const int ng = g1 - g0;
  for (int i = 0; i < D - 1 && i < ng; ++i) issue(g0 + i, i);

  v4f acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
  const v4f zero = {0.f, 0.f, 0.f, 0.f};
  const uint32_t one2 = kBf16 ? 0x3F803F80u : 0x3C003C00u;
  const u32x4 ones = {one2, one2, one2, one2};
  const int xrow = (lane & 15) & (MX - 1);
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
    u32x4 xa[4];
    v4f rs = zero;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      xa[q] = *reinterpret_cast<const u32x4*>(sp + S::kOffX + xrow * 256 + 16 * ((4 * kq + q) ^ xrow));
#pragma unroll
    for (int q = 0; q < 4; ++q) rs = mfma16<kBf16>(xa[q], ones, rs);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const u32x4 bw = *reinterpret_cast<const u32x4*>(sp + t * 1024 + 16 * lane);
      const uint32_t szw = *reinterpret_cast<const uint32_t*>(sp + S::kOffSz + 4 * (16 * t + col));
      const float sc = f16_to_f32(szw), zz = __builtin_fmaf(sc, 8.0f, f16_to_f32(szw >> 16));
      const uint32_t w[4] = {bw.x, bw.y, bw.z, bw.w};
      v4f T = zero;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t lo = w[q] & 0x0F0F0F0Fu, hi = (w[q] >> 4) & 0x0F0F0F0Fu;
        const u32x4 b = {codes16<kBf16, false>(lo), codes16<kBf16, true>(lo), codes16<kBf16, false>(hi), codes16<kBf16, true>(hi)};
        T = mfma16<kBf16>(xa[q], b, T);
      }
#pragma unroll
      for (int i = 0; i < MR; ++i) acc[t][i] += sc * T[i] - zz * rs[i];
    }
    slot = slot + 1 == D ? 0 : slot + 1;
  }

  __syncthreads();   // every ring has drained: the reduction reuses that LDS
  constexpr int R = 16 * NT + 4;   // the 4 extra words put every fourth row a quarter of the banks further
  float* sred = reinterpret_cast<float*>(smem);   // [waves][16 rows][16 NT], rows padded
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < MR; ++i) sred[(wave * 16 + 4 * kq + i) * R + 16 * t + col] = acc[t][i];
  __syncthreads();
  const int half = (c1 - c0) >> 1, pairs = M * half;   // c0, c1 and ldy even: 4-byte stores
  for (int idx = tid; idx < pairs; idx += 64 * kMvWaves) {
    const int m = idx / half, c = c0 - n0 + 2 * (idx % half);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int w = 0; w < kMvWaves; ++w) {
      const float2 q = *reinterpret_cast<const float2*>(sred + (w * 16 + m) * R + c);
      s0 += q.x;
      s1 += q.y;
    }
    *reinterpret_cast<uint32_t*>(y + static_cast<size_t>(m) * ldy + n0 + c) = out_bf16 ? bf16x2_rn(s0, s1) : f16x2_rn(s0, s1);
  }
}

template <bool kBf16, int MR, int MX>
__global__ __launch_bounds__(64 * kMvWaves, 1) void matvec_kernel(
    const uint16_t* __restrict__ x, int64_t ldx, int M, int K, const u32x4* __restrict__ wpk,
    const uint32_t* __restrict__ sz, int N, DecodeMap map, uint16_t* __restrict__ y, int64_t ldy, int out_bf16) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kMvLds];
  const int b = blockIdx.x, W = map.wg0[3];
  const int r = map.xcd ? (b % 8) * (W / 8) + b / 8 : b;
  const int q = (r >= map.wg0[1]) + (r >= map.wg0[2]);          // partition
  const int nwq = map.wg0[q + 1] - map.wg0[q], rq = r - map.wg0[q];
  const int base = map.nq[q] / nwq, extra = map.nq[q] % nwq;
  const int cnt = base + (rq < extra);
  const int c0 = map.c0[q] + 4 * (rq * base + (rq < extra ? rq : extra));
  const int c1 = c0 + 4 * cnt;
  const int nt = ((c1 - 1) >> 4) - (c0 >> 4) + 1;
  const uint16_t* xp = x + static_cast<size_t>(q) * M * ldx;
#define PQ_MATVEC_CASE(n) \
  case n: matvec_body<n, MR, MX, kBf16>(xp, ldx, M, K, wpk, sz, N, c0, c1, y, ldy, out_bf16 != 0, smem); break;
  constexpr int most = mv_max_tiles(MX);
  switch (nt) {
    PQ_MATVEC_CASE(1) PQ_MATVEC_CASE(2) PQ_MATVEC_CASE(3) PQ_MATVEC_CASE(4) PQ_MATVEC_CASE(5)
    default: break;
  }
#define PQ_MATVEC_WIDE(n) \
  if constexpr (most >= n) { if (nt == n) matvec_body<n, MR, MX, kBf16>(xp, ldx, M, K, wpk, sz, N, c0, c1, y, ldy, out_bf16 != 0, smem); }
  PQ_MATVEC_WIDE(6) PQ_MATVEC_WIDE(7) PQ_MATVEC_WIDE(8) PQ_MATVEC_WIDE(9)
#undef PQ_MATVEC_WIDE
#undef PQ_MATVEC_CASE
}

}  // namespace pq

extern "C" {

int pq_matvec(const uint16_t* x_d, int64_t ldx, int x_type, int M, int K, int P, const void* wpk_d,
              const uint16_t* sz_d, int N, int pb1, int pb2, uint16_t* y_d, int64_t ldy, int y_type,
              pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_matvec";
  if (M < 0 || M > 16) return set_error(PQ_ERR_SHAPE, "%s: M=%d must be in 0..16", what, M);
  if (K <= 0 || K % PQ_GROUP || K > (1 << 24)) return set_error(PQ_ERR_SHAPE, "%s: K=%d must be a positive multiple of 128", what, K);
  if (N <= 0 || N % 16 || N > (1 << 24)) return set_error(PQ_ERR_SHAPE, "%s: N=%d must be a positive multiple of 16", what, N);
  if ((x_type != PQ_F16 && x_type != PQ_BF16) || (y_type != PQ_F16 && y_type != PQ_BF16))
    return set_error(PQ_ERR_SHAPE, "%s: types x %d, y %d must be f16 or bf16", what, x_type, y_type);
  if (ldx < K || ldx % 8 || ldx > (1 << 26)) return set_error(PQ_ERR_SHAPE, "%s: ldx=%lld must be a multiple of 8 in K..2^26", what, static_cast<long long>(ldx));
  if (ldy < N || (ldy & 1)) return set_error(PQ_ERR_SHAPE, "%s: ldy=%lld must be even and >= N=%d", what, static_cast<long long>(ldy), N);
  const int perr = check_partitions(P, pb1, pb2, N);
  if (perr != PQ_OK) return perr;
  if (M == 0) return PQ_OK;
  if (!x_d || !wpk_d || !sz_d || !y_d) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (!aligned(x_d, 16) || !aligned(wpk_d, 16) || !aligned(sz_d, 4) || !aligned(y_d, 4))
    return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  DecodeMap map;
  // As few rounds of one range per CU as the longest ranges allow, all of about the same length; a partition rounds its number
  // of ranges up, so somewhat longer ones are tried before another round is taken (M=12, N=24576 19.9 -> 15.5 us in two).
  const int maxq = mv_max_quarters(M), cus = cu_count();
  for (int slots = cus, done = 0; !done; slots += cus) {
    if (static_cast<int64_t>(slots) * maxq < N / 4) continue;
    for (int want = slots; want > std::max(0, slots - 8) && !done; --want) {
      decode_map(N, pb1, pb2, want, maxq, &map);
      done = map.wg0[3] <= slots;
    }
  }
  const u32x4* wpk = static_cast<const u32x4*>(wpk_d);
  const uint32_t* sz = reinterpret_cast<const uint32_t*>(sz_d);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipError_t launched;
#define PQ_MATVEC_LAUNCH(MR, MX)                                                                                            \
  do {                                                                                                                      \
    auto kern = x_type == PQ_BF16 ? matvec_kernel<true, MR, MX> : matvec_kernel<false, MR, MX>;                             \
    launched = launch_kernel(kern, dim3(map.wg0[3]), dim3(64 * kMvWaves), 0, s, x_d, ldx, M, K, wpk, sz, N, map, y_d, ldy, \
                             y_type == PQ_BF16 ? 1 : 0);                                                                    \
  } while (0)
  if (M == 1) PQ_MATVEC_LAUNCH(1, 1);
  else if (M <= 4) PQ_MATVEC_LAUNCH(4, 4);
  else if (M <= 8) PQ_MATVEC_LAUNCH(4, 8);
  else PQ_MATVEC_LAUNCH(4, 16);
#undef PQ_MATVEC_LAUNCH
  return launch_status(what, launched);
}

}  // extern "C"
