// The norms before and after a block, fused with the block's gate and the residual scale
// (pq_block_norms): per token row
//   n  = x * rstd(x) * w_post'                      (or x where there is no post-norm)
//   h  = fl_R(res_scale * res + scale * a(gate) * n)
//   hs = fl_T(h * rstd(h) * w_pre')                  (absent where there is no pre-norm)
// with rstd(v) = 1 / sqrt(mean_k v^2 + eps), w' = w or 1 + w, everything in binary32 and one rounding
// where h and hs are stored; the second norm reads the stored (rounded) h, as the next block will.
//
// Both norms need the whole row before any of its elements can be written, so a row stays in
// registers: one workgroup per row, thread t holding the 8-element chunks t, t + T, ... (NC of them,
// T threads) of x and res as loaded, then of h as stored. The row is read once and written once; the two sums of
// squares are reduced over the wave by lane permutations and over the waves through LDS, in an order
// that depends on the shape alone, so results do not change from run to run.
//
// Memory bounds it from about 1000 rows on, the latency of load, two reductions and store below. What
// that decided, at M=8192, K=5120 (bf16 x, f16 stream; 335 MB) unless said otherwise:
//  - every load is one 16-byte instruction that every thread issues (the row's last chunk again past its end): 61.0 us
//    (5.5 TB/s) against 71.5 with loads under a condition, which the compiler split into four words; one row 3.35 against 3.8.
//  - x and res as nontemporal loads, h and hs as nontemporal stores: 73 us against 94 with plain loads, 98 with
//    both plain. A f32 stream's loads stay plain (90 against 92 us, M=4096, K=1000 11.9 against 13.7).
//  - norm weights and the gate read where they are used, not with the row: no faster earlier (one row 3.35 against
//    3.45, M=1024 with gate rows and a f32 stream 14.1 against 17.5).
//  - one chunk per thread up to 512 rows and for K <= 2048, else two, more only past 1024 threads. M=512 6.1 / 6.2
//    / 6.6 us with 1, 2, 3 chunks, 1024 rows 11.8 / 8.4 / 9.1, 8192 67.0 / 59.9 / 60.8; M=2048, K=17408 54 with 3, 69
//    with 4; M=9600, K=1024 18.0 / 18.1 / 18.8.
//  - one wave per row (no barriers): 81 us when this kernel took 73; persistent workgroups that keep the weights in
//    registers: 127. Neither kept.
#include <algorithm>

#include "pq_device.h"
#include "pq_internal.h"

namespace pq {

constexpr int kNormMaxNC = 4;                       // chunks of 8 elements per thread
constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxK = 8 * kNormMaxNC * kNormMaxThreads;   // 32768

struct NormArgs {
  const void* x;
  const void* res;
  const void* w_post;    // null: no post-norm
  const void* gate;      // null: no gate
  const void* w_pre;     // null: no pre-norm
  void* res_out;
  void* hs;
  int64_t ldx, ldr, ldg, ldo, ldh;
  int M, K;
  int gate_cols;                    // K, or 1 (one value per row)
  int gate_act;
  float eps, scale, res_scale, one; // one: 1 for w' = 1 + w, else 0
};

typedef uint32_t norm_u32x4 __attribute__((ext_vector_type(4)));

// 8 values of a 16-bit type from 16 loaded bytes.
template <bool kBf16>
__device__ __forceinline__ void unpack8(const norm_u32x4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (kBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = f16_to_f32(w[i]);
      v[2 * i + 1] = f16_to_f32(w[i] >> 16);
    }
  }
}

// 8 values rounded (to nearest even) to a 16-bit type.
template <bool kBf16>
__device__ __forceinline__ norm_u32x4 pack8(const float (&v)[8]) {
  uint32_t w[4];
  if constexpr (kBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16x2_rn(v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f16x2_rn(v[2 * i], v[2 * i + 1]);
  }
  return norm_u32x4{w[0], w[1], w[2], w[3]};
}

// The hardware's exp2 and reciprocal are within 1 ulp (2 u, u = 2^-24). Infinite gates give the functions' limits, NaN stays.
//  - sigmoid: relative error at most (5 + 2 |t|) u, the exponent's two roundings counting |t| each, where it is a normal number
//    (t > -87.3); below, the reciprocal's result is 0. expf and a division made 8192 rows of 5120 with a channel gate 68.4 us,
//    this 61.5; one row with its own gates 4.5, this 3.8.
//  - tanh: below 1/2 its Taylor series to t^13 (the next term is 1.5 u, the sum's roundings 3 u), above 1 - 2 / (1 + exp(2 |t|)),
//    where at 1/2 the quotient's 6 u count 1.2 and the difference rounds once: at most 8 u. tanhf made the 8192 rows
//    67.6 us, this 64.1; the one row 4.6, this 4.2.
__device__ __forceinline__ float gate_value(float t, int act) {
  if (act == PQ_GATE_SIGMOID) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504089f * t));
  if (act == PQ_GATE_TANH) {
    const float x = t * t;
    float p = __builtin_fmaf(x, 21844.0f / 6081075.0f, -1382.0f / 155925.0f);
    p = __builtin_fmaf(x, p, 62.0f / 2835.0f);
    p = __builtin_fmaf(x, p, -17.0f / 315.0f);
    p = __builtin_fmaf(x, p, 2.0f / 15.0f);
    p = __builtin_fmaf(x, p, -1.0f / 3.0f);
    const float low = __builtin_fmaf(t * x, p, t);
    const float high = __builtin_fmaf(-2.0f, __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(2.88539008178f * __builtin_fabsf(t))), 1.0f);
    return __builtin_fabsf(t) < 0.5f ? low : __builtin_copysignf(high, t);
  }
  return t;
}

// 16 bytes, and 16 bytes that nothing reads again before they have left the caches.
__device__ __forceinline__ norm_u32x4 load16(const void* p) { return *reinterpret_cast<const norm_u32x4*>(p); }
__device__ __forceinline__ norm_u32x4 load_nt(const void* p) { return __builtin_nontemporal_load(reinterpret_cast<const norm_u32x4*>(p)); }
__device__ __forceinline__ void store_nt(void* p, const norm_u32x4& v) { __builtin_nontemporal_store(v, reinterpret_cast<norm_u32x4*>(p)); }

__device__ __forceinline__ float wave_sum(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, true));    // pairs
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, true));    // quads
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x141, 0xF, 0xF, true));   // 8 lanes
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x140, 0xF, 0xF, true));   // 16 lanes
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// kX, kO: x and gate, hs and the norm weights are bf16 (else f16); kR: the stream's pq_type.
template <int NC, bool kX, int kR, bool kO>
__global__ __launch_bounds__(kNormMaxThreads) void block_norms_kernel(NormArgs a) {
  constexpr bool kRes32 = kR == PQ_F32;
  constexpr int kMaxWaves = kNormMaxThreads / 64;
  __shared__ __attribute__((aligned(16))) float red[2][kMaxWaves];
  const uint32_t tid = threadIdx.x, T = blockDim.x, waves = T >> 6, wave = tid >> 6;
  const int64_t m = blockIdx.x;
  const uint32_t chunks = static_cast<uint32_t>(a.K) >> 3;
  if (tid < 2 * kMaxWaves && tid % kMaxWaves >= waves) red[tid / kMaxWaves][tid % kMaxWaves] = 0.0f;   // waves that are not there add 0

  // Chunk c = tid + j T of a row; a thread past the row's end loads the last chunk again (every load is
  // issued, without branches), adds nothing to the sums and stores nothing.
  auto chunk = [&](int j) { return tid + j * T; };
  auto at = [&](const void* row, int j, uint32_t bytes) { return static_cast<const uint8_t*>(row) + bytes * min(chunk(j), chunks - 1); };

  norm_u32x4 xq[NC], rq[NC][kRes32 ? 2 : 1];
  const uint16_t* xr = static_cast<const uint16_t*>(a.x) + m * a.ldx;
  const uint16_t* gr = static_cast<const uint16_t*>(a.gate) + m * a.ldg;
  const void* rr = static_cast<const uint8_t*>(a.res) + m * a.ldr * (kRes32 ? 4 : 2);
  const bool gate_row = a.gate && a.gate_cols != 1, gate_one = a.gate && a.gate_cols == 1;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    xq[j] = load_nt(at(xr, j, 16));
    if constexpr (kRes32) {
      rq[j][0] = load16(at(rr, j, 32));
      rq[j][1] = load16(at(rr, j, 32) + 16);
    } else {
      rq[j][0] = load_nt(at(rr, j, 16));
    }
  }
  uint32_t g1q = 0;
  if (gate_one) g1q = gr[0];

  // sum over the row's threads, the same value in every one: the waves' sums in order
  auto total = [&](float s, float* slot) {
    s = wave_sum(s);
    if ((tid & 63) == 0) slot[wave] = s;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kMaxWaves; w += 4) {
      const float4 q = *reinterpret_cast<const float4*>(slot + w);
      t = (((t + q.x) + q.y) + q.z) + q.w;
    }
    return t;
  };
  auto rstd = [&](float ss) { return 1.0f / __builtin_sqrtf(ss / static_cast<float>(a.K) + a.eps); };

  float rx = 1.0f;
  if (a.w_post) {
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float v[8], s = ss;
      unpack8<kX>(xq[j], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i] * v[i];
      ss = chunk(j) < chunks ? s : ss;
    }
    rx = rstd(total(ss, red[0]));
  }
  norm_u32x4 wq[NC], gq[NC];   // before the stores to res_out, which the compiler lets no load pass
  if (a.w_post) {
#pragma unroll
    for (int j = 0; j < NC; ++j) wq[j] = load16(at(a.w_post, j, 16));
  }
  if (gate_row) {
#pragma unroll
    for (int j = 0; j < NC; ++j) gq[j] = load16(at(gr, j, 16));
  }
  const float g1 = gate_one ? gate_value(kX ? bf16_to_f32(g1q) : f16_to_f32(g1q), a.gate_act) : 1.0f;
  // h, rounded as it is stored
  float hh = 0.0f;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const uint32_t c = chunk(j);
    float v[8], r[8];
    unpack8<kX>(xq[j], v);
    if (a.w_post) {
      float w[8];
      unpack8<kO>(wq[j], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (v[i] * rx) * (a.one + w[i]);
    }
    if (gate_row) {
      float g[8];
      unpack8<kX>(gq[j], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= gate_value(g[i], a.gate_act);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= g1;
    }
    if constexpr (kRes32) {
      const uint32_t w[8] = {rq[j][0].x, rq[j][0].y, rq[j][0].z, rq[j][0].w, rq[j][1].x, rq[j][1].y, rq[j][1].z, rq[j][1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = __builtin_bit_cast(float, w[i]);
    } else {
      unpack8<kR == PQ_BF16>(rq[j][0], r);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = a.res_scale * r[i] + a.scale * v[i];
    if constexpr (kRes32) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __builtin_bit_cast(uint32_t, v[i]);
      rq[j][0] = norm_u32x4{w[0], w[1], w[2], w[3]};
      rq[j][1] = norm_u32x4{w[4], w[5], w[6], w[7]};
      if (c < chunks) {
        float* o = static_cast<float*>(a.res_out) + m * a.ldo + 8 * c;
        store_nt(o, rq[j][0]);
        store_nt(o + 4, rq[j][1]);
      }
    } else {
      rq[j][0] = pack8<kR == PQ_BF16>(v);
      if (c < chunks) store_nt(static_cast<uint16_t*>(a.res_out) + m * a.ldo + 8 * c, rq[j][0]);
      unpack8<kR == PQ_BF16>(rq[j][0], v);
    }
    float s = hh;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i] * v[i];
    hh = c < chunks ? s : hh;
  }
  if (!a.w_pre) return;
#pragma unroll
  for (int j = 0; j < NC; ++j) wq[j] = load16(at(a.w_pre, j, 16));
  const float rh = rstd(total(hh, red[1]));
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const uint32_t c = chunk(j);
    float v[8], w[8];
    if constexpr (kRes32) {
      const uint32_t q[8] = {rq[j][0].x, rq[j][0].y, rq[j][0].z, rq[j][0].w, rq[j][1].x, rq[j][1].y, rq[j][1].z, rq[j][1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __builtin_bit_cast(float, q[i]);
    } else {
      unpack8<kR == PQ_BF16>(rq[j][0], v);
    }
    unpack8<kO>(wq[j], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (v[i] * rh) * (a.one + w[i]);
    if (c < chunks) store_nt(static_cast<uint16_t*>(a.hs) + m * a.ldh + 8 * c, pack8<kO>(v));
  }
}

// Chunks per thread (one, or two for long rows where there are more rows than two a CU) and threads per row.
static void norms_shape(int M, int K, int* nc, int* threads) {
  const int chunks = K / 8, least = (chunks + kNormMaxThreads - 1) / kNormMaxThreads;
  *nc = std::max(least, M > 512 && chunks > 256 ? 2 : 1);
  *threads = ((chunks + *nc - 1) / *nc + 63) / 64 * 64;
}

template <bool kX, int kR, bool kO>
static hipError_t norms_launch(const NormArgs& a, hipStream_t s) {
  int nc, threads;
  norms_shape(a.M, a.K, &nc, &threads);
#define PQ_NORM_LAUNCH(NC) \
  return launch_kernel((block_norms_kernel<NC, kX, kR, kO>), dim3(static_cast<unsigned>(a.M)), dim3(threads), 0, s, a)
  if (nc == 1) PQ_NORM_LAUNCH(1);
  if (nc == 2) PQ_NORM_LAUNCH(2);
  if (nc == 3) PQ_NORM_LAUNCH(3);
  PQ_NORM_LAUNCH(4);
#undef PQ_NORM_LAUNCH
}
template <bool kX, int kR>
static hipError_t norms_for_out(const NormArgs& a, int out_type, hipStream_t s) {
  return out_type == PQ_BF16 ? norms_launch<kX, kR, true>(a, s) : norms_launch<kX, kR, false>(a, s);
}
template <bool kX>
static hipError_t norms_for_res(const NormArgs& a, int res_type, int out_type, hipStream_t s) {
  if (res_type == PQ_F32) return norms_for_out<kX, PQ_F32>(a, out_type, s);
  return res_type == PQ_BF16 ? norms_for_out<kX, PQ_BF16>(a, out_type, s) : norms_for_out<kX, PQ_F16>(a, out_type, s);
}
static hipError_t norms_for_x(const NormArgs& a, int x_type, int res_type, int out_type, hipStream_t s) {
  return x_type == PQ_BF16 ? norms_for_res<true>(a, res_type, out_type, s) : norms_for_res<false>(a, res_type, out_type, s);
}

// Whether any byte of the M rows of `wa` bytes every `lda` bytes at a is one of b's rows. Exact where
// the strides agree (two column ranges of one buffer do not overlap); else by the whole ranges.
static bool rows_overlap(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb, int64_t M) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + static_cast<uintptr_t>((M - 1) * lda + wa), b1 = b0 + static_cast<uintptr_t>((M - 1) * ldb + wb);
  if (a1 <= b0 || b1 <= a0) return false;
  if (lda != ldb || lda <= 0) return true;
  const int64_t d = static_cast<int64_t>(b0 > a0 ? b0 - a0 : a0 - b0) % lda;
  const int64_t off = b0 > a0 ? d : (lda - d) % lda;   // b's rows start `off` bytes into a's
  return off < wa || off + wb > lda;
}

}  // namespace pq

extern "C" {

int pq_block_norms(const void* x_d, int64_t ldx, int x_type, const void* res_d, int64_t ldr, int res_type,
                   const void* w_post_d, const void* gate_d, int64_t ldg, int gate_cols, int gate_act,
                   const void* w_pre_d, float eps, float scale, float res_scale, int gemma, int M, int K,
                   void* res_out_d, int64_t ldo, void* hs_d, int64_t ldh, int out_type, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_block_norms";
  if (M < 0) return set_error(PQ_ERR_SHAPE, "%s: M=%d < 0", what, M);
  if (K <= 0 || K % 8 || K > kNormMaxK)
    return set_error(PQ_ERR_SHAPE, "%s: K=%d must be a positive multiple of 8, at most %d", what, K, kNormMaxK);
  if ((x_type != PQ_F16 && x_type != PQ_BF16) || (out_type != PQ_F16 && out_type != PQ_BF16) ||
      (res_type != PQ_F16 && res_type != PQ_BF16 && res_type != PQ_F32))
    return set_error(PQ_ERR_SHAPE, "%s: types (x %d, res %d, out %d): x and out f16 or bf16, res f16, bf16 or f32", what,
                     x_type, res_type, out_type);
  if (gate_act != PQ_GATE_NONE && gate_act != PQ_GATE_SIGMOID && gate_act != PQ_GATE_TANH)
    return set_error(PQ_ERR_SHAPE, "%s: gate_act=%d", what, gate_act);
  if (!(eps > 0.0f) || !(eps < __builtin_inff())) return set_error(PQ_ERR_SHAPE, "%s: eps must be positive and finite", what);
  const int rstep = res_type == PQ_F32 ? 4 : 8;   // rows of 16-byte aligned chunks
  if (ldx < K || ldr < K || ldo < K || ldx % 8 || ldr % rstep || ldo % rstep || (w_pre_d && (ldh < K || ldh % 8)))
    return set_error(PQ_ERR_SHAPE, "%s: row strides must be >= K=%d and whole 16-byte steps", what, K);
  if (gate_d) {
    if (gate_cols != K && gate_cols != 1) return set_error(PQ_ERR_SHAPE, "%s: gate_cols=%d must be K=%d or 1", what, gate_cols, K);
    if (ldg < 0 || (gate_cols == K && (ldg % 8 || (ldg && ldg < K))))
      return set_error(PQ_ERR_SHAPE, "%s: gate row stride %lld", what, static_cast<long long>(ldg));
  }
  int nc, threads;
  norms_shape(M, K, &nc, &threads);
  if (static_cast<int64_t>(M) * threads > 0xFFFFFFFFll)   // the runtime counts a launch's threads in 32 bits
    return set_error(PQ_ERR_SHAPE, "%s: M=%d rows too many for one call (split the rows)", what, M);
  if (M == 0) return PQ_OK;
  if (!x_d || !res_d || !res_out_d || (w_pre_d && !hs_d)) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (!aligned(x_d, 16) || !aligned(res_d, 16) || !aligned(res_out_d, 16) || !aligned(w_post_d, 16) || !aligned(w_pre_d, 16) ||
      (w_pre_d && !aligned(hs_d, 16)) || !aligned(gate_d, gate_cols == 1 ? 2 : 16))
    return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  // Outputs may not overlap inputs or each other, but for the residual updated in place (the same rows:
  // a thread writes an element after it has read it, and what other threads may read of it, past the row's
  // end of their own, they do not use).
  const int64_t rb = res_type == PQ_F32 ? 4 : 2, kr = rb * K, k2 = 2 * static_cast<int64_t>(K);
  const bool inplace = res_out_d == res_d && ldo == ldr;
  auto clashes = [&](const void* p, int64_t ld, int64_t width, const void* o, int64_t lo, int64_t wo) {
    // a broadcast row (ld 0) is one row against the whole output
    if (!p) return false;
    if (ld == 0) {
      const uintptr_t p0 = reinterpret_cast<uintptr_t>(p), o0 = reinterpret_cast<uintptr_t>(o);
      return p0 < o0 + static_cast<uintptr_t>((M - 1) * lo + wo) && o0 < p0 + static_cast<uintptr_t>(width);
    }
    return rows_overlap(p, ld, width, o, lo, wo, M);
  };
  const int64_t gw = 2 * static_cast<int64_t>(gate_cols);
  bool clash = !inplace && clashes(res_d, rb * ldr, kr, res_out_d, rb * ldo, kr);
  clash = clash || clashes(x_d, 2 * ldx, k2, res_out_d, rb * ldo, kr) || clashes(gate_d, 2 * ldg, gw, res_out_d, rb * ldo, kr) ||
          clashes(w_post_d, 0, k2, res_out_d, rb * ldo, kr) || clashes(w_pre_d, 0, k2, res_out_d, rb * ldo, kr);
  if (w_pre_d)
    clash = clash || clashes(x_d, 2 * ldx, k2, hs_d, 2 * ldh, k2) || clashes(res_d, rb * ldr, kr, hs_d, 2 * ldh, k2) ||
            clashes(res_out_d, rb * ldo, kr, hs_d, 2 * ldh, k2) || clashes(gate_d, 2 * ldg, gw, hs_d, 2 * ldh, k2) ||
            clashes(w_post_d, 0, k2, hs_d, 2 * ldh, k2) || clashes(w_pre_d, 0, k2, hs_d, 2 * ldh, k2);
  if (clash) return set_error(PQ_ERR_SHAPE, "%s: an output overlaps an input or the other output", what);

  NormArgs a{x_d, res_d, w_post_d, gate_d, w_pre_d, res_out_d, hs_d, ldx, ldr, ldg, ldo, ldh, M, K,
             gate_cols, gate_act, eps, scale, res_scale, gemma ? 1.0f : 0.0f};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return launch_status(what, norms_for_x(a, x_type, res_type, out_type, s));
}

}  // extern "C"
