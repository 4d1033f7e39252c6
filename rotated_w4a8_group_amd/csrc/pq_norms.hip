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
// T threads). The row is read once and written once; the two sums of squares are reduced over the
// wave by lane permutations and over the waves through LDS, in an order that depends on the shape
// alone, so results do not change from run to run. Up to 2 chunks per thread every load of the row,
// weights and gate included, is issued before anything waits; at 4 the norm weights are read where
// they are used (from L2: every row reads the same ones), which keeps 1024 threads within 128
// registers each.
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
  int x_bf16, out_bf16, res_bf16;   // 16-bit types: 0 = f16, 1 = bf16
  int gate_cols;                    // K, or 1 (one value per row)
  int gate_act;
  float eps, scale, res_scale, one; // one: 1 for w' = 1 + w, else 0
};

// 8 values of a 16-bit type from 16 loaded bytes.
__device__ __forceinline__ void unpack8(const uint4& q, int bf16, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (bf16) {
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
__device__ __forceinline__ uint4 pack8(const float (&v)[8], int bf16) {
  uint32_t w[4];
  if (bf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16x2_rn(v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f16x2_rn(v[2 * i], v[2 * i + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float gate_value(float t, int act) {
  if (act == PQ_GATE_SIGMOID) return 1.0f / (1.0f + expf(-t));
  if (act == PQ_GATE_TANH) return tanhf(t);
  return t;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <int NC, bool kRes32>
__global__ __launch_bounds__(kNormMaxThreads) void block_norms_kernel(NormArgs a) {
  __shared__ float red[2][kNormMaxThreads / 64];
  const int tid = threadIdx.x, T = blockDim.x, waves = T >> 6, wave = tid >> 6;
  const int64_t m = blockIdx.x;
  const int chunks = a.K >> 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  constexpr bool kLate = NC > 2;
  uint4 xq[NC], rq[NC][kRes32 ? 2 : 1], pq[NC], gq[NC], wq[NC];
  const uint16_t* xr = static_cast<const uint16_t*>(a.x) + m * a.ldx;
  const uint16_t* gr = static_cast<const uint16_t*>(a.gate) + m * a.ldg;
  const bool gate_row = a.gate && a.gate_cols != 1;
  auto weights = [&](const void* w, int c) {
    return c < chunks && w ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + 8 * c) : zero;
  };
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = tid + j * T;
    const bool on = c < chunks;
    xq[j] = on ? *reinterpret_cast<const uint4*>(xr + 8 * c) : zero;
    if constexpr (kRes32) {
      const uint4* rr = reinterpret_cast<const uint4*>(static_cast<const float*>(a.res) + m * a.ldr + 8 * c);
      rq[j][0] = on ? rr[0] : zero;
      rq[j][1] = on ? rr[1] : zero;
    } else {
      rq[j][0] = on ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.res) + m * a.ldr + 8 * c) : zero;
    }
    gq[j] = on && gate_row ? *reinterpret_cast<const uint4*>(gr + 8 * c) : zero;
    if constexpr (!kLate) {
      pq[j] = weights(a.w_post, c);
      wq[j] = weights(a.w_pre, c);
    }
  }
  float g1 = 1.0f;
  if (a.gate && !gate_row) {
    const uint32_t b = gr[0];
    g1 = gate_value(a.x_bf16 ? bf16_to_f32(b) : f16_to_f32(b), a.gate_act);
  }

  // sum over the workgroup, the same value in every thread
  auto total = [&](float s, float* slot) {
    s = wave_sum(s);
    if ((tid & 63) == 0) slot[wave] = s;
    __syncthreads();
    float t = slot[0];
    for (int w = 1; w < waves; ++w) t += slot[w];
    return t;
  };
  auto rstd = [&](float ss) { return 1.0f / __builtin_sqrtf(ss / static_cast<float>(a.K) + a.eps); };

  float v[NC][8];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    unpack8(xq[j], a.x_bf16, v[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += v[j][i] * v[j][i];
  }
  if (a.w_post) {
    const float r = rstd(total(ss, red[0]));
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float w[8];
      unpack8(kLate ? weights(a.w_post, tid + j * T) : pq[j], a.out_bf16, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = (v[j][i] * r) * (a.one + w[i]);
    }
  }
  // h, rounded as it is stored
  float hh = 0.0f;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = tid + j * T;
    float g[8], r[8];
    if (gate_row) {
      unpack8(gq[j], a.x_bf16, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = gate_value(g[i], a.gate_act);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = g1;
    }
    if constexpr (kRes32) {
      const uint32_t w[8] = {rq[j][0].x, rq[j][0].y, rq[j][0].z, rq[j][0].w, rq[j][1].x, rq[j][1].y, rq[j][1].z, rq[j][1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = __builtin_bit_cast(float, w[i]);
    } else {
      unpack8(rq[j][0], a.res_bf16, r);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = a.res_scale * r[i] + a.scale * (v[j][i] * g[i]);
    if constexpr (kRes32) {
      if (c < chunks) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.res_out) + m * a.ldo + 8 * c);
        o[0] = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
        o[1] = make_float4(v[j][4], v[j][5], v[j][6], v[j][7]);
      }
    } else {
      const uint4 o = pack8(v[j], a.res_bf16);
      if (c < chunks) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.res_out) + m * a.ldo + 8 * c) = o;
      unpack8(o, a.res_bf16, v[j]);
    }
    if (c < chunks) {
#pragma unroll
      for (int i = 0; i < 8; ++i) hh += v[j][i] * v[j][i];
    }
  }
  if (!a.w_pre) return;
  const float r = rstd(total(hh, red[1]));
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = tid + j * T;
    float w[8];
    unpack8(kLate ? weights(a.w_pre, c) : wq[j], a.out_bf16, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = (v[j][i] * r) * (a.one + w[i]);
    if (c < chunks) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.hs) + m * a.ldh + 8 * c) = pack8(v[j], a.out_bf16);
  }
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
  if (M == 0) return PQ_OK;
  if (!x_d || !res_d || !res_out_d || (w_pre_d && !hs_d)) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (!aligned(x_d, 16) || !aligned(res_d, 16) || !aligned(res_out_d, 16) || !aligned(w_post_d, 16) || !aligned(w_pre_d, 16) ||
      (w_pre_d && !aligned(hs_d, 16)) || !aligned(gate_d, gate_cols == 1 ? 2 : 16))
    return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  // Outputs may not overlap inputs or each other, but for the residual updated in place (the same rows:
  // a thread writes an element after it has read it, and no other thread reads it).
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
             x_type == PQ_BF16, out_type == PQ_BF16, res_type == PQ_BF16, gate_cols, gate_act,
             eps, scale, res_scale, gemma ? 1.0f : 0.0f};
  const int chunks = K / 8;
  // threads for about two chunks each, at least one wave, and no more chunks per thread than needed
  int nc = 1;
  while (nc < kNormMaxNC && (chunks + nc - 1) / nc > 512) nc *= 2;
  const int threads = ((chunks + nc - 1) / nc + 63) / 64 * 64;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
#define PQ_NORM_LAUNCH(NC)                                                                              \
  do {                                                                                                  \
    auto kern = res_type == PQ_F32 ? block_norms_kernel<NC, true> : block_norms_kernel<NC, false>;      \
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(M)), dim3(threads), 0, s, a);                   \
  } while (0)
  if (nc == 1) PQ_NORM_LAUNCH(1);
  else if (nc == 2) PQ_NORM_LAUNCH(2);
  else PQ_NORM_LAUNCH(4);
#undef PQ_NORM_LAUNCH
  return launch_status(what);
}

}  // extern "C"
