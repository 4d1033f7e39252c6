// Attention over packed prompts (pq_attn_prefill): o[h] = sum_j softmax_j(scale q[h] . k_j) v_j, causal, grouped heads.
//
// One pass over the keys with a running maximum and sum. A wave owns 32 queries of one head and walks the keys in tiles that
// the workgroup's waves share through LDS. Both products run on the matrix core transposed, so that a lane
// owns one query throughout:
//   S^T = K Q^T   (32x32x16: keys x channels times channels x queries); lane l holds query l % 32, and of 32 keys the 16
//                 with bit 2 equal to l / 32 - the maximum and the sum are in-lane but for one exchange of the wave's halves;
//   O^T = V^T P^T (channels x keys times keys x queries): P^T is needed with 8 keys a lane, and as the order of the keys in
//                 the contraction is free, a lane's own 8 are taken as they lie - P never leaves its registers - and V^T
//                 follows that order: two transposing LDS reads of 4 keys each per 16 keys and 32 channels.
// Scores, sums and O are binary32. P is rounded to v's type for the second product (half a step of it, 2^-8 or 2^-11 of each
// weight); the sum takes the unrounded p.
//
// K and V tiles go global -> LDS by direct loads, row-major with the 16-byte chunks of a row permuted (kswizzle, vswizzle) so
// that the 16 lanes of an operand read, and the 4 keys of a transposing one, lie in different banks.
//
// The maximum that p is taken against is raised only when a score passes it by more than 2^8 (a wave-wide vote): p stays below
// 2^8, and the 16 D / 32 multiplications of O are rare. Keys that a query does not see get the score -inf, in the tiles
// that need it only. Their values still enter the product, with weight 0: a row whose result is not finite is
// recomputed key by key (attend_row), so that an infinity or a NaN in a row that it does not see cannot reach it.
#include <algorithm>

#include "pq_attn.h"

namespace pq {

typedef float f32x16 __attribute__((ext_vector_type(16)));

struct PrefillArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t ldq, hsq, ldk, hsk, ldv, hsv;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk, Hq, Hkv, causal;
  float scale_log2;
  uint16_t* o;
  int out_type;
};

// What a workgroup works on: rows r0 .. of sequence b, whose queries start at q0 (nq of them) and keys at k0 (nk of them).
struct PrefillItem {
  int r0, q0, nq, k0, nk;
};

template <bool kBf16>
__device__ __forceinline__ f32x16 mfma_32(const attn_u32x4& a, const attn_u32x4& b, const f32x16& c) {
  if constexpr (kBf16) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <int D>
struct PrefillTile {
  static constexpr int kWaves = 4;
  static constexpr int kRows = 32 * kWaves;             // queries of a workgroup
  static constexpr int kKeys = D == 256 ? 32 : 64;      // keys of a tile
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kChunks = D / 8;                 // 16-byte chunks of a row
  static constexpr int kPart = kKeys * kRowBytes;       // bytes of K, or of V, of one tile
  static constexpr int kLds = 2 * 2 * kPart;
  static constexpr int kLoads = kPart / 1024 / kWaves;  // direct loads a wave makes for K, or for V

  // The place of chunk c of row r: 16 rows (a K read: the same chunk of 16 rows) and 4 rows (a V read: 64 bytes of each) in
  // different banks of the 256-byte line.
  static __device__ __forceinline__ int kswizzle(int r) { return D == 64 ? (r >> 1) & 7 : r & 15; }
  static __device__ __forceinline__ int vswizzle(int r) { return D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2; }
};

// One row key by key, exactly as the formula reads: keys j < keys.
template <int D, bool kBf16>
__device__ __attribute__((noinline)) void attend_row(const PrefillArgs& a, int64_t t, int hq, int k0, int keys) {
  const int h = hq / (a.Hq / a.Hkv);
  float q[D / 64], k[D / 64], v[D / 64];
  lane_values<D, kBf16>(a.q + t * a.ldq + hq * a.hsq, q);
  RowState<D> r;
  for (int j = 0; j < keys; ++j) {
    lane_values<D, kBf16>(a.k + static_cast<int64_t>(k0 + j) * a.ldk + h * a.hsk, k);
    lane_values<D, kBf16>(a.v + static_cast<int64_t>(k0 + j) * a.ldv + h * a.hsv, v);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) s += q[i] * k[i];
    r.add(lanes_sum(s), a.scale_log2, v);
  }
  store_row<D>(a.o + (t * a.Hq + hq) * D, r, keys > 0, a.out_type);
}

// The item of tile number `tile` (rows of kRows; a sequence's tiles from its end, where a causal one is longest): false past the last.
template <int kRows>
__device__ __forceinline__ bool find_item(const PrefillArgs& a, int tile, PrefillItem* it) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int b = b0 + lane;
    int q0 = 0, nq = 0;
    if (b < a.B) {
      q0 = std::min(std::max(a.cu_q[b], 0), a.Tq);
      nq = std::max(std::min(a.cu_q[b + 1], a.Tq) - q0, 0);
    }
    const int n = (nq + kRows - 1) / kRows;
    int sum = n;   // inclusive prefix sum
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const int o = __shfl_up(sum, m);
      sum += lane >= m ? o : 0;
    }
    const uint64_t here = __ballot(before + sum > tile);
    if (here) {
      const int first = __builtin_ctzll(here);
      const int at = tile - before - (__builtin_amdgcn_readlane(sum, first) - __builtin_amdgcn_readlane(n, first));
      const int s = b0 + first;
      it->q0 = __builtin_amdgcn_readlane(q0, first);
      it->nq = __builtin_amdgcn_readlane(nq, first);
      it->r0 = (__builtin_amdgcn_readlane(n, first) - 1 - at) * kRows;
      it->k0 = __builtin_amdgcn_readfirstlane(std::min(std::max(a.cu_k[s], 0), a.Tk));
      it->nk = __builtin_amdgcn_readfirstlane(std::max(std::min(a.cu_k[s + 1], a.Tk) - it->k0, 0));
      return true;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

template <int D, bool kBf16>
__global__ __launch_bounds__(256, 2) void attn_prefill_kernel(PrefillArgs a) {
  using Tile = PrefillTile<D>;
  constexpr int kDB = D / 32, kKB = Tile::kKeys / 32, kSteps = D / 16;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Tile::kLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 31, half = lane >> 5;

  // Workgroup -> (tile, head). Workgroups go round the 8 XCDs, so with Hq a multiple of 8 each XCD keeps its own Hq / 8 heads (the
  // queries that share a key head meet in one L2).
  int hq, tile;
  if (a.Hq % 8 == 0) {
    const int per = a.Hq / 8, i = blockIdx.x >> 3;
    hq = (blockIdx.x & 7) * per + i % per;
    tile = i / per;
  } else {
    hq = blockIdx.x % a.Hq;
    tile = blockIdx.x / a.Hq;
  }
  PrefillItem it;
  if (!find_item<Tile::kRows>(a, tile, &it)) return;
  const int h = hq / (a.Hq / a.Hkv);
  const int shift = a.causal ? it.nk - it.nq + 1 : it.nk;              // row r sees min(nk, r + shift) keys (causal)
  const int row = it.r0 + 32 * wave + n;                               // this lane's query; rows past the end repeat the last
  const int seen = a.causal ? std::max(std::min(it.nk, std::min(row, it.nq - 1) + shift), 0) : it.nk;
  const int last_row = std::min(it.r0 + Tile::kRows, it.nq) - 1;
  const int keys = a.causal ? std::max(std::min(it.nk, last_row + shift), 0) : it.nk;
  const int tiles = (keys + Tile::kKeys - 1) / Tile::kKeys;
  // of this wave's rows: the fewest and the most keys that one sees
  const int wr0 = std::min(it.r0 + 32 * wave, it.nq - 1), wr1 = std::min(it.r0 + 32 * wave + 31, it.nq - 1);
  const int least = a.causal ? std::max(std::min(it.nk, wr0 + shift), 0) : it.nk;
  const int most = it.r0 + 32 * wave >= it.nq ? 0 : a.causal ? std::max(std::min(it.nk, wr1 + shift), 0) : it.nk;

  // queries: channels 16 s + 8 half .. + 7 of step s
  attn_u32x4 q[kSteps];
  {
    const uint16_t* p = a.q + static_cast<int64_t>(it.q0 + std::min(row, it.nq - 1)) * a.ldq + hq * a.hsq + 8 * half;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const attn_u32x4*>(p + 16 * s);
  }

  const uint16_t* kbase = a.k + static_cast<int64_t>(it.k0) * a.ldk + h * a.hsk;
  const uint16_t* vbase = a.v + static_cast<int64_t>(it.k0) * a.ldv + h * a.hsv;
  const uint32_t lds0 = lds_addr(smem);
  // Direct loads of tile j into buffer j % 2: load i of a wave fills 1 KiB, 64 chunks in LDS order; rows past the last key repeat it.
  auto load = [&](int j) {
    const int left = it.nk - j * Tile::kKeys - 1;
    const void* kb = scalar_addr(kbase + static_cast<int64_t>(j) * Tile::kKeys * a.ldk);
    const void* vb = scalar_addr(vbase + static_cast<int64_t>(j) * Tile::kKeys * a.ldv);
    const uint32_t to = lds0 + (j & 1) * 2 * Tile::kPart;
#pragma unroll
    for (int i = 0; i < Tile::kLoads; ++i) {
      const int piece = wave * Tile::kLoads + i, at = piece * 64 + lane, r = at / Tile::kChunks, c = at % Tile::kChunks;
      const uint32_t from = static_cast<uint32_t>(std::min(r, left));
      lds_dma16_s(kb, (from * static_cast<uint32_t>(a.ldk) + 8 * (c ^ Tile::kswizzle(r))) * 2, to + piece * 1024);
    }
#pragma unroll
    for (int i = 0; i < Tile::kLoads; ++i) {
      const int piece = wave * Tile::kLoads + i, at = piece * 64 + lane, r = at / Tile::kChunks, c = at % Tile::kChunks;
      const uint32_t from = static_cast<uint32_t>(std::min(r, left));
      lds_dma16_s(vb, (from * static_cast<uint32_t>(a.ldv) + 8 * (c ^ Tile::vswizzle(r))) * 2, to + Tile::kPart + piece * 1024);
    }
  };

  f32x16 o[kDB] = {};
  float m = -__builtin_inff(), mc = 0.0f, l = 0.0f;   // the maximum that p is taken against, m * c, the sum of this lane's keys
  const float c = a.scale_log2;

  if (tiles > 0) load(0);
  for (int j = 0; j < tiles; ++j) {
    // this wave's loads of tile j have landed and its reads of tile j - 1 are done; behind the barrier every wave's
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (j + 1 < tiles) load(j + 1);
    const int k0 = j * Tile::kKeys;
    if (k0 >= most) continue;                          // nothing here for this wave's rows
    const uint8_t* kt = smem + (j & 1) * 2 * Tile::kPart;
    const uint8_t* vt = kt + Tile::kPart;

    f32x16 s[kKB];
#pragma unroll
    for (int kb = 0; kb < kKB; ++kb) {
      s[kb] = f32x16{};
      const int r = 32 * kb + n;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const attn_u32x4 k = *reinterpret_cast<const attn_u32x4*>(kt + r * Tile::kRowBytes + 16 * ((2 * st + half) ^ Tile::kswizzle(r)));
        s[kb] = mfma_32<kBf16>(k, q[st], s[kb]);
      }
    }
    if (k0 + Tile::kKeys > least) {
      const int limit = seen - k0 - 4 * half;
#pragma unroll
      for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][i] = 32 * kb + (i & 3) + 8 * (i >> 2) < limit ? s[kb][i] : -__builtin_inff();
    }
    float mt = s[0][0];
#pragma unroll
    for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) mt = __builtin_fmaxf(mt, s[kb][i]);
    mt = __builtin_fmaxf(both_halves_max(mt), m);
    if (__any((mt - m) * c > 8.0f)) {
      const float f = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m * c - mt * c);
      m = mt;
      mc = m == -__builtin_inff() ? 0.0f : m * c;
      l *= f;
#pragma unroll
      for (int db = 0; db < kDB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] *= f;
    }
    uint32_t p[kKB][8];
#pragma unroll
    for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], c, -mc)), y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i + 1], c, -mc));
        l += x + y;
        p[kb][i / 2] = pack2<kBf16>(x, y);
      }
#pragma unroll
    for (int kb = 0; kb < 2 * kKB; ++kb) {             // 16 keys each
      const attn_u32x4 w = {p[kb / 2][4 * (kb % 2)], p[kb / 2][4 * (kb % 2) + 1], p[kb / 2][4 * (kb % 2) + 2], p[kb / 2][4 * (kb % 2) + 3]};
      const int r = 16 * kb + 4 * half + ((lane & 15) >> 2);   // this lane's key of the first transposing read; r + 8 of the second
#pragma unroll
      for (int db = 0; db < kDB; ++db) {
        const int ch = 4 * db + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), byte = 8 * (lane & 1);
        const uint2 v0 = lds_read_transposed(vt + r * Tile::kRowBytes + 16 * (ch ^ Tile::vswizzle(r)) + byte);
        const uint2 v1 = lds_read_transposed(vt + (r + 8) * Tile::kRowBytes + 16 * (ch ^ Tile::vswizzle(r + 8)) + byte);
        o[db] = mfma_32<kBf16>(attn_u32x4{v0.x, v0.y, v1.x, v1.y}, w, o[db]);
      }
    }
  }

  l = both_halves_sum(l);
  // Rows that saw a key and whose values are not all finite: key by key. (A sum of 0 has every score at -inf: NaN by the formula.)
  float t = l > 0.0f ? 0.0f : __builtin_nanf("");
#pragma unroll
  for (int db = 0; db < kDB; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) t = __builtin_fmaf(o[db][i], 0.0f, t);
  const uint64_t odd = __ballot(seen > 0 && row < it.nq && !(t == 0.0f));
  const uint32_t again = static_cast<uint32_t>(odd | odd >> 32);
  const float inv = seen > 0 ? 1.0f / l : 0.0f;
  if (row < it.nq && !(again >> n & 1)) {
    uint16_t* out = a.o + (static_cast<int64_t>(it.q0 + row) * a.Hq + hq) * D;
#pragma unroll
    for (int db = 0; db < kDB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g) {                    // channels 32 db + 8 g + 4 half .. + 3
        const float x[4] = {o[db][4 * g] * inv, o[db][4 * g + 1] * inv, o[db][4 * g + 2] * inv, o[db][4 * g + 3] * inv};
        const uint2 w = a.out_type == PQ_BF16 ? make_uint2(pack2<true>(x[0], x[1]), pack2<true>(x[2], x[3])) : make_uint2(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]));
        *reinterpret_cast<uint2*>(out + 32 * db + 8 * g + 4 * half) = w;
      }
  }
  for (uint32_t left = again; left; left &= left - 1) {
    const int r = it.r0 + 32 * wave + __builtin_ctz(left);
    attend_row<D, kBf16>(a, it.q0 + r, hq, it.k0, a.causal ? std::max(std::min(it.nk, r + shift), 0) : it.nk);
  }
}

template <int D>
static hipError_t prefill_launch(const PrefillArgs& a, int type, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.Tq / PrefillTile<D>::kRows + a.B) * static_cast<int64_t>(a.Hq))), block(256);
  return type == PQ_BF16 ? launch_kernel((attn_prefill_kernel<D, true>), grid, block, 0, s, a)
                         : launch_kernel((attn_prefill_kernel<D, false>), grid, block, 0, s, a);
}

}  // namespace pq

extern "C" {

size_t pq_attn_prefill_workspace_bytes(int B, int Tq, int Tk, int Hq, int Hkv, int D) { return 0; }

int pq_attn_prefill(const uint16_t* q_d, int64_t ldq, int64_t hsq, const uint16_t* k_d, int64_t ldk, int64_t hsk, const uint16_t* v_d, int64_t ldv,
                    int64_t hsv, int type, const int32_t* cu_q_d, const int32_t* cu_k_d, int B, int Tq, int Tk, int Hq, int Hkv, int D, float scale,
                    int causal, uint16_t* o_d, int out_type, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_attn_prefill";
  if (B < 0 || Tq < 0 || Tk < 0) return set_error(PQ_ERR_SHAPE, "%s: B=%d, Tq=%d, Tk=%d: negative", what, B, Tq, Tk);
  int rc = check_attention(what, type, out_type, Hq, Hkv, D, scale);
  if (rc == PQ_OK) rc = check_heads(what, "q", q_d, ldq, hsq, Tq, Hq, D);
  if (rc == PQ_OK) rc = check_heads(what, "k", k_d, ldk, hsk, Tk, Hkv, D);
  if (rc == PQ_OK) rc = check_heads(what, "v", v_d, ldv, hsv, Tk, Hkv, D);
  if (rc != PQ_OK) return rc;
  if ((Tq / 128 + static_cast<int64_t>(B)) * Hq * 256 > 0xFFFFFFFFll)   // the runtime counts a launch's threads in 32 bits
    return set_error(PQ_ERR_SHAPE, "%s: Tq=%d rows of B=%d sequences too many for one call", what, Tq, B);
  if (Tq == 0 || B == 0) return PQ_OK;
  if (!o_d || !cu_q_d || !cu_k_d) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (!aligned(o_d, 16) || !aligned(cu_q_d, 4) || !aligned(cu_k_d, 4)) return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  PrefillArgs a{q_d, k_d, v_d, ldq, hsq, ldk, hsk, ldv, hsv, cu_q_d, cu_k_d, B, Tq, Tk, Hq, Hkv, causal, scale * 1.44269504088896340736f, o_d, out_type};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return launch_status(what, D == 64 ? prefill_launch<64>(a, type, s) : D == 128 ? prefill_launch<128>(a, type, s) : prefill_launch<256>(a, type, s));
}

}  // extern "C"
