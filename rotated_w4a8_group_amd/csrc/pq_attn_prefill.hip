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
// weight, and 2^-32 of the largest for f16: kF16Lift), which is what the output's own rounding costs. Only where o is f16 and v bf16 would it be the larger by far (6.6e-4 of the norm
// against 1.9e-4): there P is held in two bf16 pieces (2^-16), each with a product of its own, for 28 to 38 % more time (9 packed
// prompts 93 -> 119 us, 8192 rows 762 -> 1053, 512 of 256 channels behind 8191 126 -> 165, 4096 rows of 24 heads of 64 71 -> 97; f16 inputs
// 96, 811, 133.5, 73.5). Figures beside each other here and below are of one run; runs on other boards differ by up to 8 %.
//
// K and V tiles go global -> LDS by direct loads, row-major with the 16-byte chunks of a row permuted (kswizzle, vswizzle) so
// that the 16 lanes of an operand read, and the 4 keys of a transposing one, lie in different banks.
//
// The score m that p = exp2(c (s - m)) is taken against is the largest of the first tile and is raised only where the weights of a
// tile pass what their type holds (their sum 2^60, or an f16 one its type: a wave-wide vote): the softmax does not depend
// on m, sums and O are binary32, and neither the maximum nor a rescaling of O is part of an ordinary tile. The sum takes the rounded p, so
// a rounding moves weight between values and leaves their sum at 1. Keys that a query does not see get the score -inf, in the tiles
// that need it only. Their values still enter the product, with weight 0: a row whose result is not finite is
// recomputed key by key (attend_row), so that an infinity or a NaN in a row that it does not see cannot reach it.
#include <algorithm>
#include <utility>

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
  int items;     // places for a head's items
  int pieces;    // pieces that a head's key tiles are cut into, about; 0: items are whole
  float* ws;
};

// What a workgroup works on: rows r0 .. of a sequence whose queries start at q0 (nq of them) and keys at k0 (nk of them), and of the
// items' key tiles the `piece`th of `pieces` parts.
struct PrefillItem {
  int r0, q0, nq, k0, nk, piece, pieces, place;   // place: of the first piece
  // Keys that row r sees.
  __device__ __forceinline__ int keys(int r, bool causal) const { return causal ? std::max(std::min(nk, r + nk - nq + 1), 0) : nk; }
};

template <bool kBf16>
__device__ __forceinline__ f32x16 mfma_32(const attn_u32x4& a, const attn_u32x4& b, const f32x16& c) {
  if constexpr (kBf16) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// log2 of what f16 weights are taken times, which divides out: f16 reaches down to 2^-24 and up to 2^16, and the largest score of the first
// tile would be 1. What rounding takes from a small weight is then 2^-32 of the largest at most, less than the output's rounding beside 1e6 such
// keys. (0, 7, 10, 13: 8192 rows of 48 heads of 128 810, 821, 830, 859 us; 9 packed prompts 95, 97, 99, 103; later maxima pass what
// is left above sooner, and a tile's weights are taken twice.)
constexpr float kF16Lift = 7.0f;

// a b, rounded to binary32 and not fused with what follows.
__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

// Four packed values, or zeros where the mask is 0: a factor of 0 would leave a NaN.
__device__ __forceinline__ uint2 kept(const uint2& v, uint32_t mask) { return make_uint2(v.x & mask, v.y & mask); }

// Key tiles of a piece, at least. (4, 8, 16: 256 rows behind 1280 keys, 24 heads of 128 23.8, 23.3, 26.2 us; 8 heads of 256 25.6, 26.1,
// 32.6; 64 behind 1500, 12 of 64 15.0, 14.9, 19.2.)
constexpr int kLeastTiles = 8;

// Two buffers of K and V are 64 KB, 32 at 64 channels, and the registers are a wave's of two a SIMD: one workgroup's softmax runs under
// the other's products. (256 channels with one wave a SIMD and 64 keys, before the pieces filled the places: 512 rows behind 8191 keys
// 183 us against 167.)
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
  static constexpr int kSlot = (D + 2) * kRows;         // floats of a piece in the workspace

  // The place of chunk c of row r: 16 rows (a K read: the same chunk of 16 rows) and 4 rows (a V read: 64 bytes of each) in
  // different banks of the 256-byte line.
  static __device__ __forceinline__ int kswizzle(int r) { return D == 64 ? (r >> 1) & 7 : r & 15; }
  static __device__ __forceinline__ int vswizzle(int r) { return D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2; }
};

// One row key by key, exactly as the formula reads: keys j < keys, four of them loaded together. A query that is not finite has no
// finite weight: its result is NaN. This is for the rare row, a wave each, and slow: a NaN in the first value of 8192 rows, which all rows of its 6
// query heads see, makes 306 ms of 0.8, in the first of 2048 23 ms of 0.08; an infinity in the last of 8192, which the rows of its tile load, 97.
template <int D, bool kBf16>
__device__ __forceinline__ void attend_row(const PrefillArgs& a, int64_t t, int hq, int k0, int keys) {
  const int h = hq / (a.Hq / a.Hkv);
  float q[D / 64], k[4][D / 64], v[4][D / 64];
  lane_values<D, kBf16>(a.q + t * a.ldq + hq * a.hsq, q);
  float finite = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) finite = __builtin_fmaf(q[i], 0.0f, finite);
  finite = lanes_sum(finite);
  RowState<D> r;
  if (!(finite == 0.0f)) r.l = finite;
  for (int j0 = 0; j0 < (finite == 0.0f ? keys : 0); j0 += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = k0 + std::min(j0 + j, keys - 1);
      lane_values<D, kBf16>(a.k + row * a.ldk + h * a.hsk, k[j]);
      lane_values<D, kBf16>(a.v + row * a.ldv + h * a.hsv, v[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j0 + j >= keys) break;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) s += q[i] * k[j][i];
      r.add(lanes_sum(s), a.scale_log2, v[j]);
    }
  }
  store_row<D>(a.o + (t * a.Hq + hq) * D, r, keys > 0, a.out_type);
}

// Sequence b's queries and keys, clamped to the rows that exist.
struct Sequence {
  int q0, nq, k0, nk;
  __device__ __forceinline__ Sequence(const PrefillArgs& a, int b) : q0(0), nq(0), k0(0), nk(0) {
    if (b < a.B) {
      q0 = std::min(std::max(a.cu_q[b], 0), a.Tq);
      nq = std::max(std::min(a.cu_q[b + 1], a.Tq) - q0, 0);
      k0 = std::min(std::max(a.cu_k[b], 0), a.Tk);
      nk = std::max(std::min(a.cu_k[b + 1], a.Tk) - k0, 0);
    }
  }
};

// The item at a place of a head's line: false past the last. kRows: queries of an item, kKeys: keys of a tile. Sequence by
// sequence, each from its end, so that its items that see the most keys begin first, and an item's pieces next to each other. (All
// items of a head by the keys that they see, found by bisection: 9 packed prompts of 4093 rows 96 us, in this order 92; 40 of 8000 87,
// 81; 5 of 6000 behind 700 keys each 102, 104.) kItems: `place` counts the items instead of their pieces.
template <int kRows, int kKeys, bool kItems = false>
__device__ __forceinline__ bool find_item(const PrefillArgs& a, int place, PrefillItem* it) {
  const int lane = threadIdx.x & 63;
  auto lane_of = [](int v, int l) { return __builtin_amdgcn_readlane(v, l); };
  // Pieces: the smallest share of key tiles with which a head's items make no more pieces than wanted (one more would be a round
  // of workgroups for itself: 512 rows behind 8191 keys, 576 pieces for 512 places 169 us, 480 144), or each stays whole.
  int per = 1;
  if (a.pieces) {
    const Sequence mine(a, lane);
    auto parts = [&](const Sequence& s, int share) { return (s.nq + kRows - 1) / kRows * std::max(((s.nk + kKeys - 1) / kKeys + share - 1) / share, 1); };
    auto count = [&](int share) {
      int n = parts(mine, share);
      for (int b = lane + 64; b < a.B; b += 64) n += parts(Sequence(a, b), share);
      return lanes_total(n);
    };
    // n items of t tiles make between n t / share and n t / share + n pieces; tiles are counted by 16, which the ends allow for. (A search
    // from every share: 256 rows behind 1280 keys, 8 heads of 256, 25.8 us, between these ends 24.9.)
    int items = 0, tiles16 = 0;
    auto add = [&](const Sequence& s) {
      const int n = (s.nq + kRows - 1) / kRows;
      items += n;
      tiles16 += static_cast<int>(static_cast<int64_t>(n) * ((s.nk + kKeys - 1) / kKeys) / 16);
    };
    add(mine);
    for (int b = lane + 64; b < a.B; b += 64) add(Sequence(a, b));
    items = lanes_total(items);
    tiles16 = lanes_total(tiles16);
    int lo = std::max(kLeastTiles, static_cast<int>(16ll * tiles16 / a.pieces)) - 1;   // but for kLeastTiles - 1, with lo there are too many,
    int hi = (a.Tk + kKeys - 1) / kKeys;                                               // with hi every item is whole
    if (items < a.pieces) hi = std::min(hi, static_cast<int>(16ll * (tiles16 + items) / (a.pieces - items)) + 1);
    hi = std::max(hi, lo + 1);
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (count(mid) > a.pieces) lo = mid;
      else hi = mid;
    }
    per = hi;
  }
  int before = 0, places = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const Sequence s(a, b0 + lane);
    const int n = (s.nq + kRows - 1) / kRows, np = a.pieces ? std::max(((s.nk + kKeys - 1) / kKeys + per - 1) / per, 1) : 1;
    const int mine = kItems ? n : n * np, sum = lanes_scan(mine), all = kItems ? lanes_scan(n * np) : sum;
    const uint64_t here = __ballot(before + sum > place);
    if (here) {
      const int f = __builtin_ctzll(here), parts = lane_of(np, f), in = place - before - (lane_of(sum, f) - lane_of(mine, f));
      const int item = kItems ? in : in / parts;
      *it = {(lane_of(n, f) - 1 - item) * kRows, lane_of(s.q0, f), lane_of(s.nq, f), lane_of(s.k0, f), lane_of(s.nk, f), kItems ? 0 : in % parts, parts,
             places + lane_of(all, f) - lane_of(n, f) * parts + item * parts};
      return true;
    }
    before += lane_of(sum, 63);
    places += lane_of(all, 63);
  }
  return false;
}

// A workgroup's head and place. Workgroups go round the 8 XCDs, so with Hq a multiple of 8 each XCD keeps its own Hq / 8 heads
// (the queries that share a key head meet in one L2).
__device__ __forceinline__ void head_and_place(const PrefillArgs& a, int block, int* hq, int* place) {
  if (a.Hq % 8 == 0) {
    const int per = a.Hq / 8, i = block >> 3;
    *hq = (block & 7) * per + i % per;
    *place = i / per;
  } else {
    *hq = block % a.Hq;
    *place = block / a.Hq;
  }
}

__device__ __forceinline__ int block_of(const PrefillArgs& a, int hq, int place) {
  if (a.Hq % 8 == 0) {
    const int per = a.Hq / 8;
    return 8 * (place * per + hq % per) + hq / per;
  }
  return place * a.Hq + hq;
}

// kSplit: the weights in two bf16 pieces, each with a product of its own.
template <int D, bool kBf16, bool kSplit>
__global__ __launch_bounds__(256, 2) void attn_prefill_kernel(PrefillArgs a) {
  using Tile = PrefillTile<D>;
  constexpr int kDB = D / 32, kKB = Tile::kKeys / 32, kSteps = D / 16;
  constexpr float kLift = kBf16 ? 0.0f : kF16Lift;
  constexpr bool kOpaque = D == 256;   // registers: at 128 channels the 1 % that it costs buys nothing
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Tile::kLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 31, half = lane >> 5;

  int hq, place;
  head_and_place(a, blockIdx.x, &hq, &place);
  PrefillItem it;
  if (!find_item<Tile::kRows, Tile::kKeys>(a, place, &it)) return;
  const int h = hq / (a.Hq / a.Hkv);
  const bool causal = a.causal;
  const int row = it.r0 + 32 * wave + n;                               // this lane's query; rows past the end repeat the last
  const int seen = it.keys(std::min(row, it.nq - 1), causal);
  const int all_tiles = (it.keys(std::min(it.r0 + Tile::kRows, it.nq) - 1, causal) + Tile::kKeys - 1) / Tile::kKeys;
  const int first = static_cast<int>(static_cast<int64_t>(all_tiles) * it.piece / it.pieces);
  const int tiles = static_cast<int>(static_cast<int64_t>(all_tiles) * (it.piece + 1) / it.pieces);
  // of this wave's rows: the fewest and the most keys that one sees
  const int least = it.keys(std::min(it.r0 + 32 * wave, it.nq - 1), causal);
  const int most = it.r0 + 32 * wave >= it.nq ? 0 : it.keys(std::min(it.r0 + 32 * wave + 31, it.nq - 1), causal);

  // queries: channels 16 s + 8 half .. + 7 of step s
  attn_u32x4 q[kSteps];
  {
    const uint16_t* p = a.q + static_cast<int64_t>(it.q0 + std::min(row, it.nq - 1)) * a.ldq + hq * a.hsq + 8 * half;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const attn_u32x4*>(p + 16 * s);
  }

  // Direct loads of a tile: load i of a wave fills 1 KiB, kStep rows, 64 chunks in LDS order. A lane's row of the kStep and its
  // chunk are fixed; the load's own rows are in the scalar base, and change the chunk's place by an exclusive or.
  constexpr int kStep = 64 / Tile::kChunks;
  const int lr = lane / Tile::kChunks, lc = lane % Tile::kChunks, wr = wave * Tile::kLoads * kStep;   // wr: the wave's first row
  const uint32_t krow = lr * static_cast<uint32_t>(a.ldk) * 2, vrow = lr * static_cast<uint32_t>(a.ldv) * 2;
  const uint32_t kch = 16 * (lc ^ Tile::kswizzle(lr)), vch = 16 * (lc ^ Tile::vswizzle(lr));
  const uint16_t* const kbase = a.k + static_cast<int64_t>(it.k0) * a.ldk + h * a.hsk;
  const uint16_t* const vbase = a.v + static_cast<int64_t>(it.k0) * a.ldv + h * a.hsv;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem) + wave * Tile::kLoads * 1024);
  auto load = [&](int j) {
    const int left = it.nk - j * Tile::kKeys;
    const uint32_t to = lds0 + (j & 1) * 2 * Tile::kPart;
    const uint16_t* const kb = kbase + static_cast<int64_t>(j) * Tile::kKeys * a.ldk;
    const uint16_t* const vb = vbase + static_cast<int64_t>(j) * Tile::kKeys * a.ldv;
    if (left >= Tile::kKeys) {
#pragma unroll
      for (int i = 0; i < Tile::kLoads; ++i)
        lds_dma16_s(scalar_addr(kb + (wr + i * kStep) * a.ldk), krow + (kch ^ (16 * Tile::kswizzle(wr + i * kStep))), to + i * 1024);
#pragma unroll
      for (int i = 0; i < Tile::kLoads; ++i)
        lds_dma16_s(scalar_addr(vb + (wr + i * kStep) * a.ldv), vrow + (vch ^ (16 * Tile::vswizzle(wr + i * kStep))), to + Tile::kPart + i * 1024);
    } else {   // rows past the last key repeat it
#pragma unroll
      for (int i = 0; i < Tile::kLoads; ++i) {
        const int r = wr + i * kStep;
        const uint32_t from = 2 * static_cast<uint32_t>(std::min(r + lr, left - 1));
        lds_dma16_s(scalar_addr(kb), from * static_cast<uint32_t>(a.ldk) + (kch ^ (16 * Tile::kswizzle(r))), to + i * 1024);
        lds_dma16_s(scalar_addr(vb), from * static_cast<uint32_t>(a.ldv) + (vch ^ (16 * Tile::vswizzle(r))), to + Tile::kPart + i * 1024);
      }
    }
  };

  f32x16 o[kDB] = {};
  float m = -__builtin_inff(), mc = 0.0f, l = 0.0f;   // the score that p is taken against, m * c, the sum of this lane's keys
  bool fresh = true;                                  // a row of the wave has no such score yet
  const float c = a.scale_log2;
  const int wave_tiles = std::min(tiles, (most + Tile::kKeys - 1) / Tile::kKeys);   // behind these nothing for this wave's rows

  // Tile j, which lies in buffer j % 2.
  auto step = [&](int j) {
    const uint8_t* const kt = smem + (j & 1) * 2 * Tile::kPart;
    const uint8_t* const vt = kt + Tile::kPart;
    const int k0 = j * Tile::kKeys;
    // Operands are read kRead products ahead of their use: an LDS read takes longer than a product. (K and V 2 and 4 ahead, 4 and 6, 8
    // and 8: 8192 rows of 48 heads of 128 779, 772, 783 us; at 256 channels registers allow 2 and 1 130, 2 and 2 127, 4 and 4, which
    // spills, 167; with weights in two pieces 2 and 1 167, 2 and 2 175.)
    constexpr int kProducts = kKB * kSteps, kRead = D == 256 ? 2 : 4;
    f32x16 s[kKB];
    const int ln = kOpaque ? opaque(lane) : lane;
    auto read_k = [&](int e) {
      const int r = 32 * (e / kSteps) + (ln & 31), st = e % kSteps;
      return *reinterpret_cast<const attn_u32x4*>(kt + r * Tile::kRowBytes + 16 * ((2 * st + (ln >> 5)) ^ Tile::kswizzle(r)));
    };
    attn_u32x4 kf[kRead];
#pragma unroll
    for (int e = 0; e < kRead; ++e) kf[e] = read_k(e);
#pragma unroll
    for (int e = 0; e < kProducts; ++e) {
      f32x16& t = s[e / kSteps];
      t = mfma_32<kBf16>(kf[e % kRead], q[e % kSteps], e % kSteps ? t : f32x16{});
      if (e + kRead < kProducts) kf[e % kRead] = read_k(e + kRead);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, kRead, 0);
#pragma unroll
    for (int e = 0; e < kProducts - kRead; ++e) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kRead, 0);
    if (k0 + Tile::kKeys > least) {
      const int limit = seen - k0 - 4 * half;
#pragma unroll
      for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][i] = 32 * kb + (i & 3) + 8 * (i >> 2) < limit ? s[kb][i] : -__builtin_inff();
    }
    auto raise = [&] {
      float mt = m;
#pragma unroll
      for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) mt = __builtin_fmaxf(mt, s[kb][i]);
      mt = both_halves_max(mt);
      // The weights so far were taken against mc as it was rounded, so the factor is the difference of the rounded ones (fused with
      // a product it would be that of others, off by 2^(half a step of mc)).
      const float to = mt == -__builtin_inff() ? 0.0f : rounded_product(mt, c) - kLift, f = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(mc - to);
      m = mt;
      mc = to;
      l *= f;
      // Scores of 2^30 and more: the step of mc may carry every weight past its type. Such a row is computed again, key by key.
      if (__builtin_fabsf(mc) >= 0x1p30f) l = __builtin_nanf("");
#pragma unroll
      for (int db = 0; db < kDB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] *= f;
      fresh = __any(m == -__builtin_inff());
    };
    uint32_t p[kKB][8], rest[kKB][kSplit ? 8 : 1];
    float sum;
    auto weights = [&] {
      float part[2] = {0.0f, 0.0f};
#pragma unroll
      for (int kb = 0; kb < kKB; ++kb)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][2 * i], c, -mc)), p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][2 * i + 1], c, -mc));
          const uint32_t w = pack2<kBf16>(p0, p1);
          p[kb][i] = w;
          if constexpr (kSplit) {
            rest[kb][i] = pack2<kBf16>(p0 - bf16_to_f32(w), p1 - bf16_to_f32(w >> 16));
            part[i & 1] += p0 + p1;
          } else {
            part[i & 1] = add_pair<kBf16>(w, part[i & 1]);
          }
        }
      sum = part[0] + part[1];
    };
    const int lv = kOpaque ? opaque(lane) : lane;
    auto read_v = [&](int e) {                         // product e: 32 channels of 16 keys
      const int kb = e / kDB, db = e % kDB;
      const int r = 16 * kb + 4 * (lv >> 5) + ((lv & 15) >> 2);   // this lane's key of the first transposing read; r + 8 of the second
      const int ch = 4 * db + 2 * ((lv >> 4) & 1) + ((lv & 3) >> 1), byte = 8 * (lv & 1);
      const uint2 v0 = lds_read_transposed(vt + r * Tile::kRowBytes + 16 * (ch ^ Tile::vswizzle(r)) + byte);
      const uint2 v1 = lds_read_transposed(vt + (r + 8) * Tile::kRowBytes + 16 * (ch ^ Tile::vswizzle(r + 8)) + byte);
      return attn_u32x4{v0.x, v0.y, v1.x, v1.y};
    };
    constexpr int kValues = 2 * kKB * kDB, kReadV = D == 256 ? (kSplit ? 1 : 2) : 6;
    attn_u32x4 vf[kReadV];
#pragma unroll
    for (int e = 0; e < kReadV; ++e) vf[e] = read_v(e);
    if (fresh) raise();
    weights();
    if (__any(!(sum <= 0x1p60f))) {   // an f16 weight past its type is an infinity, and so is the sum
      raise();
      weights();
    }
    l += sum;
#pragma unroll
    for (int e = 0; e < kValues; ++e) {
      const int kb = e / kDB;
      auto of = [&](auto& p) { return attn_u32x4{p[kb / 2][4 * (kb % 2)], p[kb / 2][4 * (kb % 2) + 1], p[kb / 2][4 * (kb % 2) + 2], p[kb / 2][4 * (kb % 2) + 3]}; };
      o[e % kDB] = mfma_32<kBf16>(vf[e % kReadV], of(p), o[e % kDB]);
      if constexpr (kSplit) o[e % kDB] = mfma_32<kBf16>(vf[e % kReadV], of(rest), o[e % kDB]);
      if (e + kReadV < kValues) vf[e % kReadV] = read_v(e + kReadV);
    }
#pragma unroll
    for (int e = 0; e < kValues - kReadV; ++e) {
      __builtin_amdgcn_sched_group_barrier(0x008, kSplit ? 2 : 1, 1);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kReadV * (kSplit ? 2 : 1), 1);
  };
  auto turn = [&](int j) {
    // this wave's loads of tile j have landed and its reads of tile j - 1 are done; behind the barrier every wave's
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (j + 1 < tiles) load(j + 1);
    if (j < wave_tiles) step(j);
  };
  if (first < tiles) load(first);
  // the queries have landed: or the loop would wait for them again, and with them for the loads it has just made
#pragma unroll
  for (int i = 0; i < kSteps; ++i) asm volatile("" : "+v"(q[i]));
  for (int j = first; j < tiles; ++j) turn(j);

  l = both_halves_sum(l);
  if (it.pieces > 1) {
    // A piece: O as 16-byte chunks [D / 4][rows], then the maximum and the sum of every row. 32 rows' chunks are one run.
    float* const p = a.ws + static_cast<int64_t>(blockIdx.x) * Tile::kSlot + 4 * (32 * wave + n);
#pragma unroll
    for (int db = 0; db < kDB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(p + (8 * db + 2 * g + half) * 4 * Tile::kRows) = make_float4(o[db][4 * g], o[db][4 * g + 1], o[db][4 * g + 2], o[db][4 * g + 3]);
    if (half == 0) *reinterpret_cast<float2*>(a.ws + static_cast<int64_t>(blockIdx.x) * Tile::kSlot + D * Tile::kRows + 2 * (32 * wave + n)) =
        make_float2(m == -__builtin_inff() ? m : mc, l);
    return;
  }
  // Rows that saw a key and whose values are not all finite: key by key. (A sum of 0 has every score at -inf: NaN by the formula.)
  float odd_sum = l > 0.0f ? 0.0f : __builtin_nanf("");
#pragma unroll
  for (int db = 0; db < kDB; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) odd_sum = __builtin_fmaf(o[db][i], 0.0f, odd_sum);
  const uint64_t odd = __ballot(seen > 0 && row < it.nq && !(odd_sum == 0.0f));
  const uint32_t again = static_cast<uint32_t>(odd | odd >> 32);
  const float inv = 1.0f / l;
  const uint32_t keep = seen > 0 ? ~0u : 0;   // a row without a key is zeros, whatever values its weights of 0 stand before
  if (row < it.nq && !(again >> n & 1)) {
    uint16_t* out = a.o + (static_cast<int64_t>(it.q0 + row) * a.Hq + hq) * D;
#pragma unroll
    for (int db = 0; db < kDB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g)                      // channels 32 db + 8 g + 4 half .. + 3
        *reinterpret_cast<uint2*>(out + 32 * db + 8 * g + 4 * half) = kept(pack4(a.out_type, o[db][4 * g] * inv, o[db][4 * g + 1] * inv, o[db][4 * g + 2] * inv, o[db][4 * g + 3] * inv), keep);
  }
  for (uint32_t left = again; left; left &= left - 1) {
    const int r = it.r0 + 32 * wave + __builtin_ctz(left);
    attend_row<D, kBf16>(a, it.q0 + r, hq, it.k0, it.keys(r, causal));
  }
}

// The pieces of 16 rows of an item together: thread (row, part) takes the 16-byte chunks part, part + 16, ... of its row.
constexpr int kJoinRows = 16;
template <int D, bool kBf16>
__global__ __launch_bounds__(256) void attn_prefill_join_kernel(PrefillArgs a) {
  using Tile = PrefillTile<D>;
  constexpr int kGroups = Tile::kRows / kJoinRows, kEach = D / 64;
  __shared__ uint32_t odd;
  const int hq = blockIdx.x / kGroups % a.Hq;
  PrefillItem it;
  if (!find_item<Tile::kRows, Tile::kKeys, true>(a, blockIdx.x / kGroups / a.Hq, &it) || it.pieces == 1) return;
  const int n = threadIdx.x % kJoinRows, part = threadIdx.x / kJoinRows, in = kJoinRows * (blockIdx.x % kGroups) + n, row = it.r0 + in;
  if (row - n >= it.nq) return;
  if (threadIdx.x == 0) odd = 0;
  __syncthreads();
  const float* const first = a.ws + static_cast<int64_t>(block_of(a, hq, it.place)) * Tile::kSlot;   // a head's places are Hq workgroups apart
  auto slot = [&](int i) { return first + static_cast<int64_t>(i) * a.Hq * Tile::kSlot; };
  auto state = [&](int i) { return *reinterpret_cast<const float2*>(slot(i) + D * Tile::kRows + 2 * in); };
  float most = -__builtin_inff();
#pragma unroll 4
  for (int i = 0; i < it.pieces; ++i) most = __builtin_fmaxf(most, state(i).x);
  float sum = 0.0f;
  float4 v[kEach] = {};
#pragma unroll 4
  for (int i = 0; i < it.pieces; ++i) {
    const float2 st = state(i);
    const float f = st.x == -__builtin_inff() ? (st.y == st.y ? 0.0f : st.y) : __builtin_amdgcn_exp2f(st.x - most);
    sum += f * st.y;
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
      const float4 u = *reinterpret_cast<const float4*>(slot(i) + (16 * c + part) * 4 * Tile::kRows + 4 * in);
      v[c].x += f * u.x, v[c].y += f * u.y, v[c].z += f * u.z, v[c].w += f * u.w;
    }
  }
  const int seen = it.keys(std::min(row, it.nq - 1), a.causal);
  float t = sum > 0.0f ? 0.0f : __builtin_nanf("");
#pragma unroll
  for (int c = 0; c < kEach; ++c) t += 0.0f * v[c].x + 0.0f * v[c].y + 0.0f * v[c].z + 0.0f * v[c].w;
  if (row < it.nq && seen > 0 && !(t == 0.0f)) atomicOr(&odd, 1u << n);
  __syncthreads();
  const uint32_t again = odd;
  if (row < it.nq && !(again >> n & 1)) {
    const float inv = 1.0f / sum;
    const uint32_t keep = seen > 0 ? ~0u : 0;
    uint16_t* out = a.o + (static_cast<int64_t>(it.q0 + row) * a.Hq + hq) * D;
#pragma unroll
    for (int c = 0; c < kEach; ++c)
      *reinterpret_cast<uint2*>(out + 4 * (16 * c + part)) = kept(pack4(a.out_type, v[c].x * inv, v[c].y * inv, v[c].z * inv, v[c].w * inv), keep);
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int i = wave; i < kJoinRows; i += 4)
    if (again >> i & 1) attend_row<D, kBf16>(a, it.q0 + row - n + i, hq, it.k0, it.keys(row - n + i, a.causal));
}

// The most items that a head can have, an item for every kRows queries of a sequence, and the pieces that they are cut into. Cut where
// the items are fewer than the workgroups that the device holds (two a CU) and a row may see more than kWholeTiles key tiles: the
// join costs what some tiles do. (256 rows behind 1280 keys, 24 heads of 128: whole 32.4 us, cut 23.3; 1000 rows of 16 heads of 128:
// 23.8, 24.9; 256 behind 768, 8 heads of 256: 43, 24.)
constexpr int kWholeTiles = 16;
constexpr int kMostRows = 1 << 30;   // of queries, and of keys: their sum stays within 32 bits
template <int D>
static void prefill_shape(int B, int Tq, int Tk, int Hq, int* pieces, int64_t* items) {
  const int64_t room = 2 * cu_count();
  *items = Tq / PrefillTile<D>::kRows + static_cast<int64_t>(B);
  *pieces = *items * Hq < room && Tk > kWholeTiles * PrefillTile<D>::kKeys ? static_cast<int>(room / Hq) : 0;
}
template <int D>
static size_t prefill_workspace(int B, int Tq, int Tk, int Hq) {
  int pieces;
  int64_t items;
  prefill_shape<D>(B, Tq, Tk, Hq, &pieces, &items);
  return pieces ? static_cast<size_t>(std::max<int64_t>(items, pieces) * Hq) * PrefillTile<D>::kSlot * sizeof(float) : 0;
}

template <int D, bool kBf16, bool kSplit>
static hipError_t prefill_kernels(const PrefillArgs& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(std::max(a.items, a.pieces)) * a.Hq);
  const hipError_t e = launch_kernel((attn_prefill_kernel<D, kBf16, kSplit>), dim3(grid), dim3(64 * PrefillTile<D>::kWaves), 0, s, a);
  if (e != hipSuccess || !a.pieces) return e;
  return launch_kernel((attn_prefill_join_kernel<D, kBf16>), dim3(static_cast<unsigned>(a.items * a.Hq) * (PrefillTile<D>::kRows / kJoinRows)), dim3(256), 0, s, a);
}
template <int D>
static hipError_t prefill_launch(PrefillArgs a, int type, hipStream_t s) {
  int64_t items;
  prefill_shape<D>(a.B, a.Tq, a.Tk, a.Hq, &a.pieces, &items);
  a.items = static_cast<int>(items);
  if (type == PQ_F16) return prefill_kernels<D, false, false>(a, s);
  return a.out_type == PQ_F16 ? prefill_kernels<D, true, true>(a, s) : prefill_kernels<D, true, false>(a, s);
}

}  // namespace pq

extern "C" {

size_t pq_attn_prefill_workspace_bytes(int B, int Tq, int Tk, int Hq, int Hkv, int D) {
  using namespace pq;
  if (B <= 0 || Tq <= 0 || Tk <= 0 || Hq <= 0) return 0;
  return D == 64 ? prefill_workspace<64>(B, Tq, Tk, Hq) : D == 128 ? prefill_workspace<128>(B, Tq, Tk, Hq) : D == 256 ? prefill_workspace<256>(B, Tq, Tk, Hq) : 0;
}

int pq_attn_prefill(const uint16_t* q_d, int64_t ldq, int64_t hsq, const uint16_t* k_d, int64_t ldk, int64_t hsk, const uint16_t* v_d, int64_t ldv,
                    int64_t hsv, int type, const int32_t* cu_q_d, const int32_t* cu_k_d, int B, int Tq, int Tk, int Hq, int Hkv, int D, float scale,
                    int causal, uint16_t* o_d, int out_type, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_attn_prefill";
  if (B < 0 || Tq < 0 || Tk < 0) return set_error(PQ_ERR_SHAPE, "%s: B=%d, Tq=%d, Tk=%d: negative", what, B, Tq, Tk);
  int rc = check_attention(what, type, out_type, Hq, Hkv, D, scale);
  if (rc == PQ_OK) rc = check_heads(what, "q", q_d, ldq, hsq, Tq);
  if (rc == PQ_OK) rc = check_heads(what, "k", k_d, ldk, hsk, Tk);
  if (rc == PQ_OK) rc = check_heads(what, "v", v_d, ldv, hsv, Tk);
  if (rc != PQ_OK) return rc;
  if (Tq > kMostRows || Tk > kMostRows) return set_error(PQ_ERR_SHAPE, "%s: Tq=%d, Tk=%d: at most 2^30 rows", what, Tq, Tk);
  if ((Tq / 128 + static_cast<int64_t>(B)) * Hq * 256 > 0xFFFFFFFFll)   // the runtime counts a launch's threads in 32 bits
    return set_error(PQ_ERR_SHAPE, "%s: Tq=%d rows of B=%d sequences too many for one call", what, Tq, B);
  if (Tq == 0 || B == 0) return PQ_OK;
  if (!o_d || !cu_q_d || !cu_k_d) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (!aligned(o_d, 16) || !aligned(cu_q_d, 4) || !aligned(cu_k_d, 4) || !aligned(ws_d, 16)) return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  const size_t need = pq_attn_prefill_workspace_bytes(B, Tq, Tk, Hq, Hkv, D);
  if (need && (!ws_d || ws_bytes < need)) return set_error(PQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, ws_d ? ws_bytes : 0, need);
  const int64_t ob = 2ll * Tq * Hq * D, qb = heads_span(ldq, hsq, Tq, Hq, D), kb = heads_span(ldk, hsk, Tk, Hkv, D), vb = heads_span(ldv, hsv, Tk, Hkv, D);
  for (const auto& [o, n] : {std::pair<const void*, int64_t>{o_d, ob}, {ws_d, static_cast<int64_t>(need)}})
    if (ranges_meet(o, n, q_d, qb) || ranges_meet(o, n, k_d, kb) || ranges_meet(o, n, v_d, vb) || ranges_meet(o, n, cu_q_d, 4ll * (B + 1ll)) ||
        ranges_meet(o, n, cu_k_d, 4ll * (B + 1ll)))
      return overlap(what);
  if (ranges_meet(o_d, ob, ws_d, static_cast<int64_t>(need))) return overlap(what);
  PrefillArgs a{q_d, k_d, v_d, ldq, hsq, ldk, hsk, ldv, hsv, cu_q_d, cu_k_d, B, Tq, Tk, Hq, Hkv, causal, scale * 1.44269504088896340736f, o_d, out_type,
                0, 0, static_cast<float*>(ws_d)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return launch_status(what, D == 64 ? prefill_launch<64>(a, type, s) : D == 128 ? prefill_launch<128>(a, type, s) : prefill_launch<256>(a, type, s));
}

}  // extern "C"
