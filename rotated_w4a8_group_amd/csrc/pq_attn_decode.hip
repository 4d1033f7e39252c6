// Attention of one new token of each sequence over the paged cache (pq_attn_decode): the heads that share a key head are
// the rows of one small product, so every cached row is read once.
//
// The cache is the traffic and bounds it; the arithmetic only has to stay beside it. A wave walks tiles of 32 keys, which go
// global -> LDS by direct loads into its own two slots, K and V of one tile: while a tile's scores are computed its V is
// in flight, while its V is used the next tile's K is. Nothing in the loop waits for another wave.
//   S^T = K Q^T   (16x16x32, twice: 16 keys x 32 channels times 32 channels x 16 query heads): lane l holds head l % 16 and, of
//                 each 16 keys, the 4 from 4 (l / 16) on;
//   O^T = V^T P^T (16 channels x 32 keys times 32 keys x 16 heads), the keys in the order in which a lane holds them, V^T by
//                 transposing LDS reads of that order.
// Codes become 16-bit values, exactly, on their way from LDS to the matrix core (of q's type for K, bf16 for V); a key's
// scale multiplies its score, a value's its weight. p is held in two 16-bit pieces, hi + lo, each with a product of its
// own: the matrix core has the time, and no rounding of p shows in an f16 output (2^-16 of it is left; of f16 pieces 2^-32 of the
// largest weight, where that is more: kF16Lift).
//
// Work is split over the cache's length: each head's tiles of a sequence are cut into pieces of at most a share of all of them
// (Cut), a workgroup each, whatever the lengths. A piece that is not the whole head leaves its maximum, sum and O in the
// workspace, and attn_join_kernel puts the pieces together in their order. Which pieces exist follows from the lengths on
// the device; the host only bounds them.
//
// Measured: 64 sequences of up to 8192 positions (8 heads of 128, 16-bit, 1.04 GB of rows) 178 us, 5.84 TB/s; one of 131071, e4m3
// (277 MB) 53 us, 5.2 TB/s; a read of as much memory and nothing else reaches 6.3. Small calls are the waits of one chain: length,
// page, row, score, and the join's launch (17 sequences of up to 4000, 4 heads of 256, e4m3, 36 MB: 17.7 us).
// "n x <= L" below is n sequences, one of length L and the others spread below it as L r^1.5, r uniform: 0.4 L on average.
#include <algorithm>
#include <utility>

#include "pq_attn.h"

namespace pq {

struct DecodeArgs {
  CacheArgs c;
  const uint16_t* q;
  int64_t ldq, hsq;
  const int32_t* lens;
  int B, Hq, G;             // G: query heads of a key head
  int hv, tiles_of_heads;   // virtual heads: a key head once for each 16 query heads that share it
  int pieces;               // pieces to cut the whole line into, about; 0: a workgroup for each sequence and virtual head
  int places, least;        // workgroups that the device holds at a time; tiles of a piece at least
  float scale_log2;
  uint16_t* o;
  int out_type;
  float* ws;
};

constexpr int kTileKeys = 32;
// While a piece for every place of the device is at most this many tiles, there are no more pieces than places, each a whole number of
// tiles for every wave: what a second round costs is the wait of its first loads (8 x <= 3000 of 4 heads of 256, 16-bit: 2 tiles a piece, 750
// pieces for 512 places 23 us, 4 tiles 17.2; 4 x <= 500, 2 tiles 9.9, 4 12, 8 16; 17 x <= 4000 of 4 of 256, e4m3, 5 tiles for 4 waves
// 17.9, 8 17.5). Longer ones are cut into wanted_pieces() of two tiles a wave at least (16 x <= 8000 of 4 of 256, 16-bit, 12 tiles in one
// round 61, 6 in two 51; 12 x <= 4000 of 8 of 128, 16-bit, 5 tiles 30.5, 8 27.9).
constexpr int kOneRound = 8;
constexpr int kTableHalves = 128;   // 16-key halves whose pages a wave holds at a time
constexpr int kMostPieces = 4096;   // of one head

// kWide: as many waves as the LDS holds, for whole heads that are no more than the CUs (1 x 509 of 8 heads of 128, e4m3: 7.5 us, else 9.6; 32 x
// <= 1000 11.7, 18.5; 60 x <= 250 of 4 of 256, 16-bit 12.2, 15.5); else several workgroups a CU (60 x <= 500 of 8 of 128, 16-bit 15.6, wide 17.4;
// 128 x <= 2000, e4m3 53.9, 58.4; but 40 x <= 1000 18.6, 16.9).
template <int D, bool kQuant, bool kWide>
struct DecodeTile {
  static constexpr int kRow = D * (kQuant ? 1 : 2);        // bytes of a row
  static constexpr int kPart = kTileKeys * kRow;           // a tile's K, or V
  static constexpr int kWaves = (2 * kPart > 16384 ? 2 : 2 * kPart > 8192 || !kWide ? 4 : 8) * (kWide ? 2 : 1);
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kLoads = kPart / 1024;              // direct loads of it
  static constexpr int kChunks = kRow / 16;                // 16-byte chunks of a row
  static constexpr int kTable = 4 * kTableHalves;
  static constexpr int kScale = kQuant ? 256 : 0;          // 32 scales of K, 32 of V
  static constexpr int kWave = 2 * kPart + 2 * kScale + kTable;
  static constexpr int kState = kWaves * 16 * 16;          // maximum, sum, seen of every wave and head
  static constexpr int kLds = kWaves * kWave + 2 * kState + 16;   // states, factors of them, and a flag
  static constexpr int kPerCu = std::min(160 * 1024 / kLds, 16 / kWaves);
  static constexpr int kSlot = 16 * D + 64;                // floats of a piece in the workspace
  static_assert(2 * kPart >= 16 * D * 4, "O of a wave fits its slots");

  // Places of chunk c of row r in a slot, so that the 16 lanes of an operand read lie in different banks: K reads the same
  // chunk of 16 rows; V 32 bytes of the 8 rows 4 g .. of two neighbouring lane groups (codes: 16 bytes of those and of the
  // rows 16 further on).
  static __device__ __forceinline__ int kswizzle(int r) { return kRow >= 256 ? r & 15 : kRow == 128 ? (r >> 1) & 7 : (r >> 2) & 3; }
  static __device__ __forceinline__ int vswizzle(int r) {
    if constexpr (kQuant) return kRow == 256 ? (r & 7) | (r >> 4 & 1) << 3 : kRow == 128 ? (r >> 1 & 3) | (r >> 4 & 1) << 2 : (r >> 2 & 1) | (r >> 4 & 1) << 1;
    else return kRow >= 256 ? (r & 7) << 1 : (r >> 1 & 3) << 1;
  }
};

template <bool kBf16>
__device__ __forceinline__ v4f mfma_16(const attn_u32x4& a, const attn_u32x4& b, const v4f& c) {
  if constexpr (kBf16) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 4 codes as 16-bit values (exact).
template <bool kBf16>
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  if constexpr (kBf16)
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)));
  else
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)));
}
template <bool kBf16>
__device__ __forceinline__ attn_u32x4 widen8(uint32_t lo, uint32_t hi) {
  const uint2 a = widen4<kBf16>(lo), b = widen4<kBf16>(hi);
  return attn_u32x4{a.x, a.y, b.x, b.y};
}

// 8 bytes a lane: lanes 2 r and 2 r + 1 of 16 give the halves of row r's 16 bytes; lane i gets byte i of the 8 rows.
__device__ __forceinline__ uint2 lds_read_transposed8(const uint8_t* p) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) i32x2* lds_ptr;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_ptr)(uintptr_t)lds_addr(p)));
}

// The lanes l, l ^ 16, l ^ 32, l ^ 48 combined.
template <typename F>
__device__ __forceinline__ float four_groups(float v, F f) {
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  const uint32_t a = r[0], b = r[1];
  const Halves x = both_halves(f(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
  return f(x.lo, x.hi);
}

// What values are taken times in a second walk: 2^31 weights of up to 2^8 times values of up to 2^128 stay below 2^120. (Smaller weights instead would
// lose those of large values; of values this takes 2^-69 a key at most, beside sums past 2^100.)
constexpr float kSmaller = 0x1p-48f;

// log2 of what the weights of f16 values are taken times, which divides out: m is raised before one passes 2^8, so 2^15 of f16's 2^16 are used, and its
// 2^-25 is 2^-32 of the largest weight.
constexpr float kF16Lift = 7.0f;

// What a state (maximum, sum, seen, the factor of its O) counts beside others, with the largest maximum.
__device__ __forceinline__ float state_factor(const float4& st, float most, float c) {
  if (st.x == -__builtin_inff()) return st.y == st.y ? 0.0f : st.y;
  return __builtin_amdgcn_exp2f((st.x - most) * c);
}

// Positions and tiles of a sequence.
__device__ __forceinline__ int seq_len(const DecodeArgs& a, int b) { return std::min(std::max(a.lens[b], 0), a.c.width << a.c.page_shift); }
__device__ __forceinline__ int tiles_of(int len) { return static_cast<int>((static_cast<uint32_t>(len) + kTileKeys - 1) / kTileKeys); }

// How the sequences are cut: a head's nt tiles into pieces of at most `per`, alike in size; the pieces stand in one line,
// sequence by sequence and head by head. The host bounds their number (a.pieces + sequences x heads), the lengths decide it.
// Sequence b is lane b % 64's of round b / 64.
struct Cut {
  int per, first_len;   // this lane's length in the first round
  __device__ __forceinline__ explicit Cut(const DecodeArgs& a) {
    const int lane = threadIdx.x & 63;
    first_len = lane < a.B ? seq_len(a, lane) : 0;
    int n = tiles_of(first_len);
    for (int b = lane + 64; b < a.B; b += 64) n += tiles_of(seq_len(a, b));
    const int all = lanes_total(n) * a.hv;
    const int one = (all + a.places - 1) / a.places;
    per = one <= kOneRound ? std::max(one + a.least - 1, a.least) / a.least * a.least : std::max((all + a.pieces - 1) / a.pieces, 2 * a.least);
  }
  __device__ __forceinline__ int len(const DecodeArgs& a, int b) const { return b < 64 ? first_len : b < a.B ? seq_len(a, b) : 0; }
  __device__ __forceinline__ int pieces(int len) const { return (tiles_of(len) + per - 1) / per; }
};

// A workgroup's piece: tiles t0 .. t1 - 1 of the nt of sequence b and virtual head hv.
struct DecodePiece {
  int b, hv, len, t0, t1, nt;
};

// Walks the piece's tiles and stores what they give. Whether a sum passed 2^100, or a NaN came: it may have passed binary32 on the way, or will
// beside other pieces', though the mean does not. Such a piece is walked a second time (kAgain) with values kSmaller times as large. (That is
// code of its own: as a loop around one walk, its registers cost the first 5 %. What a thread's number gives is computed in each, not
// kept for the second.)
template <int D, bool kBf16, bool kQuant, bool kWide, bool kAgain>
__device__ __forceinline__ bool decode_walk(const DecodeArgs& a, const DecodePiece& piece, uint8_t* smem) {
  using Tile = DecodeTile<D, kQuant, kWide>;
  constexpr int kDB = D / 16, kSteps = D / 32;
  constexpr bool kVBf16 = kQuant || kBf16;
  const int b = piece.b, hv = piece.hv, len = piece.len, t0 = piece.t0, t1 = piece.t1, nt = piece.nt;
  const float c = a.scale_log2;
  const int64_t page_mask = (1ll << a.c.page_shift) - 1;
  const int h = hv / a.tiles_of_heads, first_head = hv % a.tiles_of_heads * 16, heads = std::min(a.G - first_head, 16);
  const int hq0 = h * a.G + first_head;
  const uint8_t* const kc = static_cast<const uint8_t*>(a.c.k);
  const uint8_t* const vc = static_cast<const uint8_t*>(a.c.v);

  const int tid = opaque(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  uint8_t* const mine = smem + wave * Tile::kWave;
  uint8_t* const kslot = mine;
  uint8_t* const vslot = mine + Tile::kPart;
  float* const scales = reinterpret_cast<float*>(mine + 2 * Tile::kPart);      // two tiles' worth
  int32_t* const table = reinterpret_cast<int32_t*>(mine + 2 * Tile::kPart + 2 * Tile::kScale);
  float* const state = reinterpret_cast<float*>(smem + Tile::kWaves * Tile::kWave);
  float* const factors = state + Tile::kState / 4;
  int* const flag = reinterpret_cast<int*>(factors + Tile::kState / 4);
  if (!kAgain && tid == 0) *flag = 0;   // not by the second walk: waves may still be reading it

  // this wave's tiles
  const int count = t1 - t0, ta = t0 + static_cast<int>(static_cast<int64_t>(count) * wave / Tile::kWaves),
            tb = t0 + static_cast<int>(static_cast<int64_t>(count) * (wave + 1) / Tile::kWaves);

  // query heads: for 16-bit rows channels 32 s + 8 g .. + 7 of step s; for codes 64 t + 16 g .. + 7 and .. + 15 of steps 2 t, 2 t + 1
  attn_u32x4 q[kSteps];
  if (ta < tb) {
    const uint16_t* p = a.q + b * a.ldq + (hq0 + std::min(n, heads - 1)) * a.hsq;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const attn_u32x4*>(p + (kQuant ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g));
  }

  int held = ta;   // the tile that the held page numbers begin with
  auto fill = [&](int t) {
    held = t;
    wait_lds_reads();
#pragma unroll
    for (int i = 0; i < kTableHalves / 64; ++i) {
      const int64_t key = (static_cast<int64_t>(t) * 2 + 64 * i + lane) * 16;
      int page = -1;
      if (key < len) {                                    // positions past the width do not exist: len stops there
        page = a.c.table[static_cast<int64_t>(b) * a.c.width + (key >> a.c.page_shift)];
        if (page < 0 || page >= a.c.pages) page = -1;
      }
      table[64 * i + lane] = page;
    }
    wait_lds_reads();
  };
  auto page_of = [&](int t, int i) { return __builtin_amdgcn_readfirstlane(table[2 * (t - held) + i]); };
  // first cache row of half i of tile t, and whether it exists; where it does not, row 0 of the cache stands in
  auto row_of = [&](int t, int i, int page) {
    const int64_t key = static_cast<int64_t>(t) * kTileKeys + 16 * i;
    return page < 0 ? 0 : ((static_cast<int64_t>(page) * a.c.Hkv + h) << a.c.page_shift) + (key & page_mask);
  };
  auto load = [&](const uint8_t* cache, uint8_t* slot, int t, bool is_k) {
    const int ln = opaque(lane), r0 = ln / Tile::kChunks, ch = ln % Tile::kChunks;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const void* base = scalar_addr(cache + row_of(t, i, page_of(t, i)) * Tile::kRow);
#pragma unroll
      for (int j = 0; j < Tile::kLoads / 2; ++j) {
        const int r = 64 / Tile::kChunks * j + r0;
        lds_dma16_nt(base, r * Tile::kRow + 16 * (ch ^ (is_k ? Tile::kswizzle(16 * i + r) : Tile::vswizzle(16 * i + r))),
                    lds_addr(slot) + (i * Tile::kLoads / 2 + j) * 1024);
      }
    }
  };
  auto load_k = [&](int t) {
    load(kc, kslot, t, true);
    if constexpr (kQuant) {   // lanes 0..31 the scales of K, 32..63 those of V
      const int64_t r0 = row_of(t, 0, page_of(t, 0)), r1 = row_of(t, 1, page_of(t, 1));
      lds_dma4((lane < 32 ? a.c.ks : a.c.vs) + ((lane & 16) ? r1 : r0) + n, lds_addr(scales + 64 * (t & 1)));
    }
  };
  auto load_v = [&](int t) { load(vc, vslot, t, false); };

  v4f o[kDB];
#pragma unroll
  for (int i = 0; i < kDB; ++i) o[i] = v4f{0.f, 0.f, 0.f, 0.f};
  float m = -__builtin_inff(), ref = 0.0f, l = 0.0f;   // ref: m, once there is one
  bool any = false;

  if (ta < tb) {
    fill(ta);
    load_k(ta);
    load_v(ta);
  }
  for (int t = ta; t < tb; ++t) {
    const bool more = t + 1 < tb;
    // which of the tile's keys exist
    const int left = std::min(len - t * kTileKeys, kTileKeys);
    uint32_t valid = left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1;
    if (page_of(t, 0) < 0) valid &= 0xFFFF0000u;
    if (page_of(t, 1) < 0) valid &= 0x0000FFFFu;
    any = any || valid;

    wait_vm<Tile::kLoads>();          // K of this tile and its scales; V may be in flight
    v4f s[2];
    const int ln = opaque(lane);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      s[kb] = v4f{0.f, 0.f, 0.f, 0.f};
      const int r = 16 * kb + (ln & 15), g = ln >> 4;
      if constexpr (kQuant) {
#pragma unroll
        for (int st = 0; st < kSteps / 2; ++st) {
          const attn_u32x4 w = *reinterpret_cast<const attn_u32x4*>(kslot + r * Tile::kRow + 16 * ((4 * st + g) ^ Tile::kswizzle(r)));
          s[kb] = mfma_16<kBf16>(widen8<kBf16>(w.x, w.y), q[2 * st], s[kb]);
          s[kb] = mfma_16<kBf16>(widen8<kBf16>(w.z, w.w), q[2 * st + 1], s[kb]);
        }
      } else {
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          const attn_u32x4 w = *reinterpret_cast<const attn_u32x4*>(kslot + r * Tile::kRow + 16 * ((4 * st + g) ^ Tile::kswizzle(r)));
          s[kb] = mfma_16<kBf16>(w, q[st], s[kb]);
        }
      }
    }
    float vs[2][4];
    if constexpr (kQuant) {
      const float* sc = scales + 64 * (t & 1);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const float4 ks4 = *reinterpret_cast<const float4*>(sc + 16 * kb + 4 * g), vs4 = *reinterpret_cast<const float4*>(sc + 32 + 16 * kb + 4 * g);
        s[kb] = v4f{s[kb][0] * ks4.x, s[kb][1] * ks4.y, s[kb][2] * ks4.z, s[kb][3] * ks4.w};
        vs[kb][0] = vs4.x, vs[kb][1] = vs4.y, vs[kb][2] = vs4.z, vs[kb][3] = vs4.w;
        if constexpr (kAgain)
#pragma unroll
          for (int i = 0; i < 4; ++i) vs[kb][i] *= kSmaller;
      }
    }
    wait_lds_reads();                 // K's slot is free
    if (more) {
      if (t + 1 - held >= kTableHalves / 2) fill(t + 1);
      load_k(t + 1);
    }
    if (valid != 0xFFFFFFFFu) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool is = valid >> (16 * kb + 4 * g + i) & 1;
          s[kb][i] = is ? s[kb][i] : -__builtin_inff();
          if constexpr (kQuant) vs[kb][i] = is ? vs[kb][i] : 0.0f;
        }
    }
    float mt = m;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 4; ++i) mt = __builtin_fmaxf(mt, s[kb][i]);
    mt = four_groups(mt, [](float u, float v) { return __builtin_fmaxf(u, v); });
    if (__any((mt - m) * c > 8.0f)) {
      const float f = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((m - mt) * c);
      m = mt;
      ref = m == -__builtin_inff() ? 0.0f : m;
      l *= f;
#pragma unroll
      for (int i = 0; i < kDB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] *= f;
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        float p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          p[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i + k] - ref, c, kVBf16 ? 0.0f : kF16Lift));   // the difference first: 0 at the largest score, whatever the scale
          l += p[k];
          if constexpr (kQuant) p[k] *= vs[kb][i + k];
        }
        const uint32_t w = pack2<kVBf16>(p[0], p[1]);
        hi[2 * kb + i / 2] = w;
        lo[2 * kb + i / 2] = kVBf16 ? pack2<true>(p[0] - bf16_to_f32(w), p[1] - bf16_to_f32(w >> 16)) : pack2<false>(p[0] - f16_to_f32(w), p[1] - f16_to_f32(w >> 16));
      }
    const attn_u32x4 ph = {hi[0], hi[1], hi[2], hi[3]}, pl = {lo[0], lo[1], lo[2], lo[3]};

    if (more) wait_vm<Tile::kLoads + (kQuant ? 1 : 0)>();   // V of this tile; the next K may be in flight
    else wait_vm<0>();
    if (valid != 0xFFFFFFFFu) {       // rows that do not exist enter the product with weight 0: as zeros, whatever the cache holds there
#pragma unroll
      for (int j = 0; j < Tile::kLoads; ++j) {
        const int r = (64 * j + lane) / Tile::kChunks;
        if (!(valid >> r & 1)) *reinterpret_cast<attn_u32x4*>(vslot + 1024 * j + 16 * lane) = attn_u32x4{0, 0, 0, 0};
      }
      wait_lds_reads();
    }
    const int lv = opaque(lane);
#pragma unroll
    for (int db = 0; db < kDB; ++db) {
      attn_u32x4 w;
      const int g = lv >> 4, lane = lv;
      if constexpr (kQuant) {
        const int i = (lane & 15) >> 1, r = 4 * g + (i & 3) + (i >> 2) * 16;
        const uint2 v = lds_read_transposed8(vslot + r * Tile::kRow + 16 * (db ^ Tile::vswizzle(r)) + 8 * (lane & 1));
        w = widen8<true>(v.x, v.y);
      } else {
        const int r = 4 * g + ((lane & 15) >> 2), ch = 2 * db + ((lane & 3) >> 1);
        const uint2 v0 = lds_read_transposed(vslot + r * Tile::kRow + 16 * (ch ^ Tile::vswizzle(r)) + 8 * (lane & 1));
        const uint2 v1 = lds_read_transposed(vslot + (r + 16) * Tile::kRow + 16 * (ch ^ Tile::vswizzle(r + 16)) + 8 * (lane & 1));
        w = attn_u32x4{v0.x, v0.y, v1.x, v1.y};
        if constexpr (kAgain) {
          float v[8];
          unpack16x8<kVBf16>(w, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= kSmaller;
          w = pack16x8<kVBf16>(v);
        }
      }
      o[db] = mfma_16<kVBf16>(w, ph, o[db]);
      o[db] = mfma_16<kVBf16>(w, pl, o[db]);
      if (db % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // no more operands in flight than this: registers
    }
    wait_lds_reads();                 // V's slot is free
    if (more) load_v(t + 1);
  }

  // The waves' states meet in LDS: O [16 heads][D] in each wave's own slots, its 16-byte chunks permuted by the head.
  l = four_groups(l, [](float u, float v) { return u + v; });
  float* const po = reinterpret_cast<float*>(mine);
#pragma unroll
  for (int db = 0; db < kDB; ++db)
    *reinterpret_cast<float4*>(po + n * D + 4 * ((4 * db + g) ^ n)) = make_float4(o[db][0], o[db][1], o[db][2], o[db][3]);
  if (g == 0) *reinterpret_cast<float4*>(state + (wave * 16 + n) * 4) = make_float4(m, l, any ? 1.0f : 0.0f, 0.0f);
  __syncthreads();
  // Each wave's factor of each head, once, beside what it gives to the sum.
  if (tid < Tile::kWaves * 16) {
    float most = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < Tile::kWaves; ++w) most = __builtin_fmaxf(most, state[(w * 16 + (tid & 15)) * 4]);
    const float4 st = *reinterpret_cast<const float4*>(state + tid * 4);
    const float f = state_factor(st, most, c);
    *reinterpret_cast<float4*>(factors + tid * 4) = make_float4(f, f * st.y, st.z, most);
  }
  __syncthreads();
  const bool whole = t0 == 0 && t1 == nt;
  for (int e = tid; e < heads * (D / 4); e += Tile::kThreads) {
    const int r = e / (D / 4), ch = e % (D / 4);
    float sum = 0.0f, seen = 0.0f, most = 0.0f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < Tile::kWaves; ++w) {
      const float4 st = *reinterpret_cast<const float4*>(factors + (w * 16 + r) * 4);
      const float4 u = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * Tile::kWave) + r * D + 4 * (ch ^ r));
      sum += st.y;
      seen += st.z;
      most = st.w;
      v.x += st.x * u.x, v.y += st.x * u.y, v.z += st.x * u.z, v.w += st.x * u.w;
    }
    if (kVBf16 && !(__builtin_fabsf(v.x) + __builtin_fabsf(v.y) + __builtin_fabsf(v.z) + __builtin_fabsf(v.w) <= 0x1p100f)) *flag = 1;
    if (whole) {
      const float inv = seen > 0.0f ? 1.0f / (sum * (kAgain ? kSmaller : 1.0f)) : 0.0f;
      *reinterpret_cast<uint2*>(a.o + (static_cast<int64_t>(b) * a.Hq + hq0 + r) * D + 4 * ch) = pack4(a.out_type, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    } else {
      float* const p = a.ws + static_cast<int64_t>(blockIdx.x) * Tile::kSlot;
      *reinterpret_cast<float4*>(p + r * D + 4 * ch) = v;
      if (ch == 0) *reinterpret_cast<float4*>(p + 16 * D + 4 * r) = make_float4(most, sum, seen, kAgain ? kSmaller : 1.0f);
    }
  }
  if constexpr (kVBf16 && !kAgain) {
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*flag);
  } else {
    return false;   // (f16 values are too small for it)
  }
}

template <int D, bool kBf16, bool kQuant, bool kWide>
__global__ __launch_bounds__((DecodeTile<D, kQuant, kWide>::kThreads), (std::max(1, DecodeTile<D, kQuant, kWide>::kPerCu * DecodeTile<D, kQuant, kWide>::kWaves / 4)))
void attn_decode_kernel(DecodeArgs a) {
  using Tile = DecodeTile<D, kQuant, kWide>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Tile::kLds];
  // this workgroup's piece: tiles t0 .. t1 - 1 of the nt of sequence b and virtual head hv
  int b, hv, len, t0 = 0, t1, nt;
  if (a.pieces) {
    const Cut cut(a);
    int before = 0, f = 0, np = 0;
    uint64_t here = 0;
    for (int b0 = 0; b0 < a.B && !here; b0 += 64) {
      const int ln = cut.len(a, b0 + (threadIdx.x & 63)), n = cut.pieces(ln), sum = lanes_scan(n * a.hv);
      here = __ballot(before + sum > static_cast<int>(blockIdx.x));
      if (here) {
        f = __builtin_ctzll(here);
        b = b0 + f;
        len = __builtin_amdgcn_readlane(ln, f);
        np = __builtin_amdgcn_readlane(n, f);
        before += __builtin_amdgcn_readlane(sum, f) - np * a.hv;
      } else {
        before += __builtin_amdgcn_readlane(sum, 63);
      }
    }
    if (!here) return;   // fewer pieces than the host allowed for
    const int in = blockIdx.x - before, i = in % np;
    hv = in / np;
    nt = tiles_of(len);
    t0 = static_cast<int>(static_cast<int64_t>(nt) * i / np);
    t1 = static_cast<int>(static_cast<int64_t>(nt) * (i + 1) / np);
  } else {
    b = blockIdx.x / a.hv;
    hv = blockIdx.x % a.hv;
    len = __builtin_amdgcn_readfirstlane(seq_len(a, b));
    t1 = nt = tiles_of(len);
  }

  const DecodePiece piece{b, hv, len, t0, t1, nt};
  if (decode_walk<D, kBf16, kQuant, kWide, false>(a, piece, smem)) decode_walk<D, kBf16, kQuant, kWide, true>(a, piece, smem);
}

// The pieces of one sequence and query head, in the order of the line: their weights first, then D / 4 threads each take 4
// channels of every kParts-th piece.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(DecodeArgs a) {
  constexpr int kLanes = D / 4, kParts = 256 / kLanes, kSlot = 16 * D + 64;
  __shared__ __attribute__((aligned(16))) float part[kParts][D];
  __shared__ float weight[kMostPieces + 1];
  __shared__ float sums[4][4];
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq;
  const int h = hq / a.G, hv = h * a.tiles_of_heads + hq % a.G / 16, r = hq % a.G % 16;
  const int tid = threadIdx.x, lane = tid % kLanes, p = tid / kLanes;
  const float c = a.scale_log2;
  const Cut cut(a);
  int before = 0, pieces = 0;
  for (int b0 = 0; b0 <= b; b0 += 64) {
    const int i = b0 + (tid & 63), n = cut.pieces(cut.len(a, i));
    before += i < b ? n : 0;
    pieces = __builtin_amdgcn_readlane(n, b & 63);   // of sequence b in the last round
  }
  uint16_t* const out = a.o + (static_cast<int64_t>(b) * a.Hq + hq) * D;
  if (pieces == 0) {
    if (p == 0) *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(0, 0);
    return;
  }
  if (pieces == 1) return;   // one workgroup held it whole, and has written it
  const float* const first = a.ws + (static_cast<int64_t>(lanes_total(before)) * a.hv + static_cast<int64_t>(hv) * pieces) * kSlot;
  auto piece = [&](int i) { return first + static_cast<int64_t>(i) * kSlot; };
  // the first pieces' channels and states are requested together: one wait for both
  constexpr int kAhead = 8;
  float4 u[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) u[j] = *reinterpret_cast<const float4*>(piece(std::min(p + j * kParts, pieces - 1)) + r * D + 4 * lane);
  auto state = [&](int i) { return *reinterpret_cast<const float4*>(piece(i) + 16 * D + 4 * r); };
  const float4 mine = state(std::min(tid, pieces - 1));
  float most = mine.x, least = mine.w;
  for (int i = tid + 256; i < pieces; i += 256) {
    const float4 st = state(i);
    most = __builtin_fmaxf(most, st.x);
    least = __builtin_fminf(least, st.w);
  }
#pragma unroll
  for (int m = 1; m < 64; m *= 2) most = __builtin_fmaxf(most, __shfl_xor(most, m));
  least = __any(least != 1.0f) ? kSmaller : 1.0f;
  if ((tid & 63) == 0) sums[0][tid >> 6] = most, sums[3][tid >> 6] = least;
  __syncthreads();
  most = __builtin_fmaxf(__builtin_fmaxf(sums[0][0], sums[0][1]), __builtin_fmaxf(sums[0][2], sums[0][3]));
  least = __builtin_fminf(__builtin_fminf(sums[3][0], sums[3][1]), __builtin_fminf(sums[3][2], sums[3][3]));
  float sum = 0.0f, seen = 0.0f;
  for (int i = tid; i < pieces; i += 256) {
    const float4 st = i == tid ? mine : state(i);
    const float f = state_factor(st, most, c);
    weight[i] = st.w == least ? f : f * kSmaller;
    sum += f * st.y;
    seen += st.z;
  }
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    sum += __shfl_xor(sum, m);
    seen += __shfl_xor(seen, m);
  }
  if ((tid & 63) == 0) sums[1][tid >> 6] = sum, sums[2][tid >> 6] = seen;
  __syncthreads();
  sum = (sums[1][0] + sums[1][1]) + (sums[1][2] + sums[1][3]);
  seen = (sums[2][0] + sums[2][1]) + (sums[2][2] + sums[2][3]);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = p + j * kParts;
    if (i < pieces) {
      const float f = weight[i];
      v.x += f * u[j].x, v.y += f * u[j].y, v.z += f * u[j].z, v.w += f * u[j].w;
    }
  }
#pragma unroll 8
  for (int i = p + kAhead * kParts; i < pieces; i += kParts) {
    const float4 w = *reinterpret_cast<const float4*>(piece(i) + r * D + 4 * lane);
    const float f = weight[i];
    v.x += f * w.x, v.y += f * w.y, v.z += f * w.z, v.w += f * w.w;
  }
  *reinterpret_cast<float4*>(&part[p][4 * lane]) = v;
  __syncthreads();
  if (p) return;
#pragma unroll
  for (int i = 1; i < kParts; ++i) {
    const float4 u = *reinterpret_cast<const float4*>(&part[i][4 * lane]);
    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
  }
  const float inv = seen > 0.0f ? 1.0f / (sum * least) : 0.0f;
  *reinterpret_cast<uint2*>(out + 4 * lane) = pack4(a.out_type, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
}

// Pieces that the line is cut into: so many that those workgroups that get their data later than others get fewer, and few enough
// for the join. (64 x <= 8192, 16-bit, two workgroups a CU: 2, 4, 6, 8 pieces a CU 191, 178, 184, 184 us; one
// of 131071, e4m3, four a CU: 4, 8, 12, 16 pieces 53.7, 58.9, 64, 67.)
static int wanted_pieces() { return std::min(kMostPieces, 4 * cu_count()); }

// A slot for each piece; every sequence and virtual head adds at most one to the wanted number.
template <int D>
static size_t decode_workspace(int64_t B, int64_t hv) {
  return (wanted_pieces() + static_cast<size_t>(B * hv)) * DecodeTile<D, true, false>::kSlot * sizeof(float);
}

template <int D, bool kBf16, bool kQuant, bool kWide>
static hipError_t decode_kernel(const DecodeArgs& a, int64_t grid, hipStream_t s) {
  return launch_kernel((attn_decode_kernel<D, kBf16, kQuant, kWide>), dim3(static_cast<unsigned>(grid)), dim3(DecodeTile<D, kQuant, kWide>::kThreads), 0, s, a);
}
template <int D, bool kBf16, bool kQuant>
static hipError_t decode_launch(DecodeArgs a, hipStream_t s) {
  const int64_t length = static_cast<int64_t>(a.c.width) << a.c.page_shift;
  const int64_t heads = static_cast<int64_t>(a.B) * a.hv;
  // By the longest sequence that the table's width allows, as the lengths are on the device (1 x 509 of 8 heads of 128, e4m3 7.6 us, with a table
  // for 2048 positions or more 9.4; 64 x <= 500, 16-bit 16, for more than 2048 26.6; 128 x <= 2000, e4m3 54.7, 66.9):
  // a head stays in one workgroup, and no join follows, while a wide one's waves have two tiles each (60 x <= 1000 of 8 heads of 128,
  // e4m3: 20.6 us, cut 25.9; 20 x <= 1000 11.1, 13.6; 2 x <= 500, 16-bit 8.8, 9.5) - one tile where sixteen waves would be few heads' only
  // ones (1 x 1000, e4m3: 10.4, cut 9.0; 8 x <= 1000 10.7, 10.5; 1 x 509 7.5, 9.0) - or where there are heads enough to fill half of the
  // places wanted and none takes so long that the others' end leaves it alone (128 x <= 2000 of 8 heads of 128, e4m3: 56, cut 63; 100 x <= 2000,
  // 16-bit 77, 84; 60 x <= 2000 50, 55; 40 x <= 2000, e4m3 33, 29; 100 x <= 2000 of 4 of 256, 16-bit 91, 86).
  using Wide = DecodeTile<D, kQuant, true>;
  const int waves = Wide::kWaves, tiles = waves < 16 || heads > cu_count() / 8 ? 2 : 1;
  if (length <= (heads >= wanted_pieces() / 2 ? 2048 : tiles * kTileKeys * waves))
    return heads <= cu_count() ? decode_kernel<D, kBf16, kQuant, true>(a, heads, s) : decode_kernel<D, kBf16, kQuant, false>(a, heads, s);
  a.pieces = wanted_pieces();
  using Tile = DecodeTile<D, kQuant, false>;
  a.places = std::min(a.pieces, Tile::kPerCu * cu_count());
  a.least = Tile::kWaves;
  const int64_t most = heads * ((length + kTileKeys * a.least - 1) / (kTileKeys * a.least));
  const hipError_t e = decode_kernel<D, kBf16, kQuant, false>(a, std::min<int64_t>(a.pieces + heads, most), s);
  return e != hipSuccess ? e : launch_kernel((attn_join_kernel<D>), dim3(static_cast<unsigned>(a.B * a.Hq)), dim3(256), 0, s, a);
}
template <int D>
static hipError_t decode_for(const DecodeArgs& a, int type, hipStream_t s) {
  if (a.c.ks) return type == PQ_BF16 ? decode_launch<D, true, true>(a, s) : decode_launch<D, false, true>(a, s);
  return type == PQ_BF16 ? decode_launch<D, true, false>(a, s) : decode_launch<D, false, false>(a, s);
}

}  // namespace pq

extern "C" {

size_t pq_attn_decode_workspace_bytes(int B, int Hq, int Hkv, int D) {
  using namespace pq;
  if (B <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv) return 0;
  const int64_t hv = Hkv * ((Hq / Hkv + 15ll) / 16);
  return D == 64 ? decode_workspace<64>(B, hv) : D == 128 ? decode_workspace<128>(B, hv) : D == 256 ? decode_workspace<256>(B, hv) : 0;
}

int pq_attn_decode(const uint16_t* q_d, int64_t ldq, int64_t hsq, int type, const void* kc_d, const void* vc_d, const float* ks_d, const float* vs_d,
                   int64_t pages, int page, const int32_t* table_d, int width, const int32_t* lens_d, int B, int Hq, int Hkv, int D, float scale,
                   uint16_t* o_d, int out_type, void* ws_d, size_t ws_bytes, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_attn_decode";
  if (B < 0 || width < 0) return set_error(PQ_ERR_SHAPE, "%s: B=%d, width=%d: negative", what, B, width);
  int rc = check_attention(what, type, out_type, Hq, Hkv, D, scale);
  if (rc == PQ_OK) rc = check_cache(what, kc_d, vc_d, ks_d, vs_d, pages, page, Hkv, D);
  if (rc == PQ_OK) rc = check_heads(what, "q", q_d, ldq, hsq, B);
  if (rc != PQ_OK) return rc;
  if (static_cast<int64_t>(B) * Hq * 512 > 0xFFFFFFFFll)   // the runtime counts a launch's threads in 32 bits
    return set_error(PQ_ERR_SHAPE, "%s: B=%d sequences of %d heads too many for one call", what, B, Hq);
  if (static_cast<int64_t>(width) * page > INT32_MAX)
    return set_error(PQ_ERR_SHAPE, "%s: width=%d pages of %d rows: sequences of at most 2^31 - 1 positions", what, width, page);
  const int G = Hq / Hkv, tiles_of_heads = (G + 15) / 16;
  if (static_cast<int64_t>(B) * Hkv * tiles_of_heads > (1 << 30) / (static_cast<int64_t>(width) * page / kTileKeys + 1))   // tiles are counted in 32 bits
    return set_error(PQ_ERR_SHAPE, "%s: B=%d tables of %d pages of %d rows too large for one call", what, B, width, page);
  if (B == 0) return PQ_OK;
  if (!o_d || !lens_d || (width && !table_d)) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (!aligned(o_d, 16) || !aligned(lens_d, 4) || !aligned(table_d, 4) || !aligned(ws_d, 16)) return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  const size_t need = pq_attn_decode_workspace_bytes(B, Hq, Hkv, D);
  if (!ws_d || ws_bytes < need) return set_error(PQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, ws_d ? ws_bytes : 0, need);
  const int64_t ob = 2ll * B * Hq * D, cb = cache_bytes(ks_d, pages, page, Hkv, D), sb = scale_bytes(ks_d, pages, page, Hkv), qb = heads_span(ldq, hsq, B, Hq, D);
  for (const auto& [o, n] : {std::pair<const void*, int64_t>{o_d, ob}, {ws_d, static_cast<int64_t>(need)}})
    if (ranges_meet(o, n, q_d, qb) || ranges_meet(o, n, kc_d, cb) || ranges_meet(o, n, vc_d, cb) || ranges_meet(o, n, ks_d, sb) || ranges_meet(o, n, vs_d, sb) ||
        ranges_meet(o, n, table_d, 4ll * B * width) || ranges_meet(o, n, lens_d, 4ll * B))
      return overlap(what);
  if (ranges_meet(o_d, ob, ws_d, static_cast<int64_t>(need))) return overlap(what);
  DecodeArgs a{{kc_d, vc_d, ks_d, vs_d, table_d, pages, pages ? width : 0, Hkv, __builtin_ctz(page)}, q_d, ldq, hsq, lens_d, B, Hq, G,
               Hkv * tiles_of_heads, tiles_of_heads, 0, 0, 0, scale * 1.44269504088896340736f, o_d, out_type, static_cast<float*>(ws_d)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return launch_status(what, D == 64 ? decode_for<64>(a, type, s) : D == 128 ? decode_for<128>(a, type, s) : decode_for<256>(a, type, s));
}

}  // extern "C"
