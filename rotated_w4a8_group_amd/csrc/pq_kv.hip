// The key-value cache of the attention layers: rows quantised as they are written into its pages (pq_kv_write)
// and sequences read back (pq_kv_read).
//
// A cache is [pages][Hkv][page][D], so a head's rows of one page are one contiguous run, which is what the
// attention streams. Rows are e4m3 codes with one binary32 scale for each (row, head) in [pages][Hkv][page], or the
// 16-bit values themselves. Per row x of D values (the encoder and the scale are those of the prologue's groups):
//   s = fl32(max |x| * fl32(1/448)),  code_i = E(fl32(x_i * fl32(1/s))),  read back as fl(code_i * s).
//
// Both kernels move bytes. D / 8 lanes hold a (row, head) pair, 8 values of k and 8 of v each, so that a wave takes 8 pairs of 64, 4 of
// 128 or 2 of 256 values, the heads of a row next to each other; a maximum is a reduction over those lanes. Writing 4038 rows
// of 8 heads of 128 (25 MB) takes 7.9 us, of which a launch is 2.6 (k and v in lanes of their own: 9.2), and every
// lane's one chain of loads, maximum, division and store most of the rest: all workgroups are on the device at once.
#include <algorithm>

#include "pq_attn.h"

namespace pq {

struct KvWriteArgs {
  const uint16_t* src[2];   // k, v
  int64_t ld[2], hs[2];
  void* cache[2];
  float* scale[2];
  const int64_t* slots;
  int64_t nslots;           // pages * page
  int T, Hkv, page_shift;
};

// The largest of a non-negative value over the L lanes of a row.
template <int L>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int m = 1; m < L; m *= 2) v = __builtin_fmaxf(v, __shfl_xor(v, m));
  return v;
}

template <int D, bool kBf16, bool kQuant>
__global__ __launch_bounds__(256) void kv_write_kernel(KvWriteArgs a) {
  constexpr int L = D / 8, R = 256 / L;   // lanes of a row, rows of a workgroup
  // unit = (token, head): the heads of a token stand next to each other in the source
  const uint32_t unit = blockIdx.x * R + threadIdx.x / L, t = unit / a.Hkv, h = unit - t * a.Hkv;
  const int lane = threadIdx.x % L;
  if (t >= static_cast<uint32_t>(a.T)) return;     // whole rows leave: the lanes of a row stay together
  const int64_t slot = a.slots[t];
  attn_u32x4 q[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) q[w] = __builtin_nontemporal_load(reinterpret_cast<const attn_u32x4*>(a.src[w] + t * a.ld[w] + h * a.hs[w] + 8 * lane));
  if (slot < 0 || slot >= a.nslots) return;
  const int64_t row = (((slot >> a.page_shift) * a.Hkv + h) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
  if constexpr (!kQuant) {
#pragma unroll
    for (int w = 0; w < 2; ++w) *reinterpret_cast<attn_u32x4*>(static_cast<uint16_t*>(a.cache[w]) + row * D + 8 * lane) = q[w];
  } else {
    float v[2][8], most[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      unpack16x8<kBf16>(q[w], v[w]);
      // a row with an infinity or a NaN gets the scale NaN and the codes 0: it reads back as NaN
      most[w] = 0.0f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        most[w] = __builtin_fmaxf(most[w], __builtin_fabsf(v[w][i]));
        bad = bad || !(__builtin_fabsf(v[w][i]) <= 3.4e38f);
      }
      if (bad) most[w] = __builtin_inff();
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      most[w] = row_max<L>(most[w]);
      float s = most[w] * (1.0f / 448.0f);
      if (s < 1.17549435e-38f) s = 0.0f;   // its reciprocal would overflow: such a row counts as zero
      const bool finite = most[w] <= 3.4e38f;
      const float inv = s > 0.0f && finite ? 1.0f / s : 0.0f;
      if (!finite) s = __builtin_nanf("");
      uint32_t c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = e4m3_encode2(v[w][4 * i] * inv, v[w][4 * i + 1] * inv) | e4m3_encode2(v[w][4 * i + 2] * inv, v[w][4 * i + 3] * inv) << 16;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.cache[w]) + row * D + 8 * lane) = make_uint2(c[0], c[1]);
      if (lane == 0) a.scale[w][row] = s;
    }
  }
}

struct KvReadArgs {
  CacheArgs c;
  const int32_t* cu;
  int B, T;
  uint16_t* out[2];
};

// kReadUnits: (row, head) pairs of a lane, whose loads are in flight together.
template <int D, bool kBf16, bool kQuant, int kReadUnits>
__global__ __launch_bounds__(256) void kv_read_kernel(KvReadArgs a) {
  constexpr int kBytes = D * (kQuant ? 1 : 2), L = D / 8, R = 256 / L;   // bytes of a row, its lanes, rows of a workgroup at a time
  const uint32_t unit0 = blockIdx.x * (R * kReadUnits) + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  uint32_t t = unit0 / a.c.Hkv;
  if (t >= static_cast<uint32_t>(a.T)) return;
  // the sequence of row t: the last b with cu[b] <= t
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= static_cast<int64_t>(t)) lo = mid;
    else hi = mid;
  }
  int64_t row[kReadUnits], to[kReadUnits];   // row -1: a page outside the cache; to -1: nothing to write
#pragma unroll
  for (int i = 0; i < kReadUnits; ++i) {
    const uint32_t unit = unit0 + i * R;
    t = unit / a.c.Hkv;
    const uint32_t h = unit - t * a.c.Hkv;
    row[i] = to[i] = -1;
    if (t < static_cast<uint32_t>(a.T)) {
      while (lo + 1 < a.B && a.cu[lo + 1] <= static_cast<int64_t>(t)) ++lo;
      const int64_t first = a.cu[lo];
      if (t >= first && t < static_cast<int64_t>(a.cu[lo + 1])) {   // rows of no sequence stay as they are
        to[i] = static_cast<int64_t>(unit) * D + 8 * lane;
        row[i] = cache_row(a.c, lo, h, t - first);
      }
    }
  }
  attn_u32x4 q[kReadUnits][2];
  float s[kReadUnits][2];
#pragma unroll
  for (int i = 0; i < kReadUnits; ++i)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      q[i][w] = attn_u32x4{0, 0, 0, 0};
      s[i][w] = 0.0f;
      if (row[i] >= 0) {
        const uint8_t* const from = static_cast<const uint8_t*>(w ? a.c.v : a.c.k) + row[i] * kBytes + kBytes / L * lane;
        if constexpr (kQuant) {
          const uint2 c = __builtin_bit_cast(uint2, __builtin_nontemporal_load(reinterpret_cast<const uint64_t*>(from)));
          q[i][w].x = c.x, q[i][w].y = c.y;
          s[i][w] = (w ? a.c.vs : a.c.ks)[row[i]];
        } else {
          q[i][w] = __builtin_nontemporal_load(reinterpret_cast<const attn_u32x4*>(from));
        }
      }
    }
#pragma unroll
  for (int i = 0; i < kReadUnits; ++i)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (to[i] < 0) continue;
      if constexpr (kQuant) {
        float v[8];
        decode8(make_uint2(q[i][w].x, q[i][w].y), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= s[i][w];
        q[i][w] = pack16x8<kBf16>(v);
      }
      __builtin_nontemporal_store(q[i][w], reinterpret_cast<attn_u32x4*>(a.out[w] + to[i]));
    }
}

template <int D>
static hipError_t write_launch(const KvWriteArgs& a, int type, unsigned grid, hipStream_t s) {
  if (a.scale[0] && type == PQ_BF16) return launch_kernel((kv_write_kernel<D, true, true>), dim3(grid), dim3(256), 0, s, a);
  if (a.scale[0]) return launch_kernel((kv_write_kernel<D, false, true>), dim3(grid), dim3(256), 0, s, a);
  return launch_kernel((kv_write_kernel<D, false, false>), dim3(grid), dim3(256), 0, s, a);   // bits are copied, whatever their type
}
// One pair a lane while all of them are on the device together (65 rows of 4 heads of 256: 2.8 us, with four 4.6), else four (7
// sequences of up to 8191 rows, 268 MB: 53.6 us, 5.0 TB/s; with one, two, eight 64, 60, 57; stores that stay in the caches 57.5; heads
// of a page one after the other instead of a row's heads side by side, so that stores are a head wide, 60 to 63).
template <int D, bool kBf16, bool kQuant>
static hipError_t read_kernel(const KvReadArgs& a, hipStream_t s) {
  constexpr int R = 256 / (D / 8);
  const int64_t pairs = static_cast<int64_t>(a.T) * a.c.Hkv, blocks = (pairs + R - 1) / R;
  if (blocks <= 8 * cu_count()) return launch_kernel((kv_read_kernel<D, kBf16, kQuant, 1>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a);
  return launch_kernel((kv_read_kernel<D, kBf16, kQuant, 4>), dim3(static_cast<unsigned>((blocks + 3) / 4)), dim3(256), 0, s, a);
}
template <int D>
static hipError_t read_launch(const KvReadArgs& a, int type, hipStream_t s) {
  if (a.c.ks) return type == PQ_BF16 ? read_kernel<D, true, true>(a, s) : read_kernel<D, false, true>(a, s);
  return read_kernel<D, false, false>(a, s);
}

constexpr int64_t kMostCacheRows = 1ll << 40;   // 70 TB of them: its bytes are counted in 64 bits

int64_t cache_bytes(const float* scales, int64_t pages, int page, int Hkv, int D) { return pages * page * Hkv * D * (scales ? 1 : 2); }
int64_t scale_bytes(const float* scales, int64_t pages, int page, int Hkv) { return scales ? 4 * pages * page * Hkv : 0; }

int check_cache(const char* what, const void* kc, const void* vc, const float* ks, const float* vs, int64_t pages, int page, int Hkv, int D) {
  if (D != 64 && D != 128 && D != 256) return set_error(PQ_ERR_SHAPE, "%s: head size D=%d must be 64, 128 or 256", what, D);
  if (Hkv <= 0 || Hkv > kAttnMaxHeads) return set_error(PQ_ERR_SHAPE, "%s: Hkv=%d must be in 1..%d", what, Hkv, kAttnMaxHeads);
  if (page < 16 || page > 1024 || (page & (page - 1)))
    return set_error(PQ_ERR_SHAPE, "%s: page=%d must be a power of two in 16..1024", what, page);
  if (pages < 0 || pages > INT32_MAX) return set_error(PQ_ERR_SHAPE, "%s: pages=%lld must be in 0..2^31-1", what, static_cast<long long>(pages));
  if (pages * page * Hkv > kMostCacheRows) return set_error(PQ_ERR_SHAPE, "%s: %lld pages of %d rows and %d heads: at most 2^40 rows of heads", what, static_cast<long long>(pages), page, Hkv);
  if (!ks != !vs) return set_error(PQ_ERR_NULL, "%s: k and v scales go together", what);
  if (pages && (!kc || !vc)) return set_error(PQ_ERR_NULL, "%s: NULL cache", what);
  if (!aligned(kc, 16) || !aligned(vc, 16) || !aligned(ks, 4) || !aligned(vs, 4)) return set_error(PQ_ERR_ALIGN, "%s: misaligned cache", what);
  return PQ_OK;
}

int check_heads(const char* what, const char* name, const void* p, int64_t ld, int64_t hs, int T) {
  if (ld % 8 || hs % 8 || ld < 0 || hs < 0 || ld > kAttnMaxStride || hs > kAttnMaxStride)
    return set_error(PQ_ERR_SHAPE, "%s: strides of %s (%lld, %lld) must be multiples of 8 in 0..2^24", what, name,
                     static_cast<long long>(ld), static_cast<long long>(hs));
  if (T > 0 && !p) return set_error(PQ_ERR_NULL, "%s: %s is NULL", what, name);
  if (!aligned(p, 16)) return set_error(PQ_ERR_ALIGN, "%s: %s must be 16-byte aligned", what, name);
  return PQ_OK;
}

}  // namespace pq

extern "C" {

int pq_kv_write(const uint16_t* k_d, int64_t ldk, int64_t hsk, const uint16_t* v_d, int64_t ldv, int64_t hsv, int type, int T, int Hkv, int D,
                const int64_t* slots_d, void* kc_d, void* vc_d, float* ks_d, float* vs_d, int64_t pages, int page, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_kv_write";
  if (T < 0) return set_error(PQ_ERR_SHAPE, "%s: T=%d < 0", what, T);
  if (type != PQ_F16 && type != PQ_BF16) return set_error(PQ_ERR_SHAPE, "%s: type %d, expected f16 or bf16", what, type);
  int rc = check_cache(what, kc_d, vc_d, ks_d, vs_d, pages, page, Hkv, D);
  if (rc == PQ_OK) rc = check_heads(what, "k", k_d, ldk, hsk, T);
  if (rc == PQ_OK) rc = check_heads(what, "v", v_d, ldv, hsv, T);
  if (rc != PQ_OK) return rc;
  const int64_t rows = static_cast<int64_t>(T) * Hkv, per = 256 / (D / 8), grid = (rows + per - 1) / per;
  if (grid * 256 > 0xFFFFFFFFll) return set_error(PQ_ERR_SHAPE, "%s: T=%d rows too many for one call (split the rows)", what, T);
  if (T == 0) return PQ_OK;
  if (!slots_d) return set_error(PQ_ERR_NULL, "%s: slots is NULL", what);
  if (!aligned(slots_d, 8)) return set_error(PQ_ERR_ALIGN, "%s: slots must be 8-byte aligned", what);
  if (pages == 0) return PQ_OK;   // no slot exists
  const int64_t cb = cache_bytes(ks_d, pages, page, Hkv, D), sb = scale_bytes(ks_d, pages, page, Hkv), kb = heads_span(ldk, hsk, T, Hkv, D), vb = heads_span(ldv, hsv, T, Hkv, D);
  const void* const out[4] = {kc_d, vc_d, ks_d, vs_d};
  const int64_t size[4] = {cb, cb, sb, sb};
  for (int i = 0; i < 4; ++i) {
    if (ranges_meet(out[i], size[i], k_d, kb) || ranges_meet(out[i], size[i], v_d, vb) || ranges_meet(out[i], size[i], slots_d, 8ll * T)) return overlap(what);
    for (int j = 0; j < i; ++j)
      if (ranges_meet(out[i], size[i], out[j], size[j])) return overlap(what);
  }
  KvWriteArgs a{{k_d, v_d}, {ldk, ldv}, {hsk, hsv}, {kc_d, vc_d}, {ks_d, vs_d}, slots_d, pages * page, T, Hkv, __builtin_ctz(page)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const unsigned g = static_cast<unsigned>(grid);
  return launch_status(what, D == 64 ? write_launch<64>(a, type, g, s) : D == 128 ? write_launch<128>(a, type, g, s) : write_launch<256>(a, type, g, s));
}

int pq_kv_read(const void* kc_d, const void* vc_d, const float* ks_d, const float* vs_d, int64_t pages, int page, const int32_t* table_d, int width,
               const int32_t* cu_d, int B, int T, int Hkv, int D, uint16_t* k_d, uint16_t* v_d, int type, pq_stream_t stream) {
  using namespace pq;
  clear_error();
  const char* what = "pq_kv_read";
  if (T < 0 || B < 0 || width < 0) return set_error(PQ_ERR_SHAPE, "%s: T=%d, B=%d, width=%d: negative", what, T, B, width);
  if (type != PQ_F16 && type != PQ_BF16) return set_error(PQ_ERR_SHAPE, "%s: type %d, expected f16 or bf16", what, type);
  const int rc = check_cache(what, kc_d, vc_d, ks_d, vs_d, pages, page, Hkv, D);
  if (rc != PQ_OK) return rc;
  if (static_cast<int64_t>(T) * Hkv * (D / 8) > 0xFFFF0000ll)   // the runtime counts a launch's threads in 32 bits
    return set_error(PQ_ERR_SHAPE, "%s: T=%d rows of %d heads too many for one call (split the sequences)", what, T, Hkv);
  if (T == 0 || B == 0) return PQ_OK;
  if (!k_d || !v_d || !cu_d || (width && !table_d)) return set_error(PQ_ERR_NULL, "%s: NULL pointer", what);
  if (!aligned(k_d, 16) || !aligned(v_d, 16) || !aligned(cu_d, 4) || !aligned(table_d, 4)) return set_error(PQ_ERR_ALIGN, "%s: misaligned pointer", what);
  const int64_t cb = cache_bytes(ks_d, pages, page, Hkv, D), sb = scale_bytes(ks_d, pages, page, Hkv), ob = 2ll * T * Hkv * D;
  for (const void* o : {static_cast<const void*>(k_d), static_cast<const void*>(v_d)})
    if (ranges_meet(o, ob, kc_d, cb) || ranges_meet(o, ob, vc_d, cb) || ranges_meet(o, ob, ks_d, sb) || ranges_meet(o, ob, vs_d, sb) ||
        ranges_meet(o, ob, table_d, 4ll * B * width) || ranges_meet(o, ob, cu_d, 4ll * (B + 1ll)))
      return overlap(what);
  if (ranges_meet(k_d, ob, v_d, ob)) return overlap(what);
  KvReadArgs a{{kc_d, vc_d, ks_d, vs_d, table_d, pages, width, Hkv, __builtin_ctz(page)}, cu_d, B, T, {k_d, v_d}};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return launch_status(what, D == 64 ? read_launch<64>(a, type, s) : D == 128 ? read_launch<128>(a, type, s) : read_launch<256>(a, type, s));
}

}  // extern "C"
