// Rows in and out of the 4-bit cache (kv4_layout.cuh).
//
// Store: for each kv head and group of 32 dims of a K or V row x,
//   scale = bf16(max|x| / 7),  code = round-half-even(x / scale) in -7 .. 7,
// the codes of exact arithmetic (x and scale have 8 significant bits, which keeps the quotients that are not
// halves away from them). A group that
// holds a NaN or an infinity gets a NaN scale and stands for NaN throughout; a group of zeros has
// scale 0 and codes 0. Load writes bf16(scale * code), rounded once.
//
// Both are bound by HBM: a (token, kv head) is 4 D bytes of bf16 K and V and 18/16 D bytes of cache.
// Eight dims per lane (one 16-byte access of the bf16 row), four lanes per group: the group's maximum
// is two shuffles.
#include "attn_common.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kv4_layout.cuh"

namespace cb {
namespace {

constexpr int kThreads = 256;
constexpr int kRunThreads = 64, kRunBlocks = 10;  // whole records: threads per block, blocks per SM at least
constexpr int64_t kRunUnits = 32768;  // (row, kv head) pairs of a call that is taken by runs, at least

struct Kv4RowParams {
  const int32_t* slots;
  int32_t n;
  int32_t hkv;
  int32_t page_size;
  int64_t n_slots;  // n_pages * page_size
  int32_t* err;
};

// The record of slot `slot`, kv head h, and the token's place in it.
template <int D>
__device__ __forceinline__ int64_t record_offset(int32_t slot, int h, int hkv, int page_size) {
  const int32_t page = slot / page_size, in_page = slot - page * page_size;
  const int32_t blocks = page_size / kKv4Block;
  return (((int64_t)page * hkv + h) * blocks + in_page / kKv4Block) * Kv4<D>::kRecord;
}

// One lane's work item: unit (row, kv head, K or V), 8 dims l * 8 of it.
template <int D>
struct Lane {
  int64_t row;
  int h, kv, l;
  int32_t slot;  // -1: nothing to do
};

template <int D>
__device__ __forceinline__ Lane<D> lane_of(const Kv4RowParams& p) {
  constexpr int kLanes = D / 8;  // lanes per (row, head, K or V)
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t unit = i / kLanes;
  Lane<D> x;
  x.l = (int)(i % kLanes);
  x.kv = (int)(unit & 1);
  const int64_t rh = unit >> 1;
  x.row = rh / p.hkv;
  x.h = (int)(rh - x.row * p.hkv);
  x.slot = x.row < p.n ? p.slots[x.row] : -1;
  if (x.slot >= p.n_slots) {
    if (x.l == 0 && x.kv == 0 && x.h == 0) record_error(p.err, kErrIndex, (int32_t)x.row);
    x.slot = -1;
  }
  return x;
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// What a group's codes are made with: its scale's bf16 bits and the scale's reciprocal (0: the scale is 0, too
// small for one, or not finite).
struct Step {
  uint32_t bits;
  float inverse;
};
// Of a group whose largest magnitude has the bf16 bits `top` (0x7f80 and up: not finite). top times
// fp32's 1 / 7 rounds to the same bf16 as the quotient: with top = m 2^e, m an integer of 8 bits, m / 7 is
// either an integer (a bf16) or at least 1 / 112 away from a midpoint of two bf16s, which are odd
// multiples of 1 / 16 there (1 / 14 of a last place among subnormals), far above fp32's error.
__device__ __forceinline__ Step step_of(uint32_t top) {
  const float seventh = __uint_as_float(top << 16) * (1.0f / 7.0f);
  const __nv_bfloat16 scale = __float2bfloat16_rn(seventh);
  Step s;
  s.bits = top < 0x7f80u ? (uint32_t)__bfloat16_as_ushort(scale) : 0x7fc0u;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.inverse) : "f"(__bfloat162float(scale)));  // within 2^-22 of it
  if (!(seventh > 1e-36f && seventh < 1e38f)) s.inverse = 0.0f;
  return s;
}

// The codes (+ 8) of two values x and y of a group, as the low bits of the halves of the result, with the
// fp32 bits of 1.5 * 2^23 above them. The quotient q = x / scale needs its ties exact. Both have 8
// significant bits, so q is a half or at least 2^-9 away from one: rounded to multiples of 2^-10 (an
// addition of 1.5 * 2^13) the product with the reciprocal, |q| 2^-21 off at most, gives a half where q is
// one and stays on q's side of it elsewhere. The second sum is exact up to its rounding to an
// integer, ties to even. |code| <= 7 since the scale is within 2^-8 of max|x| / 7. A division per value
// took three times as long as the kernel's loads and stores.
constexpr float kSnap = 12288.0f, kWhole = 12582912.0f;
constexpr uint32_t kWholeBits = 0x4b400000u;
__device__ __forceinline__ uint64_t codes2(uint64_t xy, uint64_t inverse2) {
  return f2_add(f2_fma(xy, inverse2, f2_pack(kSnap, kSnap)), f2_pack(kWhole + 8.0f - kSnap, kWhole + 8.0f - kSnap));
}
// Pairs of codes as nibbles: the code of value i, shifted to at(i) (a compile-time position), summed; the bits
// above each code add up to a constant.
template <int N, typename At>
__device__ __forceinline__ uint32_t nibbles(const uint32_t (&x)[N], const Step& s, At at) {
  const uint64_t inverse2 = f2_pack(s.inverse, s.inverse);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float a, b;
    f2_unpack(codes2(f2_pack(lo16(x[i]), hi16(x[i])), inverse2), a, b);
    word += ((__float_as_uint(a) - kWholeBits) << at(2 * i)) + ((__float_as_uint(b) - kWholeBits) << at(2 * i + 1));
  }
  return word;
}
// The same of a group whose scale has no reciprocal in fp32: zeros, subnormal steps (a division each) and groups
// that are not finite (codes 0).
template <int N, typename At>
__device__ __forceinline__ uint32_t odd_nibbles(const uint32_t (&x)[N], uint32_t bits, At at) {
  const float scale = __uint_as_float(bits << 16);
  uint32_t word = 0;
#pragma unroll 1
  for (int i = 0; i < 2 * N; ++i) {
    const float v = i % 2 ? hi16(x[i / 2]) : lo16(x[i / 2]);
    const float c = scale > 0.0f ? rintf(__fdiv_rn(v, scale)) : 0.0f;
    word |= (uint32_t)((int)fminf(fmaxf(c, -7.0f), 7.0f) + 8) << at(i);
  }
  return word;
}
__device__ __noinline__ uint32_t odd_k(uint4 x, uint32_t bits) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  return odd_nibbles(w, bits, [](int e) { return 4 * (e / 2) + 16 * (e % 2); });
}
__device__ __noinline__ uint32_t odd_v(uint2 x, uint32_t bits) {
  const uint32_t w[2] = {x.x, x.y};
  return odd_nibbles(w, bits, [](int e) { return 4 * e; });
}
// 8 values of a K row, values e and e + 1 in the halves; 4 of a V row, one behind the other.
__device__ __forceinline__ uint32_t k_word(const uint4& x, const Step& s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  return s.inverse != 0.0f ? nibbles(w, s, [](int e) { return 4 * (e / 2) + 16 * (e % 2); }) : odd_k(x, s.bits);
}
__device__ __forceinline__ uint32_t v_word(const uint2& x, const Step& s) {
  const uint32_t w[2] = {x.x, x.y};
  return s.inverse != 0.0f ? nibbles(w, s, [](int e) { return 4 * e; }) : odd_v(x, s.bits);
}

// One work item of a converged warp: its values, and what becomes of them.
template <int D>
__device__ __forceinline__ uint4 row_values(const uint8_t* k, const uint8_t* v, const Kv4RowParams& p, const Lane<D>& x) {
  return x.slot >= 0 ? ld_stream((x.kv ? v : k) + ((x.row * p.hkv + x.h) * D + x.l * 8) * 2) : make_uint4(0, 0, 0, 0);
}
template <int D>
__device__ __forceinline__ void store_row(const uint4& raw, uint8_t* cache, const Kv4RowParams& p, const Lane<D>& x) {
  // the group's largest magnitude as bf16 bits (ordered like the magnitudes; 0x7f80 and up: not finite)
  uint32_t top = 0;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (x.slot < 0) return;
  const Step step = step_of(top);
  constexpr int NG = Kv4<D>::kGroups;
  const int g = x.l / 4, c = x.l % 4, t = x.slot % kKv4Block;
  uint8_t* rec = cache + record_offset<D>(x.slot, x.h, p.hkv, p.page_size);
  if (x.kv == 0) {
    *reinterpret_cast<uint32_t*>(rec + t * (D / 2) + (c * NG + g) * 4) = k_word(raw, step);
  } else {
    uint8_t* vb = rec + Kv4<D>::kV + (t / 8) * Kv4<D>::kPlane + (t % 8 / 2) * (4 * NG) + g * 4 + (t % 2) * 2;
    *reinterpret_cast<uint16_t*>(vb + 2 * c * (16 * NG)) = (uint16_t)v_word(make_uint2(raw.x, raw.y), step);
    *reinterpret_cast<uint16_t*>(vb + (2 * c + 1) * (16 * NG)) = (uint16_t)v_word(make_uint2(raw.z, raw.w), step);
  }
  if (c == 0)
    *reinterpret_cast<uint16_t*>(rec + Kv4<D>::kScales + t * (4 * NG) + x.kv * (2 * NG) + g * 2) = (uint16_t)step.bits;
}

// A lane's 8 codes of a stored row (two values of K in the halves, four of V one behind the other; + 8) and their
// scale's bits.
struct Codes {
  uint32_t word, scale;
};
template <int D>
__device__ __forceinline__ Codes row_codes(const uint8_t* cache, const Kv4RowParams& p, const Lane<D>& x) {
  Codes r{0, 0};
  if (x.slot < 0) return r;
  constexpr int NG = Kv4<D>::kGroups;
  const int g = x.l / 4, c = x.l % 4, t = x.slot % kKv4Block;
  const uint8_t* rec = cache + record_offset<D>(x.slot, x.h, p.hkv, p.page_size);
  r.scale = __ldg(reinterpret_cast<const uint16_t*>(rec + Kv4<D>::kScales + t * (4 * NG) + x.kv * (2 * NG) + g * 2));
  if (x.kv == 0) {
    r.word = __ldg(reinterpret_cast<const uint32_t*>(rec + t * (D / 2) + (c * NG + g) * 4));
  } else {
    const uint8_t* vb = rec + Kv4<D>::kV + (t / 8) * Kv4<D>::kPlane + (t % 8 / 2) * (4 * NG) + g * 4 + (t % 2) * 2;
    r.word = __ldg(reinterpret_cast<const uint16_t*>(vb + 2 * c * (16 * NG))) |
             (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(vb + (2 * c + 1) * (16 * NG))) << 16;
  }
  return r;
}
template <int D>
__device__ __forceinline__ void load_row(uint8_t* k, uint8_t* v, const Codes& r, const Kv4RowParams& p, const Lane<D>& x) {
  if (x.slot < 0) return;
  const float step = __uint_as_float(r.scale << 16);
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    f[e] = step * (float)((int)(r.word >> (x.kv == 0 ? 4 * (e / 2) + 16 * (e % 2) : 4 * e) & 15) - 8);
  st_stream((x.kv ? v : k) + ((x.row * p.hkv + x.h) * D + x.l * 8) * 2, pack8(f));
}

template <int D, bool STORE>
__global__ void __launch_bounds__(kThreads) kv4_rows_kernel(uint8_t* k, uint8_t* v, uint8_t* cache, const Kv4RowParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const Lane<D> x = lane_of<D>(p);
  if (STORE)
    store_row<D>(row_values<D>(k, v, p, x), cache, p, x);
  else
    load_row<D>(k, v, row_codes<D>(cache, p, x), p, x);
}

// ---- whole records ---------------------------------------------------------------------------------
//
// Chunks fill pages in order, so most rows of a large call come in runs of 16 neighbours that are one
// record (slots 16 m .. 16 m + 15). A warp takes one kv head of such a run with the decode kernel's lane
// layout: 16-byte accesses of the record, 64-byte pieces of the bf16 rows, groups reduced by shuffles,
// and two values per instruction where the arithmetic is exact in bf16 (a nibble widened to
// 128 + nibble; minus 136; times the scale, one rounding). A warp asks for all its bytes first (the store's 8 KB
// of K and V: 64 registers a lane) and blocks are of two warps: of eight, they hold their registers until the last
// warp is through, and the store takes 40 us instead of 31; with registers for 12 blocks an SM, 36.
// 32,768 rows of 8 heads of 128 dims (172 MB, 25.7 us at the copy rate): store 31 us, load 27; row by row, where
// V's nibbles are 2-byte accesses in eight sectors per row, 70 and 59.

// What a warp finds in the 16 rows from `row0` on.
struct Window {
  int start;      // row of a whole record that begins here, -1: none
  uint32_t rest;  // rows (bit i: row0 + i) that belong to no whole record and have a slot
};

__device__ __forceinline__ Window look_at(const Kv4RowParams& p, int64_t row0, int lane) {
  // slots of rows row0 - 16 .. row0 + 47, two per lane (-1 outside the rows)
  const int64_t a = row0 - 16 + lane, b = a + 32;
  const int32_t sa = a >= 0 && a < p.n ? p.slots[a] : -1, sb = b < p.n ? p.slots[b] : -1;
  // bit i: row row0 - 16 + i is followed by the next slot
  const int32_t sa1 = __shfl_down_sync(0xffffffffu, sa, 1), sb1 = __shfl_down_sync(0xffffffffu, sb, 1);
  const int32_t sb0 = __shfl_sync(0xffffffffu, sb, 0);
  const bool fa = sa >= 0 && sa == (lane == 31 ? sb0 : sa1) - 1, fb = lane < 31 && sb >= 0 && sb == sb1 - 1;
  const uint64_t follows = (uint64_t)__ballot_sync(0xffffffffu, fb) << 32 | __ballot_sync(0xffffffffu, fa);
  // bit i: a whole record inside the cache begins at row row0 - 16 + i (i < 32)
  const bool whole = sa >= 0 && sa % kKv4Block == 0 && (int64_t)sa + kKv4Block <= p.n_slots &&
                     ((follows >> lane) & 0x7fffu) == 0x7fffu;
  const uint32_t starts = __ballot_sync(0xffffffffu, whole);
  uint32_t covered = 0;  // bit i: row row0 + i
#pragma unroll
  for (int d = 0; d < kKv4Block; ++d) covered |= (uint32_t)(((uint64_t)starts << d) >> 16);
  Window w;
  w.start = starts >> 16 ? __ffs(starts >> 16) - 1 : -1;
  // slots of the window's rows: lanes 16 .. 31
  w.rest = (__ballot_sync(0xffffffffu, sa >= 0) >> 16) & ~covered & 0xffffu;
  return w;
}

__device__ __forceinline__ uint2 ld_stream2(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {  // of two bf16 pairs' magnitudes, by half
  return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t shuffled_max2(uint32_t x, int d) {
  return __vmaxu2(x, __shfl_xor_sync(0xffffffffu, x, d));
}

template <int NG>
__device__ __forceinline__ void put_words(uint8_t* p, const uint32_t (&w)[NG]) {
  if constexpr (NG == 4)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int NG>
__device__ __forceinline__ void get_words(const uint8_t* p, uint32_t (&w)[NG]) {
  if constexpr (NG == 4) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x, w[1] = x.y;
  }
}

// Rows row .. row + 15 of kv head h into their record.
template <int D>
__device__ __forceinline__ void store_record(const uint8_t* k, const uint8_t* v, uint8_t* rec, int64_t row, int h,
                                             int hkv, int lane) {
  constexpr int NG = Kv4<D>::kGroups;
  const int r = lane / 4, c = lane % 4;
  const int64_t pitch = (int64_t)hkv * D * 2, base = row * pitch + (int64_t)h * D * 2;
  // K: tokens r and r + 8, 8 dims of each group per lane
  uint4 kx[2][NG];
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int g = 0; g < NG; ++g) kx[half][g] = ld_stream(k + base + (r + 8 * half) * pitch + g * 64 + c * 16);
  // V: tokens 8 half + 2 c and + 1, dims 32 g + 4 r .. of each group per lane
  uint2 vx[2][2][NG];
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int g = 0; g < NG; ++g)
        vx[half][o][g] = ld_stream2(v + base + (8 * half + 2 * c + o) * pitch + g * 64 + r * 8);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t word[NG], bits[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint4& x = kx[half][g];
      uint32_t m = __vmaxu2(abs_max2(x.x, x.y), abs_max2(x.z, x.w));
      m = shuffled_max2(shuffled_max2(m, 1), 2);
      const Step step = step_of(max(m & 0xffffu, m >> 16));
      bits[g] = step.bits;
      word[g] = k_word(x, step);
    }
    put_words<NG>(rec + half * Kv4<D>::kPlane + lane * (4 * NG), word);
    if (c == 0)
#pragma unroll
      for (int g = 0; g < NG; g += 2)
        *reinterpret_cast<uint32_t*>(rec + Kv4<D>::kScales + (r + 8 * half) * (4 * NG) + g * 2) = bits[g] | bits[g + 1] << 16;
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t word[NG], bits[2][NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // both tokens' maxima in one register
      const uint2 &x0 = vx[half][0][g], &x1 = vx[half][1][g];
      const uint32_t m0 = abs_max2(x0.x, x0.y), m1 = abs_max2(x1.x, x1.y);
      uint32_t m = __vmaxu2(__byte_perm(m0, m1, 0x5410), __byte_perm(m0, m1, 0x7632));
      m = shuffled_max2(shuffled_max2(shuffled_max2(m, 4), 8), 16);
      const Step s0 = step_of(m & 0xffffu), s1 = step_of(m >> 16);
      bits[0][g] = s0.bits;
      bits[1][g] = s1.bits;
      word[g] = v_word(x0, s0) + (v_word(x1, s1) << 16);
    }
    put_words<NG>(rec + Kv4<D>::kV + half * Kv4<D>::kPlane + lane * (4 * NG), word);
    if (r == 0)
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int g = 0; g < NG; g += 2)
          *reinterpret_cast<uint32_t*>(rec + Kv4<D>::kScales + (8 * half + 2 * c + o) * (4 * NG) + 2 * NG + g * 2) =
              bits[o][g] | bits[o][g + 1] << 16;
  }
}

// A pair of nibbles at bits 0 and 16 as bf16 codes (exact), times a pair of scales (one rounding).
__device__ __forceinline__ uint32_t codes_times(uint32_t nibbles, uint32_t scales) {
  const uint32_t w = (nibbles & 0x000f000fu) | 0x43004300u;  // 128 + nibble
  const __nv_bfloat162 code = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&w), __floats2bfloat162_rn(136.0f, 136.0f));
  const __nv_bfloat162 x = __hmul2_rn(code, *reinterpret_cast<const __nv_bfloat162*>(&scales));
  return *reinterpret_cast<const uint32_t*>(&x);
}

// A record's 16 rows of kv head h.
template <int D>
__device__ __forceinline__ void load_record(uint8_t* k, uint8_t* v, const uint8_t* rec, int64_t row, int h, int hkv,
                                            int lane) {
  constexpr int NG = Kv4<D>::kGroups;
  const int r = lane / 4, c = lane % 4;
  const int64_t pitch = (int64_t)hkv * D * 2, base = row * pitch + (int64_t)h * D * 2;
  uint32_t kw[2][NG], vw[2][NG], ksc[2][NG / 2], vsc[2][2][NG / 2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    get_words<NG>(rec + half * Kv4<D>::kPlane + lane * (4 * NG), kw[half]);
    get_words<NG>(rec + Kv4<D>::kV + half * Kv4<D>::kPlane + lane * (4 * NG), vw[half]);
#pragma unroll
    for (int g = 0; g < NG / 2; ++g) {
      const uint8_t* sc = rec + Kv4<D>::kScales + g * 4;
      ksc[half][g] = __ldg(reinterpret_cast<const uint32_t*>(sc + (r + 8 * half) * (4 * NG)));
#pragma unroll
      for (int o = 0; o < 2; ++o)
        vsc[half][o][g] = __ldg(reinterpret_cast<const uint32_t*>(sc + (8 * half + 2 * c + o) * (4 * NG) + 2 * NG));
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // K: dims 8 c .. of the group, two neighbours per product
      const uint32_t s2 = __byte_perm(ksc[half][g / 2], 0, g % 2 ? 0x3232 : 0x1010);
      const uint32_t w = kw[half][g];
      st_stream(k + base + (r + 8 * half) * pitch + g * 64 + c * 16,
                make_uint4(codes_times(w, s2), codes_times(w >> 4, s2), codes_times(w >> 8, s2), codes_times(w >> 12, s2)));
      // V: dims 4 r .. of the group, tokens 2 c (low halves) and 2 c + 1 (high) per product
      const uint32_t t2 = __byte_perm(vsc[half][0][g / 2], vsc[half][1][g / 2], g % 2 ? 0x7632 : 0x5410);
      const uint32_t y = vw[half][g];
      const uint32_t d0 = codes_times(y, t2), d1 = codes_times(y >> 4, t2), d2 = codes_times(y >> 8, t2),
                     d3 = codes_times(y >> 12, t2);
      uint8_t* to = v + base + (8 * half + 2 * c) * pitch + g * 64 + r * 8;
      *reinterpret_cast<uint2*>(to) = make_uint2(__byte_perm(d0, d1, 0x5410), __byte_perm(d2, d3, 0x5410));
      *reinterpret_cast<uint2*>(to + pitch) = make_uint2(__byte_perm(d0, d1, 0x7632), __byte_perm(d2, d3, 0x7632));
    }
}

// A warp per 16 rows and kv head: the whole record that begins in them, then the rows of no whole
// record one by one (half a warp for K, half for V).
template <int D, bool STORE>
__global__ void __launch_bounds__(kRunThreads, kRunBlocks)
    kv4_runs_kernel(uint8_t* k, uint8_t* v, uint8_t* cache, const Kv4RowParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const int64_t unit = ((int64_t)blockIdx.x * kRunThreads + threadIdx.x) / 32;
  const int64_t row0 = unit / p.hkv * kKv4Block;
  const int h = (int)(unit % p.hkv);
  if (row0 >= p.n) return;
  const Window w = look_at(p, row0, lane);
  if (w.start >= 0) {
    const int64_t row = row0 + w.start;
    uint8_t* rec = cache + record_offset<D>(p.slots[row], h, p.hkv, p.page_size);
    if (STORE)
      store_record<D>(k, v, rec, row, h, p.hkv, lane);
    else
      load_record<D>(k, v, rec, row, h, p.hkv, lane);
  }
  for (uint32_t rest = w.rest; rest != 0;) {  // four rows at a time, so that their reads overlap
    constexpr int kRows = 4;
    Lane<D> x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      x[i].row = row0 + (rest != 0 ? __ffs(rest) - 1 : 0);
      x[i].h = h;
      x[i].kv = lane / 16;
      x[i].l = lane % 16;
      x[i].slot = rest != 0 && x[i].l < D / 8 ? p.slots[x[i].row] : -1;
      if (x[i].slot >= p.n_slots) {
        if (h == 0 && lane == 0) record_error(p.err, kErrIndex, (int32_t)x[i].row);
        x[i].slot = -1;
      }
      rest &= rest - 1;  // (stays 0)
    }
    if constexpr (STORE) {
      uint4 raw[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) raw[i] = row_values<D>(k, v, p, x[i]);
#pragma unroll
      for (int i = 0; i < kRows; ++i) store_row<D>(raw[i], cache, p, x[i]);
    } else {
      Codes r[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) r[i] = row_codes<D>(cache, p, x[i]);
#pragma unroll
      for (int i = 0; i < kRows; ++i) load_row<D>(k, v, r[i], p, x[i]);
    }
  }
}

template <int D, bool STORE>
cudaError_t launch_rows(void* k, void* v, void* cache, const Kv4RowParams& p, cudaStream_t s) {
  // By runs from kRunUnits (row, kv head) pairs on, where there are warps enough that take 16 rows each; row by row
  // below. Whole pages, by runs against row by row, store / load in us: 8 heads of 128 dims 2,048 rows 6.1 / 4.7 against
  // 5.2 / 4.6, 4,096 rows 6.6 / 4.5 against 9.1 / 7.8; 2 heads of 128, 8,192 rows 6.0 / 4.7 against 5.2 / 4.6, 16,384 rows
  // 6.5 / 4.5 against 9.1 / 7.8; one head of 64, 16,384 rows 4.0 / 2.9 against 3.4 / 3.0, 32,768 rows 4.4 / 3.8 against
  // 5.2 / 4.5; 16 heads of 128, 1,024 rows 6.1 / 4.6 against 5.3 / 4.6, 2,048 rows 6.7 / 4.5 against 9.4 / 7.8. (Loads
  // of whole pages are up to 1.1 faster by runs from 2,048 pairs on.) Scattered slots cost the other way: 32,768 pairs
  // 13.7 / 11.8 against 9.1 / 7.8 with 128 dims, 17.2 / 16.4 against 5.3 / 4.6 with 64, 8,192 pairs 9.8 / 8.8 against
  // 3.4 / 3.0; 262,144 pairs 72 / 66 against 71 / 65.
  const bool runs = (int64_t)p.n * p.hkv >= kRunUnits;
  const int64_t lanes = runs ? ((int64_t)p.n + kKv4Block - 1) / kKv4Block * p.hkv * 32 : (int64_t)p.n * p.hkv * 2 * (D / 8);
  const int threads = runs ? kRunThreads : kThreads;
  const int64_t blocks = (lanes + threads - 1) / threads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_pdl(runs ? kv4_runs_kernel<D, STORE> : kv4_rows_kernel<D, STORE>, dim3((unsigned)blocks), dim3(threads), 0, s,
                    static_cast<uint8_t*>(k), static_cast<uint8_t*>(v), static_cast<uint8_t*>(cache), p);
}

}  // namespace

cudaError_t launch_kv4_rows(bool store, void* k, void* v, const int32_t* slots, int32_t n, void* cache,
                            int32_t n_pages, int32_t page_size, int32_t hkv, int32_t head_dim, int32_t* err,
                            cudaStream_t s) {
  if (n <= 0) return cudaSuccess;
  const Kv4RowParams p{slots, n, hkv, page_size, (int64_t)n_pages * page_size, err};
  if (head_dim == 128) return store ? launch_rows<128, true>(k, v, cache, p, s) : launch_rows<128, false>(k, v, cache, p, s);
  if (head_dim == 64) return store ? launch_rows<64, true>(k, v, cache, p, s) : launch_rows<64, false>(k, v, cache, p, s);
  return cudaErrorInvalidValue;
}

}  // namespace cb
