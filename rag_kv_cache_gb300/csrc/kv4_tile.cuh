// Tiles of 128 cached tokens of one kv head widened from the 4-bit cache's records (kv4_layout.cuh) into operands of
// tcgen05.mma in shared memory, shared by the kernels that multiply with them (kv4_chunk.cu, kv4_weights.cu).
//
// fp16 holds a product scale * code exactly (8 significant bits times 3) as long as its exponent fits, which bf16,
// with 8 bits, does not. So a tile is scaled by a power of two: 2^-e_k for its keys, 2^-e_v for its values, from
// the largest scale of each, which puts that scale into [2^12, 2^13), and eight times it below fp16's largest value. Products
// of scales down to 2^-29 of the largest are exact, those of smaller ones within 2^-25 (after scaling): a group of dims
// whose values lie far below the others' keeps its own precision. The powers leave through the softmax's factor and the
// output's.
//   A nibble n = code + 8 under the bits of 1024 is the half 1024 + n, at bits 4 .. 7 1024 + 16 n: a sum with -1032, or a
//   multiply-add with 1/16 and -72, gives the code, a product the value. (From subnormals n 2^-24 one multiply-add with
//   2^24 scale and -8 scale gives it, nine instructions for eight values in place of thirteen, but 2^24 scale must stay below
//   2^16, which leaves 2^-8 between the largest scale and the first that loses bits.)
#pragma once

#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "common.cuh"
#include "kv4_layout.cuh"
#include "tc_common.cuh"

namespace cb {
namespace {

constexpr int kUnitRecords = 4;  // records of a unit of the ring of codes
constexpr int kUnitKeys = kUnitRecords * kKv4Block;
constexpr int kTileUnits = 2;
constexpr int kTileTokens = kUnitKeys * kTileUnits;
constexpr uint32_t kNoRecord = 0xffffffffu;
constexpr int kLeastExponent = -120;  // of a tile's power of two (its factors stay inside fp32)

// Records in shared memory. They come by TMA, one copy for the records of a unit that lie in one page, as lines of 128 bytes
// whose 16-byte chunks are swizzled by the line (18 D / 128 lines a record, an even number at D = 128, so that eight lanes
// that read (record, half) 0 .. 7 meet four different groups of banks and not one). The scales come a second time, on their
// own, further ahead.
template <int D>
struct Kv4Raw {
  static constexpr int kLines = 18 * D / 128;                                // of a record
  static constexpr int kUnitBytes = (kUnitRecords * 18 * D + 1023) / 1024 * 1024;  // the swizzle goes by address
  static constexpr int kScaleRecord = 2 * D;  // bytes of a record's scales
  static constexpr int kScaleBytes = kTileUnits * kUnitRecords * kScaleRecord;
};
__device__ __forceinline__ uint32_t swizzled(uint32_t at) { return at ^ (at >> 3 & 0x70u); }

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 h2_of(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

template <int N>
__device__ __forceinline__ void lds(uint32_t (&w)[N], uint32_t at) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}
__device__ __forceinline__ void sts4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts1(uint32_t at, uint32_t a) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(a) : "memory");
}

// The four pairs of a word's nibbles (bits 4 i of its halves), times the scale: 13 instructions for 8 values.
__device__ __forceinline__ void widen_word(uint32_t w, __half2 scale, uint32_t (&x)[4]) {
  const __half2 low = __float2half2_rn(-1032.0f), by = __float2half2_rn(0.0625f), high = __float2half2_rn(-72.0f);
  const uint32_t v = w >> 8;
  x[0] = h2_bits(__hmul2(__hadd2(h2_of((w & 0x000f000fu) | 0x64006400u), low), scale));
  x[1] = h2_bits(__hmul2(__hfma2(h2_of((w & 0x00f000f0u) | 0x64006400u), by, high), scale));
  x[2] = h2_bits(__hmul2(__hadd2(h2_of((v & 0x000f000fu) | 0x64006400u), low), scale));
  x[3] = h2_bits(__hmul2(__hfma2(h2_of((v & 0x00f000f0u) | 0x64006400u), by, high), scale));
}

// The scales of a tile, in place, by one converged warp: bf16 [128 tokens][K NG, V NG] become, for every 8 tokens, fp16 scales
// of K [8 tokens][NG], then of V [NG][8 tokens]. Tokens from `valid` on, and those of records in `bad`, get 0. e_k and
// e_v: the tile's exponents; e_v is least_v at least, and kNoExponent where all values are 0. A V scale that is not finite
// gets 0, and nan_from[its group] the least of what it was and first + its token. Two passes of four turns, 32 tokens each, in
// few instructions: the roles of a kernel share its instruction cache.
//   mixed: not every row sees every token. Where one's largest scale then lies more than 2^20 below the tile's, it returns
// true, each token has exponents of its own, and `own` [128 tokens] holds them (global memory).
constexpr int kNoExponent = -1000;
constexpr int kCommonRange = 20;  // the other 9 of 29 powers of two are left to the groups of a token
// The exponent of a tile whose largest scale has the bits `top`: one in [2^x, 2^(x+1)) times 2^-e, e >= x - 12, lies below
// 2^13, eight times it (a bf16's 8 bits) below fp16's largest value.
__device__ __forceinline__ int exponent_of(uint32_t top) { return max((int)(top >> 7) - 127 - 12, kLeastExponent); }
template <int D>
__device__ __forceinline__ bool prepare_scales(uint32_t at, int valid, uint32_t bad, int lane, int first, int* nan_from,
                                               int least_v, bool mixed, float2* own, int& e_k, int& e_v) {
  constexpr int NG = Kv4<D>::kGroups;
  auto there = [&](int tok) -> bool { return tok < valid && !(bad >> (tok / kKv4Block) & 1); };
  uint32_t top_k = 0, top_v = 0;  // of both halves of the words
#pragma unroll 1
  for (int k = 0; k < kTileTokens / 32; ++k) {
    uint32_t w[NG];
    lds<NG>(w, at + (32 * k + lane) * (4 * NG));
    if (there(32 * k + lane))
#pragma unroll
      for (int i = 0; i < NG / 2; ++i) {
        top_k = __vmaxu2(top_k, w[i] & 0x7fff7fffu);
        top_v = __vmaxu2(top_v, w[NG / 2 + i] & 0x7fff7fffu);
      }
  }
  __syncwarp();
  top_k = __reduce_max_sync(0xffffffffu, max(top_k & 0xffffu, top_k >> 16));
  top_v = __reduce_max_sync(0xffffffffu, max(top_v & 0xffffu, top_v >> 16));
  const bool odd = max(top_k, top_v) >= 0x7f80u;  // rare: a scale that is no number
  if (odd) {
    top_k = top_v = 0;
#pragma unroll 1
    for (int k = 0; k < kTileTokens / 32; ++k) {
      const int tok = 32 * k + lane;
#pragma unroll 1
      for (int i = 0; i < 2 * NG; ++i) {
        uint32_t w;
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w) : "r"(at + tok * (4 * NG) + 2 * i));
        w &= 0x7fffu;
        if (!there(tok)) continue;
        if (w >= 0x7f80u) {
          if (i >= NG) atomicMin(nan_from + i - NG, first + tok);
        } else if (i < NG) {
          top_k = max(top_k, w);
        } else {
          top_v = max(top_v, w);
        }
      }
    }
    __syncwarp();
    top_k = __reduce_max_sync(0xffffffffu, top_k);
    top_v = __reduce_max_sync(0xffffffffu, top_v);
  }
  e_k = exponent_of(top_k);
  e_v = max(exponent_of(top_v), least_v);
  const float fk = power_of_2(-e_k), fv = power_of_2(-e_v);  // e_k, e_v: -120 .. 115
  bool wide = false;
  if (mixed) {  // (a tile or two of an item)
#pragma unroll 1
    for (int i = 0; i < 2 * kTileTokens / 32; ++i) {
      const int tok = i / 2 * 32 + lane;
      uint32_t w[NG / 2];
      lds<NG / 2>(w, at + tok * (4 * NG) + i % 2 * (2 * NG));
      const uint32_t x = __vmaxu2(w[0] & 0x7fff7fffu, w[NG / 2 - 1] & 0x7fff7fffu), top = max(x & 0xffffu, x >> 16);
      wide = wide || (there(tok) && top > 0 && top + (kCommonRange << 7) < (i % 2 == 0 ? top_k : top_v));
    }
    wide = __any_sync(0xffffffffu, wide);
  }
  if (wide) {  // rare: the tokens' scales to the size of the tile's largest
#pragma unroll 1
    for (int i = 0; i < 2 * kTileTokens / 32; ++i) {
      const int tok = i / 2 * 32 + lane, v = i % 2;
      const uint32_t scales = at + tok * (4 * NG) + v * (2 * NG);
      uint32_t top = 0, w;
#pragma unroll 1
      for (int g = 0; g < NG && there(tok); ++g) {
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w) : "r"(scales + 2 * g) : "memory");
        if ((w & 0x7fffu) < 0x7f80u) top = max(top, w & 0x7fffu);
      }
      const int e = exponent_of(top), by = (v == 0 ? e_k : e_v) - e;  // by: 0 .. 235
#pragma unroll 1
      for (int g = 0; g < NG && there(tok); ++g) {
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w) : "r"(scales + 2 * g) : "memory");
        const float x = __uint_as_float(w << 16) * power_of_2(by >> 1) * power_of_2(by - (by >> 1));
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(scales + 2 * g), "h"((uint16_t)(__float_as_uint(x) >> 16)) : "memory");
      }
      (v == 0 ? own[tok].x : own[tok].y) = (float)e;
    }
    __threadfence();
    __syncwarp();
  }
  if (top_v == 0) e_v = kNoExponent;
#pragma unroll 1
  for (int k = 0; k < kTileTokens / 32; ++k) {
    const int tok = 32 * k + lane;
    uint32_t w[NG];
    lds<NG>(w, at + tok * (4 * NG));
    __syncwarp();  // the eight tokens are read
    const bool is = there(tok);
    const uint32_t block = at + tok / 8 * (32 * NG);
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) {
      const uint32_t x = is ? w[i] : 0u;
      sts1(block + tok % 8 * (2 * NG) + 4 * i,
           h2_bits(__floats2half2_rn(__uint_as_float(x << 16) * fk, __uint_as_float(x & 0xffff0000u) * fk)));
      uint32_t y = is ? w[NG / 2 + i] : 0u;
      if (odd) {
        if ((y & 0x7f80u) == 0x7f80u) y &= 0xffff0000u;
        if ((y & 0x7f800000u) == 0x7f800000u) y &= 0xffffu;
      }
      const uint32_t h = h2_bits(__floats2half2_rn(__uint_as_float(y << 16) * fv, __uint_as_float(y & 0xffff0000u) * fv));
      const uint32_t to = block + 16 * NG + 2 * i * 16 + tok % 8 * 2;
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"((uint16_t)(h & 0xffffu)) : "memory");
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 16), "h"((uint16_t)(h >> 16)) : "memory");
    }
  }
  return wide;
}

// Keys of unit u: records first .. first + count - 1 of the unit at `raw` into the K-major tile at `tile` (rows of 64
// dims, 128 bytes, swizzled; boxes of 64 dims one behind the other), with the tile's prepared scales at `scales`. By one
// converged warp. Eight lanes that store together hold the four words of tokens x and x + 4: eight different chunks.
template <int D>
__device__ __forceinline__ void widen_keys(uint32_t tile, uint32_t raw, uint32_t scales, int u, int first, int count,
                                           int lane) {
  constexpr int NG = Kv4<D>::kGroups;
  const int c = lane & 3, in_half = (lane >> 3) + 4 * (lane >> 2 & 1);
#pragma unroll 1
  for (int k = 0; k < 2 * count; ++k) {  // by half records
    const int rec = first + k / 2, t = 8 * (k % 2) + in_half, key = u * kUnitKeys + rec * kKv4Block + t;
    uint32_t w[NG], s[NG / 2];
    lds<NG>(w, raw + swizzled(rec * (18 * D) + (t * 4 + c) * (4 * NG)));
    lds<NG / 2>(s, scales + key / 8 * (32 * NG) + key % 8 * (2 * NG));
    uint32_t to = tile + key * 128 + (uint32_t)((c ^ (key & 7)) * 16);
#pragma unroll 1
    for (int box = 0; box < NG / 2; ++box) {  // (in a loop, the words moving up: few instructions)
      uint32_t x[4];
      widen_word(w[0], __low2half2(h2_of(s[0])), x);
      sts4(to, x[0], x[1], x[2], x[3]);
      widen_word(w[1], __high2half2(h2_of(s[0])), x);
      sts4(to ^ 64, x[0], x[1], x[2], x[3]);
      if constexpr (NG == 4) w[0] = w[2], w[1] = w[3], s[0] = s[1];
      to += kTileTokens * 128;
    }
  }
}

// Values of unit u: dims 32 g + 4 r + .. of its 64 keys for r = r0 .. r0 + 3, g = g0 and g0 + 1 into the tile at `tile`,
// whose rows are dims (64 keys, 128 bytes, swizzled; unit u at u * D * 128). By one converged warp; eight lanes that store
// together hold the eight chunks (record, half) of one dim.
template <int D>
__device__ __forceinline__ void widen_values(uint32_t tile, uint32_t raw, uint32_t scales, int u, int r0, int g0, int lane) {
  constexpr int NG = Kv4<D>::kGroups;
  const int half = lane & 1, rec = lane >> 1 & 3, r = r0 + (lane >> 3), chunk = 2 * rec + half;
  const uint32_t at = rec * (18 * D) + Kv4<D>::kV + half * Kv4<D>::kPlane + r * (16 * NG) + g0 * 4;
  const uint32_t s_at = scales + (u * kUnitRecords * 2 + chunk) * (32 * NG) + 16 * NG;
  const uint32_t to = tile + u * (D * 128) + 4 * r * 128;
  uint32_t w[4][2];
#pragma unroll
  for (int c = 0; c < 4; ++c) lds<2>(w[c], raw + swizzled(at + c * (4 * NG)));
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    uint32_t s[4];
    lds<4>(s, s_at + (g0 + e) * 16);
    uint32_t x[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      widen_word(w[c][0], h2_of(s[c]), x[c]);
      w[c][0] = w[c][1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sts4(to + (32 * (g0 + e) + i) * 128 + (uint32_t)((chunk ^ ((4 * r + i) & 7)) * 16), x[0][i], x[1][i], x[2][i], x[3][i]);
  }
}

// Bulk copy into shared memory; both addresses and the size are multiples of 16.
__device__ __forceinline__ void copy_bulk(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// A bounded wait by a converged warp. *abort_flag holds the site of the first wait of the CTA that gave up (0: none), which the
// kernel records at its end; every other wait gives up then too. In few instructions: the roles of these kernels
// share 32 KB of instruction cache, and with the general wait of tc_common.cuh at each place one of them ran at a quarter
// of its speed.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int site, uint32_t limit_us) {
  bool ok = true;
  uint32_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
    if (n % 4 != 0) continue;  // (reading the clock takes hundreds of cycles)
    const uint32_t t = (uint32_t)(global_timer() >> 10) | 1u;  // in 1.024 us
    if (t0 == 0) t0 = t;
    if (t - t0 > limit_us) *abort_flag = site;
    if (*abort_flag != 0) {
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The tensor maps of a cache: records as lines of 128 bytes, swizzled, and their scales alone; `records` of them (which lie
// in one page) per copy. Coordinates [.., line or record in the page, kv head, page].
inline bool encode_cache_maps(CUtensorMap* codes, CUtensorMap* scales, const void* cache, int32_t n_pages, int32_t page_size,
                              int32_t hkv, int32_t head_dim, int32_t records) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t rec = 18 * (cuuint64_t)head_dim, per_page = page_size / kKv4Block, heads = hkv, pages = n_pages;
  const cuuint64_t dims[2][4] = {{64, per_page * rec / 128, heads, pages}, {(cuuint64_t)head_dim, per_page, heads, pages}};
  const cuuint64_t strides[2][3] = {{128, per_page * rec, heads * per_page * rec}, {rec, per_page * rec, heads * per_page * rec}};
  const cuuint32_t box[2][4] = {{64, (cuuint32_t)(records * rec / 128), 1, 1}, {(cuuint32_t)head_dim, (cuuint32_t)records, 1, 1}};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (enc(i == 0 ? codes : scales, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<uint8_t*>(static_cast<const uint8_t*>(cache) + (i == 0 ? 0 : 16 * head_dim)), dims[i], strides[i], box[i], es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, i == 0 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

// Low half of a K-major operand's shared-memory descriptor (see sdesc); the high half is the same for all.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4 & 0x3fffu) | 1u << 16; }
constexpr uint32_t kDescHi = 1024 >> 4 | 1u << 14 | 2u << 29;

// mma_ss and mma_ts with descriptors by their low halves: fewer instructions for the one lane that issues them.
__device__ __forceinline__ void mma_ss_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}

// Instruction descriptor, kind::f16: fp16 A and B, both K-major, fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

}  // namespace
}  // namespace cb
