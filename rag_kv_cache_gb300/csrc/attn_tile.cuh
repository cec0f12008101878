// The softmax of one row's 128 scores, shared by the kernels with one softmax thread per query row
// (attention_pp.cu, prompt_attention.cu). Internal linkage: each translation unit gets its own copy.
#pragma once

#include "attn_common.cuh"
#include "common.cuh"
#include "tmem_ops.cuh"

namespace cb {
namespace {

constexpr int kTileKeys = 128;  // keys per key tile

// One row's P for a key tile: P = 2^(s * scale - m_ref) for its 128 scores (m_ref = -inf only for
// a row with nothing visible yet, whose scores are then all -inf), packed to bf16 and written to
// TMEM as 32 columns per 64 keys from taddr_p; returns the row sum of P (fp32, +inf if an exponent
// overflowed).
__device__ __forceinline__ float softmax_p(const uint32_t (&sv)[kTileKeys], float m_ref, float scale_log2,
                                           uint32_t taddr_p) {
  const float neg_m = m_ref == -INFINITY ? 0.0f : -m_ref;
  const uint64_t sc2 = f2_pack(scale_log2, scale_log2), nm2 = f2_pack(neg_m, neg_m);
  uint64_t ps2[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) ps2[q] = f2_pack(0.0f, 0.0f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int c = 64 * h + 2 * e;
      float x0, x1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sc2, nm2), x0, x1);
      const float p0 = ex2(x0), p1 = ex2(x1);
      ps2[e & 3] = f2_add(ps2[e & 3], f2_pack(p0, p1));
      pk[e] = pack2(p0, p1);
    }
    tmem_st_x32(taddr_p + 32 * h, pk);
  }
  float sa, sb;
  f2_unpack(f2_add(f2_add(ps2[0], ps2[1]), f2_add(ps2[2], ps2[3])), sa, sb);
  return sa + sb;
}

}  // namespace
}  // namespace cb
