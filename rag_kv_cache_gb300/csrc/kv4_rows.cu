// Rows in and out of the 4-bit cache (kv4_layout.cuh).
//
// Store: for each kv head and group of 32 dims of a K or V row x,
//   scale = bf16(max|x| / 7),  code = round-half-even(x / scale) in -7 .. 7,
// with the quotient in IEEE fp32: x and scale have 8 significant bits, so the fp32 quotient lies on a
// half exactly when the real one does, and the codes are those of exact arithmetic. A group that
// holds a NaN or an infinity gets a NaN scale and stands for NaN throughout; a group of zeros has
// scale 0 and codes 0. Load writes bf16(scale * code), the product exact in fp32.
//
// Both are bound by HBM: a (token, kv head) is 4 D bytes of bf16 K and V and 18/16 D bytes of cache.
// Eight dims per lane (one 16-byte access of the bf16 row), four lanes per group: the group's maximum
// is two shuffles.
#include "common.cuh"
#include "kernels.h"
#include "kv4_layout.cuh"

namespace cb {
namespace {

constexpr int kThreads = 256;

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

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_store_kernel(const uint8_t* k, const uint8_t* v, uint8_t* cache,
                                                             const Kv4RowParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const Lane<D> x = lane_of<D>(p);
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (x.slot >= 0) raw = ld_stream((x.kv ? v : k) + ((x.row * p.hkv + x.h) * D + x.l * 8) * 2);
  // the group's largest magnitude as bf16 bits (ordered like the magnitudes; 0x7f80 and up: not finite)
  uint32_t top = 0;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (x.slot < 0) return;
  const bool finite = top < 0x7f80u;
  const __nv_bfloat16 scale = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top << 16), 7.0f));
  const float step = __bfloat162float(scale);
  float f[8];
  unpack8(raw, f);
  uint32_t nib[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float c = finite && step > 0.0f ? rintf(__fdiv_rn(f[e], step)) : 0.0f;
    nib[e] = (uint32_t)((int)fminf(fmaxf(c, -7.0f), 7.0f) + 8);  // |c| may pass 7 for subnormal scales
  }
  constexpr int NG = Kv4<D>::kGroups;
  const int g = x.l / 4, c = x.l % 4, t = x.slot % kKv4Block;
  uint8_t* rec = cache + record_offset<D>(x.slot, x.h, p.hkv, p.page_size);
  if (x.kv == 0) {
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) word |= nib[2 * i] << (4 * i) | nib[2 * i + 1] << (16 + 4 * i);
    *reinterpret_cast<uint32_t*>(rec + t * (D / 2) + (c * NG + g) * 4) = word;
  } else {
    uint8_t* vb = rec + Kv4<D>::kV + (t / 8) * Kv4<D>::kPlane + (t % 8 / 2) * (4 * NG) + g * 4 + (t % 2) * 2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {  // dims 8 c + 4 q .. of the group: r = 2 c + q
      const uint32_t half = nib[4 * q] | nib[4 * q + 1] << 4 | nib[4 * q + 2] << 8 | nib[4 * q + 3] << 12;
      *reinterpret_cast<uint16_t*>(vb + (2 * c + q) * (16 * NG)) = (uint16_t)half;
    }
  }
  if (c == 0)
    *reinterpret_cast<uint16_t*>(rec + Kv4<D>::kScales + t * (4 * NG) + x.kv * (2 * NG) + g * 2) =
        finite ? __bfloat16_as_ushort(scale) : (uint16_t)0x7fc0u;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(uint8_t* k, uint8_t* v, const uint8_t* cache,
                                                            const Kv4RowParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const Lane<D> x = lane_of<D>(p);
  if (x.slot < 0) return;
  constexpr int NG = Kv4<D>::kGroups;
  const int g = x.l / 4, c = x.l % 4, t = x.slot % kKv4Block;
  const uint8_t* rec = cache + record_offset<D>(x.slot, x.h, p.hkv, p.page_size);
  const float step = __uint_as_float(
      (uint32_t)*reinterpret_cast<const uint16_t*>(rec + Kv4<D>::kScales + t * (4 * NG) + x.kv * (2 * NG) + g * 2) << 16);
  int nib[8];
  if (x.kv == 0) {
    const uint32_t word = *reinterpret_cast<const uint32_t*>(rec + t * (D / 2) + (c * NG + g) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      nib[2 * i] = word >> (4 * i) & 15;
      nib[2 * i + 1] = word >> (16 + 4 * i) & 15;
    }
  } else {
    const uint8_t* vb = rec + Kv4<D>::kV + (t / 8) * Kv4<D>::kPlane + (t % 8 / 2) * (4 * NG) + g * 4 + (t % 2) * 2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t half = *reinterpret_cast<const uint16_t*>(vb + (2 * c + q) * (16 * NG));
#pragma unroll
      for (int i = 0; i < 4; ++i) nib[4 * q + i] = half >> (4 * i) & 15;
    }
  }
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = step * (float)(nib[e] - 8);
  st_stream((x.kv ? v : k) + ((x.row * p.hkv + x.h) * D + x.l * 8) * 2, pack8(f));
}

template <int D>
cudaError_t launch_rows(bool store, const void* k, const void* v, const void* cache, const Kv4RowParams& p,
                        cudaStream_t s) {
  const int64_t lanes = (int64_t)p.n * p.hkv * 2 * (D / 8);
  const int64_t blocks = (lanes + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  uint8_t *kb = static_cast<uint8_t*>(const_cast<void*>(k)), *vb = static_cast<uint8_t*>(const_cast<void*>(v)),
          *cb = static_cast<uint8_t*>(const_cast<void*>(cache));
  if (store) return launch_pdl(kv4_store_kernel<D>, dim3((unsigned)blocks), dim3(kThreads), 0, s, kb, vb, cb, p);
  return launch_pdl(kv4_load_kernel<D>, dim3((unsigned)blocks), dim3(kThreads), 0, s, kb, vb, cb, p);
}

}  // namespace

cudaError_t launch_kv4_rows(bool store, void* k, void* v, const int32_t* slots, int32_t n, void* cache,
                            int32_t n_pages, int32_t page_size, int32_t hkv, int32_t head_dim, int32_t* err,
                            cudaStream_t s) {
  if (n <= 0) return cudaSuccess;
  const Kv4RowParams p{slots, n, hkv, page_size, (int64_t)n_pages * page_size, err};
  if (head_dim == 128) return launch_rows<128>(store, k, v, cache, p, s);
  if (head_dim == 64) return launch_rows<64>(store, k, v, cache, p, s);
  return cudaErrorInvalidValue;
}

}  // namespace cb
