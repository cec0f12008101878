// Decode attention over a paged cache held in 4 bits (kv4_layout.cuh), one new token per request:
//
//   out[s, h] = sum_{j < len_s} softmax_j(scale q[s, h] . k[s, j, g]) v[s, j, g],  g = h / G,
//
// with k and v = code * (scale of the row's group of 32 dims).
//
// Bound by HBM: a (key, kv head) is 18/16 D bytes. At 6.7 TB/s an SM receives 23 bytes per cycle, so
// it has about 6 cycles per (key, kv head) at D = 128. Widening the codes to bf16 in shared memory for
// tcgen05 would write and read 512 bytes per key there, 8 cycles at 128 bytes per cycle, more than the
// bound; so the codes are widened in registers, straight into the operand layout of mma.sync, which
// costs 7 instructions per 8 codes:
//   (word >> 4 i & 0x000f000f) | 0x43004300 = two bf16 of value 128 + nibble = 136 + code (exact),
// so that no subtraction or conversion is needed. The offset 136 leaves through the accumulators:
//   scores   S^T = K Q^T (M = 16 keys, N = 8 heads, inner = dims), one accumulator per group of 32
//            dims that starts at -136 * sum of q over the group, then times the key's scale;
//   output   O^T += V^T P^T (M = 16 dims, N = 8 heads, inner = 16 keys) with P_g = bf16(p * scale of
//            the key's group g), and one more product per group with ones in place of V, which sums
//            the same rounded P_g: O - 136 * that sum is the result, so the offset adds no rounding.
// P (keys x heads) becomes the second product's operand by an 8 x 8 transpose between lanes
// (movmatrix). Products are bf16 x bf16 in fp32; softmax statistics and sums are fp32; rounding
// p * scale to bf16 (2^-9 relative) is the one rounding before the output's.
//
// Work split: the records (16 keys of one request and kv head) of the whole batch, in the order
// request, kv head, position, are dealt to the warps of one wave of CTAs in equal contiguous runs, so
// a batch of any mix of lengths is balanced and a single long request fills the GPU. A run that ends
// inside a (request, kv head) leaves a partial result (max, sum, unnormalised O): the CTA merges those
// of its warps in shared memory, and a (request, kv head) that spans CTAs is merged by the last of
// them to finish, over partials in the plan's scratch (a ticket per CTA that begins one). The merge
// order is fixed by position, so results do not change from run to run.
#include "common.cuh"
#include "kernels.h"
#include "attn_common.cuh"
#include "kv4_layout.cuh"

namespace cb {
namespace {

constexpr float kRescale = 8.0f;          // log2 units: a max that grows by less leaves the reference alone
constexpr float kOffset = 136.0f;         // value of a widened nibble of code 0
constexpr uint32_t kNibbles = 0x000f000fu;
constexpr uint32_t kBias = 0x43004300u;   // two bf16 of 128: the last place is 1
constexpr uint32_t kOnes = 0x3f803f80u;   // two bf16 of 1

struct Kv4DecodeParams {
  const uint8_t* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* lens;
  uint8_t* out;
  int32_t n_seqs;
  int32_t n_pages;
  int32_t page_size;
  int32_t width;  // pages per row of the table
  int32_t hkv;
  int32_t G;      // query heads per kv head
  float scale_log2;
  float* part_o;     // [CTA][2][16 heads][D]
  float2* part_ml;   // [CTA][2][16 heads]
  int32_t* tickets;  // [CTA]
  int32_t* err;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t widen(uint32_t word, int i) { return (word >> (4 * i) & kNibbles) | kBias; }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// One lane's share of a record: K words of tokens r and r + 8, V words of both halves, and the
// scales of tokens r and r + 8 ([K NG, V NG] bf16 each).
template <int NG>
struct Words {
  uint32_t k[2][NG], v[2][NG], sc[2][NG];
};

template <int NG>
__device__ __forceinline__ void load_vec(uint32_t (&w)[NG], const uint8_t* p) {
  if constexpr (NG == 4) {
    const uint4 x = ld_stream(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x, w[1] = x.y;
  }
}

template <int D>
__device__ __forceinline__ void load_record(Words<Kv4<D>::kGroups>& w, const uint8_t* rec, int lane) {
  constexpr int NG = Kv4<D>::kGroups;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_vec<NG>(w.k[h], rec + h * Kv4<D>::kPlane + lane * (4 * NG));
    load_vec<NG>(w.v[h], rec + Kv4<D>::kV + h * Kv4<D>::kPlane + lane * (4 * NG));
    load_vec<NG>(w.sc[h], rec + Kv4<D>::kScales + (lane / 4 + 8 * h) * (4 * NG));
  }
}

// Running state of a warp over one (request, kv head): heads 8 t + 2 c and + 1 per lane (c = lane % 4).
template <int D, int NT>
struct State {
  static constexpr int NG = Kv4<D>::kGroups;
  float o[NT][2 * NG][4];   // O^T + 136 * sum, dims 32 g + 4 r + .. (r = lane / 4)
  float ones[NT][NG][4];    // the sums of the rounded P_g (every row the same)
  float m[NT][2], l[NT][2];  // reference (log2 units, the same in all lanes of a head), this lane's share of the sum
};

template <int D, int NT>
__device__ __forceinline__ void reset(State<D, NT>& st) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < 2 * State<D, NT>::NG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[t][i][e] = 0.0f;
#pragma unroll
    for (int g = 0; g < State<D, NT>::NG; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.ones[t][g][e] = 0.0f;
    st.m[t][0] = st.m[t][1] = -INFINITY;
    st.l[t][0] = st.l[t][1] = 0.0f;
  }
}

// Query operand of one (request, kv head): pairs of dims 32 g + 8 c + .. of head 8 t + r, and
// -136 * (sum of the group's dims) of heads 8 t + 2 c and + 1.
template <int D, int NT>
struct Query {
  static constexpr int NG = Kv4<D>::kGroups;
  uint32_t b[NT][NG][4];
  float c0[NT][NG][2];
};

template <int D, int NT>
__device__ __forceinline__ void load_query(Query<D, NT>& qf, const uint8_t* q, int G, int lane) {
  constexpr int NG = Kv4<D>::kGroups;
  const int r = lane / 4, c = lane % 4;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (8 * t + r < G) x = __ldg(reinterpret_cast<const uint4*>(q + ((8 * t + r) * D + 32 * g + 8 * c) * 2));
      qf.b[t][g][0] = x.x, qf.b[t][g][1] = x.y, qf.b[t][g][2] = x.z, qf.b[t][g][3] = x.w;
      float f[8];
      unpack8(x, f);
      float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);  // head 8 t + r
      qf.c0[t][g][0] = -kOffset * __shfl_sync(0xffffffffu, sum, 8 * c);
      qf.c0[t][g][1] = -kOffset * __shfl_sync(0xffffffffu, sum, 8 * c + 4);
    }
}

// One record of up to 16 keys, the first `valid` of them in the request.
template <int D, int NT>
__device__ __forceinline__ void step(State<D, NT>& st, const Query<D, NT>& qf, Words<Kv4<D>::kGroups>& w, int valid,
                                     float scale_log2, int lane) {
  constexpr int NG = Kv4<D>::kGroups;
  const int r = lane / 4;
  if (valid < kKv4Block) {  // scales of slots behind the request's end may be anything: 0 keeps them finite
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (r + 8 * h >= valid)
#pragma unroll
        for (int g = 0; g < NG; ++g) w.sc[h][g] = 0;
  }
  // K scales of group g: element g of [K NG, V NG] bf16
  auto ks = [&](int h, int g) { return g % 2 ? bf16_hi(w.sc[h][g / 2]) : bf16_lo(w.sc[h][g / 2]); };
  auto vs = [&](int h, int g) {
    return g % 2 ? bf16_hi(w.sc[h][NG / 2 + g / 2]) : bf16_lo(w.sc[h][NG / 2 + g / 2]);
  };
  float s[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    uint32_t a[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[2 * i] = widen(w.k[0][g], i);
      a[2 * i + 1] = widen(w.k[1][g], i);
    }
    const float s0 = ks(0, g), s1 = ks(1, g);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float acc[4] = {qf.c0[t][g][0], qf.c0[t][g][1], qf.c0[t][g][0], qf.c0[t][g][1]};
      mma_bf16(acc, a[0], a[1], a[2], a[3], qf.b[t][g][0], qf.b[t][g][1]);
      mma_bf16(acc, a[4], a[5], a[6], a[7], qf.b[t][g][2], qf.b[t][g][3]);
      s[t][0] = fmaf(s0, acc[0], s[t][0]);
      s[t][1] = fmaf(s0, acc[1], s[t][1]);
      s[t][2] = fmaf(s1, acc[2], s[t][2]);
      s[t][3] = fmaf(s1, acc[3], s[t][3]);
    }
  }
  // scores in log2 units; -inf behind the request's end
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[t][e] *= scale_log2;
      if (valid < kKv4Block && r + 8 * (e / 2) >= valid) s[t][e] = -INFINITY;
    }
  // the record's max per head, and a new reference where it passes the old one by more than 2^8
  float top[NT][2];
  bool up = false;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(s[t][e], s[t][e + 2]);
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
      top[t][e] = x;
      up |= x > st.m[t][e] + kRescale;
    }
  if (__any_sync(0xffffffffu, up)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool move = top[t][e] > st.m[t][e] + kRescale;
        alpha[e] = move ? ex2(st.m[t][e] - top[t][e]) : 1.0f;  // 0 where the head had nothing
        if (move) st.m[t][e] = top[t][e];
        st.l[t][e] *= alpha[e];
      }
#pragma unroll
      for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[t][i][e] *= alpha[e % 2];
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.ones[t][g][e] *= alpha[e % 2];
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ref = st.m[t][e % 2];
      s[t][e] = ex2(s[t][e] - (ref == -INFINITY ? 0.0f : ref));
    }
    st.l[t][0] += s[t][0] + s[t][2];
    st.l[t][1] += s[t][1] + s[t][3];
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const uint32_t v0 = w.v[0][g], v1 = w.v[1][g];
    const float s0 = vs(0, g), s1 = vs(1, g);
    const uint32_t a0 = widen(v0, 0), a1 = widen(v0, 1), a2 = widen(v1, 0), a3 = widen(v1, 1);
    const uint32_t a4 = widen(v0, 2), a5 = widen(v0, 3), a6 = widen(v1, 2), a7 = widen(v1, 3);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t b0 = transpose8x8(pack2(s[t][0] * s0, s[t][1] * s0));  // keys 0-7
      const uint32_t b1 = transpose8x8(pack2(s[t][2] * s1, s[t][3] * s1));  // keys 8-15
      mma_bf16(st.o[t][2 * g], a0, a1, a2, a3, b0, b1);
      mma_bf16(st.o[t][2 * g + 1], a4, a5, a6, a7, b0, b1);
      mma_bf16(st.ones[t][g], kOnes, kOnes, kOnes, kOnes, b0, b1);
    }
  }
}

// Warps of a CTA: two n-tiles of heads take twice the registers and half the warps.
template <int NT>
constexpr int kWarpsOf = NT == 1 ? 16 : 8;

// A partial result in shared memory: O [heads][D] and (reference, sum) [heads].
template <int D, int NT>
constexpr int kSlotFloats = 8 * NT * (D + 2);

struct SlotInfo {
  int64_t p0, p1;  // the records of its (request, kv head) in the batch's order
  int32_t pair;    // request * hkv + kv head, -1: empty
};

// Four values of dims 4 d4 .. of head h, times `inv`, as bf16 into the output.
__device__ __forceinline__ void write_out4(uint8_t* out, int64_t row, int D, int d4, const float4 a, float inv) {
  *reinterpret_cast<uint2*>(out + (row * D + d4 * 4) * 2) = make_uint2(pack2(a.x * inv, a.y * inv), pack2(a.z * inv, a.w * inv));
}

// 1 / l, and 0 for a sum over nothing.
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

template <int D, int NT>
__global__ void __launch_bounds__(kWarpsOf<NT> * 32, 1) kv4_decode_kernel(const Kv4DecodeParams p) {
  constexpr int NG = Kv4<D>::kGroups;
  constexpr int kWarps = kWarpsOf<NT>, kThreads = kWarps * 32;
  constexpr int kSlot = kSlotFloats<D, NT>;
  extern __shared__ float slots[];  // [2 kWarps][kSlot]
  __shared__ SlotInfo info[2 * kWarps];
  __shared__ int64_t s_start[kWarps];  // first record of the request that a warp's run begins in
  __shared__ int32_t s_seq[kWarps];    // that request
  __shared__ int64_t w_sum[kWarps];
  __shared__ int s_last;

  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int r = lane / 4, c = lane % 4;
  const int64_t room = (int64_t)p.width * p.page_size;
  auto len_of = [&](int s) -> int32_t {
    const int32_t n = p.lens[s];
    return n < 0 ? 0 : (n < room ? n : (int32_t)room);
  };
  auto records_of = [&](int s) -> int64_t { return ((int64_t)len_of(s) + kKv4Block - 1) / kKv4Block; };

  // The batch's records, and where each warp's run of them begins.
  const int run = (p.n_seqs + kThreads - 1) / kThreads;
  const int q0 = min(tid * run, p.n_seqs), q1 = min(q0 + run, p.n_seqs);
  int64_t mine = 0;
  for (int s = q0; s < q1; ++s) mine += records_of(s) * p.hkv;
  int64_t up = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, up, d);
    if (lane >= d) up += x;
  }
  if (lane == 31) w_sum[warp] = up;
  if (tid < 2 * kWarps) info[tid].pair = -1;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += w_sum[w];
    all += w_sum[w];
  }
  before += up - mine;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  const int64_t quota = (all + warps - 1) / warps;  // records per warp
  const int64_t cta0 = blockIdx.x * kWarps * quota;
  if (mine > 0) {
    for (int w = 0; w < kWarps; ++w) {
      const int64_t a = cta0 + w * quota;
      if (a < before || a >= before + mine) continue;
      int64_t at = before;
      int s = q0;
      while (a >= at + records_of(s) * p.hkv) at += records_of(s++) * p.hkv;
      s_seq[w] = s;
      s_start[w] = at;
    }
  }
  // Requests without keys get zeros; lengths outside [0, room] are recorded.
  for (int s = blockIdx.x; s < p.n_seqs; s += gridDim.x) {
    const int32_t n = p.lens[s];
    if ((n < 0 || n > room) && tid == 0) record_error(p.err, kErrIndex, s);
    if (n <= 0)
      for (int i = tid; i < p.hkv * p.G * D / 8; i += kThreads)
        reinterpret_cast<uint4*>(p.out)[(int64_t)s * p.hkv * p.G * D / 8 + i] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  if (cta0 >= all) return;

  const int blocks = p.page_size / kKv4Block;  // records per page and kv head
  const int64_t a0 = cta0 + warp * quota;
  int64_t a = a0;
  const int64_t a_end = min(a0 + quota, all);
  if (a < a_end) {
    int s = s_seq[warp];
    int64_t n = records_of(s);
    int h = (int)((a - s_start[warp]) / n);
    int64_t b = (a - s_start[warp]) - h * n;
    State<D, NT> st;
    Query<D, NT> qf;
    while (a < a_end) {
      const int64_t count = min(n - b, a_end - a);
      const int32_t len = len_of(s);
      load_query<D, NT>(qf, p.q + ((int64_t)s * p.hkv + h) * p.G * D * 2, p.G, lane);
      reset(st);
      for (int64_t i = b; i < b + count; ++i) {
        const int32_t page = p.table[(int64_t)s * p.width + i / blocks];
        int valid = (int)min((int64_t)len - i * kKv4Block, (int64_t)kKv4Block);
        Words<NG> w;
        if (page >= 0 && page < p.n_pages) {
          load_record<D>(w, p.cache + (((int64_t)page * p.hkv + h) * blocks + i % blocks) * Kv4<D>::kRecord, lane);
        } else {
          if (lane == 0) record_error(p.err, kErrIndex, s);
          valid = 0;
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int g = 0; g < NG; ++g) w.k[x][g] = w.v[x][g] = w.sc[x][g] = 0;
        }
        step<D, NT>(st, qf, w, valid, p.scale_log2, lane);
      }
      // sums over the lanes of a head
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = st.l[t][e];
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          st.l[t][e] = x;
        }
      const bool whole = b == 0 && count == n;
      const int slot = 2 * warp + (a == a0 ? 0 : 1);
      float* so = slots + slot * kSlot;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int head = 8 * t + 2 * c + e;
          if (head >= p.G) continue;
          const float inv = inverse(st.l[t][e]);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float off = kOffset * st.ones[t][g][e];
            const float4 x = make_float4(st.o[t][2 * g][e] - off, st.o[t][2 * g][e + 2] - off,
                                         st.o[t][2 * g + 1][e] - off, st.o[t][2 * g + 1][e + 2] - off);
            if (whole)
              write_out4(p.out, ((int64_t)s * p.hkv + h) * p.G + head, D, 8 * g + r, x, inv);
            else
              *reinterpret_cast<float4*>(so + head * D + 32 * g + 4 * r) = x;
          }
          if (!whole && r == 0) {
            so[8 * NT * D + 2 * head] = st.m[t][e];
            so[8 * NT * D + 2 * head + 1] = st.l[t][e];
          }
        }
      if (!whole && lane == 0) {
        info[slot].pair = s * p.hkv + h;
        info[slot].p0 = a - b;
        info[slot].p1 = a - b + n;
      }
      a += count;
      b = 0;
      if (++h == p.hkv && a < a_end) {
        h = 0;
        do {
          ++s;
          n = records_of(s);
        } while (n == 0);
      }
    }
  }
  __syncthreads();

  // Merge the partials of each (request, kv head) of this CTA; then those of a (request, kv head) that
  // spans CTAs, by the last of them.
  const int64_t cta_records = kWarps * quota;
  const int64_t cta1 = min(cta0 + cta_records, all);
  const int n4 = p.G * D / 4;
  for (int i = 0; i < 2 * kWarps;) {
    const int pair = info[i].pair;
    if (pair < 0) {
      ++i;
      continue;
    }
    int j = i + 1;  // slots i .. j - 1 hold it, some of them may be empty
    while (j < 2 * kWarps && (info[j].pair == pair || info[j].pair < 0)) ++j;
    const int64_t p0 = info[i].p0, p1 = info[i].p1;
    const bool inside = p0 >= cta0 && p1 <= cta1;
    const int part = blockIdx.x * 2 + (p0 < cta0 ? 0 : 1);
    for (int x = tid; x < n4; x += kThreads) {
      const int head = x * 4 / D;
      float m = -INFINITY;
      for (int k = i; k < j; ++k)
        if (info[k].pair >= 0) m = fmaxf(m, slots[k * kSlot + 8 * NT * D + 2 * head]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.0f;
      for (int k = i; k < j; ++k) {
        if (info[k].pair < 0) continue;
        const float* so = slots + k * kSlot;
        const float mk = so[8 * NT * D + 2 * head];
        const float wk = mk == -INFINITY ? 0.0f : ex2(mk - m);
        const float4 v = *reinterpret_cast<const float4*>(so + x * 4);
        l = fmaf(wk, so[8 * NT * D + 2 * head + 1], l);
        acc.x = fmaf(wk, v.x, acc.x);
        acc.y = fmaf(wk, v.y, acc.y);
        acc.z = fmaf(wk, v.z, acc.z);
        acc.w = fmaf(wk, v.w, acc.w);
      }
      if (inside) {
        write_out4(p.out, (int64_t)pair * p.G + head, D, x % (D / 4), acc, inverse(l));
      } else {
        *reinterpret_cast<float4*>(p.part_o + ((int64_t)part * 16 * D + x * 4)) = acc;
        if (x % (D / 4) == 0) p.part_ml[part * 16 + head] = make_float2(m, l);
      }
    }
    if (!inside) {
      const int c0 = (int)(p0 / cta_records), c1 = (int)((p1 - 1) / cta_records);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(&p.tickets[c0], 1) == c1 - c0;
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int x = tid; x < n4; x += kThreads) {
          const int head = x * 4 / D;
          float m = -INFINITY;
          for (int k = c0; k <= c1; ++k) m = fmaxf(m, __ldcg(&p.part_ml[(2 * k + (k == c0)) * 16 + head]).x);
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          float l = 0.0f;
          for (int k = c0; k <= c1; ++k) {
            const int64_t at = 2 * k + (k == c0);
            const float2 ml = __ldcg(&p.part_ml[at * 16 + head]);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * 16 * D + x * 4));
            const float wk = ml.x == -INFINITY ? 0.0f : ex2(ml.x - m);
            l = fmaf(wk, ml.y, l);
            acc.x = fmaf(wk, v.x, acc.x);
            acc.y = fmaf(wk, v.y, acc.y);
            acc.z = fmaf(wk, v.z, acc.z);
            acc.w = fmaf(wk, v.w, acc.w);
          }
          write_out4(p.out, (int64_t)pair * p.G + head, D, x % (D / 4), acc, inverse(l));
        }
        if (tid == 0) p.tickets[c0] = 0;  // ready for the next call
      }
      __syncthreads();
    }
    i = j;
  }
}

template <int D, int NT>
cudaError_t launch_t(const Kv4DecodeParams& p, int32_t sms, cudaStream_t s) {
  constexpr int kWarps = kWarpsOf<NT>;
  const int64_t most = (int64_t)p.n_seqs * p.hkv * p.width * (p.page_size / kKv4Block);  // records at most
  const int64_t ctas = (most + kWarps - 1) / kWarps;
  const int grid = (int)(ctas < sms ? (ctas > 0 ? ctas : 1) : sms);
  const size_t smem = sizeof(float) * 2 * kWarps * kSlotFloats<D, NT>;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = set_smem_limit_once(kv4_decode_kernel<D, NT>, (int)smem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_decode_kernel<D, NT>, dim3(grid), dim3(kWarps * 32), smem, s, p);
}

}  // namespace

cudaError_t launch_kv4_decode(const void* q, const void* cache, int32_t n_pages, int32_t page_size,
                              const int32_t* table, int32_t width, const int32_t* lens, int32_t n_seqs, int32_t hq,
                              int32_t hkv, int32_t head_dim, float scale, void* out, const Kv4Scratch& ws,
                              int32_t* err, cudaStream_t s) {
  Kv4DecodeParams p;
  p.q = static_cast<const uint8_t*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.table = table;
  p.lens = lens;
  p.out = static_cast<uint8_t*>(out);
  p.n_seqs = n_seqs;
  p.n_pages = n_pages;
  p.page_size = page_size;
  p.width = width;
  p.hkv = hkv;
  p.G = hq / hkv;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.part_o = ws.part_o;
  p.part_ml = ws.part_ml;
  p.tickets = ws.tickets;
  p.err = err;
  const bool wide = p.G > 8;
  if (head_dim == 128) return wide ? launch_t<128, 2>(p, ws.sms, s) : launch_t<128, 1>(p, ws.sms, s);
  if (head_dim == 64) return wide ? launch_t<64, 2>(p, ws.sms, s) : launch_t<64, 1>(p, ws.sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace cb
