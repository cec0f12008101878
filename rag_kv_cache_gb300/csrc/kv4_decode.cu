// Decode attention over a paged cache held in 4 bits (kv4_layout.cuh), one new token per request:
//
//   out[s, h] = sum_{j < len_s} softmax_j(scale q[s, h] . k[s, j, g]) v[s, j, g],  g = h / G,
//
// with k and v = code * (scale of the row's group of 32 dims).
//
// Floor: a (key, kv head) is 18/16 D bytes. At 6.7 TB/s an SM receives 23 bytes per cycle, so it has
// about 6 cycles per (key, kv head) at D = 128. The codes are widened in registers, straight into the
// operand layout of mma.sync, which leaves shared memory out of it; the batch below takes 12 cycles. (tcgen05 reads
// at least one operand from shared memory: widened codes there are 512 bytes per key to write and read, 8 cycles at 128
// bytes per cycle. The kernel that does so, kv4_chunk.cu, takes 373 us for requests of one token where this one's form for
// few rows takes 172: not for that traffic, but for the 3,800 cycles of its roles' chain per 128 keys.)
//   K   word & 0x000f000f and word & 0x00f000f0 are pairs of fp16 of value nibble * 2^-24 and * 2^-20
//       (subnormals, exact): 5 instructions per 8 codes;
//   V   (word >> 4 i & 0x000f000f) | 0x43004300 is a pair of bf16 of value 128 + nibble = 136 + code
//       (exact): 7 per 8 codes. In bf16, since the weights times V's scales need its range.
// No subtraction or conversion is needed. The offsets leave through the accumulators:
//   scores   S^T = K Q^T (M = 16 keys, N = 8 heads, inner = dims), one accumulator per group of 32
//            dims, times the key's scale, added to one more product of the keys' scales with -8 * (sum
//            of q over the group), the latter as three bf16 terms; q is scaled into fp16's range;
//   output   O^T += V^T P^T (M = 16 dims, N = 8 heads, inner = 16 keys) with P_g = bf16(p * scale of
//            the key's group g), and before it one more product with -136 in place of V. Record by
//            record: taken off at the end of a run (one product per group with ones, summing P_g), the
//            offsets left their fp32 rounding, 2^-24 of 136 times all weights: 2 us less for
//            the batch below, but its output 0.0029 instead of 0.0023 off (relative, root mean square).
// P (keys x heads) becomes the second product's operand by an 8 x 8 transpose between lanes
// (movmatrix). Sums of products, softmax statistics and sums are fp32; rounding p * scale to bf16 (2^-8
// relative) is the one rounding before the output's.
//
// Work split: the records (16 keys of one request and kv head) of the whole batch, in the order
// request, kv head, position, are dealt to the warps of one wave of CTAs in equal contiguous runs, so
// a batch of any mix of lengths is balanced and a single long request fills the GPU. A run that ends
// inside a (request, kv head) leaves a partial result (max, sum, unnormalised O): the CTA merges those
// of its warps in shared memory, and a (request, kv head) that spans CTAs is merged by the last of
// them to finish, over partials in the plan's scratch (a ticket per CTA that begins one). The merge
// order is fixed by position, so results do not change from run to run. Small batches of short requests
// take a CTA per (request, kv head), which spares that last merge: 4 requests of up to
// 545 keys and 2 kv heads of 64 dims 6.7 against 11.2 us. Up to 32 requests are dealt out by each
// warp for itself, a request per lane, so that no barrier stands before its first copies (6.9 us with one).
//
// Feeding: each warp asks for its own records by bulk copies into a ring of its own, five ahead (eight
// with 8 warps), and waits for them alone; no warp waits for another one until the merge.
//
// Measured (8 kv heads of 128 dims): 64 requests of up to 8,449 keys, 64 query heads (308 MB, 46 us at
// the copy rate) 89.6 us, 0.51 of that rate (89.2 before the form for few rows); one request of 32,897 keys, 32 query heads
// (38 MB, 5.7 us) 22 us: the first records arrive after 3.3 us, a warp's ten take 9, the merges 5 (a CTA's own, the ticket, the parts).
// With 16 query heads per kv head (8 warps) and other sizes: 64 requests of 4,225 keys, 8 kv heads of 128 dims, 125 us
// against 82 with 8 query heads (0.37 and 0.56 of the copy rate), of 64 dims 90 against 59 (0.26 and 0.39);
// one request of 32,897 keys, 16 query heads on one kv head of 128 dims, 49 us, of 64 dims 30; one of 4,096,
// 8,192, 16,384 keys, 8 kv heads of 128 dims, 10, 14 and 17 us.
// Runs of equal length by CTA instead of by warp are slower, 92 us for the batch. What bounds the batch
// is latency: a record costs a warp about 360 instructions, 175 of them on the integer pipe, which takes one every
// other cycle, and three warps per scheduler are too few to fill any pipe (issue slots 50% in use while active, integer
// 49%, tensor 27%). Of the 6.0 cycles per instruction of a warp 1.0 is its issue, 1.7 are fixed latencies, 0.9 a
// busy pipe, 0.8 another warp's turn, 0.4 branches, 0.3 each barriers and memory, 0.6 shared memory, dispatch and
// instruction fetch. With 14 and 16 warps, of fewer
// registers, the batch takes 96 and 94 us. Records two to a copy (92 us then) or two at a time through the
// registers (88 against 89), Q in shared memory to make room for 16 warps (105), shifts as multiplications (96),
// and K in e4m3 with Q in two terms (102; 3 instructions per 8 codes, but such a product costs more than
// two in fp16) were slower or no gain.
//
// The same kernel (CHUNK) takes the requests of few rows, several tokens among them, of a chunk attention call (kv4_chunk.cu),
// whose weights have to keep 11 bits: V is widened as K is, into fp16, and P_g is held as fp16(p * scale 2^-e) with e from the
// largest of V's scales that the row has seen, which moves O's units as the references do. 64 requests of 8,192 keys of one
// token and 4 query heads on each of 8 kv heads: 172 us with a launch of the other kernel for no request, 373 on that one.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "attn_common.cuh"
#include "kv4_layout.cuh"
#include "kv4_scores.cuh"
#include "tc_common.cuh"

namespace cb {
namespace {

constexpr float kHigh = 256.0f;           // a weight above it moves the reference
constexpr float kLow = -3e38f;            // reference of a head that has seen nothing
constexpr int kMaxCtas = 160;             // of a launch (one wave: one per SM)
constexpr uint32_t kBias = 0x43004300u;   // two bf16 of 128: the last place is 1
constexpr uint32_t kMinus = 0xc308c308u;  // two bf16 of -136, what a widened nibble of V is above its code

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Adds one; the CTA's writes before it (behind a barrier) are seen by who reads the sum, whose reads come after.
__device__ __forceinline__ int take_ticket(int32_t* at) {
  int before;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(at) : "memory");
  return before;
}

// The wait for a record's copy; false if the limit ran out: the timeout is recorded and the warp's abort flag raised,
// so that its later waits return at once; the call's result is void.
__device__ __noinline__ bool wait_record(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* err,
                                         uint64_t limit_ns) {
  return !*abort_flag && mbar_spin_slow_body(bar, parity, abort_flag, err, 80, limit_ns);
}
// After it: the lane that asks for the records waits once more for those in flight, from stage `stage` of the ring on,
// for as long as the limit again for all of them together, and asks for no more (returns false): a barrier whose phase
// has not completed must not be armed again. So no copy is under way when the ring is used for something else or
// the CTA ends, unless it takes longer than both limits. (The flag that the lane tests before each request and the
// wait's result cost 1 us of 88.)
__device__ __noinline__ bool stop_requests(uint32_t bar0, int stage, uint32_t parity, int stages, int in_flight,
                                           uint64_t limit_ns) {
  const uint64_t t0 = global_timer();
  for (int k = 0; k < in_flight; ++k) {
    while (!mbar_try_wait_sleep(bar0 + 8 * stage, parity) && global_timer() - t0 <= limit_ns) {
    }
    if (++stage == stages) stage = 0, parity ^= 1;
  }
  return false;
}

// CHUNK: two fp16 of -8 codes, 2^-24 and 2^-20 each
constexpr uint32_t kMinusLow = 0x80088008u, kMinusHigh = 0x80808080u;

struct Masks {
  uint32_t nibbles, higher, bias, minus;
};

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
  Masks masks;
  float* part_o;     // [CTA][2][16 heads][D]
  float2* part_ml;   // [CTA][2][16 heads]
  int32_t* tickets;  // [CTA]
  int32_t* err;
};
// CHUNK: request s has rows cu[s] .. cu[s + 1] - 1 of q, out [n_rows, heads, D], which G counts as if they were heads. (A struct
// of its own, and branches that the decode does not compile at all: four more members cost it 7 registers, tests of constants
// another order of its instructions; 64 requests 90.1 us in place of 89.6, with 16 query heads per kv head 127.5 for 124.8.)
struct Kv4FewParams : Kv4DecodeParams {
  const int32_t* cu;
  float* lse;
  int32_t n_rows;
  int32_t lg;  // log2 of the query heads per kv head
};
template <bool CHUNK>
using ParamsOf = std::conditional_t<CHUNK, Kv4FewParams, Kv4DecodeParams>;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Pairs `from` and from + 1 of the four pairs of nibbles of a word, widened:
// (word >> 4 i & 0x000f000f) | 0x43004300.
__device__ __forceinline__ void widen(uint32_t word, int from, const Masks& k, uint32_t (&x)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) x[i] = (word >> (4 * (from + i)) & k.nibbles) | k.bias;
}

// Running state of a warp over one (request, kv head): heads 8 t + 2 c and + 1 per lane (c = lane % 4).
template <int D, int NT>
struct State {
  static constexpr int NG = Kv4<D>::kGroups;
  float o[NT][2 * NG][4];    // O^T, dims 32 g + 4 r + .. (r = lane / 4)
  float m[NT][2], l[NT][2];  // reference (log2 units, the same in all lanes of a head), this lane's share of the sum
  int top[NT][2];  // CHUNK: the largest exponent of V's scales that the row has seen so far (biased); o is in units of
                   // 2^(top - 133 - 24) for the dims of codes in low nibbles, of 2^(top - 133 - 20) for the others
};

template <int D, int NT>
__device__ __forceinline__ void reset(State<D, NT>& st) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < 2 * State<D, NT>::NG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[t][i][e] = 0.0f;
    st.m[t][0] = st.m[t][1] = kLow;
    st.top[t][0] = st.top[t][1] = 15;  // a weight (to 2^8) times 2^(133 - top) is a float
    st.l[t][0] = st.l[t][1] = 0.0f;
  }
}

// One record of up to 16 keys, the first `valid` of them in the request; row 8 t + 2 c + e sees those below sees[t][e]
// (CHUNK only).
template <int D, int NT, bool WHOLE, bool CHUNK>
__device__ __forceinline__ void step(State<D, NT>& st, const Query<D, NT>& qf, uint32_t rec, int valid,
                                     const int (&sees)[NT][2], const Masks& mk, int lane) {
  constexpr int NG = Kv4<D>::kGroups;
  const int r = lane / 4;
  uint32_t sc[2][NG];  // scales of tokens r and r + 8: [K NG, V NG] bf16
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_vec<NG>(sc[h], rec + Kv4<D>::kScales + (r + 8 * h) * (4 * NG));
    // slots behind the request's end may hold any scales: 0 keeps what they give finite
    if (!WHOLE && r + 8 * h >= valid)
#pragma unroll
      for (int g = 0; g < NG; ++g) sc[h][g] = 0;
  }
  auto vs = [&](int h, int g) {
    return g % 2 ? bf16_hi(sc[h][NG / 2 + g / 2]) : bf16_lo(sc[h][NG / 2 + g / 2]);
  };
  float s[NT][4];
  record_scores<D, NT>(s, qf, rec, sc, mk.nibbles, mk.higher, lane);
  uint32_t w[2][NG];
  // -inf behind the request's end
  if (!WHOLE) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r + 8 * (e / 2) >= valid || (CHUNK && r + 8 * (e / 2) >= sees[t][e % 2])) s[t][e] = -INFINITY;
  }
  // P = 2^(s scale - m) against the reference. The references are raised only where a weight passes 2^8
  // (or, at a request's first record, where there is none): the max costs 8 comparisons and 6
  // shuffles per record.
  float pr[NT][4];
  float most = 0.0f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int e = 0; e < 4; ++e) pr[t][e] = ex2(fmaf(s[t][e], qf.scale[t][e % 2], -st.m[t][e % 2]));
    most = fmaxf(max3(most, pr[t][0], pr[t][1]), fmaxf(pr[t][2], pr[t][3]));
  }
  bool larger = false;  // CHUNK: than the scales so far
  if constexpr (CHUNK) {
    uint32_t scale_top = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int g = NG / 2; g < NG; ++g) scale_top = __vmaxu2(scale_top, sc[h][g] & 0x7fff7fffu);
    scale_top = max(scale_top >> 16, scale_top & 0xffffu) >> 7;
#pragma unroll
    for (int t = 0; t < NT; ++t) larger = larger || (int)scale_top > min(st.top[t][0], st.top[t][1]);
  }
  const bool high = most > kHigh || larger;
  if (__any_sync(0xffffffffu, high)) {
    int token_top[2] = {0, 0};  // CHUNK: of tokens r and r + 8, of the scales that are finite
    if constexpr (CHUNK) {
#pragma unroll
      for (int i = 0; i < 2 * NG; ++i) {
        const int e = sc[i / NG][NG / 2 + i % NG / 2] >> (i % 2 ? 23 : 7) & 0xffu;
        if (e < 255) token_top[i / NG] = max(token_top[i / NG], e);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = fmaxf(s[t][e], s[t][e + 2]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)) * qf.scale[t][e];
        const bool move = top > st.m[t][e];
        alpha[e] = move ? ex2(st.m[t][e] - top) : 1.0f;  // 0 where the head had nothing
        if (move) st.m[t][e] = top;
        st.l[t][e] *= alpha[e];
        if constexpr (CHUNK) {  // the units follow the scales of the tokens that the row sees
          int seen = max(WHOLE || r < sees[t][e] ? token_top[0] : 0, WHOLE || r + 8 < sees[t][e] ? token_top[1] : 0);
          seen = max(seen, __shfl_xor_sync(0xffffffffu, seen, 4));
          seen = max(seen, __shfl_xor_sync(0xffffffffu, seen, 8));
          seen = max(max(seen, __shfl_xor_sync(0xffffffffu, seen, 16)), st.top[t][e]);
          alpha[e] *= power_of_2(max(st.top[t][e] - seen, -126));  // (what is below 2^-126 of the new ones rounds to nothing)
          st.top[t][e] = seen;
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[t][i][e] *= alpha[e % 2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // (CHUNK: scores of any size, whose references are products rounded as here)
        pr[t][e] = CHUNK ? ex2(__fadd_rn(__fmul_rn(s[t][e], qf.scale[t][e % 2]), -st.m[t][e % 2]))
                         : ex2(fmaf(s[t][e], qf.scale[t][e % 2], -st.m[t][e % 2]));
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    st.l[t][0] += pr[t][0] + pr[t][2];
    st.l[t][1] += pr[t][1] + pr[t][3];
  }
  // V words of both halves
#pragma unroll
  for (int h = 0; h < 2; ++h) load_vec<NG>(w[h], rec + Kv4<D>::kV + h * Kv4<D>::kPlane + lane * (4 * NG));
  if constexpr (CHUNK) {  // weights to 2^8, scales below 2: P to 2^15
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) pr[t][e] *= power_of_2(133 - st.top[t][e % 2]);
  }
  uint32_t pb[NT][NG][2];  // P times the scales of group g: keys 0-7, keys 8-15
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float s0 = vs(0, g), s1 = vs(1, g);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[4] = {pr[t][0] * s0, pr[t][1] * s0, pr[t][2] * s1, pr[t][3] * s1};
      if (CHUNK && !WHOLE)  // a key that another row sees may have any scale: 0 times it may be NaN
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = r + 8 * (e / 2) >= sees[t][e % 2] ? 0.0f : x[e];
      if constexpr (CHUNK) {
        const __half2 h0 = __floats2half2_rn(x[0], x[1]), h1 = __floats2half2_rn(x[2], x[3]);
        pb[t][g][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&h0));
        pb[t][g][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&h1));
      } else {
        pb[t][g][0] = transpose8x8(pack2(x[0], x[1]));
        pb[t][g][1] = transpose8x8(pack2(x[2], x[3]));
      }
    }
  }
  // the offset first, for all groups, so that the two products of an accumulator stand apart
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if constexpr (CHUNK)
          mma_f16(st.o[t][2 * g + half], kMinusLow, kMinusHigh, kMinusLow, kMinusHigh, pb[t][g][0], pb[t][g][1]);
        else
          mma_bf16(st.o[t][2 * g + half], mk.minus, mk.minus, mk.minus, mk.minus, pb[t][g][0], pb[t][g][1]);
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t x[2], y[2];  // tokens of half 0, half 1
      if constexpr (CHUNK) {
        const uint32_t u = w[0][g] >> (8 * half), v = w[1][g] >> (8 * half);
        x[0] = u & mk.nibbles, x[1] = u & mk.higher, y[0] = v & mk.nibbles, y[1] = v & mk.higher;
      } else {
        widen(w[0][g], 2 * half, mk, x);
        widen(w[1][g], 2 * half, mk, y);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (CHUNK)
          mma_f16(st.o[t][2 * g + half], x[0], x[1], y[0], y[1], pb[t][g][0], pb[t][g][1]);
        else
          mma_bf16(st.o[t][2 * g + half], x[0], x[1], y[0], y[1], pb[t][g][0], pb[t][g][1]);
      }
    }
}

// Warps of a CTA: two n-tiles of heads take twice the registers and half the warps.
template <int NT>
constexpr int kWarpsOf = NT == 1 ? 12 : 8;

// Records per warp up to which a CTA takes a (request, kv head) alone, where the batch has no more of them than the launch
// has CTAs. Alone against split, us, 1 to 16 requests of one length:
//   64 dims, 12 warps (2 kv heads): 960 keys (5 records per warp) 7.5 - 7.8 against 8.3 - 9.0, 1,152 (6) 8.1 - 8.4 against
//     8.3 - 9.0, 1,280 (7) 8.8 - 8.9 against 8.4 - 9.3;
//   128 dims, 12 warps (2 and 8 kv heads): 768 (4) 8.5 - 9.0 against 8.9 - 9.2, 960 (5) 9.5 - 10.0 against 9.0 - 10.5, 1,152 (6)
//     10.4 - 10.8 against 9.0 - 11.0;
//   16 query heads per kv head, 8 warps (1 and 2 kv heads): 880 keys (7) 9.7 - 13.4 against 9.7 - 17.2, 1,024 (8) 10.4 - 14.5
//     against 9.8 - 13.0.
// (A batch of 128 pairs is faster alone at all these lengths, by 3 - 4 us at some.)
template <int D, int NT>
constexpr int kAlone = NT == 2 ? 7 : D == 128 ? 5 : 6;

// A partial result's O [heads][D] in shared memory (its references and sums lie in s_ml).
template <int D, int NT>
constexpr int kSlotFloats = 8 * NT * D;

// Records on their way to one warp, or held for it: about 36 KB per SM keep HBM busy.
template <int NT>
constexpr int kStagesOf = NT == 1 ? 5 : 8;

// Bytes of a warp's shared memory: the partial result of its first (request, kv head), then its ring,
// which holds the partial result of the last one when the warp is through.
template <int D, int NT>
constexpr int kWarpBytes = kSlotFloats<D, NT> * 4 + kStagesOf<NT> * Kv4<D>::kRecord;

// A warp's place in the batch's records.
struct Place {
  int s, h, i, n;  // request, kv head, record of it, its records
};

struct SlotInfo {
  int32_t p0, p1;  // the records of its (request, kv head) in the batch's order
  int32_t pair;    // request * hkv + kv head, -1: empty
};

// Four values of dims 4 d4 .. of head h, times `inv`, as bf16 into the output.
__device__ __forceinline__ void write_out4(uint8_t* out, int64_t row, int D, int d4, const float4 a, float inv) {
  *reinterpret_cast<uint2*>(out + (row * D + d4 * 4) * 2) = make_uint2(pack2(a.x * inv, a.y * inv), pack2(a.z * inv, a.w * inv));
}

// 1 / l, and 0 for a sum over nothing.
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

// PROBE: the wait-timeout probe (test support only): every warp arms the barrier of its second record but never
// copies it, and the waits give up after kProbeTimeoutNs, so each warp with two records or more takes its failure
// path. Compiled out of the kernel itself.
// CHUNK: requests of a few rows each (chunk attention): up to 8 NT of tokens times heads take the places of the heads, and
// requests that have more are left to kv4_chunk.cu. Keys are hidden by row, out and lse go to the rows' places.
template <int D, int NT, bool PROBE = false, bool CHUNK = false>
__global__ void __launch_bounds__(kWarpsOf<NT> * 32, 1) kv4_decode_kernel(const ParamsOf<CHUNK> p) {
  constexpr uint64_t kLimit = PROBE ? kProbeTimeoutNs : kTimeoutNs;
  constexpr int NG = Kv4<D>::kGroups;
  constexpr int kWarps = kWarpsOf<NT>, kThreads = kWarps * 32;
  constexpr int kSlot = kSlotFloats<D, NT>;
  constexpr int kStages = kStagesOf<NT>;
  constexpr int kRecord = Kv4<D>::kRecord;
  static_assert(kStages * kRecord >= kSlot * 4 && kSlot % 4 == 0, "a partial result fits a warp's ring");
  extern __shared__ __align__(16) uint8_t smem[];  // [kWarps] first partial result, ring
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ int s_abort[kWarps];
  constexpr int kSlots = 2 * kWarps, kHeads = 8 * NT;
  __shared__ SlotInfo info[kSlots];
  __shared__ float2 s_ml[kSlots][kHeads];     // (reference, sum) of the partial results
  __shared__ float s_weight[kSlots][kHeads];  // their weights in their groups
  __shared__ float2 s_group[kSlots][kHeads];  // (max, sum) of the group that begins at a slot
  __shared__ int32_t s_start[kWarps];         // first record of the request that a warp's run begins in
  __shared__ int32_t s_seq[kWarps];           // that request
  __shared__ int32_t w_sum[kWarps];
  __shared__ int s_last[2];

  pdl_launch_dependents();
  // What a warp uses until the merge is its own.
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (lane < kStages) mbar_init(smem_u32(&full[warp][lane]), 1);
  if (lane < 2) info[2 * warp + lane].pair = -1;
  if (lane == 0) s_abort[warp] = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  pdl_wait();
  auto slot_at = [&](int slot) -> float* {
    return reinterpret_cast<float*>(smem + (slot / 2) * kWarpBytes<D, NT> + (slot % 2) * kSlot * 4);
  };
  const int r = lane / 4, c = lane % 4;
  const int32_t room = p.width * p.page_size;  // fits: the host checks
  auto row0_of = [&](int s) -> int {
    if constexpr (CHUNK) return min(max(__ldg(p.cu + s), 0), p.n_rows);
    return 0;
  };
  // CHUNK: the rows (tokens) of a request, 0 where this kernel does not take it
  auto tokens_of = [&](int s) -> int {
    if constexpr (CHUNK) {
      const int m = max(row0_of(s + 1) - row0_of(s), 0);
      return m <= 8 * NT >> p.lg ? m : 0;
    }
    return 1;
  };
  auto len_of = [&](int s) -> int32_t {
    if constexpr (CHUNK)
      if (tokens_of(s) == 0) return 0;
    return min(max(__ldg(p.lens + s), 0), room);
  };
  // Row n (of its group of heads) of request s and kv head h in out and lse, -1: there is none.
  auto out_row = [&](int s, int h, int n) -> int64_t {
    if constexpr (CHUNK) {
      if (n >= tokens_of(s) << p.lg) return -1;
      return (((int64_t)row0_of(s) + (n >> p.lg)) * p.hkv + h << p.lg) + (n & ((1 << p.lg) - 1));
    }
    return ((int64_t)s * p.hkv + h) * p.G + n;
  };
  auto write_lse = [&](int64_t row, float m, float l) {
    if constexpr (CHUNK)
      if (p.lse != nullptr) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  };
  auto records_of = [&](int s) -> int { return (int)(((int64_t)len_of(s) + kKv4Block - 1) / kKv4Block); };

  // The batch's records, and where each warp's run of them begins (32 bits hold them: the host checks).
  const int warps = gridDim.x * kWarps;
  int quota, cta_records, cta0, cta1;  // records per warp, per CTA, this CTA's first and last
  int run_seq = 0, run_start = 0;      // the request that this warp's run begins in, that request's first record
  auto alone = [&](int longest) -> bool { return p.n_seqs * p.hkv <= (int)gridDim.x && longest <= kAlone<D, NT> * kWarps; };
  // A small batch of short requests: a CTA for each (request, kv head), so that none is merged over CTAs.
  auto split_alone = [&]() {
    const int s = blockIdx.x / p.hkv, h = blockIdx.x - s * p.hkv;
    const int n = s < p.n_seqs ? records_of(s) : 0;
    quota = (n + kWarps - 1) / kWarps;
    cta_records = n;
    cta0 = h * n;  // counted from the request's first record
    cta1 = cta0 + n;
    run_seq = s;
  };
  auto split = [&](int all) {
    quota = (int)(((uint32_t)all + warps - 1) / (uint32_t)warps);
    cta_records = kWarps * quota;
    cta0 = (int)min((int64_t)blockIdx.x * cta_records, (int64_t)all);
    cta1 = (int)min((int64_t)cta0 + cta_records, (int64_t)all);
  };
  auto scan_up = [&](int x) -> int {  // inclusive, over the warp
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    return x;
  };
  if (p.n_seqs <= 32) {  // each warp for itself, a request per lane
    const int n = lane < p.n_seqs ? records_of(lane) : 0;
    if (alone(__reduce_max_sync(0xffffffffu, n))) {
      split_alone();
    } else {
      const int end = scan_up(n * p.hkv), begin = end - n * p.hkv;
      split(__shfl_sync(0xffffffffu, end, 31));
      const int a = cta0 + warp * quota;
      const uint32_t here = __ballot_sync(0xffffffffu, a >= begin && a < end);
      run_seq = here ? __ffs(here) - 1 : 0;
      run_start = __shfl_sync(0xffffffffu, begin, run_seq);
    }
  } else {
    const int run_s = (p.n_seqs + kThreads - 1) / kThreads;
    const int q0 = min(tid * run_s, p.n_seqs), q1 = min(q0 + run_s, p.n_seqs);
    int mine = 0, longest = 0;
    for (int s = q0; s < q1; ++s) {
      const int n = records_of(s);
      mine += n * p.hkv;
      longest = max(longest, n);
    }
    const int up = scan_up(mine);
    if (lane == 31) w_sum[warp] = up;
    if (__syncthreads_and(alone(longest))) {
      split_alone();
    } else {
      const int sums = scan_up(lane < kWarps ? w_sum[lane] : 0);
      const int earlier = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
      const int before = (warp > 0 ? earlier : 0) + up - mine;
      split(__shfl_sync(0xffffffffu, sums, 31));
      if (before < cta1 && before + mine > cta0)
        for (int w = 0; w < kWarps; ++w) {
          const int a = cta0 + w * quota;
          if (a < before || a >= before + mine) continue;
          int at = before, s = q0;
          for (int n; a >= at + (n = records_of(s) * p.hkv); ++s) at += n;
          s_seq[w] = s;
          s_start[w] = at;
        }
      __syncthreads();
      run_seq = s_seq[warp];
      run_start = s_start[warp];
    }
  }
  // Requests without keys get zeros; lengths outside [0, room] are recorded.
  auto check_requests = [&]() {
    for (int s = blockIdx.x * kWarps + warp; s < p.n_seqs; s += warps) {
      if constexpr (CHUNK) {  // (what is recorded, kv4_chunk.cu records)
        const int rows = tokens_of(s) * p.hkv << p.lg;
        if (rows == 0 || len_of(s) > 0) continue;
        const int64_t at = (int64_t)row0_of(s) * p.hkv << p.lg;
        for (int i = lane; i < rows * (D / 8); i += 32) reinterpret_cast<uint4*>(p.out)[at * (D / 8) + i] = make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr)
          for (int i = lane; i < rows; i += 32) p.lse[at + i] = -INFINITY;
        continue;
      }
      const int32_t n = __ldg(p.lens + s);
      if ((n < 0 || n > room) && lane == 0) record_error(p.err, kErrIndex, s);
      if (n <= 0 || room == 0)
        for (int i = lane; i < p.hkv * p.G * D / 8; i += 32)
          reinterpret_cast<uint4*>(p.out)[(int64_t)s * p.hkv * p.G * D / 8 + i] = make_uint4(0, 0, 0, 0);
    }
  };
  if (cta0 >= cta1) {
    check_requests();
    return;
  }

  const int blocks = p.page_size / kKv4Block;  // records per page and kv head
  const int a0 = cta0 + warp * quota, a_end = min(a0 + quota, cta1);
  if (a0 < a_end) {
    int rest = a_end - a0;  // records still to take
    volatile int* abort_flag = &s_abort[warp];
    const uint32_t ring = smem_u32(smem) + warp * kWarpBytes<D, NT> + kSlot * 4;
    Place at;
    at.s = run_seq;
    at.n = records_of(at.s);
    at.h = (a0 - run_start) / at.n;
    at.i = a0 - run_start - at.h * at.n;
    auto next = [&](Place& x) {
      if (++x.i < x.n) return;
      x.i = 0;
      if (++x.h < p.hkv) return;
      x.h = 0;
      do {
        ++x.s;
        x.n = x.s < p.n_seqs ? records_of(x.s) : 1;
      } while (x.n == 0);
    };
    // The warp's own producer: records in the order of its run, kStages ahead. `run` records from src on
    // are neighbours in a page; behind them the next page's id comes from lane (page index - w0) of a
    // window of 32 entries of the table's row. All lanes keep the producer's state, the leader (lane 0, until a
    // wait of its own gives up) acts.
    bool leader = lane == 0;
    Place to = at;       // first record behind the neighbours
    int left = rest;     // records still to request
    int run = 0, w0 = 0, ws = -1;
    int32_t win = -1;
    bool page_ok = false;
    const uint8_t* src = nullptr;
    uint32_t bad = 0;  // stages whose record's page is none
    const uint32_t bar0 = smem_u32(&full[warp][0]);
    uint32_t fill_bar = bar0, fill_dst = ring, fill_bit = 1;
    auto next_page = [&]() {
      const int pi = to.i / blocks, in_page = to.i - pi * blocks;
      if (to.s != ws || pi < w0 || pi >= w0 + 32) {
        ws = to.s;
        w0 = pi;
        win = (int64_t)(pi + lane) * blocks < to.n ? p.table[(int64_t)ws * p.width + pi + lane] : -1;
      }
      const int32_t page = __shfl_sync(0xffffffffu, win, pi - w0);
      page_ok = page >= 0 && page < p.n_pages;
      src = p.cache + (((int64_t)(page_ok ? page : 0) * p.hkv + to.h) * blocks + in_page) * kRecord;
      if (!page_ok && lane == 0) record_error(p.err, kErrIndex, to.s);
      run = min(blocks - in_page, to.n - to.i);
      to.i += run - 1;
      next(to);
    };
    auto request = [&]() {
      if (left == 0) return;
      if (run == 0) next_page();
      if (page_ok) {
        bad &= ~fill_bit;
        if (leader) {
          mbar_expect_tx(fill_bar, kRecord);
          if (!(PROBE && left == a_end - a0 - 1))
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(fill_dst),
                "l"(src), "r"(kRecord), "r"(fill_bar)
                : "memory");
        }
      } else {
        bad |= fill_bit;
        if (leader) mbar_arrive(fill_bar);  // the phase passes without a copy
      }
      src += kRecord;
      --run;
      --left;
      const bool wrap = fill_bit == 1u << (kStages - 1);
      fill_bar = wrap ? bar0 : fill_bar + 8;
      fill_dst = wrap ? ring : fill_dst + kRecord;
      fill_bit = wrap ? 1 : fill_bit << 1;
    };
    for (int k = 0; k < kStages; ++k) request();
    check_requests();  // while the first records come
    int stage = 0, parity = 0;
    State<D, NT> st;
    Query<D, NT> qf;
    bool first = true;
    while (rest > 0) {
      const int s = at.s, h = at.h;
      const int count = min(at.n - at.i, rest);
      int m = 1, sees[NT][2] = {};  // CHUNK: rows; keys that each row sees, from the record on
      if constexpr (CHUNK) {
        m = tokens_of(s);
        load_query<D, NT>(qf, [&](int n) { return p.q + out_row(s, h, n) * (D * 2); }, m << p.lg, p.scale_log2, lane);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) sees[t][e] = len_of(s) - m + ((8 * t + 2 * c + e) >> p.lg) + 1 - at.i * kKv4Block;
      } else {
        const uint8_t* q = p.q + ((int64_t)s * p.hkv + h) * p.G * D * 2;
        load_query<D, NT>(qf, [&](int head) { return q + head * (D * 2); }, p.G, p.scale_log2, lane);
      }
      reset(st);
      int keys = len_of(s) - at.i * kKv4Block;  // from the record on
      for (int i = 0; i < count; ++i, keys -= kKv4Block) {
        // (after a wait that gave up, the rest of the run goes over whatever the stages hold)
        if (!mbar_test(bar0 + 8 * stage, parity) &&
            !wait_record(bar0 + 8 * stage, parity, abort_flag, p.err, kLimit) && leader)
          leader = stop_requests(bar0, stage, parity, kStages, rest - i - left, kLimit);
        __syncwarp();
        const uint32_t rec = ring + stage * kRecord;
        if (keys >= kKv4Block + (CHUNK ? m - 1 : 0) && !(bad >> stage & 1))
          step<D, NT, true, CHUNK>(st, qf, rec, kKv4Block, sees, p.masks, lane);
        else  // without its page, a stage holds an earlier record: weight 0
          step<D, NT, false, CHUNK>(st, qf, rec, bad >> stage & 1 ? 0 : min(keys, kKv4Block), sees, p.masks, lane);
        if constexpr (CHUNK) {
#pragma unroll
          for (int t = 0; t < NT; ++t) sees[t][0] -= kKv4Block, sees[t][1] -= kKv4Block;
        }
        __syncwarp();
        request();  // into the stage just read
        if (++stage == kStages) stage = 0, parity ^= 1;
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
      const bool whole = count == at.n;
      const int slot = 2 * warp + (first ? 0 : 1);
      float* so = slot_at(slot);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int head = 8 * t + 2 * c + e;
          if (head >= p.G) continue;
          const float inv = inverse(st.l[t][e]);
          const int64_t to = CHUNK && !whole ? 0 : out_row(s, h, head);
          if (CHUNK && whole && to >= 0 && r == 0) write_lse(to, st.m[t][e], st.l[t][e]);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float4 x = make_float4(st.o[t][2 * g][e], st.o[t][2 * g][e + 2], st.o[t][2 * g + 1][e],
                                   st.o[t][2 * g + 1][e + 2]);
            if constexpr (CHUNK) {
              const float unit = power_of_2(st.top[t][e] - 133);
              x = make_float4(x.x * 16777216.0f * unit, x.y * 1048576.0f * unit, x.z * 16777216.0f * unit,
                              x.w * 1048576.0f * unit);
            }
            if (CHUNK && to < 0) continue;
            if (whole)
              write_out4(p.out, to, D, 8 * g + r, x, inv);
            else
              *reinterpret_cast<float4*>(so + head * D + 32 * g + 4 * r) = x;
          }
          if (!whole && r == 0) s_ml[slot][head] = make_float2(st.m[t][e], st.l[t][e]);
        }
      if (!whole && lane == 0) {
        info[slot].pair = s * p.hkv + h;
        info[slot].p0 = a_end - rest - at.i;
        info[slot].p1 = info[slot].p0 + at.n;
      }
      rest -= count;
      at.i += count - 1;
      next(at);
      first = false;
    }
  } else {
    check_requests();
  }
  __syncthreads();

  // Merge the partial results of each (request, kv head) of this CTA, then those of a (request, kv head)
  // that spans CTAs, by the last of them. Slots of one (request, kv head) are neighbours (a group, with
  // empty slots among them); lane k of every warp looks at slot k; groups begin at the set bits of `groups`.
  const int n4 = p.G * D / 4;
  const int my_pair = lane < kSlots ? info[lane].pair : -1;
  const uint32_t held = __ballot_sync(0xffffffffu, my_pair >= 0);
  const int prev = 31 - __clz(held & ((1u << lane) - 1));  // -1: none
  const int prev_pair = __shfl_sync(0xffffffffu, my_pair, prev < 0 ? 0 : prev);
  const uint32_t groups = __ballot_sync(0xffffffffu, my_pair >= 0 && (prev < 0 || prev_pair != my_pair));
  auto group_end = [&](int k) -> int {  // one past the group that begins at slot k
    const uint32_t later = groups & ~((2u << k) - 1);
    return later ? __ffs(later) - 1 : kSlots;
  };
  // Weights: a warp per head, sums and maxima over the lanes of a group by segmented scans.
  {
    const uint32_t upto = groups & ((2u << lane) - 1);
    const int g0 = upto ? 31 - __clz(upto) : 0;
    const int end = min(upto ? group_end(g0) : lane + 1, 32) - 1;
    for (int head = warp; head < p.G; head += kWarps) {
      const float2 ml = my_pair >= 0 ? s_ml[lane][head] : make_float2(kLow, 0.0f);
      float m = ml.x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, m, d);
        if (lane - d >= g0) m = fmaxf(m, x);
      }
      m = __shfl_sync(0xffffffffu, m, end);
      const float wk = my_pair >= 0 ? ex2(ml.x - m) : 0.0f;
      float l = wk * ml.y;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, l, d);
        if (lane - d >= g0) l += x;
      }
      l = __shfl_sync(0xffffffffu, l, end);
      if (my_pair >= 0) {
        s_weight[lane][head] = wk;
        if (lane == g0) s_group[lane][head] = make_float2(m, l);
      }
    }
  }
  __syncthreads();
  uint32_t to_do = groups;
  for (int at = tid; to_do != 0;) {  // all groups' elements in one range
    if (at >= n4) {
      at -= n4;
      to_do &= to_do - 1;
      continue;
    }
    const int g0 = __ffs(to_do) - 1, head = at * 4 / D;
    const int g1 = group_end(g0);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t some = held & (0xffffffffu >> (32 - g1)) & ~((1u << g0) - 1); some != 0;) {
      // Up to four slots at a time. A slot that holds something is added whatever its weight: 0 times a NaN is
      // NaN here as within a warp's run and over CTAs, so a value that is not finite shows however the batch was split.
      const int here = __popc(some);
      float wk[4];
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = u < here ? __ffs(some) - 1 : g0;
        wk[u] = s_weight[k][head];
        some &= some - 1;
        v[u] = *reinterpret_cast<const float4*>(slot_at(k) + at * 4);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u >= here) continue;
        acc.x = fmaf(wk[u], v[u].x, acc.x);
        acc.y = fmaf(wk[u], v[u].y, acc.y);
        acc.z = fmaf(wk[u], v[u].z, acc.z);
        acc.w = fmaf(wk[u], v[u].w, acc.w);
      }
    }
    const SlotInfo& x = info[g0];
    const float2 ml = s_group[g0][head];
    if (x.p0 >= cta0 && x.p1 <= cta1) {
      if constexpr (CHUNK) {
        const int64_t to = out_row(x.pair / p.hkv, x.pair % p.hkv, head);
        if (to >= 0) write_out4(p.out, to, D, at % (D / 4), acc, inverse(ml.y));
        if (to >= 0 && at % (D / 4) == 0) write_lse(to, ml.x, ml.y);
      } else {
        write_out4(p.out, (int64_t)x.pair * p.G + head, D, at % (D / 4), acc, inverse(ml.y));
      }
    } else {
      const int part = blockIdx.x * 2 + (x.p0 < cta0 ? 0 : 1);
      *reinterpret_cast<float4*>(p.part_o + part * kKv4MaxGroup * D + at * 4) = acc;
      if (at % (D / 4) == 0) p.part_ml[part * kKv4MaxGroup + head] = ml;
    }
    at += kThreads;
  }
  // At most the first and the last group reach past this CTA.
  const int edge[2] = {groups ? __ffs(groups) - 1 : -1, groups ? 31 - __clz(groups) : -1};
  auto reaches = [&](int e) -> bool {
    if (edge[e] < 0 || (e == 1 && edge[1] == edge[0])) return false;
    const SlotInfo& x = info[edge[e]];
    return x.p0 < cta0 || x.p1 > cta1;
  };
  if (!reaches(0) && !reaches(1)) return;
  __syncthreads();  // the CTA's parts are written
  if (tid < 2) {
    s_last[tid] = 0;
    if (reaches(tid)) {
      const SlotInfo& x = info[edge[tid]];
      const int c0 = x.p0 / cta_records, c1 = (x.p1 - 1) / cta_records;
      if (take_ticket(&p.tickets[c0]) == c1 - c0) {
        s_last[tid] = 1;
        p.tickets[c0] = 0;  // ready for the next call
      }
    }
  }
  __syncthreads();
  if (s_last[0] + s_last[1] == 0) return;
  // Both, where this CTA is the last of both, side by side (one after the other they took 3 us longer).
  float* scratch = reinterpret_cast<float*>(smem);  // the partial results in it have been read
  constexpr int kSums = kMaxCtas * kKv4MaxGroup, kTops = kSums + kKv4MaxGroup;
  constexpr int kWeights = kTops + kKv4MaxGroup;  // of one of the two
  static_assert(kWarps * kWarpBytes<D, NT> >= (2 * kWeights + 2 * 4 * kThreads) * 4, "scratch of the merge over CTAs");
  int c0[2], parts[2], pair[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    c0[e] = parts[e] = pair[e] = 0;
    if (!s_last[e]) continue;
    const SlotInfo x = info[edge[e]];
    c0[e] = x.p0 / cta_records;
    parts[e] = (x.p1 - 1) / cta_records - c0[e] + 1;
    pair[e] = x.pair;
  }
  auto part_of = [&](int e, int k) -> int { return (2 * (c0[e] + k) + (k == 0 ? 1 : 0)) * kKv4MaxGroup; };
  // weights of the parts, a warp per head: scratch [part][head], then the heads' sums
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float* weights = scratch + e * kWeights;
    // the warps from the last one down take the second's heads
    for (int head = e == 0 ? warp : kWarps - 1 - warp; head < p.G && parts[e] > 0; head += kWarps) {
      // parts lane, lane + 32, ..; most launches have no more than 32
      auto ml_of = [&](int k) -> float2 {
        return k < parts[e] ? __ldcg(&p.part_ml[part_of(e, k) + head]) : make_float2(kLow, 0.0f);
      };
      const float2 ml = ml_of(lane);
      float m = ml.x;
#pragma unroll 1
      for (int k = lane + 32; k < parts[e]; k += 32) m = fmaxf(m, ml_of(k).x);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      float wk = ex2(ml.x - m), l = wk * ml.y;
      if (lane < parts[e]) weights[lane * kKv4MaxGroup + head] = wk;
#pragma unroll 1
      for (int k = lane + 32; k < parts[e]; k += 32) {
        const float2 more = ml_of(k);
        wk = ex2(more.x - m);
        l = fmaf(wk, more.y, l);
        weights[k * kKv4MaxGroup + head] = wk;
      }
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      if (lane == 0) {
        weights[kSums + head] = l;
        if (CHUNK) weights[kTops + head] = m;
      }
    }
  }
  __syncthreads();
  auto write_joined = [&](int e, int pr, int head, int i, const float4 a) {
    const float l = scratch[e * kWeights + kSums + head];
    const int64_t to = CHUNK ? out_row(pr / p.hkv, pr % p.hkv, head) : (int64_t)pr * p.G + head;
    if (!CHUNK || to >= 0) write_out4(p.out, to, D, i % (D / 4), a, inverse(l));
    if (CHUNK && to >= 0 && i % (D / 4) == 0) write_lse(to, scratch[e * kWeights + kTops + head], l);
  };
  // the threads in teams of n4 (a power of two), each taking every (kThreads / n4)-th part
  const int teams = kThreads >= n4 ? kThreads / n4 : 1;
  if (tid < teams * n4 || teams == 1)
    for (int at = tid & (n4 - 1), team = teams > 1 ? tid / n4 : 0; at < n4; at += kThreads) {
      const int head = at * 4 / D;
      float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      for (int k = team; k < max(parts[0], parts[1]); k += 4 * teams) {
        float4 v[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (k + u * teams < parts[e])
              v[e][u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + part_of(e, k + u * teams) * D + at * 4));
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (k + u * teams >= parts[e]) continue;
            const float wk = scratch[e * kWeights + (k + u * teams) * kKv4MaxGroup + head];
            acc[e].x = fmaf(wk, v[e][u].x, acc[e].x);
            acc[e].y = fmaf(wk, v[e][u].y, acc[e].y);
            acc[e].z = fmaf(wk, v[e][u].z, acc[e].z);
            acc[e].w = fmaf(wk, v[e][u].w, acc[e].w);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (parts[e] == 0) continue;
        if (teams > 1)
          *reinterpret_cast<float4*>(scratch + 2 * kWeights + 4 * (e * kThreads + team * n4 + at)) = acc[e];
        else
          write_joined(e, pair[e], head, at, acc[e]);
      }
    }
  if (teams == 1) return;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (parts[e] == 0 || tid >= n4) continue;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int team = 0; team < teams; ++team) {
      const float4 v = *reinterpret_cast<const float4*>(scratch + 2 * kWeights + 4 * (e * kThreads + team * n4 + tid));
      acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
    }
    write_joined(e, pair[e], tid * 4 / D, tid, acc);
  }
}

template <int D, int NT, bool PROBE = false, bool CHUNK = false>
cudaError_t launch_t(const ParamsOf<CHUNK>& p, int32_t sms, cudaStream_t s) {
  constexpr int kWarps = kWarpsOf<NT>;
  const int64_t most = (int64_t)p.n_seqs * p.hkv * p.width * (p.page_size / kKv4Block);  // records at most
  const int64_t pairs = (int64_t)p.n_seqs * p.hkv;
  if (sms > kMaxCtas) sms = kMaxCtas;
  int64_t grid = (most + kWarps - 1) / kWarps;
  if (pairs > grid) grid = pairs;
  if (grid > sms) grid = sms;
  if (grid < 1) grid = 1;
  const size_t smem = (size_t)kWarps * kWarpBytes<D, NT>;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = set_smem_limit_once(kv4_decode_kernel<D, NT, PROBE, CHUNK>, (int)smem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_decode_kernel<D, NT, PROBE, CHUNK>, dim3((unsigned)grid), dim3(kWarps * 32), smem, s, p);
}

Kv4DecodeParams params_of(const void* q, const void* cache, int32_t n_pages, int32_t page_size, const int32_t* table,
                          int32_t width, const int32_t* lens, int32_t n_seqs, int32_t hq, int32_t hkv, float scale,
                          void* out, const Kv4Scratch& ws, int32_t* err) {
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
  p.masks = Masks{kNibbles, kNibbles << 4, kBias, kMinus};
  p.part_o = ws.part_o;
  p.part_ml = ws.part_ml;
  p.tickets = ws.tickets;
  p.err = err;
  return p;
}

}  // namespace

cudaError_t launch_kv4_decode(const void* q, const void* cache, int32_t n_pages, int32_t page_size,
                              const int32_t* table, int32_t width, const int32_t* lens, int32_t n_seqs, int32_t hq,
                              int32_t hkv, int32_t head_dim, float scale, void* out, const Kv4Scratch& ws,
                              int32_t* err, cudaStream_t s) {
  const Kv4DecodeParams p =
      params_of(q, cache, n_pages, page_size, table, width, lens, n_seqs, hq, hkv, scale, out, ws, err);
  const bool wide = p.G > 8;
  if (head_dim == 128) return wide ? launch_t<128, 2>(p, ws.sms, s) : launch_t<128, 1>(p, ws.sms, s);
  if (head_dim == 64) return wide ? launch_t<64, 2>(p, ws.sms, s) : launch_t<64, 1>(p, ws.sms, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_decode_timeout_probe(const void* q, const void* cache, int32_t n_pages, int32_t page_size,
                                            const int32_t* table, int32_t width, const int32_t* lens, int32_t n_seqs,
                                            int32_t hq, int32_t hkv, float scale, void* out, const Kv4Scratch& ws,
                                            int32_t* err, cudaStream_t s) {
  const Kv4DecodeParams p =
      params_of(q, cache, n_pages, page_size, table, width, lens, n_seqs, hq, hkv, scale, out, ws, err);
  return launch_t<128, 1, true>(p, ws.sms, s);
}

cudaError_t launch_kv4_chunk_few(const Kv4Batch& b, int32_t head_dim, void* out, float* lse, const Kv4Scratch& ws,
                                 cudaStream_t s) {
  Kv4FewParams p;
  static_cast<Kv4DecodeParams&>(p) = params_of(b.q, b.cache, b.n_pages, b.page_size, b.table, b.width, b.kv_lens, b.n_seqs,
                                               b.hq, b.hkv, b.scale, out, ws, b.err);
  p.cu = b.cu;
  p.lse = lse;
  p.n_rows = b.n_rows;
  p.lg = 31 - __builtin_clz(p.G);
  p.G = kv4_chunk_few_rows(b);
  const bool wide = p.G > 8;
  if (head_dim == 128) return wide ? launch_t<128, 2, false, true>(p, ws.sms, s) : launch_t<128, 1, false, true>(p, ws.sms, s);
  if (head_dim == 64) return wide ? launch_t<64, 2, false, true>(p, ws.sms, s) : launch_t<64, 1, false, true>(p, ws.sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace cb
