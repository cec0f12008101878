// Attention of each request's new tokens over a paged cache held in 4 bits (kv4_layout.cuh):
//
//   out[t, h] = sum_{j <= p} softmax_j(scale q[t, h] . k_j[g]) v_j[g],  lse[t, h] = log sum_{j <= p} exp(..),  g = h / G,
//
// for row i of a request of m rows and len cached tokens at place p = len - m + i.
//
// Requests of few rows in a batch of many go to the decode kernel (kv4_decode.cu: a key costs it two thirds as much for one tile
// of 8 rows, as much for two), the others to this one.
//
// A work item is a request, a kv head and 256 rows (two tiles of 128: TQ = 128 / G tokens times the G heads that
// share the kv head), so that a key is read and widened once for all of them. S_i = Q_i K^T and O_i += P_i V are
// tcgen05.mma with S, P and O in tensor memory; per round of 128 keys the warps take these parts:
//   0 .. 7    softmax, a thread per row: the two tiles' warps alternate with the products;
//   8 .. 15   keys (four) and values (four) widened from the records' codes into operands in shared memory (kv4_tile.cuh, fp16,
//             exact but for a power of two per round);
//   16        records and, further ahead, their scales by TMA into rings; the list of items; 17 the scales' powers of two and
//             factors; 18 the products; 19 checks the requests.
// Where a request's rows fill no more than a tile on the average (ONE), items have one, whose even and odd rounds the two
// tiles' warps take in turn, each with a softmax of its own, and which are joined at the item's end. Such items against those of
// two tiles, us (8 kv heads of 128 dims, 4 query heads each): one request of 32,768 keys and 64, 128, 192, 256, 512 rows per kv
// head 66 and 72, 70 and 76, 83 and 83, 85 and 87, 122 and 111; 8 of 8,192 87 and 100, 90 and 103, 131 and 111, 133 and 116,
// 226 and 184; 40 of 8,192 270 and 346, 275 and 349, 501 and 377.
//
// Measured (8 kv heads of 128 dims): 2,048 tokens over 30,720, 32 query heads, 1.05 ms (1.06 TFLOP, 0.53 of the burst rate of a
// library product, which also has no softmax); 128 over 32,768 111 us; 64 requests of up to 8,453 keys, up to 5
// tokens of 64 query heads each, 347 us (378 MB, 56 us at the copy rate); 40 requests, 5 with chunks of up to 512
// tokens, 307 us; three short ones 14 us. What bounds it: a round of 128 keys takes 4,700 cycles with 256 rows, of which the
// tensor cores work 2,050, and 3,800 with few rows. No role is busy all the time (softmax 2,200 to 2,800 cycles of a tile's
// round, widening 1,650 to 2,100, scales 1,600 to 1,800, issuing products 1,300 to 2,300); each waits for another one's
// latency: two tiles of scores, K and V each is all that tensor memory and shared memory hold. Leaving out the softmax of
// warps without rows gains nothing (24 of 128 rows). Instructions count twice: all roles together run from 32 KB of
// instruction cache, so loops are rolled and waits are small (2.81 ms with everything unrolled, 1.08 ms rolled); codes
// through registers in place of a ring of records were slower (1.27 against 1.13 ms).
//
// Work split: the rounds of all items, in the order request, kv head, rows, keys, are dealt to one CTA per SM in
// equal contiguous runs, so any mix of lengths is balanced and a single request fills the GPU. An item that
// spans CTAs leaves partial results (normalised rows, reference, sum) in the plan's scratch, which a second kernel
// joins, in the order of the keys.
//
// Powers of two. Keys are held as k 2^-e_k of their round, a row of q as q 2^up (largest magnitude in [2^14,
// 2^15)): both leave through the factor a of the row's scores in that round. Values are held as v 2^-e_v; P is formed as
// 2^(score a + e_v - ref), in fp16 with at most 2^15, so P V = 2^(score a - ref) v; the sum of the weights takes
// 2^(e_b - e_v) per round, with e_b of the run's first round, and out = O 2^e_b / l. So each weight is rounded once to
// 11 bits, relative to what it contributes: to 2^-25 where the largest weight times its values' power is 2^6 or more.
// The sum itself must not depend on the values: an e_v lies 60 below the largest one of the run so far at most (a weight 2^-60
// of the largest is still summed; values below 2^-85 of the largest become 0), and where a reference has to move up because
// the values do, e_b moves with it.
//
// Nor may a row depend on keys that it does not see, which may be of any size. Those behind an item's last row count as zeros.
// Where the keys of a round that some of its rows do not see lie more than 2^20 apart, each has a power of its own for its key
// and its value, and the round's softmax goes by columns, three times over the scores (`wide`, rare: not made fast). So do
// rounds whose scores may pass 2^24.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "attn_common.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kv4_batch.cuh"
#include "kv4_tile.cuh"
#include "tmem_ops.cuh"

namespace cb {
namespace {

constexpr int kBM = 128;             // rows per tile
constexpr int kTiles = 2;            // tiles of an item
constexpr int kBN = kTileTokens;     // keys per round
constexpr int kQuarter = kBN / 4;    // keys that a softmax thread takes at a time
constexpr int kStages = 2;           // widened K and V tiles
constexpr int kItems = 8;            // ring of items; also of the rounds' constants
// Units of codes on their way or held: what shared memory leaves. And rounds of scales: kScaleStages.
__host__ __device__ constexpr int units_of(int d, bool one) { return d == 128 ? (one ? 6 : 3) : (one ? 8 : 6); }
constexpr int kThreads = 640;
constexpr int kSoftmaxThreads = 128;
constexpr int kWarpWiden = 8;        // 8 .. 11: keys; 12 .. 15: values
constexpr int kWidenWarps = 8;
constexpr int kWarpProducer = 16;
constexpr int kWarpScales = 17;
constexpr int kWarpMma = 18;
constexpr int kItemReaders = 18;     // warps that walk the items: scales, widening, MMA, softmax
constexpr uint32_t kTmemCols = 512;
constexpr int kSoftmaxRegs = 152, kWidenRegs = 56, kOtherRegs = 64;
constexpr float kHeadroom = 6.0f;         // log2 of P at the reference: what lies 2^-31 below it still counts
constexpr float kRescaleThreshold = 6.0f; // log2 units
constexpr float kHalfSumLimit = 32768.0f; // half a round whose P sums to more moves the reference (P fits fp16)
// log2 of a row's factor up to which its scores (at most 2^38 times it) stay below 2^24: there a reference rounded to 24 bits
// may still be taken off an exact product.
constexpr int kFactorExponent = -14;
constexpr int kValueRange = 60;           // powers of two that a round's e_v may lie below one before it

__host__ __device__ constexpr uint32_t col_s(int i) { return (uint32_t)(i * kBN); }
__host__ __device__ constexpr uint32_t col_o(int i, int d) { return 256u + (uint32_t)(i * d); }

// A run of rounds of one item, which one CTA takes.
struct Item {
  int row0;    // first row of its first token
  int tokens;  // its tokens (at most 2 TQ)
  int place0;  // place of its first token in the cache
  int g;       // kv head
  int j0;      // first round of keys
  int rounds;  // 0: no more items
  int two;     // its rows reach the second tile (not ONE)
  int part;    // where its partial result goes (of the CTA's two), -1: the run is the whole item
};
struct Round {
  float e_k;  // exponents of the round's keys and values (kNoExponent: all values are 0)
  float e_v;
  int bad;    // its records whose page is none
  int wide;   // its keys have exponents of their own
};
// What the join needs of an item that begins in a CTA and goes on in the next.
struct Part {
  int row0, tokens, g;
  int parts;  // 0: there is none
};

template <int kScaleStages>
struct Bars {
  uint64_t item[kItems], item_empty[kItems];
  uint64_t sc_full[kScaleStages], sc_ready[kScaleStages], sc_empty[kScaleStages];
  uint64_t k_full[kStages], v_full[kStages];
  uint64_t k_free[kStages], v_free[kStages];  // the products that read the stage are complete
  // Per tile, one phase for each of its rounds, none of which can pass before its warps are done with the one before.
  uint64_t s_full[kTiles], p_full[kTiles], o_done[kTiles];
  uint64_t q_full[kTiles];           // one for each item
  uint64_t stats_full, stats_read;  // ONE: what an item's odd rounds gave
  uint64_t drain;
};

struct ChunkParams {
  Kv4Batch b;
  uint8_t* out;
  float* lse;
  float* part_o;    // [CTA][2][256 rows][D]
  float2* part_ml;  // [CTA][2][256 rows]
  Part* parts;      // [CTA]
  float2* own;      // [CTA][kItems][128 keys]: exponents of a wide round's keys and values
  int lg;           // log2 of the query heads per kv head
  int few;          // requests of so many rows or fewer are another kernel's
  int run;          // records per copy: the four of a unit or two, where a page holds so many or a multiple, else 1
};

// Rounds of the item of rows 256 t .. of a request per kv head: those up to its last row's place. (Where there are more
// rows than tokens, as if the first sat at place 0.)
struct Shape {
  int base;  // place of the first row, at least 0
  int m;
  int per;   // log2 of the tokens per item
  __device__ __forceinline__ int tiles() const { return m > 0 ? ((m - 1) >> per) + 1 : 0; }
  __device__ __forceinline__ int rounds_of(int t) const { return (base + min((t + 1) << per, m) - 1) / kBN + 1; }  // at least 1
  // rounds of items 0 .. t - 1, all of which are full
  __device__ __forceinline__ int rounds_before(int t) const {
    if (per >= 7) {  // an item covers 1 or 2 rounds of keys itself
      const int step = 1 << (per - 7);
      return t * (base > 0 ? (base - 1) / kBN + 1 : 0) + step * (t * (t + 1) / 2);
    }
    const int lq = 7 - per;  // items per round of keys
    const int b = base > 0 ? ((base - 1) >> per) + 1 : 0, a = b >> lq, r = b & ((1 << lq) - 1);
    return t * a + ceils(r + t, lq) - ceils(r, lq);
  }
  __device__ __forceinline__ int all() const {
    const int t = tiles();
    return t == 0 ? 0 : rounds_before(t - 1) + rounds_of(t - 1);
  }
  // sum_{u = 1 .. n} ceil(u / 2^lq)
  static __device__ __forceinline__ int ceils(int n, int lq) {
    const int a = n >> lq, r = n & ((1 << lq) - 1);
    return (a * (a + 1) / 2 << lq) + r * (a + 1);
  }
};
template <bool ONE>
__device__ __forceinline__ Shape shape_of(const Kv4Request& r, int lg, int few) {
  return Shape{max(r.len - r.m, 0), r.m <= few ? 0 : r.m, (ONE ? 7 : 8) - lg};
}

// One row's P for a quarter of a round: 2^(s a + off) for 32 scores, packed to fp16; their sum is added to `sum`.
__device__ __forceinline__ void quarter_p(const uint32_t (&sv)[kQuarter], float a, float off, uint32_t (&pk)[kQuarter / 2],
                                          float& sum) {
  const uint64_t a2 = f2_pack(a, a), off2 = f2_pack(off, off);
  uint64_t ps2[2] = {f2_pack(sum, 0.0f), f2_pack(0.0f, 0.0f)};
#pragma unroll
  for (int e = 0; e < kQuarter / 2; ++e) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), a2, off2), x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    ps2[e & 1] = f2_add(ps2[e & 1], f2_pack(p0, p1));
    pk[e] = h2_bits(__floats2half2_rn(p0, p1));
  }
  float sa, sb;
  f2_unpack(f2_add(ps2[0], ps2[1]), sa, sb);
  sum = sa + sb;
}

// The largest of a row's 32 scores.
__device__ __forceinline__ float quarter_max(const uint32_t (&sv)[kQuarter]) {
  float tm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < kQuarter; c += 8)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      tm[u] = max3(tm[u], __uint_as_float(sv[c + 2 * u]), __uint_as_float(sv[c + 2 * u + 1]));
  return fmaxf(fmaxf(tm[0], tm[1]), fmaxf(tm[2], tm[3]));
}

// Scores of columns past `lim`, and of records in `bad` (bit 0: the first 16 columns), become -inf.
__device__ __forceinline__ void hide(uint32_t (&sv)[kQuarter], int lim, int bad) {
  __syncwarp();  // keeps its callers' branch around it one: else its selections run in every round
#pragma unroll
  for (int c = 0; c < kQuarter; ++c)
    if (c > lim || (bad >> (c / kKv4Block) & 1)) sv[c] = 0xff800000u;
}

// PROBE: the wait-timeout probe (test support only): the second unit of the second round of every CTA is never copied, and
// the waits give up after kProbeTimeoutNs. Compiled out of the kernel itself.
// ONE: items of one tile.
template <int D, bool ONE, bool PROBE = false>
__global__ void __launch_bounds__(kThreads, 1)
    kv4_chunk_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_scales,
                     const ChunkParams p) {
  constexpr uint64_t kLimit = PROBE ? kProbeTimeoutNs : kTimeoutNs;
  constexpr uint32_t kLimitUs = (uint32_t)(kLimit / 1024);
  using Raw = Kv4Raw<D>;
  constexpr int kUnits = units_of(D, ONE), kScaleStages = ONE ? 4 : 2;
  constexpr uint32_t kQBytes = kBM * D * 2;
  constexpr uint32_t kKVBytes = kBN * D * 2;
  constexpr uint32_t kBox = kBM * 128;       // 64 columns of a Q or K tile
  constexpr uint32_t kVBox = D * 128;        // 64 keys of a V tile

  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars<kScaleStages> bars;
  __shared__ uint64_t raw_full[kUnits], raw_empty[kUnits];
  __shared__ Item items[kItems];
  __shared__ int nan_from[kItems][4];  // first place of the item's run whose V is not finite, per group of dims
  __shared__ Round rounds_info[kItems];
  __shared__ float s_ref[kBM], s_sum[kBM], s_exp[kBM];  // the odd rounds' references, sums and the sums' exponents
  __shared__ int2 scale_info[kScaleStages];  // (valid tokens, bad records)
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_seq, s_before;
  __shared__ int64_t w_sum[kThreads / 32];

  pdl_launch_dependents();
  const Kv4Batch& b = p.b;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base;
  const uint32_t sK0 = sQ + (ONE ? 1 : 2) * kQBytes;
  const uint32_t sV0 = sK0 + kStages * kKVBytes;
  const uint32_t sRaw = sV0 + kStages * kKVBytes;
  const uint32_t sScale = sRaw + kUnits * Raw::kUnitBytes;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (warp == kWarpProducer && lane == 0) {
    for (int i = 0; i < kItems; ++i) {
      mbar_init(smem_u32(&bars.item[i]), 1);
      mbar_init(smem_u32(&bars.item_empty[i]), kItemReaders);
    }
    for (int i = 0; i < kScaleStages; ++i) {
      mbar_init(smem_u32(&bars.sc_full[i]), 1);
      mbar_init(smem_u32(&bars.sc_ready[i]), 1);
      mbar_init(smem_u32(&bars.sc_empty[i]), kWidenWarps);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_u32(&raw_full[i]), 1);
      mbar_init(smem_u32(&raw_empty[i]), kWidenWarps);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bars.k_full[i]), kWidenWarps / 2);
      mbar_init(smem_u32(&bars.v_full[i]), kWidenWarps / 2);
      mbar_init(smem_u32(&bars.k_free[i]), 1);
      mbar_init(smem_u32(&bars.v_free[i]), 1);
    }
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(smem_u32(&bars.s_full[t]), 1);
      mbar_init(smem_u32(&bars.o_done[t]), 1);
      mbar_init(smem_u32(&bars.p_full[t]), 4);
      mbar_init(smem_u32(&bars.q_full[t]), 4);
    }
    mbar_init(smem_u32(&bars.stats_full), 4);
    mbar_init(smem_u32(&bars.stats_read), 4);
    mbar_init(smem_u32(&bars.drain), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  // The batch's rounds, and where this CTA's run of them begins. 31 bits hold them (the host checks), unless offsets that
  // rise again behind a fall give the same rows to several requests: then nothing is computed past that limit.
  const int run_s = (b.n_seqs + kThreads - 1) / kThreads;
  const int q0 = min(tid * run_s, b.n_seqs), q1 = min(q0 + run_s, b.n_seqs);
  int64_t mine = 0;
  for (int s = q0; s < q1; ++s) mine += shape_of<ONE>(kv4_request(b, s), p.lg, p.few).all() * b.hkv;
  int64_t up = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, up, d);
    if (lane >= d) up += y;
  }
  if (lane == 31) w_sum[warp] = up;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t all_rounds = 0, before = up - mine;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += w_sum[w];
    all_rounds += w_sum[w];
  }
  const int total = all_rounds <= kKv4MostTiles ? (int)all_rounds : 0;
  const int quota = (total + gridDim.x - 1) / gridDim.x;
  const int run0 = (int)min((int64_t)blockIdx.x * quota, (int64_t)total);
  const int run1 = (int)min((int64_t)run0 + quota, (int64_t)total);
  if (before <= run0 && run0 < before + mine && total > 0) {
    int at = (int)before, s = q0;
    for (int n; run0 >= at + (n = shape_of<ONE>(kv4_request(b, s), p.lg, p.few).all() * b.hkv); ++s) at += n;
    s_seq = s;
    s_before = at;
  }
  __syncthreads();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  // Rounds of the it-th item of this CTA, which lies in items[it % kItems]; 0 at the end (or after a failure).
  auto item_at = [&](int it) -> int {
    const bool there = wait_warp(smem_u32(&bars.item[it % kItems]), (it / kItems) & 1, abort_flag, 100, kLimitUs);
    return there ? items[it % kItems].rounds : 0;
  };
  auto leave_item = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.item_empty[it % kItems]));
  };
  auto wait = [&](uint64_t& bar, uint32_t parity, int site) -> bool {
    return wait_warp(smem_u32(&bar), parity, abort_flag, site, kLimitUs);
  };

  if (warp >= kWarpProducer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kWarpProducer) {
      Part mine_part{0, 0, 0, 0};
      int seq = s_seq, at = run0 - s_before;  // the request, and the round in it
      const int per_page = b.page_size / kKv4Block;
      const bool acts = lane < 8 && (lane & (p.run - 1)) == 0;
      int it = 0, r = 0, left = run1 - run0, unit = 0, unit_phase = 0;
      int units = 0, scales = 0;  // units, rounds of scales asked for
      bool ok = true;
      // lane l: record l of the next four rounds' 32
      while (left > 0 && ok) {
        const Kv4Request rq = kv4_request(b, seq);
        const Shape sh = shape_of<ONE>(rq, p.lg, p.few);
        const int per_head = sh.all();
        if (at >= per_head * b.hkv) {  // (also a request without rows)
          at -= per_head * b.hkv;
          ++seq;
          continue;
        }
        const int g = at / per_head, rest = at - g * per_head;
        int t = 0;  // the item that holds round `rest` of the head: the last with rounds_before(t) <= rest
        for (int step = 1 << (31 - __clz(sh.tiles())); step > 0; step >>= 1)
          if (t + step < sh.tiles() && sh.rounds_before(t + step) <= rest) t += step;
        const int n = sh.rounds_of(t), j0 = rest - sh.rounds_before(t), count = min(n - j0, left);
        Item x;
        x.row0 = rq.row0 + (t << sh.per);
        x.tokens = min(rq.m - (t << sh.per), 1 << sh.per);
        x.place0 = rq.len - rq.m + (t << sh.per);
        x.g = g;
        x.j0 = j0;
        x.rounds = count;
        x.two = !ONE && x.tokens > kBM >> p.lg;
        x.part = j0 > 0 ? 0 : count < n ? 1 : -1;
        if (x.part == 1) mine_part = Part{x.row0, x.tokens, g, (n - count + quota - 1) / quota + 1};
        ok = it < kItems || wait(bars.item_empty[it % kItems], (it / kItems - 1) & 1, 120);
        if (!ok) break;
        if (lane == 0) items[it % kItems] = x;
        if (lane < 4) nan_from[it % kItems][lane] = 0x7fffffff;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.item[it % kItems]));
        int32_t page = -1, place = 0;  // and the record's place in it
#pragma unroll 1
        for (int j = 0; j < count; ++j, ++r) {
          const int rec0 = (j0 + j) * (kBN / kKv4Block), st = r % kScaleStages;
          if (j % 4 == 0) {  // pages of the next 32 records
            const int i = rec0 + lane;
            page = -1;
            if (i * kKv4Block < rq.len && i < rec0 + (count - j) * 8) {
              const int nth = i / per_page;
              place = i - nth * per_page;
              page = __ldg(b.table + (int64_t)seq * b.width + nth);
              if (page < 0 || page >= b.n_pages) {
                record_error(b.err, kErrIndex, seq);
                page = -2;
              }
            }
          }
          // lanes 0 .. 7: the round's records; those that begin a copy act
          const int from = (j % 4) * 8 + lane % 8;
          const int32_t my_page = __shfl_sync(0xffffffffu, page, from);
          const int in_page = __shfl_sync(0xffffffffu, place, from);
          const bool there = my_page >= 0 && acts;
          const uint32_t held = __ballot_sync(0xffffffffu, there);
          const uint32_t bad = __ballot_sync(0xffffffffu, my_page == -2 && lane < 8);
          ok = r < kScaleStages || wait(bars.sc_empty[st], (r / kScaleStages - 1) & 1, 101);
          if (!ok) break;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the scales were rewritten in place
          if (lane == 0) {
            scale_info[st] = make_int2(max(min(rq.len, x.place0 + x.tokens) - (j0 + j) * kBN, 0), (int)bad);
            if (held != 0)
              mbar_expect_tx(smem_u32(&bars.sc_full[st]), __popc(held) * p.run * Raw::kScaleRecord);
            else
              mbar_arrive(smem_u32(&bars.sc_full[st]));
          }
          ++scales;
          __syncwarp();
          if (there)
            tma_load_4d(sScale + st * Raw::kScaleBytes + lane * Raw::kScaleRecord, &tm_scales, smem_u32(&bars.sc_full[st]), 0,
                        in_page, g, my_page);
#pragma unroll 1
          for (int u = 0; u < kTileUnits; ++u) {
            ok = 2 * r + u < kUnits || wait(raw_empty[unit], unit_phase ^ 1, 102);
            if (!ok) break;
            const uint32_t here = held >> (u * kUnitRecords) & 15u, bar = smem_u32(&raw_full[unit]);
            if (lane == 0) {
              if (here != 0)
                mbar_expect_tx(bar, __popc(here) * p.run * (18 * D));
              else
                mbar_arrive(bar);
            }
            __syncwarp();
            if (there && lane / kUnitRecords == u && !(PROBE && 2 * r + u == 3))
              tma_load_4d(sRaw + unit * Raw::kUnitBytes + (lane % kUnitRecords) * (18 * D), &tm_codes, bar, 0,
                          in_page * Raw::kLines, g, my_page);
            ++units;
            if (++unit == kUnits) unit = 0, unit_phase ^= 1;
          }
          if (!ok) break;
        }
        at += count;
        left -= count;
        ++it;
      }
      ok = ok && (it < kItems || wait(bars.item_empty[it % kItems], (it / kItems - 1) & 1, 120));
      if (lane == 0) {
        if (ok) items[it % kItems].rounds = 0;  // (else the abort flag ends every warp's list)
        if (ok) mbar_arrive(smem_u32(&bars.item[it % kItems]));
        p.parts[blockIdx.x] = mine_part;
      }
      __syncwarp();
      // Before the CTA can exit, every copy issued must have landed (also after an abort). The last kUnits units and
      // kScaleStages rounds may be on their way: unit u of the ring's current turn has phase unit_phase for u < unit.
      if (lane == 0) {
#pragma unroll 1
        for (int k = 0; k < kUnits + kScaleStages; ++k) {
          const int st = k - kUnits;
          if (k < kUnits ? k < unit || units >= kUnits : st < scales)
            mbar_wait_inl(k < kUnits ? smem_u32(&raw_full[k]) : smem_u32(&bars.sc_full[st]),
                          k < kUnits ? (k < unit ? unit_phase : unit_phase ^ 1) : ((scales - 1 - st) / kScaleStages) & 1,
                          abort_flag, b.err, 103, false, kLimit);
        }
      }
    } else if (warp == kWarpScales) {
      int r = 0;
      bool ok = true;
      for (int it = 0, n; ok && (n = item_at(it)) > 0; ++it) {
        const int j0 = items[it % kItems].j0, place0 = items[it % kItems].place0;
        int most_v = kNoExponent;  // of the run so far
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++r) {
          const int st = r % kScaleStages;
          ok = wait(bars.sc_full[st], (r / kScaleStages) & 1, 105);
          if (!ok) break;
          const int2 info = scale_info[st];
          int e_k, e_v;
          const bool wide = prepare_scales<D>(sScale + st * Raw::kScaleBytes, info.x, (uint32_t)info.y, lane, (j0 + j) * kBN,
                                              nan_from[it % kItems], most_v - kValueRange,
                                              (j0 + j) * kBN + min(info.x, kBN) - 1 > place0,
                                              p.own + ((int)blockIdx.x * kItems + r % kItems) * kBN, e_k, e_v);
          most_v = max(most_v, e_v);
          if (lane == 0) rounds_info[r % kItems] = Round{(float)e_k, (float)e_v, info.y, wide};
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.sc_ready[st]));
        }
        leave_item(it);
      }
    } else if (warp == kWarpMma) {
      constexpr uint32_t idesc_s = idesc_f16(kBM, kBN);
      constexpr uint32_t idesc_o = idesc_f16(kBM, D);
      // S_i = Q_i K^T of round r; elected lane only. last: no other tile needs the round's keys.
      auto issue_s = [&](int i, int r, bool last) {
        const int st = r % kStages;
        const uint32_t dq = desc_lo(sQ + (ONE ? 0 : i) * kQBytes), dk = desc_lo(sK0 + st * kKVBytes), d = tmem + col_s(i);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t at = ((ks / 4) * kBox + ks % 4 * 32) >> 4;
          mma_ss_lo(d, dq + at, dk + at, idesc_s, ks > 0 ? 1u : 0u);
        }
        tc_commit(smem_u32(&bars.s_full[i]));
        if (last) tc_commit(smem_u32(&bars.k_free[st]));
      };
      // O_i (+)= P_i V of round r: P from TMEM (16 keys = 8 columns per MMA).
      auto issue_pv = [&](int i, int r, bool first, bool last) {
        const int st = r % kStages;
        const uint32_t dv = desc_lo(sV0 + st * kKVBytes), d = tmem + col_o(i, D), a = tmem + col_s(i);
#pragma unroll
        for (int ks = 0; ks < kBN / 16; ++ks)
          mma_ts_lo(d, a + ks * 8, dv + (((ks / 4) * kVBox + ks % 4 * 32) >> 4), idesc_o, (ks > 0 || !first) ? 1u : 0u);
        tc_commit(smem_u32(&bars.o_done[i]));
        if (last) tc_commit(smem_u32(&bars.v_free[st]));
      };
      int r = 0, n_p = 0, n_q = 0;  // bit i: parity of tile i's next P, q
      bool ok = true;
      for (int it = 0, n; ok && (n = item_at(it)) > 0; ++it) {
        // Per round and tile the products, then the scores of the tile's next round (`step` later).
        const bool two = items[it % kItems].two != 0;
        constexpr int step = ONE ? 2 : 1;
#pragma unroll 1
        for (int j = -step; j < n && ok; ++j) {
          const int i1 = ONE ? j & 1 : two ? 1 : 0;
#pragma unroll 1
          for (int i = ONE ? i1 : 0; i <= i1 && ok; ++i) {
            if (j >= 0) {
              const int rr = r + j;
              ok = wait(bars.p_full[i], n_p >> i & 1, 108) && wait(bars.v_full[rr % kStages], (rr / kStages) & 1, 109);
              n_p ^= 1 << i;
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) issue_pv(i, rr, j < step, i == i1);
              __syncwarp();
            }
            if (j + step >= n) continue;
            const int next = r + j + step;
            if (j < 0 && (!ONE || j == -step)) {
              ok = wait(bars.q_full[i], n_q >> i & 1, 106);
              n_q ^= 1 << i;
            }
            ok = ok && wait(bars.k_full[next % kStages], (next / kStages) & 1, 107);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) issue_s(i, next, i == i1);
            __syncwarp();
          }
        }
        r += n;
        leave_item(it);
      }
      // All tensor-core work issued by this CTA completes before TMEM is freed.
      if (elect_one()) tc_commit(smem_u32(&bars.drain));
      __syncwarp();
      mbar_wait_inl(smem_u32(&bars.drain), 0, abort_flag, b.err, 110, false, kLimit);
    } else {
      for (int s = blockIdx.x * 32 + lane; s < b.n_seqs; s += gridDim.x * 32) kv4_check_request(b, s);
    }
    __syncwarp();
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
    return;
  } else if (warp >= kWarpWiden) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWidenRegs));
    const int part = warp % 4;  // keys: a record of each unit; values: half of the r, a pair of groups (or a unit)
    const bool keys = warp < kWarpWiden + kWidenWarps / 2;
    int r = 0, unit = 0, unit_phase = 0;
    bool ok = true;
    for (int it = 0, n; ok && (n = item_at(it)) > 0; ++it) {
      for (int j = 0; j < n && ok; ++j, ++r) {
        const int st = r % kStages, ss = r % kScaleStages;
        const uint32_t scales = sScale + ss * Raw::kScaleBytes;
        ok = wait(bars.sc_ready[ss], (r / kScaleStages) & 1, 111) &&
             // the stage of round r - 2 is free once the products that read it are complete
             (r < kStages || wait(keys ? bars.k_free[st] : bars.v_free[st], (r / kStages - 1) & 1, 112));
#pragma unroll 1
        for (int u = 0; u < kTileUnits && ok; ++u) {
          ok = wait(raw_full[unit], unit_phase, 113);
          if (!ok) break;
          const uint32_t raw = sRaw + unit * Raw::kUnitBytes;
          if (keys)
            widen_keys<D>(sK0 + st * kKVBytes, raw, scales, u, part, 1, lane);
          else if (D == 128 || part / 2 == u)
            widen_values<D>(sV0 + st * kKVBytes, raw, scales, u, part % 2 * 4, D == 128 ? part / 2 * 2 : 0, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&raw_empty[unit]));
          if (++unit == kUnits) unit = 0, unit_phase ^= 1;
        }
        if (!ok) break;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read what was written
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars.sc_empty[ss]));
          mbar_arrive(smem_u32(keys ? &bars.k_full[st] : &bars.v_full[st]));
        }
      }
      leave_item(it);
    }
    __syncwarp();
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
    return;
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int ti = warp / 4;  // this warpgroup's tile
    const int row = tid % kBM;
    const uint32_t lane_base = tmem + ((uint32_t)((warp % 4) * 32) << 16);
    const int tq = kBM >> p.lg, group = 1 << p.lg;
    int r = 0;
    bool ok = true;
    float a_row = 0.0f, e_row = 0.0f;  // scale in log2 units, and the power of two of the row's q
    float most_e_k = 0.0f;
    const int scale_exponent = (int)(__float_as_uint(b.scale * 1.4426950408889634f) >> 23 & 255u) - 126;
    // This thread's row of the item's q into shared memory, in fp16 (rows past the item's end repeat its last token).
    auto load_q = [&](const Item& x) {
      const int token = min((ONE ? 0 : ti * tq) + (row >> p.lg), x.tokens - 1);
      const uint8_t* src = b.q + (((int64_t)(x.row0 + token) * b.hq + (x.g << p.lg) + (row & (group - 1))) * D) * 2;
      uint4 v[D / 8];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, w[e] >> 16 & 0x7fffu));
      }
      const int by = 141 - max((int)(top >> 7), 1);  // puts the largest magnitude into [2^14, 2^15): -114 .. 140
      const float f0 = power_of_2(by >> 1), f1 = power_of_2(by - (by >> 1));
      a_row = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : b.scale * 1.4426950408889634f;
      e_row = (float)-by;
      // the keys' exponents up to which the factors of this warp's rows stay within the limit
      most_e_k = (float)__reduce_min_sync(0xffffffffu, top >= 0x7f80u ? 1000 : kFactorExponent + by - scale_exponent);
      if (ONE && ti == 1) return;  // the first tile's warps write it for both
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * f0 * f1;
        sts4(sQ + ti * kQBytes + (i / 8) * kBox + row * 128 + (uint32_t)(((i % 8) ^ (row & 7)) * 16),
             h2_bits(__floats2half2_rn(f[0], f[1])), h2_bits(__floats2half2_rn(f[2], f[3])),
             h2_bits(__floats2half2_rn(f[4], f[5])), h2_bits(__floats2half2_rn(f[6], f[7])));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.q_full[ti]));
    };
    // Item `it` after item it - 1's rounds and before its output, so that the first scores form while that is written.
    int n = 0, done = 0;                   // done: this tile's rounds so far
    int odd = 0, handed = 0;               // ONE: odd rounds so far; items whose odd rounds' result was handed over
    bool not_read = false;                 // (the last of them may not have been read)
#pragma unroll 1
    for (int it = -1; it < 0 || n > 0; ++it) {
      const Item x = items[max(it, 0) % kItems];  // (before the first: not used)
      const bool work = it >= 0 && (ONE || ti == 0 || x.two);
      constexpr int step = ONE ? 2 : 1;
      const int first = ONE ? ti : 0;  // this tile's rounds: from here on every step-th
      const int my_token = min((ONE ? 0 : ti * tq) + (row >> p.lg), x.tokens - 1), my_place = x.place0 + my_token;
      float m_ref = -INFINITY, l = 0.0f, e_b = 0.0f;  // reference (log2 units) that O_ti and l are scaled to, exponent
      bool has_b = false;                             // that l is for
      // One round, by halves of 64 keys (in a loop: the roles share the instruction cache), a quarter's scores on their way
      // from TMEM while the one before is worked on; false if a wait gave up (the abort flag is raised then).
      auto tile = [&](int j) -> bool {
        const int rr = r + j;
        tc_fence_after();
        const uint32_t taddr = lane_base + col_s(ti);  // a half's P lies over the first half's scores, which have been read
        uint32_t s0[kQuarter], s1[kQuarter];
        tmem_ld_x32_async(taddr, s0);
        const Round info = rounds_info[rr % kItems];
        // the row's factor for keys of exponent e_k (not 0, which times -infinity, a hidden key's score, is NaN)
        auto factor = [&](float e_k) -> float {
          const float e = e_k + e_row, eh = floorf(0.5f * e);
          return fmaxf(a_row * ex2(eh) * ex2(e - eh), 1.2e-38f) + (a_row - a_row);
        };
        const int lim = my_place - (x.j0 + j) * kBN;  // columns c <= lim are visible to this row
        if (__builtin_expect(info.wide != 0 || info.e_k > most_e_k, 0)) {
          tmem_wait_ld(s0);
          const float2* own = p.own + ((int)blockIdx.x * kItems + rr % kItems) * kBN;
          // Columns 16 u .. + 15: their scores (log2 units) and values' exponents.
          auto columns = [&](int u, float (&y)[16], float (&ev)[16]) {
            uint32_t z[16];
            tmem_ld_x16(taddr + 16 * u, z);
            const bool gone = info.bad >> u & 1;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 e = make_float2(info.e_k, info.e_v == (float)kNoExponent ? e_b : info.e_v);
              if (info.wide != 0) e = __ldcg(own + 16 * u + i);
              y[i] = gone || 16 * u + i > lim ? -INFINITY : __uint_as_float(z[i]) * factor(e.x);
              ev[i] = e.y;
            }
          };
          float y[16], ev[16];
          float most = -INFINITY, rel = -INFINITY;  // the largest score; of what a key gives, relative to it
#pragma unroll 1
          for (int u = 0; u < kBN / 16; ++u) {
            columns(u, y, ev);
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, y[i]);
          }
#pragma unroll 1
          for (int u = 0; u < kBN / 16; ++u) {
            columns(u, y, ev);
#pragma unroll
            for (int i = 0; i < 16; ++i) rel = fmaxf(rel, (y[i] - most) + ev[i]);
          }
          // The weights are 2^(score - ref) here, and P 2^(ev - e_b) times that: scores may be so large that a value's exponent
          // is lost beside them, so m_ref = ref + e_b is no measure for both.
          float ref = m_ref == -INFINITY ? 0.0f : m_ref - e_b, f = 1.0f;
          if (most != -INFINITY) {
            const float ref0 = m_ref - e_b;
            ref = fmaxf(ref0, most - kHeadroom);
            const float up = ref - ref0;
            float e = e_b - floorf(up);  // O is not scaled up,
            const float need = ceilf((most - ref) + rel - kHeadroom);  // and P lies about 2^6 at most
            if (need > e + kRescaleThreshold) e = need;
            f = ex2(e_b - e - up);
            l *= ex2(-up);
            e_b = e;
            m_ref = ref + e;
            has_b = true;
          }
          if (j > first && __any_sync(0xffffffffu, f != 1.0f)) {
            if (!wait(bars.o_done[ti], (done - 1) & 1, 116 + ti)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int i0 = 0; i0 < D; i0 += 16) {
              uint32_t o[16];
              tmem_ld_x16(lane_base + col_o(ti, D) + i0, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st_x16(lane_base + col_o(ti, D) + i0, o);
            }
          }
#pragma unroll 1
          for (int u = 0; u < kBN / 16; ++u) {  // (a column of P lies over scores that have been read)
            columns(u, y, ev);
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float a = y[i] - ref, b = y[i + 1] - ref;
              l += ex2(a) + ex2(b);
              pk[i / 2] = h2_bits(__floats2half2_rn(ex2(a + (ev[i] - e_b)), ex2(b + (ev[i + 1] - e_b))));
            }
            tmem_st_x8(taddr + 8 * u, pk);
          }
          tmem_st_wait();
          return true;
        }
        const float a = factor(info.e_k);
        float e_v = e_b;
        if (info.e_v != (float)kNoExponent) {
          e_v = info.e_v;
          if (!has_b) {  // nothing in O yet: the reference moves with the exponent that it is for
            m_ref += e_v - e_b;
            e_b = e_v;
            has_b = true;
          }
        }
        float to_l = ex2(fminf(fmaxf(e_b - e_v, -126.0f), 126.0f));
        const bool hidden = info.bad != 0 || __any_sync(0xffffffffu, lim < kBN - 1);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int c0 = 2 * kQuarter * h;
          uint32_t pk[kQuarter];
          uint32_t(&pk0)[kQuarter / 2] = *reinterpret_cast<uint32_t(*)[kQuarter / 2]>(&pk[0]);
          uint32_t(&pk1)[kQuarter / 2] = *reinterpret_cast<uint32_t(*)[kQuarter / 2]>(&pk[kQuarter / 2]);
          tmem_wait_ld(s0);
          tmem_ld_x32_async(taddr + c0 + kQuarter, s1);
          if (hidden) hide(s0, lim - c0, info.bad >> (4 * h));
          // Halves run against a reference and take their max only where their sum shows that it is too low. The
          // first one's is the max of its first 32 columns: the rest is within 2^9 of it but for rare rows, which the
          // check finds.
          if (j == first && h == 0) {
            const float top = quarter_max(s0);
            if (top != -INFINITY) m_ref = fmaf(top, a, e_v - kHeadroom);
          }
          float sum = 0.0f;
          quarter_p(s0, a, e_v - m_ref, pk0, sum);
          tmem_wait_ld(s1);
          tmem_ld_x32_async(taddr + (c0 + 2 * kQuarter) % kBN, s0);  // (behind the second half not used)
          if (hidden) hide(s1, lim - c0 - kQuarter, info.bad >> (4 * h + 2));
          quarter_p(s1, a, e_v - m_ref, pk1, sum);
          if (!__all_sync(0xffffffffu, sum <= kHalfSumLimit && m_ref != -INFINITY)) {
            // Rare: against the half's max (also where nothing is visible or a score is no number).
            float top = -INFINITY;
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              tmem_ld_x32(taddr + c0 + kQuarter * i, s1);
              if (hidden) hide(s1, lim - c0 - kQuarter * i, info.bad >> (4 * h + 2 * i));
              top = fmaxf(top, quarter_max(s1));
            }
            const float mt = top == -INFINITY ? -INFINITY : fmaf(top, a, e_v - kHeadroom);
            const bool raise = mt > m_ref + kRescaleThreshold;  // always, at a row's first visible key
            if (__any_sync(0xffffffffu, raise)) {
              const float alpha = raise ? ex2(m_ref - mt) : 1.0f;  // 0 for a row that had nothing visible
              const bool scale_o = raise && m_ref != -INFINITY;
              if (raise) {
                // what of it the values ask for, and not the scores, leaves the sum as it is
                const float up = floorf(fminf(fmaxf(e_v - e_b, 0.0f), mt - m_ref));
                l *= ex2(m_ref - mt + up);
                e_b += up;
                to_l = ex2(fminf(fmaxf(e_b - e_v, -126.0f), 126.0f));
                m_ref = mt;
              }
              const float f = scale_o ? alpha : 1.0f;
              // O_ti holds the sum through its round before (wait for that product), the other half's P lies in TMEM
              if ((j > first || h > 0) && __any_sync(0xffffffffu, scale_o)) {
                if (j > first && !wait(bars.o_done[ti], (done - 1) & 1, 116 + ti)) return false;
                tc_fence_after();
                tmem_st_wait();
#pragma unroll 1
                for (int i0 = j > first ? 0 : D; i0 < D + 32 * h; i0 += 16) {
                  const uint32_t at = i0 < D ? lane_base + col_o(ti, D) + i0 : taddr + i0 - D;
                  uint32_t o[16];
                  tmem_ld_x16(at, o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const float2 y = __half22float2(h2_of(o[i]));
                    o[i] = i0 < D ? __float_as_uint(__uint_as_float(o[i]) * f) : h2_bits(__floats2half2_rn(y.x * f, y.y * f));
                  }
                  tmem_st_x16(at, o);
                }
                tmem_st_wait();
              }
            }
            const float off = m_ref == -INFINITY ? 0.0f : e_v - m_ref;
            sum = 0.0f;
            tmem_ld_x32(taddr + c0, s1);
            if (hidden) hide(s1, lim - c0, info.bad >> (4 * h));
            quarter_p(s1, a, off, pk0, sum);
            tmem_ld_x32(taddr + c0 + kQuarter, s1);
            if (hidden) hide(s1, lim - c0 - kQuarter, info.bad >> (4 * h + 2));
            quarter_p(s1, a, off, pk1, sum);
          }
          l = fmaf(sum, to_l, l);
          tmem_st_x32(taddr + kQuarter * h, pk);
        }
        tmem_wait_ld(s0);
        tmem_st_wait();
        return true;
      };
      if (ONE && not_read) {  // before O and the statistics change
        ok = ok && wait(bars.stats_read, (handed - 1) & 1, 121);
        not_read = false;
      }
#pragma unroll 1
      for (int j = work ? first : n; j < n; j += step, ++done) {
        ok = ok && wait(bars.s_full[ti], done & 1, 114 + ti) && tile(j);
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[ti]));
      }
      r += n;
      const int rounds = n;
      // Its tile in shared memory is free: the last scores are formed (ONE: the odd rounds' too).
      if (ONE && ti == 0) {
        ok = ok && (rounds < 2 || wait(bars.s_full[1], (odd + rounds / 2 - 1) & 1, 114));
        odd += rounds / 2;
      }
      n = ok ? item_at(it + 1) : 0;
      if (n > 0 && (ONE || ti == 0 || items[(it + 1) % kItems].two)) load_q(items[(it + 1) % kItems]);
      if (!work) {
        if (it >= 0) leave_item(it);
        continue;
      }
      ok = ok && (rounds <= first || wait(bars.o_done[ti], (done - 1) & 1, 118 + ti)) && !*abort_flag;
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (ONE && ti == 1) {  // the first tile's warps join the two
        s_ref[row] = m_ref;
        s_sum[row] = l;
        s_exp[row] = e_b;
        ++handed;
        not_read = true;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.stats_full));
        leave_item(it);
        continue;
      }
      // Both relative to the larger reference; weights of O_0 and O_1.
      float w0 = 1.0f, w1 = 0.0f;
      bool odd_too = false;
      if (ONE) {
        ok = wait(bars.stats_full, handed++ & 1, 122);
        if (!ok) break;
        tc_fence_after();
        const float m1 = s_ref[row], l1 = s_sum[row], e1 = s_exp[row];
        const float r0 = m_ref - e_b, r1 = m1 - e1, r = fmaxf(r0, r1);  // the sums' own references
        odd_too = rounds > 1;
        if (odd_too && r != -INFINITY) {
          const float d0 = r0 - r, d1 = r1 - r, e = ceilf(fmaxf(d0 + e_b, d1 + e1));
          w0 = ex2(d0 + (e_b - e));
          w1 = ex2(d1 + (e1 - e));
          l = l * ex2(d0) + l1 * ex2(d1);
          e_b = e;
          m_ref = r + e;
        }
      }
      const float e_out = e_b, m_out = m_ref, l_out = l;
      // out = O_ti 2^e_b / l, each thread its row.
      const float inv = l_out == 0.0f ? 0.0f : 1.0f / l_out;
      const float eh = floorf(0.5f * e_out), f0 = ex2(eh), f1 = ex2(e_out - eh);
      const bool stored = (ONE ? 0 : ti * tq) + (row >> p.lg) < x.tokens;
      const int64_t at = ((int64_t)(x.row0 + my_token) * b.hq + (x.g << p.lg) + (row & (group - 1)));
      const int64_t part = x.part < 0 ? 0 : ((int64_t)blockIdx.x * 2 + x.part) * (kTiles * kBM) + ti * kBM + row;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld_x32(lane_base + col_o(ti, D) + c0, o);
        if (ONE && odd_too) {
          uint32_t o1[32];
          tmem_ld_x32(lane_base + col_o(1, D) + c0, o1);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), w1, __uint_as_float(o[i]) * w0));
        }
        const bool no_number = nan_from[it % kItems][c0 / kKv4Group] <= my_place;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float y = __uint_as_float(o[i]) * inv * f0 * f1;
          o[i] = no_number ? 0x7fc00000u : __float_as_uint(y);
        }
        if (stored) {
          if (x.part < 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float f[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[8 * i + e]);
              *reinterpret_cast<uint4*>(p.out + (at * D + c0 + 8 * i) * 2) = pack8(f);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(p.part_o + part * D + c0 + 4 * i) =
                  make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        __syncwarp();  // the next load of TMEM is warp-aligned
      }
      if (ONE) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.stats_read));
      }
      if (stored) {
        const float m = m_out - e_out;  // the sum is l 2^m
        if (x.part >= 0)
          p.part_ml[part] = make_float2(m, l_out);
        else if (p.lse != nullptr)
          p.lse[at] = l_out == 0.0f ? -INFINITY : (m + log2f(l_out)) * 0.6931471805599453f;
      }
      leave_item(it);
    }
    __syncwarp();
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
    if (warp == 0) {
      tc_fence_after();
      if (lane == 0 && s_abort != 0) record_error(b.err, kErrTimeout, s_abort);
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
  }
}

// Joins the partial results of the items that span CTAs: block (c, y) takes rows 32 y .. of the item that begins in
// CTA c and ends in a later one. A warp per row, a lane per four (two) dims.
constexpr int kJoinRows = 32;
template <int D>
__global__ void __launch_bounds__(256) kv4_join_kernel(const ChunkParams p) {
  constexpr int kPer = D / 32;
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x, lane = threadIdx.x % 32;
  const Part it = p.parts[c];
  for (int k = threadIdx.x / 32; k < kJoinRows; k += 8) {
    const int row = blockIdx.y * kJoinRows + k;
    if (row >= it.tokens << p.lg || it.parts == 0) return;
    auto at = [&](int i) -> int64_t { return ((int64_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * (kTiles * kBM) + row; };
    float m = -INFINITY;
    for (int i = lane; i < it.parts; i += 32) {
      const float2 ml = __ldcg(&p.part_ml[at(i)]);
      if (ml.y != 0.0f) m = fmaxf(m, ml.x);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float o[kPer] = {}, l = 0.0f;
    for (int i = 0; i < it.parts; ++i) {
      const float2 ml = __ldcg(&p.part_ml[at(i)]);
      const float w = ml.y == 0.0f ? 0.0f : ml.y * ex2(ml.x - m);
      l += w;
      const float* src = p.part_o + at(i) * D + lane * kPer;
#pragma unroll
      for (int d = 0; d < kPer; d += 2) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(src + d));
        o[d] = fmaf(w, v.x, o[d]);
        o[d + 1] = fmaf(w, v.y, o[d + 1]);
      }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t dst = (int64_t)(it.row0 + (row >> p.lg)) * p.b.hq + (it.g << p.lg) + (row & ((1 << p.lg) - 1));
#pragma unroll
    for (int d = 0; d < kPer; d += 2)
      *reinterpret_cast<uint32_t*>(p.out + (dst * D + lane * kPer + d) * 2) = pack2(o[d] * inv, o[d + 1] * inv);
    if (p.lse != nullptr && lane == 0) p.lse[dst] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

template <int D, bool ONE, bool PROBE = false>
cudaError_t launch_t(const Kv4Batch& b, void* out, float* lse, const Kv4ChunkScratch& ws, cudaStream_t s) {
  // The register split: see prompt_attention.cu; a build with fewer registers than it needs would wait forever.
  static std::atomic<int> known{-1};
  int regs = known.load(std::memory_order_relaxed);
  if (regs < 0) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, kv4_chunk_kernel<D, ONE, PROBE>);
    if (e != cudaSuccess) return e;
    regs = a.numRegs;
    known.store(regs, std::memory_order_relaxed);
  }
  if (regs * kThreads < kSoftmaxThreads * (kTiles * kSoftmaxRegs + kWidenWarps / 4 * kWidenRegs + kOtherRegs))
    return cudaErrorNotSupported;
  ChunkParams p;
  p.b = b;
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.part_o = ws.part_o;
  p.part_ml = ws.part_ml;
  p.parts = static_cast<Part*>(ws.parts);
  p.own = ws.own;
  p.lg = 31 - __builtin_clz(b.hq / b.hkv);
  p.few = PROBE ? 0 : kv4_chunk_few_rows(b) >> p.lg;
  // (1.15 ms for 2,048 tokens over 30,720 where each record has a copy of its own, 1.13 with four to a copy)
  p.run = b.page_size % 64 == 0 ? 4 : b.page_size % 32 == 0 ? 2 : 1;
  static_assert(kUnitRecords == 4, "records per copy");
  CUtensorMap codes, scales;
  // (without pages nothing is read: any address will do)
  if (!encode_cache_maps(&codes, &scales, b.n_pages > 0 ? b.cache : b.q, std::max(b.n_pages, 1), b.page_size, b.hkv, D, p.run))
    return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)((ONE ? 1 : 2) * kBM + 2 * kStages * kBN) * D * 2 + units_of(D, ONE) * Kv4Raw<D>::kUnitBytes +
                      (ONE ? 4 : 2) * Kv4Raw<D>::kScaleBytes;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = set_smem_limit_once(kv4_chunk_kernel<D, ONE, PROBE>, (int)smem, configured);
  if (e != cudaSuccess) return e;
  // no more CTAs than there can be rounds
  const int64_t items_at_most = ((int64_t)b.n_rows / ((ONE ? 1 : 2) * kBM >> p.lg) + b.n_seqs) * b.hkv;
  const int64_t most = items_at_most * ((int64_t)b.width * b.page_size / kBN + 1);
  const int grid = (int)std::min<int64_t>(most, ws.sms);
  e = launch_pdl(kv4_chunk_kernel<D, ONE, PROBE>, dim3((unsigned)grid), dim3(kThreads), smem, s, codes, scales, p);
  if (e != cudaSuccess) return e;
  const int rows = (int)std::min<int64_t>((int64_t)b.n_rows << p.lg, (ONE ? 1 : 2) * kBM);
  return launch_pdl(kv4_join_kernel<D>, dim3((unsigned)grid, (unsigned)((rows + kJoinRows - 1) / kJoinRows)), dim3(256), 0, s, p);
}

}  // namespace

size_t kv4_chunk_part_rows(int32_t sms) { return (size_t)sms * 2 * kTiles * kBM; }
size_t kv4_chunk_parts_bytes(int32_t sms) { return (size_t)sms * sizeof(Part); }
size_t kv4_chunk_own_keys(int32_t sms) { return (size_t)sms * kItems * kBN; }

// (Request, kv head) pairs of a batch from which on its requests of few rows are worth a launch of their own, whether it has
// any or not; where the mean request has so few rows, fewer are enough. With and without the launch, us, 32 query on 8 kv
// heads of 128 dims:
//   32 requests (256 pairs), one in eight of 256 tokens, the others of one: 512 keys 84 and 82, 2,048 keys 126 and 156, 8,192
//   keys 259 and 400; all of 64 tokens: 84 and 76, 141 and 133, 321 and 311;
//   16 requests (128 pairs), one in eight of 256: 66 and 57, 94 and 97, 162 and 225; all of 64: 45 and 36, 93 and 85, 185 and 176;
//   all of one token: 8 requests (64 pairs) of 8,192 keys 47 and 66; 16 requests 24 and 25, 39 and 50, 63 and 107; 64 requests
//   of 128 keys 28 and 46; but 2 requests (16 pairs) of 128, 1,024 and 8,192 keys 22 and 19, 26 and 21, 35 and 33.
constexpr int64_t kFewPairs = 256, kAllFewPairs = 64;

int32_t kv4_chunk_few_rows(const Kv4Batch& b) {
  const int group = b.hq / b.hkv, few = group > 8 ? 16 : 8;
  // its records are counted in 31 bits
  if ((int64_t)b.n_seqs * b.hkv * b.width * (b.page_size / kKv4Block) >= (1 << 30)) return 0;
  const bool all = (int64_t)b.n_rows * group <= (int64_t)few * b.n_seqs;
  return (int64_t)b.n_seqs * b.hkv >= (all ? kAllFewPairs : kFewPairs) ? few : 0;
}

cudaError_t launch_kv4_chunk(const Kv4Batch& b, int32_t head_dim, void* out, float* lse, const Kv4ChunkScratch& ws,
                             cudaStream_t s) {
  const int few = kv4_chunk_few_rows(b);
  const int64_t rows = (int64_t)b.n_rows * (b.hq / b.hkv);
  if (few > 0) {
    const cudaError_t e = launch_kv4_chunk_few(b, head_dim, out, lse, ws.few, s);
    if (e != cudaSuccess) return e;
  }
  // Items of one tile where a request's rows fill no more on the average (both measured above).
  const bool one = rows <= (int64_t)kBM * b.n_seqs;
  if (head_dim == 128) return one ? launch_t<128, true>(b, out, lse, ws, s) : launch_t<128, false>(b, out, lse, ws, s);
  if (head_dim == 64) return one ? launch_t<64, true>(b, out, lse, ws, s) : launch_t<64, false>(b, out, lse, ws, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_chunk_timeout_probe(const Kv4Batch& b, void* out, const Kv4ChunkScratch& ws, cudaStream_t s) {
  return launch_t<128, false, true>(b, out, nullptr, ws, s);
}

}  // namespace cb
