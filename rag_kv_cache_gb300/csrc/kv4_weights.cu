// Accumulated attention weights over a paged cache held in 4 bits (kv4_layout.cuh):
//
//   weights[s, g, j] = earlier[s, g, j] + sum_{t, h in g} exp(scale q[t, h] . k_j[g] - lse[t, h])
//
// over the request's last `window` rows t that see token j.
//
// The scores are formed transposed, S^T = K Q^T (tcgen05.mma, fp16, fp32 accumulators in tensor memory): a token is a lane
// and its weight a sum along the lane's columns, 128 rows (tokens times heads of the kv head) at a time, so nothing
// passes between threads and the order of the sum is fixed. Every token is owned by one CTA: no atomics, and its codes
// are read and widened once. A unit of work is four tiles of 128 tokens of one (request, kv head), which share
// the conversion of the rows to fp16.
//
// Requests of few rows go to a kernel on mma.sync (kv4_weights_few.cu).
//
// Bound: a token and kv head costs 5/8 D bytes of the cache (and D / 16 of V's scales, which lie between K's), 8 of weights;
// a (row, token) pair 2 D flops (an SM takes 32 pairs' per cycle at D = 128) and one exponential (32).
//
// Parts: twelve warps in three groups of 128 threads take the products (tile x 128 rows) in turn, a thread per token, and leave the
// sums of tiles that another group writes in shared memory; eight warps widen the codes and convert the rows, which come by
// TMA, in place (loaded by these warps through registers they waited 4,100 cycles per 128 rows: 173 us for the prompts below);
// one issues the products, one asks for rows, one makes the list of units. The rows' lse have a ring of their own, since they
// are needed until the last exponential and the rows only until the last product (one ring: 159 us).
//
// Work split: the tiles of all requests and kv heads in a row, in one contiguous run per CTA, of equal cost (one for a tile,
// one for each 128 rows that see it; 194 us before, with all of a request's tiles of equal cost, 171 with it).
//
// Measured (32 query on 8 kv heads of 128 dims): eight pieces of prompts of up to 1,024 tokens over up to 2,048, 139 us (27 us
// of products at the burst rate); the last 32 rows over 32,896 tokens 31 us. The first is bound by the latency of the
// exponentials' loop: a product takes a group 3,900 cycles with three at work (2,730 with two; 512 cycles of a scheduler's
// transcendental pipe, which is in use 25% of the time).
// Scores loaded 32 columns at a time in place of 16 ahead: 140 us.
//
// Powers of two: a key is held as k 2^-e_k (its lane's factor; no key, seen or not, takes bits from another), rows as q 2^-e_q
// per 128 rows.
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

constexpr int kTile = 128;        // tokens per tile
constexpr int kTiles = 4;         // tiles per unit; tile q of a unit has stage q of K; stages of S, taken in turn
constexpr int kRows = 128;        // rows per chunk
constexpr int kQStages = 2;       // of rows
constexpr int kLseStages = 4;     // of their lse, which are needed for longer
constexpr int kUnits = 8;         // ring of units
constexpr int kRecords = 2;       // records on their way to a widening warp, or held for it
constexpr int kGroups = 3;        // of 128 threads, which take the products in turn
constexpr int kExpWarps = 4 * kGroups;
constexpr int kWarpWiden = kExpWarps;  // 12 .. 19: a record of each tile, 16 of each chunk's rows
constexpr int kWidenWarps = 8;
constexpr int kWarpMma = kWarpWiden + kWidenWarps;
constexpr int kWarpRows = kWarpMma + 1;   // asks for the rows
constexpr int kWarpUnits = kWarpRows + 1; // makes the list of units
constexpr int kUnitReaders = kWarpUnits;  // all other warps
constexpr int kThreads = 32 * (kWarpUnits + 1);
constexpr uint32_t kTmemCols = 512;
constexpr int kBadRecord = -128;  // in place of a token's exponent: its page is none
// Units whose tokens' exponents are held. A unit's keys are widened once the last product of the unit before is complete, which
// was issued once the scores of the fourth product before it were taken; a unit has one product at least.
constexpr int kHeldUnits = kTiles + 1;

struct WeightsParams {
  Kv4Batch b;
  const float* lse;
  const float* earlier;
  float* weights;
  int window;
  int lg;   // log2 of the query heads per kv head
  int few;  // requests of so many row tokens or fewer are another kernel's
};

struct Bars {
  uint64_t unit[kUnits], unit_free[kUnits];
  uint64_t raw[kWidenWarps][kRecords];
  uint64_t k_full[kTiles], k_free[kTiles];
  uint64_t s_full[kTiles], s_free[kTiles];
  uint64_t q_raw[kQStages], q_full[kQStages], q_free[kQStages];  // rows as they are, in fp16, no longer needed
  uint64_t lse_full[kLseStages], lse_free[kLseStages];
  uint64_t top;  // the largest magnitudes of a chunk's rows are known
  uint64_t part[kGroups];  // a group's sums of the others' tiles are there
  uint64_t drain;
};

// What of a request counts.
struct Share {
  int tiles;   // per kv head
  int rows0;   // first row (in q), the place in the cache of its token
  int place0;
  int tokens;  // row tokens
  int chunks;
  int len, old;  // the request's tokens, those before its rows
};
__device__ __forceinline__ Share share_of(const WeightsParams& p, int s) {
  const Kv4Request r = kv4_request(p.b, s);
  Share x;
  x.tokens = p.window > 0 ? min(p.window, r.m) : r.m;
  x.tiles = x.tokens > p.few && r.len > 0 ? (r.len - 1) / kTile + 1 : 0;
  x.rows0 = r.row0 + r.m - x.tokens;
  x.place0 = r.len - x.tokens;
  x.chunks = ((x.tokens << p.lg) + kRows - 1) / kRows;
  x.len = r.len;
  x.old = r.len - r.m;
  return x;
}

// The first chunk that a row of which sees the tile's first token.
__device__ __forceinline__ int first_chunk(const Share& x, int tile, int lg) { return max(tile * kTile - x.place0, 0) >> (7 - lg); }

// What the tiles 0 .. n - 1 of a kv head cost: one each, and one for each chunk that sees it.
__device__ __forceinline__ int64_t cost_before(const Share& x, int n, int lg) {
  const int t1 = (max(x.place0, 0) + kTile - 1) / kTile, k = max(n - t1, 0);  // from t1 on one chunk per head fewer and fewer
  return (int64_t)n * (x.chunks + 1) - (int64_t)k * first_chunk(x, t1, lg) - ((int64_t)k * (k - 1) / 2 << lg);
}

// Up to four tiles of one request and kv head.
struct Unit {
  Share r;
  int s, g, t;  // request, kv head, first tile
  int n;        // its tiles, 0: no more units
  int first;    // first chunk that sees one of them
  int fresh;    // its rows are not those of the unit before (of one chunk)
  int last;     // nor those of the unit behind
  __device__ __forceinline__ int chunk_tokens(int c, int lg) const { return min(r.tokens - c * (kRows >> lg), kRows >> lg); }
  // Tiles whose first token the last row of chunk c sees.
  __device__ __forceinline__ int seen(int c, int lg) const {
    return min(n, (r.place0 + min((c + 1) * (kRows >> lg), r.tokens) - 1) / kTile - t + 1);
  }
};

// PROBE: the wait-timeout probe (test support only): the second record of every widening warp is never copied, and the
// waits give up after kProbeTimeoutNs. Compiled out of the kernel itself.
template <int D, bool PROBE = false>
__global__ void __launch_bounds__(kThreads, 1)
    kv4_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const WeightsParams p) {
  constexpr uint64_t kLimit = PROBE ? kProbeTimeoutNs : kTimeoutNs;
  constexpr uint32_t kLimitUs = (uint32_t)(kLimit / 1024);
  constexpr int NG = Kv4<D>::kGroups;
  constexpr uint32_t kKBytes = kTile * D * 2, kBox = kTile * 128, kRaw = 10 * D;  // K's codes and all scales of a record
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ Unit units[kUnits];
  __shared__ alignas(16) float s_lse[kLseStages][kRows];  // -lse in log2 units, -inf where there is no row
  __shared__ float s_eq[kLseStages];                     // the rows' exponent
  __shared__ int8_t s_ek[kHeldUnits][kTiles][kTile];  // the tokens' exponents, by unit (the next ones' keys may come while
                                                      // the last scores are worked on)
  __shared__ float s_part[2][kGroups - 1][kTiles][kTile];    // sums for the group that writes a tile, from those after it
  __shared__ uint32_t s_top[2][kWidenWarps];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_seq[2], s_tile[2], s_index[2];
  __shared__ int64_t w_cost[kThreads / 32];
  __shared__ int w_tiles[kThreads / 32];

  pdl_launch_dependents();
  const Kv4Batch& b = p.b;
  const uint32_t sK = (smem_u32(smem_raw) + 1023u) & ~1023u, sQ = sK + kTiles * kKBytes, sRaw = sQ + kQStages * kRows * D * 2;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 32 * kWarpMma) {
#pragma unroll 1
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_u32(&bars.unit[i]), 1);
      mbar_init(smem_u32(&bars.unit_free[i]), kUnitReaders);
    }
#pragma unroll 1
    for (int i = 0; i < kWidenWarps * kRecords; ++i) mbar_init(smem_u32(&bars.raw[0][0] + i), 1);
#pragma unroll 1
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(smem_u32(&bars.k_full[i]), kWidenWarps);
      mbar_init(smem_u32(&bars.k_free[i]), 1);
      mbar_init(smem_u32(&bars.s_full[i]), 1);
      mbar_init(smem_u32(&bars.s_free[i]), 4);
    }
#pragma unroll 1
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(smem_u32(&bars.q_raw[i]), 1);
      mbar_init(smem_u32(&bars.q_full[i]), kWidenWarps);
      mbar_init(smem_u32(&bars.q_free[i]), 1);
    }
#pragma unroll 1
    for (int i = 0; i < kLseStages; ++i) {
      mbar_init(smem_u32(&bars.lse_full[i]), kWidenWarps);
      mbar_init(smem_u32(&bars.lse_free[i]), kExpWarps);
    }
    mbar_init(smem_u32(&bars.top), kWidenWarps);
#pragma unroll 1
    for (int i = 0; i < kGroups; ++i) mbar_init(smem_u32(&bars.part[i]), 4);
    mbar_init(smem_u32(&bars.drain), 1);
    s_abort = 0;
    s_index[0] = s_index[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  // Costs of all tiles, and where this CTA's run begins and ends: its tiles are those whose cost begins inside its share.
  const int run_s = (b.n_seqs + kThreads - 1) / kThreads;
  const int q0 = min(tid * run_s, b.n_seqs), q1 = min(q0 + run_s, b.n_seqs);
  int64_t mine = 0;
  int mine_tiles = 0;
#pragma unroll 1
  for (int s = q0; s < q1; ++s) {
    const Share x = share_of(p, s);
    mine += cost_before(x, x.tiles, p.lg) * b.hkv;
    mine_tiles += x.tiles * b.hkv;
  }
  int64_t up = mine;
  int up_tiles = mine_tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, up, d);
    const int z = __shfl_up_sync(0xffffffffu, up_tiles, d);
    if (lane >= d) up += y, up_tiles += z;
  }
  if (lane == 31) w_cost[warp] = up, w_tiles[warp] = up_tiles;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t total = 0, before = up - mine;
  int tiles_before = up_tiles - mine_tiles, all_tiles = 0;
#pragma unroll 1
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += w_cost[i], tiles_before += w_tiles[i];
    total += w_cost[i];
    all_tiles += w_tiles[i];
  }
  // A tile costs one and one for each product, of which the host bounds the number: no more than twice its limit, unless offsets
  // that rise again behind a fall give the same rows to several requests. Nothing is computed then.
  if (total > 2 * kKv4MostTiles) total = 0;
  const int64_t quota = (total + gridDim.x - 1) / gridDim.x;
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const int64_t at = (blockIdx.x + e) * quota;
    if (at >= total) {
      if (tid == 0) s_index[e] = all_tiles;
    } else if (before <= at && at < before + mine) {
      int64_t c0 = before;
      int i0 = tiles_before;
#pragma unroll 1
      for (int s = q0; s < q1; ++s) {
        const Share x = share_of(p, s);
        const int64_t head = cost_before(x, x.tiles, p.lg);
        if (at < c0 + head * b.hkv) {
          const int g = (int)((at - c0) / head);
          int low = 0, high = x.tiles;  // the first tile that begins there or later; may be none of the head's
          while (low < high) {
            const int half = (low + high) / 2;
            if (cost_before(x, half, p.lg) < at - c0 - g * head)
              low = half + 1;
            else
              high = half;
          }
          s_seq[e] = s;
          s_tile[e] = g * x.tiles + low;
          s_index[e] = i0 + s_tile[e];
          break;
        }
        c0 += head * b.hkv;
        i0 += x.tiles * b.hkv;
      }
    }
  }
  __syncthreads();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  const int count = s_index[1] - s_index[0];  // this CTA's tiles
  auto wait = [&](uint64_t& bar, uint32_t parity, int site) -> bool {
    return wait_warp(smem_u32(&bar), parity, abort_flag, site, kLimitUs);
  };
  // Tiles of the un-th unit of this CTA, which lies in units[un % kUnits]; 0 at the end (or after a failure).
  auto unit_at = [&](int un) -> int { return wait(bars.unit[un % kUnits], (un / kUnits) & 1, 138) ? units[un % kUnits].n : 0; };
  auto leave_unit = [&](int un) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.unit_free[un % kUnits]));
  };

  if (warp < kExpWarps) {
    const int grp = warp / 4, row = tid % kTile;
    const uint32_t lane_base = tmem + ((uint32_t)((warp % 4) * 32) << 16);
    const float scale_log2 = b.scale * 1.4426950408889634f;
    int qn = 0;       // rows' chunks before this one
    uint32_t sn = 0;  // products before this one, which the groups take in turn
    int turn = grp;   // this group's next one, from sn on
    bool ok = true;
#pragma unroll 1
    for (int un = 0, n; ok && (n = unit_at(un)) > 0; ++un) {
      const Unit& w = units[un % kUnits];
      // This thread writes the weights of tokens j0 and (the first group) j0 + kGroups kTile.
      const int chunks = w.r.chunks, j0 = (w.t + grp) * kTile + row;
      const bool more = grp + kGroups < n;
      const int64_t base = ((int64_t)w.s * b.hkv + w.g) * b.width * b.page_size;
      float sum[kTiles] = {}, old0 = 0.0f, old1 = 0.0f;
      if (p.earlier != nullptr) {
        if (grp < n && j0 < w.r.old) old0 = p.earlier[base + j0];
        if (more && j0 + kGroups * kTile < w.r.old) old1 = p.earlier[base + j0 + kGroups * kTile];
      }
      qn -= !w.fresh;
#pragma unroll 1
      for (int c = w.first; c < chunks && ok; ++c, ++qn) {
        const int st = qn % kLseStages, cols = w.chunk_tokens(c, p.lg) << p.lg;
        ok = wait(bars.lse_full[st], (qn / kLseStages) & 1, 130);
        if (!ok) break;
        const float eq = s_eq[st];
        const int first = w.r.place0 + c * (kRows >> p.lg);  // place of the chunk's first row
        const int seen = w.seen(c, p.lg);
#pragma unroll 1
        for (int q = turn; q < seen && ok; q += kGroups) {
          const int buf = (sn + q) % kTiles;
          ok = wait(bars.s_full[buf], (sn + q) / kTiles & 1, 131);
          tc_fence_after();
          const int ek = s_ek[un % kHeldUnits][q][row];
          // the lane's factor (not 0, which times -infinity is NaN)
          const float e = (float)ek + eq, eh = floorf(0.5f * e);
          const float a = fmaxf(scale_log2 * ex2(eh) * ex2(e - eh), 1.2e-38f);
          // columns below are rows before the token
          const int hidden = min(max((w.t + q) * kTile + row - first, 0), kRows) << p.lg;
          const int most_hidden = __reduce_max_sync(0xffffffffu, hidden);
          const uint64_t a2 = f2_pack(a, a);
          const uint64_t zero = f2_pack(0.0f, 0.0f);
          uint64_t ac[4] = {zero, zero, zero, zero};
          const float* lse = s_lse[st];
          // 16 columns at a time, the next ones on their way (behind the last: some that are not used)
          uint32_t x[16], y[16];
          const uint32_t taddr = lane_base + (uint32_t)(buf * kRows);
          auto add = [&](uint32_t (&z)[16], int c0) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 m = *reinterpret_cast<const float4*>(lse + c0 + k);
              f2_unpack(f2_fma(f2_pack(__uint_as_float(z[k]), __uint_as_float(z[k + 1])), a2, f2_pack(m.x, m.y)), v[k], v[k + 1]);
              f2_unpack(f2_fma(f2_pack(__uint_as_float(z[k + 2]), __uint_as_float(z[k + 3])), a2, f2_pack(m.z, m.w)), v[k + 2],
                        v[k + 3]);
            }
            if (c0 < most_hidden) {  // (the result: its lse may be no number)
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (c0 + k < hidden) v[k] = -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < 16; k += 2) ac[k / 2 % 4] = f2_add(ac[k / 2 % 4], f2_pack(ex2(v[k]), ex2(v[k + 1])));
          };
          tmem_ld_x16_async(taddr, x);
#pragma unroll 1
          for (int c0 = 0; c0 < cols; c0 += 32) {
            tmem_wait_ld16(x);
            tmem_ld_x16_async(taddr + c0 + 16, y);
            add(x, c0);
            tmem_wait_ld16(y);
            tmem_ld_x16_async(taddr + (c0 + 32) % kRows, x);
            if (c0 + 16 < cols) add(y, c0 + 16);
          }
          tmem_wait_ld16(x);
          float s0, s1;
          f2_unpack(f2_add(f2_add(ac[0], ac[1]), f2_add(ac[2], ac[3])), s0, s1);
          s0 = ek == kBadRecord ? 0.0f : s0 + s1;
#pragma unroll
          for (int k = 0; k < kTiles; ++k) sum[k] += k == q ? s0 : 0.0f;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.s_free[buf]));
        }
        sn += seen;
        turn = (turn + 4 * kGroups - seen) % kGroups;
        __syncwarp();
        if (lane == 0 && (chunks > 1 || w.last)) mbar_arrive(smem_u32(&bars.lse_free[st]));
      }
      // Each group writes its share of the tiles: the others' sums of them come through shared memory.
      float(*part)[kTiles][kTile] = s_part[un & 1];
#pragma unroll
      for (int k = 0; k < kTiles; ++k) {
        const int from = (grp + kGroups - k % kGroups) % kGroups;  // 0: this group's own tile
        if (from > 0) part[from - 1][k][row] = sum[k];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.part[grp]));
#pragma unroll 1
      for (int i = 0; i < kGroups; ++i) ok = ok && (i == grp || wait(bars.part[i], un & 1, 143));
      if (ok) {
        float mine = 0.0f, last = sum[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) mine += k == grp ? sum[k] : 0.0f;
#pragma unroll
        for (int i = 0; i < kGroups - 1; ++i) {
          mine += part[i][grp][row];
          last += part[i][kGroups][row];
        }
        if (grp < n && j0 < w.r.len) p.weights[base + j0] = old0 + mine;
        if (more && j0 + kGroups * kTile < w.r.len) p.weights[base + j0 + kGroups * kTile] = old1 + last;
      }
      leave_unit(un);
    }
  } else if (warp < kWarpMma) {
    // A record of each tile, whose codes and scales come by bulk copies, kRecords tiles ahead, into a ring of the warp's
    // own. Lane l holds the page of tile l of a window of 32. And 16 rows of each chunk, in fp16 after a power of two that puts the
    // largest of all 128 into [2^14, 2^15), in place: a row by D / 8 lanes.
    const int mine_rec = warp - kWarpWiden, per_page = b.page_size / kKv4Block;
    const int c = lane & 3, t0 = (lane >> 3) + 4 * (lane >> 2 & 1);  // token of a half record; see widen_keys in kv4_tile.cuh
    const uint32_t ring = sRaw + mine_rec * kRecords * kRaw;
    bool ok = true;
    // the walk of what is asked for: unit, its tiles, next tile of it
    int un = 0, n = unit_at(0), tile = 0, asked = 0;
    int win_s = -1, win0 = 0;
    uint32_t win = kNoRecord;  // the record of kv head 0, or why there is none
    uint32_t meta = 0;       // 9 bits per slot of the ring: stage of K, valid tokens << 2, its page is none << 7
    auto request = [&](int slot) {
      uint32_t it = 0;
      const uint32_t bar = smem_u32(&bars.raw[mine_rec][slot]);
      bool copy = false;
      if (n > 0) {
        const Unit& w = units[un % kUnits];
        const int t = w.t + tile;
        if (win_s != w.s || t >= win0 + 32 || t < win0) {
          win_s = w.s;
          win0 = t;
          const int rec = (t + lane) * (kTile / kKv4Block) + mine_rec, at = rec / per_page;
          win = kNoRecord;
          if (rec * kKv4Block < w.r.len) {
            const int32_t page = __ldg(b.table + (int64_t)w.s * b.width + at);
            if (page >= 0 && page < b.n_pages) win = (uint32_t)page * b.hkv * per_page + rec - at * per_page;
          }
        }
        const uint32_t id = __shfl_sync(0xffffffffu, win, t - win0);
        const int left = w.r.len - (t * (kTile / kKv4Block) + mine_rec) * kKv4Block;
        copy = left > 0 && id != kNoRecord;
        it = tile | (copy ? min(left, kKv4Block) : 0) << 2;
        if (copy) {
          if (lane == 0) {
            const uint8_t* src = b.cache + (uint64_t)(id + (uint32_t)w.g * per_page) * Kv4<D>::kRecord;
            const uint32_t dst = ring + slot * kRaw;
            mbar_expect_tx(bar, kRaw);
            if (!(PROBE && asked == 1)) {
              copy_bulk(dst, src, 8 * D, bar);
              copy_bulk(dst + 8 * D, src + Kv4<D>::kScales, 2 * D, bar);
            }
          }
        } else if (left > 0) {
          if (lane == 0) record_error(b.err, kErrIndex, w.s);
          it |= 128;
        }
        if (++tile == n) {
          tile = 0;
          n = unit_at(++un);
        }
        ++asked;
      }
      if (lane == 0 && !copy) mbar_arrive(bar);  // the phase passes without a copy
      meta = (meta & ~(511u << (9 * slot))) | it << (9 * slot);
      __syncwarp();
    };
#pragma unroll 1
    for (int i = 0; i < kRecords; ++i) request(i);
    int slot = 0, phase = 0;
    uint32_t uses = 0, used = 0;  // bit q: parity of the uses of stage q so far; whether there was one
    auto widen = [&](int un) {
      const uint32_t it = meta >> (9 * slot);
      const int stage = it & 3, valid = it >> 2 & 31;
      ok = wait(bars.raw[mine_rec][slot], phase, 139) &&
           (!(used >> stage & 1) || wait(bars.k_free[stage], (uses >> stage & 1) ^ 1, 132));
      if (!ok) return;
      // the tokens' exponents
      const uint32_t raw = ring + slot * kRaw;
      uint32_t top = 0, sc[NG / 2];
      lds<NG / 2>(sc, raw + 8 * D + lane % kKv4Block * (4 * NG));
#pragma unroll
      for (int i = 0; i < NG / 2; ++i) {
        sc[i] = lane % kKv4Block < valid ? sc[i] : 0u;
        const uint32_t lo = sc[i] & 0x7fffu, hi = sc[i] >> 16 & 0x7fffu;
        top = max(top, max(lo >= 0x7f80u ? 0u : lo, hi >= 0x7f80u ? 0u : hi));
      }
      const int e_k = exponent_of(top);
      const float fk = power_of_2(-e_k);
#pragma unroll
      for (int i = 0; i < NG / 2; ++i)
        sc[i] = h2_bits(__floats2half2_rn(__uint_as_float(sc[i] << 16) * fk, __uint_as_float(sc[i] & 0xffff0000u) * fk));
      if (lane < kKv4Block) s_ek[un % kHeldUnits][stage][mine_rec * kKv4Block + lane] = (int8_t)(it & 128 ? kBadRecord : e_k);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int key = mine_rec * kKv4Block + 8 * half + t0;
        uint32_t s[NG / 2], w[NG];
        lds<NG>(w, raw + ((8 * half + t0) * 4 + c) * (4 * NG));
#pragma unroll
        for (int i = 0; i < NG / 2; ++i) s[i] = __shfl_sync(0xffffffffu, sc[i], 8 * half + t0);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint32_t y[4];
          widen_word(w[g], g % 2 ? __high2half2(h2_of(s[g / 2])) : __low2half2(h2_of(s[g / 2])), y);
          sts4(sK + stage * kKBytes + (g / 2) * kBox + key * 128 + (uint32_t)(((4 * (g % 2) + c) ^ (key & 7)) * 16), y[0], y[1], y[2],
               y[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read it
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.k_full[stage]));
      uses ^= 1u << stage;
      used |= 1u << stage;
      request(slot);
      if (++slot == kRecords) slot = 0, phase ^= 1;
    };
    constexpr int kPer = 256 / D, kLoads = 16 / kPer;  // rows per access; accesses
    const int row0 = mine_rec * 16 + lane / (D / 8), piece = lane % (D / 8), group = 1 << p.lg;
    const int my_row = mine_rec * 16 + lane % 16;      // whose lse this lane loads
    float lse = 0.0f;
    auto load_lse = [&](const Unit& w, int c) {
      const int64_t first = (int64_t)(w.r.rows0 + c * (kRows >> p.lg)) * b.hq + (w.g << p.lg);
      const bool is = my_row < w.chunk_tokens(c, p.lg) << p.lg;
      lse = is ? __ldg(p.lse + first + (int64_t)(my_row >> p.lg) * b.hq + (my_row & (group - 1))) : -INFINITY;
    };
    int qn = 0;  // chunks before this one
    bool loaded = false;
#pragma unroll 1
    for (int cur = 0, m; ok && (m = unit_at(cur)) > 0; ++cur) {
      const Unit& w = units[cur % kUnits];
      const int first = w.first, chunks = w.fresh ? w.r.chunks : 0;
#pragma unroll 1
      for (int c = first; (c < chunks || c == first) && ok; ++c) {
        if (c < chunks) {
          const int st = qn % kQStages, cols = w.chunk_tokens(c, p.lg) << p.lg;
          if (!loaded) load_lse(w, c);
          ok = wait(bars.q_raw[st], (qn / kQStages) & 1, 144);
          if (!ok) break;
          const uint32_t at = sQ + st * (kRows * D * 2) + (piece / 8) * kBox;
          // rows of others, or behind the last, and rows that add nothing, whatever their q is
          const uint32_t none = __ballot_sync(0xffffffffu, lse == -INFINITY);
          uint32_t v[kLoads][4], top = 0;
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int r = row0 + i * kPer;
            lds<4>(v[i], at + r * 128 + (uint32_t)(((piece % 8) ^ (r & 7)) * 16));
            if (none >> (r % 16) & 1) v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0;
            const uint32_t x = __vmaxu2(__vmaxu2(v[i][0] & 0x7fff7fffu, v[i][1] & 0x7fff7fffu),
                                        __vmaxu2(v[i][2] & 0x7fff7fffu, v[i][3] & 0x7fff7fffu));
            const uint32_t y = max(x & 0xffffu, x >> 16);
            top = max(top, y >= 0x7f80u ? 0u : y);  // what is no number takes no part
          }
          top = __reduce_max_sync(0xffffffffu, top);
          if (lane == 0) {
            s_top[qn & 1][mine_rec] = top;
            mbar_arrive(smem_u32(&bars.top));
          }
          ok = wait(bars.top, qn & 1, 142);
          if (!ok) break;
          top = __reduce_max_sync(0xffffffffu, s_top[qn & 1][lane % kWidenWarps]);
          const int by = min(141 - max((int)(top >> 7), 1), 127);  // -114 .. 127 (below 2^-112 the rows stay smaller)
          const uint64_t f2 = f2_pack(power_of_2(by), power_of_2(by));
          if (mine_rec * 16 < cols)  // (a product reads 16 rows or a multiple)
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
              const int r = row0 + i * kPer;
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float lo, hi;
                f2_unpack(f2_mul(f2_pack(__uint_as_float(v[i][e] << 16), __uint_as_float(v[i][e] & 0xffff0000u)), f2), lo, hi);
                h[e] = h2_bits(__floats2half2_rn(lo, hi));
              }
              sts4(at + r * 128 + (uint32_t)(((piece % 8) ^ (r & 7)) * 16), h[0], h[1], h[2], h[3]);
            }
          const int ls = qn % kLseStages;
          ok = qn < kLseStages || wait(bars.lse_free[ls], (qn / kLseStages - 1) & 1, 146);
          if (!ok) break;
          if (lane < 16) s_lse[ls][my_row] = lse == -INFINITY ? lse : lse * -1.4426950408889634f;
          if (mine_rec == 0 && lane == 0) s_eq[ls] = (float)-by;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&bars.lse_full[ls]));
            mbar_arrive(smem_u32(&bars.q_full[st]));
          }
          ++qn;
          loaded = c + 1 < chunks;
          if (loaded) load_lse(w, c + 1);
        }
        if (c == first)
#pragma unroll 1
          for (int q = 0; q < m && ok; ++q) widen(cur);
      }
      leave_unit(cur);
    }
    // Before the CTA can exit, every copy issued must have landed (also after a failure).
    if (lane == 0)
#pragma unroll 1
      for (int i = 0; i < kRecords; ++i) {
        mbar_wait(smem_u32(&bars.raw[mine_rec][slot]), phase, abort_flag, b.err, 140, false, kLimit);
        if (++slot == kRecords) slot = 0, phase ^= 1;
      }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // S^T of tile q and chunk c, keys by rows; elected lane only.
    int qn = 0;
    uint32_t uses = 0;                // bit q: parity of the uses of stage q before this unit
    uint32_t sn = 0;                  // products before this one, which have the stages of S in turn
    bool ok = true;
#pragma unroll 1
    for (int un = 0, n; ok && (n = unit_at(un)) > 0; ++un) {
      const Unit& w = units[un % kUnits];
      const int chunks = w.r.chunks;
      int ready = 0;  // tiles of keys waited for
      qn -= !w.fresh;
#pragma unroll 1
      for (int c = w.first; c < chunks && ok; ++c, ++qn) {
        const int st = qn % kQStages, cols = w.chunk_tokens(c, p.lg) << p.lg;
        const uint32_t idesc = idesc_f16(kTile, 16) - (2u << 17) + ((uint32_t)((cols + 15) / 16 * 16 >> 3) << 17);
        ok = wait(bars.q_full[st], (qn / kQStages) & 1, 134);
        const int seen = w.seen(c, p.lg);
        const bool last = c + 1 == chunks;
#pragma unroll 1
        for (int q = 0; q < seen && ok; ++q, ++sn) {
          if (q >= ready) {  // (the last rows see every tile)
            ok = wait(bars.k_full[q], uses >> q & 1, 135);
            ++ready;
          }
          const int buf = sn % kTiles;
          ok = ok && (sn < kTiles || wait(bars.s_free[buf], (sn / kTiles & 1) ^ 1, 136));  // the scores before were taken
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t dk = desc_lo(sK + q * kKBytes), dq = desc_lo(sQ + st * (kRows * D * 2));
            const uint32_t d = tmem + (uint32_t)(buf * kRows);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t at = ((ks / 4) * kBox + ks % 4 * 32) >> 4;
              mma_ss_lo(d, dk + at, dq + at, idesc, ks > 0 ? 1u : 0u);
            }
            tc_commit(smem_u32(&bars.s_full[buf]));
            if (last) tc_commit(smem_u32(&bars.k_free[q]));
          }
          __syncwarp();
        }
        if (ok && (chunks > 1 || w.last)) {
          if (elect_one()) tc_commit(smem_u32(&bars.q_free[st]));
          __syncwarp();
        }
      }
      uses ^= (1u << n) - 1;
      leave_unit(un);
    }
    // All tensor-core work issued by this CTA completes before TMEM is freed.
    if (elect_one()) tc_commit(smem_u32(&bars.drain));
    __syncwarp();
    mbar_wait(smem_u32(&bars.drain), 0, abort_flag, b.err, 137, false, kLimit);
  } else if (warp == kWarpRows) {
    int qn = 0;
    bool ok = true;
#pragma unroll 1
    for (int un = 0, n; ok && (n = unit_at(un)) > 0; ++un) {
      const Unit& w = units[un % kUnits];
      const int chunks = w.fresh ? w.r.chunks : 0;
#pragma unroll 1
      for (int c = w.first; c < chunks && ok; ++c) {
        const int st = qn % kQStages;
        ok = qn < kQStages || wait(bars.q_free[st], (qn / kQStages - 1) & 1, 133);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&bars.q_raw[st]);
          mbar_expect_tx(bar, kRows * D * 2);
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
            tma_load_3d(sQ + st * (kRows * D * 2) + k * kBox, &tm_q, bar, 64 * k, w.g << p.lg, w.r.rows0 + c * (kRows >> p.lg));
        }
        ++qn;
        __syncwarp();
      }
      leave_unit(un);
    }
    // Before the CTA can exit, every copy issued must have landed (also after a failure).
    if (lane == 0)
#pragma unroll 1
      for (int k = max(qn - kQStages, 0); k < qn; ++k)
        mbar_wait(smem_u32(&bars.q_raw[k % kQStages]), (k / kQStages) & 1, abort_flag, b.err, 145, false, kLimit);
    __syncwarp();
  } else {  // kWarpUnits
    // The CTA's units, one after the other.
    int left = max(count, 0), s = 0, at = 0;
    if (left > 0) {
      s = s_seq[0];
      at = s_tile[0];
    }
    bool fresh = true, ok = true;
    int un = 0;
#pragma unroll 1
    for (; left > 0 && ok; ++un) {
      Unit w;
      w.r = share_of(p, s);
      if (at >= w.r.tiles * b.hkv) {  // (also a request without rows)
        at -= w.r.tiles * b.hkv;
        ++s;
        --un;
        continue;
      }
      w.s = s;
      w.g = at / w.r.tiles;
      w.t = at - w.g * w.r.tiles;
      w.n = min(min(kTiles, w.r.tiles - w.t), left);
      w.first = first_chunk(w.r, w.t, p.lg);
      left -= w.n;
      at += w.n;
      w.fresh = fresh || w.r.chunks > 1;
      w.last = w.r.chunks > 1 || left == 0 || w.t + w.n == w.r.tiles;
      fresh = w.last;
      ok = un < kUnits || wait(bars.unit_free[un % kUnits], (un / kUnits - 1) & 1, 141);
      if (ok && lane == 0) {
        units[un % kUnits] = w;
        mbar_arrive(smem_u32(&bars.unit[un % kUnits]));
      }
      __syncwarp();
    }
    ok = ok && (un < kUnits || wait(bars.unit_free[un % kUnits], (un / kUnits - 1) & 1, 141));
    if (ok && lane == 0) {  // (else the abort flag ends every warp's list)
      units[un % kUnits].n = 0;
      mbar_arrive(smem_u32(&bars.unit[un % kUnits]));
    }
    __syncwarp();
    for (int i = blockIdx.x * 32 + lane; i < b.n_seqs; i += gridDim.x * 32) kv4_check_request(b, i);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    if (lane == 0 && s_abort != 0) record_error(b.err, kErrTimeout, s_abort);
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

template <int D, bool PROBE = false>
cudaError_t launch_t(const Kv4Batch& b, const float* lse, int32_t window, const float* earlier, float* weights, int32_t sms,
                     cudaStream_t s) {
  const WeightsParams p{b, lse, earlier, weights, window, 31 - __builtin_clz(b.hq / b.hkv), PROBE ? 0 : kv4_weights_few(b, window)};
  CUtensorMap rows;
  const int tokens = kRows >> p.lg;  // of a chunk
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)b.hq, (cuuint64_t)b.n_rows};
  const cuuint64_t strides[2] = {D * 2, (cuuint64_t)b.hq * D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(b.hq / b.hkv), (cuuint32_t)tokens};
  if (!encode_map(&rows, b.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)(kTiles * kTile + kQStages * kRows) * D * 2 + kWidenWarps * kRecords * 10 * D;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = set_smem_limit_once(kv4_weights_kernel<D, PROBE>, (int)smem, configured);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)b.n_seqs * b.hkv * (((int64_t)b.width * b.page_size + kTile - 1) / kTile);
  const int grid = (int)std::min<int64_t>(std::max<int64_t>(most, 1), sms);
  return launch_pdl(kv4_weights_kernel<D, PROBE>, dim3((unsigned)grid), dim3(kThreads), smem, s, rows, p);
}

}  // namespace

cudaError_t launch_kv4_weights(const Kv4Batch& b, int32_t head_dim, const float* lse, int32_t window,
                               const float* earlier, float* weights, int32_t sms, cudaStream_t s) {
  if (const int32_t few = kv4_weights_few(b, window); few > 0) {
    const cudaError_t e = launch_kv4_weights_few(b, head_dim, lse, window, earlier, weights, sms, s);
    // no request can have more rows
    if (e != cudaSuccess || b.n_rows <= few || (window > 0 && window <= few)) return e;
  }
  if (head_dim == 128) return launch_t<128>(b, lse, window, earlier, weights, sms, s);
  if (head_dim == 64) return launch_t<64>(b, lse, window, earlier, weights, sms, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_weights_timeout_probe(const Kv4Batch& b, const float* lse, float* weights, int32_t sms, cudaStream_t s) {
  return launch_t<128, true>(b, lse, 0, nullptr, weights, sms, s);
}

}  // namespace cb
