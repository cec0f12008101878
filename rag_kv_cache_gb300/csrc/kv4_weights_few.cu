// Accumulated attention weights (see kv4_weights.cu) where requests bring a few rows each (a decode step, guessed tokens):
//
//   weights[s, g, j] = earlier[s, g, j] + sum_{t, h in g} exp(scale q[t, h] . k_j[g] - lse[t, h])
//
// Every warp takes a contiguous run of the batch's records (16 tokens of one request and kv head, in that order), whose K codes
// and scales come by bulk copies into a ring of its own, and forms their scores with up to 8 NT rows on mma.sync
// (kv4_scores.cuh): about 150 instructions a record, against 500 for widened operands of tcgen05.mma in shared
// memory, which this many rows do not repay. A token's weight is a sum over the four lanes that hold its scores, in a fixed
// order; nothing passes between warps. Requests of more rows are left to kv4_weights.cu.
//
// Measured: a step of 64 requests of up to 8,449 tokens, 8 query heads on each of 8 kv heads of 128 dims, added to earlier
// weights, 68 us (171 MB, 25 us at the copy rate; 160 on the other kernel); bound by its warps' own latencies as the decode kernel
// is (kv4_decode.cu), whose keys' half this is: issue slots 45%, integer pipe 48%.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "kv4_batch.cuh"
#include "kv4_scores.cuh"
#include "kv4_tile.cuh"

namespace cb {
namespace {

struct FewParams {
  Kv4Batch b;
  const float* lse;
  const float* earlier;
  float* weights;
  int window;
  int lg;    // log2 of the query heads per kv head
  int most;  // row tokens of a request that this kernel takes
  uint32_t nibbles, higher;
};

// Four n-tiles take twice the registers of one.
template <int NT>
constexpr int kWarpsOf = NT == 4 ? 12 : 16;
constexpr int kStages = 6;  // records on their way to a warp, or held for it

template <int D, int NT>
__global__ void __launch_bounds__(kWarpsOf<NT> * 32, 1) kv4_weights_few_kernel(const FewParams p) {
  constexpr int NG = Kv4<D>::kGroups, kWarps = kWarpsOf<NT>, kRaw = 10 * D;  // K's codes and all scales of a record
  constexpr uint32_t kLimitUs = (uint32_t)(kTimeoutNs / 1024);
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ int s_abort[kWarps];
  pdl_launch_dependents();
  // What a warp uses is its own.
  const Kv4Batch& b = p.b;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
  if (lane < kStages) mbar_init(smem_u32(&full[warp][lane]), 1);
  if (lane == 0) s_abort[warp] = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  pdl_wait();
  auto tokens_of = [&](const Kv4Request& x) -> int { return p.window > 0 ? min(p.window, x.m) : x.m; };
  auto records_of = [&](int s) -> int {
    const Kv4Request x = kv4_request(b, s);
    return x.m > 0 && x.len > 0 && tokens_of(x) <= p.most ? (x.len - 1) / kKv4Block + 1 : 0;
  };
  // The batch's records, and where this warp's run of them begins (31 bits hold them: the host checks).
  const int warps = gridDim.x * kWarps, me = blockIdx.x * kWarps + warp;
  int total = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < b.n_seqs; s0 += 32)
    total += __reduce_add_sync(0xffffffffu, s0 + lane < b.n_seqs ? records_of(s0 + lane) * b.hkv : 0);
  const int quota = (total + warps - 1) / warps;
  const int a0 = (int)min((int64_t)me * quota, (int64_t)total), a1 = (int)min((int64_t)a0 + quota, (int64_t)total);
  for (int s = me * 32 + lane; s < b.n_seqs; s += warps * 32) kv4_check_request(b, s);
  if (a0 >= a1) return;
  int s = 0, first = 0;  // the request that record a0 lies in, that request's first record
  {
    int before = 0;
#pragma unroll 1
    for (int s0 = 0;; s0 += 32) {
      const int n = s0 + lane < b.n_seqs ? records_of(s0 + lane) * b.hkv : 0;
      int up = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += y;
      }
      const uint32_t here = __ballot_sync(0xffffffffu, a0 >= before + up - n && a0 < before + up);
      if (here != 0) {
        const int at = __ffs(here) - 1;
        s = s0 + at;
        first = before + __shfl_sync(0xffffffffu, up - n, at);
        break;
      }
      before += __shfl_sync(0xffffffffu, up, 31);
    }
  }
  struct Place {
    int s, h, i, n;  // request, kv head, record of it, its records
  };
  auto next = [&](Place& x) {
    if (++x.i < x.n) return;
    x.i = 0;
    if (++x.h < b.hkv) return;
    x.h = 0;
    do {
      ++x.s;
      x.n = x.s < b.n_seqs ? records_of(x.s) : 1;
    } while (x.n == 0);
  };
  Place at;
  at.s = s;
  at.n = records_of(s);
  at.h = (a0 - first) / at.n;
  at.i = a0 - first - at.h * at.n;
  // The warp's own producer: lane l holds the place of record win0 + l of request win_s (of kv head 0).
  const int per_page = b.page_size / kKv4Block;
  const uint32_t ring = smem_u32(smem) + warp * (kStages * kRaw), bar0 = smem_u32(&full[warp][0]);
  Place to = at;
  int left = a1 - a0, win_s = -1, win0 = 0;
  uint32_t win = kNoRecord, bad = 0;  // bit k: the page of stage k's record is none
  auto request = [&](int stage) {
    if (left == 0) return;
    --left;
    if (to.s != win_s || to.i < win0 || to.i >= win0 + 32) {
      win_s = to.s;
      win0 = to.i;
      win = kNoRecord;
      const int i = to.i + lane, nth = i / per_page;
      if (i < to.n) {
        const int32_t page = __ldg(b.table + (int64_t)to.s * b.width + nth);
        if (page >= 0 && page < b.n_pages) win = (uint32_t)page * b.hkv * per_page + i - nth * per_page;
      }
    }
    const uint32_t id = __shfl_sync(0xffffffffu, win, to.i - win0);
    const uint32_t bar = bar0 + 8 * stage;
    bad = id == kNoRecord ? bad | 1u << stage : bad & ~(1u << stage);
    if (lane == 0) {
      if (id == kNoRecord) {
        record_error(b.err, kErrIndex, to.s);
        mbar_arrive(bar);  // the phase passes without a copy
      } else {
        const uint8_t* src = b.cache + (uint64_t)(id + (uint32_t)(to.h * per_page)) * Kv4<D>::kRecord;
        mbar_expect_tx(bar, kRaw);
        copy_bulk(ring + stage * kRaw, src, 8 * D, bar);
        copy_bulk(ring + stage * kRaw + 8 * D, src + Kv4<D>::kScales, 2 * D, bar);
      }
    }
    __syncwarp();
    next(to);
  };
#pragma unroll 1
  for (int k = 0; k < kStages; ++k) request(k);
  const float scale_log2 = b.scale * 1.4426950408889634f;
  int stage = 0, phase = 0, rest = a1 - a0, under_way = min(kStages, rest);
  bool ok = true;
  Query<D, NT> qf;
  float nl[NT][2];  // -lse (log2 units) of rows 8 t + 2 c and + 1, -inf where there is none
#pragma unroll 1
  while (rest > 0 && ok) {
    const Kv4Request rq = kv4_request(b, at.s);
    const int tokens = tokens_of(rq), rows = tokens << p.lg;
    const int64_t q0 = (int64_t)(rq.row0 + rq.m - tokens) * b.hq + (at.h << p.lg);
    const int place0 = rq.len - tokens, old = rq.len - rq.m, group = 1 << p.lg;
    const int64_t base = ((int64_t)at.s * b.hkv + at.h) * b.width * b.page_size;
    auto row_of = [&](int n) -> int64_t { return q0 + (int64_t)(n >> p.lg) * b.hq + (n & (group - 1)); };
    bool none = false;  // a row adds nothing, whatever its q is
    load_query<D, NT>(qf, [&](int n) { return b.q + row_of(n) * (D * 2); }, rows, scale_log2, lane);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = 8 * t + 2 * c + e;
        const float x = n < rows ? __ldg(p.lse + row_of(n)) : -INFINITY;
        nl[t][e] = x == -INFINITY ? x : x * -1.4426950408889634f;
        none = none || (n < rows && x == -INFINITY);
      }
    none = __any_sync(0xffffffffu, none);
    const int count = min(at.n - at.i, rest);
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const int key0 = (at.i + i) * kKv4Block, mine = key0 + r + 8 * (c & 1);  // this lane's token of the weights (c < 2)
      float before = 0.0f;
      if (p.earlier != nullptr && c < 2 && mine < old) before = p.earlier[base + mine];
      ok = wait_warp(bar0 + 8 * stage, phase, &s_abort[warp], 150, kLimitUs);
      if (!ok) break;
      const uint32_t rec = ring + stage * kRaw;
      float sum[2] = {0.0f, 0.0f};  // tokens r and r + 8
      if (!(bad >> stage & 1)) {
        uint32_t sc[2][NG / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) lds<NG / 2>(sc[h], rec + 8 * D + (r + 8 * h) * (4 * NG));
        float x[NT][4];
        record_scores<D, NT>(x, qf, rec, sc, p.nibbles, p.higher, lane);
        const bool some = key0 + kKv4Block - 1 > place0 || none;  // a row that does not see all keys
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[t][e] = fmaf(x[t][e], qf.scale[t][e % 2], nl[t][e % 2]);
          if (some) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (place0 + ((8 * t + 2 * c + e % 2) >> p.lg) < key0 + r + 8 * (e / 2) || nl[t][e % 2] == -INFINITY)
                x[t][e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e / 2] += ex2(x[t][e]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
          sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
        }
      }
      if (c < 2 && mine < rq.len) p.weights[base + mine] = before + (c == 0 ? sum[0] : sum[1]);
      __syncwarp();
      under_way -= left == 0;
      request(stage);  // into the stage just read
      if (++stage == kStages) stage = 0, phase ^= 1;
    }
    rest -= count;
    at.i += count - 1;
    next(at);
  }
  if (!ok) {  // what is under way lands before the CTA ends
    if (lane == 0) {
#pragma unroll 1
      for (int k = 0; k < under_way; ++k) {
        mbar_wait(bar0 + 8 * stage, phase, &s_abort[warp], b.err, 151, false);
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
      record_error(b.err, kErrTimeout, 150);
    }
    __syncwarp();
  }
}

template <int D, int NT>
cudaError_t launch_t(const FewParams& p, int32_t sms, cudaStream_t s) {
  constexpr int kWarps = kWarpsOf<NT>;
  const size_t smem = (size_t)kWarps * kStages * 10 * D;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = set_smem_limit_once(kv4_weights_few_kernel<D, NT>, (int)smem, configured);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)p.b.n_seqs * p.b.hkv * p.b.width * (p.b.page_size / kKv4Block);
  const int grid = (int)std::min<int64_t>(std::max<int64_t>((most + kWarps - 1) / kWarps, 1), sms);
  return launch_pdl(kv4_weights_few_kernel<D, NT>, dim3((unsigned)grid), dim3(kWarps * 32), smem, s, p);
}

template <int D>
cudaError_t launch_d(const FewParams& p, int tiles, int32_t sms, cudaStream_t s) {
  if (tiles == 1) return launch_t<D, 1>(p, sms, s);
  if (tiles == 2) return launch_t<D, 2>(p, sms, s);
  return launch_t<D, 4>(p, sms, s);
}

}  // namespace

// Mean rows of a request and kv head up to which this kernel takes all requests that have no more, and (request, kv head)
// pairs from which on it takes those of up to 8 rows in any batch. With its launch (and the other's where a request may have
// more rows) and without, us, 32 query on 8 kv heads of 128 dims:
//   64 requests of 8,192 keys, of 1, 2, 4, 8 tokens (4 to 32 rows) 103, 103, 140, 219 and 274 - 277;
//   8 of 8,192: 29, 28, 35, 45 and 50; 4 of 1,024: 17, 17, 17, 23 and 19;
//   one request in eight of 256 tokens, the others of one: 64 requests of 2,048 keys 104 and 152, 32 of 8,192 171 and 263,
//   16 of 512 36 and 38, 8 (64 pairs) of 8,192 66 and 85;
//   its launch for nothing (all of 64 tokens): 0 - 2.
constexpr int kFewRows = 32;
constexpr int64_t kFewPairs = 64;

// Row tokens of a request up to which this kernel takes it (0: none): with 8, 16 or 32 rows (tokens times heads per kv head), as the
// mean asks for.
int32_t kv4_weights_few(const Kv4Batch& b, int32_t window) {
  const int group = b.hq / b.hkv;
  // its records are counted in 31 bits
  if ((int64_t)b.n_seqs * b.hkv * b.width * (b.page_size / kKv4Block) >= (1 << 30)) return 0;
  const int64_t rows = std::min<int64_t>(b.n_rows, window > 0 ? (int64_t)window * b.n_seqs : b.n_rows) * group;
  const int64_t n = b.n_seqs;
  const bool few = rows <= kFewRows * n;
  if (!few && n * b.hkv < kFewPairs) return 0;
  return std::max(group, !few || rows <= 8 * n ? 8 : rows <= 16 * n ? 16 : kFewRows) / group;
}

cudaError_t launch_kv4_weights_few(const Kv4Batch& b, int32_t head_dim, const float* lse, int32_t window,
                                   const float* earlier, float* weights, int32_t sms, cudaStream_t s) {
  const int lg = 31 - __builtin_clz(b.hq / b.hkv), most = kv4_weights_few(b, window);
  const FewParams p{b, lse, earlier, weights, window, lg, most, kNibbles, kNibbles << 4};
  if (head_dim == 128) return launch_d<128>(p, (most << lg) / 8, sms, s);
  if (head_dim == 64) return launch_d<64>(p, (most << lg) / 8, sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace cb
