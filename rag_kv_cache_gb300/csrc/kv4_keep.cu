// The tokens that each kv head keeps of a request under a budget, and their rows moved into other pages.
//
// Keep: of n tokens the last r, the first f and the `want` heaviest between them (ties to the lower index). A block
// per (request, kv head), or a cluster of eight for a few long rows, holds the weights' order-preserving keys in shared memory
// (up to kHeldKeys per block; longer rows that have no cluster are read from L2 in each pass), finds the key of the want-th
// heaviest by a radix select of 11, 11 and 10 bits, and writes the indices in order: every warp takes a contiguous part of the
// row, counts what it keeps, and after one scan over the warps writes it. A cluster's blocks add their bins into the first
// one's, which picks the digit and tells the others (bins read from one another's memory: 62 us where this takes 12). Bound by
// latency: four passes over a row that is read once, eleven barriers. Measured: 64 requests of up to 8,449 tokens, 8 kv heads,
// a quarter kept, 22 us (11 MB, 1.6 us at the copy rate); one of 32,896 tokens, 15% kept, 12 us.
//
// Move: a warp per record (16 kept tokens of one kv head) of the pages written. K words and scales of a token are
// contiguous; V words hold a pair of tokens, whose halves come from two places. Bound by HBM: a kept token costs 18/16 D
// bytes written and, where few of its record's neighbours are kept, up to 2.4 times as many read (sectors of 32 bytes).
// Measured, 8 kv heads of 128 dims: a quarter of 64 requests of up to 8,449 tokens 51 us; 15% of one of 32,896 tokens 8 us.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "kv4_layout.cuh"

namespace cb {
namespace {

constexpr int kBins = 2048;

// Keys in the order of the weights: a NaN lowest, both zeros alike.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct KeepParams {
  const float* weights;
  const int32_t* lens;
  const int32_t* budgets;
  int32_t* kept;
  int32_t* kept_lens;
  int32_t* err;
  int32_t width;       // weights per (request, kv head)
  int32_t kept_width;
  int32_t hkv;
  int32_t first, recent;
};

// Inclusive sum over the block.
template <int WARPS>
__device__ __forceinline__ int block_scan(int x, int* warps) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  return x + __reduce_add_sync(0xffffffffu, lane < warp && lane < WARPS ? warps[lane] : 0);
}

// Shared memory of another block of the cluster.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* at, int rank) {
  uint32_t x;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"((uint32_t)__cvta_generic_to_shared(at)), "r"(rank));
  return x;
}
__device__ __forceinline__ int load_remote(const int* at, int rank) {
  int x;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(remote(at, rank)) : "memory");
  return x;
}
__device__ __forceinline__ void add_remote(int* at, int rank, int x) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(remote(at, rank)), "r"(x) : "memory");
}
__device__ __forceinline__ void store_remote(int* at, int rank, int x) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote(at, rank)), "r"(x) : "memory");
}

constexpr int kHeldKeys = 45056;  // 176 KB, per block
constexpr int kCluster = 8;       // blocks that share a long row
// Rows up to which they do: as many clusters as run at once, and more where a block alone cannot hold its row. A cluster against a
// block each, us: 8 rows of 16,384, 32,768 and 45,000 weights 11.5 and 14.6, 13 and 21, 15 and 26; 16 rows 21 and 15, 23 and 21
// (32,768); of 60,000 and 131,072: 8 rows 16 and 57, 20 and 115, 32 rows 43 and 57, 55 and 116, 64 rows of 45,000 65 and 27.
constexpr int kClusterRows = 8, kLongClusterRows = 32;
// Weights per row up to which a block has 512 threads, in place of 1,024: where there are more rows than SMs, so that blocks
// share one, and else. 512 against 1,024 threads, us: 512 rows of 1,024, 8,192, 16,384 and 32,768 weights 13 and 23, 25 and
// 38, 43 and 54, 105 and 83; 256 rows 10 and 13, 19 and 20, 23 and 28, 53 and 42; 128 rows of 1,024, 4,096, 8,192 and 16,384
// weights 6 and 7, 9.5 and 9, 13 and 11, 21 and 16.
constexpr int kShortRow = 16384, kShorterRow = 6144;

// HELD: every row fits shared memory. REP counters per bin, for the lanes in turn: most weights lie within a few powers of
// two, and a warp's additions to one counter follow one another.
// CL: blocks (a cluster) that share a row, each a contiguous part of it.
template <int THREADS, int REP, bool HELD, int CL>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 4 : 1) kv4_keep_kernel(const KeepParams p) {
  constexpr int kThreads = THREADS, kWarps = THREADS / 32, kPer = kBins / THREADS;
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ alignas(16) uint32_t bins[kBins * REP];
  __shared__ int warps[2][kWarps];
  __shared__ int s_part[2];  // CL > 1: above, equal in this block's part
  __shared__ int s_digit, s_above;
  __shared__ int sums[CL > 1 ? kBins : 1];  // CL > 1: the row's bins, in the cluster's first block
  pdl_launch_dependents();
  pdl_wait();
  const int pair = blockIdx.x / CL, rank = blockIdx.x % CL, s = pair / p.hkv, g = pair - s * p.hkv;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int len = __ldg(p.lens + s), given = __ldg(p.budgets + s);
  const int n = min(max(len, 0), p.width);
  const int budget = min(max(given, 0), p.kept_width);
  const int count = min(n, budget);
  if (g == 0 && rank == 0 && tid == 0) {
    p.kept_lens[s] = count;
    if (len < 0 || len > p.width || given < 0 || min(n, max(given, 0)) > p.kept_width) record_error(p.err, kErrIndex, s);
  }
  if (count == 0) return;
  int32_t* kept = p.kept + (int64_t)pair * p.kept_width;
  if (n <= budget) {
    for (int i = rank * kThreads + tid; i < n; i += CL * kThreads) kept[i] = i;
    return;
  }
  const int late = min(p.recent, budget), early = min(p.first, budget - late), want = budget - late - early;
  for (int i = rank * kThreads + tid; i < early; i += CL * kThreads) kept[i] = i;
  for (int i = rank * kThreads + tid; i < late; i += CL * kThreads) kept[budget - late + i] = n - late + i;
  if (want == 0) return;
  // keys p0 .. p0 + m - 1 of those between the first and the last are this block's
  const int all = n - late - early;  // > want
  const int share = (all + CL - 1) / CL, p0 = min(rank * share, all), m = min(p0 + share, all) - p0;
  const float* w = p.weights + (int64_t)pair * p.width + early + p0;
  // weights from w + head on by 16 bytes; their keys lie as they do
  const int head = min((int)(-(reinterpret_cast<uintptr_t>(w) >> 2) & 3), m), quads = (m - head) / 4;
  uint32_t* held = smem + ((4 - head) & 3);
  auto key_at = [&](int i) -> uint32_t { return HELD ? held[i] : order_key(__ldg(w + i)); };
  for (int i = tid; i < kBins * REP; i += kThreads) bins[i] = 0;
  if (CL > 1)
    for (int i = tid; i < kBins; i += kThreads) sums[i] = 0;
  if (CL > 1) cluster_sync();
  __syncthreads();
  // the key of the want-th heaviest
  uint32_t key = 0, known = 0;  // its bits so far, and which
  int left = want;              // its rank among the keys that agree with them
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    if (HELD && pass == 0) {
      auto take = [&](float x) -> uint32_t {
        const uint32_t k = order_key(x);
        atomicAdd(&bins[(k >> 21) * REP + lane % REP], 1u);
        return k;
      };
#pragma unroll 4
      for (int i = tid; i < quads; i += kThreads) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(w + head) + i);
        *reinterpret_cast<uint4*>(held + head + 4 * i) = make_uint4(take(x.x), take(x.y), take(x.z), take(x.w));
      }
      for (int i = tid; i < m - 4 * quads; i += kThreads) {  // before and behind them
        const int at = i < head ? i : 4 * quads + i;
        held[at] = take(__ldg(w + at));
      }
    } else {
#pragma unroll 8
      for (int i = tid; i < m; i += kThreads) {
        const uint32_t k = key_at(i);
        if ((k & known) == key) atomicAdd(&bins[((k >> shift) & mask) * REP + lane % REP], 1u);
      }
    }
    __syncthreads();
    if constexpr (CL > 1) {  // the blocks' bins to the first one's
      for (int i = tid; i < kBins; i += kThreads) {
        int x = 0;
#pragma unroll
        for (int r = 0; r < REP; ++r) x += (int)bins[i * REP + r], bins[i * REP + r] = 0;
        if (x > 0) add_remote(&sums[i], 0, x);
      }
      cluster_sync();
    }
    if (CL == 1 || rank == 0) {
      // from the top bin down, kPer bins a thread, which are 0 again for the next pass
      int in_bin[kPer], mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = kBins - 1 - kPer * tid - i;
        if constexpr (CL > 1) {
          in_bin[i] = sums[at];
          sums[at] = 0;
        } else {
          in_bin[i] = 0;
#pragma unroll
          for (int r = 0; r < REP; ++r) in_bin[i] += (int)bins[at * REP + r], bins[at * REP + r] = 0;
        }
        mine += in_bin[i];
      }
      int before = block_scan<kWarps>(mine, warps[pass & 1]) - mine;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (before < left && before + in_bin[i] >= left) {
          const int digit = kBins - 1 - kPer * tid - i;
#pragma unroll 1
          for (int r = 1; r < CL; ++r) store_remote(&s_digit, r, digit), store_remote(&s_above, r, before);
          s_digit = digit;
          s_above = before;
        }
        before += in_bin[i];
      }
    }
    if (CL > 1) cluster_sync();
    __syncthreads();
    key |= (uint32_t)s_digit << shift;
    known |= mask << shift;
    left -= s_above;
  }
  // In order: keys above, and the first `left` equal ones; a warp takes keys i0 .. i1 - 1.
  const int part = (m + kThreads - 1) / kThreads * 32, i0 = min(warp * part, m), i1 = min(i0 + part, m);
  int above = 0, same = 0;  // of the warp
#pragma unroll 4
  for (int i = i0 + lane; i < i0 + part; i += 32) {
    const uint32_t k = i < i1 ? key_at(i) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i < i1 && k > key));
    same += __popc(__ballot_sync(0xffffffffu, i < i1 && k == key));
  }
  __syncthreads();  // (the digits have been read)
  if (lane == 0) warps[0][warp] = above, warps[1][warp] = same;
  __syncthreads();
  int a0 = lane < warp && lane < kWarps ? warps[0][lane] : 0, e0 = lane < warp && lane < kWarps ? warps[1][lane] : 0;
  a0 = __reduce_add_sync(0xffffffffu, a0);  // above, equal before this warp's part
  e0 = __reduce_add_sync(0xffffffffu, e0);
  if constexpr (CL > 1) {  // and in the blocks before
    if (tid == kThreads - 1) s_part[0] = a0 + above, s_part[1] = e0 + same;
    cluster_sync();
    for (int r = 0; r < rank; ++r) a0 += load_remote(&s_part[0], r), e0 += load_remote(&s_part[1], r);
    cluster_sync();  // no block ends while another reads it
  }
  int32_t* to = kept + early;
  const uint32_t below = (1u << lane) - 1;
#pragma unroll 2
  for (int i = i0 + lane; i < i0 + part; i += 32) {
    const uint32_t k = i < i1 ? key_at(i) : 0u;
    const uint32_t up = __ballot_sync(0xffffffffu, i < i1 && k > key), eq = __ballot_sync(0xffffffffu, i < i1 && k == key);
    const int a = a0 + __popc(up & below), e = e0 + __popc(eq & below);
    if (up >> lane & 1)
      to[a + min(e, left)] = early + p0 + i;
    else if ((eq >> lane & 1) && e < left)
      to[a + e] = early + p0 + i;
    a0 += __popc(up);
    e0 += __popc(eq);
  }
}

struct MoveParams {
  uint8_t* cache;
  const int32_t* table;
  const int32_t* kept;
  const int32_t* kept_lens;
  const int32_t* table_to;
  const float* weights;
  float* weights_to;
  int32_t* err;
  int32_t n_pages, page_size, hkv;
  int32_t width, kept_width, to_width;
  int32_t records;  // per (request, kv head), at most
};

constexpr int kMoveWarps = 4;

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32) kv4_move_kernel(const MoveParams p, int64_t units) {
  constexpr int NG = Kv4<D>::kGroups;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const int64_t unit = (int64_t)blockIdx.x * kMoveWarps + threadIdx.x / 32;
  if (unit >= units) return;
  // records of one (request, kv head) are neighbours, kv heads of a request next
  const int64_t pair = unit / p.records;
  const int rec = (int)(unit - pair * p.records), s = (int)(pair / p.hkv), g = (int)(pair - (int64_t)s * p.hkv);
  const int given = __ldg(p.kept_lens + s), most = min(p.kept_width, p.to_width * p.page_size);
  const int count = min(max(given, 0), most);
  if (g == 0 && rec == 0 && lane == 0 && (given < 0 || given > most)) record_error(p.err, kErrIndex, s);
  const int i0 = rec * kKv4Block;
  if (i0 >= count) return;
  const int per_page = p.page_size / kKv4Block;
  const int page_to = __ldg(p.table_to + (int64_t)s * p.to_width + rec / per_page);
  if (page_to < 0 || page_to >= p.n_pages) {
    if (lane == 0) record_error(p.err, kErrIndex, s);
    return;
  }
  uint8_t* dst = p.cache + (((int64_t)page_to * p.hkv + g) * per_page + rec % per_page) * Kv4<D>::kRecord;
  // lane t < 16: token t's source record, and its place there
  const uint8_t* src = nullptr;
  int t_from = 0;
  if (lane < kKv4Block && i0 + lane < count) {
    const int j = __ldg(p.kept + pair * p.kept_width + i0 + lane);
    if (j >= 0 && j < p.width * p.page_size) {
      const int page = __ldg(p.table + (int64_t)s * p.width + j / p.page_size);
      if (page >= 0 && page < p.n_pages) {
        src = p.cache + (((int64_t)page * p.hkv + g) * per_page + j % p.page_size / kKv4Block) * Kv4<D>::kRecord;
        t_from = j % kKv4Block;
        if (p.weights != nullptr)
          p.weights_to[pair * p.to_width * p.page_size + i0 + lane] = __ldg(p.weights + pair * p.width * p.page_size + j);
      }
    }
    if (src == nullptr) record_error(p.err, kErrIndex, s);
  }
  auto source = [&](int t, int& from) -> const uint8_t* {
    from = __shfl_sync(0xffffffffu, t_from, t);
    return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), t));
  };
  // K: D / 2 bytes a token, 16 a lane
  constexpr int kLanes = D / 32, kAtOnce = 32 / kLanes;
#pragma unroll
  for (int t0 = 0; t0 < kKv4Block; t0 += kAtOnce) {
    const int t = t0 + lane / kLanes, at = lane % kLanes * 16;
    int from;
    const uint8_t* x = source(t, from);
    if (x != nullptr)
      *reinterpret_cast<uint4*>(dst + t * (D / 2) + at) = *reinterpret_cast<const uint4*>(x + from * (D / 2) + at);
  }
  // scales: 4 NG bytes a token
  {
    int from;
    const uint8_t* x = source(lane % kKv4Block, from);
    if (x != nullptr && lane < kKv4Block) {
      uint32_t* to = reinterpret_cast<uint32_t*>(dst + Kv4<D>::kScales + lane * (4 * NG));
      const uint32_t* at = reinterpret_cast<const uint32_t*>(x + Kv4<D>::kScales + from * (4 * NG));
#pragma unroll
      for (int i = 0; i < NG; ++i) to[i] = at[i];
    }
  }
  // V: lane 4 r + c holds the words of tokens 8 half + 2 c and + 1
  const int r = lane / 4, c = lane % 4;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[2][NG];
    bool there[2];
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      int from;
      const uint8_t* x = source(8 * half + 2 * c + odd, from);
      there[odd] = x != nullptr;
      if (there[odd]) {
        const uint32_t* at = reinterpret_cast<const uint32_t*>(
            x + Kv4<D>::kV + (from / 8) * Kv4<D>::kPlane + (r * 4 + from % 8 / 2) * (4 * NG));
#pragma unroll
        for (int i = 0; i < NG; ++i) w[odd][i] = (from & 1 ? at[i] >> 16 : at[i] & 0xffffu);
      }
    }
    uint32_t* to = reinterpret_cast<uint32_t*>(dst + Kv4<D>::kV + half * Kv4<D>::kPlane + lane * (4 * NG));
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      if (there[0] && there[1]) {
        to[i] = w[0][i] | w[1][i] << 16;
      } else {  // the other token's half stays
        if (there[0]) reinterpret_cast<uint16_t*>(to + i)[0] = (uint16_t)w[0][i];
        if (there[1]) reinterpret_cast<uint16_t*>(to + i)[1] = (uint16_t)w[1][i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv4_keep(const float* weights, int32_t weights_width, const int32_t* lens, const int32_t* budgets,
                            int32_t n_seqs, int32_t hkv, int32_t first, int32_t recent, int32_t* kept,
                            int32_t kept_width, int32_t* kept_lens, int32_t sms, int32_t* err, cudaStream_t s) {
  const KeepParams p{weights, lens, budgets, kept, kept_lens, err, weights_width, kept_width, hkv, first, recent};
  const dim3 grid((unsigned)(n_seqs * hkv));
  static std::atomic<uint64_t> configured[3];
  if (weights_width <= (n_seqs * hkv > sms ? kShortRow : kShorterRow)) {
    // no more shared memory than the rows need, so that blocks of short ones share an SM
    const cudaError_t e = set_smem_limit_once(kv4_keep_kernel<512, 2, true, 1>, kShortRow * 4 + 16, configured[0]);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv4_keep_kernel<512, 2, true, 1>, grid, dim3(512), (size_t)weights_width * 4 + 16, s, p);
  }
  if (n_seqs * hkv <= (weights_width > kHeldKeys ? kLongClusterRows : kClusterRows) && weights_width <= kCluster * kHeldKeys) {
    const size_t smem = (size_t)((weights_width + kCluster - 1) / kCluster) * 4 + 16;
    const cudaError_t e = set_smem_limit_once(kv4_keep_kernel<1024, 4, true, kCluster>, kHeldKeys * 4 + 16, configured[1]);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid.x * kCluster);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv4_keep_kernel<1024, 4, true, kCluster>, p);
  }
  if (weights_width > kHeldKeys) return launch_pdl(kv4_keep_kernel<1024, 4, false, 1>, grid, dim3(1024), 0, s, p);
  const cudaError_t e = set_smem_limit_once(kv4_keep_kernel<1024, 4, true, 1>, kHeldKeys * 4 + 16, configured[2]);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_keep_kernel<1024, 4, true, 1>, grid, dim3(1024), (size_t)weights_width * 4 + 16, s, p);
}

cudaError_t launch_kv4_move(void* cache, int32_t n_pages, int32_t page_size, int32_t hkv, int32_t head_dim,
                            const int32_t* table, int32_t width, const int32_t* kept, int32_t kept_width,
                            const int32_t* kept_lens, int32_t n_seqs, const int32_t* table_to, int32_t to_width,
                            const float* weights, float* weights_to, int32_t* err, cudaStream_t s) {
  MoveParams p{static_cast<uint8_t*>(cache), table, kept, kept_lens, table_to, weights, weights_to, err, n_pages, page_size,
               hkv, width, kept_width, to_width, 0};
  // (at least one, so that lengths past an empty table are recorded)
  p.records = std::max((std::min(kept_width, to_width * page_size) + kKv4Block - 1) / kKv4Block, 1);
  const int64_t units = (int64_t)n_seqs * hkv * p.records;
  const dim3 grid((unsigned)((units + kMoveWarps - 1) / kMoveWarps));
  if (head_dim == 128) return launch_pdl(kv4_move_kernel<128>, grid, dim3(kMoveWarps * 32), 0, s, p, units);
  if (head_dim == 64) return launch_pdl(kv4_move_kernel<64>, grid, dim3(kMoveWarps * 32), 0, s, p, units);
  return cudaErrorInvalidValue;
}

}  // namespace cb
