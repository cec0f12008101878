// Page tables, slot map and packed offsets of one serving step, from the requests' lengths.
//
// With P = page_size, request s holds have_s = ceil(ctx_s / P) pages and needs
// need_s = ceil((ctx_s + new_s) / P) - have_s more. It takes free[first_s .. first_s + need_s), where
// first_s = from + sum of need over the requests before it. Its new tokens are the packed rows
// cu_s .. cu_s + new_s - 1 (cu: exclusive sum of new), row r at position ctx_s + r - cu_s and in slot
// table[s][position / P] * P + position % P.
//
// Bound by latency: a step reads 8 bytes per request and writes 8 bytes per new row, so the design
// is one launch without any wait between blocks. Every block forms both prefix sums over all
// requests in its shared memory (12 bytes per request) and then takes its own share of the pages and
// of the rows, finding each one's request by a binary search. A page that a row falls in is looked
// up where its owner finds it (the old table or the free list), never in an entry that another block
// writes in the same launch. 64 requests that decode take 3.5 us on the device, 512 prompts of 2,048 tokens at most
// (540,000 rows, 4.3 MB out: 0.7 us at the copy rate) 8.0: 2.5 for a launch that does nothing but the sums (of 64
// requests or 512), 2.5 more where 264 blocks also write padding for every row, 2.6 more for the rows' searches and the pages
// that they look up, 0.4 for 34,000 table entries. The Python call takes 8.9.
#include "common.cuh"
#include "kernels.h"

namespace cb {
namespace {

constexpr int kThreads = 512;
constexpr int kRowsPerBlock = 2048;  // rows a block takes (4 per thread) while the grid is below kMaxBlocks
constexpr int kMaxBlocks = 304;      // two blocks per SM; larger steps loop

struct PageTableParams {
  const int32_t* ctx;
  const int32_t* added;
  int32_t n_seqs;
  int32_t page_size;
  const int32_t* free_pages;
  int32_t n_free;
  const int32_t* free_from;
  int32_t* table;
  int32_t width;
  int32_t* cu;
  int32_t* kv_lens;
  int32_t* positions;
  int32_t* slots;
  int32_t n_rows;
  int32_t* free_to;
  int32_t* err;
  uint64_t inverse;  // ceil(2^34 / (page_size / 16))
};

// Index of the last element of a[0 .. n) that is <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Lengths of request s, negative ones taken as 0. Their sum fits 32 bits without a sign.
struct Req {
  uint32_t ctx, added;
};
__device__ __forceinline__ Req request(const PageTableParams& p, int s) {
  const int32_t c = p.ctx[s], a = p.added[s];
  return Req{(uint32_t)max(c, 0), (uint32_t)max(a, 0)};
}
// t / page_size by a product: page_size = 16 m with m <= 64, and n = t / 16 < 2^28, so with M = ceil(2^34 / m)
// n M = n 2^34 / m + (less than 2^34 / m): the quotient's integer part. (Divisions took most of the kernel's time.)
__device__ __forceinline__ uint32_t page_index(const PageTableParams& p, uint32_t t) {
  return (uint32_t)((uint64_t)(t >> 4) * p.inverse >> 34);
}
// Pages that t tokens take, at most the table's width.
__device__ __forceinline__ int32_t pages_of(const PageTableParams& p, uint32_t t) {
  const uint32_t whole = page_index(p, t), n = whole + (t != whole * (uint32_t)p.page_size ? 1 : 0);
  return (int32_t)min(n, (uint32_t)p.width);
}

__global__ void __launch_bounds__(kThreads) page_tables_kernel(const PageTableParams p) {
  extern __shared__ int32_t smem[];
  int32_t* s_cu = smem;                  // [n_seqs] first row of each request, at most n_rows
  int32_t* s_first = smem + p.n_seqs;    // [n_seqs] pages taken by the requests before it
  uint32_t* s_ctx = reinterpret_cast<uint32_t*>(smem) + 2 * p.n_seqs;  // [n_seqs] tokens that it holds
  __shared__ int64_t w_rows[kThreads / 32];
  __shared__ int32_t w_pages[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int32_t from = p.free_from ? *p.free_from : 0;
  if (from < 0) {
    if (blockIdx.x == 0 && tid == 0) record_error(p.err, kErrIndex, from);
    from = 0;
  }

  // Both exclusive sums: each thread adds up a run of requests, the block adds up the threads.
  const int run = (p.n_seqs + kThreads - 1) / kThreads;
  const int s0 = min(tid * run, p.n_seqs), s1 = min(s0 + run, p.n_seqs);
  int64_t rows = 0;
  int32_t pages = 0;
  for (int s = s0; s < s1; ++s) {
    const Req q = request(p, s);
    rows += q.added;
    pages += pages_of(p, q.ctx + q.added) - pages_of(p, q.ctx);
  }
  int64_t rows_up = rows;
  int32_t pages_up = pages;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t r = __shfl_up_sync(0xffffffffu, rows_up, d);
    const int32_t g = __shfl_up_sync(0xffffffffu, pages_up, d);
    if (lane >= d) rows_up += r, pages_up += g;
  }
  if (lane == 31) w_rows[warp] = rows_up, w_pages[warp] = pages_up;
  __syncthreads();
  int64_t rows_before = 0, rows_all = 0;
  int32_t pages_before = 0, pages_all = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) rows_before += w_rows[w], pages_before += w_pages[w];
    rows_all += w_rows[w], pages_all += w_pages[w];
  }
  rows = rows_before + rows_up - rows;
  pages = pages_before + pages_up - pages;
  for (int s = s0; s < s1; ++s) {
    const Req q = request(p, s);
    s_cu[s] = (int32_t)(rows < p.n_rows ? rows : p.n_rows);
    s_first[s] = pages;
    s_ctx[s] = q.ctx;
    if (blockIdx.x == 0) {
      p.cu[s] = s_cu[s];
      const int64_t room = (int64_t)p.width * p.page_size, len = (int64_t)q.ctx + q.added;
      p.kv_lens[s] = (int32_t)(len < room ? len : room);
      if (p.ctx[s] < 0 || p.added[s] < 0 || len > room) record_error(p.err, kErrIndex, s);
    }
    rows += q.added;
    pages += pages_of(p, q.ctx + q.added) - pages_of(p, q.ctx);
  }
  const int32_t n_rows_used = (int32_t)(rows_all < p.n_rows ? rows_all : p.n_rows);
  if (blockIdx.x == 0 && tid == 0) {
    p.cu[p.n_seqs] = n_rows_used;
    const int64_t left = (int64_t)p.n_free - from;
    p.free_to[0] = from + (int32_t)(pages_all < left ? pages_all : (left > 0 ? left : 0));
    if (pages_all > left && pages_all > 0) record_error(p.err, kErrIndex, p.n_free);
    if (rows_all > p.n_rows) record_error(p.err, kErrIndex, p.n_rows);
  }
  __syncthreads();

  // The i-th page taken in this step: -1 where the free list is at its end or holds no page id.
  const int32_t max_page = 0x7fffffff / p.page_size - 1;
  auto taken = [&](int64_t i) -> int32_t {
    const int64_t at = from + i;
    if (at >= p.n_free) return -1;
    const int32_t id = p.free_pages[at];
    return id > max_page ? -1 : id;
  };
  const int64_t first = (int64_t)blockIdx.x * kThreads + tid, stride = (int64_t)gridDim.x * kThreads;
  // A request without new pages shares its first page with the next one's; the search returns the
  // last request that starts at or before the page, which is the one that takes it.
  for (int64_t u = first; u < pages_all; u += stride) {
    const int s = last_at_most(s_first, p.n_seqs, (int)u);
    const int32_t col = pages_of(p, s_ctx[s]) + (int32_t)u - s_first[s];
    const int32_t id = taken(u);
    if (id < 0 && from + u < p.n_free) record_error(p.err, kErrIndex, s);
    p.table[(int64_t)s * p.width + col] = id;
  }
  // Four rows per thread, one behind the other, where the requests add four and more on average: one search, and
  // one look at a page, do for most fours (512 prompts, 0.5 M rows: 8.0 us on the device against 11.1 row
  // by row). One otherwise, as each has a request of its own (64 requests that decode: 3.9 against 5.7).
  const int per = p.n_rows / 4 >= p.n_seqs ? 4 : 1;
  const bool wide = per == 4 && ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
  for (int64_t r0 = per * first; r0 < p.n_rows; r0 += per * stride) {
    int32_t pos[4], slot[4];
    int s = -1;                        // request of the row
    uint32_t ctx = 0, start = 0, end = 0, have = 0;  // its tokens held, first row, first row behind it, pages held
    uint32_t col = 0xffffffffu;        // page of the row before, which is page `page` of the cache
    int32_t page = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pos[i] = 0, slot[i] = -1;
      const uint32_t r = (uint32_t)r0 + i;
      if (i >= per || r >= (uint32_t)n_rows_used) continue;
      if (s < 0 || r >= end) {
        s = last_at_most(s_cu, p.n_seqs, (int)r);
        ctx = s_ctx[s];
        start = s_cu[s];
        end = s + 1 < p.n_seqs ? s_cu[s + 1] : n_rows_used;
        have = (uint32_t)pages_of(p, ctx);
        col = 0xffffffffu;
      }
      const uint32_t at = ctx + (r - start), c = page_index(p, at);
      pos[i] = (int32_t)min(at, 0x7fffffffu);
      if (c != col) {
        col = c;
        page = -1;
        if (c < (uint32_t)p.width) {
          if (c < have) {
            page = p.table[(int64_t)s * p.width + c];  // held before this step: nobody writes it now
            if (page < 0 || page > max_page) {
              record_error(p.err, kErrIndex, s);
              page = -1;
            }
          } else {
            page = taken((int64_t)s_first[s] + (c - have));
          }
        }
      }
      if (page >= 0) slot[i] = page * p.page_size + (int32_t)(at - c * (uint32_t)p.page_size);
    }
    if (wide && r0 + 4 <= p.n_rows) {
      *reinterpret_cast<int4*>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(p.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < per && r0 + i < p.n_rows) p.positions[r0 + i] = pos[i], p.slots[r0 + i] = slot[i];
    }
  }
}

}  // namespace

cudaError_t launch_page_tables(const int32_t* ctx, const int32_t* added, int32_t n_seqs, int32_t page_size,
                               const int32_t* free_pages, int32_t n_free, const int32_t* free_from, int32_t* table,
                               int32_t width, int32_t* cu, int32_t* kv_lens, int32_t* positions, int32_t* slots,
                               int32_t n_rows, int32_t* free_to, int32_t* err, cudaStream_t s) {
  const PageTableParams p{ctx, added, n_seqs,  page_size, free_pages, n_free, free_from, table,
                          width, cu, kv_lens, positions, slots, n_rows, free_to, err,
                          ((1ull << 34) + page_size / 16 - 1) / (uint64_t)(page_size / 16)};
  // pages are at most one per new row and request, so the rows set the grid
  int64_t blocks = ((int64_t)n_rows + n_seqs + kRowsPerBlock - 1) / kRowsPerBlock;
  blocks = blocks < 1 ? 1 : (blocks > kMaxBlocks ? kMaxBlocks : blocks);
  const size_t smem = sizeof(int32_t) * 3 * (size_t)n_seqs;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e =
      set_smem_limit_once(page_tables_kernel, (int)(sizeof(int32_t) * 3 * kPageTablesMaxSeqs), configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(page_tables_kernel, dim3((unsigned)blocks), dim3(kThreads), smem, s, p);
}

}  // namespace cb
