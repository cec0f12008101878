// Causal grouped-query attention over whole prompts, packed one after the other:
//
//   out[t, h] = sum_{j <= t} softmax_j(scale * q[t, h] . k[j, g]) v[j, g],  g = h / G,
//
// for tokens t and j of the same sequence; sequence s is rows cu[s] .. cu[s + 1] - 1 of q, k, v, out.
//
// Bound by the tensor cores from a few hundred tokens per sequence on (4 hq D flops per visible pair),
// by HBM below that. The tile loop is the paired-tile kernel's (attention_pp.cu): a work item is one
// kv head and two query tiles of 128 rows (tile i: TQ = 128 / G tokens times the G heads), whose
// softmax and tensor-core work alternate, so that each softmax hides behind the other tile's MMAs.
//
// What differs, and why:
//   Persistent CTAs. A chunk of 2,048 tokens has items of 1 to 16 key tiles, 8.5 rounds of 1.4 us
//   on average, and starting a CTA (TMEM, barriers, first loads) costs about 3 us, a quarter of that.
//   One CTA per SM takes items in turn; the rings of K and V run on across items, and the next
//   item's first tiles load while the last softmax of the current one runs.
//   No tile list. The lengths are known on the device only. The grid has a block for every item that
//   the row count allows; blocks stand for the items in the order of `Order`, and a running CTA claims the
//   next block that has not started (cluster launch control) when it has requested its last K tile. The
//   producer warp finds a block's item by counting sequences. Taken in turn instead, by index modulo
//   the number of CTAs in alternating direction, the items of 40 prompts of 1 to 1,087 tokens ended between
//   290 and 327 us on the various SMs; claimed they end within 4 us of one another.
//   Order. Longest first, so that the SMs end together, but by groups of sequences whose K and V (48 MB
//   at the mean length) stay in L2: over all sequences at once, 16 chunks of 2,048 tokens read theirs
//   from HBM again and again (64% of L2's reads missed): 472 us against 425, the 40 prompts 293 against
//   282, 64 prompts of 512 tokens 186 against 172. Groups of 8, 16, 32 and 64 MB: 436, 438, 429 and 429 us for
//   the chunks, 289, 283, 282 and 284 for the prompts; each sequence a group of its own 435, 299 and 204.
//   Four or eight levels of a sequence as neighbours are slower too.
//   Rows of other sequences. A key tile that reaches past its sequence's end holds the next one's
//   rows, and one on the diagonal holds keys that some of the rows must not see; their weight is 0, but
//   0 * V is NaN where V is infinite or NaN. In those tiles (the ones with a key that some row of the
//   item does not see) the waiter warp looks for such values and sets them to 0 in shared memory; an
//   item where it found any adds them back to the rows that do see them, in the epilogue. The search
//   runs while the tile waits for its softmax.
//   Output. Each softmax warp stages 64 columns of its 32 rows in shared memory of its own and sends
//   them off as one box by TMA, which runs on while the warp goes to its next item (stores from
//   registers or staged ones held the warps for 3,000 - 4,000 cycles per item, an SM's store path taking
//   about 30 bytes per cycle). A warp whose rows pass the sequence's end, which belong to others, stores
//   those inside itself. The query tiles' buffers stay free for the next item.
//   Next scores. Behind an item's last products the issuer forms the next item's first scores, while
//   the softmax warps write their output. Boxes of 32 columns, two in flight, instead of the output's boxes
//   of 64 held the warps longer: 306 against 293 us for the 40 prompts.
// Roles, TMEM columns, register split and bounded waits are those of attention_pp.cu; "round" counts
// the key tiles of all the CTA's items, and ring stage and parity follow from it. Item descriptions
// pass from the producer to the other warps through a ring of eight: the producer requests item i + 7's
// keys only once both tiles' scores of item i + 5 are formed, for which the softmax warps are through with
// item i + 3. After a wait that gave up (abort flag) every warp still walks through the rounds of the
// current item, without work, and the producer ends the list, so no named barrier is left short.
//
// Measured (8 kv heads of 128 dims): 16 chunks of 2,048 tokens, 32 query heads, 427 us with new inputs in each
// call, 394 with the same (284 us at the tensor cores' rate, 100 of HBM); 40 prompts of 1 to 1,087 tokens,
// 64 query heads, 283 us (135 and 117); one prompt of 16,384 tokens 1.32 ms, 0.86 of that rate. Other head layouts, 16
// chunks of 2,048 tokens: 16 query heads on 16 kv heads of 128 dims 227 us (142; tile 0 runs an item's last round masked
// whole), on one 197; of 64 dims 16 on one 169 (71), 32 on 16 329 (142): there a score costs the softmax as much for
// half the products. 64 prompts of 64 tokens, 32 query heads, 23 us.
// A round (a key tile against both query tiles) takes 2,750 - 2,850 cycles, of which the tensor cores need 2,504;
// an item adds about 6,000: on its softmax warps' path the masks of the diagonal tile (600), the last product
// (1,000), the output (2,000), the next item and the first maximum (600).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "attn_common.cuh"
#include "attn_tile.cuh"
#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"
#include "tmem_ops.cuh"

namespace cb {
namespace {

constexpr int kBM = 128;      // rows per query tile
constexpr int kTiles = 2;     // query tiles per item
constexpr int kBN = kTileKeys;  // keys per key tile
constexpr int kStages = 2;    // depth of the K and of the V ring
constexpr int kItems = 8;     // depth of the item ring
constexpr uint32_t kOutWarp = 32 * 128;  // output staging of one softmax warp
constexpr int kThreads = 384;
constexpr int kSoftmaxThreads = 128;
constexpr int kWarpProducerK = 8;
constexpr int kWarpMma = 9;
constexpr int kWarpProducerV = 10;
constexpr int kWarpWaiter = 11;
constexpr int kBarExit = 1;   // all 384 threads, before the tensor memory is freed
constexpr int kBarTile0 = 2;  // WG0 + issuer + waiter (192 threads), once per key tile
constexpr int kBarTile1 = 3;  // WG1 + issuer (160 threads), once per key tile
constexpr uint32_t kTmemCols = 512;
constexpr int kSoftmaxRegs = 216;  // per thread of WG0 / WG1 after setmaxnreg.inc
constexpr int kOtherRegs = 72;     // per thread of WG2 after setmaxnreg.dec
constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale O only when the max grows by > 2^8
constexpr float kTileSumLimit = 65536.0f;  // a later tile whose P sum exceeds 2^16 moves the reference
constexpr int64_t kGroupBytes = 48 << 20;  // K and V of the sequences that are taken side by side
// Limit of the wait for an item, of a kernel whose other waits give up after limit_ns. It must not run out while the
// producer lives, since roles that see different lists would miss one another at the named barriers: the producer
// makes two waits at most before it ends the list, each over at the first look at the clock past its limit (every 1.6 ms).
__host__ __device__ constexpr uint64_t item_limit(uint64_t limit_ns) { return 5 * limit_ns + 50000000ull; }

__host__ __device__ constexpr uint32_t col_s(int i) { return (uint32_t)(i * kBN); }
__host__ __device__ constexpr uint32_t col_o(int i, int d) { return 256u + (uint32_t)(i * d); }

struct Item {
  int row0;   // first row of the sequence
  int len;    // its rows
  int t0;     // first token (in the sequence) of query tile 0
  int g;      // kv head
  int n_kv;   // key tiles, 0: no more items
  int fixed;  // set by the waiter: a V tile held values that are not finite
};

// First key that is searched for values that are not finite: the first that some row of the item does
// not see is t0 + 1, and the search goes by 32 keys.
__device__ __forceinline__ int hidden_from(int t0) { return (t0 + 1) / 32 * 32; }

struct Bars {
  uint64_t q_full[kTiles];
  uint64_t k_full[kStages];
  uint64_t v_full[kStages];
  uint64_t s_full[kTiles][kStages];  // S_i of a round complete (commit); [1][s] also: K stage s free
  uint64_t o_done[kTiles][kStages];  // P_i V of a round complete (commit); [1][s] also: V stage s free
  uint64_t item[kItems];
  uint64_t claim;  // the answer to a claim of another block has arrived
  uint64_t drain;
};

struct PromptParams {
  const uint8_t* v;
  const int32_t* cu;
  uint8_t* out;
  int n_seqs;
  int n_rows;
  int hq;
  int hkv;
  int group;  // query heads per kv head, 1 << lg
  int lg;
  int tq;     // query tokens per tile = 128 / group
  int seqs_per_group;  // of the items' order
  float scale_log2;
  int32_t* err;
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void named_sync(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Cluster launch control: ask for a block of this grid that has not been launched yet, to run its work
// here. The 16-byte answer arrives in shared memory on an mbarrier.
__device__ __forceinline__ void claim_block(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
               "r"(bar)
               : "memory");
}
// The claimed block's index, -1 where none was left (no further claim may follow then).
__device__ __forceinline__ int claimed_block(uint32_t answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(answer)
      : "memory");
  return got != 0 ? (int)x : -1;
}

// First row of each sequence, inside [0, n_rows].
__device__ __forceinline__ int row_at(const PromptParams& p, int s) {
  const int r = __ldg(p.cu + s);
  return r < 0 ? 0 : min(r, p.n_rows);
}

// The launch's items in the order in which blocks stand for them, for a converged warp: by groups of
// p.seqs_per_group sequences (at most 32, one per lane); in a group by level (the index of an item in its
// sequence) from the highest down, so the longest first; in a level by sequence and kv head.
struct Order {
  int s0, group_end;   // the group's first sequence, index behind its last item
  int items;           // per kv head, of this lane's sequence
  int level, end;      // current level, index behind its last item
  uint32_t has;        // the sequences that have it
  int latest;          // last index asked for

  // Items per kv head of sequence s.
  __device__ __forceinline__ int items_of(const PromptParams& p, int s) const {
    const int n = row_at(p, s + 1) - row_at(p, s), per = kTiles * p.tq;
    return n > 0 ? (n + per - 1) >> (__ffs(per) - 1) : 0;
  }
  // The group from sequence s on, whose first item has index `first`.
  __device__ __forceinline__ void enter(const PromptParams& p, int s, int first, int lane) {
    s0 = s;
    items = lane < p.seqs_per_group && s + lane < p.n_seqs ? items_of(p, s + lane) : 0;
    group_end = first + __reduce_add_sync(0xffffffffu, items) * p.hkv;
    level = __reduce_max_sync(0xffffffffu, items);
    end = first;
  }
  __device__ __forceinline__ void start(const PromptParams& p, int lane) {
    latest = 0;
    enter(p, 0, 0, lane);
  }
  // Item idx: false past the last one. Indices come in rising order but for rare cases, which begin anew.
  __device__ __forceinline__ bool find(const PromptParams& p, int idx, int lane, int& seq, int& head) {
    if (idx < latest) start(p, lane);
    latest = idx;
    while (idx >= group_end) {
      if (s0 + p.seqs_per_group >= p.n_seqs) return false;
      enter(p, s0 + p.seqs_per_group, group_end, lane);
    }
    while (idx >= end) {
      has = __ballot_sync(0xffffffffu, items >= level);
      --level;
      end += __popc(has) * p.hkv;
    }
    const uint32_t rel = idx - (end - __popc(has) * p.hkv), nth = rel / (uint32_t)p.hkv;
    head = (int)(rel - nth * p.hkv);
    uint32_t left = has;
    for (uint32_t i = 0; i < nth; ++i) left &= left - 1;
    seq = s0 + __ffs(left) - 1;
    return true;
  }
};

// Rows from .. kBN - 1 (from a multiple of 32) of a V tile in shared memory (boxes of 64 columns, 128
// bytes per row): values that are not finite become 0. True (in every lane) if there were any. Called
// by a converged warp; eight loads in flight per lane (one at a time took 4,200 cycles per tile,
// longer than a round of the tile loop).
template <int BOXES>
__device__ __forceinline__ bool zero_not_finite(uint32_t tile, int from, int lane) {
  bool found = false;
#pragma unroll 1
  for (int b = 0; b < BOXES; ++b) {
#pragma unroll 1
    for (int r = from; r < kBN; r += 32) {
      const uint32_t at = tile + (uint32_t)(b * kBN * 128 + r * 128 + lane * 16);
      uint32_t bad = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[u][0]), "=r"(w[u][1]), "=r"(w[u][2]), "=r"(w[u][3])
                       : "r"(at + (uint32_t)(h * 4 + u) * 512));
        // an exponent of all ones, plus one unit of it, carries into the sign bit of its half
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) bad |= (w[u][e] & 0x7f807f80u) + 0x00800080u;
      }
      if (__any_sync(0xffffffffu, bad & 0x80008000u)) {
        found = true;
#pragma unroll 1
        for (int u = 0; u < 32; ++u) {
          uint32_t x;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(at + u / 4 * 512 + u % 4 * 4) : "memory");
          if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
          if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + u / 4 * 512 + u % 4 * 4), "r"(x) : "memory");
        }
      }
    }
  }
  if (found) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read it next
  return found;
}

// PROBE: the wait-timeout probe (test support only): the K producer of every CTA arms the barrier of its second key
// tile but never copies the tile, and the waits give up after kProbeTimeoutNs, so each CTA with two key tiles or more
// takes its failure path. Compiled out of the kernel itself.
template <int D, bool PROBE = false>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                            const PromptParams p) {
  constexpr uint64_t kLimit = PROBE ? kProbeTimeoutNs : kTimeoutNs;
  constexpr int kBoxes = D / 64;
  constexpr uint32_t kQBytes = kBM * D * 2;  // one query tile
  constexpr uint32_t kKVBytes = kBN * D * 2;
  constexpr uint32_t kQBox = kBM * 128;   // bytes of one 64-column box of a query tile
  constexpr uint32_t kKVBox = kBN * 128;  // bytes of one 64-column box of a K or V tile

  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ Item items[kItems];
  __shared__ alignas(16) uint4 s_claim;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_round_ok[2];

  pdl_launch_dependents();
  if (threadIdx.x == 32 * kWarpWaiter) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_q) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_v) : "memory");
  }
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base;                        // query tile i at sQ + i kQBytes
  const uint32_t sK0 = base + kTiles * kQBytes;    // K stage s at sK0 + s kKVBytes
  const uint32_t sV0 = sK0 + kStages * kKVBytes;   // V stage s at sV0 + s kKVBytes
  const uint32_t sOut = sV0 + kStages * kKVBytes;  // softmax warp w stages 32 rows of 64 columns at sOut + w kOutWarp
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (warp == kWarpProducerK && lane == 0) {
    for (int i = 0; i < kTiles; ++i) mbar_init(smem_u32(&bars.q_full[i]), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&bars.k_full[s]), 1);
      mbar_init(smem_u32(&bars.v_full[s]), 1);
      for (int i = 0; i < kTiles; ++i) {
        mbar_init(smem_u32(&bars.s_full[i][s]), 1);
        mbar_init(smem_u32(&bars.o_done[i][s]), 1);
      }
    }
    for (int i = 0; i < kItems; ++i) mbar_init(smem_u32(&bars.item[i]), 1);
    mbar_init(smem_u32(&bars.claim), 1);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  // Key tiles of the it-th item of this CTA, which lies in items[it % kItems]; 0 at the end (and, never
  // expected, if it does not come).
  auto item_at = [&](int it) -> int {
    const uint32_t bar = smem_u32(&bars.item[it % kItems]);
    bool there = mbar_test(bar, (it / kItems) & 1);
    if (!there) {
      const uint64_t t0 = global_timer();
      for (uint32_t n = 1; !(there = mbar_try_wait_sleep(bar, (it / kItems) & 1)); ++n)
        if ((n & 7u) == 0 && global_timer() - t0 > item_limit(kLimit)) break;
    }
    there = __all_sync(0xffffffffu, there);
    if (there) return items[it % kItems].n_kv;
    *abort_flag = 1;
    record_error(p.err, kErrTimeout, 40);
    return 0;
  };

  if (warp >= kTiles * (kSoftmaxThreads / 32)) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    pdl_wait();  // q, k, v and the offsets come from the kernels before this one
    if (warp == kWarpProducerK) {
      if (blockIdx.x == 0)  // offsets that fall or leave the rows are recorded (and read as empty or clipped)
        for (int s = lane; s < p.n_seqs; s += 32) {
          const int a = __ldg(p.cu + s), b = __ldg(p.cu + s + 1);
          if (a < 0 || b > p.n_rows) record_error(p.err, kErrIndex, s);
          if (b < a) record_error(p.err, kErrOrder, s);
        }
      Order order;
      order.start(p, lane);
      int rounds = 0;  // rounds of the items before
      int nk = 0;      // K tiles requested, by round
      // The first item is the block's own; each further one is that of a block which has not started,
      // claimed when the K tiles of the item before have been requested.
      int idx = blockIdx.x, claims = 0;
      for (int it = 0;;) {
        Item x{0, 0, 0, 0, 0, 0};
        int seq, head;
        bool give_up = __any_sync(0xffffffffu, *abort_flag != 0);
        if (!give_up && idx >= 0 && order.find(p, idx, lane, seq, head)) {
          x.row0 = row_at(p, seq);
          x.len = row_at(p, seq + 1) - x.row0;
          x.t0 = order.level * kTiles * p.tq;
          x.g = head;
          x.n_kv = (min(x.t0 + kTiles * p.tq, x.len) - 1) / kBN + 1;
        }
        const bool end = give_up || idx < 0;  // a block past the last item has none: claim the next
        if (lane == 0 && (end || x.n_kv > 0)) {
          items[it % kItems] = x;
          mbar_arrive(smem_u32(&bars.item[it % kItems]));
          const int n = x.n_kv;
          auto load_k = [&](int j) -> bool {
            const int r = rounds + j, st = r % kStages;
            // K of round r - 2 held this stage: free once S_1 of that round (issued after S_0) is complete
            if (r >= kStages &&
                !mbar_wait_inl(smem_u32(&bars.s_full[1][st]), ((r / kStages) - 1) & 1, abort_flag, p.err, 41, true,
                               kLimit))
              return false;
            const uint32_t kb = smem_u32(&bars.k_full[st]);
            mbar_expect_tx(kb, kKVBytes);
            if (!(PROBE && r == 1)) tma_load_4d(sK0 + st * kKVBytes, &tm_k, kb, 0, x.row0 + j * kBN, 0, x.g);
            nk = r + 1;
            return true;
          };
          bool ok = true;
          for (int j = 0; j < n && ok; ++j) ok = load_k(j);
        }
        __syncwarp();
        if (end) break;
        if (x.n_kv > 0) ++it;
        rounds += x.n_kv;
        const uint32_t cb = smem_u32(&bars.claim);
        if (lane == 0) {
          mbar_expect_tx(cb, 16);
          claim_block(smem_u32(&s_claim), cb);
        }
        __syncwarp();
        // not honouring the abort flag: the answer must have landed before the CTA exits
        const bool there =
            __all_sync(0xffffffffu, mbar_wait_inl(cb, claims & 1, abort_flag, p.err, 44, false, kLimit));
        ++claims;
        idx = there ? claimed_block(smem_u32(&s_claim)) : -1;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // read before the next answer is written
        __syncwarp();
      }
      // Before the CTA can exit, every copy issued must have landed (also after an abort).
      if (lane == 0) {
        for (int r = nk < kStages ? 0 : nk - kStages; r < nk; ++r)
          mbar_wait_inl(smem_u32(&bars.k_full[r % kStages]), (r / kStages) & 1, abort_flag, p.err, 57, false, kLimit);
      }
    } else if (warp == kWarpProducerV) {
      int rounds = 0, nv = 0, nq = 0;  // V tiles, query tiles requested
      bool ok = true;
      for (int it = 0;; ++it) {
        const int n_kv = item_at(it);
        if (n_kv == 0) break;
        if (lane == 0) {
          const int row0 = items[it % kItems].row0, t0 = items[it % kItems].t0, g = items[it % kItems].g;
          auto load_v = [&](int j) {
            const int r = rounds + j, st = r % kStages;
            // V of round r - 2 held this stage: free once P_1 V of that round (after P_0 V) is complete
            ok = r < kStages ||
                 mbar_wait_inl(smem_u32(&bars.o_done[1][st]), ((r / kStages) - 1) & 1, abort_flag, p.err, 43, true, kLimit);
            if (!ok) return;
            const uint32_t vb = smem_u32(&bars.v_full[st]);
            mbar_expect_tx(vb, kKVBytes);
            tma_load_4d(sV0 + st * kKVBytes, &tm_v, vb, 0, row0 + j * kBN, 0, g);
            nv = r + 1;
          };
          // Query tile i: its buffer is free once S_i of the round before (the last of the item before)
          // is complete. Rows past the sequence's end are other sequences' (or the fill value).
          auto load_q = [&](int i) {
            const int r = rounds - 1;
            ok = ok && (r < 0 || mbar_wait_inl(smem_u32(&bars.s_full[i][r % kStages]), (r / kStages) & 1, abort_flag,
                                               p.err, 42, true, kLimit));
            if (!ok) return;
            const uint32_t qb = smem_u32(&bars.q_full[i]);
            mbar_expect_tx(qb, kQBytes);
            tma_load_5d(sQ + i * kQBytes, &tm_q, qb, 0, 0, row0 + t0 + i * p.tq, 0, g);
            ++nq;
          };
          // in the order in which the buffers become free
          load_q(0);
          if (ok) load_v(0);
          load_q(1);
          for (int j = 1; j < n_kv && ok; ++j) load_v(j);
        }
        __syncwarp();
        rounds += n_kv;
      }
      // Before the CTA can exit, every copy issued must have landed (also after an abort).
      if (lane == 0)
        for (int i = 0; i < kTiles; ++i) {
          const int n = (nq + 1 - i) / kTiles;  // tiles i requested
          if (n > 0) mbar_wait_inl(smem_u32(&bars.q_full[i]), (n - 1) & 1, abort_flag, p.err, 56, false, kLimit);
        }
      if (lane == 0)
        for (int r = nv < kStages ? 0 : nv - kStages; r < nv; ++r)
          mbar_wait_inl(smem_u32(&bars.v_full[r % kStages]), (r / kStages) & 1, abort_flag, p.err, 58, false, kLimit);
    } else if (warp == kWarpWaiter) {
      // Per round, its V tile and the item's next K tile, published to the issuer through shared memory
      // before the waiter meets the issuer (and WG0) on a named barrier. Every round is joined, also
      // after a failure.
      auto spin_all = [&](uint32_t bar, uint32_t parity, int site) -> bool {
        return __all_sync(0xffffffffu, mbar_spin_inl(bar, parity, abort_flag, p.err, site, kLimit));
      };
      int rounds = 0;
      bool ok = true;
      for (int it = 0;; ++it) {
        const int n_kv = item_at(it);
        if (n_kv == 0) break;
        const int hidden = hidden_from(items[it % kItems].t0), first_edge = items[it % kItems].t0 + 1;
        for (int j = 0; j < n_kv; ++j) {
          const int r = rounds + j, st = r % kStages;
          ok = ok && spin_all(smem_u32(&bars.v_full[st]), (r / kStages) & 1, 47);
          // a tile with a key that the item's first row does not see
          if (ok && (j + 1) * kBN > first_edge &&
              zero_not_finite<kBoxes>(sV0 + st * kKVBytes, max(hidden - j * kBN, 0), lane) && lane == 0)
            items[it % kItems].fixed = 1;
          ok = ok && (j + 1 >= n_kv ||
                      spin_all(smem_u32(&bars.k_full[(r + 1) % kStages]), ((r + 1) / kStages) & 1, 48));
          if (lane == 0) s_round_ok[r & 1] = ok ? 1 : 0;
          __syncwarp();  // bar.sync is warp-aligned: reach it converged
          named_sync(kBarTile0, 192);
        }
        rounds += n_kv;
      }
    } else if (warp == kWarpMma) {
      constexpr uint32_t idesc_s = idesc_bf16(kBM, kBN, false);
      constexpr uint32_t idesc_o = idesc_bf16(kBM, D, true);
      const uint64_t dk0 = sdesc(sK0, 16, 1024);
      const uint64_t dv0 = sdesc(sV0, kKVBox, 1024);
      // S_i = Q_i K^T of round r; elected lane only.
      auto issue_s = [&](int i, int r) {
        const int st = r % kStages;
        const uint64_t dq = sdesc(sQ + i * kQBytes, 16, 1024);
        const uint64_t dk = dk0 + (uint64_t)((st * kKVBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int bx = ks / 4, kk = ks % 4;
          mma_ss(tmem + col_s(i), dq + (uint64_t)((bx * kQBox + kk * 32) >> 4),
                 dk + (uint64_t)((bx * kKVBox + kk * 32) >> 4), idesc_s, ks > 0 ? 1u : 0u);
        }
        tc_commit(smem_u32(&bars.s_full[i][st]));
      };
      // O_i (+)= P_i V of round r: P from TMEM (16 keys = 8 columns per MMA), V MN-major in shared memory.
      auto issue_pv = [&](int i, int r, bool first) {
        const int st = r % kStages;
        const uint64_t dv = dv0 + (uint64_t)((st * kKVBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < kBN / 16; ++ks)
          mma_ts(tmem + col_o(i, D), tmem + col_s(i) + ks * 8, dv + (uint64_t)((ks * 16 * 128) >> 4), idesc_o,
                 (ks > 0 || !first) ? 1u : 0u);
        tc_commit(smem_u32(&bars.o_done[i][st]));
      };
      // This warp's own wait for query tile i and the first K tile of item it (round r).
      auto inputs = [&](int i, int it, int r) -> bool {
        const bool there = mbar_spin_inl(smem_u32(&bars.q_full[i]), it & 1, abort_flag, p.err, 45 + i, kLimit) &&
                           mbar_spin_inl(smem_u32(&bars.k_full[r % kStages]), (r / kStages) & 1, abort_flag, p.err, 47,
                                         kLimit);
        return __all_sync(0xffffffffu, there);
      };
      // An item's first S_i, once per item: as a loop, which leaves the registers to the rounds' products.
      auto first_s = [&](int i, int r) {
        tc_fence_after();
        if (elect_one()) {
          const int st = r % kStages;
#pragma unroll 1
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ss(tmem + (uint32_t)(i * kBN), sdesc(sQ + i * kQBytes + (ks / 4) * kQBox + ks % 4 * 32, 16, 1024),
                   sdesc(sK0 + st * kKVBytes + (ks / 4) * kKVBox + ks % 4 * 32, 16, 1024), idesc_s, ks > 0 ? 1u : 0u);
          tc_commit(smem_u32(&bars.s_full[i][st]));
        }
        __syncwarp();
      };
      int rounds = 0;
      bool ok = true;
      for (int it = 0;; ++it) {
        const int n_kv = item_at(it);
        if (n_kv == 0) break;
        // Behind the item before's last products: its output takes the softmax warps longer than these scores.
        // (Tile 0's before tile 1's last product would hold that one up until the query tile is there.)
#pragma unroll 1
        for (int i = 0; i < kTiles; ++i) {
          ok = ok && inputs(i, it, rounds);
          if (ok) first_s(i, rounds);
        }
        for (int j = 0; j < n_kv; ++j) {
          const int r = rounds + j;
          const bool last = j + 1 == n_kv;
          // Tile i's P is in TMEM; this round's V and the item's next K are loaded (the waiter meets
          // tile 0's barrier).
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            __syncwarp();
            if (i == 0) {
              named_sync(kBarTile0, 192);
              ok = ok && s_round_ok[r & 1] != 0;
            } else {
              named_sync(kBarTile1, 160);
            }
            ok = ok && !*abort_flag;
            if (ok) {
              tc_fence_after();
              if (elect_one()) {
                issue_pv(i, r, j == 0);
                if (!last) issue_s(i, r + 1);
              }
              __syncwarp();
            }
          }
        }
        rounds += n_kv;
      }
      // All tensor-core work issued by this CTA completes before TMEM is freed.
      if (elect_one()) tc_commit(smem_u32(&bars.drain));
      __syncwarp();
      mbar_wait_inl(smem_u32(&bars.drain), 0, abort_flag, p.err, 49, false, kLimit);
    }
    // The two register regions end separately (no common tail after the branch): every warp
    // meets on named barrier 1 before warp 0 frees the tensor memory.
    __syncwarp();
    tc_fence_before();
    named_sync(kBarExit, kThreads);
    return;
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    pdl_wait();
    const int ti = warp / 4;  // this warpgroup's query tile
    const int row = threadIdx.x % kBM;
    const uint32_t lane_base = tmem + ((uint32_t)((warp % 4) * 32) << 16);
    int rounds = 0;
    bool ok = true;
    int n_kv = item_at(0);
    for (int it = 0; n_kv > 0; ++it) {
      // Position of this thread's row in the sequence; rows past its end repeat the last one and are
      // never stored.
      const int my_pos = min(items[it % kItems].t0 + ti * p.tq + (row >> p.lg), items[it % kItems].len - 1);
      float m_ref = -INFINITY, l = 0.0f;  // reference max (log2 units) that O_ti and l are scaled to
      auto wait_o = [&](int r, int site) -> bool {
        const bool w =
            mbar_spin_inl(smem_u32(&bars.o_done[ti][r % kStages]), (r / kStages) & 1, abort_flag, p.err, site, kLimit);
        return __all_sync(0xffffffffu, w);
      };
      // One key tile; false if a wait gave up (the abort flag is raised then).
      auto tile = [&](int j) -> bool {
        const int r = rounds + j;
        if (!__all_sync(0xffffffffu, mbar_spin_inl(smem_u32(&bars.s_full[ti][r % kStages]), (r / kStages) & 1,
                                                   abort_flag, p.err, 50 + ti, kLimit)))
          return false;
        tc_fence_after();
        uint32_t sv[kBN];  // this row's 128 scores
        {
          uint32_t(&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sv[0]);
          uint32_t(&s1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sv[32]);
          uint32_t(&s2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sv[64]);
          uint32_t(&s3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sv[96]);
          tmem_ld_x32_async(lane_base + col_s(ti), s0);
          tmem_ld_x32_async(lane_base + col_s(ti) + 32, s1);
          tmem_ld_x32_async(lane_base + col_s(ti) + 64, s2);
          tmem_ld_x32_async(lane_base + col_s(ti) + 96, s3);
          tmem_wait_ld(s0);
          tmem_wait_ld(s1);
          tmem_wait_ld(s2);
          tmem_wait_ld(s3);
        }
        const int lim = my_pos - j * kBN;  // columns c <= lim are visible to this row
        if (__any_sync(0xffffffffu, lim < kBN - 1)) {  // diagonal tiles only
          // by 32 columns: only those that a row of the warp does not see (its first row sees the fewest)
          const int first = __shfl_sync(0xffffffffu, lim, 0);
#pragma unroll
          for (int c0 = 0; c0 < kBN; c0 += 32) {
            if (first < c0 + 31)
#pragma unroll
              for (int c = c0; c < c0 + 32; ++c)
                if (c > lim) sv[c] = 0xff800000u;  // -inf
          }
        }
        // As in attention_pp.cu, tiles run against a reference and take their max only where their P
        // sum shows that the reference is too low. The first tile's reference is the max of its first
        // 32 columns (every row sees column 0): the rest is within 2^16 of it but for rare rows, which
        // the check finds.
        const uint32_t taddr_p = lane_base + col_s(ti);
        if (j == 0) {
          float tm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 32; c += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              tm[u] = max3(tm[u], __uint_as_float(sv[c + 2 * u]), __uint_as_float(sv[c + 2 * u + 1]));
          m_ref = fmaxf(fmaxf(tm[0], tm[1]), fmaxf(tm[2], tm[3])) * p.scale_log2;
        }
        bool move_ref = !__all_sync(0xffffffffu, m_ref != -INFINITY);
        float sum = 0.0f;
        if (!move_ref) {
          sum = softmax_p(sv, m_ref, p.scale_log2, taddr_p);
          move_ref = !__all_sync(0xffffffffu, sum <= kTileSumLimit);  // rare: the max jumped
        }
        if (move_ref) {
          // Four independent chains of three-input max.
          float tm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < kBN; c += 8) {
            tm[0] = max3(tm[0], __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            tm[1] = max3(tm[1], __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
            tm[2] = max3(tm[2], __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 5]));
            tm[3] = max3(tm[3], __uint_as_float(sv[c + 6]), __uint_as_float(sv[c + 7]));
          }
          const float mt = fmaxf(fmaxf(tm[0], tm[1]), fmaxf(tm[2], tm[3])) * p.scale_log2;
          const bool up = mt > m_ref + kRescaleThreshold;  // always, at a row's first tile
          if (__any_sync(0xffffffffu, up)) {
            const float alpha = up ? ex2(m_ref - mt) : 1.0f;  // 0 for a row that had nothing visible
            const bool scale_o = up && m_ref != -INFINITY;
            if (up) {
              l *= alpha;
              m_ref = mt;
            }
            // O_ti holds the sum through the tile before: wait for that product, then scale it.
            if (j > 0 && __any_sync(0xffffffffu, scale_o)) {
              if (!wait_o(r - 1, 52 + ti)) return false;
              tc_fence_after();
              const float a = scale_o ? alpha : 1.0f;
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tmem_ld_x32(lane_base + col_o(ti, D) + c0, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                tmem_st_x32(lane_base + col_o(ti, D) + c0, o);
              }
              tmem_st_wait();
            }
          }
          sum = softmax_p(sv, m_ref, p.scale_log2, taddr_p);  // these stores replace any earlier P
        }
        l += sum;
        tmem_st_wait();
        return true;
      };
      // Every softmax warp syncs once per key tile on its tile's named barrier, also after a failed
      // wait (then without work), so every round of the issuer and the waiter completes.
      for (int j = 0; j < n_kv; ++j) {
        if (ok) ok = tile(j);
        tc_fence_before();
        __syncwarp();
        if (ti == 0)
          named_sync(kBarTile0, 192);
        else
          named_sync(kBarTile1, 160);
      }
      rounds += n_kv;
      n_kv = item_at(it + 1);  // while the last product runs
      if (ok) ok = wait_o(rounds - 1, 54 + ti);
      // Epilogue: out = O_ti / l, each thread its row.
      if (__all_sync(0xffffffffu, ok && !*abort_flag)) {
        tc_fence_after();
        const float inv = 1.0f / l;
        const Item x = items[it % kItems];
        const bool fixed = x.fixed != 0;
        const uint32_t stage = sOut + (uint32_t)warp * kOutWarp;
        const int tokens = x.len - x.t0 - ti * p.tq;  // of this tile that are in the sequence (may be <= 0 or many)
        const bool whole = tokens >= ((warp % 4) * 32 + 32) >> p.lg;  // every row of this warp is
        const int token_bytes = p.hq * D * 2;
        uint8_t* dst = p.out + ((int64_t)(x.row0 + x.t0 + ti * p.tq) * p.hq + x.g * p.group) * (D * 2) + (lane & 7) * 16;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 64) {
          uint32_t o[64];
          uint32_t(&o0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&o[0]);
          uint32_t(&o1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&o[32]);
          tmem_ld_x32_async(lane_base + col_o(ti, D) + c0, o0);
          tmem_ld_x32_async(lane_base + col_o(ti, D) + c0 + 32, o1);
          tmem_wait_ld(o0);
          tmem_wait_ld(o1);
          if (fixed) {  // the values that were set to 0, of the keys that this row does see
            for (int key = hidden_from(x.t0); key <= my_pos; ++key) {
              const uint8_t* src = p.v + (((int64_t)(x.row0 + key) * p.hkv + x.g) * D + c0) * 2;
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                float f[8];
                unpack8(*reinterpret_cast<const uint4*>(src + q * 16), f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (!isfinite(f[e])) o[q * 8 + e] = __float_as_uint(__uint_as_float(o[q * 8 + e]) + f[e]);
              }
            }
            __syncwarp();  // the next load of TMEM is warp-aligned
          }
          // the rows staged before have been read
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[q * 8 + e]) * inv;
            const uint4 pk = pack8(f);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + (uint32_t)((q ^ (lane & 7)) * 16)),
                         "r"(pk.x), "r"(pk.y), "r"(pk.z), "r"(pk.w)
                         : "memory");
          }
          if (whole) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              asm volatile("cp.async.bulk.tensor.5d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4, %5}], [%6];" ::"l"(&tm_o),
                           "r"(0), "r"(0), "r"(x.row0 + x.t0 + ti * p.tq + (((warp % 4) * 32) >> p.lg)), "r"(c0 / 64), "r"(x.g), "r"(stage)
                           : "memory");
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            __syncwarp();
            continue;
          }
          __syncwarp();
          // 8 lanes per row: 128 bytes of four rows per instruction, all loads first
          uint4 pk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rl = 4 * i + lane / 8;  // row in the warp
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(pk[i].x), "=r"(pk[i].y), "=r"(pk[i].z), "=r"(pk[i].w)
                         : "r"(stage + rl * 128 + (uint32_t)(((lane & 7) ^ (rl & 7)) * 16)));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rt = (warp % 4) * 32 + 4 * i + lane / 8;  // row in the tile
            if ((rt >> p.lg) < tokens)
              *reinterpret_cast<uint4*>(dst + c0 * 2 + (rt >> p.lg) * token_bytes + (rt & (p.group - 1)) * (D * 2)) = pk[i];
          }
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // before shared memory goes
    __syncwarp();
    tc_fence_before();
    named_sync(kBarExit, kThreads);
    if (warp == 0) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
  }
}

template <int D, bool PROBE = false>
cudaError_t launch_prompt_t(const void* q, const void* k, const void* v, const int32_t* cu, int32_t n_seqs,
                            int32_t n_rows, int32_t hq, int32_t hkv, float scale, void* out, int32_t* err,
                            cudaStream_t s) {
  const int group = hq / hkv;
  const int tq = kBM / group;
  // The register split: the block is launched with numRegs per thread and setmaxnreg moves them
  // between the warpgroups; a build with fewer than the split needs would wait forever in
  // setmaxnreg.inc, so it is never launched.
  static std::atomic<int> known{-1};  // (threads may make their first calls at once)
  int regs = known.load(std::memory_order_relaxed);
  if (regs < 0) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, prompt_attention_kernel<D, PROBE>);
    if (e != cudaSuccess) return e;
    regs = a.numRegs;
    known.store(regs, std::memory_order_relaxed);
  }
  if (regs * kThreads < kTiles * kSoftmaxThreads * kSoftmaxRegs + kSoftmaxThreads * kOtherRegs)
    return cudaErrorNotSupported;
  CUtensorMap tq_map, tk_map, tv_map, to_map;
  // Columns in blocks of 64 (128 bytes, the swizzle's span) as a dimension of their own, so that one copy
  // brings a tile's blocks one behind the other: [64, heads of g, tokens, block, g] and [64, keys, block, g].
  const cuuint64_t qd[5] = {64, (cuuint64_t)group, (cuuint64_t)n_rows, D / 64, (cuuint64_t)hkv};
  const cuuint64_t qs[4] = {(cuuint64_t)D * 2, (cuuint64_t)hq * D * 2, 128, (cuuint64_t)group * D * 2};
  const cuuint32_t qb[5] = {64, (cuuint32_t)group, (cuuint32_t)tq, D / 64, 1};
  const cuuint32_t ob[5] = {64, (cuuint32_t)group, (cuuint32_t)(32 / group), 1, 1};  // the rows of a softmax warp
  const cuuint64_t kd[4] = {64, (cuuint64_t)n_rows, D / 64, (cuuint64_t)hkv};
  const cuuint64_t ks[3] = {(cuuint64_t)hkv * D * 2, 128, (cuuint64_t)D * 2};
  const cuuint32_t kbx[4] = {64, (cuuint32_t)kBN, D / 64, 1};
  if (!encode_map(&tq_map, q, 5, qd, qs, qb) || !encode_map(&tk_map, k, 4, kd, ks, kbx) ||
      !encode_map(&tv_map, v, 4, kd, ks, kbx) || !encode_map(&to_map, out, 5, qd, qs, ob))
    return cudaErrorInvalidValue;
  PromptParams p;
  p.v = static_cast<const uint8_t*>(v);
  p.cu = cu;
  p.out = static_cast<uint8_t*>(out);
  p.n_seqs = n_seqs;
  p.n_rows = n_rows;
  p.hq = hq;
  p.hkv = hkv;
  p.group = group;
  p.lg = 31 - __builtin_clz(group);
  p.tq = tq;
  const int64_t seq_bytes = (int64_t)n_rows / n_seqs * hkv * D * 4 + 1;  // K and V of a sequence of the mean length
  p.seqs_per_group = (int)std::min<int64_t>(std::max<int64_t>(kGroupBytes / seq_bytes, 1), 32);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.err = err;
  const size_t smem = 1024 + (size_t)(kTiles * kBM + 2 * kStages * kBN) * D * 2 + 2 * kSoftmaxThreads / 32 * kOutWarp;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = set_smem_limit_once(prompt_attention_kernel<D, PROBE>, (int)smem, configured);
  if (e != cudaSuccess) return e;
  const int64_t most = prompt_items(n_seqs, n_rows, hq, hkv);
  return launch_pdl(prompt_attention_kernel<D, PROBE>, dim3((unsigned)most), dim3(kThreads), smem, s,
                    tq_map, tk_map, tv_map, to_map, p);
}

}  // namespace

int64_t prompt_items(int32_t n_seqs, int32_t n_rows, int32_t hq, int32_t hkv) {
  const int64_t per = kTiles * (kBM / (hq / hkv));  // tokens per item; each sequence may end inside one
  return ((int64_t)n_rows / per + n_seqs) * hkv;
}

cudaError_t launch_prompt_attention(const void* q, const void* k, const void* v, const int32_t* cu, int32_t n_seqs,
                                    int32_t n_rows, int32_t hq, int32_t hkv, int32_t head_dim, float scale, void* out,
                                    int32_t* err, cudaStream_t s) {
  if (n_seqs <= 0 || n_rows <= 0) return cudaSuccess;
  if (head_dim == 128)
    return launch_prompt_t<128>(q, k, v, cu, n_seqs, n_rows, hq, hkv, scale, out, err, s);
  if (head_dim == 64) return launch_prompt_t<64>(q, k, v, cu, n_seqs, n_rows, hq, hkv, scale, out, err, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_prompt_timeout_probe(const void* q, const void* k, const void* v, const int32_t* cu, int32_t n_seqs,
                                        int32_t n_rows, int32_t hq, int32_t hkv, float scale, void* out, int32_t* err,
                                        cudaStream_t s) {
  if (n_seqs <= 0 || n_rows <= 0) return cudaSuccess;
  return launch_prompt_t<128, true>(q, k, v, cu, n_seqs, n_rows, hq, hkv, scale, out, err, s);
}

}  // namespace cb
