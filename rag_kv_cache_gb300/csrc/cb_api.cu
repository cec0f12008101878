// C ABI of the blend (declared in include/cacheblend.h): host-side argument
// checks, the plan (RoPE table, device error word, scratch), and the
// per-layer driver that enqueues the kernels of one layer on the caller's
// stream without any host synchronisation.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <string>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "../../include/cacheblend.h"
#include "common.cuh"
#include "kernels.h"

static_assert(CB_PAGE_TABLES_MAX_SEQS == cb::kPageTablesMaxSeqs, "page table limit");

// Streams that run consecutive layers' attention in cb_blend_request (the caller's stream and
// CB_ATTN_STREAMS - 1 of the plan's): a layer's attention overlaps the tails of the layers before it.
#ifndef CB_ATTN_STREAMS
#define CB_ATTN_STREAMS 2
#endif
constexpr int kAttnStreams = CB_ATTN_STREAMS;
static_assert(kAttnStreams >= 1 && kAttnStreams <= 8, "attention streams");

struct cb_plan {
  cb_config cfg;
  int device;
  int32_t n_ctx;
  int32_t n_tokens;
  float2* rope_tab;  // [n_tokens][head_dim / 2]
  int32_t* err;      // [0] flags, [1] first offending index (-1 = none)
  cudaStream_t aux_stream;  // cb_blend_request: every layer's deviation, top-k and fuse (with the query encoding)
  cudaStream_t aux_attn[kAttnStreams];  // cb_blend_request: attention of layer l on stream (l - 1) % kAttnStreams
                                        // ([0] unused: that one is the caller's stream)
  cudaEvent_t ev_fork, ev_ready, ev_join;
  cb::DecodeScratch decode;  // cb_decode_attention's split partials and ticket counters
  cb::Kv4Scratch kv4;        // cb_kv4_decode_attention's partials and ticket counters
  cb::Kv4ChunkScratch chunk; // cb_kv4_chunk_attention's partials
};

namespace {

// Every entry point is one NVTX range named after it, so a profile of a request reads by call
// (a push and a pop through an unset function pointer when no tool collects NVTX).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};
#define CB_NVTX_RANGE() const NvtxRange cb_nvtx_range_(__func__)

thread_local std::string g_last_error = "no error";

cb_status fail(cb_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

cb_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return CB_OK;
  return fail(CB_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

cb_status need_tensor(const void* p, const char* name) {
  if (p == nullptr) return fail(CB_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(CB_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return CB_OK;
}

cb_status need_ptr(const void* p, const char* name) {
  if (p == nullptr) return fail(CB_ERR_INVALID_ARG, "%s is NULL", name);
  return CB_OK;
}

cb_status need_words(const void* p, const char* name) {
  if (p == nullptr) return fail(CB_ERR_INVALID_ARG, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return fail(CB_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
  return CB_OK;
}

#define CB_TRY(expr)                  \
  do {                                \
    const cb_status _s = (expr);      \
    if (_s != CB_OK) return _s;       \
  } while (0)

cb_status check_plan(const cb_plan* plan) {
  if (plan == nullptr) return fail(CB_ERR_INVALID_ARG, "plan is NULL");
  return CB_OK;
}

// The serving calls check that the plan's device is the current one: its scratch and error word live there.
cb_status check_device(const cb_plan* plan) {
  int dev = -1;
  CB_TRY(cuda_status(cudaGetDevice(&dev), "cudaGetDevice"));
  if (dev != plan->device)
    return fail(CB_ERR_INVALID_ARG, "the plan belongs to device %d, the current device is %d", plan->device, dev);
  return CB_OK;
}

// Shape of a 4-bit cache: pages of whole 16-token records, slots that fit an int32.
cb_status check_kv4_cache(int32_t n_pages, int32_t page_size) {
  if (n_pages < 0) return fail(CB_ERR_INVALID_ARG, "n_pages < 0");
  if (page_size <= 0 || page_size % 16 != 0 || page_size > CB_KV4_MAX_PAGE)
    return fail(CB_ERR_INVALID_ARG, "page_size %d: a multiple of 16 up to %d is required", page_size, CB_KV4_MAX_PAGE);
  if ((int64_t)n_pages * page_size > 0x7fffffffll)
    return fail(CB_ERR_INVALID_ARG, "n_pages * page_size above 2^31 - 1");
  return CB_OK;
}

// A buffer of a call, for the check that what it writes lies apart from what it reads.
struct Span {
  const void* at;
  int64_t bytes;
  const char* name;
};
bool meet(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at != nullptr && b.at != nullptr && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes &&
         y < x + (uintptr_t)a.bytes;
}
// No output may overlap an input or another output, not in part either.
cb_status check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meet(*o, i)) return fail(CB_ERR_INVALID_ARG, "%s overlaps %s", o->name, i.name);
    for (const Span* other = outs.begin(); other != o; ++other)
      if (meet(*o, *other)) return fail(CB_ERR_INVALID_ARG, "%s overlaps %s", o->name, other->name);
  }
  return CB_OK;
}

Span cache_span(const cb_plan* plan, const void* cache, int32_t n_pages, int32_t page_size) {
  return Span{cache, (int64_t)n_pages * plan->cfg.hkv * (page_size / 16 * 18 * plan->cfg.head_dim), "cache"};
}

cb::RopeTable table(const cb_plan* p) { return cb::RopeTable{p->rope_tab, p->n_tokens}; }

int32_t k_for_ratio(int32_t r_pct, int32_t n_ctx) {
  return static_cast<int32_t>((static_cast<int64_t>(r_pct) * n_ctx) / 100);
}

}  // namespace

namespace cb {
cb_status set_last_error(cb_status s, const char* msg) { return fail(s, "%s", msg); }
}  // namespace cb

extern "C" {

int32_t cb_version(void) { return 100; }

const char* cb_last_error_string(void) { return g_last_error.c_str(); }

cb_status cb_plan_create(const cb_config* cfg, cb_plan** out) {
  CB_NVTX_RANGE();
  CB_TRY(need_ptr(cfg, "cfg"));
  CB_TRY(need_ptr(out, "out"));
  *out = nullptr;
  const cb_config& c = *cfg;
  if (c.n_chunks < 0 || c.chunk_len <= 0 || c.n_suffix < 0)
    return fail(CB_ERR_INVALID_ARG, "n_chunks >= 0, chunk_len > 0 and n_suffix >= 0 required");
  const int64_t n_tokens = (int64_t)c.n_chunks * c.chunk_len + c.n_suffix;
  if (n_tokens <= 0 || n_tokens > (1 << 24)) return fail(CB_ERR_INVALID_ARG, "n_tokens must be in [1, 2^24]");
  if (c.hkv <= 0 || c.hq <= 0 || c.hq % c.hkv != 0)
    return fail(CB_ERR_INVALID_ARG, "hq must be a positive multiple of hkv");
  const int group = c.hq / c.hkv;
  if (group != 1 && group != 2 && group != 4 && group != 8 && group != 16)
    return fail(CB_ERR_UNSUPPORTED, "hq / hkv = %d; supported: 1, 2, 4, 8, 16", group);
  if (c.head_dim != 64 && c.head_dim != 128) return fail(CB_ERR_UNSUPPORTED, "head_dim %d; supported: 64, 128", c.head_dim);
  if (c.hkv * c.head_dim > 2048) return fail(CB_ERR_UNSUPPORTED, "hkv * head_dim above 2048");
  if (!(c.rope_theta > 1.0) || !std::isfinite(c.rope_theta)) return fail(CB_ERR_INVALID_ARG, "rope_theta must be > 1");
  if (c.rope_style != CB_ROPE_HALF && c.rope_style != CB_ROPE_INTERLEAVED)
    return fail(CB_ERR_INVALID_ARG, "unknown rope_style %d", c.rope_style);
  if (c.r1_pct < 0 || c.r1_pct > 100 || c.r2_pct < 0 || c.r2_pct > c.r1_pct)
    return fail(CB_ERR_INVALID_ARG, "need 0 <= r2_pct <= r1_pct <= 100");
  if (c.deviation != CB_DEV_V && c.deviation != CB_DEV_KV)
    return fail(CB_ERR_INVALID_ARG, "unknown deviation %d", c.deviation);
  if (c.filter != CB_FILTER_KEEP && c.filter != CB_FILTER_RESELECT)
    return fail(CB_ERR_INVALID_ARG, "unknown filter %d", c.filter);

  cb_plan* p = new cb_plan();
  p->cfg = c;
  p->n_ctx = c.n_chunks * c.chunk_len;
  p->n_tokens = (int32_t)n_tokens;
  cudaError_t e = cudaGetDevice(&p->device);
  if (e == cudaSuccess) e = cudaMalloc(&p->rope_tab, sizeof(float2) * (size_t)n_tokens * (c.head_dim / 2));
  if (e == cudaSuccess) e = cudaMalloc(&p->err, 2 * sizeof(int32_t));
  if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&p->aux_stream, cudaStreamNonBlocking);
  for (int a = 1; a < kAttnStreams && e == cudaSuccess; ++a)
    e = cudaStreamCreateWithFlags(&p->aux_attn[a], cudaStreamNonBlocking);
  if (e == cudaSuccess) e = cudaEventCreateWithFlags(&p->ev_fork, cudaEventDisableTiming);
  if (e == cudaSuccess) e = cudaEventCreateWithFlags(&p->ev_ready, cudaEventDisableTiming);
  if (e == cudaSuccess) e = cudaEventCreateWithFlags(&p->ev_join, cudaEventDisableTiming);
  if (e == cudaSuccess) {
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, p->device);
    p->decode.sms = sms > 0 ? sms : 1;
  }
  const size_t dec_units = (size_t)c.hq * cb::decode_max_splits();  // (kv head, split, q head) triples
  if (e == cudaSuccess) e = cudaMalloc(&p->decode.part_o, sizeof(float) * dec_units * c.head_dim);
  if (e == cudaSuccess) e = cudaMalloc(&p->decode.part_ml, sizeof(float2) * dec_units);
  if (e == cudaSuccess) e = cudaMalloc(&p->decode.tickets, sizeof(int32_t) * c.hkv);
  if (e == cudaSuccess) e = cudaMemset(p->decode.tickets, 0, sizeof(int32_t) * c.hkv);

  p->kv4.sms = p->decode.sms;
  const size_t kv4_units = (size_t)p->kv4.sms * 2 * cb::kKv4MaxGroup;
  if (e == cudaSuccess) e = cudaMalloc(&p->kv4.part_o, sizeof(float) * kv4_units * c.head_dim);
  if (e == cudaSuccess) e = cudaMalloc(&p->kv4.part_ml, sizeof(float2) * kv4_units);
  if (e == cudaSuccess) e = cudaMalloc(&p->kv4.tickets, sizeof(int32_t) * p->kv4.sms);
  if (e == cudaSuccess) e = cudaMemset(p->kv4.tickets, 0, sizeof(int32_t) * p->kv4.sms);

  p->chunk.sms = p->decode.sms;
  const size_t chunk_rows = cb::kv4_chunk_part_rows(p->chunk.sms);
  if (e == cudaSuccess) e = cudaMalloc(&p->chunk.part_o, sizeof(float) * chunk_rows * c.head_dim);
  if (e == cudaSuccess) e = cudaMalloc(&p->chunk.part_ml, sizeof(float2) * chunk_rows);
  if (e == cudaSuccess) e = cudaMalloc(&p->chunk.parts, cb::kv4_chunk_parts_bytes(p->chunk.sms));
  if (e == cudaSuccess) e = cudaMalloc(&p->chunk.own, sizeof(float2) * cb::kv4_chunk_own_keys(p->chunk.sms));
  p->chunk.few.sms = p->chunk.sms;
  if (e == cudaSuccess) e = cudaMalloc(&p->chunk.few.part_o, sizeof(float) * kv4_units * c.head_dim);
  if (e == cudaSuccess) e = cudaMalloc(&p->chunk.few.part_ml, sizeof(float2) * kv4_units);
  if (e == cudaSuccess) e = cudaMalloc(&p->chunk.few.tickets, sizeof(int32_t) * p->chunk.sms);
  if (e == cudaSuccess) e = cudaMemset(p->chunk.few.tickets, 0, sizeof(int32_t) * p->chunk.sms);

  if (e == cudaSuccess) {
    const int32_t init[2] = {0, -1};
    e = cudaMemcpy(p->err, init, sizeof(init), cudaMemcpyHostToDevice);
  }
  if (e == cudaSuccess) {
    // (cos, sin) of p * theta^(-2j/D): the exponent (-2j)/D, theta^x, the angle and cos / sin in
    // fp64 with the C library's routines, then rounded to fp32.
    const int half = c.head_dim / 2;
    std::vector<double> inv(half);
    for (int j = 0; j < half; ++j) inv[j] = std::pow(c.rope_theta, (-2.0 * j) / c.head_dim);
    std::vector<float2> tab((size_t)n_tokens * half);
    for (int64_t pos = 0; pos < n_tokens; ++pos)
      for (int j = 0; j < half; ++j) {
        const double a = (double)pos * inv[j];
        tab[(size_t)pos * half + j] = make_float2((float)std::cos(a), (float)std::sin(a));
      }
    e = cudaMemcpy(p->rope_tab, tab.data(), sizeof(float2) * tab.size(), cudaMemcpyHostToDevice);
  }
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cb_plan_destroy(p);
    return cuda_status(e, "cb_plan_create");
  }
  *out = p;
  return CB_OK;
}

cb_status cb_plan_destroy(cb_plan* plan) {
  CB_NVTX_RANGE();
  if (plan == nullptr) return CB_OK;
  cudaDeviceSynchronize();
  cudaFree(plan->rope_tab);
  cudaFree(plan->err);
  cudaFree(plan->decode.part_o);
  cudaFree(plan->decode.part_ml);
  cudaFree(plan->decode.tickets);
  cudaFree(plan->kv4.part_o);
  cudaFree(plan->kv4.part_ml);
  cudaFree(plan->kv4.tickets);
  cudaFree(plan->chunk.part_o);
  cudaFree(plan->chunk.part_ml);
  cudaFree(plan->chunk.parts);
  cudaFree(plan->chunk.own);
  cudaFree(plan->chunk.few.part_o);
  cudaFree(plan->chunk.few.part_ml);
  cudaFree(plan->chunk.few.tickets);
  if (plan->aux_stream) cudaStreamDestroy(plan->aux_stream);
  for (int a = 1; a < kAttnStreams; ++a)
    if (plan->aux_attn[a]) cudaStreamDestroy(plan->aux_attn[a]);
  if (plan->ev_fork) cudaEventDestroy(plan->ev_fork);
  if (plan->ev_ready) cudaEventDestroy(plan->ev_ready);
  if (plan->ev_join) cudaEventDestroy(plan->ev_join);
  delete plan;
  return CB_OK;
}

cb_status cb_layer_sizes(const cb_plan* plan, int32_t layer, int32_t* n_cand, int32_t* k, int32_t* mq,
                         int32_t* selects) {
  CB_TRY(check_plan(plan));
  if (layer < 1) return fail(CB_ERR_INVALID_ARG, "layer is 1-based, got %d", layer);
  const int32_t k1 = k_for_ratio(plan->cfg.r1_pct, plan->n_ctx);
  const int32_t k2 = k_for_ratio(plan->cfg.r2_pct, plan->n_ctx);
  int32_t c, kk, sel;
  if (layer == 1) {
    c = plan->n_ctx, kk = k1, sel = 1;
  } else if (layer == 2) {
    c = k1, kk = k2, sel = 1;
  } else if (plan->cfg.filter == CB_FILTER_RESELECT) {
    c = k1, kk = k2, sel = 1;
  } else {
    c = k2, kk = k2, sel = 0;
  }
  if (n_cand) *n_cand = c;
  if (k) *k = kk;
  if (mq) *mq = kk + plan->cfg.n_suffix;
  if (selects) *selects = sel;
  return CB_OK;
}

cb_status cb_rope_rerotate(cb_plan* plan, void* out, const void* x, const int32_t* in_rows,
                           const int32_t* out_rows, const int32_t* pos_from, const int32_t* pos_to, int32_t n,
                           int32_t n_heads, int32_t x_rows, int32_t out_rows_total, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (n < 0 || n_heads <= 0 || x_rows < 0 || out_rows_total < 0)
    return fail(CB_ERR_INVALID_ARG, "negative size or n_heads <= 0");
  if (n == 0) return CB_OK;
  CB_TRY(need_tensor(out, "out"));
  CB_TRY(need_tensor(x, "x"));
  CB_TRY(need_ptr(pos_to, "pos_to"));
  if (out == x && (in_rows != nullptr || out_rows != nullptr))
    return fail(CB_ERR_INVALID_ARG, "in-place rotation needs in_rows == out_rows == NULL");
  const cb::RowMap im{in_rows, n, 0, x_rows};
  const cb::RowMap om{out_rows, n, 0, out_rows_total};
  return cuda_status(cb::launch_rope_rows(out, x, im, om, pos_from, pos_to, nullptr, n, n_heads,
                                          plan->cfg.head_dim, plan->cfg.rope_style, table(plan), plan->err,
                                          static_cast<cudaStream_t>(stream)),
                     "cb_rope_rerotate");
}

cb_status cb_kv_deviation(cb_plan* plan, const void* v_new, const void* v_old, const int32_t* cand, int32_t m,
                          float* dev, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (m < 0) return fail(CB_ERR_INVALID_ARG, "m < 0");
  if (m == 0) return CB_OK;
  if (cand == nullptr && m > plan->n_ctx) return fail(CB_ERR_INVALID_ARG, "m > n_ctx without a candidate list");
  CB_TRY(need_tensor(v_new, "v_new"));
  CB_TRY(need_tensor(v_old, "v_old"));
  CB_TRY(need_ptr(dev, "dev"));
  return cuda_status(cb::launch_kv_deviation(nullptr, nullptr, v_new, v_old, cand, m, plan->n_ctx, plan->cfg.hkv,
                                             plan->cfg.head_dim, 1, 0, table(plan), dev, plan->err,
                                             static_cast<cudaStream_t>(stream)),
                     "cb_kv_deviation");
}

cb_status cb_kv_deviation_kv(cb_plan* plan, const void* k_new, const void* k_old, const void* v_new,
                             const void* v_old, const int32_t* cand, int32_t m, float* dev, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (m < 0) return fail(CB_ERR_INVALID_ARG, "m < 0");
  if (m == 0) return CB_OK;
  if (cand == nullptr && m > plan->n_ctx) return fail(CB_ERR_INVALID_ARG, "m > n_ctx without a candidate list");
  CB_TRY(need_tensor(k_new, "k_new"));
  CB_TRY(need_tensor(k_old, "k_old"));
  CB_TRY(need_tensor(v_new, "v_new"));
  CB_TRY(need_tensor(v_old, "v_old"));
  CB_TRY(need_ptr(dev, "dev"));
  const auto& c = plan->cfg;
  return cuda_status(cb::launch_kv_deviation(k_new, k_old, v_new, v_old, cand, m, plan->n_ctx, c.hkv, c.head_dim,
                                             c.chunk_len, c.rope_style, table(plan), dev, plan->err,
                                             static_cast<cudaStream_t>(stream)),
                     "cb_kv_deviation_kv");
}

cb_status cb_hkvd_topk(cb_plan* plan, const float* dev, const int32_t* cand, int32_t m, int32_t k,
                       int32_t* sel_tok, int32_t* sel_row, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (m < 0 || k < 0 || k > m) return fail(CB_ERR_INVALID_ARG, "need 0 <= k <= m (k=%d, m=%d)", k, m);
  if (k == 0) return CB_OK;
  CB_TRY(need_ptr(dev, "dev"));
  CB_TRY(need_ptr(sel_tok, "sel_tok"));
  CB_TRY(need_ptr(sel_row, "sel_row"));
  return cuda_status(cb::launch_hkvd_topk(dev, cand, m, k, sel_tok, sel_row, plan->err,
                                          static_cast<cudaStream_t>(stream)),
                     "cb_hkvd_topk");
}

cb_status cb_fuse_scatter(cb_plan* plan, void* k_fused, void* v_fused, const void* k_new, const void* v_new,
                          const int32_t* sel_tok, int32_t k, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (k < 0 || k > plan->n_ctx) return fail(CB_ERR_INVALID_ARG, "need 0 <= k <= n_ctx");
  if (k + plan->cfg.n_suffix == 0) return CB_OK;
  CB_TRY(need_tensor(k_fused, "k_fused"));
  CB_TRY(need_tensor(v_fused, "v_fused"));
  CB_TRY(need_tensor(k_new, "k_new"));
  CB_TRY(need_tensor(v_new, "v_new"));
  if (k > 0) CB_TRY(need_ptr(sel_tok, "sel_tok"));
  return cuda_status(cb::launch_fuse_scatter(k_fused, v_fused, k_new, v_new, sel_tok, k, plan->n_ctx,
                                             plan->n_tokens, plan->cfg.hkv, plan->cfg.head_dim,
                                             plan->cfg.rope_style, table(plan), plan->err,
                                             static_cast<cudaStream_t>(stream)),
                     "cb_fuse_scatter");
}

cb_status cb_hkvd_attention(cb_plan* plan, const void* q, const int32_t* q_pos, int32_t mq, const void* k,
                            const void* v, int32_t n_keys, float scale, void* out, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (mq < 0 || n_keys < 0) return fail(CB_ERR_INVALID_ARG, "negative size");
  if (mq == 0) return CB_OK;
  if (n_keys == 0) return fail(CB_ERR_INVALID_ARG, "n_keys == 0 with queries to answer");
  CB_TRY(need_tensor(q, "q"));
  CB_TRY(need_ptr(q_pos, "q_pos"));
  CB_TRY(need_tensor(k, "k"));
  CB_TRY(need_tensor(v, "v"));
  CB_TRY(need_tensor(out, "out"));
  if (!(scale > 0.0f)) scale = 1.0f / std::sqrt((float)plan->cfg.head_dim);
  const cb::QueryPositions qp{q_pos, mq, 0, true};
  return cuda_status(cb::launch_hkvd_attention(q, qp, mq, k, v, n_keys, plan->cfg.hq, plan->cfg.hkv,
                                               plan->cfg.head_dim, scale, out, plan->err,
                                               static_cast<cudaStream_t>(stream)),
                     "cb_hkvd_attention");
}

int32_t cb_attention_uses_paired_tiles(const cb_plan* plan, int32_t mq) {
  if (plan == nullptr) return 0;
  return cb::attention_pp_eligible(mq, plan->cfg.hq, plan->cfg.hkv, plan->cfg.head_dim) ? 1 : 0;
}

cb_status cb_test_attention_wait_timeout(cb_plan* plan, const void* q, const int32_t* q_pos, int32_t mq,
                                         const void* k, const void* v, int32_t n_keys, void* out, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (plan->cfg.head_dim != 128) return fail(CB_ERR_UNSUPPORTED, "the wait-timeout probe needs head_dim 128");
  if (mq <= 0 || n_keys <= 128) return fail(CB_ERR_INVALID_ARG, "the wait-timeout probe needs mq > 0, n_keys > 128");
  CB_TRY(need_tensor(q, "q"));
  CB_TRY(need_ptr(q_pos, "q_pos"));
  CB_TRY(need_tensor(k, "k"));
  CB_TRY(need_tensor(v, "v"));
  CB_TRY(need_tensor(out, "out"));
  const cb::QueryPositions qp{q_pos, mq, 0, true};
  return cuda_status(cb::launch_attention_timeout_probe(q, qp, mq, k, v, n_keys, plan->cfg.hq, plan->cfg.hkv,
                                                        1.0f / std::sqrt(128.0f), out, plan->err,
                                                        static_cast<cudaStream_t>(stream)),
                     "cb_test_attention_wait_timeout");
}

cb_status cb_test_decode_wait_timeout(cb_plan* plan, const void* q, const void* k, const void* v, int32_t n_keys,
                                      void* out, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (plan->cfg.head_dim != 128) return fail(CB_ERR_UNSUPPORTED, "the wait-timeout probe needs head_dim 128");
  if (n_keys <= 128) return fail(CB_ERR_INVALID_ARG, "the wait-timeout probe needs n_keys > 128");
  CB_TRY(need_tensor(q, "q"));
  CB_TRY(need_tensor(k, "k"));
  CB_TRY(need_tensor(v, "v"));
  CB_TRY(need_tensor(out, "out"));
  const auto& c = plan->cfg;
  return cuda_status(cb::launch_decode_timeout_probe(q, k, v, n_keys, c.hq, c.hkv, 1.0f / std::sqrt(128.0f), out,
                                                     plan->decode, plan->err, static_cast<cudaStream_t>(stream)),
                     "cb_test_decode_wait_timeout");
}

cb_status cb_test_projection_wait_timeout(cb_plan* plan, const void* x, int32_t d_model, int32_t m,
                                          const void* w_qkv, void* q, void* k, void* v, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (plan->cfg.head_dim != 128) return fail(CB_ERR_UNSUPPORTED, "the wait-timeout probe needs head_dim 128");
  if (m <= 0 || m > plan->n_tokens) return fail(CB_ERR_INVALID_ARG, "the wait-timeout probe needs 0 < m <= n_tokens");
  if (d_model < 128 || d_model % 64 != 0)
    return fail(CB_ERR_INVALID_ARG, "the wait-timeout probe needs d_model >= 128, a multiple of 64");
  CB_TRY(need_tensor(x, "x"));
  CB_TRY(need_tensor(w_qkv, "w_qkv"));
  CB_TRY(need_tensor(q, "q"));
  CB_TRY(need_tensor(k, "k"));
  CB_TRY(need_tensor(v, "v"));
  const auto& c = plan->cfg;
  return cuda_status(cb::launch_projection_timeout_probe(x, d_model, m, w_qkv, plan->n_tokens, c.hq, c.hkv, q, k, v,
                                                         plan->err, static_cast<cudaStream_t>(stream)),
                     "cb_test_projection_wait_timeout");
}

cb_status cb_attention_sparsity(cb_plan* plan, const void* q, const int32_t* q_pos, int32_t mq, const void* k,
                                const void* v, int32_t n_keys, float scale, float eps, void* out, void* row_stats,
                                int32_t* counts, uint64_t* total, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (mq < 0 || n_keys < 0) return fail(CB_ERR_INVALID_ARG, "negative size");
  if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(CB_ERR_INVALID_ARG, "eps must be positive and finite");
  CB_TRY(need_ptr(total, "total"));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (mq == 0) return cuda_status(cudaMemsetAsync(total, 0, sizeof(uint64_t), s), "cb_attention_sparsity");
  if (n_keys == 0) return fail(CB_ERR_INVALID_ARG, "n_keys == 0 with queries to answer");
  CB_TRY(need_tensor(q, "q"));
  CB_TRY(need_ptr(q_pos, "q_pos"));
  CB_TRY(need_tensor(k, "k"));
  CB_TRY(need_tensor(v, "v"));
  CB_TRY(need_tensor(out, "out"));
  CB_TRY(need_tensor(row_stats, "row_stats"));
  CB_TRY(need_ptr(counts, "counts"));
  const auto& c = plan->cfg;
  if (!(scale > 0.0f)) scale = 1.0f / std::sqrt((float)c.head_dim);
  const cb::QueryPositions qp{q_pos, mq, 0, true};
  cb::AttentionDiag first;  // pass 1: the attention and each row's (max, sum)
  first.row_stats = static_cast<float2*>(row_stats);
  CB_TRY(cuda_status(cb::launch_hkvd_attention(q, qp, mq, k, v, n_keys, c.hq, c.hkv, c.head_dim, scale, out, plan->err,
                                               s, first),
                     "cb_attention_sparsity (statistics pass)"));
  cb::AttentionDiag second;  // pass 2: the same scores against each row's threshold
  second.count_stats = static_cast<const float2*>(row_stats);
  second.log2_eps = std::log2(eps);
  second.counts = counts;
  CB_TRY(cuda_status(cb::launch_hkvd_attention(q, qp, mq, k, v, n_keys, c.hq, c.hkv, c.head_dim, scale, out, plan->err,
                                               s, second),
                     "cb_attention_sparsity (counting pass)"));
  return cuda_status(cb::launch_sum_counts(counts, (int64_t)mq * c.hq, reinterpret_cast<unsigned long long*>(total), s),
                     "cb_attention_sparsity (sum)");
}

cb_status cb_output_deviation(cb_plan* plan, const void* o, const void* o_ref, int32_t rows, double* sums,
                              void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (rows < 0) return fail(CB_ERR_INVALID_ARG, "rows < 0");
  CB_TRY(need_ptr(sums, "sums"));
  if (rows > 0) {
    CB_TRY(need_tensor(o, "o"));
    CB_TRY(need_tensor(o_ref, "o_ref"));
  }
  const int64_t n = (int64_t)rows * plan->cfg.hq * plan->cfg.head_dim;
  return cuda_status(cb::launch_output_deviation(o, o_ref, n, sums, static_cast<cudaStream_t>(stream)),
                     "cb_output_deviation");
}

static cb_status qkv_projection(const char* fn, cb_plan* plan, const void* x, int32_t x_rows, int32_t d_model,
                                const int32_t* x_index, const int32_t* tokens, int32_t m, const void* w_qkv,
                                int32_t encode, void* x_gathered, void* q, void* k, void* v, void* stream) {
  CB_TRY(check_plan(plan));
  if (m < 0 || x_rows < 0) return fail(CB_ERR_INVALID_ARG, "negative size");
  if (m == 0) return CB_OK;
  if (!cb::qkv_projection_supported(d_model))
    return fail(CB_ERR_UNSUPPORTED, "d_model %d: a positive multiple of 64 is required", d_model);
  if (x_index == nullptr && m > x_rows) return fail(CB_ERR_INVALID_ARG, "m > x_rows without an index list");
  if (tokens == nullptr && m > plan->n_tokens) return fail(CB_ERR_INVALID_ARG, "m > n_tokens without a token list");
  CB_TRY(need_tensor(x, "x"));
  CB_TRY(need_tensor(w_qkv, "w_qkv"));
  CB_TRY(need_tensor(q, "q"));
  CB_TRY(need_tensor(k, "k"));
  CB_TRY(need_tensor(v, "v"));
  if (x_index != nullptr) CB_TRY(need_tensor(x_gathered, "x_gathered"));
  const auto& c = plan->cfg;
  return cuda_status(cb::launch_qkv_projection(x, x_rows, d_model, x_index, tokens, m, x_gathered, w_qkv,
                                               plan->n_tokens, c.hq, c.hkv, c.head_dim, encode ? 1 : 0, c.rope_style,
                                               table(plan), q, k, v, plan->err, static_cast<cudaStream_t>(stream)),
                     fn);
}

cb_status cb_qkv_projection(cb_plan* plan, const void* x, int32_t x_rows, int32_t d_model, const int32_t* rows,
                            int32_t m, const void* w_qkv, int32_t encode, void* x_gathered, void* q, void* k, void* v,
                            void* stream) {
  CB_NVTX_RANGE();
  return qkv_projection("cb_qkv_projection", plan, x, x_rows, d_model, rows, rows, m, w_qkv, encode, x_gathered, q,
                        k, v, stream);
}

cb_status cb_qkv_projection_indexed(cb_plan* plan, const void* x, int32_t x_rows, int32_t d_model,
                                    const int32_t* x_index, const int32_t* tokens, int32_t m, const void* w_qkv,
                                    int32_t encode, void* x_gathered, void* q, void* k, void* v, void* stream) {
  CB_NVTX_RANGE();
  return qkv_projection("cb_qkv_projection_indexed", plan, x, x_rows, d_model, x_index, tokens, m, w_qkv, encode,
                        x_gathered, q, k, v, stream);
}

cb_status cb_decode_attention(cb_plan* plan, const void* q, const void* k, const void* v, int32_t n_keys,
                              float scale, void* out, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (n_keys < 0) return fail(CB_ERR_INVALID_ARG, "n_keys < 0");
  if (n_keys == 0) return CB_OK;
  CB_TRY(need_tensor(q, "q"));
  CB_TRY(need_tensor(k, "k"));
  CB_TRY(need_tensor(v, "v"));
  CB_TRY(need_tensor(out, "out"));
  const auto& c = plan->cfg;
  if (!(scale > 0.0f)) scale = 1.0f / std::sqrt((float)c.head_dim);
  if (!cb::decode_tc_supported(c.hq, c.hkv, c.head_dim))
    return fail(CB_ERR_UNSUPPORTED, "decode: hq / hkv = %d, head_dim %d", c.hq / c.hkv, c.head_dim);
  return cuda_status(cb::launch_decode_tc(q, k, v, n_keys, c.hq, c.hkv, c.head_dim, scale, out, plan->decode,
                                          plan->err, static_cast<cudaStream_t>(stream)),
                     "cb_decode_attention");
}

int32_t cb_kv4_page_bytes(const cb_plan* plan, int32_t page_size) {
  if (check_plan(plan) != CB_OK || check_kv4_cache(0, page_size) != CB_OK) return 0;
  return page_size / 16 * 18 * plan->cfg.head_dim;
}

cb_status cb_page_tables(cb_plan* plan, const int32_t* ctx_lens, const int32_t* new_lens, int32_t n_seqs,
                         int32_t page_size, const int32_t* free_pages, int32_t n_free, const int32_t* free_from,
                         int32_t* table, int32_t table_width, int32_t* cu_seqlens, int32_t* kv_lens,
                         int32_t* positions, int32_t* slots, int32_t n_rows, int32_t* free_to, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  CB_TRY(check_kv4_cache(0, page_size));
  if (n_seqs < 0 || n_free < 0 || table_width < 0 || n_rows < 0) return fail(CB_ERR_INVALID_ARG, "negative size");
  if (n_seqs > CB_PAGE_TABLES_MAX_SEQS)
    return fail(CB_ERR_UNSUPPORTED, "n_seqs %d above %d", n_seqs, CB_PAGE_TABLES_MAX_SEQS);
  if ((int64_t)n_seqs * table_width > (1 << 30) || (int64_t)table_width * page_size > 0x7fffffffll)
    return fail(CB_ERR_INVALID_ARG, "page table too large: n_seqs * table_width above 2^30 or a row above 2^31 - 1 slots");
  if (n_seqs > 0) {
    CB_TRY(need_ptr(ctx_lens, "ctx_lens"));
    CB_TRY(need_ptr(new_lens, "new_lens"));
    CB_TRY(need_ptr(kv_lens, "kv_lens"));
    if (table_width > 0) CB_TRY(need_ptr(table, "table"));
  }
  if (n_free > 0) CB_TRY(need_ptr(free_pages, "free_pages"));
  if (n_rows > 0) {
    CB_TRY(need_ptr(positions, "positions"));
    CB_TRY(need_ptr(slots, "slots"));
  }
  CB_TRY(need_ptr(cu_seqlens, "cu_seqlens"));
  CB_TRY(need_ptr(free_to, "free_to"));
  // Every block reads all lengths, the start of the free list and the pages that it gives out, each at a time of its
  // own, so no block may write over them.
  if (n_seqs > 0 && (kv_lens == ctx_lens || kv_lens == new_lens))
    return fail(CB_ERR_INVALID_ARG, "kv_lens must not be ctx_lens or new_lens");
  if (free_to == free_from) return fail(CB_ERR_INVALID_ARG, "free_to must not be free_from");
  const int64_t per_request = 4 * (int64_t)n_seqs, per_row = 4 * (int64_t)n_rows;
  CB_TRY(check_apart({{table, per_request * table_width, "table"},
                      {cu_seqlens, per_request + 4, "cu_seqlens"},
                      {kv_lens, per_request, "kv_lens"},
                      {positions, per_row, "positions"},
                      {slots, per_row, "slots"},
                      {free_to, 4, "free_to"}},
                     {{ctx_lens, per_request, "ctx_lens"},
                      {new_lens, per_request, "new_lens"},
                      {free_pages, 4 * (int64_t)n_free, "free_pages"},
                      {free_from, 4, "free_from"}}));
  CB_TRY(check_device(plan));
  return cuda_status(cb::launch_page_tables(ctx_lens, new_lens, n_seqs, page_size, free_pages, n_free, free_from, table,
                                            table_width, cu_seqlens, kv_lens, positions, slots, n_rows, free_to,
                                            plan->err, static_cast<cudaStream_t>(stream)),
                     "cb_page_tables");
}

static cb_status kv4_rows(const char* fn, bool store, cb_plan* plan, void* k, void* v, const int32_t* slots, int32_t n,
                          void* cache, int32_t n_pages, int32_t page_size, void* stream) {
  CB_TRY(check_plan(plan));
  CB_TRY(check_kv4_cache(n_pages, page_size));
  if (n < 0) return fail(CB_ERR_INVALID_ARG, "n < 0");
  if (n == 0) return CB_OK;
  CB_TRY(need_tensor(k, "k"));
  CB_TRY(need_tensor(v, "v"));
  CB_TRY(need_ptr(slots, "slots"));
  if (n_pages > 0) CB_TRY(need_tensor(cache, "cache"));
  const int64_t rows = (int64_t)n * plan->cfg.hkv * plan->cfg.head_dim * 2;
  const Span ks{k, rows, "k"}, vs{v, rows, "v"}, ss{slots, 4 * (int64_t)n, "slots"}, cs = cache_span(plan, cache, n_pages, page_size);
  CB_TRY(store ? check_apart({cs}, {ks, vs, ss}) : check_apart({ks, vs}, {cs, ss}));
  CB_TRY(check_device(plan));
  return cuda_status(cb::launch_kv4_rows(store, k, v, slots, n, cache, n_pages, page_size, plan->cfg.hkv,
                                         plan->cfg.head_dim, plan->err, static_cast<cudaStream_t>(stream)),
                     fn);
}

cb_status cb_kv4_store(cb_plan* plan, const void* k, const void* v, const int32_t* slots, int32_t n, void* cache,
                       int32_t n_pages, int32_t page_size, void* stream) {
  CB_NVTX_RANGE();
  return kv4_rows("cb_kv4_store", true, plan, const_cast<void*>(k), const_cast<void*>(v), slots, n, cache, n_pages,
                  page_size, stream);
}

cb_status cb_kv4_load(cb_plan* plan, const void* cache, int32_t n_pages, int32_t page_size, const int32_t* slots,
                      int32_t n, void* k, void* v, void* stream) {
  CB_NVTX_RANGE();
  return kv4_rows("cb_kv4_load", false, plan, k, v, slots, n, const_cast<void*>(cache), n_pages, page_size, stream);
}

static cb_status kv4_decode(const char* fn, bool probe, cb_plan* plan, const void* q, const void* cache, int32_t n_pages,
                            int32_t page_size, const int32_t* table, int32_t table_width, const int32_t* kv_lens,
                            int32_t n_seqs, float scale, void* out, void* stream) {
  CB_TRY(check_plan(plan));
  CB_TRY(check_kv4_cache(n_pages, page_size));
  const auto& c = plan->cfg;
  if (n_seqs < 0 || table_width < 0) return fail(CB_ERR_INVALID_ARG, "negative size");
  if ((int64_t)n_seqs * c.hkv > 0x7fffffffll || (int64_t)table_width * page_size > 0x7fffffffll)
    return fail(CB_ERR_INVALID_ARG, "n_seqs * hkv or table_width * page_size above 2^31 - 1");
  if ((int64_t)n_seqs * c.hkv * ((int64_t)table_width * page_size / 16) >= (1ll << 30))
    return fail(CB_ERR_UNSUPPORTED, "n_seqs * hkv * table_width * page_size above 2^34");
  if (n_seqs == 0) return CB_OK;
  CB_TRY(need_tensor(q, "q"));
  if (n_pages > 0) CB_TRY(need_tensor(cache, "cache"));
  if (table_width > 0) CB_TRY(need_ptr(table, "table"));
  CB_TRY(need_ptr(kv_lens, "kv_lens"));
  CB_TRY(need_tensor(out, "out"));
  if (out == q) return fail(CB_ERR_INVALID_ARG, "out must not be q");
  const int64_t rows = (int64_t)n_seqs * c.hq * c.head_dim * 2;
  CB_TRY(check_apart({{out, rows, "out"}}, {{q, rows, "q"},
                                            cache_span(plan, cache, n_pages, page_size),
                                            {table, 4 * (int64_t)n_seqs * table_width, "table"},
                                            {kv_lens, 4 * (int64_t)n_seqs, "kv_lens"}}));
  CB_TRY(check_device(plan));
  if (!(scale > 0.0f)) scale = 1.0f / std::sqrt((float)c.head_dim);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(probe ? cb::launch_kv4_decode_timeout_probe(q, cache, n_pages, page_size, table, table_width, kv_lens,
                                                                 n_seqs, c.hq, c.hkv, scale, out, plan->kv4, plan->err, s)
                           : cb::launch_kv4_decode(q, cache, n_pages, page_size, table, table_width, kv_lens, n_seqs, c.hq,
                                                   c.hkv, c.head_dim, scale, out, plan->kv4, plan->err, s),
                     fn);
}

cb_status cb_kv4_decode_attention(cb_plan* plan, const void* q, const void* cache, int32_t n_pages, int32_t page_size,
                                  const int32_t* table, int32_t table_width, const int32_t* kv_lens, int32_t n_seqs,
                                  float scale, void* out, void* stream) {
  CB_NVTX_RANGE();
  return kv4_decode("cb_kv4_decode_attention", false, plan, q, cache, n_pages, page_size, table, table_width, kv_lens,
                    n_seqs, scale, out, stream);
}

cb_status cb_test_kv4_decode_wait_timeout(cb_plan* plan, const void* q, const void* cache, int32_t n_pages,
                                          int32_t page_size, const int32_t* table, int32_t table_width,
                                          const int32_t* kv_lens, int32_t n_seqs, void* out, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (plan->cfg.head_dim != 128 || plan->cfg.hq > 8 * plan->cfg.hkv)
    return fail(CB_ERR_UNSUPPORTED, "the wait-timeout probe needs head_dim 128 and hq / hkv of at most 8");
  return kv4_decode("cb_test_kv4_decode_wait_timeout", true, plan, q, cache, n_pages, page_size, table, table_width,
                    kv_lens, n_seqs, 0.0f, out, stream);
}

static cb_status prompt_attention(const char* fn, bool probe, cb_plan* plan, const void* q, const void* k, const void* v,
                                  const int32_t* cu_seqlens, int32_t n_seqs, int32_t n_rows, float scale, void* out,
                                  void* stream) {
  CB_TRY(check_plan(plan));
  const auto& c = plan->cfg;
  if (n_seqs < 0 || n_rows < 0) return fail(CB_ERR_INVALID_ARG, "negative size");
  if (n_seqs > CB_PROMPT_MAX_SEQS) return fail(CB_ERR_UNSUPPORTED, "n_seqs above 16384");
  if (n_seqs == 0 || n_rows == 0) return CB_OK;
  if (cb::prompt_items(n_seqs, n_rows, c.hq, c.hkv) > (1 << 30))
    return fail(CB_ERR_INVALID_ARG, "n_rows and n_seqs make more than 2^30 work items");
  CB_TRY(need_tensor(q, "q"));
  CB_TRY(need_tensor(k, "k"));
  CB_TRY(need_tensor(v, "v"));
  CB_TRY(need_ptr(cu_seqlens, "cu_seqlens"));
  CB_TRY(need_tensor(out, "out"));
  if (out == q || out == k || out == v) return fail(CB_ERR_INVALID_ARG, "out must not be q, k or v");
  const int64_t q_row = (int64_t)c.hq * c.head_dim * 2, kv_row = (int64_t)c.hkv * c.head_dim * 2;
  CB_TRY(check_apart({{out, n_rows * q_row, "out"}}, {{q, n_rows * q_row, "q"},
                                                      {k, n_rows * kv_row, "k"},
                                                      {v, n_rows * kv_row, "v"},
                                                      {cu_seqlens, 4 * ((int64_t)n_seqs + 1), "cu_seqlens"}}));
  CB_TRY(check_device(plan));
  if (!(scale > 0.0f)) scale = 1.0f / std::sqrt((float)c.head_dim);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(probe ? cb::launch_prompt_timeout_probe(q, k, v, cu_seqlens, n_seqs, n_rows, c.hq, c.hkv, scale, out,
                                                             plan->err, s)
                           : cb::launch_prompt_attention(q, k, v, cu_seqlens, n_seqs, n_rows, c.hq, c.hkv, c.head_dim,
                                                         scale, out, plan->err, s),
                     fn);
}

cb_status cb_prompt_attention(cb_plan* plan, const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                              int32_t n_seqs, int32_t n_rows, float scale, void* out, void* stream) {
  CB_NVTX_RANGE();
  return prompt_attention("cb_prompt_attention", false, plan, q, k, v, cu_seqlens, n_seqs, n_rows, scale, out, stream);
}

cb_status cb_test_prompt_wait_timeout(cb_plan* plan, const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                                      int32_t n_seqs, int32_t n_rows, void* out, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (plan->cfg.head_dim != 128) return fail(CB_ERR_UNSUPPORTED, "the wait-timeout probe needs head_dim 128");
  return prompt_attention("cb_test_prompt_wait_timeout", true, plan, q, k, v, cu_seqlens, n_seqs, n_rows, 0.0f, out, stream);
}

// The checks that the calls over a batch's pages share; `b` is filled in.
static cb_status kv4_batch(cb_plan* plan, const void* q, const void* cache, int32_t n_pages, int32_t page_size,
                           const int32_t* table, int32_t table_width, const int32_t* cu_seqlens, const int32_t* kv_lens,
                           int32_t n_seqs, int32_t n_rows, float scale, cb::Kv4Batch* b) {
  const auto& c = plan->cfg;
  CB_TRY(check_kv4_cache(n_pages, page_size));
  if (n_seqs < 0 || n_rows < 0 || table_width < 0) return fail(CB_ERR_INVALID_ARG, "negative size");
  if (n_seqs > CB_PROMPT_MAX_SEQS) return fail(CB_ERR_UNSUPPORTED, "n_seqs above 16384");
  if ((int64_t)table_width * page_size > 0x7fffffffll)
    return fail(CB_ERR_INVALID_ARG, "table_width * page_size above 2^31 - 1");
  // (the kernels count tokens of a tile or two past it)
  if ((int64_t)table_width * page_size > (1 << 30)) return fail(CB_ERR_UNSUPPORTED, "table_width * page_size above 2^30");
  if ((int64_t)n_seqs * table_width > (1 << 30))
    return fail(CB_ERR_INVALID_ARG, "page table too large: n_seqs * table_width above 2^30");
  // row tiles times key tiles of all kv heads, 128 rows or keys each
  const int64_t tiles = ((int64_t)n_rows / (128 / (c.hq / c.hkv)) + n_seqs) * c.hkv;
  if (tiles * (std::max<int64_t>((int64_t)table_width * page_size, n_rows) / 128 + 1) > cb::kKv4MostTiles)
    return fail(CB_ERR_UNSUPPORTED, "n_rows, n_seqs and table_width * page_size make more than 2^30 tiles");
  if (n_seqs == 0 || n_rows == 0) return CB_OK;
  CB_TRY(need_tensor(q, "q"));
  if (n_pages > 0) CB_TRY(need_tensor(cache, "cache"));
  if (table_width > 0) CB_TRY(need_words(table, "table"));
  CB_TRY(need_words(cu_seqlens, "cu_seqlens"));
  CB_TRY(need_words(kv_lens, "kv_lens"));
  b->q = static_cast<const uint8_t*>(q);
  b->cache = static_cast<const uint8_t*>(cache);
  b->table = table;
  b->cu = cu_seqlens;
  b->kv_lens = kv_lens;
  b->n_pages = n_pages;
  b->page_size = page_size;
  b->width = table_width;
  b->n_seqs = n_seqs;
  b->n_rows = n_rows;
  b->hq = c.hq;
  b->hkv = c.hkv;
  b->scale = scale > 0.0f ? scale : 1.0f / std::sqrt((float)c.head_dim);
  b->err = plan->err;
  return CB_OK;
}

static cb_status kv4_chunk(const char* fn, bool probe, cb_plan* plan, const void* q, const void* cache, int32_t n_pages,
                           int32_t page_size, const int32_t* table, int32_t table_width, const int32_t* cu_seqlens,
                           const int32_t* kv_lens, int32_t n_seqs, int32_t n_rows, float scale, void* out, float* lse,
                           void* stream) {
  CB_TRY(check_plan(plan));
  const auto& c = plan->cfg;
  cb::Kv4Batch b;
  CB_TRY(kv4_batch(plan, q, cache, n_pages, page_size, table, table_width, cu_seqlens, kv_lens, n_seqs, n_rows, scale, &b));
  if (n_seqs == 0 || n_rows == 0) return CB_OK;
  CB_TRY(need_tensor(out, "out"));
  if (lse != nullptr) CB_TRY(need_words(lse, "lse"));
  const int64_t rows = (int64_t)n_rows * c.hq * c.head_dim * 2;
  CB_TRY(check_apart({{out, rows, "out"}, {lse, 4 * (int64_t)n_rows * c.hq, "lse"}},
                     {{q, rows, "q"},
                      cache_span(plan, cache, n_pages, page_size),
                      {table, 4 * (int64_t)n_seqs * table_width, "table"},
                      {cu_seqlens, 4 * ((int64_t)n_seqs + 1), "cu_seqlens"},
                      {kv_lens, 4 * (int64_t)n_seqs, "kv_lens"}}));
  CB_TRY(check_device(plan));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(probe ? cb::launch_kv4_chunk_timeout_probe(b, out, plan->chunk, s)
                           : cb::launch_kv4_chunk(b, c.head_dim, out, lse, plan->chunk, s),
                     fn);
}

cb_status cb_kv4_chunk_attention(cb_plan* plan, const void* q, const void* cache, int32_t n_pages, int32_t page_size,
                                 const int32_t* table, int32_t table_width, const int32_t* cu_seqlens,
                                 const int32_t* kv_lens, int32_t n_seqs, int32_t n_rows, float scale, void* out,
                                 float* lse, void* stream) {
  CB_NVTX_RANGE();
  return kv4_chunk("cb_kv4_chunk_attention", false, plan, q, cache, n_pages, page_size, table, table_width, cu_seqlens,
                   kv_lens, n_seqs, n_rows, scale, out, lse, stream);
}

cb_status cb_test_kv4_chunk_wait_timeout(cb_plan* plan, const void* q, const void* cache, int32_t n_pages,
                                         int32_t page_size, const int32_t* table, int32_t table_width,
                                         const int32_t* cu_seqlens, const int32_t* kv_lens, int32_t n_seqs,
                                         int32_t n_rows, void* out, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (plan->cfg.head_dim != 128) return fail(CB_ERR_UNSUPPORTED, "the wait-timeout probe needs head_dim 128");
  return kv4_chunk("cb_test_kv4_chunk_wait_timeout", true, plan, q, cache, n_pages, page_size, table, table_width,
                   cu_seqlens, kv_lens, n_seqs, n_rows, 0.0f, out, nullptr, stream);
}

static cb_status kv4_weights(const char* fn, bool probe, cb_plan* plan, const void* q, const float* lse,
                             const void* cache, int32_t n_pages, int32_t page_size, const int32_t* table,
                             int32_t table_width, const int32_t* cu_seqlens, const int32_t* kv_lens, int32_t n_seqs,
                             int32_t n_rows, int32_t window, float scale, const float* earlier, float* weights,
                             void* stream) {
  CB_TRY(check_plan(plan));
  const auto& c = plan->cfg;
  if (window < 0) return fail(CB_ERR_INVALID_ARG, "window < 0");
  cb::Kv4Batch b;
  CB_TRY(kv4_batch(plan, q, cache, n_pages, page_size, table, table_width, cu_seqlens, kv_lens, n_seqs, n_rows, scale, &b));
  if (n_seqs == 0 || n_rows == 0 || table_width == 0) return CB_OK;
  CB_TRY(need_words(lse, "lse"));
  CB_TRY(need_words(weights, "weights"));
  if (earlier != nullptr) CB_TRY(need_words(earlier, "earlier"));
  const int64_t bytes = 4 * (int64_t)n_seqs * c.hkv * table_width * page_size;
  CB_TRY(check_apart({{weights, bytes, "weights"}},
                     {{q, (int64_t)n_rows * c.hq * c.head_dim * 2, "q"},
                      {lse, 4 * (int64_t)n_rows * c.hq, "lse"},
                      cache_span(plan, cache, n_pages, page_size),
                      {table, 4 * (int64_t)n_seqs * table_width, "table"},
                      {cu_seqlens, 4 * ((int64_t)n_seqs + 1), "cu_seqlens"},
                      {kv_lens, 4 * (int64_t)n_seqs, "kv_lens"},
                      {earlier == weights ? nullptr : earlier, bytes, "earlier"}}));
  CB_TRY(check_device(plan));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(probe ? cb::launch_kv4_weights_timeout_probe(b, lse, weights, plan->chunk.sms, s)
                           : cb::launch_kv4_weights(b, c.head_dim, lse, window, earlier, weights, plan->chunk.sms, s),
                     fn);
}

cb_status cb_kv4_attention_weights(cb_plan* plan, const void* q, const float* lse, const void* cache, int32_t n_pages,
                                   int32_t page_size, const int32_t* table, int32_t table_width,
                                   const int32_t* cu_seqlens, const int32_t* kv_lens, int32_t n_seqs, int32_t n_rows,
                                   int32_t window, float scale, const float* earlier, float* weights, void* stream) {
  CB_NVTX_RANGE();
  return kv4_weights("cb_kv4_attention_weights", false, plan, q, lse, cache, n_pages, page_size, table, table_width,
                     cu_seqlens, kv_lens, n_seqs, n_rows, window, scale, earlier, weights, stream);
}

cb_status cb_test_kv4_weights_wait_timeout(cb_plan* plan, const void* q, const float* lse, const void* cache,
                                           int32_t n_pages, int32_t page_size, const int32_t* table,
                                           int32_t table_width, const int32_t* cu_seqlens, const int32_t* kv_lens,
                                           int32_t n_seqs, int32_t n_rows, float* weights, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (plan->cfg.head_dim != 128) return fail(CB_ERR_UNSUPPORTED, "the wait-timeout probe needs head_dim 128");
  return kv4_weights("cb_test_kv4_weights_wait_timeout", true, plan, q, lse, cache, n_pages, page_size, table,
                     table_width, cu_seqlens, kv_lens, n_seqs, n_rows, 0, 0.0f, nullptr, weights, stream);
}

cb_status cb_kv4_keep(cb_plan* plan, const float* weights, int32_t weights_width, const int32_t* kv_lens,
                      const int32_t* budgets, int32_t n_seqs, int32_t first, int32_t recent, int32_t* kept,
                      int32_t kept_width, int32_t* kept_lens, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  const int64_t hkv = plan->cfg.hkv;
  if (weights_width < 0 || n_seqs < 0 || kept_width < 0) return fail(CB_ERR_INVALID_ARG, "negative size");
  if (first < 0 || recent < 0) return fail(CB_ERR_INVALID_ARG, "first < 0 or recent < 0");
  if (weights_width > (1 << 30)) return fail(CB_ERR_UNSUPPORTED, "weights_width above 2^30");
  if (n_seqs > CB_PROMPT_MAX_SEQS) return fail(CB_ERR_UNSUPPORTED, "n_seqs above 16384");
  if (n_seqs == 0) return CB_OK;
  if (weights_width > 0) CB_TRY(need_words(weights, "weights"));
  CB_TRY(need_words(kv_lens, "kv_lens"));
  CB_TRY(need_words(budgets, "budgets"));
  if (kept_width > 0) CB_TRY(need_words(kept, "kept"));
  CB_TRY(need_words(kept_lens, "kept_lens"));
  CB_TRY(check_apart({{kept, 4 * n_seqs * hkv * kept_width, "kept"}, {kept_lens, 4 * (int64_t)n_seqs, "kept_lens"}},
                     {{weights, 4 * n_seqs * hkv * weights_width, "weights"},
                      {kv_lens, 4 * (int64_t)n_seqs, "kv_lens"},
                      {budgets, 4 * (int64_t)n_seqs, "budgets"}}));
  CB_TRY(check_device(plan));
  return cuda_status(cb::launch_kv4_keep(weights, weights_width, kv_lens, budgets, n_seqs, plan->cfg.hkv, first, recent,
                                         kept, kept_width, kept_lens, plan->chunk.sms, plan->err,
                                         static_cast<cudaStream_t>(stream)),
                     "cb_kv4_keep");
}

cb_status cb_kv4_move(cb_plan* plan, void* cache, int32_t n_pages, int32_t page_size, const int32_t* table,
                      int32_t table_width, const int32_t* kept, int32_t kept_width, const int32_t* kept_lens,
                      int32_t n_seqs, const int32_t* table_to, int32_t to_width, const float* weights,
                      float* weights_to, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  CB_TRY(check_kv4_cache(n_pages, page_size));
  const int64_t hkv = plan->cfg.hkv;
  if (n_seqs < 0 || table_width < 0 || kept_width < 0 || to_width < 0) return fail(CB_ERR_INVALID_ARG, "negative size");
  if (n_seqs > CB_PROMPT_MAX_SEQS) return fail(CB_ERR_UNSUPPORTED, "n_seqs above 16384");
  if ((int64_t)table_width * page_size > 0x7fffffffll || (int64_t)to_width * page_size > 0x7fffffffll)
    return fail(CB_ERR_INVALID_ARG, "table_width or to_width times page_size above 2^31 - 1");
  if ((int64_t)table_width * page_size > (1 << 30) || (int64_t)to_width * page_size > (1 << 30))
    return fail(CB_ERR_UNSUPPORTED, "table_width or to_width times page_size above 2^30");
  if ((int64_t)n_seqs * table_width > (1 << 30) || (int64_t)n_seqs * to_width > (1 << 30))
    return fail(CB_ERR_INVALID_ARG, "page table too large: n_seqs times its width above 2^30");
  if (n_seqs * hkv * (kept_width / 16 + 1ll) > (1 << 30))
    return fail(CB_ERR_UNSUPPORTED, "n_seqs * hkv * kept_width above 2^34");
  if ((weights == nullptr) != (weights_to == nullptr))
    return fail(CB_ERR_INVALID_ARG, "weights and weights_to: both or neither");
  if (n_seqs == 0 || kept_width == 0) return CB_OK;
  if (n_pages > 0) CB_TRY(need_tensor(cache, "cache"));
  if (table_width > 0) CB_TRY(need_words(table, "table"));
  CB_TRY(need_words(kept, "kept"));
  CB_TRY(need_words(kept_lens, "kept_lens"));
  if (to_width > 0) CB_TRY(need_words(table_to, "table_to"));
  if (weights != nullptr) {
    CB_TRY(need_words(weights, "weights"));
    CB_TRY(need_words(weights_to, "weights_to"));
  }
  CB_TRY(check_apart({cache_span(plan, cache, n_pages, page_size),
                      {weights_to, 4 * n_seqs * hkv * to_width * page_size, "weights_to"}},
                     {{table, 4 * (int64_t)n_seqs * table_width, "table"},
                      {kept, 4 * n_seqs * hkv * kept_width, "kept"},
                      {kept_lens, 4 * (int64_t)n_seqs, "kept_lens"},
                      {table_to, 4 * (int64_t)n_seqs * to_width, "table_to"},
                      {weights, 4 * n_seqs * hkv * table_width * page_size, "weights"}}));
  CB_TRY(check_device(plan));
  return cuda_status(cb::launch_kv4_move(cache, n_pages, page_size, plan->cfg.hkv, plan->cfg.head_dim, table, table_width,
                                         kept, kept_width, kept_lens, n_seqs, table_to, to_width, weights, weights_to,
                                         plan->err, static_cast<cudaStream_t>(stream)),
                     "cb_kv4_move");
}

struct LayerShape {
  int32_t n_cand, k, mq, selects;
};

// Host checks of one layer's buffers; `cand` is the candidate list the layer will read.
static cb_status validate_io(cb_plan* plan, int32_t layer, const cb_layer_io* io, const int32_t* cand,
                             LayerShape* sh) {
  CB_TRY(need_ptr(io, "io"));
  CB_TRY(cb_layer_sizes(plan, layer, &sh->n_cand, &sh->k, &sh->mq, &sh->selects));
  CB_TRY(need_tensor(io->k_old, "io.k_old"));
  CB_TRY(need_tensor(io->v_old, "io.v_old"));
  CB_TRY(need_tensor(io->k_new, "io.k_new"));
  CB_TRY(need_tensor(io->v_new, "io.v_new"));
  CB_TRY(need_tensor(io->q, "io.q"));
  CB_TRY(need_tensor(io->k_fused, "io.k_fused"));
  CB_TRY(need_tensor(io->v_fused, "io.v_fused"));
  if (sh->mq > 0) {
    CB_TRY(need_tensor(io->q_rot, "io.q_rot"));
    CB_TRY(need_tensor(io->out, "io.out"));
  }
  if (sh->k > 0) {
    CB_TRY(need_ptr(io->sel_tok, "io.sel_tok"));
    CB_TRY(need_ptr(io->sel_row, "io.sel_row"));
  }
  if (layer >= 2 && sh->n_cand > 0) CB_TRY(need_ptr(cand, "io.cand"));
  if (sh->selects && sh->n_cand > 0) CB_TRY(need_ptr(io->dev, "io.dev"));
  return CB_OK;
}

// One stage of layer `layer` on `s`; `cand` is the candidate list the layer reads (ignored at
// layer 1, where the candidates are all context tokens). S_l is sel_tok at selecting layers and
// the candidates themselves elsewhere; the fuse pass then copies them out to sel_tok / sel_row.
// inputs_by_event: the attention's inputs are ordered by an event on its stream (cb_blend_request),
// so it need not wait for the kernel before it on that stream, which it does not read from.
static cb_status enqueue_stage(cb_plan* plan, int32_t layer, const cb_layer_io* io, const int32_t* cand,
                               const LayerShape& sh, int32_t stage, cudaStream_t s, bool inputs_by_event = false) {
  const auto& c = plan->cfg;
  if (layer == 1) cand = nullptr;
  const int32_t* sel = sh.selects ? io->sel_tok : cand;
  switch (stage) {
    case CB_STAGE_DEVIATION: {
      if (!sh.selects) return CB_OK;
      const bool kv = c.deviation == CB_DEV_KV;
      return cuda_status(cb::launch_kv_deviation(kv ? io->k_new : nullptr, kv ? io->k_old : nullptr, io->v_new,
                                                 io->v_old, cand, sh.n_cand, plan->n_ctx, c.hkv, c.head_dim,
                                                 c.chunk_len, c.rope_style, table(plan), io->dev, plan->err, s),
                         "deviation");
    }
    case CB_STAGE_TOPK:
      if (!sh.selects) return CB_OK;
      return cuda_status(cb::launch_hkvd_topk(io->dev, cand, sh.n_cand, sh.k, io->sel_tok, io->sel_row, plan->err, s),
                         "top-k");
    case CB_STAGE_FUSE: {
      // One launch: the fused cache and the query encoding (both read the layer's selection list).
      // Small blocks on the layers whose attention runs the paired-tile kernel (see the fuse kernel).
      const bool copy_out = !sh.selects && sh.k > 0;
      const bool narrow = cb::attention_pp_eligible(sh.mq, c.hq, c.hkv, c.head_dim);
      return cuda_status(cb::launch_blend_fuse(io->k_fused, io->v_fused, io->k_old, io->v_old, io->k_new, io->v_new,
                                               sel, sh.k, copy_out ? io->sel_tok : nullptr,
                                               copy_out ? io->sel_row : nullptr, plan->n_ctx, c.chunk_len,
                                               plan->n_tokens, c.hkv, c.head_dim, c.rope_style, table(plan),
                                               sh.mq > 0 ? io->q : nullptr, sh.mq > 0 ? io->q_rot : nullptr, sh.mq,
                                               c.hq, narrow, plan->err, s),
                         "fuse");
    }
    case CB_STAGE_ATTENTION: {
      if (sh.mq == 0) return CB_OK;
      // query row t sits at sel[t] (t < k) or n_ctx + t - k
      const cb::QueryPositions qp{sel, sh.k, plan->n_ctx, !inputs_by_event};
      return cuda_status(cb::launch_hkvd_attention(io->q_rot, qp, sh.mq, io->k_fused, io->v_fused, plan->n_tokens,
                                                   c.hq, c.hkv, c.head_dim, 1.0f / std::sqrt((float)c.head_dim),
                                                   io->out, plan->err, s),
                         "attention");
    }
    default:
      return fail(CB_ERR_INVALID_ARG, "unknown stage %d", stage);
  }
}

// The selections of layers 2..n_layers (all from cand = S_1, k_2 each), kSelectBatchMax layers per
// pair of launches.
static cb_status enqueue_select_batches(cb_plan* plan, int32_t n_layers, const cb_layer_io* ios,
                                        const int32_t* cand, const LayerShape& sh, cudaStream_t s) {
  const auto& c = plan->cfg;
  const bool kv = c.deviation == CB_DEV_KV;
  for (int32_t l0 = 2; l0 <= n_layers; l0 += cb::kSelectBatchMax) {
    cb::SelectBatch b = {};
    b.n = std::min<int32_t>(cb::kSelectBatchMax, n_layers - l0 + 1);
    for (int i = 0; i < b.n; ++i) {
      const cb_layer_io& io = ios[l0 - 1 + i];
      b.k_new[i] = kv ? io.k_new : nullptr;
      b.k_old[i] = kv ? io.k_old : nullptr;
      b.v_new[i] = io.v_new;
      b.v_old[i] = io.v_old;
      b.dev[i] = io.dev;
      b.sel_tok[i] = io.sel_tok;
      b.sel_row[i] = io.sel_row;
    }
    CB_TRY(cuda_status(cb::launch_select_batch(b, cand, sh.n_cand, sh.k, plan->n_ctx, c.hkv, c.head_dim, c.chunk_len,
                                               c.rope_style, table(plan), plan->err, s),
                       "batched selection"));
  }
  return CB_OK;
}

cb_status cb_blend_layer(cb_plan* plan, int32_t layer, const cb_layer_io* io, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  LayerShape sh;
  CB_TRY(validate_io(plan, layer, io, io ? io->cand : nullptr, &sh));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t st = CB_STAGE_DEVIATION; st <= CB_STAGE_ATTENTION; ++st)
    CB_TRY(enqueue_stage(plan, layer, io, io->cand, sh, st, s));
  return CB_OK;
}

cb_status cb_blend_stage(cb_plan* plan, int32_t layer, const cb_layer_io* io, int32_t stage, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (stage < CB_STAGE_DEVIATION || stage > CB_STAGE_ATTENTION) return fail(CB_ERR_INVALID_ARG, "unknown stage %d", stage);
  LayerShape sh;
  CB_TRY(validate_io(plan, layer, io, io ? io->cand : nullptr, &sh));
  return enqueue_stage(plan, layer, io, io->cand, sh, stage, static_cast<cudaStream_t>(stream));
}

cb_status cb_blend_request(cb_plan* plan, int32_t n_layers, const cb_layer_io* ios, void* stream) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  if (n_layers < 1) return fail(CB_ERR_INVALID_ARG, "n_layers must be >= 1");
  CB_TRY(need_ptr(ios, "ios"));
  // C_l is the selection of layer l - 1, or of layer 1 when every layer re-selects from its pool.
  const bool reselect = plan->cfg.filter == CB_FILTER_RESELECT;
  auto cand_of = [&](int32_t l) -> const int32_t* {
    return l == 1 ? nullptr : ios[(reselect ? 1 : l - 1) - 1].sel_tok;
  };
  for (int32_t l = 1; l <= n_layers; ++l) {
    LayerShape sh;
    CB_TRY(validate_io(plan, l, &ios[l - 1], cand_of(l), &sh));
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaStream_t attn_stream[kAttnStreams];
  attn_stream[0] = s;
  for (int a = 1; a < kAttnStreams; ++a) attn_stream[a] = plan->aux_attn[a];
  CB_TRY(cuda_status(cudaEventRecord(plan->ev_fork, s), "fork"));
  CB_TRY(cuda_status(cudaStreamWaitEvent(plan->aux_stream, plan->ev_fork, 0), "fork"));
  for (int a = 1; a < kAttnStreams; ++a)
    CB_TRY(cuda_status(cudaStreamWaitEvent(attn_stream[a], plan->ev_fork, 0), "fork"));
  // Re-selection: every layer >= 2 selects k_2 from the same candidates S_1, so their deviations and
  // top-k go out as two batched launches right after layer 1's selection (instead of a deviation and
  // a one-block top-k ahead of every fuse), and the fuses then run ahead of the attention as they do
  // when the set is kept.
  const bool batch_select = reselect && n_layers >= 2;
  for (int32_t l = 1; l <= n_layers; ++l) {
    const cb_layer_io* io = &ios[l - 1];
    const int32_t* cand = cand_of(l);
    LayerShape sh;
    CB_TRY(validate_io(plan, l, io, cand, &sh));
    if (batch_select && l >= 2) {
      if (l == 2) CB_TRY(enqueue_select_batches(plan, n_layers, ios, ios[0].sel_tok, sh, plan->aux_stream));
      CB_TRY(enqueue_stage(plan, l, io, cand, sh, CB_STAGE_FUSE, plan->aux_stream));
    } else {
      for (int32_t st = CB_STAGE_DEVIATION; st <= CB_STAGE_FUSE; ++st)
        CB_TRY(enqueue_stage(plan, l, io, cand, sh, st, plan->aux_stream));
    }
    const cudaStream_t a = attn_stream[(l - 1) % kAttnStreams];
    CB_TRY(cuda_status(cudaEventRecord(plan->ev_ready, plan->aux_stream), "layer inputs ready"));
    CB_TRY(cuda_status(cudaStreamWaitEvent(a, plan->ev_ready, 0), "layer inputs ready"));
    CB_TRY(enqueue_stage(plan, l, io, cand, sh, CB_STAGE_ATTENTION, a, true));
  }
  for (int a = 1; a < kAttnStreams; ++a) {
    CB_TRY(cuda_status(cudaEventRecord(plan->ev_join, attn_stream[a]), "join"));
    CB_TRY(cuda_status(cudaStreamWaitEvent(s, plan->ev_join, 0), "join"));
  }
  CB_TRY(cuda_status(cudaEventRecord(plan->ev_join, plan->aux_stream), "join"));
  return cuda_status(cudaStreamWaitEvent(s, plan->ev_join, 0), "join");
}

cb_status cb_check(cb_plan* plan) {
  CB_NVTX_RANGE();
  CB_TRY(check_plan(plan));
  int32_t h[2] = {0, -1};
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(h, plan->err, sizeof(h), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) {
    const int32_t init[2] = {0, -1};
    e = cudaMemcpy(plan->err, init, sizeof(init), cudaMemcpyHostToDevice);
  }
  if (e != cudaSuccess) return cuda_status(e, "cb_check");
  if (h[0] == 0) return CB_OK;
  const bool timeout = (h[0] & cb::kErrTimeout) != 0;
  return fail(timeout ? CB_ERR_TIMEOUT : CB_ERR_DEVICE_CHECK,
              "device check failed: flags 0x%x (1 rope range, 2 index, 4 order, 8 timeout), first at %d", h[0], h[1]);
}

}  // extern "C"
