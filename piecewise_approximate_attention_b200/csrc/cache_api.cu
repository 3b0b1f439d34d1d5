// Host entry points of the paged key/value cache (pisa_cache.h): validation and dispatch.
#include <cmath>

#include "cache.cuh"
#include "pisa_testing.h"

namespace pisa {
namespace cache {
namespace {

// test-only fault injection (pisa_testing.h)
int g_test_fault = PISA_TESTING_FAULT_NONE;
unsigned long long g_test_wait_ns = 0;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pisa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PISA_OK : PISA_ERR_CUDA; }

pisa_status check_sizes(const pisa_cache* c) {
  if (!c || c->num_pages < 1 || c->kv_heads < 1 || c->page < 1 || c->head_dim < 1) return PISA_ERR_INVALID_ARG;
  if (c->dtype != PISA_CACHE_BF16 && c->dtype != PISA_CACHE_FP32 && c->dtype != PISA_CACHE_E4M3)
    return PISA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return PISA_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return PISA_ERR_UNSUPPORTED;
  // pages are addressed by 32-bit row numbers; no divisions that overflow: kv_heads * page first
  if (c->kv_heads > 65535 || (long long)c->num_pages * ((long long)c->kv_heads * c->page) >= 0x80000000LL)
    return PISA_ERR_UNSUPPORTED;
  return PISA_OK;
}

pisa_status check_cache(const pisa_cache* c, Pool* p) {
  const pisa_status s = check_sizes(c);
  if (s != PISA_OK) return s;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return PISA_ERR_INVALID_ARG;
  if (c->dtype == PISA_CACHE_E4M3 && (!c->k_exp || !c->v_exp || !aligned16(c->k_exp) || !aligned16(c->v_exp)))
    return PISA_ERR_INVALID_ARG;
  p->k = static_cast<const char*>(c->k);
  p->v = static_cast<const char*>(c->v);
  p->k_exp = c->k_exp;
  p->v_exp = c->v_exp;
  p->num_pages = c->num_pages;
  p->kv_heads = c->kv_heads;
  p->page = c->page;
  p->page_log2 = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  p->dtype = c->dtype;
  return PISA_OK;
}

// *empty: nothing to do (no sequence, or none with a new token).
pisa_status check_seqs(const pisa_cache* c, const pisa_sequences* q, void* ws, size_t ws_bytes, Seqs* s, bool* empty) {
  if (!q || q->batch < 0 || q->max_pages < 0 || q->max_len < 0 || q->max_new < 0) return PISA_ERR_INVALID_ARG;
  if (q->max_len > (long long)q->max_pages * c->page) return PISA_ERR_INVALID_ARG;
  if (q->starts && q->counts) return PISA_ERR_INVALID_ARG;
  if (q->batch > 65535) return PISA_ERR_UNSUPPORTED;
  *empty = q->batch == 0 || q->max_new == 0;
  if (!*empty && (!q->lens || (q->max_len > 0 && !q->page_table))) return PISA_ERR_INVALID_ARG;
  const void* p[] = {q->lens, q->page_table, q->starts, q->counts};
  for (const void* x : p)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return PISA_ERR_INVALID_ARG;   // views of larger int32 tensors are fine
  if (!ws || !aligned16(ws) || ws_bytes < pisa_cache_workspace_bytes(c)) return PISA_ERR_INVALID_ARG;
  s->batch = q->batch;
  s->max_pages = q->max_pages;
  s->max_len = q->max_len;
  s->max_new = q->max_new;
  s->table = q->page_table;
  s->lens = q->lens;
  s->starts = q->starts;
  s->counts = q->counts;
  s->status = static_cast<int*>(ws);
  return PISA_OK;
}

// written: an output, whose rows must not fall on one another.
pisa_status check_rows(const pisa_rows* r, const pisa_cache* c, const Seqs& s, int heads, bool written, Rows* out) {
  // packed tensors may be empty (every sequence waits): then there is no address, and nothing to check
  if (!r || r->rows < 0 || !aligned16(r->data) || (!r->data && (r->rows > 0 || !s.starts))) return PISA_ERR_INVALID_ARG;
  const int esz = c->dtype == PISA_CACHE_FP32 ? 4 : 2;
  const bool packed = s.starts != nullptr;
  if (!packed && r->rows < s.max_new) return PISA_ERR_INVALID_ARG;
  const long long st[3] = {packed ? 0 : r->seq_stride, r->row_stride, r->head_stride};
  const long long n[3] = {packed ? 1 : s.batch, r->rows, heads};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < 0 || st[i] > (1LL << 48) || (st[i] * esz) % 16) return PISA_ERR_INVALID_ARG;
    if (written && st[i] < c->head_dim) return PISA_ERR_INVALID_ARG;
  }
  out->data = static_cast<char*>(r->data);
  out->rows = r->rows;
  out->seq = n[0] <= 1 ? 0 : st[0] * esz;
  out->row = n[1] <= 1 ? 0 : st[1] * esz;
  out->head = n[2] <= 1 ? 0 : st[2] * esz;
  return PISA_OK;
}

}  // namespace
}  // namespace cache
}  // namespace pisa

using namespace pisa;
using namespace pisa::cache;

extern "C" {

size_t pisa_cache_workspace_bytes(const pisa_cache* c) {
  if (check_sizes(c) != PISA_OK) return 0;
  return kPartialsAt + partials_bytes(c->head_dim);
}

namespace {
pisa_status move_rows(bool append, const pisa_cache* c, const pisa_sequences* q, const pisa_rows* k, const pisa_rows* v,
                      void* ws, size_t ws_bytes, pisa_stream_t stream) {
  Pool pool;
  Seqs seqs;
  Rows kr, vr;
  bool empty;
  pisa_status s = check_cache(c, &pool);
  if (s != PISA_OK) return s;
  if ((s = check_seqs(c, q, ws, ws_bytes, &seqs, &empty)) != PISA_OK) return s;
  if (empty) return PISA_OK;
  if ((s = check_rows(k, c, seqs, c->kv_heads, !append, &kr)) != PISA_OK) return s;
  if ((s = check_rows(v, c, seqs, c->kv_heads, !append, &vr)) != PISA_OK) return s;
  if (!kr.data || !vr.data) return kr.data == vr.data ? PISA_OK : PISA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(append ? launch_append(pool, c->head_dim, seqs, kr, vr, st)
                            : launch_read(pool, c->head_dim, seqs, kr, vr, st));
}
}  // namespace

pisa_status pisa_cache_append(const pisa_cache* cache, const pisa_sequences* seqs, const pisa_rows* k, const pisa_rows* v,
                              void* ws, size_t ws_bytes, pisa_stream_t stream) {
  return move_rows(true, cache, seqs, k, v, ws, ws_bytes, stream);
}

pisa_status pisa_cache_read(const pisa_cache* cache, const pisa_sequences* seqs, const pisa_rows* k, const pisa_rows* v,
                            void* ws, size_t ws_bytes, pisa_stream_t stream) {
  return move_rows(false, cache, seqs, k, v, ws, ws_bytes, stream);
}

pisa_status pisa_cache_attention(const pisa_cache* cache, const pisa_sequences* seqs, int32_t heads, int32_t causal,
                                 int32_t window, float softmax_scale, const pisa_rows* q, const pisa_rows* o, float* lse,
                                 void* ws, size_t ws_bytes, pisa_stream_t stream) {
  AttnArgs a;
  bool empty;
  pisa_status s = check_cache(cache, &a.pool);
  if (s != PISA_OK) return s;
  if (heads < 1 || heads % cache->kv_heads || window < 0) return PISA_ERR_INVALID_ARG;
  if (heads > 65535) return PISA_ERR_UNSUPPORTED;
  if (!std::isfinite(softmax_scale * 1.4426950408889634f) || !(softmax_scale > 0.f)) return PISA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return PISA_ERR_INVALID_ARG;
  if ((s = check_seqs(cache, seqs, ws, ws_bytes, &a.seqs, &empty)) != PISA_OK) return s;
  if (empty) return PISA_OK;
  // the rows of one sequence and key/value head are numbered in 31 bits, and so are its pairs of a tile of rows and
  // one of keys (at least 16 and 32 of them)
  const long long head_rows = (long long)seqs->max_new * (heads / cache->kv_heads);
  if (head_rows >= 0x7fff0000LL || (head_rows / 16 + 1) * ((long long)seqs->max_len / 32 + 16) >= 0x7fff0000LL)
    return PISA_ERR_UNSUPPORTED;
  if ((s = check_rows(q, cache, a.seqs, heads, false, &a.q)) != PISA_OK) return s;
  if ((s = check_rows(o, cache, a.seqs, heads, true, &a.o)) != PISA_OK) return s;
  if ((q->data == o->data && q->data) || o->rows < q->rows) return PISA_ERR_INVALID_ARG;
  if (!q->data) return PISA_OK;
  a.lse = lse;
  a.heads = heads;
  a.group = heads / cache->kv_heads;
  a.group_mul = a.group == 1 ? 0u : (unsigned)((1ull << 32) / (unsigned)a.group + 1);
  a.causal = causal != 0;
  a.window = window >= seqs->max_len ? 0 : window;          // no position is that far back (and none less its window passes 32 bits)
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cache->dtype == PISA_CACHE_FP32) return cuda_status(launch_attention_fp32(a, cache->head_dim, ws, st));
  const unsigned long long wait_ns = g_test_wait_ns ? g_test_wait_ns : kWaitLimitNs;
  if ((long long)seqs->max_new * a.group <= kMaxFewRows)
    return cuda_status(launch_attention_few(a, cache->head_dim, ws, wait_ns, g_test_fault, st));
  return cuda_status(launch_attention_chunk(a, cache->head_dim, ws, wait_ns, g_test_fault, st));
}

pisa_status pisa_testing_set_cache_fault(int32_t fault, uint64_t wait_limit_ns) {
  if (fault != PISA_TESTING_FAULT_NONE && fault != PISA_TESTING_FAULT_SKIP_KEYS_LOAD) return PISA_ERR_INVALID_ARG;
  g_test_fault = fault;
  g_test_wait_ns = wait_limit_ns;
  return PISA_OK;
}

}  // extern "C"
