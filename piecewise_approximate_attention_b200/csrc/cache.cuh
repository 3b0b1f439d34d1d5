// Shared definitions of the paged key/value cache kernels (internal; the C ABI is pisa_cache.h).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "pisa_cache.h"

namespace pisa {
namespace cache {

constexpr int kExpBias = 127;
constexpr int kExpLimit = 50;      // stored scales lie in [2^-50, 2^50] (pisa_cache.h)

// Token tensor with its element size applied: byte strides.
struct Rows {
  char* data;
  int rows;
  long long seq, row, head;
};

// What every kernel needs to find tokens; passed by value.
struct Pool {
  const char* k;
  const char* v;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  int num_pages, kv_heads, page, page_log2, dtype;
};

struct Seqs {
  int batch, max_pages, max_len, max_new;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* starts;
  const int32_t* counts;
  int* status;
};

// Sequence b as the device arrays describe it: its length, its new tokens and its first row.
struct Seq {
  int len, n, row0;
};

// False if its count or start is out of range (nothing of it may be read or written); a length out
// of range counts as empty.  Both set the status word.
__device__ __forceinline__ bool load_seq(const Seqs& s, int b, int rows, Seq* q) {
  q->len = s.lens[b];
  if (q->len < 0 || q->len > s.max_len) {
    set_status(s.status, PISA_DEVERR_BAD_LENGTH);
    q->len = 0;
  }
  q->row0 = 0;
  if (s.starts) {
    const int a = s.starts[b], e = s.starts[b + 1];
    q->row0 = a;
    q->n = 0;
    if (a < 0 || e < a || e > rows || e - a > s.max_new) {
      set_status(s.status, PISA_DEVERR_BAD_LENGTH);
      return false;
    }
    q->n = e - a;
  } else {
    q->n = s.counts ? s.counts[b] : s.max_new;
    if (q->n < 0 || q->n > s.max_new) {
      set_status(s.status, PISA_DEVERR_BAD_LENGTH);
      q->n = 0;
      return false;
    }
  }
  return true;
}

// Page of position p (p < len <= max_pages * page), -1 if the table holds no page of the pool.
__device__ __forceinline__ int load_page(const Seqs& s, const Pool& c, int b, int p) {
  const int pg = s.table[(size_t)b * s.max_pages + (p >> c.page_log2)];
  if (pg < 0 || pg >= c.num_pages) {
    set_status(s.status, PISA_DEVERR_BAD_PAGE);
    return -1;
  }
  return pg;
}

// Two e4m3 codes (low byte first) as fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// One attention call.
struct AttnArgs {
  Pool pool;
  Seqs seqs;
  Rows q, o;
  float* lse;
  int heads, group, causal, window;
  unsigned group_mul;              // floor(2^32 / group) + 1, 0 for group 1
  float scale_log2;                // softmax_scale * log2(e)
};

// x / group for 0 <= x < 2^31.  The product with group_mul exceeds x * 2^32 / group by x * e / group with
// 0 < e <= group: exact while x * group < 2^32, else a division.
__device__ __forceinline__ int token_of(const AttnArgs& a, int x) {
  if (a.group_mul == 0u) return x;
  if ((unsigned long long)(unsigned)x * (unsigned)a.group >> 32) return x / a.group;
  return (int)__umulhi((unsigned)x, a.group_mul);
}

// Keys that position p of a sequence of `len` tokens sees: [first, last).
__device__ __forceinline__ void visible(const AttnArgs& a, int len, int p, int* first, int* last) {
  *last = a.causal ? min(len, p + 1) : len;
  *first = a.window > 0 ? max(0, min(*last, p - a.window + 1)) : 0;
  if (*last < 0) *last = 0;
  if (*first > *last) *first = *last;
}

__device__ __forceinline__ float* lse_at(const AttnArgs& a, int b, const Seq& s, int i, int h) {
  if (!a.lse) return nullptr;
  return a.seqs.starts ? a.lse + ((size_t)(s.row0 + i) * a.heads + h)
                       : a.lse + ((size_t)b * a.heads + h) * a.q.rows + i;
}

// Workspace: status word, counters of the few-row kernel's blocks (zero between calls), words for the
// chunk kernel's joining, partial results of items that several blocks share: per block two of them (the end of one item, the beginning of another).
constexpr int kMaxFewBlocks = 296, kMaxFewRows = 64;       // few-row attention: two blocks on each of 148 SMs
constexpr size_t kCountersAt = kStatusBytes;
constexpr size_t kSplitAt = kCountersAt + (kMaxFewBlocks * sizeof(int) + 255) / 256 * 256;
constexpr int kMaxChunkBlocks = 148, kMaxChunkRows = 256;  // chunk attention: one block an SM
constexpr size_t kPartialsAt = kSplitAt + (kMaxChunkBlocks * sizeof(int4) + 255) / 256 * 256;
inline size_t partials_bytes(int d) {
  const size_t few = (size_t)kMaxFewBlocks * kMaxFewRows, chunk = (size_t)kMaxChunkBlocks * kMaxChunkRows;
  return 2 * (few > chunk ? few : chunk) * (d + 2) * sizeof(float);
}

// Launches a kernel that may be scheduled while the one before it in the stream still runs
// (programmatic stream serialization).  Such a kernel begins with sm100.cuh's griddep_wait() in every
// thread, before it touches global memory, so that a stream's kernels still follow one another.
template <typename... K, typename... A>
cudaError_t launch_after(void (*kernel)(K...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) cudaGetLastError();      // reported here, not by the next call that asks
  return e;
}

// ---- launchers ----
cudaError_t launch_append(const Pool& pool, int head_dim, const Seqs& seqs, const Rows& k, const Rows& v, cudaStream_t st);
cudaError_t launch_read(const Pool& pool, int head_dim, const Seqs& seqs, const Rows& k, const Rows& v, cudaStream_t st);
// fp32 pools.
cudaError_t launch_attention_fp32(const AttnArgs& a, int head_dim, void* ws, cudaStream_t st);
// wait_ns: the limit of the kernels' waits; fault: test-only fault injection (pisa_testing.h), 0 in normal calls.
// bf16 and e4m3 pools, at most kMaxFewRows rows (new tokens times query heads of a key/value head).
cudaError_t launch_attention_few(const AttnArgs& a, int head_dim, void* ws, unsigned long long wait_ns, int fault, cudaStream_t st);
// bf16 and e4m3 pools, any number of rows.
cudaError_t launch_attention_chunk(const AttnArgs& a, int head_dim, void* ws, unsigned long long wait_ns, int fault, cudaStream_t st);

}  // namespace cache
}  // namespace pisa
