// Attention over the paged cache, plain form: one warp per new token and head.
//
// For each run of 32 keys, lane j computes the logit of key j (the query sits in shared memory, read
// as broadcasts), the warp joins them into the running maximum and sum of the softmax, and then lane
// c adds the keys' values to its head_dim / 32 columns.  Only keys that the token sees are read.
#include "cache.cuh"

namespace pisa {
namespace cache {
namespace {

constexpr int kWarps = 4;

// 16 bytes of a pool row as floats (4 fp32, 8 bf16 or 16 e4m3 numbers).
__device__ __forceinline__ void piece(const float*, uint4 u, float* x) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void piece(const __nv_bfloat16*, uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ float2 codes2(uint16_t c) {
  const uint32_t h = e4m3x2_to_f16x2(c);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ void piece(const uint8_t*, uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = codes2((uint16_t)w[i]), b = codes2((uint16_t)(w[i] >> 16));
    x[4 * i] = a.x;
    x[4 * i + 1] = a.y;
    x[4 * i + 2] = b.x;
    x[4 * i + 3] = b.y;
  }
}

// K: element of the pool (float, bf16, uint8_t for e4m3 codes); T: element of q and o.
template <typename K, typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) attn_simt(const AttnArgs a) {
  constexpr int kPer = 16 / (int)sizeof(K);        // elements of a 16-byte piece
  constexpr int kCols = D / 32;
  __shared__ float qs[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  Seq s;
  if (!load_seq(a.seqs, b, a.q.rows, &s)) return;
  const long long row = (long long)blockIdx.x * kWarps + warp;
  const int i = (int)(row / a.heads), h = (int)(row % a.heads);
  if (i >= s.n) return;
  const int kvh = h / a.group;
  const long long qi = s.row0 + i;
  const T* q = reinterpret_cast<const T*>(a.q.data + b * a.q.seq + qi * a.q.row + (long long)h * a.q.head);
  for (int c = lane; c < D; c += 32) qs[warp][c] = to_f32(q[c]);
  __syncwarp();
  int first, last;
  visible(a, s.len, s.len - s.n + i, &first, &last);
  float m = -INFINITY, l = 0.f, acc[kCols] = {};
  for (int j0 = first & ~31; j0 < last; j0 += 32) {
    const int j = j0 + lane;
    int slot = -1;
    if (j >= first && j < last) {
      const int pg = load_page(a.seqs, a.pool, b, j);
      if (pg >= 0) slot = (pg * a.pool.kv_heads + kvh) * a.pool.page + (j & (a.pool.page - 1));
    }
    float sc = -INFINITY, vs = 1.f;
    if (slot >= 0) {
      const uint4* k = reinterpret_cast<const uint4*>(a.pool.k + (size_t)slot * D * sizeof(K));
      float dot = 0.f;
#pragma unroll
      for (int c = 0; c < D / kPer; ++c) {
        float x[kPer];
        piece(static_cast<const K*>(nullptr), k[c], x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) dot = fmaf(qs[warp][c * kPer + e], x[e], dot);
      }
      if (sizeof(K) == 1) {
        dot *= pow2((int)a.pool.k_exp[slot] - kExpBias);
        vs = pow2((int)a.pool.v_exp[slot] - kExpBias);
      }
      sc = dot * a.scale_log2;
    }
    float mx = sc;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float m_new = fmaxf(m, mx), base = m_new == -INFINITY ? 0.f : m_new;
    const float f = exp2f(m - base), p = slot >= 0 ? exp2f(sc - base) : 0.f;
    m = m_new;
    float sum = p;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = l * f + sum;
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] *= f;
    const float w = p * vs;
    for (int jj = 0; jj < 32; ++jj) {
      const float wj = __shfl_sync(0xffffffffu, w, jj);
      const int sj = __shfl_sync(0xffffffffu, slot, jj);
      if (sj < 0) continue;
      const K* v = reinterpret_cast<const K*>(a.pool.v) + (size_t)sj * D;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        float x;
        if constexpr (sizeof(K) == 1) x = codes2(v[c * 32 + lane]).x;
        else x = to_f32(v[c * 32 + lane]);
        acc[c] = fmaf(wj, x, acc[c]);
      }
    }
  }
  T* o = reinterpret_cast<T*>(a.o.data + b * a.o.seq + qi * a.o.row + (long long)h * a.o.head);
  const float inv = l == 0.f ? 0.f : 1.f / l;      // NaN sums stay NaN
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c * 32 + lane] = from_f32<T>(acc[c] * inv);
  float* lse = lse_at(a, b, s, i, h);
  if (lse && lane == 0) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <typename K, typename T, int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  const long long blocks = ((long long)a.seqs.max_new * a.heads + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  attn_simt<K, T, D><<<dim3((unsigned)blocks, a.seqs.batch), kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_simt(const AttnArgs& a, int d, cudaStream_t st) {
  switch (a.pool.dtype) {
    case PISA_CACHE_FP32:
      return d == 64 ? launch<float, float, 64>(a, st) : launch<float, float, 128>(a, st);
    case PISA_CACHE_E4M3:
      return d == 64 ? launch<uint8_t, __nv_bfloat16, 64>(a, st) : launch<uint8_t, __nv_bfloat16, 128>(a, st);
    default:
      return d == 64 ? launch<__nv_bfloat16, __nv_bfloat16, 64>(a, st)
                     : launch<__nv_bfloat16, __nv_bfloat16, 128>(a, st);
  }
}

}  // namespace cache
}  // namespace pisa
