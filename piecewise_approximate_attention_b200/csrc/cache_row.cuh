// One query row over a run of cached keys by one warp: what the tiled kernels fall back to for data
// that their products cannot take (values that are not finite and not seen by all rows of a tile).
#pragma once

#include "cache.cuh"
#include "sm100.cuh"

namespace pisa {
namespace cache {

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

// Keys [first, last) of sequence b and key/value head kvh; q: the query row in shared memory (float).
// For each run of 32 keys, lane j computes the logit of key j, the warp joins them into the running
// maximum m (base 2) and sum l, and lane c adds the values to columns c, c + 32, ... of the row (acc).
// K: element of the pool (float, bf16, uint8_t for e4m3 codes).  alive: where to say every 1024 keys that the warp is at
// work (cache_pipe.cuh), if not null.
template <typename K, int D>
__device__ __forceinline__ void row_attention(const AttnArgs& a, int b, int kvh, const float* q, int first, int last, float* m_out,
                              float* l_out, float* acc, volatile unsigned long long* alive = nullptr) {
  constexpr int kPer = 16 / (int)sizeof(K), kCols = D / 32;
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
  for (int j0 = first & ~31; j0 < last; j0 += 32) {
    if (alive && lane == 0 && (j0 & 1023) == 0) *alive = sm100::globaltimer_ns();
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
        for (int e = 0; e < kPer; ++e) dot = fmaf(q[c * kPer + e], x[e], dot);
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
  *m_out = m;
  *l_out = l;
}

}  // namespace cache
}  // namespace pisa
