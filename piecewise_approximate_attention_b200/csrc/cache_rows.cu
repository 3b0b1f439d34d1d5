// Appending tokens to the paged cache and reading them back (pisa_cache_append, pisa_cache_read).
//
// Both move rows of head_dim elements between a strided token tensor and the pages; e4m3 pools
// quantise on the way in (one power-of-two scale per row) and give exact bf16 values on the way out.
// HBM-bound: each row is read once and written once.  A thread moves 16 bytes of the token tensor
// and of the pool's matching piece; kRows rows of K and of V per thread are loaded before any is
// stored, so that enough bytes are in flight.  A block takes consecutive tokens of one head, which
// are consecutive in a page and (for [B, H, L, d] tensors) in the token tensor.  Read back: 32760 tokens
// of 12 heads in 62.7 us (bf16, 6.42 TB/s) and 49.4 us (e4m3, 6.1 TB/s).
#include "cache.cuh"
#include "sm100.cuh"

namespace pisa {
namespace cache {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 2;             // tokens a thread moves (32760 tokens, 12 heads, e4m3: 53.9 us with 1, 49.4 with 2, 49.9 with 3)

// Elements of one 16-byte piece of a token tensor.
template <typename T> constexpr int kPiece = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack8(uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Quantises the 8 elements that each of D/8 neighbouring lanes holds of one row.
template <int D>
__device__ __forceinline__ uint2 quantise(uint4 u, uint8_t* exp_byte) {
  float x[8];
  unpack8(u, x);
  uint32_t m = 0;                    // magnitudes of finite numbers order like their bit patterns
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
    m = max(m, b <= 0x7f800000u ? b : 0u);   // NaN has no part in the scale
  }
#pragma unroll
  for (int d = D / 16; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  // m = f * 2^E, 448 = 1.75 * 2^8: the smallest e with m <= 448 * 2^e is E - 8 if f <= 1.75, else E - 7
  int e = (int)((m + 0x1fffffu) >> 23) - 8 - kExpBias;
  e = max(-kExpLimit, min(kExpLimit, e));
  const float inv = pow2(-e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
  *exp_byte = (uint8_t)(e + kExpBias);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// 8 codes times 2^e as bf16, exact: |e| <= 50, and a code is a multiple of 2^-9 up to 448.
__device__ __forceinline__ uint4 dequantise(uint2 c, uint8_t exp_byte) {
  const float s = pow2((int)exp_byte - kExpBias);
  uint32_t w[4];
  const uint32_t in[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_to_f16x2((uint16_t)(in[i >> 1] >> (16 * (i & 1))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// T: element of the token tensors.  kF8: e4m3 pool (T is bf16).  kAppend: into the pool, else out of it.
template <typename T, int D, bool kF8, bool kAppend>
__global__ void __launch_bounds__(kThreads) move_rows_kernel(Pool pool, Seqs seqs, Rows kr, Rows vr) {
  constexpr int kLanes = D / kPiece<T>;          // threads a row
  constexpr int kTokens = kThreads / kLanes;     // rows a step
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int b = blockIdx.y, head = blockIdx.x % pool.kv_heads;
  const int t0 = blockIdx.x / pool.kv_heads * (kTokens * kRows);
  Seq s;
  if (!load_seq(seqs, b, min(kr.rows, vr.rows), &s) || t0 >= s.n) return;
  if (s.n > s.len) {
    set_status(seqs.status, PISA_DEVERR_BAD_LENGTH);
    return;
  }
  const int lane = threadIdx.x % kLanes, t = t0 + threadIdx.x / kLanes;
  const long long kbase = (long long)b * kr.seq + (long long)head * kr.head + lane * 16;
  const long long vbase = (long long)b * vr.seq + (long long)head * vr.head + lane * 16;
  int slot[kRows];                               // row number in the pool, -1: nothing to move
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int i = t + u * kTokens, p = s.len - s.n + i;
    slot[u] = -1;
    if (i < s.n) {
      const int pg = load_page(seqs, pool, b, p);
      if (pg >= 0) slot[u] = (pg * pool.kv_heads + head) * pool.page + (p & (pool.page - 1));
    }
  }
  constexpr int kBytes = kF8 ? D : D * (int)sizeof(T);   // of a pool row
  constexpr int kOut = kF8 ? 8 : 16;                     // of a thread's piece of it
  char* pk = const_cast<char*>(pool.k) + lane * kOut;
  char* pv = const_cast<char*>(pool.v) + lane * kOut;
  if (kAppend) {
    uint4 k[kRows], v[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      k[u] = v[u] = make_uint4(0, 0, 0, 0);
      if (slot[u] >= 0) {
        const long long r = s.row0 + t + u * kTokens;
        k[u] = *reinterpret_cast<const uint4*>(kr.data + kbase + r * kr.row);
        v[u] = *reinterpret_cast<const uint4*>(vr.data + vbase + r * vr.row);
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if constexpr (kF8) {
        uint8_t ke, ve;                          // the whole warp takes part in the reductions
        const uint2 kc = quantise<D>(k[u], &ke), vc = quantise<D>(v[u], &ve);
        if (slot[u] >= 0) {
          *reinterpret_cast<uint2*>(pk + (size_t)slot[u] * kBytes) = kc;
          *reinterpret_cast<uint2*>(pv + (size_t)slot[u] * kBytes) = vc;
          if (lane == 0) {
            const_cast<uint8_t*>(pool.k_exp)[slot[u]] = ke;
            const_cast<uint8_t*>(pool.v_exp)[slot[u]] = ve;
          }
        }
      } else if (slot[u] >= 0) {
        *reinterpret_cast<uint4*>(pk + (size_t)slot[u] * kBytes) = k[u];
        *reinterpret_cast<uint4*>(pv + (size_t)slot[u] * kBytes) = v[u];
      }
    }
  } else {
    using Piece = typename std::conditional<kF8, uint2, uint4>::type;
    Piece k[kRows], v[kRows];
    uint8_t ke[kRows], ve[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (slot[u] >= 0) {
        k[u] = *reinterpret_cast<const Piece*>(pk + (size_t)slot[u] * kBytes);
        v[u] = *reinterpret_cast<const Piece*>(pv + (size_t)slot[u] * kBytes);
        if constexpr (kF8) {
          ke[u] = pool.k_exp[slot[u]];
          ve[u] = pool.v_exp[slot[u]];
        }
      }
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (slot[u] >= 0) {
        const long long r = s.row0 + t + u * kTokens;
        uint4 ko, vo;
        if constexpr (kF8) {
          ko = dequantise(k[u], ke[u]);
          vo = dequantise(v[u], ve[u]);
        } else {
          ko = k[u];
          vo = v[u];
        }
        *reinterpret_cast<uint4*>(kr.data + kbase + r * kr.row) = ko;
        *reinterpret_cast<uint4*>(vr.data + vbase + r * vr.row) = vo;
      }
  }
}

template <typename T, int D, bool kF8, bool kAppend>
cudaError_t launch(const Pool& pool, const Seqs& seqs, const Rows& k, const Rows& v, cudaStream_t st) {
  constexpr int kTile = kThreads / (D / kPiece<T>) * kRows;
  const long long chunks = ((long long)seqs.max_new + kTile - 1) / kTile;
  if (chunks * pool.kv_heads > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_after(move_rows_kernel<T, D, kF8, kAppend>, dim3((unsigned)(chunks * pool.kv_heads), seqs.batch), kThreads, 0, st,
                      pool, seqs, k, v);
}

template <bool kAppend>
cudaError_t launch_any(const Pool& pool, int d, const Seqs& seqs, const Rows& k, const Rows& v, cudaStream_t st) {
  switch (pool.dtype) {
    case PISA_CACHE_FP32:
      return d == 64 ? launch<float, 64, false, kAppend>(pool, seqs, k, v, st)
                     : launch<float, 128, false, kAppend>(pool, seqs, k, v, st);
    case PISA_CACHE_E4M3:
      return d == 64 ? launch<__nv_bfloat16, 64, true, kAppend>(pool, seqs, k, v, st)
                     : launch<__nv_bfloat16, 128, true, kAppend>(pool, seqs, k, v, st);
    default:
      return d == 64 ? launch<__nv_bfloat16, 64, false, kAppend>(pool, seqs, k, v, st)
                     : launch<__nv_bfloat16, 128, false, kAppend>(pool, seqs, k, v, st);
  }
}

}  // namespace

cudaError_t launch_append(const Pool& pool, int d, const Seqs& seqs, const Rows& k, const Rows& v, cudaStream_t st) {
  return launch_any<true>(pool, d, seqs, k, v, st);
}

cudaError_t launch_read(const Pool& pool, int d, const Seqs& seqs, const Rows& k, const Rows& v, cudaStream_t st) {
  return launch_any<false>(pool, d, seqs, k, v, st);
}

}  // namespace cache
}  // namespace pisa
