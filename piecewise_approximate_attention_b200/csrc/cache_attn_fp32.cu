// Attention over the paged cache in full precision (fp32 pools): fp32 FMAs, shared out like the other
// kernels (cache_walk.cuh).
//
// An item is 16 or 64 rows (kRI rows a thread) against tiles of 64 keys, loaded by cp.async two tiles
// deep.  A thread holds kRI x 4 scores and kRI x D / 16 outputs; both products read float4 from shared
// memory and run on packed pairs (fma.f32x2): the scores' pairs are two neighbouring d, so each sum has
// two halves, the outputs' pairs two neighbouring columns.  Scores pass through shared memory between
// the products, where four threads a row keep its maximum and sum.  64 rows: bound by the FMA pipe,
// 2 * 64 * 64 * D FMAs a tile; 16 rows: 64 keys of K and V take the FMAs about as long as HBM takes to
// bring them.
// A tile that holds a value which is not finite where only some rows see it is flagged, and the rows
// of the share are computed again by row_attention, which reads only what a row sees.
#include "cache_row.cuh"
#include "cache_walk.cuh"
#include "sm100.cuh"

namespace pisa {
namespace cache {
namespace {
using namespace sm100;

constexpr int kThreads = 256;
constexpr unsigned FULL = 0xffffffffu;

template <int D, int kRI>
struct alignas(16) Smem {
  static constexpr int kKeys = D == 128 ? 32 : 64;          // two blocks fit an SM
  static constexpr int kRows = 16 * kRI, kLd = D + 4;       // padded: 8 rows' float4 fall on all banks
  float q[kRows][kLd];
  float k[2][kKeys][kLd];
  float v[2][kKeys][kLd];
  float s[kRows][kKeys + 4];
  float f[kRows];                       // what O is scaled by before a tile's products
  float m[kRows], l[kRows];
  uint32_t bad[2][kKeys / 32];                   // keys of a tile whose page is missing
  uint8_t bad4[2][8];                   // the same, four keys a byte
  WalkScratch<kThreads / 32> walk;
  int last;
};

struct Params {
  AttnArgs a;
  int* counters;             // one a block, zero between calls
  float2* part_ml;           // [2 * blocks][64]
  float* part_o;             // [2 * blocks][64][D]
};

__device__ __forceinline__ void cp16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D, int kRI>
__global__ void __launch_bounds__(kThreads, 2) attn_fp32(const Params p) {
  using S = Smem<D, kRI>;
  constexpr int kRows = S::kRows, kKeys = S::kKeys;
  constexpr int kCols = D / 64, kKJ = kKeys / 16;           // a thread: float4 columns of O, keys of a row's scores
  constexpr int kQuads = kThreads / kKeys;                  // threads that load a key
  extern __shared__ __align__(16) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  griddep_wait();
  Walk<kKeys> w;
  if (!w.template start<kThreads>(a, sm.walk, kRI == 4 ? 6 : 4, 2, 1)) return;
  // products: rows rx + 16 i, keys kx + 16 j, columns 4 (kx) + 64 j
  const int rx = (lane >> 3) + 4 * (warp & 3), kx = (lane & 7) + 8 * (warp >> 2);
  // softmax: four threads a row (kRows * 4 threads)
  const int sr = tid >> 2, sq = tid & 3;
  const bool soft = sr < kRows;

  do {
    if (w.t_begin >= w.t_end) continue;
    const int rows = w.it.rows;
    __syncthreads();                                        // the item before is done with shared memory
    // kQuads threads a key.  The page of a tile's key is looked up a tile ahead of its loads.
    const int key_l = tid / kQuads;
    int page = -1;
    const auto look_up = [&](int t) {
      const int j = t * kKeys + key_l;
      page = t < w.t_end && j < w.s.len && j >= w.it.first ? load_page(a.seqs, a.pool, w.b, j) : -1;
    };
    const auto load_tile = [&](int t) {
      const int buf = t & 1, j = t * kKeys + key_l;
      const bool there = page >= 0;
      const size_t slot = there ? (size_t)((page * a.pool.kv_heads + w.h) * a.pool.page + (j & (a.pool.page - 1))) : 0;
      const float* ks = reinterpret_cast<const float*>(a.pool.k) + slot * D;
      const float* vs = reinterpret_cast<const float*>(a.pool.v) + slot * D;
#pragma unroll
      for (int x = 0; x < D / 4 / kQuads; ++x) {
        const int c = tid % kQuads + x * kQuads;
        cp16(&sm.k[buf][key_l][4 * c], ks + 4 * c, there);        // zeros where there is no key
        cp16(&sm.v[buf][key_l][4 * c], vs + 4 * c, there);
      }
      cp_commit();
      // a warp's 32 / kQuads keys: bits of the missing ones
      const unsigned miss = __ballot_sync(FULL, !there);
      if (lane == 0) {
        uint32_t bits = 0;
#pragma unroll
        for (int x = 0; x < 32 / kQuads; ++x) bits |= ((miss >> (kQuads * x)) & 1u) << x;
        if (kQuads == 4) reinterpret_cast<uint8_t*>(sm.bad[buf])[warp] = (uint8_t)bits;
        else sm.bad4[buf][warp] = (uint8_t)bits;
      }
      look_up(t + 1);
    };
    look_up(w.t_begin);
    load_tile(w.t_begin);
    for (int e = tid; e < kRows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int gr = w.row0() + r, i = token_of(a, gr), hh = w.h * a.group + gr - i * a.group;
        x = *reinterpret_cast<const float4*>(a.q.data + w.b * a.q.seq + (long long)(w.s.row0 + i) * a.q.row +
                                             (long long)hh * a.q.head + c * 16);
      }
      *reinterpret_cast<float4*>(&sm.q[r][4 * c]) = x;
    }
    int first = 0, last = w.s.len;                          // of my softmax row
    if (soft && sr < rows) visible(a, w.s.len, w.s.len - w.s.n + token_of(a, w.row0() + sr), &first, &last);
    float m = -INFINITY, l = 0.f;
    // keys that all rows see: tiles inside need no care
    int af, al;
    {
      int f1, l1;
      visible(a, w.s.len, w.s.len - w.s.n + token_of(a, w.row0()), &af, &al);
      visible(a, w.s.len, w.s.len - w.s.n + token_of(a, w.row0() + rows - 1), &f1, &l1);
      af = max(af, f1);
      al = min(al, l1);
    }
    uint64_t o[kRI][kCols][2];
#pragma unroll
    for (int i = 0; i < kRI; ++i)
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[i][c][0] = o[i][c][1] = 0ull;
    bool odd = false;

    for (int t = w.t_begin; t < w.t_end; ++t) {
      const int buf = t & 1;
      if (t + 1 < w.t_end) {
        load_tile(t + 1);
        cp_wait<1>();
      } else {
        cp_wait<0>();
      }
      __syncthreads();
      const int j0 = t * kKeys;
      if (j0 < af || j0 + kKeys > al) {                     // a value that is not finite and not seen by all
        bool here = false;
        for (int e = tid; e < kKeys * (D / 4); e += kThreads) {
          const float4 x = *reinterpret_cast<const float4*>(&sm.v[buf][e / (D / 4)][e % (D / 4) * 4]);
          here = here || !isfinite(x.x) || !isfinite(x.y) || !isfinite(x.z) || !isfinite(x.w);
        }
        odd = __syncthreads_or(here) || odd;
      }
      // ---- scores ----
      uint64_t acc[kRI][kKJ];
#pragma unroll
      for (int i = 0; i < kRI; ++i)
#pragma unroll
        for (int j = 0; j < kKJ; ++j) acc[i][j] = 0ull;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        ulonglong2 qv[kRI], kv[kKJ];
#pragma unroll
        for (int i = 0; i < kRI; ++i) qv[i] = *reinterpret_cast<const ulonglong2*>(&sm.q[rx + 16 * i][d]);
#pragma unroll
        for (int j = 0; j < kKJ; ++j) kv[j] = *reinterpret_cast<const ulonglong2*>(&sm.k[buf][kx + 16 * j][d]);
#pragma unroll
        for (int i = 0; i < kRI; ++i)
#pragma unroll
          for (int j = 0; j < kKJ; ++j) {
            acc[i][j] = f2_fma(qv[i].x, kv[j].x, acc[i][j]);
            acc[i][j] = f2_fma(qv[i].y, kv[j].y, acc[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < kRI; ++i)
#pragma unroll
        for (int j = 0; j < kKJ; ++j) {
          float x, y;
          f2_unpack(acc[i][j], x, y);
          sm.s[rx + 16 * i][kx + 16 * j] = (x + y) * a.scale_log2;
        }
      __syncthreads();
      // ---- weights: my keys are sq, sq + 4, ... ----
      if (soft) {
        uint32_t bad[kKeys / 32];
        if (kQuads == 4) {
#pragma unroll
          for (int e = 0; e < kKeys / 32; ++e) bad[e] = sm.bad[buf][e];
        } else {
          bad[0] = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) bad[0] |= (uint32_t)sm.bad4[buf][e] << (4 * e);
        }
        constexpr int kMine = kKeys / 4;
        float x[kMine], mx = -INFINITY;
        const bool care = j0 < af || j0 + kKeys > al || (bad[0] | bad[kKeys / 32 - 1]);
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
          const int key = sq + 4 * e;
          x[e] = sm.s[sr][key];
          if (care && (j0 + key < first || j0 + key >= last || ((bad[key >> 5] >> (key & 31)) & 1u))) x[e] = -INFINITY;
          mx = fmaxf(mx, x[e]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
        const float m_new = fmaxf(m, mx), base = m_new == -INFINITY ? 0.f : m_new;
        const float f = exp2f(m - base);                    // 0 when m = -inf
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
          x[e] = exp2f(x[e] - base);
          sum += x[e];
          sm.s[sr][sq + 4 * e] = x[e];
        }
        m = m_new;
        l = l * f + sum;                                    // of my keys
        if (sq == 0) sm.f[sr] = f;
      }
      __syncthreads();
      // ---- O = O f + P V ----
#pragma unroll
      for (int i = 0; i < kRI; ++i) {
        const float f = sm.f[rx + 16 * i];
        const uint64_t f2 = f2_pack(f, f);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          o[i][c][0] = f2_fma(o[i][c][0], f2, 0ull);
          o[i][c][1] = f2_fma(o[i][c][1], f2, 0ull);
        }
      }
#pragma unroll 2
      for (int key = 0; key < kKeys; key += 4) {
        float4 pw[kRI];
#pragma unroll
        for (int i = 0; i < kRI; ++i) pw[i] = *reinterpret_cast<const float4*>(&sm.s[rx + 16 * i][key]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ulonglong2 vv[kCols];
#pragma unroll
          for (int c = 0; c < kCols; ++c) vv[c] = *reinterpret_cast<const ulonglong2*>(&sm.v[buf][key + e][4 * kx + 64 * c]);
#pragma unroll
          for (int i = 0; i < kRI; ++i) {
            const float x = e == 0 ? pw[i].x : e == 1 ? pw[i].y : e == 2 ? pw[i].z : pw[i].w;
            const uint64_t x2 = f2_pack(x, x);
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              o[i][c][0] = f2_fma(x2, vv[c].x, o[i][c][0]);
              o[i][c][1] = f2_fma(x2, vv[c].y, o[i][c][1]);
            }
          }
        }
      }
      __syncthreads();                                      // the tile's buffers may be filled again
    }
    // ---- the rows' results: complete, or a part of an item that other blocks work on too ----
    l += __shfl_xor_sync(FULL, l, 1);
    l += __shfl_xor_sync(FULL, l, 2);
    if (soft && sq == 0) {
      sm.m[sr] = m;
      sm.l[sr] = l;
    }
    __syncthreads();
    const int c0 = w.first_block(), c1 = w.last_block();
    const size_t part = (size_t)w.part() * kMaxFewRows;
    const auto finish = [&](int r, float mr, float lr) {    // once a row
      const int gr = w.row0() + r, i = token_of(a, gr), hh = w.h * a.group + gr - i * a.group;
      float* lse = lse_at(a, w.b, w.s, i, hh);
      if (lse) *lse = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * 0.6931471805599453f;
    };
    const auto out_row = [&](int r) {
      const int gr = w.row0() + r, i = token_of(a, gr), hh = w.h * a.group + gr - i * a.group;
      return reinterpret_cast<float*>(a.o.data + w.b * a.o.seq + (long long)(w.s.row0 + i) * a.o.row + (long long)hh * a.o.head);
    };
    if (odd) {
      // rare: row by row, a warp a row
      for (int r = warp; r < rows; r += kThreads / 32) {
        int f0, l0;
        visible(a, w.s.len, w.s.len - w.s.n + token_of(a, w.row0() + r), &f0, &l0);
        float mr, lr, acc[D / 32];
        row_attention<float, D>(a, w.b, w.h, sm.q[r], max(f0, w.t_begin * kKeys), min(l0, w.t_end * kKeys), &mr, &lr, acc);
        const float inv = lr == 0.f ? 0.f : 1.f / lr;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          if (c0 == c1) out_row(r)[c * 32 + lane] = acc[c] * inv;
          else p.part_o[(part + r) * D + c * 32 + lane] = acc[c];
        }
        if (lane == 0) {
          if (c0 == c1) finish(r, mr, lr);
          else p.part_ml[part + r] = make_float2(mr, lr);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRI; ++i) {
        const int r = rx + 16 * i;
        if (r >= rows) continue;
        const float lr = sm.l[r], inv = c0 != c1 ? 1.f : lr == 0.f ? 0.f : 1.f / lr;      // NaN sums stay NaN
        float* dst = c0 == c1 ? out_row(r) : p.part_o + (part + r) * D;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          float4 x;
          f2_unpack(o[i][c][0], x.x, x.y);
          f2_unpack(o[i][c][1], x.z, x.w);
          *reinterpret_cast<float4*>(dst + 4 * kx + 64 * c) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        }
        if (kx == 0) {
          if (c0 == c1) finish(r, sm.m[r], lr);
          else p.part_ml[part + r] = make_float2(sm.m[r], lr);
        }
      }
    }
    if (c0 != c1) {
      // the block that ends last joins the parts, in their order
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const bool done = atomicAdd(p.counters + c0, 1) == c1 - c0;
        if (done) p.counters[c0] = 0;                       // as the next call finds it
        sm.last = done;
      }
      __syncthreads();
      if (sm.last) {
        __threadfence();
        constexpr int kLanes = D / 4;
        const int col = (tid % kLanes) * 4;
        for (int r = tid / kLanes; r < rows; r += kThreads / kLanes) {
          float mm = -INFINITY;
          for (int c = c0; c <= c1; ++c) mm = fmaxf(mm, __ldcg(&p.part_ml[(size_t)(2 * c + (c == c0)) * kMaxFewRows + r]).x);
          const float base = mm == -INFINITY ? 0.f : mm;
          float ll = 0.f;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int c = c0; c <= c1; ++c) {
            const size_t at = (size_t)(2 * c + (c == c0)) * kMaxFewRows + r;
            const float2 ml = __ldcg(&p.part_ml[at]);
            const float4 po = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + col));
            const float f = exp2f(ml.x - base);
            ll = fmaf(ml.y, f, ll);
            x.x = fmaf(po.x, f, x.x);
            x.y = fmaf(po.y, f, x.y);
            x.z = fmaf(po.z, f, x.z);
            x.w = fmaf(po.w, f, x.w);
          }
          const float inv = ll == 0.f ? 0.f : 1.f / ll;
          *reinterpret_cast<float4*>(out_row(r) + col) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
          if (col == 0) finish(r, mm, ll);
        }
      }
    }
  } while (w.next(a));
}

template <int D, int kRI>
cudaError_t launch(const Params& p, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(Smem<D, kRI>);
  if ((e = set_max_dynamic_smem(reinterpret_cast<const void*>(attn_fp32<D, kRI>), smem))) return e;
  const int per_sm = smem <= 113 * 1024 ? 2 : 1;
  return launch_after(attn_fp32<D, kRI>, dim3(min(per_sm * sms, kMaxFewBlocks)), kThreads, smem, st, p);
}

}  // namespace

cudaError_t launch_attention_fp32(const AttnArgs& a, int d, void* ws, cudaStream_t st) {
  Params p;
  p.a = a;
  char* w = static_cast<char*>(ws);
  p.counters = reinterpret_cast<int*>(w + kCountersAt);
  p.part_ml = reinterpret_cast<float2*>(w + kPartialsAt);
  p.part_o = reinterpret_cast<float*>(w + kPartialsAt + sizeof(float2) * 2 * kMaxFewBlocks * kMaxFewRows);
  const bool few = (long long)a.seqs.max_new * a.group <= 16;
  if (d == 64) return few ? launch<64, 1>(p, st) : launch<64, 4>(p, st);
  return few ? launch<128, 1>(p, st) : launch<128, 4>(p, st);
}

}  // namespace cache
}  // namespace pisa
