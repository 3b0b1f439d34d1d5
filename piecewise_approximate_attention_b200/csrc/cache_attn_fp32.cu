// Attention over the paged cache in full precision (fp32 pools), shared out like the other kernels
// (cache_walk.cuh): two kernels, for at most 16 rows a key/value head (attn_few) and for more
// (attn_split).  Parts of an item are joined by the block that ends last.
//
// attn_few: 16 rows against tiles of 32 (D = 128) or 64 keys, loaded by cp.async two tiles deep, by fp32
// FMAs on packed pairs (fma.f32x2): the scores' pairs are two neighbouring d, so each sum has two
// halves, the outputs' pairs two neighbouring columns.  Scores pass through shared memory between the
// products, where four threads a row keep its maximum and sum.  Bound by what shared memory returns: four
// cycles for each warp's 16-byte loads.  One token, 16 heads on 4 (D = 128): 577 positions 15.5 us,
// 2000 18.5, 8000 35.5; 40 heads on 8, 4 sequences of up to 32760 positions 459 us.
//
// attn_split: 64 rows, 16 a warp, by the matrix pipe (mma.m16n8k16).  Every number is cut into three bf16
// pieces, h + m + l, which keep 24 bits; of the nine products of pieces the six that weigh 2^-16 and
// more are taken (h h, h m, m h, m m, h l, l h), so a product is off by at most 2^-22 of its size, as
// are fp32 sums of a few terms.  The tensor cores do not round their sums to nearest: the five
// small products are summed apart from h h, and a tile's P V is summed from zero and added to O by one
// fp32 FMA, so that no long sum runs through them.  Tiles of 32 (64) keys arrive as fp32 by cp.async
// while the tile before them is worked on, and are cut once for all four warps.  64 x 64 keys x D take 6 mma for
// each FMA's worth and still end in 2/3 of the time that FMAs fed from shared memory took: 333 tokens a
// sequence in a window of 1024 (two sequences, 8 heads, D = 64) 62 -> 45 us; 1000 tokens over 8000 (12
// heads, D = 128) 1489 -> 950 us, 52 TFLOP/s of fp32 work.  Two blocks of four warps an SM (255
// registers): the tensor pipe is busy 23% of the time, the rest is latency between a warp's steps.
//
// A tile that holds a value which is not finite (attn_few: where only some rows see it; attn_split: anywhere,
// and in Q, whose pieces would turn inf into NaN) is flagged, and the rows of the share are computed
// again by row_attention, which reads only what a row sees.
#include "cache_row.cuh"
#include "cache_walk.cuh"
#include "sm100.cuh"

namespace pisa {
namespace cache {
namespace {
using namespace sm100;

constexpr int kThreads = 256;
constexpr unsigned FULL = 0xffffffffu;

template <int D>
struct alignas(128) Smem {
  static constexpr int kKeys = D == 128 ? 32 : 64;          // two blocks fit an SM
  static constexpr int kRows = 16, kLd = D + 4;       // padded: 8 rows' float4 fall on all banks
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

// True in the block that ends last of those that share an item: it joins the parts.
__device__ __forceinline__ bool ends_last(const Params& p, int& joins, int c0, int c1) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool done = atomicAdd(p.counters + c0, 1) == c1 - c0;
    if (done) p.counters[c0] = 0;                           // as the next call finds it
    joins = done;
  }
  __syncthreads();
  if (!joins) return false;
  __threadfence();
  return true;
}
__device__ __forceinline__ size_t part_row(int c, int c0, int r) { return (size_t)(2 * c + (c == c0)) * kMaxFewRows + r; }
__device__ __forceinline__ void add_scaled(float4& x, float f, float4 y) {
  x.x = fmaf(y.x, f, x.x);
  x.y = fmaf(y.y, f, x.y);
  x.z = fmaf(y.z, f, x.z);
  x.w = fmaf(y.w, f, x.w);
}
__device__ __forceinline__ float4 scaled(float4 x, float f) { return make_float4(x.x * f, x.y * f, x.z * f, x.w * f); }

// Few rows can have many parts: each group of D / 4 threads sums every kGroups-th, then the groups' sums are added,
// in their order (2000 positions, 63 parts: 24 us with the parts one after another).  `sums`: [kGroups][16][D].
template <int D, int kT, typename Out, typename Finish>
__device__ __forceinline__ void join_few(const Params& p, float* top, float* total, float* sums, int rows, int c0, int c1,
                                         Out out_row, Finish finish) {
  constexpr int kLanes = D / 4, kGroups = kT / kLanes;
  const int tid = threadIdx.x, lane = tid & 31, g = tid / kLanes, col = (tid % kLanes) * 4;
  for (int r = tid >> 5; r < rows; r += kT / 32) {          // a warp a row: its maximum and sum
    float mm = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) mm = fmaxf(mm, __ldcg(&p.part_ml[part_row(c, c0, r)]).x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(FULL, mm, d));
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    for (int c = c0 + lane; c <= c1; c += 32) {
      const float2 ml = __ldcg(&p.part_ml[part_row(c, c0, r)]);
      ll = fmaf(ml.y, exp2f(ml.x - base), ll);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ll += __shfl_xor_sync(FULL, ll, d);
    if (lane == 0) {
      top[r] = base;
      total[r] = ll;
      finish(r, mm, ll);
    }
  }
  __syncthreads();
  for (int r = 0; r < rows; ++r) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = c0 + g; c <= c1; c += kGroups) {
      const size_t at = part_row(c, c0, r);
      add_scaled(x, exp2f(__ldcg(&p.part_ml[at]).x - top[r]), __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + col)));
    }
    *reinterpret_cast<float4*>(sums + (g * 16 + r) * D + col) = x;
  }
  __syncthreads();
  for (int r = g; r < rows; r += kGroups) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int y = 0; y < kGroups; ++y) add_scaled(x, 1.f, *reinterpret_cast<const float4*>(sums + (y * 16 + r) * D + col));
    *reinterpret_cast<float4*>(out_row(r) + col) = scaled(x, total[r] == 0.f ? 0.f : 1.f / total[r]);
  }
}

// Many rows: four of a thread's in flight.
template <int D, int kT, typename Out, typename Finish>
__device__ __forceinline__ void join(const Params& p, float* top, int rows, int c0, int c1, Out out_row, Finish finish) {
  const int tid = threadIdx.x;
  if (tid < rows) {
    float mm = -INFINITY;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) mm = fmaxf(mm, __ldcg(&p.part_ml[part_row(c, c0, tid)]).x);
    top[tid] = mm;
  }
  __syncthreads();
  constexpr int kLanes = D / 4, kStep = kT / kLanes, kBatch = 4;
  const int col = (tid % kLanes) * 4;
  for (int r0 = tid / kLanes; r0 < rows; r0 += kBatch * kStep) {
    float mm[kBatch], base[kBatch], ll[kBatch];
    float4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      mm[i] = top[min(r0 + i * kStep, rows - 1)];
      base[i] = mm[i] == -INFINITY ? 0.f : mm[i];
      ll[i] = 0.f;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 2
    for (int c = c0; c <= c1; ++c) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const size_t at = part_row(c, c0, min(r0 + i * kStep, rows - 1));
        const float2 ml = __ldcg(&p.part_ml[at]);
        const float f = exp2f(ml.x - base[i]);
        ll[i] = fmaf(ml.y, f, ll[i]);
        add_scaled(x[i], f, __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + col)));
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * kStep;
      if (r >= rows) break;
      *reinterpret_cast<float4*>(out_row(r) + col) = scaled(x[i], ll[i] == 0.f ? 0.f : 1.f / ll[i]);
      if (col == 0) finish(r, mm[i], ll[i]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) attn_few(const Params p) {
  using S = Smem<D>;
  constexpr int kRows = S::kRows, kKeys = S::kKeys;
  constexpr int kCols = D / 64, kKJ = kKeys / 16;           // a thread: float4 columns of O, keys of a row's scores
  constexpr int kQuads = kThreads / kKeys;                  // threads that load a key
  extern __shared__ __align__(128) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  griddep_wait();
  Walk<kKeys> w;
  if (!w.template start<kThreads>(a, sm.walk, 4, 2, 1)) return;
  // products: row rx, keys kx + 16 j, columns 4 (kx) + 64 j
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
    uint64_t o[kCols][2];
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[c][0] = o[c][1] = 0ull;
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
      uint64_t acc[kKJ];
#pragma unroll
      for (int j = 0; j < kKJ; ++j) acc[j] = 0ull;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        ulonglong2 kv[kKJ];
        const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(&sm.q[rx][d]);
#pragma unroll
        for (int j = 0; j < kKJ; ++j) kv[j] = *reinterpret_cast<const ulonglong2*>(&sm.k[buf][kx + 16 * j][d]);
#pragma unroll
        for (int j = 0; j < kKJ; ++j) {
          acc[j] = f2_fma(qv.x, kv[j].x, acc[j]);
          acc[j] = f2_fma(qv.y, kv[j].y, acc[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < kKJ; ++j) {
        float x, y;
        f2_unpack(acc[j], x, y);
        sm.s[rx][kx + 16 * j] = (x + y) * a.scale_log2;
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
      {
        const float f = sm.f[rx];
        const uint64_t f2 = f2_pack(f, f);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          o[c][0] = f2_fma(o[c][0], f2, 0ull);
          o[c][1] = f2_fma(o[c][1], f2, 0ull);
        }
      }
#pragma unroll 2
      for (int key = 0; key < kKeys; key += 4) {
        const float4 pw = *reinterpret_cast<const float4*>(&sm.s[rx][key]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ulonglong2 vv[kCols];
#pragma unroll
          for (int c = 0; c < kCols; ++c) vv[c] = *reinterpret_cast<const ulonglong2*>(&sm.v[buf][key + e][4 * kx + 64 * c]);
          const float x = e == 0 ? pw.x : e == 1 ? pw.y : e == 2 ? pw.z : pw.w;
          const uint64_t x2 = f2_pack(x, x);
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            o[c][0] = f2_fma(x2, vv[c].x, o[c][0]);
            o[c][1] = f2_fma(x2, vv[c].y, o[c][1]);
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
      const int r = rx;
      if (r < rows) {
        const float lr = sm.l[r], inv = c0 != c1 ? 1.f : lr == 0.f ? 0.f : 1.f / lr;      // NaN sums stay NaN
        float* dst = c0 == c1 ? out_row(r) : p.part_o + (part + r) * D;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          float4 x;
          f2_unpack(o[c][0], x.x, x.y);
          f2_unpack(o[c][1], x.z, x.w);
          *reinterpret_cast<float4*>(dst + 4 * kx + 64 * c) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        }
        if (kx == 0) {
          if (c0 == c1) finish(r, sm.m[r], lr);
          else p.part_ml[part + r] = make_float2(sm.m[r], lr);
        }
      }
    }
    if (c0 != c1 && ends_last(p, sm.last, c0, c1)) {
      static_assert(sizeof(sm.k) + sizeof(sm.v) >= kThreads / (D / 4) * 16 * D * sizeof(float), "the groups' sums");
      join_few<D, kThreads>(p, sm.m, sm.l, &sm.k[0][0][0], rows, c0, c1, out_row, finish);      // over K and V
    }
  } while (w.next(a));
}

// ---- more than 16 rows: the matrix pipe on split numbers ----

// a = h + m + l with 8 significant bits each, and at most 2^-24 |a| left out; for two numbers at once.
__device__ __forceinline__ void split2(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  const auto pack = [](float a, float b) {
    uint32_t u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(b), "f"(a));
    return u;
  };
  h = pack(x, y);
  x -= __uint_as_float(h << 16);
  y -= __uint_as_float(h & 0xffff0000u);
  m = pack(x, y);
  l = pack(x - __uint_as_float(m << 16), y - __uint_as_float(m & 0xffff0000u));
}
// a bit for each of two bf16 numbers that is not finite
__device__ __forceinline__ uint32_t not_finite2(uint32_t h) { return ((h & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

constexpr int kSplitThreads = 128;

template <int D>
struct alignas(128) SplitSmem {
  static constexpr int kKeys = D == 128 ? 32 : 64;
  uint8_t piece[2][3][kKeys * D * 2];   // K, V: h, m, l as rows of bf16, 16-byte units swizzled; before that Q's
  float raw[2][kKeys][D];               // K, V as they are stored
  float m[kMaxFewRows], l[kMaxFewRows];
  uint8_t bad[2][kKeys / 8];            // keys of a tile whose page is missing
  WalkScratch<kSplitThreads / 32> walk;
  int last;
};

// `n` rows of D floats into three arrays of bf16 pieces, `stride` bytes apart; src(row, c): float4 number c of a row
template <int D, typename Src>
__device__ __forceinline__ uint32_t split_rows(uint8_t* dst, int stride, int n, Src src) {
  constexpr int kUnits = D / 4;
  uint32_t bad = 0;
#pragma unroll 8
  for (int e = threadIdx.x; e < n * kUnits; e += kSplitThreads) {
    const int r = e / kUnits, c = e % kUnits;
    const float4 x = src(r, c);
    uint2 h, m, l;
    split2(x.x, x.y, h.x, m.x, l.x);
    split2(x.z, x.w, h.y, m.y, l.y);
    bad |= not_finite2(h.x) | not_finite2(h.y);
    const int at = r * (D * 2) + (((c >> 1) ^ (r & 7)) << 4) + ((c & 1) << 3);
    *reinterpret_cast<uint2*>(dst + at) = h;
    *reinterpret_cast<uint2*>(dst + stride + at) = m;
    *reinterpret_cast<uint2*>(dst + 2 * stride + at) = l;
  }
  return bad;
}

template <int D>
__global__ void __launch_bounds__(kSplitThreads, 2) attn_split(const Params p) {
  using S = SplitSmem<D>;
  constexpr int kKeys = S::kKeys, kT = kSplitThreads;
  constexpr int kPiece = kKeys * D * 2;                     // bytes of an array of pieces
  constexpr int kQuads = kT / kKeys;                        // threads that load a key
  static_assert(kMaxFewRows * D * 2 <= 2 * kPiece, "Q's pieces fit where K's and V's are");
  extern __shared__ __align__(128) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  griddep_wait();
  Walk<kKeys> w;
  if (!w.template start<kT>(a, sm.walk, 6, 2, 1)) return;
  const uint32_t pieces = smem_u32(sm.piece);
  // ldmatrix rows of this lane: A and V take (8 rows, 8 more) x (8 columns, 8 more), K the other way round
  const int r_av = lane & 15, c_av = lane >> 4, r_k = (lane & 7) + ((lane >> 4) << 3), c_k = (lane >> 3) & 1;
  const auto at = [](int row, int unit) { return (uint32_t)(row * (D * 2) + ((unit ^ (row & 7)) << 4)); };

  do {
    if (w.t_begin >= w.t_end) continue;
    const int rows = w.it.rows;
    __syncthreads();                                        // the item before is done with shared memory
    const int key_l = tid / kQuads;
    int page = -1;
    const auto look_up = [&](int t) {                       // a tile ahead of its loads
      const int j = t * kKeys + key_l;
      page = t < w.t_end && j < w.s.len && j >= w.it.first ? load_page(a.seqs, a.pool, w.b, j) : -1;
    };
    const auto load_tile = [&](int t) {
      const int j = t * kKeys + key_l;
      const bool there = page >= 0;
      const size_t slot = there ? (size_t)((page * a.pool.kv_heads + w.h) * a.pool.page + (j & (a.pool.page - 1))) : 0;
      const float* ks = reinterpret_cast<const float*>(a.pool.k) + slot * D;
      const float* vs = reinterpret_cast<const float*>(a.pool.v) + slot * D;
#pragma unroll
      for (int x = 0; x < D / 4 / kQuads; ++x) {
        const int c = tid % kQuads + x * kQuads;
        cp16(&sm.raw[0][key_l][4 * c], ks + 4 * c, there);  // zeros where there is no key
        cp16(&sm.raw[1][key_l][4 * c], vs + 4 * c, there);
      }
      cp_commit();
      const unsigned miss = __ballot_sync(FULL, !there);    // a warp's 32 / kQuads keys
      if (lane == 0) {
        uint32_t bits = 0;
#pragma unroll
        for (int x = 0; x < 32 / kQuads; ++x) bits |= ((miss >> (kQuads * x)) & 1u) << x;
        if (kQuads == 4) sm.bad[t & 1][warp] = (uint8_t)bits;
        else *reinterpret_cast<uint16_t*>(&sm.bad[t & 1][2 * warp]) = (uint16_t)bits;
      }
      look_up(t + 1);
    };
    look_up(w.t_begin);
    load_tile(w.t_begin);
    uint32_t odd = split_rows<D>(&sm.piece[0][0][0], kMaxFewRows * D * 2, kMaxFewRows, [&](int r, int c) {
      if (r >= rows) return make_float4(0.f, 0.f, 0.f, 0.f);
      const int gr = w.row0() + r, i = token_of(a, gr), hh = w.h * a.group + gr - i * a.group;
      return *reinterpret_cast<const float4*>(a.q.data + w.b * a.q.seq + (long long)(w.s.row0 + i) * a.q.row +
                                              (long long)hh * a.q.head + c * 16);
    });
    __syncthreads();
    uint32_t q[3][D / 16][4];
#pragma unroll
    for (int x = 0; x < 3; ++x)
#pragma unroll
      for (int k = 0; k < D / 16; ++k) ldsm4(pieces + x * (kMaxFewRows * D * 2) + at(16 * warp + r_av, 2 * k + c_av), q[x][k]);
    // my rows: r and r + 8
    const int r = 16 * warp + (lane >> 2);
    const bool work = 16 * warp < rows;
    int first[2] = {0, 0}, last[2] = {w.s.len, w.s.len};
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (r + 8 * x < rows) visible(a, w.s.len, w.s.len - w.s.n + token_of(a, w.row0() + r + 8 * x), &first[x], &last[x]);
    int af, al;                                             // keys that all rows see: tiles inside need no care
    {
      int f1, l1;
      visible(a, w.s.len, w.s.len - w.s.n + token_of(a, w.row0()), &af, &al);
      visible(a, w.s.len, w.s.len - w.s.n + token_of(a, w.row0() + rows - 1), &f1, &l1);
      af = max(af, f1);
      al = min(al, l1);
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[n][x] = 0.f;

    for (int t = w.t_begin; t < w.t_end; ++t) {
      const int j0 = t * kKeys;
      cp_wait<0>();
      __syncthreads();                                      // the tile is there, the pieces of the one before are free
      odd |= split_rows<D>(&sm.piece[0][0][0], kPiece, kKeys, [&](int r, int c) { return *reinterpret_cast<const float4*>(&sm.raw[0][r][4 * c]); });
      odd |= split_rows<D>(&sm.piece[1][0][0], kPiece, kKeys, [&](int r, int c) { return *reinterpret_cast<const float4*>(&sm.raw[1][r][4 * c]); });
      __syncthreads();
      if (t + 1 < w.t_end) load_tile(t + 1);
      if (!work) continue;
      // ---- scores: products with 16 bits of weight and below apart from h h, which are added last ----
      float s[kKeys / 8][4];
#pragma unroll
      for (int n4 = 0; n4 < kKeys / 8; n4 += 4) {
        float low[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[n4 + n][x] = low[n][x] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[3][2][4];
#pragma unroll
          for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int n = 0; n < 2; ++n) ldsm4(pieces + x * kPiece + at(8 * n4 + 16 * n + r_k, 2 * k + c_k), b[x][n]);
          const auto mul = [&](int qx, int kx, float (*acc)[4]) {
#pragma unroll
            for (int n = 0; n < 4; ++n) mma16816<false>(acc[n], q[qx][k], b[kx][n >> 1][2 * (n & 1)], b[kx][n >> 1][2 * (n & 1) + 1]);
          };
          mul(2, 0, low);
          mul(0, 2, low);
          mul(0, 0, &s[n4]);
          mul(1, 1, low);
          mul(1, 0, low);
          mul(0, 1, low);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[n4 + n][x] = (s[n4 + n][x] + low[n][x]) * a.scale_log2;
      }
      // ---- weights ----
      uint32_t missing = 0;
#pragma unroll
      for (int x = 0; x < kKeys / 32; ++x) missing |= reinterpret_cast<const uint32_t*>(sm.bad[t & 1])[x];
      if (j0 < af || j0 + kKeys > al || missing) {
#pragma unroll
        for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = 8 * n + 2 * (lane & 3) + (x & 1);
            if (j0 + key < first[x >> 1] || j0 + key >= last[x >> 1] || ((sm.bad[t & 1][n] >> (key & 7)) & 1)) s[n][x] = -INFINITY;
          }
      }
      float f[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < kKeys / 8; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * x], s[n][2 * x + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
        const float m_new = fmaxf(m[x], mx), base = m_new == -INFINITY ? 0.f : m_new;
        f[x] = exp2f(m[x] - base);                          // 0 when m = -inf
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < kKeys / 8; ++n) {
          s[n][2 * x] = exp2f(s[n][2 * x] - base);
          s[n][2 * x + 1] = exp2f(s[n][2 * x + 1] - base);
          sum += s[n][2 * x] + s[n][2 * x + 1];
        }
        m[x] = m_new;
        l[x] = l[x] * f[x] + sum;                           // of my keys
      }
      uint32_t pw[kKeys / 16][3][4];
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float* e = &s[2 * k + (x >> 1)][2 * (x & 1)];
          split2(e[0], e[1], pw[k][0][x], pw[k][1][x], pw[k][2][x]);
        }
      // ---- O = O f + P V: a tile's products by themselves, added with one rounding ----
#pragma unroll
      for (int n4 = 0; n4 < D / 8; n4 += 4) {
        float high[4][4], low[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) high[n][x] = low[n][x] = 0.f;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) {
          uint32_t b[3][2][4];
#pragma unroll
          for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int n = 0; n < 2; ++n) ldsm4t(pieces + (3 + x) * kPiece + at(16 * k + r_av, n4 + 2 * n + c_av), b[x][n]);
          const auto mul = [&](int px, int vx, float (*acc)[4]) {
#pragma unroll
            for (int n = 0; n < 4; ++n) mma16816<false>(acc[n], pw[k][px], b[vx][n >> 1][2 * (n & 1)], b[vx][n >> 1][2 * (n & 1) + 1]);
          };
          mul(2, 0, low);
          mul(0, 2, low);
          mul(0, 0, high);
          mul(1, 1, low);
          mul(1, 0, low);
          mul(0, 1, low);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[n4 + n][x] = fmaf(o[n4 + n][x], f[x >> 1], high[n][x] + low[n][x]);
      }
    }
    // ---- the rows' results: complete, or a part of an item that other blocks work on too ----
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(FULL, l[x], 1);
      l[x] += __shfl_xor_sync(FULL, l[x], 2);
    }
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
    if (__syncthreads_or(odd != 0)) {
      // rare: row by row, a warp a row
      float* qr = &sm.raw[0][warp][0];
      for (int r = warp; r < rows; r += kT / 32) {
        const int gr = w.row0() + r, i = token_of(a, gr), hh = w.h * a.group + gr - i * a.group;
        const float* src = reinterpret_cast<const float*>(a.q.data + w.b * a.q.seq + (long long)(w.s.row0 + i) * a.q.row + (long long)hh * a.q.head);
        __syncwarp();
        for (int c = lane; c < D; c += 32) qr[c] = src[c];
        __syncwarp();
        int f0, l0;
        visible(a, w.s.len, w.s.len - w.s.n + i, &f0, &l0);
        float mr, lr, acc[D / 32];
        row_attention<float, D>(a, w.b, w.h, qr, max(f0, w.t_begin * kKeys), min(l0, w.t_end * kKeys), &mr, &lr, acc);
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
      for (int x = 0; x < 2; ++x) {
        const int rr = r + 8 * x;
        if (rr >= rows) continue;
        const float inv = c0 != c1 ? 1.f : l[x] == 0.f ? 0.f : 1.f / l[x];                // NaN sums stay NaN
        float* dst = c0 == c1 ? out_row(rr) : p.part_o + (part + rr) * D;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2*>(dst + 8 * n + 2 * (lane & 3)) = make_float2(o[n][2 * x] * inv, o[n][2 * x + 1] * inv);
        if ((lane & 3) == 0) {
          if (c0 == c1) finish(rr, m[x], l[x]);
          else p.part_ml[part + rr] = make_float2(m[x], l[x]);
        }
      }
    }
    if (c0 != c1 && ends_last(p, sm.last, c0, c1)) join<D, kT>(p, sm.m, rows, c0, c1, out_row, finish);
  } while (w.next(a));
}

template <int D>
cudaError_t launch_few(const Params& p, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(Smem<D>);
  if ((e = set_max_dynamic_smem(reinterpret_cast<const void*>(attn_few<D>), smem))) return e;
  static_assert(sizeof(Smem<D>) <= 113 * 1024, "two blocks' shared memory fits an SM");
  return launch_after(attn_few<D>, dim3(min(2 * sms, kMaxFewBlocks)), kThreads, smem, st, p);
}

template <int D>
cudaError_t launch_split(const Params& p, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(SplitSmem<D>);
  if ((e = set_max_dynamic_smem(reinterpret_cast<const void*>(attn_split<D>), smem))) return e;
  return launch_after(attn_split<D>, dim3(min(2 * sms, kMaxFewBlocks)), kSplitThreads, smem, st, p);
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
  if (d == 64) return few ? launch_few<64>(p, st) : launch_split<64>(p, st);
  return few ? launch_few<128>(p, st) : launch_split<128>(p, st);
}

}  // namespace cache
}  // namespace pisa
