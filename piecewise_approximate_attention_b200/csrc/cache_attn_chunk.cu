// Attention over the paged cache for chunks of new tokens: bf16 and e4m3 pools, TMA + tcgen05.
//
// The new tokens of a sequence times the group of query heads that share a key/value head are the
// rows of one product with that head's keys.  An item is up to 256 of these rows: two tiles ("slots")
// of 128 that walk the same tiles of 128 keys together, so a key tile is read from L2 once for 256
// rows, and one slot's softmax runs while the tensor core works on the other's products.  Where no item
// has more than 128 rows (kDual), both slots hold the same rows and take the key tiles in turn, and
// slot 1 hands its result to slot 0 at the end.  The work is shared out as in cache_walk.cuh; items that several
// blocks share leave partial results (O, maximum, sum) that a second small kernel joins.
//
// Block (one an SM, 16 warps):
//   warps 0-3, 4-7   softmax and output of slot 0 and 1: thread r owns row r (TMEM lane r).  Per tile
//                    and half of 64 keys: scores from TMEM, weights against a maximum that is moved only
//                    when a row outgrows it by 2^15, P back over the scores' columns, release to warp 13
//   warps 8-11       values made ready: see below; thread r owns key r of the tile
//   warp 12          follows the page table, TMA loads into two K and two V stages
//   warp 13          issues the MMAs: S = Q K^T (M 128, N 128), O += P V per half (P from TMEM), the slots in
//                    turn: that keeps their softmaxes apart (each slot with an issuer of its own, they fell
//                    into step and fought for the exponential unit: 1860 instead of 1480 cycles a tile)
// TMEM: S/P of the slots at columns 0 and 128, O at 256 and 384.
//
// bf16 pools: K and V are used as stored; P is bf16, as the type of V asks of the MMA (each weight is
// off by 2^-8 at most, like the output's own rounding; the error against float64 is 2.33e-3 where the output's rounding
// alone is 1.66e-3).  Weights in two bf16 parts, as cache_attn_few.cu has them for few rows, would take half as long again
// (frame of 1560 tokens 399 -> 608 us, prompts 210 -> 319).  What is done: the maximum is also moved where a half outweighs
// kPart times all that its row has so far, so that a key which holds four fifths of a row or more weighs exactly 1 and
// such a row is not off by its rounding (frame +1%, prompts +3%).
//
// e4m3 pools: warps 8-11 turn codes into fp16 tiles in shared memory, once for both slots, as
// code * 2^(e - E): e the row's own exponent, E the largest of the first tile of the share that has rows other than
// zeros.  That is exact for e - E in [-15, 7], so scores need one factor 2^E a share and P (fp16, 11 bits) multiplies
// values that are all in one unit.  q becomes fp16 with a power of two per row, exactly.
//
// What does not fit is computed again: a share in which a row's exponent leaves that window, or that
// holds a value which is not finite in a tile that only some rows see (0 * NaN would reach the rows
// that do not), is flagged and its rows are computed by the plain routine of cache_row.cuh.  That takes long (256 rows of
// 8192 keys: some tens of milliseconds), and the block's other warps wait meanwhile for longer than their limit if need
// be: it counts from the last sign of life of the warps at it.  V rows of
// stale slots and of missing pages are zeroed.
#include <cfloat>
#include <type_traits>

#include "cache_pipe.cuh"
#include "cache_row.cuh"
#include "cache_walk.cuh"
#include "sm100.cuh"

namespace pisa {
namespace cache {
namespace {
using namespace sm100;

constexpr int kKeys = 128;                   // keys of a tile
constexpr int kRows = 128;                   // rows of a slot
constexpr int kThreads = 512;
constexpr float kPart = 4.f;                  // bf16 pools: see above
// e4m3 pools: weights reach 2^8 where the maximum is moved, so those that are normal fp16 numbers reach down to 2^-22 of a
// row's largest, and what is lost below is at most 2^-33 of it a key: many small weights can matter beside a large one
// whose values are small.
template <bool kF8> constexpr float kLift = kF8 ? 8.f : 0.f;
constexpr float kRoom = 32768.f;              // weights of a half that P (fp16 at least) takes as they are
constexpr unsigned FULL = 0xffffffffu;
constexpr uint32_t kColO = 256;
constexpr int kStages = 2;
constexpr int kNoUnit = 1 << 20;
constexpr int kBelow = 15, kAbove = 7;       // exponents that fp16 holds exactly around E

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool softmax_or(bool x) {
  int y;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
               : "=r"(y) : "r"((int)x) : "memory");
  return y != 0;
}
__device__ __forceinline__ void aux_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }

template <int D, bool kF8>
struct alignas(1024) Smem {
  static constexpr int kHalf = kKeys * 128;              // 128 rows of 64 16-bit columns
  static constexpr int kTile = D / 64 * kHalf;
  uint8_t q[2][kTile];
  uint8_t k[kStages][kTile];
  uint8_t v[kStages][kTile];
  uint8_t raw[kF8 ? 2 : 1][kF8 ? kKeys * D : 16];        // e4m3 codes as loaded, K and V in turn
  uint8_t raw_exp[2][kKeys];
  float row_scale[2 * kRows];                            // raw score -> base-2 logit, but for 2^E; at an item's end slot 1's (maximum, sum)
  uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages], vready[kStages];
  uint64_t rawfull[2], rawempty[2];
  uint64_t qfull[2], sfull[2], pfull[2][2], odone[2][2], drain;
  uint32_t bad[4][4];                                    // tile of the block & 3: keys whose page is missing
  int unit[4][2], odd[4];                                // item & 3: E of K and V, kNoUnit before they are known; to be computed again
  WalkScratch<kThreads / 32> walk;
  uint32_t tmem;
  int abort;
  unsigned long long alive;                              // when a warp that computes rows by themselves was last seen at it, ns
};

struct Params {
  AttnArgs a;
  int4* split;               // one a block: the item that begins in it and is shared (sequence, head, pair, parts), parts = 0 for none
  float2* part_ml;           // [2 * blocks][256]
  float* part_o;             // [2 * blocks][D / 4][256][4]: a warp's rows next to one another
  int log_rows;              // rows of an item: 2^7 or 2^8
  int item_cost;             // what an item costs besides its tiles, in tiles; < 0: items are not cut (cache_walk.cuh)
  unsigned long long wait_ns;
  int fault;
};

template <typename S>
__device__ __forceinline__ bool wait(S& sm, uint64_t* bar, uint32_t parity, const Params& p) {
  return wait_for(sm, bar, parity, p.wait_ns, p.a.seqs.status);
}
// The same where what is waited for may itself have to wait for rows that are computed one by one: all that hangs on the
// next item's queries.  (In every wait of the softmax's loops it costs D = 128 6 to 8%.)
template <typename S>
__device__ __forceinline__ bool wait_long(S& sm, uint64_t* bar, uint32_t parity, const Params& p) {
  return wait_for(sm, bar, parity, p.wait_ns, p.a.seqs.status, &sm.alive);
}

// E of one side of tile t: the largest exponent of its rows that are there and not zero; false if there is none.  A row
// of zeros is stored with the smallest exponent, so only where no row has another do the codes themselves tell.  Each
// of the four warps finds out by itself.
template <int D, typename S>
__device__ __forceinline__ bool first_unit(const S& sm, int side, int t, int len, const uint32_t* bad, int* unit) {
  const int lane = threadIdx.x & 31;
  const uint32_t exps = reinterpret_cast<const uint32_t*>(sm.raw_exp[side])[lane];      // of rows 4 lane ... 4 lane + 3
  int e = -kExpLimit;
  bool any = false;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * lane + i;
    if (t * kKeys + r >= len || ((bad[r >> 5] >> (r & 31)) & 1u)) continue;
    const int x = (int)((exps >> (8 * i)) & 0xffu) - kExpBias;
    e = max(e, x);
    if (x == -kExpLimit && !any) {
      const uint4* row = reinterpret_cast<const uint4*>(sm.raw[side] + r * D);
      for (int c = 0; c < D / 16; ++c) any = any || ((row[c].x | row[c].y | row[c].z | row[c].w) & 0x7f7f7f7fu);
    }
  }
  *unit = __reduce_max_sync(FULL, e);
  if (*unit > -kExpLimit || __any_sync(FULL, any)) return true;
  *unit = 0;
  return false;
}

// Bits of 32 keys from j0 on that lie in [first, last).
__device__ __forceinline__ uint32_t range_bits(int j0, int first, int last) {
  const int lo = first - j0, hi = last - j0;
  uint32_t m = hi >= 32 ? FULL : hi > 0 ? (1u << hi) - 1u : 0u;
  if (lo > 0) m &= lo >= 32 ? 0u : ~((1u << lo) - 1u);
  return m;
}

// Out of line, the rare path's registers stay out of the softmax's (frame of 1560 tokens, head_dim 64: 389 -> 362 us;
// bf16 with head_dim 128 is better off without the call: prompts 230 -> 220 us).
template <typename K, int D>
__device__ __noinline__ void row_apart(const AttnArgs& a, int b, int kvh, const float* q, int first, int last, float* m, float* l,
                                       float* acc, volatile unsigned long long* alive) {
  row_attention<K, D>(a, b, kvh, q, first, last, m, l, acc, alive);
}

template <int D, bool kF8, bool kDual>
__global__ void __launch_bounds__(kThreads, 1)
attn_chunk(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Params p) {
  using S = Smem<D, kF8>;
  extern __shared__ uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- set-up, and this block's share of the line ----
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.kfull[i], kF8 ? 4 : 1);
      mbar_init(&sm.kempty[i], 1);
      mbar_init(&sm.vfull[i], 1);
      mbar_init(&sm.vempty[i], 1);
      mbar_init(&sm.vready[i], 4);
      mbar_init(&sm.rawfull[i], 1);
      mbar_init(&sm.rawempty[i], 4);
      mbar_init(&sm.qfull[i], 4);
      mbar_init(&sm.sfull[i], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sm.pfull[i][h], 4);
        mbar_init(&sm.odone[i][h], 1);
      }
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    sm.alive = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  griddep_wait();
  if (threadIdx.x == 0) p.split[blockIdx.x] = make_int4(0, 0, 0, 0);
  Walk<kKeys> w;
  if (w.template start<kThreads>(a, sm.walk, p.log_rows, p.item_cost, p.item_cost < 0 ? 1 : 1 + p.item_cost)) {
    if (warp < 8) {
      // =========================== softmax and output ===========================
      const int slot = warp >> 2, r = threadIdx.x & (kRows - 1);
      const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16), ts = trow + 128 * slot, to = trow + kColO + 128 * slot;
      uint32_t n_tile = 0, all_tiles = 0;          // this slot's tiles so far, the block's
      do {
        if (w.t_begin >= w.t_end) continue;
        const uint32_t tile0 = all_tiles;
        all_tiles += w.t_end - w.t_begin;
        const bool active = kDual || slot * kRows < w.it.rows;
        const int row = (kDual ? 0 : slot * kRows) + r, grow_ = w.row0() + row;          // of the item, of the head's rows
        const bool valid = row < w.it.rows;
        const int tok = valid ? token_of(a, grow_) : 0, head = w.h * a.group + (valid ? grow_ - tok * a.group : 0);
        float m = -INFINITY, l = 0.f;
        int first = 0, last = w.s.len;
        if (valid) visible(a, w.s.len, w.s.len - w.s.n + tok, &first, &last);
        if (active) {
          // ---- the slot's queries into shared memory: each warp its own 32 rows, D / 8 lanes a row ----
          constexpr int kLanes = D / 8, kPer = 32 / kLanes;    // rows a step
          const int c = lane % kLanes, q0 = (warp & 3) * 32 + lane / kLanes;
          const auto q_at = [&](int qr) { return sm.q[slot] + (c >> 3) * S::kHalf + qr * 128 + (((c & 7) ^ (qr & 7)) << 4); };
          {
            const int gr0 = w.row0() + (kDual ? 0 : slot * kRows) + q0;
            int i = token_of(a, gr0), gm = gr0 - i * a.group;  // token and head of the group, stepped
#pragma unroll 2
            for (int x = 0; x < kLanes; ++x) {
              const bool there = gr0 + x * kPer < w.row0() + w.it.rows;       // zeros behind the last row
              const char* src = there ? a.q.data + w.b * a.q.seq + (long long)(w.s.row0 + i) * a.q.row +
                                            (long long)(w.h * a.group + gm) * a.q.head + c * 16
                                      : a.q.data;
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(q_at(q0 + x * kPer))), "l"(src),
                           "r"(there ? 16 : 0) : "memory");
              gm += kPer;
              while (gm >= a.group) {
                gm -= a.group;
                ++i;
              }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
          }
          if constexpr (kF8) {
#pragma unroll 2
            for (int x4 = 0; x4 < kLanes; ++x4) {              // each lane what it has loaded itself
              const int qr = q0 + x4 * kPer;
              uint4* at = reinterpret_cast<uint4*>(q_at(qr));
              const uint4 u = *at;
              const uint32_t x[4] = {u.x, u.y, u.z, u.w};
              uint32_t mx = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) mx = max(mx, max((x[e] << 16) & 0x7fff0000u, x[e] & 0x7fff0000u));
#pragma unroll
              for (int d = kLanes / 2; d > 0; d >>= 1) mx = max(mx, __shfl_xor_sync(FULL, mx, d));
              // largest magnitude to [2^14, 2^15): every bf16 down to 2^-31 of it is an fp16 number
              const int eq = max(-100, min(112, (int)(mx >> 23) - 127 - 14));
              const float sc = pow2(-eq);
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = pack_f16x2(__uint_as_float(x[e] << 16) * sc, __uint_as_float(x[e] & 0xffff0000u) * sc);
              *at = make_uint4(y[0], y[1], y[2], y[3]);
              if (c == 0) sm.row_scale[slot * kRows + qr] = a.scale_log2 * pow2(eq);
            }
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.qfull[slot]);
          // keys that all of the warp's rows see
          int all_first = first, all_last = last;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) {
            all_first = max(all_first, __shfl_xor_sync(FULL, all_first, d));
            all_last = min(all_last, __shfl_xor_sync(FULL, all_last, d));
          }
          float sl = a.scale_log2;       // raw score -> base-2 logit
          bool open = true;              // e4m3: no E yet
          const int t_first = w.t_begin + (kDual ? slot : 0);
          if (t_first < w.t_end) wait_long(sm, &sm.sfull[slot], n_tile & 1, p);         // the other slot may keep the item waiting
          for (int t = t_first; t < w.t_end; t += kDual ? 2 : 1, ++n_tile) {
            const uint32_t par = n_tile & 1;
            wait(sm, &sm.sfull[slot], par, p);
            __syncwarp();
            tc_fence_after();
            if (kF8 && open) {
              // E may come with a later tile than the first; scores before that are zero.  The factor stays a normal
              // number: -inf of a masked score times 0, or a zero score times inf, would be NaN (scores whose logits that
              // changes are zero, or the logits below 2^-80 or past fp32 anyway).
              const int e = sm.unit[w.count & 3][0];
              open = e == kNoUnit;
              sl = sm.row_scale[slot * kRows + r] * pow2(open ? 0 : e);
              sl = fminf(fmaxf(sl, FLT_MIN), FLT_MAX);
            }
            const uint32_t* bad = sm.bad[(tile0 + t - w.t_begin) & 3];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const int j0 = t * kKeys + 64 * hh;
              uint32_t vm0 = FULL, vm1 = FULL;
              if (j0 < all_first || j0 + 64 > all_last || (bad[2 * hh] | bad[2 * hh + 1])) {
                vm0 = range_bits(j0, first, last) & ~bad[2 * hh];
                vm1 = range_bits(j0 + 32, first, last) & ~bad[2 * hh + 1];
                if (__all_sync(FULL, (vm0 | vm1) == 0u)) {
                  // nothing to see for any of the warp's rows: P = 0, and m and l stay
                  uint32_t zero[16];
#pragma unroll
                  for (int x = 0; x < 16; ++x) zero[x] = 0u;
                  tmem_st16(ts + 64 * hh, zero);
                  tmem_st16(ts + 64 * hh + 16, zero);
                  tmem_st_wait();
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&sm.pfull[slot][hh]);
                  continue;
                }
              }
              float s[64];
              tmem_ld32(ts + 64 * hh, s);
              tmem_ld32(ts + 64 * hh + 32, s + 32);
              tmem_ld_wait();
              if (vm0 != FULL) {
#pragma unroll
                for (int x = 0; x < 32; ++x) s[x] = ((vm0 >> x) & 1u) ? s[x] : -INFINITY;
              }
              if (vm1 != FULL) {
#pragma unroll
                for (int x = 0; x < 32; ++x) s[32 + x] = ((vm1 >> x) & 1u) ? s[32 + x] : -INFINITY;
              }
              // Weights against the maximum so far, without looking for the half's own first: their sum says
              // whether a row outgrew it (each weight is at most the sum, so below kRoom P holds them all).
              float ls = 0.f;
              const auto weights = [&]() {
                const float mb = m == -INFINITY ? 0.f : m;
                const uint64_t sc2 = f2_pack(sl, sl), nmb2 = f2_pack(-mb, -mb);
                uint64_t acc2 = f2_pack(0.f, 0.f);
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                  uint32_t pk[16];
#pragma unroll
                  for (int x = 0; x < 32; x += 2) {
                    const int c = 32 * ch + x;
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), sc2, nmb2), x0, x1);
                    const float p0 = ex2(x0), p1 = ex2(x1);
                    acc2 = f2_add(acc2, f2_pack(p0, p1));
                    pk[x >> 1] = kF8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                  }
                  tmem_st16(ts + 64 * hh + 16 * ch, pk);
                }
                float ls0, ls1;
                f2_unpack(acc2, ls0, ls1);
                ls = ls0 + ls1;
              };
              const auto largest = [&]() {
                float t0 = fmaxf(s[0], s[1]), t1 = fmaxf(s[2], s[3]), t2 = fmaxf(s[4], s[5]), t3 = fmaxf(s[6], s[7]);
#pragma unroll
                for (int c = 8; c < 64; c += 8) {
                  t0 = fmax3(t0, s[c], s[c + 1]);
                  t1 = fmax3(t1, s[c + 2], s[c + 3]);
                  t2 = fmax3(t2, s[c + 4], s[c + 5]);
                  t3 = fmax3(t3, s[c + 6], s[c + 7]);
                }
                return fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
              };
              const bool first_half = t == t_first && hh == 0;
              if (!first_half) weights();
              // bf16: no weight yet, or one that may dominate the row, or one that does not fit; rows of NaN stay as they are
              if (__any_sync(FULL, kF8 ? first_half || ls > kRoom || m == -INFINITY : m == -INFINITY || ls > fminf(kRoom, kPart * l))) {
                // rare but for the first half: move the maximum, and with it l and O
                const float m_new = fmaxf(m, largest() * sl - kLift<kF8>);         // base-2 units
                const float f = m_new == -INFINITY ? 1.f : ex2(m - m_new);         // 0 when m = -inf
                l *= f;
                m = m_new;
                if (!first_half) {
                  // O holds the products of the halves before this one
                  wait(sm, &sm.odone[slot][hh ^ 1], hh ? par : par ^ 1u, p);
                  __syncwarp();
                  tc_fence_after();
#pragma unroll 1
                  for (int ch = 0; ch < D / 16; ++ch) {
                    float ov[16];
                    tmem_ld16(to + 16 * ch, ov);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 16; ++x) ov[x] *= f;
                    tmem_st16(to + 16 * ch, reinterpret_cast<const uint32_t*>(ov));
                  }
                }
                weights();
              }
              l += ls;
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.pfull[slot][hh]);
            }
          }
          if (t_first < w.t_end) {
            wait(sm, &sm.odone[slot][1], (n_tile - 1) & 1, p);
            __syncwarp();
            tc_fence_after();
          }
        }
        // ---- dual: slot 1 hands its maximum, sum and O over, through the queries' room ----
        // (both slots' products have read the queries, and what one knows of odd values in its last tiles goes for both:
        // they have to agree on it whatever happens, barriers depend on it)
        bool odd = *reinterpret_cast<volatile int*>(&sm.odd[w.count & 3]) != 0;
        if (kDual) odd = softmax_or(odd);
        const int ev = kF8 ? sm.unit[w.count & 3][1] : 0;
        const float unit = ev == kNoUnit ? 1.f : pow2(ev);                 // O's
        const bool joined = kDual && w.t_end - w.t_begin > 1 && !odd;                 // slot 1 had tiles, too
        float4* hand = reinterpret_cast<float4*>(sm.q[0]) + r;                       // [D / 4][128]
        float2* hand_ml = reinterpret_cast<float2*>(sm.row_scale);
        float f_own = 1.f, f_other = 0.f;
        if (joined) {
          if (slot == 1) {
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              float ov[32];
              __syncwarp();
              tmem_ld32(to + 32 * ch, ov);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 8; ++x) hand[(8 * ch + x) * kRows] = make_float4(ov[4 * x], ov[4 * x + 1], ov[4 * x + 2], ov[4 * x + 3]);
            }
            tc_fence_before();
            hand_ml[r] = make_float2(m, l);
          }
          softmax_sync();
          if (slot == 0) {
            const float2 o = hand_ml[r];
            const float mn = fmaxf(m, o.x), base = mn == -INFINITY ? 0.f : mn;
            f_own = ex2(m - base);
            f_other = ex2(o.x - base);
            m = mn;
            l = l * f_own + o.y * f_other;
          }
        }
        const bool writes = kDual ? slot == 0 : active;
        // ---- the rows' results: complete, or a part of an item that other blocks work on too ----
        const int c0 = w.first_block(), c1 = w.last_block();
        const size_t part = (size_t)w.part() * 256;
        const auto out_row = [&](int i, int hh) {
          return a.o.data + w.b * a.o.seq + (long long)(w.s.row0 + i) * a.o.row + (long long)hh * a.o.head;
        };
        if (writes && odd) {
          // rare: what the operands could not hold, row by row; this warp's rows of the query tile are free as scratch
          float* qs = reinterpret_cast<float*>(sm.q[slot] + (warp & 3) * 32 * 128);
          for (int rr = 0; rr < 32; ++rr) {
            const int ir = (kDual ? 0 : slot * kRows) + (warp & 3) * 32 + rr;
            if (ir >= w.it.rows) break;
            const int gr = w.row0() + ir, i = token_of(a, gr), hh = w.h * a.group + gr - i * a.group;
            const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(
                a.q.data + w.b * a.q.seq + (long long)(w.s.row0 + i) * a.q.row + (long long)hh * a.q.head);
            for (int c = lane; c < D; c += 32) qs[c] = to_f32(q[c]);
            __syncwarp();
            int f0, l0;
            visible(a, w.s.len, w.s.len - w.s.n + i, &f0, &l0);
            float mr, lr, acc[D / 32];
            if (lane == 0) *reinterpret_cast<volatile unsigned long long*>(&sm.alive) = globaltimer_ns();
            const int j_first = max(f0, w.t_begin * kKeys), j_last = min(l0, w.t_end * kKeys);
            if constexpr (D == 128 && !kF8) row_attention<__nv_bfloat16, D>(a, w.b, w.h, qs, j_first, j_last, &mr, &lr, acc, &sm.alive);
            else row_apart<typename std::conditional<kF8, uint8_t, __nv_bfloat16>::type, D>(a, w.b, w.h, qs, j_first, j_last, &mr, &lr, acc, &sm.alive);
            __syncwarp();
            const float inv = lr == 0.f ? 0.f : 1.f / lr;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              if (c0 == c1) reinterpret_cast<__nv_bfloat16*>(out_row(i, hh))[c * 32 + lane] = from_f32<__nv_bfloat16>(acc[c] * inv);
              else p.part_o[part * D + ((c * 32 + lane) / 4 * kMaxChunkRows + ir) * 4 + lane % 4] = acc[c];
            }
            if (lane == 0) {
              float* lse = lse_at(a, w.b, w.s, i, hh);
              if (c0 != c1) p.part_ml[part + ir] = make_float2(mr, lr);
              else if (lse) *lse = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * 0.6931471805599453f;
            }
          }
        } else if (writes) {
          const float inv = (l == 0.f ? 0.f : 1.f / l) * unit;
#pragma unroll
          for (int ch = 0; ch < D / 32; ++ch) {
            float ov[32];
            __syncwarp();
            tmem_ld32(to + 32 * ch, ov);
            tmem_ld_wait();
            if (joined) {
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const float4 o = hand[(8 * ch + x) * kRows];
                ov[4 * x] = ov[4 * x] * f_own + o.x * f_other;
                ov[4 * x + 1] = ov[4 * x + 1] * f_own + o.y * f_other;
                ov[4 * x + 2] = ov[4 * x + 2] * f_own + o.z * f_other;
                ov[4 * x + 3] = ov[4 * x + 3] * f_own + o.w * f_other;
              }
            }
            if (!valid) {
            } else if (c0 == c1) {
              uint4* dst = reinterpret_cast<uint4*>(out_row(tok, head) + 64 * ch);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                dst[x] = make_uint4(pack_bf16x2(ov[8 * x] * inv, ov[8 * x + 1] * inv), pack_bf16x2(ov[8 * x + 2] * inv, ov[8 * x + 3] * inv),
                                    pack_bf16x2(ov[8 * x + 4] * inv, ov[8 * x + 5] * inv), pack_bf16x2(ov[8 * x + 6] * inv, ov[8 * x + 7] * inv));
            } else {
              float4* dst = reinterpret_cast<float4*>(p.part_o + part * D) + 8 * ch * kMaxChunkRows + row;
#pragma unroll
              for (int x = 0; x < 8; ++x)
                dst[x * kMaxChunkRows] = make_float4(ov[4 * x] * unit, ov[4 * x + 1] * unit, ov[4 * x + 2] * unit, ov[4 * x + 3] * unit);
            }
          }
          if (valid) {
            if (c0 != c1) p.part_ml[part + row] = make_float2(m, l);
            else if (float* lse = lse_at(a, w.b, w.s, tok, head)) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
          }
          tc_fence_before();             // O is read before the next item's first product overwrites it
        }
        if (kDual) softmax_sync();       // what was handed over has been read: the queries' room is free
        // the block that begins an item which others go on with leaves word of it for the joining kernel
        if (threadIdx.x == 0 && c0 != c1 && !w.began_before()) p.split[blockIdx.x] = make_int4(w.b, w.h, w.p, c1 - c0 + 1);
        ++w.count;
      } while (w.next(a));
    } else if (warp < 12) {
      // =========================== values made ready ===========================
      const int r = threadIdx.x & 127;   // my key of the tile
      uint32_t n_tile = 0;
      do {
        if (w.t_begin >= w.t_end) continue;
        const int it4 = w.count & 3;
        if (r == 0) sm.odd[it4] = 0, sm.unit[it4][0] = sm.unit[it4][1] = kNoUnit;
        aux_sync();
        // keys that all of the item's rows see: tiles inside need no care
        int f0, l0, f1, l1;
        visible(a, w.s.len, w.s.len - w.s.n + token_of(a, w.row0()), &f0, &l0);
        visible(a, w.s.len, w.s.len - w.s.n + token_of(a, w.row0() + w.it.rows - 1), &f1, &l1);
        const int all_first = max(f0, f1), all_last = min(l0, l1);
        int eu[2] = {0, 0}, has_unit = 0;         // E of K and of V, as far as there are (bits 1 and 2): 0 before
        for (int t = w.t_begin; t < w.t_end; ++t, ++n_tile) {
          const int st = n_tile & 1;
          const uint32_t ph = (n_tile >> 1) & 1;
          if constexpr (!kF8) {
            wait_long(sm, &sm.vfull[st], ph, p);
            const uint32_t* bad = sm.bad[n_tile & 3];
            if (t * kKeys < all_first || (t + 1) * kKeys > all_last || (bad[0] | bad[1] | bad[2] | bad[3])) {
              const bool there = t * kKeys + r < w.s.len && !((bad[r >> 5] >> (r & 31)) & 1u);
              bool odd = false;
#pragma unroll 4
              for (int c = 0; c < D / 8; ++c) {
                uint4* x = reinterpret_cast<uint4*>(sm.v[st] + (c >> 3) * S::kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                uint4 u = there ? *x : make_uint4(0, 0, 0, 0);
                uint32_t y[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((y[e] & 0x7f80u) == 0x7f80u) { odd = true; y[e] &= 0xffff0000u; }
                  if ((y[e] & 0x7f800000u) == 0x7f800000u) { odd = true; y[e] &= 0x0000ffffu; }
                }
                *x = make_uint4(y[0], y[1], y[2], y[3]);
              }
              if (odd) *reinterpret_cast<volatile int*>(&sm.odd[it4]) = 1;
              fence_async_shared();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.vready[st]);
          } else {
#pragma unroll 1
            for (int side = 0; side < 2; ++side) {
              wait_long(sm, &sm.rawfull[side], n_tile & 1, p);
              const uint32_t* bad = sm.bad[n_tile & 3];
              const bool there = t * kKeys + r < w.s.len && !((bad[r >> 5] >> (r & 31)) & 1u);
              const int e = there ? (int)sm.raw_exp[side][r] - kExpBias : -kExpLimit;
              if (!(has_unit & (1 << side))) {
                if (first_unit<D>(sm, side, t, w.s.len, bad, &eu[side])) {
                  has_unit |= 1 << side;
                  if (r == 0) sm.unit[it4][side] = eu[side];
                }
              }
              const int de = e - eu[side];
              const bool far = de > kAbove || de < -kBelow;
              const __half f16 = __float2half_rn(there ? pow2(max(-24, min(kAbove, de))) : 0.f);
              const __half2 f2 = __half2half2(f16);
              // the converted stage is free
              if (n_tile >= kStages) wait_long(sm, side ? &sm.vempty[st] : &sm.kempty[st], ph ^ 1u, p);
              uint8_t* dst = side ? sm.v[st] : sm.k[st];
              const bool edge = t * kKeys < all_first || (t + 1) * kKeys > all_last;
              bool odd = false;
              const uint8_t* src = sm.raw[side] + r * D;
              uint8_t* row = dst + r * 128;
              const int src_x = D == 128 ? r & 7 : (r >> 1) & 3, dst_x = r & 7;       // the swizzles' part of the row
              const auto chunk = [&](int c, uint32_t* y) {     // 16 codes, times the row's factor
                const uint4 u = *reinterpret_cast<const uint4*>(src + ((c ^ src_x) << 4));
                const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint32_t h = e4m3x2_to_f16x2((uint16_t)(x[i >> 1] >> (16 * (i & 1))));
                  const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&h), f2);
                  y[i] = *reinterpret_cast<const uint32_t*>(&z);
                }
                return ((x[0] | x[1] | x[2] | x[3]) & 0x7f7f7f7fu) != 0u;       // -0 is a zero, too
              };
              const auto store = [&](int c, const uint32_t* y) {
                uint8_t* at = row + (c >> 2) * S::kHalf;
                const int ch = (2 * c) & 7;
                *reinterpret_cast<uint4*>(at + ((ch ^ dst_x) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(at + (((ch + 1) ^ dst_x) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
              };
              if (__all_sync(FULL, there && !far) && !(edge && side)) {
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t y[8];
                  chunk(c, y);
                  store(c, y);
                }
              } else {
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t y[8];
                  const bool any = chunk(c, y);
                  if (there && far && any) odd = true;
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const bool inf = (y[i] & 0x7c00u) == 0x7c00u || (y[i] & 0x7c000000u) == 0x7c000000u;
                    if (there && edge && side && inf) odd = true;
                    if (!there || (edge && side && inf)) y[i] = 0u;     // a stale NaN times zero
                  }
                  store(c, y);
                }
              }
              if (odd) *reinterpret_cast<volatile int*>(&sm.odd[it4]) = 1;
              fence_async_shared();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(&sm.rawempty[side]);
                mbar_arrive(side ? &sm.vready[st] : &sm.kfull[st]);
              }
            }
          }
        }
        ++w.count;
      } while (w.next(a));
    } else if (warp == 12) {
      // =============================== producer ===============================
      if (lane == 0) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
      }
      const int box = a.pool.page, log_box = a.pool.page_log2, boxes = kKeys >> log_box;
      constexpr int kHalves = kF8 ? 1 : D / 64;
      const uint32_t box_bytes = (uint32_t)box * D * (kF8 ? 1 : 2) + (kF8 ? (uint32_t)box : 0u);
      constexpr int kDeep = kF8 ? 1 : kStages;             // tiles loaded ahead (e4m3: converted into two more)
      uint32_t n_tile = 0, sides = 0;                      // sides: of tiles loaded so far, K and V in turn
      bool ok = true;
      do {
        for (int t = w.t_begin; ok && t < w.t_end; ++t, ++n_tile) {
          const int st = n_tile % kDeep;
          int row = -1;                  // lane i < boxes: the box's first row of the pool
          const int pos = t * kKeys + lane * box;
          if (lane < boxes && pos < w.s.len && pos + box > w.it.first) {
            const int pg = load_page(a.seqs, a.pool, w.b, pos);
            if (pg >= 0) row = (pg * a.pool.kv_heads + w.h) * box;
          }
          const unsigned have = __ballot_sync(FULL, row >= 0);
#pragma unroll 1
          for (int side = 0; side < 2; ++side, ++sides) {
            uint64_t* full = kF8 ? &sm.rawfull[side] : side ? &sm.vfull[st] : &sm.kfull[st];
            uint64_t* empty = kF8 ? &sm.rawempty[side] : side ? &sm.vempty[st] : &sm.kempty[st];
            // warps that gave up on a copy hand its stage back all the same, after they set the abort word
            if (n_tile >= kDeep) ok = __all_sync(FULL, wait_long(sm, empty, (n_tile / kDeep - 1) & 1, p) && !aborted(sm));
            if (!ok) break;
            if (p.fault && sides == 0) continue;             // a test's: the keys that never come
            if (side == 0 && lane < 4) { // the tile's missing keys, before anything of it is released
              uint32_t bits = 0;
              for (int i = 0; i < 32; i += 16)
                if (!((have >> ((lane * 32 + i) >> log_box)) & 1u)) bits |= 0xffffu << i;
              sm.bad[n_tile & 3][lane] = bits;
            }
            __syncwarp();
            if (lane == 0) mbar_expect_tx(full, __popc(have) * box_bytes);
            __syncwarp();
            const int i = lane / kHalves, half = lane % kHalves;        // boxes * halves <= 16
            const int rr = __shfl_sync(FULL, row, i);
            if (i < boxes && rr >= 0) {
              uint8_t* dst = kF8 ? sm.raw[side] + i * box * D : (side ? sm.v[st] : sm.k[st]) + half * S::kHalf + i * box * 128;
              tma_load_3d(dst, side ? &vmap : &kmap, full, half * 64, rr, 0);
              if (kF8) bulk_load(sm.raw_exp[side] + i * box, (side ? a.pool.v_exp : a.pool.k_exp) + rr, box, full);
            }
          }
        }
      } while (ok && w.next(a));
      // every copy lands before this block's shared memory is released
      if (lane == 0)
        for (uint32_t x = sides > 2 * kDeep ? sides - 2 * kDeep : 0; x < sides; ++x) {
          const uint32_t i = x >> 1, side = x & 1;
          mbar_drain(kF8 ? &sm.rawfull[side] : side ? &sm.vfull[i % kDeep] : &sm.kfull[i % kDeep], (i / kDeep) & 1, p.wait_ns);
        }
    } else if (warp == 13 && lane == 0) {
      // =============================== MMA issuer ===============================
      constexpr uint32_t idesc_s = kF8 ? idesc_f16_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t idesc_pv = kF8 ? idesc_f16_f32(128, D, false, true) : idesc_bf16_f32(128, D, false, true);
      uint32_t n_tile = 0, n_slot0 = 0, n_slot1 = 0, n_item0 = 0, n_item1 = 0;       // tiles of the block, tiles and items of each slot
      uint64_t qd[2], kd[2], vd[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qd[i] = smem_desc_sw128(smem_u32(sm.q[i]), 16, 1024);
        kd[i] = smem_desc_sw128(smem_u32(sm.k[i]), 16, 1024);
        vd[i] = smem_desc_sw128(smem_u32(sm.v[i]), S::kHalf, 1024);
      }
      // S of the block's n-th tile (stage n & 1) in a slot; `done`: no other slot needs the tile's keys
      const auto scores = [&](auto slot_tag, uint32_t n, bool done) {
        constexpr int slot = decltype(slot_tag)::value;
        const int st = n & 1;
        wait(sm, &sm.kfull[st], (n >> 1) & 1, p);
        tc_fence_after();
        const uint64_t k = st ? kd[1] : kd[0];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * S::kHalf + (kk & 3) * 32) >> 4;
          mma_ss(tmem + 128 * slot, qd[slot] + off, k + off, idesc_s, kk > 0);
        }
        mma_commit(&sm.sfull[slot]);
        if (done) mma_commit(&sm.kempty[st]);
      };
      // O += P V of the same tile, half by half
      const auto values = [&](auto slot_tag, uint32_t n, bool fresh, bool done) {
        constexpr int slot = decltype(slot_tag)::value;
        const int st = n & 1;
        uint32_t& n_slot = slot ? n_slot1 : n_slot0;
        const uint64_t v = st ? vd[1] : vd[0];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          wait(sm, &sm.pfull[slot][hh], n_slot & 1, p);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(tmem + kColO + 128 * slot, tmem + 128 * slot + 64 * hh + kk * 8, v + ((8192 * hh + kk * 2048) >> 4), idesc_pv,
                   (!fresh || hh > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&sm.odone[slot][hh]);
        }
        ++n_slot;
        if (done) mma_commit(&sm.vempty[st]);
      };
      const auto ready = [&](uint32_t n) {
        wait(sm, &sm.vready[n & 1], (n >> 1) & 1, p);
        tc_fence_after();
      };
      constexpr std::integral_constant<int, 0> s0{};
      constexpr std::integral_constant<int, 1> s1{};
      do {
        if (w.t_begin >= w.t_end) continue;
        const int n = w.t_end - w.t_begin;
        const bool both = kDual || w.it.rows > kRows;
        wait_long(sm, &sm.qfull[0], n_item0++ & 1, p);
        if (both) wait_long(sm, &sm.qfull[1], n_item1++ & 1, p);
        if constexpr (kDual) {                     // the slots take the tiles in turn
          scores(s0, n_tile, true);
          if (n > 1) scores(s1, n_tile + 1, true);
#pragma unroll 1
          for (int i = 0; i < n; i += 2) {
            ready(n_tile + i);
            values(s0, n_tile + i, i == 0, true);
            if (i + 2 < n) scores(s0, n_tile + i + 2, true);
            if (i + 1 < n) {
              ready(n_tile + i + 1);
              values(s1, n_tile + i + 1, i == 0, true);
              if (i + 3 < n) scores(s1, n_tile + i + 3, true);
            }
          }
        } else {
          scores(s0, n_tile, !both);
          if (both) scores(s1, n_tile, true);
#pragma unroll 1
          for (int i = 0; i < n; ++i) {
            ready(n_tile + i);
            values(s0, n_tile + i, i == 0, !both);
            if (i + 1 < n) scores(s0, n_tile + i + 1, !both);
            if (both) {
              values(s1, n_tile + i, i == 0, true);
              if (i + 1 < n) scores(s1, n_tile + i + 1, true);
            }
          }
        }
        n_tile += n;
      } while (w.next(a));
      mma_commit(&sm.drain);
      mbar_drain(&sm.drain, 0, p.wait_ns);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  __syncwarp();
  if (warp == 13) tmem_dealloc(tmem, 512);
  griddep_launch_dependents();
}

// Joins the parts of the items that several blocks worked on.  Block (i, y): the item that begins in
// block i of the attention kernel, its rows [64 y, 64 y + 64), a warp 8 of them, a lane four columns of
// one row at a time.
template <int D>
__global__ void __launch_bounds__(256) attn_join(const Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const AttnArgs& a = p.a;
  const int4 item = p.split[blockIdx.x];
  if (item.w == 0) return;
  const int b = item.x, h = item.y, parts = item.w, lane = threadIdx.x & 31;
  Seq s;
  if (!load_seq(a.seqs, b, a.q.rows, &s)) return;
  const int r = blockIdx.y * 64 + (threadIdx.x >> 5) * 8 + (lane & 7);
  const int gr = (item.z << p.log_rows) + r;
  if (r >> p.log_rows || gr >= s.n * a.group) return;
  const auto slot_of = [&](int x) { return (size_t)(2 * (blockIdx.x + x) + (x == 0)) * kMaxChunkRows; };
  float m = -INFINITY, l = 0.f;
  for (int x = 0; x < parts; ++x) m = fmaxf(m, p.part_ml[slot_of(x) + r].x);
  const float base = m == -INFINITY ? 0.f : m;
  float4 o[D / 16];
#pragma unroll
  for (int c = 0; c < D / 16; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int x = 0; x < parts; ++x) {
    const float2 ml = p.part_ml[slot_of(x) + r];
    const float f = ex2(ml.x - base);
    const float4* src = reinterpret_cast<const float4*>(p.part_o + slot_of(x) * D) + (lane >> 3) * kMaxChunkRows + r;
    l = fmaf(ml.y, f, l);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const float4 v = src[4 * c * kMaxChunkRows];
      o[c].x = fmaf(v.x, f, o[c].x);
      o[c].y = fmaf(v.y, f, o[c].y);
      o[c].z = fmaf(v.z, f, o[c].z);
      o[c].w = fmaf(v.w, f, o[c].w);
    }
  }
  const int i = token_of(a, gr), hh = h * a.group + gr - i * a.group;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2* dst = reinterpret_cast<uint2*>(a.o.data + b * a.o.seq + (long long)(s.row0 + i) * a.o.row + (long long)hh * a.o.head);
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
    dst[4 * c + (lane >> 3)] = make_uint2(pack_bf16x2(o[c].x * inv, o[c].y * inv), pack_bf16x2(o[c].z * inv, o[c].w * inv));
  float* lse = lse_at(a, b, s, i, hh);
  if (lse && lane < 8) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, bool kF8, bool kDual>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& vm, const Params& p, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(Smem<D, kF8>) + 1024;
  if ((e = set_max_dynamic_smem(reinterpret_cast<const void*>(attn_chunk<D, kF8, kDual>), smem))) return e;
  const int blocks = min(sms, kMaxChunkBlocks);
  if ((e = launch_after(attn_chunk<D, kF8, kDual>, dim3(blocks), kThreads, smem, st, km, vm, p)) != cudaSuccess) return e;
  if (p.item_cost < 0) return cudaSuccess;      // no item is cut
  return launch_after(attn_join<D>, dim3(blocks, kMaxChunkRows / 64), 256, 0, st, p);
}

}  // namespace

cudaError_t launch_attention_chunk(const AttnArgs& a, int d, void* ws, unsigned long long wait_ns, int fault, cudaStream_t st) {
  CUtensorMap km, vm;
  const uint64_t rows = (uint64_t)a.pool.num_pages * a.pool.kv_heads * a.pool.page;
  const int esz = a.pool.dtype == PISA_CACHE_E4M3 ? 1 : 2;
  if (!encode_rows(&km, a.pool.k, esz, d, rows, a.pool.page) || !encode_rows(&vm, a.pool.v, esz, d, rows, a.pool.page))
    return cudaErrorInvalidValue;
  Params p;
  p.a = a;
  char* w = static_cast<char*>(ws);
  p.split = reinterpret_cast<int4*>(w + kSplitAt);
  p.part_ml = reinterpret_cast<float2*>(w + kPartialsAt);
  p.part_o = reinterpret_cast<float*>(w + kPartialsAt + sizeof(float2) * 2 * kMaxChunkBlocks * kMaxChunkRows);
  // Short items of which each can have a block to itself are not cut: joining costs 3 us, a tile 2.
  const long long rows_max = (long long)a.seqs.max_new * a.group, pieces = (rows_max + kRows - 1) / kRows;
  const long long span = a.window > 0 ? min((long long)a.seqs.max_len, (long long)a.window + a.seqs.max_new - 1) : a.seqs.max_len;
  const bool whole = span <= 8 * kKeys && pieces * a.pool.kv_heads * a.seqs.batch <= kMaxChunkBlocks;
  // e4m3 tiles are not ready fast enough for two slots that each want their own (190 against 185 us at 4 x 16 heads,
  // 100 rows, 30000 keys; bf16 133 against 149, with head_dim 64 107 against 146)
  const bool dual = whole || (rows_max <= kRows && esz == 2);
  p.log_rows = dual ? 7 : 8;
  p.item_cost = whole ? -1 : 2;
  p.wait_ns = wait_ns;
  p.fault = fault;
  const auto go = [&](auto f8, auto dual) {
    return d == 64 ? launch<64, decltype(f8)::value, decltype(dual)::value>(km, vm, p, st)
                   : launch<128, decltype(f8)::value, decltype(dual)::value>(km, vm, p, st);
  };
  const std::true_type yes;
  const std::false_type no;
  if (esz == 1) return dual ? go(yes, yes) : go(yes, no);
  return dual ? go(no, yes) : go(no, no);
}

}  // namespace cache
}  // namespace pisa
