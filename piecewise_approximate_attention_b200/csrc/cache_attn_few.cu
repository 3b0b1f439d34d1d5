// Attention over the paged cache for few query rows a key/value head (single tokens, a handful of
// tokens): bf16 and e4m3 pools.
//
// The new tokens of a sequence times the group of query heads that share a key/value head are the
// rows (at most 64) of one small matrix product with that head's keys, so every stored key and value
// is read from HBM once and serves all of them; the kernel is bound by that stream.
//
// Work: an item is (sequence, key/value head); its keys are cut into tiles of 64 (e4m3: 128, the same
// bytes).  All items' tiles form one line that is cut into equal shares, one a block, whatever the
// lengths: a block walks through the end of one item, whole items, and the beginning of another.
// Items that several blocks share leave partial results (O, maximum, sum) in the workspace; the block
// that finishes last joins them in the order of the blocks, so the result does not depend on which
// that is.  Short items with a block each are not cut.
//
// Block: a producer warp that follows the page table and fills a ring of shared-memory stages with
// TMA (a 128-byte-swizzled box a page), and 4 consumer warps, which multiply by mma.m16n8k16 (rows are
// too few to fill a tcgen05 tile), keep running maxima and sums of their own, and are joined at the
// item's end.  At most 8 rows (attn_row8): keys are the MMA's 16 rows and the query rows its 8 columns,
// so no half of it is empty; each warp takes a quarter of the tile's keys.  Up to 16, 32 and 64 rows (attn_few, MT
// row tiles of 16): MT row groups x 4 / MT key groups.  O is rescaled only when a row's maximum grows by
// more than 2^8 (weights stay finite, sums are fp32).
//
// Measured: 32 sequences of up to 32760 tokens, 40 heads on 8, bf16: 328 us (6.8 TB/s: the stream, a
// little of it from L2); 64 sequences of up to 4608 tokens, 24 heads, e4m3: 159 us (5.9 TB/s).  More than 16 rows of an e4m3
// pool are bound by latency between a warp's steps instead (30 rows 358 us where the stream takes 169; issue slots 41%,
// tensor pipe 27%, 8 warps an SM): the warps of a key group convert the same codes, each for its row tile.
//
// bf16 pools: the type of V asks for bf16 weights.  At most 16 rows, a weight enters as two bf16 numbers, itself and
// what rounding left over (16 bits), which costs nothing beside the stream (326.4 and 327.0 us above; the error against
// float64 falls from 2.35e-3, the output's rounding and the weights', to 1.67e-3, the output's alone).  Above, where
// the second product would cost 23% (30 rows) to 38% (60), weights are bf16, off by 2^-8 at most, and the maximum is
// also moved where a key outweighs twice what its lane has of the row so far, so that a key which holds two thirds of a
// row or more weighs exactly 1 and such a row is not off by its rounding (60 rows 548 -> 555 us).
//
// e4m3 pools: codes become fp16 exactly (one instruction for two), q becomes fp16 with a power of
// two per row, also exactly, and a key's scales act on the logits: with x_j = s_j + e_j (e_j the
// exponent of v_j's scale, in base-2 logits) the weight of code row j is 2^(x_j - M), M the maximum of
// the x, and the sum takes 2^(x_j - M) 2^-e_j.  So the fp16 weights keep 11 bits for what counts most
// in O, however the rows' scales differ.  (x_j is rounded like a number of e_j's size, so a log-sum-exp is off by up to
// 2^-18 where scales are as far from 1 as they may be.)
//
// Positions that a row does not see get weight zero; the V rows behind the last position (stale
// slots) are zeroed in registers, because 0 * NaN is NaN, and a value that is not finite where only
// some rows see it is taken out of the product and added to those rows alone.
#include <type_traits>

#include "cache_pipe.cuh"
#include "cache_walk.cuh"
#include "sm100.cuh"

namespace pisa {
namespace cache {
namespace {
using namespace sm100;

constexpr int kConsumers = 128;
constexpr int kThreads = kConsumers + 32;
constexpr float kLazyLog2 = 8.f;
constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int D, bool kF8>
struct Layout {
  static constexpr int kTile = kF8 ? 128 : 64;                    // keys: the same bytes either way
  static constexpr int kRowBytes = kF8 ? D : 128;                 // of a swizzled tile's row
  static constexpr int kHalves = kF8 ? 1 : D / 64;                // 64-column bf16 halves
  static constexpr int kSide = kTile * D * (kF8 ? 1 : 2);         // bytes of a K or V tile
  static constexpr int kStages = D == 128 ? 3 : 6;
};

template <int D, bool kF8>
struct alignas(1024) Smem {
  using L = Layout<D, kF8>;
  uint8_t k[L::kStages][L::kSide];
  uint8_t v[L::kStages][L::kSide];
  uint8_t ke[L::kStages][kF8 ? L::kTile : 16];
  uint8_t ve[L::kStages][kF8 ? L::kTile : 16];
  uint64_t full[L::kStages], empty[L::kStages];
  unsigned long long bad[L::kStages][L::kTile / 64];      // keys of the tile whose page is no page of the pool, or is not there
  long long scan[kThreads / 32], before;
  int items[kThreads / 32], longest[kThreads / 32];
  float4 join[kConsumers * 2];               // joining the parts of an item: the groups' O, maxima and sums
  float2 join_ml[16];
  float2 ml[4][16];                          // maximum and sum of the rows that a warp hands over
  int start_b, abort, last;
};

struct Params {
  AttnArgs a;
  int* counters;             // one a block, zero between calls
  float2* part_ml;           // [2 * blocks][64]: maximum and sum of a partial result's rows
  float* part_o;             // [2 * blocks][64][D]
  int item_cost, fault;      // what an item costs besides its tiles, in tiles
  unsigned long long wait_ns;
};

// An item's keys in tiles: tiles [t0, t0 + n) of the sequence, n = 0 for no new token.
struct Item {
  Seq s;
  int t0, n, first;             // first: the first key that any row sees
};
template <int kTile>
__device__ __forceinline__ Item load_item(const AttnArgs& a, int b) {
  Item it;
  it.t0 = it.n = it.first = 0;
  if (!load_seq(a.seqs, b, a.q.rows, &it.s) || it.s.n == 0) return it;
  const int first = a.window > 0 ? max(0, min(it.s.len, it.s.len - it.s.n - a.window + 1)) : 0;
  it.first = first;
  it.t0 = first / kTile;
  it.n = max(1, (it.s.len + kTile - 1) / kTile - it.t0);      // an empty sequence's rows are written too
  return it;
}

template <typename S>
__device__ __forceinline__ bool wait(S& sm, uint64_t* bar, uint32_t parity, const Params& p) {
  return wait_for(sm, bar, parity, p.wait_ns, p.a.seqs.status);
}

// Byte offset of 16-byte chunk c of row r in a tile as TMA wrote it.
template <int D, bool kF8>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if (kF8) return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  return (c >> 3) * (64 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Element (row r, column c) of a V tile.
template <int D, bool kF8>
__device__ __forceinline__ float value_at(const uint8_t* tile, int r, int c) {
  if (kF8) {
    const uint32_t h = e4m3x2_to_f16x2(tile[chunk_at<D, true>(r, c >> 4) + (c & 15)]);
    return __half2float(__ushort_as_half((unsigned short)h));
  }
  return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(tile + chunk_at<D, false>(r, c >> 3) + 2 * (c & 7)));
}

// A block's share of the line, and where it is in it; every warp walks its own copy.
//
// In the line an item takes n places for its tiles and then item_cost for what it costs besides them.  Shares are at
// least two places long, and no item is cut in more than 24 parts or so: past that, joining them costs more than the
// shorter shares save (16 heads on 4, 8000 tokens: 13.2 us, 14.3 with 48 parts, 15.6 with 96).  Short items of which each
// can have a block to itself are not cut, and take one place each: joining parts costs 3 us (200 tokens, 4 heads: 6.4 us
// whole, 8.2 cut; 577 tokens: 10.3 and 8.8).  All of this goes by the lengths and the window that the device finds: the
// caller's bound may be far above them (a captured step; 4 heads, a window of 1024 in 75600 tokens: 37.9 us by the bound, 10.1 so).
constexpr int kMostParts = 24, kWholeTiles = 6, kWholeItems = 148;
template <int kTile>
struct FewWalk {
  long long u0, u1, share, item0;     // places: this block's, how long shares are, the item's first
  int b, h, t_begin, t_end, item_cost;      // item_cost < 0: items are not cut
  Item it;

  __device__ __forceinline__ int cost(int tiles) const { return tiles == 0 ? 0 : item_cost < 0 ? 1 : tiles + item_cost; }

  // Whole block; false if the line ends before this block's share.
  template <typename S>
  __device__ __forceinline__ bool start(const AttnArgs& a, S& sm, int cost_of_item) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const auto tiles = [&](int b) { return b < a.seqs.batch ? load_item<kTile>(a, b).n : 0; };
    const auto scan = [&](long long n) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long up = __shfl_up_sync(FULL, n, d);
        if (lane >= d) n += up;
      }
      return n;
    };
    long long before = 0;
    if (a.seqs.batch <= 32) {         // each warp by itself
      const int mine = tiles(lane);
      const int longest = __reduce_max_sync(FULL, mine);
      choose(a, longest, cost_of_item);
      const long long n = (long long)cost(mine) * a.pool.kv_heads, upto = scan(n);
      shares(__shfl_sync(FULL, upto, 31), longest);
      if (u0 >= u1) return false;
      const int w = __ffs(__ballot_sync(FULL, upto > u0)) - 1;
      b = w;
      before = __shfl_sync(FULL, upto - n, w);
    } else {
      long long total = 0;
      int items = 0, longest = 0;
      for (int i = threadIdx.x; i < a.seqs.batch; i += kThreads) {
        const int n = tiles(i);
        total += n;
        items += n > 0;
        longest = max(longest, n);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(FULL, total, d);
      items = __reduce_add_sync(FULL, items);
      longest = __reduce_max_sync(FULL, longest);
      if (lane == 0) {
        sm.scan[warp] = total;
        sm.items[warp] = items;
        sm.longest[warp] = longest;
      }
      __syncthreads();
      total = items = longest = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        total += sm.scan[w];
        items += sm.items[w];
        longest = max(longest, sm.longest[w]);
      }
      choose(a, longest, cost_of_item);
      shares((item_cost < 0 ? items : total + (long long)items * item_cost) * a.pool.kv_heads, longest);
      if (u0 >= u1) return false;
      if (warp == 0) {                // 32 sequences at a time
        long long base = 0;
        for (int b0 = 0; b0 < a.seqs.batch; b0 += 32) {
          const long long n = (long long)cost(tiles(b0 + lane)) * a.pool.kv_heads, upto = scan(n);
          const unsigned hit = __ballot_sync(FULL, base + upto > u0);
          if (hit) {
            const int w = __ffs(hit) - 1;
            if (lane == w) {
              sm.start_b = b0 + w;
              sm.before = base + upto - n;
            }
            break;
          }
          base += __shfl_sync(FULL, upto, 31);
        }
      }
      __syncthreads();
      b = sm.start_b;
      before = sm.before;
    }
    it = load_item<kTile>(a, b);
    h = (int)quotient(u0 - before, cost(it.n));
    item0 = before + (long long)h * cost(it.n);
    enter();
    return true;
  }
  __device__ __forceinline__ void choose(const AttnArgs& a, int longest, int cost_of_item) {
    item_cost = longest <= kWholeTiles && (long long)a.seqs.batch * a.pool.kv_heads <= kWholeItems ? -1 : cost_of_item;
  }
  __device__ __forceinline__ void shares(long long total, int longest) {
    const int least = item_cost < 0 ? 1 : max(2, (longest + kMostParts - 1) / kMostParts);
    share = max((long long)least, quotient(total + gridDim.x - 1, gridDim.x));
    u0 = share * blockIdx.x;
    u1 = min(total, u0 + share);
  }
  // the tiles of the item that are this block's: none where its share holds only the item's last places
  __device__ __forceinline__ void enter() {
    if (item_cost < 0) {              // items are not cut
      t_begin = it.t0;
      t_end = it.t0 + it.n;
      return;
    }
    t_begin = it.t0 + (int)min((long long)it.n, max(0LL, u0 - item0));
    t_end = it.t0 + (int)min((long long)it.n, u1 - item0);
  }
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    item0 += cost(it.n);
    if (item0 >= u1) return false;
    if (++h == a.pool.kv_heads) {
      h = 0;
      do it = load_item<kTile>(a, ++b); while (it.n == 0);   // the line goes on: there is one
    }
    enter();
    return true;
  }
  // Blocks that work on the item, and this block's part of it: the end (2 * block) or the beginning (+ 1).
  __device__ __forceinline__ int first_block() const { return (int)quotient(item0, share); }
  __device__ __forceinline__ int last_block() const { return item_cost < 0 ? first_block() : (int)quotient(item0 + it.n - 1, share); }
  __device__ __forceinline__ size_t part() const { return (size_t)(2 * blockIdx.x + (item0 < u0 ? 0 : 1)) * kMaxFewRows; }
};
__device__ __forceinline__ size_t part_of(int block, int first) { return (size_t)(2 * block + (block == first)) * kMaxFewRows; }

// The producer warp: follows the page table and fills the ring.  kJoin: a stage after each item's tiles
// is left to the consumers, to join their results in.
template <int D, bool kF8, bool kJoin, bool kCheck, typename S>
__device__ __forceinline__ void produce(S& sm, const CUtensorMap& kmap, const CUtensorMap& vmap, const Params& p,
                                        FewWalk<Layout<D, kF8>::kTile>& w) {
  using L = Layout<D, kF8>;
  constexpr int kTile = L::kTile, kStages = L::kStages;
  const AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  const int box = min(a.pool.page, kTile), log_box = min(a.pool.page_log2, kF8 ? 7 : 6), pages = kTile >> log_box;   // boxes of a tile
  constexpr int per = 2 * L::kHalves;                                  // copies of a box
  const uint32_t box_bytes = 2u * box * D * (kF8 ? 1 : 2) + (kF8 ? 2u * box : 0u);
  int skip = p.fault != 0, ring = skip;                                // stages used so far; skip: a test's stage that never fills
  bool ok = true;
  do {
    for (int t = w.t_begin + skip; t < w.t_end; ++t, ++ring) {
      const int st = ring % kStages;
      // lane i < pages looks box i's page up
      int row = -1;
      const int pos = t * kTile + lane * box;
      if (lane < pages && pos < w.it.s.len && pos + box > w.it.first) {
        const int pg = load_page(a.seqs, a.pool, w.b, pos);
        if (pg >= 0) row = (pg * a.pool.kv_heads + w.h) * a.pool.page + (pos & (a.pool.page - 1));
      }
      if (ring >= kStages) ok = wait(sm, &sm.empty[st], (ring / kStages - 1) & 1, p) && !(kCheck && aborted(sm));
      // one vote for the pages (at most 8) and whether there is room, for all lanes what the last one saw
      const unsigned have = __ballot_sync(FULL, lane < 31 ? row >= 0 : !ok);
      ok = !(have >> 31);
      if (!ok) break;
      if (lane < kTile / 64) {
        unsigned long long bits = 0;
        for (int i = 0; i < 64; i += 16)
          if (!((have >> ((lane * 64 + i) >> log_box)) & 1u)) bits |= 0xffffull << i;
        sm.bad[st][lane] = bits;
      }
      __syncwarp();
      if (lane == 0) mbar_expect_tx(&sm.full[st], __popc(have) * box_bytes);
      __syncwarp();
      // copies (box, K or V, half) over the lanes: at most 32
      const int i = lane / per, side = lane % per & 1, half = lane % per >> 1;
      const int r = __shfl_sync(FULL, row, i);
      if (i < pages && r >= 0) {
        uint8_t* dst = (side ? sm.v[st] : sm.k[st]) + half * (kTile * 128) + i * box * L::kRowBytes;
        tma_load_3d(dst, side ? &vmap : &kmap, &sm.full[st], half * 64, r, 0);
        if (kF8) bulk_load((side ? sm.ve[st] : sm.ke[st]) + i * box, (side ? a.pool.v_exp : a.pool.k_exp) + r, box, &sm.full[st]);
      }
    }
    skip = 0;
    if (kJoin && ok && w.t_begin < w.t_end) {
      const int st = ring % kStages;
      if (ring >= kStages) ok = __all_sync(FULL, wait(sm, &sm.empty[st], (ring / kStages - 1) & 1, p) && !(kCheck && aborted(sm)));
      if (ok && lane == 0) mbar_arrive(&sm.full[st]);
      ring += ok;
    }
  } while (ok && w.next(a));
  // every copy lands before this block's shared memory is released
  if (lane == 0)
    for (int i = max(0, ring - kStages); i < ring; ++i) mbar_drain(&sm.full[i % kStages], (i / kStages) & 1, p.wait_ns);
}

// Barriers, and whether the block has a share.
template <int D, bool kF8, typename S>
__device__ __forceinline__ bool set_up(S& sm, const Params& p, FewWalk<Layout<D, kF8>::kTile>& w) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < Layout<D, kF8>::kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 4);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  griddep_launch_dependents();
  griddep_wait();
  const bool any = w.start(p.a, sm, p.item_cost);
  __syncthreads();
  return any;
}

// Whether this block is the last to end of those that share an item.  Consumer warps only.
template <typename S>
__device__ __forceinline__ bool ends_last(S& sm, const Params& p, int c0, int c1) {
  __threadfence();
  consumer_sync();
  if (threadIdx.x == 0) {
    const bool done = atomicAdd(p.counters + c0, 1) == c1 - c0;
    if (done) p.counters[c0] = 0;                            // as the next call finds it
    sm.last = done;
  }
  consumer_sync();
  const bool last = sm.last;
  if (last) __threadfence();
  return last;
}
// Joins the parts of an item, in the order of the blocks.  A group of D / 8 threads (eight columns each)
// takes a row, or, when there are fewer rows than groups, every kSub-th part of one.
template <int D, typename S>
__device__ __forceinline__ void join_parts(S& sm, const Params& p, const Item& it, int b, int h, int c0, int c1) {
  constexpr int kLanes = D / 8, kGroups = kConsumers / kLanes;
  const AttnArgs& a = p.a;
  const int x = threadIdx.x % kLanes, grp = threadIdx.x / kLanes, rows = it.s.n * a.group, parts = c1 - c0 + 1;
  int subs = 1;                                              // groups a row
  while (subs < 8 && subs * 2 * rows <= kGroups) subs *= 2;
  const int sub = grp % subs;
  // uniform trips: the shuffles take whole warps
  for (int r0 = 0; r0 < rows; r0 += kGroups / subs) {
    const int r = r0 + grp / subs, rr = min(r, rows - 1);
    float m = -INFINITY, l = 0.f;
    float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int y0 = 0; y0 < parts; y0 += kLanes * subs) {      // lane x: part y0 + x * subs + sub
      const int mine = y0 + x * subs + sub;
      const float2 ml = mine < parts ? __ldcg(&p.part_ml[part_of(c0 + mine, c0) + rr]) : make_float2(-INFINITY, 0.f);
      float mx = ml.x;
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, d, kLanes));
      const float m_new = fmaxf(m, mx), base = m_new == -INFINITY ? 0.f : m_new;
      const float f0 = ex2(m - base), fx = ex2(ml.x - base);
      float sum = ml.y * fx;
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d, kLanes);
      l = l * f0 + sum;
      m = m_new;
#pragma unroll
      for (int e = 0; e < 2; ++e) o[e] = make_float4(o[e].x * f0, o[e].y * f0, o[e].z * f0, o[e].w * f0);
      const int left = parts - y0, turns = min(kLanes, (left + subs - 1) / subs);
#pragma unroll 8
      for (int y = 0; y < turns; ++y) {
        const int part = y0 + y * subs + sub;
        const float f = __shfl_sync(FULL, fx, y, kLanes);
        if (part < parts) {
          const float4* src = reinterpret_cast<const float4*>(p.part_o + (part_of(c0 + part, c0) + rr) * D) + 2 * x;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 v = __ldcg(src + e);
            o[e].x = fmaf(v.x, f, o[e].x);
            o[e].y = fmaf(v.y, f, o[e].y);
            o[e].z = fmaf(v.z, f, o[e].z);
            o[e].w = fmaf(v.w, f, o[e].w);
          }
        }
      }
    }
    if (subs > 1) {                                          // the groups of a row, in their order
      consumer_sync();
      float4* at = reinterpret_cast<float4*>(sm.join) + grp * 2 * kLanes + 2 * x;
      at[0] = o[0];
      at[1] = o[1];
      if (x == 0) sm.join_ml[grp] = make_float2(m, l);
      consumer_sync();
      if (sub == 0) {
        float mm = -INFINITY;
        for (int y = 0; y < subs; ++y) mm = fmaxf(mm, sm.join_ml[grp + y].x);
        const float base = mm == -INFINITY ? 0.f : mm;
        m = mm;
        l = 0.f;
        o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int y = 0; y < subs; ++y) {
          const float f = ex2(sm.join_ml[grp + y].x - base);
          l = fmaf(sm.join_ml[grp + y].y, f, l);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 v = at[y * 2 * kLanes + e];
            o[e].x = fmaf(v.x, f, o[e].x);
            o[e].y = fmaf(v.y, f, o[e].y);
            o[e].z = fmaf(v.z, f, o[e].z);
            o[e].w = fmaf(v.w, f, o[e].w);
          }
        }
      }
    }
    if (r >= rows || sub != 0) continue;
    const int i = token_of(a, r), hh = h * a.group + r - i * a.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    char* dst = a.o.data + b * a.o.seq + (long long)(it.s.row0 + i) * a.o.row + (long long)hh * a.o.head;
    *reinterpret_cast<uint4*>(dst + x * 16) = make_uint4(pack_bf16x2(o[0].x * inv, o[0].y * inv), pack_bf16x2(o[0].z * inv, o[0].w * inv),
                                                        pack_bf16x2(o[1].x * inv, o[1].y * inv), pack_bf16x2(o[1].z * inv, o[1].w * inv));
    float* lse = lse_at(a, b, it.s, i, hh);
    if (lse && x == 0) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

// Two weights as bf16 numbers, and what their rounding left over.
__device__ __forceinline__ void split_bf16x2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// At most 8 rows: the keys are the 16 rows of the MMA's A operand and the queries its 8 columns, which
// takes half the instructions and half the accumulators of the form below.  S^T = K Q^T, O^T += V^T P^T;
// P^T is turned from the scores' layout to the operand's by movmatrix.  Each warp takes kTile / 4 keys
// of a tile.  The warps' O meet in a stage of the ring, 16 threads finish a row.
template <int D, bool kF8>
__global__ void __launch_bounds__(kThreads, 2)
attn_row8(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Params p) {
  using L = Layout<D, kF8>;
  constexpr int kStages = L::kStages, kTile = L::kTile, kSub = kTile / 64;     // 16-key pieces of a warp's keys
  extern __shared__ uint8_t smem_raw[];
  Smem<D, kF8>& sm = *reinterpret_cast<Smem<D, kF8>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  FewWalk<kTile> wk;
  if (!set_up<D, kF8>(sm, p, wk)) return;
  if (warp == 4) {
    produce<D, kF8, true, false>(sm, kmap, vmap, p, wk);
    return;
  }
  const int g = lane >> 2, q4 = lane & 3;
  int ring = 0;                                               // stages used so far
  do {
    if (wk.t_begin >= wk.t_end) continue;
    const Item& it = wk.it;
    const int b = wk.b, h = wk.h, rows = it.s.n * a.group;
    // query row g into the B fragments
    uint32_t qb[D / 16][2];
    float rs_g = a.scale_log2;                                // raw score -> base-2 logit
    {
      const char* src = nullptr;
      if (g < rows) {
        const int i = token_of(a, g), hh = h * a.group + g - i * a.group;
        src = a.q.data + b * a.q.seq + (long long)(it.s.row0 + i) * a.q.row + (long long)hh * a.q.head;
      }
      if constexpr (kF8) {
        // K fragments hold codes 4 q4 ... 4 q4 + 3 of a 16-code chunk as their k positions 2 q4, 2 q4 + 1 and +8
        uint2 x[D / 16];
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          x[c] = src ? *reinterpret_cast<const uint2*>(src + c * 32 + q4 * 8) : make_uint2(0, 0);
          mx = max(mx, max(max((x[c].x << 16) & 0x7fff0000u, x[c].x & 0x7fff0000u),
                           max((x[c].y << 16) & 0x7fff0000u, x[c].y & 0x7fff0000u)));
        }
        mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
        mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
        // largest magnitude to [2^14, 2^15): every bf16 down to 2^-31 of it is an fp16 number
        const int eq = max(-100, min(112, (int)(mx >> 23) - 127 - 14));
        const float s = pow2(-eq);
        rs_g *= pow2(eq);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          qb[c][0] = pack_f16x2(__uint_as_float(x[c].x << 16) * s, __uint_as_float(x[c].x & 0xffff0000u) * s);
          qb[c][1] = pack_f16x2(__uint_as_float(x[c].y << 16) * s, __uint_as_float(x[c].y & 0xffff0000u) * s);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          qb[c][0] = src ? *reinterpret_cast<const uint32_t*>(src + c * 32 + q4 * 4) : 0u;
          qb[c][1] = src ? *reinterpret_cast<const uint32_t*>(src + c * 32 + 16 + q4 * 4) : 0u;
        }
      }
    }
    // rows 2 q4 and 2 q4 + 1: the columns of my scores
    float rs[2];
    int first[2], last[2], all_first = 0, all_last = it.s.len;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * q4 + e;
      rs[e] = __shfl_sync(FULL, rs_g, r * 4);
      first[e] = last[e] = 0;
      if (r < rows) {
        visible(a, it.s.len, it.s.len - it.s.n + token_of(a, r), &first[e], &last[e]);
        all_first = max(all_first, first[e]);
        all_last = min(all_last, last[e]);
      }
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {                         // keys that all rows see: only those tiles need no masks
      all_first = max(all_first, __shfl_xor_sync(FULL, all_first, d));
      all_last = min(all_last, __shfl_xor_sync(FULL, all_last, d));
    }
    float acc[D / 16][4];                                     // rows 2 q4, 2 q4 + 1 of two columns (d_of)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
    const auto d_of = [&](int c, int e) { return kF8 ? 16 * c + 2 * g + e : 16 * c + g + 8 * e; };
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int t = wk.t_begin; t < wk.t_end; ++t, ++ring) {
      const int st = ring % kStages;
      const bool landed = wait(sm, &sm.full[st], (ring / kStages) & 1, p);
      const uint32_t kb = smem_u32(sm.k[st]), vb = smem_u32(sm.v[st]);
      const int k0 = warp * (kTile / 4), j0 = t * kTile + k0;
      const unsigned bad_bits = (unsigned)(sm.bad[st][k0 >> 6] >> (k0 & 63)) & (kSub == 1 ? 0xffffu : FULL);
      // this warp's keys of the tile; edge: some row does not see some of them
      const auto keys = [&](auto edge_tag) {
        constexpr bool edge = decltype(edge_tag)::value;
        // ---- scores: keys g and g + 8 of each piece, rows 2 q4 and 2 q4 + 1 ----
        float s[kSub][4] = {};
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            const int key = k0 + 16 * u + ((lane >> 3) & 1) * 8 + (lane & 7);
            uint32_t x[4];
            if constexpr (kF8) {
              if (c & 1) continue;
              ldsm4(kb + chunk_at<D, true>(key, c + (lane >> 4)), x);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t lo = x[2 * e], hi = x[2 * e + 1];
                const uint32_t A[4] = {e4m3x2_to_f16x2((uint16_t)lo), e4m3x2_to_f16x2((uint16_t)hi),
                                       e4m3x2_to_f16x2((uint16_t)(lo >> 16)), e4m3x2_to_f16x2((uint16_t)(hi >> 16))};
                mma16816<true>(s[u], A, qb[c + e][0], qb[c + e][1]);
              }
            } else {
              ldsm4(kb + chunk_at<D, false>(key, 2 * c + (lane >> 4)), x);
              mma16816<false>(s[u], x, qb[c][0], qb[c][1]);
            }
          }
        // ---- base-2 logits (e4m3: plus the exponent of the value's scale) ----
        float inv[kSub][2];                                   // e4m3: 2^-e of my keys' values
        unsigned seen[kSub];
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          seen[u] = 0xfu;
          if (edge) seen[u] = 0u;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int kk = 16 * u + 8 * x + g;
            float ks = 1.f, ef = 0.f;
            if (kF8) {
              const uint32_t vx = sm.ve[st][k0 + kk];
              ks = __uint_as_float((uint32_t)sm.ke[st][k0 + kk] << 23);
              ef = (float)((int)vx - kExpBias);
              inv[u][x] = __uint_as_float((254u - vx) << 23);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& y = s[u][2 * x + e];
              y = kF8 ? fmaf(y * ks, rs[e], ef) : y * a.scale_log2;
              if (edge) {
                const int j = j0 + kk;
                if (j >= first[e] && j < last[e] && !((bad_bits >> kk) & 1u)) seen[u] |= 1u << (2 * x + e);
                else y = -INFINITY;
              }
              top[e] = fmaxf(top[e], y);
            }
          }
        }
        // ---- running maximum: moved only when a row outgrows it by 2^8 ----
        if (__any_sync(FULL, top[0] > m[0] + kLazyLog2 || top[1] > m[1] + kLazyLog2)) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(FULL, top[e], d));
            const float mn = fmaxf(m[e], top[e]);
            f[e] = mn == -INFINITY ? 1.f : ex2(m[e] - mn);
            m[e] = mn;
            l[e] *= f[e];
          }
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[c][x] *= f[x & 1];
        }
        const float mb[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        [[maybe_unused]] uint32_t pb[kSub][2], pl[kSub][2];   // pl: bf16 weights' second parts
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& y = s[u][2 * x + e];
              y = ex2(y - mb[e]);
              if (kF8) {
                if (!edge || ((seen[u] >> (2 * x + e)) & 1u)) l[e] = fmaf(y, inv[u][x], l[e]);
              } else {
                l[e] += y;
              }
            }
            if constexpr (kF8) {
              pb[u][x] = transpose8x8(pack_f16x2(s[u][2 * x], s[u][2 * x + 1]));
            } else {
              uint32_t hi, lo;
              split_bf16x2(s[u][2 * x], s[u][2 * x + 1], hi, lo);
              pb[u][x] = transpose8x8(hi);
              pl[u][x] = transpose8x8(lo);
            }
          }
        // ---- O^T += V^T P^T; A fragments hold keys 2 q4, 2 q4 + 1 and +8 ----
        uint32_t keep[kSub][2];
        if (edge) {
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              keep[u][n] = 0;
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int kk = 16 * u + 8 * n + 2 * q4 + x;
                if (j0 + kk < it.s.len && !((bad_bits >> kk) & 1u)) keep[u][n] |= 0xffffu << (16 * x);
              }
            }
        }
        constexpr uint32_t kInf = kF8 ? 0x7c007c00u : 0x7f807f80u;
        bool odd = false;                                     // a value that is not finite where not all rows see it
        const auto clean = [&](uint32_t x, int u, int n) -> uint32_t {
          if (!edge) return x;
          x &= keep[u][n];
          const bool lo = (x & kInf & 0xffffu) == (kInf & 0xffffu), hi = (x & kInf & 0xffff0000u) == (kInf & 0xffff0000u);
          odd = odd || lo || hi;
          if (lo) x &= 0xffff0000u;
          if (hi) x &= 0x0000ffffu;
          return x;
        };
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t x[4];
            if constexpr (kF8) {
              if (c & 1) continue;
              ldsm4t(vb + chunk_at<D, true>(k0 + 16 * u + ((lane >> 3) & 1) * 8 + (lane & 7), c + (lane >> 4)), x);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // bytes (key, d), (key, d + 1), (key + 1, d), (key + 1, d + 1) -> pairs of keys for d and for d + 1
                const uint32_t lo = __byte_perm(x[2 * e], 0, 0x3120), hi = __byte_perm(x[2 * e + 1], 0, 0x3120);
                const uint32_t A[4] = {clean(e4m3x2_to_f16x2((uint16_t)lo), u, 0), clean(e4m3x2_to_f16x2((uint16_t)(lo >> 16)), u, 0),
                                       clean(e4m3x2_to_f16x2((uint16_t)hi), u, 1), clean(e4m3x2_to_f16x2((uint16_t)(hi >> 16)), u, 1)};
                mma16816<true>(acc[c + e], A, pb[u][0], pb[u][1]);
              }
            } else {
              ldsm4t(vb + chunk_at<D, false>(k0 + 16 * u + (lane >> 4) * 8 + (lane & 7), 2 * c + ((lane >> 3) & 1)), x);
              const uint32_t A[4] = {clean(x[0], u, 0), clean(x[1], u, 0), clean(x[2], u, 1), clean(x[3], u, 1)};
              mma16816<false>(acc[c], A, pb[u][0], pb[u][1]);
              mma16816<false>(acc[c], A, pl[u][0], pl[u][1]);
            }
          }
        if (edge && __any_sync(FULL, odd)) {
          // rare: add what was taken out, to the rows that see it
#pragma unroll 1
          for (int kk = 0; kk < 16 * kSub; ++kk) {
            if (j0 + kk >= it.s.len || ((bad_bits >> kk) & 1u)) continue;
            const int src = (kk & 7) * 4 + q4, x = (kk >> 3) & 1;
            float wk2[2];
            bool sk[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float y = 0.f;
              unsigned z = 0;
#pragma unroll
              for (int u = 0; u < kSub; ++u)
                if (u == kk >> 4) {
                  y = x ? s[u][2 + e] : s[u][e];
                  z = seen[u];
                }
              wk2[e] = __shfl_sync(FULL, y, src);
              sk[e] = (__shfl_sync(FULL, z, src) >> (2 * x + e)) & 1u;
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float val = value_at<D, kF8>(sm.v[st], k0 + kk, d_of(c, y));
                if (isfinite(val)) continue;
                if (sk[0]) acc[c][2 * y] = fmaf(wk2[0], val, acc[c][2 * y]);
                if (sk[1]) acc[c][2 * y + 1] = fmaf(wk2[1], val, acc[c][2 * y + 1]);
              }
          }
        }
      };
      if (j0 < all_first || j0 + kTile / 4 > all_last || bad_bits) keys(std::true_type());
      else keys(std::false_type());
      __syncwarp();
      if (lane == 0 && landed) mbar_arrive(&sm.empty[st]);
    }

    // ---- the warps' results meet in a stage: rows of D + 4 floats ----
    const int st = ring % kStages;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(FULL, l[e], d);
    const bool landed = wait(sm, &sm.full[st], (ring / kStages) & 1, p);
    constexpr int kLd = D + 4;
    static_assert(2 * 8 * kLd * 4 <= L::kSide, "two warps' O fit one side of a stage");
    const auto scratch = [&](int w) { return reinterpret_cast<float*>(w & 2 ? sm.v[st] : sm.k[st]) + (w & 1) * 8 * kLd; };
    {
      float* buf = scratch(warp);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* at = buf + (2 * q4 + e) * kLd;
          if (kF8) {
            *reinterpret_cast<float2*>(at + d_of(c, 0)) = make_float2(acc[c][e], acc[c][2 + e]);
          } else {
            at[d_of(c, 0)] = acc[c][e];
            at[d_of(c, 1)] = acc[c][2 + e];
          }
        }
      if (g == 0) {
        sm.ml[warp][2 * q4] = make_float2(m[0], l[0]);
        sm.ml[warp][2 * q4 + 1] = make_float2(m[1], l[1]);
      }
    }
    consumer_sync();
    const int c0 = wk.first_block(), c1 = wk.last_block();
    {
      const int r = threadIdx.x >> 4, x = threadIdx.x & 15;   // 16 threads a row, float4 columns x + 16 y
      float mm = -INFINITY, ll = 0.f, f[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sm.ml[w][r].x);
      const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[w] = ex2(sm.ml[w][r].x - base);
        ll = fmaf(sm.ml[w][r].y, f[w], ll);
      }
      if (r < rows) {
        const int i = token_of(a, r), hh = h * a.group + r - i * a.group;
        const float sc = c0 != c1 ? 1.f : ll == 0.f ? 0.f : 1.f / ll;
        char* dst = a.o.data + b * a.o.seq + (long long)(it.s.row0 + i) * a.o.row + (long long)hh * a.o.head;
        const size_t part = wk.part() + r;
#pragma unroll
        for (int y = 0; y < D / 64; ++y) {
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(scratch(w) + r * kLd + 4 * x + 64 * y);
            o.x = fmaf(v.x, f[w], o.x);
            o.y = fmaf(v.y, f[w], o.y);
            o.z = fmaf(v.z, f[w], o.z);
            o.w = fmaf(v.w, f[w], o.w);
          }
          if (c0 == c1)
            *reinterpret_cast<uint2*>(dst + (4 * x + 64 * y) * 2) = make_uint2(pack_bf16x2(o.x * sc, o.y * sc), pack_bf16x2(o.z * sc, o.w * sc));
          else
            *reinterpret_cast<float4*>(p.part_o + part * D + 4 * x + 64 * y) = o;
        }
        if (x == 0) {
          if (c0 != c1) p.part_ml[part] = make_float2(mm, ll);
          else if (float* lse = lse_at(a, b, it.s, i, hh)) *lse = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
        }
      }
    }
    fence_async_shared();                                     // the stage goes back to TMA
    consumer_sync();
    if (lane == 0 && landed) mbar_arrive(&sm.empty[st]);
    ++ring;
    if (c0 != c1 && ends_last(sm, p, c0, c1)) join_parts<D>(sm, p, it, b, h, c0, c1);
  } while (wk.next(a));
}

template <int D, bool kF8, int MT>
__global__ void __launch_bounds__(kThreads, 2)
attn_few(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Params p) {
  using L = Layout<D, kF8>;
  constexpr int kStages = L::kStages, kTile = L::kTile;
  constexpr int kKeyGroups = 4 / MT, kSteps = kTile / 16 / kKeyGroups;     // 16-key steps of a warp in a tile
  constexpr bool kTwoParts = !kF8 && MT == 1;                    // of bf16 weights
  extern __shared__ uint8_t smem_raw[];
  Smem<D, kF8>& sm = *reinterpret_cast<Smem<D, kF8>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  FewWalk<kTile> wk;
  if (!set_up<D, kF8>(sm, p, wk)) return;
  if (warp == 4) {
    produce<D, kF8, (kKeyGroups > 1), (MT > 1)>(sm, kmap, vmap, p, wk);
  } else {
    // =============================== consumers ===============================
    const int rt = warp % MT, kg = warp / MT;                 // row tile, key group
    const int g = lane >> 2, q4 = lane & 3;
    int ring = 0;                                               // stages used so far
    do {
      if (wk.t_begin >= wk.t_end) continue;
      const Item& it = wk.it;
      const int b = wk.b, h = wk.h, t_begin = wk.t_begin, t_end = wk.t_end;
      const int rows = it.s.n * a.group;
      // my two rows: r0 = 16 rt + g and r0 + 8; queries straight into the A fragments
      const int r0 = rt * 16 + g;
      uint32_t qa[D / 16][4];
      float rs[2] = {a.scale_log2, a.scale_log2};             // raw score -> base-2 logit
      int first[2], last[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + 8 * e;
        first[e] = last[e] = 0;
        const char* src = nullptr;
        if (r < rows) {
          const int i = token_of(a, r), hh = h * a.group + r - i * a.group;
          visible(a, it.s.len, it.s.len - it.s.n + i, &first[e], &last[e]);
          src = a.q.data + b * a.q.seq + (long long)(it.s.row0 + i) * a.q.row + (long long)hh * a.q.head;
        }
        if constexpr (kF8) {
          // K fragments hold codes 4 q4 ... 4 q4 + 3 of a 16-code chunk as their k positions 2 q4, 2 q4 + 1 and +8
          uint2 w[D / 16];
          uint32_t m = 0;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            w[c] = src ? *reinterpret_cast<const uint2*>(src + c * 32 + q4 * 8) : make_uint2(0, 0);
            m = max(m, max(max((w[c].x << 16) & 0x7fff0000u, w[c].x & 0x7fff0000u),
                           max((w[c].y << 16) & 0x7fff0000u, w[c].y & 0x7fff0000u)));
          }
          m = max(m, __shfl_xor_sync(FULL, m, 1));
          m = max(m, __shfl_xor_sync(FULL, m, 2));
          // largest magnitude to [2^14, 2^15): every bf16 down to 2^-31 of it is an fp16 number
          const int eq = max(-100, min(112, (int)(m >> 23) - 127 - 14));
          const float s = pow2(-eq);
          rs[e] *= pow2(eq);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            qa[c][e] = pack_f16x2(__uint_as_float(w[c].x << 16) * s, __uint_as_float(w[c].x & 0xffff0000u) * s);
            qa[c][2 + e] = pack_f16x2(__uint_as_float(w[c].y << 16) * s, __uint_as_float(w[c].y & 0xffff0000u) * s);
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            qa[c][e] = src ? *reinterpret_cast<const uint32_t*>(src + c * 32 + q4 * 4) : 0u;
            qa[c][2 + e] = src ? *reinterpret_cast<const uint32_t*>(src + c * 32 + 16 + q4 * 4) : 0u;
          }
        }
      }
      // keys that all of the warp's rows see: only those tiles need no masks
      int all_first = r0 < rows ? first[0] : 0, all_last = r0 < rows ? last[0] : 0x7fffffff;
      if (r0 + 8 < rows) {
        all_first = max(all_first, first[1]);
        all_last = min(all_last, last[1]);
      }
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        all_first = max(all_first, __shfl_xor_sync(FULL, all_first, d));
        all_last = min(all_last, __shfl_xor_sync(FULL, all_last, d));
      }
      all_last = min(all_last, it.s.len);
      float acc[D / 8][4];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

      for (int t = t_begin; t < t_end; ++t, ++ring) {
        const int st = ring % kStages;
        const bool landed = wait(sm, &sm.full[st], (ring / kStages) & 1, p);
        const uint32_t kb = smem_u32(sm.k[st]), vb = smem_u32(sm.v[st]);
        // 16 keys from k0 on; edge: some row does not see some of them
        const auto keys16 = [&](auto edge_tag, const int k0) {
          constexpr bool edge = decltype(edge_tag)::value;
          const int j0 = t * kTile + k0;
          const unsigned bad16 = (unsigned)(sm.bad[st][k0 >> 6] >> (k0 & 63)) & 0xffffu;
          // ---- scores of 16 rows x 16 keys ----
          float s[2][4] = {};
          if (kF8) {
#pragma unroll
            for (int c = 0; c < D / 16; c += 2) {
              uint32_t x[4];
              ldsm4(kb + chunk_at<D, true>(k0 + ((lane >> 3) & 1) * 8 + (lane & 7), c + (lane >> 4)), x);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                mma16816<true>(s[0], qa[c + e], e4m3x2_to_f16x2((uint16_t)x[2 * e]), e4m3x2_to_f16x2((uint16_t)(x[2 * e] >> 16)));
                mma16816<true>(s[1], qa[c + e], e4m3x2_to_f16x2((uint16_t)x[2 * e + 1]), e4m3x2_to_f16x2((uint16_t)(x[2 * e + 1] >> 16)));
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t x[4];
              ldsm4(kb + chunk_at<D, false>(k0 + (lane >> 4) * 8 + (lane & 7), 2 * c + ((lane >> 3) & 1)), x);
              mma16816<false>(s[0], qa[c], x[0], x[1]);
              mma16816<false>(s[1], qa[c], x[2], x[3]);
            }
          }
          // ---- base-2 logits; my keys are 8 n + 2 q4 + {0, 1} ----
          float inv[2][2];                                    // e4m3: 2^-e of my keys' values
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (kF8) {
              const int at = k0 + 8 * n + 2 * q4;
              const uint32_t ke = *reinterpret_cast<const uint16_t*>(&sm.ke[st][at]);
              const uint32_t ve = *reinterpret_cast<const uint16_t*>(&sm.ve[st][at]);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t kx = (ke >> (8 * x)) & 0xffu, vx = (ve >> (8 * x)) & 0xffu;
                const float ks = __uint_as_float(kx << 23), ef = (float)((int)vx - kExpBias);
                inv[n][x] = __uint_as_float((254u - vx) << 23);
                s[n][x] = fmaf(s[n][x] * ks, rs[0], ef);
                s[n][2 + x] = fmaf(s[n][2 + x] * ks, rs[1], ef);
              }
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x) s[n][x] *= a.scale_log2;
            }
          }
          unsigned seen = 0xffu;                              // bit 4 n + x
          if (edge) {
            seen = 0;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int kk = 8 * n + 2 * q4 + (x & 1), j = j0 + kk;
                if (j >= first[x >> 1] && j < last[x >> 1] && !((bad16 >> kk) & 1u)) seen |= 1u << (4 * n + x);
                else s[n][x] = -INFINITY;
              }
          }
          // ---- running maximum: moved only when a row outgrows it by 2^8, or (bf16 in one part) twice what the lane has of it ----
          float lag[2] = {kLazyLog2, kLazyLog2};
          if constexpr (!kF8 && !kTwoParts) {
#pragma unroll
            for (int e = 0; e < 2; ++e) lag[e] = fminf(kLazyLog2, fmaxf(0.f, 1.f + __log2f(l[e])));
          }
          const float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
          const float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
          if (__any_sync(FULL, x0 > m[0] + lag[0] || x1 > m[1] + lag[1])) {
            float mx[2] = {x0, x1}, f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mx[e] = fmaxf(mx[e], __shfl_xor_sync(FULL, mx[e], 1));
              mx[e] = fmaxf(mx[e], __shfl_xor_sync(FULL, mx[e], 2));
              const float mn = fmaxf(m[e], mx[e]);
              f[e] = mn == -INFINITY ? 1.f : ex2(m[e] - mn);
              m[e] = mn;
              l[e] *= f[e];
            }
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              acc[c][0] *= f[0];
              acc[c][1] *= f[0];
              acc[c][2] *= f[1];
              acc[c][3] *= f[1];
            }
          }
          const float mb[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
          float w[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              w[n][x] = ex2(s[n][x] - mb[x >> 1]);
              if (kF8) {
                if (!edge || ((seen >> (4 * n + x)) & 1u)) l[x >> 1] = fmaf(w[n][x], inv[n][x & 1], l[x >> 1]);
              } else {
                l[x >> 1] += w[n][x];
              }
            }
          [[maybe_unused]] uint32_t pa[4], pl[4];             // pl: bf16 weights' second parts
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = 2 * n + e;
              if constexpr (kTwoParts) split_bf16x2(w[n][2 * e], w[n][2 * e + 1], pa[i], pl[i]);
              else pa[i] = kF8 ? pack_f16x2(w[n][2 * e], w[n][2 * e + 1]) : pack_bf16x2(w[n][2 * e], w[n][2 * e + 1]);
            }
          // ---- O += P V ----
          uint32_t keep[2] = {FULL, FULL};                    // edge: my V rows (keys 2 q4, +1, and +8) that exist
          if (edge) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              keep[n] = 0;
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int kk = 8 * n + 2 * q4 + x;
                if (j0 + kk < it.s.len && !((bad16 >> kk) & 1u)) keep[n] |= 0xffffu << (16 * x);
              }
            }
          }
          constexpr uint32_t kInf = kF8 ? 0x7c007c00u : 0x7f807f80u;
          bool odd = false;                                   // a value that is not finite where not all rows see it
          const auto clean = [&](uint32_t x, int n) -> uint32_t {
            if (!edge) return x;
            x &= keep[n];
            const bool lo = (x & kInf & 0xffffu) == (kInf & 0xffffu), hi = (x & kInf & 0xffff0000u) == (kInf & 0xffff0000u);
            odd = odd || lo || hi;
            if (lo) x &= 0xffff0000u;
            if (hi) x &= 0x0000ffffu;
            return x;
          };
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t x[4];
            if constexpr (kF8) {
              if (c & 1) continue;
              ldsm4t(vb + chunk_at<D, true>(k0 + ((lane >> 3) & 1) * 8 + (lane & 7), c + (lane >> 4)), x);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // bytes (key, d), (key, d + 1), (key + 1, d), (key + 1, d + 1) -> pairs of keys for d and for d + 1
                const uint32_t lo = __byte_perm(x[2 * e], 0, 0x3120), hi = __byte_perm(x[2 * e + 1], 0, 0x3120);
                mma16816<true>(acc[2 * (c + e)], pa, clean(e4m3x2_to_f16x2((uint16_t)lo), 0), clean(e4m3x2_to_f16x2((uint16_t)hi), 1));
                mma16816<true>(acc[2 * (c + e) + 1], pa, clean(e4m3x2_to_f16x2((uint16_t)(lo >> 16)), 0),
                               clean(e4m3x2_to_f16x2((uint16_t)(hi >> 16)), 1));
              }
            } else {
              ldsm4t(vb + chunk_at<D, false>(k0 + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * c + (lane >> 4)), x);
              if constexpr (kTwoParts) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint32_t v0 = clean(x[2 * y], 0), v1 = clean(x[2 * y + 1], 1);
                  mma16816<false>(acc[2 * c + y], pa, v0, v1);
                  mma16816<false>(acc[2 * c + y], pl, v0, v1);
                }
              } else {
                mma16816<false>(acc[2 * c], pa, clean(x[0], 0), clean(x[1], 1));
                mma16816<false>(acc[2 * c + 1], pa, clean(x[2], 0), clean(x[3], 1));
              }
            }
          }
          if (edge && __any_sync(FULL, odd)) {
            // rare: add what was taken out, to the rows that see it
#pragma unroll 1
            for (int kk = 0; kk < 16; ++kk) {
              if (j0 + kk >= it.s.len || ((bad16 >> kk) & 1u)) continue;
              const int src = (lane & ~3) | ((kk & 7) >> 1);
              const int n = kk >> 3, x = kk & 1;
              float wk[2];
              bool sk[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float mine_w = n ? (x ? w[1][2 * e + 1] : w[1][2 * e]) : (x ? w[0][2 * e + 1] : w[0][2 * e]);
                wk[e] = __shfl_sync(FULL, mine_w, src);
                sk[e] = (__shfl_sync(FULL, seen, src) >> (4 * n + 2 * e + x)) & 1u;
              }
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int col = kF8 ? 16 * (c >> 1) + 4 * q4 + 2 * y + (c & 1) : 8 * c + 2 * q4 + y;
                  const float val = value_at<D, kF8>(sm.v[st], k0 + kk, col);
                  if (isfinite(val)) continue;
                  if (sk[0]) acc[c][y] = fmaf(wk[0], val, acc[c][y]);
                  if (sk[1]) acc[c][2 + y] = fmaf(wk[1], val, acc[c][2 + y]);
                }
            }
          }
        };
#pragma unroll 1
        for (int step = 0; step < kSteps; ++step) {
          const int k0 = (kg * kSteps + step) * 16, j0 = t * kTile + k0;
          if (j0 < all_first || j0 + 16 > all_last || ((sm.bad[st][k0 >> 6] >> (k0 & 63)) & 0xffffu)) keys16(std::true_type(), k0);
          else keys16(std::false_type(), k0);
        }
        __syncwarp();
        if (lane == 0 && (MT > 1 || landed)) mbar_arrive(&sm.empty[st]);
      }
      // ---- the row sums of the four lanes of a row, then the key groups ----
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(FULL, l[e], 1);
        l[e] += __shfl_xor_sync(FULL, l[e], 2);
      }
      if (kKeyGroups > 1) {
        const int st = ring % kStages;
        const bool landed = wait(sm, &sm.full[st], (ring / kStages) & 1, p);
        // one side of the stage takes the O of one warp, element by element a lane; at most two give at a time
        static_assert(L::kSide >= 16 * D * 4, "");
#pragma unroll
        for (int from = kKeyGroups / 2; from > 0; from >>= 1) {
          const int pair = (kg % from) * MT + rt;              // groups [from, 2 from) give theirs to [0, from)
          float* buf = reinterpret_cast<float*>(pair ? sm.v[st] : sm.k[st]) + lane;
          if (kg >= from && kg < 2 * from) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
#pragma unroll
              for (int x = 0; x < 4; ++x) buf[(4 * c + x) * 32] = acc[c][x];
            if (q4 == 0) {
              sm.ml[pair][g] = make_float2(m[0], l[0]);
              sm.ml[pair][g + 8] = make_float2(m[1], l[1]);
            }
          }
          consumer_sync();
          if (kg < from) {
            float f[2], fo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 o = sm.ml[pair][g + 8 * e];
              const float mn = fmaxf(m[e], o.x), base = mn == -INFINITY ? 0.f : mn;
              f[e] = ex2(m[e] - base);
              fo[e] = ex2(o.x - base);
              m[e] = mn;
              l[e] = l[e] * f[e] + o.y * fo[e];
            }
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
#pragma unroll
              for (int x = 0; x < 4; ++x) acc[c][x] = acc[c][x] * f[x >> 1] + buf[(4 * c + x) * 32] * fo[x >> 1];
          }
          consumer_sync();
        }
        fence_async_shared();                                  // the stage goes back to TMA
        __syncwarp();
        if (lane == 0 && (MT > 1 || landed)) mbar_arrive(&sm.empty[st]);
        ++ring;
      }

      // ---- the rows' results: complete, or a part of an item that other blocks work on too ----
      const int c0 = wk.first_block(), c1 = wk.last_block();
      if (kg == 0) {
        const size_t part = wk.part();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + 8 * e;
          if (r >= rows) continue;
          if (c0 == c1) {
            const int i = token_of(a, r), hh = h * a.group + r - i * a.group;
            char* dst = a.o.data + b * a.o.seq + (long long)(it.s.row0 + i) * a.o.row + (long long)hh * a.o.head;
            const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const float x = acc[c][2 * e] * inv, y = acc[c][2 * e + 1] * inv;
              if constexpr (kF8) {
                if (c & 1) continue;
                const float x1 = acc[c + 1][2 * e] * inv, y1 = acc[c + 1][2 * e + 1] * inv;
                *reinterpret_cast<uint2*>(dst + (8 * c + 4 * q4) * 2) = make_uint2(pack_bf16x2(x, x1), pack_bf16x2(y, y1));
              } else {
                *reinterpret_cast<uint32_t*>(dst + (8 * c + 2 * q4) * 2) = pack_bf16x2(x, y);
              }
            }
            float* lse = lse_at(a, b, it.s, i, hh);
            if (lse && q4 == 0) *lse = l[e] == 0.f ? -INFINITY : (m[e] + log2f(l[e])) * 0.6931471805599453f;
          } else {
            float* dst = p.part_o + (part + r) * D;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              if constexpr (kF8) {
                if (c & 1) continue;
                *reinterpret_cast<float4*>(dst + 8 * c + 4 * q4) =
                    make_float4(acc[c][2 * e], acc[c + 1][2 * e], acc[c][2 * e + 1], acc[c + 1][2 * e + 1]);
              } else {
                *reinterpret_cast<float2*>(dst + 8 * c + 2 * q4) = make_float2(acc[c][2 * e], acc[c][2 * e + 1]);
              }
            }
            if (q4 == 0) p.part_ml[part + r] = make_float2(m[e], l[e]);
          }
        }
      }
      if (c0 != c1 && ends_last(sm, p, c0, c1)) join_parts<D>(sm, p, it, b, h, c0, c1);
    } while (wk.next(a));
  }
}

// MT row tiles of 16; 0: at most 8 rows
template <int D, bool kF8, int MT>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& vm, const Params& p, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(Smem<D, kF8>) + 1024;
  const auto kernel = [] {
    if constexpr (MT == 0) return attn_row8<D, kF8>;
    else return attn_few<D, kF8, MT>;
  }();
  if ((e = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem))) return e;
  // no more blocks than there can be places
  constexpr int kTile = Layout<D, kF8>::kTile;
  const long long items = (long long)p.a.seqs.batch * p.a.pool.kv_heads, tiles = ((long long)p.a.seqs.max_len + kTile - 1) / kTile;
  const long long places = tiles <= kWholeTiles && items <= kWholeItems ? items : items * (tiles + 1 + p.item_cost);
  const int blocks = (int)min((long long)min(2 * sms, kMaxFewBlocks), places);
  return launch_after(kernel, dim3(blocks), kThreads, smem, st, km, vm, p);
}

template <int D, bool kF8>
cudaError_t launch_rows(const CUtensorMap& km, const CUtensorMap& vm, const Params& p, cudaStream_t st) {
  const long long rows = (long long)p.a.seqs.max_new * p.a.group;
  if (rows <= 8) return launch<D, kF8, 0>(km, vm, p, st);
  if (rows <= 16) return launch<D, kF8, 1>(km, vm, p, st);
  if (rows <= 32) return launch<D, kF8, 2>(km, vm, p, st);
  return launch<D, kF8, 4>(km, vm, p, st);
}

}  // namespace

cudaError_t launch_attention_few(const AttnArgs& a, int d, void* ws, unsigned long long wait_ns, int fault, cudaStream_t st) {
  CUtensorMap km, vm;
  const uint64_t rows = (uint64_t)a.pool.num_pages * a.pool.kv_heads * a.pool.page;
  const int esz = a.pool.dtype == PISA_CACHE_E4M3 ? 1 : 2;
  const int tile = esz == 1 ? 128 : 64;
  const uint32_t box = a.pool.page < tile ? a.pool.page : tile;
  if (!encode_rows(&km, a.pool.k, esz, d, rows, box) || !encode_rows(&vm, a.pool.v, esz, d, rows, box))
    return cudaErrorInvalidValue;
  Params p;
  p.a = a;
  char* w = static_cast<char*>(ws);
  p.counters = reinterpret_cast<int*>(w + kCountersAt);
  p.part_ml = reinterpret_cast<float2*>(w + kPartialsAt);
  p.part_o = reinterpret_cast<float*>(w + kPartialsAt + sizeof(float2) * 2 * kMaxFewBlocks * kMaxFewRows);
  // What an item costs besides its tiles (queries, the warps' join, output), in tiles: without it the blocks with
  // many short sequences end last (64 sequences x 24 heads of up to 4608 tokens, e4m3: 186 us with 1, 155 with 4).
  p.item_cost = esz == 1 ? 4 : 3;
  p.wait_ns = wait_ns;
  p.fault = fault;
  if (esz == 1) return d == 64 ? launch_rows<64, true>(km, vm, p, st) : launch_rows<128, true>(km, vm, p, st);
  return d == 64 ? launch_rows<64, false>(km, vm, p, st) : launch_rows<128, false>(km, vm, p, st);
}

}  // namespace cache
}  // namespace pisa
