// How attention over the cache is shared out among the blocks of a launch.
//
// An item is up to 2^log_rows rows of one sequence and key/value head (rows: its new tokens times the group
// of query heads, token by token), with the keys that any of them sees in tiles of kKeys.  All items
// form one line, sequence by sequence, head by head; in it an item takes a place for each of its tiles
// and then item_cost places for what it costs besides them.  The line is cut into equal shares, one a
// block, so a block works on the end of one item, whole items, and the beginning of another, whatever
// the lengths.  Everything is computed on the device, from the lengths there.
#pragma once

#include "cache.cuh"

namespace pisa {
namespace cache {

// a / b for a >= 0 and b > 0, by 32 bits where they do.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 31) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

template <int kWarps>
struct WalkScratch {                  // in shared memory
  long long scan[kWarps], before;
  int b, h, p;
};

// Every role of a block walks its own copy.
template <int kKeys>
struct Walk {
  struct Item {
    int t0, n, rows, first;           // its tiles are [t0, t0 + n) of the sequence; first: the first key any row sees
    int places, cost;                 // places of its tiles, and with what it costs besides
  };
  int b, h, p, pieces, count;         // sequence, head, piece of its rows (of `pieces`); count: for the caller's use
  Seq s;
  Item it;
  long long item0, u0, u1, share;     // places: the item's first, this block's share, and how long shares are
  int t_begin, t_end, item_cost, log_rows;      // this block's tiles of the item: none where its share holds only the last places

  __device__ __forceinline__ int pieces_of(const AttnArgs& a, const Seq& s) const { return (s.n * a.group + (1 << log_rows) - 1) >> log_rows; }
  __device__ __forceinline__ int row0() const { return p << log_rows; }
  __device__ __forceinline__ Item item_of(const AttnArgs& a, const Seq& s, int p) const {
    Item it;
    it.rows = min(1 << log_rows, s.n * a.group - (p << log_rows));
    int f0, l0, f1, l1;
    const int pos = s.len - s.n;
    visible(a, s.len, pos + token_of(a, p << log_rows), &f0, &l0);
    visible(a, s.len, pos + token_of(a, (p << log_rows) + it.rows - 1), &f1, &l1);
    // rows that see nothing (before the cache's first position) leave the range to the others
    const int first = l0 > f0 ? f0 : 0, last = max(l0, l1);
    it.first = first;
    it.t0 = first / kKeys;
    it.n = max(1, (last + kKeys - 1) / kKeys - it.t0);      // rows that see nothing are written too
    it.places = item_cost < 0 ? 1 : it.n;
    it.cost = item_cost < 0 ? 1 : it.places + item_cost;
    return it;
  }

  __device__ __forceinline__ void shares(long long total, int min_share) {
    share = max((long long)min_share, quotient(total + gridDim.x - 1, gridDim.x));
    u0 = share * blockIdx.x;
    u1 = min(total, u0 + share);
  }

  // Whole block of kThreads; false if the line ends before this block's share.  cost_of_item < 0: items
  // are not cut, each takes one place (for calls with no more of them than blocks).
  template <int kThreads, typename Scratch>
  __device__ __forceinline__ bool start(const AttnArgs& a, Scratch& sc, int log2_rows, int cost_of_item, int min_share) {
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    item_cost = cost_of_item;
    log_rows = log2_rows;
    count = 0;
    // the piece of head h that place u0 falls into, `at` places into the line at the head's first; a warp
    const auto find_piece = [&](const Seq& sq, long long at, int* piece, long long* before) {
      for (int i0 = 0;; i0 += 32) {
        const int n = i0 + lane < pieces_of(a, sq) ? item_of(a, sq, i0 + lane).cost : 0;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, at + upto > u0);
        if (hit || i0 + 32 >= pieces_of(a, sq)) {
          const int w = hit ? __ffs(hit) - 1 : 0;
          *piece = i0 + w;
          *before = at + __shfl_sync(0xffffffffu, upto - n, w);
          return;
        }
        at += __shfl_sync(0xffffffffu, upto, 31);
      }
    };
    if (a.seqs.batch <= 32) {         // each warp by itself, lane i for sequence i
      Seq mine;
      int cost = 0, np = 0;
      if (lane < a.seqs.batch && load_seq(a.seqs, lane, a.q.rows, &mine)) np = pieces_of(a, mine);
      else mine.n = mine.len = mine.row0 = 0;
      if (__any_sync(0xffffffffu, np > 4)) {
        for (int i = 0; i < a.seqs.batch; ++i) {              // lanes over a sequence's pieces
          Seq sq;
          sq.len = __shfl_sync(0xffffffffu, mine.len, i);
          sq.n = __shfl_sync(0xffffffffu, mine.n, i);
          int c = 0;
          for (int x = lane; x < pieces_of(a, sq); x += 32) c += item_of(a, sq, x).cost;
          c = __reduce_add_sync(0xffffffffu, c);
          if (lane == i) cost = c;
        }
      } else {
        for (int x = 0; x < np; ++x) cost += item_of(a, mine, x).cost;
      }
      const long long n = (long long)cost * a.pool.kv_heads;
      long long upto = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += up;
      }
      shares(__shfl_sync(0xffffffffu, upto, 31), min_share);
      if (u0 >= u1) return false;
      b = __ffs(__ballot_sync(0xffffffffu, upto > u0)) - 1;
      const long long at = __shfl_sync(0xffffffffu, upto - n, b);
      const int per = __shfl_sync(0xffffffffu, cost, b);
      s.len = __shfl_sync(0xffffffffu, mine.len, b);
      s.n = __shfl_sync(0xffffffffu, mine.n, b);
      s.row0 = __shfl_sync(0xffffffffu, mine.row0, b);
      pieces = pieces_of(a, s);
      h = (int)quotient(u0 - at, per);
      find_piece(s, at + (long long)h * per, &p, &item0);
      enter(a);
      return true;
    }
    // places of a sequence and head: a warp a sequence, lanes over its pieces
    const auto seq_cost = [&](int seq) -> long long {
      Seq sq;
      long long c = 0;
      if (seq < a.seqs.batch && load_seq(a.seqs, seq, a.q.rows, &sq))
        for (int i = lane; i < pieces_of(a, sq); i += 32) c += item_of(a, sq, i).cost;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
      return c;
    };
    long long mine = 0;
    for (int seq = warp; seq < a.seqs.batch; seq += kWarps) mine += seq_cost(seq);
    if (lane == 0) sc.scan[warp] = mine;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sc.scan[w];
    total *= a.pool.kv_heads;
    shares(total, min_share);
    if (u0 >= u1) return false;
    __syncthreads();                  // scan is used again
    long long base = 0;
    for (int b0 = 0; b0 < a.seqs.batch; b0 += kWarps) {
      const long long c = seq_cost(b0 + warp) * a.pool.kv_heads;
      if (lane == 0) sc.scan[warp] = c;
      __syncthreads();
      long long run = base;
      int found = -1;
      for (int w = 0; w < kWarps && found < 0; ++w) {
        if (u0 < run + sc.scan[w]) found = w;
        else run += sc.scan[w];
      }
      if (found >= 0) {
        if (warp == found) {          // the head, then the piece of rows, in it
          Seq sq;
          load_seq(a.seqs, b0 + warp, a.q.rows, &sq);
          const long long per = c / a.pool.kv_heads;
          const int head = (int)((u0 - run) / per);
          run += head * per;
          int piece;
          long long before;
          find_piece(sq, run, &piece, &before);
          if (lane == 0) {
            sc.b = b0 + warp;
            sc.h = head;
            sc.p = piece;
            sc.before = before;
          }
        }
        break;
      }
      base = run;
      __syncthreads();
    }
    __syncthreads();
    b = sc.b;
    h = sc.h;
    p = sc.p;
    item0 = sc.before;
    load_seq(a.seqs, b, a.q.rows, &s);
    pieces = pieces_of(a, s);
    enter(a);
    return true;
  }

  __device__ __forceinline__ void enter(const AttnArgs& a) {
    it = item_of(a, s, p);
    if (item_cost < 0) {
      t_begin = it.t0;
      t_end = it.t0 + it.n;
      return;
    }
    t_begin = it.t0 + (int)min((long long)it.n, max(0LL, u0 - item0));
    t_end = it.t0 + (int)min((long long)it.n, u1 - item0);
  }

  // The next item of this block, false at its share's end.
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    item0 += it.cost;
    if (item0 >= u1) return false;
    if (++p == pieces) {
      p = 0;
      if (++h == a.pool.kv_heads) {
        h = 0;
        do {
          if (!load_seq(a.seqs, ++b, a.q.rows, &s)) s.n = 0;
          pieces = pieces_of(a, s);
        } while (pieces == 0);        // the line goes on: there is one
      }
    }
    enter(a);
    return true;
  }

  // Blocks that work on the item; a block has at most two items that it shares: the one that began before its
  // share (part 2 * block) and the one that goes on after it (part 2 * block + 1).
  __device__ __forceinline__ int first_block() const { return (int)quotient(item0, share); }
  __device__ __forceinline__ int last_block() const { return (int)quotient(item0 + it.places - 1, share); }
  __device__ __forceinline__ bool began_before() const { return item0 < u0; }
  __device__ __forceinline__ int part() const { return 2 * blockIdx.x + (began_before() ? 0 : 1); }
};

}  // namespace cache
}  // namespace pisa
