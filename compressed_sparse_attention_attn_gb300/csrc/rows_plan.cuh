// rows_plan.cuh -- the plan of an attention of many rows (k_rows_attn.cu): its items and the CTAs' parts of them.  One CTA makes it: of
// k_paged_attn's, where that runs before k_rows_attn (the rows' own pages, requests of one token), else of a launch of its own.
#pragma once

#include "paged_common.cuh"

namespace csa {
namespace rows {

constexpr int kSub = 128;      // rows of a product
constexpr int kMinPlaces = 2;  // places a CTA has at least

// Rows row0 .. row0 + rows - 1 of the segment whose first token is tok0; positions begin .. end - 1 behind table row seg are all that
// any of them attends.  Token t of a prompt stands at t + shift; of a prefix shift is its length.
// end0, begin1: of its first 128 rows, of the others.  at0 .. at1: positions that every row attends (with a window in a prefix: none).
struct Item {
  int tok0, row0, rows, seg, begin, end, shift, end0, begin1, at0, at1, spare;
};
// A CTA's part of the places (a kv head's items one behind the other, head after head): first .. end - 1, of which the first is in item
// `item` of head kvh; `items` of a head, `places` of a head.  No places: first == end.
struct Part {
  unsigned long long first, end, places, start;  // start: first place of the item
  int item, kvh, items, spare;
  Item d;
};

struct Plan {
  RowsAttnArgs a;
  paged::FastDiv page, g;
  int rows_log2, tile_log2;    // an item has up to 2^rows_log2 rows, a tile 2^tile_log2 positions
  int end_tiles;
  Part *part;                  // [ctas + 1] (of the last one: first)
  int ctas;
  Item *item;                  // [cap]
  unsigned long long *start;   // [cap + 1]: first place of an item
  int cap;
  bool single;                 // prompts: segments of one token are k_paged_attn's
};

// Inclusive over the CTA's threads; sum: of all.
template <int NT>
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long *warp_sum, unsigned long long &sum) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) warp_sum[wid] = v;
  __syncthreads();
  unsigned long long w = lane < NT / 32 ? warp_sum[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  sum = __shfl_sync(0xffffffffu, w, 31);
  const unsigned long long before = __shfl_sync(0xffffffffu, w, wid > 0 ? wid - 1 : 0);
  return v + (wid > 0 ? before : 0);
}

// Shared memory of the CTA that makes the plan.
constexpr int kStartsKept = 2048;
template <int NT>
struct PlanRoom {
  int4 seg[NT];  // first token, tokens, length, items up to and with this segment's
  unsigned long long sum[32];
  unsigned long long start[kStartsKept];  // first places of the first items
};

// By all NT threads of a CTA, behind the wait for what came before.  (What is run once costs its fetches: a thread with four segments,
// items and parts at a time, unrolled, took 18.5 us where this takes 6.)
template <int NT>
__device__ __forceinline__ void make_plan(const Plan P, PlanRoom<NT> &room) {
  const RowsAttnArgs &a = P.a;
  const int tid = threadIdx.x, RL = P.rows_log2, KL = P.tile_log2;
  const int64_t cap = min((int64_t)a.width * a.c.page, (int64_t)0x7fffffff);
  unsigned long long places = 0;
  int items = 0;
  bool full = false;
#pragma unroll 1
  for (int s0 = 0; s0 < a.S; s0 += NT) {
    const int s = s0 + tid, segs = min(NT, a.S - s0);
    int t0 = 0, n = 0, len = 0;
    if (s < a.S) {
      int t1 = a.N;
      if (a.cu) t0 = a.cu[s], t1 = a.cu[s + 1];
      len = a.len[s];
      bool bad = t0 < 0 || t1 < t0 || t1 > a.N;
      n = bad ? 0 : t1 - t0;
      if (n > 0) {
        if (len < 0 || len > cap) bad = true;
        if (a.pos == nullptr && len < n) {
          bad = true;
          n = 0;
        }
        if (a.pos) len = max(len, 0);
      }
      if (bad) atomicOr(a.status, kStatusBadIndex);
      if (n == 1 && P.single) n = 0;
    }
    unsigned long long sum;
    const unsigned long long tiles = ((unsigned long long)n * P.g.d + (1 << RL) - 1) >> RL, to = block_scan<NT>(tiles, room.sum, sum);
    room.seg[tid] = make_int4(t0, n, len, (int)min(to, 0x7fffffffull));
    __syncthreads();
    const int left = P.cap - items, all = (int)min(sum, (unsigned long long)left);
    full = full || sum > (unsigned long long)left;
#pragma unroll 1
    for (int i0 = 0; i0 < all; i0 += NT) {
      const int i = i0 + tid;
      unsigned long long mine = 0;
      if (i < all) {
        int lo = 0, hi = segs - 1;  // the first segment with more than i items up to its end
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (room.seg[mid].w > i) hi = mid;
          else lo = mid + 1;
        }
        const int4 sg = room.seg[lo];
        const int first = lo ? room.seg[lo - 1].w : 0;
        Item it{};
        it.tok0 = sg.x;
        it.row0 = (i - first) << RL;
        it.rows = (int)min(1ll << RL, (long long)sg.y * P.g.d - it.row0);
        it.seg = s0 + lo;
        if (a.pos) {  // (a row's own part begins at len or behind it: the window reaches back to len - window at most)
          it.shift = sg.z;
          it.begin = it.begin1 = a.window > 0 ? max(0, sg.z - a.window) : 0;
          it.end = it.end0 = (int)min((int64_t)sg.z, cap);
          it.at0 = 0;
          it.at1 = a.window > 0 ? 0 : it.end;
        } else {
          it.shift = sg.z - sg.x - sg.y;
          auto pos = [&](int r) { return (int64_t)sg.x + P.g.div(it.row0 + min(r, it.rows - 1)) + it.shift; };  // of a row
          auto first = [&](int64_t p) { return (int)(a.window > 0 ? max((int64_t)0, p - a.window + 1) : 0); };
          it.begin = first(pos(0));
          it.begin1 = first(pos(kSub));
          it.end0 = (int)min(pos(kSub - 1) + 1, cap);
          it.end = (int)min(pos(it.rows - 1) + 1, cap);
          it.at0 = first(pos(it.rows - 1));
          it.at1 = (int)min(pos(0) + 1, cap);
        }
        mine = (it.end > it.begin ? ((it.end - 1) >> KL) - (it.begin >> KL) + 1 : 1) + P.end_tiles;
        reinterpret_cast<int4 *>(P.item + items + i)[0] = make_int4(it.tok0, it.row0, it.rows, it.seg);
        reinterpret_cast<int4 *>(P.item + items + i)[1] = make_int4(it.begin, it.end, it.shift, it.end0);
        reinterpret_cast<int4 *>(P.item + items + i)[2] = make_int4(it.begin1, it.at0, it.at1, 0);
      }
      const unsigned long long at = places + block_scan<NT>(mine, room.sum, sum) - mine;
      if (i < all) {
        P.start[items + i] = at;
        if (items + i < kStartsKept) room.start[items + i] = at;
      }
      places += sum;
    }
    items += all;
    __syncthreads();
  }
  if (tid == 0) {
    P.start[items] = places;
    if (full) atomicOr(a.status, kStatusBadIndex);  // (more items than rows can make: requests that overlap)
  }
  __syncthreads();
  const unsigned long long total = places * a.c.kv_heads;
  const int parts = (int)min((unsigned long long)P.ctas, max(1ull, total / kMinPlaces));
  const unsigned long long each = total / parts, more = total % parts;
  const unsigned long long *starts = items <= kStartsKept ? room.start : P.start;
#pragma unroll 1
  for (int c = tid; c <= P.ctas; c += NT) {
    const int n = min(c, parts);
    Part q{};
    q.first = each * n + more * n / parts;
    q.places = places;
    q.items = items;
    q.end = c < parts ? each * (n + 1) + more * (n + 1) / parts : q.first;
    if (q.first < q.end) {
      q.kvh = (int)(q.first / places);
      const unsigned long long in = q.first - places * q.kvh;
      int lo = 0, hi = items - 1;  // the last item that begins at `in` or before
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= in) lo = mid;
        else hi = mid - 1;
      }
      q.item = lo;
      q.start = starts[lo];
      q.d = P.item[lo];
    }
    P.part[c] = q;
  }
}

}  // namespace rows
}  // namespace csa
