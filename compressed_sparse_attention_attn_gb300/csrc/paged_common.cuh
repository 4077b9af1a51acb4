// paged_common.cuh -- what the paged-attention kernels share: how ragged rows are dealt over the CTAs, and how
// the shares of a row that several CTAs worked on are joined.
//
// A segment is the work of one (row, head group): its positions in units of U rows, at least one (an empty row
// writes zeros), and behind them W places in which nothing is read, for the time that its end takes.  The segments'
// places stand one behind the other (row, head group, place); of their total T each of G CTAs takes T / G in a
// row (the first T mod G CTAs one more), so every CTA has as much to do as any other whatever the lengths are, and at
// most the first and the last segment of its range are shared with others.  The host knows no lengths: every CTA
// sums the units itself.  (W 0 left the CTAs with the shortest rows 1.4 times the mean time over 48 rows of 0 to 9000.)
//
// A CTA's share of a segment is (M, L, O): its running maximum (base 2), sum of weights and weighted sum of
// values relative to M, in f32, in one of its two slots (0: a segment that began in an earlier CTA, 1: one
// that begins here).  Up to 256 features, twelve consecutive shares of a segment are a group.  The CTA that completes a
// group joins it (in the order of the shares, whoever is last); with more than one group the joined shares go
// to the group's first slot, and twelve groups are joined in the same way.  So a long row over 400 CTAs is joined
// in three steps, and nothing waits (in two, of 12 and of 38 shares, one row of 46000 took 20.0 against 17.4 us).  The
// counters return to zero.  Shares of latent rows, 128 KB each, are joined by a second kernel (k_paged_attn_tc.cu).
#pragma once

#include "csa_internal.cuh"
#include "tc_ptx.cuh"

namespace csa {
namespace paged {

constexpr int kJoin = 12;          // shares of a group
constexpr int kMaxCtas = 640;

// x / d for 0 <= x < 2^31 by a multiplication: m = ceil(2^(31+s) / d), s = ceil(log2 d); m d - 2^(31+s) < d <=
// 2^s, so the error x (m d - 2^(31+s)) / (d 2^(31+s)) stays below 1 / d (Granlund and Montgomery, 1994).
struct FastDiv {
  uint32_t d = 1, m = 0x80000000u;
  int s = 31;
  FastDiv() = default;
  explicit FastDiv(uint32_t d_) : d(d_) {
    int b = 0;
    while ((1ull << b) < d) ++b;
    s = 31 + b;
    m = (uint32_t)(((1ull << s) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t div(uint32_t x) const { return (uint32_t)(((uint64_t)x * m) >> s); }
};

struct Params {
  PagedAttnArgs a;
  FastDiv page;
  int g, sub, Hg;       // query heads a kv head, head groups a kv head, segments a row
  float scale_log2;     // softmax scale * log2(e)
  float *share_o;       // [2 G][heads of a group][padded head_dim]
  float *share_ml;      // [2 G][heads of a group][2]: M, L (latent rows: L of the weights as the product takes them)
  float *share_l;       // latent rows: [2 G][heads of a group], L of the weights as they were
  int *counters;        // [3][2][kMaxCtas]: for each step of joining, groups past a segment's first, first groups
  int2 *split;          // latent rows: of the segments that several CTAs shared, the first CTA and how many
  int ctas;             // CTAs launched
  int by_segment;       // `split` is by segment (no more of them than CTAs), else by first CTA
};

// The positions first + lead .. first + rows - 1 of row n; units of U rows from `first` on (0: a row that is left alone).
// ALIGN: `first` is a multiple of U (with a window it may lie before the first position that counts), else lead is 0.
struct Row {
  int req, first, lead, rows, units;
};
template <int U, bool ALIGN>
__device__ __forceinline__ Row row_of(const PagedAttnArgs &a, int n, bool report) {
  Row r;
  r.req = a.req ? a.req[n] : n;
  const int pos = a.pos[n];
  r.first = r.lead = r.rows = r.units = 0;
  if (r.req < 0 || pos < -1) return r;
  if (r.req >= a.R) {
    if (report) atomicOr(a.status, kStatusBadIndex);
    return r;
  }
  const int cap = (int)min((int64_t)a.width * a.c.page, (int64_t)0x7fffffff);
  int end;  // one past the last position
  if (pos >= cap) {
    if (report) atomicOr(a.status, kStatusBadIndex);
    end = cap;
  } else {
    end = pos + 1;
  }
  if (a.window > 0) r.first = max(0, pos - a.window + 1);
  r.rows = max(0, end - r.first);
  if (ALIGN && r.rows > 0) {
    r.lead = r.first % U;
    r.first -= r.lead;
    r.rows += r.lead;
  }
  r.units = r.rows > 0 ? (r.rows - 1) / U + 1 : 1;  // (rows may be 2^31 - 1: positions of the last unit pass 31 bits)
  return r;
}

// A CTA's range: the row, head group and unit it begins with and its units.  Places are counted in 31 bits: a call whose
// segments come to 2^31 or more of them (an empty row has 1 + W too) does nothing but report it.
struct Range {
  int row, hg, t;        // t may be behind the segment's units (then the next segment's first unit is meant)
  uint32_t base;         // first place of that segment
  uint32_t each, more;   // places a CTA; the first `more` CTAs have one more
  uint32_t u0, u1;       // units before its first place and before its end
  int c0, parts;         // parts > 0: all its units are of one segment, dealt over CTAs c0 .. c0 + parts - 1
  int n_units;
};
// The first rows of a CTA's range, kept in shared memory: the cursors read a new row there and not through two
// dependent loads from global memory.
constexpr int kRowsKept = 32;
struct Rows {
  int n0;
  Row row[kRowsKept];
  template <int U, bool ALIGN>
  __device__ __forceinline__ Row get(const PagedAttnArgs &a, int n) const {
    return (unsigned)(n - n0) < (unsigned)kRowsKept ? row[n - n0] : row_of<U, ALIGN>(a, n, false);
  }
};

// Where a thread is in its CTA's range: segment (row n, head group hg) of `units` units from place `base` on, unit t of it.
struct Cursor {
  int n, hg, t, units;
  uint32_t base;
};
template <int U, bool ALIGN, int W>
__device__ __forceinline__ void advance(const PagedAttnArgs &a, int Hg, const Rows &rows, Cursor &c) {
  if (++c.t < c.units) return;
  c.t = 0;
  c.base += c.units + W;
  if (++c.hg < Hg) return;
  c.hg = 0;
  do {
    if (++c.n >= a.N) return;  // (past the last unit: not used any more)
    c.units = rows.get<U, ALIGN>(a, c.n).units;
  } while (c.units == 0);
}

// Sums of units and of segments, held at 2^31 - 1 once they reach it.
struct Two {
  uint32_t units, segs;
};
__device__ __forceinline__ Two plus(Two a, Two b) { return {min(a.units + b.units, 0x7fffffffu), min(a.segs + b.segs, 0x7fffffffu)}; }
__device__ __forceinline__ Two warp_scan(Two v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Two o{__shfl_up_sync(0xffffffffu, v.units, d), __shfl_up_sync(0xffffffffu, v.segs, d)};
    if (lane >= d) v = plus(v, o);
  }
  return v;
}

// Called by all NT threads of the CTA.  scratch: Two [NT / 32], rows, out: all in shared memory.  Returns how many
// units the CTA has (-1: more than can be counted in all).  Up to 32 rows the first warp finds it alone, and the CTA meets
// once.  WHOLE: few segments (and rows) get whole CTAs, as many as ceil(its units / q) says, if such a q close to
// the even share exists: a CTA then has one segment's end and not two (32 latent rows of about 20 tiles: 20.9
// against 22.6 us, 128 shares of 128 KB instead of 184; up to 256 features, where ends are cheap, one row of 8000 lost 1 us).
template <int U, int NT, bool ALIGN, int W, bool WHOLE>
__device__ __forceinline__ int find_range(const Params &P, Two *scratch, Rows &rows, Range &out) {
  const PagedAttnArgs &a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t Hg = (uint32_t)P.Hg, G = gridDim.x;
  const bool report = blockIdx.x == 0;
  auto of_row = [&](int n, Row &r) -> Two {
    r = Row{0, 0, 0, 0, 0};
    if (n < a.N) r = row_of<U, ALIGN>(a, n, report);
    return {(uint32_t)r.units, r.units > 0 ? 1u : 0u};
  };
  auto places = [&](Two v) -> int64_t { return ((int64_t)v.units + (int64_t)W * v.segs) * Hg; };
  // no more CTAs than there are places, so that none between two has none
  uint32_t begin = 0, end = 0;
  auto shares = [&](Two sum, bool tell) -> int {  // this CTA's places; 0: it has some
    const int64_t all = places(sum);
    if (all > 0x7fffffff) {
      if (report && tell) atomicOr(a.status, kStatusBadIndex);
      return -1;
    }
    const uint32_t total = (uint32_t)all, ctas = min(G, total);
    if (blockIdx.x >= ctas) return 1;
    const uint32_t each = total / ctas, more = total - each * ctas;
    begin = each * blockIdx.x + min(blockIdx.x, more);
    end = begin + each + (blockIdx.x < more ? 1 : 0);
    if (tell) {
      out.each = each;
      out.more = more;
      out.parts = 0;
    }
    return 0;
  };
  auto look = [&](Two from, uint32_t u, int n) -> bool {  // at row n of u units a segment; whether the range begins there
    const uint32_t lo = (uint32_t)places(from), hi = lo + (u ? (u + W) * Hg : 0u), before = from.units * Hg;
    if (end > lo && end <= hi) {
      const uint32_t in = end - lo, hg = in / (u + W), t = in - hg * (u + W);
      out.u1 = before + hg * u + min(t, u);
    }
    if (begin < lo || begin >= hi) return false;
    const uint32_t in = begin - lo, hg = in / (u + W), t = in - hg * (u + W);
    out.row = n;
    out.hg = (int)hg;
    out.t = (int)t;
    out.base = begin - t;
    out.u0 = before + hg * u + min(t, u);
    return true;
  };

  if (a.N <= 32) {
    if (wid == 0) {
      Row row;
      const Two mine = of_row(lane, row), incl = warp_scan(mine, lane);
      const Two sum{__shfl_sync(0xffffffffu, incl.units, 31), __shfl_sync(0xffffffffu, incl.segs, 31)};
      const int none = shares(sum, lane == 0);
      __syncwarp();  // (out.parts may be written again)
      bool here = false, whole = WHOLE && none >= 0 && sum.segs > 0 && sum.segs * Hg <= G;
      if (whole) {
        const uint32_t u = mine.units, q = (sum.units * Hg + G - 1) / G;
        const Two c{(u + q - 1) / q, (u + q) / (q + 1)}, to = warp_scan(c, lane);
        const bool first = __shfl_sync(0xffffffffu, to.units, 31) * Hg <= G;
        whole = first || __shfl_sync(0xffffffffu, to.segs, 31) * Hg <= G;
        const uint32_t n = first ? c.units : c.segs, in = blockIdx.x - ((first ? to.units : to.segs) - n) * Hg;
        if (whole && in < n * Hg) {  // (a CTA before the row's: wraps)
          const uint32_t hg = in / n, part = in - hg * n, one = u / n, rest = u - one * n;
          here = true;
          out.row = lane;
          out.hg = (int)hg;
          out.t = (int)(part * one + min(part, rest));
          out.base = out.u0 = 0;
          out.u1 = one + (part < rest ? 1 : 0);
          out.c0 = (int)(blockIdx.x - part);
          out.parts = (int)n;
        }
      }
      if (!whole && none == 0) here = look(Two{incl.units - mine.units, incl.segs - mine.segs}, mine.units, lane);
      const uint32_t who = __ballot_sync(0xffffffffu, here);
      const int first_row = __ffs(who) - 1;
      if (lane >= first_row) rows.row[lane - max(first_row, 0)] = row;
      __syncwarp();
      if (lane == 0) {
        rows.n0 = first_row;
        out.n_units = none < 0 ? -1 : who ? (int)(out.u1 - out.u0) : 0;
      }
    }
    __syncthreads();
    return out.n_units;
  }

  auto scan = [&](Two v, Two &sum) -> Two {  // inclusive over the CTA; sum: of all
    v = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) scratch[wid] = v;
    __syncthreads();
    sum = {0, 0};
    Two before{0, 0};
#pragma unroll 1
    for (int w = 0; w < NT / 32; ++w) {
      if (w == wid) before = sum;
      sum = plus(sum, scratch[w]);
    }
    return plus(v, before);
  };
  Two mine{0, 0}, sum;
  Row row;
  for (int n = tid; n < a.N; n += NT) mine = plus(mine, of_row(n, row));
  scan(mine, sum);
  const int none = shares(sum, tid == 0);
  if (none) return none < 0 ? -1 : 0;
  Two base{0, 0};
  for (int n0 = 0; n0 < a.N; n0 += NT) {
    mine = of_row(n0 + tid, row);
    const Two incl = plus(base, scan(mine, sum));
    look(Two{incl.units - mine.units, incl.segs - mine.segs}, mine.units, n0 + tid);
    base = plus(base, sum);
    if (end <= places(base)) break;
  }
  __syncthreads();
  if (tid == 0) rows.n0 = out.row;
  if (tid < kRowsKept) {
    of_row(out.row + tid, row);
    rows.row[tid] = row;
  }
  __syncthreads();
  return (int)(out.u1 - out.u0);
}
// The cursor at the first unit of a range that has one.
template <int U, bool ALIGN, int W>
__device__ __forceinline__ Cursor first_unit(const PagedAttnArgs &a, int Hg, const Range &r, const Rows &rows) {
  Cursor c;
  c.n = r.row;
  c.units = rows.row[0].units;
  c.hg = r.hg;
  c.base = r.base;
  c.t = r.t;
  if (c.t >= c.units) {  // (behind a segment's units)
    c.t = c.units - 1;
    advance<U, ALIGN, W>(a, Hg, rows, c);
  }
  return c;
}

// 2^x; results below the smallest normal number are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The CTA that place u belongs to.
__device__ __forceinline__ int cta_of(uint32_t u, const Range &r) {
  const uint32_t first = r.more * (r.each + 1);  // places of the CTAs with one more
  return (int)(u < first ? u / (r.each + 1) : r.more + (u - first) / r.each);
}

// The CTAs that share the cursor's segment: c0 .. c0 + (returned) - 1.
__device__ __forceinline__ int sharers(const Range &r, const Cursor &c, int &c0) {
  c0 = r.parts ? r.c0 : cta_of(c.base, r);
  return r.parts ? r.parts : cta_of(c.base + c.units - 1, r) - c0 + 1;
}

// One more arrival at a counter of `of` (by one thread, after a CTA barrier behind the writes it publishes);
// true for the last, which finds the others' writes.
__device__ __forceinline__ bool arrive_last(int *counter, int of) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  if (old != of - 1) return false;
  *counter = 0;
  return true;
}

// O of a row and head from its joined (M, L, O): the factor on O, with the sink in the denominator only.
__device__ __forceinline__ float out_factor(float M, float L, const float *sink, int h) {
  const float s2 = sink ? sink[h] * 1.4426950408889634f : -INFINITY;
  const float top = fmaxf(M, s2);
  const float em = M == -INFINITY ? 0.f : exp2f(M - top);
  const float st = s2 == -INFINITY ? 0.f : (s2 == INFINITY ? INFINITY : exp2f(s2 - top));
  const float below = L * em + st;
  return below == 0.f ? 0.f : em / below;
}

// Join `parts` shares, shares i of slots slot(i), of NH heads x HD features by the NT threads of the CTA.  fin: write O
// and lse of heads h0 .. h0+nh-1 of row n; else the joined share to slot `to` (one of the slots: a thread writes
// only what it alone has read, the maxima and sums behind a barrier).  A thread reads the maxima and sums of its
// head itself, with the values: one round trip a dozen shares, and no barrier.
template <int NH, int HD, int NT, class Slot>
__device__ __forceinline__ void join(const Params &P, int parts, Slot slot, bool fin, int to, int n, int h0, int nh) {
  const PagedAttnArgs &a = P.a;
  const int hd = a.c.head_dim;
  float M = -INFINITY, L = 0.f;
  constexpr int kRounds = (NH * (HD / 4) + NT - 1) / NT;
  float keep_m[kRounds], keep_l[kRounds];
#pragma unroll
  for (int rd = 0; rd < kRounds; ++rd) {
    const int i = threadIdx.x + rd * NT, h = i / (HD / 4), d = (i % (HD / 4)) * 4;
    keep_m[rd] = keep_l[rd] = 0.f;
    if (h >= nh || d >= hd) continue;
    M = -INFINITY;
    L = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += kJoin) {
      float2 ml[kJoin];
      float4 x[kJoin];
#pragma unroll
      for (int u = 0; u < kJoin; ++u) {
        ml[u] = make_float2(-INFINITY, 0.f);
        x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p0 + u < parts) {
          const int64_t at = (int64_t)slot(p0 + u) * NH + h;
          ml[u] = __ldcg(reinterpret_cast<const float2 *>(P.share_ml) + at);
          x[u] = __ldcg(reinterpret_cast<const float4 *>(P.share_o + at * HD + d));
        }
      }
      float top = M;
#pragma unroll
      for (int u = 0; u < kJoin; ++u) top = fmaxf(top, ml[u].x);
      const float ref = top == -INFINITY ? 0.f : top, f0 = ex2(M - ref);  // (2^-inf = 0)
      M = top;
      L *= f0;
      v.x *= f0;
      v.y *= f0;
      v.z *= f0;
      v.w *= f0;
#pragma unroll
      for (int u = 0; u < kJoin; ++u) {
        const float f = ex2(ml[u].x - ref);
        L = fmaf(ml[u].y, f, L);
        v.x = fmaf(x[u].x, f, v.x);
        v.y = fmaf(x[u].y, f, v.y);
        v.z = fmaf(x[u].z, f, v.z);
        v.w = fmaf(x[u].w, f, v.w);
      }
    }
    keep_m[rd] = M;
    keep_l[rd] = L;
    if (fin) {
      const float f = out_factor(M, L, a.sink, h0 + h);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * f, v.y * f), hi = __floats2bfloat162_rn(v.z * f, v.w * f);
      *reinterpret_cast<uint2 *>(a.o + (int64_t)n * a.o_t + (int64_t)(h0 + h) * hd + d) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
      if (a.lse && d == 0) a.lse[(int64_t)n * a.H + h0 + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    } else {
      *reinterpret_cast<float4 *>(P.share_o + ((int64_t)to * NH + h) * HD + d) = v;
    }
  }
  if (fin) return;
  __syncthreads();  // every thread has read the slots' maxima and sums
#pragma unroll
  for (int rd = 0; rd < kRounds; ++rd) {
    const int i = threadIdx.x + rd * NT, h = i / (HD / 4), d = (i % (HD / 4)) * 4;
    if (h < nh && d == 0)
      *reinterpret_cast<float2 *>(P.share_ml + ((int64_t)to * NH + h) * 2) = make_float2(keep_m[rd], keep_l[rd]);
  }
}

// Publish this CTA's share of the segment that CTAs c0 .. c0 + parts - 1 share (already written to its slot by the CTA's threads)
// and join what it completes: a dozen shares, a dozen of such groups, and so on.  flag: an int in shared memory.
template <int NH, int HD, int NT>
__device__ __forceinline__ void publish(const Params &P, int c0, int parts, int n, int h0, int nh, int *flag) {
  auto slot_of = [c0](int p) { return p == 0 ? 2 * c0 + 1 : 2 * (c0 + p); };
  int mine = (int)blockIdx.x - c0, step = 1;  // of `parts` joined shares, `step` CTAs apart
#pragma unroll 1
  for (int *counters = P.counters + c0;; counters += 2 * kMaxCtas) {
    const int first = mine / kJoin * kJoin, in_grp = min(kJoin, parts - first);
    __syncthreads();
    // (a segment's first group and another's later one may belong to one CTA: each has a counter of its own)
    if (threadIdx.x == 0) *flag = arrive_last(counters + (first == 0 ? kMaxCtas : first * step), in_grp) ? 1 : 0;
    __syncthreads();
    if (!*flag) return;
    const bool fin = parts <= kJoin;
    join<NH, HD, NT>(P, in_grp, [&](int p) { return slot_of((first + p) * step); }, fin, slot_of(first * step), n, h0, nh);
    if (fin) return;
    mine = first / kJoin;
    parts = (parts + kJoin - 1) / kJoin;
    step *= kJoin;
  }
}

}  // namespace paged
}  // namespace csa
