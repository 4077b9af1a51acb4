// paged_common.cuh -- what the paged-attention kernels share: how ragged rows are dealt over the CTAs, and how
// the shares of a row that several CTAs worked on are joined.
//
// A segment is the work of one (row, head group): its positions in units of U rows, at least one (an empty row
// writes zeros).  The segments' units stand one behind the other (row, head group, unit); of their total T
// CTA c of G takes [T c / G, T (c + 1) / G), so every CTA has the same number of rows to read whatever the
// lengths are, and at most the first and the last segment of its range are shared with others.  The host knows
// no lengths: every CTA sums the units itself.
//
// A CTA's share of a segment is (M, L, O): its running maximum (base 2), sum of weights and weighted sum of
// values relative to M, in f32, in one of its two slots (0: a segment that began in an earlier CTA, 1: one
// that begins here).  Twenty consecutive shares of a segment are a group.  The CTA that completes a group
// joins it (in the order of the shares, whoever is last); with more than one group the joined shares go to
// the group's first slot, and the CTA that completes the last group joins those.  So a long row over 300
// CTAs is joined in two steps of at most 20, and nothing waits.  The counters return to zero.
#pragma once

#include "csa_internal.cuh"
#include "tc_ptx.cuh"

namespace csa {
namespace paged {

constexpr int kJoin = 20;          // shares of a group
constexpr int kMaxJoin = 32;       // groups of a segment
constexpr int kMaxCtas = kJoin * kMaxJoin;

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
  float *share_ml;      // [2 G][heads of a group][2]
  int *counters;        // [3][kMaxCtas]: groups past a segment's first, first groups, segments
  int2 *split;          // latent rows: of the segments that several CTAs shared, the first CTA and how many
  int ctas;             // CTAs launched
  int by_segment;       // `split` is by segment (no more of them than CTAs), else by first CTA
};

// The positions first .. first + rows - 1 of row n; units of U rows (0: a row that is left alone).
struct Row {
  int req, first, rows, units;
};
template <int U>
__device__ __forceinline__ Row row_of(const PagedAttnArgs &a, int n, bool report) {
  Row r;
  r.req = a.req ? a.req[n] : n;
  const int pos = a.pos[n];
  r.first = r.rows = r.units = 0;
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
  r.units = max(1, (r.rows + U - 1) / U);
  return r;
}

// A CTA's range of units and the row its first unit lies in.
struct Range {
  int64_t total, begin, end;  // units
  int ctas;                   // CTAs that share them: no more than there are units, so that none between two has nothing
  int row;
  int64_t before;             // units (of all its segments) before that row
};
// Called by all NT threads of the CTA.  scratch: int64 [NT / 32 + 4] in shared memory.
template <int U, int NT>
__device__ __forceinline__ Range find_range(const Params &P, int64_t *scratch) {
  const PagedAttnArgs &a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  constexpr int NW = NT / 32;
  int64_t *found = scratch + NW;  // row, before, total
  const bool report = blockIdx.x == 0;
  auto scan = [&](int64_t v, int64_t &sum) -> int64_t {  // inclusive over the CTA; sum: of all
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += o;
    }
    __syncthreads();
    if (lane == 31) scratch[wid] = x;
    __syncthreads();
    int64_t b = 0;
    sum = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < wid) b += scratch[w];
      sum += scratch[w];
    }
    return x + b;
  };
  Range r;
  int64_t mine = 0;
  for (int n = tid; n < a.N; n += NT) mine += row_of<U>(a, n, report).units;
  int64_t sum;
  int64_t incl = scan(mine, sum);
  r.total = sum * P.Hg;
  r.ctas = (int)min((int64_t)gridDim.x, r.total);
  const bool works = (int)blockIdx.x < r.ctas;
  r.begin = works ? r.total * blockIdx.x / r.ctas : 0;
  r.end = works ? r.total * (blockIdx.x + 1) / r.ctas : 0;
  r.row = 0;
  r.before = 0;
  if (r.begin >= r.end) return r;
  int64_t base = 0;
  for (int n0 = 0; n0 < a.N; n0 += NT) {  // one round for up to NT rows
    if (a.N > NT) {
      mine = n0 + tid < a.N ? row_of<U>(a, n0 + tid, false).units : 0;
      incl = scan(mine, sum);
    }
    const int64_t lo = (base + incl - mine) * P.Hg, hi = (base + incl) * P.Hg;
    if (r.begin >= lo && r.begin < hi) {
      found[0] = n0 + tid;
      found[1] = lo;
    }
    base += sum;
    if (r.begin < base * P.Hg) break;
  }
  __syncthreads();
  r.row = (int)found[0];
  r.before = found[1];
  return r;
}

// The CTA that unit u belongs to: the largest c with T c / G <= u.
__device__ __forceinline__ int cta_of(int64_t u, const Range &r) { return (int)(((u + 1) * r.ctas - 1) / r.total); }

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

// Barrier of the NT threads that join: the whole CTA (BAR 0) or named barrier BAR.
template <int NT, int BAR>
__device__ __forceinline__ void join_sync() {
  if constexpr (BAR == 0)
    __syncthreads();
  else
    tc::named_bar(BAR, NT);
}

// Join `parts` shares, shares i of slots slot(i), of NH heads x HD features by NT threads (tid of them).  fin: write
// O and lse of heads h0 .. h0+nh-1 of row n; else the joined share to slot `to`.
// sf: kJoinFloats<NH> floats of shared memory.
template <int NH>
constexpr int kJoinFloats = (kMaxJoin + 2) * NH;
template <int NH, int HD, int NT, int BAR, class Slot>
__device__ __forceinline__ void join(const Params &P, int tid, int parts, Slot slot, bool fin, int to, int n, int h0, int nh,
                                     float *sf) {
  const PagedAttnArgs &a = P.a;
  float *sM = sf + kMaxJoin * NH, *sL = sM + NH;
  for (int i = tid; i < parts * nh; i += NT) {
    const int p = i / nh, h = i % nh;
    sf[p * NH + h] = __ldcg(P.share_ml + ((int64_t)slot(p) * NH + h) * 2);
  }
  join_sync<NT, BAR>();
  if (tid < nh) {
    float M = -INFINITY;
    for (int p = 0; p < parts; ++p) M = fmaxf(M, sf[p * NH + tid]);
    float L = 0.f;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float m = sf[p * NH + tid];
      const float f = m == -INFINITY ? 0.f : exp2f(m - M);
      sf[p * NH + tid] = f;
      L = fmaf(__ldcg(P.share_ml + ((int64_t)slot(p) * NH + tid) * 2 + 1), f, L);
    }
    sL[tid] = L;
    if (fin) {
      sM[tid] = out_factor(M, L, a.sink, h0 + tid);
      if (a.lse) a.lse[(int64_t)n * a.H + h0 + tid] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    } else {
      sM[tid] = M;
    }
  }
  join_sync<NT, BAR>();
  const int hd = a.c.head_dim;
  for (int i = tid; i < nh * (HD / 4); i += NT) {
    const int h = i / (HD / 4), d = (i % (HD / 4)) * 4;
    if (d >= hd) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += 8) {
      float4 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (p0 + u < parts) x[u] = __ldcg(reinterpret_cast<const float4 *>(P.share_o + ((int64_t)slot(p0 + u) * NH + h) * HD + d));
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (p0 + u < parts) {
          const float f = sf[(p0 + u) * NH + h];
          v.x = fmaf(x[u].x, f, v.x);
          v.y = fmaf(x[u].y, f, v.y);
          v.z = fmaf(x[u].z, f, v.z);
          v.w = fmaf(x[u].w, f, v.w);
        }
    }
    if (fin) {
      const float f = sM[h];
      __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * f, v.y * f), hi = __floats2bfloat162_rn(v.z * f, v.w * f);
      uint2 w = make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
      *reinterpret_cast<uint2 *>(a.o + (int64_t)n * a.o_t + (int64_t)(h0 + h) * hd + d) = w;
    } else {
      *reinterpret_cast<float4 *>(P.share_o + ((int64_t)to * NH + h) * HD + d) = v;
    }
  }
  if (!fin && tid < nh) {
    float2 ml = make_float2(sM[tid], sL[tid]);
    *reinterpret_cast<float2 *>(P.share_ml + ((int64_t)to * NH + tid) * 2) = ml;
  }
  join_sync<NT, BAR>();
}

// Publish this CTA's share of the segment of units [sb, se) (already written to its slot by the NT threads, or
// by threads they have synchronised with) and join what it completes.  flag: an int in shared memory.
template <int NH, int HD, int NT, int BAR>
__device__ __forceinline__ void publish(const Params &P, int tid, int64_t sb, int64_t se, const Range &r, int n, int h0, int nh,
                                        float *sf, int *flag) {
  const int c0 = cta_of(sb, r), c1 = cta_of(se - 1, r);
  const int parts = c1 - c0 + 1, mine = (int)blockIdx.x - c0, grp = mine / kJoin, ngrp = (parts + kJoin - 1) / kJoin;
  const int in_grp = min(kJoin, parts - grp * kJoin);
  auto slot_of = [c0](int p) { return p == 0 ? 2 * c0 + 1 : 2 * (c0 + p); };
  join_sync<NT, BAR>();
  if (tid == 0) {
    int *ctr = grp == 0 ? P.counters + kMaxCtas + c0 : P.counters + c0 + grp * kJoin;
    *flag = arrive_last(ctr, in_grp) ? 1 : 0;
  }
  join_sync<NT, BAR>();
  if (!*flag) return;
  const int first = grp * kJoin;
  join<NH, HD, NT, BAR>(P, tid, in_grp, [&](int p) { return slot_of(first + p); }, ngrp == 1, slot_of(first), n, h0, nh, sf);
  if (ngrp == 1) return;
  if (tid == 0) *flag = arrive_last(P.counters + 2 * kMaxCtas + c0, ngrp) ? 1 : 0;
  join_sync<NT, BAR>();
  if (!*flag) return;
  join<NH, HD, NT, BAR>(P, tid, ngrp, [&](int p) { return slot_of(p * kJoin); }, true, 0, n, h0, nh, sf);
}

}  // namespace paged
}  // namespace csa
