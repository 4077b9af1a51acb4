// k_rows_attn.cu -- attention of many rows over a paged cache: the new tokens of prompts, and decode rows that share a prefix.
//
// A warp takes one row (token n, query head h) and goes through its positions 32 at a time: a lane the score of one position, then
// a lane eight features of the weighted values.  Softmax statistics are f32 (base 2), one pass with the running maximum and sum.
#include "paged_common.cuh"

namespace csa {
namespace rows {

struct Params {
  RowsAttnArgs a;
  paged::FastDiv page;
  float scale_log2;
};

// The positions first .. last of a table's row that token n (of the segment with rows t0 .. t1 - 1) attends.
struct Span {
  const int32_t *pages;
  int64_t first, last;
};

__global__ void __launch_bounds__(128) k_rows_attn(const __grid_constant__ Params P) {
  const RowsAttnArgs &a = P.a;
  const int lane = threadIdx.x & 31, hd = a.c.head_dim;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  dependency_wait();
  if (i >= (int64_t)a.N * a.H) return;
  const int n = (int)(i / a.H), h = (int)(i - (int64_t)n * a.H), kvh = h / (a.H / a.c.kv_heads);
  int seg = -1, t0 = 0, t1 = a.N;
  if (a.cu) {
    for (int s = 0; s < a.S; ++s) {
      const int lo = a.cu[s], hi = a.cu[s + 1];
      if (lo < 0 || hi < lo || hi > a.N) {
        if (i == 0 && lane == 0) atomicOr(a.status, kStatusBadIndex);
        continue;
      }
      if (seg < 0 && n >= lo && n < hi) seg = s, t0 = lo, t1 = hi;
    }
  } else {
    seg = 0;
  }
  if (seg < 0) return;
  Span sp[2];
  int spans = 1;
  const int64_t cap = min((int64_t)a.width * a.c.page, (int64_t)0x7fffffff);
  int64_t len = a.len[seg];
  if (a.pos) {  // a prefix, and the row's own pages
    const int req = a.req ? a.req[n] : n, pos = a.pos[n];
    if (req < 0 || pos < -1) return;
    const int64_t own = min((int64_t)a.own_width * a.c.page, (int64_t)0x7fffffff);
    if (req >= a.R) {
      if (lane == 0) atomicOr(a.status, kStatusBadIndex);
      return;
    }
    if (lane == 0 && (pos >= own || len < 0 || len > cap)) atomicOr(a.status, kStatusBadIndex);
    len = max((int64_t)0, len);
    const int64_t first = a.window > 0 ? max((int64_t)0, len + pos + 1 - a.window) : 0;
    sp[0] = {a.table + (int64_t)seg * a.width, first, min(len, cap) - 1};
    sp[1] = {a.own_table + (int64_t)req * a.own_width, max((int64_t)0, first - len), min((int64_t)pos, own - 1)};
    spans = 2;
  } else {
    if (len < t1 - t0) {
      if (lane == 0) atomicOr(a.status, kStatusBadIndex);
      return;
    }
    const int64_t at = len - t1 + n;
    if (lane == 0 && len > cap) atomicOr(a.status, kStatusBadIndex);
    sp[0] = {a.table + (int64_t)seg * a.width, a.window > 0 ? max((int64_t)0, at + 1 - a.window) : 0, min(at, cap - 1)};
  }
  const bf16 *q = a.q + (int64_t)n * a.q_t + (int64_t)h * hd;
  const bf16 *kb = reinterpret_cast<const bf16 *>(a.c.k) + kvh * a.c.k_head;
  const bf16 *vb = a.c.v ? reinterpret_cast<const bf16 *>(a.c.v) + kvh * a.c.v_head : kb;
  const int64_t v_page = a.c.v ? a.c.v_page : a.c.k_page, v_row = a.c.v ? a.c.v_row : a.c.k_row;
  float m = -INFINITY, l = 0.f, acc[8] = {};
  for (int s = 0; s < spans; ++s)
    for (int64_t j0 = sp[s].first; j0 <= sp[s].last; j0 += 32) {
      const int64_t j = j0 + lane;
      int64_t vo = -1;
      float x = -INFINITY;
      if (j <= sp[s].last) {
        const int pg = (int)P.page.div((uint32_t)j), r = (int)j - pg * a.c.page, id = sp[s].pages[pg];
        if (id >= 0 && id < a.c.n_pages) {
          const bf16 *k = kb + (int64_t)id * a.c.k_page + (int64_t)r * a.c.k_row;
          vo = (int64_t)id * v_page + (int64_t)r * v_row;
          x = 0.f;
          for (int d = 0; d < hd; ++d) x = fmaf(__bfloat162float(q[d]), __bfloat162float(k[d]), x);
          x *= P.scale_log2;
        } else {
          atomicOr(a.status, kStatusBadIndex);
        }
      }
      float mx = x;
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(m, mx);
      const float ref = mx == -INFINITY ? 0.f : mx, f = paged::ex2(m - ref), p = vo < 0 ? 0.f : paged::ex2(x - ref);
      m = mx;
      l = l * f + p;
      for (int e = 0; e < 8; ++e) acc[e] *= f;
      for (int u = 0; u < 32; ++u) {
        const int64_t off = __shfl_sync(0xffffffffu, vo, u);
        const float w = __shfl_sync(0xffffffffu, p, u);
        if (off < 0) continue;
        for (int e = 0; e < 8; ++e)
          if (e * 32 + lane < hd) acc[e] = fmaf(w, __bfloat162float(vb[off + e * 32 + lane]), acc[e]);
      }
    }
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float f = paged::out_factor(m, l, a.sink, h);
  bf16 *out = a.o + (int64_t)n * a.o_t + (int64_t)h * hd;
  for (int e = 0; e < 8; ++e)
    if (e * 32 + lane < hd) out[e * 32 + lane] = __float2bfloat16(acc[e] * f);
  if (a.lse && lane == 0) a.lse[(int64_t)n * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace rows

cudaError_t launch_rows_attn(const RowsAttnArgs &a, float *ws, size_t ws_bytes, int *counters, int num_sms, cudaStream_t s) {
  rows::Params p;
  p.a = a;
  p.page = paged::FastDiv((uint32_t)a.c.page);
  p.scale_log2 = (float)(a.scale * 1.4426950408889634);
  return launch_dependent(rows::k_rows_attn, dim3((unsigned)(((int64_t)a.N * a.H + 3) / 4)), dim3(128), 0, s, 1, p);
}

}  // namespace csa
