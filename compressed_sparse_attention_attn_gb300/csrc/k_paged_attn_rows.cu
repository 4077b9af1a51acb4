// k_paged_attn_rows.cu -- attention of single tokens over a paged cache of wide latent rows (head_dim above 256).
//
// Row n, head h: S_j = scale q_h . K_j over the rows j = first .. pos of its request, O = sum e^{S_j} V_j /
// (e^{sink} + sum e^{S_j}).  One CTA a (row, head): each warp takes every fourth row with a running maximum
// and sum in f32, the lanes holding the features; the four warps are joined through shared memory.
#include "csa_internal.cuh"
#include "rowops.cuh"

namespace csa {
namespace paged {
namespace {

constexpr int kRowWarps = 4;
constexpr int kMaxPer = 16;  // features a lane (head_dim <= 512)

__global__ void __launch_bounds__(kRowWarps * 32) k_paged_attn_simple(PagedAttnArgs a) {
  __shared__ float s_acc[kRowWarps][512], s_m[kRowWarps], s_l[kRowWarps];
  const int n = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hd = a.c.head_dim, kvh = h / (a.H / a.c.kv_heads);
  const int req = a.req ? a.req[n] : n;
  int pos = a.pos[n];
  if (req < 0 || pos < -1) return;
  if (req >= a.R) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadIndex);
    return;
  }
  const int64_t cap = (int64_t)a.width * a.c.page;
  if (pos >= cap) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadIndex);
  }
  const int64_t first = a.window > 0 ? max((int64_t)0, (int64_t)pos + 1 - a.window) : 0;
  const int64_t end = min((int64_t)pos + 1, cap);
  const bf16 *q = a.q + n * a.q_t + (int64_t)h * hd;
  float qv[kMaxPer], acc[kMaxPer];
#pragma unroll
  for (int u = 0; u < kMaxPer; ++u) {
    const int d = lane + 32 * u;
    qv[u] = d < hd ? __bfloat162float(q[d]) : 0.f;
    acc[u] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const bf16 *kb = reinterpret_cast<const bf16 *>(a.c.k) + kvh * a.c.k_head;
  const bf16 *vb = a.c.v ? reinterpret_cast<const bf16 *>(a.c.v) + kvh * a.c.v_head : kb;
  const int64_t vp = a.c.v ? a.c.v_page : a.c.k_page, vr = a.c.v ? a.c.v_row : a.c.k_row;
  for (int64_t j = first + warp; j < end; j += kRowWarps) {
    const int id = a.table[(int64_t)req * a.width + j / a.c.page];
    if (id < 0 || id >= a.c.n_pages) {
      if (lane == 0) atomicOr(a.status, kStatusBadIndex);
      continue;
    }
    const int64_t r = j % a.c.page;
    const bf16 *k = kb + id * a.c.k_page + r * a.c.k_row, *v = vb + id * vp + r * vr;
    float d = 0.f;
#pragma unroll
    for (int u = 0; u < kMaxPer; ++u)
      if (lane + 32 * u < hd) d = fmaf(qv[u], __bfloat162float(k[lane + 32 * u]), d);
    const float s = warp_sum(d) * a.scale;
    const float mn = fmaxf(m, s), c = mn == -INFINITY ? 1.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
    l = l * c + p;
#pragma unroll
    for (int u = 0; u < kMaxPer; ++u)
      if (lane + 32 * u < hd) acc[u] = fmaf(p, __bfloat162float(v[lane + 32 * u]), acc[u] * c);
    m = mn;
  }
#pragma unroll
  for (int u = 0; u < kMaxPer; ++u)
    if (lane + 32 * u < hd) s_acc[warp][lane + 32 * u] = acc[u];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY;
  for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, s_m[w]);
  const float sink = a.sink ? a.sink[h] : -INFINITY;
  const float T = fmaxf(M, sink);
  float L = 0.f, f[kRowWarps];
  for (int w = 0; w < kRowWarps; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.f : expf(s_m[w] - M);  // (towards the rows' own maximum: a sink far above it
    L += s_l[w] * f[w];                                   //  leaves lse its digits)
  }
  const float em = M == -INFINITY ? 0.f : expf(M - T);
  const float below = L * em + (a.sink ? expf(sink - T) : 0.f);
  for (int d = threadIdx.x; d < hd; d += blockDim.x) {
    float o = 0.f;
    for (int w = 0; w < kRowWarps; ++w) o += s_acc[w][d] * f[w];
    a.o[n * a.o_t + (int64_t)h * hd + d] = __float2bfloat16_rn(below > 0.f ? o * em / below : 0.f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[(int64_t)n * a.H + h] = L > 0.f ? M + logf(L) : -INFINITY;
}

}  // namespace

cudaError_t launch_rows(const PagedAttnArgs &a, cudaStream_t s) {
  k_paged_attn_simple<<<dim3(a.N, a.H), kRowWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace csa
