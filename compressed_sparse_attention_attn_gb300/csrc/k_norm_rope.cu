// k_norm_rope.cu -- RMSNorm of each query and key head, the position rotation and the write into a paged
// cache, in one pass over the rows.
//
// A head's row (head_dim features) is held by a group of 4 to 32 lanes, V vectors of 8 features a lane
// (vector lane + G*u of the row), so the sum of squares is a few shuffles and a row is read once:
//   y = x r w,  r = 1 / sqrt(mean(x^2) + eps);  (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c) over the pairs
// of the turned part, everything in f32, one rounding to bf16 at the store (a normed value rounded before
// its turn would add a second error of the same size).  Adjacent pairs lie in one lane's vector.  Pairs half
// the turned part apart do not: a lane reads its partners' vectors too (the L1 lines its neighbours have
// just fetched), which needs no rule on where a partner's lane is.
//
// Bound by HBM: a row is read and written once; the angles of a token are shared by its heads through L1.
// Value rows are copies of the same shape.
#include "csa_internal.cuh"
#include "rowops.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack(const uint4 &w, float (&v)[8]) {
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __low2float(h[e]);
    v[2 * e + 1] = __high2float(h[e]);
  }
}
__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
  uint4 w;
  __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&w);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
  return w;
}

// 8 floats of w at feature f (ones where w is NULL)
__device__ __forceinline__ void load_w(const float *w, int f, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = w ? __ldg(w + f + e) : 1.f;
}

// Turn the 8 normed features y at f .. f+7 of a row.  xr: the row's bf16 values in memory, scale r and weights w for
// the partners.  FAST: the turned part starts and ends on vector borders, as do its halves.
template <bool FAST>
__device__ __forceinline__ void turn(const NormRopeArgs &a, const bf16 *xr, const uint4 &partner, const float2 *tp, float r,
                                     const float *w, int f, float (&y)[8]) {
  const int h2 = a.rd >> 1;
  if (FAST) {
    if (f < a.at || f >= a.at + a.rd) return;
    if (a.half) {
      const bool low = f < a.at + h2;
      const int i0 = low ? f - a.at : f - a.at - h2;
      float z[8], wz[8];
      unpack(partner, z);
      load_w(w, low ? f + h2 : f - h2, wz);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 cs = __ldg(reinterpret_cast<const float4 *>(tp + i0 + e));
        const float z0 = z[e] * r * wz[e], z1 = z[e + 1] * r * wz[e + 1];
        y[e] = low ? y[e] * cs.x - z0 * cs.y : z0 * cs.y + y[e] * cs.x;
        y[e + 1] = low ? y[e + 1] * cs.z - z1 * cs.w : z1 * cs.w + y[e + 1] * cs.z;
      }
    } else {
      const int i0 = (f - a.at) >> 1;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 cs = __ldg(reinterpret_cast<const float4 *>(tp + i0 + e / 2));
        const float a0 = y[e], b0 = y[e + 1], a1 = y[e + 2], b1 = y[e + 3];
        y[e] = a0 * cs.x - b0 * cs.y;
        y[e + 1] = a0 * cs.y + b0 * cs.x;
        y[e + 2] = a1 * cs.z - b1 * cs.w;
        y[e + 3] = a1 * cs.w + b1 * cs.z;
      }
    }
  } else {
    float out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = f + e - a.at;  // feature of the turned part
      out[e] = y[e];
      if (d < 0 || d >= a.rd) continue;
      const bool first = a.half ? d < h2 : !(d & 1);
      const int i = a.half ? (first ? d : d - h2) : d >> 1;
      const int fp = a.half ? (first ? f + e + h2 : f + e - h2) : (first ? f + e + 1 : f + e - 1);
      const float z = __bfloat162float(xr[fp]) * r * (w ? __ldg(w + fp) : 1.f);
      const float2 cs = __ldg(tp + i);
      out[e] = first ? y[e] * cs.x - z * cs.y : z * cs.y + y[e] * cs.x;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = out[e];
  }
}

// G lanes a row, V vectors a lane (head_dim <= 8 G V).  Items are (token, head) with a token's query, key and value
// heads in a row.
template <int G, int V, bool FAST>
__global__ void __launch_bounds__(kThreads) k_norm_rope(NormRopeArgs a, int per_token, int64_t items) {
  const int lane = threadIdx.x & (G - 1);
  const int hd = a.c.head_dim, Hk = a.c.kv_heads;
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / G;
  const bool in = item < items;
  const int n = in ? (int)(item / per_token) : 0;
  const int h = in ? (int)(item - (int64_t)n * per_token) : 0;
  const int kind = h < a.H ? 0 : (h < a.H + Hk ? 1 : 2);  // query, key, value
  const int hh = kind == 0 ? h : (kind == 1 ? h - a.H : h - a.H - Hk);
  const int p = in ? a.pos[n] : -1;
  const int64_t rows = (int64_t)a.c.n_pages * a.c.page;
  const int64_t slot = !in ? -1 : (a.slot ? a.slot[n] : n);
  bool live = in && p >= 0;
  const bool bad = live && ((a.rd > 0 && p >= a.tab_rows) || slot < -1 || slot >= rows);
  if (bad) {
    if (h == 0 && lane == 0) atomicOr(a.status, kStatusBadIndex);
    live = false;
  }
  if (kind != 0 && slot < 0) live = false;
  const bf16 *x = kind == 0 ? a.q + n * a.q_t + hh * a.q_h
                            : (kind == 1 ? a.k + n * a.k_t + hh * a.k_h : a.v + n * a.v_t + hh * a.v_h);
  bf16 *y;
  if (kind == 0) {
    y = a.q_out + n * a.o_t + hh * a.o_h;
  } else {
    const int64_t pg = live ? slot / a.c.page : 0, row = live ? slot % a.c.page : 0;
    y = kind == 1 ? reinterpret_cast<bf16 *>(a.c.k) + pg * a.c.k_page + row * a.c.k_row + hh * a.c.k_head
                  : reinterpret_cast<bf16 *>(a.c.v) + pg * a.c.v_page + row * a.c.v_row + hh * a.c.v_head;
  }
  const int h2 = a.rd >> 1;
  const bool turns = kind != 2 && a.rd > 0;
  uint4 xv[V], xp[V];
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int f = 8 * (lane + G * u);
    xv[u] = xp[u] = make_uint4(0, 0, 0, 0);
    if (live && f < hd) {
      xv[u] = *reinterpret_cast<const uint4 *>(x + f);
      if (FAST && turns && a.half && f >= a.at && f < a.at + a.rd)
        xp[u] = *reinterpret_cast<const uint4 *>(x + (f < a.at + h2 ? f + h2 : f - h2));
    }
  }
  float r = 1.f;
  const float *w = kind == 0 ? a.q_norm : a.k_norm;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    float v[8];
    unpack(xv[u], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (kind != 2 && w) r = 1.0f / sqrtf(ss / (float)hd + a.eps);
  const float2 *tp = reinterpret_cast<const float2 *>(a.tab) + (int64_t)(live && a.rd > 0 ? p : 0) * h2;
  uint4 out[V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int f = 8 * (lane + G * u);
    out[u] = xv[u];
    if (live && f < hd && kind != 2) {
      float v[8], wv[8];
      unpack(xv[u], v);
      load_w(w, f, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= r * wv[e];
      if (turns) turn<FAST>(a, x, xp[u], tp, r, w, f, v);
      out[u] = pack(v);
    }
  }
  __syncwarp();  // (q_out may be q: every lane has read its partners)
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int f = 8 * (lane + G * u);
    if (live && f < hd) *reinterpret_cast<uint4 *>(y + f) = out[u];
  }
}

template <int G, int V>
cudaError_t launch(const NormRopeArgs &a, cudaStream_t s) {
  const int per_token = a.H + a.c.kv_heads * (a.v ? 2 : 1);
  const int64_t items = (int64_t)a.N * per_token;
  const int64_t blocks = (items * G + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  // vectors of angles and partners: the turned part (and its halves) on vector borders, 16-byte angles
  const bool fast = a.at % 8 == 0 && a.rd % (a.half ? 16 : 8) == 0 && ((uintptr_t)a.tab & 15) == 0;
  if (fast)
    k_norm_rope<G, V, true><<<(unsigned)blocks, kThreads, 0, s>>>(a, per_token, items);
  else
    k_norm_rope<G, V, false><<<(unsigned)blocks, kThreads, 0, s>>>(a, per_token, items);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t s) {
  const int hd = a.c.head_dim;
  if (hd <= 32) return launch<4, 1>(a, s);
  if (hd <= 64) return launch<8, 1>(a, s);
  if (hd <= 128) return launch<16, 1>(a, s);
  if (hd <= 256) return launch<32, 1>(a, s);
  if (hd <= 512) return launch<32, 2>(a, s);
  return launch<32, 4>(a, s);
}

}  // namespace csa
