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
#include <algorithm>

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
template <bool FAST>
__device__ __forceinline__ void load_w(const float *w, int f, float (&v)[8]) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.f;
  } else if (FAST) {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4 *>(w + f + e));
      v[e] = x.x;
      v[e + 1] = x.y;
      v[e + 2] = x.z;
      v[e + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __ldg(w + f + e);
  }
}

// The (cos, sin) that the 8 features from f on are turned by, and the sign with which the partner enters: (y, z) ->
// y c + z s' with s' = -s for the first of a pair.  FAST: the turned part and its halves start and end on
// vector borders.  Outside the turned part: c = 1, s' = 0.
template <bool FAST>
__device__ __forceinline__ void load_angles(const NormRopeArgs &a, const float2 *tp, int f, float (&c)[8], float (&s)[8]) {
  const int h2 = a.rd >> 1;
  if (FAST && (f < a.at || f >= a.at + a.rd)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
  } else if (FAST && a.half) {
    const bool low = f < a.at + h2;
    const int i0 = low ? f - a.at : f - a.at - h2;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float4 x = __ldg(reinterpret_cast<const float4 *>(tp + i0 + e));
      c[e] = x.x;
      c[e + 1] = x.z;
      s[e] = low ? -x.y : x.y;
      s[e + 1] = low ? -x.w : x.w;
    }
  } else if (FAST) {
    const int i0 = (f - a.at) >> 1;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4 *>(tp + i0 + e / 2));
      c[e] = c[e + 1] = x.x;
      s[e] = -x.y;
      s[e + 1] = x.y;
      c[e + 2] = c[e + 3] = x.z;
      s[e + 2] = -x.w;
      s[e + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = f + e - a.at;  // feature of the turned part
      c[e] = 1.f;
      s[e] = 0.f;
      if (d < 0 || d >= a.rd) continue;
      const bool first = a.half ? d < h2 : !(d & 1);
      const float2 x = __ldg(tp + (a.half ? (first ? d : d - h2) : d >> 1));
      c[e] = x.x;
      s[e] = first ? -x.y : x.y;
    }
  }
}

// The partners' normed values (before the scale r): features half the turned part away, from the row in memory.
template <bool FAST>
__device__ __forceinline__ void load_partners(const NormRopeArgs &a, const bf16 *x, int f, uint4 &z) {
  const int h2 = a.rd >> 1;
  z = make_uint4(0, 0, 0, 0);
  if (FAST) {
    if (f >= a.at && f < a.at + a.rd) z = *reinterpret_cast<const uint4 *>(x + (f < a.at + h2 ? f + h2 : f - h2));
  } else {
    bf16 *zb = reinterpret_cast<bf16 *>(&z);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = f + e - a.at;
      if (d >= 0 && d < a.rd) zb[e] = x[d < h2 ? f + e + h2 : f + e - h2];
    }
  }
}
template <bool FAST>
__device__ __forceinline__ void load_partner_w(const NormRopeArgs &a, const float *w, int f, float (&v)[8]) {
  const int h2 = a.rd >> 1;
  if (FAST) {
    load_w<true>(w, f >= a.at && f < a.at + a.rd ? (f < a.at + h2 ? f + h2 : f - h2) : f, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = f + e - a.at;
      v[e] = w && d >= 0 && d < a.rd ? __ldg(w + (d < h2 ? f + e + h2 : f + e - h2)) : 1.f;
    }
  }
}

// G lanes a row, V vectors a lane (head_dim <= 8 G V).  A group of lanes takes `per` heads of one kind (query, key,
// value) of one token, U at a time with the next U's vectors in flight; the norm's weights and the token's angles,
// multiplied together, stay in registers for all of them.  Items are (token, block of `per` heads), a token's
// query, key and value blocks in a row.
template <int G, int V, int U, bool HALF, bool FAST>
__global__ void __launch_bounds__(kThreads, V == 4 ? 1 : (V == 2 && HALF ? 2 : 3)) k_norm_rope(const __grid_constant__ NormRopeArgs a, int per, int q_blocks,
                                                           int k_blocks, int per_token, int64_t items) {
  const int lane = threadIdx.x & (G - 1);
  const int hd = a.c.head_dim;
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / G;
  const bool in = item < items;
  const int n = in ? (int)(item / per_token) : 0;
  const int jb = in ? (int)(item - (int64_t)n * per_token) : 0;
  const int kind = jb < q_blocks ? 0 : (jb < q_blocks + k_blocks ? 1 : 2);  // query, key, value
  const int h0 = (kind == 0 ? jb : (kind == 1 ? jb - q_blocks : jb - q_blocks - k_blocks)) * per;
  const int nh = min(per, (kind == 0 ? a.H : a.c.kv_heads) - h0);
  const int64_t x_h = kind == 0 ? a.q_h : (kind == 1 ? a.k_h : a.v_h);
  const bf16 *x = (kind == 0 ? a.q + n * a.q_t : (kind == 1 ? a.k + n * a.k_t : a.v + n * a.v_t)) + h0 * x_h;
  uint4 cur[U][V], nxt[U][V];
  auto load = [&](uint4 (&d)[U][V], int t0) {
#pragma unroll
    for (int t = 0; t < U; ++t)
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int f = 8 * (lane + G * u);
        d[t][u] = make_uint4(0, 0, 0, 0);
        if (in && t0 + t < nh && f < hd) d[t][u] = *reinterpret_cast<const uint4 *>(x + (int64_t)(t0 + t) * x_h + f);
      }
  };
  load(cur, 0);  // (the rows of padding tokens exist too)
  const int p = in ? a.pos[n] : -1;
  const int rows = a.c.n_pages * a.c.page;
  const int slot = !in ? -1 : (a.slot ? a.slot[n] : n);
  bool live = in && p >= 0;
  if (live && ((a.rd > 0 && p >= a.tab_rows) || slot < -1 || slot >= rows)) {
    if (jb == 0 && lane == 0) atomicOr(a.status, kStatusBadIndex);
    live = false;
  }
  if (kind != 0 && slot < 0) live = false;
  int64_t y_h;
  bf16 *y;
  if (kind == 0) {
    y_h = a.o_h;
    y = a.q_out + n * a.o_t + h0 * y_h;
  } else {
    const int pg = live ? (int)((uint32_t)slot / (uint32_t)a.c.page) : 0, row = live ? slot - pg * a.c.page : 0;
    y_h = kind == 1 ? a.c.k_head : a.c.v_head;
    y = (kind == 1 ? reinterpret_cast<bf16 *>(a.c.k) + pg * a.c.k_page + row * a.c.k_row
                   : reinterpret_cast<bf16 *>(a.c.v) + pg * a.c.v_page + row * a.c.v_row) + h0 * y_h;
  }
  const float *w = kind == 0 ? a.q_norm : a.k_norm;
  const bool plain = kind == 2, turns = !plain && a.rd > 0;
  // y = r (x c + z s) with z the partner's value: c = weight x cos, s = partner's weight x (+-sin)
  float c[V][8], s[V][8];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int f = 8 * (lane + G * u);
#pragma unroll
    for (int e = 0; e < 8; ++e) c[u][e] = 1.f, s[u][e] = 0.f;
    if (!live || plain || f >= hd) continue;
    float wv[8];
    load_w<FAST>(w, f, wv);
    if (turns) {
      const float2 *tp = reinterpret_cast<const float2 *>(a.tab) + (int64_t)p * (a.rd >> 1);
      load_angles<FAST>(a, tp, f, c[u], s[u]);
      float wp[8];
      if (HALF) load_partner_w<FAST>(a, w, f, wp);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[u][e] *= HALF ? wp[e] : wv[e ^ 1];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) c[u][e] *= wv[e];
  }
  // (every group of the warp goes through as many rounds: the shuffles below are the warp's)
  int rounds = (max(nh, 0) + U - 1) / U;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) rounds = max(rounds, __shfl_xor_sync(0xffffffffu, rounds, o));
  for (int rnd = 0; rnd < rounds; ++rnd) {
    const int t0 = rnd * U;
    load(nxt, t0 + U);
    uint4 xp[U][V];  // the partners' vectors, from the lines just read
    if (HALF) {
#pragma unroll
      for (int t = 0; t < U; ++t)
#pragma unroll
        for (int u = 0; u < V; ++u) {
          const int f = 8 * (lane + G * u);
          xp[t][u] = make_uint4(0, 0, 0, 0);
          if (live && turns && t0 + t < nh && f < hd) load_partners<FAST>(a, x + (int64_t)(t0 + t) * x_h, f, xp[t][u]);
        }
    }
    float r[U];
#pragma unroll
    for (int t = 0; t < U; ++t) {
      r[t] = 0.f;
#pragma unroll
      for (int u = 0; u < V; ++u) {
        float v[8];
        unpack(cur[t][u], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[t] = fmaf(v[e], v[e], r[t]);
      }
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
      for (int t = 0; t < U; ++t) r[t] += __shfl_xor_sync(0xffffffffu, r[t], o);
#pragma unroll
    for (int t = 0; t < U; ++t) r[t] = !plain && w ? 1.0f / sqrtf(r[t] / (float)hd + a.eps) : 1.f;
    __syncwarp();  // (q_out may be q: every lane has read its partners)
#pragma unroll
    for (int t = 0; t < U; ++t) {
      if (!live || t0 + t >= nh) continue;
      bf16 *yt = y + (int64_t)(t0 + t) * y_h;
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int f = 8 * (lane + G * u);
        if (f >= hd) continue;
        if (plain) {
          *reinterpret_cast<uint4 *>(yt + f) = cur[t][u];
          continue;
        }
        float v[8], z[8], o[8];
        unpack(cur[t][u], v);
        if (HALF) unpack(xp[t][u], z);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // (outside the turned part there is no partner, which may be infinite)
          if (!HALF) z[e] = turns && f + e >= a.at && f + e < a.at + a.rd ? v[e ^ 1] : 0.f;
          o[e] = r[t] * fmaf(v[e], c[u][e], z[e] * s[u][e]);
        }
        *reinterpret_cast<uint4 *>(yt + f) = pack(o);
      }
    }
#pragma unroll
    for (int t = 0; t < U; ++t)
#pragma unroll
      for (int u = 0; u < V; ++u) cur[t][u] = nxt[t][u];
  }
}

template <int G, int V, int U>
cudaError_t launch(const NormRopeArgs &a, int num_sms, cudaStream_t s) {
  // Heads a group: as many (up to 16) as still leave a full complement of warps (24 an SM), at least U where there
  // are rows enough, else one, which spreads few rows over more SMs.
  const int most = std::max(a.H, a.c.kv_heads);
  auto blocks_of = [](int h, int per) { return (h + per - 1) / per; };
  auto per_token_of = [&](int per) { return blocks_of(a.H, per) + blocks_of(a.c.kv_heads, per) * (a.v ? 2 : 1); };
  int per = 1;
  while (per < 16 && per < most && (int64_t)a.N * per_token_of(2 * per) * G >= (int64_t)num_sms * 24 * 32) per *= 2;
  const int q_blocks = blocks_of(a.H, per), k_blocks = blocks_of(a.c.kv_heads, per), per_token = per_token_of(per);
  const int64_t items = (int64_t)a.N * per_token;
  const int64_t blocks = (items * G + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  // vectors of weights, angles and partners: 16-byte aligned, the turned part (and its halves) on vector borders
  const bool fast = a.at % 8 == 0 && a.rd % (a.half ? 16 : 8) == 0 &&
                    (((uintptr_t)a.tab | (uintptr_t)a.q_norm | (uintptr_t)a.k_norm) & 15) == 0;
  auto *k = a.half ? (fast ? k_norm_rope<G, V, U, true, true> : k_norm_rope<G, V, U, true, false>)
                   : (fast ? k_norm_rope<G, V, U, false, true> : k_norm_rope<G, V, U, false, false>);
  k<<<(unsigned)blocks, kThreads, 0, s>>>(a, per, q_blocks, k_blocks, per_token, items);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, int num_sms, cudaStream_t s) {
  const int hd = a.c.head_dim;
  if (hd <= 32) return launch<4, 1, 2>(a, num_sms, s);
  if (hd <= 64) return launch<8, 1, 2>(a, num_sms, s);
  if (hd <= 128) return launch<16, 1, 2>(a, num_sms, s);
  if (hd <= 256) return launch<32, 1, 2>(a, num_sms, s);
  if (hd <= 512) return launch<32, 2, 1>(a, num_sms, s);
  return launch<32, 4, 1>(a, num_sms, s);
}

}  // namespace csa
