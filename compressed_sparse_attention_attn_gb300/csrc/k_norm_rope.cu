// k_norm_rope.cu -- RMSNorm of each query and key head, the position rotation and the write into a paged
// cache, in one pass over the rows.
//
//   y = x r w,  r = 1 / sqrt(mean(x^2) + eps);  (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c) over the pairs
// of the turned part, everything in f32, one rounding to bf16 at the store (a normed value rounded before its
// turn would add a second error of the same size).  A group of 2 to 32
// lanes holds two rows, whose angles and weights come from L1 (all rows of a token, and all tokens, share them).
//
// Bound by HBM: a row is read and written once (4096 tokens of 64 x 512 and one 512-wide key row, 546 MB: 89 us, 6.2
// TB/s; 8000 tokens of 32 + 8 + 8 heads of 128, 201 MB: 39 us, 5.2 TB/s, with halves 42 us).  The instructions and L1 come close to
// it at 64 to 128 features, so the arithmetic is on pairs of f32 and a lane holds both vectors of a pair of halves:
// nothing is read twice, and only the sum of squares crosses lanes.
#include <algorithm>

#include "csa_internal.cuh"
#include "paged_common.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;
// CTAs an SM: of two rows of two vectors a group (4 against 3 with adjacent pairs, 4096 x 64 x 512: 89 against 100 us; 3 against 2
// with halves, 8000 tokens of 48 x 128: 42 against 52; one more spills)
template <int V, bool HALF>
constexpr int kResident = V > 2 ? 1 : HALF ? 3 : 4;

// ---- two f32 at a time ----
struct f2 {
  float x, y;
};
__device__ __forceinline__ unsigned long long pk(f2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ f2 up(unsigned long long r) {
  f2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)), "l"(pk(c)));
  return up(r);
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)));
  return up(r);
}
// four pairs of a 16-byte vector of bf16
__device__ __forceinline__ void unpack(const uint4 &w, f2 (&v)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = {__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u)};
}
__device__ __forceinline__ uint32_t pack2(f2 a) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// What the two kernels share: the row a group of lanes works on, and whether it is written.
struct Item {
  bool in, live, plain;  // plain: a value row, copied
  int n, pos, rows;      // rows: heads of the item
  const bf16 *x;
  bf16 *y;
  const float *w;
  int64_t x_h, y_h;      // to the next of its heads
};
struct Grid {  // items are (token, `each` heads of one kind), a token's query, key and value heads in a row
  int items, nq, nk;       // nq, nk: items of a token's queries, of its keys
  paged::FastDiv per_token, page;
};
template <int R>
__device__ __forceinline__ int find_item(const NormRopeArgs &a, const Grid &g, int64_t i, Item &t) {
  t.in = i < g.items;
  const int item = t.in ? (int)i : 0;
  t.n = (int)g.per_token.div((uint32_t)item);
  const int h = item - t.n * (int)g.per_token.d;
  const int kind = h < g.nq ? 0 : (h < g.nq + g.nk ? 1 : 2);
  const int hh = R * (kind == 0 ? h : (kind == 1 ? h - g.nq : h - g.nq - g.nk));
  t.plain = kind == 2;
  t.rows = min(R, (kind == 0 ? a.H : a.c.kv_heads) - hh);
  t.x_h = kind == 0 ? a.q_h : (kind == 1 ? a.k_h : a.v_h);
  t.x = (kind == 0 ? a.q + t.n * a.q_t : (kind == 1 ? a.k + t.n * a.k_t : a.v + t.n * a.v_t)) + hh * t.x_h;
  t.w = kind == 0 ? a.q_norm : (kind == 1 ? a.k_norm : nullptr);
  return h;
}
template <int R>
__device__ __forceinline__ void find_place(const NormRopeArgs &a, const Grid &g, int h, int lane, Item &t) {
  t.pos = a.pos[t.n];
  const int slot = a.slot ? a.slot[t.n] : t.n;
  t.live = t.in && t.pos >= 0;
  if (t.live && ((a.rd > 0 && t.pos >= a.tab_rows) || slot < -1 || slot >= a.c.n_pages * a.c.page)) {
    if (h == 0 && lane == 0) atomicOr(a.status, kStatusBadIndex);
    t.live = false;
  }
  if (h < g.nq) {
    t.y_h = a.o_h;
    t.y = a.q_out + t.n * a.o_t + R * h * a.o_h;
  } else {
    if (slot < 0) t.live = false;
    const int pg = t.live ? (int)g.page.div((uint32_t)slot) : 0, row = t.live ? slot - pg * a.c.page : 0;
    const int hk = R * (h - g.nq - (t.plain ? g.nk : 0));
    t.y_h = t.plain ? a.c.v_head : a.c.k_head;
    t.y = (t.plain ? reinterpret_cast<bf16 *>(a.c.v) + pg * a.c.v_page + row * a.c.v_row
                   : reinterpret_cast<bf16 *>(a.c.k) + pg * a.c.k_page + row * a.c.k_row) + hk * t.y_h;
  }
}

__device__ __forceinline__ void load8(const float *w, f2 (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float4 x = __ldg(reinterpret_cast<const float4 *>(w + 2 * e));
    v[e] = {x.x, x.y};
    v[e + 1] = {x.z, x.w};
  }
}

// G lanes a row, V (even) vectors of 8 features a lane, head_dim <= 8 G V a multiple of 16; the turned part and its halves
// start and end on vector borders.  Adjacent pairs lie inside a vector; with HALF vectors u and u + 1 (u even) of a lane are
// partners, rd / 2 features apart, or lie both outside the turned part.  R rows a group and no loop: what hides the
// latency is many resident warps, each with its rows in flight.  Two heads of a token take each weight and angle
// once (with one row they are twice the row's own bytes on their way from L1; 4096 x 64 x 512: 97 us, 8000 tokens of 48
// x 128 42.6 against 38.8 with adjacent pairs, 46.1 against 42.1 with halves); more rows, looped over with weights
// and angles in registers, needed 80 to 128 of them and took 113 us.
template <int G, int V, bool HALF, int R>
__global__ void __launch_bounds__(kThreads, kResident<V, HALF>) k_norm_rope(const __grid_constant__ NormRopeArgs a,
                                                                                const __grid_constant__ Grid g) {
  const int lane = threadIdx.x & (G - 1);
  const int hd = a.c.head_dim, h2 = a.rd >> 1;
  Item t;
  const int h = find_item<R>(a, g, ((int64_t)blockIdx.x * kThreads + threadIdx.x) / G, t);
  dependency_wait();
  int f[V];  // first feature of this lane's vectors (hd: none)
  uint4 x[R][V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    if (HALF) {
      const int j = lane + G * (u >> 1), turned = h2 >> 3;  // pair of vectors j
      if (j < turned) {
        f[u] = a.at + 8 * j + (u & 1) * h2;
      } else {
        const int v = 8 * (2 * (j - turned) + (u & 1));
        f[u] = v < a.at ? v : v + a.rd;
      }
    } else {
      f[u] = 8 * (lane + G * u);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      x[i][u] = make_uint4(0, 0, 0, 0);
      if (f[u] < hd && i < t.rows) x[i][u] = *reinterpret_cast<const uint4 *>(t.x + i * t.x_h + f[u]);
    }
  }
  find_place<R>(a, g, h, lane, t);
  f2 v[R][V][4];
  float r[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    f2 q[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int u = 0; u < V; ++u) {
      unpack(x[i][u], v[i][u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e & 1] = fma2(v[i][u][e], v[i][u][e], q[e & 1]);
    }
    r[i] = (q[0].x + q[0].y) + (q[1].x + q[1].y);
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < R; ++i) r[i] += __shfl_xor_sync(0xffffffffu, r[i], o);
  if (!t.live) return;
  if (t.plain) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (f[u] < hd && i < t.rows) *reinterpret_cast<uint4 *>(t.y + i * t.y_h + f[u]) = x[i][u];
    return;
  }
  if (t.w) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      r[i] = rsqrtf(r[i] / (float)hd + a.eps);  // (within 2 units of the last place: 2^-22, far below the result's 2^-8)
#pragma unroll
    for (int u = 0; u < V; ++u) {
      if (f[u] >= hd) continue;
      f2 w[4];
      load8(t.w + f[u], w);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][u][e] = mul2(mul2(v[i][u][e], f2{r[i], r[i]}), w[e]);
    }
  }
  const float2 *tp = reinterpret_cast<const float2 *>(a.tab) + (int64_t)t.pos * h2;
#pragma unroll
  for (int u = 0; u < V; u += HALF ? 2 : 1) {
    if (f[u] < a.at || f[u] >= a.at + a.rd) continue;
    if (HALF) {
      const float4 *ap = reinterpret_cast<const float4 *>(tp + (f[u] - a.at));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 cs = __ldg(ap + e);
        const f2 c = {cs.x, cs.z}, s = {cs.y, cs.w}, m = {-cs.y, -cs.w};
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const f2 lo = v[i][u][e], hi = v[i][u + 1][e];
          v[i][u][e] = fma2(hi, m, mul2(lo, c));
          v[i][u + 1][e] = fma2(lo, s, mul2(hi, c));
        }
      }
    } else {
      const float4 *ap = reinterpret_cast<const float4 *>(tp + ((f[u] - a.at) >> 1));
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float4 cs = __ldg(ap + e / 2);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const f2 y = v[i][u][e], z = v[i][u][e + 1];
          v[i][u][e] = fma2(f2{y.y, y.x}, f2{-cs.y, cs.y}, mul2(y, f2{cs.x, cs.x}));
          v[i][u][e + 1] = fma2(f2{z.y, z.x}, f2{-cs.w, cs.w}, mul2(z, f2{cs.z, cs.z}));
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (f[u] < hd && i < t.rows)
        *reinterpret_cast<uint4 *>(t.y + i * t.y_h + f[u]) =
            make_uint4(pack2(v[i][u][0]), pack2(v[i][u][1]), pack2(v[i][u][2]), pack2(v[i][u][3]));
}

// Any even turned part and alignment of weights and angles.  Adjacent pairs still lie inside a vector; halves meet through shared
// memory, where a row's normed features wait for their partners (one row a group, 11475 tokens of 56 x 80 with 4 features
// turned: 74 us; partners read from the row again, a feature at a time: 147).
template <int G, int V>
__global__ void __launch_bounds__(kThreads) k_norm_rope_any(const __grid_constant__ NormRopeArgs a,
                                                            const __grid_constant__ Grid g) {
  __shared__ __align__(16) float s_row[kThreads / G][8 * G * V];
  const int lane = threadIdx.x & (G - 1);
  const int hd = a.c.head_dim, h2 = a.rd >> 1;
  float *mine = s_row[threadIdx.x / G];
  Item t;
  const int h = find_item<1>(a, g, ((int64_t)blockIdx.x * kThreads + threadIdx.x) / G, t);
  dependency_wait();
  uint4 x[V];
  f2 v[V][4], q = {0.f, 0.f};
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int f = 8 * (lane + G * u);
    x[u] = f < hd ? *reinterpret_cast<const uint4 *>(t.x + f) : make_uint4(0, 0, 0, 0);
  }
  find_place<1>(a, g, h, lane, t);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    unpack(x[u], v[u]);
#pragma unroll
    for (int e = 0; e < 4; ++e) q = fma2(v[u][e], v[u][e], q);
  }
  float r = q.x + q.y;
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  if (t.w) {
    r = rsqrtf(r / (float)hd + a.eps);
    const bool whole = ((uintptr_t)t.w & 15) == 0;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int f = 8 * (lane + G * u);
      if (f >= hd) continue;
      f2 w[4];
      if (whole) {
        load8(t.w + f, w);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = {__ldg(t.w + f + 2 * e), __ldg(t.w + f + 2 * e + 1)};
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[u][e] = mul2(mul2(v[u][e], f2{r, r}), w[e]);
    }
  }
  const bool turn = t.live && !t.plain;
  const float2 *tp = reinterpret_cast<const float2 *>(a.tab) + (int64_t)(turn ? t.pos : 0) * h2;
  if (a.half) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      float4 *to = reinterpret_cast<float4 *>(mine + 8 * (lane + G * u));
      to[0] = make_float4(v[u][0].x, v[u][0].y, v[u][1].x, v[u][1].y);
      to[1] = make_float4(v[u][2].x, v[u][2].y, v[u][3].x, v[u][3].y);
    }
    __syncwarp();
  }
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int f = 8 * (lane + G * u);
    if (f >= hd || !t.live) continue;
    uint4 out = x[u];
    if (turn) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = f + 2 * e - a.at;  // (even, as `at` and rd are; rd / 2 may be odd)
        if (d < 0 || d >= a.rd) continue;
        if (a.half) {
          const bool lo = d < h2, lo1 = d + 1 < h2;
          const float2 c0 = __ldg(tp + (lo ? d : d - h2)), c1 = __ldg(tp + (lo1 ? d + 1 : d + 1 - h2));
          const float *p = mine + a.at + d;
          const float p0 = lo ? p[h2] : p[-h2], p1 = lo1 ? p[1 + h2] : p[1 - h2];
          v[u][e] = {fmaf(lo ? -p0 : p0, c0.y, v[u][e].x * c0.x), fmaf(lo1 ? -p1 : p1, c1.y, v[u][e].y * c1.x)};
        } else {
          const float2 cs = __ldg(tp + (d >> 1));
          const f2 y = v[u][e];
          v[u][e] = fma2(f2{y.y, y.x}, f2{-cs.y, cs.y}, mul2(y, f2{cs.x, cs.x}));
        }
      }
      out = make_uint4(pack2(v[u][0]), pack2(v[u][1]), pack2(v[u][2]), pack2(v[u][3]));
    }
    *reinterpret_cast<uint4 *>(t.y + f) = out;
  }
}

using Kernel = void (*)(NormRopeArgs, Grid);

cudaError_t launch(Kernel k, int G, int R, const NormRopeArgs &a, cudaStream_t s) {
  const int nq = (a.H + R - 1) / R, nk = (a.c.kv_heads + R - 1) / R, per_token = nq + nk * (a.v ? 2 : 1);
  const int64_t items = (int64_t)a.N * per_token;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;  // (refused by the entry)
  const Grid g{(int)items, nq, nk, paged::FastDiv((uint32_t)per_token), paged::FastDiv((uint32_t)a.c.page)};
  return launch_dependent(k, dim3((unsigned)((items * G + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, 1, a, g);
}
template <int G, int V, int R>
cudaError_t launch_vectors(const NormRopeArgs &a, cudaStream_t s) {
  return launch(a.half ? (Kernel)k_norm_rope<G, V, true, R> : (Kernel)k_norm_rope<G, V, false, R>, G, R, a, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t s) {
  const int hd = a.c.head_dim;
  // whole vectors: weights and angles 16-byte aligned, the turned part (and its halves) on vector borders
  const bool vectors = hd % 16 == 0 && a.at % 8 == 0 && a.rd % (a.half ? 16 : 8) == 0 &&
                       (((uintptr_t)a.tab | (uintptr_t)a.q_norm | (uintptr_t)a.k_norm) & 15) == 0;
  if (!vectors) {
    if (hd <= 64) return launch(k_norm_rope_any<4, 2>, 4, 1, a, s);
    if (hd <= 128) return launch(k_norm_rope_any<8, 2>, 8, 1, a, s);
    if (hd <= 256) return launch(k_norm_rope_any<16, 2>, 16, 1, a, s);
    return launch(hd <= 512 ? (Kernel)k_norm_rope_any<32, 2> : (Kernel)k_norm_rope_any<32, 4>, 32, 1, a, s);
  }
  if (hd <= 32) return launch_vectors<2, 2, 2>(a, s);
  if (hd <= 64) return launch_vectors<4, 2, 2>(a, s);
  if (hd <= 128) return launch_vectors<8, 2, 2>(a, s);
  if (hd <= 256) return launch_vectors<16, 2, 2>(a, s);
  if (hd <= 512) return launch_vectors<32, 2, 2>(a, s);
  return launch_vectors<32, 4, 1>(a, s);
}

}  // namespace csa
