// k_paged_attn.cu -- attention of single tokens over a paged key-value cache (head_dim up to 256).
//
// Row n, query head h over kv head h / g: S_j = scale q_h . K_j over the positions j of its request, O = sum_j
// e^{S_j} V_j / (e^{sink} + sum_j e^{S_j}).  Up to 16 query heads of one kv head are the rows (up to 8: the columns) of an m16n8k16
// product, so a cache row is read once for all of them (a kv head with more query heads takes several head
// groups).  A decode step does 4 g flops a byte of cache: at g = 8 that is 54 TFLOP/s at the card's copy
// rate, far below what warp-level products give, and their accumulators stay in registers -- no trip
// through tensor memory between the scores and the values.
//
// A unit is 16 positions for each of a CTA's warps (four; at 256 features three, or six with more than eight heads a kv head).  Every warp streams its own tiles (16 key rows,
// 16 value rows) through a ring of its own in shared memory, with no barrier between the warps before the
// end of a segment; the ring runs on across segments.  Rows come by 16-byte cp.async from the page of each
// position (looked up two tiles ahead), rows past the end and features past head_dim as zeros; chunks are
// XOR-swizzled by the row so that ldmatrix reads without conflicts.  Softmax statistics are f32 (base 2); the
// weights enter the second product as two bf16 terms (their sum carries 16 bits), so the only rounding that
// counts is the result's.  At the end of a segment each warp leaves its accumulators in the stage it has
// just read (exactly as large: 16 rows of keys and values in bf16 are 16 heads of f32), and the CTA joins them.  How CTAs share the rows: paged_common.cuh.
//
// Bound by HBM: 4 rows of 50 to 65 thousand (64 heads over 8 of 128) 150 us, 94 % of a copy; 32 rows of 300 to 4000 (32 over 8 of
// 128) 37 us, 77 %; 48 windows of up to 1000 (16 of 256) 53 us, 79 %: what is left is the start and the segments' ends.
#include <algorithm>
#include <cstring>

#include "attn_common.cuh"
#include "paged_common.cuh"

namespace csa {
namespace paged {

constexpr int kTile = 16;  // positions of a warp's tile
constexpr int kEnd = 1;    // units that the end of a segment counts for (2 to 4 thousand cycles, as one unit takes)

// Warps and ring stages are set so that the rings fill an SM's shared memory and 64 to 128 KB are in flight: 4 x 3 x 4 KB
// x 4 (or 3) CTAs at 64 features, 4 x 2 x 8 KB x 3 (x 3 x 8 KB x 2 where 16 heads' accumulators need the
// registers) at 128, 3 x 2 x 16 KB x 2 at 256 (one CTA of 6: 83 against 74 us over 48 windows of 16 heads, whose segments end
// every few units), 6 x 2 x 16 KB x 1 with 16 heads (two CTAs of 3 spill: 90 against 47 us over 16 rows of 32 x 256).
template <int HD, int NH>
struct Shape {
  static constexpr int kWarps = HD == 256 ? (NH == 8 ? 3 : 6) : 4;
  static constexpr int kStages = HD == 256 || (HD == 128 && NH == 8) ? 2 : 3;
  static constexpr int kCtas = HD == 64 ? (NH == 8 ? 4 : 3) : (HD == 128 ? (NH == 8 ? 3 : 2) : NH == 8 ? 2 : 1);  // resident an SM
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kUnit = kWarps * kTile;            // positions of a unit
  static constexpr int kStageBytes = 2 * kTile * HD * 2;  // key rows, value rows
  // q as fragments in registers, but in shared memory where its 64 registers and 128 of accumulators are too many
  static constexpr bool kQShared = HD == 256 && NH == 16;
  static constexpr int kQAt = kWarps * kStages * kStageBytes, kSmem = kQAt + (kQShared ? NH * HD * 2 : 0);
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit values, a row in the four lanes of a quad.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t *>(&v); }
// (hi, lo): two values as bf16 and what the rounding left, as bf16
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  hi = bits(h);
  lo = bits(__floats2bfloat162_rn(x - __low2float(h), y - __high2float(h)));
}

// Where a thread's values of a 16-bit or f32 fragment lie in a row of a segment's accumulators in shared memory.
template <int NH>
__device__ __forceinline__ int swizzle(int h) {
  return (NH == 8 ? (h >> 1) & 3 : h & 3) << 3;
}

template <int HD, int NH>
__global__ void __launch_bounds__((Shape<HD, NH>::kThreads), (Shape<HD, NH>::kCtas)) k_paged_attn(const __grid_constant__ Params P) {
  using S = Shape<HD, NH>;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kUnit = S::kUnit, kHeads = NH;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Two s_scan[kWarps];
  __shared__ float s_ml[2][kWarps][kHeads];
  __shared__ float s_f[kWarps][kHeads];
  __shared__ float s_out[kHeads];
  __shared__ int s_flag;
  const PagedAttnArgs &a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hd = a.c.head_dim;
  __shared__ Rows rows;
  __shared__ Range rg;
  dependency_wait();
  const int nunits = find_range<kUnit, kThreads, false, kEnd, false>(P, s_scan, rows, rg);
  if (nunits <= 0) return;
  const uint32_t ring = tc::smem_u32(smem) + warp * (S::kStages * S::kStageBytes);
  uint8_t *ring_p = smem + warp * (S::kStages * S::kStageBytes);
  Cursor cl = first_unit<kUnit, false, kEnd>(a, P.Hg, rg, rows), cc = cl;  // of the lookups, of the products
  const bf16 *kbase = reinterpret_cast<const bf16 *>(a.c.k);
  const bf16 *vbase = a.c.v ? reinterpret_cast<const bf16 *>(a.c.v) : kbase;
  const int64_t v_page = a.c.v ? a.c.v_page : a.c.k_page, v_row = a.c.v ? a.c.v_row : a.c.k_row,
                v_head = a.c.v ? a.c.v_head : a.c.k_head;
  // Two tiles ahead of the copies: the page of this lane's position (the tables' latency passes while the tiles before are
  // copied).  pos -1: no such position.
  struct Found {
    int page, pos, kvh;
  };
  int todo = nunits;  // units not yet looked up
  auto lookup = [&]() -> Found {
    Found f{0, -1, -1};
    if (todo > 0) {
      const uint32_t j = (uint32_t)cl.t * kUnit + warp * kTile + (lane & (kTile - 1));
      f.kvh = cl.hg / P.sub;
      const Row row = rows.get<kUnit, false>(a, cl.n);
      if (j < (uint32_t)row.rows) {
        f.pos = row.first + (int)j;
        f.page = a.table[(int64_t)row.req * a.width + P.page.div((uint32_t)f.pos)];
      }
      --todo;
      const int hg0 = cl.hg, n0 = cl.n;
      advance<kUnit, false, kEnd>(a, P.Hg, rows, cl);
      if (warp == 0 && todo > 0 && (cl.hg != hg0 || cl.n != n0)) {  // the next segment's q on its way to L1
        const int kv2 = cl.hg / P.sub, sg = cl.hg - kv2 * P.sub, nq = min(NH, P.g - sg * NH);
        const bf16 *q = a.q + (int64_t)cl.n * a.q_t + (int64_t)(kv2 * P.g + sg * NH) * hd;
        for (int i = lane * 64; i < nq * hd; i += 32 * 64) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + i));
      }
    }
    return f;
  };
  constexpr uint32_t kAll = (1u << kTile) - 1;
  Found f0 = lookup(), f1 = lookup();
  // Copy the tile looked up first into a stage; returns the mask of its positions that are there.
  auto issue = [&](int stage) -> uint32_t {
    uint32_t ok = 0;
    const Found f = f0;
    f0 = f1;
    f1 = lookup();
    if (f.kvh >= 0) {
      const bool there = f.pos >= 0, good = there && f.page >= 0 && f.page < a.c.n_pages;
      if (there && !good && lane < kTile) atomicOr(a.status, kStatusBadIndex);
      ok = __ballot_sync(0xffffffffu, good) & kAll;
      const uint32_t p = (uint32_t)f.pos, r = p - P.page.div(p) * P.page.d;
      const int64_t ko = good ? (int64_t)f.page * a.c.k_page + (int64_t)r * a.c.k_row : -1;
      const int64_t vo = good ? (int64_t)f.page * v_page + (int64_t)r * v_row : -1;
      const bf16 *kh = kbase + (int64_t)f.kvh * a.c.k_head, *vh = vbase + (int64_t)f.kvh * v_head;
      // Eight lanes a row, four rows at a time, 128 bytes of a row at a time (its further parts one constant apart).  Rows
      // that are not there as zeros: their weights are 0, but 0 x NaN is not.
      const int ch = lane & 7, r0 = lane >> 3;
      const uint32_t st = ring + stage * S::kStageBytes + r0 * (HD * 2);
#pragma unroll
      for (int i = 0; i < kTile / 4; ++i) {
        const int row = r0 + 4 * i;
        const int64_t k_off = __shfl_sync(0xffffffffu, ko, row), v_off = __shfl_sync(0xffffffffu, vo, row);
        const bool in = k_off >= 0;
        const bf16 *ks = in ? kh + k_off + ch * 8 : kbase, *vs = in ? vh + v_off + ch * 8 : vbase;
        const uint32_t dst = st + i * (4 * HD * 2) + ((ch ^ (row & 7)) << 4);
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
          const bool f_in = in && ch * 8 + c * 64 < hd;
          attn::cp_async16(dst + c * 128, f_in ? ks + c * 64 : kbase, f_in);
          attn::cp_async16(dst + c * 128 + kTile * HD * 2, f_in ? vs + c * 64 : vbase, f_in);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return ok;
  };

  // NH 16: heads are the rows of both products (q and the weights their first operands).  NH 8: positions are the
  // rows of the first product, features of the second, and the heads the columns of both: half the products,
  // exponentials and registers where a kv head has no more than eight query heads.
  constexpr int QR = NH == 16 ? 4 : 2, AT = NH == 16 ? HD / 8 : HD / 16;
  uint32_t qf[S::kQShared ? 1 : HD / 16][QR];
  float acc[AT][4], m[2], l[2];  // m, l: of heads qr, qr + 8 (NH 16) or qc, qc + 1 (NH 8); l of this thread's positions
  int h0 = 0, nh = 0;
  int seg = 0;  // the CTA's first unit of the current segment
  const int qr = lane >> 2, qc = 2 * (lane & 3);
  auto begin_segment = [&]() {
    const int kvh = cc.hg / P.sub, sg = cc.hg - kvh * P.sub;
    h0 = kvh * P.g + sg * kHeads;
    nh = min(kHeads, P.g - sg * kHeads);
    const bf16 *q = a.q + (int64_t)cc.n * a.q_t + (int64_t)h0 * hd;
    if constexpr (S::kQShared) {  // (between two barriers: the one before this, and this one)
      for (int i = tid; i < NH * (HD / 8); i += kThreads) {
        const int h = i / (HD / 8), ch = i % (HD / 8);
        const uint4 x = h < nh && ch * 8 < hd ? *reinterpret_cast<const uint4 *>(q + h * hd + ch * 8) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(smem + S::kQAt + h * (HD * 2) + ((ch ^ (h & 7)) << 4)) = x;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
        for (int e = 0; e < QR; ++e) {
          const int h = NH == 16 ? qr + 8 * (e & 1) : qr, d = 16 * kk + qc + 8 * (NH == 16 ? e >> 1 : e);
          qf[kk][e] = h < nh && d < hd ? *reinterpret_cast<const uint32_t *>(q + h * hd + d) : 0u;
        }
    }
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  };
  begin_segment();

  uint32_t masks[S::kStages] = {};  // of the tiles in flight, the oldest first
  int stage = 1;  // of unit u, which goes around the ring with u
  for (int u = 1 - S::kStages; u < nunits; ++u) {  // (the first rounds only fill the ring)
    if (u >= 0) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
      __syncwarp();
    }
    masks[S::kStages - 1] = issue(stage == 0 ? S::kStages - 1 : stage - 1);
    const uint32_t ok = masks[0];
    const uint32_t sk = ring + stage * S::kStageBytes, sv = sk + kTile * HD * 2;
    if (u >= 0 && ok) {
      // ---- scores: c[t][e], of the head with statistics si(e)
      constexpr int NT = NH == 16 ? 2 : 1;
      float c[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[t][e] = 0.f;
      const int krow = NH == 16 ? (lane >> 4) * 8 + (lane & 7) : lane & 15, kch = NH == 16 ? (lane >> 3) & 1 : lane >> 4;
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        uint32_t b[4];
        ldsm4(b, sk + krow * (HD * 2) + (((2 * kk + kch) ^ (krow & 7)) << 4));
        if constexpr (S::kQShared) {
          uint32_t qa[4];
          ldsm4(qa, tc::smem_u32(smem) + S::kQAt + (lane & 15) * (HD * 2) + (((2 * kk + (lane >> 4)) ^ (lane & 7)) << 4));
          mma16816(c[0], qa, b[0], b[1]);
          mma16816(c[1], qa, b[2], b[3]);
        } else if constexpr (NH == 16) {
          mma16816(c[0], qf[kk], b[0], b[1]);
          mma16816(c[1], qf[kk], b[2], b[3]);
        } else {
          mma16816(c[0], b, qf[kk][0], qf[kk][1]);
        }
      }
      auto si = [](int e) { return NH == 16 ? e >> 1 : e & 1; };
      // ---- running maxima and sums (NH 16: a head's scores lie in the four lanes of a quad; NH 8: in every fourth lane)
      float mx[2] = {m[0], m[1]};
      if (ok == kAll) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[t][e] *= P.scale_log2;
            mx[si(e)] = fmaxf(mx[si(e)], c[t][e]);
          }
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = NH == 16 ? 8 * t + qc + (e & 1) : qr + 8 * (e >> 1);
            c[t][e] = (ok >> j) & 1u ? c[t][e] * P.scale_log2 : -INFINITY;
            mx[si(e)] = fmaxf(mx[si(e)], c[t][e]);
          }
      }
#pragma unroll
      for (int o = NH == 16 ? 1 : 4; o < (NH == 16 ? 4 : 32); o <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f[i] = m[i] == -INFINITY ? 0.f : ex2(m[i] - mx[i]);
          l[i] *= f[i];
          m[i] = mx[i];
        }
#pragma unroll
        for (int t = 0; t < AT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][e] *= f[si(e)];
      }
      const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
      uint32_t ph[2 * NT], pl[2 * NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[t][e] = ex2(c[t][e] - ref[si(e)]);
          l[si(e)] += c[t][e];
        }
        split2(c[t][0], c[t][1], ph[2 * t], pl[2 * t]);
        split2(c[t][2], c[t][3], ph[2 * t + 1], pl[2 * t + 1]);
      }
      // ---- weighted values
      const int vrow = NH == 16 ? lane & 15 : (lane >> 4) * 8 + (lane & 7), vch = NH == 16 ? lane >> 4 : (lane >> 3) & 1;
      if constexpr (NH == 8) {
#pragma unroll
        for (int t = 0; t < 2 * NT; ++t) {
          ph[t] = transpose8(ph[t]);
          pl[t] = transpose8(pl[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < HD / 16; ++t) {
        uint32_t b[4];
        ldsm4_t(b, sv + vrow * (HD * 2) + (((2 * t + vch) ^ (vrow & 7)) << 4));
        if constexpr (NH == 16) {
          mma16816(acc[2 * t], ph, b[0], b[1]);
          mma16816(acc[2 * t + 1], ph, b[2], b[3]);
          mma16816(acc[2 * t], pl, b[0], b[1]);
          mma16816(acc[2 * t + 1], pl, b[2], b[3]);
        } else {
          mma16816(acc[t], b, ph[0], ph[1]);
          mma16816(acc[t], b, pl[0], pl[1]);
        }
      }
    }
    if (u >= 0 && (cc.t == cc.units - 1 || u + 1 == nunits)) {
      // ---- the segment's end in this CTA: the warps' accumulators joined
      float *mine = reinterpret_cast<float *>(ring_p + stage * S::kStageBytes);
      __syncwarp();
#pragma unroll
      for (int t = 0; t < AT; ++t) {
        if constexpr (NH == 16) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int h = qr + 8 * i;
            *reinterpret_cast<float2 *>(mine + h * HD + ((8 * t + qc) ^ swizzle<NH>(h))) = make_float2(acc[t][2 * i], acc[t][2 * i + 1]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = qc + (e & 1), d = 16 * t + qr + 8 * (e >> 1);
            mine[h * HD + (d ^ swizzle<NH>(h))] = acc[t][e];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = NH == 16 ? 1 : 4; o < (NH == 16 ? 4 : 32); o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        if (NH == 16 ? (lane & 3) == 0 : lane < 4) {
          s_ml[0][warp][NH == 16 ? qr + 8 * i : qc + i] = m[i];
          s_ml[1][warp][NH == 16 ? qr + 8 * i : qc + i] = l[i];
        }
      }
      __syncthreads();
      const int sb = u - cc.t, se = sb + cc.units;  // the whole segment, from this CTA's first unit
      const bool whole = sb >= 0 && se <= nunits;
      const int slot = 2 * blockIdx.x + (seg == sb ? 1 : 0);
      if (tid < nh) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[0][w][tid]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = s_ml[0][w][tid] == -INFINITY ? 0.f : exp2f(s_ml[0][w][tid] - M);
          s_f[w][tid] = f;
          L = fmaf(s_ml[1][w][tid], f, L);
        }
        if (whole) {
          s_out[tid] = out_factor(M, L, a.sink, h0 + tid);
          if (a.lse) a.lse[(int64_t)cc.n * a.H + h0 + tid] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float2 *>(P.share_ml + ((int64_t)slot * kHeads + tid) * 2) = make_float2(M, L);
        }
      }
      __syncthreads();
      for (int i = tid; i < nh * (HD / 4); i += kThreads) {
        const int h = i / (HD / 4), d = (i % (HD / 4)) * 4;
        if (d >= hd) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float *src = reinterpret_cast<const float *>(smem + w * (S::kStages * S::kStageBytes) + stage * S::kStageBytes);
          const float4 x = *reinterpret_cast<const float4 *>(src + h * HD + (d ^ swizzle<NH>(h)));
          const float f = s_f[w][h];
          v.x = fmaf(x.x, f, v.x);
          v.y = fmaf(x.y, f, v.y);
          v.z = fmaf(x.z, f, v.z);
          v.w = fmaf(x.w, f, v.w);
        }
        if (whole) {
          const float f = s_out[h];
          *reinterpret_cast<uint2 *>(a.o + (int64_t)cc.n * a.o_t + (int64_t)(h0 + h) * hd + d) =
              make_uint2(bits(__floats2bfloat162_rn(v.x * f, v.y * f)), bits(__floats2bfloat162_rn(v.z * f, v.w * f)));
        } else {
          *reinterpret_cast<float4 *>(P.share_o + ((int64_t)slot * kHeads + h) * HD + d) = v;
        }
      }
      __syncthreads();  // the stage may be refilled
      if (!whole) {
        int c0;
        const int parts = sharers(rg, cc, c0);
        publish<kHeads, HD, kThreads>(P, c0, parts, cc.n, h0, nh, &s_flag);
      }
      if (u + 1 < nunits) {
        advance<kUnit, false, kEnd>(a, P.Hg, rows, cc);
        seg = u + 1;
        begin_segment();
      }
    } else if (u >= 0) {
      ++cc.t;
    }
#pragma unroll
    for (int i = 0; i + 1 < S::kStages; ++i) masks[i] = masks[i + 1];
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int HD, int NH>
cudaError_t launch_heads(Params p, float *ws, size_t ws_bytes, int num_sms, cudaStream_t s) {
  using S = Shape<HD, NH>;
  static SmemAttr attr;
  cudaError_t e = attr.ensure((const void *)k_paged_attn<HD, NH>, S::kSmem);
  if (e != cudaSuccess) return e;
  const PagedAttnArgs &a = p.a;
  p.sub = (p.g + NH - 1) / NH;
  p.Hg = p.sub * a.c.kv_heads;
  // no more CTAs than there can be units
  const int64_t rows = a.window > 0 ? std::min<int64_t>(a.window, (int64_t)a.width * a.c.page) : (int64_t)a.width * a.c.page;
  const int64_t units = (int64_t)a.N * p.Hg * std::max<int64_t>(1, (rows + S::kUnit - 1) / S::kUnit);
  const int64_t grid = std::min<int64_t>(std::min(units, (int64_t)num_sms * S::kCtas), kMaxCtas);
  p.share_o = ws;
  p.share_ml = ws + 2 * grid * NH * HD;
  if (sizeof(float) * 2 * grid * NH * (HD + 2) > ws_bytes) return cudaErrorInvalidValue;
  return launch_dependent(k_paged_attn<HD, NH>, dim3((unsigned)grid), dim3(S::kThreads), S::kSmem, s, 1, p);
}
template <int HD>
cudaError_t launch(Params p, float *ws, size_t ws_bytes, int num_sms, cudaStream_t s) {
  p.g = p.a.H / p.a.c.kv_heads;
  return p.g <= 8 ? launch_heads<HD, 8>(p, ws, ws_bytes, num_sms, s) : launch_heads<HD, 16>(p, ws, ws_bytes, num_sms, s);
}

// (head_dim above 256: k_paged_attn_tc.cu)
cudaError_t launch_latent(Params p, float *ws, size_t ws_bytes, int num_sms, cudaStream_t s);

}  // namespace paged

cudaError_t launch_paged_attn(const PagedAttnArgs &a, float *ws, size_t ws_bytes, int *counters, int num_sms,
                              cudaStream_t s) {
  static_assert(kPagedCounters == 3 * 2 * paged::kMaxCtas && paged::kJoin * paged::kJoin * paged::kJoin >= paged::kMaxCtas, "the context's counters");
  paged::Params p;
  p.a = a;
  p.page = paged::FastDiv((uint32_t)a.c.page);
  p.scale_log2 = (float)(a.scale * 1.4426950408889634);
  p.counters = counters;
  const int hd = a.c.head_dim;
  if (hd <= 64) return paged::launch<64>(p, ws, ws_bytes, num_sms, s);
  if (hd <= 128) return paged::launch<128>(p, ws, ws_bytes, num_sms, s);
  if (hd <= 256) return paged::launch<256>(p, ws, ws_bytes, num_sms, s);
  return paged::launch_latent(p, ws, ws_bytes, num_sms, s);
}

}  // namespace csa
