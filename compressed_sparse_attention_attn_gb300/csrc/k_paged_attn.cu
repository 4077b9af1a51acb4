// k_paged_attn.cu -- attention of single tokens over a paged key-value cache (head_dim up to 256).
//
// Row n, query head h over kv head h / g: S_j = scale q_h . K_j over the positions j of its request, O = sum_j
// e^{S_j} V_j / (e^{sink} + sum_j e^{S_j}).  Up to 16 query heads of one kv head are the rows of an m16n8k16
// product, so a cache row is read once for all of them (a kv head with more query heads takes several head
// groups).  A decode step does 4 g flops a byte of cache: at g = 8 that is 54 TFLOP/s at the card's copy
// rate, far below what warp-level products give, and their accumulators stay in registers -- no trip
// through tensor memory between the scores and the values.
//
// A unit is 64 positions: 16 for each of a CTA's four warps.  Every warp streams its own tiles (16 key rows,
// 16 value rows) through a ring of its own in shared memory, with no barrier between the warps before the
// end of a segment; the ring runs on across segments.  Rows come by 16-byte cp.async from the page of each
// position (looked up one tile ahead), rows past the end and features past head_dim as zeros; chunks are
// XOR-swizzled by the row so that ldmatrix reads without conflicts.  Softmax statistics are f32 (base 2); the
// weights enter the second product as two bf16 terms (their sum carries 16 bits), so the only rounding that
// counts is the result's.  At the end of a segment each warp leaves its accumulators in the stage it has
// just read (exactly as large: 16 rows of keys and values in bf16 are 16 heads of f32), and the CTA joins the
// four.  How CTAs share the rows: paged_common.cuh.
#include <algorithm>
#include <cstring>

#include "attn_common.cuh"
#include "paged_common.cuh"

namespace csa {
namespace paged {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;               // positions of a warp's tile
constexpr int kUnit = kWarps * kTile;   // positions of a unit
constexpr int kHeads = 16;              // query heads of a head group

template <int HD>
struct Shape {
  static constexpr int kStages = 3;
  static constexpr int kStageBytes = 2 * kTile * HD * 2;          // key rows, value rows
  static constexpr int kCtas = HD == 64 ? 4 : (HD == 128 ? 2 : 1);  // resident an SM
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
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

// Where a CTA is in its range: segment (row n, head group hg), unit t of it.
struct Cursor {
  int n, hg, t;
  Row row;
};

template <int HD>
__global__ void __launch_bounds__(kThreads, Shape<HD>::kCtas) k_paged_attn(const __grid_constant__ Params P) {
  using S = Shape<HD>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[kWarps + 4];
  __shared__ float s_ml[2][kWarps][kHeads];
  __shared__ float s_f[kWarps][kHeads];
  __shared__ float s_join[kJoinFloats<kHeads>];
  __shared__ float s_out[2][kHeads];
  __shared__ int s_flag;
  const PagedAttnArgs &a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hd = a.c.head_dim;
  const Range rg = find_range<kUnit, kThreads>(P, s_scan);
  if (rg.begin >= rg.end) return;
  const int64_t nunits = rg.end - rg.begin;
  const uint32_t ring = tc::smem_u32(smem) + warp * (S::kStages * S::kStageBytes);
  uint8_t *ring_p = smem + warp * (S::kStages * S::kStageBytes);

  Cursor cl;  // of the copies
  cl.n = rg.row;
  cl.row = row_of<kUnit>(a, cl.n, false);
  {
    const int64_t in = rg.begin - rg.before;
    cl.hg = (int)(in / cl.row.units);
    cl.t = (int)(in - (int64_t)cl.hg * cl.row.units);
  }
  Cursor cc = cl;  // of the products
  auto advance = [&](Cursor &c) {
    if (++c.t < c.row.units) return;
    c.t = 0;
    if (++c.hg < P.Hg) return;
    c.hg = 0;
    do {
      ++c.n;
      if (c.n >= a.N) {
        c.row.units = 1;
        c.row.rows = 0;
        return;
      }
      c.row = row_of<kUnit>(a, c.n, false);
    } while (c.row.units == 0);
  };
  const bf16 *kbase = reinterpret_cast<const bf16 *>(a.c.k);
  const bf16 *vbase = a.c.v ? reinterpret_cast<const bf16 *>(a.c.v) : kbase;
  const int64_t v_page = a.c.v ? a.c.v_page : a.c.k_page, v_row = a.c.v ? a.c.v_row : a.c.k_row,
                v_head = a.c.v ? a.c.v_head : a.c.k_head;
  // lanes 0-15: the page of this lane's position of a tile (-1: no such position)
  auto lookup = [&](const Cursor &c, bool in) -> int {
    const int j = c.t * kUnit + warp * kTile + (lane & 15);
    if (!in || j >= c.row.rows) return -1;
    return a.table[(int64_t)c.row.req * a.width + P.page.div((uint32_t)(c.row.first + j))];
  };
  int64_t todo = nunits;  // units not yet copied
  int pid = lookup(cl, true);
  // Copy the cursor's tile into a stage; returns the mask of its positions that are there.
  auto issue = [&](int stage) -> uint32_t {
    uint32_t ok = 0;
    if (todo > 0) {
      const int j = cl.t * kUnit + warp * kTile + (lane & 15);
      const bool there = j < cl.row.rows, good = there && pid >= 0 && pid < a.c.n_pages;
      if (there && !good && lane < 16) atomicOr(a.status, kStatusBadIndex);
      ok = __ballot_sync(0xffffffffu, good) & 0xffffu;
      const uint32_t p = (uint32_t)(cl.row.first + j), r = p - P.page.div(p) * P.page.d;
      const int kvh = cl.hg / P.sub;
      const int64_t ko = good ? (int64_t)pid * a.c.k_page + (int64_t)r * a.c.k_row : -1;
      const int64_t vo = good ? (int64_t)pid * v_page + (int64_t)r * v_row : -1;
      const bf16 *kh = kbase + (int64_t)kvh * a.c.k_head, *vh = vbase + (int64_t)kvh * v_head;
      constexpr int CH = HD / 8;  // 16-byte chunks of a row
      const uint32_t st = ring + stage * S::kStageBytes;
      // rows of the tile that hold something (the others' weights are 0, but 0 x NaN is not: they are zeroed)
#pragma unroll
      for (int i = 0; i < kTile * CH / 32; ++i) {
        const int e = lane + 32 * i, row = e / CH, ch = e % CH;
        const int64_t k_off = __shfl_sync(0xffffffffu, ko, row), v_off = __shfl_sync(0xffffffffu, vo, row);
        const bool in = k_off >= 0 && ch * 8 < hd;
        const uint32_t dst = st + row * (HD * 2) + ((ch ^ (row & 7)) << 4);
        attn::cp_async16(dst, in ? kh + k_off + ch * 8 : kbase, in);
        attn::cp_async16(dst + kTile * HD * 2, in ? vh + v_off + ch * 8 : vbase, in);
      }
      --todo;
      advance(cl);
      pid = lookup(cl, todo > 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return ok;
  };

  uint32_t masks[S::kStages];  // of the tiles in flight, the oldest first
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) masks[i] = issue(i);

  uint32_t qf[HD / 16][4];
  float acc[HD / 8][4], m[2], l[2];
  int h0 = 0, nh = 0;
  int64_t seg = rg.begin;  // the CTA's first unit of the current segment
  const int qr = lane >> 2, qc = 2 * (lane & 3);
  auto begin_segment = [&]() {
    const int kvh = cc.hg / P.sub, sg = cc.hg - kvh * P.sub;
    h0 = kvh * P.g + sg * kHeads;
    nh = min(kHeads, P.g - sg * kHeads);
    const bf16 *q = a.q + (int64_t)cc.n * a.q_t + (int64_t)h0 * hd;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = qr + 8 * (e & 1), d = 16 * kk + qc + 8 * (e >> 1);
        qf[kk][e] = h < nh && d < hd ? *reinterpret_cast<const uint32_t *>(q + h * hd + d) : 0u;
      }
#pragma unroll
    for (int t = 0; t < HD / 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  };
  begin_segment();

  int stage = 0;
  for (int64_t u = rg.begin; u < rg.end; ++u) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
    __syncwarp();
    masks[S::kStages - 1] = issue((stage + S::kStages - 1) % S::kStages);
    const uint32_t ok = masks[0];
    const uint32_t sk = ring + stage * S::kStageBytes, sv = sk + kTile * HD * 2;
    if (ok) {
      // ---- scores of 16 heads x 16 positions
      float c[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[t][e] = 0.f;
      const int krow = (lane >> 4) * 8 + (lane & 7), kch = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        uint32_t b[4];
        ldsm4(b, sk + krow * (HD * 2) + (((2 * kk + kch) ^ (krow & 7)) << 4));
        mma16816(c[0], qf[kk], b[0], b[1]);
        mma16816(c[1], qf[kk], b[2], b[3]);
      }
      // ---- running maximum and sum (a head's 16 scores lie in the four lanes of a quad)
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * t + qc + (e & 1);
          c[t][e] = (ok >> j) & 1u ? c[t][e] * P.scale_log2 : -INFINITY;
          mx[e >> 1] = fmaxf(mx[e >> 1], c[t][e]);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f[i] = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mx[i]);
          l[i] *= f[i];
          m[i] = mx[i];
        }
#pragma unroll
        for (int t = 0; t < HD / 8; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][e] *= f[e >> 1];
      }
      uint32_t ph[4], pl[4];
      {
        const float r0 = m[0] == -INFINITY ? 0.f : m[0], r1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[t][e] = exp2f(c[t][e] - (e < 2 ? r0 : r1));
            l[e >> 1] += c[t][e];
          }
          split2(c[t][0], c[t][1], ph[2 * t], pl[2 * t]);
          split2(c[t][2], c[t][3], ph[2 * t + 1], pl[2 * t + 1]);
        }
      }
      // ---- weighted values
      const int vrow = lane & 15, vch = lane >> 4;
#pragma unroll
      for (int t = 0; t < HD / 16; ++t) {
        uint32_t b[4];
        ldsm4_t(b, sv + vrow * (HD * 2) + (((2 * t + vch) ^ (vrow & 7)) << 4));
        mma16816(acc[2 * t], ph, b[0], b[1]);
        mma16816(acc[2 * t + 1], ph, b[2], b[3]);
        mma16816(acc[2 * t], pl, b[0], b[1]);
        mma16816(acc[2 * t + 1], pl, b[2], b[3]);
      }
    }
    const bool last = cc.t == cc.row.units - 1;
    if (last || u + 1 == rg.end) {
      // ---- the segment's end in this CTA: the four warps' accumulators joined
      float *mine = reinterpret_cast<float *>(ring_p + stage * S::kStageBytes);
      __syncwarp();
#pragma unroll
      for (int t = 0; t < HD / 8; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = qr + 8 * i;
          *reinterpret_cast<float2 *>(mine + h * HD + ((8 * t + qc) ^ ((h & 3) << 3))) = make_float2(acc[t][2 * i], acc[t][2 * i + 1]);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if ((lane & 3) == 0) {
          s_ml[0][warp][qr + 8 * i] = m[i];
          s_ml[1][warp][qr + 8 * i] = l[i];
        }
      }
      __syncthreads();
      const int64_t sb = u - cc.t, se = sb + cc.row.units;  // the whole segment
      const bool whole = sb >= rg.begin && se <= rg.end;
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
          s_out[0][tid] = out_factor(M, L, a.sink, h0 + tid);
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
          const float4 x = *reinterpret_cast<const float4 *>(src + h * HD + (d ^ ((h & 3) << 3)));
          const float f = s_f[w][h];
          v.x = fmaf(x.x, f, v.x);
          v.y = fmaf(x.y, f, v.y);
          v.z = fmaf(x.z, f, v.z);
          v.w = fmaf(x.w, f, v.w);
        }
        if (whole) {
          const float f = s_out[0][h];
          *reinterpret_cast<uint2 *>(a.o + (int64_t)cc.n * a.o_t + (int64_t)(h0 + h) * hd + d) =
              make_uint2(bits(__floats2bfloat162_rn(v.x * f, v.y * f)), bits(__floats2bfloat162_rn(v.z * f, v.w * f)));
        } else {
          *reinterpret_cast<float4 *>(P.share_o + ((int64_t)slot * kHeads + h) * HD + d) = v;
        }
      }
      __syncthreads();  // the stage may be refilled
      if (!whole) publish<kHeads, HD, kThreads, 0>(P, tid, sb, se, rg, cc.n, h0, nh, s_join, &s_flag);
      if (u + 1 < rg.end) {
        advance(cc);
        seg = u + 1;
        begin_segment();
      }
    } else {
      ++cc.t;
    }
#pragma unroll
    for (int i = 0; i + 1 < S::kStages; ++i) masks[i] = masks[i + 1];
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int HD>
cudaError_t launch(Params p, float *ws, size_t ws_bytes, int num_sms, cudaStream_t s) {
  using S = Shape<HD>;
  static SmemAttr attr;
  cudaError_t e = attr.ensure((const void *)k_paged_attn<HD>, S::kSmem);
  if (e != cudaSuccess) return e;
  const PagedAttnArgs &a = p.a;
  p.g = a.H / a.c.kv_heads;
  p.sub = (p.g + kHeads - 1) / kHeads;
  p.Hg = p.sub * a.c.kv_heads;
  // no more CTAs than there can be units
  const int64_t rows = a.window > 0 ? std::min<int64_t>(a.window, (int64_t)a.width * a.c.page) : (int64_t)a.width * a.c.page;
  const int64_t units = (int64_t)a.N * p.Hg * std::max<int64_t>(1, (rows + kUnit - 1) / kUnit);
  const int64_t grid = std::min<int64_t>(std::min(units, (int64_t)num_sms * S::kCtas), kMaxCtas);
  p.share_o = ws;
  p.share_ml = ws + 2 * grid * kHeads * HD;
  if (sizeof(float) * 2 * grid * kHeads * (HD + 2) > ws_bytes) return cudaErrorInvalidValue;
  k_paged_attn<HD><<<(unsigned)grid, kThreads, S::kSmem, s>>>(p);
  return cudaGetLastError();
}

// (head_dim above 256: k_paged_attn_tc.cu)
cudaError_t launch_latent(Params p, float *ws, size_t ws_bytes, int num_sms, cudaStream_t s);

}  // namespace paged

cudaError_t launch_paged_attn(const PagedAttnArgs &a, float *ws, size_t ws_bytes, int *counters, int num_sms,
                              cudaStream_t s) {
  static_assert(kPagedCounters == 3 * paged::kMaxCtas, "the context's counters");
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
