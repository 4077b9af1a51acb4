// k_paged_attn_tc.cu -- attention of single tokens over a paged cache of latent rows (head_dim above 256, the key
// rows are the values) on the 5th-generation tensor cores.
//
// Up to 64 query heads share a row of 512 features that is key and value: 4 x 64 x 512 flops for 1 KB, 860
// TFLOP/s at the card's copy rate, which warp-level products do not reach.  A CTA an SM works through its
// range of 48-position tiles (paged_common.cuh), the accumulators in tensor memory:
//   S[h][r] = sum_d q[h][d] K[r][d]       M = 64 heads (the first 16 lanes of each quarter), N = 48 positions, K = 512
//   p = exp2(S scale - m), bf16           a quad of lanes a head: the running maximum m and the sum stay in their registers;
//                                         m is raised only by more than 2^8 (the sums so far are then rescaled)
//   O^T[d][h] += sum_r K[r][d] p[h][r]    M = 4 x 128 features, N = 64 heads, K = 48 positions (the same tile read
//                                         as an MN-major operand)
// p is rounded to bf16, by at most 2^-8 of itself: a second term for what the rounding leaves would double the products of
// the values, and its tiles do not fit beside q and three tiles of rows.  O's denominator adds up the rounded
// p, so that its weights still add up to 1 (with the sink's): O moves by at most 2^-8 sum_r w_r |K_rd - O_d|, and a feature
// that all rows share by nothing.  lse is of the p as they were.  Scores, maxima, sums and O are f32.
//
// Shared memory holds q (64 KB) and three tiles (48 KB each): one whose values are used, one whose scores are, one in flight
// (two of 64 positions took 217 against 182 us over 64 rows of 12 to 16 thousand).  Tiles come by TMA, boxes of up to 16 rows inside
// a page, where pages hold whole boxes of 8 rows at least, else by cp.async from the page of each position.  One thread issues
// whichever product is ready first, the next tile's scores or this tile's values, so a buffer is handed back
// as soon as its weights are there.  Four warps do the softmax, and load the next segment's q behind the last
// scores that read it; four rescale O and write it out.  All waits are time-bounded.
//
// 64 x 1 over 12 to 16 thousand rows: 176 us, 5.3 TB/s (79 % of a copy); of the 2550 cycles that an SM is active for each of its
// 124 tiles, the segments' ends among them, the products take 1300, and most of the rest is what their hand-overs take:
// scores to softmax to values.  32 x 1 over about 900 rows (4 tiles a CTA): 20 us, of which the shares' 128 KB a CTA take 2 us to
// write and 5 us to join.
#include <algorithm>
#include <cstring>

#include "attn_common.cuh"
#include "paged_common.cuh"

namespace csa {

// 4-D bf16 tensor map with 128-byte swizzle, boxes {box_inner, 1, box_rows, 1} (defined with the GEMM's TMA helpers).
bool tma_map_pages_bf16(CUtensorMap *m, const void *base, const uint64_t (&dims)[4], const uint64_t (&strides)[3], uint32_t box_inner,
                        uint32_t box_rows);

namespace paged {
namespace latent {

constexpr int kHD = 512;
constexpr int kHeads = 64;              // query heads of a head group
constexpr int kUnit = 48;               // positions of a tile
constexpr int kEnd = 2;                 // tiles that the end of a segment counts for (its share takes 2 us to write)
constexpr int kJ = kUnit / 8;
constexpr int kBufs = 3;                // tile buffers
constexpr int kBlock = kUnit * 128;     // bytes of a 64-feature block of a tile
constexpr int kQBlock = kHeads * 128;   // and of q
constexpr int kS = 64;                  // columns of a score accumulator (kUnit used)
constexpr uint32_t kHalf = 0xffffffu;   // the positions of half a tile
constexpr int kBlocks = kHD / 64;
// warps 0-3 softmax; 4-7 O; 8 products; from 9 on copies: by TMA (four, a quarter of the features each) or by cp.async (two
// for each tile buffer)
constexpr int kFirstCopy = 9;
template <bool TMA>
constexpr int kThreads = (kFirstCopy + (TMA ? 4 : 2 * kBufs)) * 32;

struct L {
  static constexpr size_t q = 0;                                             // [8][64][128 B]
  static constexpr size_t t = q + (size_t)kBlocks * kQBlock;                 // [3][8][48][128 B]
  static constexpr size_t p = t + (size_t)kBufs * kBlocks * kBlock;          // [2][64][128 B]
  static constexpr size_t alpha = p + (size_t)2 * kHeads * 128;              // float [2][64]
  static constexpr size_t f = alpha + 2 * kHeads * 4;                        // float [2][64]
  static constexpr size_t scan = f + 2 * kHeads * 4;                         // Two [16]
  static constexpr size_t range = scan + 16 * 8;                             // Range
  static constexpr size_t rows = range + ((sizeof(Range) + 7) & ~7);         // Rows
  static constexpr size_t bars = rows + ((sizeof(Rows) + 7) & ~7);           // u64 [16]
  static constexpr size_t misc = bars + 16 * 8;                              // masks [3][2], flags [2][4], slot, abort
  static constexpr size_t total = misc + 96;
};
static_assert(L::total <= 232448, "one CTA's shared memory");

// Every lane waits (each acquires what the barrier publishes); the warp goes on only if all succeeded.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  const bool ok = tc::mbar_wait(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}
// What a CTA's copies need beyond the parameters (TMA): the map of the pages [page][row][kv head][feature], boxes of
// box_rows rows x 64 features inside a page, a power of two that divides `page`.
struct Pages {
  CUtensorMap map;
  int box_rows;
};

template <bool TMA>
__global__ void __launch_bounds__(kThreads<TMA>, 1) k_paged_attn_latent(const __grid_constant__ Params P,
                                                                        const __grid_constant__ Pages PG) {
  constexpr bool ALIGN = TMA;  // (tiles then hold whole boxes)
  extern __shared__ __align__(1024) uint8_t smem[];  // (all of the kernel's shared memory: the swizzled tiles come first)
  const uint32_t s_q = tc::smem_u32(smem + L::q), s_t = tc::smem_u32(smem + L::t), s_p = tc::smem_u32(smem + L::p);
  float *alpha_sm = reinterpret_cast<float *>(smem + L::alpha), *f_sm = reinterpret_cast<float *>(smem + L::f);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bars);
  // full, empty [3]: a tile has landed, has been used
  uint64_t *full = bars, *empty = bars + kBufs, *s_full = bars + 2 * kBufs, *p_full = s_full + 2, *stat = s_full + 4,
           *fin = s_full + 6, *q_full = s_full + 8, *drain = s_full + 9;
  uint32_t *masks = reinterpret_cast<uint32_t *>(smem + L::misc);  // [3][2]: positions of a tile that are there (24 each)
  int *flags = reinterpret_cast<int *>(masks + 2 * kBufs);         // [2][4]: a maximum was raised (by warp)
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(flags + 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const PagedAttnArgs &a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hd = a.c.head_dim;
  const int nkb = (hd + 63) / 64;

  Rows &rows = *reinterpret_cast<Rows *>(smem + L::rows);
  Range &rg = *reinterpret_cast<Range *>(smem + L::range);
  if (tid == 0) {
    for (int i = 0; i < kBufs; ++i) {
      tc::mbar_init(&full[i], TMA ? 4 : 64);  // the four warps, or the lanes of the buffer's two
      tc::mbar_init(&empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&s_full[b], 1);
      tc::mbar_init(&p_full[b], 128 + 128);
      tc::mbar_init(&stat[b], 128);
    }
    tc::mbar_init(&fin[0], 128);
    tc::mbar_init(&fin[1], 128);
    tc::mbar_init(q_full, 128);
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  dependency_wait();
  if (warp == 8) tc::tmem_alloc(tmem_slot, 512);  // (a block of the kernel before may still ask for tensor memory until then)
  tc::tc_fence_before();
  const int nt = find_range<kUnit, kThreads<TMA>, ALIGN, kEnd, true>(P, gridDim.x, reinterpret_cast<Two *>(smem + L::scan), rows, rg);  // this CTA's tiles
  if (nt <= 0) {  // (< 0: more units than can be counted, so that no segment is told of)
    if (tid == 0 && (nt < 0 || !P.by_segment)) P.split[blockIdx.x] = make_int2(0, 0);
    if (warp == 8) {
      tc::tc_fence_after();
      tc::tmem_dealloc(*tmem_slot, 512);
    }
    return;
  }
  Cursor c = first_unit<kUnit, ALIGN, kEnd>(a, P.Hg, rg, rows);
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot, tO = tmem + 2 * kS;  // S: 2 x 64 columns, O^T: 4 x 64
  // Scores, weights and what goes with them alternate by tile (phases: par), tile buffers go round.
  auto par = [](int i) { return (uint32_t)((i >> 1) & 1); };
  struct Ring {  // buffer and phase of a tile
    int b = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
      if (++b == kBufs) b = 0, ph ^= 1u;
    }
  };
  auto last_of = [&](int i) { return c.t == c.units - 1 || i + 1 == nt; };  // of a segment, in this CTA

  if (warp < 4) {
    // ------------------------------------------------------------------------------ softmax
    // The scores' 64 rows lie in the first 16 lanes of each quarter of tensor memory; a thread holds 12 positions of two
    // heads, hA and hB = hA + 8, a head's 48 positions the four lanes of a quad.
    const int hA = 16 * warp + (lane >> 2), qc = 2 * (lane & 3);
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    auto load_q = [&](const Cursor &k) {
      const int kvh = k.hg / P.sub, sg = k.hg - kvh * P.sub;
      const int h0 = kvh * P.g + sg * kHeads, nh = min(kHeads, P.g - sg * kHeads);
      const bf16 *q = a.q + (int64_t)k.n * a.q_t + (int64_t)h0 * hd;
      const int cc = lane & 7;
#pragma unroll 1
      for (int kb = 0; kb < nkb; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = warp * 16 + 4 * i + (lane >> 3), d = kb * 64 + cc * 8;
          const bool in = r < nh && d < hd;
          attn::cp_async16(s_q + kb * kQBlock + r * 128 + ((cc ^ (r & 7)) << 4), in ? q + (int64_t)r * hd + d : a.q, in);
        }
    };
    load_q(c);
    attn::cp_async_wait_all();
    attn::fence_proxy_async();
    tc::mbar_arrive(q_full);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lr[2] = {0.f, 0.f};  // l, lr: of this thread's positions; lr as rounded
    int nseg = 0;
    bool first = true;
    int seg = 0;  // the segment's first tile here
    Ring tile;
    for (int i = 0; i < nt; ++i, tile.next()) {
      const int b = i & 1;
      if (!warp_wait(&full[tile.b], tile.ph, abort_flag)) break;  // (its mask)
      uint32_t ok0 = masks[2 * tile.b], ok1 = masks[2 * tile.b + 1];
      if (!warp_wait(&s_full[b], par(i), abort_flag)) break;
      tc::tc_fence_after();
      const bool last = last_of(i);
      Cursor nx = c;
      if (last && i + 1 < nt) {  // q's last reader is done: the next segment's q on its way
        nx.t = nx.units - 1;
        advance<kUnit, ALIGN, kEnd>(a, P.Hg, rows, nx);
        load_q(nx);
      }
      float s[4 * kJ];  // s[4 j + 2 x + e]: position 8 j + qc + e of head x
      {
        uint32_t r[4 * kJ];
        tc::tmem_ld_16x48_wait(tmem + (uint32_t)(b * kS) + lane_off, r);
#pragma unroll
        for (int k = 0; k < 4 * kJ; ++k) s[k] = __uint_as_float(r[k]);
      }
      float sc = P.scale_log2;
      if ((ok0 & ok1) != kHalf) {  // positions that are not there: -inf (scaled here, so that a scale of 0 is right)
        ok0 >>= qc;
        ok1 >>= qc;
#pragma unroll
        for (int k = 0; k < 4 * kJ; ++k)
          s[k] = ((k < 2 * kJ ? ok0 : ok1) >> (8 * ((k >> 2) % (kJ / 2)) + (k & 1))) & 1u ? s[k] * sc : -INFINITY;
        sc = 1.f;
      }
      float al[2];
      bool raised = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = s[2 * x];  // the largest scaled score, of a scale of either sign
        if (sc < 0.f) {
#pragma unroll
          for (int k = 0; k < 2 * kJ; ++k) mx = fminf(mx, s[4 * (k >> 1) + 2 * x + (k & 1)]);
        } else {
#pragma unroll
          for (int k = 0; k < 2 * kJ; ++k) mx = fmaxf(mx, s[4 * (k >> 1) + 2 * x + (k & 1)]);
        }
        mx *= sc;
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        al[x] = 1.f;
        if (first) {
          m[x] = mx;
        } else if (mx > m[x] + 8.f || (m[x] == -INFINITY && mx > m[x])) {
          al[x] = m[x] == -INFINITY ? 0.f : exp2f(m[x] - mx);
          m[x] = mx;
          raised = true;
        }
        if (qc == 0) alpha_sm[b * kHeads + hA + 8 * x] = al[x];
      }
      const bool any = __any_sync(0xffffffffu, raised);
      if (lane == 0) flags[4 * b + warp] = any ? 1 : 0;
      __syncwarp();
      tc::mbar_arrive(&stat[b]);
      uint32_t pk[2][kJ];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float ref = m[x] == -INFINITY ? 0.f : m[x];
        const int h = hA + 8 * x;
        const uint32_t prow = s_p + b * kHeads * 128 + h * 128 + 2 * qc;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const float p0 = ex2(fmaf(s[4 * j + 2 * x], sc, -ref)), p1 = ex2(fmaf(s[4 * j + 2 * x + 1], sc, -ref));
          sum += p0 + p1;
          const __nv_bfloat162 pr = __floats2bfloat162_rn(p0, p1);
          pk[x][j] = *reinterpret_cast<const uint32_t *>(&pr);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(prow + ((j ^ (h & 7)) << 4)), "r"(pk[x][j]) : "memory");
        }
        l[x] = l[x] * al[x] + sum;
      }
      attn::fence_proxy_async();
      tc::tc_fence_before();
      tc::mbar_arrive(&p_full[b]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // (behind what the products wait for)
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kJ; ++j) sum += __uint_as_float(pk[x][j] << 16) + __uint_as_float(pk[x][j] & 0xffff0000u);
        lr[x] = lr[x] * al[x] + sum;
      }
      first = false;
      if (last) {
        const int kvh = c.hg / P.sub, sg = c.hg - kvh * P.sub;
        const int h0 = kvh * P.g + sg * kHeads, nh = min(kHeads, P.g - sg * kHeads);
        const int sb = i - c.t, se = sb + c.units;  // the whole segment, from this CTA's first tile
        const bool whole = sb >= 0 && se <= nt;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
          l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
          lr[x] += __shfl_xor_sync(0xffffffffu, lr[x], 1);
          lr[x] += __shfl_xor_sync(0xffffffffu, lr[x], 2);
          const int h = hA + 8 * x;
          float fo = 1.f;
          if (qc == 0 && h < nh) {
            if (whole) {
              fo = out_factor(m[x], lr[x], a.sink, h0 + h);
              if (a.lse)
                a.lse[(int64_t)c.n * a.H + h0 + h] = l[x] == 0.f ? -INFINITY : (m[x] + log2f(l[x])) * 0.6931471805599453f;
            } else {
              const int slot = 2 * blockIdx.x + (seg == sb ? 1 : 0);
              *reinterpret_cast<float2 *>(P.share_ml + ((int64_t)slot * kHeads + h) * 2) = make_float2(m[x], lr[x]);
              P.share_l[(int64_t)slot * kHeads + h] = l[x];
            }
          }
          if (qc == 0) f_sm[(nseg & 1) * kHeads + h] = fo;
          m[x] = -INFINITY;
          l[x] = lr[x] = 0.f;
        }
        __syncwarp();
        tc::mbar_arrive(&fin[nseg & 1]);
        ++nseg;
        seg = i + 1;
        first = true;
        if (i + 1 < nt) {
          attn::cp_async_wait_all();
          attn::fence_proxy_async();
          tc::mbar_arrive(q_full);
        }
        c = nx;
      } else {
        ++c.t;
      }
    }
    attn::cp_async_wait_all();
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------------------------ O: rescaling, results, joins
    const int quad = warp - 4, jt = tid - 128;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    bool first = true, told = false;
    int nseg = 0;
    int seg = 0;
    Ring tile, before;  // this tile's buffer, the one's before
    for (int i = 0; i < nt; ++i, before = tile, tile.next()) {
      const int b = i & 1;
      if (TMA) {
        // positions that are not there hold what the page holds (or an older tile): their weights are 0, but 0 x NaN is not,
        // so their rows are zeroed before the values' products read them
        if (!warp_wait(&full[tile.b], tile.ph, abort_flag)) break;
        const uint32_t ok0 = masks[2 * tile.b], ok1 = masks[2 * tile.b + 1];
        if ((ok0 & ok1) != kHalf) {
          for (int r = jt >> 6; r < kUnit; r += 2)
            if (!(((r < kUnit / 2 ? ok0 : ok1) >> (r % (kUnit / 2))) & 1u))
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                               s_t + (tile.b * kBlocks + ((jt >> 3) & 7)) * kBlock + r * 128 + (jt & 7) * 16),
                           "r"(0)
                           : "memory");
          attn::fence_proxy_async();
        }
      }
      if (!warp_wait(&stat[b], par(i), abort_flag)) break;
      if (!first && (flags[4 * b] | flags[4 * b + 1] | flags[4 * b + 2] | flags[4 * b + 3])) {
        if (!warp_wait(&empty[before.b], before.ph, abort_flag)) break;
        tc::tc_fence_after();
#pragma unroll 1
        for (int cq = 0; cq < 4 * 4; ++cq) {
          if ((cq >> 2) * 128 >= hd) break;
          uint32_t v[16];
          const uint32_t ta = tO + (uint32_t)(cq * 16) + lane_off;
          float av[16];
          attn::lds16(av, alpha_sm + b * kHeads + (cq & 3) * 16);
          tc::tmem_ld16_wait(ta, v);
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * av[k]);
          attn::tmem_st16(ta, v);
        }
        attn::tmem_st_wait();
        tc::tc_fence_before();
      }
      const bool last = last_of(i);
      tc::mbar_arrive(&p_full[b]);
      first = false;
      if (!last) {
        ++c.t;
        continue;
      }
      if (!warp_wait(&fin[nseg & 1], (uint32_t)((nseg >> 1) & 1), abort_flag)) break;
      if (!warp_wait(&empty[tile.b], tile.ph, abort_flag)) break;
      tc::tc_fence_after();
      const int kvh = c.hg / P.sub, sg = c.hg - kvh * P.sub;
      const int h0 = kvh * P.g + sg * kHeads, nh = min(kHeads, P.g - sg * kHeads);
      const int sb = i - c.t, se = sb + c.units;
      const bool whole = sb >= 0 && se <= nt;
      const int slot = 2 * blockIdx.x + (seg == sb ? 1 : 0);
#pragma unroll 1
      for (int cq = 0; cq < 4 * 2; ++cq) {
        const int hh = (cq & 1) * 32, d = (cq >> 1) * 128 + quad * 32 + lane;
        if ((cq >> 1) * 128 >= hd) break;
        if (hh >= nh) continue;
        float v[32];
        attn::tmem_ld_32cols(tO + (uint32_t)((cq >> 1) * kHeads + hh) + lane_off, v);
        if (whole) {
          // (all factors first, and no branch a store: with both inside the loop a result took 14 thousand cycles, not 5; two
          // features a store, exchanged between lanes, are no faster)
          float f[16];
          bf16 *o = a.o + (int64_t)c.n * a.o_t + (int64_t)(h0 + hh) * hd + d;
#pragma unroll
          for (int k = 0; k < 32; k += 16) {
            attn::lds16(f, f_sm + (nseg & 1) * kHeads + hh + k);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[k + e] *= f[e];
          }
          if (hh + 32 <= nh && (cq >> 1) * 128 + quad * 32 + 32 <= hd) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k * hd] = __float2bfloat16(v[k]);
          } else if (d < hd) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (hh + k < nh) o[k * hd] = __float2bfloat16(v[k]);
          }
        } else if (d < hd) {
          float *o = P.share_o + ((int64_t)slot * kHeads + hh) * kHD + d;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (hh + k < nh) o[k * kHD] = v[k];
        }
      }
      tc::tc_fence_before();
      if (seg == sb && jt == 0) {  // (the segment begins here)
        int c0;
        const int parts = whole ? 0 : sharers(rg, c, c0);
        if (P.by_segment) {
          P.split[(int64_t)c.n * P.Hg + c.hg] = make_int2(blockIdx.x, parts);
        } else if (!whole) {
          P.split[blockIdx.x] = make_int2(c.n * P.Hg + c.hg, parts);
          told = true;
        }
      }
      first = true;
      ++nseg;
      seg = i + 1;
      c.t = c.units - 1;
      if (i + 1 < nt) advance<kUnit, ALIGN, kEnd>(a, P.Hg, rows, c);
    }
    if (!P.by_segment && jt == 0 && !told) P.split[blockIdx.x] = make_int2(0, 0);
  } else if (warp == 8) {
    // ------------------------------------------------------------------------------ products
    // One elected lane (by elect.sync, which lets the operands' descriptors stay in uniform registers: issued by `lane == 0`
    // each product cost about 115 cycles, of which it computes 40 or 57).
    if (tc::elect_one()) {
      const uint32_t id1 = tc::idesc_bf16_f32(kHeads, kUnit);
      const uint32_t id2 = tc::idesc_bf16_f32(128, kHeads, /*a_mn_major=*/true, /*b_mn_major=*/false);
      // the operands' descriptors differ in their lower words (address, leading offset) only
      const uint32_t dq = (uint32_t)tc::sdesc_sw128(s_q, 16, 1024), dk = (uint32_t)tc::sdesc_sw128(s_t, 16, 1024),
                     dv = (uint32_t)tc::sdesc_sw128(s_t, kBlock, 1024), dp = (uint32_t)tc::sdesc_sw128(s_p, 16, 1024);
      const uint32_t hi = (uint32_t)(tc::sdesc_sw128(0, 16, 1024) >> 32);
      constexpr uint32_t kStep = kBlock >> 4, kQStep = kQBlock >> 4;  // a block, in descriptor units
      auto mma = [hi](uint32_t d, uint32_t al, uint32_t bl, uint32_t id, uint32_t acc) {
        tc::mma_bf16(d, (uint64_t)hi << 32 | al, (uint64_t)hi << 32 | bl, id, acc);
      };
      // (Rolled loops: unrolled, the products' code is fetched anew for every tile while eleven other warps run theirs.)
      auto scores = [&](int b, int sb) {
        const uint32_t d = tmem + (uint32_t)(sb * kS);
        uint32_t al = dq, bl = dk + b * kBlocks * kStep;
#pragma unroll 1
        for (int kb = 0; kb < nkb; ++kb, al += kQStep, bl += kStep) {
          mma(d, al, bl, id1, kb ? 1u : 0u);
#pragma unroll
          for (int k4 = 1; k4 < 4; ++k4) mma(d, al + 2 * k4, bl + 2 * k4, id1, 1u);
        }
        tc::mma_commit(&s_full[sb]);
      };
      auto values = [&](int b, int sb, bool first) {
        tc::tc_fence_after();
        const uint32_t p0 = dp + sb * (kHeads * 128 >> 4);
#pragma unroll 1
        for (int ch = 0; ch * 128 < hd; ++ch) {
          const uint32_t v0 = dv + (b * kBlocks + 2 * ch) * kStep;
#pragma unroll
          for (int ii = 0; ii < kUnit / 16; ++ii)
            mma(tO + (uint32_t)(ch * kHeads), v0 + ii * 128, p0 + ii * 2, id2, (first && ii == 0) ? 0u : 1u);
        }
        tc::mma_commit(&empty[b]);
      };
      bool ok = tc::mbar_wait(q_full, 0, abort_flag), first = true;
      int nq = 1;  // segments whose q has been waited for
      if (ok && (ok = tc::mbar_wait(&full[0], 0, abort_flag))) scores(0, 0);
      Ring tile, nx;
      nx.next();
      for (int i = 0; i < nt && ok; ++i, tile = nx, nx.next()) {
        const int sb = i & 1;
        const bool last = last_of(i);
        // this tile's values and the next tile's scores, whichever is ready (a new segment's q, and so its scores,
        // only behind the values)
        bool pv = false, qk = i + 1 == nt;
        uint64_t t0 = 0;  // (when it first had to wait: the timer is slow to read)
        uint32_t spins = 0;
        while (!pv || !qk) {
          // (both barriers asked at once: a read of shared memory takes 250 cycles beside the products' operands)
          const bool p_ready = tc::mbar_test_wait(&p_full[sb], par(i)), t_ready = tc::mbar_test_wait(&full[nx.b], nx.ph);
          if (!pv && p_ready) {
            values(tile.b, sb, first);
            pv = true;
            if (last && !qk) {
              if (!(ok = tc::mbar_wait(q_full, (uint32_t)(nq & 1), abort_flag))) break;
              ++nq;
            }
          }
          if (!qk && (pv || !last) && t_ready) {
            scores(nx.b, sb ^ 1);
            qk = true;
          }
          if ((++spins & 63) == 0) {
            if (t0 == 0) t0 = tc::global_ns();
            if (*abort_flag || tc::global_ns() - t0 > tc::kWaitLimitNs) {
              *abort_flag = 1;
              ok = false;
              break;
            }
          }
        }
        if (!ok) break;
        first = last;
        if (last) {
          c.t = c.units - 1;
          if (i + 1 < nt) advance<kUnit, ALIGN, kEnd>(a, P.Hg, rows, c);
        } else {
          ++c.t;
        }
      }
      // nothing may still read shared memory, write TMEM or arrive when the CTA ends
      tc::mma_commit(drain);
      const uint64_t t1 = tc::global_ns();
      while (!tc::mbar_try_wait(drain, 0) && tc::global_ns() - t1 < tc::kWaitLimitNs) {
      }
    }
    __syncwarp();
  } else if (TMA) {
    // ------------------------------------------------------------------------------ copies by TMA: a quarter of the features a warp
    const int w = warp - kFirstCopy, R = PG.box_rows, nbox = kUnit / R, r_log = __ffs(R) - 1;
    const int nb_kb = max(0, min(2, nkb - 2 * w));  // its 64-feature blocks
    if (lane == 0) tc::prefetch_tmap(&PG.map);
    // Box k of a tile (its positions k R .. k R + R - 1, which lie in one page) is lane k's; m0, m1: the tile's positions
    // that are there.  A tile is looked up two tiles ahead, so that nothing but the copies is left to do when its buffer
    // is handed back.
    struct Tile {
      uint32_t boxes, m0, m1;
      int kvh, page, row;
    };
    int looked = 0, issued = 0;
    auto look = [&]() {
      Tile x{0, 0, 0, 0, 0, 0};
      if (looked < nt) {
        const Row row = rows.get<kUnit, ALIGN>(a, c.n);
        const int lo = max(row.lead - c.t * kUnit, 0), hi = min(row.rows - c.t * kUnit, kUnit);  // positions lo .. hi - 1
        x.kvh = c.hg / P.sub;
        const bool wanted = lane < nbox && lane * R < hi && (lane + 1) * R > lo;
        const uint32_t pos = (uint32_t)row.first + c.t * kUnit + lane * R, pg = P.page.div(pos);
        x.row = (int)(pos - pg * P.page.d);
        x.page = wanted ? a.table[(int64_t)row.req * a.width + pg] : 0;
        const bool good = wanted && x.page >= 0 && x.page < a.c.n_pages;
        if (wanted && !good) atomicOr(a.status, kStatusBadIndex);
        x.boxes = __ballot_sync(0xffffffffu, good);
        constexpr int kH = kUnit / 2;
        x.m0 = __ballot_sync(0xffffffffu, lane < kH && lane >= lo && lane < hi && ((x.boxes >> (lane >> r_log)) & 1u));
        x.m1 = __ballot_sync(0xffffffffu, lane < kH && lane + kH >= lo && lane + kH < hi && ((x.boxes >> ((lane + kH) >> r_log)) & 1u));
        if (++looked < nt) advance<kUnit, ALIGN, kEnd>(a, P.Hg, rows, c);
      }
      return x;
    };
    Tile t0 = look(), t1 = look();
    Ring tile;
    for (int i = 0; i < nt; ++i, tile.next()) {
      if (i >= kBufs && !warp_wait(&empty[tile.b], tile.ph ^ 1u, abort_flag)) break;
      uint64_t *bar = &full[tile.b];
      if (lane == 0) {
        if (w == 0) {  // (the mask of the tile before has been read: its values are done)
          masks[2 * tile.b] = t0.m0;
          masks[2 * tile.b + 1] = t0.m1;
        }
        tc::mbar_expect_tx(bar, (uint32_t)(__popc(t0.boxes) * nb_kb * R * 128));
      }
      __syncwarp();
      if ((t0.boxes >> lane) & 1u)
        for (int kb = 0; kb < nb_kb; ++kb)
          tc::tma_load_4d(s_t + (tile.b * kBlocks + 2 * w + kb) * kBlock + lane * R * 128, &PG.map, bar, (2 * w + kb) * 64, t0.kvh,
                          t0.row, t0.page);
      t0 = t1;
      t1 = look();
      issued = i + 1;
    }
    // nothing is in flight when the CTA ends, even after a wait that ran out
    for (int i = max(issued - kBufs, 0); i < issued; ++i) {
      const uint64_t t2 = tc::global_ns();
      while (!tc::mbar_try_wait(&full[i % kBufs], (uint32_t)((i / kBufs) & 1)) && tc::global_ns() - t2 < tc::kWaitLimitNs) {
      }
    }
  } else {
    // ------------------------------------------------------------------------------ copies by cp.async: 24 positions a warp
    const int b = (warp - kFirstCopy) >> 1, part = (warp - kFirstCopy) & 1;
    const bf16 *kbase = reinterpret_cast<const bf16 *>(a.c.k);
    const int cc = lane & 7;
    constexpr int kH = kUnit / 2;
    for (int k = 0; k < b && k + 1 < nt; ++k) advance<kUnit, ALIGN, kEnd>(a, P.Hg, rows, c);
    uint32_t ph = 1;
    for (int i = b; i < nt; i += kBufs, ph ^= 1u) {
      const Row row = rows.get<kUnit, ALIGN>(a, c.n);
      const uint32_t j = (uint32_t)c.t * kUnit + part * kH + lane;
      const bool there = lane < kH && j < (uint32_t)row.rows;
      const uint32_t pos = row.first + j, pg = P.page.div(pos);
      const int id = there ? a.table[(int64_t)row.req * a.width + pg] : 0;
      const bool good = there && id >= 0 && id < a.c.n_pages;
      if (there && !good) atomicOr(a.status, kStatusBadIndex);
      const int64_t off = good ? (int64_t)id * a.c.k_page + (int64_t)(pos - pg * P.page.d) * a.c.k_row +
                                     (int64_t)(c.hg / P.sub) * a.c.k_head
                               : -1;
      const uint32_t mask = __ballot_sync(0xffffffffu, good);
      int64_t ro[kH / 4];  // positions 4 u + lane / 8 of this warp's 24
#pragma unroll
      for (int u = 0; u < kH / 4; ++u) ro[u] = __shfl_sync(0xffffffffu, off, 4 * u + (lane >> 3));
      const uint32_t dst = s_t + b * kBlocks * kBlock + (part * kH + (lane >> 3)) * 128;
      if (i >= kBufs && !warp_wait(&empty[b], ph, abort_flag)) break;
      if (lane == 0) masks[2 * b + part] = mask;
#pragma unroll 1
      for (int kb = 0; kb < nkb; ++kb) {
        const bool f_in = kb * 64 + cc * 8 < hd;
#pragma unroll
        for (int u = 0; u < kH / 4; ++u) {
          const bool in = ro[u] >= 0 && f_in;
          const int r7 = (4 * u + (lane >> 3)) & 7;
          attn::cp_async16(dst + kb * kBlock + u * 512 + ((cc ^ r7) << 4), in ? kbase + ro[u] + kb * 64 + cc * 8 : kbase, in);
        }
      }
      attn::cp_async_wait_all();
      attn::fence_proxy_async();
      tc::mbar_arrive(&full[b]);
      for (int k = 1; k <= kBufs && i + k < nt; ++k) advance<kUnit, ALIGN, kEnd>(a, P.Hg, rows, c);
    }
    attn::cp_async_wait_all();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && *abort_flag) atomicOr(a.status, kStatusTimeout);
}

// Join the shares of the segments that several CTAs worked on: block x a segment (or the CTA that a split segment
// began in), its heads and 64-feature chunks dealt over the blocks y.  A share is 128 KB, which the last CTA to finish
// alone would take tens of microseconds to read; here the whole device reads them, 16 lanes a chunk of a share, every
// load of a group in flight at once.  One group adds up to six shares of an item, two or four groups the shares of a segment that
// more CTAs had (up to sixteen: the same within 1 us from 2 to 152 shares).  Shares are added in an order that their number alone
// sets.  32 segments of 4 to 5 shares (17 MB): 5 us with the launch; the shares' way through L2 bounds it.  (Eight
// shares, or four, 1 to 2 us more; a fifth block an SM spills.)
constexpr int kJoinThreads = 256, kJoinChunk = 64, kJoinLanes = kJoinChunk / 4, kJoinGroups = kJoinThreads / kJoinLanes;
constexpr int kJoinShares = 6, kJoinSplit = 4;
__global__ void __launch_bounds__(kJoinThreads, 4) k_paged_join_latent(const __grid_constant__ Params P) {
  __shared__ float4 s_v[kJoinGroups][kJoinLanes];
  __shared__ float3 s_ml[kJoinGroups];
  const PagedAttnArgs &a = P.a;
  dependency_wait();
  const int2 sp = P.split[blockIdx.x];
  const int n_hg = P.by_segment ? (int)blockIdx.x : sp.x, n = n_hg / P.Hg, hg = n_hg - n * P.Hg, parts = sp.y;
  if (P.by_segment && row_of<kUnit, false>(a, n, false).units == 0) return;  // (a row that was left alone: nothing told)
  const int c0 = P.by_segment ? sp.x : (int)blockIdx.x;
  // (after a wait that ran out the notes may be those of another call: nothing outside the workspace is read)
  if (parts <= 1 || c0 < 0 || parts > P.ctas - c0 || n < 0 || n >= a.N) return;
  const int kvh = hg / P.sub, sg = hg - kvh * P.sub, h0 = kvh * P.g + sg * kHeads, nh = min(kHeads, P.g - sg * kHeads);
  const int hd = a.c.head_dim, lane = threadIdx.x % kJoinLanes, grp = threadIdx.x / kJoinLanes;
  const int chunks = (hd + kJoinChunk - 1) / kJoinChunk;
  int G = 1;  // groups an item
  while (G < kJoinSplit && G * kJoinShares < parts) G *= 2;
  const int sub = grp & (G - 1), per = kJoinGroups / G;
  for (int it0 = blockIdx.y * per; it0 < nh * chunks; it0 += gridDim.y * per) {
    const int it = it0 + grp / G, h = it / chunks, d = (it - h * chunks) * kJoinChunk + lane * 4;
    const bool in = h < nh && d < hd;
    float M = -INFINITY, Lr = 0.f;  // (of the rounded weights)
    float L = 0.f;                  // of the weights as they were: share u of a round in lane u
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = sub; p0 < parts && h < nh; p0 += G * kJoinShares) {
      float4 x[kJoinShares];
      float2 ml[kJoinShares];
      const int pl = p0 + lane * G;
      const float l = lane < kJoinShares && pl < parts
                          ? __ldcg(P.share_l + (int64_t)(pl == 0 ? 2 * c0 + 1 : 2 * (c0 + pl)) * kHeads + h)
                          : 0.f;
#pragma unroll
      for (int u = 0; u < kJoinShares; ++u) {
        const int p = p0 + u * G;
        ml[u] = make_float2(-INFINITY, 0.f);
        x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < parts) {
          const int64_t r = (int64_t)(p == 0 ? 2 * c0 + 1 : 2 * (c0 + p)) * kHeads + h;
          ml[u] = __ldcg(reinterpret_cast<const float2 *>(P.share_ml + r * 2));
          if (in) x[u] = __ldcg(reinterpret_cast<const float4 *>(P.share_o + r * kHD + d));
        }
      }
      float mx = M;
#pragma unroll
      for (int u = 0; u < kJoinShares; ++u) mx = fmaxf(mx, ml[u].x);
      const float f0 = M == -INFINITY ? 0.f : exp2f(M - mx);
      M = mx;
      Lr *= f0;
      L *= f0;
      v.x *= f0, v.y *= f0, v.z *= f0, v.w *= f0;
#pragma unroll
      for (int u = 0; u < kJoinShares; ++u) {
        const float e = ml[u].x == -INFINITY ? 0.f : exp2f(ml[u].x - M);
        Lr = fmaf(ml[u].y, e, Lr);
        if (lane == u) L = fmaf(l, e, L);
        v.x = fmaf(x[u].x, e, v.x);
        v.y = fmaf(x[u].y, e, v.y);
        v.z = fmaf(x[u].z, e, v.z);
        v.w = fmaf(x[u].w, e, v.w);
      }
    }
#pragma unroll
    for (int o = kJoinLanes / 2; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (G > 1) {  // (uniform over the block)
      s_v[grp][lane] = v;
      if (lane == 0) s_ml[grp] = make_float3(M, Lr, L);
      __syncthreads();
      if (sub == 0) {
        for (int k = 1; k < G; ++k) M = fmaxf(M, s_ml[grp + k].x);
        Lr = L = 0.f;
        v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < G; ++k) {
          const float3 ml = s_ml[grp + k];
          const float4 x = s_v[grp + k][lane];
          const float e = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
          Lr = fmaf(ml.y, e, Lr);
          L = fmaf(ml.z, e, L);
          v.x = fmaf(x.x, e, v.x);
          v.y = fmaf(x.y, e, v.y);
          v.z = fmaf(x.z, e, v.z);
          v.w = fmaf(x.w, e, v.w);
        }
      }
      __syncthreads();
    }
    if (sub == 0 && in) {
      const float fo = out_factor(M, Lr, a.sink, h0 + h);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * fo, v.y * fo), hi = __floats2bfloat162_rn(v.z * fo, v.w * fo);
      *reinterpret_cast<uint2 *>(a.o + (int64_t)n * a.o_t + (int64_t)(h0 + h) * hd + d) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
      if (a.lse && d == 0) a.lse[(int64_t)n * a.H + h0 + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
  }
}

}  // namespace latent

cudaError_t launch_latent(Params p, float *ws, size_t ws_bytes, int num_sms, cudaStream_t s) {
  using namespace latent;
  const PagedAttnArgs &a = p.a;
  // TMA where pages hold whole boxes of at least 8 rows (the swizzle's period), up to a tile; cp.async for other pages
  Pages pg;
  memset(&pg, 0, sizeof(pg));
  pg.box_rows = std::min(a.c.page & -a.c.page, kUnit & -kUnit);
  bool tma = pg.box_rows >= 8;
  if (tma) {
    const uint64_t dims[4] = {(uint64_t)a.c.head_dim, (uint64_t)a.c.kv_heads, (uint64_t)a.c.page, (uint64_t)a.c.n_pages};
    // (strides of dimensions of size 1 may be anything: a row's)
    const uint64_t row = 2 * (uint64_t)a.c.head_dim;
    const uint64_t strides[3] = {a.c.kv_heads > 1 ? 2 * (uint64_t)a.c.k_head : row, 2 * (uint64_t)a.c.k_row,
                                 a.c.n_pages > 1 ? 2 * (uint64_t)a.c.k_page : row};
    tma = tma_map_pages_bf16(&pg.map, a.c.k, dims, strides, 64, (uint32_t)pg.box_rows);
  }
  static SmemAttr attr_tma, attr_copy;
  const size_t smem = L::total;
  cudaError_t e = tma ? attr_tma.ensure((const void *)k_paged_attn_latent<true>, (int)smem)
                      : attr_copy.ensure((const void *)k_paged_attn_latent<false>, (int)smem);
  if (e != cudaSuccess) return e;
  p.g = a.H / a.c.kv_heads;
  p.sub = (p.g + kHeads - 1) / kHeads;
  p.Hg = p.sub * a.c.kv_heads;
  const int64_t rows = a.window > 0 ? std::min<int64_t>(a.window, (int64_t)a.width * a.c.page) : (int64_t)a.width * a.c.page;
  const int64_t units = (int64_t)a.N * p.Hg * std::max<int64_t>(1, (rows + kUnit - 1) / kUnit + (a.window > 0 ? 1 : 0));
  const int64_t grid = std::min<int64_t>(std::min<int64_t>(units, num_sms), kMaxCtas);
  const int64_t segments = (int64_t)a.N * p.Hg;
  p.share_o = ws;
  p.share_ml = ws + 2 * grid * kHeads * kHD;
  p.split = reinterpret_cast<int2 *>(p.share_ml + 2 * grid * kHeads * 2);
  p.share_l = reinterpret_cast<float *>(p.split + grid);
  p.by_segment = segments <= grid;
  p.ctas = (int)grid;
  if (sizeof(float) * 2 * grid * kHeads * (kHD + 3) + sizeof(int2) * grid > ws_bytes) return cudaErrorInvalidValue;
  e = tma ? launch_dependent(k_paged_attn_latent<true>, dim3((unsigned)grid), dim3(kThreads<true>), smem, s, 1, p, pg)
          : launch_dependent(k_paged_attn_latent<false>, dim3((unsigned)grid), dim3(kThreads<false>), smem, s, 1, p, pg);
  if (e != cudaSuccess || segments == units) return e;  // (one tile a segment: nothing is shared)
  // blocks of the join: one group an item, and four blocks an SM where segments are few and so split over many CTAs
  const int64_t x = std::min(segments, grid), items = (int64_t)std::min(p.g, kHeads) * ((a.c.head_dim + kJoinChunk - 1) / kJoinChunk);
  const int64_t y = std::min(items, std::max((items + kJoinGroups - 1) / kJoinGroups, 4 * num_sms / x));
  return launch_dependent(k_paged_join_latent, dim3((unsigned)x, (unsigned)y), dim3(kJoinThreads), 0, s, 1, p);
}

}  // namespace paged
}  // namespace csa
