// k_rows_attn.cu -- attention of many rows over a paged cache (head_dim up to 256): the new tokens of prompts, and decode rows that
// share a prefix, on the 5th-generation tensor cores.
//
// The g query heads of a kv head and the tokens of a segment (a request's new tokens, the rows of a prefix) are rows of one
// product: row i of a segment is token i / g, head i mod g, whatever g is, so a cache row is read once for all of them.
// An item is a tile of up to QT x 128 such rows of one kv head with the tiles of KVT positions that any of them attends:
//   S[i][j] = sum_d q[i][d] K[j][d]       M = 128 rows, N = KVT positions, K = head_dim
//   p = exp2(S scale - m), bf16           a lane a row: the running maximum m and the sums stay in its registers; m is
//                                         raised only by more than 2^8 (the sums so far are then rescaled)
//   O[i][d] += sum_j p[i][j] V[j][d]      N = head_dim, K = KVT: p from tensor memory, where it lies over S
// p is rounded to bf16, by at most 2^-8 of itself (a second term would double that product); O's denominator adds up the
// rounded p, so that its weights still add up to 1 (with the sink's), lse the p as they were.  Scores, maxima, sums and O are f32.
//
// Up to 192 features two tiles of 128 rows share the keys and values, and one's softmax runs while the other's products do; at 256, where
// O takes half of tensor memory, one tile has two score buffers instead.
//
// A plan lists the items with the number of their position tiles (rows_plan.cuh); the tiles of all items and kv heads stand one
// behind the other, with places for each item's end, and each CTA takes an equal part of them in a row, so every CTA has as much to do
// as any other whatever the lengths and masks are.  An item that several CTAs worked on is joined from their shares (M, L, O), in the
// order of the CTAs, by k_rows_join.  The rows of a prefix batch's own pages come from k_paged_attn as one more share, and it takes a
// prompt batch's requests of one token (single_tokens below); its last CTA then makes the plan, beside the others' work.
//
// A CTA an SM: four warps a tile of rows for the softmax and the results, a warp that issues its products, and the copies (whole
// tiles by TMA, boxes of up to 128 rows inside a page where pages hold whole boxes of 8 rows at least; ragged tiles and other pages by
// cp.async, rows that are not there as zeros).  Shared memory holds q (64 KB at 128 features) and a ring of five tiles of keys or values.
// All waits are time-bounded.
//
// Bound by the way of a tile through its stages: scores to softmax (1600 cycles, of which 64 pairs of exponentials take 770 at least),
// softmax to values and the next scores (768 cycles of products, behind the other tile's).  The products alone take 2700 cycles for two
// tiles of rows and a tile of positions (2048 by the measured peak: two products read q and the keys from shared memory at
// 128 bytes a cycle, all of its rate), with the softmax 3400.  16384 tokens of 64 heads over 8 of 128: 3.34 ms, 1316 TFLOP/s, 68 % of
// the measured bf16 rate (76 % of the sustained one); 12 ragged prompts of 100 to 4000 tokens (32 over 8 of 128) 311 us, 45 %:
// the ends of their items.  64 decodes of 1 to 5000 beside two prompts (40 over 8 of 80) 100 us.  256 rows behind 32768 shared ones (64
// over 8 of 128) 350 us, of which their own pages take 115.
#include <algorithm>
#include <cstring>

#include "attn_common.cuh"
#include "rows_plan.cuh"

namespace csa {

// 4-D bf16 tensor map with 128-byte swizzle, boxes {box_inner, 1, box_rows, 1} (defined with the GEMM's TMA helpers).
bool tma_map_pages_bf16(CUtensorMap *m, const void *base, const uint64_t (&dims)[4], const uint64_t (&strides)[3], uint32_t box_inner,
                        uint32_t box_rows);

namespace rows {

// Tiles that the end of an item counts for: its last tiles' masks and values looked over, the wait for the last product, results, the next
// q, 10 thousand cycles in all where a tile takes 3.4.  (4096 tokens of 64 heads over 8 of 128: 322, 282, 276 and 280 us for 1 to 4.)
// At 256 features a tile is half as long, and one tile of rows has nothing beside its end (32 over 8 of 256, 4096 tokens: 298, 282, 265 and
// 263 us for 3 to 6, 6 chunks behind 5000 to 30000, 16 over 2: 581, 586, 599, 606) -- but where its rows come by cp.async, tiles are longer
// (windows in pages of 17: 209 and 218 us for 3 and 5).
template <int HDP>
constexpr int end_tiles(bool tma) { return HDP == 256 && tma ? 5 : 3; }
constexpr int kNote = 8;      // tiles whose notes are kept: more than the copies can be ahead
constexpr float kRaise = 8.f;

struct Params : Plan {
  float scale_log2;
  int wide;                    // o's rows are whole 32 bytes on such borders
  float *share_o;              // [2 ctas][QT * 128][HDP]
  float4 *share_ml;            // [2 ctas][QT * 128]: M, L of the rounded weights, L
  int4 *split;                 // [ctas]: the item that began in this CTA and goes on behind it: item, kv head, CTAs
  const float *own_o;          // prefix: [N][H][head_dim], the share of each row's own pages
  const float2 *own_ml;        // [N][H]: M, L
};

// Sizes by padded head_dim.
template <int HDP>
struct Shape {
  static constexpr int QT = HDP == 256 ? 1 : 2;             // tiles of 128 rows an item
  static constexpr int KVT = HDP <= 128 ? 128 : 64;         // positions of a tile
  static constexpr int NP = HDP / 64;                       // 64-feature panels
  static constexpr int kQBytes = kSub * HDP * 2, kStage = KVT * HDP * 2;
  static constexpr int NST = HDP == 64 ? 8 : 5;             // stages: a tile's keys or values
  static constexpr int kSoft = 4 * QT, kMma = QT, kLoad = 4 - QT;  // warps
  static constexpr int kThreads = (kSoft + kMma + kLoad) * 32;
  // Registers a thread, softmax and the others: a row's 128 scores do not fit in the 168 that 384 threads get each.  They add up
  // to what the block is launched with: 256 x 208 + 128 x 88 = 384 x 168.
  static constexpr bool kSplit = HDP <= 128;
  static constexpr int kRegsSoft = 208, kRegsRest = 88;
  static constexpr int kQ = 0, kRing = QT * kQBytes, kBars = kRing + NST * kStage;
  static constexpr int kSlots = kBars + 32 * 8 + kNote * 16 + 160;
  static constexpr int kSmem = kSlots + (kSoft + kMma) * 2 * 64;  // (all that the kernel has: the swizzled tiles come first)
  static constexpr int kColO = 2 * KVT;                     // columns of tensor memory: two score buffers, then QT x HDP of O
};

// ------------------------------------------------------------------------------------------------ plan

constexpr int kPlanThreads = 512;  // (1024: 1 us more for every step's barriers)

// (Where k_paged_attn does not make it.)
__global__ void __launch_bounds__(kPlanThreads) k_rows_plan(const __grid_constant__ Plan P) {
  __shared__ PlanRoom<kPlanThreads> room;
  dependency_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (k_rows_attn may start, up to its own wait)
  make_plan<kPlanThreads>(P, room);
}

// ------------------------------------------------------------------------------------------------ a CTA's part

// An item as the plan has it, and its first place.
struct Slot {
  int4 a, b, c;
  unsigned long long start, spare;
};
// A role's way through its CTA's items.  SLOT: the next item's description is on its way to shared memory (two slots a warp, by cp.async)
// while one is worked on: from global memory it would take two trips in a row at the end of every item.
template <int KVT, bool SLOT>
struct Walk {
  const Params *P;
  const Part *rg;  // (in shared memory)
  Slot *slot;
  unsigned long long base = 0;
  int i, kvh, seq = -1;  // seq: items so far
  Item d;
  int kt0, tiles;               // the item's tiles of positions
  int u0, u1;                   // of these, the CTA's

  __device__ __forceinline__ void fetch(int to, int item, bool by) const {
    if (!by) return;
    const uint32_t dst = tc::smem_u32(slot + to);
    const int4 *src = reinterpret_cast<const int4 *>(P->item + item);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n\tcp.async.cg.shared.global [%0 + 16], [%1 + 16], 16;\n\t"
                 "cp.async.cg.shared.global [%0 + 32], [%1 + 32], 16;" ::"r"(dst), "l"(src)
                 : "memory");
    asm volatile("cp.async.ca.shared.global [%0 + 48], [%1], 8;" ::"r"(dst), "l"(P->start + item) : "memory");
  }
  // The item's place and parts from its description; false: it is behind the CTA's part.
  __device__ __forceinline__ bool set(int4 x, int4 y, int4 z, unsigned long long start) {
    const unsigned long long p0 = rg->first, p1 = rg->end;
    base = rg->places * kvh + start;
    if (base >= p1) return false;
    d = Item{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, 0};
    kt0 = d.begin / KVT;
    tiles = d.end > d.begin ? (d.end - 1) / KVT - kt0 + 1 : 1;
    u0 = base < p0 ? (int)min(p0 - base, 0x7fffffffull) : 0;
    u1 = (int)min((unsigned long long)tiles, p1 - base);
    return true;
  }
  __device__ __forceinline__ bool load() {
    if (kvh >= P->a.c.kv_heads) return false;
    const int4 *at = reinterpret_cast<const int4 *>(P->item + i);
    // (past L1: this kernel may begin before the plan has written them)
    return set(__ldcg(at), __ldcg(at + 1), __ldcg(at + 2), __ldcg(P->start + i));
  }
  __device__ __forceinline__ void step() {
    if (++i == rg->items) i = 0, ++kvh;
  }
  __device__ __forceinline__ void ahead(bool by) {  // the item after this one on its way
    if (SLOT) fetch((seq + 1) & 1, i + 1 == rg->items ? 0 : i + 1, by);
  }
  // The first item (all lanes that use the slots together; `by`: the one that copies).
  __device__ __forceinline__ bool first(bool by) {
    const int4 *at = reinterpret_cast<const int4 *>(&rg->d);
    bool more = set(at[0], at[1], at[2], rg->start);
    if (more && u0 >= u1) {  // (the part begins in the place of an item's end)
      step();
      more = load();
    }
    seq = 0;
    if (more) ahead(by);
    return more;
  }
  __device__ __forceinline__ bool peek() {  // on to the next item (copies waited for by whoever made them)
    step();
    if (!SLOT) return load();
    if (kvh >= P->a.c.kv_heads) return false;
    const Slot &n = slot[(seq + 1) & 1];
    return set(n.a, n.b, n.c, n.start);
  }
  __device__ __forceinline__ bool next(bool by) {
    const bool more = peek();
    ++seq;
    if (more) ahead(by);
    return more;
  }
  __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == tiles; }
};

// The rows of position tile j that are filled, and multiplied with: up to the item's last position, in steps of a product.
template <int KVT>
__device__ __forceinline__ int tile_rows(int end, int j) {
  const int left = max(end - j * KVT, 1);
  return left >= KVT ? KVT : (left + 15) & ~15;
}

// The first row of the item that the warps of tile of rows t have, -1: none.  An item of no more than 128 rows is tile 0's or tile 1's
// by turns, so that the end of one and the beginning of the next pass beside each other (64 decodes and two
// prompts, with the decodes as items here: 125 against 127 us).
template <int KVT, bool SLOT>
__device__ __forceinline__ int sub_rows(const Walk<KVT, SLOT> &w, int t, bool two) {
  if (!two) return 0;
  if (w.d.rows > kSub) return kSub * t;
  return (w.seq & 1) == t ? 0 : -1;
}
// The position tiles x .. y - 1, of the CTA's, that the warps of tile of rows t have to do with.
template <int KVT, bool SLOT>
__device__ __forceinline__ void sub_range(const Walk<KVT, SLOT> &w, int t, bool two, int &x, int &y) {
  const int sub = sub_rows(w, t, two);
  const int j0 = w.kt0 + w.u0, j1 = w.kt0 + w.u1, lo = sub > 0 ? w.d.begin1 : w.d.begin, end = sub > 0 ? w.d.end : w.d.end0;
  x = max(j0, lo / KVT);
  y = min(j1, (end - 1) / KVT + 1);  // (all of them not negative)
  if (sub < 0 || end <= lo || y < x) x = y = j0;
}

// ------------------------------------------------------------------------------------------------ building blocks

// (The kernel's code is larger than the instruction cache next to the schedulers, and a line that is not there costs as much as 15
// instructions: what is rarely run is out of line, loops are rolled where that costs little.)
__device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *abort) { return tc::mbar_wait(bar, parity, abort); }
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return tc::mbar_try_wait(bar, parity) || wait_on(bar, parity, abort);
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  const bool ok = tc::mbar_wait(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}
// D += A B: A (128 x 16 bf16) from tensor memory, B from shared memory.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Keeps the uses of loaded registers behind the wait above it.
__device__ __forceinline__ void tie32(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
// 32 bytes by one lane: a row's whole sector (16 at a time, a row a lane, each store would touch 32 sectors twice).
__device__ __forceinline__ void store32(void *p, const uint32_t *u) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]),
               "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}
__device__ __forceinline__ void lds4(uint32_t (&z)[4], uint32_t at) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(z[0]), "=r"(z[1]), "=r"(z[2]), "=r"(z[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// sum + both halves (bf16), each added in f32
__device__ __forceinline__ void add_halves(uint32_t v, float &x, float &y) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
      : "+f"(x), "+f"(y)
      : "r"(v));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ bool not_finite(uint32_t v) {  // either half
  return (v & 0x7f80u) == 0x7f80u || (v & 0x7f800000u) == 0x7f800000u;
}

// What goes below O and on it: factors of a row's share (m, lr) and of its own pages' (own), and lse.  (Powers as those of the
// weights, 2^-22 off; the logarithm and the division in full, as k_paged_attn's: where one score outweighs the others lse is little
// more than the error of the short logarithm.  Full powers too cost a long prompt 1.3 %.)
struct Finish {
  float f, f_own, lse;
};
__device__ __forceinline__ Finish finish(float m, float lr, float l, float2 own, const float *sink, int h) {
  const float M = fmaxf(m, own.x), ref = M == -INFINITY ? 0.f : M;
  const float e = paged::ex2(m - ref), eo = paged::ex2(own.x - ref);  // (2^-inf = 0)
  const float below = fmaf(own.y, eo, lr * e), sum = fmaf(own.y, eo, l * e);
  float top = ref, with = 0.f;  // with the sink's term
  if (sink) {
    const float s2 = sink[h] * 1.4426950408889634f;
    top = M == -INFINITY && s2 == -INFINITY ? 0.f : fmaxf(M, s2);
    with = s2 == INFINITY ? INFINITY : paged::ex2(s2 - top);
  }
  const float em = M == -INFINITY ? 0.f : paged::ex2(M - top), all = fmaf(below, em, with);
  const float f = all == 0.f ? 0.f : em / all;
  return {f * e, f * eo, sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f};
}
// Whether a row of the prefix form is there, and not padding.
__device__ __forceinline__ bool row_live(const RowsAttnArgs &a, int n) {
  if (!a.pos) return true;
  const int req = a.req ? a.req[n] : n;
  return a.pos[n] >= -1 && req >= 0 && req < a.R;
}

// A row's scores of a tile, which the lane finds in its KVT columns from tS on, times `by` and -inf where the row attends nothing: it
// attends positions from .. to of the tile as far as `there` has them.  (Rolled, and apart from the weights: few tiles need it.)
template <int KVT>
__device__ __forceinline__ void mask_scores(uint32_t tS, float by, int from, int to, const uint32_t *there) {
#pragma unroll 1
  for (int k = 0; k < KVT / 32; ++k, tS += 32, from -= 32, to -= 32) {
    const int f = min(max(from, 0), 32), e = min(max(to, -1), 31) + 1;
    const uint32_t mask = (e == 32 ? 0xffffffffu : (1u << e) - 1u) & (f == 32 ? 0u : 0xffffffffu << f) & there[k];
    if (by == 1.f && __all_sync(0xffffffffu, mask == 0xffffffffu)) continue;
    float v[32];
    attn::tmem_ld_32cols(tS, v);
    uint32_t u[16];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      u[c & 15] = __float_as_uint((mask >> c) & 1u ? v[c] * by : -INFINITY);
      if ((c & 15) == 15) attn::tmem_st16(tS + (c & 16), u);
    }
  }
  attn::tmem_st_wait();
}

// The row's weights where its scores were: exponentials by the maximum, which is raised by more than 2^8 only, in two halves, so that
// the first one's product begins beside the second's exponentials.  An exponential takes a warp 4 cycles at least, two with what goes
// with them 12: 64 such pairs are most of a tile's time.
template <int HDP, class Done>
__device__ __forceinline__ bool weights(float sc, float &m, float &l, float &lr, bool first, uint32_t tS, uint32_t tO, int hd16,
                                        uint64_t *p_half, uint64_t *p_full, int lane, Done &&values_done) {
  constexpr int KVT = Shape<HDP>::KVT, kW = KVT / 32;
  float2 s[KVT / 2], l4[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  {
    uint32_t v[kW][32];
#pragma unroll
    for (int k = 0; k < kW; ++k) tc::tmem_ld32(tS + 32 * k, v[k]);
    tc::tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < kW; ++k) {
      tie32(v[k]);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[16 * k + e] = make_float2(__uint_as_float(v[k][2 * e]), __uint_as_float(v[k][2 * e + 1]));
    }
  }
  float q4[4];  // (four chains, so that one's latency passes in the others)
#pragma unroll
  for (int k = 0; k < 4; ++k) q4[k] = fmaxf(s[k].x, s[k].y);
#pragma unroll
  for (int k = 4; k < KVT / 2; ++k) q4[k & 3] = max3(q4[k & 3], s[k].x, s[k].y);
  const float mx = fmaxf(max3(q4[0], q4[1], q4[2]), q4[3]);
  const bool raise = (mx - m) * sc > kRaise || (m == -INFINITY && mx > m);
  if (first) {
    m = mx;
  } else if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
    const float al = raise ? (m == -INFINITY ? 0.f : paged::ex2((m - mx) * sc)) : 1.f;
    if (raise) m = mx;
    l *= al;
    lr *= al;
    if (!values_done()) return false;
    tc::tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < hd16; c += 16) {
      uint32_t v[16];
      tc::tmem_ld16_wait(tO + c, v);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * al);
      attn::tmem_st16(tO + c, v);
    }
  }
  const float ref = m == -INFINITY ? 0.f : m * sc;
  const float2 sc2 = make_float2(sc, sc), ref2 = make_float2(-ref, -ref);
  uint32_t pk[KVT / 2];
#pragma unroll
  for (int k = 0; k < KVT / 32; ++k) {
    uint32_t v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 z = __ffma2_rn(s[16 * k + e], sc2, ref2), p = make_float2(paged::ex2(z.x), paged::ex2(z.y));
      l4[e & 1] = __fadd2_rn(l4[e & 1], p);
      v[e] = pk[16 * k + e] = pack2(p.x, p.y);
    }
    attn::tmem_st16(tS + 16 * k, v);
    if (k == KVT / 64 - 1 || k == KVT / 32 - 1) {
      attn::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(k == KVT / 64 - 1 ? p_half : p_full);
    }
  }
  // (behind what the product waits for)
  l += (l4[0].x + l4[0].y) + (l4[1].x + l4[1].y);
  l4[0] = l4[1] = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < KVT / 2; ++k) add_halves(pk[k], l4[k & 1].x, l4[k & 1].y);
  lr += (l4[0].x + l4[0].y) + (l4[1].x + l4[1].y);
  return true;
}

// Between which of the CTA's items, and between which tiles of positions, values that are not finite were taken out.
struct OddTiles {
  int seq0, seq1, j0, j1;
  __device__ __forceinline__ void note(int seq, int j) {
    atomicMin(&seq0, seq);
    atomicMax(&seq1, seq);
    atomicMin(&j0, j);
    atomicMax(&j1, j);
  }
  __device__ __forceinline__ bool any() const {
    const volatile OddTiles &v = *this;
    return v.seq0 <= v.seq1;
  }
};
// A lane's share of a tile of values, 16 bytes of every 2 KB: those that are not finite, in the tile's first `rows` rows (behind them lies
// what was there before), become 0, and the tile (the CTA's item seq, tile j of its positions) is noted.
template <int KVT>
__device__ __noinline__ void clear_odd(uint32_t at, int n, int r, int rows, OddTiles *odd, int seq, int j) {
  for (int i = 0; i < n; ++i, at += kSub * 16) {
    if ((i * kSub + r) / 8 % KVT >= rows) continue;
    uint32_t z[4];
    lds4(z, at);
    if (!(not_finite(z[0]) || not_finite(z[1]) || not_finite(z[2]) || not_finite(z[3]))) continue;
    odd->note(seq, j);  // (before they are gone: the other tile of rows may find them gone)
    __threadfence_block();
    for (int k = 0; k < 4; ++k) {
      if ((z[k] & 0x7f80u) == 0x7f80u) z[k] &= 0xffff0000u;
      if ((z[k] & 0x7f800000u) == 0x7f800000u) z[k] &= 0xffffu;
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(z[0]), "r"(z[1]), "r"(z[2]), "r"(z[3]) : "memory");
  }
}

// A row's result with the share of its own pages (own, none: NULL): O from the columns from tO on (there: if it was computed), times f.
// o NULL: nothing is written.  (Out of line: prompts run the code around it.)
__device__ __noinline__ void out_with_own(uint32_t tO, bool there, float f, const float *own, float f_own, int hd, bf16 *o) {
#pragma unroll 1
  for (int c = 0; c < hd; c += 8) {
    uint32_t u[8] = {};
    __syncwarp();
    if (there)
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                   : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                   : "r"(tO + c)
                   : "memory");
    if (!o) continue;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(u[k]) * f;
    if (own) {
      const float4 z0 = *reinterpret_cast<const float4 *>(own + c), z1 = *reinterpret_cast<const float4 *>(own + c + 4);
      const float z[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fmaf(z[k], f_own, v[k]);
    }
    *reinterpret_cast<uint4 *>(o + c) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  }
}

// Positions lo .. hi that token tok attends, as far as the segment has them.  (hi of a prefix: all.)
__device__ __forceinline__ void span(const RowsAttnArgs &a, int tok, int shift, int &lo, int &hi) {
  if (!a.pos) {
    hi = tok + shift;
    if (a.window > 0) lo = max(0, hi - a.window + 1);
  } else if (a.window > 0) {
    const int64_t first = (int64_t)shift + a.pos[tok] + 1 - a.window;
    lo = (int)max((int64_t)0, min(first, (int64_t)0x7fffffff));
  }
}

// Values that are not finite were left out of the products of tiles that not every row attends: here each is added to the rows that
// attend it, in their shares or results (whatever else is in the sum, it is not finite).  The softmax warps come here once, behind all
// of the CTA's items, when nothing waits for them any more, however many such tiles there are: each goes through those between the first
// and the last with such values, for the rows that it had, a lane a row as before, 32 positions at a time.  (Loops rolled: the tile loop is
// as fast as its code is short and well placed; 4 or 8 loads a round here cost it 1 %.)  40 thousand rows of a prefix's window of a
// million positions, 128 features: 20 ms with one such value or none, 74 with two half a window apart, 264 with one in every tile.
template <int HDP>
__device__ __forceinline__ void odd_values(const Params &P, const Part *rg, const OddTiles *odd) {  // (inline: a call cost a spill)
  using S = Shape<HDP>;
  constexpr int QT = S::QT, KVT = S::KVT;
  const RowsAttnArgs &a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = warp >> 2, row0 = (warp & 3) * 32, hd = a.c.head_dim, g = P.g.d;
  const OddTiles in = *odd;
  const bool vals = a.c.v != nullptr;
  Walk<KVT, false> w;
  w.P = &P;
  w.rg = rg;
  w.i = rg->item;
  w.kvh = rg->kvh;
  for (bool more = w.first(false); more && w.seq <= in.seq1; more = w.next(false)) {
    const Item &d = w.d;
    const int sub = sub_rows(w, t, QT == 2);
    if (w.seq < in.seq0 || sub < 0 || sub + row0 >= d.rows) continue;
    int x, y, lo = 0, hi = 0x7fffffff;
    sub_range(w, t, QT == 2, x, y);
    x = max(x, in.j0);
    y = min(y, in.j1 + 1);
    const int R = sub + row0 + lane;
    float *share = nullptr;
    bf16 *o = nullptr;
    if (R < d.rows) {
      const int q = (int)P.g.div(d.row0 + R), tok = d.tok0 + q, h = w.kvh * g + (d.row0 + R - q * g);
      span(a, tok, d.shift, lo, hi);
      if (!w.whole()) share = P.share_o + ((int64_t)(2 * blockIdx.x + (w.u0 == 0 ? 1 : 0)) * (QT * kSub) + R) * HDP;
      else if (row_live(a, tok)) o = a.o + (int64_t)tok * a.o_t + (int64_t)h * hd;
    }
    const bf16 *vb = reinterpret_cast<const bf16 *>(vals ? a.c.v : a.c.k) + w.kvh * (vals ? a.c.v_head : a.c.k_head);
#pragma unroll 1
    for (int j = x; j < y; ++j) {
      if (j * KVT >= d.at0 && d.at1 - j * KVT >= KVT) {  // (tiles that all attend have theirs already)
        j = d.at1 / KVT - 1;
        continue;
      }
#pragma unroll 1
      for (int k = 0; k < KVT; k += 32) {
        const uint32_t p = (uint32_t)j * KVT + k + lane, pg = P.page.div(p);
        const int id = p >= (uint32_t)d.begin && p < (uint32_t)d.end ? a.table[(int64_t)d.seg * a.width + pg] : -1;
        const bool there = id >= 0 && id < a.c.n_pages;
        const bf16 *src =
            there ? vb + id * (vals ? a.c.v_page : a.c.k_page) + (int64_t)(p - pg * P.page.d) * (vals ? a.c.v_row : a.c.k_row) : vb;
        uint32_t any = 0;
#pragma unroll 1
        for (int c = 0; c < hd; c += 8) {
          const uint4 z = *reinterpret_cast<const uint4 *>(src + c);
          any |= not_finite(z.x) || not_finite(z.y) || not_finite(z.z) || not_finite(z.w);
        }
        if (!__any_sync(0xffffffffu, there && any)) continue;
#pragma unroll 1
        for (int c = 0; c < hd; c += 8) {
          const uint4 z = *reinterpret_cast<const uint4 *>(src + c);
          const uint32_t u[4] = {z.x, z.y, z.z, z.w};
          const bool bad = there && (not_finite(z.x) || not_finite(z.y) || not_finite(z.z) || not_finite(z.w));
          float add[8] = {};
          for (uint32_t who = __ballot_sync(0xffffffffu, bad); who; who &= who - 1) {
            const int by = __ffs(who) - 1, pos = j * KVT + k + by;
            const bool here = pos >= lo && pos <= hi;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t v = __shfl_sync(0xffffffffu, u[e], by);
              if (here && !isfinite(low(v))) add[2 * e] += low(v);
              if (here && !isfinite(high(v))) add[2 * e + 1] += high(v);
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (add[e] == 0.f) continue;
            if (share) share[c + e] += add[e];
            else if (o) o[c + e] = __float2bfloat16(__bfloat162float(o[c + e]) + add[e]);
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------ attention

// Maps of the pages [page][row][kv head][feature], boxes of box_rows rows x 64 features inside a page (0: none).
struct Maps {
  CUtensorMap k, v;
  int box_rows;
};

template <int HDP>
__global__ void __launch_bounds__(Shape<HDP>::kThreads, 1) k_rows_attn(const __grid_constant__ Params P, const __grid_constant__ Maps G) {
  using S = Shape<HDP>;
  constexpr int QT = S::QT, KVT = S::KVT, NP = S::NP, NST = S::NST, kSoft = S::kSoft, kW = KVT / 32;
  extern __shared__ __align__(1024) uint8_t smem[];
  const RowsAttnArgs &a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hd = a.c.head_dim, g = P.g.d;
  const int hd16 = (hd + 15) & ~15;
  const uint32_t s_q = tc::smem_u32(smem + S::kQ), s_ring = tc::smem_u32(smem + S::kRing);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kBars);
  // full, empty: a stage has landed, has been used; s_full, p_full: scores, weights; pv_done: values added up; q_full
  uint64_t *full = bars, *empty = bars + NST, *s_full = bars + 2 * NST, *p_full = s_full + 2, *pv_done = s_full + 4,
           *q_full = s_full + 6, *p_half = s_full + 8, *drain = s_full + 10;
  uint32_t *masks = reinterpret_cast<uint32_t *>(bars + 32);  // [kNote][4]: positions of a tile that are there
  uint32_t *tmem_slot = masks + 4 * kNote;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *issue_lock = reinterpret_cast<int *>(tmem_slot + 2);
  Part &rg = *reinterpret_cast<Part *>(tmem_slot + 4);
  OddTiles &odd = *reinterpret_cast<OddTiles *>(&rg + 1);
  static_assert(2 * NST + 11 <= 32 && NST / 2 + 2 < kNote, "barriers, notes");

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      tc::mbar_init(&full[i], 32);
      tc::mbar_init(&empty[i], QT);   // both tiles of rows
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&s_full[b], 2);   // the products' completion, and the issuing thread (which has seen the stage's notes)
      tc::mbar_init(&p_half[b], 4);   // a warp of the four each
      tc::mbar_init(&p_full[b], 4);
      tc::mbar_init(&pv_done[b], 2);
      tc::mbar_init(&q_full[b], 128);
    }
    tc::mbar_init(drain, S::kMma);
    odd = OddTiles{0x7fffffff, -1, 0x7fffffff, -1};
    *abort_flag = 0;
    *issue_lock = 0;
    tc::fence_barrier_init();
  }
  dependency_wait();
  const int cta = blockIdx.x;
  if (P.part[cta].first == P.part[cta].end) {
    if (tid == 0) P.split[cta] = make_int4(0, 0, 0, 0);
    return;
  }
  if (tid < (int)sizeof(Part) / 16) reinterpret_cast<int4 *>(&rg)[tid] = reinterpret_cast<const int4 *>(P.part + cta)[tid];
  if (warp == kSoft) tc::tmem_alloc(tmem_slot, 512);  // (behind the wait: a block of the kernel before may still ask for tensor memory)
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto begin = [&](auto &w) {
    w.P = &P;
    w.rg = &rg;
    w.slot = reinterpret_cast<Slot *>(smem + S::kSlots) + 2 * warp;  // (of the warps that have slots)
    w.i = rg.item;
    w.kvh = rg.kvh;
  };

  if (warp < kSoft) {
    // ------------------------------------------------------------------------------ softmax and results: a lane a row
    if constexpr (S::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsSoft));
    const int t = warp >> 2, quad = warp & 3, r = quad * 32 + lane;  // of tile t of the item
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16, tO = tmem + S::kColO + t * HDP + lane_off;
    auto load_q = [&](const Item &d, int kvh, int sub) {
      const int cc = lane & 7;
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {
        const int row = quad * 32 + 4 * i + (lane >> 3), R = d.row0 + sub + row;
        const bool in = sub + row < d.rows;
        const int tok = (int)P.g.div(R), h = R - tok * g;
        const bf16 *q = in ? a.q + (int64_t)(d.tok0 + tok) * a.q_t + (int64_t)(kvh * g + h) * hd + cc * 8 : a.q;
#pragma unroll
        for (int kb = 0; kb < NP; ++kb) {
          const bool f_in = in && kb * 64 + cc * 8 < hd;
          attn::cp_async16(s_q + t * S::kQBytes + kb * (kSub * 128) + row * 128 + ((cc ^ (row & 7)) << 4), f_in ? q + kb * 64 : a.q, f_in);
        }
      }
    };
    Walk<KVT, true> w;
    begin(w);
    bool more = w.first(lane == 0);
    auto has_rows = [&](const Walk<KVT, true> &x) {  // whether tile t has anything to do in this CTA's part of the item
      int from, to;
      sub_range(x, t, QT == 2, from, to);
      return to > from;
    };
    auto slot_there = [&]() {  // what lane 0 has copied, for the warp
      attn::cp_async_wait_all();
      __syncwarp();
    };
    if (more && has_rows(w)) {
      load_q(w.d, w.kvh, sub_rows(w, t, QT == 2));
      attn::cp_async_wait_all();
      attn::fence_proxy_async();
      tc::mbar_arrive(&q_full[t]);
    }
    int n_s = 0, n_pv = 0, tile0 = 0;  // scores taken, products of values asked for, first tile of the item
    // The last product of values asked for is done, and all before it.  (With two score buffers their products take turns at two
    // barriers: the one before the last may not be done either when the last is waited for.)
    auto values_done = [&]() {
      const int n = n_pv - 1;
      return QT == 2 ? warp_wait(&pv_done[t], n & 1, abort_flag) : warp_wait(&pv_done[n & 1], (n >> 1) & 1, abort_flag);
    };
    // (a negative scale would make the largest score the smallest, and 0 times a mask's -inf is not -inf: scores are then scaled first)
    const bool odd_scale = !(P.scale_log2 > 0.f);
    const float sc = odd_scale ? 1.f : P.scale_log2;
    bool ok = true;
    int4 split = make_int4(0, 0, 0, 0);
    while (more) {
      int x, y, lo = 0, hi = 0x7fffffff;  // (a row that is not there attends all: no mask for its sake)
      sub_range(w, t, QT == 2, x, y);
      const int sub = sub_rows(w, t, QT == 2);
      const bool work = sub >= 0 && sub + quad * 32 < w.d.rows;  // (of the warp)
      if (work && sub + r < w.d.rows) {
        span(a, w.d.tok0 + (int)P.g.div(w.d.row0 + sub + r), w.d.shift, lo, hi);
      }
      float m = -INFINITY, l = 0.f, lr = 0.f;
      const int note0 = tile0 - (w.kt0 + w.u0);
      tile0 += w.u1 - w.u0;
      for (int j = x; j < y; ++j) {
        const int b = QT == 2 ? t : n_s & 1, at = j * KVT;
        const bool in_part = odd_scale || !__all_sync(0xffffffffu, lo <= at && hi - at >= KVT - 1);  // some row attends not all of the tile
        if (!(ok = warp_wait(&s_full[b], QT == 2 ? n_s & 1 : (n_s >> 1) & 1, abort_flag))) break;
        tc::tc_fence_after();
        if (at < w.d.at0 || w.d.at1 - at < KVT) {  // (at + KVT may pass 31 bits)
          // A weight of 0 does not undo a NaN: in a tile that not every row of the item attends, values that are not finite are
          // taken out before the product (by both tiles of rows, whichever comes first), and the rows that attend them get them
          // at the CTA's end.  (Behind the scores: only then is the stage's barrier in the phase that is asked for, or the next.)
          const int stage = 2 * (note0 + j) + 1, rows = tile_rows<KVT>(w.d.end, j);
          if (!(ok = warp_wait(&full[stage % NST], (uint32_t)((stage / NST) & 1), abort_flag))) break;
          const uint32_t v_at = s_ring + (stage % NST) * S::kStage + r * 16;
          uint32_t bits = 0;
#pragma unroll 4
          for (int i = 0; i < S::kStage / 16 / kSub; ++i) {
            uint32_t z[4];
            lds4(z, v_at + i * (kSub * 16));
#pragma unroll
            for (int k = 0; k < 4; ++k) bits |= (z[k] & 0x7f807f80u) + 0x00800080u;  // (a carry where an exponent is all ones)
          }
          if (__builtin_expect((bits & 0x80008000u) != 0, 0))
            clear_odd<KVT>(v_at, S::kStage / 16 / kSub, r, rows, &odd, w.seq, j);
          attn::fence_proxy_async();
        }
        if (work) {
          const uint32_t tS = tmem + b * KVT + lane_off;
          const uint32_t *there = masks + 4 * ((note0 + j) & (kNote - 1));  // positions that are there
          const uint4 mk = *reinterpret_cast<const uint4 *>(there);
          if (__builtin_expect(in_part || (kW == 4 ? (mk.x & mk.y & mk.z & mk.w) : (mk.x & mk.y)) != 0xffffffffu, 0))
            mask_scores<KVT>(tS, odd_scale ? P.scale_log2 : 1.f, lo - at, hi - at, there);
          ok = weights<HDP>(sc, m, l, lr, j == x, tS, tO, hd16, &p_half[b], &p_full[b], lane, values_done);
          if (!ok) break;
        } else {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(&p_half[b]);
            tc::mbar_arrive(&p_full[b]);
          }
        }
        ++n_s;
        ++n_pv;
      }
      if (!ok) break;
      // ---- the end of the item in this CTA; the next one's q comes beside the last values (its last reader is done; w stays, not to
      // hold two items in registers)
      bool q_next = false;
      {
        slot_there();
        Walk<KVT, true> nx = w;
        const bool there = nx.peek();
        ++nx.seq;
        if (there && has_rows(nx)) {
          load_q(nx.d, nx.kvh, sub_rows(nx, t, QT == 2));
          q_next = true;
        }
      }
      if (y > x) {
        if (!(ok = values_done())) break;
        tc::tc_fence_after();
      }
      if (q_next) {
        attn::cp_async_wait_all();
        attn::fence_proxy_async();
        tc::mbar_arrive(&q_full[t]);
      }
      if (work) {
        const Item &d = w.d;
        const int R = sub + r, q = (int)P.g.div(d.row0 + R), tok = d.tok0 + q, h = w.kvh * g + (d.row0 + R - q * g);
        const bool whole = w.whole(), mine = R < d.rows, live = mine && row_live(a, tok);
        if (m != -INFINITY) m *= sc;
        float f = 1.f, f_own = 0.f;
        float *share = nullptr;
        bf16 *o = nullptr;
        const float *own = nullptr;
        if (whole) {
          float2 oml = make_float2(-INFINITY, 0.f);
          if (live && P.own_o) {
            oml = P.own_ml[(int64_t)tok * a.H + h];
            own = P.own_o + ((int64_t)tok * a.H + h) * hd;
          }
          const Finish fin = finish(m, lr, l, oml, a.sink, h);
          f = fin.f;
          f_own = fin.f_own;
          if (live && a.lse) a.lse[(int64_t)tok * a.H + h] = fin.lse;
          o = a.o + (int64_t)tok * a.o_t + (int64_t)h * hd;
        } else {
          const int64_t at = (int64_t)(2 * cta + (w.u0 == 0 ? 1 : 0)) * (QT * kSub) + R;
          share = P.share_o + at * HDP;
          if (mine) P.share_ml[at] = make_float4(m, lr, l, 0.f);
        }
        if (whole && P.own_o) {
          out_with_own(tO, y > x, f, own, f_own, hd, live ? o : nullptr);
        } else {
#pragma unroll 1
          for (int c = 0; c < hd; c += 16) {
            uint32_t u[16];
            __syncwarp();
            if (y > x) {
              tc::tmem_ld16_wait(tO + c, u);
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k) u[k] = 0u;
            }
            if (share) {
              if (mine) {
                store32(share + c, u);
                store32(share + c + 8, u + 8);
              }
            } else if (live) {
              float v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(u[k]) * f;
#pragma unroll
              for (int k = 0; k < 8; ++k) u[k] = pack2(v[2 * k], v[2 * k + 1]);
              if (P.wide) {  // (rows of whole 32 bytes, on their borders)
                store32(o + c, u);
              } else {
                *reinterpret_cast<uint4 *>(o + c) = make_uint4(u[0], u[1], u[2], u[3]);
                if (c + 8 < hd) *reinterpret_cast<uint4 *>(o + c + 8) = make_uint4(u[4], u[5], u[6], u[7]);
              }
            }
          }
        }
        tc::tc_fence_before();
      }
      if (tid == 0 && w.u0 == 0 && w.u1 < w.tiles) {  // (the CTA's last item: it goes on in the next ones)
        const unsigned long long last_place = w.base + w.tiles - 1;
        int c = cta;
        while (c + 1 < P.ctas && P.part[c + 1].first < P.part[c + 1].end && P.part[c + 1].first <= last_place) ++c;
        split = make_int4(w.i, w.kvh, c - cta + 1, 0);
      }
      slot_there();
      more = w.next(lane == 0);
    }
    attn::cp_async_wait_all();
    if (tid == 0) P.split[cta] = split;
  } else {
    if constexpr (S::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsRest));
    if (warp < kSoft + S::kMma) {
      // ------------------------------------------------------------------------------ products, issued by one elected lane
      if (tc::elect_one()) {
        const uint32_t id_s = tc::idesc_bf16_f32(kSub, KVT), id_v = tc::idesc_bf16_f32(kSub, hd16, false, /*b_mn_major=*/true);
        const uint32_t dq = (uint32_t)tc::sdesc_sw128(s_q, 16, 1024), dk = (uint32_t)tc::sdesc_sw128(s_ring, 16, 1024),
                       dv = (uint32_t)tc::sdesc_sw128(s_ring, KVT * 128, 1024);
        const uint64_t hi = tc::sdesc_sw128(0, 16, 1024) & 0xffffffff00000000ull;
        const int ks = hd16 / 16;
        int s = 0;  // stages so far
        auto stage_ready = [&](int i) { return wait(&full[i % NST], (uint32_t)((i / NST) & 1), abort_flag); };
        // A warp has one tile of rows of each item, and lets the stages that the tile attends nothing of pass by.
        const int t = warp - kSoft;
        Walk<KVT, true> w;
        begin(w);
        bool more = w.first(true);
        uint32_t n_q = 0, n_s = 0, n_p = 0;
        const uint32_t dO = tmem + S::kColO + t * HDP;
        auto buffer = [&](uint32_t n) { return QT == 2 ? (uint32_t)t : n & 1; };
        auto phase = [&](uint32_t n) { return QT == 2 ? n & 1 : (n >> 1) & 1; };
        auto scores = [&](int stage) {
          const uint32_t A = dq + t * (S::kQBytes >> 4), B = dk + (stage % NST) * (S::kStage >> 4), b = buffer(n_s++);
          const uint32_t d = tmem + b * KVT;
          uint32_t al = A, bl = B;
          int k = 0;
#pragma unroll 1
          for (; k + 4 <= ks; k += 4, al += kSub * 128 >> 4, bl += KVT * 128 >> 4)
#pragma unroll
            for (int e = 0; e < 4; ++e) tc::mma_bf16(d, hi | (al + 2 * e), hi | (bl + 2 * e), id_s, e ? 1u : (k ? 1u : 0u));
#pragma unroll 1
          for (; k < ks; ++k, al += 2, bl += 2) tc::mma_bf16(d, hi | al, hi | bl, id_s, k ? 1u : 0u);
          tc::mma_commit(&s_full[b]);
          tc::mbar_arrive(&s_full[b]);
        };
        auto values = [&](int stage, int half, int rows, bool first) {  // (the half's weights are there)
          tc::tc_fence_after();
          const uint32_t A = tmem + buffer(n_p) * KVT, B = dv + (stage % NST) * (S::kStage >> 4);
          if (rows == KVT) {  // (known counts: 2 % of a long prompt's time)
#pragma unroll 2
            for (int k = 0; k < KVT / 32; ++k) {
              const int kk = half * (KVT / 32) + k;
              mma_ts(dO, A + 8 * kk, hi | (B + kk * 128), id_v, first && kk == 0 ? 0u : 1u);
            }
          } else {
#pragma unroll 1
            for (int k = half * (KVT / 32); k < min((half + 1) * (KVT / 32), rows / 16); ++k)
              mma_ts(dO, A + 8 * k, hi | (B + k * 128), id_v, first && k == 0 ? 0u : 1u);
          }
        };
        // The two warps' products come in groups, each as a whole behind the other's: one tile's scores are then there while the other's
        // are computed (product by product in turn, both would be late, and both softmaxes run at once).
        auto lock = [&]() -> bool {
          uint32_t spins = 0;
          uint64_t t0 = 0;
          while (QT == 2 && atomicCAS(issue_lock, 0, 1) != 0)
            if ((++spins & 255) == 0) {
              if (t0 == 0) t0 = tc::global_ns();
              if (*abort_flag || tc::global_ns() - t0 > tc::kWaitLimitNs) return false;
            }
          return true;
        };
        auto unlock = [&]() {
          if (QT == 2) atomicExch(issue_lock, 0);
        };
        bool ok = true;
        while (more) {
          const int j0 = w.kt0 + w.u0, j1 = w.kt0 + w.u1;
          int x, y;
          sub_range(w, t, QT == 2, x, y);
          auto keys_there = [&](int j, int stage) {
            return stage_ready(stage) && (j != x || x == y || wait(&q_full[t], n_q++ & 1, abort_flag));
          };
          auto keys = [&](int j, int stage) {  // tile j's scores
            if (x <= j && j < y) scores(stage);
            tc::mma_commit(&empty[stage % NST]);
          };
          ok = keys_there(j0, s) && lock();
          if (!ok) break;
          keys(j0, s);
          unlock();
          for (int j = j0; j < j1; ++j, s += 2) {
            const bool live = x <= j && j < y, next = j + 1 < j1;
            const int rows = tile_rows<KVT>(w.d.end, j);
            if (QT == 1 && next) {  // (the other score buffer: before this tile's values)
              if (!(ok = keys_there(j + 1, s + 2))) break;
              keys(j + 1, s + 2);
            }
            if (!(ok = stage_ready(s + 1))) break;
            if (live) {
              const uint32_t b = buffer(n_p), ph = phase(n_p);
              if (!(ok = wait(&p_half[b], ph, abort_flag))) break;
              values(s + 1, 0, rows, j == x);
              if (!(ok = wait(&p_full[b], ph, abort_flag))) break;
            }
            if (QT == 2 && next) {
              if (!(ok = keys_there(j + 1, s + 2))) break;
            }
            ok = lock();
            if (!ok) break;
            if (live) {
              values(s + 1, 1, rows, false);
              const uint32_t b = buffer(n_p++);
              tc::mma_commit(&pv_done[b]);
              tc::mbar_arrive(&pv_done[b]);
            }
            tc::mma_commit(&empty[(s + 1) % NST]);
            if (QT == 2 && next) keys(j + 1, s + 2);
            unlock();
          }
          if (!ok) break;
          attn::cp_async_wait_all();
          more = w.next(true);
        }
        // nothing may still read shared memory, write tensor memory or arrive when the CTA ends
        tc::mma_commit(drain);
        const uint64_t t1 = tc::global_ns();
        while (!tc::mbar_try_wait(drain, 0) && tc::global_ns() - t1 < tc::kWaitLimitNs) {
        }
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------------------ copies: a warp every second or third stage
      // The pages of a warp's next stage are looked up while its copies are in flight.
      const int lw = warp - kSoft - S::kMma, cc = lane & 7;
      Walk<KVT, false> w;
      begin(w);
      bool more = w.first(false);
      struct Look {
        int page[kW];
        uint32_t at;     // first position
        int kvh, seg, begin, end, tile;
        bool values;
      };
      int s = lw, x = lw, tile0 = 0;  // stage, stage of the item, first tile of the item
      auto look = [&](Look &f) __attribute__((always_inline)) -> bool {
        while (more && x >= 2 * (w.u1 - w.u0)) {
          x -= 2 * (w.u1 - w.u0);
          tile0 += w.u1 - w.u0;
          more = w.next(false);
        }
        if (!more) return false;
        const Item &d = w.d;
        f.at = (uint32_t)(w.kt0 + w.u0 + (x >> 1)) * KVT;
        f.values = x & 1;
        f.kvh = w.kvh;
        f.begin = d.begin;
        f.end = d.end;
        f.seg = d.seg;
        f.tile = tile0 + (x >> 1);
#pragma unroll
        for (int k = 0; k < kW; ++k) {
          const uint32_t p = f.at + 32 * k + lane;
          const bool in = p >= (uint32_t)d.begin && p < (uint32_t)d.end;
          f.page[k] = in ? a.table[(int64_t)d.seg * a.width + P.page.div(p)] : 0;
        }
        return true;
      };
      Look f{};
      if (G.box_rows && lane == 0) {
        tc::prefetch_tmap(&G.k);
        if (a.c.v) tc::prefetch_tmap(&G.v);
      }
      for (bool begun = false, have = true; have; begun = true) {  // (from the second round on with a stage to fill)
        const uint32_t dst = s_ring + (s % NST) * S::kStage + (lane >> 3) * 128;
        const int cur = s;
        bool copied = false;  // by cp.async
        if (begun) {
          const bool vals = f.values && a.c.v;
          const bf16 *src = reinterpret_cast<const bf16 *>(vals ? a.c.v : a.c.k) + f.kvh * (vals ? a.c.v_head : a.c.k_head) + cc * 8;
          const int64_t st_page = vals ? a.c.v_page : a.c.k_page, st_row = vals ? a.c.v_row : a.c.k_row;
          const int buf = s % NST;
          uint32_t there[kW], all = 0xffffffffu;  // positions that are there
#pragma unroll
          for (int k = 0; k < kW; ++k) {
            const uint32_t p = f.at + 32 * k + lane;
            const bool in = p >= (uint32_t)f.begin && p < (uint32_t)f.end, good = in && f.page[k] >= 0 && f.page[k] < a.c.n_pages;
            if (in && !good) atomicOr(a.status, kStatusBadIndex);
            all &= there[k] = __ballot_sync(0xffffffffu, good);
          }
          if (s >= NST && !warp_wait(&empty[buf], (uint32_t)((s / NST - 1) & 1), abort_flag)) break;
          if (!f.values && lane == 0)
#pragma unroll
            for (int k = 0; k < kW; ++k) masks[4 * (f.tile & (kNote - 1)) + k] = there[k];
          if (G.box_rows && all == 0xffffffffu) {
            // A whole tile: by TMA, a lane a box.
            const int R = G.box_rows, first = lane * R;
            int page = 0;
#pragma unroll
            for (int k = 0; k < kW; ++k) {
              const int x0 = __shfl_sync(0xffffffffu, f.page[k], first & 31);
              if ((first >> 5) == k) page = x0;
            }
            if (lane == 0) tc::mbar_expect_tx(&full[buf], S::kStage);
            __syncwarp();
            if (first < KVT) {
              const uint32_t p = f.at + first;
              const int row = (int)(p - P.page.div(p) * P.page.d);
#pragma unroll
              for (int kb = 0; kb < NP; ++kb)
                tc::tma_load_4d(s_ring + buf * S::kStage + kb * (KVT * 128) + first * 128, vals ? &G.v : &G.k, &full[buf], kb * 64,
                                f.kvh, row, page);
            }
            if (lane != 0) tc::mbar_arrive(&full[buf]);
          } else {
            copied = true;
            const int rows = tile_rows<KVT>(f.end, (int)(f.at / KVT));
#pragma unroll 1
            for (int k = 0; 32 * k < rows; ++k) {  // (rolled: four times the code would be fetched anew for every stage)
              int page = f.page[0];
              uint32_t good = there[0];
#pragma unroll
              for (int e = 1; e < kW; ++e)
                if (k == e) page = f.page[e], good = there[e];
              const uint32_t p = f.at + 32 * k + lane;
              const int64_t off = (good >> lane) & 1u ? page * st_page + (int64_t)(p - P.page.div(p) * P.page.d) * st_row : -1;
#pragma unroll 2
              for (int i = 0; i < 8; ++i) {  // four rows at a time, eight lanes 128 bytes of a row
                if (32 * k + 4 * i >= rows) break;
                const int r7 = (4 * i + (lane >> 3)) & 7;
                const int64_t o = __shfl_sync(0xffffffffu, off, 4 * i + (lane >> 3));
#pragma unroll
                for (int kb = 0; kb < NP; ++kb) {
                  const bool in = o >= 0 && kb * 64 + cc * 8 < hd;
                  attn::cp_async16(dst + kb * (KVT * 128) + k * 4096 + i * 512 + ((cc ^ r7) << 4), in ? src + o + kb * 64 : src, in);
                }
              }
            }
          }
          s += S::kLoad;
          x += S::kLoad;
        }
        have = look(f);
        if (!copied) continue;
        attn::cp_async_wait_all();
        attn::fence_proxy_async();
        tc::mbar_arrive(&full[cur % NST]);
      }
      attn::cp_async_wait_all();
      // Nothing is in flight when the CTA ends.  The products wait for every stage; after a wait that ran out, they do not.
      if (*abort_flag)
        for (int i = s - S::kLoad; i >= 0 && i > s - S::kLoad - NST; i -= S::kLoad) {
          const uint64_t t1 = tc::global_ns();
          while (!tc::mbar_try_wait(&full[i % NST], (uint32_t)((i / NST) & 1)) && tc::global_ns() - t1 < 10000000) {
          }
        }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kSoft) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && *abort_flag) atomicOr(a.status, kStatusTimeout);
  // (a share or result is its lane's own; *abort_flag: results are lost anyway)
  if (warp < kSoft && !*abort_flag && __any_sync(0xffffffffu, odd.any())) odd_values<HDP>(P, &rg, &odd);
}

// ------------------------------------------------------------------------------------------------ joining

constexpr int kJoinThreads = 256, kJoinAhead = 6;

template <int HDP>
__global__ void __launch_bounds__(kJoinThreads) k_rows_join(const __grid_constant__ Params P, int ctas) {
  constexpr int kRows = Shape<HDP>::QT * kSub, kLanes = HDP / 4;
  const RowsAttnArgs &a = P.a;
  dependency_wait();
  const int c0 = blockIdx.x;
  const int4 sp = P.split[c0];
  const int parts = sp.z, hd = a.c.head_dim, g = P.g.d;
  // (after a wait that ran out the notes may be those of another call: nothing outside the workspace is read)
  if (parts <= 1 || parts > ctas - c0 || sp.x < 0 || sp.x >= P.part[0].items || sp.y < 0 || sp.y >= a.c.kv_heads) return;
  const int4 x = reinterpret_cast<const int4 *>(P.item + sp.x)[0];
  for (int i = blockIdx.y * kJoinThreads + threadIdx.x; i < x.z * kLanes; i += gridDim.y * kJoinThreads) {
    const int r = i / kLanes, dd = (i - r * kLanes) * 4;
    if (dd >= hd) continue;
    const int q = (int)P.g.div(x.y + r), tok = x.x + q, h = sp.y * g + (x.y + r - q * g);
    if (tok >= a.N || !row_live(a, tok)) continue;
    float M = -INFINITY, Lr = 0.f, L = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += kJoinAhead) {
      float4 o[kJoinAhead], ml[kJoinAhead];
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) {
        ml[u] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
        o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p0 + u < parts) {
          const int64_t at = (int64_t)(p0 + u == 0 ? 2 * c0 + 1 : 2 * (c0 + p0 + u)) * kRows + r;
          ml[u] = __ldcg(P.share_ml + at);
          o[u] = __ldcg(reinterpret_cast<const float4 *>(P.share_o + at * HDP + dd));
        }
      }
      float top = M;
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) top = fmaxf(top, ml[u].x);
      const float ref = top == -INFINITY ? 0.f : top, f0 = exp2f(M - ref);
      M = top;
      L *= f0;
      Lr *= f0;
      v.x *= f0;
      v.y *= f0;
      v.z *= f0;
      v.w *= f0;
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) {
        const float f = exp2f(ml[u].x - ref);
        Lr = fmaf(ml[u].y, f, Lr);
        L = fmaf(ml[u].z, f, L);
        v.x = fmaf(o[u].x, f, v.x);
        v.y = fmaf(o[u].y, f, v.y);
        v.z = fmaf(o[u].z, f, v.z);
        v.w = fmaf(o[u].w, f, v.w);
      }
    }
    float2 oml = make_float2(-INFINITY, 0.f);
    float4 own = make_float4(0.f, 0.f, 0.f, 0.f);
    if (P.own_o) {
      oml = P.own_ml[(int64_t)tok * a.H + h];
      own = *reinterpret_cast<const float4 *>(P.own_o + ((int64_t)tok * a.H + h) * hd + dd);
    }
    const Finish fin = finish(M, Lr, L, oml, a.sink, h);
    *reinterpret_cast<uint2 *>(a.o + (int64_t)tok * a.o_t + (int64_t)h * hd + dd) =
        make_uint2(pack2(fmaf(own.x, fin.f_own, v.x * fin.f), fmaf(own.y, fin.f_own, v.y * fin.f)),
                   pack2(fmaf(own.z, fin.f_own, v.z * fin.f), fmaf(own.w, fin.f_own, v.w * fin.f)));
    if (a.lse && dd == 0) a.lse[(int64_t)tok * a.H + h] = fin.lse;
  }
}

// ------------------------------------------------------------------------------------------------ launch

// Hands out parts of the workspace.
struct Room {
  uint8_t *at, *end;
  template <class T>
  T *take(size_t n) {
    uint8_t *p = at;
    at += (n * sizeof(T) + 255) / 256 * 256;
    return reinterpret_cast<T *>(p);
  }
};

// What runs beside the plan: the rows' own pages, or the segments of one token.  (In one grid: 64 rows of 40 to 700 own positions behind
// 8192 53.5 us, two launches in a row 57.7; 2 x 500 20.7, 22.9.)
struct Beside {
  PagedAttnArgs a;
  float *shares;
  int *counters;
};

template <int HDP>
cudaError_t launch(Params p, Room room, const Beside *beside, int num_sms, cudaStream_t s) {
  using S = Shape<HDP>;
  const RowsAttnArgs &a = p.a;
  constexpr int TR = S::QT * kSub;
  static SmemAttr attr;
  cudaError_t e = attr.ensure((const void *)k_rows_attn<HDP>, S::kSmem);
  if (e != cudaSuccess) return e;
  const int g = a.H / a.c.kv_heads;
  const int64_t cap = ((int64_t)a.N * g + TR - 1) / TR + a.S;
  // no more CTAs than can get places (so that their number, and with it the split, does not go by rows that are padding)
  const int64_t rows = (int64_t)a.width * a.c.page;
  const int64_t tiles = (a.window > 0 ? std::min<int64_t>(rows, (int64_t)a.window + TR) : rows) / S::KVT + 2;
  const bool one = rows <= S::KVT;  // (every item has one tile: nothing is shared)
  const int64_t each = one ? 1 : std::max(tiles, (tiles + end_tiles<HDP>(true) + 1) / kMinPlaces);
  const int64_t most = (double)cap * a.c.kv_heads * each > 1e9 ? num_sms : cap * a.c.kv_heads * each;
  const int grid = (int)std::min<int64_t>(num_sms, most);
  p.cap = (int)cap;
  p.part = room.take<Part>(grid + 1);
  p.ctas = grid;
  p.item = room.take<Item>(cap);
  p.start = room.take<unsigned long long>(cap + 1);
  p.split = room.take<int4>(grid);
  p.share_ml = room.take<float4>((size_t)2 * grid * TR);
  p.share_o = room.take<float>((size_t)2 * grid * TR * HDP);
  if (room.at > room.end || cap > (1 << 24)) return cudaErrorInvalidValue;
  // TMA where pages hold whole boxes of 8 rows (the swizzle's period) or more, up to a tile
  Maps maps;
  memset((void *)&maps, 0, sizeof(maps));
  const int box = std::min(a.c.page & -a.c.page, S::KVT);
  if (box >= 8) {
    auto map = [&](CUtensorMap *m, const void *base, int64_t page, int64_t row, int64_t head) {
      if ((a.c.kv_heads > 1 && head == 0) || (a.c.page > 1 && row == 0) || (a.c.n_pages > 1 && page == 0)) return false;  // (one for all)
      const uint64_t dims[4] = {(uint64_t)a.c.head_dim, (uint64_t)a.c.kv_heads, (uint64_t)a.c.page, (uint64_t)a.c.n_pages};
      const uint64_t one_row = 2 * (uint64_t)a.c.head_dim;  // (strides of dimensions of size 1 may be anything)
      const uint64_t strides[3] = {a.c.kv_heads > 1 ? 2 * (uint64_t)head : one_row, a.c.page > 1 ? 2 * (uint64_t)row : one_row,
                                   a.c.n_pages > 1 ? 2 * (uint64_t)page : one_row};
      return tma_map_pages_bf16(m, base, dims, strides, 64, (uint32_t)box);
    };
    if (map(&maps.k, a.c.k, a.c.k_page, a.c.k_row, a.c.k_head) &&
        (!a.c.v || map(&maps.v, a.c.v, a.c.v_page, a.c.v_row, a.c.v_head)))
      maps.box_rows = box;
  }
  p.end_tiles = end_tiles<HDP>(maps.box_rows > 0);
  p.rows_log2 = TR == 256 ? 8 : 7;
  p.tile_log2 = S::KVT == 128 ? 7 : 6;
  const Plan &plan = p;
  e = beside ? launch_paged_attn(beside->a, beside->shares, kPagedShareBytes, beside->counters, num_sms, s, &plan)
             : launch_dependent(k_rows_plan, dim3(1), dim3(kPlanThreads), 0, s, 1, plan);
  if (e == cudaSuccess) e = launch_dependent(k_rows_attn<HDP>, dim3(grid), dim3(S::kThreads), S::kSmem, s, 1, p, maps);
  if (e != cudaSuccess || one) return e;
  // blocks of the join: a thread a quarter of 16 features; more of them an item where items are few, and so split over many CTAs
  const int64_t all = (int64_t)TR * HDP / 4 / kJoinThreads, few = std::min<int64_t>(cap * a.c.kv_heads, grid);
  const int64_t y = std::min(all, std::max<int64_t>(4, 8 * num_sms / few));
  return launch_dependent(k_rows_join<HDP>, dim3(grid, (unsigned)y), dim3(kJoinThreads), 0, s, 1, p, grid);
}

}  // namespace rows

// Whether a prompt batch's segments of one token go to k_paged_attn: up to 8 query heads a kv head, always, so that neither the other
// requests nor padding rows change how a token is computed.  There it takes half the time over them (64 of up to 5000 positions, 32 heads
// over 8 of 128: 41 against 73 us; 32 of up to 64000 beside a chunk of 2000 309, 330; 15 of 16 to 64 thousand beside one of 8200 1185,
// 1262; 15 of 1 to 32 thousand beside 8200, 32 over 8 of 64, 820, 858; four of 64000 beside 8200 1033, 1062), and where there are none it
// costs no more than the plan alone (4096 tokens 277, 276 us; 12 prompts of 100 to 4000 312 both).  It is slower where few single tokens are
// short (one beside 4 windows of up to 6001, 16 of 256: 214, 209; 4 of up to 64000 beside 2000: 224, 217).  With 16 heads a kv head it is
// not faster (32 of 2000 to 8000, 32 over 2 of 128: 48 against 46 us; 16 of 3000 to 9000, 32 over 2 of 256: 64, 51).
static bool single_tokens(const RowsAttnArgs &a) { return !a.pos && a.H / a.c.kv_heads <= 8; }

// Bytes of workspace that launch_rows_attn needs (an upper bound).
size_t rows_attn_bytes(const RowsAttnArgs &a, int num_sms) {
  const size_t hd = (size_t)(a.c.head_dim + 63) / 64 * 64, items = (size_t)a.N * (a.H / a.c.kv_heads) / 128 + 1 + a.S;
  const size_t shares = (size_t)2 * num_sms * (hd == 256 ? 128 : 256) * (hd * 4 + 16);
  const size_t own = a.pos ? (size_t)a.N * a.H * (a.c.head_dim * 4 + 8) : 0;
  return items * 56 + shares + own + (a.pos || single_tokens(a) ? kPagedShareBytes : 0) + (num_sms + 1) * 112 + 8192;
}

cudaError_t launch_rows_attn(const RowsAttnArgs &a, float *ws, size_t ws_bytes, int *counters, int num_sms, cudaStream_t s) {
  rows::Params p;
  memset((void *)&p, 0, sizeof(p));
  p.a = a;
  p.page = paged::FastDiv((uint32_t)a.c.page);
  p.g = paged::FastDiv((uint32_t)(a.H / a.c.kv_heads));
  p.scale_log2 = (float)(a.scale * 1.4426950408889634);
  p.wide = ((uintptr_t)a.o | (uintptr_t)(a.o_t * 2) | (uintptr_t)(a.c.head_dim * 2)) % 32 == 0;
  rows::Room room{reinterpret_cast<uint8_t *>(ws), reinterpret_cast<uint8_t *>(ws) + ws_bytes};
  rows::Beside beside{};
  PagedAttnArgs &o = beside.a;
  p.single = single_tokens(a);
  if (a.pos || p.single) {
    o.q = a.q;
    o.q_t = a.q_t;
    o.H = a.H;
    o.c = a.c;
    o.scale = a.scale;
    o.window = a.window;
    o.status = a.status;
    beside.counters = counters;
    if (a.pos) {
      o.N = a.N;
      o.table = a.own_table;
      o.R = a.R;
      o.width = a.own_width;
      o.req = a.req;
      o.pos = a.pos;
      p.own_o = o.part_o = room.take<float>((size_t)a.N * a.H * a.c.head_dim);
      p.own_ml = o.part_ml = room.take<float2>((size_t)a.N * a.H);
    } else {
      o.N = o.R = a.S;
      o.table = a.table;
      o.width = a.width;
      o.cu = a.cu;
      o.len = a.len;
      o.tokens = a.N;
      o.sink = a.sink;
      o.o = a.o;
      o.o_t = a.o_t;
      o.lse = a.lse;
    }
    beside.shares = room.take<float>(kPagedShareBytes / 4);
  }
  const rows::Beside *b = a.pos || p.single ? &beside : nullptr;
  const int hd = a.c.head_dim;
  if (hd <= 64) return rows::launch<64>(p, room, b, num_sms, s);
  if (hd <= 128) return rows::launch<128>(p, room, b, num_sms, s);
  if (hd <= 192) return rows::launch<192>(p, room, b, num_sms, s);
  return rows::launch<256>(p, room, b, num_sms, s);
}

}  // namespace csa
