// k_page_step.cu -- the token maps and block tables of one step of a continuous batch, from the requests'
// lengths.
//
// With add_r = max(new_r, 0), have_r = ceil(length_r / page), need_r = ceil((length_r + add_r) / page) - have_r
// and back_r = have_r of a request that ended (else 0), everything follows from the three running sums over r:
// token t belongs to the first r whose running sum of add exceeds t, at position length_r + t - (tokens before
// r); taken page i goes to the first r whose running sum of need exceeds i, and is entry head + i of the ring;
// released page i likewise.  A page of a token is either one the request had (its table entry, which this
// step does not write) or one it takes now (a ring entry), so no thread reads what another one writes.
//
// Bound by latency: a 64-token step moves 2 KB and takes 3.2 us, 1500 requests 8.8 us (device times).
// One CTA does small steps; larger ones (above 2048 tokens or requests, or with long tables) take one cluster of
// eight CTAs, each of which forms the sums for itself (R <= 14000 lengths from L2, kept in its shared memory)
// and takes an eighth of the tokens and pages.  The hardware's cluster barrier, after everything has been
// read, lets length_out and state_out be length and state: one launch, and no counter that two calls could
// share.
#include "csa_internal.cuh"
#include "paged_common.cuh"

namespace csa {
namespace {

constexpr int kClusterCtas = 8;
constexpr uint32_t kCap = 1u << 30;  // the sums saturate here, above every count that is accepted (two of them fit 32 bits)

__device__ __forceinline__ uint32_t sat(uint32_t a, uint32_t b) { return min(a + b, kCap); }

struct Sums {
  uint32_t add, need, back;
};
__device__ __forceinline__ Sums plus(Sums a, Sums b) { return {sat(a.add, b.add), sat(a.need, b.need), sat(a.back, b.back)}; }
__device__ __forceinline__ Sums shfl_up(Sums v, int d) {
  return {__shfl_up_sync(0xffffffffu, v.add, d), __shfl_up_sync(0xffffffffu, v.need, d),
          __shfl_up_sync(0xffffffffu, v.back, d)};
}

// The first index of the non-decreasing incl[0..n) whose value exceeds x (x below the last one).
__device__ __forceinline__ int first_above(const uint32_t *incl, int n, uint32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (incl[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(1024) k_page_step(const __grid_constant__ PageStepArgs a, const __grid_constant__ paged::FastDiv a_page) {
  extern __shared__ uint32_t sm[];  // running sums of add, need, back and the lengths: [R] each
  uint32_t *s_add = sm, *s_need = sm + a.R, *s_back = sm + 2 * a.R;
  int *s_len = reinterpret_cast<int *>(sm + 3 * a.R);
  __shared__ Sums s_warp[32];
  __shared__ int s_err;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, wid = tid >> 5, nw = nt >> 5;
  const int gt = blockIdx.x * nt + tid, gn = gridDim.x * nt;  // over the cluster
  if (tid == 0) s_err = 0;
  dependency_wait();
  const int head = a.state[0], count = a.state[1];
  __syncthreads();
  // ---- the running sums: a thread takes `per` requests in a row
  const int per = (a.R + nt - 1) / nt, r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
  Sums mine{0, 0, 0};
  int err = 0;
  for (int r = r0; r < r1; ++r) {
    const int len = a.length[r], nw_r = a.new_len[r];
    s_len[r] = len;
    const int have = len < 0 ? 0 : (int)a_page.div((uint32_t)min((int64_t)len + a.page - 1, (int64_t)0x7fffffff));
    Sums one{0, 0, 0};
    if (len < 0 || have > a.width) {
      err |= 2;
    } else if (nw_r > a.N) {
      err |= 1;
    } else if (nw_r > 0) {
      const int64_t after = a_page.div((uint32_t)min((int64_t)len + nw_r + a.page - 1, (int64_t)0x7fffffff));
      if (after > a.width)
        err |= 2;
      else
        one = {(uint32_t)nw_r, (uint32_t)(after - have), 0};
    } else if (nw_r < 0) {
      one.back = (uint32_t)have;
    }
    mine = plus(mine, one);
    s_add[r] = mine.add;
    s_need[r] = mine.need;
    s_back[r] = mine.back;
  }
  if (err) atomicOr(&s_err, err);
  Sums incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shfl_up(incl, d);
    if (lane >= d) incl = plus(incl, o);
  }
  if (lane == 31) s_warp[wid] = incl;
  __syncthreads();
  if (wid == 0) {
    Sums w = lane < nw ? s_warp[lane] : Sums{0, 0, 0};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums o = shfl_up(w, d);
      if (lane >= d) w = plus(w, o);
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  Sums before = shfl_up(incl, 1);
  if (lane == 0) before = {0, 0, 0};
  if (wid > 0) before = plus(before, s_warp[wid - 1]);
  for (int r = r0; r < r1; ++r) {
    s_add[r] = sat(s_add[r], before.add);
    s_need[r] = sat(s_need[r], before.need);
    s_back[r] = sat(s_back[r], before.back);
  }
  const Sums total = s_warp[nw - 1];
  err = s_err;
  if (total.add > (uint32_t)a.N) err |= 1;
  if (head < 0 || head >= a.n_pages || count < 0 || count > a.n_pages || total.back > (uint32_t)(a.n_pages - count))
    err |= 8;
  else if (total.need > (uint32_t)count)
    err |= 4;
  __syncthreads();
  // ---- tokens, four a thread at a time (their searches and loads side by side)
  const int n_tok = err ? 0 : (int)total.add;
  constexpr int kAtOnce = 4;
  for (int t0 = gt; t0 < a.N; t0 += kAtOnce * gn) {
    int req[kAtOnce], pos[kAtOnce], id[kAtOnce], at[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int t = t0 + k * gn;
      req[k] = pos[k] = -1;
      if (t < n_tok) {
        req[k] = first_above(s_add, a.R, (uint32_t)t);
        pos[k] = t - (int)(req[k] ? s_add[req[k] - 1] : 0u);
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (req[k] >= 0) pos[k] += s_len[req[k]];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      id[k] = -1;
      at[k] = 0;
      if (req[k] < 0) continue;
      const uint32_t p = a_page.div((uint32_t)pos[k]), have = a_page.div((uint32_t)(s_len[req[k]] + a.page - 1));
      at[k] = pos[k] - (int)p * a.page;
      if (p < have) {
        id[k] = a.table[(int64_t)req[k] * a.width + p];
      } else {
        const uint32_t i = (uint32_t)head + (req[k] ? s_need[req[k] - 1] : 0u) + (p - have);  // (below 2 n_pages)
        id[k] = a.free_ring[i >= (uint32_t)a.n_pages ? i - (uint32_t)a.n_pages : i];
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int t = t0 + k * gn;
      if (t >= a.N) continue;
      a.tok_req[t] = req[k];
      a.tok_pos[t] = pos[k];
      a.tok_slot[t] = id[k] >= 0 && id[k] < a.n_pages ? id[k] * a.page + at[k] : -1;
    }
  }
  auto wrap = [&](uint32_t i) { return i >= (uint32_t)a.n_pages ? i - (uint32_t)a.n_pages : i; };
  // ---- pages taken into the tables, pages released behind the ring's end
  if (!err) {
    for (int i = gt; i < (int)total.need; i += gn) {
      const int r = first_above(s_need, a.R, (uint32_t)i);
      const int have = (int)a_page.div((uint32_t)(s_len[r] + a.page - 1));
      a.table[(int64_t)r * a.width + have + (i - (int)(r ? s_need[r - 1] : 0u))] =
          a.free_ring[wrap((uint32_t)head + (uint32_t)i)];
    }
    for (int i = gt; i < (int)total.back; i += gn) {
      const int r = first_above(s_back, a.R, (uint32_t)i);
      a.free_ring[((uint32_t)head + (uint32_t)count + (uint32_t)i) % (uint32_t)a.n_pages] =
          a.table[(int64_t)r * a.width + (i - (int)(r ? s_back[r - 1] : 0u))];
    }
  }
  // ---- the state after the step, once every CTA has read the one before
  if (gridDim.x > 1)
    tc::cluster_sync();
  else
    __syncthreads();
  for (int r = gt; r < a.R; r += gn) {
    const int len = s_len[r], nw_r = a.new_len[r];
    a.length_out[r] = err ? len : (nw_r < 0 ? 0 : len + nw_r);
    if (a.cu) a.cu[r + 1] = err ? 0 : (int)s_add[r];
  }
  if (gt == 0) {
    if (a.cu) a.cu[0] = 0;
    a.state_out[0] = err ? head : (int)(((uint32_t)head + total.need) % (uint32_t)a.n_pages);
    a.state_out[1] = err ? count : count - (int)total.need + (int)total.back;
    a.info[0] = n_tok;
    a.info[1] = err ? 0 : (int)total.need;
    a.info[2] = err ? 0 : (int)total.back;
    a.info[3] = err;
  }
}

}  // namespace

cudaError_t launch_page_step(const PageStepArgs &a, cudaStream_t s) {
  static SmemAttr attr;
  const size_t smem = 4 * sizeof(uint32_t) * (size_t)a.R;
  cudaError_t e = attr.ensure((const void *)k_page_step, (int)smem);
  if (e != cudaSuccess) return e;
  // One CTA against eight: 1000 requests 5.2 against 6.0 us, 2000 tokens 4.2 / 4.4, 4000 tokens 5.0 / 4.5, 4000 requests 12.2 /
  // 9.1, 1400 requests of which 113 end with up to 1700 pages each 28 / 9.5 (what a step releases is not known here, only how
  // wide the tables are).  256 threads against 1024: 200 requests 3.4 / 3.9, 300 4.4 / 4.3, 1000 6.7 / 5.2.
  const bool large = a.N > 2048 || a.R > 2048 || (a.R > 256 && a.width > 1024);
  const unsigned ctas = large ? kClusterCtas : 1;
  return launch_dependent(k_page_step, dim3(ctas), dim3(a.N <= 256 && a.R <= 256 ? 256 : 1024), smem, s, ctas, a,
                          paged::FastDiv((uint32_t)a.page));
}

}  // namespace csa
