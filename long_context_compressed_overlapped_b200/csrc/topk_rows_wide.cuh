// Top-k of few score rows ("Paper Breakdown: DeepSeek-V4", section 4, DSA on
// Compressed KV: the top-k entries by I_{t,s}): rows of up to kTopkSmemMaxN
// keys, no more of them than SMs.
//
// Such a call is bound by its chain of steps, not by HBM (18 rows of 16,384
// keys are 1.2 MB), so a row gets a CTA of 1,024 threads, which asks for all
// of it at once and keeps it in registers: warp w holds a contiguous range, key
// j0 + 32 x + lane in its x-th register.  The exact key T of the k-th largest
// and how many keys equal to T are taken come from three histograms (bits 31..21,
// 20..10, 9..0).  Few bins hold most scores, and atomics on one bin wait for
// one another: in rows above 4,096 keys a histogram of every eighth 32-key
// segment first gives a bound, and the some 5 k / 4 keys that reach it go to a
// list for the histograms (fewer than k of them, or more than the list holds:
// the registers are counted).  The warps then place their keys > T and
// lowest-index keys == T by ballots, in index order.
//
// indexer_topk with the selection's scores, 18 queries, k = 1,024, here / with
// 256 threads a row and the scores read back by another kernel: 4,096 keys
// 18 / 29 us, 16,384 keys 25 / 54 us, 32,768 keys 35 / 76 us (k = 4,096, where the
// lists of 256 threads run over: 37 / 192 us); 148 queries of 16,384 keys
// 56 / 86 us.
#pragma once
#include "topk.cuh"

namespace csahca {

constexpr int kTopkWideThreads = 1024;
constexpr int kTopkWideWarps = kTopkWideThreads / 32;
constexpr int kTopkWideSampleFrom = 4096;            // keys of a row from which a sample pays
constexpr int kTopkWideList = 8192;

struct TopkWideSmem {
  uint32_t hist[2048];
  uint32_t wsum[kTopkWideWarps];
  uint32_t digit, need;
  int sampled, listed;
  int wcnt[kTopkWideWarps][2];                       // per warp: keys > T, keys == T
  uint32_t list[kTopkWideList];
};

// The largest digit d of nb (2048 or 1024) with sum_{e >= d} hist[e] >= need, and
// need - sum_{e > d} hist[e]; digit = ~0 if all bins together hold fewer.
__device__ __forceinline__ void topk_wide_digit(TopkWideSmem& sm, int nb, uint32_t need) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int per = nb / kTopkWideThreads;             // bins of a thread, top bins first
  const int hi = nb - threadIdx.x * per;
  uint32_t local = 0;
  for (int e = 0; e < per; ++e) local += sm.hist[hi - 1 - e];
  uint32_t incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm.wsum[wid] = incl;
  if (threadIdx.x == 0) sm.digit = ~0u;
  __syncthreads();
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < wid ? sm.wsum[lane] : 0u);
  uint32_t cum = before + incl - local;              // keys in the bins above this thread's
  if (cum < need && cum + local >= need) {
    for (int e = 0; e < per; ++e) {
      const int b = hi - 1 - e;
      if (cum + sm.hist[b] >= need) { sm.digit = (uint32_t)b; sm.need = need - cum; break; }
      cum += sm.hist[b];
    }
  }
  __syncthreads();
}

// The score of an order key (zero's sign is lost).
__device__ __forceinline__ float topk_wide_score(uint32_t u) {
  return __uint_as_float(u == kOrderKeyNan ? 0x7fffffffu : (u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// f(x) for the registers that a row with ranges of L keys fills, eight at a time.
template <int KPL, typename F> __device__ __forceinline__ void topk_wide_each(int L, F f) {
  constexpr int G = KPL < 8 ? KPL : 8;
#pragma unroll
  for (int g = 0; g < KPL; g += G) {
    if (32 * g < L) {
#pragma unroll
      for (int x = g; x < g + G; ++x) f(x);
    }
  }
}

// KPL: keys a lane holds, at least ceil(N / 1024).  sel (optional): the scores of
// the selection, -inf behind it.
template <int KPL>
__global__ void __launch_bounds__(kTopkWideThreads, 1) topk_rows_wide_kernel(TopkParams p, float* sel) {
  __shared__ TopkWideSmem sm;
  griddep_wait();
  griddep_launch_dependents();
  const TopkRow r = topk_row(p);
  const int v = r.v;
  int* const out = r.out;
  float* const so = sel ? sel + (out - p.idx) : nullptr;
  if (v <= p.k) {
    for (int j = threadIdx.x; j < p.k; j += blockDim.x) {
      out[j] = j < v ? j : -1;
      if (so) so[j] = j < v ? __ldg(r.s + j) : -INFINITY;
    }
    return;
  }
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const uint32_t lt = (1u << lane) - 1u, k = (uint32_t)p.k;
  const int L = (v + kTopkWideThreads - 1) / kTopkWideThreads * 32;      // <= 32 KPL
  const int j0 = wid * L, j1 = min(v, j0 + L);
  uint32_t u[KPL];                                   // order keys; no key: 0
  topk_wide_each<KPL>(L, [&](int x) {
    const int j = j0 + 32 * x + lane;
    u[x] = j < j1 ? __float_as_uint(__ldg(r.s + j)) : 0u;
  });
  if (threadIdx.x == 0) sm.sampled = sm.listed = 0;
  for (int x = threadIdx.x; x < 2048; x += kTopkWideThreads) sm.hist[x] = 0u;
  topk_wide_each<KPL>(L, [&](int x) { u[x] = j0 + 32 * x + lane < j1 ? order_key(__uint_as_float(u[x])) : 0u; });
  __syncthreads();

  // ---- a bound that about 5 k / 4 keys reach
  uint32_t lo = 1u;
  if (KPL > 4 && v > kTopkWideSampleFrom) {
    int n = 0;
#pragma unroll
    for (int x = 0; x < KPL; x += 8) {
      if (32 * x < L) {
        if (u[x]) atomicAdd(&sm.hist[u[x] >> 21], 1u);
        n += __popc(__ballot_sync(0xffffffffu, u[x] != 0u));
      }
    }
    if (lane == 0 && n) atomicAdd(&sm.sampled, n);
    __syncthreads();
    const int ns = sm.sampled;
    const int ks0 = (int)(((int64_t)p.k * ns + v - 1) / v);
    topk_wide_digit(sm, 2048, (uint32_t)min(ns, ks0 + max(64, ks0 / 4)));
    lo = max(1u, sm.digit << 21);                    // (the sample's keys are all counted: there is a digit)
    for (int x = threadIdx.x; x < 2048; x += kTopkWideThreads) sm.hist[x] = 0u;
    __syncthreads();
  }

  // ---- the keys that reach the bound, in any order, to a list (if it holds them)
  int keep = 0;
  topk_wide_each<KPL>(L, [&](int x) { keep += u[x] >= lo; });
  int incl = keep;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  int at = lane == 31 ? atomicAdd(&sm.listed, incl) : 0;
  at = __shfl_sync(0xffffffffu, at, 31) + incl - keep;
  if (at + keep <= kTopkWideList) {
    topk_wide_each<KPL>(L, [&](int x) {
      if (u[x] >= lo) sm.list[at++] = u[x];
    });
  }
  __syncthreads();
  const int nl = sm.listed;
  if (nl < (int)k) lo = 1u;                          // the sample misled: every key
  const bool listed = nl >= (int)k && nl <= kTopkWideList;

  // ---- the k-th largest key T: three digits of 11, 11, 10 bits
  uint32_t T = 0u, need = k;
#pragma unroll
  for (int dgt = 0; dgt < 3; ++dgt) {
    const int sh = dgt == 0 ? 21 : dgt == 1 ? 10 : 0, hs = dgt == 1 ? 21 : 10, nb = dgt == 2 ? 1024 : 2048;
    if (dgt > 0) {
      for (int x = threadIdx.x; x < nb; x += kTopkWideThreads) sm.hist[x] = 0u;
      __syncthreads();
    }
    const auto count = [&](uint32_t key) {
      if (dgt == 0 || (key >> hs) == T) atomicAdd(&sm.hist[(key >> sh) & (uint32_t)(nb - 1)], 1u);
    };
    if (listed) {
      for (int x = threadIdx.x; x < nl; x += kTopkWideThreads) count(sm.list[x]);
    } else {
      topk_wide_each<KPL>(L, [&](int x) {
        if (u[x] >= lo) count(u[x]);
      });
    }
    __syncthreads();
    topk_wide_digit(sm, nb, need);
    T = dgt == 0 ? sm.digit : (T << (dgt == 1 ? 11 : 10)) | sm.digit;
    need = sm.need;
  }

  // ---- each warp's place in the output, then its keys in index order
  unsigned n_gt = 0, n_eq = 0;
  topk_wide_each<KPL>(L, [&](int x) {
    n_gt += u[x] > T;
    n_eq += u[x] == T;
  });
  n_gt = __reduce_add_sync(0xffffffffu, n_gt);
  n_eq = __reduce_add_sync(0xffffffffu, n_eq);
  if (lane == 0) { sm.wcnt[wid][0] = (int)n_gt; sm.wcnt[wid][1] = (int)n_eq; }
  __syncthreads();
  // lane w: warp w's ties, those before it, and what it takes of them
  const int eq_w = sm.wcnt[lane][1];
  int eq_incl = eq_w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, eq_incl, o);
    if (lane >= o) eq_incl += y;
  }
  const int take_w = max(0, min(eq_w, (int)need - (eq_incl - eq_w)));
  int pos = (int)__reduce_add_sync(0xffffffffu, lane < wid ? (unsigned)(sm.wcnt[lane][0] + take_w) : 0u);
  const int eq_take = __shfl_sync(0xffffffffu, take_w, wid);
  const auto put = [&](int x, int o) {
    out[o] = j0 + 32 * x + lane;
    if (so) so[o] = topk_wide_score(u[x]);
  };
  if (eq_take == 0 || eq_take == (int)n_eq) {        // no tie is split here
    const uint32_t thr = eq_take == 0 ? T + 1u : T;  // (a key is at most that of +inf)
    topk_wide_each<KPL>(L, [&](int x) {
      const uint32_t tb = __ballot_sync(0xffffffffu, u[x] >= thr);
      if (u[x] >= thr) put(x, pos + __popc(tb & lt));
      pos += __popc(tb);
    });
  } else {
    int eq_seen = 0;
    topk_wide_each<KPL>(L, [&](int x) {
      const uint32_t eqb = __ballot_sync(0xffffffffu, u[x] == T);
      const bool take = u[x] > T || (u[x] == T && eq_seen + __popc(eqb & lt) < eq_take);
      const uint32_t tb = __ballot_sync(0xffffffffu, take);
      if (take) put(x, pos + __popc(tb & lt));
      pos += __popc(tb);
      eq_seen += __popc(eqb);
    });
  }
}

}  // namespace csahca
