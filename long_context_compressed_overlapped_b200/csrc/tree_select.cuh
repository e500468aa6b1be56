// Drafted entries among a tree node's selection ("Paper Breakdown:
// DeepSeek-V4", section 4, DSA on Compressed KV: lightning indexer, top-k).
//
// indexer_topk has left each node's k best committed entries with their
// scores.  A node also sees the entries that its own path completes, so its
// selection is the top k of both: a drafted entry stays if it beats one of the
// candidates that must then go (ties to the lower index: the committed one).
// Scores are compared as order keys throughout, as in the top-k, so that a NaN
// ranks last on either side.
// With f free places and the node's drafted scores in descending order, the
// r-th (from 0) stays iff f plus the number of candidates below it exceeds r.
// The y that stay push out the y - f lowest candidates (of equal scores the
// higher index first), found one after another: mostly none or very few.
//
// One CTA per node.  The drafted scores need only the call's inputs, which were
// complete before the kernels of this call began (each of them waits for its
// predecessor before it lets its successor start): they are formed while the
// top-k of the committed entries still runs.
#pragma once
#include "norm_rope.cuh"
#include "topk.cuh"

namespace csahca {

constexpr int kTsThreads = 256;
constexpr int kTsMaxK = 4096;

struct TreeSelectParams {
  const int* parents; const int* pos;
  const void* qI; const float* w;          // [nodes, HI, dI], [nodes, HI]
  const void* kI; const float* kI_scale;   // drafted keys [B, T, dI], [B, T, dI / 128]
  int q_bf16, k_dtype;                     // k_dtype: 0 fp32, 1 bf16, 2 e4m3
  int T, HI, dI, m, N, k;
  const float* scores;                     // [nodes, k]
  int* idx;                                // [nodes, k] in and out
};

__device__ __forceinline__ float ts_q(const TreeSelectParams& p, int64_t o) {
  return p.q_bf16 ? to_f32(static_cast<const __nv_bfloat16*>(p.qI)[o]) : static_cast<const float*>(p.qI)[o];
}
__device__ __forceinline__ float ts_k(const TreeSelectParams& p, int64_t row, int x) {
  const int64_t o = row * p.dI + x;
  if (p.k_dtype == 0) return static_cast<const float*>(p.kI)[o];
  if (p.k_dtype == 1) return to_f32(static_cast<const __nv_bfloat16*>(p.kI)[o]);
  return e4m3_to_f32(static_cast<const uint8_t*>(p.kI)[o]) * p.kI_scale[row * (p.dI / 128) + x / 128];
}

__global__ void __launch_bounds__(kTsThreads) tree_select_kernel(const __grid_constant__ TreeSelectParams p) {
  extern __shared__ __align__(16) uint8_t ts_smem[];
  int* idx_s = reinterpret_cast<int*>(ts_smem);                   // [k], -1 once pushed out
  uint32_t* key_s = reinterpret_cast<uint32_t*>(idx_s + p.k);     // [k] order keys of the scores
  __shared__ TreeNode node_s;
  __shared__ int dnode[kTreeMaxNodes], rank_s[kTreeMaxNodes], below[kTreeMaxNodes];
  __shared__ uint32_t dkey[kTreeMaxNodes];
  __shared__ float part_s[kTsThreads / 32];
  __shared__ int nd_s, valid_s, scan_s[kTsThreads / 32];
  __shared__ unsigned long long min_s;
  const int node = blockIdx.x, b = node / p.T, i = node - b * p.T;
  const int t = tree_node(p.parents, p.pos, b, p.T, i, &node_s);
  // (a CTA that leaves waits all the same: the attention behind this kernel reads
  // what the one before it wrote)
  if (t < 0) {
    griddep_wait();
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) {
    int nd = 0;
    const int end = tree_entries_end(t, p.m, p.N);
    for (int64_t q = tree_first_end(node_s.pos0, p.m); q <= end; q += p.m) dnode[nd++] = node_s.at((int)q);
    nd_s = nd;
    valid_s = 0;
  }
  if (tid < kTreeMaxNodes) below[tid] = 0;
  __syncthreads();
  const int nd = nd_s;
  if (nd == 0) {
    griddep_wait();
    return;
  }
  // scores of the drafted entries: a warp takes every eighth head
  for (int x = 0; x < nd; ++x) {
    const int64_t krow = (int64_t)b * p.T + dnode[x];
    float sum = 0.f;
    for (int h = wid; h < p.HI; h += kTsThreads / 32) {
      const int64_t qo = ((int64_t)node * p.HI + h) * p.dI;
      float dot = 0.f;
      for (int c = lane; c < p.dI; c += 32) dot = fmaf(ts_q(p, qo + c), ts_k(p, krow, c), dot);
      dot = warp_sum(dot);
      sum = fmaf(fmaxf(dot, 0.f), p.w[(int64_t)node * p.HI + h], sum);
    }
    if (lane == 0) part_s[wid] = sum;
    __syncthreads();
    if (tid == 0) {
      float s = 0.f;
      for (int k = 0; k < kTsThreads / 32; ++k) s += part_s[k];
      dkey[x] = order_key(s);
    }
    __syncthreads();
  }
  griddep_wait();
  griddep_launch_dependents();
  // descending rank of each drafted entry (ties: the earlier one first)
  if (tid < nd) {
    int r = 0;
    for (int x = 0; x < nd; ++x) r += dkey[x] > dkey[tid] || (dkey[x] == dkey[tid] && x < tid);
    rank_s[tid] = r;
  }
  int mine = 0;
  for (int j = tid; j < p.k; j += kTsThreads) {
    const int e = p.idx[(int64_t)node * p.k + j];
    idx_s[j] = e;
    key_s[j] = e >= 0 ? order_key(p.scores[(int64_t)node * p.k + j]) : 0u;
    mine += e >= 0;
  }
  if (mine) atomicAdd(&valid_s, mine);
  __syncthreads();
  for (int x = 0; x < nd; ++x) {
    int c = 0;
    for (int j = tid; j < p.k; j += kTsThreads) c += idx_s[j] >= 0 && key_s[j] < dkey[x];
    c = (int)__reduce_add_sync(0xffffffffu, (unsigned)c);
    if (lane == 0 && c) atomicAdd(&below[x], c);
  }
  __syncthreads();
  const int free_places = p.k - valid_s;
  int y = 0;
  for (int x = 0; x < nd; ++x) y += free_places + below[x] > rank_s[x];
  if (y == 0) return;                                // (uniform) the selection stays as it is
  for (int drop = y - free_places; drop > 0; --drop) {
    // the lowest candidate left: (score, higher index first)
    unsigned long long mn = ~0ull;
    int at = -1;
    for (int j = tid; j < p.k; j += kTsThreads) {
      if (idx_s[j] < 0) continue;
      const unsigned long long key = ((unsigned long long)key_s[j] << 32) | (0xFFFFFFFFu - (uint32_t)idx_s[j]);
      if (key < mn) { mn = key; at = j; }
    }
    if (tid == 0) min_s = ~0ull;
    __syncthreads();
    if (at >= 0) atomicMin(&min_s, mn);
    __syncthreads();
    if (at >= 0 && mn == min_s) idx_s[at] = -1;
    __syncthreads();
  }
  // candidates that stay in index order, then the drafted entries in path order
  int base = 0;
  for (int j0 = 0; j0 < p.k; j0 += kTsThreads) {
    const int j = j0 + tid;
    const int e = j < p.k ? idx_s[j] : -1;
    const unsigned keep = __ballot_sync(0xffffffffu, e >= 0);
    if (lane == 0) scan_s[wid] = __popc(keep);
    __syncthreads();
    int before = base, total = 0;
    for (int k = 0; k < kTsThreads / 32; ++k) {
      before += k < wid ? scan_s[k] : 0;
      total += scan_s[k];
    }
    if (e >= 0) p.idx[(int64_t)node * p.k + before + __popc(keep & ((1u << lane) - 1u))] = e;
    base += total;
    __syncthreads();
  }
  if (tid == 0) {
    for (int x = 0; x < nd; ++x)
      if (free_places + below[x] > rank_s[x]) p.idx[(int64_t)node * p.k + base++] = p.N + dnode[x];
  }
  for (int j = valid_s - max(0, y - free_places) + y + tid; j < p.k; j += kTsThreads) p.idx[(int64_t)node * p.k + j] = -1;
}

}  // namespace csahca
