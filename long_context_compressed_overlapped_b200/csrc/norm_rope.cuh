// Norms of query and key heads with the position rotation ("Paper Breakdown:
// DeepSeek-V4", section 4, Additional Techniques: query/KV RMSNorm, partial
// RoPE), for any tokens' rows, and for the drafted tokens of a tree.
//
//   y = RoPE_pos(x / sqrt(mean(x^2) + eps) * gain), the last r dims rotated.
//
// One CTA = one token x a run of its heads.  The rows go through registers
// once (read, summed, scaled, rotated, written: 2 d e bytes a row, so HBM is
// the bound); the token's r/2 rotation angles are the same for every head, so
// the CTA forms them once, in double, while its first rows are in flight.
// LPR lanes share a row (a power of two, so that a row of 64 bf16 dims takes 8
// lanes and a warp 4 rows), each with NCH 16-byte pieces; a lane keeps the
// pieces of up to four rows in flight, packed.  Arithmetic is fp32 and the one
// rounding is the store's.
//
// kTree: the tokens are the nodes of draft trees.  A node's position is pos[b]
// plus its depth, found by walking its parents; the CTA of a node's first
// heads also writes the node's plan (TreePlan) for the attention.
#pragma once
#include "common.cuh"

namespace csahca {

constexpr int kNrThreads = 256;
constexpr int kNrMaxPairs = 256;       // rope dims <= 512
constexpr int kTreeMaxNodes = 64;

// Row codes of a node's own key list: window rows by position, then (HCA) the
// drafted entries on its path.
constexpr int kRowShift = 29;
constexpr int kRowMask = (1 << kRowShift) - 1;
enum : int { ROW_RING = 0, ROW_TREE = 1, ROW_DRAFT = 2 };

struct TreePlan {
  const int* parents;       // [B, T]: < own index; -1 first drafted token; < -1 no node
  const int* pos;           // [B] position of the first drafted token
  int T, w, m, N;
  int list_drafts;          // append the path's drafted entries to the list (HCA)
  int* node_pos;            // [B, T] position of the node, -1: no node
  int* sel_pos;             // [B, T] pos - 1 (the committed tokens' last position), -1: no node
  int* list;                // [B, T][w + T] row codes
  int4* info;               // [B, T] {position, visible committed entries, length of the list, 0}
};

struct NormRopeParams {
  const void* x[2]; void* y[2];         // queries, keys
  const float* gain[2];
  int64_t xs[2][3], ys[2][3];           // element strides of batch, token, head
  int heads[2], norm[2];
  const int* pos;                       // [B, n]; < 0: the token's rows are left as they are
  int n, d, rope_dims, rows_per_cta;
  float eps;
  TreePlan plan;
  double theta[kNrMaxPairs];
};

// The path of node i: path[0] the first drafted token .. path[depth] = i.
// Returns the depth, or -1 if i or one of its ancestors is no node.  A parent
// that is not below its child ends the walk as no node (error word 2), so the
// walk always ends.
__device__ __forceinline__ int tree_path(const int* parents, int i, int* path) {
  int up = 0;
  for (int j = i; j >= 0;) {
    const int p = parents[j];
    if (p < -1) return -1;
    if (p >= j) { raise_device_error(DEVERR_BAD_INDEX); return -1; }
    path[up++] = j;
    j = p;
  }
  for (int a = 0, b = up - 1; a < b; ++a, --b) { const int s = path[a]; path[a] = path[b]; path[b] = s; }
  return up - 1;
}

// Position of the token, or -1 for none; every thread of the CTA calls it.
__device__ __forceinline__ int tree_node(const int* parents, const int* pos, int b, int T, int i, int* par_s,
                                         int* path_s, int* t_s) {
  for (int j = threadIdx.x; j <= i; j += blockDim.x) par_s[j] = parents[(int64_t)b * T + j];
  __syncthreads();
  if (threadIdx.x == 0) {
    const int p0 = pos[b];
    const int depth = p0 < 0 ? -1 : tree_path(par_s, i, path_s);
    *t_s = depth < 0 || p0 > INT32_MAX - kTreeMaxNodes ? -1 : p0 + depth;
  }
  __syncthreads();
  return *t_s;
}

template <typename T> __device__ __forceinline__ void unpack16(const uint4& raw, float* o);
template <> __device__ __forceinline__ void unpack16<float>(const uint4& raw, float* o) {
  o[0] = __uint_as_float(raw.x); o[1] = __uint_as_float(raw.y);
  o[2] = __uint_as_float(raw.z); o[3] = __uint_as_float(raw.w);
}
template <> __device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4& raw, float* o) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(w[i] << 16);
    o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <typename T, int LPR, int NCH, bool kTree>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int VEC = Vec16<T>::N;
  constexpr int RPW = 32 / LPR;                       // rows a warp takes at once
  constexpr int RPC = RPW * (kNrThreads / 32);        // rows the CTA takes at once
  constexpr int U = NCH >= 4 ? 2 : 4;                 // rows of a lane in flight
  __shared__ float2 cs_s[kNrMaxPairs];
  __shared__ int par_s[kTree ? kTreeMaxNodes : 1], path_s[kTree ? kTreeMaxNodes : 1], t_s;
  griddep_wait();
  griddep_launch_dependents();
  const int tok = blockIdx.x, b = tok / p.n, i = tok - b * p.n;
  const int lane = threadIdx.x & 31, sub = lane % LPR;
  const int slot = (threadIdx.x >> 5) * RPW + lane / LPR;
  const int rows = p.heads[0] + p.heads[1];
  const int r_begin = blockIdx.y * p.rows_per_cta, r_end = min(rows, r_begin + p.rows_per_cta);
  const int nch = p.d / VEC;

  int t = 0;
  if constexpr (kTree) {
    t = tree_node(p.plan.parents, p.plan.pos, b, p.n, i, par_s, path_s, &t_s);
    if (blockIdx.y == 0) {
      const TreePlan& L = p.plan;
      if (threadIdx.x == 0) {
        L.node_pos[tok] = t;
        L.sel_pos[tok] = t < 0 ? -1 : L.pos[b] - 1;
      }
      int* list = L.list + (int64_t)tok * (L.w + L.T);
      int count = 0;
      if (t >= 0) {
        const int p0 = L.pos[b], lo = max(0, t - L.w + 1);
        const int nwin = L.w > 0 ? t - lo + 1 : 0;
        for (int j = threadIdx.x; j < nwin; j += blockDim.x) {
          const int q = lo + j;
          list[j] = q < p0 ? (ROW_RING << kRowShift) | (b * L.w + q % L.w)
                           : (ROW_TREE << kRowShift) | (b * L.T + path_s[q - p0]);
        }
        count = nwin;
        if (L.list_drafts && threadIdx.x == 0) {
          for (int q = p0; q <= t; ++q)
            if ((q + 1) % L.m == 0 && (q + 1) / L.m - 1 < L.N)
              list[count++] = (ROW_DRAFT << kRowShift) | (b * L.T + path_s[q - p0]);
        }
      }
      if (threadIdx.x == 0) L.info[tok] = make_int4(t, t < 0 ? 0 : min(L.N, L.pos[b] / L.m), count, 0);
    }
  } else {
    t = p.pos[tok];
  }
  if (t < 0) return;

  bool have_cs = false;
  int which = -1;
  float gain[NCH][VEC];
  for (int r0 = r_begin; r0 < r_end; r0 += U * RPC) {
    uint4 raw[U][NCH];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = r0 + u * RPC + slot;
      const int k = row >= p.heads[0];
      const T* x = static_cast<const T*>(p.x[k]) + b * p.xs[k][0] + i * p.xs[k][1] +
                   (row - k * p.heads[0]) * p.xs[k][2];
#pragma unroll
      for (int q = 0; q < NCH; ++q) {
        const int ch = sub + LPR * q;
        if (row < r_end && ch < nch) raw[u][q] = __ldg(reinterpret_cast<const uint4*>(x + ch * VEC));
      }
    }
    if (!have_cs) {
      // (uniform over the CTA: the first turn of every warp)
      for (int j = threadIdx.x; j < p.rope_dims / 2; j += blockDim.x)
        rope_sincos((double)t, p.theta[j], &cs_s[j].x, &cs_s[j].y);
      __syncthreads();
      have_cs = true;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = r0 + u * RPC + slot;
      if (r0 + u * RPC >= r_end) break;               // (uniform over the CTA)
      const int k = row >= p.heads[0];
      if (k != which) {
        which = k;
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
          const int ch = sub + LPR * q;
#pragma unroll
          for (int e = 0; e < VEC; e += 4) {
            float4 g = make_float4(1.f, 1.f, 1.f, 1.f);
            if (p.norm[k] && p.gain[k] && ch < nch)
              g = __ldg(reinterpret_cast<const float4*>(p.gain[k] + ch * VEC + e));
            gain[q][e] = g.x; gain[q][e + 1] = g.y; gain[q][e + 2] = g.z; gain[q][e + 3] = g.w;
          }
        }
      }
      float v[NCH][VEC];
      float ss = 0.f;
#pragma unroll
      for (int q = 0; q < NCH; ++q) {
        if (row < r_end && sub + LPR * q < nch) {
          unpack16<T>(raw[u][q], v[q]);
#pragma unroll
          for (int e = 0; e < VEC; ++e) ss = fmaf(v[q][e], v[q][e], ss);
        }
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = p.norm[k] ? rsqrtf(ss / (float)p.d + p.eps) : 1.f;
      T* y = static_cast<T*>(p.y[k]) + b * p.ys[k][0] + i * p.ys[k][1] + (row - k * p.heads[0]) * p.ys[k][2];
#pragma unroll
      for (int q = 0; q < NCH; ++q) {
        const int ch = sub + LPR * q;
        if (row < r_end && ch < nch) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[q][e] *= inv * gain[q][e];
          const int j0 = ch * VEC - (p.d - p.rope_dims);
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            if (j0 + e >= 0) {
              const float2 c = cs_s[(j0 + e) >> 1];
              const float x0 = v[q][e], x1 = v[q][e + 1];
              v[q][e] = x0 * c.x - x1 * c.y;
              v[q][e + 1] = x0 * c.y + x1 * c.x;
            }
          }
          store16(y + ch * VEC, v[q]);
        }
      }
    }
  }
}

}  // namespace csahca
