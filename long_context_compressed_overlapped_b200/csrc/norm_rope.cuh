// Norms of query and key heads with the position rotation ("Paper Breakdown:
// DeepSeek-V4", section 4, Additional Techniques: query/KV RMSNorm, partial
// RoPE), for any tokens' rows, and for the drafted tokens of a tree.
//
//   y = RoPE_pos(x / sqrt(mean(x^2) + eps) * gain), the last r dims rotated.
//
// The rows go through registers once (read, summed, scaled, rotated, written:
// 2 d e bytes a row, so HBM is the bound).  One CTA = one token x a run of its
// heads, or several tokens where a token has few (a CTA per token of 5 rows of
// 64 dims left HBM at 780 GB/s).  A token's r/2 rotation angles are the same for
// every head, so the CTA forms them once, in double, while its first rows are
// in flight.  LPR lanes share a row (a power of two, so that a row of 64 bf16
// dims takes 8 lanes and a warp 4 rows), each with NCH 16-byte pieces; a lane
// keeps the pieces of its next two or four rows in flight, packed, while it works
// on one.  bf16 rows are bound by instructions
// before HBM: the arithmetic is in pairs (two fp32 lanes an instruction).
// Arithmetic is fp32 and the one rounding is the store's.
//
// kTree: the tokens are the nodes of draft trees.  A node's position is pos[b]
// plus its depth, found by walking its parents; the CTA of a node's first
// heads also writes the node's plan (TreePlan) for the attention.
#pragma once
#include "common.cuh"

namespace csahca {

constexpr int kNrThreads = 256;
constexpr int kNrMaxPairs = 256;       // rope dims <= 512
constexpr int kNrTable = 512;          // angles of a CTA: its tokens x r / 2
constexpr int kNrMaxTokens = 64;       // tokens of a CTA
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
  float2* turn;             // [B, T][r / 2] cos, sin of the node's angles (optional)
  uint4* zero;              // [B, T][zero_n]: rows of places without a node become zeros (optional)
  int zero_n;
};

struct NormRopeParams {
  const void* x[2]; void* y[2];         // queries, keys
  const float* gain[2];
  int64_t xs[2][3], ys[2][3];           // element strides of batch, token, head
  int heads[2], norm[2];
  int zero_rest;                        // bit k: rows of y[k] of a token with pos < 0 become zeros
  const int* pos;                       // [B, n]; < 0: the token's rows are left as they are
  int tokens, n, d, rope_dims;
  int tpc, rows_per_cta;                // tokens of a CTA; rows of its token (tpc = 1) that it takes
  float eps, inv_d;
  TreePlan plan;
  double theta[kNrMaxPairs];
};

// A node of a draft tree, as the threads of its CTA see it: its sequence's
// first position, its own (-1: no node), and up[k], its k-th ancestor (up[0] the
// node itself, up[t - pos0] a first drafted token).
struct TreeNode {
  int par[kTreeMaxNodes], up[kTreeMaxNodes];
  int pos0, t;
  __device__ __forceinline__ int at(int position) const { return up[t - position]; }   // path node at a position >= pos0
};

// Fills it; every thread of the CTA calls it, and gets the node's position.  A
// parent that is not below its child ends the walk as no node (error word 2),
// so the walk always ends.
__device__ __forceinline__ int tree_node(const int* parents, const int* pos, int b, int T, int i, TreeNode* nd) {
  const int p0 = threadIdx.x == 0 ? pos[b] : 0;
  for (int j = threadIdx.x; j <= i; j += blockDim.x) nd->par[j] = parents[(int64_t)b * T + j];
  __syncthreads();
  if (threadIdx.x == 0) {
    int depth = -1;
    if (p0 >= 0 && p0 <= INT32_MAX - kTreeMaxNodes) {
      for (int j = i; j >= 0;) {
        const int p = nd->par[j];
        if (p < -1) { depth = -1; break; }
        if (p >= j) { raise_device_error(DEVERR_BAD_INDEX); depth = -1; break; }
        nd->up[++depth] = j;
        j = p;
      }
    }
    nd->pos0 = p0;
    nd->t = depth < 0 ? -1 : p0 + depth;
  }
  __syncthreads();
  return nd->t;
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

// The positions at which a path completes stored entries: from the first
// block end at or after pos0, every m, up to the last one <= t whose entry is < N.
// (64-bit: a step past a position near 2^31 must not wrap)
__device__ __forceinline__ int64_t tree_first_end(int pos0, int m) { return (int64_t)pos0 + (m - 1 - pos0 % m); }
__device__ __forceinline__ int tree_entries_end(int t, int m, int N) {
  const int64_t last = (int64_t)N * m - 1;          // the block end of entry N - 1
  return last < t ? (int)last : t;
}

// Pairs of fp32 in one 64-bit register.
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <typename T> __device__ __forceinline__ void f2_load(const uint4& raw, uint64_t* o);
template <> __device__ __forceinline__ void f2_load<float>(const uint4& raw, uint64_t* o) {
  o[0] = f2_pack(__uint_as_float(raw.x), __uint_as_float(raw.y));
  o[1] = f2_pack(__uint_as_float(raw.z), __uint_as_float(raw.w));
}
template <> __device__ __forceinline__ void f2_load<__nv_bfloat16>(const uint4& raw, uint64_t* o) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <typename T> __device__ __forceinline__ uint4 f2_store(const uint64_t* v);
template <> __device__ __forceinline__ uint4 f2_store<float>(const uint64_t* v) {
  const float2 a = f2_unpack(v[0]), b = f2_unpack(v[1]);
  return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
}
template <> __device__ __forceinline__ uint4 f2_store<__nv_bfloat16>(const uint64_t* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f2_unpack(v[i]);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows [row_begin, row_end) of a CTA's padding tokens as zeros, a warp a row.
template <typename T>
__device__ __forceinline__ void zero_padding(const NormRopeParams& p, const int* pos_s, const int64_t (*off_s)[kNrMaxTokens],
                                             int tok0, int row_begin, int row_end) {
  constexpr int VEC = Vec16<T>::N;
#pragma unroll 1
  for (int q = 0; q < p.tpc; ++q) {
    if (tok0 + q >= p.tokens || pos_s[q] >= 0) continue;
#pragma unroll 1
    for (int r = row_begin + (threadIdx.x >> 5); r < row_end; r += kNrThreads / 32) {
      const int k = r >= p.heads[0];
      if (!(p.zero_rest >> k & 1)) continue;
      T* y = static_cast<T*>(p.y[k]) + (off_s[2 + k][q] + (r - k * p.heads[0]) * p.d);
#pragma unroll 1
      for (int c = threadIdx.x & 31; c < p.d / VEC; c += 32) *reinterpret_cast<uint4*>(y + c * VEC) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

// kFull: every lane's NCH pieces exist (d = LPR * NCH * VEC).
template <typename T, int LPR, int NCH, bool kFull, bool kTree>
__global__ void __launch_bounds__(kNrThreads, NCH >= 4 ? 2 : NCH == 2 ? 3 : 4) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int VEC = Vec16<T>::N, V2 = VEC / 2;
  constexpr int RPW = 32 / LPR;                       // rows a warp takes at once
  constexpr int RPC = RPW * (kNrThreads / 32);        // rows the CTA takes at once
  constexpr int U = NCH >= 2 ? 2 : 4;                 // rows of a lane in flight
  // long rows are asked for one by one as their slots come free, short ones a
  // turn at a time (measured: 396 against 410 us for 16,384 x 65 rows of 512, 46
  // against 51 for as many tokens of 17 rows of 128)
  constexpr bool kAhead = NCH >= 2;
  __shared__ float2 cs_s[kNrTable];
  __shared__ int pos_s[kNrMaxTokens];
  __shared__ int64_t off_s[4][kNrMaxTokens];          // token's offset in q, k, q_out, k_out
  __shared__ TreeNode node_s;                         // (kTree)
  griddep_wait();
  griddep_launch_dependents();
  const int tok0 = blockIdx.x * p.tpc;
  const int lane = threadIdx.x & 31, sub = lane % LPR;
  const int slot = (threadIdx.x >> 5) * RPW + lane / LPR;
  const int heads = p.heads[0] + p.heads[1];
  const int npair = p.rope_dims >> 1;

  // rows of this CTA: [row_begin, row_end) of one token, or all of tpc tokens
  const int row_begin = blockIdx.y * p.rows_per_cta;
  const int row_end = p.tpc > 1 ? heads : min(heads, row_begin + p.rows_per_cta);
  const int n_rows = p.tpc > 1 ? p.tpc * heads : row_end - row_begin;
  const int nch = p.d / VEC;
  int tk = 0, row = row_begin + slot;                 // this lane group's next row
  if (p.tpc > 1) { tk = slot / heads; row = slot - tk * heads; }
  const int step_t = p.tpc > 1 ? RPC / heads : 0, step_r = RPC - step_t * heads;
  int which = -1;
  uint64_t gain[NCH][V2];
  uint4 raw[U][NCH];
  T* out[U];
  int ut[U];                                          // token of the row (-1: nothing to do)
  bool uk[U];
  // asks for this lane group's next row, r0 rows of the CTA's on
  const auto load_row = [&](int u, int r0) {
    const bool in = r0 + slot < n_rows && (kTree || pos_s[tk] >= 0);
    const int k = row >= p.heads[0];
    ut[u] = in ? tk : -1;
    uk[u] = k;
    if (in) {
      const int h = row - k * p.heads[0];
      const int64_t xo = kTree ? (int64_t)tok0 * p.xs[k][1] : off_s[k][tk];
      const int64_t yo = kTree ? (int64_t)tok0 * p.ys[k][1] : off_s[2 + k][tk];
      const T* x = static_cast<const T*>(p.x[k]) + (xo + h * p.xs[k][2] + sub * VEC);
      out[u] = static_cast<T*>(p.y[k]) + (yo + h * p.d + sub * VEC);
#pragma unroll
      for (int q = 0; q < NCH; ++q) {
        if (kFull || sub + LPR * q < nch) raw[u][q] = __ldg(reinterpret_cast<const uint4*>(x + LPR * q * VEC));
      }
    }
    row += step_r;
    tk += step_t;
    if (p.tpc > 1 && row >= heads) { row -= heads; ++tk; }
  };
  bool padding = false;                               // (this thread's token, then any of the CTA's) becomes zeros
  // a node's rows are asked for before its place in the tree is known
  if constexpr (kTree) {
#pragma unroll
    for (int u = 0; u < U; ++u) load_row(u, u * RPC);
  }

  if constexpr (kTree) {
    const int b = tok0 / p.n, i = tok0 - b * p.n;
    const int t = tree_node(p.plan.parents, p.plan.pos, b, p.n, i, &node_s);
    const int p0 = node_s.pos0;
    if (blockIdx.y == 0) {
      const TreePlan& L = p.plan;
      if (threadIdx.x == 0) {
        L.node_pos[tok0] = t;
        L.sel_pos[tok0] = t < 0 ? -1 : p0 - 1;
      }
      int* list = L.list + (int64_t)tok0 * (L.w + L.T);
      int count = 0;
      if (t >= 0) {
        const int lo = max(0, t - L.w + 1);
        const int nwin = L.w > 0 ? t - lo + 1 : 0;
        for (int j = threadIdx.x; j < nwin; j += blockDim.x) {
          const int q = lo + j;
          list[j] = q < p0 ? (ROW_RING << kRowShift) | (b * L.w + q % L.w)
                           : (ROW_TREE << kRowShift) | (b * L.T + node_s.at(q));
        }
        count = nwin;
        if (L.list_drafts && threadIdx.x == 0) {
          const int end = tree_entries_end(t, L.m, L.N);
          for (int64_t q = tree_first_end(p0, L.m); q <= end; q += L.m)
            list[count++] = (ROW_DRAFT << kRowShift) | (b * L.T + node_s.at((int)q));
        }
      }
      if (threadIdx.x == 0) L.info[tok0] = make_int4(t, t < 0 ? 0 : min(L.N, p0 / L.m), count, 0);
    }
    if (t < 0) {
      if (p.plan.zero) {
        uint4* z = p.plan.zero + (int64_t)tok0 * p.plan.zero_n;
        for (int j = blockIdx.y * blockDim.x + threadIdx.x; j < p.plan.zero_n; j += gridDim.y * blockDim.x)
          z[j] = make_uint4(0u, 0u, 0u, 0u);
      }
      return;
    }
    if (threadIdx.x == 0) pos_s[0] = t;
  } else {
    if (threadIdx.x < p.tpc) {
      const bool in = tok0 + threadIdx.x < p.tokens;
      const int t = in ? p.pos[tok0 + threadIdx.x] : -1;
      pos_s[threadIdx.x] = t;
      padding = in && t < 0 && p.zero_rest;
    }
  }
  if (threadIdx.x < 4 * p.tpc) {
    const int w = threadIdx.x & 3, q = threadIdx.x >> 2, tok = tok0 + q, b = tok / p.n, i = tok - b * p.n;
    const int64_t* st = w < 2 ? p.xs[w] : p.ys[w - 2];
    off_s[w][q] = b * st[0] + i * st[1];
  }
  // (one vote: a test of the flag alone moved the compiler's schedule of the
  // main loop, 409 against 405 us for 16,384 x 65 rows of 512)
  if constexpr (kTree) __syncthreads();
  else padding = __syncthreads_or(padding);

  if constexpr (!kTree) {
    if (padding) zero_padding<T>(p, pos_s, off_s, tok0, row_begin, row_end);
#pragma unroll
    for (int u = 0; u < U; ++u) load_row(u, u * RPC);
  }
  for (int j = threadIdx.x; j < p.tpc * npair; j += blockDim.x) {
    const int q = j / npair;
    float2 c;
    rope_sincos((double)pos_s[q], p.theta[j - q * npair], &c.x, &c.y);
    cs_s[j] = c;
    if constexpr (kTree) {
      if (p.plan.turn && blockIdx.y == 0) p.plan.turn[(int64_t)tok0 * npair + j] = c;
    }
  }
  __syncthreads();
  for (int r0 = 0; r0 < n_rows; r0 += U * RPC) {
    if (!kAhead && r0 > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_row(u, r0 + u * RPC);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r0 + u * RPC >= n_rows) break;              // (uniform over the CTA)
      const bool in = ut[u] >= 0;
      if (LPR == 32 && !in) {                         // (the warp's one row)
        if (kAhead) load_row(u, r0 + (U + u) * RPC);
        continue;
      }
      const int k = uk[u], cs0 = ut[u] * npair;
      T* const y = out[u];
      if (k != which) {
        which = k;
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
          const int ch = sub + LPR * q;
#pragma unroll
          for (int e = 0; e < V2; e += 2) {
            float4 g = make_float4(1.f, 1.f, 1.f, 1.f);
            if (p.norm[k] && p.gain[k] && ch < nch)
              g = __ldg(reinterpret_cast<const float4*>(p.gain[k] + ch * VEC + 2 * e));
            gain[q][e] = f2_pack(g.x, g.y);
            gain[q][e + 1] = f2_pack(g.z, g.w);
          }
        }
      }
      uint64_t v[NCH][V2], s2 = 0;
#pragma unroll
      for (int q = 0; q < NCH; ++q) {
        if ((LPR == 32 || in) && (kFull || sub + LPR * q < nch)) {
          f2_load<T>(raw[u][q], v[q]);
#pragma unroll
          for (int e = 0; e < V2; ++e) s2 = f2_fma(v[q][e], v[q][e], s2);
        }
      }
      if (kAhead) load_row(u, r0 + (U + u) * RPC);    // this slot's next row is on its way while this one is worked on
      const float2 s1 = f2_unpack(s2);
      float ss = s1.x + s1.y;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = p.norm[k] ? rsqrtf(fmaf(ss, p.inv_d, p.eps)) : 1.f;
      const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
      for (int q = 0; q < NCH; ++q) {
        const int ch = sub + LPR * q;
        if ((LPR == 32 || in) && (kFull || ch < nch)) {
#pragma unroll
          for (int e = 0; e < V2; ++e) v[q][e] = f2_mul(f2_mul(v[q][e], gain[q][e]), inv2);
          const int j0 = (ch * VEC - (p.d - p.rope_dims)) >> 1;
          const float2* cs = cs_s + cs0 + j0;
          if (j0 >= 0) {
#pragma unroll
            for (int e = 0; e < V2; ++e) {
              const float2 c = cs[e], x = f2_unpack(v[q][e]);
              v[q][e] = f2_pack(x.x * c.x - x.y * c.y, x.x * c.y + x.y * c.x);
            }
          } else if (j0 + V2 > 0) {                   // the rope dims begin inside the piece
#pragma unroll
            for (int e = 0; e < V2; ++e) {
              if (j0 + e >= 0) {
                const float2 c = cs[e], x = f2_unpack(v[q][e]);
                v[q][e] = f2_pack(x.x * c.x - x.y * c.y, x.x * c.y + x.y * c.x);
              }
            }
          }
          *reinterpret_cast<uint4*>(y + LPR * q * VEC) = f2_store<T>(v[q]);
        }
      }
    }
  }
}

}  // namespace csahca
