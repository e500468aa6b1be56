// Attention of draft-tree nodes on CUDA cores: fp32, and bf16 shapes other than
// 64 heads of 512 dims ("Paper Breakdown: DeepSeek-V4", section 4: MQA core
// attention, sliding window, HCA, attention sink).
//
// One CTA = one node x up to four heads x one split of its keys: the node's
// compressed keys (the selected entries, or every committed one), then its
// plan's list.  Each warp takes every kWarps-th tile of 32 keys by itself: it
// copies the rows to its own shared-memory tile as fp32 (rows d + 4 floats
// apart, so that 16-byte reads of one row per lane meet no bank twice), forms
// the scores with a key per lane (one read of a key for the four heads), keeps
// an online softmax per head, and accumulates O with d / 32 dims per lane.  The
// warps are joined at the end.  Bound by shared-memory reads and latency: these
// are small shapes (16 heads of 128 dims, 22 nodes, 203 keys: 57 us with 32
// keys a CTA at a time and element-wise copies).
#pragma once
#include "norm_rope.cuh"

namespace csahca {

constexpr int kTsaHeads = 4;
constexpr int kTsaKeys = 32;
constexpr int kTsaMaxSplits = 512;
// warps of a CTA for rows of d dims (32 x (d + 4) floats each)
__host__ __device__ constexpr int tsa_warps(int dpl) { return dpl <= 4 ? 8 : dpl <= 8 ? 4 : 2; }

struct TreeSimtParams {
  const void* q; const float* q_gain; const float* sinks;
  int q_norm; float eps, scale; int rope_dims;
  int T, H, d;
  const void* kv; int N;
  const int* idx; int k;                 // CSA: [nodes, k]; null: HCA
  const void* rows[3];                   // ROW_RING, ROW_TREE, ROW_DRAFT bases
  const int* list; const int4* info; int list_stride;
  int splits;
  void* out;                             // [nodes, H, d]
  float* partial;                        // [nodes, H, splits][d + 4]: m, l, -, -, acc (null: one split)
  double theta[kNrMaxPairs];
};

template <typename T>
__device__ __forceinline__ const T* tsa_row(const TreeSimtParams& p, int node, int j, int ncomp) {
  if (j >= ncomp) {
    const int code = __ldg(p.list + (int64_t)node * p.list_stride + (j - ncomp));
    const int kind = code >> kRowShift;
    const void* base = kind == ROW_RING ? p.rows[0] : kind == ROW_TREE ? p.rows[1] : p.rows[2];
    return static_cast<const T*>(base) + (int64_t)(code & kRowMask) * p.d;
  }
  const int e = p.idx ? __ldg(p.idx + (int64_t)node * p.k + j) : j;
  const int64_t b = node / p.T;
  if (e < 0) return nullptr;
  if (e < p.N) return static_cast<const T*>(p.kv) + (b * p.N + e) * p.d;
  if (e - p.N < p.T && p.rows[ROW_DRAFT]) return static_cast<const T*>(p.rows[ROW_DRAFT]) + (b * p.T + (e - p.N)) * p.d;
  raise_device_error(DEVERR_BAD_INDEX);
  return nullptr;
}

// o of one head (d values in shared memory, unnormalised, relative to m) with
// its sink, rope dims turned back by -t, into out.
template <typename T>
__device__ __forceinline__ void tsa_write(const float* o, float m, float l, float z, int t, int d, int rope_dims,
                                          const double* theta, T* out, int lane, int lanes) {
  const float M = fmaxf(m, z);
  // no key, or all weight on an infinite sink: 0
  const float f = m == -INFINITY || z == INFINITY ? 0.f : expf(m - M) / (expf(z - M) + l * expf(m - M));
  const int r0 = d - rope_dims;
  for (int x = 2 * lane; x < d; x += 2 * lanes) {
    float a = o[x] * f, b = o[x + 1] * f;
    if (x >= r0) {
      float cs, sn;
      rope_sincos(-(double)t, theta[(x - r0) >> 1], &cs, &sn);
      const float a0 = a;
      a = a0 * cs - b * sn;
      b = a0 * sn + b * cs;
    }
    out[x] = from_f32<T>(a);
    out[x + 1] = from_f32<T>(b);
  }
}

// DPL: at least d / 32.
template <typename T, int DPL>
__global__ void __launch_bounds__(32 * tsa_warps(DPL))
attn_tree_simt_kernel(const __grid_constant__ TreeSimtParams p) {
  constexpr int kWarps = tsa_warps(DPL), VEC = Vec16<T>::N;
  extern __shared__ __align__(16) float tsa_smem[];
  griddep_wait();
  griddep_launch_dependents();
  const int node = blockIdx.x, h0 = blockIdx.y * kTsaHeads, split = blockIdx.z;
  const int4 info = p.info[node];
  if (info.x < 0) return;                            // no node: its rows are left as they are
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d = p.d, ld = d + 4, dpl = d / 32, nh = min(kTsaHeads, p.H - h0);
  float* qs = tsa_smem;                              // [4][d]
  float* tile = qs + kTsaHeads * d + warp * kTsaKeys * ld;
  __shared__ float m_s[kWarps][kTsaHeads], l_s[kWarps][kTsaHeads];

  // queries: RMSNorm * gain, RoPE at t, times the softmax scale
  for (int h = warp; h < kTsaHeads; h += kWarps) {
    float v[DPL], ss = 0.f;
    const T* Q = static_cast<const T*>(p.q) + ((int64_t)node * p.H + h0 + min(h, nh - 1)) * d;
#pragma unroll
    for (int e = 0; e < DPL; ++e)
      if (e < dpl) { v[e] = to_f32(Q[lane + 32 * e]); ss = fmaf(v[e], v[e], ss); }
    const float inv = p.q_norm ? rsqrtf(warp_sum(ss) / (float)d + p.eps) : 1.f;
#pragma unroll
    for (int e = 0; e < DPL; ++e) {
      if (e < dpl) {
        const int dim = lane + 32 * e, r0 = d - p.rope_dims;
        v[e] *= inv * (p.q_norm && p.q_gain ? p.q_gain[dim] : 1.f);
        const float o = __shfl_xor_sync(0xffffffffu, v[e], 1);
        if (dim >= r0) {
          float cs, sn;
          rope_sincos((double)info.x, p.theta[(dim - r0) >> 1], &cs, &sn);
          v[e] = (dim & 1) ? fmaf(o, sn, v[e] * cs) : fmaf(-o, sn, v[e] * cs);
        }
        qs[h * d + dim] = v[e];
      }
    }
  }
  __syncthreads();

  const int ncomp = p.idx ? p.k : info.y, J = ncomp + info.z;
  const int tiles = (J + kTsaKeys - 1) / kTsaKeys;
  const int t0 = (int)((int64_t)tiles * split / p.splits), t1 = (int)((int64_t)tiles * (split + 1) / p.splits);
  const int nch = d / VEC;                           // 16-byte pieces of a row
  const int lpr = nch >= 32 ? 32 : nch > 16 ? 32 : nch > 8 ? 16 : nch > 4 ? 8 : 4;   // lanes that share a row's copy
  const int rpi = 32 / lpr, sub = lane & (lpr - 1), rsub = lane / lpr;
  float m[kTsaHeads], l[kTsaHeads], acc[kTsaHeads][DPL];
#pragma unroll
  for (int h = 0; h < kTsaHeads; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < DPL; ++e) acc[h][e] = 0.f;
  }
  for (int tl = t0 + warp; tl < t1; tl += kWarps) {
    const int j = tl * kTsaKeys + lane;
    const T* mine = j < J ? tsa_row<T>(p, node, j, ncomp) : nullptr;
    const int nk = min(kTsaKeys, J - tl * kTsaKeys);
    // copy the tile (a row that is no key: zeros)
    for (int c0 = 0; c0 < nch; c0 += lpr) {
      const int ch = c0 + sub;
#pragma unroll 8
      for (int r = 0; r < kTsaKeys; r += rpi) {
        const T* src = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, (unsigned long long)mine, r + rsub));
        float x[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = 0.f;
        if (ch < nch) {
          if (src) unpack16<T>(__ldg(reinterpret_cast<const uint4*>(src + ch * VEC)), x);
          float4* dst = reinterpret_cast<float4*>(tile + (r + rsub) * ld + ch * VEC);
#pragma unroll
          for (int e = 0; e < VEC / 4; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
      }
    }
    __syncwarp();
    // scores: this lane's key, four heads
    float s[kTsaHeads] = {0.f, 0.f, 0.f, 0.f};
    const float4* kr = reinterpret_cast<const float4*>(tile + lane * ld);
    const float4* q4 = reinterpret_cast<const float4*>(qs);
#pragma unroll 4
    for (int c = 0; c < d / 4; ++c) {
      const float4 kf = kr[c];
#pragma unroll
      for (int h = 0; h < kTsaHeads; ++h) {
        const float4 qf = q4[h * (d / 4) + c];
        s[h] = fmaf(qf.x, kf.x, s[h]);
        s[h] = fmaf(qf.y, kf.y, s[h]);
        s[h] = fmaf(qf.z, kf.z, s[h]);
        s[h] = fmaf(qf.w, kf.w, s[h]);
      }
    }
#pragma unroll
    for (int h = 0; h < kTsaHeads; ++h) {
      const float sc = mine ? s[h] * p.scale : -INFINITY;
      const float mn = fmaxf(m[h], warp_max(sc));
      const float ms = mn == -INFINITY ? 0.f : mn;
      const float pr = expf(sc - ms), corr = expf(m[h] - ms);
      l[h] = l[h] * corr + warp_sum(pr);
      m[h] = mn;
      s[h] = pr;
#pragma unroll
      for (int e = 0; e < DPL; ++e) acc[h][e] *= corr;
    }
#pragma unroll 4
    for (int kk = 0; kk < nk; ++kk) {
      float pk[kTsaHeads];
#pragma unroll
      for (int h = 0; h < kTsaHeads; ++h) pk[h] = __shfl_sync(0xffffffffu, s[h], kk);
#pragma unroll
      for (int e = 0; e < DPL; ++e) {
        if (e < dpl) {
          const float x = tile[kk * ld + lane + 32 * e];
#pragma unroll
          for (int h = 0; h < kTsaHeads; ++h) acc[h][e] = fmaf(pk[h], x, acc[h][e]);
        }
      }
    }
    __syncwarp();
  }
  // join the warps: every warp's O relative to the common maximum, in its tile
  if (lane == 0) {
#pragma unroll
    for (int h = 0; h < kTsaHeads; ++h) { m_s[warp][h] = m[h]; l_s[warp][h] = l[h]; }
  }
  __syncthreads();
  float M[kTsaHeads];
#pragma unroll
  for (int h = 0; h < kTsaHeads; ++h) {
    M[h] = m_s[0][h];
    for (int w = 1; w < kWarps; ++w) M[h] = fmaxf(M[h], m_s[w][h]);
    const float f = m[h] == -INFINITY ? 0.f : expf(m[h] - M[h]);
#pragma unroll
    for (int e = 0; e < DPL; ++e)
      if (e < dpl) tile[h * d + lane + 32 * e] = acc[h][e] * f;
  }
  __syncthreads();
  for (int x = threadIdx.x; x < nh * d; x += blockDim.x) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w) o += qs[kTsaHeads * d + w * kTsaKeys * ld + x];
    qs[x] = o;                                       // (the queries are no longer needed)
  }
  __syncthreads();
  for (int h = warp; h < nh; h += kWarps) {
    float lsum = 0.f, mh = m_s[0][h];
    for (int w = 1; w < kWarps; ++w) mh = fmaxf(mh, m_s[w][h]);
    for (int w = 0; w < kWarps; ++w)
      lsum += m_s[w][h] == -INFINITY ? 0.f : l_s[w][h] * expf(m_s[w][h] - mh);
    const int64_t row = (int64_t)node * p.H + h0 + h;
    if (p.partial) {
      float* P = p.partial + (row * p.splits + split) * (d + 4);
      if (lane == 0) { P[0] = mh; P[1] = lsum; }
      for (int x = lane; x < d; x += 32) P[4 + x] = qs[h * d + x];
    } else {
      tsa_write<T>(qs + h * d, mh, lsum, p.sinks[h0 + h], info.x, d, p.rope_dims, p.theta,
                   static_cast<T*>(p.out) + row * d, lane, 32);
    }
  }
}

// Join of a row's splits: one CTA per (node, head).
template <typename T>
__global__ void __launch_bounds__(128) tree_simt_combine_kernel(const __grid_constant__ TreeSimtParams p) {
  __shared__ float w_s[kTsaMaxSplits], o_s[512];
  __shared__ float stat[2];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int t = p.info[row / p.H].x;
  if (t < 0) return;
  const int d = p.d;
  const float* P = p.partial + row * p.splits * (d + 4);
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    float M = -INFINITY, l = 0.f;
    for (int s = lane; s < p.splits; s += 32) M = fmaxf(M, P[(int64_t)s * (d + 4)]);
    M = warp_max(M);
    for (int s = lane; s < p.splits; s += 32) {
      const float ms = P[(int64_t)s * (d + 4)];
      const float f = ms == -INFINITY ? 0.f : expf(ms - M);
      w_s[s] = f;
      l = fmaf(P[(int64_t)s * (d + 4) + 1], f, l);
    }
    l = warp_sum(l);
    if (lane == 0) { stat[0] = M; stat[1] = l; }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < d; x += blockDim.x) {
    float o = 0.f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) o = fmaf(P[(int64_t)s * (d + 4) + 4 + x], w_s[s], o);
    o_s[x] = o;
  }
  __syncthreads();
  tsa_write<T>(o_s, stat[0], stat[1], p.sinks[row % p.H], t, d, p.rope_dims, p.theta, static_cast<T*>(p.out) + row * d,
               threadIdx.x, blockDim.x);
}

}  // namespace csahca
