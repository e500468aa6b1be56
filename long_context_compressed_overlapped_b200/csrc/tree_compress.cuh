// Compressed entries that drafted tokens complete ("Paper Breakdown:
// DeepSeek-V4", section 4: CSA KV compression, HCA, Additional Techniques).
//
// Node i of a draft tree stands at position t = pos[b] + depth.  If t ends a
// block, (t + 1) % m == 0, the path to the node completes entry
// (t + 1) / m - 1: per channel the softmax-weighted pool of the block's m
// tokens (CSA: and of the preceding block's, 2m logits jointly), token p from
// the path's node at depth p - pos where p >= pos and from the ring of the
// committed tokens' raw streams otherwise.  Siblings that complete the same
// entry pool different tokens, so every node has its own row.
//
// One CTA = one node; a node that completes nothing leaves at once.  A thread
// owns a 16-byte vector of channels and every G-th token of the pool, so that
// all rows of the pool are asked for in one or few round trips to L2: the call
// is bound by those and by the walk up the tree, not by its few hundred KB.
// The G partial softmaxes (max, sum, weighted sum) are joined in shared
// memory, a channel a thread.  256 threads for the 2m rows of CSA (three CTAs an
// SM; 512 at one an SM ran in four waves, 22 us instead of 9 for 512 nodes),
// 512 for the m' of HCA.
#pragma once
#include "norm_rope.cuh"
#include "tc_common.cuh"

namespace csahca {

constexpr int kTcpMaxTokens = 512;      // 2m (CSA), m (HCA)
constexpr float kLog2eF = 1.4426950408889634f;

template <bool kCSA> __host__ __device__ constexpr int tree_compress_threads() { return kCSA ? 256 : 512; }
template <typename T, bool kCSA> constexpr int tree_compress_smem() {
  return 3 * Vec16<T>::N * tree_compress_threads<kCSA>() * 4;
}

struct TreeCompressParams {
  const int* parents; const int* pos;
  const void* nw[4];                    // drafted tokens' streams [B, T, c]: a, b, za, zb (HCA: a, za)
  const void* ring;                     // [B, R, S, c]
  const float* bias_a; const float* bias_b; const float* gain;
  void* out; float* out_scale;          // [B, T, c]; e4m3: codes, [B, T, c / 128]
  int T, c, m, rms_norm, rope_dims, e4m3;
  int64_t kv_row_bytes;                 // > 0: out holds FP8 KV rows of so many bytes
  int64_t out_row_bytes; int zero_rest; // rows that no entry fills become zeros
  float eps;
  double theta[kNrMaxPairs];
};

template <typename T, bool kCSA>
__global__ void __launch_bounds__(tree_compress_threads<kCSA>(), kCSA ? 3 : 1)
tree_compress_kernel(const __grid_constant__ TreeCompressParams p) {
  constexpr int VEC = Vec16<T>::N, kThreads = tree_compress_threads<kCSA>();
  constexpr int S = kCSA ? 4 : 2;
  constexpr int kTcpBatch = kCSA ? 2 : 4;             // tokens of a thread in flight
  // partial softmaxes by vector element: thread x's element e at [e][x], conflict-free
  extern __shared__ __align__(16) float tcp_smem[];
  float (*st_mx)[kThreads] = reinterpret_cast<float (*)[kThreads]>(tcp_smem);
  float (*st_s)[kThreads] = st_mx + VEC;
  float (*st_acc)[kThreads] = st_s + VEC;
  __shared__ int src_s[kTcpMaxTokens];  // >= 0: node of the tree; < 0: ring slot -1 - src
  __shared__ TreeNode node_s;
  __shared__ float red_s[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int tok = blockIdx.x, b = tok / p.T, i = tok - b * p.T;
  const int t = tree_node(p.parents, p.pos, b, p.T, i, &node_s);
  const int m = p.m, c = p.c;
  if (t < 0 || (t + 1) % m != 0) {
    // (a row of out is a multiple of 8 bytes: c % 128 codes, 16-byte vectors, or an FP8 KV row)
    uint2* z = p.zero_rest ? reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + tok * p.out_row_bytes) : nullptr;
    for (int j = threadIdx.x; z && j < (int)(p.out_row_bytes / 8); j += kThreads) z[j] = make_uint2(0u, 0u);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31;
  const int R = kCSA ? 2 * m : m;
  const int p0 = node_s.pos0;
  const int blk = (t + 1) / m - 1;
  const int J0 = (kCSA && blk == 0) ? m : 0;          // entry 0 has no preceding block
  for (int j = J0 + tid; j < R; j += kThreads) {
    const int q = t + 1 - R + j;                      // token j of the pool (CSA: preceding block first)
    src_s[j] = q >= p0 ? node_s.at(q) : -1 - q % R;
  }
  __syncthreads();

  const int nv = c / VEC, G = kThreads / nv;          // nv <= 128: G >= 2
  const int vec = tid % nv, grp = tid / nv, ch0 = vec * VEC;
  float mx[VEC], s[VEC], acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) { mx[e] = -INFINITY; s[e] = 0.f; acc[e] = 0.f; }
  if (grp < G) {
    for (int jb = J0 + grp; jb < R; jb += G * kTcpBatch) {
      uint4 rv[kTcpBatch], rz[kTcpBatch];
      float4 rb[kTcpBatch][VEC / 4];
#pragma unroll
      for (int u = 0; u < kTcpBatch; ++u) {
        const int j = jb + u * G;
        if (j < R) {
          const int sb = (kCSA && j < m) ? 1 : 0;     // CSA: the preceding block reads stream b
          const int src = src_s[j];
          const T* rv_p; const T* rz_p;
          if (src >= 0) {
            const int64_t o = ((int64_t)b * p.T + src) * c + ch0;
            rv_p = static_cast<const T*>(p.nw[sb]) + o;
            rz_p = static_cast<const T*>(p.nw[S / 2 + sb]) + o;
          } else {
            const T* ring = static_cast<const T*>(p.ring) + (((int64_t)b * R + (-1 - src)) * S) * c + ch0;
            rv_p = ring + (int64_t)sb * c;
            rz_p = ring + (int64_t)(S / 2 + sb) * c;
          }
          rv[u] = __ldg(reinterpret_cast<const uint4*>(rv_p));
          rz[u] = __ldg(reinterpret_cast<const uint4*>(rz_p));
          const float* bias = kCSA ? (j < m ? p.bias_b + (int64_t)j * c : p.bias_a + (int64_t)(j - m) * c)
                                   : p.bias_a + (int64_t)j * c;
#pragma unroll
          for (int e = 0; e < VEC / 4; ++e) rb[u][e] = __ldg(reinterpret_cast<const float4*>(bias + ch0) + e);
        }
      }
      // the batch's logits in log2 units (-inf: weight 0, and where there is no
      // token), one new maximum and one rescale of the running sums a channel
      float z[kTcpBatch][VEC];
#pragma unroll
      for (int u = 0; u < kTcpBatch; ++u) {
        if (jb + u * G < R) {
          unpack16<T>(rz[u], z[u]);
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            z[u][e] = (z[u][e] + reinterpret_cast<const float*>(&rb[u][e / 4])[e % 4]) * kLog2eF;
        } else {
          rv[u] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int e = 0; e < VEC; ++e) z[u][e] = -INFINITY;
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float M = mx[e];
#pragma unroll
        for (int u = 0; u < kTcpBatch; ++u) M = fmaxf(M, z[u][e]);
        const float Ms = M == -INFINITY ? 0.f : M, f = fast_exp2(mx[e] - Ms);
        mx[e] = M;
        s[e] *= f;
        acc[e] *= f;
#pragma unroll
        for (int u = 0; u < kTcpBatch; ++u) {
          z[u][e] = fast_exp2(z[u][e] - Ms);
          s[e] += z[u][e];
        }
      }
#pragma unroll
      for (int u = 0; u < kTcpBatch; ++u) {
        float v[VEC];
        unpack16<T>(rv[u], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          acc[e] = z[u][e] != 0.f ? fmaf(z[u][e], v[e], acc[e]) : acc[e];   // (a token of weight 0 is not read into the sum)
      }
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) { st_mx[e][tid] = mx[e]; st_s[e][tid] = s[e]; st_acc[e][tid] = acc[e]; }
  __syncthreads();
  // element x = e * nv + vec of the row by thread x mod kThreads: the groups'
  // partials joined; the pooled values then go back through st_mx[e][vec]
  float ss = 0.f;
  for (int x = tid; x < VEC * nv; x += kThreads) {
    const int e = x / nv, w = x - e * nv;
    float M = -INFINITY;
    for (int g = 0; g < G; ++g) M = fmaxf(M, st_mx[e][g * nv + w]);
    float sum = 0.f, a = 0.f;
    for (int g = 0; g < G; ++g) {
      const float mg = st_mx[e][g * nv + w];
      const float f = mg == M ? 1.f : exp2f(mg - M);  // (a group without tokens: exp2f(-inf) = 0)
      sum = fmaf(st_s[e][g * nv + w], f, sum);
      a = fmaf(st_acc[e][g * nv + w], f, a);
    }
    const float r = a / sum;
    st_mx[e][w] = r;                                  // (this thread alone reads column w of row e)
    ss = fmaf(r, r, ss);
  }
  float inv = 1.f;
  if (p.rms_norm) {
    ss = warp_sum(ss);
    if (lane == 0) red_s[tid >> 5] = ss;
    __syncthreads();
    float tot = 0.f;
    for (int k = 0; k < kThreads / 32; ++k) tot += red_s[k];
    inv = rsqrtf(tot / (float)c + p.eps);
  } else {
    __syncthreads();
  }
  float y[VEC];                                       // the first nv threads: a vector of the row
  if (tid < nv) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      y[e] = st_mx[e][tid] * (p.rms_norm ? inv * (p.gain ? __ldg(p.gain + ch0 + e) : 1.f) : 1.f);
    const int j0 = ch0 - (c - p.rope_dims);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      if (j0 + e >= 0) {
        float cs, sn;
        rope_sincos((double)blk * (double)m, p.theta[(j0 + e) >> 1], &cs, &sn);
        const float x0 = y[e], x1 = y[e + 1];
        y[e] = x0 * cs - x1 * sn;
        y[e + 1] = x0 * sn + x1 * cs;
      }
    }
  }
  if (p.kv_row_bytes > 0) {
    // FP8 KV row: 64-dim blocks of codes with one fp32 scale each (the cache's
    // rule), the rope dims as bf16; 8 lanes hold a block
    if (p.zero_rest) {                                // (and what fills the row up to 128 bytes)
      uint32_t* row = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + tok * p.kv_row_bytes);
      for (int j = (c + p.rope_dims) / 4 + (c - p.rope_dims) / 64 + tid; j < (int)(p.kv_row_bytes / 4); j += kThreads)
        row[j] = 0u;
    }
    if (tid < (nv + 31) / 32 * 32) {
      float amax = 0.f;
      if (tid < nv) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fabsf(y[e]));
      }
#pragma unroll
      for (int o = 64 / VEC / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (tid < nv) {
        uint8_t* row = static_cast<uint8_t*>(p.out) + (int64_t)tok * p.kv_row_bytes;
        const int nope = c - p.rope_dims;
        if (ch0 < nope) {
          const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            row[ch0 + e] = __nv_cvt_float_to_fp8(__fdiv_rn(y[e], scale), __NV_SATFINITE, __NV_E4M3);
          if (ch0 % 64 == 0) *reinterpret_cast<float*>(row + c + p.rope_dims + 4 * (ch0 / 64)) = scale;
        } else {
          store16(reinterpret_cast<__nv_bfloat16*>(row + nope) + (ch0 - nope), y);
        }
      }
    }
    return;
  }
  if (!p.e4m3) {
    if (tid < nv) store16(static_cast<T*>(p.out) + (int64_t)tok * c + ch0, y);
    return;
  }
  // e4m3 codes with one fp32 scale per 128 channels, amax / 448 (1 for an
  // all-zero block): the cache's rule (the pooled values are decode_compress's to
  // some ulps, being summed in another order, and codes next to a border differ)
  // (nv is a multiple of 128 / VEC lanes, which divides a warp)
  constexpr int LB = 128 / VEC;
  if (tid < (nv + 31) / 32 * 32) {
    float amax = 0.f;
    if (tid < nv) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fabsf(y[e]));
    }
#pragma unroll
    for (int o = LB / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (tid < nv) {
      const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
      uint8_t* o = static_cast<uint8_t*>(p.out) + (int64_t)tok * c + ch0;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        o[e] = __nv_cvt_float_to_fp8(__fdiv_rn(y[e], scale), __NV_SATFINITE, __NV_E4M3);
      if (ch0 % 128 == 0) p.out_scale[(int64_t)tok * (c / 128) + ch0 / 128] = scale;
    }
  }
}

}  // namespace csahca
