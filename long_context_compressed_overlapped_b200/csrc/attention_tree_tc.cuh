// Attention of draft-tree nodes on the tensor cores (64 heads of 512 dims,
// bf16; "Paper Breakdown: DeepSeek-V4", section 4: MQA core attention,
// sliding window, HCA, attention sink; one query per drafted token).
//
// Both products are written transposed, as in the decode kernel, so that one
// copy of a key tile serves both (K = V) and O^T [512 x 64] fits TMEM beside
// S^T:  S^T [128 keys x 64 heads] = K . Q^T,  O^T += V^T . P^T.
//
// A node's keys are two runs.  Tiles of 128 consecutive committed entries
// (HCA) arrive by TMA, two 64-dim chunks a box (an SM completes about one TMA
// op per 580 cycles whatever its size, so 32 KB boxes).  Everything else is
// the node's row list, gathered row by row: the selected entries (CSA) or the
// entries past the last whole tile (HCA), then the plan's list (window rows by
// position out of the ring or the path, and the path's drafted entries).  Rows
// of the list that are no key, and the rows that fill its last MMA step, are
// written as zeros: nothing that a mask hides is read, so NaN there cannot
// reach O.
//
// Roles (896 threads): warps 0-7 softmax and epilogue (two groups of four
// warps, group g owns heads 32g .. 32g + 31; thread i of a group is key slot i
// of S^T and dim slot i of each O^T M-tile), warps 8-23 producers, then the
// S and the P.V MMA issuers.  Each producer warp copies 8 rows of a gathered
// tile, waits for its own copies of a chunk pair and arrives once (a barrier
// arrival per lane and chunk was 4,096 of them a tile).
//
// Work items: (node, split of its tiles).  With one split the item writes the
// final row, otherwise a partial for tree_combine_kernel.
#pragma once
#include "attention_tc.cuh"
#include "norm_rope.cuh"

namespace csahca {

constexpr int kTreeProducers = 16;
constexpr int kTreeThreads = 32 * (8 + kTreeProducers + 4);
constexpr int kTreePairs = kAttnChunks / 2;              // chunk pairs of a tile (= O^T M-tiles)
static_assert(kTreePairs == kAttnMT, "a chunk pair is one O^T M-tile's rows");
static_assert(256 * kAttnRegsSoftmax + 32 * kTreeProducers * kAttnRegsProducer + 128 * kAttnRegsMma <= 72 * kTreeThreads,
              "the register split fits a 72-register launch");

struct TreeAttnParams {
  const __nv_bfloat16* kv;               // [B * N, D]
  const __nv_bfloat16* rows[3];          // ROW_RING, ROW_TREE, ROW_DRAFT bases
  const int* idx;                        // CSA: [nodes, k]; null: HCA
  const int* list; const int4* info;
  const float* sinks;
  int list_stride;                       // w + T
  int k, N, T;
  int n_items, splits;
  float scale_log2;
  int rope_dims;
  __nv_bfloat16* out;                    // [nodes, H, D]
  char* partial;                         // [nodes][splits] blocks of kTcPartialBytes
  double theta[64];
};

struct TreeItem { int node, split, t, full, tail, nlist, tile0, tile1; };

__device__ __forceinline__ int4 tree_info(const TreeAttnParams& p, int id) {
  return id < p.n_items ? __ldg(p.info + id / p.splits) : make_int4(-1, 0, 0, 0);
}
__device__ __forceinline__ TreeItem tree_item(const TreeAttnParams& p, int id, const int4& f) {
  TreeItem it;
  it.node = id / p.splits;
  it.split = id - it.node * p.splits;
  it.t = f.x;
  it.full = p.idx ? 0 : f.y >> 7;
  it.tail = p.idx ? p.k : f.y & 127;
  it.nlist = it.tail + f.z;
  const int total = f.x < 0 ? 0 : it.full + ((it.nlist + 127) >> 7);
  it.tile0 = (int)((int64_t)total * it.split / p.splits);
  it.tile1 = (int)((int64_t)total * (it.split + 1) / p.splits);
  return it;
}
// Row j of the node's list, or null if it is no key.
__device__ __forceinline__ const __nv_bfloat16* tree_row(const TreeAttnParams& p, const TreeItem& it, int j) {
  if (j >= it.nlist) return nullptr;
  const int b = it.node / p.T;
  if (j >= it.tail) {
    const int code = __ldg(p.list + (int64_t)it.node * p.list_stride + (j - it.tail));
    const int kind = code >> kRowShift;
    const __nv_bfloat16* base = kind == ROW_RING ? p.rows[0] : kind == ROW_TREE ? p.rows[1] : p.rows[2];
    return base + (int64_t)(code & kRowMask) * kAttnD;
  }
  if (!p.idx) return p.kv + ((int64_t)b * p.N + it.full * 128 + j) * kAttnD;
  const int e = __ldg(p.idx + (int64_t)it.node * p.k + j);
  if (e < 0) return nullptr;
  if (e < p.N) return p.kv + ((int64_t)b * p.N + e) * kAttnD;
  if (e - p.N < p.T && p.rows[ROW_DRAFT]) return p.rows[ROW_DRAFT] + ((int64_t)b * p.T + (e - p.N)) * kAttnD;
  raise_device_error(DEVERR_BAD_INDEX);
  return nullptr;
}
__device__ __forceinline__ bool tree_key_valid(const TreeAttnParams& p, const TreeItem& it, int j) {
  if (j >= it.nlist) return false;
  if (!p.idx || j >= it.tail) return true;
  const int e = __ldg(p.idx + (int64_t)it.node * p.k + j);
  return e >= 0 && (e < p.N || (e - p.N < p.T && p.rows[ROW_DRAFT]));
}

// 16 bytes global -> shared, or 16 zero bytes if !live (nothing is read then).
__device__ __forceinline__ void cp_async16_or_zero(void* dst_smem, const void* src_gmem, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst_smem)), "l"(src_gmem),
               "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

__global__ void __launch_bounds__(kTreeThreads, 1)
attn_tree_tc_kernel(const __grid_constant__ CUtensorMap comp_rows, const __grid_constant__ CUtensorMap q_rows,
                    const __grid_constant__ CUtensorMap part_rows, const __grid_constant__ TreeAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sK = sQ + AttnSmem::Q_BYTES;
  uint8_t* sP = sK + AttnSmem::K_BYTES;
  // bar_pv[j]: the tile's P.V MMAs of O^T M-tiles 0 .. j have completed (key
  // chunk pair j is free; j = 3: O^T and P^T may be touched again)
  __shared__ uint64_t bar_kfull[kTreePairs], bar_pv[kTreePairs];
  __shared__ uint64_t bar_q_full, bar_q_empty, bar_s_full, bar_s_empty, bar_p_full, bar_done;
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  __shared__ float red[2][4 * 32];
  __shared__ __align__(16) float stat_a[kAttnH];
  __shared__ __align__(16) float m_use[kAttnH];
  __shared__ __align__(16) float alpha[kAttnH];
  __shared__ float l_run[kAttnH];
  __shared__ double theta_s[64];
  __shared__ int need_rescale[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarpS = 8 + kTreeProducers, kWarpPV = kWarpS + 1;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int c = 0; c < kTreePairs; ++c) {
      mbar_init(&bar_kfull[c], kTreeProducers);
      mbar_init(&bar_pv[c], 1);
    }
    mbar_init(&bar_q_full, 1);
    mbar_init(&bar_q_empty, 1);
    mbar_init(&bar_s_full, 1);
    mbar_init(&bar_s_empty, 256);
    mbar_init(&bar_p_full, 256);
    mbar_init(&bar_done, 2);
    mbar_fence_init();
  }
  if (threadIdx.x < 64) theta_s[threadIdx.x] = p.theta[threadIdx.x];
  if (warp == kWarpS) tmem_alloc(&tmem_base_sh, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const uint32_t tS = tmem;                              // S^T: H columns
  const uint32_t tO = tmem + 128;                        // O^T M-tile j: columns [128 + j H, ...)
  const uint32_t tL = tmem + 128 + kAttnMT * kAttnH;     // per-key-slot sums of p
  // the plan, the finished rows and the selection come from earlier kernels
  griddep_wait();
  griddep_launch_dependents();

  if (warp >= 8 && warp < kWarpS) {
    setmaxnreg_dec<kAttnRegsProducer>();
    // ------------------------------------------------------------ producers
    const int pw = warp - 8;
    if (lane == 0) {
      tma_prefetch_desc(&comp_rows);
      tma_prefetch_desc(&q_rows);
    }
    const int piece = lane & 7, rg = lane >> 3;
    const int r0 = 4 * pw + rg, r1 = r0 + 64;            // this lane's rows of a gathered tile
    uint32_t tcount = 0, icount = 0;
    bool stop = false;                                   // warp-uniform
    int4 f = tree_info(p, blockIdx.x);
    for (int id = blockIdx.x; id < p.n_items && !stop; id += gridDim.x) {
      const TreeItem it = tree_item(p, id, f);
      f = tree_info(p, id + gridDim.x);
      if (it.tile1 <= it.tile0) continue;
      if (pw == 0) {
        int ok = 1;
        if (lane == 0) {
          ok = mbar_wait(&bar_q_empty, (icount & 1) ^ 1, &abort_flag);
          if (ok) {
            mbar_expect_tx(&bar_q_full, AttnSmem::Q_BYTES);
            tma_load_3d(sQ, &q_rows, 0, it.node * kAttnH, 0, &bar_q_full);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) { stop = true; break; }
        ++icount;
      }
      const __nv_bfloat16 *n0 = nullptr, *n1 = nullptr;  // the next gathered tile's rows
      bool have_next = false;
      for (int tile = it.tile0; tile < it.tile1 && !stop; ++tile, ++tcount) {
        const uint32_t ph = tcount & 1;
        if (tile < it.full) {
          // 128 consecutive entries: box c (two chunks) by producer warp c
          const int row0 = (it.node / p.T) * p.N + tile * 128;
          for (int c = 0; c < kTreePairs; ++c) {
            int ok = 1;
            if (lane == 0) {
              ok = mbar_wait(&bar_pv[c], ph ^ 1, &abort_flag);
              if (ok) {
                if (c == pw) {
                  mbar_expect_tx(&bar_kfull[c], 2 * AttnSmem::K_CHUNK);
                  tma_load_3d(sK + 2 * c * AttnSmem::K_CHUNK, &comp_rows, 0, row0, 2 * c, &bar_kfull[c]);
                } else {
                  mbar_arrive(&bar_kfull[c]);
                }
              }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) { stop = true; break; }
          }
          continue;
        }
        const int off = (tile - it.full) * 128;
        const int fill = min(128, (it.nlist - off + 15) & ~15);   // rows that the P.V MMAs read
        const __nv_bfloat16* s0 = have_next ? n0 : tree_row(p, it, off + r0);
        const __nv_bfloat16* s1 = have_next ? n1 : tree_row(p, it, off + r1);
        const bool l0 = s0 != nullptr, l1 = s1 != nullptr;
        if (!l0) s0 = p.kv;
        if (!l1) s1 = p.kv;
        for (int c = 0; c < kTreePairs; ++c) {
          int ok = 1;
          if (lane == 0) ok = mbar_wait(&bar_pv[c], ph ^ 1, &abort_flag);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) { stop = true; break; }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint8_t* dst = sK + (2 * c + h) * AttnSmem::K_CHUNK;
            const int o = (2 * c + h) * 64 + piece * 8;
            if (r0 < fill) cp_async16_or_zero(dst + sw128_offset(r0, piece * 16), s0 + o, l0);
            if (r1 < fill) cp_async16_or_zero(dst + sw128_offset(r1, piece * 16), s1 + o, l1);
          }
          cp_async_commit();
        }
        // the next tile's rows, and their lines into L2 behind this tile's copies
        have_next = tile + 1 < it.tile1;
        if (have_next) {
          n0 = tree_row(p, it, off + 128 + r0);
          n1 = tree_row(p, it, off + 128 + r1);
          if (n0) prefetch_l2_line(n0 + piece * 64);
          if (n1) prefetch_l2_line(n1 + piece * 64);
        }
        if (stop) break;
        // every lane's own copies of pair c have landed and are made visible
        // to the MMAs (async proxy) before the warp's one arrival
#pragma unroll
        for (int c = 0; c < kTreePairs; ++c) {
          if (c == 0) cp_async_wait<3>();
          else if (c == 1) cp_async_wait<2>();
          else if (c == 2) cp_async_wait<1>();
          else cp_async_wait<0>();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_kfull[c]);
        }
      }
    }
    // copies in flight end before the CTA may exit: this lane's gathers here,
    // the boxes and the query by their barriers
    cp_async_wait<0>();
    if (lane == 0 && pw < kTreePairs && tcount > 0) mbar_wait(&bar_kfull[pw], (tcount - 1) & 1, &abort_flag);
    if (lane == 0 && pw == 0 && icount > 0) mbar_wait(&bar_q_full, (icount - 1) & 1, &abort_flag);
  } else if (warp >= kWarpS) {
    setmaxnreg_dec<kAttnRegsMma>();
    if (warp == kWarpS && lane == 0) {
      // ---------------------------------------------------------- S issuer
      constexpr uint32_t idesc_s = umma_idesc_bf16(128, kAttnH, 0, 0);
      const uint64_t kdesc = umma_desc_kmajor(smem_u32(sK)), qdesc = umma_desc_kmajor(smem_u32(sQ));
      uint32_t tcount = 0, icount = 0;
      bool stop = false;
      int4 f = tree_info(p, blockIdx.x);
      for (int id = blockIdx.x; id < p.n_items && !stop && !abort_flag; id += gridDim.x) {
        const TreeItem it = tree_item(p, id, f);
        f = tree_info(p, id + gridDim.x);
        if (it.tile1 <= it.tile0) continue;
        if (!mbar_wait(&bar_q_full, icount & 1, &abort_flag)) break;
        ++icount;
        for (int tile = it.tile0; tile < it.tile1 && !stop; ++tile, ++tcount) {
          const uint32_t ph = tcount & 1;
          if (!mbar_wait(&bar_s_empty, ph ^ 1, &abort_flag)) { stop = true; break; }
          tc_fence_after();
          for (int c = 0; c < kTreePairs; ++c) {
            if (!mbar_wait(&bar_kfull[c], ph, &abort_flag)) { stop = true; break; }
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t kd = kdesc + (uint64_t)((2 * c + h) * (AttnSmem::K_CHUNK >> 4));
              const uint64_t qd = qdesc + (uint64_t)((2 * c + h) * (AttnSmem::Q_CHUNK >> 4));
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) umma_bf16(tS, kd + 2 * ks, qd + 2 * ks, idesc_s, (c | h | ks) != 0);
            }
          }
          if (stop) break;
          umma_commit(&bar_s_full);
          if (tile == it.tile1 - 1) umma_commit(&bar_q_empty);
        }
      }
      umma_commit(&bar_done);
      mbar_wait(&bar_done, 0, &abort_flag);
    } else if (warp == kWarpPV && lane == 0) {
      // -------------------------------------------------------- P.V issuer
      constexpr uint32_t idesc_pv = umma_idesc_bf16(128, kAttnH, 1, 1);
      const uint64_t vdesc = umma_desc_mnmajor(smem_u32(sK), AttnSmem::K_CHUNK);
      const uint64_t pdesc = umma_desc_mnmajor(smem_u32(sP), AttnSmem::P_BYTES);
      uint32_t tcount = 0;
      bool stop = false;
      int4 f = tree_info(p, blockIdx.x);
      for (int id = blockIdx.x; id < p.n_items && !stop && !abort_flag; id += gridDim.x) {
        const TreeItem it = tree_item(p, id, f);
        f = tree_info(p, id + gridDim.x);
        for (int tile = it.tile0; tile < it.tile1; ++tile, ++tcount) {
          if (!mbar_wait(&bar_p_full, tcount & 1, &abort_flag)) { stop = true; break; }
          tc_fence_after();
          const bool first = tile == it.tile0;
          // a list's last tile: P is 0 past its last row, the steps there are skipped
          const int hi = tile < it.full ? 128 : it.nlist - (tile - it.full) * 128;
          const int nks = min(8, (hi + 15) >> 4);
#pragma unroll
          for (int mt = 0; mt < kAttnMT; ++mt) {
            const uint64_t vd = vdesc + (uint64_t)((2 * mt) * (AttnSmem::K_CHUNK >> 4));
            if (nks == 8) {
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                umma_bf16(tO + mt * kAttnH, vd + 128 * ks, pdesc + 128 * ks, idesc_pv, !(first && ks == 0));
            } else {
              for (int ks = 0; ks < nks; ++ks)
                umma_bf16(tO + mt * kAttnH, vd + 128 * ks, pdesc + 128 * ks, idesc_pv, !(first && ks == 0));
            }
            umma_commit(&bar_pv[mt]);
          }
        }
      }
      umma_commit(&bar_done);
      mbar_wait(&bar_done, 0, &abort_flag);
    }
  } else {
    setmaxnreg_inc<kAttnRegsSoftmax>();
    // --------------------------------------------------- softmax / epilogue
    const int g = warp >> 2, gid = 1 + g;
    const int tid = threadIdx.x & 127, st = threadIdx.x;
    const int h0 = 32 * g;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t tcount = 0;
    const int r0 = kAttnD - p.rope_dims;
    const float4* mu4 = reinterpret_cast<const float4*>(m_use + h0);
    int4 f = tree_info(p, blockIdx.x);
    for (int id = blockIdx.x; id < p.n_items; id += gridDim.x) {
      const TreeItem it = tree_item(p, id, f);
      f = tree_info(p, id + gridDim.x);
      const bool empty = it.tile1 <= it.tile0;
      bool bad = false;                      // uniform over the group; both groups leave together
      if (tid < 32) m_use[h0 + tid] = -INFINITY;
      group_sync(gid);
      for (int tile = it.tile0; tile < it.tile1; ++tile, ++tcount) {
        if (bad) continue;
        const uint32_t ph = tcount & 1;
        const bool first = tile == it.tile0;
        const bool valid = tile < it.full || tree_key_valid(p, it, (tile - it.full) * 128 + tid);
        if (!mbar_wait_group(gid, &bar_s_full, ph, &abort_flag)) { bad = true; continue; }
        tc_fence_after();
        float v[32];
        tmem_ld32(tS + lane_base + h0, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = valid ? v[e] * p.scale_log2 : -INFINITY;
        // the running max is raised only where a score exceeds it by more than
        // 2^8 (or on the item's first tile)
        bool exceed = first;
        if (!first) {
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            const float4 mu = mu4[e4];
            exceed |= (v[4 * e4 + 0] > mu.x + kRescaleThreshold) | (v[4 * e4 + 1] > mu.y + kRescaleThreshold) |
                      (v[4 * e4 + 2] > mu.z + kRescaleThreshold) | (v[4 * e4 + 3] > mu.w + kRescaleThreshold);
          }
        }
        exceed = group_any(gid, exceed);
        bool rescale = false;
        if (exceed) {
          {
            float x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = v[e];
            reduce_group32<true>(x, red[g], stat_a + h0, gid);
          }
          if (tid == 0) need_rescale[g] = 0;
          group_sync(gid);
          if (tid < 32) {
            const int h = h0 + tid;
            const float mt = stat_a[h], mo = m_use[h];
            float a = 1.f;
            if (mt > mo + kRescaleThreshold || (mo == -INFINITY && mt != -INFINITY)) {
              a = (mo == -INFINITY) ? 0.f : exp2f(mo - mt);
              m_use[h] = mt;
              if (!first) need_rescale[g] = 1;
            }
            alpha[h] = a;
          }
          group_sync(gid);
          rescale = need_rescale[g] != 0;
        }
        // the previous tile's P.V has finished: P^T may be overwritten and
        // O^T / the sums rescaled
        if (!first) {
          if (!mbar_wait_group(gid, &bar_pv[kAttnMT - 1], ph ^ 1, &abort_flag)) { bad = true; continue; }
          tc_fence_after();
        }
        if (rescale) {
          const float4* al4 = reinterpret_cast<const float4*>(alpha + h0);
#pragma unroll 1
          for (int mt = 0; mt <= kAttnMT; ++mt) {
            float o[32];
            const uint32_t a = (mt < kAttnMT ? tO + mt * kAttnH : tL) + lane_base + h0;
            tmem_ld32(a, o);
            tmem_wait_ld();
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
              const float4 al = al4[e4];
              o[4 * e4 + 0] *= al.x; o[4 * e4 + 1] *= al.y; o[4 * e4 + 2] *= al.z; o[4 * e4 + 3] *= al.w;
            }
            tmem_st32(a, o);
          }
          tmem_wait_st();
        }
        // p = 2^(s - m), 0 for a key slot that is no key
#pragma unroll
        for (int e4 = 0; e4 < 8; ++e4) {
          const float4 mu = mu4[e4];
          v[4 * e4 + 0] = valid ? fast_exp2(v[4 * e4 + 0] - mu.x) : 0.f;
          v[4 * e4 + 1] = valid ? fast_exp2(v[4 * e4 + 1] - mu.y) : 0.f;
          v[4 * e4 + 2] = valid ? fast_exp2(v[4 * e4 + 2] - mu.z) : 0.f;
          v[4 * e4 + 3] = valid ? fast_exp2(v[4 * e4 + 3] - mu.w) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 o;
          store16(reinterpret_cast<__nv_bfloat16*>(&o), v + 8 * j);
          *reinterpret_cast<uint4*>(sP + sw128_offset(tid, (4 * g + j) * 16)) = o;
        }
        {
          const uint32_t la = tL + lane_base + h0;
          if (!first) {
            float l[32];
            tmem_ld32(la, l);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] += l[e];
          }
          tmem_st32(la, v);
          tmem_wait_st();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bar_s_empty);
        mbar_arrive(&bar_p_full);
      }
      // ---- epilogue
      if (!empty && !bad) {
        if (!mbar_wait_group(gid, &bar_pv[kAttnMT - 1], (tcount - 1) & 1, &abort_flag)) bad = true;
        else tc_fence_after();
      }
      if (!empty && !bad) {
        float v[32];
        tmem_ld32(tL + lane_base + h0, v);
        tmem_wait_ld();
        reduce_group32<false>(v, red[g], l_run + h0, gid);
      }
      bad = softmax_any256(bad);
      if (!bad && it.t >= 0) {
        if (p.splits > 1) {
          // m[H] (log2 units) and l[H] in fp32, then O / l as bf16 [D][H]; a
          // split without keys writes its header only (m = -inf, l = 0)
          float* hdr = reinterpret_cast<float*>(p.partial + (int64_t)id * kTcPartialBytes);
          if (tid < 32) {
            const int h = h0 + tid;
            const float l = empty ? 0.f : l_run[h];
            hdr[h] = l > 0.f ? m_use[h] : -INFINITY;
            hdr[kAttnH + h] = l;
            stat_a[h] = l > 0.f ? 1.f / l : 0.f;
          }
          group_sync(gid);
          if (!empty) {
            const float4* f4 = reinterpret_cast<const float4*>(stat_a + h0);
            const bool own_k = p.n_items <= (int)gridDim.x;   // the CTA's only item: stage in the key buffer
#pragma unroll 1
            for (int mt = 0; mt < kAttnMT; ++mt) {
              uint8_t* stg = own_k ? sK + mt * AttnSmem::K_CHUNK : sP;
              float o[32];
              tmem_ld32(tO + lane_base + mt * kAttnH + h0, o);
              tmem_wait_ld();
#pragma unroll
              for (int e4 = 0; e4 < 8; ++e4) {
                const float4 fc = f4[e4];
                o[4 * e4 + 0] *= fc.x; o[4 * e4 + 1] *= fc.y; o[4 * e4 + 2] *= fc.z; o[4 * e4 + 3] *= fc.w;
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint4 w;
                store16(reinterpret_cast<__nv_bfloat16*>(&w), o + 8 * q);
                *reinterpret_cast<uint4*>(stg + sw128_offset(tid, (4 * g + q) * 16)) = w;
              }
              fence_proxy_async_smem();
              softmax_sync256();
              if (st == 0) {
                tma_store_2d(&part_rows, stg, 0, id * kTcPartialRows + kTcPartialHeaderRows + mt * 128);
                bulk_commit();
                if (!own_k) bulk_wait_read<0>();
              }
              if (!own_k) softmax_sync256();
            }
            if (st == 0) bulk_wait_read<0>();
          }
        } else {
          // o = O / (l + e^{z - m}), rope dims rotated back by -t
          __nv_bfloat16* O = p.out + (int64_t)it.node * kAttnH * kAttnD;
          if (tid < 32) {
            const int h = h0 + tid;
            const float z2 = p.sinks[h] * kLog2e;
            const float mu = empty ? -INFINITY : m_use[h];
            const float M = fmaxf(mu, z2);
            const float den = exp2f(z2 - M) + (mu == -INFINITY ? 0.f : l_run[h] * exp2f(mu - M));
            // no key, or all weight on an infinite sink: o = 0
            stat_a[h] = (mu == -INFINITY || z2 == INFINITY) ? 0.f : exp2f(mu - M) / den;
          }
          group_sync(gid);
          __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(sP) + g * 32 * 128;   // [32 heads][128 dims]
          const float4* fac4 = reinterpret_cast<const float4*>(stat_a + h0);
#pragma unroll 1
          for (int mt = 0; mt < kAttnMT; ++mt) {
            const int dim = mt * 128 + tid;
            const bool mt_rope = mt * 128 + 127 >= r0;
            const bool rot = dim >= r0;
            float cs = 1.f, sn = 0.f;
            if (rot) rope_sincos(-(double)it.t, theta_s[(dim - r0) >> 1], &cs, &sn);
            float o[32];
            if (!empty) {
              tmem_ld32(tO + lane_base + mt * kAttnH + h0, o);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0.f;
            }
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
              const float4 fc = fac4[e4];
              o[e4 * 4 + 0] *= fc.x; o[e4 * 4 + 1] *= fc.y; o[e4 * 4 + 2] *= fc.z; o[e4 * 4 + 3] *= fc.w;
            }
            if (mt_rope) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float partner = __shfl_xor_sync(0xffffffffu, o[e], 1);
                if (rot) o[e] = (dim & 1) ? fmaf(partner, sn, o[e] * cs) : fmaf(-partner, sn, o[e] * cs);
              }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) stage[e * 128 + tid] = __float2bfloat16_rn(o[e]);
            group_sync(gid);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int pc = tid + 128 * i;                // 16-byte piece: head pc / 16
              const int h = pc >> 4, off = (pc & 15) * 8;
              const uint4 val = *reinterpret_cast<const uint4*>(stage + h * 128 + off);
              *reinterpret_cast<uint4*>(O + (int64_t)(h0 + h) * kAttnD + mt * 128 + off) = val;
            }
            group_sync(gid);
          }
        }
      }
      tc_fence_before();
      if (softmax_any256(bad)) break;        // also: both groups are done with the item
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpS) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Join of a node's splits with the sink, and the output de-rotation:
// o = sum_s f_s (O_s / l_s), f_s = l_s 2^(m_s - M) / (2^(z - M) + sum_s l_s 2^(m_s - M)).
// One CTA per (node, 64 dims).  The partials are in L2; each thread reads its
// dim pair's 8 heads of four splits at a time, so the kernel is two or three
// L2 round trips.
constexpr int kTreeCombineThreads = 256;
constexpr int kTreeMaxSplits = 148;

struct TreeCombineParams {
  const char* partial; const float* sinks; const int* node_pos;
  __nv_bfloat16* out;
  int splits, rope_dims;
  double theta[64];
};

__global__ void __launch_bounds__(kTreeCombineThreads) tree_combine_kernel(const __grid_constant__ TreeCombineParams p) {
  __shared__ float w_s[kTreeMaxSplits][kAttnH];
  __shared__ __align__(16) __nv_bfloat16 stage[kAttnH][64 + 8];
  __shared__ float red[4][kAttnH];
  griddep_wait();
  griddep_launch_dependents();
  const int node = blockIdx.x, d0 = blockIdx.y * 64;
  const int t = p.node_pos[node];
  if (t < 0) return;
  const int tid = threadIdx.x;
  const char* P = p.partial + (int64_t)node * p.splits * kTcPartialBytes;
  // weights: thread (head h, part) takes the splits part, part + 4, ...
  {
    const int h = tid & 63, part = tid >> 6;
    const float z2 = p.sinks[h] * kLog2e;
    float mx = -INFINITY;
    for (int s = part; s < p.splits; s += 4) {
      const float m = *reinterpret_cast<const float*>(P + (int64_t)s * kTcPartialBytes + h * 4);
      w_s[s][h] = m;
      mx = fmaxf(mx, m);
    }
    red[part][h] = mx;
    __syncthreads();
    const float mk = fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h]));
    const float M = fmaxf(mk, z2);
    float den = 0.f;
    for (int s = part; s < p.splits; s += 4) {
      const float m = w_s[s][h];
      const float f = m == -INFINITY ? 0.f
                      : *reinterpret_cast<const float*>(P + (int64_t)s * kTcPartialBytes + (kAttnH + h) * 4) * exp2f(m - M);
      w_s[s][h] = f;
      den += f;
    }
    __syncthreads();
    red[part][h] = den;
    __syncthreads();
    den = red[0][h] + red[1][h] + red[2][h] + red[3][h] + exp2f(z2 - M);
    // no key, or all weight on an infinite sink: o = 0
    const float inv = (mk == -INFINITY || z2 == INFINITY) ? 0.f : 1.f / den;
    for (int s = part; s < p.splits; s += 4) {
      const float f = w_s[s][h];
      w_s[s][h] = f > 0.f ? f * inv : 0.f;
    }
  }
  __syncthreads();
  const int dp = tid >> 3, hg = tid & 7;                 // dims d0 + 2 dp, + 1; heads 8 hg ..
  const char* src = P + kTcPartialHeader + ((int64_t)(d0 + 2 * dp) * kAttnH + 8 * hg) * 2;
  float a0[8], a1[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) { a0[e] = 0.f; a1[e] = 0.f; }
  for (int s0 = 0; s0 < p.splits; s0 += 4) {
    uint4 x[4], y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (s0 + u < p.splits) {
        x[u] = *reinterpret_cast<const uint4*>(src + (int64_t)(s0 + u) * kTcPartialBytes);
        y[u] = *reinterpret_cast<const uint4*>(src + (int64_t)(s0 + u) * kTcPartialBytes + kAttnH * 2);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (s0 + u < p.splits) {
        float f0[8], f1[8];
        unpack16<__nv_bfloat16>(x[u], f0);
        unpack16<__nv_bfloat16>(y[u], f1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = w_s[s0 + u][8 * hg + e];
          // (a split of weight 0 may hold no O: its bytes are not used)
          a0[e] += w != 0.f ? w * f0[e] : 0.f;
          a1[e] += w != 0.f ? w * f1[e] : 0.f;
        }
      }
    }
  }
  const int j0 = d0 + 2 * dp - (kAttnD - p.rope_dims);
  if (j0 >= 0) {
    float cs, sn;
    rope_sincos(-(double)t, p.theta[j0 >> 1], &cs, &sn);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x0 = a0[e], x1 = a1[e];
      a0[e] = x0 * cs - x1 * sn;
      a1[e] = x0 * sn + x1 * cs;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    *reinterpret_cast<__nv_bfloat162*>(&stage[8 * hg + e][2 * dp]) = __floats2bfloat162_rn(a0[e], a1[e]);
  __syncthreads();
  __nv_bfloat16* O = p.out + (int64_t)node * kAttnH * kAttnD + d0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = tid + 256 * i, h = x >> 3, pc = (x & 7) * 8;
    *reinterpret_cast<uint4*>(O + (int64_t)h * kAttnD + pc) = *reinterpret_cast<const uint4*>(&stage[h][pc]);
  }
}

}  // namespace csahca
