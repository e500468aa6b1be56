// Attention of draft-tree nodes on the tensor cores (64 heads of 512 dims,
// bf16; "Paper Breakdown: DeepSeek-V4", section 4: MQA core attention,
// sliding window, HCA, attention sink; one query per drafted token).
//
// Both products are written transposed, as in the decode kernel, so that one
// copy of a key tile serves both (K = V) and O^T [512 x 64] fits TMEM beside
// S^T:  S^T [64 keys x 64 heads] = K . Q^T,  O^T += V^T . P^T.
//
// The tensor pipe reads its operands from shared memory at 128 bytes a cycle,
// and at N = 64 that is what an MMA costs: 48 cycles for M = 128, 32 for M = 64
// (measured; 32 and 16 by arithmetic).  Two key tiles are in flight, so that
// the scores of tile i + 1 are formed and its successor loads while tile i is
// in the softmax: tiles of 64 keys (64 KB), since 128 KB of keys fit beside
// the query.  M = 64 for S^T costs 1,033 + 776 cycles of operand reads a tile
// (3,620 per 128 keys, against 3,090 with tiles of 128 keys), but one tile of
// 128 at a time left the pipe idle for the softmax and the load: 7,250 cycles
// per 128 keys.  With all SMs at work a tile takes some 3,000 cycles: 64 KB a
// tile and node is 5.9 TB/s out of L2, near the 7.3 to 7.7 TB/s that a bare
// stream of boxes reaches, so the tiles' way out of L2 bounds HCA calls of many
// nodes (64 nodes over 8,192 entries: 106 us for 0.56 GB, start and end included;
// dealing the tiles out evenly over all SMs instead of two items a node changed
// nothing).  A CTA
// cannot keep two nodes: O^T of one is half of TMEM.
//
// A node's keys are two runs.  Tiles of 64 consecutive committed entries
// (HCA) arrive by TMA, four 64-dim chunks a box (an SM completes about one TMA
// op per 580 cycles whatever its size, so 32 KB boxes).  Everything else is
// the node's row list, gathered row by row: the selected entries (CSA) or the
// entries past the last whole tile (HCA), then the plan's list (window rows by
// position out of the ring or the path, and the path's drafted entries).  Rows
// of the list that are no key, and the rows that fill its last MMA step, are
// written as zeros: nothing that a mask hides is read, so NaN there cannot
// reach O.
//
// Roles (896 threads): warps 0-7 softmax and epilogue (two groups of four
// warps, group g owns heads 32g .. 32g + 31; S^T is read in the 16 x 256-bit
// shape, a thread holding two keys of eight heads, with its heads' running
// maxima and sums in registers), warps 8-23 producers, then the S and the P.V
// MMA issuers.  Each producer warp copies 4 rows of a gathered tile, waits
// for its own copies of a half tile and arrives once (a barrier arrival per
// lane and chunk was 4,096 of them per 128 keys).
//
// Roundings to bf16: the finished query (once, by the plan's kernel), the
// weights p, and the output; sums, statistics and split partials are fp32.  The
// decode kernel rounds the same way, so a verified token sees what a decoded one
// does: 2.6e-3 of the result's norm in all, against 1.7e-3 for the output's
// rounding alone.  Weights as the sum of two bf16 (a second P.V) gave 2.3e-3 and
// took 22 to 26 % longer on HCA calls of many nodes.
//
// Work items: (node, split of its tiles).  With one split the item writes the
// final row, otherwise a partial for tree_combine_kernel.
#pragma once
#include "attention_tc.cuh"
#include "norm_rope.cuh"

namespace csahca {

constexpr int kTreeProducers = 16;
constexpr int kTreeThreads = 32 * (8 + kTreeProducers + 4);
constexpr int kTreeTile = 64;                            // keys of a tile
constexpr int kTreeHalfChunks = kAttnChunks / 2;         // a half tile: 4 chunks of 64 dims
static_assert(kTreeProducers * 4 == kTreeTile, "a producer lane group copies one row of a gathered tile");
struct TreeSmem {
  static constexpr int K_CHUNK = kTreeTile * 128;              // 8 KB
  static constexpr int K_BYTES = kAttnChunks * K_CHUNK;        // 64 KB a tile
  static constexpr int P_BYTES = kTreeTile * 128;              // 8 KB
  static constexpr int TOTAL = 1024 + AttnSmem::Q_BYTES + 2 * K_BYTES + 2 * P_BYTES;
};
static_assert(256 * kAttnRegsSoftmax + 32 * kTreeProducers * kAttnRegsProducer + 128 * kAttnRegsMma <= 72 * kTreeThreads,
              "the register split fits a 72-register launch");

// Partial of one (node, split), fp32: m[H], l[H] (l = -1: a split without keys,
// which has no more than this header), then O / l as [2 head groups][D]
// rows of 32 heads, 128 bytes each, whose 16-byte piece j holds heads
// 4 (j ^ (dim & 7)) .. + 3: as the threads write them into shared memory without
// conflicts, so that a bulk copy takes 16 KB of it at once (stored from the
// registers, 16 bytes a lane and 256 bytes apart, a partial took 10,600 cycles).
constexpr int kTreePartialFloats = 2 * kAttnH + kAttnD * kAttnH;
constexpr int kTreePartialBytes = kTreePartialFloats * 4;
__host__ __device__ __forceinline__ int tree_partial_at(int dim, int head) {   // head % 4 == 0
  return 2 * kAttnH + ((head >> 5) * kAttnD + dim) * 32 + ((((head & 31) >> 2) ^ (dim & 7)) << 2);
}

struct TreeAttnParams {
  const uint8_t* kv;                     // cache rows [B * N]
  const uint8_t* rows[3];                // ROW_RING, ROW_TREE (bf16 rows), ROW_DRAFT (as the cache's) bases
  int row_bytes;                         // of a cache row: 2 D, or an FP8 KV row's
  int nope_chunks;                       // FP8 KV rows: 64-dim chunks of codes, (D - rope_dims) / 64
  const int* idx;                        // CSA: [nodes, k]; null: HCA
  const int* list; const int4* info;
  const float2* turn;                    // [nodes][rope_dims / 2] cos, sin of the node's angles
  const float* sinks;
  int list_stride;                       // w + T
  int k, N, T;
  int idx_given;                         // idx is the caller's, not an earlier kernel's
  int n_items, splits;
  float scale_log2;
  int rope_dims;
  __nv_bfloat16* out;                    // [nodes, H, D]
  char* partial;                         // [nodes][splits] blocks of kTreePartialBytes
};

struct TreeItem { int node, split, t, full, tail, nlist, tile0, tile1; };

__device__ __forceinline__ int4 tree_info(const TreeAttnParams& p, int id) {
  return id < p.n_items ? __ldg(p.info + id / p.splits) : make_int4(-1, 0, 0, 0);
}
// First tile of a split: the first total % splits of them take one more.
__device__ __forceinline__ int tree_tile0(int total, int split, int splits) {
  const int q = total / splits;
  return q * split + min(split, total - q * splits);
}
template <bool kF8>
__device__ __forceinline__ TreeItem tree_item(const TreeAttnParams& p, int id, const int4& f) {
  TreeItem it;
  it.node = id / p.splits;
  it.split = id - it.node * p.splits;
  it.t = f.x;
  it.full = kF8 || p.idx ? 0 : f.y / kTreeTile;        // (FP8 rows are widened on their way: all gathered)
  it.tail = p.idx ? p.k : f.y - it.full * kTreeTile;
  it.nlist = it.tail + f.z;
  const int total = f.x < 0 ? 0 : it.full + (it.nlist + kTreeTile - 1) / kTreeTile;
  it.tile0 = tree_tile0(total, it.split, p.splits);
  it.tile1 = tree_tile0(total, it.split + 1, p.splits);
  return it;
}
// Entry j of the node's list as it stands in memory (the selection's index or
// the plan's code; asked for a tile ahead), and the row it names, or null if
// it is no key.
__device__ __forceinline__ int tree_entry(const TreeAttnParams& p, const TreeItem& it, int j) {
  if (j >= it.nlist) return -1;
  if (j >= it.tail) return __ldg(p.list + (int64_t)it.node * p.list_stride + (j - it.tail));
  return p.idx ? __ldg(p.idx + (int64_t)it.node * p.k + j) : it.full * kTreeTile + j;
}
// (*cached: a row of the cache's or the drafted entries' kind)
__device__ __forceinline__ const uint8_t* tree_row(const TreeAttnParams& p, const TreeItem& it, int j, int e, bool* cached) {
  *cached = true;
  if (e < 0) return nullptr;
  if (j >= it.tail) {
    const int kind = e >> kRowShift;
    const int64_t r = e & kRowMask;
    *cached = kind == ROW_DRAFT;
    return kind == ROW_RING ? p.rows[0] + r * (2 * kAttnD) : kind == ROW_TREE ? p.rows[1] + r * (2 * kAttnD)
                                                                              : p.rows[2] + r * p.row_bytes;
  }
  const int b = it.node / p.T;
  if (e < p.N) return p.kv + ((int64_t)b * p.N + e) * p.row_bytes;
  if (e - p.N < p.T && p.rows[ROW_DRAFT]) return p.rows[ROW_DRAFT] + ((int64_t)b * p.T + (e - p.N)) * p.row_bytes;
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
// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// MMA and commit issued by the elected lane, in code that the whole warp runs:
// the descriptors stay warp-uniform values (issued from a lane-0 branch, the
// scalar work around an MMA took 80 to 118 cycles of the pipe's 49).
__device__ __forceinline__ void umma_bf16_if(uint32_t leader, uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                             uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}"
      ::"r"(d_tmem), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader));
}
__device__ __forceinline__ void umma_commit_if(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(leader) : "memory");
}
// A converged warp's wait: every lane leaves with the same answer.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort)) != 0;
}
// 16 lanes x 32 columns of 32 bits: thread t gets lanes t / 4 and t / 4 + 8 of
// columns 8 j + 2 (t % 4) + {0, 1}: v[4 j + {0, 1}] and v[4 j + {2, 3}].
__device__ __forceinline__ void tmem_ld16x256_x4(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// Every committed bulk group of this thread has completed, its writes made.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Contiguous shared -> global copy (bulk-group completion).
__device__ __forceinline__ void bulk_store(void* dst_gmem, const void* src_smem, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst_gmem), "r"(smem_u32(src_smem)),
               "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// 8 e4m3 codes times the block scale as 8 bf16.
__device__ __forceinline__ uint4 f8x8_to_bf16(uint2 codes, float scale) {
  const uint32_t c[2] = {codes.x, codes.y};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((c[i >> 1] >> (16 * (i & 1))) & 0xffffu), __NV_E4M3)));
    w[i] = pack_bf16x2(f.x * scale, f.y * scale);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// FP8 KV rows of a sequence's committed entries and of its drafted ones, as the
// bf16 rows they stand for: HCA calls of several nodes a sequence read every
// entry once a node, so that widening them once and running the bf16 kernel
// costs less than widening in every gather.  64 threads a row, 8 dims each;
// bound by HBM.
struct KvWidenParams {
  const uint8_t* kv; const uint8_t* draft; const int* pos;
  __nv_bfloat16* kv_out; __nv_bfloat16* draft_out;     // [B, N, D], [B, T, D]
  int B, N, T, m, row_bytes, rope_dims;
};
__global__ void __launch_bounds__(256) kv_widen_kernel(const __grid_constant__ KvWidenParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x, v = p.pos[b] < 0 ? 0 : min(p.N, p.pos[b] / p.m);
  const int rows = v + (p.draft ? p.T : 0), piece = threadIdx.x & 63, chunk = piece >> 3;
  const int nope = (kAttnD - p.rope_dims) / 64;
  for (int r = blockIdx.y * 4 + (threadIdx.x >> 6); r < rows; r += gridDim.y * 4) {
    const uint8_t* src = r < v ? p.kv + ((int64_t)b * p.N + r) * p.row_bytes
                               : p.draft + ((int64_t)b * p.T + (r - v)) * p.row_bytes;
    uint4 w;
    if (chunk < nope)
      w = f8x8_to_bf16(__ldg(reinterpret_cast<const uint2*>(src + piece * 8)),
                       __ldg(reinterpret_cast<const float*>(src + kAttnD + p.rope_dims + 4 * chunk)));
    else
      w = __ldg(reinterpret_cast<const uint4*>(src + nope * 64 + (piece - 8 * nope) * 16));
    __nv_bfloat16* dst = r < v ? p.kv_out + ((int64_t)b * p.N + r) * kAttnD
                               : p.draft_out + ((int64_t)b * p.T + (r - v)) * kAttnD;
    *reinterpret_cast<uint4*>(dst + piece * 8) = w;
  }
}

// kF8: the cache and the drafted entries are FP8 KV rows.  Every tile is
// gathered, and the producers widen the codes to bf16 between the load and the
// shared-memory row (through registers, half a tile at a time), as a row stands
// for decode(code) * scale; ring and tree rows are bf16 and are copied.
template <bool kF8>
__global__ void __launch_bounds__(kTreeThreads, 1)
attn_tree_tc_kernel(const __grid_constant__ CUtensorMap comp_rows, const __grid_constant__ CUtensorMap q_rows,
                    const __grid_constant__ TreeAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sK = sQ + AttnSmem::Q_BYTES;                  // two tiles
  uint8_t* sP = sK + 2 * TreeSmem::K_BYTES;              // two
  // Tile n uses buffer n & 1 of keys, S^T and P^T, phase (n >> 1) & 1.
  // bar_pv[b][h]: the P.V MMAs of the half's two O^T M-tiles have completed (its
  // four key chunks are free; h = 1: P^T too, and O^T may be touched)
  __shared__ uint64_t bar_kfull[2][2], bar_pv[2][2], bar_s_full[2], bar_s_free[2], bar_p_full[2];
  __shared__ uint64_t bar_q_full, bar_q_empty, bar_done;
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  __shared__ __align__(16) float red[2][4][32];
  __shared__ __align__(16) float stat_a[kAttnH];
  __shared__ float m_run[kAttnH], l_run[kAttnH];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarpS = 8 + kTreeProducers, kWarpPV = kWarpS + 1;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int x = 0; x < 2; ++x) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&bar_kfull[x][h], kTreeProducers);
        mbar_init(&bar_pv[x][h], 1);
      }
      mbar_init(&bar_s_full[x], 1);
      mbar_init(&bar_s_free[x], 256);
      mbar_init(&bar_p_full[x], 256);
    }
    mbar_init(&bar_q_full, 1);
    mbar_init(&bar_q_empty, 1);
    mbar_init(&bar_done, 2);
    mbar_fence_init();
  }
  if (warp == kWarpS) tmem_alloc(&tmem_base_sh, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const uint32_t tS = tmem;                              // S^T of buffer b: columns [64 b, ...), M = 64: keys 16 q ..
                                                         // 16 q + 15 in lanes 32 q .. 32 q + 15
  const uint32_t tO = tmem + 128;                        // O^T M-tile j: columns [128 + j H, ...)
  // the plan, the finished rows and the selection come from earlier kernels; a
  // selection that the caller gave is an input, and the rows that it names for
  // the first tile (as it would be for a whole window) go to L2 meanwhile
  if (p.idx_given && warp >= 8 && warp < kWarpS) {
    const int node = blockIdx.x / p.splits;
    const int tiles = (p.k + p.list_stride - p.T + kTreeTile - 1) / kTreeTile;
    const int j = tree_tile0(tiles, blockIdx.x - node * p.splits, p.splits) * kTreeTile + 4 * (warp - 8) + (lane >> 3);
    const int e = j < p.k ? __ldg(p.idx + (int64_t)node * p.k + j) : -1;
    if (e >= 0 && e < p.N)
      prefetch_l2_line(p.kv + ((int64_t)(node / p.T) * p.N + e) * p.row_bytes + min((lane & 7) * 128, p.row_bytes - 16));
  }
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
    const int piece = lane & 7, row = 4 * pw + (lane >> 3);   // this lane's row of a gathered tile
    uint32_t tcount = 0, icount = 0;
    bool stop = false;                                   // warp-uniform
    int4 f = tree_info(p, blockIdx.x);
    for (int id = blockIdx.x; id < p.n_items && !stop; id += gridDim.x) {
      const TreeItem it = tree_item<kF8>(p, id, f);
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
      // the entry of this lane's row in the next gathered tile
      int e = tree_entry(p, it, (max(it.tile0, it.full) - it.full) * kTreeTile + row);
      for (int tile = it.tile0; tile < it.tile1 && !stop; ++tile, ++tcount) {
        const int buf = tcount & 1;
        const uint32_t ph = (tcount >> 1) & 1;
        uint8_t* dst = sK + buf * TreeSmem::K_BYTES;
        const bool box = tile < it.full;
        const int off = (tile - it.full) * kTreeTile;
        const int fill = box ? 0 : (it.nlist - off + 15) & ~15;   // rows that the P.V MMAs read
        const uint8_t* src = nullptr;
        bool cached = true;
        if (!box) {
          src = tree_row(p, it, off + row, e, &cached);
          e = tree_entry(p, it, off + kTreeTile + row);
        }
        const bool live = src != nullptr;
        if constexpr (kF8) {
          const bool codes = cached;
          for (int h = 0; h < 2; ++h) {
            // this lane's 8 dims of the half's four chunks, asked for before the buffer is free
            uint4 raw[kTreeHalfChunks];
            float scale[kTreeHalfChunks];
#pragma unroll
            for (int c = 0; c < kTreeHalfChunks; ++c) {
              const int cc = h * kTreeHalfChunks + c;
              raw[c] = make_uint4(0u, 0u, 0u, 0u);
              scale[c] = 0.f;
              if (live) {
                if (codes && cc < p.nope_chunks) {
                  const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + cc * 64 + piece * 8));
                  raw[c].x = v.x;
                  raw[c].y = v.y;
                  scale[c] = __ldg(reinterpret_cast<const float*>(src + kAttnD + p.rope_dims + 4 * cc));
                } else {
                  const int o = codes ? p.nope_chunks * 64 + (cc - p.nope_chunks) * 128 : cc * 128;
                  raw[c] = __ldg(reinterpret_cast<const uint4*>(src + o + piece * 16));
                }
              }
            }
            int ok = 1;
            if (lane == 0) ok = mbar_wait(&bar_pv[buf][h], ph ^ 1, &abort_flag);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) { stop = true; break; }
            if (row < fill) {
#pragma unroll
              for (int c = 0; c < kTreeHalfChunks; ++c) {
                const int cc = h * kTreeHalfChunks + c;
                const uint4 w = live && codes && cc < p.nope_chunks
                                    ? f8x8_to_bf16(make_uint2(raw[c].x, raw[c].y), scale[c]) : raw[c];
                *reinterpret_cast<uint4*>(dst + cc * TreeSmem::K_CHUNK + sw128_offset(row, piece * 16)) = w;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_kfull[buf][h]);
          }
          if (!stop && tile + 1 < it.tile1) {
            bool nc;
            const uint8_t* nx = tree_row(p, it, off + kTreeTile + row, e, &nc);
            if (nx && piece * 128 < (nc ? p.row_bytes : 2 * kAttnD)) prefetch_l2_line(nx + piece * 128);
          }
          continue;
        }
        if (!live) src = p.kv;
        for (int h = 0; h < 2; ++h) {
          int ok = 1;
          if (lane == 0) {
            ok = mbar_wait(&bar_pv[buf][h], ph ^ 1, &abort_flag);
            if (ok && box) {
              // 64 consecutive entries: half h (four chunks) by producer warp h
              if (h == pw) {
                mbar_expect_tx(&bar_kfull[buf][h], kTreeHalfChunks * TreeSmem::K_CHUNK);
                tma_load_3d(dst + h * kTreeHalfChunks * TreeSmem::K_CHUNK, &comp_rows, 0,
                            (it.node / p.T) * p.N + tile * kTreeTile, h * kTreeHalfChunks, &bar_kfull[buf][h]);
              } else {
                mbar_arrive(&bar_kfull[buf][h]);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) { stop = true; break; }
          if (!box) {
            if (row < fill) {
#pragma unroll
              for (int c = 0; c < kTreeHalfChunks; ++c) {
                const int cc = h * kTreeHalfChunks + c;
                cp_async16_or_zero(dst + cc * TreeSmem::K_CHUNK + sw128_offset(row, piece * 16),
                                   src + cc * 128 + piece * 16, live);
              }
            }
            cp_async_commit();
          }
        }
        if (box || stop) continue;
        // every lane's own copies of a half have landed and are made visible
        // to the MMAs (async proxy) before the warp's one arrival
        cp_async_wait<1>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_kfull[buf][0]);
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_kfull[buf][1]);
        if (tile + 1 < it.tile1) {
          // the next tile's lines into L2, while its buffer is still in use
          const uint8_t* nx = tree_row(p, it, off + kTreeTile + row, e, &cached);
          if (nx) prefetch_l2_line(nx + piece * 128);
        }
      }
    }
    // copies in flight end before the CTA may exit: this lane's gathers here,
    // the boxes and the query by their barriers
    cp_async_wait<0>();
    if (lane == 0 && pw < 2) {
      for (uint32_t n = tcount < 2 ? 0 : tcount - 2; n < tcount; ++n)
        mbar_wait(&bar_kfull[n & 1][pw], (n >> 1) & 1, &abort_flag);
    }
    if (lane == 0 && pw == 0 && icount > 0) mbar_wait(&bar_q_full, (icount - 1) & 1, &abort_flag);
  } else if (warp >= kWarpS) {
    setmaxnreg_dec<kAttnRegsMma>();
    if (warp == kWarpS) {
      // ---------------------------------------------------------- S issuer
      const uint32_t leader = elect_one();
      constexpr uint32_t idesc_s = umma_idesc_bf16(kTreeTile, kAttnH, 0, 0);
      // (descriptors by halves: only the low word, the address, changes)
      const uint64_t kdesc = umma_desc_kmajor(smem_u32(sK)), qdesc = umma_desc_kmajor(smem_u32(sQ));
      const uint32_t k_lo = (uint32_t)kdesc, k_hi = (uint32_t)(kdesc >> 32);
      const uint32_t q_lo = (uint32_t)qdesc, q_hi = (uint32_t)(qdesc >> 32);
      uint32_t tcount = 0, icount = 0;
      bool stop = false;
      int4 f = tree_info(p, blockIdx.x);
      for (int id = blockIdx.x; id < p.n_items && !stop; id += gridDim.x) {
        const TreeItem it = tree_item<kF8>(p, id, f);
        f = tree_info(p, id + gridDim.x);
        if (it.tile1 <= it.tile0) continue;
        if (!mbar_wait_warp(&bar_q_full, icount & 1, &abort_flag)) break;
        ++icount;
        for (int tile = it.tile0; tile < it.tile1 && !stop; ++tile, ++tcount) {
          const int buf = tcount & 1;
          const uint32_t ph = (tcount >> 1) & 1;
          if (!mbar_wait_warp(&bar_s_free[buf], ph ^ 1, &abort_flag)) { stop = true; break; }
          const uint32_t kb = k_lo + buf * (TreeSmem::K_BYTES >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!mbar_wait_warp(&bar_kfull[buf][h], ph, &abort_flag)) { stop = true; break; }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kTreeHalfChunks; ++c) {
              const int cc = h * kTreeHalfChunks + c;
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                umma_bf16_if(leader, tS + buf * kAttnH, kb + cc * (TreeSmem::K_CHUNK >> 4) + 2 * ks, k_hi,
                             q_lo + cc * (AttnSmem::Q_CHUNK >> 4) + 2 * ks, q_hi, idesc_s, (cc | ks) != 0);
            }
          }
          if (stop) break;
          umma_commit_if(leader, &bar_s_full[buf]);
          if (tile == it.tile1 - 1) umma_commit_if(leader, &bar_q_empty);
        }
      }
      umma_commit_if(leader, &bar_done);
      mbar_wait_warp(&bar_done, 0, &abort_flag);
    } else if (warp == kWarpPV) {
      // -------------------------------------------------------- P.V issuer
      const uint32_t leader = elect_one();
      constexpr uint32_t idesc_pv = umma_idesc_bf16(128, kAttnH, 1, 1);
      const uint64_t vdesc = umma_desc_mnmajor(smem_u32(sK), TreeSmem::K_CHUNK);
      const uint64_t pdesc = umma_desc_mnmajor(smem_u32(sP), TreeSmem::P_BYTES);
      const uint32_t v_lo = (uint32_t)vdesc, v_hi = (uint32_t)(vdesc >> 32);
      const uint32_t p_lo = (uint32_t)pdesc, p_hi = (uint32_t)(pdesc >> 32);
      uint32_t tcount = 0;
      bool stop = false;
      int4 f = tree_info(p, blockIdx.x);
      for (int id = blockIdx.x; id < p.n_items && !stop; id += gridDim.x) {
        const TreeItem it = tree_item<kF8>(p, id, f);
        f = tree_info(p, id + gridDim.x);
        for (int tile = it.tile0; tile < it.tile1; ++tile, ++tcount) {
          const int buf = tcount & 1;
          if (!mbar_wait_warp(&bar_p_full[buf], (tcount >> 1) & 1, &abort_flag)) { stop = true; break; }
          tc_fence_after();
          const uint32_t first = tile == it.tile0;
          // a list's last tile: P is 0 past its last row, the steps there are skipped
          const int hi = tile < it.full ? kTreeTile : it.nlist - (tile - it.full) * kTreeTile;
          const int nks = min(kTreeTile / 16, (hi + 15) >> 4);
          const uint32_t vb = v_lo + buf * (TreeSmem::K_BYTES >> 4), pb = p_lo + buf * (TreeSmem::P_BYTES >> 4);
#pragma unroll
          for (int mt = 0; mt < kAttnMT; ++mt) {
#pragma unroll
            for (int ks = 0; ks < kTreeTile / 16; ++ks)
              if (ks < nks)
                umma_bf16_if(leader, tO + mt * kAttnH, vb + (2 * mt) * (TreeSmem::K_CHUNK >> 4) + 128 * ks, v_hi,
                             pb + 128 * ks, p_hi, idesc_pv, ks > 0 || !first);
            if (mt & 1) umma_commit_if(leader, &bar_pv[buf][mt >> 1]);
          }
        }
      }
      umma_commit_if(leader, &bar_done);
      mbar_wait_warp(&bar_done, 0, &abort_flag);
    }
  } else {
    setmaxnreg_inc<kAttnRegsSoftmax>();
    // --------------------------------------------------- softmax / epilogue
    const int g = warp >> 2, gid = 1 + g;
    const int tid = threadIdx.x & 127;
    const int h0 = 32 * g;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t tcount = 0;
    const int r0 = kAttnD - p.rope_dims;
    const int wq = warp & 3;
    const int key0 = 16 * wq + (lane >> 2);              // this thread's keys: key0, key0 + 8
    const int hl = 2 * (lane & 3);                       // its heads: h0 + 8 j + hl + {0, 1}, j = 0 .. 3
    const float z2 = p.sinks[h0 + lane] * kLog2e;        // (of head h0 + lane)
    int4 f = tree_info(p, blockIdx.x);
    for (int id = blockIdx.x; id < p.n_items; id += gridDim.x) {
      const TreeItem it = tree_item<kF8>(p, id, f);
      f = tree_info(p, id + gridDim.x);
      const bool empty = it.tile1 <= it.tile0;
      bool bad = false;                      // uniform over the group; both groups leave together
      // this thread's dim of the last M-tile turns back by this angle (rope_dims <= 128)
      float2 turn = make_float2(1.f, 0.f);
      const bool rot = 3 * 128 + tid >= r0;
      if (rot && it.t >= 0 && p.splits == 1)
        turn = __ldg(p.turn + (int64_t)it.node * (p.rope_dims >> 1) + ((3 * 128 + tid - r0) >> 1));
      float m[8], l[8];                      // [2 j + {0, 1}]: running max (log2 units) and this thread's share of the sum
#pragma unroll
      for (int x = 0; x < 8; ++x) { m[x] = -INFINITY; l[x] = 0.f; }
      for (int tile = it.tile0; tile < it.tile1; ++tile, ++tcount) {
        if (bad) continue;
        const int buf = tcount & 1;
        const uint32_t ph = (tcount >> 1) & 1;
        bool v0 = true, v1 = true;
        if (tile >= it.full) {
          v0 = tree_key_valid(p, it, (tile - it.full) * kTreeTile + key0);
          v1 = tree_key_valid(p, it, (tile - it.full) * kTreeTile + key0 + 8);
        }
        // (a wait that gives up is settled with the vote below: until then its
        // threads work on what the buffers hold)
        const bool ok = mbar_wait(&bar_s_full[buf], ph, &abort_flag);
        tc_fence_after();
        float v[16];
        tmem_ld16x256_x4(tS + buf * kAttnH + lane_base + h0, v);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(&bar_s_free[buf]);
        // scaled to log2 units; v[4 j + x]: key 0 for x < 2, key 1 else
        bool exceed = !ok;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float sc = (x < 2 ? v0 : v1) ? v[4 * j + x] * p.scale_log2 : -INFINITY;
            v[4 * j + x] = sc;
            exceed |= sc > m[2 * j + (x & 1)] + kRescaleThreshold;
          }
        // the running max is raised only where a score exceeds it by more than
        // 2^8 (or is the item's first)
        if (group_any(gid, exceed)) {
          if (!group_all(gid, ok)) { bad = true; continue; }
          float t[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int j = x >> 1, e = x & 1;
            t[x] = fmaxf(v[4 * j + e], v[4 * j + 2 + e]);
            t[x] = fmaxf(t[x], __shfl_xor_sync(0xffffffffu, t[x], 4));
            t[x] = fmaxf(t[x], __shfl_xor_sync(0xffffffffu, t[x], 8));
            t[x] = fmaxf(t[x], __shfl_xor_sync(0xffffffffu, t[x], 16));
          }
          if (lane < 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<float2*>(&red[g][wq][8 * j + hl]) = make_float2(t[2 * j], t[2 * j + 1]);
          }
          group_sync(gid);
          bool rescale = false;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 mt = *reinterpret_cast<const float2*>(&red[g][0][8 * j + hl]);
#pragma unroll
            for (int w = 1; w < 4; ++w) {
              const float2 o = *reinterpret_cast<const float2*>(&red[g][w][8 * j + hl]);
              mt.x = fmaxf(mt.x, o.x);
              mt.y = fmaxf(mt.y, o.y);
            }
            float al[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float tm = e ? mt.y : mt.x, mo = m[2 * j + e];
              al[e] = 1.f;
              if (tm > mo + kRescaleThreshold) {          // (true of any score while mo = -inf)
                al[e] = mo == -INFINITY ? 0.f : exp2f(mo - tm);
                m[2 * j + e] = tm;
                rescale |= mo != -INFINITY;
              }
              l[2 * j + e] *= al[e];
            }
            if (wq == 0 && lane < 4) *reinterpret_cast<float2*>(&stat_a[h0 + 8 * j + hl]) = make_float2(al[0], al[1]);
          }
          // O^T is rescaled where a head had keys already, once the P.V of the
          // tile before has completed (the barrier also publishes stat_a)
          if (group_any(gid, rescale)) {
            const uint32_t n = tcount - 1;               // (a head with keys: not the item's first tile)
            if (!mbar_wait_group(gid, &bar_pv[n & 1][1], (n >> 1) & 1, &abort_flag)) { bad = true; continue; }
            tc_fence_after();
            const float4* al4 = reinterpret_cast<const float4*>(stat_a + h0);
#pragma unroll 1
            for (int mt = 0; mt < kAttnMT; ++mt) {
              float o[32];
              const uint32_t a = tO + mt * kAttnH + lane_base + h0;
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
            tc_fence_before();
          }
        }
        // (the P^T buffer is free: these scores' keys were loaded once the P.V of
        // the tile before the last had completed)
        // p = 2^(s - m), 0 for a key slot that is no key (m = -inf: no key yet)
        uint8_t* P = sP + buf * TreeSmem::P_BYTES;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float ma = m[2 * j] == -INFINITY ? 0.f : m[2 * j], mb = m[2 * j + 1] == -INFINITY ? 0.f : m[2 * j + 1];
          const float p0 = fast_exp2(v[4 * j] - ma), p1 = fast_exp2(v[4 * j + 1] - mb);
          const float p2 = fast_exp2(v[4 * j + 2] - ma), p3 = fast_exp2(v[4 * j + 3] - mb);
          l[2 * j] += p0 + p2;
          l[2 * j + 1] += p1 + p3;
          const uint32_t piece = (4 * g + j) * 16;
          *reinterpret_cast<uint32_t*>(P + sw128_offset(key0, piece) + 2 * hl) = pack_bf16x2(p0, p1);
          *reinterpret_cast<uint32_t*>(P + sw128_offset(key0 + 8, piece) + 2 * hl) = pack_bf16x2(p2, p3);
        }
        fence_proxy_async_smem();
        mbar_arrive(&bar_p_full[buf]);
      }
      // ---- epilogue
      if (!empty && !bad) {
        const uint32_t n = tcount - 1;
        if (!mbar_wait_group(gid, &bar_pv[n & 1][1], (n >> 1) & 1, &abort_flag)) bad = true;
        else tc_fence_after();
      }
      if (!empty && !bad) {
        // the group's 64 key slots' sums
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          l[x] += __shfl_xor_sync(0xffffffffu, l[x], 4);
          l[x] += __shfl_xor_sync(0xffffffffu, l[x], 8);
          l[x] += __shfl_xor_sync(0xffffffffu, l[x], 16);
        }
        if (lane < 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<float2*>(&red[g][wq][8 * j + hl]) = make_float2(l[2 * j], l[2 * j + 1]);
            if (wq == 0) { m_run[h0 + 8 * j + hl] = m[2 * j]; m_run[h0 + 8 * j + hl + 1] = m[2 * j + 1]; }
          }
        }
        group_sync(gid);
        if (tid < 32) l_run[h0 + tid] = red[g][0][tid] + red[g][1][tid] + red[g][2][tid] + red[g][3][tid];
      }
      bad = softmax_any256(bad);
      if (!bad && it.t >= 0) {
        if (p.splits > 1) {
          // m[H] (log2 units), l[H] and O / l [D][H], all fp32 (a node's splits
          // are joined without a rounding in between); a split without keys
          // writes its header only (m = -inf, l = -1).  NaN among the scores
          // makes l NaN, which has to reach the join: with no other score of the
          // head m is still -inf, and 0 in the header
          float* blk = reinterpret_cast<float*>(p.partial + (int64_t)id * kTreePartialBytes);
          if (tid < 32) {
            const int h = h0 + tid;
            const float l = empty ? -1.f : l_run[h], m = empty ? -INFINITY : m_run[h];
            blk[h] = l != l && m == -INFINITY ? 0.f : m;
            blk[kAttnH + h] = l;
            stat_a[h] = l == 0.f ? 0.f : 1.f / l;      // (l = 0: every score was -inf, and O 0 or 0 x inf)
          }
          group_sync(gid);
          if (!empty) {
            // staged as the partial's rows: all four M-tiles in the key buffers
            // where this is the CTA's last item (its last P.V has completed and
            // no further keys come), else 64 dims at a time in P^T's buffers
            const float4* f4 = reinterpret_cast<const float4*>(stat_a + h0);
            const bool last = id + (int)gridDim.x >= p.n_items;
#pragma unroll 1
            for (int mt = 0; mt < kAttnMT; ++mt) {
              float o[32];
              tmem_ld32(tO + lane_base + mt * kAttnH + h0, o);
              tmem_wait_ld();
              float* dst = blk + 2 * kAttnH + (g * kAttnD + mt * 128) * 32;
#pragma unroll 1
              for (int half = 0; half < (last ? 1 : 2); ++half) {
                uint8_t* stg = last ? sK + (g * kAttnMT + mt) * 16384 : sP + g * TreeSmem::P_BYTES;
                const int row = last ? tid : tid & 63;
                if (last || half == tid >> 6) {
#pragma unroll
                  for (int e4 = 0; e4 < 8; ++e4) {
                    const float4 fc = f4[e4];
                    *reinterpret_cast<float4*>(stg + sw128_offset(row, 16 * e4)) =
                        make_float4(o[4 * e4] * fc.x, o[4 * e4 + 1] * fc.y, o[4 * e4 + 2] * fc.z, o[4 * e4 + 3] * fc.w);
                  }
                }
                fence_proxy_async_smem();
                group_sync(gid);
                if (tid == 0) {
                  bulk_store(dst + half * 64 * 32, stg, last ? 16384 : 8192);
                  bulk_commit();
                  if (!last) bulk_wait_read<0>();
                }
                if (!last) group_sync(gid);
              }
            }
            if (tid == 0) bulk_wait_all();             // written before the CTA may exit
          }
        } else {
          // o = O / (l + e^{z - m}), rope dims rotated back by -t.  A thread
          // stores its dim of each head, a warp 64 contiguous bytes (two whole
          // sectors): turning the tile through shared memory first took 9,000
          // cycles an item, most of them cold instructions and barriers
          if (tid < 32) {                    // (this warp wrote l_run; m_run: see the barrier above)
            const int h = h0 + tid;
            const float mu = empty ? -INFINITY : m_run[h];
            const float M = fmaxf(mu, z2);
            const float den = exp2f(z2 - M) + (mu == -INFINITY ? 0.f : l_run[h] * exp2f(mu - M));
            // no key, or all weight on an infinite sink: o = 0
            stat_a[h] = (mu == -INFINITY || z2 == INFINITY) ? 0.f : exp2f(mu - M) / den;
          }
          group_sync(gid);
          const float4* fac4 = reinterpret_cast<const float4*>(stat_a + h0);
          __nv_bfloat16* O = p.out + ((int64_t)it.node * kAttnH + h0) * kAttnD + tid;
#pragma unroll 1
          for (int mt = 0; mt < kAttnMT; ++mt) {
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
            if (mt == kAttnMT - 1 && r0 < kAttnD) {
              // pair partners are neighbouring lanes
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float partner = __shfl_xor_sync(0xffffffffu, o[e], 1);
                if (rot) o[e] = (tid & 1) ? fmaf(-partner, turn.y, o[e] * turn.x) : fmaf(partner, turn.y, o[e] * turn.x);
              }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) O[(int64_t)e * kAttnD + mt * 128] = __float2bfloat16_rn(o[e]);
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
// One CTA per (node, 32 dims).  The partials are in L2; each thread reads its
// dim pair's 4 heads of four splits at a time, the first ones together with the
// headers, so that a few splits cost one round trip (10 us with the position,
// the maxima, the sums and O read one after another).  Up to 16 splits a head's
// maxima and sums stay in registers between its sum and the weights; the
// weights carry 1 / den, once a head and split instead of in every thread (64
// nodes of two splits: some 1 us less; 64 dims a CTA, one wave instead of two: 0.5 us
// less again, not worth a second form).
constexpr int kTreeCombineDims = 32;
constexpr int kTreeCombineThreads = 256;
constexpr int kTreeMaxSplits = 148;
__host__ __device__ constexpr int tree_combine_smem(int splits) { return splits * kAttnH * 4; }

struct TreeCombineParams {
  const char* partial; const float* sinks; const int* node_pos;
  __nv_bfloat16* out;
  int splits, rope_dims;
  double theta[64];
};

__global__ void __launch_bounds__(kTreeCombineThreads, 4) tree_combine_kernel(const __grid_constant__ TreeCombineParams p) {
  constexpr int U = 4;                                   // splits of a thread in flight
  extern __shared__ __align__(16) float cmb_s[];
  float (*w_s)[kAttnH] = reinterpret_cast<float (*)[kAttnH]>(cmb_s);
  __shared__ __align__(16) __nv_bfloat16 stage[kAttnH][kTreeCombineDims + 8];
  __shared__ float red[4][kAttnH], red2[4][kAttnH];
  griddep_wait();
  griddep_launch_dependents();
  const int node = blockIdx.x, d0 = blockIdx.y * kTreeCombineDims;
  const int tid = threadIdx.x;
  const float* P = reinterpret_cast<const float*>(p.partial) + (int64_t)node * p.splits * kTreePartialFloats;
  const int dp = tid >> 4, h4 = (tid & 15) * 4;          // dims d0 + 2 dp, + 1; heads h4 .. h4 + 3
  // the position, the headers and the first splits' O are asked for together
  // (the partial blocks of a place without a node hold no numbers, but exist)
  const int t = p.node_pos[node];
  const int h = tid & 63, part = tid >> 6;
  const float z2 = p.sinks[h] * kLog2e;
  float4 x[U], y[U];
  const auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u < p.splits) {
        const float* src = P + (int64_t)(s0 + u) * kTreePartialFloats;
        x[u] = *reinterpret_cast<const float4*>(src + tree_partial_at(d0 + 2 * dp, h4));
        y[u] = *reinterpret_cast<const float4*>(src + tree_partial_at(d0 + 2 * dp + 1, h4));
      }
    }
  };
  load(0);
  // head h: the maximum M and the sum over the splits part, part + 4, ...
  float M = -INFINITY, den = 0.f, ms[4], ls[4];
  for (int s0 = part; s0 < p.splits; s0 += 16) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + 4 * u;
      ms[u] = s < p.splits ? P[(int64_t)s * kTreePartialFloats + h] : -INFINITY;
      ls[u] = s < p.splits ? P[(int64_t)s * kTreePartialFloats + kAttnH + h] : 0.f;
    }
    float Mn = M;
#pragma unroll
    for (int u = 0; u < 4; ++u) Mn = fmaxf(Mn, ms[u]);
    const float Ms = Mn == -INFINITY ? 0.f : Mn;
    den *= exp2f(M - Ms);
#pragma unroll
    for (int u = 0; u < 4; ++u) den = ms[u] == -INFINITY ? den : fmaf(ls[u], exp2f(ms[u] - Ms), den);
    M = Mn;
  }
  if (t < 0) return;
  red[part][h] = M;
  red2[part][h] = den;
  __syncthreads();
  // the head's over all splits and the sink
  float Mt = z2;
#pragma unroll
  for (int u = 0; u < 4; ++u) Mt = fmaxf(Mt, red[u][h]);
  const float Ms = Mt == -INFINITY ? 0.f : Mt;
  den = exp2f(z2 - Ms);
#pragma unroll
  for (int u = 0; u < 4; ++u) den = red[u][h] == -INFINITY ? den : fmaf(red2[u][h], exp2f(red[u][h] - Ms), den);
  // the splits' weights (0: every score -inf, or all weight on an infinite sink;
  // -1: no key, and no O)
  const float inv = z2 == INFINITY ? 0.f : 1.f / den;
  const auto weight = [&](int s, float m, float l) {
    // (formed whether or not there are keys: with l tested first, m was asked for a
    // round trip later, 22.6 against 21.7 us for 3 nodes of 18 splits)
    const float w = m == -INFINITY || z2 == INFINITY ? 0.f : l * exp2f(m - Ms) * inv;
    w_s[s][h] = l < 0.f ? -1.f : w;
  };
  if (p.splits <= 16) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (part + 4 * u < p.splits) weight(part + 4 * u, ms[u], ls[u]);
  } else {
    for (int s = part; s < p.splits; s += 4)
      weight(s, P[(int64_t)s * kTreePartialFloats + h], P[(int64_t)s * kTreePartialFloats + kAttnH + h]);
  }
  __syncthreads();
  float a0[4] = {0.f, 0.f, 0.f, 0.f}, a1[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < p.splits; s0 += U) {
    if (s0 > 0) load(s0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u < p.splits) {
        const float4 w = *reinterpret_cast<const float4*>(&w_s[s0 + u][h4]);
        const float ws[4] = {w.x, w.y, w.z, w.w};
        const float xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, ys[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (no O: the bytes are not used)
          a0[e] += ws[e] < 0.f ? 0.f : ws[e] * xs[e];
          a1[e] += ws[e] < 0.f ? 0.f : ws[e] * ys[e];
        }
      }
    }
  }
  const int j0 = d0 + 2 * dp - (kAttnD - p.rope_dims);
  if (j0 >= 0) {
    float cs, sn;
    rope_sincos(-(double)t, p.theta[j0 >> 1], &cs, &sn);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x0 = a0[e], x1 = a1[e];
      a0[e] = x0 * cs - x1 * sn;
      a1[e] = x0 * sn + x1 * cs;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    *reinterpret_cast<__nv_bfloat162*>(&stage[h4 + e][2 * dp]) = __floats2bfloat162_rn(a0[e], a1[e]);
  __syncthreads();
  const int ho = tid >> 2, pc = (tid & 3) * 8;
  *reinterpret_cast<uint4*>(p.out + ((int64_t)node * kAttnH + ho) * kAttnD + d0 + pc) =
      *reinterpret_cast<const uint4*>(&stage[ho][pc]);
}

}  // namespace csahca
