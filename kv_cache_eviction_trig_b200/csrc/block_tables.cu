// Block tables and slot maps of a paged cache from the lengths on the GPU (serving with a paged
// KV cache: dimensionstp.github.io review, section 6, Limitations).
//
// One cluster: in every CTA thread b < B works out what sequence b needs, and two prefix sums
// over the sequences give every block that changes hands its place in the pool's ring.  Groups
// of warps, over all CTAs, move a sequence's blocks: those past the need to the ring's tail,
// then, after a cluster barrier, the missing ones from its head.  A second grid (chained by
// programmatic dependent launch) maps the tokens to slots; few slots are mapped by the first.
// Bound by latency: the lengths, the blocks that change hands, the barrier.  Eight CTAs where
// the table is large (kTableWide entries), as one CTA's warps take long rows one after
// another; a single one, whose barriers are cheaper, below that.
#include <cooperative_groups.h>

#include "tree.cuh"

namespace cg = cooperative_groups;

namespace tria {

namespace {

constexpr int kTableThreads = 1024;
constexpr int kMapThreads = 256;
constexpr int kTableCluster = 8;
// Table entries above which the cluster of eight is taken.  One CTA and eight, per call: 2304
// entries 4.2 and 4.9 us, 4608 4.5 and 5.2, 9216 5.6 and 5.6, 18432 7.5 and 5.6.
constexpr int64_t kTableWide = 8192;
// Slots up to which the first grid maps them itself.  Itself and by a second grid, on the device:
// 1024 slots 4.3 and 5.1 us, 4096 5.9 and 5.9, 8192 5.5 to 6.4 and 5.3 to 6.1, 16384 7.7 and 6.3.
// Back to back a second launch also costs the host 2 us: 4096 slots 7.4 and 9.5 us a call, 8192 7.6 and
// 9.7, 16384 8.3 and 9.7.  So 8192, where the device's times are the same.
constexpr int64_t kMapInline = 8192;

struct Ask {
  int32_t len, n;
  bool ok;  // the length and n are in range and within the sequence's capacity
};

__device__ __forceinline__ Ask ask_of(const BlockTablesParams &p, int b, int *bad) {
  Ask a{p.seq_len[b], p.n_new[b], true};
  const int64_t cap = p.seg_cap[b];
  *bad = 0;
  if (a.len < 0 || a.len > cap || a.n < 0 || a.n > p.max_new) *bad = TRIA_DEVERR_SEQ_LEN;
  else if ((int64_t)a.len + a.n > cap) *bad = TRIA_DEVERR_SEGMENT_FULL;
  a.ok = *bad == 0;
  return a;
}

// Blocks that a sequence can hold: its row's entries, and those of the largest segment (so the
// sums over the sequences below stay within 32 bits, whatever the counts say).
__device__ __forceinline__ int32_t most_held(const BlockTablesParams &p) {
  return min(p.max_blocks, TRIA_MAX_SEGMENT >> p.shift);
}
static_assert((int64_t)TRIA_MAX_BATCH * (TRIA_MAX_SEGMENT >> 4) < INT32_MAX, "sums of block counts");

// Slots of sequence b's next tokens: W of its row's entries at a time, first, first + step, ....
template <int W>
__device__ __forceinline__ void map_row(const BlockTablesParams &p, int b, int32_t len, int32_t n,
                                        bool served, int first, int step) {
  const int32_t *row = p.table + (int64_t)b * p.max_blocks;
  int32_t *to = p.slot_map + (int64_t)b * p.max_new;
  const bool whole = W == 4 && p.max_new % 4 == 0 && (reinterpret_cast<uintptr_t>(p.slot_map) & 15) == 0;
  for (int i = W * first; i < p.max_new; i += W * step) {
    int32_t slot[4];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int32_t t = len + i + k;
      slot[k] = -1;
      if (served && i + k < n) {
        const int32_t id = row[t >> p.shift];
        if (id >= 0 && id < p.n_blocks) slot[k] = (id << p.shift) + (t & ((1 << p.shift) - 1));
        else dev::set_error(p.err, TRIA_DEVERR_PAGES);
      }
    }
    if (W == 4 && whole) {
      *reinterpret_cast<int4 *>(to + i) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k)
        if (i + k < p.max_new) to[i + k] = slot[k];
    }
  }
}

// Place `at` of the ring (at < 3 n: the head, the free blocks and those that change hands).
__device__ __forceinline__ int32_t ring_place(int32_t at, int32_t n) {
  at = at >= n ? at - n : at;
  return at >= n ? at - n : at;
}

// Inclusive prefix sums of two values over the block's first 256 threads.
__device__ __forceinline__ void scan2(int32_t (&v)[2], int32_t (*sums)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t x = __shfl_up_sync(0xffffffffu, v[k], o);
      if (lane >= o) v[k] += x;
    }
  if (lane == 31) {
    sums[warp][0] = v[0];
    sums[warp][1] = v[1];
  }
  __syncthreads();
  for (int w = 0; w < warp && w < 8; ++w) {
    v[0] += sums[w][0];
    v[1] += sums[w][1];
  }
}

template <int CL>
__global__ void __launch_bounds__(kTableThreads)
    block_tables_kernel(const __grid_constant__ BlockTablesParams p, int map_inline) {
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  auto sync = [&]() {
    if (CL > 1) cl.sync();
    else __syncthreads();
  };
  // per sequence: what it holds, what it gets to hold, its places among the blocks that
  // are released and taken
  __shared__ int32_t s_old[TRIA_MAX_BATCH], s_new[TRIA_MAX_BATCH], s_rel[TRIA_MAX_BATCH],
      s_take[TRIA_MAX_BATCH], s_len[TRIA_MAX_BATCH], s_n[TRIA_MAX_BATCH];
  __shared__ int32_t sums[kTableThreads / 32][2], totals[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = CL * kTableThreads / 32;
  if (tid == 0) dev::pdl_launch_dependents();
  const int32_t head = p.ring_state[0], count = p.ring_state[1];
  int32_t old = 0, need = 0, v[2] = {0, 0}, bad = 0;
  Ask a{0, 0, false};
  if (tid < p.B) {
    a = ask_of(p, tid, &bad);
    old = p.held[tid];
    if (old < 0 || old > most_held(p)) {
      bad |= TRIA_DEVERR_PAGES;
      a.ok = false;
    }
    need = old;
    if (a.ok) {
      need = (int32_t)(((int64_t)a.len + a.n + (1 << p.shift) - 1) >> p.shift);
      v[0] = max(0, old - need);
      v[1] = max(0, need - old);
    }
  }
  const int32_t rel = v[0], shortage = v[1];
  scan2(v, sums);
  if (tid == TRIA_MAX_BATCH - 1) {
    totals[0] = v[0];
    totals[1] = v[1];
  }
  __syncthreads();
  const bool ring_ok = head >= 0 && head < p.n_blocks && count >= 0 && count <= p.n_blocks &&
                       (int64_t)count + totals[0] <= p.n_blocks;
  const int32_t pool = ring_ok ? count + totals[0] : 0;
  if (tid < p.B) {
    if (!ring_ok) need = old;
    else if (shortage > 0 && v[1] > pool) {
      bad |= TRIA_DEVERR_POOL;
      need = old;
    }
    s_old[tid] = old;
    s_new[tid] = need;
    s_rel[tid] = v[0] - rel;
    s_take[tid] = v[1] - shortage;
    s_len[tid] = a.len;
    s_n[tid] = a.ok && (int64_t)a.len + a.n <= ((int64_t)need << p.shift) ? a.n : -1;
  }
  if (tid == 0 && !ring_ok) bad |= TRIA_DEVERR_PAGES;
  if (bad && rank == 0) dev::set_error(p.err, bad);
  __syncthreads();
  // a group of warps per sequence
  const int all = rank * (kTableThreads / 32) + warp;
  const int per = max(1, kWarps / p.B), group = all / per, groups = kWarps / per;
  const int first = (all - group * per) * 32 + lane, step = per * 32;
  for (int b = group; b < p.B; b += groups) {
    const int32_t n0 = s_new[b], n1 = s_old[b];
    if (n1 <= n0) continue;
    int32_t *row = p.table + (int64_t)b * p.max_blocks;
    for (int j0 = n0 + first; j0 < n1; j0 += 4 * step) {  // four loads under way
      int32_t id[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j0 + k * step < n1) id[k] = row[j0 + k * step];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + k * step;
        if (j < n1) {
          p.ring[ring_place(head + count + s_rel[b] + (j - n0), p.n_blocks)] = id[k];
          row[j] = -1;
        }
      }
    }
  }
  sync();  // what was released can be taken, and every CTA has read the counts and the ring's state
  for (int b = group; b < p.B; b += groups) {
    const int32_t n0 = s_old[b], n1 = s_new[b];
    int32_t *row = p.table + (int64_t)b * p.max_blocks;
    for (int j0 = n0 + first; j0 < n1; j0 += 4 * step) {
      int32_t id[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + k * step;
        if (j < n1) id[k] = p.ring[ring_place(head + s_take[b] + (j - n0), p.n_blocks)];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + k * step;
        if (j < n1) {
          if (id[k] < 0 || id[k] >= p.n_blocks) dev::set_error(p.err, TRIA_DEVERR_PAGES);
          row[j] = id[k];
        }
      }
    }
  }
  if (rank == 0 && tid < p.B) p.held[tid] = s_new[tid];
  if (rank == 0 && warp == 0) {
    int32_t all = 0;
    for (int b = lane; b < p.B; b += 32) all += max(0, s_new[b] - s_old[b]);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane == 0 && ring_ok) {
      p.ring_state[0] = (int32_t)(((int64_t)head + all) % p.n_blocks);
      p.ring_state[1] = pool - all;
    }
  }
  if (!map_inline) return;
  sync();  // the rows are complete
  for (int b = group; b < p.B; b += groups) map_row<1>(p, b, s_len[b], s_n[b], s_n[b] >= 0, first, step);
}

__global__ void __launch_bounds__(kMapThreads) slot_map_kernel(const __grid_constant__ BlockTablesParams p) {
  dev::pdl_wait();
  const int b = blockIdx.y;
  int bad;
  const Ask a = ask_of(p, b, &bad);
  const int32_t held = p.held[b];
  const bool served = a.ok && held >= 0 && held <= most_held(p) &&
                      (int64_t)a.len + a.n <= ((int64_t)held << p.shift);
  map_row<4>(p, b, a.len, a.n, served, blockIdx.x * kMapThreads + threadIdx.x, gridDim.x * kMapThreads);
}

}  // namespace

cudaError_t launch_block_tables(const BlockTablesParams &p, cudaStream_t s) {
  const bool small = (int64_t)p.B * p.max_new <= kMapInline;
  const bool wide = (int64_t)p.B * p.max_blocks > kTableWide;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(wide ? kTableCluster : 1, 1, 1);
  cfg.blockDim = dim3(kTableThreads, 1, 1);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = wide ? kTableCluster : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, block_tables_kernel<kTableCluster>, p, small ? 1 : 0)
                             : cudaLaunchKernelEx(&cfg, block_tables_kernel<1>, p, small ? 1 : 0);
  if (e != cudaSuccess || small) return e;
  const int64_t per = ((int64_t)p.max_new + 4 * kMapThreads - 1) / (4 * kMapThreads);
  cfg.gridDim = dim3((unsigned)(per < 1024 ? per : 1024), (unsigned)p.B, 1);
  cfg.blockDim = dim3(kMapThreads, 1, 1);
  attr[0] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, slot_map_kernel, p);
}

}  // namespace tria
