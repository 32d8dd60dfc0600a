// The accepted path of every drafted tree joins the cache: tria_append for several tokens
// per sequence (the cache grows by decoded tokens, romaanj.github.io review, "Background";
// the paper decodes one at a time).
//
// A block takes one sequence and lg_per_block of its (layer, KV head) rows.  It brings the
// sequence's parents into shared memory, walks from the accepted node to the root, and its
// warps copy the path's K and V rows (16-byte vectors, four per lane under way) to the next
// slots; every block reads the length before it reports, and the sequence's last block to
// report advances the lengths, so the step is one launch.  A sequence that cannot take its
// path is left as it is by every block, for the same reason.
// Bound by the rows' bytes (8 D + 4 per token and (layer, KV head) row).
#include "tree.cuh"

namespace tria {

namespace {

constexpr int kCommitThreads = 256;

__global__ void __launch_bounds__(kCommitThreads)
    tree_commit_kernel(const __grid_constant__ TreeCommitParams p) {
  __shared__ int32_t parent[TRIA_MAX_NODES];
  __shared__ int32_t path[TRIA_MAX_NODES];  // leaf first
  __shared__ int32_t slots[TRIA_MAX_NODES];
  __shared__ int32_t depth;
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t rows = (int64_t)p.L * p.Hkv;
  const int64_t cap_b = p.seg_start[b + 1] - p.seg_start[b];
  // everything that the sequence's blocks decide by, in one round of loads
  static_assert(kCommitThreads >= TRIA_MAX_NODES, "a thread per node");
  const int32_t last = p.last[b], n = p.n_nodes[b], cur = p.cur_pos[b];
  const int32_t T0 = p.unit_len ? 0 : p.seq_len[b];
  const int32_t up = tid < p.N ? p.parent[(int64_t)b * p.N + tid] : -1;
  const int32_t slot = p.slot_map && tid < p.max_new ? p.slot_map[(int64_t)b * p.max_new + tid] : -1;
  int bad = n < 0 || n > p.N || last < -1 || last >= n ? TRIA_DEVERR_TREE : 0;
  if (bad || last < 0) {  // the same decision in every block of the sequence
    if (bad && blockIdx.y == 0 && tid == 0) dev::set_error(p.err, bad);
    return;
  }
  if (tid <= last) {
    const bool fine = up >= -1 && up < tid;
    if (!fine && blockIdx.y == 0) dev::set_error(p.err, TRIA_DEVERR_TREE);
    parent[tid] = fine ? up : -1;
  }
  slots[tid] = slot;
  __syncthreads();
  if (tid == 0) {
    int d = 0;
    for (int i = last; i >= 0; i = parent[i]) path[d++] = i;  // parents precede their children
    depth = d;
  }
  __syncthreads();
  const int len = depth;
  if (p.unit_len) {
    for (int64_t lg = tid; lg < rows; lg += kCommitThreads) {
      const int32_t T = p.unit_len[lg * p.B + b];
      if (T < 0 || (int64_t)T > cap_b) bad |= TRIA_DEVERR_SEQ_LEN;
      else if ((int64_t)T + len > cap_b) bad |= TRIA_DEVERR_SEGMENT_FULL;
    }
  } else if (T0 < 0 || (int64_t)T0 > cap_b) {
    bad = TRIA_DEVERR_SEQ_LEN;
  } else if ((int64_t)T0 + len > cap_b) {
    bad = TRIA_DEVERR_SEGMENT_FULL;
  }
  // (a path longer than the map finds -1s behind it)
  if (p.slot_map && tid < len && (slot < 0 || (int64_t)slot >= p.cap)) bad |= TRIA_DEVERR_PAGES;
  if (__syncthreads_or(bad)) {
    if (blockIdx.y == 0 && bad) dev::set_error(p.err, bad);
    return;
  }
  const int nv = p.D >> 3;  // 16-byte vectors per row
  for (int64_t lg = (int64_t)blockIdx.y * p.lg_per_block + warp;
       lg < rows && lg < (int64_t)(blockIdx.y + 1) * p.lg_per_block; lg += kCommitThreads / 32) {
    const int64_t T = p.slot_map ? 0 : p.seg_start[b] + (p.unit_len ? p.unit_len[lg * p.B + b] : T0);
    const uint4 *ks = reinterpret_cast<const uint4 *>(p.k_new) + (lg * p.B + b) * p.N * nv;
    const uint4 *vs = reinterpret_cast<const uint4 *>(p.v_new) + (lg * p.B + b) * p.N * nv;
    uint4 *kd = reinterpret_cast<uint4 *>(p.k) + lg * p.cap * nv;
    uint4 *vd = reinterpret_cast<uint4 *>(p.v) + lg * p.cap * nv;
    // the path's 16-byte vectors, K's of a row before V's, four per lane under way
    const int row_vecs = 2 * nv, vecs = len * row_vecs;
    auto slot_of = [&](int j) { return p.slot_map ? (int64_t)slots[j] : T + j; };
    for (int i0 = lane; i0 < vecs; i0 += 128) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + 32 * k, j = i / row_vecs, e = i - j * row_vecs;
        if (i < vecs) {
          const int64_t node = path[len - 1 - j];
          v[k] = e < nv ? ks[node * nv + e] : vs[node * nv + e - nv];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + 32 * k, j = i / row_vecs, e = i - j * row_vecs;
        if (i < vecs) {
          const int64_t slot = slot_of(j);
          if (e < nv) kd[slot * nv + e] = v[k];
          else vd[slot * nv + e - nv] = v[k];
        }
      }
    }
    for (int j = lane; j < len; j += 32) p.pos[lg * p.cap + slot_of(j)] = cur + 1 + j;
  }
  // the sequence's last block advances its lengths: the others have read them
  __syncthreads();
  __shared__ int mine;
  if (tid == 0) {
    __threadfence();
    mine = atomicAdd(p.arrived + b, 1) == (int)gridDim.y - 1;
  }
  __syncthreads();
  if (!mine) return;
  if (p.unit_len) {
    for (int64_t lg = tid; lg < rows; lg += kCommitThreads) p.unit_len[lg * p.B + b] += len;
  } else if (tid == 0) {
    p.seq_len[b] = T0 + len;
  }
  if (tid == 0) {
    p.cur_pos[b] = cur + len;
    p.arrived[b] = 0;
  }
}

}  // namespace

cudaError_t launch_tree_commit(const TreeCommitParams &params, cudaStream_t s) {
  TreeCommitParams p = params;
  // a row per warp while the blocks are resident at once (eight per SM), else more: a second
  // wave would repeat the sequences' loads (64 sequences of 288 rows: 25 us with 8 rows per
  // block, 22 us with 16; one sequence: 4.2 us with 8, 4.6 us with 16)
  p.lg_per_block = kCommitThreads / 32;
  while ((int64_t)p.B * (((int64_t)p.L * p.Hkv + p.lg_per_block - 1) / p.lg_per_block) > 8ll * device_sm_count() &&
         p.lg_per_block < 64)
    p.lg_per_block *= 2;
  // (a grid is at most 65535 blocks high; rows < 2^31)
  while (((int64_t)p.L * p.Hkv + p.lg_per_block - 1) / p.lg_per_block > 65535) p.lg_per_block *= 2;
  const int64_t chunks = ((int64_t)p.L * p.Hkv + p.lg_per_block - 1) / p.lg_per_block;
  tree_commit_kernel<<<dim3((unsigned)p.B, (unsigned)chunks), kCommitThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace tria
