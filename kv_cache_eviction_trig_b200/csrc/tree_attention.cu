// Attention of drafted trees over the cache (like tria_decode_attention it reads the
// budgeted cache, romaanj.github.io review, "Results").  For node i of sequence b and
// query head h of KV head g = h / G
//   out[b][i][h] = sum_x softmax_x(scale * q[b][i][h] . k_x) v_x
// over the live cached tokens and the nodes on the path from the root to i.
//
// One warp per (sequence, node, query head): 32 keys at a time, a lane per key for the
// products with the query, then a lane per D / 32 output dims for those with V; a running
// maximum and sum (online softmax), float32 throughout.
#include <cuda_bf16.h>
#include <math.h>

#include "tree.cuh"

namespace tria {

namespace {

constexpr int kRowWarps = 8;

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32)
    tree_rows_kernel(const __grid_constant__ TreeAttnParams p) {
  constexpr int E = D / 32;
  __shared__ float qs[kRowWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kRowWarps + warp;  // (b * N + i) * Hq + h
  if (row >= (int64_t)p.B * p.N * p.Hq) return;
  const int h = (int)(row % p.Hq), i = (int)(row / p.Hq % p.N), b = (int)(row / p.Hq / p.N);
  const int g = h / p.G;
  const int64_t lg = (int64_t)p.layer * p.Hkv + g;
  const int32_t n = p.n_nodes[b];
  const int32_t T = p.unit_len ? p.unit_len[lg * p.B + b] : p.seq_len[b];
  int bad = 0;
  if (n < 0 || n > p.N) bad |= TRIA_DEVERR_TREE;
  if (T < 0 || (int64_t)T > p.seg_start[b + 1] - p.seg_start[b]) bad |= TRIA_DEVERR_SEQ_LEN;
  if (bad || i >= n) {
    if (bad && i == 0 && lane == 0) dev::set_error(p.err, bad);
    return;
  }
  for (int d = lane; d < D; d += 32) qs[warp][d] = bf(p.q[row * D + d]);
  __syncwarp();
  float m = -INFINITY, l = 0.0f, o[E] = {};
  // one group of 32 keys: key rows kr, value rows vr (null: not seen)
  auto take = [&](const uint16_t *kr, const uint16_t *vr) {
    float s = -INFINITY;
    if (kr) {
      s = 0.0f;
      for (int d = 0; d < D; ++d) s = fmaf(bf(kr[d]), qs[warp][d], s);
      s *= p.scale;
    }
    float mx = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) return;
    const float a = expf(m - mn), w = kr ? expf(s - mn) : 0.0f;
    float sum = w;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * a + sum;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= a;
    for (int x = 0; x < 32; ++x) {
      const uint16_t *v = reinterpret_cast<const uint16_t *>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vr), x));
      const float wx = __shfl_sync(0xffffffffu, w, x);
      if (!v) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(wx, bf(v[lane + 32 * e]), o[e]);
    }
  };
  for (int t0 = 0; t0 < T; t0 += 32) {
    const int t = t0 + lane;
    const uint16_t *kr = nullptr, *vr = nullptr;
    if (t < T) {
      int64_t slot = p.seg_start[b] + t;
      if (p.pages.table) {
        const int32_t id = p.pages.table[(int64_t)b * p.pages.max_blocks + (t >> p.pages.shift)];
        if (id < 0 || id >= p.pages.n_blocks) dev::set_error(p.err, TRIA_DEVERR_PAGES);
        slot = ((int64_t)min(max(id, 0), p.pages.n_blocks - 1) << p.pages.shift) +
               (t & ((1 << p.pages.shift) - 1));
      }
      kr = p.k + (lg * p.cap + slot) * D;
      vr = p.v + (lg * p.cap + slot) * D;
    }
    take(kr, vr);
  }
  for (int j0 = 0; j0 <= i; j0 += 32) {
    // the path's nodes of this group of 32
    bool seen = false;
    for (int j = i; j >= j0;) {
      if (j == j0 + lane) seen = true;
      const int32_t up = p.parent[(int64_t)b * p.N + j];
      const bool fine = up >= -1 && up < j;
      if (!fine) dev::set_error(p.err, TRIA_DEVERR_TREE);
      j = fine ? up : -1;
    }
    const int64_t node = (lg * p.B + b) * p.N + j0 + lane;
    take(seen ? p.kd + node * D : nullptr, seen ? p.vd + node * D : nullptr);
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.out[row * D + lane + 32 * e] = __bfloat16_as_ushort(__float2bfloat16_rn(l == 0.0f ? 0.0f : o[e] / l));
}

}  // namespace

size_t tree_attention_scratch(int D, int G, int N) {
  (void)D;
  (void)G;
  (void)N;
  return 0;
}

cudaError_t launch_tree_attention(const TreeAttnParams &p, cudaStream_t s) {
  const int64_t blocks = ((int64_t)p.B * p.N * p.Hq + kRowWarps - 1) / kRowWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  switch (p.D) {
    case 64: tree_rows_kernel<64><<<(unsigned)blocks, kRowWarps * 32, 0, s>>>(p); break;
    case 128: tree_rows_kernel<128><<<(unsigned)blocks, kRowWarps * 32, 0, s>>>(p); break;
    case 256: tree_rows_kernel<256><<<(unsigned)blocks, kRowWarps * 32, 0, s>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace tria
