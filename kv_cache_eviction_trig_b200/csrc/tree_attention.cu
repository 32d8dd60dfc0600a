// Attention of drafted trees over the cache (like tria_decode_attention it reads the
// budgeted cache, romaanj.github.io review, "Results").  For node i of sequence b and
// query head h of KV head g = h / G
//   out[b][i][h] = sum_x softmax_x(scale * q[b][i][h] . k_x) v_x
// over the live cached tokens and the nodes on the path from the root to i.
//
// Design (sm_100a).  The G heads of a group share keys, so the rows of one product are
// (node, head) pairs: 128 of them per M tile.  A unit is (sequence, KV head, group of MT M
// tiles); its keys come in tiles of 128, the cached ones first, the drafted nodes last.  The
// host does not know the lengths, so every CTA adds them up and takes an equal share of the
// list of all units' tiles (a persistent grid, one CTA per SM), whatever unit it starts or
// ends in.  Within a CTA
//   warp 0        streams K and V tiles into a shared-memory ring by TMA (128-byte swizzle;
//                 a box per block of a paged cache), and the units' queries;
//   warp 1        one thread issues the tensor products: S = Q K^T into tensor memory, and
//                 O += P V with P read from tensor memory, where it overlays S;
//   warps 4..     two warpgroups of softmax: S from tensor memory, the running maximum and
//                 sum, P = 2^((S - m) c) as bf16 back to tensor memory.  MT = 1: two threads per
//                 row, each takes half of a tile's keys, and they exchange their maxima.
//                 MT = 2: a thread per row of either M tile.
// The next tile's S is computed while this one's softmax runs (MT = 1: two S buffers; MT = 2:
// the M tiles alternate).  P is computed with the maximum so far; only if the tile's own is
// larger by more than 2^8 is it computed again and O, which stays in tensor memory, rescaled
// (P is at most 2^8 otherwise; float32 sums lose nothing; rescaling only past such a bound is a
// published technique).  A separate pass for the maximum first took 0.5 of 2.6 thousand cycles
// per tile.  The maximum is one of S, and its difference to S is formed before the scale: rounded
// after it, a maximum past 2^31 would be off by factors of 2^128 (the extra operation: 61.9 us
// against 60.6 for 32768 keys and 64 nodes).
// A unit that lies in one CTA is written from there.  The parts of the others go to the
// workspace with their maxima and sums; once a CTA is through with its share it waits for the
// other CTAs of its first and of its last unit and merges its share of their rows and columns,
// the parts in the order of the keys, so results do not depend on timing.  (The launch is
// cooperative: all CTAs are resident, and each reports its parts before it waits.  A merge
// kernel of its own took 7 us from the last part to the last row, this one 2 us.)
//
// Rounding: S, maxima, sums and O are float32.  P is rounded to bf16 for the product with the
// bf16 V; the sum is of the rounded P, so that the weights add up to one and the error is at
// most about that of the bf16 output's own rounding (1.0 to 1.45 times the output's alone, by
// how even the weights are).  P as a bf16 pair high + low takes that away but doubles the
// products with V: 313 us against 272 us for 16 x 8K..32K keys, 436 against 360 for 4 x 131072.
//
// Masks.  Columns past the length, and nodes off a row's path, are set to -inf in S.  V rows
// past the length are zeroed in shared memory (P is 0 there, but 0 * NaN is not), and
// so are Inf and NaN in the drafted V rows; the rows that do see such a node get them back
// in the epilogue.
//
// What bounds it (B200, 148 SMs).  Long keys with up to 128 rows per KV head: the K and V bytes;
// 4 x 131072 keys of 8 heads, D = 128, 16 nodes: 2.15 GB in 356 us, 0.93 of the measured copy
// rate; 16 x 8192..32768 keys, 16 to 32 nodes in pages of 64: 1.48 GB in 280 us, 0.82 (back to
// back the SM clock falls, the softmax warps' 2.4 thousand cycles per tile show: 415 to 435
// us and 285 to 325).  More rows: the chain product, softmax, product of an M tile
// (4.2 thousand cycles per tile for the two M tiles, of which the tensor core works 2.0); a
// chunk of up to 255 tokens over 4 x 8.2K keys with 8 heads per KV head: 256 GFLOP in 354 us, 0.43
// of the measured matrix rate.  Short keys: latency; 2048 keys, 32 nodes: 13 us on the device, of which
// 3 pass before the first K tile arrives and 6 between the last O and the last merged row.
// D = 64 carries half the bytes and products of D = 128 per softmax step: 0.15 of the floor with 49 nodes
// of 8 heads over 23 x 3.9K..7.8K keys (84 us), 0.37 with 11 nodes over 9 x 3.6K..10.8K (58).
// Tried and slower: streams that split a tile's keys with an O of their own (288 us against
// 269 on the long case above), softmax steps of 64 keys for two M tiles (61 us against 55 for
// 32768 keys and 64 nodes: the products with N = 64 are not worth their reads of Q), four
// warpgroups of softmax for two M tiles (78 us against 69: 96 registers per thread), a quarter
// of the exponentials by a polynomial on the FMA pipes (278 us against 268), P rounded there
// (276).
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include <cudaTypedefs.h>

#include "mma_sync.cuh"
#include "ring.cuh"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace tria {

namespace {

constexpr int kTile = 128;   // keys per tile, rows per M tile
constexpr int kPartSlots = 2;  // parts that a CTA can leave: of its first and of its last unit
constexpr int kArriveStride = 32;  // words from one unit's counter to the next: a line each

// A unit of which a CTA has a part.
struct TreePart {
  int32_t b, head0, node0, n, first, last;  // first, last: the CTAs with its first and last tile
};

template <int D, int MT>
struct TreeShape {
  static constexpr int TB = kTile * D * 2;               // a K or V tile, or an M tile of queries
  static constexpr int SLAB = kTile * 128;               // 128 rows of 64 columns
  static constexpr int QB = D == 64 ? 2 : 1;              // query buffers
  static constexpr int NS = D == 256 ? 2 : D == 64 ? 8 : MT == 2 ? 4 : 5;  // ring slots
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = QB * MT * TB;
  static constexpr int OFF_CTL = OFF_RING + NS * TB;
  static constexpr int NH = MT == 2 ? 1 : 2;             // threads per row
  static constexpr int THREADS = 128 + 128 * NH * MT;
};

struct TreeCtl {
  uint64_t full[8], empty[8], q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_free[2], done;
  uint32_t tmem;
  int32_t abort;
  int4 start;                          // where this CTA's share starts: sequence, head, M group, tile
  int32_t warp_sums[8];
  uint32_t poison[4];                  // drafted V rows of the tile with Inf or NaN
  float swap[2][2][2][kTile];          // what a row's two threads exchange: in turn, by M tile and half
  uint32_t tn[TRIA_MAX_BATCH];         // live length (0 with per-unit lengths) << 9 | nodes (0: skipped)
  uint32_t path[TRIA_MAX_NODES / 32][TRIA_MAX_NODES];  // word w of the node's path
  int16_t jump[TRIA_MAX_NODES];
};
static_assert(TRIA_MAX_NODES < 512 && TRIA_MAX_SEGMENT < (1 << 23), "lengths and nodes in one word");

template <int D, int MT>
constexpr int tree_smem() {
  return TreeShape<D, MT>::OFF_CTL + (int)sizeof(TreeCtl) + 1024;  // + room to align to 1024
}

// Waits that ran out make every later wait return at once; all roles then run through
// their loops without issuing copies or products.
__device__ __forceinline__ bool tree_wait(TreeCtl &c, uint64_t *bar, uint32_t parity, int32_t *err) {
  uint32_t done;  // a plain test first: most barriers have completed by the time they are awaited
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(dev::smem_addr(bar)), "r"(parity)
      : "memory");
  if (done) return true;
  for (uint32_t i = 0; i < 2000000u; ++i) {
    if (*reinterpret_cast<volatile int32_t *>(&c.abort)) return false;
    if (dev::mbar_try_wait(bar, parity)) return true;
  }
  *reinterpret_cast<volatile int32_t *>(&c.abort) = 1;
  dev::set_error(err, TRIA_DEVERR_TIMEOUT);
  return false;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const void *map, int32_t x, int32_t y,
                                            int32_t z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dev::smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(dev::smem_addr(bar))
      : "memory");
}

// A named barrier that tells whether any of its threads gave true.
__device__ __forceinline__ bool barrier_any(uint32_t id, uint32_t threads, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"((uint32_t)mine)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two float32 products and sums at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// The tiles [k0, k1) of unit (b, g, mg), which has K tiles, KT of them cached.
struct Piece {
  int b, g, mg, k0, k1, K, KT, T, n;
};

// Walks a CTA's share of the tile list, a piece at a time.
template <int MT>
struct Walk {
  const TreeAttnParams &p;
  const TreeCtl &c;
  int b, g, mg, kt, left;

  __device__ __forceinline__ int length(int b_, int g_) const {
    if (!p.unit_len) return (int)(c.tn[b_] >> 9);
    const int32_t t = p.unit_len[((int64_t)p.layer * p.Hkv + g_) * p.B + b_];
    return t < 0 || (int64_t)t > p.seg_start[b_ + 1] - p.seg_start[b_] ? -1 : t;
  }
  __device__ __forceinline__ int nodes(int b_) const { return (int)(c.tn[b_] & 511u); }
  // M groups of sequence b, and key tiles of a unit with T cached tokens (none if T < 0)
  __device__ __forceinline__ int groups(int b_) const {
    return (nodes(b_) * p.G + MT * kTile - 1) / (MT * kTile);
  }
  __device__ __forceinline__ int tiles(int b_, int T) const {
    return T < 0 ? 0 : (T + kTile - 1) / kTile + (nodes(b_) + kTile - 1) / kTile;
  }
  __device__ __forceinline__ Walk(const TreeAttnParams &p_, const TreeCtl &c_, int left_)
      : p(p_), c(c_), b(c_.start.x), g(c_.start.y), mg(c_.start.z), kt(c_.start.w), left(left_) {}
  __device__ __forceinline__ bool next(Piece &x) {
    while (left > 0) {
      if (g == p.Hkv || nodes(b) == 0) {
        g = 0;
        ++b;
        continue;
      }
      const int T = length(b, g), K = tiles(b, T);
      if (K == 0) {
        ++g;
        continue;
      }
      x.b = b;
      x.g = g;
      x.mg = mg;
      x.k0 = kt;
      x.k1 = min(K, kt + left);
      x.K = K;
      x.KT = (T + kTile - 1) / kTile;
      x.T = T;
      x.n = nodes(b);
      left -= x.k1 - x.k0;
      kt = 0;
      if (++mg == groups(b)) {
        mg = 0;
        ++g;
      }
      return true;
    }
    return false;
  }
};

// Where tile x of a CTA's X tiles stands in the ring's order of K and V tiles.
template <int MT>
__device__ __forceinline__ int k_seq(int x) {
  return MT == 2 ? 2 * x : x == 0 ? 0 : 2 * x - 1;  // MT = 1: K0 K1 V0 K2 V1 ...
}
template <int MT>
__device__ __forceinline__ int v_seq(int x, int X) {
  return MT == 2 ? 2 * x + 1 : x < X - 1 ? 2 * x + 2 : 2 * x + 1;
}

__device__ __forceinline__ int64_t share_start(int64_t total, int c, int ctas) {
  return total * c / ctas;
}

// Merges a unit's parts, in the order of the keys: warp `rank` of `warps` takes every warps-th
// item of 32 rows by DC output dims, lane = row, AT parts under way at a time (the loads'
// latency bounds it: many parts want few dims at a time, few parts many).
template <int D, int ROWS, int DC, int AT>
__device__ __forceinline__ void merge_items(const TreeAttnParams &p, const TreePart &t, int rank, int warps) {
  constexpr int PART = ROWS * (D + 2);
  const int lane = threadIdx.x & 31, parts = t.last - t.first + 1;
  const float sl = p.scale * 1.4426950408889634f;
  const int rows = min((t.n - t.node0) * p.G, ROWS), groups = (rows + 31) / 32;
  for (int it = rank; it < groups * (D / DC); it += warps) {
    const int d0 = it / groups * DC, r = (it % groups) * 32 + lane;
    if (r >= rows) continue;
    const float *src = p.scratch + (size_t)t.first * kPartSlots * PART + r;
    float M = -INFINITY, L = 0.0f, o[DC] = {};
    for (int i0 = 0; i0 < parts; i0 += AT) {
      float v[AT][DC + 2];
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        if (i0 + i < parts) {
          const float *y = src + ((size_t)(i0 + i) * kPartSlots + (i0 + i == 0 ? 1 : 0)) * PART;
#pragma unroll
          for (int e = 0; e < DC; ++e) v[i][e] = __ldcg(y + (d0 + e) * ROWS);
          v[i][DC] = __ldcg(y + D * ROWS);
          v[i][DC + 1] = __ldcg(y + (D + 1) * ROWS);
        }
      }
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        if (i0 + i < parts) {
          // a part that saw nothing (its sum is 0) adds 0; a NaN in it stays one
          const float mc = v[i][DC], l1 = v[i][DC + 1], top = fmaxf(M, mc), ref = top == -INFINITY ? 0.0f : top;
          const float a = exp2_approx((M - ref) * sl);  // (0 for the first part)
          const float w = mc == -INFINITY ? (l1 == 0.0f ? 0.0f : 1.0f) : exp2_approx((mc - ref) * sl);
          M = top;
          L = fmaf(L, a, w * l1);
#pragma unroll
          for (int e = 0; e < DC; ++e) o[e] = fmaf(o[e], a, w * v[i][e]);
        }
      }
    }
    const float inv = 1.0f / L;  // (0 only where all logits are -inf: such a row becomes NaN)
    uint2 *to = reinterpret_cast<uint2 *>(p.out + (((int64_t)t.b * p.N + t.node0 + r / p.G) * p.Hq + t.head0 + r % p.G) * D + d0);
#pragma unroll
    for (int e = 0; e < DC; e += 4)
      to[e / 4] = make_uint2(pack_bf16x2(o[e] * inv, o[e + 1] * inv), pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv));
  }
}

template <int D, int MT>
__global__ void __launch_bounds__(TreeShape<D, MT>::THREADS, 1)
    tree_attention_kernel(const __grid_constant__ TreeAttnParams p) {
  using S = TreeShape<D, MT>;
  constexpr int TB = S::TB, SLAB = S::SLAB, NS = S::NS, QB = S::QB, NB = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024u - (dev::smem_addr(smem_raw) & 1023u)) & 1023u);
  TreeCtl &c = *reinterpret_cast<TreeCtl *>(sm + S::OFF_CTL);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;

  // ---------------------------------------------------------------- setup
  // (the segments' bounds by ordinary loads: a constant-bank read takes one address at a time)
  const int64_t *starts = p.seg_start;
  asm volatile("" : "+l"(starts));
  if (tid == 96) {
    const CUtensorMap *maps[] = {&p.tq, &p.tk, &p.tv, &p.tkd, &p.tvd};
    for (const CUtensorMap *t : maps)
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(t)) : "memory");
  }
  int tiles_b = 0;
  if (tid < TRIA_MAX_BATCH) {
    if (tid < p.B) {
      int n = p.n_nodes[tid], T = p.unit_len ? 0 : p.seq_len[tid], bad = 0;
      if (n < 0 || n > p.N) {
        bad = TRIA_DEVERR_TREE;
        n = 0;
      }
      const int64_t cap_b = starts[tid + 1] - starts[tid];
      const int M = (n * p.G + MT * kTile - 1) / (MT * kTile), DT = (n + kTile - 1) / kTile;
      if (p.unit_len) {
        for (int g = 0; g < p.Hkv; ++g) {
          const int32_t t = p.unit_len[((int64_t)p.layer * p.Hkv + g) * p.B + tid];
          if (t < 0 || (int64_t)t > cap_b) bad |= TRIA_DEVERR_SEQ_LEN;
          else tiles_b += M * ((t + kTile - 1) / kTile + DT);
        }
      } else {
        if (T < 0 || (int64_t)T > cap_b) {
          bad |= TRIA_DEVERR_SEQ_LEN;
          n = T = 0;
        } else {
          tiles_b = M * p.Hkv * ((T + kTile - 1) / kTile + DT);
        }
      }
      if (bad && cta == 0) dev::set_error(p.err, bad);
      c.tn[tid] = (uint32_t)T << 9 | (uint32_t)n;
    }
  }
  if (warp == 1) tc::tmem_alloc<512>(&c.tmem);
  if (tid == 64) {
    for (int i = 0; i < NS; ++i) {
      dev::mbar_init(&c.full[i], 1);
      dev::mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      dev::mbar_init(&c.q_full[i], 1);
      dev::mbar_init(&c.q_empty[i], 1);
      dev::mbar_init(&c.s_full[i], 1);
      dev::mbar_init(&c.p_full[i], 128 * S::NH);
      dev::mbar_init(&c.o_full[i], 1);
      dev::mbar_init(&c.o_free[i], 128 * S::NH);
    }
    dev::mbar_init(&c.done, 1);
    dev::fence_mbar_init();
    c.abort = 0;
  }
  // prefix sums of the sequences' tiles
  int incl = tiles_b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (warp < 8 && lane == 31) c.warp_sums[warp] = incl;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  int64_t total = 0;
  for (int w = 0; w < 8; ++w) {
    if (w < warp) incl += c.warp_sums[w];
    total += c.warp_sums[w];
  }
  // no share is empty but those of the last CTAs, where there are fewer tiles than CTAs
  const int ctas = (int)min((int64_t)gridDim.x, total);
  const int w0 = cta < ctas ? (int)share_start(total, cta, ctas) : 0;
  const int w1 = cta < ctas ? (int)share_start(total, cta + 1, ctas) : 0;
  const int X = w1 - w0;
  if (X > 0 && tid < TRIA_MAX_BATCH && w0 >= incl - tiles_b && w0 < incl) {
    const int n = (int)(c.tn[tid] & 511u), M = (n * p.G + MT * kTile - 1) / (MT * kTile);
    int rem = w0 - (incl - tiles_b), g = 0, K = (int)(c.tn[tid] >> 9);
    K = (K + kTile - 1) / kTile + (n + kTile - 1) / kTile;
    if (p.unit_len) {
      for (;; ++g) {
        const int32_t t = p.unit_len[((int64_t)p.layer * p.Hkv + g) * p.B + tid];
        const bool fine = t >= 0 && (int64_t)t <= starts[tid + 1] - starts[tid];
        K = fine ? (t + kTile - 1) / kTile + (n + kTile - 1) / kTile : 0;
        if (rem < K * M) break;
        rem -= K * M;
      }
    } else {
      g = rem / (K * M);
      rem -= g * K * M;
    }
    c.start = make_int4(tid, g, rem / K, rem % K);
  }
  __syncthreads();
  const uint32_t tmem = c.tmem;
  const uint32_t tm_s[2] = {tmem, tmem + 128}, tm_o[2] = {tmem + 256, tmem + 256 + (MT == 2 ? D : 0)};

  if (X > 0) {
  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    Walk<MT> walk(p, c, X);
    Piece u;
    int x = 0, pi = 0;
    int tiles = 0, queries = 0;  // copies issued: of K and V tiles (in the order of `seq`), of queries
    // a tile's K or V rows into ring place `seq`
    auto load = [&](const Piece &q, int kt, bool v, int seq, int32_t id) {
      const int s = seq % NS, use = seq / NS;
      if (use > 0) tree_wait(c, &c.empty[s], (use - 1) & 1, p.err);
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int32_t *>(&c.abort))) return;
      ++tiles;
      uint8_t *to = sm + S::OFF_RING + s * TB;
      const int lg = p.layer * p.Hkv + q.g;
      if (kt >= q.KT) {  // drafted nodes
        if (lane == 0) {
          dev::mbar_arrive_expect_tx(&c.full[s], (uint32_t)(NB * p.draft_rows * 128));
          for (int cb = 0; cb < NB; ++cb)
            tma_load_3d(to + cb * SLAB, v ? &p.tvd : &p.tkd, cb * 64, (kt - q.KT) * kTile,
                        lg * p.B + q.b, &c.full[s]);
        }
      } else if (!p.pages.table) {
        if (lane == 0) {
          dev::mbar_arrive_expect_tx(&c.full[s], (uint32_t)TB);
          for (int cb = 0; cb < NB; ++cb)
            tma_load_3d(to + cb * SLAB, v ? &p.tv : &p.tk, cb * 64,
                        (int32_t)p.seg_start[q.b] + kt * kTile, lg, &c.full[s]);
        }
      } else {
        // lane j takes block j of the tile (blocks of 256: its half)
        const int rows = min(kTile, 1 << p.pages.shift);
        const int need = (min(kTile, q.T - kt * kTile) + rows - 1) / rows;
        if (lane == 0) dev::mbar_arrive_expect_tx(&c.full[s], (uint32_t)(NB * need * rows * 128));
        __syncwarp();
        if (lane < need) {
          const int32_t slot = (id << p.pages.shift) + (kt * kTile & ((1 << p.pages.shift) - 1) & ~(rows - 1));
          for (int cb = 0; cb < NB; ++cb)
            tma_load_3d(to + cb * SLAB + lane * rows * 128, v ? &p.tv : &p.tk, cb * 64, slot, lg,
                        &c.full[s]);
        }
      }
    };
    // block id of lane j's rows in cached tile kt
    auto block_of = [&](const Piece &q, int kt) -> int32_t {
      if (!p.pages.table || kt >= q.KT) return 0;
      const int rows = min(kTile, 1 << p.pages.shift);
      const int t = kt * kTile + lane * rows;
      if (lane * rows >= kTile || t >= q.T) return 0;
      const int32_t id = p.pages.table[(int64_t)q.b * p.pages.max_blocks + (t >> p.pages.shift)];
      if (id < 0 || id >= p.pages.n_blocks) {
        dev::set_error(p.err, TRIA_DEVERR_PAGES);
        return 0;
      }
      return id;
    };
    // the V of a tile follows the next tile's K (MT = 1), which may be another unit's
    Piece vu = {};
    int vkt = -1, vx = 0;
    int32_t vid = 0;
    while (walk.next(u)) {
      const int qb = pi % QB, quse = pi / QB;
      if (quse > 0) tree_wait(c, &c.q_empty[qb], (quse - 1) & 1, p.err);
      if (lane == 0 && !*reinterpret_cast<volatile int32_t *>(&c.abort)) {
        ++queries;
        dev::mbar_arrive_expect_tx(&c.q_full[qb], (uint32_t)(MT * TB));
        for (int m = 0; m < MT; ++m)
          for (int cb = 0; cb < NB; ++cb)
            tma_load_3d(sm + S::OFF_Q + (qb * MT + m) * TB + cb * SLAB, &p.tq, cb * 64, u.g * p.G,
                        u.b * p.N + (u.mg * MT + m) * (kTile / p.G), &c.q_full[qb]);
      }
      __syncwarp();
      for (int kt = u.k0; kt < u.k1; ++kt, ++x) {
        const int32_t id = block_of(u, kt);
        load(u, kt, false, k_seq<MT>(x), id);
        if (MT == 2) {
          load(u, kt, true, v_seq<MT>(x, X), id);
        } else {
          if (x > 0) load(vu, vkt, true, v_seq<MT>(vx, X), vid);
          vu = u;
          vkt = kt;
          vx = x;
          vid = id;
        }
      }
      ++pi;
    }
    if (MT == 1) load(vu, vkt, true, v_seq<MT>(vx, X), vid);
    if (*reinterpret_cast<volatile int32_t *>(&c.abort)) {
      // copies in flight land before the shared memory is given up (lane 0 has issued the queries')
      if (lane == 0) {
        auto landed = [](uint64_t *bar, uint32_t parity) {
          for (int k = 0; k < 2000 && !dev::mbar_try_wait(bar, parity); ++k) {
          }
        };
        drain_ring(tiles, NS, [&](int i, uint32_t parity) { landed(&c.full[i], parity); });
        drain_ring(queries, QB, [&](int i, uint32_t parity) { landed(&c.q_full[i], parity); });
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    const uint32_t one = tc::elect_one();
    Walk<MT> walk(p, c, X), ahead(p, c, X);
    Piece u, ua;
    int ka = 0, pa = -1;       // the next S product's tile and piece
    bool more = ahead.next(ua);
    if (more) {
      ka = ua.k0;
      pa = 0;
    }
    bool gone = false;         // a wait ran out: nothing is issued any more
    auto await = [&](uint64_t *bar, int phase) {
      if (!tree_wait(c, bar, phase & 1, p.err)) gone = true;
    };
    auto settled = [&]() {     // the warp is together again, and of one mind
      gone = __any_sync(0xffffffffu, gone);
      tc::fence_after();
      return !gone;
    };
    const uint32_t base_lo = __shfl_sync(0xffffffffu, dev::smem_addr(sm), 0);
    // S of the tile ahead, x, M tile m
    auto scores = [&](int x, int m) {
      const int qb = pa % QB, s = k_seq<MT>(x) % NS, buf = MT == 2 ? m : x & 1;
      const uint64_t qd = tc::desc(base_lo + S::OFF_Q + (qb * MT + m) * TB, 16);
      const uint64_t kd = tc::desc(base_lo + S::OFF_RING + s * TB, 16);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((uint32_t)(k >> 2) * SLAB + (uint32_t)(k & 3) * 32) >> 4;
        tc::mma_ss(tm_s[buf], qd + off, kd + off, tc::instr(kTile, false), k > 0, one);
      }
      tc::commit(&c.s_full[buf], one);
      if (m == MT - 1) {
        tc::commit(&c.empty[s], one);
        if (ka + 1 == ua.k1) tc::commit(&c.q_empty[qb], one);
      }
    };
    // its operands have arrived
    auto await_scores = [&](int x, int m) {
      if (m > 0) return;
      if (ka == ua.k0) await(&c.q_full[pa % QB], pa / QB);
      await(&c.full[k_seq<MT>(x) % NS], k_seq<MT>(x) / NS);
    };
    // O of tile x, M tile m
    auto output = [&](int x, int m, bool first) {
      const int s = v_seq<MT>(x, X) % NS, buf = MT == 2 ? m : x & 1;
      const uint64_t vd = tc::desc(base_lo + S::OFF_RING + s * TB, SLAB);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        tc::mma_ts(tm_o[m], tm_s[buf] + 8 * k, vd + (2048 >> 4) * k, tc::instr(D, true), !first || k > 0, one);
      tc::commit(&c.o_full[m], one);
      if (m == MT - 1) tc::commit(&c.empty[s], one);
    };
    auto await_output = [&](int x, int m, bool first, int pi) {
      if (m == 0) await(&c.full[v_seq<MT>(x, X) % NS], v_seq<MT>(x, X) / NS);
      if (first && pi > 0) await(&c.o_free[m], pi - 1);
      await(&c.p_full[MT == 2 ? m : x & 1], MT == 2 ? x : x >> 1);
    };
    auto step_ahead = [&]() {
      if (++ka == ua.k1) {
        more = ahead.next(ua);
        if (more) {
          ka = ua.k0;
          ++pa;
        }
      }
    };
    await_scores(0, 0);
    if (settled())
      for (int m = 0; m < MT; ++m) scores(0, m);
    step_ahead();
    int x = 0, pi = 0;
    while (walk.next(u)) {
      for (int kt = u.k0; kt < u.k1; ++kt, ++x) {
        for (int m = 0; m < MT; ++m) {
          if (MT == 1 && more) {
            await_scores(x + 1, m);
            if (settled()) scores(x + 1, m);
          }
          // (two M tiles: the next S goes out right behind the product with V, so its operands
          // are awaited before the P)
          const bool first = kt == u.k0;
          if (MT == 2 && more) await_scores(x + 1, m);
          await_output(x, m, first, pi);
          if (settled()) {
            output(x, m, first);
            if (MT == 2 && more) scores(x + 1, m);
          }
        }
        if (more) step_ahead();
      }
      ++pi;
    }
    if (gone) {  // products in flight complete before tensor memory is given up
      tc::commit(&c.done, one);
      for (int k = 0; k < 2000 && !dev::mbar_try_wait(&c.done, 0); ++k) {
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax
    constexpr int NH = S::NH, HK = kTile / NH, HD = D / NH;    // keys and output dims per thread
    const int q4 = warp & 3, m = (warp - 4) / (4 * NH), half = NH == 2 ? ((warp - 4) >> 2) & 1 : 0;
    const int kid = tid - 128, row = q4 * 32 + lane, part_id = half * 128 + row;  // row of M tile m; its thread
    const uint32_t lane_off = (uint32_t)q4 << 21;              // 32 lanes of tensor memory
    const float sl = p.scale * 1.4426950408889634f;            // c: from S to powers of two
    const int per = kTile / p.G;                               // nodes per M tile
    const uint32_t pair = 2 + m * 4 + q4;                      // barrier of a row's two warps (NH = 2)
    Walk<MT> walk(p, c, X);
    Piece u;
    constexpr int ALL = 128 * NH * MT;
    static_assert(ALL >= TRIA_MAX_NODES, "a thread per parent");
    int x = 0, swaps = 0;
    // the units of which this CTA has a part: what their merge needs
    constexpr int ROWS = MT * kTile;
    int pending = 0;
    TreePart todo[2];
    // The products with V up to that of tile x - 1 have completed.  (A parity tells only the
    // last two phases of a barrier apart.  While this row's P of tile x is outstanding, that of
    // x - 1 or x - 2 is the last that can have completed, as S of x came after x - 2.)
    auto outputs_before = [&](int x) {
      if (x > 0) tree_wait(c, &c.o_full[m], (x - 1) & 1, p.err);
      __syncwarp();
    };
    while (walk.next(u)) {
      const int node0 = (u.mg * MT + m) * per;
      const int node = node0 + row / p.G, head = u.g * p.G + row % p.G;
      const bool live = node < u.n;
      const bool any = node0 + (row & ~31) / p.G < u.n;  // the warp has a live row
      int32_t up = -1;
      if (u.k1 > u.KT && kid < u.n) {  // the parents, ahead of their use
        up = p.parent[(int64_t)u.b * p.N + kid];
        if (up < -1 || up >= kid) {
          dev::set_error(p.err, TRIA_DEVERR_TREE);
          up = -1;
        }
      }
      float mr = -INFINITY, l = 0.0f;
      uint32_t hurt[2][4] = {};  // nodes on this row's path whose V has Inf or NaN
      for (int kt = u.k0; kt < u.k1; ++kt, ++x) {
        const int buf = MT == 2 ? m : x & 1;
        const bool draft = kt >= u.KT;
        const int valid = draft ? u.n - (kt - u.KT) * kTile : u.T - kt * kTile;  // columns (may pass 128)
        const bool masked = draft || valid < kTile;
        uint32_t on[4] = {~0u, ~0u, ~0u, ~0u};  // the tile's columns that this row sees
        if (draft) {
          constexpr int PW = TRIA_MAX_NODES / 32;
          dev::named_barrier(1, ALL);  // the last tile's paths and marks have been read
          if (kid < 4) c.poison[kid] = 0;
          if (kt == max(u.KT, u.k0)) {
            // Every node's path as bits, once per piece, a thread per node, by doubling: what
            // its path is known to hold joins what that of the node `to` holds, the first one
            // not known yet, and `to` moves on to that node's.
            uint32_t bits[PW];
            int to = up;
#pragma unroll
            for (int w = 0; w < PW; ++w) c.path[w][kid] = bits[w] = w == kid >> 5 ? 1u << (kid & 31) : 0u;
            c.jump[kid] = (int16_t)to;
            dev::named_barrier(1, ALL);
            for (;;) {
              uint32_t more[PW];
              int next = -1;
              if (to >= 0) {
#pragma unroll
                for (int w = 0; w < PW; ++w) more[w] = c.path[w][to];
                next = c.jump[to];
              }
              if (!barrier_any(1, ALL, to >= 0)) break;  // (and all have read)
              if (to >= 0) {
#pragma unroll
                for (int w = 0; w < PW; ++w) c.path[w][kid] = bits[w] |= more[w];
                c.jump[kid] = (int16_t)(to = next);
              }
              dev::named_barrier(1, ALL);
            }
          }
          dev::named_barrier(1, ALL);
#pragma unroll
          for (int e = 0; e < 4; ++e) on[e] = live ? c.path[(kt - u.KT) * (kTile / 32) + e][node] : 0u;
        } else if (masked) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            on[e] = valid >= 32 * (e + 1) ? ~0u : valid <= 32 * e ? 0u : (1u << (valid - 32 * e)) - 1u;
        }
        tree_wait(c, &c.s_full[buf], (MT == 2 ? x : x >> 1) & 1, p.err);
        __syncwarp();
        tc::fence_after();
        if (any) {
          const uint32_t ts = tm_s[buf] + lane_off;
          // columns [32 e, 32 e + 32) of this thread's keys: asked for, and arrived
          auto ask = [&](int e, float *s) {
            tc::ld32(ts + half * HK + 32 * e, reinterpret_cast<uint32_t *>(s));
          };
          if (masked) {  // -inf into the columns that this row does not see
#pragma unroll 1
            for (int e = 0; e < HK / 32; ++e) {
              const int w4 = e + (NH == 2 ? 2 * half : 0);
              const uint32_t bits = w4 == 0 ? on[0] : w4 == 1 ? on[1] : w4 == 2 ? on[2] : on[3];
              float s[32];
              ask(e, s);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(bits >> i & 1u)) s[i] = -INFINITY;
              tc::st32(ts + half * HK + 32 * e, reinterpret_cast<uint32_t *>(s));
            }
            tc::wait_st();
          }
          // the larger of the two threads' values
          auto both = [&](float v) {
            if (NH == 1) return v;
            c.swap[swaps & 1][m][half][row] = v;
            dev::named_barrier(pair, 64);
            v = fmaxf(v, c.swap[swaps & 1][m][half ^ 1][row]);
            ++swaps;
            return v;
          };
          if (kt == u.k0) {  // the first maximum
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
            for (int e = 0; e < HK / 32; ++e) {
              float s[32];
              ask(e, s);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) mx[i & 1] = fmaxf(mx[i & 1], s[i]);
            }
            mr = both(fmaxf(mx[0], mx[1]));
          }
          // P with the maximum so far, which as a rule stands (within 2^8), 64 keys at a time;
          // if theirs is larger, once more with that.  A maximum grows by whole powers of two
          // of P, so that a change of scale is exact up to the rounding of the maximum.
#pragma unroll 1
          for (int h = 0; h < HK / 64; ++h) {
            float2 sum;
            uint32_t w[32];
            for (;;) {
              const float base = mr == -INFINITY ? 0.0f : mr;
              // the difference first: scale * maximum may be so large that its rounding alone
              // is a factor of many powers of two
              const float2 scale2 = make_float2(sl, sl), base2 = make_float2(-base, -base);
              float2 sums[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
              float mx[2] = {-INFINITY, -INFINITY};
              float s[2][32];
              ask(2 * h, s[0]);
              tc::wait_ld();
              ask(2 * h + 1, s[1]);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (e == 1) tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float2 y = mul2(add2(make_float2(s[e][2 * i], s[e][2 * i + 1]), base2), scale2);
                  mx[0] = fmaxf(mx[0], s[e][2 * i]);
                  mx[1] = fmaxf(mx[1], s[e][2 * i + 1]);
                  const float2 a = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                  const uint32_t r2 = pack_bf16x2(a.x, a.y);
                  sums[i & 1] = add2(sums[i & 1], make_float2(dev::bf16lo(r2), dev::bf16hi(r2)));
                  w[16 * e + i] = r2;
                }
              }
              sum = add2(sums[0], sums[1]);
              const float top = both(fmaxf(mx[0], mx[1]));
              const float rise = mr == -INFINITY ? (top == mr ? 0.0f : INFINITY) : (top - mr) * sl;
              if (!__any_sync(0xffffffffu, rise > 8.0f)) break;
              // (what it rises by past 2^128 leaves nothing of the terms before it)
              const float mn = rise > 128.0f ? top
                             : rise > 8.0f   ? fminf(fmaxf(top, mr + ceilf(rise) / sl), FLT_MAX)
                                             : mr;
              const float a = mn == mr ? 1.0f : exp2_approx((mr - mn) * sl);
              tc::wait_st();  // O, or the first half of P, as the last change of scale left it
              if (kt > u.k0) {
                outputs_before(x);
                tc::fence_after();
#pragma unroll 1
                for (int d = half * HD; d < (half + 1) * HD; d += 32) {
                  uint32_t o[32];
                  tc::ld32(tm_o[m] + lane_off + d, o);
                  tc::wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                  tc::st32(tm_o[m] + lane_off + d, o);
                }
              }
              if (h > 0) {  // and the tile's first half of P
                uint32_t o[32];
                tc::ld32(ts, o);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = pack_bf16x2(dev::bf16lo(o[i]) * a, dev::bf16hi(o[i]) * a);
                tc::st32(ts, o);
              }
              l *= a;
              mr = mn;
            }
            l += sum.x + sum.y;
            // (both threads of the row have read the S that this overwrites)
            tc::st32(ts + (HK / 2) * half + 32 * h, w);
          }
        }
        if (masked) {
          // this tile's V in shared memory: rows past `valid` become zero, and in a tile of
          // nodes so do Inf and NaN
          const int seq = v_seq<MT>(x, X), s = seq % NS;
          if (NS < 4) outputs_before(x);  // (a ring of two: the tile before in this place has arrived)
          tree_wait(c, &c.full[s], (seq / NS) & 1, p.err);
          uint8_t *vt = sm + S::OFF_RING + s * TB;
          if (draft) {
            for (int i = kid; i < kTile * D / 8; i += ALL) {
              uint4 *at = reinterpret_cast<uint4 *>(vt) + i;
              const int r = (i >> 3) & (kTile - 1);
              if (r >= valid) {
                *at = make_uint4(0u, 0u, 0u, 0u);
                continue;
              }
              uint4 v = *at;
              uint32_t *vs = &v.x;
              bool bad = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((vs[e] & 0x7f80u) == 0x7f80u) {
                  vs[e] &= 0xffff0000u;
                  bad = true;
                }
                if ((vs[e] & 0x7f800000u) == 0x7f800000u) {
                  vs[e] &= 0x0000ffffu;
                  bad = true;
                }
              }
              if (bad) {
                *at = v;
                atomicOr(&c.poison[r >> 5], 1u << (r & 31));
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            dev::named_barrier(1, ALL);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (kt > u.KT) hurt[1][e] = on[e] & c.poison[e];
              else hurt[0][e] = on[e] & c.poison[e];
            }
          } else {
            for (int i = part_id; i < (kTile - valid) * (D / 8); i += 128 * NH) {
              const int r = valid + i / (D / 8), q = i % (D / 8);
              *(reinterpret_cast<uint4 *>(vt + (q >> 3) * SLAB + r * 128) + (q & 7)) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
        if (kt + 1 == u.k1) outputs_before(x);  // for the wait below, while it is certain which phase is next
        tc::wait_st();
        tc::fence_before();
        dev::mbar_arrive(&c.p_full[buf]);
      }
      // ------------------------------------------------------------ the unit, or its part
      if (any && NH == 2) {  // the row's sum
        c.swap[swaps & 1][m][half][row] = l;
        dev::named_barrier(pair, 64);
        const float other = c.swap[swaps & 1][m][half ^ 1][row];
        ++swaps;
        l = half ? other + l : l + other;
      }
      outputs_before(x);
      tc::fence_after();
      const bool whole = u.k0 == 0 && u.k1 == u.K;
      const int r = m * kTile + row;
      if (any) {
        const float inv = 1.0f / l;  // (l is 0 only where all logits are -inf: such a row becomes NaN)
        uint4 *to = reinterpret_cast<uint4 *>(p.out + (((int64_t)u.b * p.N + node) * p.Hq + head) * D);
        float *part = p.scratch + ((size_t)cta * kPartSlots + (u.k0 > 0 ? 0 : 1)) * (size_t)(MT * kTile) * (D + 2) + r;
        bool any_hurt = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) any_hurt |= (hurt[0][e] | hurt[1][e]) != 0;
#pragma unroll 1
        for (int d = half * HD; d < (half + 1) * HD; d += 32) {
          float o[32];
          __syncwarp();
          tc::ld32(tm_o[m] + lane_off + d, reinterpret_cast<uint32_t *>(o));
          tc::wait_ld();
          if (any_hurt) {
            for (int e = 0; e < 8; ++e)
              for (uint32_t bits = hurt[e >> 2][e & 3]; bits; bits &= bits - 1) {
                const int j = 32 * e + __ffs(bits) - 1;
                const uint16_t *v = p.vd + ((((int64_t)p.layer * p.Hkv + u.g) * p.B + u.b) * p.N + j) * D + d;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float f = __uint_as_float((uint32_t)v[i] << 16);
                  if (!isfinite(f)) o[i] += f;
                }
              }
          }
          if (live && whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              to[(d + i) / 8] = make_uint4(pack_bf16x2(o[i] * inv, o[i + 1] * inv),
                                           pack_bf16x2(o[i + 2] * inv, o[i + 3] * inv),
                                           pack_bf16x2(o[i + 4] * inv, o[i + 5] * inv),
                                           pack_bf16x2(o[i + 6] * inv, o[i + 7] * inv));
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) part[(d + i) * (MT * kTile)] = o[i];
          }
        }
        if (!whole && live && half == 0) {
          part[D * (MT * kTile)] = mr;
          part[(D + 1) * (MT * kTile)] = l;
        }
      }
      tc::fence_before();
      dev::mbar_arrive(&c.o_free[m]);
      if (!whole) {  // reported once all threads have stored it
        const int64_t from = (int64_t)w0 + x - (u.k1 - u.k0) - u.k0, to = from + u.K;  // the unit's tiles
        TreePart &t = todo[pending++];
        t.b = u.b;
        t.head0 = u.g * p.G;
        t.node0 = u.mg * MT * per;
        t.n = u.n;
        t.first = (int32_t)(((from + 1) * ctas + total - 1) / total) - 1;
        t.last = (int32_t)((to * ctas + total - 1) / total) - 1;
        __threadfence();
        dev::named_barrier(1, ALL);
        if (kid == 0) atomicAdd(p.arrived + t.first * kArriveStride, 1);
      }
    }
    // ---------------------------------------------------------------- merge
    for (int k = 0; k < pending; ++k) {
      const TreePart t = todo[k];
      const int parts = t.last - t.first + 1;
      int32_t *arrived = p.arrived + t.first * kArriveStride;
      if (kid == 0) {
        int32_t seen = 0;
        for (uint32_t i = 0; i < 3000000u && seen < parts; ++i) {
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(arrived) : "memory");
          if (*reinterpret_cast<volatile int32_t *>(&c.abort)) break;
        }
        if (seen < parts) dev::set_error(p.err, TRIA_DEVERR_TIMEOUT);
      }
      dev::named_barrier(1, ALL);
      // its items (32 rows by some output dims) over the warps of the unit's CTAs
      const int rank = (cta - t.first) * (ALL / 32) + (kid >> 5);
      // Few dims and many parts at a time, or many dims and few parts; both for all units, us against
      // this rule's: 17 parts of 2048 keys 16.5, 19.1 against 16.5; 16 x 2.1K keys, units over
      // one to three CTAs, 63.3, 57.8 against 55.5; 32 nodes over 32768 keys 47.6, 51.3 against 46.6;
      // 4 x 32 nodes over 8192 keys, units over five or six CTAs, 68.5, 67.5 against 69.7.
      if (parts > 4) merge_items<D, ROWS, MT == 2 ? 8 : 4, MT == 2 ? 8 : 10>(p, t, rank, parts * (ALL / 32));
      else merge_items<D, ROWS, 16, 4>(p, t, rank, parts * (ALL / 32));
      // the last of the unit's CTAs to be done leaves the counter at zero
      if (kid == 0 && atomicAdd(arrived, 1) == 2 * parts - 1) atomicExch(arrived, 0);
    }
  }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 1) tc::tmem_free<512>(tmem);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, []() {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return encode;
}

// bf16 [z][y][D], boxes of 64 columns x by x bz.
bool map_3d(CUtensorMap *map, const void *base, int D, int64_t y, int64_t z, int by, int bz) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)(y > 0 ? y : 1), (cuuint64_t)z};  // (an empty cache is not read)
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * (cuuint64_t)y};
  const cuuint32_t box[3] = {64, (cuuint32_t)by, (cuuint32_t)bz};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
                estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// M tiles per unit: two as soon as one does not hold the tree's rows (K and V are then read
// once for 256 rows), but for D = 256, whose accumulator fills tensor memory.  By the tree's
// capacity, as the host does not know the nodes.  Two and one M tile per unit, us: 255 tokens
// over 4 x 4K..9K keys, 8 heads per KV head, D = 128 311 and 316, D = 64 250 and 267; 64 x 200 nodes, one head
// per KV head 199 and 217; 4 x 32 nodes of 8 heads over 100..300 keys 22.6 and 25.8; 64 nodes of 4 heads
// over 2048 keys 21.2 and 25.8, over 32768 62.1 and 62.1.  One is faster where few units have long
// keys: 4 x 32 nodes of 8 heads over 8192 keys 70.8 and 67.7, over 2048 44.2 and 34.6.
int m_tiles(int D, int G, int N) { return D < 256 && N * G > kTile ? 2 : 1; }

template <int D, int MT>
cudaError_t launch(const TreeAttnParams &p, int ctas, cudaStream_t s) {
  auto kern = tree_attention_kernel<D, MT>;
  constexpr int smem = tree_smem<D, MT>();
  static_assert(smem <= 227 * 1024, "shared memory");
  static bool set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(TreeShape<D, MT>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // CTAs wait for one another
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

size_t tree_attention_scratch(int D, int G, int N) {
  return (size_t)device_sm_count() * kPartSlots * (size_t)(m_tiles(D, G, N) * kTile) * (D + 2) * sizeof(float);
}

cudaError_t launch_tree_attention(const TreeAttnParams &params, cudaStream_t s) {
  TreeAttnParams p = params;
  const int mt = m_tiles(p.D, p.G, p.N);
  // the most tiles that there can be: all segments full
  int64_t most = 0;
  for (int b = 0; b < p.B; ++b)
    most += (p.seg_start[b + 1] - p.seg_start[b] + kTile - 1) / kTile + (p.N + kTile - 1) / kTile;
  most *= (int64_t)p.Hkv * ((p.N * p.G + mt * kTile - 1) / (mt * kTile));
  const int64_t heads = (int64_t)p.L * p.Hkv;
  if (most > INT32_MAX || p.cap > INT32_MAX || heads * p.B > INT32_MAX) return cudaErrorNotSupported;
  if (most == 0) return cudaSuccess;
  p.draft_rows = p.N < kTile ? p.N : kTile;
  const int rows = p.pages.table && p.pages.shift < 7 ? 1 << p.pages.shift : kTile;
  if (!map_3d(&p.tk, p.k, p.D, p.cap, heads, rows, 1) || !map_3d(&p.tv, p.v, p.D, p.cap, heads, rows, 1) ||
      !map_3d(&p.tkd, p.kd, p.D, p.N, heads * p.B, p.draft_rows, 1) ||
      !map_3d(&p.tvd, p.vd, p.D, p.N, heads * p.B, p.draft_rows, 1) ||
      !map_3d(&p.tq, p.q, p.D, p.Hq, (int64_t)p.B * p.N, p.G, kTile / p.G))
    return cudaErrorInvalidValue;
  const int sms = device_sm_count(), ctas = (int)(most < sms ? most : sms);
  if (p.D == 64) return mt == 2 ? launch<64, 2>(p, ctas, s) : launch<64, 1>(p, ctas, s);
  if (p.D == 128) return mt == 2 ? launch<128, 2>(p, ctas, s) : launch<128, 1>(p, ctas, s);
  return launch<256, 1>(p, ctas, s);
}

}  // namespace tria
