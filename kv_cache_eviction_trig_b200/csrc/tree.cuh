// Speculative decoding over the cache: attention of drafted trees, the commit of their accepted
// paths, and the block tables of a paged cache (which the prune does not take).
#pragma once

#include "tria_internal.cuh"

namespace tria {

// Where a sequence's tokens live: in its segment, or in the blocks of its table row.
struct PageParams {
  const int32_t *table;     // [B][max_blocks], or null: segments
  int32_t max_blocks, n_blocks;
  int32_t shift;            // log2 of the block size
};

struct BlockTablesParams {
  int32_t *table;           // [B][max_blocks]
  int32_t *held;            // [B]
  int32_t *ring;            // [n_blocks]
  int32_t *ring_state;      // [2] head, free
  const int32_t *seq_len;   // [B]
  const int32_t *n_new;     // [B]
  int32_t *slot_map;        // [B][max_new]
  int32_t *err;
  int32_t B, max_new, max_blocks, n_blocks, shift;
  int32_t seg_cap[TRIA_MAX_BATCH];
};
cudaError_t launch_block_tables(const BlockTablesParams &p, cudaStream_t s);

struct TreeCommitParams {
  const int32_t *parent;    // [B][N]
  const int32_t *n_nodes;   // [B]
  const int32_t *last;      // [B]
  const int32_t *slot_map;  // [B][max_new], or null: segments
  const uint8_t *k_new;     // bf16 [L][Hkv][B][N][D]
  const uint8_t *v_new;
  uint8_t *k;               // bf16 [L][Hkv][cap][D]
  uint8_t *v;
  int32_t *pos;             // [L][Hkv][cap]
  int32_t *seq_len;         // [B]
  int32_t *unit_len;        // [L][Hkv][B] per-unit lengths (instead of seq_len), or null
  int32_t *cur_pos;         // [B]
  int32_t *arrived;         // [B] blocks that are done with a sequence, zero at rest
  int32_t *err;
  int64_t cap;
  int32_t L, Hkv, B, D, N, max_new, lg_per_block;
  int64_t seg_start[TRIA_MAX_BATCH + 1];
};
cudaError_t launch_tree_commit(const TreeCommitParams &params, cudaStream_t s);

struct alignas(64) TreeAttnParams {
  CUtensorMap tk, tv;       // K and V as [L*Hkv][cap][D], boxes of 64 columns x 128 rows (or a block)
  CUtensorMap tkd, tvd;     // the nodes' as [L*Hkv*B][N][D], boxes of 64 x draft_rows
  CUtensorMap tq;           // the queries as [B*N][Hq][D], boxes of 64 x G heads x 128 / G nodes
  float *scratch;           // two parts per CTA: unnormalised output [D][rows], maxima, sums
  int32_t *arrived;         // per CTA, a line apart: reports on the unit that starts there; zero at rest
  const int32_t *parent;    // [B][N]
  const int32_t *n_nodes;   // [B]
  const uint16_t *q;        // bf16 [B][N][Hq][D]
  const uint16_t *k;        // bf16 [L][Hkv][cap][D]
  const uint16_t *v;
  const uint16_t *kd;       // bf16 [L][Hkv][B][N][D]
  const uint16_t *vd;
  const int32_t *seq_len;   // [B]
  const int32_t *unit_len;  // [L][Hkv][B] per-unit lengths (instead of seq_len), or null
  uint16_t *out;            // bf16 [B][N][Hq][D]
  int32_t *err;
  PageParams pages;
  int64_t cap;
  int32_t layer, L, B, N, Hkv, Hq, G, D, draft_rows;
  float scale;
  int64_t seg_start[TRIA_MAX_BATCH + 1];
};
// The tensor maps and what depends on the launch are filled in here; scratch holds
// tree_attention_scratch bytes.
cudaError_t launch_tree_attention(const TreeAttnParams &params, cudaStream_t s);
size_t tree_attention_scratch(int D, int G, int N);

}  // namespace tria
