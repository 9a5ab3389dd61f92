// kda_lin_tc.cuh -- work items and workspace of the tensor-core prompts of the
// linear attention with a decay for each head.
#pragma once

#include "kda_attn_tc.cuh"
#include "kda_lin.cuh"

namespace kda {

constexpr int kLinChunk = 128;  // tokens of a chunk: the rows of a tensor-core tile

// One chain: tokens [tok0, tok0 + len) of a head's columns [tile * DV, ...).
// from, to: the state it starts from and leaves, a place of the workspace's
// states (>= 0), row -2 - x of the pool (<= -2), or none (-1).
struct LinItem {
  int32_t tok0, len, head, tile, from, to;
};

struct LinTcArgs {
  const LinItem* items;    // null: CTA b takes chain b of sequence, head, tile
  const int32_t* num_items;
  float* states;           // [places][H][dk][dv]
  int32_t tiles;           // column tiles of a head
  int32_t o_wide;          // o is 32-byte aligned
};

}  // namespace kda
