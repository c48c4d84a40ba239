// The tensor-core kernel of the shared prefix: its arguments.
#pragma once

#include <cuda.h>

#include "attn.cuh"

namespace idx {

struct AttnTcArgs {
  AttnArgs a;
  int row_tiles;     // pairs of 128-row tiles of a KV head
  int cells_k;       // pieces of the keys
  int blocks;        // grid
  bool whole_cells;  // a block takes one (KV head, piece, row tile pair) instead of an even share of the key tiles
};

bool make_tmap_3d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t rows,
                  uint64_t planes, uint64_t row_bytes, uint64_t plane_bytes, uint32_t box_inner, uint32_t box_rows);
cudaError_t launch_attn_tc(const AttnTcArgs& t, cudaStream_t st);

}  // namespace idx
