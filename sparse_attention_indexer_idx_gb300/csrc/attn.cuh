// Attention of a decode step over a shared prefix and private caches: what its
// kernels have in common (arguments, partial results, row limits).
//
// A row is (request b, token t, query head hq).  Its softmax is computed in
// pieces: each (part of the prefix or of the private cache) leaves the
// unnormalised sum  o = sum 2^(y - m) v  with y = log2(e) scale q.k, its
// maximum m and its sum l = sum 2^(y - m), all fp32; the finish kernel joins a
// row's pieces:  M = max m_i,  out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace idx {

struct AttnArgs {
  attn_problem p;
  float scale_log2;    // scale * log2(e)
  int G;               // query heads of one KV head
  int parts_prefix;    // pieces of a row from the prefix, then from the private cache
  int parts_private;
  float* po;           // [rows, parts, D] unnormalised sums, rows = B*T*Hq
  float2* pml;         // [rows, parts] (m, l); l == 0: the piece is empty and po is not written
  float* sc;           // [rows, sc_ld] private scores y, or NULL
  int64_t sc_ld;
  void* out;
  float* lse;
  float* mass;
  int mass_heads;
};

// Keys of a tile of the streaming kernel.
__host__ __device__ constexpr int stream_tile(int D) { return D == 128 ? 16 : 32; }

// Private slots that token t of request b sees under KV head h.
__device__ __forceinline__ int attn_len(const attn_problem& p, int b, int h) {
  if (!p.len) return 0;
  int n = p.len[p.len_per_head ? (int64_t)b * p.n_kv + h : b];
  if (n < 0 || n > p.S) {
    atomicOr(&g_device_error, DEVERR_BAD_ROW);
    n = 0;
  }
  return n;
}
__device__ __forceinline__ int64_t attn_prefix_len(const attn_problem& p, int b) {
  if (!p.prefix_len) return p.P;
  int n = p.prefix_len[b];
  if (n < 0 || n > p.P) {
    atomicOr(&g_device_error, DEVERR_BAD_ROW);
    n = 0;
  }
  return n;
}

// Units of request b's cache on the streaming kernel's line: by its longest
// head, at least one, so that every sequence has a place.
__device__ __forceinline__ int cache_units(const attn_problem& p, int b, int unit_shift) {
  int n = 0;
  for (int h = 0; h < (p.len_per_head ? p.n_kv : 1); h++) {
    const int x = p.len[p.len_per_head ? (int64_t)b * p.n_kv + h : b];
    if (x <= p.S) n = max(n, x);
  }
  return max(1, (n + (1 << unit_shift) - 1) >> unit_shift);
}

__device__ __forceinline__ float attn_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The streaming kernel's line of key units and its cut (see attn_stream.cu).
struct StreamLine {
  bool after;        // the tensor-core kernel comes before: it writes nothing that this one reads
  int unit_shift;    // a unit is 2^unit_shift keys: a tile, two or four
  int row_tile;      // 16 or 32 rows of a warp
  int members;       // warps of a group: KV heads times row tiles
  int groups;
  int prefix_units;  // of the prefix, if its rows need no more row tiles than the caches' do
  int seqs;          // private sequences: requests, or (request, token) lists
  int uniform;       // units that every private sequence counts as, or 0: as many as its length asks
  int least;         // smallest share of a group, so that no sequence has more parts than planned
  // a short prefix under many rows: a line of its own, taken by the first blocks
  int own_blocks, own_members, own_groups, own_units;
};
cudaError_t launch_attn_stream(const AttnArgs& a, const StreamLine& line, cudaStream_t st);
cudaError_t launch_attn_finish(const AttnArgs& a, cudaStream_t st);

}  // namespace idx
