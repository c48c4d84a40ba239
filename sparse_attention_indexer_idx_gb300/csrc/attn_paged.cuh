// Attention over caches in pages: what its kernels have in common.
#pragma once

#include "attn_tc.cuh"

namespace idx {

struct PagedArgs {
  paged_problem p;
  float scale_log2;  // scale * log2(e)
  int G;             // query heads of a KV head
  // Partial results.  The line of sequences is cut into the groups' shares; from one
  // pair of a group and a sequence that meet to the next, either the group or the
  // sequence goes up by one, so the pair (g, s) has place g + s to itself, and there
  // are groups + sequences places however the lengths are.
  int rows;          // of a sequence: T*Hq, or Hq of a list
  float* po;         // [places, rows, D] unnormalised sums
  float2* pml;       // [places, rows] maximum (of log2 units) and sum; sum 0: empty, po is not written
  int2* ends;        // [sequences] first and last group of each
  int box;           // keys of a box (kTiles)
};

struct PagedMaps {
  CUtensorMap m[2];  // keys, values (kTiles)
};

// The line of key units and its cut.
struct PagedLine {
  int unit_shift;  // a unit is 2^unit_shift keys
  int members;     // warps of a group: KV heads times row tiles
  int groups;
  int seqs;        // requests, or (request, token) lists
  int uniform;     // units that every sequence counts as, or 0: as many as its length asks
  int least;       // smallest share of a group
};

__device__ __forceinline__ int paged_len(const paged_problem& p, int b) {
  const int n = p.len[b];
  if (n >= 0 && n <= p.max_len) return n;
  atomicOr(&g_device_error, DEVERR_BAD_ROW);
  return 0;
}
__device__ __forceinline__ int units_of(const paged_problem& p, int b, int shift) {
  const int n = p.len[b];
  return n <= p.max_len ? max(1, (n + (1 << shift) - 1) >> shift) : 1;
}

// The scale of the exponents, above zero: a negative one's sign goes into the queries
// (flip), and a scale of zero becomes one that takes every score to zero but leaves
// -inf alone.
__device__ __forceinline__ float scale_of(const PagedArgs& a) { return fmaxf(fabsf(a.scale_log2), 0x1p-149f); }
__device__ __forceinline__ uint32_t flip_of(const PagedArgs& a) { return a.scale_log2 < 0.f ? 0x80008000u : 0u; }

// Weights are lifted, 2^(y - m + kLift): as fp16 they reach down to 2^-14 before they
// lose bits, up to 2^16 at most, and sums, outputs and the join's factors scale alike.
// bf16 has fp32's range and needs none of it.  (Without it, fp16 weights below 2^-25 of
// a warp's largest were 0 in the product and yet in the sum that divides it: 4 % of a
// row of 30,000 weights of 2^-27 got lost.)
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 15.f;
// lse in log2 units, from a maximum and a sum of lifted weights.
template <bool BF16>
__device__ __forceinline__ float log2_sum(float m, float sum) {
  return m + log2f(sum * (BF16 ? 1.f : 0x1p-15f));
}

// Rows beyond 16 over long caches, on the 5th-generation tensor cores.
cudaError_t launch_attn_paged_tc(const PagedArgs& a, const PagedMaps& maps, const PagedLine& line, cudaStream_t st);
// Joins the places of every row.
cudaError_t launch_attn_paged_join(const PagedArgs& a, int seqs, int groups, void* out, float* lse, cudaStream_t st);

}  // namespace idx
