// Attention over caches in pages, last step: the partial results of each row joined.
//
// With pieces (m_i, l_i, o_i):  M = max m_i,  out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
// A row's pieces are the places of its sequence, from its first group's to its last
// one's.  A warp has a row, two to eight where a sequence has many pieces and the rows
// leave warps free; it loads eight pieces' sums before it adds them.  Bound by the
// chain of loads, from the ends to (m, l) to the sums: 3 to 6 us behind the kernel
// before it.
#include "attn_mma.cuh"
#include "attn_paged.cuh"

#include <algorithm>

namespace idx {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) attn_paged_join_kernel(const __grid_constant__ PagedArgs a, int seqs, int groups,
                                                                    int share, void* out, float* lse) {
  __shared__ float s_acc[kWarps][D];
  __shared__ float2 s_ml[kWarps];
  grid_wait();
  grid_let_next_start();
  constexpr int E = D / 32;  // elements of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % share;
  const int64_t r = (int64_t)blockIdx.x * (kWarps / share) + warp / share, rows = (int64_t)seqs * a.rows;
  int64_t at = 0;  // of the warp's first piece; the next one is a.rows further on
  int n = 0;
  if (r < rows) {
    const int seq = (int)(r / a.rows);
    const int2 ends = a.ends[seq];
    // (a kernel whose waits gave up may not have written them)
    const bool there = ends.x >= 0 && ends.x <= ends.y && ends.y < groups;
    const int all = there ? ends.y - ends.x + 1 : 0, each = (all + share - 1) / share, first = min(all, sub * each);
    n = min(each, all - first);
    at = (int64_t)((there ? ends.x : 0) + first + seq) * a.rows + (r - (int64_t)seq * a.rows);
  }
  float top = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; e++) acc[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    // lane i has piece i0 + i; a piece is empty where its sum is 0, and only there
    const float2 x = i0 + lane < n ? a.pml[at + (int64_t)(i0 + lane) * a.rows] : make_float2(-INFINITY, 0.f);
    float most = x.y != 0.f ? x.x : -INFINITY;
#pragma unroll
    for (int s = 16; s; s >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
    most = fmaxf(most, top);
    const float base = most == -INFINITY ? 0.f : most, scale = attn_ex2(top - base);
    top = most;
    const float w = x.y != 0.f ? attn_ex2(x.x - base) : 0.f;
    l = l * scale + w * x.y;
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] *= scale;
    unsigned some = __ballot_sync(0xffffffffu, w != 0.f);  // the others' sums count nothing, or are not there
    while (some) {
      constexpr int U = 8;
      float v[U][E], wi[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int i = some ? __ffs(some) - 1 : -1;
        some &= some - 1;
        wi[u] = __shfl_sync(0xffffffffu, w, i < 0 ? 0 : i);
        if (i < 0) wi[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; e++) v[u][e] = 0.f;
        if (i >= 0) {
          const float* o = a.po + (at + (int64_t)(i0 + i) * a.rows) * D + lane * E;
          if constexpr (E == 4)
            *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(o);
          else
            *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(o);
        }
      }
#pragma unroll
      for (int u = 0; u < U; u++)
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] += wi[u] * v[u][e];
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  if (share > 1) {
#pragma unroll
    for (int e = 0; e < E; e++) s_acc[warp][lane * E + e] = acc[e];
    if (lane == 0) s_ml[warp] = make_float2(top, l);
    __syncthreads();
    if (sub) return;
    for (int i = 0; i < share; i++)
      if (s_ml[warp + i].y != 0.f) top = fmaxf(top, s_ml[warp + i].x);
    const float base = top == -INFINITY ? 0.f : top;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] = 0.f;
    for (int i = 0; i < share; i++) {
      const float2 x = s_ml[warp + i];
      const float w = x.y != 0.f ? attn_ex2(x.x - base) : 0.f;
      l += w * x.y;
#pragma unroll
      for (int e = 0; e < E; e++) acc[e] += w * s_acc[warp + i][lane * E + e];
    }
  }
  if (r >= rows) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  uint32_t* to = reinterpret_cast<uint32_t*>(out) + (r * D + lane * E) / 2;
#pragma unroll
  for (int e = 0; e < E / 2; e++) to[e] = pack2<BF16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (lane == 0 && lse) lse[r] = l != 0.f ? log2_sum<BF16>(top, l) * 0.693147180559945309f : -INFINITY;
}

template <int D, bool BF16>
cudaError_t launch(const PagedArgs& a, int seqs, int groups, void* out, float* lse, cudaStream_t st) {
  const int64_t rows = (int64_t)seqs * a.rows;
  int share = 1;
  while (share < kWarps && groups / seqs > 16 * share && rows * share < 8 * sm_count()) share *= 2;
  const int64_t blocks = (rows * share + kWarps - 1) / kWarps;
  return launch_early(attn_paged_join_kernel<D, BF16>, dim3((unsigned)blocks), kThreads, 0, st, a, seqs, groups, share, out, lse);
}

}  // namespace

cudaError_t launch_attn_paged_join(const PagedArgs& a, int seqs, int groups, void* out, float* lse, cudaStream_t st) {
  const bool bf = a.p.dtype == IDX_BF16;
  if (a.p.D == 128) return bf ? launch<128, true>(a, seqs, groups, out, lse, st) : launch<128, false>(a, seqs, groups, out, lse, st);
  return bf ? launch<64, true>(a, seqs, groups, out, lse, st) : launch<64, false>(a, seqs, groups, out, lse, st);
}

}  // namespace idx
