// Eviction from private caches by accumulated attention weight.
//
// evict_select_kernel finds, per (request, mass head) row, the n_keep best slots
// of the order (rank desc, slot asc) and where each of them goes.  A row is
// spread over a cluster of 1 to 8 blocks; each reads its slice of masses and
// positions once and keeps the slice's 32-bit ranking keys in shared memory, so
// the three digit passes (11, 11, 10 bits) of the search for the n_keep-th key
// run on chip: per pass the blocks exchange a histogram through distributed
// shared memory.  What stays is then a bitmap; the rows behind the new length
// that stay ("late") and the freed slots before it ("holes") are ranked by
// warp-wide prefix counts and paired, late row i with hole i.  Bound: 8 bytes
// read per slot, 12 written per kept slot.
//
// evict_move_kernel copies the rows of the planes: late rows and holes are
// disjoint, so it needs no order.  Bound: each moved row read and written once.
#include <cooperative_groups.h>

#include <algorithm>

#include "internal.h"

namespace idx {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kSelWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 49152;  // keys of one block: 192 KB of shared memory

struct EvictArgs {
  evict_problem p;
  int32_t* src;
  int32_t* out_len;
  int32_t* out_pos;
  float* out_mass;
  int64_t out_stride;
  int slice_max;  // keys that a block has room for
};

struct SelShared {
  alignas(16) uint32_t hist[2][kBins];  // read four bins at a time
  uint32_t bitmap[kMaxSlice / 32];
  uint32_t wcount[kSelWarps];
  uint32_t wcount2[kSelWarps];
  uint32_t scan[kSelWarps];
  uint32_t found_bin, found_above;
  uint32_t ties, late, holes;  // this block's counts, read by the cluster
};

__device__ __forceinline__ uint32_t rank_key(float m, bool guard) {
  if (guard) return score_key(INFINITY);
  if (m != m) m = -INFINITY;
  return score_key(m);
}

// Exclusive sum of one value per warp (lane 0's), and their total.
__device__ __forceinline__ uint32_t warps_before(const uint32_t* count, int warp, uint32_t* total) {
  uint32_t before = 0, all = 0;
  for (int w = 0; w < kSelWarps; w++) {
    const uint32_t c = count[w];
    if (w < warp) before += c;
    all += c;
  }
  *total = all;
  return before;
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];  // [slice_max]; later the late rows' slots
  grid_let_next_start();
  __shared__ SelShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const evict_problem& p = a.p;
  const int C = (int)cl.num_blocks(), c = (int)cl.block_rank();
  const int64_t row = blockIdx.x / C;
  const int b = (int)(row / p.mass_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int n = p.len[row];
  if (n < 0 || n > p.S) {
    if (tid == 0) atomicOr(&g_device_error, DEVERR_BAD_ROW);
    n = 0;
  }
  const int keep = (int)min((int64_t)p.n_keep, p.S);
  const int nk = min(n, keep);
  const float* mass = p.mass + row * p.stride;
  const int32_t* pos = p.pos ? p.pos + row * p.stride : nullptr;
  int32_t* src = a.src + row * p.n_keep;
  int32_t* opos = a.out_pos ? a.out_pos + row * a.out_stride : nullptr;
  float* omass = a.out_mass ? a.out_mass + row * a.out_stride : nullptr;
  const bool trim = n > keep;

  // this block's slots [s0, s1), a multiple of 32 but for the last
  const int slice = ((n + C - 1) / C + 31) & ~31;
  const int s0 = min(n, slice * c), s1 = min(n, s0 + slice);
  const int cnt = s1 - s0;
  const int words = (cnt + 31) >> 5;
  // a warp's words [w0, w1) for the ordered passes
  const int wper = (words + kSelWarps - 1) / kSelWarps;
  const int w0 = min(words, warp * wper), w1 = min(words, w0 + wper);

  uint32_t before_late = 0, before_holes = 0;
  if (trim) {
    for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = sh.hist[1][i] = 0;
    __syncthreads();
    const int64_t cur = p.cur ? p.cur[b] : n;
    for (int i = tid; i < cnt; i += kThreads) {
      const int s = s0 + i;
      const int64_t at = pos ? pos[s] : s;
      const uint32_t k = rank_key(mass[s], at < p.n_first || at >= cur - p.n_last);
      keys[i] = k;
      atomicAdd(&sh.hist[0][k >> 21], 1u);
    }
    // digits from the top: after each, `prefix` holds the found digits and
    // `need` how many keys of that prefix stay
    uint32_t prefix = 0, need = (uint32_t)keep;
#pragma unroll
    for (int pass = 0; pass < 3; pass++) {
      uint32_t* hist = sh.hist[pass & 1];
      if (pass > 0) {
        const int shift = pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 1 ? 2047u : 1023u;
        const int top = pass == 1 ? 21 : 10;
        for (int i = tid; i < cnt; i += kThreads) {
          const uint32_t k = keys[i];
          if ((k >> top) == (prefix >> top)) atomicAdd(&hist[(k >> shift) & mask], 1u);
        }
      }
      cl.sync();
      // the cluster's histogram, four bins a thread, largest bin first
      uint32_t v[4], mine = 0;
      const int b0 = kBins - 4 * (tid + 1);
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] = 0;
      for (int r = 0; r < C; r++) {
        const uint4 x = *reinterpret_cast<const uint4*>(cl.map_shared_rank(hist, r) + b0);
        v[0] += x.x;
        v[1] += x.y;
        v[2] += x.z;
        v[3] += x.w;
      }
      mine = v[0] + v[1] + v[2] + v[3];
      uint32_t incl = mine;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += y;
      }
      if (lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      uint32_t all;
      uint32_t above = warps_before(sh.scan, warp, &all) + incl - mine;
      if (above < need && need <= above + mine) {
#pragma unroll
        for (int j = 3; j >= 0; j--) {
          if (above < need && need <= above + v[j]) {
            sh.found_bin = b0 + j;
            sh.found_above = above;
          }
          above += v[j];
        }
      }
      // every block has read hist[(pass - 1) & 1] before this pass's cluster
      // barrier: it can be cleared for the next pass
      if (pass == 1)
        for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = 0;
      __syncthreads();
      need -= sh.found_above;
      prefix |= sh.found_bin << (pass == 0 ? 21 : pass == 1 ? 10 : 0);
    }
    // ties of the last kept key: the lowest slots stay
    uint32_t t = 0;
    for (int w = w0; w < w1; w++) {
      const int i = w * 32 + lane;
      t += __popc(__ballot_sync(0xffffffffu, i < cnt && keys[i] == prefix));
    }
    if (lane == 0) sh.wcount[warp] = t;
    __syncthreads();
    uint32_t total;
    uint32_t tie = warps_before(sh.wcount, warp, &total);
    if (tid == 0) sh.ties = total;
    cl.sync();
    for (int r = 0; r < c; r++) tie += *cl.map_shared_rank(&sh.ties, r);
    uint32_t late = 0, holes = 0;
    for (int w = w0; w < w1; w++) {
      const int i = w * 32 + lane;
      const uint32_t k = i < cnt ? keys[i] : 0;
      const bool eq = i < cnt && k == prefix;
      const unsigned eqs = __ballot_sync(0xffffffffu, eq);
      const bool stay = i < cnt && (k > prefix || (eq && tie + __popc(eqs & ((1u << lane) - 1)) < need));
      tie += __popc(eqs);
      const unsigned word = __ballot_sync(0xffffffffu, stay);
      late += __popc(__ballot_sync(0xffffffffu, stay && s0 + i >= nk));
      holes += __popc(__ballot_sync(0xffffffffu, i < cnt && !stay && s0 + i < nk));
      if (lane == 0) sh.bitmap[w] = word;
    }
    if (lane == 0) {
      sh.wcount[warp] = late;
      sh.wcount2[warp] = holes;
    }
    __syncthreads();  // the keys are read, the bitmap is whole: the late rows' slots take the keys' place
    uint32_t all_late, all_holes;
    before_late = warps_before(sh.wcount, warp, &all_late);
    before_holes = warps_before(sh.wcount2, warp, &all_holes);
    if (tid == 0) {
      sh.late = all_late;
      sh.holes = all_holes;
    }
    uint32_t at = before_late;
    for (int w = w0; w < w1; w++) {
      const int i = w * 32 + lane;
      const bool is = i < cnt && s0 + i >= nk && ((sh.bitmap[w] >> lane) & 1);
      const unsigned m = __ballot_sync(0xffffffffu, is);
      if (is) keys[at + __popc(m & ((1u << lane) - 1))] = (uint32_t)(s0 + i);
      at += __popc(m);
    }
    cl.sync();
    for (int r = 0; r < c; r++) before_holes += *cl.map_shared_rank(&sh.holes, r);
  }

  // where each new slot comes from
  for (int w = w0; w < w1; w++) {
    const int i = w * 32 + lane;
    const int s = s0 + i;
    if (s0 + w * 32 >= nk) break;
    const bool in = i < cnt && s < nk;
    const bool hole = in && trim && !((sh.bitmap[w] >> lane) & 1);
    const unsigned m = __ballot_sync(0xffffffffu, hole);
    int from = s;
    if (hole) {
      uint32_t r = before_holes + __popc(m & ((1u << lane) - 1));
      int q = 0;
      while (q < C - 1) {
        const uint32_t l = *cl.map_shared_rank(&sh.late, q);
        if (r < l) break;
        r -= l;
        q++;
      }
      from = (int)*cl.map_shared_rank(keys + r, q);
    }
    before_holes += __popc(m);
    if (in) {
      src[s] = from;
      if (opos) opos[s] = pos ? pos[from] : from;
      if (omass) omass[s] = mass[from];
    }
  }
  for (int64_t s = nk + (int64_t)c * kThreads + tid; s < p.n_keep; s += (int64_t)C * kThreads) {
    src[s] = -1;
    if (opos) opos[s] = -1;
    if (omass) omass[s] = 0.f;
  }
  cl.sync();  // nobody reads this block's shared memory or the late rows' masses any more
  if (trim) {
    // outputs in place: the slots that the row no longer has start afresh
    const bool clear_pos = opos && opos == pos, clear_mass = omass && omass == mass;
    if (clear_pos || clear_mass)
      for (int s = max(s0, nk) + tid; s < s1; s += kThreads) {
        if (clear_pos) opos[s] = -1;
        if (clear_mass) omass[s] = 0.f;
      }
  }
  if (c == 0 && tid == 0 && a.out_len) a.out_len[row] = nk;
}

// ------------------------------------------------------------------- moves --
constexpr int kMoveThreads = 256;
constexpr int kMoveSlots = 256;  // new slots that a block looks at

struct MoveArgs {
  const int32_t* src;  // [B, mass_heads, n_keep]
  int64_t n_keep;
  int mass_heads, n_planes;
  evict_plane plane[IDX_MAX_PLANES];
  int first[IDX_MAX_PLANES + 1];  // of the grid's y axis: plane i's heads start here
};

template <class V>
__device__ __forceinline__ void move_rows(const int2* list, int n, char* base, int64_t ss, int64_t row_bytes) {
  const int per = (int)(row_bytes / (int64_t)sizeof(V));  // vectors of a row
  const int64_t all = (int64_t)n * per;
  constexpr int U = 4;
  for (int64_t i0 = threadIdx.x; i0 < all; i0 += (int64_t)U * kMoveThreads) {
    V x[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t i = i0 + (int64_t)u * kMoveThreads;
      if (i < all) x[u] = reinterpret_cast<const V*>(base + list[i / per].y * ss)[i % per];
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t i = i0 + (int64_t)u * kMoveThreads;
      if (i < all) reinterpret_cast<V*>(base + list[i / per].x * ss)[i % per] = x[u];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ MoveArgs a) {
  __shared__ int2 list[kMoveSlots];  // (new slot, slot it comes from)
  __shared__ int count;
  int pl = 0;
  while (pl + 1 < a.n_planes && (int)blockIdx.y >= a.first[pl + 1]) pl++;
  const evict_plane& q = a.plane[pl];
  const int64_t chunks = (a.n_keep + kMoveSlots - 1) / kMoveSlots;
  const int64_t row = blockIdx.x / chunks;
  const int64_t s = (blockIdx.x % chunks) * kMoveSlots + threadIdx.x;
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  grid_wait();
  const int from = s < a.n_keep ? a.src[row * a.n_keep + s] : -1;
  const bool moves = from >= 0 && from != s;
  const unsigned m = __ballot_sync(0xffffffffu, moves);
  int at = 0;
  if ((threadIdx.x & 31) == 0 && m) at = atomicAdd(&count, __popc(m));
  at = __shfl_sync(0xffffffffu, at, 0);
  if (moves) list[at + __popc(m & ((1u << (threadIdx.x & 31)) - 1))] = make_int2((int)s, from);
  __syncthreads();
  const int n = count;
  if (n == 0) return;
  const int64_t b = row / a.mass_heads;
  const int h = a.mass_heads == 1 ? (int)blockIdx.y - a.first[pl] : (int)(row % a.mass_heads);
  char* base = (char*)q.base + b * q.stride_b + h * q.stride_h;
  switch (q.reserved) {  // widest access that the plane's addresses allow
    case 16: move_rows<uint4>(list, n, base, q.stride_s, q.row_bytes); break;
    case 8: move_rows<uint2>(list, n, base, q.stride_s, q.row_bytes); break;
    case 4: move_rows<uint32_t>(list, n, base, q.stride_s, q.row_bytes); break;
    case 2: move_rows<uint16_t>(list, n, base, q.stride_s, q.row_bytes); break;
    default: move_rows<uint8_t>(list, n, base, q.stride_s, q.row_bytes); break;
  }
}

}  // namespace

int64_t evict_max_slots() { return (int64_t)kMaxCluster * kMaxSlice; }

cudaError_t launch_evict(const evict_problem& p, int32_t* src, int32_t* out_len, int32_t* out_pos, float* out_mass,
                         int64_t out_stride, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.mass_heads;
  EvictArgs a{p, src, out_len, out_pos, out_mass, out_stride, 0};
  // blocks of a row: as many as its keys need, more while the rows leave SMs
  // idle and a block still has a few thousand keys
  int C = 1;
  while (C < kMaxCluster && (p.S > (int64_t)C * kMaxSlice || (rows * C < sm_count() && p.S > (int64_t)C * 4096))) C *= 2;
  a.slice_max = (int)(((p.S + C - 1) / C + 31) & ~int64_t(31));
  const size_t smem = (size_t)std::max(a.slice_max, 32) * 4;
  static KernelReady ready;
  cudaError_t e = ready.once([] {
    return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSlice * 4);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
  if (e != cudaSuccess || p.n_planes == 0) return e;

  MoveArgs m{};
  m.src = src;
  m.n_keep = p.n_keep;
  m.mass_heads = p.mass_heads;
  for (int i = 0; i < p.n_planes; i++) {
    evict_plane q = p.planes[i];
    if (q.row_bytes == 0) continue;
    const uint64_t all = (uint64_t)q.base | (uint64_t)q.row_bytes | (uint64_t)q.stride_b | (uint64_t)q.stride_s |
                         (uint64_t)q.stride_h;
    q.reserved = all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
    m.plane[m.n_planes] = q;
    m.first[m.n_planes + 1] = m.first[m.n_planes] + (p.mass_heads == 1 ? q.heads : 1);
    m.n_planes++;
  }
  if (m.n_planes == 0) return cudaSuccess;
  const int64_t chunks = (p.n_keep + kMoveSlots - 1) / kMoveSlots;
  const dim3 grid((unsigned)(rows * chunks), (unsigned)m.first[m.n_planes]);
  return launch_after(evict_move_kernel, grid, kMoveThreads, 0, st, true, m);
}

}  // namespace idx
