// Eviction from private caches by accumulated attention weight.
//
// evict_select_kernel finds, per (request, mass head) row, the n_keep best slots
// of the order (rank desc, slot asc) and where each of them goes.  A row is
// spread over a cluster of 1 to 8 blocks; each reads its slice of masses and
// positions once and keeps the slice's 32-bit ranking keys in shared memory, so
// the three digit passes (11, 11, 10 bits) of the search for the n_keep-th key
// run on chip: per pass the blocks look up the counts of 64 groups of bins, then
// of one group's bins, in one another's shared memory.  What stays is then a
// bitmap; the rows behind the new length that stay ("late") and the freed slots
// before it ("holes") are ranked by warp-wide prefix counts and paired, late row
// i with hole i.
//
// The bytes (8 read per slot, 12 written per kept slot) are little; what bounds
// it is the chain of steps that wait for one another: loads, three passes of two
// barriers each, counts, late rows, new slots.  8 rows of 1,040 slots take 6.6
// us, 512 rows of 4,160 (a block each, 3.4 to an SM) 18 us, 96 rows of 10,007
// (two blocks each) 18.5 us, 4 rows of 131,072 (eight blocks each) 19 us.
//
// evict_move_kernel copies the rows of the planes: late rows and holes are
// disjoint, so it needs no order.  Bound by each moved row read and written
// once, at rows of 128 or 256 bytes spread over a cache: 55,000 slots of 8
// heads' keys and values and an index key, 256 bytes each (480 MB both ways),
// take 76 us, 6.3 TB/s.
#include <cooperative_groups.h>

#include <algorithm>

#include "internal.h"

namespace idx {

namespace {

namespace cg = cooperative_groups;

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
  bool vec4;  // rows of mass and pos start on 16 bytes
};

struct SelShared {
  alignas(16) uint32_t hist[2][kBins];        // read several bins at a time
  alignas(16) uint32_t coarse[2][kBins / 32];  // sums of 32 bins
  uint32_t wcount[32];
  uint32_t found_bin, found_above, found_count;
  uint32_t ties, late, holes;  // this block's counts, read by the cluster
};

// Words of a slice that a thread of a block of NT has at most.
template <int NT>
constexpr int kMaxWords = (kMaxSlice / 32 + NT - 1) / NT;

__device__ __forceinline__ uint32_t rank_key(float m, bool guard) {
  if (guard) return score_key(INFINITY);
  if (m != m) m = -INFINITY;
  return score_key(m);
}

// The lowest n bits, n clamped to 0..32.
__device__ __forceinline__ unsigned low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }

// Sum of the values of the warps before this one, and of all (a value per
// warp, at most 32).
__device__ __forceinline__ uint32_t warps_before(const uint32_t* count, int warps, int warp, uint32_t* total) {
  const int lane = threadIdx.x & 31;
  const uint32_t v = lane < warps ? count[lane] : 0;
  *total = __reduce_add_sync(0xffffffffu, v);
  return __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
}

// The cluster of a row, or the one block that has it all: there the exchange
// needs no cluster barriers and no distributed addresses.
template <bool ONE>
struct RowGroup {
  __device__ __forceinline__ int blocks() const { return ONE ? 1 : (int)cg::this_cluster().num_blocks(); }
  __device__ __forceinline__ int rank() const { return ONE ? 0 : (int)cg::this_cluster().block_rank(); }
  __device__ __forceinline__ void sync() const {
    if (ONE)
      __syncthreads();
    else
      cg::this_cluster().sync();
  }
  template <class T>
  __device__ __forceinline__ T* at(T* x, int r) const {
    return ONE ? x : cg::this_cluster().map_shared_rank(x, r);
  }
};

// NT threads; each takes U slots, or words of 32 slots, at a time, so that U
// loads are in flight.
template <int NT, bool ONE>
__global__ void __launch_bounds__(NT, 1024 / NT) evict_select_kernel(const __grid_constant__ EvictArgs a, int slice_max) {
  constexpr int W = NT / 32, U = 8;
  // the slice's keys, later the late rows' slots; a bitmap of the slots that
  // stay; and the slice's holes before each word of it
  extern __shared__ __align__(16) uint32_t keys[];
  uint32_t* bitmap = keys + slice_max;
  uint16_t* rank = reinterpret_cast<uint16_t*>(bitmap + slice_max / 32);
  __shared__ SelShared sh;
  grid_wait();
  grid_let_next_start();
  const RowGroup<ONE> cl;
  const evict_problem& p = a.p;
  const int C = cl.blocks(), c = cl.rank();
  const int64_t row = blockIdx.x / (unsigned)C;
  const int b = (int)((unsigned)row / (unsigned)p.mass_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int n = p.len[row];
  const int cur = p.cur ? p.cur[b] : 0;
  for (int i = tid; i < kBins; i += NT) sh.hist[0][i] = sh.hist[1][i] = 0;
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

  if (trim) {
    // positions from here on are protected
    const int recent = (int)max((int64_t)INT32_MIN, (p.cur ? cur : n) - (int64_t)p.n_last);
    __syncthreads();
    auto take = [&](int i, float x, int at) {
      const uint32_t k = rank_key(x, at < p.n_first || at >= recent);
      keys[i] = k;
      atomicAdd(&sh.hist[0][k >> 21], 1u);
    };
    int done = 0;
    if (a.vec4) {  // four slots a load; the slice's start is a multiple of 32
      const int quads = cnt >> 2;
      const float4* m4 = reinterpret_cast<const float4*>(mass + s0);
      const int4* p4 = reinterpret_cast<const int4*>(pos + s0);
      for (int i0 = tid; i0 < quads; i0 += NT * 4) {
        float4 x[4];
        int4 at[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const int i = i0 + u * NT;
          if (i < quads) {
            x[u] = m4[i];
            const int s = s0 + 4 * i;
            at[u] = pos ? p4[i] : make_int4(s, s + 1, s + 2, s + 3);
          }
        }
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const int i = i0 + u * NT;
          if (i < quads) {
            take(4 * i, x[u].x, at[u].x);
            take(4 * i + 1, x[u].y, at[u].y);
            take(4 * i + 2, x[u].z, at[u].z);
            take(4 * i + 3, x[u].w, at[u].w);
          }
        }
      }
      done = quads * 4;
    }
    for (int i0 = done + tid; i0 < cnt; i0 += NT * U) {
      float x[U];
      int at[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int i = i0 + u * NT;
        x[u] = i < cnt ? mass[s0 + i] : 0.f;
        at[u] = i < cnt && pos ? pos[s0 + i] : s0 + i;
      }
#pragma unroll
      for (int u = 0; u < U; u++)
        if (i0 + u * NT < cnt) take(i0 + u * NT, x[u], at[u]);
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
        auto look = [&](uint32_t k) {
          if ((k >> top) == (prefix >> top)) atomicAdd(&hist[(k >> shift) & mask], 1u);
        };
        const uint4* k4 = reinterpret_cast<const uint4*>(keys);
        for (int i = tid; i < cnt >> 2; i += NT) {
          const uint4 k = k4[i];
          look(k.x);
          look(k.y);
          look(k.z);
          look(k.w);
        }
        if (tid < (cnt & 3)) look(keys[(cnt & ~3) + tid]);
      }
      __syncthreads();
      // Sums of 32 bins; then one warp of every block finds the group with the
      // need-th key among all blocks' sums, and its bin among the group's 32 (the
      // whole histograms added up in shares took 2 us longer for blocks of 5,000).
      constexpr int V = kBins / NT;  // bins of a thread: 2 to 8
      uint32_t sum = 0;
#pragma unroll
      for (int j = 0; j < V / 2; j++) {
        const uint2 x = reinterpret_cast<const uint2*>(hist + V * tid)[j];
        sum += x.x + x.y;
      }
#pragma unroll
      for (int d = 1; d < 32 / V; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (tid % (32 / V) == 0) sh.coarse[pass & 1][tid * V / 32] = sum;
      cl.sync();
      if (warp == 0) {
        auto before = [&](uint32_t x) {  // sum over the lanes before this one
          uint32_t incl = x;
#pragma unroll
          for (int s = 1; s < 32; s <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, s);
            if (lane >= s) incl += y;
          }
          return incl - x;
        };
        uint32_t hi = 0, lo = 0;  // groups 63 - 2 lane and 62 - 2 lane: the largest bins first
#pragma unroll
        for (int r = 0; r < (ONE ? 1 : kMaxCluster); r++)
          if (r < C) {
            const uint2 x = reinterpret_cast<const uint2*>(cl.at(sh.coarse[pass & 1], r))[31 - lane];
            lo += x.x;
            hi += x.y;
          }
        uint32_t above = before(hi + lo);
        const bool upper = need <= above + hi;
        const int at = __ffs(__ballot_sync(0xffffffffu, above < need && need <= above + hi + lo)) - 1;
        const int g = __shfl_sync(0xffffffffu, upper ? 63 - 2 * lane : 62 - 2 * lane, at);
        above = __shfl_sync(0xffffffffu, upper ? above : above + hi, at);
        uint32_t v = 0;
#pragma unroll
        for (int r = 0; r < (ONE ? 1 : kMaxCluster); r++)
          if (r < C) v += cl.at(hist, r)[g * 32 + 31 - lane];
        above += before(v);
        if (above < need && need <= above + v) {
          sh.found_bin = g * 32 + 31 - lane;
          sh.found_above = above;
          sh.found_count = v;
        }
      }
      // every block has read hist[0] before the second pass's cluster barrier
      if (pass == 1)
        for (int i = tid; i < kBins; i += NT) sh.hist[0][i] = 0;
      __syncthreads();
      need -= sh.found_above;
      prefix |= sh.found_bin << (pass == 0 ? 21 : pass == 1 ? 10 : 0);
    }
    // A thread forms whole words of 32 slots: those above the last kept key stay,
    // and of those equal to it the lowest.  (Lanes read their words' quads in
    // turn, so that they meet different banks.)
    uint32_t tie = 0;
    const bool all_ties = need == sh.found_count;
    auto word_bits = [&](int w, uint32_t* above, uint32_t* equal) {
      const uint4* k4 = reinterpret_cast<const uint4*>(keys) + w * 8;
      uint32_t gt = 0, eq = 0;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int q = (j + lane) & 7;
        const uint4 k = k4[q];
        gt |= (uint32_t)((k.x > prefix) | (k.y > prefix) << 1 | (k.z > prefix) << 2 | (k.w > prefix) << 3) << (4 * q);
        eq |= (uint32_t)((k.x == prefix) | (k.y == prefix) << 1 | (k.z == prefix) << 2 | (k.w == prefix) << 3) << (4 * q);
      }
      const uint32_t valid = low_bits(cnt - w * 32);
      *above = gt & valid;
      *equal = eq & valid;
    };
    if (!ONE && !all_ties) {
      // ties in the blocks before this one
      uint32_t t = 0;
      for (int w = tid; w < words; w += NT) {
        uint32_t gt, eq;
        word_bits(w, &gt, &eq);
        t += __popc(eq);
      }
      t = __reduce_add_sync(0xffffffffu, t);
      if (lane == 0) sh.wcount[warp] = t;
      __syncthreads();
      uint32_t all;
      warps_before(sh.wcount, W, warp, &all);
      if (tid == 0) sh.ties = all;
      cl.sync();
      for (int r = 0; r < c; r++) tie += *cl.at(&sh.ties, r);
    }
    // sums over the threads before this one; the counts of a slice fit 16 bits
    auto before = [&](uint32_t x, uint32_t* all) {
      uint32_t incl = x;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += y;
      }
      __syncthreads();
      if (lane == 31) sh.wcount[warp] = incl;
      __syncthreads();
      return warps_before(sh.wcount, W, warp, all) + incl - x;
    };
    uint32_t holes_late = 0;  // of the words so far: holes, and late rows in the upper half
    uint32_t mine[kMaxWords<NT>];
    uint32_t at[kMaxWords<NT>];
#pragma unroll
    for (int x = 0; x < kMaxWords<NT>; x++) {
      if (x * NT >= words) break;
      const int w = x * NT + tid;
      uint32_t gt = 0, eq = 0, all;
      if (w < words) word_bits(w, &gt, &eq);
      if (all_ties) {
        gt |= eq;
      } else {
        const uint32_t ahead = tie + before(__popc(eq), &all);
        uint32_t take = ahead >= need ? 0 : need - ahead, low = eq;
        if (take >= (uint32_t)__popc(eq)) {
          gt |= eq;
        } else {
          for (; take; take--) {
            gt |= low & (0u - low);
            low &= low - 1;
          }
        }
        tie += all;
      }
      const uint32_t low = low_bits(nk - (s0 + w * 32)), valid = w < words ? low_bits(cnt - w * 32) : 0u;
      const uint32_t both = __popc(~gt & valid & low) | __popc(gt & ~low) << 16;
      const uint32_t first = holes_late + before(both, &all);
      holes_late += all;
      if (w < words) {
        bitmap[w] = gt;
        rank[w] = (uint16_t)first;
      }
      mine[x] = w < words ? gt & ~low : 0u;
      at[x] = first >> 16;
    }
    if (tid == 0) {
      sh.late = holes_late >> 16;
      sh.holes = holes_late & 0xffff;
    }
    __syncthreads();  // the keys are read: the late rows' slots take their place
#pragma unroll
    for (int x = 0; x < kMaxWords<NT>; x++) {
      if (x * NT >= words) break;
      uint32_t m = mine[x], to = at[x];
      while (m) {
        keys[to++] = (uint32_t)(s0 + (x * NT + tid) * 32 + __ffs(m) - 1);
        m &= m - 1;
      }
    }
    cl.sync();
  }

  // where each new slot comes from: words of 32 new slots in turn over the
  // warps of the whole cluster
  uint32_t holes_of = 0, late_of = 0;  // lane r: holes and late rows of the blocks before block r
  uint32_t late_before[kMaxCluster] = {};
  if (trim && !ONE) {
    uint32_t h = lane < C ? *cl.at(&sh.holes, lane) : 0;
    uint32_t l = lane < C ? *cl.at(&sh.late, lane) : 0;
    holes_of = h;
    late_of = l;
#pragma unroll
    for (int s = 1; s < kMaxCluster; s <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, holes_of, s), y = __shfl_up_sync(0xffffffffu, late_of, s);
      if (lane >= s) {
        holes_of += x;
        late_of += y;
      }
    }
    holes_of -= h;
    late_of -= l;
#pragma unroll
    for (int x = 1; x < kMaxCluster; x++) late_before[x] = x < C ? __shfl_sync(0xffffffffu, late_of, x) : ~0u;
  }
  const int new_words = (nk + 31) >> 5, stride = C * W;
  constexpr int F = 8;
  for (int v0 = c * W + warp; v0 < new_words; v0 += stride * F) {
    int from[F], slot[F];
    // lane u: the holes of word u, and how many come before them in the row
    uint32_t m_l = 0, nth_l = 0;
    if (trim) {
      const int v = min(v0 + (lane % F) * stride, new_words - 1);
      const int q = ONE ? 0 : (int)((uint32_t)(v * 32) / (uint32_t)slice), w = v - q * (slice >> 5);  // its block
      m_l = ~cl.at(bitmap, q)[w] & low_bits(nk - v * 32);
      nth_l = (ONE ? 0 : __shfl_sync(0xffffffffu, holes_of, q)) + cl.at(rank, q)[w];
    }
#pragma unroll
    for (int u = 0; u < F; u++) {
      const int v = v0 + u * stride;
      const int s = v * 32 + lane;
      slot[u] = v < new_words && s < nk ? s : -1;
      from[u] = s;
      const uint32_t m = __shfl_sync(0xffffffffu, m_l, u);
      const uint32_t r = __shfl_sync(0xffffffffu, nth_l, u) + __popc(m & ((1u << lane) - 1));
      if (slot[u] >= 0 && ((m >> lane) & 1)) {
        int z = 0;  // the block that has late row r
        uint32_t first = 0;
        if (!ONE) {
#pragma unroll
          for (int x = 1; x < kMaxCluster; x++)
            if (r >= late_before[x]) {
              z = x;
              first = late_before[x];
            }
        }
        from[u] = (int)*cl.at(keys + (r - first), z);
      }
    }
    int ps[F];
    float ms[F];
#pragma unroll
    for (int u = 0; u < F; u++) {
      ps[u] = slot[u] >= 0 && opos && pos ? pos[from[u]] : from[u];
      ms[u] = slot[u] >= 0 && omass ? mass[from[u]] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < F; u++)
      if (slot[u] >= 0) {
        src[slot[u]] = from[u];
        if (opos) opos[slot[u]] = ps[u];
        if (omass) omass[slot[u]] = ms[u];
      }
  }
  for (int64_t s = nk + (int64_t)c * NT + tid; s < p.n_keep; s += (int64_t)C * NT) {
    src[s] = -1;
    if (opos) opos[s] = -1;
    if (omass) omass[s] = 0.f;
  }
  cl.sync();  // nobody reads this block's shared memory or the late rows' masses any more
  if (trim) {
    // outputs in place: the slots that the row no longer has start afresh
    const bool clear_pos = opos && opos == pos, clear_mass = omass && omass == mass;
    if (clear_pos || clear_mass)
      for (int s = max(s0, nk) + tid; s < s1; s += NT) {
        if (clear_pos) opos[s] = -1;
        if (clear_mass) omass[s] = 0.f;
      }
  }
  if (c == 0 && tid == 0 && a.out_len) a.out_len[row] = nk;
}

// ------------------------------------------------------------------- moves --
constexpr int kMoveThreads = 256;

struct MoveArgs {
  const int32_t* src;  // [B, mass_heads, n_keep]
  int64_t n_keep;
  int mass_heads, n_planes;
  evict_plane plane[IDX_MAX_PLANES];
  int first[IDX_MAX_PLANES + 1];  // planes' heads in one row: plane i's start here
};

template <class V>
__device__ __forceinline__ void move_rows(const int2* list, int n, char* base, int64_t ss, int64_t row_bytes) {
  const uint32_t per = (uint32_t)(row_bytes / (int64_t)sizeof(V));  // vectors of a row
  const uint32_t all = n * per;  // at most 1024 rows of 2^20 bytes
  constexpr uint32_t U = 4;
  for (uint32_t i0 = threadIdx.x; i0 < all; i0 += U * kMoveThreads) {
    V x[U];
    V* to[U];
#pragma unroll
    for (uint32_t u = 0; u < U; u++) {
      const uint32_t i = i0 + u * kMoveThreads;
      if (i < all) {
        const uint32_t r = i / per, e = i - r * per;
        const int2 mv = list[r];
        x[u] = reinterpret_cast<const V*>(base + mv.y * ss)[e];
        to[u] = reinterpret_cast<V*>(base + mv.x * ss) + e;
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < U; u++)
      if (i0 + u * kMoveThreads < all) *to[u] = x[u];
  }
}

// SLOTS: new slots that a block looks at.
template <int SLOTS>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ MoveArgs a) {
  __shared__ int2 list[SLOTS];  // (new slot, slot it comes from)
  __shared__ int count;
  const int64_t chunks = (a.n_keep + SLOTS - 1) / SLOTS;
  const int64_t row = blockIdx.x / (unsigned)chunks;
  const int64_t s0 = (int64_t)(blockIdx.x % (unsigned)chunks) * SLOTS + threadIdx.x;
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  grid_wait();
  constexpr int U = SLOTS / kMoveThreads;
  int from[U];
  bool some = false;
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t s = s0 + u * kMoveThreads;
    from[u] = s < a.n_keep ? a.src[row * a.n_keep + s] : -1;
  }
#pragma unroll
  for (int u = 0; u < U; u++) some |= from[u] >= 0 && from[u] != (int)s0 + u * kMoveThreads;
  if (__any_sync(0xffffffffu, some)) {  // few do where a cache is just over its budget
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int s = (int)s0 + u * kMoveThreads;
      const bool moves = from[u] >= 0 && from[u] != s;
      const unsigned m = __ballot_sync(0xffffffffu, moves);
      int at = 0;
      if ((threadIdx.x & 31) == 0 && m) at = atomicAdd(&count, __popc(m));
      at = __shfl_sync(0xffffffffu, at, 0);
      if (moves) list[at + __popc(m & ((1u << (threadIdx.x & 31)) - 1))] = make_int2(s, from[u]);
    }
  }
  __syncthreads();
  const int n = count;
  if (n == 0) return;
  const int64_t b = row / a.mass_heads;
  int pl = 0;
  while ((int)blockIdx.y >= a.first[pl + 1]) pl++;
  const evict_plane& q = a.plane[pl];
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

template <int NT, bool ONE>
static cudaError_t launch_select(const EvictArgs& a, int64_t rows, int C, cudaStream_t st) {
  auto bytes = [](int64_t slice) { return (size_t)(slice * 4 + slice / 32 * 6); };
  const int64_t slice = std::max<int64_t>(((a.p.S + C - 1) / C + 31) & ~int64_t(31), 32);
  auto kern = evict_select_kernel<NT, ONE>;
  static KernelReady ready;
  cudaError_t e =
      ready.once([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes(kMaxSlice)); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = bytes(slice);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)C;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = ONE ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kern, a, (int)slice);
}

cudaError_t launch_evict(const evict_problem& p, int32_t* src, int32_t* out_len, int32_t* out_pos, float* out_mass,
                         int64_t out_stride, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.mass_heads;
  const bool vec4 = p.stride % 4 == 0 && ((uintptr_t)p.mass | (uintptr_t)p.pos) % 16 == 0;
  const EvictArgs a{p, src, out_len, out_pos, out_mass, out_stride, vec4};
  // blocks of a row: as many as its keys need, more while the rows leave SMs
  // idle and a block still has a few thousand keys
  int C = 1;
  while (C < kMaxCluster && (p.S > (int64_t)C * kMaxSlice || (rows * C < sm_count() && p.S > (int64_t)C * 4096))) C *= 2;
  cudaError_t e;
  // a thread for each 16 keys or so: blocks of a whole SM's threads only where a
  // slice has work for them
  const int64_t slice = (p.S + C - 1) / C;
  if (C > 1)
    e = slice > 8192 ? launch_select<1024, false>(a, rows, C, st) : launch_select<512, false>(a, rows, C, st);
  else if (slice > 8192)
    e = launch_select<1024, true>(a, rows, C, st);
  else
    e = launch_select<256, true>(a, rows, C, st);
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
  // a block looks at 1024 new slots, or at 256 where that leaves SMs short of blocks
  const int64_t wide = rows * ((p.n_keep + 1023) / 1024), narrow = rows * ((p.n_keep + 255) / 256);
  const unsigned ph = (unsigned)m.first[m.n_planes];
  return wide * ph >= 16 * sm_count()
             ? launch_early(evict_move_kernel<1024>, dim3((unsigned)wide, ph), kMoveThreads, 0, st, m)
             : launch_early(evict_move_kernel<256>, dim3((unsigned)narrow, ph), kMoveThreads, 0, st, m);
}

}  // namespace idx
