// Attention, last step: the pieces of each row joined, and the attention weight
// of every private slot added to its mass.
//
// Both parts read what the pieces left (po, and the private scores: 4 bytes a row
// and slot).  One launch holds both: blocks 0 .. join_blocks - 1 join rows, a
// warp or more each; the others add masses.  A mass block takes its rows'
// normalisers from the pieces' (m, l) itself, so it need not wait for the join.
// Large calls are bound by those reads and an exponential a score (16 caches of
// 24,576 slots on average under 64 rows: 100 MB in 34 us), small ones by the
// chain of loads from the pieces to a block's sums, 6 to 10 us.
//
// A piece is empty where its sum is 0, and only there: a sum that is NaN (a
// score was) makes the row's output, its lse and its weights NaN.
#include "attn.cuh"

#include <algorithm>

namespace idx {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlots = 4;    // consecutive slots of a thread: one 16-byte load per row
constexpr int kRowsAt = 512; // rows whose normalisers are held at a time
constexpr int kBatch = 8;    // rows loaded before the first is used (dense masses)

// A row is the work of `share` warps (1 to 8), each of a run of its pieces.
template <int D, bool BF16>
__device__ void join_rows(const AttnArgs& a, int share) {
  __shared__ float s_acc[kWarps][D];
  __shared__ float2 s_ml[kWarps];
  const int all_parts = a.parts_prefix + a.parts_private;
  const int64_t rows = (int64_t)a.p.B * a.p.T * a.p.Hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * (kWarps / share) + warp / share;
  const int sub = warp % share;
  const int each = (all_parts + share - 1) / share;
  const int p0 = min(all_parts, sub * each);
  const int parts = r < rows ? min(each, all_parts - p0) : 0;  // of this warp
  const float2* ml = a.pml + r * all_parts + p0;
  // lane i holds piece i (of the first 32; the others are read again)
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 first = lane < parts ? ml[lane] : none;
  float top = first.y != 0.f ? first.x : -INFINITY;
  for (int i = lane + 32; i < parts; i += 32) {
    const float2 x = ml[i];
    if (x.y != 0.f) top = fmaxf(top, x.x);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  const float base = top == -INFINITY ? 0.f : top;
  float l = 0.f;
  constexpr int E = D / 32;  // elements of a lane
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; e++) acc[e] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    const float2 x = i0 == 0 ? first : i0 + lane < parts ? ml[i0 + lane] : none;
    const float w = x.y != 0.f ? attn_ex2(x.x - base) : 0.f;
    l += w * x.y;
    unsigned some = __ballot_sync(0xffffffffu, w != 0.f);  // empty pieces hold no data
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
          const float* o = a.po + (r * all_parts + p0 + i0 + i) * D + lane * E;
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
    for (int i = 0; i < share; i++) top = fmaxf(top, s_ml[warp + i].x);
    const float all = top == -INFINITY ? 0.f : top;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] = 0.f;
    for (int i = 0; i < share; i++) {
      const float2 x = s_ml[warp + i];
      const float w = attn_ex2(x.x - all);
      l += w * x.y;
#pragma unroll
      for (int e = 0; e < E; e++) acc[e] += w * s_acc[warp + i][lane * E + e];
    }
  }
  if (r >= rows) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  uint32_t pk[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; e++) {
    if (BF16) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      pk[e] = *reinterpret_cast<const uint32_t*>(&x);
    } else {
      const __half2 x = __floats2half2_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      pk[e] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out) + (r * D + lane * E) / 2;
#pragma unroll
  for (int e = 0; e < E / 2; e++) out[e] = pk[e];
  if (lane == 0 && a.lse) a.lse[r] = l != 0.f ? (top + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

// What a mass block needs of a row: its log2 normaliser, how many private slots
// it sees, and its number.
struct MassRows {
  float lse2[kRowsAt];    // +inf for a row that sees no private slot, or nothing
  int lim[kRowsAt];
  int row[kRowsAt];       // (b*T + t)*Hq + hq
  int longest, shortest;  // of lim
};

// Rows (b, t, hq): the i-th is t = t0 + i / heads, hq = hq0 + i % heads, for i0
// <= i < i0 + n.  Reads only the call's inputs: it runs before grid_wait().
__device__ __forceinline__ void set_rows(const AttnArgs& a, MassRows& s, int b, int t0, int hq0, int heads, int i0,
                                         int n) {
  const attn_problem& p = a.p;
  if (threadIdx.x == 0) {
    s.longest = 0;
    s.shortest = INT32_MAX;
  }
  __syncthreads();
  int longest = 0, shortest = INT32_MAX;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int dt = (i0 + i) / heads, t = t0 + dt, hq = hq0 + (i0 + i) - dt * heads;
    const int len = p.len[p.len_per_head ? (int64_t)b * p.n_kv + hq / a.G : b];
    const int lim = len < 0 || len > p.S ? 0 : max(0, len - p.T + t + 1);
    s.lim[i] = lim;
    s.row[i] = (b * p.T + t) * p.Hq + hq;
    longest = max(longest, lim);
    shortest = min(shortest, lim);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  shortest = __reduce_min_sync(0xffffffffu, shortest);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&s.longest, longest);
    atomicMin(&s.shortest, shortest);
  }
  __syncthreads();
}

// The normalisers of the n rows.  A warp takes four rows at a time, eight lanes
// to a row's pieces, or sixteen rows where eight lanes hold all of them.
__device__ __forceinline__ void load_norms(const AttnArgs& a, MassRows& s, int n) {
  const int parts = a.parts_prefix + a.parts_private;
  const int lane = threadIdx.x & 31, sub = lane & 7;
  if (parts <= 8) {
    for (int i0 = (threadIdx.x >> 5) * 4; i0 < n; i0 += kWarps * 16) {
      float2 x[4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const int i = i0 + u * kWarps * 4 + (lane >> 3);
        x[u] = i < n && sub < parts ? a.pml[(int64_t)s.row[i] * parts + sub] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int u = 0; u < 4; u++) {
        if (i0 + u * kWarps * 4 >= n) break;
        const int i = i0 + u * kWarps * 4 + (lane >> 3);
        float m = x[u].y > 0.f ? x[u].x : -INFINITY;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        float l = x[u].y > 0.f ? x[u].y * attn_ex2(x[u].x - m) : x[u].y;  // 0 or NaN
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (i < n && sub == 0) s.lse2[i] = s.lim[i] > 0 && l != 0.f ? m + log2f(l) : INFINITY;
      }
    }
    __syncthreads();
    return;
  }
  for (int i = (threadIdx.x >> 5) * 4 + (lane >> 3); i < ((n + 3) & ~3); i += kWarps * 4) {
    const bool live = i < n;
    const float2* ml = a.pml + (int64_t)s.row[live ? i : 0] * parts;
    float top = -INFINITY, l = 0.f;
    for (int j0 = 0; j0 < parts; j0 += 32) {  // four pieces of a lane at a time
      float2 x[4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const int j = j0 + u * 8 + sub;
        x[u] = live && j < parts ? ml[j] : make_float2(-INFINITY, 0.f);
      }
      float m = top;
#pragma unroll
      for (int u = 0; u < 4; u++)
        if (x[u].y > 0.f)
          m = fmaxf(m, x[u].x);
        else
          l += x[u].y;  // 0 or NaN
      if (m == -INFINITY) continue;
      l *= attn_ex2(top - m);
      top = m;
#pragma unroll
      for (int u = 0; u < 4; u++)
        if (x[u].y > 0.f) l += x[u].y * attn_ex2(x[u].x - top);
    }
    float m = top;
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    l = m == -INFINITY ? l : l * attn_ex2(top - m);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (live && sub == 0) s.lse2[i] = s.lim[i] > 0 && l != 0.f ? m + log2f(l) : INFINITY;
  }
  __syncthreads();
}

// Mass of every slot.  A slot's rows are split over `groups` threads in equal
// runs; each sums its own in row order, then the runs are added in order.  A
// block takes every per-th run of slots: the rows' normalisers, which take more
// instructions than the sums of a few hundred slots, are formed once for them.
// The old masses are fetched before the kernels that come first are done, the
// first scores beside the pieces of the normalisers.
__device__ __forceinline__ void mass_dense(const AttnArgs& a, int64_t block, int per, int groups) {
  __shared__ MassRows s;
  __shared__ float4 s_add[kThreads];
  const attn_problem& p = a.p;
  const int lanes = kThreads / groups;  // threads next to one another in the slots
  const int64_t bm = block / per;
  const int mine = threadIdx.x % lanes, run = threadIdx.x / lanes;
  const int b = (int)(bm / a.mass_heads), m = (int)(bm % a.mass_heads);
  const int heads = p.Hq / a.mass_heads;  // query heads of the mass head
  const int rows = heads * p.T;
  const int first = (int)(block % per) * lanes * kSlots;
  for (int r0 = 0; r0 < rows; r0 += kRowsAt) {
    const int n = min(kRowsAt, rows - r0);
    const int len = (n + groups - 1) / groups;
    const int i0 = min(n, run * len), i1 = min(n, i0 + len);  // this thread's rows of those held
    __syncthreads();
    set_rows(a, s, b, 0, m * heads, heads, r0, n);
    if (first >= s.longest) continue;
    float old[kSlots];
    auto fetch_old = [&](int slot) {
      const float* from = a.mass + bm * p.S + slot;
#pragma unroll
      for (int e = 0; e < kSlots; e++) old[e] = run == 0 && slot + e < s.longest ? from[e] : 0.f;
    };
    float4 y[kBatch];
    // scores of rows i ..; a row's memory goes on behind its last one for these four
    auto fetch = [&](int slot, int i) {
#pragma unroll
      for (int u = 0; u < kBatch; u++)
        if (i + u < i1) y[u] = *reinterpret_cast<const float4*>(a.sc + (int64_t)s.row[i + u] * a.sc_ld + slot);
    };
    const int slot0 = first + mine * kSlots;
    fetch_old(slot0);
    grid_wait();
    if (slot0 < s.longest) fetch(slot0, i0);
    load_norms(a, s, n);
    for (int at = first; at < s.longest; at += per * lanes * kSlots) {
      const int slot = at + mine * kSlots;
      if (at != first) fetch_old(slot);
      float add[kSlots] = {};
      const bool all = slot + kSlots <= s.shortest;  // every row sees all four slots
      if (slot < s.longest)
        for (int i = i0; i < i1; i += kBatch) {
          if (at != first || i != i0) fetch(slot, i);
#pragma unroll
          for (int u = 0; u < kBatch; u++)
            if (i + u < i1) {
              const float z = s.lse2[i + u];
              const int left = all ? kSlots : s.lim[i + u] - slot;  // of the four, those that the row sees
              add[0] += left > 0 ? attn_ex2(y[u].x - z) : 0.f;
              add[1] += left > 1 ? attn_ex2(y[u].y - z) : 0.f;
              add[2] += left > 2 ? attn_ex2(y[u].z - z) : 0.f;
              add[3] += left > 3 ? attn_ex2(y[u].w - z) : 0.f;
            }
        }
      if (groups > 1) {
        __syncthreads();
        s_add[threadIdx.x] = make_float4(add[0], add[1], add[2], add[3]);
        __syncthreads();
        if (run > 0) continue;
        for (int g = 1; g < groups; g++) {
          const float4 x = s_add[g * lanes + mine];
          add[0] += x.x;
          add[1] += x.y;
          add[2] += x.z;
          add[3] += x.w;
        }
      }
      float* to = a.mass + bm * p.S + slot;
#pragma unroll
      for (int e = 0; e < kSlots; e++)
        if (slot + e < s.longest) to[e] = old[e] + add[e];
    }
  }
  grid_wait();
}

// Sum of an entry's weights over those of n rows that see it.
__device__ __forceinline__ float seen_only(const float* sc, int64_t ld, const float* lse2, int n) {
  float add = 0.f;
#pragma unroll 1
  for (int i = 0; i < n; i++) {
    const float y = sc[i * ld];
    if (y != -INFINITY) add += attn_ex2(fminf(y, 3e38f) - lse2[i]);
  }
  return add;
}

// Mass of listed slots.  One list holds a slot at most once, so its threads add
// to different slots; lists that can share a slot (another token's, or another
// KV head's when all heads share the mass) are added one after the other by one
// block.  The lists' entries form one line; a thread takes E of them, and several
// rows of each, at a time: ids and scores of whatever lists they belong to are
// loaded together, only the additions follow the lists' order.
template <int E>
__device__ __forceinline__ void mass_listed(const AttnArgs& a, int64_t block, int64_t per) {
  __shared__ MassRows s;
  constexpr int kBatch = E == 1 ? 16 : 8;
  const attn_problem& p = a.p;
  const int lists_h = p.ids_per_head && a.mass_heads == 1 ? p.n_kv : 1;
  const int lists = p.T * lists_h;
  const int lane = threadIdx.x & 31;
  const int64_t bm = block / per;
  const int b = (int)(bm / a.mass_heads), m = (int)(bm % a.mass_heads);
  const int all = p.Hq / a.mass_heads;  // query heads of the mass head
  const int heads = all / lists_h;      // of these, the ones that read one list
  float* mass = a.mass + bm * p.S;
  // rows (t, query head) of the mass head: list q has rows q * heads ..
  const int held = min(heads, kRowsAt);            // rows of a list at a time
  const int many = min(lists, kRowsAt / held);     // lists at a time
  const uint32_t W = ((uint32_t)p.W + 31) & ~31u;  // below 2^31; a warp's entries are of one list
  for (int q0 = 0; q0 < lists; q0 += many)
    for (int r0 = 0; r0 < heads; r0 += held) {
      const int nl = min(many, lists - q0), nh = min(held, heads - r0), n = nl * nh;
      __syncthreads();
      set_rows(a, s, b, 0, m * all, all, q0 * heads + r0, n);
      const int64_t line = nl * (int64_t)W;
      bool ready = false;
      for (int64_t x0 = block % per * kThreads; x0 < line; x0 += per * kThreads * E) {
        // the round's first entry: entry w0 of list l0 (counted from q0)
        const int l0 = lists > 1 ? (int)(x0 / W) : 0;
        const uint32_t w0 = (uint32_t)(x0 - (int64_t)l0 * W);
        int id[E], list[E];
        const float* sc[E];
        float add[E] = {};
        // lane e: what the warp's entries of chunk e have in common
        int list_l, sc_l, ids_l;
        uint32_t w_l;
        {
          const uint32_t off = (uint32_t)(lane % E * per) * kThreads + (threadIdx.x & ~31u);
          const uint32_t d = lists > 1 ? (w0 + off) / W : 0;
          list_l = min(l0 + (int)d, nl - 1);
          w_l = l0 + (int)d < nl ? w0 + off - d * W : W;  // W: none
          const int q = q0 + list_l;
          const int t = q / lists_h, hq = m * all + (q - t * lists_h) * heads, bt = b * p.T + t;
          sc_l = bt * p.Hq + hq + r0;
          ids_l = p.ids_per_head ? bt * p.n_kv + hq / a.G : bt;
        }
#pragma unroll
        for (int e = 0; e < E; e++) {
          const uint32_t w = __shfl_sync(0xffffffffu, w_l, e) + lane;
          const int64_t sc_row = __shfl_sync(0xffffffffu, sc_l, e), ids_row = __shfl_sync(0xffffffffu, ids_l, e);
          const bool live = w < p.W;
          list[e] = __shfl_sync(0xffffffffu, list_l, e);
          sc[e] = a.sc + sc_row * a.sc_ld + (live ? w : 0);
          id[e] = live ? p.ids[ids_row * p.W + w] : -1;
        }
        grid_wait();
        for (int i0 = 0; i0 < nh; i0 += kBatch) {
          float y[kBatch][E];
#pragma unroll
          for (int u = 0; u < kBatch; u++)
#pragma unroll
            for (int e = 0; e < E; e++) y[u][e] = i0 + u < nh ? sc[e][(i0 + u) * a.sc_ld] : 0.f;
          if (!ready) load_norms(a, s, n);
          ready = true;
          // Scores of entries that a row does not see are -inf.  A row that sees no
          // slot has no scores, and one whose list holds none of its slots may see
          // nothing at all: their normaliser is +inf (fminf: so that whatever the
          // memory of absent scores holds becomes 0).
#pragma unroll
          for (int u = 0; u < kBatch; u++)
            if (i0 + u < nh)
#pragma unroll
              for (int e = 0; e < E; e++) {
                const int i = list[e] * nh + i0 + u;
                add[e] += attn_ex2(fminf(y[u][e], 3e38f) - s.lse2[i]);
              }
        }
        // A row whose normaliser is NaN counts only where it sees the entry.  (The
        // choice in the loop above took 1.5 us of 27 and of 65.)
#pragma unroll
        for (int e = 0; e < E; e++)
          if (add[e] != add[e]) add[e] = seen_only(sc[e], a.sc_ld, s.lse2 + list[e] * nh, nh);
        // with several lists (then per is 1) those of this round in turn
        const int l1 = lists > 1 ? min(nl - 1, l0 + (int)((w0 + kThreads * E - 1) / W)) : l0;
        for (int l = l0; l <= l1; l++) {
          if (lists > 1) __syncthreads();  // the additions of the list before are done
#pragma unroll
          for (int e = 0; e < E; e++)
            if (list[e] == l && id[e] >= 0 && id[e] < s.longest) atomicAdd(mass + id[e], add[e]);
        }
      }
    }
  grid_wait();
}

// MASS: 0 every slot, else the entries that a thread of the listed form takes.
template <int D, bool BF16, int MASS>
__global__ void __launch_bounds__(kThreads, MASS == 4 ? 3 : 4)
    attn_finish_kernel(const __grid_constant__ AttnArgs a, int64_t join_blocks, int share, int64_t per, int row_groups) {
  if (blockIdx.x < join_blocks) {
    grid_wait();
    join_rows<D, BF16>(a, share);
  } else if constexpr (MASS == 0) {
    mass_dense(a, blockIdx.x - join_blocks, (int)per, row_groups);
  } else {
    mass_listed<MASS>(a, blockIdx.x - join_blocks, per);
  }
}

template <int D, bool BF16>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  const attn_problem& p = a.p;
  const int64_t rows = (int64_t)p.B * p.T * p.Hq;
  // A warp for a row; where the rows leave warps free, one for each 16 pieces of
  // it (2 requests of 28 heads behind 45,840 tokens, 456 pieces a row: 74 us for
  // the call with one, 39 with eight).
  const int parts = a.parts_prefix + a.parts_private;
  int share = 1;
  while (share < kWarps && parts > 16 * share && rows * share < 8 * sm_count()) share *= 2;
  const int64_t join = (rows * share + kWarps - 1) / kWarps;
  // A slot's rows are spread over up to four threads where there are many, and
  // over up to 32 while the slots are too few to give every SM a block (7 rows of
  // 170 slots under 256 rows: 27 us with four threads).
  const int mass_rows = p.Hq / a.mass_heads * p.T;
  int groups = mass_rows >= 32 ? 4 : mass_rows >= 16 ? 2 : 1;
  auto mass_blocks = [&] { return (p.S + kThreads / groups * kSlots - 1) / (kThreads / groups * kSlots); };
  while (groups < 32 && mass_rows >= 16 * groups && (int64_t)p.B * a.mass_heads * mass_blocks() < sm_count()) groups *= 2;
  auto kern = attn_finish_kernel<D, BF16, 0>;
  int64_t per = 0;  // mass blocks of one (b, mass head)
  if (a.mass && a.parts_private) {
    const int64_t bms = (int64_t)p.B * a.mass_heads;
    per = std::min(mass_blocks(), std::max<int64_t>(1, (4 * sm_count() + bms - 1) / bms));  // four blocks fit an SM
    if (p.ids) {
      // lists that share slots are one block's; another list's entries are spread
      // over blocks
      const bool one = p.T == 1 && !(p.ids_per_head && a.mass_heads == 1 && p.n_kv > 1);
      per = one ? (p.W + kThreads - 1) / kThreads : 1;
      kern = one && p.Hq / a.mass_heads > 8 ? attn_finish_kernel<D, BF16, 1> : attn_finish_kernel<D, BF16, 4>;
    }
  }
  const int64_t blocks = join + (int64_t)p.B * a.mass_heads * per;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_early(kern, dim3((unsigned)blocks), kThreads, 0, st, a, join, share, per, groups);
}

}  // namespace

cudaError_t launch_attn_finish(const AttnArgs& a, cudaStream_t st) {
  const bool bf = a.p.dtype == IDX_BF16;
  if (a.p.D == 128) return bf ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return bf ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

}  // namespace idx
