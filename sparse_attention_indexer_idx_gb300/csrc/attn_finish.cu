// Attention, last step: the pieces of each row joined, and the attention weight
// of every private slot added to its mass.
//
// Both parts are bound by reading what the pieces left (po, and the private
// scores).  One launch holds both: blocks 0 .. join_blocks - 1 join rows, a warp
// each; the others add masses.  A mass block takes its rows' normalisers from
// the pieces' (m, l) itself, so it need not wait for the join.
#include "attn.cuh"

namespace idx {

namespace {

constexpr int kJoinWarps = 4;
constexpr int kThreads = 32 * kJoinWarps;

// log2 of sum_i 2^(m_i) l_i over a row's pieces; -inf for a row without keys.
__device__ __forceinline__ float row_lse2(const float2* ml, int parts) {
  float top = -INFINITY;
  for (int i = 0; i < parts; i++) {
    const float2 x = ml[i];
    if (x.y > 0.f) top = fmaxf(top, x.x);
  }
  if (top == -INFINITY) return top;
  float l = 0.f;
  for (int i = 0; i < parts; i++) {
    const float2 x = ml[i];
    if (x.y > 0.f) l += x.y * attn_ex2(x.x - top);
  }
  return top + log2f(l);
}

template <int D, bool BF16>
__device__ void join_rows(const AttnArgs& a) {
  const int parts = a.parts_prefix + a.parts_private;
  const int64_t rows = (int64_t)a.p.B * a.p.T * a.p.Hq;
  const int64_t r = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= rows) return;
  const float2* ml = a.pml + r * parts;
  // every lane takes pieces lane, lane + 32, ...
  float top = -INFINITY, l = 0.f;
  for (int i = lane; i < parts; i += 32) {
    const float2 x = ml[i];
    if (x.y > 0.f) top = fmaxf(top, x.x);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  const float base = top == -INFINITY ? 0.f : top;
  for (int i = lane; i < parts; i += 32) {
    const float2 x = ml[i];
    if (x.y > 0.f) l += x.y * attn_ex2(x.x - base);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  const float inv = l > 0.f ? 1.f / l : 0.f;

  constexpr int E = D / 32;  // elements of a lane
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; e++) acc[e] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < parts) {
      const float2 x = ml[i0 + lane];
      if (x.y > 0.f) w = attn_ex2(x.x - base) * inv;
    }
    const unsigned some = __ballot_sync(0xffffffffu, w != 0.f);
    const int n = min(32, parts - i0);
#pragma unroll 4
    for (int i = 0; i < n; i++) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      if (!((some >> i) & 1)) continue;  // empty pieces hold no data
      const float* o = a.po + (r * parts + i0 + i) * D + lane * E;
      if (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(o);
        acc[0] += wi * x.x;
        acc[1] += wi * x.y;
        acc[E - 2] += wi * x.z;
        acc[E - 1] += wi * x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(o);
        acc[0] += wi * x.x;
        acc[1] += wi * x.y;
      }
    }
  }
  uint32_t pk[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; e++) {
    if (BF16) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[2 * e], acc[2 * e + 1]);
      pk[e] = *reinterpret_cast<const uint32_t*>(&x);
    } else {
      const __half2 x = __floats2half2_rn(acc[2 * e], acc[2 * e + 1]);
      pk[e] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out) + (r * D + lane * E) / 2;
#pragma unroll
  for (int e = 0; e < E / 2; e++) out[e] = pk[e];
  if (lane == 0 && a.lse) a.lse[r] = l > 0.f ? (top + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

// Mass of every slot: a thread per slot sums its rows' weights in row order.
__device__ void mass_dense(const AttnArgs& a, int64_t block) {
  __shared__ float s_lse[kThreads];
  const attn_problem& p = a.p;
  const int parts = a.parts_prefix + a.parts_private;
  const int64_t per = (p.S + kThreads - 1) / kThreads;  // blocks of one (b, mass head)
  const int64_t bm = block / per;
  const int64_t slot = (block % per) * kThreads + threadIdx.x;
  const int b = (int)(bm / a.mass_heads), m = (int)(bm % a.mass_heads);
  const int heads = p.Hq / a.mass_heads;  // query heads of the mass head
  const int rows = heads * p.T;
  float add = 0.f;
  bool any = false;
  for (int r0 = 0; r0 < rows; r0 += kThreads) {
    __syncthreads();
    if (r0 + (int)threadIdx.x < rows) {
      const int r = r0 + threadIdx.x;
      const int64_t row = ((int64_t)b * p.T + r / heads) * p.Hq + (int64_t)m * heads + r % heads;
      s_lse[threadIdx.x] = row_lse2(a.pml + row * parts, parts);
    }
    __syncthreads();
    const int n = min(kThreads, rows - r0);
    int h_have = -1, len = 0;
    for (int i = 0; i < n; i++) {
      const int t = (r0 + i) / heads, hq = m * heads + (r0 + i) % heads;
      const int h = hq / a.G;
      if (h != h_have) {
        h_have = h;
        len = p.len[p.len_per_head ? (int64_t)b * p.n_kv + h : b];
        if (len > p.S) len = 0;
      }
      if (slot < (int64_t)len - p.T + t + 1) {
        const float y = a.sc[(((int64_t)b * p.T + t) * p.Hq + hq) * a.sc_ld + slot];
        add += attn_ex2(y - s_lse[i]);
        any = true;
      }
    }
  }
  if (any) a.mass[bm * p.S + slot] += add;
}

// Mass of listed slots.  One list holds a slot at most once, so its threads add
// to different slots; lists that can share a slot (another token's, or another
// KV head's when all heads share the mass) follow one another in one block.
__device__ void mass_listed(const AttnArgs& a, int64_t block) {
  __shared__ float s_lse[kThreads];
  const attn_problem& p = a.p;
  const int parts = a.parts_prefix + a.parts_private;
  const int lists_h = p.ids_per_head && a.mass_heads == 1 ? p.n_kv : 1;
  const int lists = p.T * lists_h;
  const int64_t per = lists == 1 ? (p.W + kThreads - 1) / kThreads : 1;
  const int64_t bm = block / per;
  const int b = (int)(bm / a.mass_heads), m = (int)(bm % a.mass_heads);
  const int64_t w0 = (block % per) * kThreads + threadIdx.x;
  const int64_t step = per * kThreads;
  const int heads = p.Hq / a.mass_heads / lists_h;  // query heads that read one list into one mass head
  float* mass = a.mass + bm * p.S;
  for (int q = 0; q < lists; q++) {
    const int t = q / lists_h;
    const int hq0 = m * (p.Hq / a.mass_heads) + (q % lists_h) * heads;
    const int32_t* list = p.ids + (p.ids_per_head ? (((int64_t)b * p.T + t) * p.n_kv + hq0 / a.G) * p.W
                                                  : ((int64_t)b * p.T + t) * p.W);
    const int64_t row0 = ((int64_t)b * p.T + t) * p.Hq + hq0;
    for (int r0 = 0; r0 < heads; r0 += kThreads) {
      __syncthreads();  // the previous list's additions are done, s_lse is free
      if (r0 + (int)threadIdx.x < heads) s_lse[threadIdx.x] = row_lse2(a.pml + (row0 + r0 + threadIdx.x) * parts, parts);
      __syncthreads();
      const int n = min(kThreads, heads - r0);
      for (int64_t w = w0; w < p.W; w += step) {
        const int id = list[w];
        float add = 0.f;
        int h_have = -1, lim = 0;
        bool any = false;
        for (int i = 0; i < n; i++) {
          const int h = (hq0 + r0 + i) / a.G;
          if (h != h_have) {
            h_have = h;
            const int len = p.len[p.len_per_head ? (int64_t)b * p.n_kv + h : b];
            lim = len > p.S ? 0 : len - p.T + t + 1;
          }
          if (id >= 0 && id < lim) {
            add += attn_ex2(a.sc[(row0 + r0 + i) * a.sc_ld + w] - s_lse[i]);
            any = true;
          }
        }
        if (any) atomicAdd(mass + id, add);
      }
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) attn_finish_kernel(const __grid_constant__ AttnArgs a, int64_t join_blocks) {
  if (blockIdx.x < join_blocks)
    join_rows<D, BF16>(a);
  else if (a.p.ids)
    mass_listed(a, blockIdx.x - join_blocks);
  else
    mass_dense(a, blockIdx.x - join_blocks);
}

}  // namespace

cudaError_t launch_attn_finish(const AttnArgs& a, cudaStream_t st) {
  const attn_problem& p = a.p;
  const int64_t rows = (int64_t)p.B * p.T * p.Hq;
  const int64_t join = (rows + kJoinWarps - 1) / kJoinWarps;
  int64_t mass = 0;
  if (a.mass && a.parts_private) {
    int64_t per = (p.S + kThreads - 1) / kThreads;
    if (p.ids) {
      const bool one = p.T == 1 && !(p.ids_per_head && a.mass_heads == 1 && p.n_kv > 1);
      per = one ? (p.W + kThreads - 1) / kThreads : 1;
    }
    mass = (int64_t)p.B * a.mass_heads * per;
  }
  const dim3 grid((unsigned)(join + mass));
  const bool bf = p.dtype == IDX_BF16;
  if (p.D == 128) {
    if (bf)
      attn_finish_kernel<128, true><<<grid, kThreads, 0, st>>>(a, join);
    else
      attn_finish_kernel<128, false><<<grid, kThreads, 0, st>>>(a, join);
  } else {
    if (bf)
      attn_finish_kernel<64, true><<<grid, kThreads, 0, st>>>(a, join);
    else
      attn_finish_kernel<64, false><<<grid, kThreads, 0, st>>>(a, join);
  }
  return cudaGetLastError();
}

}  // namespace idx
