// Attention over few rows per key sequence, bound by reading keys and values:
// the private caches of a decode step, and a shared prefix under a small batch.
//
// Mapping.  The key sequences (the prefix, then every request's cache or list)
// form one line of key units; it is cut evenly over groups of blocks, with one
// block of a group for each KV head (and tile of up to 32 rows).  The heads of a
// group run side by side, so their rows of a cache, which lie next to one
// another, are read together, and all groups end together however ragged the
// lengths are.  A group that starts or ends inside a sequence leaves one of
// several partial results of it.
//
// A block's four warps are independent streams: warp w takes every fourth tile
// of KT keys, copies the keys and values with 16-byte cp.async into a ring of
// its own (swizzled, so ldmatrix is free of bank conflicts) and keeps the
// running maximum, sum and output of its keys in registers; nothing but the
// warp itself waits for a copy.  The four results are joined through shared
// memory at the end of a sequence or of the block's share.
//
// The products use mma.sync (16 x 8 x 16): a decode row group is 1 to 32 rows,
// so the tensor work is a few percent of the time the bytes take, and the
// register layout of its accumulators is the operand layout of the second
// product, so the weights never leave registers.  Sequences with many rows
// take the tcgen05 kernel instead.
#include "attn.cuh"

namespace idx {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void cp_async_16z(uint32_t dst, const void* src, bool live) {
  // live == false: no bytes are read, the 16 bytes become zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int D, int MT>
struct StreamCfg {
  // Ring slots of a warp.  With up to 16 rows two of them leave room for three
  // blocks on an SM (registers allow no more), whose twelve tiles in flight
  // cover the latency of HBM; with more rows two blocks fit, and a third slot.
  static constexpr int kStages = MT == 1 ? 2 : 3;
  static constexpr int KT = D == 128 ? 16 : 32;  // keys of a warp's tile: 4 KB of keys, 4 KB of values
  static constexpr int ROWB = D * 2;
  static constexpr int CH = ROWB / 16;            // 16-byte chunks of a row
  static constexpr int STAGE = 2 * KT * ROWB;
  static constexpr int UNIT = kWarps * KT;        // keys of the four warps' tiles
  static constexpr int RING = kWarps * kStages * STAGE;
  static constexpr int SLOTS = kWarps * kStages * KT * 4;  // slot numbers of gathered tiles
};

// Chunk c of row r in a swizzled tile of rows of CH chunks.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

// What a block works on at a time: the units [u0, u1) of a key sequence (or of
// an id list), and up to 16*MT rows that read it.
struct StreamItem {
  const char* k;
  const char* v;
  int64_t ks, vs;   // bytes between keys
  int64_t k0, k1;
  int rows, row0;   // rows row0 .. of `rows`
};

// b, t: request, and token of a gathered list; [u0, u1): this block's units of
// the sequence's `units`; part: number of the partial result.
template <int D, int MT, bool BF16, bool GATHER, bool PREFIX>
__device__ __forceinline__ void stream_item(const AttnArgs& a, int h, int tile, int b, int t, int u0, int u1, int units,
                                            int part) {
  using C = StreamCfg<D, MT>;
  constexpr int KT = C::KT, NT = KT / 8, KS = D / 16, CH = C::CH, kStages = C::kStages;
  constexpr int R = 16 * MT;
  extern __shared__ __align__(1024) char smem[];
  char* sring = smem;
  int* sslot = reinterpret_cast<int*>(smem + C::RING);
  char* sq = smem + C::RING + C::SLOTS;
  __shared__ int s_rowid[R];      // (b*T + t)*Hq + hq (below 2^30), or -1
  __shared__ int s_lim[R];        // keys below this index are visible to the row
  __shared__ float2 s_ml[kWarps][R];
  __shared__ float2 s_tot[R];

  const attn_problem& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  StreamItem it;
  it.rows = PREFIX ? p.B * p.T * a.G : GATHER ? a.G : p.T * a.G;
  it.row0 = tile * R;
  const int nrow = min(R, it.rows - it.row0);
  if (nrow <= 0) return;  // a tile that only other sequences have
  if (PREFIX) {
    it.k = (const char*)p.pk + 2 * h * p.pk_stride_h;
    it.v = (const char*)p.pv + 2 * h * p.pv_stride_h;
    it.ks = 2 * p.pk_stride_s;
    it.vs = 2 * p.pv_stride_s;
  } else {
    it.k = (const char*)p.k + 2 * ((int64_t)b * p.k_stride_b + h * p.k_stride_h);
    it.v = (const char*)p.v + 2 * ((int64_t)b * p.v_stride_b + h * p.v_stride_h);
    it.ks = 2 * p.k_stride_s;
    it.vs = 2 * p.v_stride_s;
  }
  const int64_t priv = PREFIX ? 0 : attn_len(p, b, h);
  if (threadIdx.x < R) {
    const int i = threadIdx.x;
    int id = -1, lim = 0;
    if (i < nrow) {
      const int r = it.row0 + i;
      const int g = r % a.G, bt = r / a.G;
      const int rb = PREFIX ? bt / p.T : b, rt = PREFIX ? bt % p.T : GATHER ? t : bt;
      lim = PREFIX ? (int)attn_prefix_len(p, rb) : max(0, (int)priv - p.T + rt + 1);
      id = (rb * p.T + rt) * p.Hq + h * a.G + g;
    }
    s_rowid[i] = id;
    s_lim[i] = lim;
  }
  __syncthreads();
  int64_t n = 0;
  if (GATHER) {
    n = s_lim[0] > 0 ? p.W : 0;
  } else {
    for (int i = 0; i < nrow; i++) n = max(n, (int64_t)s_lim[i]);
  }
  it.k0 = (int64_t)u0 * C::UNIT;
  it.k1 = min(n, (int64_t)u1 * C::UNIT);
  const int parts_all = a.parts_prefix + a.parts_private;
  const int parts = PREFIX ? a.parts_prefix : a.parts_private, at = PREFIX ? 0 : a.parts_prefix;
  // the block with a sequence's last unit marks the partial results that the
  // sequence does not have
  if (u1 == units && threadIdx.x < nrow)
    for (int i = part + 1; i < parts; i++) a.pml[(int64_t)s_rowid[threadIdx.x] * parts_all + at + i] = make_float2(-INFINITY, 0.f);
  part += at;
  if (it.k0 >= it.k1) {
    if (threadIdx.x < nrow) a.pml[(int64_t)s_rowid[threadIdx.x] * parts_all + part] = make_float2(-INFINITY, 0.f);
    __syncthreads();
    return;
  }

  // ---- this warp's tiles: w, w + kWarps, ... of the piece
  const int ntile = (int)((it.k1 - it.k0 + KT - 1) / KT);
  const int mine = (ntile - warp + kWarps - 1) / kWarps;
  const uint32_t ring = smem_u32(sring) + warp * kStages * C::STAGE;
  int* slots = sslot + warp * kStages * KT;
  const int32_t* list = nullptr;
  if (GATHER)
    list = p.ids + (p.ids_per_head ? (((int64_t)b * p.T + t) * p.n_kv + h) * p.W : ((int64_t)b * p.T + t) * p.W);
  const int glim = GATHER ? s_lim[0] : 0;

  int32_t next_id = -1;  // GATHER: lane i holds list entry i of the next tile to copy
  auto load_ids = [&](int j) {
    if (!GATHER) return;
    const int64_t at = it.k0 + (int64_t)(warp + j * kWarps) * KT + lane;
    next_id = (lane < KT && j < mine && at < it.k1) ? __ldg(list + at) : -1;
  };
  auto copy_tile = [&](int j) {
    if (j < mine) {
      const uint32_t sk = ring + (j % kStages) * C::STAGE, sv = sk + C::STAGE / 2;
      const int64_t base = it.k0 + (int64_t)(warp + j * kWarps) * KT;
      if (GATHER && lane < KT) slots[(j % kStages) * KT + lane] = (next_id >= 0 && next_id < glim) ? next_id : -1;
      constexpr int RPI = 32 / CH;  // rows of one warp-wide copy
      const int c = lane % CH;
#pragma unroll
      for (int i = 0; i < KT / RPI; i++) {
        const int r = i * RPI + lane / CH;
        int64_t key;
        bool live;
        if (GATHER) {
          const int id = __shfl_sync(0xffffffffu, next_id, r);
          live = id >= 0 && id < glim;
          key = live ? id : 0;
        } else {
          live = base + r < it.k1;
          key = live ? base + r : it.k0;
        }
        cp_async_16z(sk + swz<D>(r, c), it.k + key * it.ks + c * 16, live);
        cp_async_16z(sv + swz<D>(r, c), it.v + key * it.vs + c * 16, live);
      }
      load_ids(j + 1);
    }
    cp_async_commit();
  };

  load_ids(0);
#pragma unroll
  for (int j = 0; j < kStages - 1; j++) copy_tile(j);

  // ---- queries: rows into shared memory, then operand fragments
  for (int i = threadIdx.x; i < R * CH; i += blockDim.x) {
    const int r = i / CH, c = i % CH;
    const int id = s_rowid[r];
    uint4 x = make_uint4(0, 0, 0, 0);
    if (id >= 0) {
      const int bt = id / p.Hq, hq = id - bt * p.Hq, rb = bt / p.T;
      const int64_t e = rb * p.q_stride_b + (bt - rb * p.T) * p.q_stride_t + hq * p.q_stride_h;
      x = __ldg(reinterpret_cast<const uint4*>((const char*)p.q + 2 * e) + c);
    }
    *reinterpret_cast<uint4*>(sq + swz<D>(r, c)) = x;
  }
  __syncthreads();
  uint32_t qf[MT][KS][4];
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int s = 0; s < KS; s++)
      ldsm_x4(qf[m][s], smem_u32(sq) + swz<D>(m * 16 + (lane & 15), 2 * s + (lane >> 4)));

  float o[MT][D / 8][4];
  float mx[MT][2], sum[MT][2];
  int lim[MT][2];
  int rid[MT][2];
#pragma unroll
  for (int m = 0; m < MT; m++) {
#pragma unroll
    for (int j = 0; j < D / 8; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[m][j][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; e++) {
      mx[m][e] = -INFINITY;
      sum[m][e] = 0.f;
      const int r = m * 16 + (lane >> 2) + 8 * e;
      lim[m][e] = GATHER ? 0 : s_lim[r];
      rid[m][e] = s_rowid[r];
    }
  }

  for (int j = 0; j < mine; j++) {
    cp_async_wait_group<kStages - 2>();
    __syncwarp();  // every lane's copies of tile j have landed, every lane is done with tile j - 1
    copy_tile(j + kStages - 1);
    const uint32_t sk = ring + (j % kStages) * C::STAGE, sv = sk + C::STAGE / 2;
    const int64_t base = it.k0 + (int64_t)(warp + j * kWarps) * KT;
    float s[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int i = 0; i < NT; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) s[m][i][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
      for (int i = 0; i < NT; i += 2) {
        uint32_t kf[4];  // keys 8i..8i+7 and the next eight, the two halves of 16 dims
        ldsm_x4(kf, sk + swz<D>(8 * i + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
#pragma unroll
        for (int m = 0; m < MT; m++) {
          mma16816<BF16>(s[m][i], qf[m][ks], kf[0], kf[1]);
          mma16816<BF16>(s[m][i + 1], qf[m][ks], kf[2], kf[3]);
        }
      }
    // scores in units of log2, masked, and the running maximum
    const int c0 = 2 * (lane & 3);
#pragma unroll
    for (int m = 0; m < MT; m++) {
      float top[2] = {mx[m][0], mx[m][1]};
#pragma unroll
      for (int i = 0; i < NT; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int col = 8 * i + c0 + (e & 1);
          const bool see = GATHER ? slots[(j % kStages) * KT + col] >= 0 : (int)base + col < lim[m][e >> 1];
          s[m][i][e] = see ? s[m][i][e] * a.scale_log2 : -INFINITY;
          top[e >> 1] = fmaxf(top[e >> 1], s[m][i][e]);
        }
      if (!PREFIX && a.sc) {
#pragma unroll
        for (int i = 0; i < NT; i++) {
          const int64_t at = base + 8 * i + c0;
#pragma unroll
          for (int e = 0; e < 2; e++)
            if (rid[m][e] >= 0 && at < it.k1)  // the pair's second half lies inside the padded row
              *reinterpret_cast<float2*>(a.sc + (int64_t)rid[m][e] * a.sc_ld + at) =
                  make_float2(s[m][i][2 * e], s[m][i][2 * e + 1]);
        }
      }
      bool grew = false;
      float scl[2];
#pragma unroll
      for (int e = 0; e < 2; e++) {
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
        const float b = top[e] == -INFINITY ? 0.f : top[e];
        scl[e] = attn_ex2(mx[m][e] - b);  // 0 for a first maximum, 1 where it stays
        grew |= top[e] != mx[m][e];
        mx[m][e] = top[e];
        top[e] = b;
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int e = 0; e < 2; e++) sum[m][e] *= scl[e];
#pragma unroll
        for (int i = 0; i < D / 8; i++)
#pragma unroll
          for (int e = 0; e < 4; e++) o[m][i][e] *= scl[e >> 1];
      }
#pragma unroll
      for (int i = 0; i < NT; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          s[m][i][e] = attn_ex2(s[m][i][e] - top[e >> 1]);
          sum[m][e >> 1] += s[m][i][e];
        }
    }
    // weights (rounded to the element type) times values
#pragma unroll
    for (int kk = 0; kk < KT / 16; kk++) {
      uint32_t pf[MT][4];
#pragma unroll
      for (int m = 0; m < MT; m++) {
        pf[m][0] = pack2<BF16>(s[m][2 * kk][0], s[m][2 * kk][1]);
        pf[m][1] = pack2<BF16>(s[m][2 * kk][2], s[m][2 * kk][3]);
        pf[m][2] = pack2<BF16>(s[m][2 * kk + 1][0], s[m][2 * kk + 1][1]);
        pf[m][3] = pack2<BF16>(s[m][2 * kk + 1][2], s[m][2 * kk + 1][3]);
      }
#pragma unroll
      for (int i = 0; i < D / 8; i += 2) {
        uint32_t vf[4];  // keys 0-7 and 8-15 of dims 8i.., then of the next eight dims
        ldsm_x4_t(vf, sv + swz<D>(kk * 16 + (lane & 15), i + (lane >> 4)));
#pragma unroll
        for (int m = 0; m < MT; m++) {
          mma16816<BF16>(o[m][i], pf[m], vf[0], vf[1]);
          mma16816<BF16>(o[m][i + 1], pf[m], vf[2], vf[3]);
        }
      }
    }
  }
  cp_async_wait_group<0>();

  // ---- join the four warps
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      sum[m][e] += __shfl_xor_sync(0xffffffffu, sum[m][e], 1);
      sum[m][e] += __shfl_xor_sync(0xffffffffu, sum[m][e], 2);
      if ((lane & 3) == 0) s_ml[warp][m * 16 + (lane >> 2) + 8 * e] = make_float2(mx[m][e], sum[m][e]);
    }
  __syncthreads();  // every warp is done with its ring: it holds the outputs now
  float* so = reinterpret_cast<float*>(sring);  // [warp][R][D]
  static_assert(kWarps * R * D * 4 <= C::RING, "the ring holds the warps' outputs");
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const int r = m * 16 + (lane >> 2) + 8 * e;
      if (r >= nrow) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; w++) top = fmaxf(top, s_ml[w][r].x);
      const float f = top == -INFINITY ? 0.f : attn_ex2(mx[m][e] - top);
#pragma unroll
      for (int i = 0; i < D / 8; i++)
        *reinterpret_cast<float2*>(so + ((size_t)warp * R + r) * D + 8 * i + 2 * (lane & 3)) =
            make_float2(o[m][i][2 * e] * f, o[m][i][2 * e + 1] * f);
    }
  if (threadIdx.x < nrow) {
    float top = -INFINITY, l = 0.f;
    for (int w = 0; w < kWarps; w++) top = fmaxf(top, s_ml[w][threadIdx.x].x);
    for (int w = 0; w < kWarps; w++)
      if (top != -INFINITY) l += s_ml[w][threadIdx.x].y * attn_ex2(s_ml[w][threadIdx.x].x - top);
    s_tot[threadIdx.x] = make_float2(top, l);
    a.pml[(int64_t)s_rowid[threadIdx.x] * parts_all + part] = make_float2(top, l);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nrow * (D / 4); i += blockDim.x) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    if (s_tot[r].y == 0.f) continue;
    float4 x = *reinterpret_cast<const float4*>(so + (size_t)r * D + d);
#pragma unroll
    for (int w = 1; w < kWarps; w++) {
      const float4 y = *reinterpret_cast<const float4*>(so + ((size_t)w * R + r) * D + d);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    *reinterpret_cast<float4*>(a.po + ((int64_t)s_rowid[r] * parts_all + part) * D + d) = x;
  }
  __syncthreads();  // the next item takes this memory
}

template <int D, int MT, bool BF16, bool GATHER>
__global__ void __launch_bounds__(32 * kWarps, MT == 1 ? 3 : 2)
    attn_stream_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ StreamLine line) {
  using C = StreamCfg<D, MT>;
  constexpr int NT = 32 * kWarps;
  __shared__ int s_sum[kWarps];
  __shared__ int s_start, s_seq;
  grid_let_next_start();
  const attn_problem& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = blockIdx.x / line.members, member = blockIdx.x - group * line.members;
  const int tile = member / p.n_kv, h = member - tile * p.n_kv;
  const int seqs = line.seqs;                                   // private sequences
  const int list_units = (int)((p.W + C::UNIT - 1) / C::UNIT);  // of a gathered list

  // the line's length (below 2^31, the plan checks), and where on it each
  // thread's share of the requests begins
  int mine = 0, total = line.prefix_units;
  const int per = (seqs + NT - 1) / NT;
  const int b0 = min(seqs, tid * per), b1 = min(seqs, b0 + per);
  if (GATHER) {
    total += seqs * list_units;
  } else {
    for (int b = b0; b < b1; b++) mine += cache_units<C::UNIT>(p, b);
    int incl = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = line.prefix_units;
    for (int w = 0; w < kWarps; w++) {
      total += s_sum[w];
      if (w < warp) before += s_sum[w];
    }
    mine = before + incl - mine;
  }
  // the cut: `groups` shares of `each` units, the first `extra` of them one longer
  const int groups = min(line.groups, max(1, total / line.least));
  const int each = total / groups, extra = total - each * groups;
  auto group_of = [&](int u) {
    const int head = extra * (each + 1);
    return u < head ? u / (each + 1) : extra + (u - head) / each;
  };
  int lo = group * each + min(group, extra);
  const int hi = group < groups ? lo + each + (group < extra ? 1 : 0) : lo;
  // The finish kernel waits for this grid alone, so it has to end behind the
  // one before it: one block waits for that (a wait of every block would keep
  // the next ones from their places).
  const bool waits = blockIdx.x == gridDim.x - 1;
  if (lo >= hi) {
    if (waits) grid_wait();
    return;
  }
  if (lo < line.prefix_units) {
    const int u1 = min(hi, line.prefix_units);
    stream_item<D, MT, BF16, false, true>(a, h, tile, 0, 0, lo, u1, line.prefix_units, group);
    lo = u1;
  }
  if (lo < hi) {
    int seq, units, start;  // the sequence that holds lo
    if (GATHER) {
      seq = (lo - line.prefix_units) / list_units;
      start = line.prefix_units + seq * list_units;
      units = list_units;
    } else {
      __syncthreads();
      int at = mine;
      for (int b = b0; b < b1; b++) {
        const int u = cache_units<C::UNIT>(p, b);
        if (at <= lo && lo < at + u) {
          s_seq = b;
          s_start = at;
        }
        at += u;
      }
      __syncthreads();
      seq = s_seq;
      start = s_start;
      units = cache_units<C::UNIT>(p, seq);
    }
    while (true) {
      const int b = GATHER ? seq / p.T : seq;
      stream_item<D, MT, BF16, GATHER, false>(a, h, tile, b, GATHER ? seq - b * p.T : 0, lo - start, min(units, hi - start),
                                              units, group - group_of(start));
      start += units;
      lo = start;
      if (lo >= hi) break;
      seq++;
      if (!GATHER) units = cache_units<C::UNIT>(p, seq);
    }
  }
  if (waits) grid_wait();
}

template <int D, int MT, bool BF16, bool GATHER>
cudaError_t launch(const AttnArgs& a, const StreamLine& line, bool after, cudaStream_t st) {
  using C = StreamCfg<D, MT>;
  static_assert(C::UNIT == stream_unit(D), "the plan counts in these units");
  const int smem = C::RING + C::SLOTS + 16 * MT * D * 2;
  auto kern = attn_stream_kernel<D, MT, BF16, GATHER>;
  static KernelReady ready;
  cudaError_t e = ready.once([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3((unsigned)(line.members * line.groups)), 32 * kWarps, smem, st, after, a, line);
}

template <int D, bool BF16, bool GATHER>
cudaError_t launch_rows(const AttnArgs& a, const StreamLine& line, bool after, cudaStream_t st) {
  return line.row_tile == 16 ? launch<D, 1, BF16, GATHER>(a, line, after, st)
                             : launch<D, 2, BF16, GATHER>(a, line, after, st);
}

template <int D, bool BF16>
cudaError_t launch_kind(const AttnArgs& a, const StreamLine& line, bool after, cudaStream_t st) {
  return a.p.ids ? launch_rows<D, BF16, true>(a, line, after, st) : launch_rows<D, BF16, false>(a, line, after, st);
}

}  // namespace

cudaError_t launch_attn_stream(const AttnArgs& a, const StreamLine& line, bool after, cudaStream_t st) {
  const bool bf = a.p.dtype == IDX_BF16;
  if (a.p.D == 128) return bf ? launch_kind<128, true>(a, line, after, st) : launch_kind<128, false>(a, line, after, st);
  return bf ? launch_kind<64, true>(a, line, after, st) : launch_kind<64, false>(a, line, after, st);
}

}  // namespace idx
