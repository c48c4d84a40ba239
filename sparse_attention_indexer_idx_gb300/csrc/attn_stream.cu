// Attention over few rows per key sequence, bound by reading keys and values:
// the private caches of a decode step, and a shared prefix under a small batch.
//
// Mapping.  The key sequences (the prefix, then every request's cache or list)
// form one line of units of one to four key tiles; it is cut evenly over groups
// of warps, with one warp of a group for each KV head (and tile of up to 32
// rows).  The heads of a group run side by side, so their rows of a cache, which
// lie next to one another, are read together, and all groups end together
// however ragged the lengths are.  A group that starts or ends inside a sequence leaves one of
// several partial results of it.
//
// Every warp is a stream of its own: it copies tiles of KT keys and values with
// 16-byte cp.async into a ring (swizzled, so ldmatrix is free of bank
// conflicts) and keeps the running maximum, sum and output in registers.
// Nothing waits for another warp: the start and the end of one warp's sequence
// pass while the others of the SM stream.  One tile of each of the SM's twelve
// warps is on its way all the time, 96 KB; refilling each half of a ring slot as
// soon as it was used, up to twice as much, cost 8 percent (272 against 251 us
// for 16 caches of 24,576 slots on average, 8 KV heads of 128: 1.61 GB, 6.4 TB/s).
// 64 lists of 2,048 ids, 4 KV heads of 128 (268 MB in rows of 256 bytes), take 53
// us, 5.1 TB/s: a list is one warp's few dozen tiles per head, and each tile's
// addresses wait for its ids.
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
  static constexpr int KT = stream_tile(D);      // keys of a tile: 4 KB of keys, 4 KB of values
  static constexpr int CH = D / 8;                // 16-byte chunks of a row
  static constexpr int HALF = KT * D * 2;         // bytes of a tile's keys, and of its values
  static constexpr int RING = 2 * 2 * HALF;       // two slots
  static constexpr int SLOTS = 2 * KT;            // slot numbers of gathered tiles
  static constexpr int WARP_BYTES = RING + SLOTS * 4;
};

// Chunk c of row r in a swizzled tile of rows of CH chunks.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

// One warp's part of a key sequence (or of an id list) for up to 16*MT rows: its
// units [u0, u1) of the sequence's `units`.  b, t: request, and token of a
// gathered list; part: number of the partial result.
template <int D, int MT, bool BF16, bool GATHER, bool PREFIX>
__device__ __forceinline__ void stream_item(const AttnArgs& a, int shift, int h, int tile, int b, int t, int u0, int u1,
                                            int units, int part) {
  using C = StreamCfg<D, MT>;
  constexpr int KT = C::KT, NT = KT / 8, KS = D / 16, CH = C::CH;
  constexpr int R = 16 * MT;
  extern __shared__ __align__(1024) char smem[];
  const attn_problem& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  int* slots = reinterpret_cast<int*>(smem + kWarps * C::RING) + warp * C::SLOTS;
  const int rows = PREFIX ? p.B * p.T * a.G : GATHER ? a.G : p.T * a.G;
  const int row0 = tile * R;
  const int nrow = min(R, rows - row0);
  if (nrow <= 0) return;  // a tile that only other sequences have

  // lane r holds row r: its number, its queries, and how many keys it sees
  int rid_l = -1, lim_l = 0;
  int64_t q_l = 0;
  if (lane < nrow) {
    const int r = row0 + lane, bt = r / a.G, g = r - bt * a.G;
    int rb = b, rt = GATHER ? t : bt;
    if (PREFIX) {
      rb = bt / p.T;
      rt = bt - rb * p.T;
      lim_l = (int)attn_prefix_len(p, rb);
    } else {
      lim_l = max(0, attn_len(p, b, h) - p.T + rt + 1);
    }
    const int hq = h * a.G + g;
    rid_l = (rb * p.T + rt) * p.Hq + hq;
    q_l = rb * p.q_stride_b + rt * p.q_stride_t + hq * p.q_stride_h;
  }
  const int most = __reduce_max_sync(0xffffffffu, lim_l);
  const int n = GATHER ? (most > 0 ? (int)p.W : 0) : most;  // keys of the sequence
  const int k0 = u0 << shift, k1 = (int)min((int64_t)n, (int64_t)u1 << shift);
  const int parts_all = a.parts_prefix + a.parts_private;
  const int parts = PREFIX ? a.parts_prefix : a.parts_private, at0 = PREFIX ? 0 : a.parts_prefix;
  // the warp with a sequence's last unit marks the partial results that the
  // sequence does not have
  if (u1 == units && lane < nrow)
    for (int i = part + 1; i < parts; i++) a.pml[(int64_t)rid_l * parts_all + at0 + i] = make_float2(-INFINITY, 0.f);
  part += at0;
  if (k0 >= k1) {
    if (lane < nrow) a.pml[(int64_t)rid_l * parts_all + part] = make_float2(-INFINITY, 0.f);
    return;
  }

  const char* kb;
  const char* vb;
  int64_t ks_b, vs_b;  // bytes between keys, and between values
  if (PREFIX) {
    kb = (const char*)p.pk + 2 * h * p.pk_stride_h;
    vb = (const char*)p.pv + 2 * h * p.pv_stride_h;
    ks_b = 2 * p.pk_stride_s;
    vs_b = 2 * p.pv_stride_s;
  } else {
    kb = (const char*)p.k + 2 * ((int64_t)b * p.k_stride_b + h * p.k_stride_h);
    vb = (const char*)p.v + 2 * ((int64_t)b * p.v_stride_b + h * p.v_stride_h);
    ks_b = 2 * p.k_stride_s;
    vs_b = 2 * p.v_stride_s;
  }
  const int mine = (k1 - k0 + KT - 1) / KT;  // tiles
  const int32_t* list = nullptr;
  if (GATHER)
    list = p.ids + (p.ids_per_head ? (((int64_t)b * p.T + t) * p.n_kv + h) * p.W : ((int64_t)b * p.T + t) * p.W);
  int next_id = -1;  // GATHER: lane i holds list entry i of the tile to copy next
  auto load_ids = [&](int j) {
    const int at = k0 + j * KT + lane;
    next_id = (lane < KT && j < mine && at < k1) ? __ldg(list + at) : -1;
  };
  // copies tile j into its ring slot
  auto copy = [&](int j) {
    if (j < mine) {
      constexpr int RPI = 32 / CH;  // rows of one warp-wide copy
      const uint32_t sk = ring + (j & 1) * 2 * C::HALF, sv = sk + C::HALF;
      const int c = lane % CH, base = k0 + j * KT;
      int slot = -1;  // GATHER: lane i's, -1: not a visible one
      if (GATHER) {
        slot = next_id >= 0 && next_id < most ? next_id : -1;
        if (lane < KT) slots[(j & 1) * KT + lane] = slot;
        load_ids(j + 1);
      }
#pragma unroll
      for (int i = 0; i < KT / RPI; i++) {
        const int r = i * RPI + lane / CH;
        int key;
        bool live;
        if (GATHER) {
          key = __shfl_sync(0xffffffffu, slot, r);
          live = key >= 0;
          key = max(key, 0);
        } else {
          key = base + r;
          live = key < k1;
          key = live ? key : k0;
        }
        cp_async_16z(sk + swz<D>(r, c), kb + key * ks_b + c * 16, live);
        cp_async_16z(sv + swz<D>(r, c), vb + key * vs_b + c * 16, live);
      }
    }
    cp_async_commit();
  };
  if (GATHER) load_ids(0);
  copy(0);

  // the queries, as operand fragments: row lane / 4 (and 8 on) of a 16-row tile,
  // pairs of dims 2 (lane % 4) (and 8 on)
  uint32_t qf[MT][KS][4];
  int lim[MT][2], rid[MT][2];
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const int r = m * 16 + (lane >> 2) + 8 * e;
      rid[m][e] = __shfl_sync(0xffffffffu, rid_l, r);
      lim[m][e] = __shfl_sync(0xffffffffu, lim_l, r);
      const int64_t q_at = __shfl_sync(0xffffffffu, q_l, r);
      const uint32_t* q = reinterpret_cast<const uint32_t*>((const char*)p.q + 2 * q_at) + (lane & 3);
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        qf[m][ks][e] = rid[m][e] >= 0 ? __ldg(q + 8 * ks) : 0u;
        qf[m][ks][e + 2] = rid[m][e] >= 0 ? __ldg(q + 8 * ks + 4) : 0u;
      }
    }

  float o[MT][D / 8][4];
  float mx[MT][2], sum[MT][2];
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
    }
  }

  for (int j = 0; j < mine; j++) {
    const uint32_t sk = ring + (j & 1) * 2 * C::HALF, sv = sk + C::HALF;
    const int base = k0 + j * KT;
    cp_async_wait_group<0>();
    __syncwarp();  // every lane's copies of tile j have landed, every lane is done with tile j - 1
    copy(j + 1);
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
          const bool see = GATHER ? slots[(j & 1) * KT + col] >= 0 : base + col < lim[m][e >> 1];
          s[m][i][e] = see ? s[m][i][e] * a.scale_log2 : -INFINITY;
          top[e >> 1] = fmaxf(top[e >> 1], s[m][i][e]);
        }
      if (!PREFIX && a.sc) {
#pragma unroll
        for (int i = 0; i < NT; i++) {
          const int at = base + 8 * i + c0;
#pragma unroll
          for (int e = 0; e < 2; e++)
            if (rid[m][e] >= 0 && at < k1)  // the pair's second half lies inside the padded row
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
    // Weights times values.  The weights are rounded to the element type, as the
    // 16-bit operand of the product has to be, one rounding of at most 2^-8 (2^-11
    // for fp16) of each weight, as large as the output's own; the sum that divides
    // them is of the unrounded ones, in 32 bits.
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
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      sum[m][e] += __shfl_xor_sync(0xffffffffu, sum[m][e], 1);
      sum[m][e] += __shfl_xor_sync(0xffffffffu, sum[m][e], 2);
      if (rid[m][e] < 0) continue;
      const int64_t at = (int64_t)rid[m][e] * parts_all + part;
      if ((lane & 3) == 0) a.pml[at] = make_float2(mx[m][e], sum[m][e]);
      if (sum[m][e] != 0.f) {  // (NaN where a score was)
#pragma unroll
        for (int i = 0; i < D / 8; i++)
          *reinterpret_cast<float2*>(a.po + at * D + 8 * i + 2 * (lane & 3)) = make_float2(o[m][i][2 * e], o[m][i][2 * e + 1]);
      }
    }
  __syncwarp();
}

template <int D, int MT, bool BF16, bool GATHER>
__global__ void __launch_bounds__(32 * kWarps, MT == 1 ? 3 : 2)
    attn_stream_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ StreamLine line) {
  using C = StreamCfg<D, MT>;
  constexpr int NT = 32 * kWarps;
  __shared__ int s_sum[kWarps];
  __shared__ int s_first[NT];
  if (!line.after) grid_wait();  // behind the tensor-core kernel, which has waited, the call's inputs are there
  grid_let_next_start();
  const attn_problem& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if ((int)blockIdx.x < line.own_blocks) {
    const int x = blockIdx.x * kWarps + warp;
    const int group = x / line.own_members, member = x - group * line.own_members;
    const int tile = member / p.n_kv;
    if (group < line.own_groups) {
      const int each = line.own_units / line.own_groups, extra = line.own_units - each * line.own_groups;
      const int lo = group * each + min(group, extra);
      const int hi = lo + each + (group < extra ? 1 : 0);
      stream_item<D, MT, BF16, false, true>(a, line.unit_shift, member - tile * p.n_kv, tile, 0, 0, lo, hi,
                                            line.own_units, group);
    }
    if (blockIdx.x == gridDim.x - 1) grid_wait();
    return;
  }
  const int w = ((int)blockIdx.x - line.own_blocks) * kWarps + warp;
  const int group = w / line.members, member = w - group * line.members;
  const int tile = member / p.n_kv, h = member - tile * p.n_kv;
  const int seqs = line.seqs;                                   // private sequences

  // the line's length (below 2^31, the plan checks), and where on it each
  // thread's share of the requests begins
  int total = line.prefix_units;
  const int per = (seqs + NT - 1) / NT;
  if (line.uniform) {
    total += seqs * line.uniform;
  } else if (!GATHER && seqs) {
    const int b0 = min(seqs, tid * per), b1 = min(seqs, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; b++) mine += cache_units(p, b, line.unit_shift);
    int incl = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = line.prefix_units;
    for (int x = 0; x < kWarps; x++) {
      total += s_sum[x];
      if (x < warp) before += s_sum[x];
    }
    s_first[tid] = before + incl - mine;
    __syncthreads();
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
  if (lo < hi && lo < line.prefix_units) {
    const int u1 = min(hi, line.prefix_units);
    stream_item<D, MT, BF16, false, true>(a, line.unit_shift, h, tile, 0, 0, lo, u1, line.prefix_units, group);
    lo = u1;
  }
  if (lo < hi) {
    int seq, units, start;  // the sequence that holds lo
    if (GATHER || line.uniform) {
      seq = (lo - line.prefix_units) / line.uniform;
      start = line.prefix_units + seq * line.uniform;
      units = line.uniform;
    } else {
      // the last thread whose requests begin at or before lo, then one by one
      int last = -1;
#pragma unroll
      for (int x = 0; x < NT; x += 32)
        last += __popc(__ballot_sync(0xffffffffu, s_first[x + lane] <= lo && (x + lane) * per < seqs));
      seq = last * per;
      start = s_first[last];
      units = cache_units(p, seq, line.unit_shift);
      while (start + units <= lo) {
        start += units;
        units = cache_units(p, ++seq, line.unit_shift);
      }
    }
    while (true) {
      const int b = GATHER ? seq / p.T : seq;
      stream_item<D, MT, BF16, GATHER, false>(a, line.unit_shift, h, tile, b, GATHER ? seq - b * p.T : 0, lo - start,
                                              min(units, hi - start), units, group - group_of(start));
      start += units;
      lo = start;
      if (lo >= hi) break;
      seq++;
      if (!GATHER && !line.uniform) units = cache_units(p, seq, line.unit_shift);
    }
  }
  // The finish kernel waits for this grid alone, so behind the tensor-core
  // kernel this one has to end later than that: one block waits for it (a wait of
  // every block would keep the next ones from their places).
  if (blockIdx.x == gridDim.x - 1) grid_wait();
}

template <int D, int MT, bool BF16, bool GATHER>
cudaError_t launch(const AttnArgs& a, const StreamLine& line, cudaStream_t st) {
  using C = StreamCfg<D, MT>;
  const int smem = kWarps * (GATHER ? C::WARP_BYTES : C::RING);
  auto kern = attn_stream_kernel<D, MT, BF16, GATHER>;
  static KernelReady ready;
  cudaError_t e = ready.once([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  const int blocks = line.own_blocks + (line.members * line.groups + kWarps - 1) / kWarps;
  return launch_early(kern, dim3((unsigned)blocks), 32 * kWarps, smem, st, a, line);
}

template <int D, bool BF16, bool GATHER>
cudaError_t launch_rows(const AttnArgs& a, const StreamLine& line, cudaStream_t st) {
  return line.row_tile == 16 ? launch<D, 1, BF16, GATHER>(a, line, st)
                             : launch<D, 2, BF16, GATHER>(a, line, st);
}

template <int D, bool BF16>
cudaError_t launch_kind(const AttnArgs& a, const StreamLine& line, cudaStream_t st) {
  return a.p.ids ? launch_rows<D, BF16, true>(a, line, st) : launch_rows<D, BF16, false>(a, line, st);
}

}  // namespace

cudaError_t launch_attn_stream(const AttnArgs& a, const StreamLine& line, cudaStream_t st) {
  const bool bf = a.p.dtype == IDX_BF16;
  if (a.p.D == 128) return bf ? launch_kind<128, true>(a, line, st) : launch_kind<128, false>(a, line, st);
  return bf ? launch_kind<64, true>(a, line, st) : launch_kind<64, false>(a, line, st);
}

}  // namespace idx
