// Attention of many rows over the shared prefix on the 5th-generation tensor
// cores: every request's query heads read the same keys and values, so the
// rows of a KV head form the M axis of one long matrix problem.
//
// A block holds two tiles of 128 rows (TMEM lane = row) and walks tiles of 128
// keys.  Per key tile and row tile:  S = Q K^T (fp32 in TMEM, both operands in
// shared memory);  one warpgroup, a thread per row, takes the row's 128 scores
// into registers, forms the weights 2^(y - m) and writes them back over S as
// 16-bit operands;  O += P V with P read from TMEM.  The two row tiles
// alternate: while one's weights are formed, the other's products run.
//
// A tile's weights are handed over in two halves of 64 keys: the product over
// the first runs while the second is formed, which takes the time that a row
// tile waits for its weights (1,350 cycles for 128 keys) below the 1,024 cycles
// of the other one's products.
//
// The reference m of a row moves only when a score passes it by more than 2^8
// (weights up to 2^8 lose nothing in fp32 sums or in the 16-bit operands), so
// the accumulator in TMEM is almost never rescaled.
//
// Work is (KV head, piece of the keys, pair of row tiles, key tile), row tiles
// inside pieces: blocks that run together read the same keys, which then come
// from L2.  The line of key tiles is cut evenly over the SMs, or piece by piece
// where the pieces fill them; a block leaves one partial result per piece it
// touched and the finish kernel joins them.
//
// 1,024 rows of each of 8 KV heads over 65,536 keys of 128 (275 GFLOP) take 174
// us alone, 1.58 PFLOP/s; a unit of two row tiles and a key tile about 2,600
// cycles, 2,048 of them its products.
//
// Warp roles: warp 0 TMA producer, warp 1 MMA issue, warp 2 TMEM allocation,
// warps 4..7 and 8..11 the two row tiles.  Waits are bounded as everywhere in
// the library; on a timeout the roles stop, the four warps of a row tile
// together, and drain what they issued.
#include "attn_tc.cuh"

namespace idx {

namespace {

constexpr int kThreadsTc = 384;
// After setmaxnreg: warps 0..3, and the softmax warps, which hold a row's 128
// scores.  4 * 72 + 8 * 216 = 12 * 168, the launch's registers.
constexpr int kRegsIssue = 72, kRegsSoftmax = 216;

template <int D>
struct TcCfg {
  static constexpr int TILE = 128 * D * 2;            // 128 rows or keys
  static constexpr int NS = D == 128 ? 5 : 8;         // ring of key and value tiles
  static constexpr int SMEM = 2 * TILE + NS * TILE + 1024;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(tmap), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], kind::f16.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// True in one lane, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// Ties the registers of a tcgen05.ld to the wait before it, so that no use of
// them can be scheduled ahead of that wait.
__device__ __forceinline__ void tie(uint32_t (&r)[32]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                    "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
  asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                    "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                    "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Values as the second operand: rows of the tile are keys (the K axis), 64
// dims to a 128-byte row, so the operand is MN-major with the 128-byte swizzle:
// 8-key groups follow at 1024 bytes, the next 64 dims at 128 keys * 128 bytes.
__device__ __forceinline__ uint64_t desc_values(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3ffffu) >> 4);
  d |= (uint64_t)(16384u >> 4) << 16;  // leading byte offset: between 64-dim chunks
  d |= (uint64_t)(1024u >> 4) << 32;   // stride byte offset: between 8-key groups
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// Barrier of the four warps of a row tile.
__device__ __forceinline__ void row_tile_sync(int i) { asm volatile("bar.sync %0, 128;" ::"r"(i + 1) : "memory"); }
// The same barrier, and whether `ok` holds in all its 128 threads.
__device__ __forceinline__ bool row_tile_all(int i, bool ok) {
  uint32_t r;
  __syncwarp();
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"((uint32_t)ok), "r"(i + 1)
               : "memory");
  return r != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// A run of key tiles [j0, j1) of one (KV head, pair of row tiles).
struct Run {
  int h, rt, j0, j1, part;
};

// The line of units and this block's share of it.
struct Line {
  int tiles, cells_k, rts, heads;  // key tiles, pieces of the keys, row tile pairs, KV heads
  int u, u0, u1;                   // the share, and how far this role has come
  int cell, longer;                // key tiles of a piece; the first `longer` pieces have one more
  bool whole;
  __device__ __forceinline__ int cell_start(int kc) const { return kc * cell + min(kc, longer); }
  __device__ __forceinline__ void init(int tiles_, const AttnTcArgs& a) {
    tiles = tiles_;
    cells_k = min(a.cells_k, tiles);
    rts = a.row_tiles;
    heads = a.a.p.n_kv;
    const int c = (int)blockIdx.x;
    whole = a.whole_cells;
    cell = cells_k ? tiles / cells_k : 0;
    longer = tiles - cell * cells_k;
    const int total = heads * rts * tiles, n = (int)gridDim.x;  // total is below 2^31, the plan checks
    if (tiles == 0) {
      u0 = u1 = 0;
    } else if (whole) {
      u0 = c;  // one cell: block index (h, kc, rt)
      u1 = c < heads * cells_k * rts ? c + 1 : c;
    } else {
      const int each = total / n, extra = total - each * n;
      u0 = c * each + min(c, extra);
      u1 = u0 + each + (c < extra ? 1 : 0);
    }
    u = u0;
  }
  // The next run of this block; false at its end.
  __device__ __forceinline__ bool next(Run* r) {
    if (u >= u1) return false;
    if (whole) {
      const int q = u / rts;
      r->rt = u - q * rts;
      r->h = q / cells_k;
      r->part = q - r->h * cells_k;
      r->j0 = cell_start(r->part);
      r->j1 = cell_start(r->part + 1);
      u++;
      return true;
    }
    // unit u lies in head h; in it, cells of (piece, row tile pair)
    const int per = rts * tiles;
    r->h = u / per;
    const int in = u - r->h * per;
    const int x = in / rts, head = longer * (cell + 1);
    const int kc = x < head ? x / (cell + 1) : longer + (x - head) / cell;
    const int s = cell_start(kc), len = cell + (kc < longer ? 1 : 0);
    const int off = in - s * rts;
    r->rt = off / len;
    const int at = off - r->rt * len;
    r->j0 = s + at;
    r->j1 = min(s + len, r->j0 + (u1 - u));
    // the cell's first unit lies in this block's share, or in the one before
    r->part = 2 * kc + (u - at < u0 ? 1 : 0);
    u += r->j1 - r->j0;
    return true;
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreadsTc, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ AttnTcArgs args) {
  using C = TcCfg<D>;
  constexpr int CH = D / 8;  // 16-byte pieces of a row of queries
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sq = smem;
  uint8_t* skv = smem + 2 * C::TILE;
  __shared__ uint64_t kv_full[C::NS], kv_empty[C::NS], q_full[2], s_full[2], p_half[2], p_ready[2], o_full[2], pv_done, drain;
  __shared__ uint32_t s_tmem;
  // where a row's queries begin, in 16 bytes; then the number of its partial result
  __shared__ int s_row[2][128];
  __shared__ int s_abort, s_vis;

  const AttnArgs& a = args.a;
  const attn_problem& p = a.p;
  // A warp index that is uniform for the compiler, and a warp that runs
  // converged around the issue of its products: their descriptors then stay in
  // uniform registers (24 cycles a product; from one lane's own it was 45, and
  // twice that next to the softmax warps, more than a product takes).
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int parts_all = a.parts_prefix + a.parts_private;

  grid_wait();
  grid_let_next_start();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; i++) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&q_full[i], 128);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 128);
      mbar_init(&p_ready[i], 128);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(&pv_done, 1);
    mbar_init(&drain, 1);
    s_abort = 0;
    s_vis = p.prefix_len ? 0 : (int)p.P;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc(&s_tmem, 512);
  if (p.prefix_len) {
    int v = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreadsTc) v = max(v, (int)attn_prefix_len(p, b));
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0 && v) atomicMax(&s_vis, v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int vis = s_vis;  // no row sees a position at or behind it
  volatile int* abort_flag = &s_abort;
  const int rows = p.B * p.T * a.G;
  Line line;
  line.init((vis + 127) / 128, args);

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue) : "memory");
  if (warp == 0) {
    if (lane == 0) {
      uint32_t cnt = 0;  // tiles loaded
      bool ok = true;
      Run r;
      while (ok && line.next(&r)) {
        for (int j = r.j0; ok && j < r.j1; j++)
          for (int kv = 0; kv < 2; kv++) {
            const int st = cnt % C::NS;
            if (cnt >= C::NS && !mbar_wait(&kv_empty[st], ((cnt / C::NS) & 1) ^ 1, abort_flag)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&kv_full[st], C::TILE);
#pragma unroll
            for (int x = 0; x < D / 64; x++)
              tma_load_3d(smem_u32(skv) + st * C::TILE + x * 16384, kv ? &tv : &tk, &kv_full[st], x * 64, j * 128,
                          r.h);
            cnt++;
          }
      }
      // the copies in flight land before the block ends
      for (uint32_t i = cnt > C::NS ? cnt - C::NS : 0; i < cnt; i++)
        mbar_wait_drain(&kv_full[i % C::NS], (i / C::NS) & 1);
    }
  } else if (warp == 1) {
    constexpr uint32_t ab = BF16 ? 1 : 0;
    constexpr uint32_t id_s = idesc_f16(128, 128, ab);
    constexpr uint32_t id_o = idesc_f16(128, D, ab) | (1u << 16);  // B is MN-major
    // descriptors of the first query tile and the first ring slot; others follow
    // at their distance (in 16 bytes)
    const uint64_t dq = smem_desc_sw128(smem_u32(sq)), dk = smem_desc_sw128(smem_u32(skv)),
                   dv = desc_values(smem_u32(skv));
    uint32_t slot = 0, phase = 0;  // of the next ring slot
    uint32_t np = 0, np1 = 0, nq0 = 0, nq1 = 0;  // uses of the barriers
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
    };
    auto advance = [&] {
      if (++slot == C::NS) {
        slot = 0;
        phase ^= 1;
      }
    };
    // S_i = Q_t K^T, then the barrier of its readers
    auto scores = [&](int i, int t, uint32_t k) {
      const uint64_t q0 = dq + t * (C::TILE / 16), k0 = dk + k * (C::TILE / 16);
#pragma unroll
      for (int s = 0; s < D / 16; s++) {
        const uint32_t off = ((s / 4) * 16384 + (s % 4) * 32) / 16;
        tc_mma_f16(tmem + 128 * i, q0 + off, k0 + off, id_s, s > 0);
      }
      tc_commit(&s_full[i]);
    };
    // O_t += P_i V over the first or the second half of the tile's keys
    auto values = [&](int i, int t, uint32_t v, int s0, bool add) {
      const uint64_t v0 = dv + v * (C::TILE / 16);
#pragma unroll
      for (int s = s0; s < s0 + 4; s++)
        tc_mma_f16_ts(tmem + 256 + 128 * t, tmem + 128 * i + 8 * s, v0 + s * (2048 / 16), id_o, add || s > 0);
    };
    Run r;
    while (ok && line.next(&r)) {
      const bool two = rows - r.rt * 256 > 128;  // both row tiles have rows
      const int n = r.j1 - r.j0;
      ok = wait(&q_full[0], nq0++ & 1);
      if (two) ok = ok && wait(&q_full[1], nq1++ & 1);
      ok = ok && wait(&kv_full[slot], phase);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        scores(0, 0, slot);
        if (two) scores(1, 1, slot);
        tc_commit(&kv_empty[slot]);
      }
      __syncwarp();
      advance();
      for (int j = 0; j < n; j++) {
        const uint32_t v = slot;
        ok = wait(&kv_full[slot], phase);
        advance();
        if (!ok) break;
        const uint32_t k = slot, k_phase = phase;
        const bool more = j + 1 < n;
        if (more) advance();
        if (!two) {
          // One row tile: its scores alternate between the two places, so that
          // the next key tile's are formed while this one's weights are.
          if (more) ok = wait(&kv_full[k], k_phase);
          if (!ok) break;
          tc_fence_after();
          if (more && elect_one()) {
            scores((j + 1) & 1, 0, k);
            tc_commit(&kv_empty[k]);
          }
          __syncwarp();
          // (a barrier for each place: with one for both, the weights of two
          // key tiles could arrive while this warp is between two looks at it)
          const int pl = j & 1;
          const uint32_t parity = (pl ? np1++ : np++) & 1;
          ok = wait(&p_half[pl], parity);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) values(pl, 0, v, 0, j > 0);
          __syncwarp();
          ok = wait(&p_ready[pl], parity);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            values(pl, 0, v, 4, true);
            tc_commit(&pv_done);
            if (!more) {
              tc_commit(&o_full[0]);
              tc_commit(&o_full[1]);  // the other row tile's warps wait for the run's end
            }
            tc_commit(&kv_empty[v]);
          }
          __syncwarp();
          continue;
        }
        ok = wait(&p_half[0], np & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) values(0, 0, v, 0, j > 0);
        __syncwarp();
        ok = wait(&p_ready[0], np++ & 1);
        if (ok && more) ok = wait(&kv_full[k], k_phase);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          values(0, 0, v, 4, true);
          if (more)
            scores(0, 0, k);
          else
            tc_commit(&o_full[0]);
        }
        __syncwarp();
        ok = wait(&p_half[1], np1 & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) values(1, 1, v, 0, j > 0);
        __syncwarp();
        ok = wait(&p_ready[1], np1++ & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          values(1, 1, v, 4, true);
          if (more)
            scores(1, 1, k);
          else
            tc_commit(&o_full[1]);
          tc_commit(&kv_empty[v]);
          if (more) tc_commit(&kv_empty[k]);
        }
        __syncwarp();
      }
    }
    // every product issued is done before the block's memory goes
    if (elect_one()) tc_commit(&drain);
    __syncwarp();
    mbar_wait_drain(&drain, 0);
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax) : "memory");
    const int i = (warp - 4) >> 2;              // row tile
    const int row = threadIdx.x - 128 - 128 * i;  // its row, = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lane_off + 256 + 128 * i;
    // 2^(c s - m): a negative scale goes into the queries' sign, and a scale of
    // zero becomes one that takes every score to zero but leaves -inf alone
    const float c = fmaxf(fabsf(a.scale_log2), 1e-37f);
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
    // ns: uses of the scores' two places; npv: products with V of runs with one row tile
    uint32_t ns0 = 0, ns1 = 0, no = 0, npv = 0, cnt = 0;
    bool ok = true;
    Run r;
    while (ok && line.next(&r)) {
      const int n = r.j1 - r.j0;
      const int rr = r.rt * 256 + i * 128 + row;
      const bool two = rows - r.rt * 256 > 128;
      if (i == 1 && !two) {
        // An empty row tile: the other one uses both places.  Its barriers are
        // this one's again when the run is over.
        ns1 += n / 2;
        ok = row_tile_all(i, mbar_wait(&o_full[1], no++ & 1, abort_flag));
        continue;
      }
      if (i == 0 && two) ns1 += n;  // the other tile's
      const bool live = rr < rows;
      int rid = -1, lim = 0;
      if (live) {
        const int bt = rr / a.G, g = rr - bt * a.G;
        const int b = bt / p.T, t = bt - b * p.T;
        const int hq = r.h * a.G + g;
        rid = bt * p.Hq + hq;
        lim = (int)attn_prefix_len(p, b);
        s_row[i][row] = (int)((b * p.q_stride_b + t * p.q_stride_t + hq * p.q_stride_h) / 8);
      }
      row_tile_sync(i);
      // the queries, in the swizzled layout of the keys: CH lanes to a row, so
      // that a row is read whole
      {
        uint4 v[CH];
#pragma unroll
        for (int x = 0; x < CH; x++) {
          const int qr = x * (128 / CH) + row / CH;
          v[x] = make_uint4(0, 0, 0, 0);
          if (r.rt * 256 + i * 128 + qr < rows)
            v[x] = __ldg(reinterpret_cast<const uint4*>(p.q) + (int64_t)s_row[i][qr] + row % CH);
        }
#pragma unroll
        for (int x = 0; x < CH; x++) {
          const int qr = x * (128 / CH) + row / CH, ch = row % CH;
          v[x].x ^= flip;
          v[x].y ^= flip;
          v[x].z ^= flip;
          v[x].w ^= flip;
          *reinterpret_cast<uint4*>(sq + i * C::TILE + (ch / 8) * 16384 + qr * 128 + (((ch & 7) ^ (qr & 7)) << 4)) = v[x];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&q_full[i]);

      float m = -INFINITY;
      uint64_t l2[4];
#pragma unroll
      for (int q = 0; q < 4; q++) l2[q] = f2_pack(0.f, 0.f);
      for (int j = r.j0; j < r.j1; j++) {
        const int place = two ? i : (j - r.j0) & 1;
        const uint32_t ts = tmem + lane_off + 128 * place;
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[place], (place ? ns1++ : ns0++) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        // the row's scores, the second half on its way while the first is used;
        // maxima and sums run in four chains each, the latency of one would be
        // longer than the products
        uint32_t s[4][32];
        float tops[4];
        const int left = lim - j * 128;  // keys of the tile that the row sees
        const bool cut = __any_sync(0xffffffffu, left < 128);
        tmem_ld_32x32b_x32(ts, s[0]);
        tmem_ld_32x32b_x32(ts + 32, s[1]);
        tmem_ld_wait();
        tie(s[0]);
        tie(s[1]);
        tmem_ld_32x32b_x32(ts + 64, s[2]);
        tmem_ld_32x32b_x32(ts + 96, s[3]);
        auto look = [&](int x) {
          if (cut) {
#pragma unroll
            for (int e = 0; e < 32; e++)
              if (32 * x + e >= left) s[x][e] = 0xff800000u;  // -inf
          }
          if (x == 0) {
#pragma unroll
            for (int q = 0; q < 4; q++) tops[q] = __uint_as_float(s[0][q]);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8)
#pragma unroll
            for (int q = 0; q < 4; q++)
              tops[q] = max3(tops[q], __uint_as_float(s[x][e + 2 * q]), __uint_as_float(s[x][e + 2 * q + 1]));
        };
        look(0);
        look(1);
        tmem_ld_wait();
        tie(s[2]);
        tie(s[3]);
        look(2);
        look(3);
        float top = max3(tops[0], tops[1], fmaxf(tops[2], tops[3]));
        top *= c;
        const bool move = top > m + 8.f;  // also from -inf to the first score
        if (__any_sync(0xffffffffu, move)) {
          const float to_m = move ? top : m;
          const float f = move ? attn_ex2(m - top) : 1.f;
          m = to_m;
          const uint64_t f2 = f2_pack(f, f), zero = f2_pack(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 4; q++) l2[q] = f2_fma(l2[q], f2, zero);
          if (j > r.j0) {
            // The accumulator has to be at rest.  With two row tiles these scores
            // were formed after the last product with V; with one they were not,
            // and that product has to be waited for.
            if (!two) mbar_wait(&pv_done, (npv + (j - r.j0) - 1) & 1, abort_flag);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < D / 32; x++) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(to + 32 * x, o);
              tmem_ld_wait();
              tie(o);
#pragma unroll
              for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x32(to + 32 * x, o);
            }
          }
        }
        if (i == 0 && vis < p.P && j * 128 + 128 > vis) {
          // positions behind every row's limit are not data: their values
          // must not reach the product, where 0 * NaN would
          const uint32_t v = cnt + 1;
          ok = mbar_wait(&kv_full[v % C::NS], (v / C::NS) & 1, abort_flag);
          if (ok && row >= vis - j * 128) {
            uint4* z = reinterpret_cast<uint4*>(skv + (v % C::NS) * C::TILE + row * 128);
#pragma unroll
            for (int x = 0; x < D / 64; x++)
#pragma unroll
              for (int e = 0; e < 8; e++) z[x * 1024 + e] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        // The weights are rounded to the element type, which the 16-bit operand has
        // to be (in error as much as the output's own rounding); their sum, which
        // divides the output, is of the unrounded ones.
        const float base = m == -INFINITY ? 0.f : m;
        const uint64_t c2 = f2_pack(c, c), b2 = f2_pack(-base, -base), one = f2_pack(1.f, 1.f);
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; e++) {
            const int y = x + e / 16, z = 2 * (e & 15);
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[y][z]), __uint_as_float(s[y][z + 1])), c2, b2), &p0, &p1);
            p0 = attn_ex2(p0);
            p1 = attn_ex2(p1);
            l2[e & 3] = f2_fma(f2_pack(p0, p1), one, l2[e & 3]);
            w[e] = pack2<BF16>(p0, p1);
          }
          tmem_st_32x32b_x32(ts + 16 * x, w);
          if (x == 0) {  // the product over the first half of the keys can start
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&p_half[place]);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_ready[place]);
        cnt += 2;
      }
      // A wait that gives up does so in one warp: another's can still succeed a
      // moment later.  The barriers below count all four warps of the row tile, so
      // they go on or leave together, by one vote a run that every one of them
      // reaches, whatever its own waits returned.
      ok = row_tile_all(i, ok && mbar_wait(&o_full[i], no++ & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      if (!two) npv += n;
      float l = 0.f;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        float l0, l1;
        f2_unpack(l2[q], &l0, &l1);
        l += l0 + l1;
      }
      const int64_t at = (int64_t)rid * parts_all + r.part;
      if (live) {
        a.pml[at] = make_float2(l != 0.f ? m : -INFINITY, l);
        // a cell that one block did alone has no second part
        if (!line.whole && (r.part & 1) == 0 && r.j1 == line.cell_start(r.part / 2 + 1))
          a.pml[at + 1] = make_float2(-INFINITY, 0.f);
      }
      s_row[i][row] = live && l != 0.f ? (int)at : -1;  // (l is NaN where a score was)
      // the sums leave through the memory of the queries, half of a row at a
      // time, so that CH lanes write one row's half next to one another
#pragma unroll
      for (int half = 0; half < 2; half++) {
        uint8_t* stage = sq + i * C::TILE;
#pragma unroll
        for (int x = 0; x < D / 64; x++) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(to + half * (D / 2) + 32 * x, o);
          tmem_ld_wait();
          tie(o);
#pragma unroll
          for (int e = 0; e < 8; e++)
            *reinterpret_cast<uint4*>(stage + row * (2 * D) + (((8 * x + e) ^ (row & 7)) << 4)) =
                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
        row_tile_sync(i);
#pragma unroll 4
        for (int x = 0; x < CH; x++) {
          const int qr = x * (128 / CH) + row / CH, ch = row % CH;
          const int64_t to_row = s_row[i][qr];
          if (to_row >= 0)
            *reinterpret_cast<uint4*>(a.po + to_row * D + half * (D / 2) + 4 * ch) =
                *reinterpret_cast<const uint4*>(stage + qr * (2 * D) + ((ch ^ (qr & 7)) << 4));
        }
        row_tile_sync(i);
      }
      tc_fence_before();
    }
    // pieces that the visible prefix does not reach
    const int used = line.cells_k * (line.whole ? 1 : 2);
    if (used < a.parts_prefix) {
      const int64_t all = (int64_t)p.B * p.T * p.Hq;
      for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x - 128; x < all; x += (int64_t)gridDim.x * 256)
        for (int y = used; y < a.parts_prefix; y++) a.pml[x * parts_all + y] = make_float2(-INFINITY, 0.f);
    }
  }
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

template <int D, bool BF16>
cudaError_t launch(const AttnTcArgs& t, cudaStream_t st) {
  using C = TcCfg<D>;
  const attn_problem& p = t.a.p;
  CUtensorMap tk, tv;
  const CUtensorMapDataType dt = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  // one head: its stride is never used, but has to be a legal one
  const int64_t kh = p.n_kv > 1 ? p.pk_stride_h : p.D, vh = p.n_kv > 1 ? p.pv_stride_h : p.D;
  const int64_t ks = p.P > 1 ? p.pk_stride_s : p.D, vs = p.P > 1 ? p.pv_stride_s : p.D;
  if (!make_tmap_3d(&tk, dt, p.pk, D, (uint64_t)p.P, (uint64_t)p.n_kv, 2 * ks, 2 * kh, 64, 128) ||
      !make_tmap_3d(&tv, dt, p.pv, D, (uint64_t)p.P, (uint64_t)p.n_kv, 2 * vs, 2 * vh, 64, 128))
    return cudaErrorInvalidValue;
  auto kern = attn_tc_kernel<D, BF16>;
  static KernelReady ready;
  cudaError_t e = ready.once([&]() -> cudaError_t {
    // setmaxnreg moves registers within the block: what the softmax warps take
    // must not exceed what the others give back from the launch count
    cudaFuncAttributes fa;
    cudaError_t x = cudaFuncGetAttributes(&fa, kern);
    if (x != cudaSuccess) return x;
    if (4 * kRegsIssue + 8 * kRegsSoftmax > 12 * fa.numRegs || fa.numRegs > kRegsSoftmax) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3((unsigned)t.blocks), kThreadsTc, C::SMEM, st, tk, tv, t);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnTcArgs& t, cudaStream_t st) {
  const bool bf = t.a.p.dtype == IDX_BF16;
  if (t.a.p.D == 128) return bf ? launch<128, true>(t, st) : launch<128, false>(t, st);
  return bf ? launch<64, true>(t, st) : launch<64, false>(t, st);
}

}  // namespace idx
