// Attention over long caches in pages under more than 16 query rows of a KV head
// (drafted tokens times grouped heads), on the 5th-generation tensor cores.
//
// mma.sync is issued by the warps that also form the weights, and from 17 rows on that
// takes longer than the keys do, no less with four warps of 16 rows on one ring of
// keys.  Here a block holds up to 128 rows (TMEM lane = row; the product is of 128 rows
// however few there are) and walks tiles of 128 keys:  S = Q K^T (fp32 in TMEM);  two
// threads a row, one of each of two warpgroups, take 64 scores each into registers,
// agree on the row's maximum, form the weights 2^(y - m) and write them back over S as
// 16-bit operands;  O += P V with P read from TMEM.  S alternates between two places, so
// that the next tile's scores are formed while this one's weights are.
//
// A tile comes in boxes of consecutive slots of a page; the ring of key and value
// tiles (160 KB) keeps on filling while one sequence ends and the next begins.
// Blocks take the line of all sequences' tiles in even shares, as the warps of the
// streaming kernel do, and leave partial results for the join.
//
// Measured, with heads of 128 in bf16 and 8 KV heads: 16 requests of 8 tokens and 8 heads
// a KV head over 25,100 slots 247 us (243 at the copy rate; the streaming kernel 543); 8
// of 8 tokens and 16 heads over 12,800 81 us (62; 289); 4 of one KV head over 81,250 45
// us (26; 150).  What is left is a block's start and the end of its runs, about 9 us,
// and where the rows fill the 128 the exponentials: two threads a row take 1 us for 128
// keys, one thread took 1.3.
//
// Warp roles: warp 0 TMA producer, warp 1 MMA issue, warp 2 TMEM allocation, warps
// 4..7 and 8..11 the rows.  Waits are bounded as everywhere in the library; on a
// timeout the roles stop, the eight warps of the rows together, and drain what they
// issued.
#include "attn_paged.cuh"
#include "attn_tc_ops.cuh"

namespace idx {

namespace {

constexpr int kThreads = 384;

template <int D>
struct TcCfg {
  static constexpr int TILE = 128 * D * 2;          // 128 rows or keys
  static constexpr int NS = D == 128 ? 5 : 10;      // ring of key and value tiles
  static constexpr int SMEM = (1 + NS) * TILE + 8 * 2048 + 1024;
};

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int line, int head, int slot,
                                         int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(smem_u32(bar)), "r"(0), "r"(line), "r"(head), "r"(slot), "r"(page)
      : "memory");
}

// A run of key tiles [j0, j1) of request b, how many keys
// its last row sees, and whether the sequence's beginning and its end are in it.
struct Run {
  int b, j0, j1, most;
  bool first, last;
};

// This block's share [lo, hi) of the line of all requests' tiles.
struct Share {
  int lo, hi, seq, units, start;
  int group, each, extra;
  // The next run of the rows that end with token `token` of a step; false at the end.
  __device__ __forceinline__ bool next(const PagedArgs& a, int token, Run* r) {
    if (lo >= hi) return false;
    const paged_problem& p = a.p;
    r->b = seq;
    r->most = max(0, paged_len(p, seq) - p.T + token + 1);
    r->j0 = lo - start;
    const int u1 = min(units, hi - start);
    r->j1 = max(r->j0, min(u1, (r->most + 127) / 128));
    r->first = lo == start;
    r->last = u1 == units;
    start += units;
    lo = start;
    seq++;
    if (lo < hi) units = units_of(p, seq, 7);
    return true;
  }
};

// Barrier of the eight warps of the rows, and whether `ok` holds in all its threads.
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool rows_all(bool ok) {
  uint32_t r;
  __syncwarp();
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"((uint32_t)ok)
               : "memory");
  return r != 0;
}
// Barrier of the two warps of 32 rows.
__device__ __forceinline__ void pair_sync(int i) { asm volatile("bar.sync %0, 64;" ::"r"(i + 2) : "memory"); }

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_tc_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedArgs a,
                         const __grid_constant__ PagedLine line) {
  using C = TcCfg<D>;
  constexpr int CH = D / 8;  // 16-byte pieces of a row of queries
  constexpr int kAhead = 16;  // more tiles than the ring can be ahead of the weights
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sq = smem;
  uint8_t* skv = smem + C::TILE;
  __shared__ uint64_t kv_full[C::NS], kv_empty[C::NS], q_full, s_full[2], p_half[2], p_ready[2], o_full, pv_done, drain;
  __shared__ uint32_t s_tmem;
  __shared__ int64_t s_row[128];  // where a row's queries begin, in 16 bytes
  __shared__ unsigned s_boxes[kAhead];  // of a tile: which boxes are there
  __shared__ int s_sum[kThreads / 32], s_first[kThreads];
  __shared__ float s_top[2][2][128], s_sums[2][128];  // maxima, by the tile's parity and the half; a run's sums
  __shared__ int s_ok[2][2][4];                      // with the maxima: no wait of the warp has given up
  __shared__ int s_abort;

  const paged_problem& p = a.p;
  // (uniform for the compiler: the products' descriptors then stay in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; i++) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(&q_full, 256);
    for (int i = 0; i < 2; i++) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 128);
      mbar_init(&p_ready[i], 128);
    }
    mbar_init(&o_full, 1);
    mbar_init(&pv_done, 1);
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 2) prefetch_tmap(&maps.m[threadIdx.x]);
  if (warp == 2) tmem_alloc(&s_tmem, 512);
  // (nothing is started early behind this kernel: 3 requests of 32 rows over 8,199 slots
  // took 19.4 us instead of 16.0)
  grid_wait();
  // where on the line each thread's share of the requests begins, and its length
  const int per = (line.seqs + kThreads - 1) / kThreads;
  int total = 0;
  {
    const int b0 = min(line.seqs, (int)threadIdx.x * per), b1 = min(line.seqs, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; b++) mine += units_of(p, b, 7);
    int incl = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int x = 0; x < kThreads / 32; x++) {
      total += s_sum[x];
      if (x < warp) before += s_sum[x];
    }
    s_first[threadIdx.x] = before + incl - mine;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;

  Share share;
  share.group = (int)blockIdx.x / line.members;
  const int member = (int)blockIdx.x - share.group * line.members;
  const int rt = member / p.n_kv, h = member - rt * p.n_kv;
  {
    const int groups = min(line.groups, max(1, total / line.least));
    share.each = total / groups;
    share.extra = total - share.each * groups;
    share.lo = share.group * share.each + min(share.group, share.extra);
    share.hi = share.group < groups ? share.lo + share.each + (share.group < share.extra ? 1 : 0) : share.lo;
    share.seq = share.units = share.start = 0;
    if (share.lo < share.hi) {
      // the last thread whose requests begin at or before lo, then one by one
      int last = -1;
#pragma unroll
      for (int x = 0; x < kThreads; x += 32)
        last += __popc(__ballot_sync(0xffffffffu, s_first[x + lane] <= share.lo && (x + lane) * per < line.seqs));
      share.seq = last * per;
      share.start = s_first[last];
      share.units = units_of(p, share.seq, 7);
      while (share.start + share.units <= share.lo) {
        share.start += share.units;
        share.units = units_of(p, ++share.seq, 7);
      }
    }
  }
  const int rows = p.T * a.G, row0 = rt * 128, nrow = min(128, rows - row0);
  const int token = (row0 + nrow - 1) / a.G;  // of the last row
  Run r;

  if (warp == 0) {
    uint32_t cnt = 0;  // tiles (of keys or values) that were issued
    bool ok = true;
    while (ok && share.next(a, token, &r)) {
      const int32_t* table = p.table + r.b * p.table_stride;
      for (int j = r.j0; ok && j < r.j1; j++) {
        // lane i has box i of the tile
        const int at = lane * a.box, key = j * 128 + at;
        int page = -1, slot = 0;
        const bool wanted = at < 128 && key < r.most;
        if (wanted) {
          const int pg = (int)((uint32_t)key / (uint32_t)p.page_size);
          page = __ldg(table + pg);
          slot = key - pg * p.page_size;
        }
        const bool there = wanted && page >= 0 && page < p.n_pages;
        if (wanted && !there) atomicOr(&g_device_error, DEVERR_BAD_ROW);
        const unsigned boxes = __ballot_sync(0xffffffffu, there);
        for (int kv = 0; kv < 2; kv++) {
          const int st = cnt % C::NS;
          if (cnt >= C::NS) {
            ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[st], ((cnt / C::NS) & 1) ^ 1, abort_flag));
            if (!ok) break;
          }
          if (lane == 0) {
            if (kv == 0) *(volatile unsigned*)&s_boxes[cnt / 2 % kAhead] = boxes;
            mbar_arrive_expect_tx(&kv_full[st], __popc(boxes) * a.box * D * 2);
          }
          __syncwarp();
          if (there)
#pragma unroll
            for (int x = 0; x < D / 64; x++)
              load_box(smem_u32(skv) + st * C::TILE + x * 16384 + at * 128, &maps.m[kv], &kv_full[st], x, h, slot, page);
          cnt++;
        }
      }
    }
    // the copies in flight land before the block ends
    for (uint32_t i = cnt > C::NS ? cnt - C::NS : 0; i < cnt; i++) mbar_wait_drain(&kv_full[i % C::NS], (i / C::NS) & 1);
  } else if (warp == 1) {
    constexpr uint32_t ab = BF16 ? 1 : 0;
    constexpr uint32_t id_s = idesc_f16(128, 128, ab);
    constexpr uint32_t id_o = idesc_f16(128, D, ab) | (1u << 16);  // B is MN-major
    // descriptors of the queries and the first ring slot; others follow at their
    // distance (in 16 bytes)
    const uint64_t dq = smem_desc_sw128(smem_u32(sq)), dk = smem_desc_sw128(smem_u32(skv)), dv = desc_values(smem_u32(skv));
    uint32_t slot = 0, phase = 0;                // of the next ring slot
    uint32_t np0 = 0, np1 = 0, nq = 0;           // uses of the barriers
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
    // S in place i = Q K^T, then the barrier of its readers
    auto scores = [&](int i, uint32_t k) {
      const uint64_t k0 = dk + k * (C::TILE / 16);
#pragma unroll
      for (int s = 0; s < D / 16; s++) {
        const uint32_t off = ((s / 4) * 16384 + (s % 4) * 32) / 16;
        tc_mma_f16(tmem + 128 * i, dq + off, k0 + off, id_s, s > 0);
      }
      tc_commit(&s_full[i]);
    };
    // O += P_i V over the first or the second half of the tile's keys
    auto values = [&](int i, uint32_t v, int s0, bool add) {
      const uint64_t v0 = dv + v * (C::TILE / 16);
#pragma unroll
      for (int s = s0; s < s0 + 4; s++)
        tc_mma_f16_ts(tmem + 256, tmem + 128 * i + 8 * s, v0 + s * (2048 / 16), id_o, add || s > 0);
    };
    while (ok && share.next(a, token, &r)) {
      const int n = r.j1 - r.j0;
      if (n == 0) continue;
      ok = wait(&q_full, nq++ & 1);
      ok = ok && wait(&kv_full[slot], phase);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        scores(0, slot);
        tc_commit(&kv_empty[slot]);
      }
      __syncwarp();
      advance();
      for (int j = 0; j < n; j++) {
        const uint32_t v = slot;
        ok = wait(&kv_full[slot], phase);
        advance();
        if (!ok) break;
        const bool more = j + 1 < n;
        if (more) {
          const uint32_t k = slot;
          ok = wait(&kv_full[k], phase);
          advance();
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            scores((j + 1) & 1, k);
            tc_commit(&kv_empty[k]);
          }
          __syncwarp();
        }
        // (a barrier for each place: with one for both, the weights of two key
        // tiles could arrive while this warp is between two looks at it)
        const int pl = j & 1;
        const uint32_t parity = (pl ? np1++ : np0++) & 1;
        ok = wait(&p_half[pl], parity);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) values(pl, v, 0, j > 0);
        __syncwarp();
        ok = wait(&p_ready[pl], parity);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          values(pl, v, 4, true);
          tc_commit(&pv_done);
          if (!more) tc_commit(&o_full);
          tc_commit(&kv_empty[v]);
        }
        __syncwarp();
      }
    }
    // every product issued is done before the block's memory goes
    if (elect_one()) tc_commit(&drain);
    __syncwarp();
    mbar_wait_drain(&drain, 0);
  } else if (warp >= 4) {
    const int wg = (warp - 4) >> 2, pair = warp & 3;  // half of a tile's keys; number of the 32 rows
    const int row = pair * 32 + lane;                 // = TMEM lane
    const bool idle = pair * 32 >= nrow;  // no row of the warp is there: its lanes of P hold anything
    const uint32_t lane_off = (uint32_t)(pair * 32) << 16;
    const uint32_t to = tmem + lane_off + 256 + wg * (D / 2);  // this half of the columns' sums
    const float c = scale_of(a);
    const uint32_t flip = flip_of(a);
    uint32_t ns0 = 0, ns1 = 0, no = 0, npv = 0, cnt = 0;  // uses of the barriers; tiles
    bool ok = true;
    const bool live = row < nrow;
    const int t_row = (row0 + row) / a.G, hq_row = h * a.G + (row0 + row - t_row * a.G);
    int lim = 0;
    auto place_of = [&](int b) { return (int64_t)(share.group + b) * a.rows + t_row * p.Hq + hq_row; };
    // The next run that has tiles (without, its rows' place is marked empty): its rows'
    // limits, its queries in shared memory, in the swizzled layout of the keys: CH lanes
    // to a row, so that a row is read whole.
    auto begin = [&] {
      while (share.next(a, token, &r)) {
        if (threadIdx.x == 128 && member == 0) {
          if (r.first) a.ends[r.b].x = share.group;
          if (r.last) a.ends[r.b].y = share.group;
        }
        if (live && wg == 0 && r.j0 == r.j1) a.pml[place_of(r.b)] = make_float2(-INFINITY, 0.f);
        if (r.j0 == r.j1) continue;
        // (rows that are not there see as much as the others: zeros)
        lim = live ? max(0, paged_len(p, r.b) - p.T + t_row + 1) : r.most;
        s_row[row] = live ? (r.b * p.q_stride_b + t_row * p.q_stride_t + hq_row * p.q_stride_h) / 8 : 0;
        rows_sync();
        const int id = threadIdx.x - 128;
        uint4 v[CH / 2];
#pragma unroll
        for (int x = 0; x < CH / 2; x++) {
          const int qr = x * (256 / CH) + id / CH;
          v[x] = make_uint4(0, 0, 0, 0);
          if (qr < nrow) v[x] = __ldg(reinterpret_cast<const uint4*>(p.q) + s_row[qr] + id % CH);
        }
#pragma unroll
        for (int x = 0; x < CH / 2; x++) {
          const int qr = x * (256 / CH) + id / CH, ch = id % CH;
          v[x].x ^= flip;
          v[x].y ^= flip;
          v[x].z ^= flip;
          v[x].w ^= flip;
          *reinterpret_cast<uint4*>(sq + (ch / 8) * 16384 + qr * 128 + (((ch & 7) ^ (qr & 7)) << 4)) = v[x];
        }
        fence_proxy_async_smem();
        rows_sync();  // (s_row is written again for the next run)
        mbar_arrive(&q_full);
        return true;
      }
      return false;
    };
    bool more_runs = begin();
    while (more_runs) {
      const int n = r.j1 - r.j0, j0 = r.j0, most = r.most, lim_run = lim;
      const int64_t at = place_of(r.b);

      float m = -INFINITY;
      uint64_t l2[4];
#pragma unroll
      for (int q = 0; q < 4; q++) l2[q] = f2_pack(0.f, 0.f);
      for (int j = j0; j < j0 + n; j++) {
        const int place = (j - j0) & 1;
        const uint32_t ts = tmem + lane_off + 128 * place;
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[place], (place ? ns1 : ns0) & 1, abort_flag));
        if (!ok && idle) break;  // (the others leave in pairs, below)
        ns0 += place ^ 1;
        ns1 += place;
        tc_fence_after();
        const int most_left = min(128, most - j * 128);
        const unsigned boxes = *(volatile unsigned*)&s_boxes[cnt / 2 % kAhead];
        const bool holes = boxes != (2u << ((most_left - 1) / a.box)) - 1;  // a page out of range
        if (most_left < 128 || holes) {
          // slots that no row sees are not data: their values must not reach the
          // product, where 0 * NaN would
          const uint32_t v = cnt + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[v % C::NS], (v / C::NS) & 1, abort_flag)) && ok;
          if (wg == 0 && ok && (row >= most_left || !(boxes >> (row / a.box) & 1))) {
            uint4* z = reinterpret_cast<uint4*>(skv + (v % C::NS) * C::TILE + row * 128);
#pragma unroll
            for (int x = 0; x < D / 64; x++)
#pragma unroll
              for (int e = 0; e < 8; e++) z[x * 1024 + e] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        cnt += 2;
        if (idle) {
          mbar_arrive(wg ? &p_ready[place] : &p_half[place]);
          continue;
        }
        // the thread's 64 scores, the second half on its way while the first is used;
        // maxima and sums run in four chains each
        uint32_t s[2][32];
        float tops[4];
        const int left = lim_run - j * 128 - 64 * wg;  // of its keys, those that the row sees
        const bool cut = holes || __any_sync(0xffffffffu, left < 64);
        tmem_ld_32x32b_x32(ts + 64 * wg, s[0]);
        tmem_ld_wait();
        tie(s[0]);
        tmem_ld_32x32b_x32(ts + 64 * wg + 32, s[1]);
        auto look = [&](int x) {
          if (cut) {
            // (boxes have 8 keys at least: a bit for each eighth of the 32)
#pragma unroll
            for (int g = 0; g < 4; g++) {
              const bool there = boxes >> ((64 * wg + 32 * x + 8 * g) / a.box) & 1;
#pragma unroll
              for (int e = 8 * g; e < 8 * g + 8; e++)
                if (!there || 32 * x + e >= left) s[x][e] = 0xff800000u;  // -inf
            }
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
        tmem_ld_wait();
        tie(s[1]);
        look(1);
        // the maximum over both halves; behind this barrier both have read the scores,
        // over which the weights are written
        float* tops_at = s_top[(j - j0) & 1][0];
        tops_at[128 * wg + row] = max3(tops[0], tops[1], fmaxf(tops[2], tops[3]));
        volatile int* oks = s_ok[(j - j0) & 1][0];
        if (lane == 0) oks[4 * wg + pair] = ok;
        tc_fence_before();
        pair_sync(pair);
        tc_fence_after();
        ok = oks[pair] && oks[4 + pair];
        if (!ok) break;  // both warps of the pair
        const float top = fmaxf(tops_at[row], tops_at[128 + row]) * c;
        // The reference moves only when a score passes it by more than 2^8 (weights
        // up to 2^8 lose nothing): the accumulator is almost never rescaled.  With fp16
        // it is set 11 below the maximum and moves at kLift.
        //   Steep scores, from 2^20 in log2 units on, leave this no room: 2^(c s - m) with c
        // s unrounded, in one fma, is 2^(half the last bit of m) for the largest score,
        // and infinite from 2^31 on.  They are multiplied first, so that the largest is
        // met exactly, and their reference is the maximum itself.
        constexpr float kSteep = 0x1p20f, below = BF16 ? 0.f : 11.f, late = BF16 ? 8.f : kLift<BF16>;
        const bool move = top > m + (fabsf(top) >= kSteep ? 0.f : late);  // also from -inf to the first score
        if (__any_sync(0xffffffffu, move)) {
          const float to_m = !move ? m : fabsf(top) >= kSteep ? top : top - below;
          const float f = move ? attn_ex2(m - to_m) : 1.f;
          m = to_m;
          const uint64_t f2 = f2_pack(f, f), zero = f2_pack(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 4; q++) l2[q] = f2_fma(l2[q], f2, zero);
          if (j > j0) {
            // the accumulator has to be at rest: the product with V of the tile before
            mbar_wait(&pv_done, (npv + (j - j0) - 1) & 1, abort_flag);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < D / 64; x++) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(to + 32 * x, o);
              tmem_ld_wait();
              tie(o);
#pragma unroll
              for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x32(to + 32 * x, o);
            }
            // (the product over the first half of the keys adds to all columns)
            tmem_st_wait();
            tc_fence_before();
            pair_sync(pair);
            tc_fence_after();
          }
        }
        // The weights are rounded to the element type, which the 16-bit operand has
        // to be (in error as much as the output's own rounding; fp16 ones below 2^-25 of
        // the largest by 2^-36 of it); their sum, which divides the output, is of the
        // unrounded ones.
        const float base = m == -INFINITY ? 0.f : m;
        const bool steep = __any_sync(0xffffffffu, fabsf(base) >= kSteep);
        const float cs = steep ? 1.f : c;
        if (steep)
#pragma unroll
          for (int e = 0; e < 64; e++) s[e / 32][e % 32] = __float_as_uint(__uint_as_float(s[e / 32][e % 32]) * c);
        const uint64_t c2 = f2_pack(cs, cs), b2 = f2_pack(-base, -base), one = f2_pack(1.f, 1.f);
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 32; e++) {
          const int y = e / 16, z = 2 * (e & 15);
          float p0, p1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(s[y][z]), __uint_as_float(s[y][z + 1])), c2, b2), &p0, &p1);
          p0 = attn_ex2(p0);
          p1 = attn_ex2(p1);
          l2[e & 3] = f2_fma(f2_pack(p0, p1), one, l2[e & 3]);
          w[e] = pack2<BF16>(p0, p1);
        }
        tmem_st_32x32b_x32(ts + 32 * wg, w);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(wg ? &p_ready[place] : &p_half[place]);
      }
      // A wait that gives up does so in one warp: another's can still succeed a
      // moment later.  The barriers below count all eight warps, so they go on or
      // leave together, by votes that every one of them reaches.
      ok = rows_all(ok);
      if (!ok) break;
      // The next run's queries take the place of this one's, whose last scores are
      // there: their product runs while the sums of this run leave.
      more_runs = begin();
      ok = rows_all(mbar_wait(&o_full, no++ & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      npv += n;
      float l = 0.f;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        float l0, l1;
        f2_unpack(l2[q], &l0, &l1);
        l += l0 + l1;
      }
      if (!idle) {
        float* sums_at = s_sums[0];
        sums_at[128 * wg + row] = l;
        pair_sync(pair);
        l = sums_at[row] + sums_at[128 + row];
        if (live && wg == 0) a.pml[at] = make_float2(l != 0.f ? m + kLift<BF16> : -INFINITY, l);
        // the sums leave through 2 KB of the warp's own, 16 columns at a time, so that
        // four lanes write 64 bytes of a row next to one another
        uint8_t* stage = smem + (1 + C::NS) * C::TILE + (warp - 4) * 2048;
        const int64_t to_row = live && l != 0.f ? at : -1;  // (l is NaN where a score was)
#pragma unroll
        for (int x = 0; x < D / 64; x++) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(to + 32 * x, o);
          tmem_ld_wait();
          tie(o);
#pragma unroll
          for (int y = 0; y < 2; y++) {
#pragma unroll
            for (int e = 0; e < 4; e++)
              *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(o[16 * y + 4 * e], o[16 * y + 4 * e + 1], o[16 * y + 4 * e + 2], o[16 * y + 4 * e + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const int qr = 8 * i + lane / 4, ch = lane & 3;
              const int64_t row_at = __shfl_sync(0xffffffffu, to_row, qr);
              if (row_at >= 0)
                *reinterpret_cast<uint4*>(a.po + row_at * D + wg * (D / 2) + 32 * x + 16 * y + 4 * ch) =
                    *reinterpret_cast<const uint4*>(stage + qr * 64 + ((ch ^ ((qr >> 1) & 3)) << 4));
            }
            __syncwarp();
          }
        }
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

template <int D, bool BF16>
cudaError_t launch(const PagedArgs& a, const PagedMaps& maps, const PagedLine& line, cudaStream_t st) {
  auto kern = attn_paged_tc_kernel<D, BF16>;
  static KernelReady ready;
  cudaError_t e = ready.once([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TcCfg<D>::SMEM); });
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3((unsigned)(line.members * line.groups)), kThreads, TcCfg<D>::SMEM, st, maps, a, line);
}

}  // namespace

cudaError_t launch_attn_paged_tc(const PagedArgs& a, const PagedMaps& maps, const PagedLine& line, cudaStream_t st) {
  const bool bf = a.p.dtype == IDX_BF16;
  if (a.p.D == 128) return bf ? launch<128, true>(a, maps, line, st) : launch<128, false>(a, maps, line, st);
  return bf ? launch<64, true>(a, maps, line, st) : launch<64, false>(a, maps, line, st);
}

}  // namespace idx
