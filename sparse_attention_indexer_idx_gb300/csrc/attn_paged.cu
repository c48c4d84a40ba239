// Attention of a decode step over caches in pages, bound by reading keys and
// values.
//
// Mathematics.  For a row of a KV head (a query head and a token), over the slots it
// sees:  y = scale log2(e) q.k,  out = sum 2^(y - m) v / sum 2^(y - m)  with the running
// maximum m, everything but the operands of the two products in fp32.  The weights are
// rounded to 16 bits for the second product, half a step each, as the values are; their
// sum is taken before the rounding.
//
// Every warp is a stream of its own: it brings tiles of KT keys and values (8 KB) into a
// ring of two and keeps the running maximum, sum and output in registers.  Tiles come
// as boxes of consecutive slots of a page by TMA; row by row with 16-byte cp.async where
// a page holds no whole box of 8 slots or no tensor map can hold the pools, and for
// lists of slots.  Lane i of a warp finds the page of the tile's i-th key one tile
// ahead of the copy, so the table's latency is waited for at a sequence's start only,
// and a page may end inside a tile, hold one slot, or lie anywhere.
//
// The products use mma.sync (16 x 8 x 16): for 1 to 16 rows a KV head the tensor work is
// a few percent of the time the bytes take, and the register layout of its accumulators
// is the operand layout of the second product, so the weights never leave registers.
// Long calls with more rows than that go to the tensor cores (attn_paged_tc.cu).
//
// Short calls.  A cluster of 1 to 16 blocks has a sequence, KV head and row tile; its
// warps take every n-th tile, and the blocks send their sums to one another's shared
// memory, each for the part of the output that it writes.  One launch, no workspace: 6
// us for one request of 1,200 slots and 8 KV heads, 11 with the line and its join.
//
// Long calls.  The key sequences (every request's cache, or every token's list) form
// one line of units of one or more key tiles, cut evenly over groups of warps, with one
// warp of a group for each KV head (and tile of up to 32 query rows).  A group that
// starts or ends inside a sequence leaves a partial result, which attn_paged_join.cu
// joins with the others.  The heads of a group run side by side, so a slot's rows, which
// lie next to one another, are read together.
//
// Measured, with keys and values of 128 in bf16, 8 KV heads: 16 caches of 25,100 slots
// on average (1.6 GB) 256 us, 6.4 TB/s; one of 524,288 331 us, 6.5 TB/s; 32 of 2,900 68
// us, 5.7 TB/s; 64 x 4 lists of 2,048 slots 55 us, 4.9 TB/s: rows of 256 bytes in no
// order.  Row by row (pages of 4 slots) instead of in boxes the first takes as long, and
// 16 requests of 4 tokens with heads of 64 15.5 us instead of 14.6.
#include <algorithm>

#include "attn_mma.cuh"
#include "attn_paged.cuh"

namespace idx {

namespace {

constexpr int kWarps = 4;

// How tiles get into the ring: in boxes of consecutive slots of a page, by TMA; row
// by row; or row by row from a list of slots.
enum Load { kTiles, kRows, kList };

// A tile's keys, and its values, in boxes are lines of 128 bytes, one or two a row,
// with TMA's 128-byte swizzle (ldmatrix meets a bank twice where they are two).
template <int D>
struct Cfg {
  static constexpr int KT = stream_tile(D);  // keys of a tile: 4 KB of keys, 4 KB of values
  static constexpr int HALF = KT * D * 2;
  static constexpr int RING = 2 * 2 * HALF;  // of a warp: two tiles
  static constexpr uint32_t FULL = KT == 32 ? ~0u : (1u << KT) - 1;
  // 16-byte chunk c of row r
  template <bool BOXES>
  __device__ __forceinline__ static uint32_t at(int r, int c) {
    if (!BOXES) return swz<D>(r, c);
    const int line = r * (D / 64) + (c >> 3);
    return (uint32_t)(line * 128 + (((c & 7) ^ (line & 7)) << 4));
  }
};

// What a warp has of its rows: lane / 4 (and 8 on) of each 16, dims 8 i + 2 (lane % 4) and the next.
template <int D, int MT>
struct Rows {
  float o[MT][D / 8][4];
  float mx[MT][2], sum[MT][2];
  int id[MT][2];  // (b*T + t)*Hq + hq, -1: none
};

// Lane r's row of a tile: its number (-1: none), how many keys it sees, and where
// its queries are.
struct LaneRow {
  int id, lim;
  int64_t q;
};
template <bool LIST>
__device__ __forceinline__ LaneRow lane_row(const PagedArgs& a, int h, int row0, int R, int b, int t) {
  const paged_problem& p = a.p;
  const int rows = LIST ? a.G : p.T * a.G, r = row0 + (int)(threadIdx.x & 31);
  const int len = paged_len(p, b);
  LaneRow w{-1, 0, 0};
  if (r < min(rows, row0 + R)) {
    const int rt = LIST ? t : r / a.G, hq = h * a.G + (LIST ? r : r - rt * a.G);
    w.lim = max(0, len - p.T + rt + 1);
    w.id = (b * p.T + rt) * p.Hq + hq;
    w.q = b * p.q_stride_b + rt * p.q_stride_t + hq * p.q_stride_h;
  }
  return w;
}

__device__ __forceinline__ const int32_t* list_of(const paged_problem& p, int h, int b, int t) {
  const int64_t token = (int64_t)b * p.T + t;
  return p.ids + (p.ids_per_head ? token * p.n_kv + h : token) * p.W;
}

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int head, int slot, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %4, %5, %6}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(bar), "r"(0), "r"(head), "r"(slot), "r"(page)
      : "memory");
}

// A warp's ring: its tiles, and for each the barriers of its keys and its values.
struct Ring {
  uint32_t at;
  uint64_t* bars;  // keys of slot 0, values of slot 0, keys of slot 1, values of slot 1
  uint32_t tiles;  // that went through it
  volatile int* stop;
};

// The lane's keys of a warp's first two tiles, looked up as far as that goes beside
// the length: their slots (or list entries), and without a list their pages and
// slots in them.
struct Ahead {
  int slot[2], page[2], in_page[2];
};
template <int D, Load LOAD>
__device__ __forceinline__ Ahead look_ahead(const PagedArgs& a, int h, int b, int t, int k0, int apart) {
  const paged_problem& p = a.p;
  const int32_t* from = LOAD == kList ? list_of(p, h, b, t) : p.table + b * p.table_stride;
  Ahead w;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int at = k0 + j * apart + (int)(threadIdx.x % Cfg<D>::KT);
    w.slot[j] = LOAD == kList ? -1 : at;
    w.page[j] = w.in_page[j] = 0;
    if (LOAD == kList) {
      if (at < p.W) w.slot[j] = __ldg(from + at);
    } else if (at < p.max_len) {
      const int pg = (int)((uint32_t)at / (uint32_t)p.page_size);
      w.page[j] = __ldg(from + pg);
      w.in_page[j] = at - pg * p.page_size;
    }
  }
  return w;
}

// One warp's tiles of a sequence (of request b, or the list of its token t) under
// up to 16*MT rows of KV head h: fills r.  They are the tiles from key k0 on, `apart`
// keys from one to the next, as far as they begin before k1.  most: keys that the
// longest row sees.  false: a wait gave up, and what the ring holds has landed.
template <int D, int MT, bool BF16, Load LOAD>
__device__ __forceinline__ bool stream_keys(const PagedArgs& a, const CUtensorMap* maps, Ring& ring, int h, int b, int t, int k0, int k1,
                                            int apart, int most, const Ahead& ahead, const LaneRow& row_l, Rows<D, MT>& r) {
  using C = Cfg<D>;
  constexpr int KT = C::KT, NT = KT / 8, KS = D / 16;
  constexpr bool LIST = LOAD == kList;
  const paged_problem& p = a.p;
  const int lane = threadIdx.x & 31, key_of = lane % KT;
  const int32_t* table = p.table + b * p.table_stride;
  const int32_t* list = LIST ? list_of(p, h, b, t) : nullptr;
  const int mine = k0 < k1 ? (k1 - k0 + apart - 1) / apart : 0;  // tiles

  // the lane's key of the tile to copy next: its slot in its page (-1: not seen)
  // and that page; with a list, also the slot of the tile after
  int next_slot, next_page, later = -1;
  auto fetch_id = [&](int j) {
    const int at = k0 + j * apart + key_of;
    later = j < mine && at < k1 ? __ldg(list + at) : -1;
  };
  auto find = [&](int slot) {
    next_slot = -1;
    next_page = 0;
    if (slot >= 0 && slot < most) {
      const int pg = (int)((uint32_t)slot / (uint32_t)p.page_size);
      next_page = __ldg(table + pg);
      next_slot = slot - pg * p.page_size;
    }
  };
  auto look_up = [&](int j) {
    const int at = k0 + j * apart + key_of;
    find(LIST ? later : j < mine && at < k1 ? at : -1);
    if (LIST) fetch_id(j + 1);
  };
  auto take_ahead = [&](int j) {  // j 0 or 1
    const bool there = j < mine && k0 + j * apart + key_of < k1;
    if (LIST) return find(there ? ahead.slot[j] : -1);
    next_slot = there && ahead.slot[j] < most ? ahead.in_page[j] : -1;
    next_page = ahead.page[j];
  };
  unsigned live_after[2] = {0, 0};  // keys of the copied tiles that are seen
  bool ok_l = false;
  auto decide = [&] {
    ok_l = next_slot >= 0;
    if (ok_l && (next_page < 0 || next_page >= p.n_pages)) {
      atomicOr(&g_device_error, DEVERR_BAD_ROW);
      ok_l = false;
    }
    live_after[0] = live_after[1];
    live_after[1] = __ballot_sync(0xffffffffu, ok_l) & C::FULL;
  };
  // A box lies in one page, and is there if its first key is seen.  half 0: keys,
  // 1: values.
  auto issue_boxes = [&](int j, int half) {
    const uint32_t to = ((ring.tiles + j) & 1) * 2 + half;
    const bool lead = lane < KT && ok_l && (lane & (a.box - 1)) == 0;
    const int boxes = __popc(__ballot_sync(0xffffffffu, lead));
    if (lane == 0) mbar_arrive_expect_tx(ring.bars + to, boxes * a.box * D * 2);
    __syncwarp();
    if (lead)
      load_box(ring.at + to * C::HALF + lane * D * 2, maps + half, smem_u32(ring.bars + to), h, next_slot, next_page);
  };
  // Keys and values row by row; rows that are not seen become 0.
  auto issue_rows = [&](int j) {
    constexpr int CH = D / 8, RPI = 32 / CH;  // chunks of a row; rows of one warp-wide copy
    const uint32_t to = ((ring.tiles + j) & 1) * 2, sk = ring.at + to * C::HALF, sv = sk + C::HALF;
    const char* kb = (const char*)p.k + 2 * h * p.k_stride_h + lane % CH * 16;
    const char* vb = (const char*)p.v + 2 * h * p.v_stride_h + lane % CH * 16;
#pragma unroll
    for (int i = 0; i < KT / RPI; i++) {
      const int row = i * RPI + lane / CH;
      const uint32_t at = C::template at<LOAD == kTiles>(row, lane % CH);
      const int page = __shfl_sync(0xffffffffu, next_page, row), slot = __shfl_sync(0xffffffffu, next_slot, row);
      const bool live = live_after[1] >> row & 1;
      cp_async_16z(sk + at, live ? kb + 2 * (page * p.k_stride_p + slot * p.k_stride_s) : (const char*)p.q, live);
      cp_async_16z(sv + at, live ? vb + 2 * (page * p.v_stride_p + slot * p.v_stride_s) : (const char*)p.q, live);
    }
    cp_async_commit();
  };
  take_ahead(0);
  if (LOAD == kTiles) {
    decide();
    issue_boxes(0, 0);
    issue_boxes(0, 1);
    take_ahead(1);
    decide();
    issue_boxes(1, 0);
    issue_boxes(1, 1);
    look_up(2);
  } else {
    decide();
    issue_rows(0);
    take_ahead(1);
    if (LIST) fetch_id(2);
  }

  // the queries, as operand fragments: row lane / 4 (and 8 on) of a 16-row tile,
  // pairs of dims 2 (lane % 4) (and 8 on)
  const float c = scale_of(a);
  const uint32_t flip = flip_of(a);
  uint32_t qf[MT][KS][4];
  int lim[MT][2];
  // what the row that sees least sees (of the ones that there are)
  const int least = (int)__reduce_min_sync(0xffffffffu, (unsigned)(row_l.id >= 0 ? row_l.lim : INT32_MAX));
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const int row = m * 16 + (lane >> 2) + 8 * e;
      r.id[m][e] = __shfl_sync(0xffffffffu, row_l.id, row);
      lim[m][e] = __shfl_sync(0xffffffffu, row_l.lim, row);
      const int64_t q_at = __shfl_sync(0xffffffffu, row_l.q, row);
      const uint32_t* q = reinterpret_cast<const uint32_t*>((const char*)p.q + 2 * q_at) + (lane & 3);
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        qf[m][ks][e] = r.id[m][e] >= 0 ? __ldg(q + 8 * ks) ^ flip : 0u;
        qf[m][ks][e + 2] = r.id[m][e] >= 0 ? __ldg(q + 8 * ks + 4) ^ flip : 0u;
      }
    }
#pragma unroll
  for (int m = 0; m < MT; m++) {
#pragma unroll
    for (int j = 0; j < D / 8; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) r.o[m][j][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; e++) {
      r.mx[m][e] = -INFINITY;
      r.sum[m][e] = 0.f;
    }
  }

  // Boxes: tiles 0 and 1 are on their way; behind tile j's products tile j + 2 takes
  // its place.  Two tiles beyond the last are issued without rows: their barriers
  // complete at once, which keeps the ring's parity.  Rows: tile j + 1 is copied
  // while tile j is worked on; a second tile on its way made lists slower (58.5
  // against 55 us for 64 lists of 2,048).
  auto drain = [&](int tile, int half) {
    const uint32_t n = ring.tiles + tile;
    mbar_wait_drain(ring.bars + 2 * (n & 1) + half, (n >> 1) & 1);
  };
  for (int j = 0; j < mine; j++) {
    const uint32_t slot = (ring.tiles + j) & 1, parity = ((ring.tiles + j) >> 1) & 1;
    const uint32_t sk = ring.at + slot * 2 * C::HALF, sv = sk + C::HALF;
    const unsigned live = live_after[LOAD == kTiles ? 0 : 1];  // (before the next tile is decided)
    const int base = k0 + j * apart;
    if (LOAD != kTiles) {
      cp_async_wait_group<0>();
      __syncwarp();  // every lane's rows of tile j have landed, every lane is done with tile j - 1
      decide();
      issue_rows(j + 1);
      look_up(j + 2);
    } else if (!__all_sync(0xffffffffu, mbar_wait(ring.bars + 2 * slot, parity, ring.stop))) {
      for (int i = 0; i < 4; i++) drain(j + i / 2, i & 1);
      return false;
    }
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
        ldsm_x4(kf, sk + C::template at<LOAD == kTiles>(8 * i + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
#pragma unroll
        for (int m = 0; m < MT; m++) {
          mma16816<BF16>(s[m][i], qf[m][ks], kf[0], kf[1]);
          mma16816<BF16>(s[m][i + 1], qf[m][ks], kf[2], kf[3]);
        }
      }
    if (LOAD == kTiles) {
      __syncwarp();  // every lane has read the keys
      decide();
      issue_boxes(j + 2, 0);
    }
    // Scores, masked, and the running maximum.  A tile that every row sees whole needs
    // no masks.
    const int c0 = 2 * (lane & 3);
    const unsigned seen = live >> c0;
    const bool whole = live == C::FULL && (LIST || base + KT <= least);
#pragma unroll
    for (int m = 0; m < MT; m++) {
      float top[2] = {r.mx[m][0], r.mx[m][1]};
      if (!whole) {
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            bool see = seen >> (8 * i + (e & 1)) & 1;
            if (!LIST) see = see && base + 8 * i + c0 + (e & 1) < lim[m][e >> 1];
            if (!see) s[m][i][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int i = 0; i < NT; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) top[e >> 1] = fmaxf(top[e >> 1], s[m][i][e]);
      bool grew = false;
      float scl[2];
#pragma unroll
      for (int e = 0; e < 2; e++) {
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
        const float x = top[e] == -INFINITY ? 0.f : top[e];
        scl[e] = attn_ex2((r.mx[m][e] - x) * c);  // 0 for a first maximum, 1 where it stays
        grew |= top[e] != r.mx[m][e];
        r.mx[m][e] = top[e];
        top[e] = x;
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int e = 0; e < 2; e++) r.sum[m][e] *= scl[e];
#pragma unroll
        for (int i = 0; i < D / 8; i++)
#pragma unroll
          for (int e = 0; e < 4; e++) r.o[m][i][e] *= scl[e >> 1];
      }
      // (the maximum is subtracted before the scale: c s - c m in one fma is not 0 for
      // the largest score but half a step of c m, and infinite from 2^31 on)
#pragma unroll
      for (int i = 0; i < NT; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          s[m][i][e] = attn_ex2(fmaf(s[m][i][e] - top[e >> 1], c, kLift<BF16>));
          r.sum[m][e >> 1] += s[m][i][e];
        }
    }
    if (LOAD == kTiles && !__all_sync(0xffffffffu, mbar_wait(ring.bars + 2 * slot + 1, parity, ring.stop))) {
      for (int i = 1; i < 5; i++) drain(j + i / 2, i & 1);
      return false;
    }
    if (LOAD == kTiles && live != C::FULL) {
      // rows that were not copied, and a page's rows behind the last key, hold
      // anything, NaN too, and a weight of zero would not cancel it
      if (lane < KT && !(live >> lane & 1))
#pragma unroll
        for (int i = 0; i < D / 8; i++)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sv + C::template at<LOAD == kTiles>(lane, i)), "r"(0) : "memory");
      fence_proxy_async_smem();
      __syncwarp();
    }
    // Weights times values.  The weights are rounded to the element type, as the
    // 16-bit operand of the product has to be, one rounding of at most 2^-8 (2^-11
    // for fp16, down to 2^-29 of the largest, below that 2^-40 of it) of each weight, as
    // large as the output's own; the sum that divides them is of the unrounded ones, in 32 bits.
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
        ldsm_x4_t(vf, sv + C::template at<LOAD == kTiles>(kk * 16 + (lane & 15), i + (lane >> 4)));
#pragma unroll
        for (int m = 0; m < MT; m++) {
          mma16816<BF16>(r.o[m][i], pf[m], vf[0], vf[1]);
          mma16816<BF16>(r.o[m][i + 1], pf[m], vf[2], vf[3]);
        }
      }
    }
    if (LOAD == kTiles) {
      __syncwarp();  // every lane has read the values
      issue_boxes(j + 2, 1);
      look_up(j + 3);
    }
  }
  ring.tiles += mine + (LOAD == kTiles ? 2 : 1);
  if (LOAD != kTiles) {
    cp_async_wait_group<0>();
    __syncwarp();
  }
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      r.mx[m][e] *= c;  // in log2 units
      r.sum[m][e] += __shfl_xor_sync(0xffffffffu, r.sum[m][e], 1);
      r.sum[m][e] += __shfl_xor_sync(0xffffffffu, r.sum[m][e], 2);
    }
  return true;
}

// One warp's units [u0, u1) of a sequence's `units`, at `place` of the partial results.
template <int D, int MT, bool BF16, Load LOAD>
__device__ __forceinline__ bool line_item(const PagedArgs& a, const CUtensorMap* maps, Ring& ring, int shift, int h, int tile, int b, int t, int u0, int u1,
                                          int units, int64_t place) {
  constexpr int R = 16 * MT;
  constexpr bool LIST = LOAD == kList;
  const paged_problem& p = a.p;
  const Ahead ahead = look_ahead<D, LOAD>(a, h, b, t, u0 << shift, Cfg<D>::KT);
  const LaneRow row = lane_row<LIST>(a, h, tile * R, R, b, t);
  const int lane = threadIdx.x & 31, rid_l = row.id, most = __reduce_max_sync(0xffffffffu, row.lim);
  const int n = LIST ? (most > 0 ? (int)p.W : 0) : most;  // keys of the sequence
  const int k0 = u0 << shift, k1 = (int)min((int64_t)n, (int64_t)u1 << shift);
  const int64_t row_0 = place * a.rows - (int64_t)(LIST ? b * p.T + t : b) * a.rows;  // of row 0 of the call
  if (k0 >= k1) {
    if (rid_l >= 0) a.pml[row_0 + rid_l] = make_float2(-INFINITY, 0.f);
    return true;
  }
  Rows<D, MT> r;
  if (!stream_keys<D, MT, BF16, LOAD>(a, maps, ring, h, b, t, k0, k1, Cfg<D>::KT, most, ahead, row, r))
    return false;
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      if (r.id[m][e] < 0) continue;
      const int64_t at = row_0 + r.id[m][e];
      if ((lane & 3) == 0) a.pml[at] = make_float2(r.mx[m][e], r.sum[m][e]);
      if (r.sum[m][e] != 0.f) {  // (NaN where a score was)
#pragma unroll
        for (int i = 0; i < D / 8; i++)
          *reinterpret_cast<float2*>(a.po + at * D + 8 * i + 2 * (lane & 3)) =
              make_float2(r.o[m][i][2 * e], r.o[m][i][2 * e + 1]);
      }
    }
  return true;
}

template <int D, int MT, bool BF16, Load LOAD>
__global__ void __launch_bounds__(32 * kWarps, MT == 1 ? 3 : 2)
    attn_paged_line_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedArgs a,
                           const __grid_constant__ PagedLine line) {
  constexpr int NT = 32 * kWarps;
  constexpr bool LIST = LOAD == kList;
  __shared__ int s_sum[kWarps];
  __shared__ int s_first[NT];
  __shared__ uint64_t s_bars[kWarps][4];
  __shared__ int s_stop;
  extern __shared__ char smem[];
  Ring ring{((smem_u32(smem) + 1023) & ~1023u) + (threadIdx.x >> 5) * Cfg<D>::RING, s_bars[threadIdx.x >> 5], 0, &s_stop};
  if (threadIdx.x == 0) s_stop = 0;
  if ((threadIdx.x & 31) < 4) mbar_init(ring.bars + (threadIdx.x & 31), 1);
  if (LOAD == kTiles && threadIdx.x < 2) prefetch_tmap(&maps.m[threadIdx.x]);
  fence_mbar_init();
  fence_proxy_async_smem();
  __syncthreads();
  // (nothing is started early behind this kernel: the next one's blocks would take the
  // room of the last warps' loads; 32 requests of 4,096 slots took 71.9 us instead of 67.8)
  grid_wait();
  const paged_problem& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w = (int)blockIdx.x * kWarps + warp;
  const int group = w / line.members, member = w - group * line.members;
  const int tile = member / p.n_kv, h = member - tile * p.n_kv;

  // the line's length (below 2^31, the plan checks), and where on it each
  // thread's share of the sequences begins
  int total = 0;
  const int per = (line.seqs + NT - 1) / NT;
  if (LIST || line.uniform) {
    total = line.seqs * line.uniform;
  } else {
    const int b0 = min(line.seqs, tid * per), b1 = min(line.seqs, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; b++) mine += units_of(p, b, line.unit_shift);
    int incl = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = 0;
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
  int lo = group * each + min(group, extra);
  const int hi = group < groups ? lo + each + (group < extra ? 1 : 0) : lo;
  if (lo >= hi) return;
  int seq, units, start;  // the sequence that holds lo
  if (LIST || line.uniform) {
    seq = lo / line.uniform;
    start = seq * line.uniform;
    units = line.uniform;
  } else {
    // the last thread whose sequences begin at or before lo, then one by one
    int last = -1;
#pragma unroll
    for (int x = 0; x < NT; x += 32)
      last += __popc(__ballot_sync(0xffffffffu, s_first[x + lane] <= lo && (x + lane) * per < line.seqs));
    seq = last * per;
    start = s_first[last];
    units = units_of(p, seq, line.unit_shift);
    while (start + units <= lo) {
      start += units;
      units = units_of(p, ++seq, line.unit_shift);
    }
  }
  while (true) {
    const int b = LIST ? seq / p.T : seq;
    if (member == 0 && lane == 0) {
      if (lo == start) a.ends[seq].x = group;
      if (hi >= start + units) a.ends[seq].y = group;
    }
    if (!line_item<D, MT, BF16, LOAD>(a, maps.m, ring, line.unit_shift, h, tile, b, LIST ? seq - b * p.T : 0, lo - start,
                                      min(units, hi - start), units, (int64_t)group + seq))
      return;
    start += units;
    lo = start;
    if (lo >= hi) break;
    seq++;
    if (!LIST && !line.uniform) units = units_of(p, seq, line.unit_shift);
  }
}

// Short calls: one block, or a cluster of up to 16, has a sequence's row tile; its
// warps take the key tiles in turn.  The warps' partial results are joined through
// shared memory, the blocks' through distributed shared memory: each block sends
// every other its share of the columns, and writes its own share out.  A piece is
// empty where the sum of its weights is 0, and only there (NaN: a score was).  No
// second launch, no workspace.
struct Short {
  int blocks;  // of a cluster
  int share;   // units (a row's four columns) that a block of a cluster writes out
  void* out;
  float* lse;
};

// Column col of row `row` in a warp's partial sums: swizzled, so that the rows of
// an accumulator do not meet in one bank.
template <int D>
__device__ __forceinline__ int sum_at(int row, int col) {
  return row * D + (col ^ ((row & 7) << 3));
}

__device__ __forceinline__ uint32_t peer(uint32_t at, int rank) {
  uint32_t far;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
  return far;
}

constexpr int kCluster = 16;  // blocks at most

template <int D, int MT, bool BF16, Load LOAD>
__global__ void __launch_bounds__(32 * kWarps, MT == 1 ? 3 : 2)
    attn_paged_short_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedArgs a,
                            const __grid_constant__ Short sh) {
  constexpr int R = 16 * MT, KT = Cfg<D>::KT;
  constexpr bool LIST = LOAD == kList;
  __shared__ uint64_t s_bars[kWarps][4];
  __shared__ int s_stop;
  __shared__ float2 s_ml[kWarps][R];
  __shared__ int s_id[R];
  extern __shared__ char smem[];
  const paged_problem& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rings = (smem_u32(smem) + 1023) & ~1023u;
  char* const rings_p = smem + (rings - smem_u32(smem));
  const int C = sh.blocks, rank = (int)(blockIdx.x % C);
  Ring ring{rings + warp * Cfg<D>::RING, s_bars[warp], 0, &s_stop};
  if (tid == 0) s_stop = 0;
  if (lane < 4) mbar_init(ring.bars + lane, 1);
  if (LOAD == kTiles && tid < 2) prefetch_tmap(&maps.m[tid]);
  fence_mbar_init();
  fence_proxy_async_smem();
  __syncthreads();
  // (what is sent to a block needs it to have begun: it is asked for just before)
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  grid_wait();
  grid_let_next_start();

  int item = (int)(blockIdx.x / C);
  const int h = item % p.n_kv;
  item /= p.n_kv;
  const int rows = (LIST ? 1 : p.T) * a.G, tiles = (rows + R - 1) / R, tile = item % tiles, seq = item / tiles;
  const int b = LIST ? seq / p.T : seq, t = LIST ? seq - b * p.T : 0;
  const int first = (rank * kWarps + warp) * KT, apart = C * kWarps * KT;
  const Ahead ahead = look_ahead<D, LOAD>(a, h, b, t, first, apart);
  const LaneRow row = lane_row<LIST>(a, h, tile * R, R, b, t);
  const int most = __reduce_max_sync(0xffffffffu, row.lim);
  const int n = LIST ? (most > 0 ? (int)p.W : 0) : most;
  const int nrow = min(R, rows - tile * R), units = nrow * (D / 4);
  if (tid < nrow) s_id[tid] = row.id;
  {
    Rows<D, MT> r;
    const bool ok = stream_keys<D, MT, BF16, LOAD>(a, maps.m, ring, h, b, t, first, n, apart, most, ahead, row, r);
    float* sums = reinterpret_cast<float*>(rings_p + warp * Cfg<D>::RING);
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int at = m * 16 + (lane >> 2) + 8 * e;
        if (at >= nrow) continue;
        if ((lane & 3) == 0) s_ml[warp][at] = ok ? make_float2(r.mx[m][e], r.sum[m][e]) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < D / 8; i++)
          *reinterpret_cast<float2*>(sums + sum_at<D>(at, 8 * i + 2 * (lane & 3))) =
              make_float2(r.o[m][i][2 * e], r.o[m][i][2 * e + 1]);
      }
  }
  __syncthreads();
  auto put = [&](int r, int col, float top, float sum, float4 v) {
    const float inv = sum != 0.f ? __fdividef(1.f, sum) : 0.f;  // (within 2 units in the last place)
    const int64_t id = s_id[r];
    *reinterpret_cast<uint2*>((char*)sh.out + 2 * (id * D + col)) =
        make_uint2(pack2<BF16>(v.x * inv, v.y * inv), pack2<BF16>(v.z * inv, v.w * inv));
    if (col == 0 && sh.lse) sh.lse[id] = sum != 0.f ? log2_sum<BF16>(top, sum) * 0.693147180559945309f : -INFINITY;
  };
  // from the blocks of the cluster, by their ranks: sums, and (maximum, sum) of the
  // weights, of this block's units
  float4* const all_sums = reinterpret_cast<float4*>(rings_p + kWarps * Cfg<D>::RING);
  float2* const all_ml = reinterpret_cast<float2*>(all_sums + C * sh.share);
  if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int u = tid; u < units; u += 32 * kWarps) {
    const int r = u / (D / 4), col = u % (D / 4) * 4;
    float2 ml[kWarps];
#pragma unroll
    for (int i = 0; i < kWarps; i++) ml[i] = s_ml[i][r];
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; i++) top = fmaxf(top, ml[i].y != 0.f ? ml[i].x : -INFINITY);
    const float base = top == -INFINITY ? 0.f : top;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kWarps; i++) {
      const float w = ml[i].y != 0.f ? attn_ex2(ml[i].x - base) : 0.f;
      const float4 x = *reinterpret_cast<const float4*>(rings_p + i * Cfg<D>::RING + sum_at<D>(r, col) * 4);
      sum += w * ml[i].y;
      v.x += w * x.x;
      v.y += w * x.y;
      v.z += w * x.z;
      v.w += w * x.w;
    }
    if (C == 1) {
      put(r, col, top, sum, v);
    } else {
      const int to = u / sh.share, at = u - to * sh.share;
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                       peer(smem_u32(all_sums + rank * sh.share + at), to)),
                   "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                   : "memory");
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                       peer(smem_u32(all_ml + rank * sh.share + at), to)),
                   "f"(top), "f"(sum)
                   : "memory");
    }
  }
  if (C == 1) return;
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  // A lane adds up to four blocks' parts of a unit, four lanes those of sixteen.
  const int mine = min(sh.share, units - rank * sh.share), lanes = C <= 4 ? 1 : C <= 8 ? 2 : 4, from = tid & (lanes - 1);
  for (int at0 = 0; at0 < mine; at0 += 32 * kWarps / lanes) {
    const int at = min(at0 + tid / lanes, mine - 1);
    float2 ml[4];
    float4 x[4];
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int src = (min(4 * from + i, C - 1)) * sh.share + at;
      ml[i] = all_ml[src];
      x[i] = all_sums[src];
      if (4 * from + i >= C) {
        ml[i] = make_float2(-INFINITY, 0.f);
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      top = fmaxf(top, ml[i].y != 0.f ? ml[i].x : -INFINITY);
    }
    for (int o = lanes >> 1; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float w = ml[i].y != 0.f ? attn_ex2(ml[i].x - base) : 0.f;
      sum += w * ml[i].y;
      v.x += w * x[i].x;
      v.y += w * x[i].y;
      v.z += w * x[i].z;
      v.w += w * x[i].w;
    }
    for (int o = lanes >> 1; o; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
      v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
    }
    const int u = rank * sh.share + at;
    if (from == 0 && at0 + tid / lanes < mine) put(u / (D / 4), u % (D / 4) * 4, top, sum, v);
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t keys_of(const paged_problem& p) { return p.max_len == 0 ? 0 : p.ids ? p.W : p.max_len; }
// Query rows of a KV head and sequence, and how many of them a warp takes.
int64_t rows_of(const paged_problem& p) { return (p.ids ? 1 : p.T) * (int64_t)(p.Hq / p.n_kv); }
int row_tile(const paged_problem& p) { return rows_of(p) <= 16 ? 16 : 32; }

// Every SM holds twelve warps of 16 rows or eight of 32 (three or two blocks), and
// every warp gets one share of the line.
PagedLine plan_line(const paged_problem& p) {
  PagedLine l{};
  const int64_t rt = row_tile(p), rows = rows_of(p);
  const int64_t tile = stream_tile(p.D), keys = keys_of(p);
  l.members = (int)(p.n_kv * ceil_div(rows, rt));
  l.seqs = p.ids ? p.B * p.T : p.B;
  const int64_t warps = (rt == 16 ? 12 : 8) * (int64_t)sm_count();
  // A unit is a tile where every share has sixteen of them or more (an even cut
  // matters), else four.
  const bool fine = l.seqs * ceil_div(keys, tile) * l.members >= 16 * warps;
  l.unit_shift = (p.D == 128 ? 4 : 5) + (fine ? 0 : 2);
  const int64_t longest = std::max<int64_t>(1, ceil_div(keys, (int64_t)1 << l.unit_shift)), total = l.seqs * longest;
  l.groups = (int)std::max<int64_t>(1, warps / l.members);
  l.least = fine ? 4 : 1;  // no shorter than the coarse units
  // Lists have one length; short lines are cut as if all caches were full, which
  // saves their blocks the look at the lengths.
  if (p.ids || (!fine && total <= 2 * (int64_t)l.groups)) l.uniform = (int)longest;
  if (l.uniform) l.groups = (int)std::min<int64_t>(l.groups, std::max<int64_t>(1, total / l.least));
  return l;
}

// Keys of a box: the largest power of two that divides the page, up to a tile; 0
// where no tensor map can hold the pools or the boxes are too small to be worth it.
int box_of(const paged_problem& p, int tile) {
  const int box = std::min(p.page_size & -p.page_size, tile);
  auto legal = [](int64_t n, int64_t stride) { return n <= 1 || (stride > 0 && stride < ((int64_t)1 << 38)); };
  const bool ok = legal(p.n_kv, p.k_stride_h) && legal(p.page_size, p.k_stride_s) && legal(p.n_pages, p.k_stride_p) &&
                  legal(p.n_kv, p.v_stride_h) && legal(p.page_size, p.v_stride_s) && legal(p.n_pages, p.v_stride_p);
  return !p.ids && ok && box >= 8 && p.n_pages > 0 && p.max_len > 0 ? box : 0;
}

// Whether a long call goes to the tensor-core kernel (not lists, and not pages that no
// box fits).  Up to 16 rows are the streaming kernel's.  With heads of 64 and up to 32
// rows it reads as fast as the other computes, and wins once there are more than about 8
// sequences and KV heads (4 x 4 KV heads of 32 rows over 75,000 slots 53 us against 58, 4
// x 8 87 against 102; 1 x 1 over 75,000, one in every group, 26 against 15, 2 x 1 29
// against 19, 4 x 1 28 against 25); with heads of 128, or more rows, it takes 1.1 to 3
// times as long.
bool tensor_cores(const paged_problem& p) {
  return rows_of(p) > 16 && box_of(p, 128) > 0 &&
         (rows_of(p) > 32 || p.D == 128 || (int64_t)p.B * p.n_kv * 16 <= sm_count());
}

// Of the blocks that there is room for, how many run at once in clusters of c, in percent.
int cluster_part(int c) { return c <= 2 ? 100 : c <= 5 ? 95 : c <= 12 ? 89 : 73; }

// Shared memory that leaves an SM room for one block, or two.
constexpr int kOneBlock = 116 << 10, kTwoBlocks = 78 << 10;

// Row tiles of all KV heads and sequences.
int64_t short_items(const paged_problem& p) {
  return (int64_t)p.B * (p.ids ? p.T : 1) * p.n_kv * ceil_div(rows_of(p), row_tile(p));
}

// Blocks of a cluster for a short call, 0: a long one.  An SM holds three blocks,
// two where more than 16 rows ask for registers, or more than 8 of 128 for room in shared
// memory (12 warps of 16 rows are no faster than 8, but for long calls).  A
// cluster stays within a part of the GPU, whose SMs it need not use up, so of the blocks
// that there is room for 0.95 or more run at once in clusters of up to 5, 0.89 or more in
// 6, 8, 10 and 12 and 0.73 in 16, as the runtime says for two and for three blocks an SM
// (4 requests of 4 KV heads of 32 rows of 64 over 6,000 slots took 17 us in 16 clusters
// of 16, 13 in 16 of 8).  Powers of two alone left up to half of the room empty: 16
// requests of 4 heads over 4,000 slots 29 us instead of 23.
int short_blocks(const paged_problem& p) {
  const int64_t items = short_items(p), room = (rows_of(p) <= (p.D == 64 ? 16 : 8) ? 3 : 2) * (int64_t)sm_count();
  const int64_t tiles = std::max<int64_t>(1, ceil_div(keys_of(p), stream_tile(p.D)));
  int blocks = 1;
  int64_t each = ceil_div(tiles, kWarps);  // tiles of a warp
  for (int c : {2, 3, 4, 5, 6, 8, 10, 12, kCluster}) {
    const int64_t n = ceil_div(tiles, kWarps * c);
    if (items * c * 100 <= room * cluster_part(c) && n < each) {
      blocks = c;
      each = n;
    }
  }
  const int64_t waves = ceil_div(items * blocks, room);
  // On the other side is the streaming kernel, whose warps share the line evenly (full:
  // tiles of a warp, of a short call that leaves no room empty) and read at DRAM's rate
  // when they are long, at the cost of a second launch: 12 to 13 tiles' time.
  //   Waves of many blocks even their lengths out by themselves: 256 requests of 8 heads
  // over 2,000 slots 230 us against 255 there, of 4 tokens and 4 heads over 1,000 72
  // against 84.
  //   Else latency bounds a call that fills little of the GPU (one request of 8 heads over
  // 16,000 slots 24 us in both, over 20,000 29 against 25), and bytes the others, where
  // the longest cache of a batch counts here and the average there: 16 requests of 4
  // tokens and 4 heads over 5,000 slots 30 us against 38, 8 of 1 token and 8 heads over
  // 16,000 71 against 74, 16 of them 134 against 132.  Heads of 64, more than 16 rows and
  // row by row loads take a tile's bytes more slowly (24 lists of 2,000 23 us against 30,
  // 64 55 in both).
  const bool boxes = box_of(p, stream_tile(p.D)) > 0, one = row_tile(p) == 16;
  const int64_t work = waves * each, full = items * tiles / (kWarps * room);
  const int64_t lead = boxes && one ? (p.D == 128 ? 250 : 160) : 120;
  bool is_short = (boxes && waves >= 3 && work <= 160) || (work <= 12 + full && 8 * work <= lead + 5 * full);
  if (tensor_cores(p)) {
    // A wave takes about 3 us and 2 for each tile, the tensor-core kernel 9 us for a run
    // of each block and 1 for a tile of 128 keys (128 requests of 32 rows, 4 KV heads
    // and 300 slots: 31 us against 40; 8 of 32 rows, 4 heads and 4,000: 23 against 21).
    const int64_t seqs = p.B * p.n_kv * ceil_div(rows_of(p), 128), n = sm_count();
    is_short = waves * (3 + 2 * each) <= ceil_div(seqs, n) * 9 + seqs * ceil_div(p.max_len, 128) / n;
  }
  return is_short && items * blocks < ((int64_t)1 << 31) ? blocks : 0;
}

// Its line: units of 128 keys, a block for each KV head and 128 rows of a group.
PagedLine plan_tc(const paged_problem& p) {
  PagedLine l{};
  l.unit_shift = 7;
  l.members = (int)(p.n_kv * ceil_div(rows_of(p), 128));
  l.seqs = p.B;
  const int64_t longest = std::max<int64_t>(1, ceil_div(p.max_len, 128)), total = l.seqs * longest;
  l.groups = (int)std::min<int64_t>(total, std::max<int64_t>(1, sm_count() / l.members));
  l.least = 1;
  return l;
}

PagedLine plan_long(const paged_problem& p) { return tensor_cores(p) ? plan_tc(p) : plan_line(p); }

PagedArgs make_args(const paged_problem& p) {
  PagedArgs a{};
  a.p = p;
  a.G = p.Hq / p.n_kv;
  a.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
  a.box = box_of(p, stream_tile(p.D));
  return a;
}

// Rows of a sequence of the line.
int64_t line_rows(const paged_problem& p) { return (p.ids ? 1 : p.T) * (int64_t)p.Hq; }

// The line and the rows are counted in 32 bits.
bool fits(const paged_problem& p) {
  const int64_t most = (int64_t)1 << 31, seqs = (int64_t)p.B * (p.ids ? p.T : 1);
  if (seqs * std::max<int64_t>(1, ceil_div(keys_of(p), stream_tile(p.D))) >= most) return false;
  return (seqs + plan_long(p).groups) * line_rows(p) < most;
}

struct Ws {
  size_t pml, ends, total;
};
Ws layout(const paged_problem& p, const PagedLine& line) {
  const size_t places = (size_t)(line.groups + (int64_t)line.seqs), rows = (size_t)line_rows(p);
  Ws w;
  WsCarver c(nullptr);
  c.take<float>(places * rows * p.D);
  w.pml = (c.used + 255) & ~size_t(255);
  c.take<float2>(places * rows);
  w.ends = (c.used + 255) & ~size_t(255);
  c.take<int2>((size_t)line.seqs);
  w.total = c.used + 256;
  return w;
}

// Maps of the pools, for boxes of `box` slots of a KV head and `lines` lines of 128
// bytes.  The two lines of a row of 256 bytes are a dimension, so that a box holds the
// rows one by one: with the lines' halves of a box behind one another 16 long caches
// took 257 us instead of 251.
bool make_maps(PagedMaps* maps, const paged_problem& p, int box, int lines) {
  auto make = [&](CUtensorMap* map, const void* base, int64_t sp, int64_t ss, int64_t sh) {
    // a dimension of one: its stride is never used, but has to be a legal one
    auto bytes = [&](int64_t n, int64_t stride) { return (uint64_t)(2 * (n > 1 ? stride : p.D)); };
    return make_tmap_5d(map, p.dtype == IDX_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        base, {64, (uint64_t)p.D / 64, (uint64_t)p.n_kv, (uint64_t)p.page_size, (uint64_t)p.n_pages},
                        {128, bytes(p.n_kv, sh), bytes(p.page_size, ss), bytes(p.n_pages, sp)},
                        {64, (uint32_t)lines, 1, (uint32_t)box, 1});
  };
  return make(&maps->m[0], p.k, p.k_stride_p, p.k_stride_s, p.k_stride_h) &&
         make(&maps->m[1], p.v, p.v_stride_p, p.v_stride_s, p.v_stride_h);
}

template <int D, int MT, bool BF16, Load LOAD>
cudaError_t launch_one(const PagedArgs& a, const PagedLine* line, const Short* sh, cudaStream_t st) {
  constexpr int kRings = kWarps * Cfg<D>::RING + 1024, kR = 16 * MT;
  // (boxes under more than 16 rows of 128 are the tensor-core kernel's, or short)
  constexpr bool kLine = LOAD != kTiles || MT == 1 || D == 64;
  auto kern = attn_paged_line_kernel<D, kLine ? MT : 1, BF16, LOAD>;
  auto kern_short = attn_paged_short_kernel<D, MT, BF16, LOAD>;
  static KernelReady ready;
  cudaError_t e = ready.once([&] {
    cudaError_t x = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRings);
    if (x == cudaSuccess)
      x = cudaFuncSetAttribute(kern_short, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               std::max(kOneBlock, kRings + (kR * D / 4 + kCluster) * 24));
    if (x == cudaSuccess) x = cudaFuncSetAttribute(kern_short, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return x;
  });
  if (e != cudaSuccess) return e;
  PagedMaps maps{};
  const paged_problem& p = a.p;
  if (LOAD == kTiles && !make_maps(&maps, p, a.box, D / 64)) return cudaErrorInvalidValue;
  if (line && !kLine) return cudaErrorInvalidValue;
  if (line) {
    const int64_t blocks = ceil_div((int64_t)line->members * line->groups, kWarps);
    return launch_early(kern, dim3((unsigned)blocks), 32 * kWarps, kRings, st, maps, a, *line);
  }
  size_t smem = kRings + (sh->blocks > 1 ? sh->blocks * sh->share * 24 : 0);
  // Blocks that need no room of three an SM (or of two, in clusters that any SM has room
  // for) ask for more shared memory than that leaves, and so spread over all SMs: 64
  // requests of 4 tokens and 4 heads over 500 slots 15.7 us, 17.9 without.
  const int64_t percent = short_items(p) * sh->blocks * 100, of_one = sm_count() * (int64_t)cluster_part(sh->blocks);
  if (percent <= 2 * of_one) smem = std::max<size_t>(smem, sh->blocks <= 2 && percent <= of_one ? kOneBlock : kTwoBlocks);
  return launch_early_cluster(kern_short, (unsigned)(short_items(p) * sh->blocks), (unsigned)sh->blocks, 32 * kWarps,
                              smem, st, maps, a, *sh);
}
template <int D, bool BF16, int MT>
cudaError_t launch_load(const PagedArgs& a, const PagedLine* line, const Short* sh, cudaStream_t st) {
  if (a.p.ids) return launch_one<D, MT, BF16, kList>(a, line, sh, st);
  return a.box ? launch_one<D, MT, BF16, kTiles>(a, line, sh, st) : launch_one<D, MT, BF16, kRows>(a, line, sh, st);
}
template <int D, bool BF16>
cudaError_t launch_kind(const PagedArgs& a, const PagedLine* line, const Short* sh, cudaStream_t st) {
  return row_tile(a.p) == 16 ? launch_load<D, BF16, 1>(a, line, sh, st) : launch_load<D, BF16, 2>(a, line, sh, st);
}
cudaError_t launch(PagedArgs a, const PagedLine* line, const Short* sh, cudaStream_t st) {
  if (line && tensor_cores(a.p)) {
    PagedMaps maps{};
    a.box = box_of(a.p, 128);
    if (!make_maps(&maps, a.p, a.box, 1)) return cudaErrorInvalidValue;
    return launch_attn_paged_tc(a, maps, *line, st);
  }
  const bool bf = a.p.dtype == IDX_BF16;
  if (a.p.D == 128) return bf ? launch_kind<128, true>(a, line, sh, st) : launch_kind<128, false>(a, line, sh, st);
  return bf ? launch_kind<64, true>(a, line, sh, st) : launch_kind<64, false>(a, line, sh, st);
}

}  // namespace

bool attn_paged_ws(const paged_problem& p, size_t* bytes) {
  if (!fits(p)) return false;
  *bytes = 0;
  if (short_blocks(p)) return true;
  *bytes = layout(p, plan_long(p)).total;
  return true;
}

idx_status launch_attn_paged(const paged_problem& p, void* out, float* lse, void* ws, size_t ws_bytes,
                             cudaStream_t st, cudaError_t* err) {
  if (!fits(p)) return IDX_ERR_UNSUPPORTED;
  PagedArgs a = make_args(p);
  if (const int blocks = short_blocks(p)) {
    const int64_t rows = std::min<int64_t>(row_tile(p), rows_of(p));
    const Short sh{blocks, (int)ceil_div(rows * p.D / 4, blocks), out, lse};
    *err = launch(a, nullptr, &sh, st);
    return *err == cudaSuccess ? IDX_OK : IDX_ERR_CUDA;
  }
  const PagedLine line = plan_long(p);
  const Ws w = layout(p, line);
  if (ws_bytes < w.total) return IDX_ERR_WORKSPACE_TOO_SMALL;
  if (!ws) return IDX_ERR_INVALID_ARG;
  char* base = (char*)(((uintptr_t)ws + 255) & ~uintptr_t(255));
  a.rows = (int)line_rows(p);
  a.po = (float*)base;
  a.pml = (float2*)(base + w.pml);
  a.ends = (int2*)(base + w.ends);
  cudaError_t e = launch(a, &line, nullptr, st);
  if (e == cudaSuccess) e = launch_attn_paged_join(a, line.seqs, line.groups, out, lse, st);
  *err = e;
  return e == cudaSuccess ? IDX_OK : IDX_ERR_CUDA;
}

}  // namespace idx
