// Attention of a decode step: the plan of a call (which kernel takes which
// part, how many pieces) and its workspace.  Host only.
#include "attn_tc.cuh"

#include <algorithm>

namespace idx {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Keys of the private part that a row can see at most.
int64_t private_keys(const attn_problem& p) { return p.S == 0 ? 0 : p.ids ? p.W : p.S; }

// Rows of a KV head that one warp of the streaming kernel takes.
constexpr int64_t kStreamRows = 16;

// How the prefix is read.
enum PrefixWay { kNone, kLine, kOwnLine, kTensorCore };

// Up to 16 rows are one warp's: the prefix is streamed on one line with the
// caches.  More rows would read it again for each 16: where that is little, the
// streaming kernel still does it, beside the caches, because the tensor-core
// kernel's launch and start take about 9 us; else it goes to that kernel, with
// TMA, if a tensor map can hold its strides.
PrefixWay prefix_way(const attn_problem& p) {
  constexpr int64_t kLittle = 32 << 20;  // bytes: about 4 us from L2
  const int64_t rows = (int64_t)p.B * p.T * (p.Hq / p.n_kv);
  if (p.P == 0) return kNone;
  if (rows <= kStreamRows) return kLine;
  if (ceil_div(rows, kStreamRows) * p.n_kv * p.P * 4 * p.D <= kLittle) return kOwnLine;
  auto legal = [](int64_t n, int64_t stride) { return n <= 1 || (stride > 0 && stride < ((int64_t)1 << 38)); };
  return legal(p.P, p.pk_stride_s) && legal(p.P, p.pv_stride_s) && legal(p.n_kv, p.pk_stride_h) &&
                 legal(p.n_kv, p.pv_stride_h)
             ? kTensorCore
             : kOwnLine;
}

// The tensor-core kernel's grid: a whole number of pieces of the keys per (KV
// head, row tile pair), so that the row tiles of a piece run in step and their
// keys come from L2, if that leaves few SMs idle; otherwise the key tiles are
// cut evenly, and a piece can end up on two blocks.  On 65536 keys under 1024
// rows of each of 8 heads, 128 whole pieces and an even cut over 152 SMs take
// the same time (190 and 192 us), on 8192 keys 39 and 51 us; with heads of 64,
// where the weights take longer than the products, the idle SMs cost more (181
// against 164 us).
//
// Beside private caches the grid is smaller: the streaming kernel, which waits
// for memory most of the time, starts on the SMs that are left.  The share
// follows the two kernels' work (1.6 us a key tile under two row tiles, 0.9 us
// under one; 55 bytes/ns of an SM that streams, caches taken as 0.6 full, their
// lengths being on the device), and a block takes eight key tiles at least, so
// that its start and end count little; but where the caches are so short that
// they need few SMs for a moment, it gets all the others (84 requests with 18
// listed slots each behind 3,309 tokens: 31 us, with eight key tiles a block 34).
// One after the other took 337 us for 128 requests with caches of 2,048 slots
// behind 65,536 tokens, side by side 289; 53 and 41 for 32 requests with 1,024
// slots behind 8,192.  Caches that are full are also best taken as 0.6 full: 330
// us for those 128 requests, 390 with a share for full ones (lengths from half to
// all: 287 and 385); the others measured do not depend on it.
AttnTcArgs plan_tc(const AttnArgs& a) {
  const attn_problem& p = a.p;
  AttnTcArgs t{};
  t.a = a;
  const int64_t tiles = ceil_div(p.P, 128), n = sm_count();
  const int64_t rows = (int64_t)p.B * p.T * a.G;
  t.row_tiles = (int)ceil_div(rows, 256);
  const int64_t items = (int64_t)p.n_kv * t.row_tiles, most = std::min(tiles, n / items);
  const bool whole = most > 0 && (most == tiles || items * most * 10 >= n * (p.D == 128 ? 8 : 9));
  int64_t pieces = whole ? most : 0;
  if (most > 0 && private_keys(p) > 0) {
    const double keys = (p.ids ? (double)p.T * p.W : (double)p.S) * p.B * p.n_kv;
    const double mine = items * (6.0 + tiles * (rows > 128 ? 1.6 : 0.9)), other = 0.6 * keys * 4 * p.D / 55e3;
    const double share = std::max(0.4, mine / (mine + other));
    int64_t k = std::min((int64_t)(n * share / items), ceil_div(tiles, 8));
    const int64_t rows_own = p.ids ? a.G : (int64_t)p.T * a.G, row_tile = rows_own <= 16 ? 16 : 32;
    const int64_t warps = p.B * (p.ids ? p.T : 1) * ceil_div(private_keys(p), 4 * stream_tile(p.D)) * p.n_kv *
                          ceil_div(rows_own, row_tile);
    k = std::max(k, std::min(most, (n - ceil_div(warps, row_tile == 16 ? 12 : 8)) / items));
    if (k < most && (pieces || items * k * 10 >= n * share * 7)) pieces = std::max<int64_t>(1, k);
  }
  t.whole_cells = pieces > 0;
  t.cells_k = (int)(pieces ? pieces : std::min(tiles, ceil_div(n, items)));
  t.blocks = (int)(pieces ? items * pieces : std::min(n, items * tiles));
  return t;
}

// The streaming kernel's groups and the parts of a sequence.  Every SM holds
// twelve warps of 16 rows or eight of 32 (three or two blocks), and every warp
// gets one share of the line: cutting it finer cost 1 to 7 percent.  The share of
// a group depends on the lengths, which only the device knows; the parts allow
// for lines down to a quarter of the longest.
StreamLine plan_stream(AttnArgs& a) {
  const attn_problem& p = a.p;
  StreamLine l{};
  const PrefixWay way = prefix_way(p);
  l.after = way == kTensorCore;
  const int64_t rows_pre = (int64_t)p.B * p.T * a.G;
  const int64_t rows = std::max<int64_t>(p.S == 0 ? 1 : p.ids ? a.G : (int64_t)p.T * a.G, way == kLine ? rows_pre : 1);
  l.row_tile = rows <= 16 ? 16 : 32;
  l.members = (int)(p.n_kv * ceil_div(rows, l.row_tile));
  const int64_t warps = (l.row_tile == 16 ? 12 : 8) * (int64_t)sm_count();
  l.seqs = private_keys(p) == 0 ? 0 : p.ids ? p.B * p.T : p.B;
  // A unit is a tile where every share has sixteen of them or more (an even cut
  // matters), else four: a sequence's start takes about the time of four tiles.
  // Where even units of two find warps for all, and do not make a row's pieces
  // many, two: a short call waits for its longest share (one request of 200 slots
  // behind 1,024: 9.4 against 10.6 us).  Beside a prefix under many rows, on the
  // tensor cores or on a line of its own, it stays four (two: 31 against 26 us).
  const int64_t tile = stream_tile(p.D);
  const int64_t tiles = (way == kLine ? ceil_div(p.P, tile) : 0) + l.seqs * ceil_div(private_keys(p), tile);
  const bool fine = tiles * l.members >= 16 * warps;
  const int64_t pieces = (way == kLine ? ceil_div(p.P, 2 * tile) : 0) + ceil_div(private_keys(p), 2 * tile);
  const bool two = (way == kNone || way == kLine) && tiles * l.members <= warps && pieces <= 96;
  l.unit_shift = (p.D == 128 ? 4 : 5) + (fine ? 0 : two ? 1 : 2);
  const int64_t unit = (int64_t)1 << l.unit_shift;
  if (way == kLine) l.prefix_units = (int)ceil_div(p.P, unit);
  if (way == kOwnLine) {
    l.own_units = (int)ceil_div(p.P, unit);
    l.own_members = (int)(p.n_kv * ceil_div(rows_pre, l.row_tile));
    l.own_groups = (int)std::min<int64_t>(l.own_units, std::max<int64_t>(1, warps / l.own_members));
    l.own_blocks = (int)ceil_div((int64_t)l.own_members * l.own_groups, 4);
    a.parts_prefix = l.own_groups;
  }
  const int64_t longest = ceil_div(private_keys(p), unit);
  const int64_t total = l.prefix_units + l.seqs * longest;
  // beside the tensor-core kernel two shares for each place: the second ones
  // begin when that kernel leaves its SMs, or where a first one ends
  l.groups = total == 0 ? 0 : (int)std::max<int64_t>(1, (way == kTensorCore ? 2 : 1) * warps / l.members);
  l.least = (int)std::max<int64_t>(1, ceil_div(total, 4 * std::max<int64_t>(1, l.groups)));
  // Lists have one length; short lines are cut as if all caches were full, which
  // saves their blocks the look at the lengths.
  if (p.ids || (!fine && total <= 2 * l.groups)) l.uniform = (int)longest;
  if (l.uniform || l.seqs == 0) l.groups = (int)std::min<int64_t>(l.groups, std::max<int64_t>(1, total / l.least));
  auto parts = [&](int64_t units) { return units == 0 ? 0 : (int)std::min(units, ceil_div(units - 1, l.least) + 1); };
  if (way == kLine) a.parts_prefix = parts(l.prefix_units);
  a.parts_private = l.seqs ? parts(longest) : 0;
  return l;
}

void plan_parts(AttnArgs& a) {
  if (prefix_way(a.p) == kTensorCore) {
    const AttnTcArgs t = plan_tc(a);
    a.parts_prefix = t.cells_k * (t.whole_cells ? 1 : 2);
  }
  plan_stream(a);
}

struct AttnWs {
  size_t po, pml, sc, total;
};

AttnWs layout(const AttnArgs& a, bool mass) {
  const attn_problem& p = a.p;
  const size_t rows = (size_t)p.B * p.T * p.Hq;
  const size_t parts = (size_t)(a.parts_prefix + a.parts_private);
  AttnWs w;
  WsCarver c(nullptr);
  c.take<float>(rows * parts * p.D);
  w.po = 0;
  w.pml = (c.used + 255) & ~size_t(255);
  c.take<float2>(rows * parts);
  w.sc = (c.used + 255) & ~size_t(255);
  if (mass) c.take<float>(rows * (size_t)a.sc_ld);
  w.total = c.used + 256;
  return w;
}

AttnArgs make_args(const attn_problem& p) {
  AttnArgs a{};
  a.p = p;
  a.G = p.Hq / p.n_kv;
  a.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
  a.sc_ld = (private_keys(p) + 4) & ~int64_t(3);  // rows of 16-byte groups, with room behind an odd last slot
  plan_parts(a);
  return a;
}

}  // namespace

// The lines of key tiles, the partial results and the rows of q (in 16 bytes)
// are counted in 32 bits.
static bool fits(const AttnArgs& a) {
  const attn_problem& p = a.p;
  const int64_t tile = stream_tile(p.D), most = (int64_t)1 << 31;
  const int64_t seqs = (int64_t)p.B * (p.ids ? p.T : 1);
  const int64_t line = ceil_div(p.P, tile) + seqs * std::max<int64_t>(1, ceil_div(private_keys(p), tile));
  const int64_t tiles = ceil_div((int64_t)p.B * p.T * a.G, 256) * p.n_kv * ceil_div(p.P, 128);
  const int64_t rows = (int64_t)p.B * p.T * p.Hq;
  auto span = [](int64_t n, int64_t stride) { return (n - 1) * (stride < 0 ? -stride : stride); };
  const int64_t q = span(p.B, p.q_stride_b) + span(p.T, p.q_stride_t) + span(p.Hq, p.q_stride_h);
  return line < most && tiles < most && rows * (a.parts_prefix + a.parts_private) < most && q / 8 < most;
}

size_t attn_shared_ws(const attn_problem& p, bool mass) {
  const AttnArgs a = make_args(p);
  return fits(a) ? layout(a, mass).total : 0;
}

idx_status launch_attn_shared(const attn_problem& p, void* out, float* lse, float* mass, int mass_heads, void* ws,
                              size_t ws_bytes, cudaStream_t st, cudaError_t* err) {
  AttnArgs a = make_args(p);
  if (!fits(a)) return IDX_ERR_UNSUPPORTED;
  const AttnWs w = layout(a, mass != nullptr);
  if (ws_bytes < w.total) return IDX_ERR_WORKSPACE_TOO_SMALL;
  if (!ws) return IDX_ERR_INVALID_ARG;
  char* base = (char*)(((uintptr_t)ws + 255) & ~uintptr_t(255));
  a.po = (float*)(base + w.po);
  a.pml = (float2*)(base + w.pml);
  a.sc = mass ? (float*)(base + w.sc) : nullptr;
  a.out = out;
  a.lse = lse;
  a.mass = mass;
  a.mass_heads = mass_heads;
  cudaError_t e = cudaSuccess;
  if (prefix_way(p) == kTensorCore) e = launch_attn_tc(plan_tc(a), st);
  const StreamLine line = plan_stream(a);
  if (e == cudaSuccess && line.own_blocks + line.prefix_units + line.seqs > 0) e = launch_attn_stream(a, line, st);
  if (e == cudaSuccess) e = launch_attn_finish(a, st);
  *err = e;
  return e == cudaSuccess ? IDX_OK : IDX_ERR_CUDA;
}

}  // namespace idx
