// Attention of a decode step: the plan of a call (which kernel takes which
// part, how many pieces) and its workspace.  Host only.
#include "attn.cuh"

#include <algorithm>

namespace idx {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Keys of the private part that a row can see at most.
int64_t private_keys(const attn_problem& p) { return p.S == 0 ? 0 : p.ids ? p.W : p.S; }

// How many pieces each part is cut into: pieces of one length everywhere, short
// enough to give every SM two blocks, not below kMinChunk keys (a block's start
// and the join of its warps cost about as much as 128 keys do).
void plan_parts(AttnArgs& a) {
  const attn_problem& p = a.p;
  constexpr int64_t kMinChunk = 128;
  auto tiles = [](int64_t rows) { return ceil_div(rows, rows <= 16 ? 16 : 32); };
  const int64_t pre = (int64_t)p.n_kv * tiles((int64_t)p.B * p.T * a.G);
  const int64_t prv = (int64_t)p.B * p.n_kv * (p.ids ? p.T * tiles(a.G) : tiles((int64_t)p.T * a.G));
  const int64_t keys = private_keys(p);
  const int64_t blocks = 2 * (int64_t)sm_count();
  const int64_t chunk = std::max(kMinChunk, ceil_div(pre * p.P + prv * keys, blocks));
  a.parts_prefix = (int)ceil_div(p.P, chunk);
  a.parts_private = (int)ceil_div(keys, chunk);
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
  a.sc_ld = (private_keys(p) + 2) & ~int64_t(1);
  plan_parts(a);
  return a;
}

}  // namespace

size_t attn_shared_ws(const attn_problem& p, bool mass) { return layout(make_args(p), mass).total; }

cudaError_t launch_attn_shared(const attn_problem& p, void* out, float* lse, float* mass, int mass_heads, void* ws,
                               cudaStream_t st) {
  AttnArgs a = make_args(p);
  const AttnWs w = layout(a, mass != nullptr);
  char* base = (char*)(((uintptr_t)ws + 255) & ~uintptr_t(255));
  a.po = (float*)(base + w.po);
  a.pml = (float2*)(base + w.pml);
  a.sc = mass ? (float*)(base + w.sc) : nullptr;
  a.out = out;
  a.lse = lse;
  a.mass = mass;
  a.mass_heads = mass_heads;
  cudaError_t e = cudaSuccess;
  if (a.parts_prefix) e = launch_attn_stream(a, true, st);
  if (e == cudaSuccess && a.parts_private) e = launch_attn_stream(a, false, st);
  if (e == cudaSuccess) e = launch_attn_finish(a, st);
  return e;
}

}  // namespace idx
