// C-ABI entry points of libidx: argument validation on the host, workspace
// carving and dispatch to the kernels.  Nothing here computes on the host.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <mutex>
#include <vector>
#include <cstring>
#include <string>

#include "internal.h"

namespace idx {

static std::vector<uint32_t (*)()>& error_words() {
  static std::vector<uint32_t (*)()> v;
  return v;
}
static std::mutex g_error_words_mu;

void register_error_word(uint32_t (*take)()) {
  std::lock_guard<std::mutex> lk(g_error_words_mu);
  error_words().push_back(take);
}

static std::vector<cudaError_t (*)(uint64_t)>& wait_limit_setters() {
  static std::vector<cudaError_t (*)(uint64_t)> v;
  return v;
}

void register_wait_limit_setter(cudaError_t (*set)(uint64_t)) {
  std::lock_guard<std::mutex> lk(g_error_words_mu);
  wait_limit_setters().push_back(set);
}

static thread_local std::string g_last_error;

idx_status fail(idx_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

static idx_status cuda_status(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return IDX_OK;
  return fail(IDX_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

// SM count of the calling thread's current device, cached per device (the
// kernels size their grids by it, and a process may switch devices).
int sm_count() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  if (cached) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 1;
  if (cached) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

static idx_status check_problem(const idx_problem* p) {
  if (!p) return fail(IDX_ERR_INVALID_ARG, "problem is NULL");
  if (p->M < 0 || p->H <= 0 || p->D <= 0 || p->n_keys < 0 || p->max_key_len < 0)
    return fail(IDX_ERR_INVALID_ARG, "negative or zero size (M=%lld H=%d D=%d n_keys=%lld max_key_len=%d)",
                (long long)p->M, p->H, p->D, (long long)p->n_keys, p->max_key_len);
  // bounds that keep every size derived from the problem (the M x max_key_len
  // scores, workspaces, key offsets) far inside 64-bit arithmetic (checked by
  // division, so the check itself cannot wrap)
  if (p->M > ((int64_t)1 << 40) || p->n_keys > ((int64_t)1 << 46) ||
      (p->max_key_len > 0 && p->M > ((int64_t)1 << 56) / p->max_key_len))
    return fail(IDX_ERR_UNSUPPORTED, "problem too large (M=%lld max_key_len=%d n_keys=%lld)", (long long)p->M,
                p->max_key_len, (long long)p->n_keys);
  if (p->M > 0 && (!p->q || !p->w || !p->key_len))
    return fail(IDX_ERR_INVALID_ARG, "q, w and key_len must be non-NULL");
  if (p->n_keys > 0 && !p->keys) return fail(IDX_ERR_INVALID_ARG, "keys is NULL");
  if (p->H > 128) return fail(IDX_ERR_UNSUPPORTED, "H=%d above 128", p->H);
  const bool f32 = p->q_dtype == IDX_F32 && p->k_dtype == IDX_F32;
  const bool bf16 = p->q_dtype == IDX_BF16 && p->k_dtype == IDX_BF16;
  const bool fp8 = p->q_dtype == IDX_BF16 && p->k_dtype == IDX_FP8_E4M3;
  if (!(f32 || bf16 || fp8))
    return fail(IDX_ERR_UNSUPPORTED, "dtype pair (q %d, keys %d) not supported", p->q_dtype, p->k_dtype);
  if (fp8 && !p->key_scale) return fail(IDX_ERR_INVALID_ARG, "FP8 keys need key_scale");
  if (!fp8 && p->key_scale) return fail(IDX_ERR_INVALID_ARG, "key_scale is only for FP8 keys");
  if ((f32 || bf16) && p->D > 256) return fail(IDX_ERR_UNSUPPORTED, "D=%d above 256", p->D);
  if ((int64_t)p->H * p->D > 16384) return fail(IDX_ERR_UNSUPPORTED, "H*D above 16384");
  if (fp8 && !score_uses_tensor_cores(*p))
    return fail(IDX_ERR_UNSUPPORTED, "FP8 keys need D=128 and H in {16,32,64,128}");
  if (!p->key_off && p->max_key_len > p->n_keys)
    return fail(IDX_ERR_INVALID_ARG, "shared keys: max_key_len %d exceeds n_keys %lld", p->max_key_len,
                (long long)p->n_keys);
  return IDX_OK;
}

static bool aligned16(const void* base, std::initializer_list<int64_t> strides) {
  if ((uintptr_t)base & 15) return false;
  for (int64_t s : strides)
    if (s & 7) return false;  // 2-byte elements
  return true;
}

static idx_status check_attn(const attn_problem* p) {
  if (!p) return fail(IDX_ERR_INVALID_ARG, "problem is NULL");
  if (p->B < 0 || p->T < 1 || p->Hq < 1 || p->n_kv < 1 || p->S < 0 || p->P < 0 || p->W < 0)
    return fail(IDX_ERR_INVALID_ARG, "negative or zero size (B=%d T=%d Hq=%d n_kv=%d S=%lld P=%lld W=%lld)", p->B,
                p->T, p->Hq, p->n_kv, (long long)p->S, (long long)p->P, (long long)p->W);
  if (p->Hq % p->n_kv) return fail(IDX_ERR_INVALID_ARG, "Hq=%d is no multiple of n_kv=%d", p->Hq, p->n_kv);
  if (p->dtype != IDX_BF16 && p->dtype != IDX_F16)
    return fail(IDX_ERR_UNSUPPORTED, "dtype %d (IDX_BF16 or IDX_F16)", p->dtype);
  if (p->D != 64 && p->D != 128) return fail(IDX_ERR_UNSUPPORTED, "D=%d (64 or 128)", p->D);
  // strides whose products with any index stay far inside 64 bits
  for (int64_t x : {p->q_stride_b, p->q_stride_t, p->q_stride_h, p->k_stride_b, p->k_stride_s, p->k_stride_h,
                    p->v_stride_b, p->v_stride_s, p->v_stride_h, p->pk_stride_s, p->pk_stride_h, p->pv_stride_s,
                    p->pv_stride_h})
    if (x > ((int64_t)1 << 40) || x < -((int64_t)1 << 40))
      return fail(IDX_ERR_UNSUPPORTED, "stride of %lld elements", (long long)x);
  // bounds that keep grids, row counts and key indices inside 32 bits
  if (p->S > (1 << 30) || p->P > (1 << 30) || p->W > (1 << 30) ||
      (int64_t)p->B * p->T > ((int64_t)1 << 30) / p->Hq || (int64_t)p->T * p->Hq > (1 << 20))
    return fail(IDX_ERR_UNSUPPORTED, "problem too large (B=%d T=%d Hq=%d S=%lld P=%lld W=%lld)", p->B, p->T, p->Hq,
                (long long)p->S, (long long)p->P, (long long)p->W);
  if (!(p->scale == p->scale) || p->scale - p->scale != 0.f) return fail(IDX_ERR_INVALID_ARG, "scale is not finite");
  if (p->B == 0) return IDX_OK;
  if (!p->q) return fail(IDX_ERR_INVALID_ARG, "q is NULL");
  if (p->S > 0 && (!p->k || !p->v || !p->len)) return fail(IDX_ERR_INVALID_ARG, "S > 0 needs k, v and len");
  if (p->P > 0 && (!p->pk || !p->pv)) return fail(IDX_ERR_INVALID_ARG, "P > 0 needs pk and pv");
  if (!p->ids && (p->W || p->ids_per_head)) return fail(IDX_ERR_INVALID_ARG, "W or ids_per_head without ids");
  if (p->ids && p->S == 0) return fail(IDX_ERR_INVALID_ARG, "ids without a private cache");
  if (!aligned16(p->q, {p->q_stride_b, p->q_stride_t, p->q_stride_h}) ||
      (p->S > 0 && (!aligned16(p->k, {p->k_stride_b, p->k_stride_s, p->k_stride_h}) ||
                    !aligned16(p->v, {p->v_stride_b, p->v_stride_s, p->v_stride_h}))) ||
      (p->P > 0 && (!aligned16(p->pk, {p->pk_stride_s, p->pk_stride_h}) ||
                    !aligned16(p->pv, {p->pv_stride_s, p->pv_stride_h}))))
    return fail(IDX_ERR_INVALID_ARG, "q, k, v, pk and pv need 16-byte aligned bases and strides");
  return IDX_OK;
}

}  // namespace idx

using namespace idx;

extern "C" {

const char* idx_last_error_string(void) { return g_last_error.c_str(); }

uint32_t idx_device_error(void) {
  cudaDeviceSynchronize();
  uint32_t v = 0;
  std::lock_guard<std::mutex> lk(g_error_words_mu);
  for (auto take : error_words()) v |= take();
  return v;
}

idx_status idx_set_wait_limit_ns(uint64_t ns) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_status(e, "idx_set_wait_limit_ns");
  std::lock_guard<std::mutex> lk(g_error_words_mu);
  for (auto set : wait_limit_setters()) {
    e = set(ns);
    if (e != cudaSuccess) return cuda_status(e, "idx_set_wait_limit_ns");
  }
  return IDX_OK;
}

idx_status idx_score(const idx_problem* p, float* scores, int64_t ld_scores, void* stream) {
  idx_status st = check_problem(p);
  if (st) return st;
  if (ld_scores < p->max_key_len) return fail(IDX_ERR_INVALID_ARG, "ld_scores < max_key_len");
  if (p->M > 0 && p->max_key_len > 0 && !scores) return fail(IDX_ERR_INVALID_ARG, "scores is NULL");
  return cuda_status(launch_score(*p, scores, ld_scores, (cudaStream_t)stream), "idx_score");
}

size_t idx_topk_workspace_size(const idx_problem* p, int32_t K) {
  if (!p || p->M <= 0) return 0;
  WsCarver c(nullptr);
  c.take<float>((size_t)p->M * (size_t)(p->max_key_len > 0 ? p->max_key_len : 1));
  c.take<char>(topk_dense_ws(p->M, p->max_key_len, K < 1 ? 1 : K));
  return c.used + 256;
}

idx_status idx_topk(const idx_problem* p, int32_t K, int32_t* out_ids, float* out_scores, void* ws, size_t ws_bytes,
                    void* stream) {
  idx_status st = check_problem(p);
  if (st) return st;
  if (K < 1 || K > IDX_MAX_K) return fail(IDX_ERR_INVALID_ARG, "K=%d outside [1, %d]", K, IDX_MAX_K);
  if (p->M > 0 && !out_ids) return fail(IDX_ERR_INVALID_ARG, "out_ids is NULL");
  if (ws_bytes < idx_topk_workspace_size(p, K)) return fail(IDX_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  if (p->M > 0 && !ws) return fail(IDX_ERR_INVALID_ARG, "workspace is NULL");
  if (p->M == 0) return IDX_OK;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t ld = p->max_key_len > 0 ? p->max_key_len : 1;
  WsCarver c(ws);
  float* scores = c.take<float>((size_t)p->M * (size_t)ld);
  char* lists = c.take<char>(topk_dense_ws(p->M, p->max_key_len, K));
  cudaError_t e = launch_score(*p, scores, ld, s);
  if (e != cudaSuccess) return cuda_status(e, "idx_topk/score");
  e = launch_topk_dense(scores, ld, nullptr, p, p->M, p->max_key_len, K, out_ids, out_scores, lists, s);
  return cuda_status(e, "idx_topk/select");
}

size_t idx_topk_prior_workspace_size(const idx_problem* p, int32_t K, int32_t prior_ld,
                                     int32_t candidate_capacity) {
  if (!p || p->M <= 0 || K < 1 || prior_ld < 1 || candidate_capacity < 1) return 0;
  return topk_prior_ws(*p, K, prior_ld, candidate_capacity);
}

static idx_status topk_prior_impl(const idx_problem* p, int32_t K, const int32_t* prior_ids, int32_t prior_ld,
                                  int32_t candidate_capacity, int32_t* out_ids, float* out_scores,
                                  int32_t* row_status, topk_prior_stats* stats, void* ws, size_t ws_bytes,
                                  void* stream, const cudaEvent_t* ev) {
  idx_status st = check_problem(p);
  if (st) return st;
  if (K < 1 || K > IDX_MAX_K) return fail(IDX_ERR_INVALID_ARG, "K=%d outside [1, %d]", K, IDX_MAX_K);
  if (prior_ld < 1) return fail(IDX_ERR_INVALID_ARG, "prior_ld=%d below 1", prior_ld);
  if (candidate_capacity < K)
    return fail(IDX_ERR_INVALID_ARG, "candidate_capacity=%d below K=%d", candidate_capacity, K);
  if (p->M == 0) return IDX_OK;
  if (!out_ids || !prior_ids) return fail(IDX_ERR_INVALID_ARG, "NULL pointer");
  if (ws_bytes < idx_topk_prior_workspace_size(p, K, prior_ld, candidate_capacity))
    return fail(IDX_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  if (!ws) return fail(IDX_ERR_INVALID_ARG, "workspace is NULL");
  return cuda_status(launch_topk_prior(*p, K, prior_ids, prior_ld, candidate_capacity, out_ids, out_scores,
                                       row_status, stats, ws, (cudaStream_t)stream, ev),
                     "idx_topk_prior");
}

idx_status idx_topk_prior(const idx_problem* p, int32_t K, const int32_t* prior_ids, int32_t prior_ld,
                          int32_t candidate_capacity, int32_t* out_ids, float* out_scores, int32_t* row_status,
                          topk_prior_stats* stats, void* ws, size_t ws_bytes, void* stream) {
  return topk_prior_impl(p, K, prior_ids, prior_ld, candidate_capacity, out_ids, out_scores, row_status, stats, ws,
                         ws_bytes, stream, nullptr);
}

idx_status idx_topk_prior_events(const idx_problem* p, int32_t K, const int32_t* prior_ids, int32_t prior_ld,
                                 int32_t candidate_capacity, int32_t* out_ids, float* out_scores,
                                 int32_t* row_status, topk_prior_stats* stats, void* ws, size_t ws_bytes,
                                 void* const* events, int32_t n_events, void* stream) {
  if (!events || n_events < 6) return fail(IDX_ERR_INVALID_ARG, "idx_topk_prior_events needs 6 events");
  cudaEvent_t ev[6];
  for (int i = 0; i < 6; ++i) ev[i] = (cudaEvent_t)events[i];
  return topk_prior_impl(p, K, prior_ids, prior_ld, candidate_capacity, out_ids, out_scores, row_status, stats, ws,
                         ws_bytes, stream, ev);
}

size_t idx_topk_scores_workspace_size(int64_t M, int32_t max_len, int32_t K) {
  if (M <= 0 || max_len <= 0) return 0;
  return topk_dense_ws(M, max_len, K < 1 ? 1 : K);
}

idx_status idx_topk_scores(const float* scores, int64_t ld, const int32_t* lens, int64_t M, int32_t max_len,
                           int32_t K, int32_t* out_ids, float* out_scores, void* ws, size_t ws_bytes,
                           void* stream) {
  if (M < 0 || max_len < 0 || ld < max_len) return fail(IDX_ERR_INVALID_ARG, "bad sizes");
  if (K < 1 || K > IDX_MAX_K) return fail(IDX_ERR_INVALID_ARG, "K=%d outside [1, %d]", K, IDX_MAX_K);
  if (M > 0 && (!lens || !out_ids || (max_len > 0 && !scores))) return fail(IDX_ERR_INVALID_ARG, "NULL pointer");
  const size_t need = idx_topk_scores_workspace_size(M, max_len, K);
  if (ws_bytes < need) return fail(IDX_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  if (need > 0 && !ws) return fail(IDX_ERR_INVALID_ARG, "workspace is NULL");
  if (M == 0) return IDX_OK;
  return cuda_status(launch_topk_dense(scores, ld, lens, nullptr, M, max_len, K, out_ids, out_scores, ws,
                                       (cudaStream_t)stream),
                     "idx_topk_scores");
}

size_t dosa_topk_workspace_size(const idx_problem* p, int32_t K, const dosa_params* dp, int32_t seed_ld) {
  if (!p || !dp || p->M <= 0) return 0;
  return dosa_ws(*p, K, *dp, seed_ld);
}

idx_status dosa_topk(const idx_problem* p, int32_t K, const dosa_params* dp, const int32_t* seed_ids,
                     int32_t seed_ld, int32_t* out_ids, float* out_scores, int32_t* row_status, dosa_stats* stats,
                     void* ws, size_t ws_bytes, void* stream) {
  idx_status st = check_problem(p);
  if (st) return st;
  if (!dp) return fail(IDX_ERR_INVALID_ARG, "params is NULL");
  if (K < 1 || K > IDX_MAX_K) return fail(IDX_ERR_INVALID_ARG, "K=%d outside [1, %d]", K, IDX_MAX_K);
  if (dp->n_seed < 0 || dp->retained_heads < 1 || dp->n_sample < 1 || dp->candidate_capacity < 0 ||
      !(dp->act_freq_min >= 0.0f && dp->act_freq_min <= 1.0f) || !(dp->margin_gamma >= 0.0f))
    return fail(IDX_ERR_INVALID_ARG, "bad dosa_params");
  if (seed_ids && seed_ld < 1) return fail(IDX_ERR_INVALID_ARG, "seed_ld < 1");
  if (p->M > 0 && !out_ids) return fail(IDX_ERR_INVALID_ARG, "out_ids is NULL");
  if (ws_bytes < dosa_topk_workspace_size(p, K, dp, seed_ids ? seed_ld : 0))
    return fail(IDX_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  if (p->M == 0) return IDX_OK;
  if (!ws) return fail(IDX_ERR_INVALID_ARG, "workspace is NULL");
  return cuda_status(launch_dosa(*p, K, *dp, seed_ids, seed_ids ? seed_ld : 0, out_ids, out_scores, row_status,
                                 stats, ws, ws_bytes, (cudaStream_t)stream),
                     "dosa_topk");
}

idx_status dosa_workspace_layout(const idx_problem* p, int32_t K, const dosa_params* dp, int32_t seed_ld,
                                 dosa_ws_layout* out) {
  idx_status st = check_problem(p);
  if (st) return st;
  if (!dp || !out) return fail(IDX_ERR_INVALID_ARG, "NULL pointer");
  if (K < 1 || K > IDX_MAX_K) return fail(IDX_ERR_INVALID_ARG, "K=%d outside [1, %d]", K, IDX_MAX_K);
  if (!dosa_layout(*p, K, *dp, seed_ld > 0 ? seed_ld : 0, out))
    return fail(IDX_ERR_UNSUPPORTED, "dosa_topk takes the unpruned path for this shape");
  return IDX_OK;
}

idx_status witness_merge(int32_t* topk_ids, int64_t rows, int32_t topk, const int32_t* context_lens,
                         int64_t n_context_lens, int32_t keep, int32_t num_segments, int32_t max_replacements,
                         void* stream) {
  if (num_segments == 0) return IDX_OK;
  if (num_segments < 0 || num_segments > IDX_MAX_SEGMENTS)
    return fail(IDX_ERR_SEGMENTS_OUT_OF_RANGE, "num_segments=%d outside [1, %d]", num_segments, IDX_MAX_SEGMENTS);
  if (keep < 0 || keep > topk) return fail(IDX_ERR_KEEP_OUT_OF_RANGE, "keep=%d outside [0, topk=%d]", keep, topk);
  if (rows < 0 || topk < 0 || max_replacements < 0) return fail(IDX_ERR_INVALID_ARG, "negative size");
  if (n_context_lens < rows)
    return fail(IDX_ERR_ROWS_MISMATCH, "%lld context lengths for %lld rows", (long long)n_context_lens,
                (long long)rows);
  const int32_t B = max_replacements < topk - keep ? max_replacements : topk - keep;
  if (B <= 0 || rows == 0) return IDX_OK;
  if (!topk_ids || !context_lens) return fail(IDX_ERR_INVALID_ARG, "NULL pointer");
  return cuda_status(launch_witness_merge(topk_ids, rows, topk, context_lens, keep, num_segments, B,
                                          (cudaStream_t)stream),
                     "witness_merge");
}

idx_status witness_indices(const int32_t* learned, int64_t rows, int32_t topk, const int32_t* context_lens,
                           int64_t n_context_lens, int32_t num_segments, int32_t* out, void* stream) {
  if (num_segments <= 0 || num_segments > IDX_MAX_SEGMENTS)
    return fail(IDX_ERR_SEGMENTS_OUT_OF_RANGE, "num_segments=%d outside [1, %d]", num_segments, IDX_MAX_SEGMENTS);
  if (rows < 0 || topk < 0) return fail(IDX_ERR_INVALID_ARG, "negative size");
  if (n_context_lens < rows)
    return fail(IDX_ERR_ROWS_MISMATCH, "%lld context lengths for %lld rows", (long long)n_context_lens,
                (long long)rows);
  if (rows == 0) return IDX_OK;
  if ((topk > 0 && !learned) || !context_lens || !out) return fail(IDX_ERR_INVALID_ARG, "NULL pointer");
  return cuda_status(launch_witness_indices(learned, rows, topk, context_lens, num_segments, out,
                                            (cudaStream_t)stream),
                     "witness_indices");
}

size_t block_select_workspace_size(int64_t Q, int32_t n_kv, int64_t L, const block_sparse_config* cfg) {
  if (!cfg || Q <= 0 || n_kv <= 0 || L <= 0) return 0;
  return block_select_ws(Q, n_kv, L, *cfg);
}

static idx_status block_select_impl(const float* index_q, const float* index_k, const int32_t* query_pos, int64_t Q,
                                    int32_t n_kv, int32_t D, int64_t L, const block_sparse_config* cfg, int32_t* out,
                                    int32_t out_width, int32_t* out_count, block_select_stats* stats, void* ws,
                                    size_t ws_bytes, void* stream, const cudaEvent_t* ev) {
  if (!cfg) return fail(IDX_ERR_INVALID_ARG, "config is NULL");
  if (Q < 0 || n_kv < 0 || D <= 0 || L < 0 || cfg->block_size < 0 || cfg->top_blocks < 0 || cfg->init_blocks < 0 ||
      cfg->local_blocks < 0)
    return fail(IDX_ERR_INVALID_ARG, "negative size or config field");
  const int64_t need_w = cfg->top_blocks > (int64_t)cfg->init_blocks + cfg->local_blocks
                             ? cfg->top_blocks
                             : (int64_t)cfg->init_blocks + cfg->local_blocks;
  if (out_width < need_w || out_width > IDX_MAX_K)
    return fail(IDX_ERR_INVALID_ARG, "out_width=%d must be in [max(top, init+local)=%lld, %d]", out_width,
                (long long)need_w, IDX_MAX_K);
  if (D > 256) return fail(IDX_ERR_UNSUPPORTED, "D=%d above 256", D);
  if (D == 128 && (((uintptr_t)index_q | (uintptr_t)index_k) & 15))
    return fail(IDX_ERR_INVALID_ARG, "index_q/index_k must be 16-byte aligned");
  if (Q * n_kv == 0) return IDX_OK;
  if (!index_q || !query_pos || !out || (L > 0 && !index_k)) return fail(IDX_ERR_INVALID_ARG, "NULL pointer");
  if (ws_bytes < block_select_workspace_size(Q, n_kv, L, cfg))
    return fail(IDX_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  if (block_select_workspace_size(Q, n_kv, L, cfg) > 0 && !ws) return fail(IDX_ERR_INVALID_ARG, "workspace is NULL");
  return cuda_status(launch_block_select(index_q, index_k, query_pos, Q, n_kv, D, L, *cfg, out, out_width, out_count,
                                         ws, (cudaStream_t)stream, stats, true, ev),
                     "block_select");
}

idx_status block_select(const float* index_q, const float* index_k, const int32_t* query_pos, int64_t Q,
                        int32_t n_kv, int32_t D, int64_t L, const block_sparse_config* cfg, int32_t* out,
                        int32_t out_width, int32_t* out_count, block_select_stats* stats, void* ws,
                        size_t ws_bytes, void* stream) {
  return block_select_impl(index_q, index_k, query_pos, Q, n_kv, D, L, cfg, out, out_width, out_count, stats, ws,
                           ws_bytes, stream, nullptr);
}

idx_status block_select_events(const float* index_q, const float* index_k, const int32_t* query_pos, int64_t Q,
                               int32_t n_kv, int32_t D, int64_t L, const block_sparse_config* cfg, int32_t* out,
                               int32_t out_width, int32_t* out_count, block_select_stats* stats, void* ws,
                               size_t ws_bytes, void* const* events, int32_t n_events, void* stream) {
  if (!events || n_events < 6) return fail(IDX_ERR_INVALID_ARG, "block_select_events needs 6 events");
  cudaEvent_t ev[6];
  for (int i = 0; i < 6; ++i) ev[i] = (cudaEvent_t)events[i];
  return block_select_impl(index_q, index_k, query_pos, Q, n_kv, D, L, cfg, out, out_width, out_count, stats, ws,
                           ws_bytes, stream, ev);
}

idx_status block_positions(const int32_t* blocks, const int32_t* counts, int64_t Q, int32_t n_kv, int32_t W,
                           const int32_t* query_pos, int64_t L, int32_t block_size, int32_t* out, int32_t out_width,
                           int32_t* out_count, void* stream) {
  if (Q < 0 || n_kv <= 0 || W < 0 || L < 0 || block_size < 0)
    return fail(IDX_ERR_INVALID_ARG, "negative size, or n_kv <= 0");
  if (W > IDX_MAX_K) return fail(IDX_ERR_INVALID_ARG, "W=%d above %d", W, IDX_MAX_K);
  if ((int64_t)out_width < (int64_t)W * block_size || out_width < 0)
    return fail(IDX_ERR_INVALID_ARG, "out_width=%d below W*block_size=%lld", out_width, (long long)W * block_size);
  if (Q * n_kv == 0) return IDX_OK;
  if ((W > 0 && !blocks) || !query_pos || (out_width > 0 && !out)) return fail(IDX_ERR_INVALID_ARG, "NULL pointer");
  return cuda_status(launch_block_positions(blocks, counts, Q * n_kv, W, query_pos, n_kv, L, block_size, out,
                                            out_width, out_count, (cudaStream_t)stream),
                     "block_positions");
}

size_t attn_shared_workspace_size(const attn_problem* p, int32_t with_mass) {
  if (!p || p->B <= 0 || check_attn(p) != IDX_OK) return 0;
  return attn_shared_ws(*p, with_mass != 0 && p->S > 0);
}

idx_status attn_shared(const attn_problem* p, void* out, float* lse, float* mass, int32_t mass_heads, void* ws,
                       size_t ws_bytes, void* stream) {
  idx_status st = check_attn(p);
  if (st) return st;
  if (mass && mass_heads != 1 && mass_heads != p->n_kv)
    return fail(IDX_ERR_INVALID_ARG, "mass_heads=%d is neither 1 nor n_kv=%d", mass_heads, p->n_kv);
  if (p->B == 0) return IDX_OK;
  if (!out) return fail(IDX_ERR_INVALID_ARG, "out is NULL");
  if (p->S == 0) mass = nullptr;
  cudaError_t e = cudaSuccess;
  st = launch_attn_shared(*p, out, lse, mass, mass ? mass_heads : 1, ws, ws_bytes, (cudaStream_t)stream, &e);
  switch (st) {
    case IDX_OK: return st;
    case IDX_ERR_CUDA: return cuda_status(e, "attn_shared");
    case IDX_ERR_WORKSPACE_TOO_SMALL: return fail(st, "workspace too small");
    case IDX_ERR_INVALID_ARG: return fail(st, "workspace is NULL");
    default:
      return fail(st, "problem too large (B=%d T=%d Hq=%d S=%lld P=%lld W=%lld)", p->B, p->T, p->Hq, (long long)p->S,
                  (long long)p->P, (long long)p->W);
  }
}

idx_status cache_evict(const evict_problem* p, int32_t* out_src, int32_t* out_len, int32_t* out_pos, float* out_mass,
                       int64_t out_stride, void* stream) {
  if (!p) return fail(IDX_ERR_INVALID_ARG, "problem is NULL");
  if (p->B < 0 || p->mass_heads < 1 || p->S < 0 || p->stride < p->S || p->n_keep < 1 || p->n_first < 0 ||
      p->n_last < 0 || p->n_planes < 0)
    return fail(IDX_ERR_INVALID_ARG, "bad size (B=%d mass_heads=%d S=%lld stride=%lld n_keep=%lld n_first=%d n_last=%d)",
                p->B, p->mass_heads, (long long)p->S, (long long)p->stride, (long long)p->n_keep, p->n_first,
                p->n_last);
  if ((int64_t)p->n_first + p->n_last > p->n_keep)
    return fail(IDX_ERR_INVALID_ARG, "n_first + n_last = %lld exceeds n_keep = %lld",
                (long long)p->n_first + p->n_last, (long long)p->n_keep);
  if (p->S > evict_max_slots() || p->n_keep > evict_max_slots())
    return fail(IDX_ERR_UNSUPPORTED, "S=%lld, n_keep=%lld: at most %lld slots", (long long)p->S, (long long)p->n_keep,
                (long long)evict_max_slots());
  if ((int64_t)p->B * p->mass_heads > (1 << 20))
    return fail(IDX_ERR_UNSUPPORTED, "B * mass_heads above 2^20");
  if (p->n_planes > IDX_MAX_PLANES)
    return fail(IDX_ERR_INVALID_ARG, "n_planes=%d above %d", p->n_planes, IDX_MAX_PLANES);
  if (p->n_planes > 0 && !p->planes) return fail(IDX_ERR_INVALID_ARG, "planes is NULL");
  int64_t heads = 0;
  for (int i = 0; i < p->n_planes; i++) {
    const evict_plane& q = p->planes[i];
    if (q.heads < 1 || q.row_bytes < 0 || (p->mass_heads > 1 && q.heads != p->mass_heads))
      return fail(IDX_ERR_INVALID_ARG, "plane %d: heads=%d for mass_heads=%d, row_bytes=%lld", i, q.heads,
                  p->mass_heads, (long long)q.row_bytes);
    if (q.row_bytes > (1 << 20)) return fail(IDX_ERR_UNSUPPORTED, "plane %d: rows above 2^20 bytes", i);
    if (!q.base && p->B > 0 && p->S > 0 && q.row_bytes > 0) return fail(IDX_ERR_INVALID_ARG, "plane %d is NULL", i);
    heads += p->mass_heads == 1 ? q.heads : 1;
  }
  if (heads > 65535) return fail(IDX_ERR_UNSUPPORTED, "planes: %lld heads in all, above 65535", (long long)heads);
  if ((out_pos || out_mass) && out_stride < p->n_keep)
    return fail(IDX_ERR_INVALID_ARG, "out_stride=%lld below n_keep=%lld", (long long)out_stride, (long long)p->n_keep);
  if (((out_mass && out_mass == p->mass) || (out_pos && out_pos == p->pos)) && out_stride != p->stride)
    return fail(IDX_ERR_INVALID_ARG, "outputs in place need out_stride == stride");
  if (p->B == 0) return IDX_OK;
  if (!p->len || !out_src || (p->S > 0 && !p->mass)) return fail(IDX_ERR_INVALID_ARG, "NULL pointer");
  return cuda_status(launch_evict(*p, out_src, out_len, out_pos, out_mass, out_stride, (cudaStream_t)stream),
                     "cache_evict");
}

}  // extern "C"
