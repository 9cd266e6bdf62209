// Host side of the C ABI: argument checks, the workspace, and kernel launches.
#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>
#include <vector>

#include "dt_internal.cuh"

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

int cuda_fail(cudaError_t e, const char* where) {
  return fail(DT_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Carver {
  size_t off = 0;
  template <typename T>
  size_t take(size_t count) {
    off = (off + 255) / 256 * 256;
    const size_t at = off;
    off += count * sizeof(T);
    return at;
  }
};

}  // namespace

extern "C" {

const char* dt_last_error_string(void) { return g_err; }

int dt_create(const dt_config* cfg, dt_handle** out) {
  if (!cfg || !out) return fail(DT_ERR_ARG, "dt_create: null argument");
  const dt_config c = *cfg;
  if (c.V < 2) return fail(DT_ERR_ARG, "V must be >= 2");
  if (c.K < 1 || c.K > dt::kMaxK || c.K > c.V) return fail(DT_ERR_ARG, "K must be in [1, min(32, V)]");
  if (c.W < 1 || c.W > dt::kMaxW) return fail(DT_ERR_ARG, "W must be in [1, 32]");
  if (c.W * c.K > dt::kCandCap) return fail(DT_ERR_ARG, "W*K must be <= 1024");
  if (c.D_max < 1 || c.D_max > dt::kMaxD) return fail(DT_ERR_ARG, "D_max must be in [1, 16]");
  if (c.P_max < 1 || c.P_max > dt::kMaxP) return fail(DT_ERR_ARG, "P_max must be in [1, 512]");
  if (c.B_max < 1 || c.B_max > 4096) return fail(DT_ERR_ARG, "B_max must be in [1, 4096]");
  if (c.dtype != DT_BF16 && c.dtype != DT_F32) return fail(DT_ERR_ARG, "dtype must be DT_BF16 or DT_F32");

  dt_handle* h = new (std::nothrow) dt_handle();
  if (!h) return fail(DT_ERR_ARG, "out of host memory");
  h->cfg = c;
  h->LW = c.W * c.K;
  h->N = 1 + c.K + (c.D_max - 1) * h->LW;
  if (h->LW < c.K) h->LW = c.K;
  h->B = 0;
  h->depth = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    delete h;
    return cuda_fail(e, "cudaGetDevice");
  }
  e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    delete h;
    return cuda_fail(e, "cudaDeviceGetAttribute");
  }

  e = dt::init_tree_attributes();
  if (e == cudaSuccess) e = dt::init_verify_attributes();
  if (e == cudaSuccess) e = dt::init_select_attributes();
  if (e == cudaSuccess) e = dt::init_meta_attributes();
  if (e == cudaSuccess) e = dt::init_block_attributes();
  if (e == cudaSuccess) e = dt::init_attn_attributes();
  if (e == cudaSuccess) e = dt::init_prompt_attributes();
  if (e != cudaSuccess) {
    delete h;
    return cuda_fail(e, "cudaFuncSetAttribute");
  }

  const size_t BN = (size_t)c.B_max * h->N;
  const size_t rows_max = (size_t)c.B_max * std::max(c.W, c.P_max);
  // the streaming passes place elements with 64-bit products (rows x V) x warps
  const double place = (double)rows_max * (double)c.V * (double)dt::stream_grid(h) * 8.0;
  if (place >= 9.0e18) {
    delete h;
    return fail(DT_ERR_ARG, "B_max * max(W, P_max) * V too large for 64-bit row placement");
  }
  Carver cv;
  const size_t o_token = cv.take<int32_t>(BN), o_parent = cv.take<int32_t>(BN), o_depth = cv.take<int32_t>(BN);
  const size_t o_logc = cv.take<float>(BN), o_value = cv.take<float>(BN), o_dd = cv.take<float2>(BN);
  const size_t o_eslot = cv.take<int32_t>(BN), o_estat = cv.take<float4>(BN);
  const size_t o_lorder = cv.take<int32_t>((size_t)c.B_max * (c.D_max + 1) * h->LW);
  const size_t o_lval = cv.take<float>((size_t)c.B_max * (c.D_max + 1) * h->LW);
  const size_t o_ltok = cv.take<int32_t>((size_t)c.B_max * (c.D_max + 1) * h->LW);
  const size_t o_lcount = cv.take<int32_t>((size_t)c.B_max * (c.D_max + 1));
  const size_t o_front = cv.take<int32_t>((size_t)c.B_max * c.W);
  const size_t o_fval = cv.take<float>((size_t)c.B_max * c.W);
  const size_t o_fcount = cv.take<int32_t>(c.B_max);
  // one partial per (row, segment) of a row-scan launch; launches clamp their segment count to it
  const size_t partial_cap = rows_max * 8 + (size_t)h->num_sms * 64;
  const size_t o_part = cv.take<dt::Partial>(partial_cap);
  const size_t o_rowc = cv.take<int32_t>(rows_max);
  const size_t o_rtau = cv.take<unsigned long long>(rows_max);
  const size_t o_reqc = cv.take<int32_t>(c.B_max);
  const size_t o_rstat = cv.take<dt::RowStat>((size_t)c.B_max * c.P_max);
  const size_t o_slin = cv.take<double>((size_t)c.B_max * c.P_max);
  const size_t o_scnt = cv.take<int32_t>(c.B_max);
  const size_t o_sids = cv.take<int32_t>((size_t)c.B_max * c.P_max);
  const size_t o_cast = cv.take<dt::CastState>(1);
  const size_t o_castr = cv.take<dt::CastState>(c.B_max);
  const size_t o_walk = cv.take<dt::WalkState>(c.B_max);
  const size_t o_bkey = cv.take<unsigned long long>(c.B_max);
  const size_t o_bcnt = cv.take<int32_t>(c.B_max);
  const size_t o_status = cv.take<int32_t>(1);
  const size_t o_ticket = cv.take<unsigned>(1);
  const size_t o_atick = cv.take<unsigned>(h->num_sms);
  const size_t o_pstate = cv.take<int32_t>(c.B_max);
  const size_t total = cv.off;

  void* base = nullptr;
  e = cudaMalloc(&base, total);
  if (e != cudaSuccess) {
    delete h;
    return cuda_fail(e, "cudaMalloc(workspace)");
  }
  e = cudaMemset(base, 0, total);
  if (e != cudaSuccess) {
    cudaFree(base);
    delete h;
    return cuda_fail(e, "cudaMemset(workspace)");
  }
  char* bp = static_cast<char*>(base);
  dt::Workspace& w = h->ws;
  w.token = reinterpret_cast<int32_t*>(bp + o_token);
  w.parent = reinterpret_cast<int32_t*>(bp + o_parent);
  w.node_depth = reinterpret_cast<int32_t*>(bp + o_depth);
  w.logc = reinterpret_cast<float*>(bp + o_logc);
  w.value = reinterpret_cast<float*>(bp + o_value);
  w.node_dd = reinterpret_cast<float2*>(bp + o_dd);
  w.exp_slot = reinterpret_cast<int32_t*>(bp + o_eslot);
  w.exp_stat = reinterpret_cast<float4*>(bp + o_estat);
  w.layer_order = reinterpret_cast<int32_t*>(bp + o_lorder);
  w.layer_val = reinterpret_cast<float*>(bp + o_lval);
  w.layer_tok = reinterpret_cast<int32_t*>(bp + o_ltok);
  w.layer_count = reinterpret_cast<int32_t*>(bp + o_lcount);
  w.frontier = reinterpret_cast<int32_t*>(bp + o_front);
  w.frontier_val = reinterpret_cast<float*>(bp + o_fval);
  w.frontier_count = reinterpret_cast<int32_t*>(bp + o_fcount);
  w.partials = reinterpret_cast<dt::Partial*>(bp + o_part);
  w.partial_cap = (int64_t)partial_cap;
  w.row_counter = reinterpret_cast<int32_t*>(bp + o_rowc);
  w.row_tau = reinterpret_cast<unsigned long long*>(bp + o_rtau);
  w.row_counter_cap = (int64_t)rows_max;
  w.req_counter = reinterpret_cast<int32_t*>(bp + o_reqc);
  w.row_stats = reinterpret_cast<dt::RowStat*>(bp + o_rstat);
  w.sorted_lin = reinterpret_cast<double*>(bp + o_slin);
  w.sorted_cnt = reinterpret_cast<int32_t*>(bp + o_scnt);
  w.sorted_ids = reinterpret_cast<int32_t*>(bp + o_sids);
  w.cast = reinterpret_cast<dt::CastState*>(bp + o_cast);
  w.cast_req = reinterpret_cast<dt::CastState*>(bp + o_castr);
  w.walk = reinterpret_cast<dt::WalkState*>(bp + o_walk);
  w.bonus_key = reinterpret_cast<unsigned long long*>(bp + o_bkey);
  w.bonus_counter = reinterpret_cast<int32_t*>(bp + o_bcnt);
  w.status = reinterpret_cast<int32_t*>(bp + o_status);
  w.ticket = reinterpret_cast<unsigned*>(bp + o_ticket);
  w.attn_tickets = reinterpret_cast<unsigned*>(bp + o_atick);
  w.page_state = reinterpret_cast<int32_t*>(bp + o_pstate);
  if (c.flags & DT_FLAG_TEST_ARRIVED) {
    const std::vector<unsigned> one(h->num_sms, 1u);
    e = cudaMemcpy(w.attn_tickets, one.data(), sizeof(unsigned) * one.size(), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) {
      cudaFree(base);
      delete h;
      return cuda_fail(e, "cudaMemcpy(workspace)");
    }
  }
  h->alloc = base;
  h->alloc_bytes = total;
  *out = h;
  return DT_OK;
}

int dt_destroy(dt_handle* h) {
  if (!h) return fail(DT_ERR_ARG, "dt_destroy: null handle");
  cudaError_t e = cudaFree(h->alloc);
  delete h;
  if (e != cudaSuccess) return cuda_fail(e, "cudaFree(workspace)");
  return DT_OK;
}

int dt_get_tree(const dt_handle* h, dt_tree_view* v) {
  if (!h || !v) return fail(DT_ERR_ARG, "dt_get_tree: null argument");
  v->B = h->B;
  v->K = h->cfg.K;
  v->W = h->cfg.W;
  v->D_max = h->cfg.D_max;
  v->N = h->N;
  v->LW = h->LW;
  v->depth = h->depth;
  v->token = h->ws.token;
  v->parent = h->ws.parent;
  v->node_depth = h->ws.node_depth;
  v->logc = h->ws.logc;
  v->value = h->ws.value;
  v->layer_order = h->ws.layer_order;
  v->layer_count = h->ws.layer_count;
  v->frontier = h->ws.frontier;
  v->frontier_count = h->ws.frontier_count;
  return DT_OK;
}

int dt_get_status(dt_handle* h, cudaStream_t s, int32_t* bits) {
  if (!h || !bits) return fail(DT_ERR_ARG, "dt_get_status: null argument");
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, h->ws.status, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_get_status");
  *bits = v;
  if (v & DT_DEV_TIMEOUT) return fail(DT_ERR_DEVICE_TIMEOUT, "device status 0x%x (a bounded wait ran out)", v);
  if (v) return fail(DT_ERR_DEVICE, "device status 0x%x", v);
  return DT_OK;
}

int dt_clear_status(dt_handle* h, cudaStream_t s) {
  if (!h) return fail(DT_ERR_ARG, "dt_clear_status: null handle");
  cudaError_t e = cudaMemsetAsync(h->ws.status, 0, sizeof(int32_t), s);
  // a call that gave up may have left arrivals behind
  if (e == cudaSuccess) e = cudaMemsetAsync(h->ws.attn_tickets, 0, sizeof(unsigned) * h->num_sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_clear_status");
  return DT_OK;
}

int dt_tree_reset(dt_handle* h, int32_t B, const int32_t* root_token, cudaStream_t s) {
  if (!h || !root_token) return fail(DT_ERR_ARG, "dt_tree_reset: null argument");
  if (B < 1 || B > h->cfg.B_max) return fail(DT_ERR_ARG, "B=%d outside [1, B_max=%d]", B, h->cfg.B_max);
  h->B = B;
  h->depth = 0;
  cudaError_t e = dt::launch_tree_reset(h, root_token, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_tree_reset");
  return DT_OK;
}

int dt_select_frontier(dt_handle* h, const int32_t* width, int32_t width_len, const int32_t* stop,
                       int32_t* frontier_token, cudaStream_t s) {
  if (!h) return fail(DT_ERR_ARG, "dt_select_frontier: null handle");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_select_frontier: no tree (call dt_tree_reset)");
  if (h->depth >= h->cfg.D_max) return fail(DT_ERR_ARG, "dt_select_frontier: tree at D_max");
  if (width && width_len != 1 && width_len != h->B) return fail(DT_ERR_ARG, "width_len must be 1 or B");
  cudaError_t e = dt::launch_select_frontier(h, width, width_len, stop, frontier_token, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_select_frontier");
  return DT_OK;
}

int dt_expand_layer(dt_handle* h, const void* logits, int64_t ld, int32_t F, cudaStream_t s) {
  if (!h || !logits) return fail(DT_ERR_ARG, "dt_expand_layer: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_expand_layer: no tree (call dt_tree_reset)");
  if (h->depth >= h->cfg.D_max) return fail(DT_ERR_ARG, "dt_expand_layer: tree already has D_max layers");
  if (F < 1 || F > h->cfg.W) return fail(DT_ERR_ARG, "F=%d outside [1, W=%d]", F, h->cfg.W);
  if (ld < h->cfg.V) return fail(DT_ERR_ARG, "ld=%lld < V", (long long)ld);
  const size_t esz = h->cfg.dtype == DT_BF16 ? 2 : 4;
  if (!aligned(logits, esz)) return fail(DT_ERR_ARG, "logits not aligned to its element size");
  cudaError_t e = dt::launch_expand(h, logits, ld, F, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_expand_layer");
  return DT_OK;
}

// Host checks shared by the CAST width/depth entry points.
static int check_cast_width_params(const dt_handle* h, const dt_prune_params* p, const dt_prune_out* out) {
  if (!p->S_T || !p->S_D) return fail(DT_ERR_ARG, "cost tables missing");
  if (p->M_rows < 1 || p->N_cols < 1) return fail(DT_ERR_ARG, "table shape must be positive");
  if (!(p->L > 0.0)) return fail(DT_ERR_ARG, "L must be > 0");
  if (p->n0 < 0) return fail(DT_ERR_ARG, "n0 must be >= 0");
  if (p->width_cap < 1 || p->width_cap > h->cfg.W || p->width_cap > p->N_cols)
    return fail(DT_ERR_ARG, "width_cap must be in [1, min(W, N_cols)]");
  if (p->R < 1 || p->R > dt::kMaxFifo) return fail(DT_ERR_ARG, "R must be in [1, 16]");
  if (!out->width || !out->stop) return fail(DT_ERR_ARG, "width and stop outputs required");
  return DT_OK;
}

static int check_policy_args(const dt_handle* h, int32_t policy, const dt_prune_params* p, const dt_prune_out* out,
                             const int32_t* width, int32_t width_len) {
  if (width && width_len != 1 && width_len != h->B) return fail(DT_ERR_ARG, "width_len must be 1 or B");
  if (policy == DT_POLICY_CAST_WIDTH_DEPTH) {
    if (!p || !out) return fail(DT_ERR_ARG, "CAST pruning needs params and outputs");
    return check_cast_width_params(h, p, out);
  }
  if (policy == DT_POLICY_GRAFT_CHECKPOINT) {
    if (!p || !out) return fail(DT_ERR_ARG, "the Graft checkpoint needs params and outputs");
    if (p->n_ckpt < 0 || p->n_ckpt > 16) return fail(DT_ERR_ARG, "n_ckpt must be in [0, 16]");
    if (!out->stop) return fail(DT_ERR_ARG, "stop output required");
    return DT_OK;
  }
  if (policy != DT_POLICY_NONE)
    return fail(DT_ERR_ARG, "policy must be DT_POLICY_NONE, DT_POLICY_CAST_WIDTH_DEPTH or "
                            "DT_POLICY_GRAFT_CHECKPOINT");
  return DT_OK;
}

int dt_expand_prune_select(dt_handle* h, const void* logits, int64_t ld, int32_t F, int32_t policy,
                           const dt_prune_params* p, const dt_prune_out* out, const int32_t* width,
                           int32_t width_len, int32_t* frontier_token, cudaStream_t s) {
  if (!h || !logits) return fail(DT_ERR_ARG, "dt_expand_prune_select: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_expand_prune_select: no tree (call dt_tree_reset)");
  if (h->depth >= h->cfg.D_max) return fail(DT_ERR_ARG, "dt_expand_prune_select: tree already has D_max layers");
  if (F < 1 || F > h->cfg.W) return fail(DT_ERR_ARG, "F=%d outside [1, W=%d]", F, h->cfg.W);
  if (ld < h->cfg.V) return fail(DT_ERR_ARG, "ld=%lld < V", (long long)ld);
  const size_t esz = h->cfg.dtype == DT_BF16 ? 2 : 4;
  if (!aligned(logits, esz)) return fail(DT_ERR_ARG, "logits not aligned to its element size");
  const int rc = check_policy_args(h, policy, p, out, width, width_len);
  if (rc != DT_OK) return rc;
  cudaError_t e = dt::launch_expand_ex(h, logits, ld, F, policy, p, out, width, width_len, frontier_token, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_expand_prune_select");
  return DT_OK;
}

int dt_expand_layer_sampled(dt_handle* h, const void* logits, int64_t ld, int32_t F, uint64_t seed, uint64_t round,
                            cudaStream_t s) {
  if (!h || !logits) return fail(DT_ERR_ARG, "dt_expand_layer_sampled: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_expand_layer_sampled: no tree (call dt_tree_reset)");
  if (h->depth >= h->cfg.D_max) return fail(DT_ERR_ARG, "dt_expand_layer_sampled: tree already has D_max layers");
  if (F < 1 || F > h->cfg.W) return fail(DT_ERR_ARG, "F=%d outside [1, W=%d]", F, h->cfg.W);
  if (ld < h->cfg.V) return fail(DT_ERR_ARG, "ld=%lld < V", (long long)ld);
  if (h->N > 4096) return fail(DT_ERR_ARG, "sampled drafts need at most 4096 nodes per request (draw counter)");
  const size_t esz = h->cfg.dtype == DT_BF16 ? 2 : 4;
  if (!aligned(logits, esz)) return fail(DT_ERR_ARG, "logits not aligned to its element size");
  cudaError_t e = dt::launch_expand(h, logits, ld, F, s, true, seed, round);
  if (e != cudaSuccess) return cuda_fail(e, "dt_expand_layer_sampled");
  return DT_OK;
}

int dt_block_expand(dt_handle* h, const void* logits, int64_t ld, int32_t L, const dt_prune_params* p,
                    const dt_prune_out* out, cudaStream_t s) {
  if (!h || !logits) return fail(DT_ERR_ARG, "dt_block_expand: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_block_expand: no tree (call dt_tree_reset)");
  if (h->depth != 0) return fail(DT_ERR_ARG, "dt_block_expand: the tree must be right after dt_tree_reset");
  if (L < 1 || L > h->cfg.D_max) return fail(DT_ERR_ARG, "L=%d outside [1, D_max=%d]", L, h->cfg.D_max);
  if ((int64_t)h->B * L > h->ws.row_counter_cap) return fail(DT_ERR_ARG, "B*L exceeds B_max*max(W, P_max)");
  if (ld < h->cfg.V) return fail(DT_ERR_ARG, "ld=%lld < V", (long long)ld);
  const size_t esz = h->cfg.dtype == DT_BF16 ? 2 : 4;
  if (!aligned(logits, esz)) return fail(DT_ERR_ARG, "logits not aligned to its element size");
  if (p) {
    if (!out || !out->stop) return fail(DT_ERR_ARG, "dt_block_expand: the gates need out->stop");
    if (p->n_ckpt < 0 || p->n_ckpt > 16) return fail(DT_ERR_ARG, "n_ckpt must be in [0, 16]");
  }
  cudaError_t e = dt::launch_block_expand(h, logits, ld, L, p, out, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_block_expand");
  return DT_OK;
}

int dt_cast_prune(dt_handle* h, int32_t policy, const dt_prune_params* p, const dt_prune_out* out,
                  cudaStream_t s) {
  if (!h || !p || !out) return fail(DT_ERR_ARG, "dt_cast_prune: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_cast_prune: no tree (call dt_tree_reset)");
  if (policy == DT_POLICY_CAST_WIDTH_DEPTH || policy == DT_POLICY_CAST_VERIFY) {
    if (!p->S_T || (policy == DT_POLICY_CAST_WIDTH_DEPTH && !p->S_D))
      return fail(DT_ERR_ARG, "cost tables missing");
    if (p->M_rows < 1 || p->N_cols < 1) return fail(DT_ERR_ARG, "table shape must be positive");
    if (!(p->L > 0.0)) return fail(DT_ERR_ARG, "L must be > 0");
    if (p->n0 < 0) return fail(DT_ERR_ARG, "n0 must be >= 0");
  }
  if (policy == DT_POLICY_CAST_WIDTH_DEPTH) {
    if (h->depth < 1) return fail(DT_ERR_ARG, "no layer to prune");
    if (p->width_cap < 1 || p->width_cap > h->cfg.W || p->width_cap > p->N_cols)
      return fail(DT_ERR_ARG, "width_cap must be in [1, min(W, N_cols)]");
    if (p->R < 1 || p->R > dt::kMaxFifo) return fail(DT_ERR_ARG, "R must be in [1, 16]");
    if (!out->width || !out->stop) return fail(DT_ERR_ARG, "width and stop outputs required");
  } else if (policy == DT_POLICY_CAST_VERIFY) {
    if (p->m_cap < 1 || p->m_cap > p->N_cols || p->m_cap > h->cfg.P_max - 1)
      return fail(DT_ERR_ARG, "m_cap must be in [1, min(N_cols, P_max-1)]");
    if (!out->m) return fail(DT_ERR_ARG, "m output required");
  } else if (policy == DT_POLICY_GRAFT_CHECKPOINT) {
    if (h->depth < 1) return fail(DT_ERR_ARG, "no layer to check");
    if (p->n_ckpt < 0 || p->n_ckpt > 16) return fail(DT_ERR_ARG, "n_ckpt must be in [0, 16]");
    if (!out->stop) return fail(DT_ERR_ARG, "stop output required");
  } else {
    return fail(DT_ERR_ARG, "unknown policy %d", policy);
  }
  cudaError_t e = dt::launch_cast_prune(h, policy, p, out, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_cast_prune");
  return DT_OK;
}

int dt_cast_verify_rerank(dt_handle* h, const dt_prune_params* p, const dt_prune_out* out, int32_t* selected,
                          cudaStream_t s) {
  if (!h || !p || !out || !selected) return fail(DT_ERR_ARG, "dt_cast_verify_rerank: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_cast_verify_rerank: no tree (call dt_tree_reset)");
  if (!p->S_T) return fail(DT_ERR_ARG, "cost tables missing");
  if (p->M_rows < 1 || p->N_cols < 1) return fail(DT_ERR_ARG, "table shape must be positive");
  if (!(p->L > 0.0)) return fail(DT_ERR_ARG, "L must be > 0");
  if (p->n0 < 0) return fail(DT_ERR_ARG, "n0 must be >= 0");
  if (p->m_cap < 1 || p->m_cap > p->N_cols || p->m_cap > h->cfg.P_max - 1)
    return fail(DT_ERR_ARG, "m_cap must be in [1, min(N_cols, P_max-1)]");
  if (!out->m) return fail(DT_ERR_ARG, "m output required");
  cudaError_t e = dt::launch_cast_verify_rerank(h, p, out, selected, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_cast_verify_rerank");
  return DT_OK;
}

int dt_cast_prune_select(dt_handle* h, const dt_prune_params* p, const dt_prune_out* out, int32_t* frontier_token,
                         cudaStream_t s) {
  if (!h || !p || !out) return fail(DT_ERR_ARG, "dt_cast_prune_select: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_cast_prune_select: no tree (call dt_tree_reset)");
  if (h->depth < 1) return fail(DT_ERR_ARG, "no layer to prune");
  const int rc = check_cast_width_params(h, p, out);
  if (rc != DT_OK) return rc;
  cudaError_t e = dt::launch_cast_prune_select(h, p, out, frontier_token, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_cast_prune_select");
  return DT_OK;
}

int dt_rerank(dt_handle* h, const int32_t* m, int32_t m_len, int32_t m_cap, int32_t* selected, cudaStream_t s) {
  if (!h || !selected) return fail(DT_ERR_ARG, "dt_rerank: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_rerank: no tree (call dt_tree_reset)");
  if (m_cap < 1 || m_cap > h->N - 1) return fail(DT_ERR_ARG, "m_cap must be in [1, N-1]");
  if (m && m_len != 1 && m_len != h->B) return fail(DT_ERR_ARG, "m_len must be 1 or B");
  cudaError_t e = dt::launch_rerank(h, m, m_len, m_cap, selected, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_rerank");
  return DT_OK;
}

int dt_graft_retrieve(dt_handle* h, const int32_t* M, const dt_template* tpl, int32_t R_cap, const int32_t* selected,
                      int32_t m_cap, int32_t* ret_token, int32_t* ret_parent, int32_t* ret_count,
                      int32_t* ret_anchor, cudaStream_t s) {
  if (!h || !M || !tpl || !ret_token || !ret_parent || !ret_count)
    return fail(DT_ERR_ARG, "dt_graft_retrieve: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_graft_retrieve: no tree (call dt_tree_reset)");
  if (tpl->n < 0 || tpl->n > 256) return fail(DT_ERR_ARG, "template size must be in [0, 256]");
  if (tpl->n > 0 && (!tpl->parent || !tpl->rank)) return fail(DT_ERR_ARG, "template arrays missing");
  for (int u = 0; u < tpl->n; ++u) {
    if (tpl->parent[u] < -1 || tpl->parent[u] >= u) return fail(DT_ERR_ARG, "template parent[%d] invalid", u);
    if (tpl->rank[u] < 0 || tpl->rank[u] >= 8) return fail(DT_ERR_ARG, "template rank[%d] invalid", u);
  }
  if (tpl->anchor != DT_ANCHOR_ROOT && tpl->anchor != DT_ANCHOR_TAIL)
    return fail(DT_ERR_ARG, "template anchor must be DT_ANCHOR_ROOT or DT_ANCHOR_TAIL");
  if (tpl->anchor == DT_ANCHOR_TAIL && (!selected || m_cap < 1 || m_cap > h->N - 1))
    return fail(DT_ERR_ARG, "a tail-anchored template needs selected and m_cap in [1, N-1]");
  if (R_cap < 1 || R_cap > dt::kMaxP) return fail(DT_ERR_ARG, "R_cap must be in [1, 512]");
  cudaError_t e = dt::launch_graft_retrieve(h, M, tpl, R_cap, selected, m_cap, ret_token, ret_parent, ret_count,
                                            ret_anchor, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_graft_retrieve");
  return DT_OK;
}

int dt_build_tree_meta(dt_handle* h, const int32_t* selected, int32_t m_cap, const int32_t* ret_token,
                       const int32_t* ret_parent, const int32_t* ret_count, const int32_t* ret_anchor,
                       int32_t R_cap, int32_t K_total, const int32_t* pos_offset, const dt_tree_meta* meta,
                       cudaStream_t s) {
  if (!h || !selected || !meta) return fail(DT_ERR_ARG, "dt_build_tree_meta: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_build_tree_meta: no tree (call dt_tree_reset)");
  if (!meta->tokens || !meta->parents || !meta->depth || !meta->node_id || !meta->mask ||
      !meta->position_ids || !meta->retrieve || !meta->n_leaves || !meta->n_pos)
    return fail(DT_ERR_ARG, "dt_build_tree_meta: a meta array is null");
  if (meta->P < 1 || meta->P > h->cfg.P_max) return fail(DT_ERR_ARG, "meta P must be in [1, P_max]");
  if (meta->D_path < 1 || meta->D_path > 64) return fail(DT_ERR_ARG, "D_path must be in [1, 64]");
  if (m_cap < 0 || m_cap > h->N - 1) return fail(DT_ERR_ARG, "m_cap out of range");
  const bool graft = ret_token != nullptr;
  if (graft && (!ret_parent || !ret_count || R_cap < 1)) return fail(DT_ERR_ARG, "retrieval arrays incomplete");
  if (1 + m_cap > meta->P) return fail(DT_ERR_ARG, "1 + m_cap exceeds P");
  cudaError_t e = dt::launch_build_meta(h, selected, m_cap, ret_token, ret_parent, ret_count,
                                        graft ? ret_anchor : nullptr, graft ? R_cap : 0, K_total, pos_offset, meta,
                                        s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_build_tree_meta");
  return DT_OK;
}

static int check_verify_args(const dt_handle* h, const char* who, const dt_tree_meta* meta, const void* logits,
                             int64_t ld, int32_t mode) {
  if (!meta || !logits) return fail(DT_ERR_ARG, "%s: null argument", who);
  if (h->B < 1) return fail(DT_ERR_ARG, "%s: no tree (call dt_tree_reset)", who);
  const int32_t base_mode = mode & ~DT_VERIFY_PACKED;
  if (base_mode != DT_GREEDY && base_mode != DT_SAMPLE)
    return fail(DT_ERR_ARG, "mode must be DT_GREEDY or DT_SAMPLE, optionally | DT_VERIFY_PACKED");
  if (meta->P < 1 || meta->P > h->cfg.P_max) return fail(DT_ERR_ARG, "meta P must be in [1, P_max]");
  if (meta->D_path < 1 || meta->D_path > 64) return fail(DT_ERR_ARG, "D_path must be in [1, 64]");
  if (ld < h->cfg.V) return fail(DT_ERR_ARG, "ld < V");
  const size_t esz = h->cfg.dtype == DT_BF16 ? 2 : 4;
  if (!aligned(logits, esz)) return fail(DT_ERR_ARG, "logits not aligned to its element size");
  if ((int64_t)h->B * meta->P > (int64_t)h->ws.row_counter_cap) return fail(DT_ERR_ARG, "B*P too large");
  return DT_OK;
}

int dt_verify_rows(dt_handle* h, const dt_tree_meta* meta, const void* logits, int64_t ld, int32_t mode,
                   int32_t with_top8, cudaStream_t s) {
  if (!h) return fail(DT_ERR_ARG, "dt_verify_rows: null handle");
  const int rc = check_verify_args(h, "dt_verify_rows", meta, logits, ld, mode);
  if (rc != DT_OK) return rc;
  cudaError_t e = dt::launch_verify_rows(h, meta, logits, ld, mode, with_top8 ? 1 : 0, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_verify_rows");
  return DT_OK;
}

int dt_verify_accept(dt_handle* h, const dt_tree_meta* meta, const void* logits, int64_t ld, int32_t mode,
                     uint64_t seed, uint64_t round, int32_t* accept_len, int32_t* accept_path, int32_t* bonus,
                     int32_t* top8, cudaStream_t s) {
  if (!h || !accept_len || !accept_path || !bonus) return fail(DT_ERR_ARG, "dt_verify_accept: null argument");
  const int rc = check_verify_args(h, "dt_verify_accept", meta, logits, ld, mode);
  if (rc != DT_OK) return rc;
  cudaError_t e = dt::launch_verify_accept(h, meta, logits, ld, mode, seed, round, accept_len, accept_path, bonus,
                                           top8, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_verify_accept");
  return DT_OK;
}

int dt_verify(dt_handle* h, const dt_tree_meta* meta, const void* logits, int64_t ld, int32_t mode,
              uint64_t seed, uint64_t round, int32_t* accept_len, int32_t* accept_path, int32_t* bonus,
              int32_t* top8, cudaStream_t s) {
  if (!h || !accept_len || !accept_path || !bonus) return fail(DT_ERR_ARG, "dt_verify: null argument");
  const int rc = check_verify_args(h, "dt_verify", meta, logits, ld, mode);
  if (rc != DT_OK) return rc;
  cudaError_t e = dt::launch_verify(h, meta, logits, ld, mode, seed, round, accept_len, accept_path, bonus, top8, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_verify");
  return DT_OK;
}

int dt_verify_sampled(dt_handle* h, const dt_tree_meta* meta, const void* logits, int64_t ld, int32_t mode,
                      const void* draft_rows, int64_t ld_d, uint64_t seed, uint64_t round, int32_t* accept_len,
                      int32_t* accept_path, int32_t* bonus, cudaStream_t s) {
  if (!h || !accept_len || !accept_path || !bonus || !draft_rows)
    return fail(DT_ERR_ARG, "dt_verify_sampled: null argument");
  if (mode != 0 && mode != DT_VERIFY_PACKED) return fail(DT_ERR_ARG, "mode must be 0 or DT_VERIFY_PACKED");
  const int rc = check_verify_args(h, "dt_verify_sampled", meta, logits, ld, DT_SAMPLE | mode);
  if (rc != DT_OK) return rc;
  if (ld_d < h->cfg.V) return fail(DT_ERR_ARG, "ld_d < V");
  const size_t esz = h->cfg.dtype == DT_BF16 ? 2 : 4;
  if (!aligned(draft_rows, esz)) return fail(DT_ERR_ARG, "draft rows not aligned to their element size");
  cudaError_t e = dt::launch_verify_sampled(h, meta, logits, ld, mode, draft_rows, ld_d, seed, round, accept_len,
                                            accept_path, bonus, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_verify_sampled");
  return DT_OK;
}

int dt_adj_update(dt_handle* h, int32_t* M, const dt_tree_meta* meta, const int32_t* top8, cudaStream_t s) {
  if (!h || !M || !meta || !top8) return fail(DT_ERR_ARG, "dt_adj_update: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_adj_update: no tree (call dt_tree_reset)");
  if (meta->P < 1 || meta->P > h->cfg.P_max) return fail(DT_ERR_ARG, "meta P must be in [1, P_max]");
  if (!aligned(M, 16) || !aligned(top8, 16)) return fail(DT_ERR_ARG, "M and top8 must be 16-byte aligned");
  cudaError_t e = dt::launch_adj_update(h, M, meta, top8, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_adj_update");
  return DT_OK;
}

int dt_commit_kv(dt_handle* h, const void* tmp_kv, int64_t tmp_pos_stride, int64_t tmp_req_stride, int32_t P,
                 void* cache, int64_t cache_pos_stride, int64_t cache_req_stride, int32_t L_max, int64_t row_bytes,
                 int32_t* cache_len, const int32_t* accept_len, const int32_t* accept_path, int32_t D_path,
                 const int32_t* tmp_row_off, cudaStream_t s) {
  if (!h || !tmp_kv || !cache || !cache_len || !accept_len || !accept_path)
    return fail(DT_ERR_ARG, "dt_commit_kv: null argument");
  if (h->B < 1) return fail(DT_ERR_ARG, "dt_commit_kv: no tree (call dt_tree_reset)");
  if (P < 1 || L_max < 1 || D_path < 1 || D_path > 64) return fail(DT_ERR_ARG, "P, L_max >= 1 and D_path in [1, 64]");
  if (row_bytes < 16) return fail(DT_ERR_ARG, "row_bytes must be >= 16");
  if (!aligned(tmp_kv, 16) || !aligned(cache, 16) || tmp_pos_stride % 16 || tmp_req_stride % 16 ||
      cache_pos_stride % 16 || cache_req_stride % 16 || row_bytes % 16)
    return fail(DT_ERR_ARG, "dt_commit_kv: pointers, strides and row_bytes must be multiples of 16 bytes");
  if (tmp_pos_stride < row_bytes || cache_pos_stride < row_bytes ||
      (!tmp_row_off && tmp_req_stride < tmp_pos_stride * P) || cache_req_stride < cache_pos_stride * L_max)
    return fail(DT_ERR_ARG, "dt_commit_kv: strides smaller than the rows they hold");
  if (!aligned(cache_len, 4) || !aligned(accept_len, 4) || !aligned(accept_path, 4) || !aligned(tmp_row_off, 4))
    return fail(DT_ERR_ARG, "dt_commit_kv: int32 arrays must be 4-byte aligned");
  cudaError_t e = dt::launch_commit_kv(h, tmp_kv, tmp_pos_stride, tmp_req_stride, P, cache, cache_pos_stride,
                                       cache_req_stride, L_max, row_bytes, cache_len, accept_len, accept_path,
                                       D_path, tmp_row_off, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_commit_kv");
  return DT_OK;
}

static int check_batch(const dt_handle* h, const char* who, int32_t B) {
  if (!h) return fail(DT_ERR_ARG, "%s: null handle", who);
  if (B < 1 || B > h->cfg.B_max) return fail(DT_ERR_ARG, "%s: B must be in [1, B_max]", who);
  return DT_OK;
}

static bool good_page(int32_t page) { return page >= 8 && page <= 256 && (page & (page - 1)) == 0; }

static int check_pool(const char* who, const dt_block_pool* p) {
  if (!p || !p->block_table || !p->n_owned || !p->free_list || !p->free_count)
    return fail(DT_ERR_ARG, "%s: null pool argument", who);
  if (!good_page(p->page)) return fail(DT_ERR_ARG, "%s: page must be a power of two in [8, 256]", who);
  if (p->n_blocks < 1 || p->max_blocks < 1) return fail(DT_ERR_ARG, "%s: n_blocks and max_blocks must be >= 1", who);
  if (!aligned(p->block_table, 4) || !aligned(p->n_owned, 4) || !aligned(p->free_list, 4) || !aligned(p->free_count, 4))
    return fail(DT_ERR_ARG, "%s: int32 arrays must be 4-byte aligned", who);
  return DT_OK;
}

int dt_kv_reserve(dt_handle* h, int32_t B, const dt_block_pool* pool, const int32_t* seq_len, const int32_t* n_new,
                  int32_t n_extra, int64_t* slots, int64_t n_slots, int32_t S, const int32_t* slot_off,
                  cudaStream_t s) {
  int rc = check_batch(h, "dt_kv_reserve", B);
  if (rc == DT_OK) rc = check_pool("dt_kv_reserve", pool);
  if (rc != DT_OK) return rc;
  if (!seq_len || !n_new || !slots) return fail(DT_ERR_ARG, "dt_kv_reserve: null argument");
  if (S < 1 || n_extra < 0) return fail(DT_ERR_ARG, "dt_kv_reserve: S >= 1 and n_extra >= 0");
  if (n_slots < 0 || (!slot_off && n_slots < (int64_t)B * S))
    return fail(DT_ERR_ARG, "dt_kv_reserve: slots holds fewer than B * S entries");
  if (!aligned(slots, 8) || !aligned(seq_len, 4) || !aligned(n_new, 4) || !aligned(slot_off, 4))
    return fail(DT_ERR_ARG, "dt_kv_reserve: misaligned array");
  cudaError_t e = dt::launch_kv_reserve(h, B, pool, seq_len, n_new, n_extra, slots, n_slots, S, slot_off, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_kv_reserve");
  return DT_OK;
}

int dt_kv_release(dt_handle* h, int32_t B, const dt_block_pool* pool, const int32_t* keep_len, cudaStream_t s) {
  int rc = check_batch(h, "dt_kv_release", B);
  if (rc == DT_OK) rc = check_pool("dt_kv_release", pool);
  if (rc != DT_OK) return rc;
  if (!keep_len) return fail(DT_ERR_ARG, "dt_kv_release: null argument");
  if (!aligned(keep_len, 4)) return fail(DT_ERR_ARG, "dt_kv_release: misaligned array");
  cudaError_t e = dt::launch_kv_release(h, B, pool, keep_len, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_kv_release");
  return DT_OK;
}

int dt_kv_fork(dt_handle* h, int32_t B, const dt_block_pool* pool, int32_t* refs, const dt_kv_pages* kv, int32_t n,
               const int32_t* src, const int32_t* dst, const int32_t* length, int32_t* seq_len, int32_t shared_len,
               cudaStream_t s) {
  int rc = check_batch(h, "dt_kv_fork", B);
  if (rc == DT_OK) rc = check_pool("dt_kv_fork", pool);
  if (rc != DT_OK) return rc;
  if (!refs || !kv || !kv->cache || !src || !dst || !seq_len) return fail(DT_ERR_ARG, "dt_kv_fork: null argument");
  if (n < 1 || n > h->cfg.B_max) return fail(DT_ERR_ARG, "dt_kv_fork: n must be in [1, B_max]");
  if (pool->n_blocks >= 1 << 30) return fail(DT_ERR_ARG, "dt_kv_fork: n_blocks must be below 2^30");
  if (shared_len < 0 || shared_len % pool->page || shared_len / pool->page > pool->max_blocks)
    return fail(DT_ERR_ARG, "dt_kv_fork: shared_len must be a multiple of page within max_blocks");
  if (kv->planes < 1 || kv->planes > 65535) return fail(DT_ERR_ARG, "dt_kv_fork: planes must be in [1, 65535]");
  if (kv->heads < 1 || kv->head_bytes < 16 || kv->heads > (int64_t)(1 << 20) / kv->head_bytes)
    return fail(DT_ERR_ARG, "dt_kv_fork: heads >= 1, head_bytes >= 16, a plane's row at most 1 MB");
  if (!aligned(kv->cache, 16) || kv->cache_plane % 16 || kv->cache_block % 16 || kv->cache_tok % 16 || kv->cache_head % 16 ||
      kv->head_bytes % 16)
    return fail(DT_ERR_ARG, "dt_kv_fork: pointers, strides and head_bytes must be multiples of 16 bytes");
  if (!aligned(refs, 4) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(length, 4) || !aligned(seq_len, 4))
    return fail(DT_ERR_ARG, "dt_kv_fork: int32 arrays must be 4-byte aligned");
  cudaError_t e = dt::launch_kv_fork(h, B, pool, refs, kv, n, src, dst, length, seq_len, shared_len, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_kv_fork");
  return DT_OK;
}

int dt_kv_release_shared(dt_handle* h, int32_t B, const dt_block_pool* pool, int32_t* refs, const int32_t* keep_len,
                         cudaStream_t s) {
  int rc = check_batch(h, "dt_kv_release_shared", B);
  if (rc == DT_OK) rc = check_pool("dt_kv_release_shared", pool);
  if (rc != DT_OK) return rc;
  if (!refs || !keep_len) return fail(DT_ERR_ARG, "dt_kv_release_shared: null argument");
  if (pool->n_blocks >= 1 << 30) return fail(DT_ERR_ARG, "dt_kv_release_shared: n_blocks must be below 2^30");
  if (!aligned(refs, 4) || !aligned(keep_len, 4)) return fail(DT_ERR_ARG, "dt_kv_release_shared: int32 arrays must be 4-byte aligned");
  cudaError_t e = dt::launch_kv_release_shared(h, B, pool, refs, keep_len, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_kv_release_shared");
  return DT_OK;
}

int dt_commit_kv_paged(dt_handle* h, int32_t B, const dt_kv_rows* kv, int32_t P, const int32_t* row_off,
                       const int32_t* path, int32_t D_path, const int32_t* n_new, int32_t n_extra,
                       const int64_t* slots, int64_t n_slots, int32_t S, const int32_t* slot_off,
                       const int32_t* seq_len, int32_t* len_out, cudaStream_t s) {
  const int rc = check_batch(h, "dt_commit_kv_paged", B);
  if (rc != DT_OK) return rc;
  if (!kv || !kv->tmp || !kv->cache || !n_new || !slots || !seq_len || !len_out)
    return fail(DT_ERR_ARG, "dt_commit_kv_paged: null argument");
  if (P < 1 || S < 1 || n_extra < 0 || (path && D_path < 1) || kv->rows < 1)
    return fail(DT_ERR_ARG, "dt_commit_kv_paged: P, S, rows, D_path >= 1 and n_extra >= 0");
  if (kv->planes < 1 || kv->planes > 65535) return fail(DT_ERR_ARG, "dt_commit_kv_paged: planes must be in [1, 65535]");
  if (!good_page(kv->page) || kv->n_blocks < 1)
    return fail(DT_ERR_ARG, "dt_commit_kv_paged: page must be a power of two in [8, 256] and n_blocks >= 1");
  if (kv->heads < 1 || kv->head_bytes < 16 || kv->heads > (int64_t)(1 << 20) / kv->head_bytes)
    return fail(DT_ERR_ARG, "dt_commit_kv_paged: heads >= 1, head_bytes >= 16, a plane's row at most 1 MB");
  if (!aligned(kv->tmp, 16) || !aligned(kv->cache, 16) || kv->tmp_plane % 16 || kv->tmp_row % 16 || kv->tmp_head % 16 ||
      kv->cache_plane % 16 || kv->cache_block % 16 || kv->cache_tok % 16 || kv->cache_head % 16 || kv->head_bytes % 16)
    return fail(DT_ERR_ARG, "dt_commit_kv_paged: pointers, strides and head_bytes must be multiples of 16 bytes");
  if (n_slots < 0 || (!slot_off && n_slots < (int64_t)B * S))
    return fail(DT_ERR_ARG, "dt_commit_kv_paged: slots holds fewer than B * S entries");
  if (!aligned(slots, 8) || !aligned(seq_len, 4) || !aligned(len_out, 4) || !aligned(n_new, 4) || !aligned(path, 4) ||
      !aligned(row_off, 4) || !aligned(slot_off, 4) || !aligned(kv->committed, 4))
    return fail(DT_ERR_ARG, "dt_commit_kv_paged: misaligned array");
  cudaError_t e = dt::launch_commit_kv_paged(h, B, kv, P, row_off, path, D_path, n_new, n_extra, slots, n_slots, S,
                                             slot_off, seq_len, len_out, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_commit_kv_paged");
  return DT_OK;
}

static int check_heads(const dt_handle* h, const char* who, int32_t B, int32_t H_q, int32_t H_kv, int32_t D) {
  const int rc = check_batch(h, who, B);
  if (rc != DT_OK) return rc;
  if (H_kv < 1 || H_q < H_kv || H_q % H_kv || H_q / H_kv > 128 || H_q > 4096)
    return fail(DT_ERR_ARG, "%s: H_q must be a multiple of H_kv, H_q / H_kv <= 128, H_q <= 4096", who);
  if (D < 8 || D > 128 || D % 8) return fail(DT_ERR_ARG, "%s: D must be a multiple of 8 in [8, 128]", who);
  return DT_OK;
}

static int check_attn_sizes(const dt_handle* h, const char* who, int32_t B, int32_t P, int32_t H_q, int32_t H_kv,
                            int32_t D) {
  const int rc = check_batch(h, who, B);
  if (rc != DT_OK) return rc;
  if (P < 1 || P > h->cfg.P_max) return fail(DT_ERR_ARG, "%s: P must be in [1, P_max]", who);
  return check_heads(h, who, B, H_q, H_kv, D);
}

int dt_tree_attention_workspace(dt_handle* h, int32_t B, int32_t P, int32_t H_q, int32_t H_kv, int32_t D,
                                int32_t shared, int64_t* bytes) {
  const int rc = check_attn_sizes(h, "dt_tree_attention_workspace", B, P, H_q, H_kv, D);
  if (rc != DT_OK) return rc;
  if (!bytes) return fail(DT_ERR_ARG, "dt_tree_attention_workspace: null argument");
  *bytes = dt::attn_workspace_bytes(h, B, P, H_q, H_kv, D, shared ? 1 : 0);
  return DT_OK;
}

int dt_tree_attention(dt_handle* h, const dt_attn_args* a, cudaStream_t s) {
  if (!h || !a) return fail(DT_ERR_ARG, "dt_tree_attention: null argument");
  const int rc = check_attn_sizes(h, "dt_tree_attention", a->B, a->P, a->H_q, a->H_kv, a->D);
  if (rc != DT_OK) return rc;
  if (!a->q || !a->out || !a->k_new || !a->v_new || !a->k_pages || !a->v_pages || !a->block_table || !a->seq_len ||
      !a->n_pos || !a->workspace)
    return fail(DT_ERR_ARG, "dt_tree_attention: null argument");
  if (a->dtype != DT_BF16 && a->dtype != DT_F16) return fail(DT_ERR_ARG, "dt_tree_attention: dtype must be DT_BF16 or DT_F16");
  if (!good_page(a->page) || a->n_blocks < 1 || a->max_blocks < 1)
    return fail(DT_ERR_ARG, "dt_tree_attention: page must be a power of two in [8, 256], n_blocks and max_blocks >= 1");
  if (a->shared_len < 0 || a->shared_len % a->page || a->shared_len / a->page > a->max_blocks)
    return fail(DT_ERR_ARG, "dt_tree_attention: shared_len must be a multiple of page within max_blocks");
  if (!(a->scale >= 1e-30f) || a->scale > 1e30f) return fail(DT_ERR_ARG, "dt_tree_attention: scale must be in [1e-30, 1e30]");
  if (a->rows < 1 || a->rows > 0x7FFFFFFFll || (!a->row_off && a->rows < (int64_t)a->B * a->P))
    return fail(DT_ERR_ARG, "dt_tree_attention: rows must hold B * P rows and fit 31 bits");
  const void* p16[] = {a->q, a->out, a->k_new, a->v_new, a->k_pages, a->v_pages};
  for (const void* p : p16)
    if (!aligned(p, 16)) return fail(DT_ERR_ARG, "dt_tree_attention: tensors must be 16-byte aligned");
  const int64_t st[] = {a->q_row,  a->q_head,  a->o_row, a->o_head, a->kn_row,  a->kn_head, a->vn_row,
                        a->vn_head, a->k_block, a->k_tok, a->k_head, a->v_block, a->v_tok,   a->v_head};
  for (int64_t x : st)
    if (x < a->D || x % 8 || x > (int64_t)1 << 38)
      return fail(DT_ERR_ARG, "dt_tree_attention: strides must be multiples of 8 elements, at least D");
  if (!aligned(a->block_table, 4) || !aligned(a->seq_len, 4) || !aligned(a->n_pos, 4) || !aligned(a->row_off, 4))
    return fail(DT_ERR_ARG, "dt_tree_attention: int32 arrays must be 4-byte aligned");
  if (!dt::attn_line_fits(a))
    return fail(DT_ERR_ARG, "dt_tree_attention: B * H_kv * rows * max_blocks * page too large");
  if (!aligned(a->workspace, 256) ||
      a->workspace_bytes < dt::attn_workspace_bytes(h, a->B, a->P, a->H_q, a->H_kv, a->D, a->shared_len > 0))
    return fail(DT_ERR_ARG, "dt_tree_attention: workspace too small (dt_tree_attention_workspace) or not 256-byte aligned");
  cudaError_t e = dt::launch_attention(h, a, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_tree_attention");
  return DT_OK;
}

int dt_prompt_attention_workspace(dt_handle* h, int32_t B, int32_t H_q, int32_t H_kv, int32_t D, int64_t* bytes) {
  const int rc = check_heads(h, "dt_prompt_attention_workspace", B, H_q, H_kv, D);
  if (rc != DT_OK) return rc;
  if (!bytes) return fail(DT_ERR_ARG, "dt_prompt_attention_workspace: null argument");
  *bytes = dt::prompt_workspace_bytes(h, D);
  return DT_OK;
}

int dt_prompt_attention(dt_handle* h, const dt_prompt_args* a, cudaStream_t s) {
  if (!h || !a) return fail(DT_ERR_ARG, "dt_prompt_attention: null argument");
  const int rc = check_heads(h, "dt_prompt_attention", a->B, a->H_q, a->H_kv, a->D);
  if (rc != DT_OK) return rc;
  if (!a->q || !a->out || !a->k_new || !a->v_new || !a->row_off || !a->workspace)
    return fail(DT_ERR_ARG, "dt_prompt_attention: null argument");
  const bool cached = a->seq_len || a->block_table || a->k_pages || a->v_pages;
  if (cached && (!a->seq_len || !a->block_table || !a->k_pages || !a->v_pages))
    return fail(DT_ERR_ARG, "dt_prompt_attention: seq_len, block_table, k_pages and v_pages come together");
  if (a->dtype != DT_BF16 && a->dtype != DT_F16) return fail(DT_ERR_ARG, "dt_prompt_attention: dtype must be DT_BF16 or DT_F16");
  if (cached && (!good_page(a->page) || a->n_blocks < 1 || a->max_blocks < 1))
    return fail(DT_ERR_ARG, "dt_prompt_attention: page must be a power of two in [8, 256], n_blocks and max_blocks >= 1");
  if (!(a->scale >= 1e-30f) || a->scale > 1e30f) return fail(DT_ERR_ARG, "dt_prompt_attention: scale must be in [1e-30, 1e30]");
  if (a->rows < 1 || a->rows > 0x7FFFFF00ll) return fail(DT_ERR_ARG, "dt_prompt_attention: rows must be in [1, 2^31 - 256]");
  const void* p16[] = {a->q, a->out, a->k_new, a->v_new, a->k_pages, a->v_pages};
  for (const void* p : p16)
    if (!aligned(p, 16)) return fail(DT_ERR_ARG, "dt_prompt_attention: tensors must be 16-byte aligned");
  const int64_t st[] = {a->q_row,   a->q_head,  a->o_row, a->o_head, a->kn_row,  a->kn_head, a->vn_row,
                        a->vn_head, a->k_block, a->k_tok, a->k_head, a->v_block, a->v_tok,   a->v_head};
  for (int k = 0; k < (cached ? 14 : 8); ++k)
    if (st[k] < a->D || st[k] % 8 || st[k] > (int64_t)1 << 38)
      return fail(DT_ERR_ARG, "dt_prompt_attention: strides must be multiples of 8 elements, at least D");
  if (!aligned(a->block_table, 4) || !aligned(a->seq_len, 4) || !aligned(a->row_off, 4))
    return fail(DT_ERR_ARG, "dt_prompt_attention: int32 arrays must be 4-byte aligned");
  if (!dt::prompt_line_fits(h, a)) return fail(DT_ERR_ARG, "dt_prompt_attention: H_kv * rows * (max_blocks * page + rows) too large");
  if (!aligned(a->workspace, 256) || a->workspace_bytes < dt::prompt_workspace_bytes(h, a->D))
    return fail(DT_ERR_ARG, "dt_prompt_attention: workspace too small (dt_prompt_attention_workspace) or not 256-byte aligned");
  cudaError_t e = dt::launch_prompt(h, a, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_prompt_attention");
  return DT_OK;
}

int dt_count_tokens(dt_handle* h, int32_t B, int32_t* counts, const int32_t* tokens, int64_t n_tokens, int32_t P,
                    const int32_t* row_off, const int32_t* path, int32_t D_path, const int32_t* n_new, int32_t n_extra, int32_t prompt,
                    cudaStream_t s) {
  const int rc = check_batch(h, "dt_count_tokens", B);
  if (rc != DT_OK) return rc;
  if (!counts || !tokens || !n_new) return fail(DT_ERR_ARG, "dt_count_tokens: null argument");
  if (P < 1 || n_extra < 0 || (path && D_path < 1)) return fail(DT_ERR_ARG, "dt_count_tokens: P, D_path >= 1 and n_extra >= 0");
  if (n_tokens < 1 || (!row_off && n_tokens < (int64_t)B * P))
    return fail(DT_ERR_ARG, "dt_count_tokens: tokens holds fewer than B * P entries");
  if (!aligned(counts, 4) || !aligned(tokens, 4) || !aligned(n_new, 4) || !aligned(path, 4) || !aligned(row_off, 4))
    return fail(DT_ERR_ARG, "dt_count_tokens: int32 arrays must be 4-byte aligned");
  cudaError_t e = dt::launch_count_tokens(h, B, counts, tokens, n_tokens, P, row_off, path, D_path, n_new, n_extra,
                                          prompt ? 1 : 0, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_count_tokens");
  return DT_OK;
}

int dt_logits_process(dt_handle* h, int32_t B, const void* logits, int64_t ld, void* out, int64_t ld_out,
                      const dt_logits_params* p, cudaStream_t s) {
  const int rc = check_batch(h, "dt_logits_process", B);
  if (rc != DT_OK) return rc;
  if (!logits || !out || !p || !p->n_pos) return fail(DT_ERR_ARG, "dt_logits_process: null argument");
  if (p->P < 1 || p->P > h->cfg.P_max) return fail(DT_ERR_ARG, "dt_logits_process: P must be in [1, P_max]");
  if (ld < h->cfg.V || ld_out < h->cfg.V) return fail(DT_ERR_ARG, "dt_logits_process: ld < V");
  if (p->rows < 1 || (!p->row_off && p->rows < (int64_t)B * p->P))
    return fail(DT_ERR_ARG, "dt_logits_process: rows must hold B * P rows");
  if (p->n_bias < 0 || p->n_bias > 4096 || (p->n_bias > 0 && p->bias_ids && !p->bias_vals))
    return fail(DT_ERR_ARG, "dt_logits_process: n_bias must be in [0, 4096], with ids and values");
  if (p->allow && p->allow_ld < (h->cfg.V + 31) / 32) return fail(DT_ERR_ARG, "dt_logits_process: allow_ld < ceil(V / 32)");
  const size_t esz = h->cfg.dtype == DT_BF16 ? 2 : 4;
  if (!aligned(logits, esz) || !aligned(out, esz)) return fail(DT_ERR_ARG, "dt_logits_process: rows not aligned to their element size");
  if (logits == out && ld != ld_out) return fail(DT_ERR_ARG, "dt_logits_process: in place needs the same ld");
  if (!aligned(p->n_pos, 4) || !aligned(p->row_off, 4) || !aligned(p->tokens, 4) || !aligned(p->counts, 4) ||
      !aligned(p->repetition, 4) || !aligned(p->frequency, 4) || !aligned(p->presence, 4) || !aligned(p->bias_ids, 4) ||
      !aligned(p->bias_vals, 4) || !aligned(p->allow, 4))
    return fail(DT_ERR_ARG, "dt_logits_process: arrays must be 4-byte aligned");
  cudaError_t e = dt::launch_logits(h, B, logits, ld, out, ld_out, p, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_logits_process");
  return DT_OK;
}

static constexpr int32_t kLogprobV = 0x7FFF0000;  // places of a row's last piece are counted in 32 bits

int dt_token_logprobs_workspace(dt_handle* h, int64_t entries, int32_t K, int64_t* bytes) {
  if (!h || !bytes) return fail(DT_ERR_ARG, "dt_token_logprobs_workspace: null argument");
  if (K < 0 || K > dt::kMaxK || K > h->cfg.V) return fail(DT_ERR_ARG, "dt_token_logprobs_workspace: K must be in [0, min(32, V)]");
  if (entries < 1 || entries > 0x7FFFFFFF) return fail(DT_ERR_ARG, "dt_token_logprobs_workspace: entries must be in [1, 2^31)");
  if (h->cfg.V > kLogprobV) return fail(DT_ERR_ARG, "dt_token_logprobs_workspace: V must be at most 2^31 - 2^16");
  *bytes = dt::logprob_workspace_bytes(h, entries, K);
  return DT_OK;
}

int dt_token_logprobs(dt_handle* h, const void* logits, int64_t ld, const dt_logprob_args* a, cudaStream_t s) {
  if (!h || !a) return fail(DT_ERR_ARG, "dt_token_logprobs: null argument");
  const int rc = check_batch(h, "dt_token_logprobs", a->B);
  if (rc != DT_OK) return rc;
  if (!logits || !a->n_new || !a->workspace) return fail(DT_ERR_ARG, "dt_token_logprobs: null argument");
  if (ld < h->cfg.V) return fail(DT_ERR_ARG, "dt_token_logprobs: ld < V");
  if (h->cfg.V > kLogprobV) return fail(DT_ERR_ARG, "dt_token_logprobs: V must be at most 2^31 - 2^16");
  if (a->P < 1 || (a->path && a->D_path < 1) || a->n_extra < 0 || (a->shift != 0 && a->shift != 1))
    return fail(DT_ERR_ARG, "dt_token_logprobs: P, D_path >= 1, n_extra >= 0, shift 0 or 1");
  if (a->rows < 1 || a->rows > 0x7FFFFFFF || (!a->row_off && a->rows < (int64_t)a->B * a->P))
    return fail(DT_ERR_ARG, "dt_token_logprobs: rows must hold B * P rows and fit 31 bits");
  const int64_t entries = a->path ? (int64_t)a->B * a->D_path : a->row_off ? a->rows : (int64_t)a->B * a->P;
  if (a->n_out < entries) return fail(DT_ERR_ARG, "dt_token_logprobs: outputs hold fewer entries than the call has");
  if (a->tokens && a->n_tokens < (a->row_off && !a->path ? 1 : (int64_t)a->B * a->P))
    return fail(DT_ERR_ARG, "dt_token_logprobs: tokens holds fewer than B * P entries");
  if ((a->logp || a->rank) && !a->tokens && !a->last) return fail(DT_ERR_ARG, "dt_token_logprobs: logp and rank need tokens or last");
  if (a->K < 0 || a->K > dt::kMaxK || a->K > h->cfg.V || (a->K > 0 && (!a->top_ids || !a->top_logp)))
    return fail(DT_ERR_ARG, "dt_token_logprobs: K must be in [0, min(32, V)], with top_ids and top_logp");
  if (!aligned(logits, h->cfg.dtype == DT_BF16 ? 2 : 4)) return fail(DT_ERR_ARG, "dt_token_logprobs: logits not aligned to their element size");
  if (!aligned(a->row_off, 4) || !aligned(a->path, 4) || !aligned(a->n_new, 4) || !aligned(a->tokens, 4) || !aligned(a->last, 4) ||
      !aligned(a->logp, 4) || !aligned(a->entropy, 4) || !aligned(a->rank, 4) || !aligned(a->top_ids, 4) || !aligned(a->top_logp, 4))
    return fail(DT_ERR_ARG, "dt_token_logprobs: arrays must be 4-byte aligned");
  if (!aligned(a->workspace, 256) || a->workspace_bytes < dt::logprob_workspace_bytes(h, entries, a->K))
    return fail(DT_ERR_ARG, "dt_token_logprobs: workspace too small (dt_token_logprobs_workspace) or not 256-byte aligned");
  if (dt::logprob_pieces(h, entries) > 0x7FFFFFFF) return fail(DT_ERR_ARG, "dt_token_logprobs: entries * V too large");
  dt_logprob_args b = *a;
  b.n_out = entries;
  cudaError_t e = dt::launch_logprobs(h, logits, ld, &b, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_token_logprobs");
  return DT_OK;
}

int dt_row_topk_static(const void* logits, int64_t ld, int32_t rows, int32_t V, int32_t K, int32_t dtype,
                       float* logp, int32_t* ids, int32_t* status, cudaStream_t s) {
  if (!logits || !logp || !ids) return fail(DT_ERR_ARG, "dt_row_topk_static: null argument");
  if (rows < 1 || rows > dt::kStaticRows)
    return fail(DT_ERR_ARG, "rows=%d outside [1, %d] (size of the static scratch)", rows, dt::kStaticRows);
  if (V < 2) return fail(DT_ERR_ARG, "V must be >= 2");
  if (K < 1 || K > dt::kMaxK || K > V) return fail(DT_ERR_ARG, "K must be in [1, min(32, V)]");
  if (dtype != DT_BF16 && dtype != DT_F32) return fail(DT_ERR_ARG, "dtype must be DT_BF16 or DT_F32");
  if (ld < V) return fail(DT_ERR_ARG, "ld=%lld < V", (long long)ld);
  const size_t esz = dtype == DT_BF16 ? 2 : 4;
  if (!aligned(logits, esz)) return fail(DT_ERR_ARG, "logits not aligned to its element size");
  if (!aligned(logp, 4) || !aligned(ids, 4) || !aligned(status, 4))
    return fail(DT_ERR_ARG, "logp, ids and status must be 4-byte aligned");
  cudaError_t e = dt::launch_row_topk_static(logits, ld, rows, V, K, dtype, logp, ids, status, s);
  if (e != cudaSuccess) return cuda_fail(e, "dt_row_topk_static");
  return DT_OK;
}

}  // extern "C"
