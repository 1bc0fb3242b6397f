// The C entry points of the attention inside packed documents: argument checks, workspace
// layout and the choice of kernel (fp32: the CUDA cores; bf16: the tensor cores).
#include <float.h>
#include <math.h>

#include "checks.h"
#include "internal.h"

namespace wan {
namespace {

float score_scale(const wan_dit_config* cfg, const wan_documents* d) {
  return d->scale != 0.f ? d->scale : static_cast<float>(1.0 / sqrt(static_cast<double>(cfg->head_dim)));
}

// The factors that the kernels work with are numbers: a score in log2 units and, with a cap, the
// argument of its tanh (an infinite factor would make NaN of a score of 0, a subnormal one
// loses its digits).
int check_factors(float scale, float cap) {
  const float log2e = 1.4426950408889634f, in = cap > 0.f ? fabsf(scale / cap) : 1.f;
  WAN_REQUIRE(isfinite(scale * log2e) && isfinite(cap * log2e), WAN_ERR_SHAPE);
  WAN_REQUIRE(isfinite(in) && in >= FLT_MIN, WAN_ERR_SHAPE);
  return WAN_OK;
}

int check_docs(const wan_dit_config* cfg, const wan_documents* d, int q_rows, int k_rows, int kv_heads) {
  WAN_TRY(check_cfg(cfg, true));
  WAN_REQUIRE(d, WAN_ERR_NULL);
  WAN_REQUIRE(q_rows >= 0 && k_rows >= 0 && d->n_docs >= 0, WAN_ERR_SHAPE);
  WAN_REQUIRE(kv_heads >= 1 && cfg->heads % kv_heads == 0 && cfg->heads <= 65535, WAN_ERR_SHAPE);
  WAN_REQUIRE(d->causal_block >= 0, WAN_ERR_SHAPE);
  WAN_REQUIRE(isfinite(d->scale) && isfinite(d->cap) && d->cap >= 0.f, WAN_ERR_SHAPE);
  WAN_TRY(check_factors(score_scale(cfg, d), d->cap));
  WAN_TRY(check_ints(d->cu_q, d->n_docs + 1));
  WAN_TRY(check_ints(d->cu_k, d->n_docs + 1));
  WAN_TRY(check_opt_ptr(d->prefix));
  WAN_TRY(check_opt_ptr(d->slopes));
  return WAN_OK;
}

PackedAttn make_packed(const wan_dit_config* cfg, const wan_documents* d, int q_rows, int k_rows, int kv_heads,
                       const wan_rows* q, const wan_rows* k, const wan_rows* v, const wan_rows* o) {
  PackedAttn p{};
  p.cu_q = d->cu_q, p.cu_k = d->cu_k, p.prefix = d->prefix, p.slopes = d->slopes;
  p.n_docs = d->n_docs, p.q_rows = q_rows, p.k_rows = k_rows;
  p.H = cfg->heads, p.Hk = kv_heads, p.d = cfg->head_dim, p.causal_block = d->causal_block;
  p.scale = score_scale(cfg, d);
  p.cap = d->cap;
  p.q = q->ptr, p.k = k->ptr, p.v = v->ptr, p.o = o->ptr;
  p.q_stride = q->row_stride, p.k_stride = k->row_stride, p.v_stride = v->row_stride, p.o_stride = o->row_stride;
  return p;
}

}  // namespace
}  // namespace wan

using namespace wan;

extern "C" {

size_t wan_attention_packed_workspace_bytes(const wan_dit_config* cfg, int q_rows, int k_rows, int n_docs,
                                            int kv_heads, int backward) {
  if (check_cfg(cfg, true) != WAN_OK || q_rows < 0 || k_rows < 0 || n_docs < 0 || kv_heads < 1 ||
      cfg->heads % kv_heads != 0)
    return 0;
  size_t bytes = 0;
  if (cfg->dtype == WAN_BF16) {
    PackedAttn a{};
    a.H = cfg->heads, a.Hk = kv_heads, a.q_rows = q_rows;
    bytes = attn_packed_tc_workspace(a);
  }
  const size_t grad = (static_cast<size_t>(cfg->heads) * q_rows * 4 + 255) / 256 * 256;
  return backward && grad > bytes ? grad : bytes;
}

int wan_attention_packed_fwd(const wan_dit_config* cfg, const wan_documents* docs, int q_rows, int k_rows,
                             int kv_heads, const wan_rows* q, const wan_rows* k, const wan_rows* v, const wan_rows* o,
                             float* lse, void* workspace, size_t ws_bytes, void* stream) {
  WAN_TRY(check_docs(cfg, docs, q_rows, k_rows, kv_heads));
  const int64_t wq = static_cast<int64_t>(cfg->heads) * cfg->head_dim, wk = static_cast<int64_t>(kv_heads) * cfg->head_dim;
  for (const wan_rows* t : {q, o}) WAN_TRY(check_view(t, q_rows, wq, cfg->dtype, true));
  for (const wan_rows* t : {k, v}) WAN_TRY(check_view(t, k_rows, wk, cfg->dtype, true));
  WAN_TRY(check_opt_ptr(lse));
  WAN_TRY(check_opt_ptr(workspace));
  if (q_rows == 0 || docs->n_docs == 0) return WAN_OK;
  PackedAttn p = make_packed(cfg, docs, q_rows, k_rows, kv_heads, q, k, v, o);
  p.lse = lse;
  if (cfg->dtype == WAN_BF16) return launch_attn_packed_tc(p, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
  return launch_attn_packed_simt(p, static_cast<cudaStream_t>(stream));
}

int wan_attention_packed_bwd(const wan_dit_config* cfg, const wan_documents* docs, int q_rows, int k_rows,
                             int kv_heads, const wan_rows* q, const wan_rows* k, const wan_rows* v, const wan_rows* o,
                             const float* lse, const wan_rows* d_o, const wan_rows* dq, const wan_rows* dk,
                             const wan_rows* dv, void* workspace, size_t ws_bytes, void* stream) {
  WAN_TRY(check_docs(cfg, docs, q_rows, k_rows, kv_heads));
  const int64_t wq = static_cast<int64_t>(cfg->heads) * cfg->head_dim, wk = static_cast<int64_t>(kv_heads) * cfg->head_dim;
  for (const wan_rows* t : {q, o, d_o, dq}) WAN_TRY(check_view(t, q_rows, wq, cfg->dtype, true));
  for (const wan_rows* t : {k, v, dk, dv}) WAN_TRY(check_view(t, k_rows, wk, cfg->dtype, true));
  WAN_TRY(check_array(lse, q_rows));
  if ((q_rows == 0 && k_rows == 0) || docs->n_docs == 0) return WAN_OK;
  const size_t need = wan_attention_packed_workspace_bytes(cfg, q_rows, k_rows, docs->n_docs, kv_heads, 1);
  if (need > 0) WAN_TRY(check_ptr(workspace));
  WAN_REQUIRE(ws_bytes >= need, WAN_ERR_WORKSPACE);
  PackedAttn p = make_packed(cfg, docs, q_rows, k_rows, kv_heads, q, k, v, o);
  p.lse = const_cast<float*>(lse);
  p.d_o = d_o->ptr, p.do_stride = d_o->row_stride;
  p.dq = dq->ptr, p.dk = dk->ptr, p.dv = dv->ptr;
  p.dq_stride = dq->row_stride, p.dk_stride = dk->row_stride, p.dv_stride = dv->row_stride;
  p.delta = static_cast<float*>(workspace);
  return launch_attn_packed_bwd(p, cfg->dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
