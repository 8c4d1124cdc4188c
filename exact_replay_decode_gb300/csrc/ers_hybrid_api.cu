// C ABI of the serving operators of gated-delta-rule and attention layers (declared in include/ers.h): host-side
// validation and dispatch.  A call that fails validation launches nothing.
#include <math.h>
#include <string.h>

#include "api_checks.h"
#include "ers.h"
#include "ers_internal.h"

using ers::check_ptr;

namespace {

ers_status finish(cudaError_t e) { return e == cudaSuccess ? ERS_OK : ERS_ECUDA; }

// ---- gated delta rule ------------------------------------------------------------------------------
ers_status check_delta(const ers_linattn_dims* d, int32_t nseq) {
  if (d == nullptr) return ERS_EINVAL;
  if (d->io_dtype != ERS_DTYPE_F32 && d->io_dtype != ERS_DTYPE_BF16) return ERS_EDTYPE;
  if (d->nheads <= 0 || d->ngroups <= 0 || d->nheads % d->ngroups != 0) return ERS_ESHAPE;
  if (d->nheads > 65535 || !ers::linattn_supported(d->dk, d->dv)) return ERS_ESHAPE;
  if (nseq < 0 || (int64_t)nseq * d->nheads > (0x7fffffff >> 3) || !isfinite(d->scale)) return ERS_EINVAL;
  return ERS_OK;
}

ers_status check_state_cache(const ers_linattn_cache* c, int32_t nseq, const int32_t* slot, const int32_t* read_page) {
  if (c == nullptr || c->nslots < 0 || c->npages < 0) return ERS_EINVAL;
  if (slot == nullptr && nseq > c->nslots) return ERS_EINVAL;
  ERS_TRY(check_ptr(c->state, true));
  ERS_TRY(check_ptr(c->table, true));
  ERS_TRY(check_ptr(slot, false));
  return check_ptr(read_page, false);
}

ers_status check_tokens(const ers::DeltaArgs& a, bool tokens) {
  for (const void* p : {a.q, a.k, a.v, (const void*)a.g, (const void*)a.beta, (const void*)a.o}) ERS_TRY(check_ptr(p, tokens));
  return check_ptr(a.status, false);
}

ers::DeltaArgs delta_args(const ers_linattn_dims* d, int32_t nseq, int64_t ntokens, int32_t max_seqlen) {
  ers::DeltaArgs a;
  memset(&a, 0, sizeof(a));
  a.H = d->nheads;
  a.G = d->ngroups;
  a.dk = d->dk;
  a.dv = d->dv;
  a.io = d->io_dtype;
  a.scale = d->scale;
  a.nseq = nseq;
  a.ntokens = ntokens;
  a.max_len = max_seqlen < ntokens ? max_seqlen : (int32_t)ntokens;
  a.len1 = 0x7fffffff;
  return a;
}

void set_tokens(ers::DeltaArgs* a, const void* q, const void* k, const void* v, const float* g, const float* beta, void* o,
                int32_t* st) {
  a->q = q;
  a->k = k;
  a->v = v;
  a->g = g;
  a->beta = beta;
  a->o = o;
  a->status = st;
}

void set_cache(ers::DeltaArgs* a, const ers_linattn_cache* c, const int32_t* slot, const int32_t* read_page) {
  a->pool = c->state;
  a->table = c->table;
  a->nslots = c->nslots;
  a->npages = c->npages;
  a->slot = slot;
  a->read_page = read_page;
}

// (a launch has a CTA for every head of every 64 tokens)
ers_status check_lengths(const ers_linattn_dims* d, int32_t nseq, int64_t ntokens, int32_t max_seqlen) {
  if (ntokens < 0 || ntokens > 0x7fffffff || max_seqlen < 0) return ERS_EINVAL;
  return (ntokens / 64 + nseq) * d->nheads > 0x7fffffff ? ERS_EINVAL : ERS_OK;
}

ers_status set_workspace(ers::DeltaArgs* a, void* workspace, size_t bytes) {
  const size_t need = ers::gdn_fwd_workspace(*a);
  if (need > 0 && (workspace == nullptr || bytes < need)) return ERS_EWORKSPACE;
  ERS_TRY(check_ptr(workspace, false));
  a->ws = workspace;
  return ERS_OK;
}

// ---- attention ---------------------------------------------------------------------------------------
ers_status check_attn(const ers_attn_dims* d, const ers_attn_cache* c, int32_t nseq, const int32_t* slot) {
  if (d == nullptr || c == nullptr) return ERS_EINVAL;
  if (d->io_dtype != ERS_DTYPE_F32 && d->io_dtype != ERS_DTYPE_BF16) return ERS_EDTYPE;
  if (d->nheads <= 0 || d->nheads > 8192 || d->kv_heads <= 0 || d->nheads % d->kv_heads != 0) return ERS_ESHAPE;
  if (d->head_dim != 64 && d->head_dim != 128) return ERS_ESHAPE;
  if (nseq < 0 || !isfinite(d->scale)) return ERS_EINVAL;
  if (c->nslots < 0 || c->npages < 0 || c->slot_pages < 1 || c->page_tokens < 1) return ERS_EINVAL;
  if ((int64_t)c->slot_pages * c->page_tokens > 0x7fffff00) return ERS_EINVAL;
  if (slot == nullptr && nseq > c->nslots) return ERS_EINVAL;
  for (const void* p : {(const void*)c->k, (const void*)c->v, (const void*)c->table, (const void*)c->refs, (const void*)c->pos})
    ERS_TRY(check_ptr(p, true));
  return check_ptr(slot, false);
}

ers::AttnArgs attn_args(const ers_attn_dims* d, const ers_attn_cache* c, int32_t nseq, const int32_t* slot, int32_t T,
                        const void* k, const void* v, int32_t* st) {
  ers::AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.H = d->nheads;
  a.KV = d->kv_heads;
  a.D = d->head_dim;
  a.io = d->io_dtype;
  a.scale = d->scale;
  a.nseq = nseq;
  a.T = T;
  if (c != nullptr) {
    a.k_pages = c->k;
    a.v_pages = c->v;
    a.table = c->table;
    a.refs = c->refs;
    a.pos = c->pos;
    a.nslots = c->nslots;
    a.slot_pages = c->slot_pages;
    a.npages = c->npages;
    a.page_tokens = c->page_tokens;
    // division by multiplication (Granlund and Montgomery, 1994): 2^shift >= page_tokens, magic = 2^32 (2^shift / page_tokens - 1) + 1
    while ((1ll << a.page_shift) < a.page_tokens) ++a.page_shift;
    a.page_magic = (uint32_t)((((1ull << a.page_shift) - (uint64_t)a.page_tokens) << 32) / (uint64_t)a.page_tokens + 1);
  }
  a.slot = slot;
  a.k = k;
  a.v = v;
  a.status = st;
  return a;
}

bool drafts_ok(const ers_attn_dims* d, int32_t nseq, int32_t T) {
  return T >= 1 && T <= ers::kMaxDrafts && (int64_t)nseq * T * d->nheads <= (0x7fffffff >> 3);
}

}  // namespace

extern "C" {

size_t ers_gdn_fwd_workspace_size(const ers_linattn_dims* dims, int32_t nseq, int64_t ntokens, int32_t max_seqlen) {
  if (check_delta(dims, nseq) != ERS_OK || check_lengths(dims, nseq, ntokens, max_seqlen) != ERS_OK || nseq == 0) return 0;
  return ers::gdn_fwd_workspace(delta_args(dims, nseq, ntokens, max_seqlen));
}

ers_status ers_gdn_fwd(const ers_linattn_dims* dims, int32_t nseq, int64_t ntokens, int32_t max_seqlen,
                       const int32_t* cu_seqlens, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const float* init_state, void* o, float* final_state, void* workspace,
                       size_t workspace_bytes, ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_delta(dims, nseq));
  ERS_TRY(check_lengths(dims, nseq, ntokens, max_seqlen));
  if (nseq == 0) return ERS_OK;
  ers::DeltaArgs a = delta_args(dims, nseq, ntokens, max_seqlen);
  set_tokens(&a, q, k, v, g, beta, o, dev_status);
  ERS_TRY(check_tokens(a, ntokens > 0));
  ERS_TRY(check_ptr(cu_seqlens, true));
  ERS_TRY(check_ptr(init_state, false));
  ERS_TRY(check_ptr(final_state, true));
  ERS_TRY(set_workspace(&a, workspace, workspace_bytes));
  a.cu = cu_seqlens;
  a.init = init_state;
  a.final_state = final_state;
  return finish(ers::gdn_fwd(a, (cudaStream_t)stream));
}

ers_status ers_gdn_prefill(const ers_linattn_dims* dims, const ers_linattn_cache* cache, int32_t nseq, int64_t ntokens,
                           int32_t max_seqlen, const int32_t* cu_seqlens, const int32_t* slot, const int32_t* read_page,
                           const void* q, const void* k, const void* v, const float* g, const float* beta, void* o,
                           void* workspace, size_t workspace_bytes, ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_delta(dims, nseq));
  ERS_TRY(check_lengths(dims, nseq, ntokens, max_seqlen));
  ERS_TRY(check_state_cache(cache, nseq, slot, read_page));
  if (nseq == 0) return ERS_OK;
  ers::DeltaArgs a = delta_args(dims, nseq, ntokens, max_seqlen);
  set_tokens(&a, q, k, v, g, beta, o, dev_status);
  ERS_TRY(check_tokens(a, ntokens > 0));
  ERS_TRY(check_ptr(cu_seqlens, true));
  ERS_TRY(set_workspace(&a, workspace, workspace_bytes));
  a.cu = cu_seqlens;
  set_cache(&a, cache, slot, read_page);
  return finish(ers::gdn_fwd(a, (cudaStream_t)stream));
}

ers_status ers_gdn_decode(const ers_linattn_dims* dims, const ers_linattn_cache* cache, int32_t nseq, const int32_t* slot,
                          const int32_t* read_page, const void* q, const void* k, const void* v, const float* g,
                          const float* beta, void* o, ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_delta(dims, nseq));
  ERS_TRY(check_state_cache(cache, nseq, slot, read_page));
  if (nseq == 0) return ERS_OK;
  ers::DeltaArgs a = delta_args(dims, nseq, nseq, 1);
  set_tokens(&a, q, k, v, g, beta, o, dev_status);
  ERS_TRY(check_tokens(a, true));
  set_cache(&a, cache, slot, read_page);
  return finish(ers::gdn_decode(a, (cudaStream_t)stream));
}

size_t ers_attn_verify_workspace_size(const ers_attn_dims* dims, int32_t nseq, int32_t T, int32_t max_len) {
  if (dims == nullptr || dims->nheads <= 0 || dims->kv_heads <= 0 || dims->nheads % dims->kv_heads != 0 || nseq < 1 ||
      max_len < 0 || !drafts_ok(dims, nseq, T))
    return 0;
  ers::AttnArgs a = attn_args(dims, nullptr, nseq, nullptr, T, nullptr, nullptr, nullptr);
  ers::attn_plan(&a, max_len);
  return ers::attn_workspace(a);
}

ers_status ers_attn_verify(const ers_attn_dims* dims, const ers_attn_cache* cache, int32_t nseq, const int32_t* slot,
                           int32_t T, int32_t max_len, const void* q, const void* k, const void* v, const int32_t* parent,
                           void* o, void* workspace, size_t workspace_bytes, ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_attn(dims, cache, nseq, slot));
  if (max_len < 0 || !drafts_ok(dims, nseq, T)) return ERS_EINVAL;
  if (nseq == 0) return ERS_OK;
  for (const void* p : {q, k, v, (const void*)o}) ERS_TRY(check_ptr(p, true));
  ERS_TRY(check_ptr(parent, false));
  ERS_TRY(check_ptr(dev_status, false));
  ers::AttnArgs a = attn_args(dims, cache, nseq, slot, T, k, v, dev_status);
  a.q = q;
  a.parent = parent;
  a.o = o;
  ers::attn_plan(&a, max_len);
  const size_t need = ers::attn_workspace(a);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return ERS_EWORKSPACE;
  ERS_TRY(check_ptr(workspace, false));
  a.part = static_cast<float*>(workspace);
  return finish(ers::attn_verify(a, (cudaStream_t)stream));
}

ers_status ers_attn_append(const ers_attn_dims* dims, const ers_attn_cache* cache, int32_t nseq, int64_t ntokens,
                           const int32_t* cu_seqlens, const int32_t* slot, const void* k, const void* v,
                           ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_attn(dims, cache, nseq, slot));
  if (ntokens < 0 || ntokens > 0x7fffffff || nseq > 0x3fffffff) return ERS_EINVAL;
  if (nseq == 0) return ERS_OK;
  ERS_TRY(check_ptr(cu_seqlens, true));
  ERS_TRY(check_ptr(k, ntokens > 0));
  ERS_TRY(check_ptr(v, ntokens > 0));
  ERS_TRY(check_ptr(dev_status, false));
  ers::AttnArgs a = attn_args(dims, cache, nseq, slot, 0, k, v, dev_status);
  a.cu = cu_seqlens;
  a.ntokens = ntokens;
  return finish(ers::attn_append(a, (cudaStream_t)stream));
}

ers_status ers_attn_commit(const ers_attn_dims* dims, const ers_attn_cache* cache, int32_t nseq, const int32_t* slot,
                           int32_t T, const int32_t* path, const int32_t* accepted, const void* k, const void* v,
                           ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_attn(dims, cache, nseq, slot));
  if (!drafts_ok(dims, nseq, T)) return ERS_EINVAL;
  if (nseq == 0) return ERS_OK;
  ERS_TRY(check_ptr(accepted, true));
  ERS_TRY(check_ptr(path, false));
  ERS_TRY(check_ptr(k, true));
  ERS_TRY(check_ptr(v, true));
  ERS_TRY(check_ptr(dev_status, false));
  ers::AttnArgs a = attn_args(dims, cache, nseq, slot, T, k, v, dev_status);
  a.path = path;
  a.accepted = accepted;
  return finish(ers::attn_commit(a, (cudaStream_t)stream));
}

}  // extern "C"
