// C ABI of the serving operators around a linear-attention layer (declared in include/ers.h): host-side
// validation and dispatch.  A call that fails validation launches nothing.
#include <math.h>
#include <string.h>

#include "api_checks.h"
#include "ers.h"
#include "ers_internal.h"

using ers::check_ptr;

namespace {

ers_status finish(cudaError_t e) { return e == cudaSuccess ? ERS_OK : ERS_ECUDA; }

// ---- linear attention ------------------------------------------------------------------------------
ers_status check_linattn(const ers_linattn_dims* d, int32_t nseq) {
  if (d == nullptr) return ERS_EINVAL;
  if (d->io_dtype != ERS_DTYPE_F32 && d->io_dtype != ERS_DTYPE_BF16) return ERS_EDTYPE;
  if (d->nheads <= 0 || d->ngroups <= 0 || d->nheads % d->ngroups != 0) return ERS_ESHAPE;
  if (d->nheads > 65535 || !ers::linattn_supported(d->dk, d->dv)) return ERS_ESHAPE;
  if (nseq < 0 || !isfinite(d->scale)) return ERS_EINVAL;
  return ERS_OK;
}

ers_status check_linattn_cache(const ers_linattn_cache* c, int32_t nseq, const int32_t* slot) {
  if (c == nullptr || c->nslots < 0 || c->npages < 0) return ERS_EINVAL;
  if (slot == nullptr && nseq > c->nslots) return ERS_EINVAL;
  ERS_TRY(check_ptr(c->state, true));
  ERS_TRY(check_ptr(c->table, true));
  return check_ptr(slot, false);
}

ers_status check_qkvo(const void* q, const void* k, const void* v, const void* o, const float* log_decay,
                      bool tokens, const int32_t* st) {
  ERS_TRY(check_ptr(q, tokens));
  ERS_TRY(check_ptr(k, tokens));
  ERS_TRY(check_ptr(v, tokens));
  ERS_TRY(check_ptr(o, tokens));
  ERS_TRY(check_ptr(log_decay, true));
  return check_ptr(st, false);
}

ers::LinAttnArgs linattn_args(const ers_linattn_dims* d, const float* log_decay, int32_t nseq, const void* q,
                              const void* k, const void* v, void* o, int32_t* st) {
  ers::LinAttnArgs a;
  memset(&a, 0, sizeof(a));
  a.H = d->nheads;
  a.G = d->ngroups;
  a.dk = d->dk;
  a.dv = d->dv;
  a.io = d->io_dtype;
  a.scale = d->scale;
  a.log_decay = log_decay;
  a.nseq = nseq;
  a.len1 = INT32_MAX;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.status = st;
  return a;
}

void set_cache(ers::LinAttnArgs* a, const ers_linattn_cache* c, const int32_t* slot, const int32_t* read_page) {
  a->pool = c->state;
  a->table = c->table;
  a->nslots = c->nslots;
  a->npages = c->npages;
  a->slot = slot;
  a->read_page = read_page;
}

// ---- pages -------------------------------------------------------------------------------------------
ers_status check_pool(const ers_page_pool* p, int32_t n, bool counted) {
  if (p == nullptr || n < 0 || p->npages < 0 || p->narrays < 0 || p->narrays > ERS_PAGE_ARRAYS_MAX) return ERS_EINVAL;
  for (int k = 0; k < p->narrays; ++k) {
    ERS_TRY(check_ptr(p->array[k], p->npages > 0));
    if (p->page_bytes[k] <= 0 || p->page_bytes[k] % 2 != 0) return ERS_ESHAPE;
  }
  if (!counted) return ERS_OK;
  if (p->nslots < 0 || p->nslots > ERS_PAGE_SLOTS_MAX || p->slot_pages < 1) return ERS_ESHAPE;
  // the deciding CTA counts in steps of 1024 in 32 bits
  if ((int64_t)p->nslots * p->slot_pages > ERS_PAGES_MAX || p->npages > ERS_PAGES_MAX || n > p->nslots) return ERS_EINVAL;
  ERS_TRY(check_ptr(p->table, p->nslots > 0));
  return check_ptr(p->refs, p->npages > 0);
}

ers::PageArgs page_args(const ers_page_pool* p, int32_t n, int32_t* st) {
  ers::PageArgs a;
  memset(&a, 0, sizeof(a));
  a.table = p->table;
  a.refs = p->refs;
  a.nslots = p->nslots;
  a.slot_pages = p->slot_pages;
  a.npages = p->npages;
  a.narrays = p->narrays;
  for (int k = 0; k < p->narrays; ++k) {
    a.array[k] = static_cast<char*>(p->array[k]);
    a.page_bytes[k] = p->page_bytes[k];
  }
  a.n = n;
  a.status = st;
  return a;
}

}  // namespace

extern "C" {

ers_status ers_linattn_fwd(const ers_linattn_dims* dims, const float* log_decay, int32_t nseq, int64_t ntokens,
                           int32_t max_seqlen, const int32_t* cu_seqlens, const void* q, const void* k, const void* v,
                           const float* init_state, void* o, float* final_state, ers_stream_t stream,
                           int32_t* dev_status) {
  ERS_TRY(check_linattn(dims, nseq));
  if (ntokens < 0 || ntokens > 0x7fffffff || max_seqlen < 0) return ERS_EINVAL;
  if (nseq == 0) return ERS_OK;
  ERS_TRY(check_qkvo(q, k, v, o, log_decay, ntokens > 0, dev_status));
  ERS_TRY(check_ptr(cu_seqlens, true));
  ERS_TRY(check_ptr(init_state, false));
  ERS_TRY(check_ptr(final_state, true));
  ers::LinAttnArgs a = linattn_args(dims, log_decay, nseq, q, k, v, o, dev_status);
  a.ntokens = ntokens;
  a.max_len = max_seqlen;
  a.cu = cu_seqlens;
  a.init = init_state;
  a.final_state = final_state;
  return finish(ers::linattn_fwd(a, (cudaStream_t)stream));
}

ers_status ers_linattn_prefill(const ers_linattn_dims* dims, const float* log_decay, const ers_linattn_cache* cache,
                               int32_t nseq, int64_t ntokens, int32_t max_seqlen, const int32_t* cu_seqlens,
                               const int32_t* slot, const int32_t* read_page, const void* q, const void* k,
                               const void* v, void* o, ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_linattn(dims, nseq));
  if (ntokens < 0 || ntokens > 0x7fffffff || max_seqlen < 0) return ERS_EINVAL;
  ERS_TRY(check_linattn_cache(cache, nseq, slot));
  if (nseq == 0) return ERS_OK;
  ERS_TRY(check_qkvo(q, k, v, o, log_decay, ntokens > 0, dev_status));
  ERS_TRY(check_ptr(cu_seqlens, true));
  ERS_TRY(check_ptr(read_page, false));
  ers::LinAttnArgs a = linattn_args(dims, log_decay, nseq, q, k, v, o, dev_status);
  a.ntokens = ntokens;
  a.max_len = max_seqlen;
  a.cu = cu_seqlens;
  set_cache(&a, cache, slot, read_page);
  return finish(ers::linattn_fwd(a, (cudaStream_t)stream));
}

ers_status ers_linattn_decode(const ers_linattn_dims* dims, const float* log_decay, const ers_linattn_cache* cache,
                              int32_t nseq, const int32_t* slot, const int32_t* read_page, const void* q,
                              const void* k, const void* v, void* o, ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_linattn(dims, nseq));
  ERS_TRY(check_linattn_cache(cache, nseq, slot));
  if (nseq == 0) return ERS_OK;
  ERS_TRY(check_qkvo(q, k, v, o, log_decay, true, dev_status));
  ERS_TRY(check_ptr(read_page, false));
  ers::LinAttnArgs a = linattn_args(dims, log_decay, nseq, q, k, v, o, dev_status);
  a.ntokens = nseq;
  set_cache(&a, cache, slot, read_page);
  return finish(ers::linattn_decode(a, (cudaStream_t)stream));
}

ers_status ers_pages_fork(const ers_page_pool* pool, int32_t n, const int32_t* src, const int32_t* dst,
                          ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_pool(pool, n, true));
  if (n == 0) return ERS_OK;
  ERS_TRY(check_ptr(src, true));
  ERS_TRY(check_ptr(dst, true));
  ERS_TRY(check_ptr(dev_status, false));
  ers::PageArgs a = page_args(pool, n, dev_status);
  a.src = src;
  a.dst = dst;
  return finish(ers::pages_fork(a, (cudaStream_t)stream));
}

size_t ers_pages_own_workspace_size(const ers_page_pool* pool, int32_t n) {
  if (pool == nullptr || n < 0 || pool->slot_pages < 1) return 0;
  return ers::align256((size_t)n * pool->slot_pages * 2 * sizeof(int32_t));
}

ers_status ers_pages_own(const ers_page_pool* pool, int32_t n, const int32_t* slot, uint32_t flags,
                         int32_t* read_page, void* workspace, size_t workspace_bytes, ers_stream_t stream,
                         int32_t* dev_status) {
  ERS_TRY(check_pool(pool, n, true));
  if ((flags & ~ERS_FLAG_COPY) != 0) return ERS_EINVAL;
  if (n == 0) return ERS_OK;
  ERS_TRY(check_ptr(slot, true));
  ERS_TRY(check_ptr(read_page, true));
  ERS_TRY(check_ptr(dev_status, false));
  if (workspace == nullptr || workspace_bytes < ers_pages_own_workspace_size(pool, n)) return ERS_EWORKSPACE;
  ERS_TRY(check_ptr(workspace, true));
  ers::PageArgs a = page_args(pool, n, dev_status);
  a.dst = slot;
  a.read_page = read_page;
  a.ws = static_cast<int32_t*>(workspace);
  return finish(ers::pages_own(a, (flags & ERS_FLAG_COPY) != 0, (cudaStream_t)stream));
}

ers_status ers_pages_clone(const ers_page_pool* pool, int32_t n, const int32_t* src, const int32_t* dst,
                           int32_t* read_page, void* workspace, size_t workspace_bytes, ers_stream_t stream,
                           int32_t* dev_status) {
  ERS_TRY(check_pool(pool, n, true));
  if (n == 0) return ERS_OK;
  ERS_TRY(check_ptr(src, true));
  ERS_TRY(check_ptr(dst, true));
  ERS_TRY(check_ptr(read_page, true));
  ERS_TRY(check_ptr(dev_status, false));
  if (workspace == nullptr || workspace_bytes < ers_pages_own_workspace_size(pool, n)) return ERS_EWORKSPACE;
  ERS_TRY(check_ptr(workspace, true));
  ers::PageArgs a = page_args(pool, n, dev_status);
  a.src = src;
  a.dst = dst;
  a.read_page = read_page;
  a.ws = static_cast<int32_t*>(workspace);
  return finish(ers::pages_clone(a, (cudaStream_t)stream));
}

ers_status ers_pages_free(const ers_page_pool* pool, int32_t n, const int32_t* slot, ers_stream_t stream,
                          int32_t* dev_status) {
  ERS_TRY(check_pool(pool, n, true));
  if (n == 0) return ERS_OK;
  ERS_TRY(check_ptr(slot, true));
  ERS_TRY(check_ptr(dev_status, false));
  ers::PageArgs a = page_args(pool, n, dev_status);
  a.dst = slot;
  return finish(ers::pages_free(a, (cudaStream_t)stream));
}

size_t ers_pages_compact_workspace_size(const ers_page_pool* pool) {
  if (pool == nullptr || pool->npages < 0) return 0;
  return ers::align256(((size_t)pool->npages * 2 + 1) * sizeof(int32_t));
}

ers_status ers_pages_compact(const ers_page_pool* pool, int32_t* remap, int32_t* live, void* workspace,
                             size_t workspace_bytes, ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_pool(pool, 0, true));
  ERS_TRY(check_ptr(remap, pool->npages > 0));
  ERS_TRY(check_ptr(live, true));
  ERS_TRY(check_ptr(dev_status, false));
  if (workspace == nullptr || workspace_bytes < ers_pages_compact_workspace_size(pool)) return ERS_EWORKSPACE;
  ERS_TRY(check_ptr(workspace, true));
  ers::PageArgs a = page_args(pool, 0, dev_status);
  a.remap = remap;
  a.live = live;
  a.ws = static_cast<int32_t*>(workspace);
  return finish(ers::pages_compact(a, (cudaStream_t)stream));
}

ers_status ers_pages_copy(const ers_page_pool* pool, int32_t n, const int32_t* src, const int32_t* dst,
                          ers_stream_t stream, int32_t* dev_status) {
  ERS_TRY(check_pool(pool, n, false));
  if (n == 0 || pool->narrays == 0) return ERS_OK;
  ERS_TRY(check_ptr(src, true));
  ERS_TRY(check_ptr(dst, true));
  ERS_TRY(check_ptr(dev_status, false));
  ers::PageArgs a = page_args(pool, n, dev_status);
  a.src = src;
  a.dst = dst;
  return finish(ers::pages_copy(a, (cudaStream_t)stream));
}

ers_status ers_token_logprobs(int32_t io_dtype, int32_t nrows, int32_t vocab, int64_t row_stride, const void* logits,
                              const int32_t* target, float scale, int32_t top_k, float* logprob, float* entropy,
                              int32_t* top_id, float* top_logprob, ers_stream_t stream, int32_t* dev_status) {
  if (io_dtype != ERS_DTYPE_F32 && io_dtype != ERS_DTYPE_BF16) return ERS_EDTYPE;
  if (nrows < 0 || vocab < 1 || vocab > 0x7fff0000 || row_stride < vocab) return ERS_EINVAL;
  if (top_k < 0 || top_k > ERS_TOP_MAX || !(scale > 0.f) || !isfinite(scale)) return ERS_EINVAL;
  if (nrows == 0) return ERS_OK;
  const uintptr_t element = io_dtype == ERS_DTYPE_BF16 ? 2 : 4;
  if (logits == nullptr || (target == nullptr) != (logprob == nullptr)) return ERS_EINVAL;
  if (reinterpret_cast<uintptr_t>(logits) % element != 0) return ERS_EPTR;
  ERS_TRY(check_ptr(target, false));
  ERS_TRY(check_ptr(logprob, false));
  ERS_TRY(check_ptr(entropy, false));
  ERS_TRY(check_ptr(top_id, top_k > 0));
  ERS_TRY(check_ptr(top_logprob, top_k > 0));
  ERS_TRY(check_ptr(dev_status, false));
  ers::LogprobArgs a;
  memset(&a, 0, sizeof(a));
  a.io = io_dtype;
  a.nrows = nrows;
  a.vocab = vocab;
  a.stride = row_stride;
  a.scale = scale;
  a.top_k = top_k;
  a.logits = logits;
  a.target = target;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_id = top_id;
  a.top_logprob = top_logprob;
  a.status = dev_status;
  return finish(ers::token_logprobs(a, (cudaStream_t)stream));
}

}  // extern "C"
