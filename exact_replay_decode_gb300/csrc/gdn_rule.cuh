// What every kernel of the gated delta rule over cached states reads of its arguments: the tokens and states of a sequence.
#pragma once

#include "ers_common.cuh"
#include "ers_internal.h"
#include "linattn.cuh"

namespace ers {

struct DeltaSeq {
  const float* in;   // the head's state [dv, dk] before the first token; null: zeros
  float* out;        // and after the last
  int t0, len;       // its tokens
};

// Sequence i, head h.  False (reported by one thread) where an index leads outside the caller's memory:
// nothing of that sequence may then be touched.  False as well where another launch takes the sequence.
__device__ __forceinline__ bool delta_seq(const DeltaArgs& a, int i, int h, DeltaSeq* s) {
  int32_t err = ERS_OK;
  s->t0 = i;
  s->len = 1;
  if (a.cu != nullptr) {
    s->t0 = a.cu[i];
    const int end = a.cu[i + 1];
    s->len = end - s->t0;
    if (s->t0 < 0 || end < s->t0 || end > a.ntokens) err = ERS_EINVAL;
  }
  const size_t head = (size_t)a.dv * a.dk;
  if (a.pool == nullptr) {
    s->in = a.init != nullptr ? a.init + ((size_t)i * a.H + h) * head : nullptr;
    s->out = a.final_state + ((size_t)i * a.H + h) * head;
  } else {
    const int slot = a.slot != nullptr ? a.slot[i] : i;
    const bool slot_ok = slot >= 0 && slot < a.nslots;
    const int own = slot_ok ? a.table[slot] : -1;
    const int from = a.read_page != nullptr ? a.read_page[i] : own;
    if (own < 0 || own >= a.npages || from < -1 || from >= a.npages) {
      err = ERS_ESLOT;
    } else {
      s->in = from < 0 ? nullptr : a.pool + ((size_t)from * a.H + h) * head;
      s->out = a.pool + ((size_t)own * a.H + h) * head;
    }
  }
  if (err != ERS_OK && threadIdx.x == 0) report(a.status, err);
  return err == ERS_OK && s->len >= a.len0 && s->len <= a.len1;
}

}  // namespace ers
