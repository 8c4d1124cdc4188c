// What every linear-attention kernel reads of its arguments: the tokens and states of a sequence.
#pragma once

#include "ers_common.cuh"
#include "ers_internal.h"

namespace ers {

struct LinAttnSeq {
  const float* in;   // the head's state [dv, dk] before the first token; null: zeros
  float* out;        // and after the last
  int t0, len;       // its tokens
};

// Sequence i, head h.  False (reported by one thread) where an index leads outside the caller's memory:
// nothing of that sequence may then be touched.  False as well where another launch takes the sequence.
__device__ __forceinline__ bool linattn_seq(const LinAttnArgs& a, int i, int h, LinAttnSeq* s) {
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

// exp(x) as the sum of two floats, for factors that a state meets once a token (or once a chunk): the rounding of a single
// float would add up over the state's whole memory (256 tokens at x = -1/256: a relative error of 4e-6).  Near 1, where
// the memory is long, 1 + expm1(x) is exact to 2^-24 |x|; further off the memory is short, and one float does.
struct Decay {
  float hi, lo;
  __device__ __forceinline__ float step(float s, float add) const { return fmaf(hi, s, fmaf(lo, s, add)); }
};
__device__ __forceinline__ Decay decay_of(float x) {
  if (fabsf(x) > 0.5f) return {expf(x), 0.f};
  const float m = expm1f(x), hi = __fadd_rn(1.f, m);
  return {hi, __fsub_rn(m, __fsub_rn(hi, 1.f))};
}

// exp(a n): of whole n, the product's rounding made good
__device__ __forceinline__ Decay decay_of_tokens(float a, int n) {
  const float x = a * (float)n, rest = fmaf(a, (float)n, -x);
  Decay d = decay_of(x);
  d.lo = fmaf(d.hi, rest, d.lo);
  return d;
}
__device__ __forceinline__ float power_of(float a, int n) {
  const Decay d = decay_of_tokens(a, n);
  return d.hi + d.lo;
}

}  // namespace ers
