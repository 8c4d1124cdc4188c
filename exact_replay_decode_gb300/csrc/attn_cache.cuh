// What every kernel of the paged attention cache reads of it.
#pragma once

#include "ers_common.cuh"
#include "ers_internal.h"

namespace ers {

// Of `all` parts of rows, the workspace holds a maximum and a sum each, then, from this float on, their outputs (16-byte aligned).
__host__ __device__ __forceinline__ size_t part_outputs(size_t all) { return (2 * all + 3) & ~size_t(3); }

struct AttnSeq {
  const int32_t* pages;   // the slot's row of the table
  int slot, pos;          // tokens of the past
};

// Sequence i's slot and how much of it is in use; the error that it has instead.  The same for every thread.
__device__ __forceinline__ int32_t attn_seq(const AttnArgs& a, int i, AttnSeq* s) {
  s->slot = a.slot != nullptr ? a.slot[i] : i;
  if (s->slot < 0 || s->slot >= a.nslots) return ERS_ESLOT;
  s->pages = a.table + (size_t)s->slot * a.slot_pages;
  s->pos = a.pos[s->slot];
  if (s->pos < 0 || s->pos > (long long)a.slot_pages * a.page_tokens) return ERS_EALIGN;
  return ERS_OK;
}

// The page of a slot that token `at` is in
__device__ __forceinline__ int page_of(const AttnArgs& a, int at) {
  return (int)((__umulhi(a.page_magic, (uint32_t)at) + (uint32_t)at) >> a.page_shift);
}

// The pool's row of token `at` of a slot, of those that the table has room for; -1 where its page is none of the pool's.
__device__ __forceinline__ long long attn_row(const AttnArgs& a, const int32_t* pages, int at) {
  const int n = page_of(a, at), page = pages[n];
  return page < 0 || page >= a.npages ? -1 : (long long)page * a.page_tokens + (at - n * a.page_tokens);
}

// The places of a draft's path, its own among them, as bits; 0 for an empty place.  parent: the sequence's, in shared memory
// (null: a chain).  bad: set where a parent is neither an earlier place in use nor -1.
__device__ __forceinline__ uint64_t path_of(const int32_t* parent, int t, bool* bad) {
  if (parent == nullptr) return ~0ull >> (63 - t);
  uint64_t m = 0;
  int at = t, p = parent[t];
  if (p == -2) return 0;
  m = 1ull << at;
  while (p != -1) {
    if (p < 0 || p >= at) {
      *bad = true;
      return 0;
    }
    at = p;
    m |= 1ull << at;
    p = parent[at];
  }
  return m;
}

}  // namespace ers
