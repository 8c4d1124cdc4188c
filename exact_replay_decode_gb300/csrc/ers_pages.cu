// Pages of a cache (include/ers.h): counted references under a table of pages per slot.
//
// The decisions (which page goes where) are whole numbers with an order, a few thousand of them, so one
// CTA takes them with prefix sums in shared memory: first everything is checked and counted, then
// either all of it is carried out or none.  The bytes are moved by a second launch over the whole GPU, at the rate of a
// device copy (128 pages of 2 MB: 81 us, 98 % of the measured bandwidth).  The decisions are latency, some 2 us each beside
// the launch; launches follow one another as programmatic dependents, so the next one is set up under the last one's work.
#include <string.h>

#include "ers_common.cuh"
#include "ers_internal.h"

namespace ers {
namespace {

constexpr int kPlan = 1024;   // threads of a deciding CTA
static_assert(ERS_PAGES_MAX <= 0x7fffffff - kPlan + 1, "its loops go one step past the last entry or page");
// CTAs that move bytes: two full waves of eight per SM.  By 1216, 2432, 4864 and 9728: 128 pages of 2 MB 80.9, 80.4, 78.8, 78.5
// us; a compaction with nothing to move 4.8, 6.0, 8.4, 13.3.
constexpr int kMovers = 2432;

// The next launch may be set up; this one's memory accesses wait for the last one to complete.
__device__ __forceinline__ void follow() {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
}

// Inclusive prefix sum over the CTA's threads; *total receives the sum.  scratch: kPlan / 32 ints.
__device__ __forceinline__ int block_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(kFull, v, off);
    if (lane >= off) v += u;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  int w = scratch[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(kFull, w, off);
    if (lane >= off) w += u;
  }
  const int before = __shfl_sync(kFull, w, warp == 0 ? 0 : warp - 1);
  *total = __shfl_sync(kFull, w, 31);
  __syncthreads();   // scratch may be written again
  return v + (warp == 0 ? 0 : before);
}

// Whether any thread found an error; the smallest code found is reported.
__device__ __forceinline__ bool failed(int32_t err, int32_t* status) {
  __shared__ int worst;
  if (threadIdx.x == 0) worst = 0x7fffffff;
  __syncthreads();
  if (err != ERS_OK) atomicMin(&worst, err);
  __syncthreads();
  const int w = worst;
  if (w != 0x7fffffff && threadIdx.x == 0) report(status, w);
  return w != 0x7fffffff;
}

// Checks the listed slots: in range, each listed once (seen: one bit per slot, shared memory).
__device__ __forceinline__ int32_t check_slots(const PageArgs& a, const int32_t* list, uint32_t* seen) {
  int32_t err = ERS_OK;
  for (int w = threadIdx.x; w < (a.nslots + 31) / 32; w += kPlan) seen[w] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kPlan) {
    const int s = list[i];
    if (s < 0 || s >= a.nslots) {
      err = ERS_ESLOT;
    } else if ((atomicOr(&seen[s >> 5], 1u << (s & 31)) >> (s & 31)) & 1u) {
      err = ERS_EINVAL;
    }
  }
  __syncthreads();
  return err;
}

// Entry e of the listed slots' table rows, one row after the other.
__device__ __forceinline__ int32_t* entry(const PageArgs& a, int e) {
  return &a.table[(size_t)a.dst[e / a.slot_pages] * a.slot_pages + e % a.slot_pages];
}
// An entry: -1, or a page of the pool that has a reference (one without counts as free: it would be handed out again).
__device__ __forceinline__ int32_t check_entry(const PageArgs& a, int p) {
  if (p < -1 || p >= a.npages) return ERS_ESLOT;
  return p >= 0 && a.refs[p] < 1 ? ERS_EINVAL : ERS_OK;
}

__global__ void __launch_bounds__(kPlan) k_pages_fork(PageArgs a) {
  extern __shared__ uint32_t seen[];
  follow();
  const int m = a.n * a.slot_pages;
  int32_t err = check_slots(a, a.dst, seen);
  for (int i = threadIdx.x; i < a.n; i += kPlan) {
    const int s = a.src[i];
    if (s < 0 || s >= a.nslots) err = ERS_ESLOT;
    else if ((seen[s >> 5] >> (s & 31)) & 1u) err = ERS_EINVAL;
  }
  if (failed(err, a.status)) return;
  for (int e = threadIdx.x; e < m; e += kPlan) {
    const int i = e / a.slot_pages, c = e % a.slot_pages;
    if (a.table[(size_t)a.dst[i] * a.slot_pages + c] != -1) err = ERS_EINVAL;   // it would be lost
    const int32_t bad = check_entry(a, a.table[(size_t)a.src[i] * a.slot_pages + c]);
    if (bad != ERS_OK) err = bad;
  }
  if (failed(err, a.status)) return;
  for (int e = threadIdx.x; e < m; e += kPlan) {
    const int i = e / a.slot_pages, c = e % a.slot_pages;
    const int p = a.table[(size_t)a.src[i] * a.slot_pages + c];
    a.table[(size_t)a.dst[i] * a.slot_pages + c] = p;
    if (p >= 0) atomicAdd(&a.refs[p], 1);
  }
}

__global__ void __launch_bounds__(kPlan) k_pages_free(PageArgs a) {
  extern __shared__ uint32_t seen[];
  follow();
  const int m = a.n * a.slot_pages;
  if (failed(check_slots(a, a.dst, seen), a.status)) return;
  int32_t err = ERS_OK;
  for (int e = threadIdx.x; e < m; e += kPlan) {
    const int p = *entry(a, e);
    if (p < -1 || p >= a.npages) err = ERS_ESLOT;
    else if (p >= 0 && atomicSub(&a.refs[p], 1) < 1) err = ERS_EINVAL;   // named more often than counted
  }
  const bool bad = failed(err, a.status);   // then all references are given back
  for (int e = threadIdx.x; e < m; e += kPlan) {
    const int p = *entry(a, e);
    if (!bad) *entry(a, e) = -1;
    else if (p >= 0 && p < a.npages) atomicAdd(&a.refs[p], 1);
  }
}

// ws: [m] rank of an entry among those that need a page (-1: it keeps its own), then [m] the free pages
__global__ void __launch_bounds__(kPlan) k_pages_own(PageArgs a) {
  extern __shared__ uint32_t seen[];
  __shared__ int scratch[kPlan / 32];
  follow();
  const int m = a.n * a.slot_pages;
  int32_t* rank = a.ws;
  int32_t* free_page = a.ws + m;
  int32_t err = check_slots(a, a.dst, seen);
  bool bad = failed(err, a.status);
  int needed = 0, found = 0;
  if (!bad) {
    for (int e0 = 0; e0 < m; e0 += kPlan) {
      const int e = e0 + threadIdx.x;
      int need = 0, p = -1;
      if (e < m) {
        p = *entry(a, e);
        const int32_t wrong = check_entry(a, p);
        if (wrong != ERS_OK) err = wrong;
        else need = p < 0 || a.refs[p] > 1;
      }
      int total;
      const int upto = block_scan(need, scratch, &total);
      if (e < m) {
        rank[e] = need ? needed + upto - 1 : -1;
        a.read_page[e] = p;
      }
      needed += total;
    }
    for (int p0 = 0; p0 < a.npages && found < needed; p0 += kPlan) {
      const int p = p0 + threadIdx.x;
      const int is_free = p < a.npages && a.refs[p] <= 0;
      int total;
      const int r = found + block_scan(is_free, scratch, &total) - 1;
      if (is_free && r < needed) free_page[r] = p;
      found += total;
    }
    if (found < needed) err = ERS_EOVERFLOW;
    bad = failed(err, a.status);
  }
  if (!bad) {
    for (int e = threadIdx.x; e < m; e += kPlan) {
      const int r = rank[e], old = a.read_page[e];
      if (r < 0) continue;
      const int p = free_page[r];
      a.refs[p] = 1;
      *entry(a, e) = p;
      if (old >= 0 && atomicSub(&a.refs[old], 1) < 1) err = ERS_EINVAL;   // named more often than counted
    }
    bad = failed(err, a.status);            // then all of it is taken back
    for (int e = threadIdx.x; bad && e < m; e += kPlan) {
      const int r = rank[e], old = a.read_page[e];
      if (r < 0) continue;
      a.refs[free_page[r]] = 0;
      *entry(a, e) = old;
      if (old >= 0) atomicAdd(&a.refs[old], 1);
    }
  }
  if (bad) {
    for (int e = threadIdx.x; e < m; e += kPlan) {
      rank[e] = -1;
      a.read_page[e] = -2;
    }
  }
}

// As free of dst, fork and own of the same lists, in one decision: every entry of dst's rows gets a page of its own, to be filled
// from src's.  ws as k_pages_own.
__global__ void __launch_bounds__(kPlan) k_pages_clone(PageArgs a) {
  extern __shared__ uint32_t seen[];
  __shared__ int scratch[kPlan / 32];
  follow();
  const int m = a.n * a.slot_pages;
  int32_t* rank = a.ws;
  int32_t* free_page = a.ws + m;
  int32_t err = check_slots(a, a.dst, seen);
  for (int i = threadIdx.x; i < a.n; i += kPlan) {
    const int s = a.src[i];
    if (s < 0 || s >= a.nslots) err = ERS_ESLOT;
    else if ((seen[s >> 5] >> (s & 31)) & 1u) err = ERS_EINVAL;
  }
  bool bad = failed(err, a.status);
  const bool given_up = !bad;
  if (!bad) {
    for (int e = threadIdx.x; e < m; e += kPlan) {
      const int p = a.table[(size_t)a.src[e / a.slot_pages] * a.slot_pages + e % a.slot_pages], old = *entry(a, e);
      a.read_page[e] = p;
      if (p < -1 || p >= a.npages || old < -1 || old >= a.npages) err = ERS_ESLOT;
      if (old >= 0 && old < a.npages && atomicSub(&a.refs[old], 1) < 1) err = ERS_EINVAL;   // named more often than counted
    }
    bad = failed(err, a.status);
  }
  if (!bad) {
    int found = 0;
    for (int e = threadIdx.x; e < m; e += kPlan) {
      const int32_t wrong = check_entry(a, a.read_page[e]);   // (what dst gave up is no longer counted)
      if (wrong != ERS_OK) err = wrong;
    }
    for (int p0 = 0; p0 < a.npages && found < m; p0 += kPlan) {
      const int p = p0 + threadIdx.x;
      const int is_free = p < a.npages && a.refs[p] <= 0;
      int total;
      const int r = found + block_scan(is_free, scratch, &total) - 1;
      if (is_free && r < m) free_page[r] = p;
      found += total;
    }
    if (found < m) err = ERS_EOVERFLOW;
    bad = failed(err, a.status);
  }
  for (int e = threadIdx.x; e < m; e += kPlan) {
    if (bad) {
      const int old = given_up ? *entry(a, e) : -1;
      if (old >= 0 && old < a.npages) atomicAdd(&a.refs[old], 1);
      rank[e] = -1;
      a.read_page[e] = -2;
    } else {
      rank[e] = e;
      a.refs[free_page[e]] = 1;
      *entry(a, e) = free_page[e];
    }
  }
}

// ws: [0] pages that move (-1: an error was found), [1, 1 + npages) where from, then [npages] where to
__global__ void __launch_bounds__(kPlan) k_pages_compact(PageArgs a) {
  __shared__ int scratch[kPlan / 32];
  follow();
  int32_t* from = a.ws + 1;
  int32_t* to = from + a.npages;
  int32_t err = ERS_OK;
  for (long long e = threadIdx.x; e < (long long)a.nslots * a.slot_pages; e += kPlan) {
    const int32_t wrong = check_entry(a, a.table[e]);
    if (wrong != ERS_OK) err = wrong;
  }
  int live = 0;
  for (int p0 = 0; p0 < a.npages; p0 += kPlan) {
    int total;
    block_scan(p0 + threadIdx.x < a.npages && a.refs[p0 + threadIdx.x] > 0, scratch, &total);
    live += total;
  }
  const bool bad = failed(err, a.status);
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < a.npages; p0 += kPlan) {
    const int p = p0 + threadIdx.x;
    const bool in = p < a.npages, used = in && a.refs[p] > 0;
    const int hole = in && !used && p < live, mover = used && p >= live;
    int total;
    int r = block_scan(hole, scratch, &total);
    if (hole) to[holes + r - 1] = p;
    holes += total;
    r = block_scan(mover, scratch, &total);
    if (mover) from[movers + r - 1] = p;
    movers += total;
    if (in) a.remap[p] = used ? p : -1;
  }
  __syncthreads();
  if (bad) movers = 0;
  for (int r = threadIdx.x; r < movers; r += kPlan) {
    a.remap[from[r]] = to[r];
    a.refs[to[r]] = a.refs[from[r]];
    a.refs[from[r]] = 0;
  }
  if (threadIdx.x == 0) {
    a.ws[0] = bad ? -1 : movers;
    *a.live = live;
  }
}

// ---- moving the bytes -----------------------------------------------------------------------------------
// A piece of a page is moved by a CTA in 16-byte words (2-byte ones where the page's size is no multiple).
constexpr long long kPiece = 32768;

__device__ __forceinline__ void move_piece(char* dst, const char* src, long long bytes, bool wide) {
  constexpr int n = kPiece / (kThreads * 16);
  if (wide && bytes == kPiece) {   // all of it under way before the first word is stored
    uint4 v[n];
#pragma unroll
    for (int i = 0; i < n; ++i)
      v[i] = src != nullptr ? __ldcs(reinterpret_cast<const uint4*>(src) + i * kThreads + threadIdx.x) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < n; ++i) __stcs(reinterpret_cast<uint4*>(dst) + i * kThreads + threadIdx.x, v[i]);
  } else if (wide) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (long long b = threadIdx.x * 16; b < bytes; b += kThreads * 16)
      *reinterpret_cast<uint4*>(dst + b) = src != nullptr ? *reinterpret_cast<const uint4*>(src + b) : z;
  } else {
    for (long long b = threadIdx.x * 2; b < bytes; b += kThreads * 2)
      *reinterpret_cast<uint16_t*>(dst + b) = src != nullptr ? *reinterpret_cast<const uint16_t*>(src + b) : uint16_t(0);
  }
}

// piece w of a page (counted through all arrays): page `to` <- page `from` (-1: zeros)
__device__ __forceinline__ void move_page_piece(const PageArgs& a, int to, int from, long long w) {
  for (int k = 0; k < a.narrays; ++k) {
    const long long size = a.page_bytes[k], pieces = (size + kPiece - 1) / kPiece;
    if (w < pieces) {
      const long long at = w * kPiece, n = size - at < kPiece ? size - at : kPiece;
      move_piece(a.array[k] + to * size + at, from < 0 ? nullptr : a.array[k] + from * size + at, n, size % 16 == 0);
      return;
    }
    w -= pieces;
  }
}

enum : int { kMoveOwn, kMoveCompact, kMoveList };

template <int kind>
__global__ void __launch_bounds__(kThreads) k_pages_move(PageArgs a, long long pieces) {
  follow();
  if (kind == kMoveCompact) {   // the tables follow
    const bool good = a.ws[0] >= 0;
    const long long entries = (long long)a.nslots * a.slot_pages;
    for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < entries; e += (long long)gridDim.x * kThreads) {
      const int p = a.table[e];
      if (good && p >= 0) a.table[e] = a.remap[p];
    }
  }
  const long long count = kind == kMoveCompact ? a.ws[0] : kind == kMoveOwn ? a.n * a.slot_pages : a.n;
  for (long long u = blockIdx.x; u < count * pieces; u += gridDim.x) {
    const int e = (int)(u / pieces);
    int to, from;
    if (kind == kMoveOwn) {
      if (a.ws[e] < 0) continue;
      to = a.ws[count + a.ws[e]];
      from = a.read_page[e];
    } else if (kind == kMoveCompact) {
      from = a.ws[1 + e];
      to = a.ws[1 + a.npages + e];
    } else {
      from = a.src[e];
      to = a.dst[e];
      if (from < 0 || from >= a.npages || to < 0 || to >= a.npages) {
        if (threadIdx.x == 0) report(a.status, ERS_ESLOT);
        continue;
      }
    }
    move_page_piece(a, to, from, u % pieces);
  }
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), long long ctas, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t move(const PageArgs& a, int kind, long long count, cudaStream_t s) {
  long long pieces = 0;
  for (int k = 0; k < a.narrays; ++k) pieces += (a.page_bytes[k] + kPiece - 1) / kPiece;
  if (count == 0 || (pieces == 0 && kind != kMoveCompact)) return cudaSuccess;
  const long long units = count > kMovers || pieces > kMovers ? kMovers : count * pieces;
  const long long ctas = units < 1 ? 1 : units > kMovers ? kMovers : units;
  if (kind == kMoveOwn) return launch(k_pages_move<kMoveOwn>, ctas, kThreads, 0, s, a, pieces);
  if (kind == kMoveCompact) return launch(k_pages_move<kMoveCompact>, ctas, kThreads, 0, s, a, pieces);
  return launch(k_pages_move<kMoveList>, ctas, kThreads, 0, s, a, pieces);
}

size_t seen_bytes(const PageArgs& a) { return (size_t)(a.nslots + 31) / 32 * sizeof(uint32_t); }

cudaError_t plan(void (*kernel)(PageArgs), const PageArgs& a, cudaStream_t s) {
  const size_t smem = seen_bytes(a);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch(kernel, 1, kPlan, smem, s, a);
}

}  // namespace

cudaError_t pages_fork(const PageArgs& a, cudaStream_t s) { return plan(k_pages_fork, a, s); }

cudaError_t pages_free(const PageArgs& a, cudaStream_t s) { return plan(k_pages_free, a, s); }

cudaError_t pages_own(const PageArgs& a, bool copy, cudaStream_t s) {
  const cudaError_t e = plan(k_pages_own, a, s);
  return e != cudaSuccess || !copy ? e : move(a, kMoveOwn, (long long)a.n * a.slot_pages, s);
}

cudaError_t pages_clone(const PageArgs& a, cudaStream_t s) {
  const cudaError_t e = plan(k_pages_clone, a, s);
  return e != cudaSuccess ? e : move(a, kMoveOwn, (long long)a.n * a.slot_pages, s);
}

cudaError_t pages_compact(const PageArgs& a, cudaStream_t s) {
  const cudaError_t e = launch(k_pages_compact, 1, kPlan, 0, s, a);
  return e != cudaSuccess ? e : move(a, kMoveCompact, a.npages, s);
}

cudaError_t pages_copy(const PageArgs& a, cudaStream_t s) { return move(a, kMoveList, a.n, s); }

}  // namespace ers
