// Attention over a paged cache (include/ers.h): drafts of a tree against their sequence's past and their own path, and the
// rows that prompts and accepted drafts add to the pages.
#include "attn_cache.cuh"
#include "ers_common.cuh"
#include "ers_internal.h"

namespace ers {
namespace {

// ---- drafts -----------------------------------------------------------------------------------------------
// fp32: the query rows of a sequence that share a head of keys, T drafts x H/KV heads, kRows of them a CTA, each warp four; tokens
// come through shared memory 32 at a time, one a lane, with a running maximum and sum a row.
constexpr int kRows = 16, kTile = 32, kWarps = 4, kEach = kRows / kWarps;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) k_attn_rows(const __grid_constant__ AttnArgs a) {
  using T = float;
  constexpr int C = D / 32;                    // output columns of a lane
  __shared__ __align__(16) float sq[kRows][D];
  __shared__ __align__(16) float sk[kTile][D + 4];
  __shared__ __align__(16) float sv[kTile][D];
  __shared__ float sp[kRows][kTile];
  __shared__ int32_t sparent[kMaxDrafts];
  const int split = blockIdx.x % a.nsplit, i = blockIdx.x / a.nsplit, kv = blockIdx.y % a.KV, row0 = blockIdx.y / a.KV * kRows;
  const int rep = a.H / a.KV, nrows = a.T * rep;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  AttnSeq s;
  int32_t err = attn_seq(a, i, &s);
  if (a.parent != nullptr && threadIdx.x < a.T) sparent[threadIdx.x] = a.parent[(size_t)i * a.T + threadIdx.x];
  __syncthreads();
  bool bad = false;
  if (threadIdx.x < a.T) path_of(a.parent != nullptr ? sparent : nullptr, threadIdx.x, &bad);
  if (__syncthreads_or(bad) && err == ERS_OK) err = ERS_EINVAL;
  const auto out_row = [&](int r) { return ((size_t)i * a.T + r / rep) * a.H + kv * rep + r % rep; };
  if (err != ERS_OK) {
    if (threadIdx.x == 0) report(a.status, err);
    if (a.nsplit > 1 && threadIdx.x < kRows && row0 + threadIdx.x < nrows)
      reinterpret_cast<float2*>(a.part)[out_row(row0 + threadIdx.x) * a.nsplit + split] = make_float2(0.f, -1.f);
    return;
  }
  for (int e = threadIdx.x; e < kRows * D; e += 32 * kWarps) {
    const int r = e / D, d = e % D;
    sq[r][d] = row0 + r < nrows ? to_f(((const T*)a.q)[out_row(row0 + r) * D + d]) : 0.f;
  }
  uint64_t path[kEach];
  float m[kEach], l[kEach], o[kEach][C];
#pragma unroll
  for (int x = 0; x < kEach; ++x) {
    const int r = row0 + warp * kEach + x;
    path[x] = r < nrows ? path_of(a.parent != nullptr ? sparent : nullptr, r / rep, &bad) : 0;
    m[x] = -INFINITY;
    l[x] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) o[x][c] = 0.f;
  }
  const bool last = split == a.nsplit - 1;
  const long long begin = (long long)split * a.per;
  const int end = last ? s.pos : (int)min((long long)s.pos, begin + a.per);
  const int past = begin < end ? (int)((end - begin + kTile - 1) / kTile) : 0, tiles = past + (last ? (a.T + kTile - 1) / kTile : 0);
  for (int n = 0; n < tiles; ++n) {
    const bool drafts = n >= past;
    const int t0 = drafts ? (n - past) * kTile : (int)begin + n * kTile;
    const int count = min(kTile, drafts ? a.T - t0 : end - t0);
    __syncthreads();                           // the last tile is no longer read
    for (int e = threadIdx.x; e < kTile * (D / 4); e += 32 * kWarps) {
      const int t = e / (D / 4), d = e % (D / 4) * 4;
      float k4[4] = {}, v4[4] = {};
      if (t < count) {
        const T *kr, *vr;
        long long row = (long long)i * a.T + t0 + t;
        if (drafts) {
          kr = (const T*)a.k;
          vr = (const T*)a.v;
        } else {
          row = attn_row(a, s.pages, t0 + t);
          kr = (const T*)a.k_pages;
          vr = (const T*)a.v_pages;
          if (row < 0) report(a.status, ERS_ESLOT);
        }
        if (row >= 0) {
          load_k<T, 4>(kr + ((size_t)row * a.KV + kv) * D + d, k4);
          load_k<T, 4>(vr + ((size_t)row * a.KV + kv) * D + d, v4);
        }
      }
      *reinterpret_cast<float4*>(&sk[t][d]) = make_float4(k4[0], k4[1], k4[2], k4[3]);
      *reinterpret_cast<float4*>(&sv[t][d]) = make_float4(v4[0], v4[1], v4[2], v4[3]);
    }
    __syncthreads();
    float x[kEach] = {};
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      const float4 k4 = *reinterpret_cast<const float4*>(&sk[lane][d]);
#pragma unroll
      for (int r = 0; r < kEach; ++r) {
        const float4 q4 = *reinterpret_cast<const float4*>(&sq[warp * kEach + r][d]);
        x[r] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, x[r]))));
      }
    }
    uint32_t seen[kEach];
#pragma unroll
    for (int r = 0; r < kEach; ++r) {
      seen[r] = count == 32 ? kFull : (1u << count) - 1;
      if (drafts) seen[r] &= (uint32_t)(path[r] >> t0);
      else if (path[r] == 0) seen[r] = 0;
      const bool mine = seen[r] >> lane & 1u;
      const float y = mine ? x[r] * a.scale : -INFINITY;
      float top = y;
#pragma unroll
      for (int off = 16; off >= 1; off /= 2) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
      top = fmaxf(top, m[r]);
      const float base = top == -INFINITY ? 0.f : top, old = m[r] == -INFINITY ? 0.f : expf(m[r] - base);
      const float p = y == -INFINITY ? 0.f : expf(y - base);
      float sum = p;
#pragma unroll
      for (int off = 16; off >= 1; off /= 2) sum += __shfl_xor_sync(kFull, sum, off);
      m[r] = top;
      l[r] = fmaf(l[r], old, sum);
#pragma unroll
      for (int c = 0; c < C; ++c) o[r][c] *= old;
      sp[warp * kEach + r][lane] = p;
    }
    __syncwarp();
#pragma unroll 4
    for (int t = 0; t < count; ++t) {
      float v[C];
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = sv[t][lane + 32 * c];
#pragma unroll
      for (int r = 0; r < kEach; ++r) {
        const float p = sp[warp * kEach + r][t];
        if (seen[r] >> t & 1u) {               // what a row does not see may be anything
#pragma unroll
          for (int c = 0; c < C; ++c) o[r][c] = fmaf(p, v[c], o[r][c]);
        }
      }
    }
  }
#pragma unroll
  for (int x = 0; x < kEach; ++x) {
    const int r = row0 + warp * kEach + x;
    if (r >= nrows) break;
    if (a.nsplit == 1) {
      const float f = l[x] == 0.f ? 0.f : 1.f / l[x];
#pragma unroll
      for (int c = 0; c < C; ++c) ((T*)a.o)[out_row(r) * D + lane + 32 * c] = from_f<T>(l[x] == 0.f ? 0.f : o[x][c] * f);
    } else {
      const size_t at = out_row(r) * a.nsplit + split, all = (size_t)a.nseq * a.T * a.H * a.nsplit;
      if (lane == 0) reinterpret_cast<float2*>(a.part)[at] = make_float2(m[x], l[x]);
#pragma unroll
      for (int c = 0; c < C; ++c) a.part[part_outputs(all) + at * D + lane + 32 * c] = o[x][c];
    }
  }
}

// The parts of a row, a warp each: o = sum_s e^(m_s - m) o_s / sum_s e^(m_s - m) l_s.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) k_attn_join(const __grid_constant__ AttnArgs a) {
  constexpr int C = D / 32;
  const size_t rows = (size_t)a.nseq * a.T * a.H, row = (size_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (row >= rows) return;
  const float2* ml = reinterpret_cast<const float2*>(a.part) + row * a.nsplit;
  const float* part = a.part + part_outputs(rows * a.nsplit) + row * a.nsplit * D;
  float m = -INFINITY;
  bool failed = false;
  for (int s = lane; s < a.nsplit; s += 32) {
    const float2 v = ml[s];
    m = fmaxf(m, v.y == 0.f ? -INFINITY : v.x);
    failed |= v.y < 0.f;
  }
#pragma unroll
  for (int off = 16; off >= 1; off /= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
  if (__any_sync(kFull, failed)) return;       // reported; nothing is written
  float l = 0.f, o[C] = {};
#pragma unroll 8
  for (int s = 0; s < a.nsplit; ++s) {
    const float2 v = ml[s];
    const bool saw = v.y != 0.f;               // (one that saw nothing may have left its outputs unwritten)
    const float f = saw ? expf(v.x - m) : 0.f;
    l = fmaf(v.y, f, l);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float x = part[(size_t)s * D + lane + 32 * c];
      o[c] = fmaf(saw ? x : 0.f, f, o[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) ((T*)a.o)[row * D + lane + 32 * c] = from_f<T>(l == 0.f ? 0.f : o[c] / l);
}

template <typename T, int D>
cudaError_t verify(const AttnArgs& a, cudaStream_t s) {
  cudaError_t e;
  if (a.io == ERS_DTYPE_BF16) {
    e = attn_tiles(a, s);
  } else {
    const int tiles = (a.T * (a.H / a.KV) + kRows - 1) / kRows;
    k_attn_rows<D><<<dim3((unsigned)(a.nseq * a.nsplit), tiles * a.KV), 32 * kWarps, 0, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || a.nsplit == 1) return e;
  const size_t rows = (size_t)a.nseq * a.T * a.H, each = kThreads / 32;
  k_attn_join<T, D><<<(unsigned)((rows + each - 1) / each), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// ---- rows into pages ------------------------------------------------------------------------------------------
// Whether n tokens can be added to the slot: the table has room, and every page that they go to is the pool's and this slot's
// alone.  Decided by all threads together, the same in every CTA of a sequence.
__device__ __forceinline__ int32_t room_for(const AttnArgs& a, int i, const AttnSeq& s, int n) {
  int32_t err = ERS_OK;
  if (a.slot != nullptr)                       // a slot listed twice has two new ends
    for (int x = threadIdx.x; x < a.nseq; x += blockDim.x)
      if (x != i && a.slot[x] == s.slot) err = ERS_EINVAL;
  if (s.pos + (long long)n > (long long)a.slot_pages * a.page_tokens) {
    err = ERS_EOVERFLOW;
  } else if (n > 0) {
    const int first = page_of(a, s.pos), last = page_of(a, s.pos + n - 1);
    for (int x = first + threadIdx.x; x <= last; x += blockDim.x) {
      const int page = s.pages[x];
      if (page < 0 || page >= a.npages) err = ERS_ESLOT;
      else if (a.refs[page] != 1) err = ERS_EINVAL;
    }
  }
  return __syncthreads_or(err == ERS_EOVERFLOW) ? ERS_EOVERFLOW : __syncthreads_or(err == ERS_ESLOT) ? ERS_ESLOT
         : __syncthreads_or(err == ERS_EINVAL) ? ERS_EINVAL : ERS_OK;
}

// Rows [begin, end) of the new ones of a slot, source(r) each, both arrays, 16 bytes a thread.
template <typename F>
__device__ __forceinline__ void copy_rows(const AttnArgs& a, const AttnSeq& s, int begin, int end, F source) {
  const int pieces = a.KV * a.D * (a.io == ERS_DTYPE_BF16 ? 2 : 4) / 16;
  for (int e = threadIdx.x; e < (end - begin) * pieces; e += blockDim.x) {
    const int r = begin + e / pieces, x = e % pieces;
    const size_t from = (size_t)source(r) * pieces + x, to = (size_t)attn_row(a, s.pages, s.pos + r) * pieces + x;
    const uint4 k = __ldcs((const uint4*)a.k + from), v = __ldcs((const uint4*)a.v + from);
    ((uint4*)a.k_pages)[to] = k;
    ((uint4*)a.v_pages)[to] = v;
  }
}

// Whether the packed rows' borders ascend within [0, ntokens], all of them: blocks are found by them.  By all threads.
__device__ __forceinline__ bool ascending(const AttnArgs& a) {
  bool ok = true;
  for (int x = threadIdx.x; x < a.nseq; x += blockDim.x) {
    const int t0 = a.cu[x], t1 = a.cu[x + 1];
    ok &= 0 <= t0 && t0 <= t1 && t1 <= a.ntokens;
  }
  return __syncthreads_and(ok);
}

constexpr int kBlockRows = 16;                 // rows of a CTA

// Sequence i's blocks are numbers t0 / kBlockRows + i on: as many as there can be lie between those of two neighbours.
__global__ void __launch_bounds__(kThreads) k_attn_append(const __grid_constant__ AttnArgs a) {
  if (!ascending(a)) return;                   // the next launch reports what is wrong
  int lo = 0, hi = a.nseq - 1;                 // the last sequence whose blocks start at or before this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if ((long long)(a.cu[mid] / kBlockRows) + mid <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  AttnSeq s;
  const int t0 = a.cu[lo], n = a.cu[lo + 1] - t0;
  if (attn_seq(a, lo, &s) != ERS_OK) return;
  const long long first = ((long long)blockIdx.x - (t0 / kBlockRows + lo)) * kBlockRows;
  if (first < 0 || first >= n || room_for(a, lo, s, n) != ERS_OK) return;
  copy_rows(a, s, (int)first, min(n, (int)first + kBlockRows), [&](int r) { return t0 + r; });
}

__global__ void __launch_bounds__(kThreads) k_attn_advance(const __grid_constant__ AttnArgs a) {
  AttnSeq s;
  const int n = a.cu[blockIdx.x + 1] - a.cu[blockIdx.x];
  int32_t err = ascending(a) ? attn_seq(a, blockIdx.x, &s) : ERS_EINVAL;
  if (err == ERS_OK) err = room_for(a, blockIdx.x, s, n);
  if (threadIdx.x != 0) return;
  if (err != ERS_OK) report(a.status, err);
  else a.pos[s.slot] = s.pos + n;
}

__global__ void __launch_bounds__(kThreads) k_attn_commit(const __grid_constant__ AttnArgs a) {
  const int i = blockIdx.x, n = a.accepted[i];
  const int32_t* path = a.path != nullptr ? a.path + (size_t)i * a.T : nullptr;
  AttnSeq s;
  int32_t err = attn_seq(a, i, &s);
  if (err == ERS_OK && (n < 0 || n > a.T)) err = ERS_ECOMMIT;
  if (err == ERS_OK) err = room_for(a, i, s, n);
  bool bad = false;
  if (err == ERS_OK && path != nullptr)
    for (int t = threadIdx.x; t < n; t += blockDim.x) bad |= path[t] < 0 || path[t] >= a.T;
  if (__syncthreads_or(bad)) err = ERS_ECOMMIT;
  if (err != ERS_OK) {
    if (threadIdx.x == 0) report(a.status, err);
    return;
  }
  copy_rows(a, s, 0, n, [&](int r) { return (long long)i * a.T + (path != nullptr ? path[r] : r); });
  if (threadIdx.x == 0) a.pos[s.slot] = s.pos + n;               // read by all before the barriers above
}

}  // namespace

// Parts of a past: what takes the least time by a model in tiles of 64 tokens, each CTA some 4 beside its own, of as many CTAs
// as run at once (two a SM on the tensor cores, four of the fp32 kernel), and a quarter for each part that a row is joined
// of (bf16; a tile of the fp32 kernel takes much longer than that).  By 1, 2, 4, 8, 16, 32 and 64 parts, us:
//   1 x 32768 tokens 593, 310, 163, 89, 54, 41, 54 (38: 40)     8 x 8192, 4 drafts 156, 89, 57, 67, 79, 98, 138
//   1 x 1000 26, 20, 16, 15, 16 (6: 12.5)                       64 x 4096, 16 drafts 186, 220, 265, 339 (175 by 1 since)
//   16 x 4096, 64 drafts 105, 148, 183, 237                     fp32, 4 x up to 1000, 7 drafts 129, 69, 40, 26, 21
void attn_plan(AttnArgs* a, int max_len) {
  const bool tiles_of = a->io == ERS_DTYPE_BF16;
  const int each = tiles_of ? 128 : kRows, slots = tiles_of ? 304 : 608, rows = a->T * (a->H / a->KV);
  const long long units = (long long)a->nseq * a->KV * ((rows + each - 1) / each), tokens = max_len;
  const int blocks = (int)((tokens + 63) / 64);
  int per = blocks < 1 ? 1 : blocks;
  long long least = 0;
  for (int n = 1; n <= 64 && n <= blocks; ++n) {
    const int p = (blocks + n - 1) / n;
    const long long parts = (blocks + p - 1) / p, cost = (units * parts + slots - 1) / slots * (p + 4) * 4 + (tiles_of && parts > 1 ? parts : 0);
    if (n == 1 || cost < least) {
      least = cost;
      per = p;
    }
  }
  a->per = (int)(per > 0x1000000 ? 0x40000000 : per * 64);
  a->nsplit = blocks < 1 ? 1 : (blocks + per - 1) / per;
}

size_t attn_workspace(const AttnArgs& a) {
  const size_t all = (size_t)a.nseq * a.T * a.H * a.nsplit;
  return a.nsplit == 1 ? 0 : align256((part_outputs(all) + all * a.D) * sizeof(float));
}

cudaError_t attn_verify(const AttnArgs& a, cudaStream_t s) {
  if (a.io == ERS_DTYPE_BF16) return a.D == 64 ? verify<__nv_bfloat16, 64>(a, s) : verify<__nv_bfloat16, 128>(a, s);
  return a.D == 64 ? verify<float, 64>(a, s) : verify<float, 128>(a, s);
}

cudaError_t attn_append(const AttnArgs& a, cudaStream_t s) {
  if (a.ntokens > 0) {
    k_attn_append<<<(unsigned)(a.ntokens / kBlockRows + a.nseq), kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  k_attn_advance<<<a.nseq, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t attn_commit(const AttnArgs& a, cudaStream_t s) {
  k_attn_commit<<<a.nseq, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ers
