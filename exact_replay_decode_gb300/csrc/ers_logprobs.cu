// Log probabilities of given tokens, entropy and top alternatives (include/ers.h).  Per row, with
// m = max_j x_j, d_j = scale (x_j - m), z = sum_j exp(d_j):
//   logprob = d_target - log z,  entropy = log z - sum_j exp(d_j) d_j / z
//
// One pass over the logits.  A thread keeps a running maximum and, relative to it, the sums of exp(d) and exp(d) d; threads,
// and the CTAs of a row's cluster where rows are few, are joined at the end.  For the alternatives the pass only notes the
// maximum of each segment (a warp's 512 bytes): the k-th largest of 256 maxima over disjoint parts is a lower bound of the
// k-th best logit, so the segments that reach it, little more than k of them, are read again (from L2) and what reaches it
// is ranked.  Should the candidates overflow, the k-th best of those found is a better bound, and the segments are read once
// more.
//
// What bounds it: 2 (4) bytes a logit from memory; 152 SMs at 6.8 TB/s leave 10.9 issue slots a bf16 logit, of which it takes 7.
#include <limits.h>
#include <math.h>
#include <string.h>

#include "ers_common.cuh"
#include "ers_internal.h"
#include "tc_common.cuh"

namespace ers {
namespace {

constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;           // segments a warp has under way
constexpr int kSegs = 2048;          // segment maxima of a CTA
constexpr int kCandidates = 512;
constexpr int kMaxSplit = 8;         // CTAs of a row
constexpr float kLog2e = 1.44269504f;

// values in order as whole numbers; -0 and +0 are equal
__device__ __forceinline__ int order_of(float x) {
  const int b = __float_as_int(x + 0.f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }
// (value, lowest index first) as one whole number: larger is better, 0 is below all
__device__ __forceinline__ unsigned long long key_of(int order, int j) {
  return ((unsigned long long)((unsigned)order ^ 0x80000000u) << 32) | (0xffffffffu - (unsigned)j);
}
__device__ __forceinline__ int key_order(unsigned long long k) { return (int)((unsigned)(k >> 32) ^ 0x80000000u); }
__device__ __forceinline__ int key_index(unsigned long long k) { return (int)(0xffffffffu - (unsigned)k); }

__device__ __forceinline__ float exp2_fast(float x) {   // 2 units in the last place, 0 below -126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T> struct Vec;   // 16 bytes of logits
template <> struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// A row as 16-byte vectors from the last aligned address at or before its start: element e of vector v is logit
// v * n + e - shift.
template <typename T>
struct Row {
  const T* base;
  int shift, vocab;
  __device__ __forceinline__ int vectors() const { return (int)(((long long)vocab + shift + Vec<T>::n - 1) / Vec<T>::n); }
  __device__ __forceinline__ bool whole(int v) const {
    return (v > 0 || shift == 0) && ((long long)v + 1) * Vec<T>::n <= (long long)vocab + shift;
  }
  __device__ __forceinline__ uint4 load(int v) const {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(base + (long long)v * Vec<T>::n));
    return r;
  }
  // a vector that the row does not fill: -inf outside
  __device__ __forceinline__ void edge(int v, float (&x)[Vec<T>::n]) const {
#pragma unroll
    for (int e = 0; e < Vec<T>::n; ++e) {
      const long long j = (long long)v * Vec<T>::n + e - shift;
      x[e] = j >= 0 && j < vocab ? to_f(base[j + shift]) : -INFINITY;
    }
  }
  __device__ __forceinline__ void get(int v, float (&x)[Vec<T>::n]) const {
    if (whole(v)) Vec<T>::unpack(load(v), x);
    else edge(v, x);
  }
};

// exp(d) and exp(d) d relative to m, in the units of x (d = c (x - m) is taken to base 2: c = scale log2 e)
struct Sums {
  float m, z, zd;
  __device__ __forceinline__ void raise(float to, float c) {
    if (z != 0.f) {
      const float f = exp2_fast((m - to) * c);
      zd = f > 0.f ? f * fmaf(z, m - to, zd) : 0.f;
      z *= f;
    }
    m = to;
  }
  __device__ __forceinline__ void join(const Sums& o, float c) {
    Sums u = o;
    if (u.m > m) raise(u.m, c);
    else u.raise(m, c);
    z += u.z;
    zd += u.zd;
  }
};

struct Shared {
  Sums sums[kWarps];
  int part_max[kThreads];
  unsigned long long candidates[kCandidates];
  int count;
  unsigned long long best[ERS_TOP_MAX];
  // of the row's first CTA: what all of them found
  Sums all_sums[kMaxSplit];
  unsigned long long all_best[kMaxSplit * ERS_TOP_MAX];
  int seg_max[kSegs];
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <typename V>
__device__ __forceinline__ V* at_first(V* p) {   // the same object of the cluster's first CTA
  uint64_t r;
  asm("mapa.u64 %0, %1, 0;" : "=l"(r) : "l"(p));
  return reinterpret_cast<V*>(r);
}

// The k best of n distinct keys in place of rank order into best[0..k), 0 beyond n.  All threads.
__device__ __forceinline__ void rank_keys(const unsigned long long* keys, int n, unsigned long long* best, int k) {
  if (threadIdx.x < k) best[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long mine = keys[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > mine;
    if (rank < k && mine != 0) best[rank] = mine;
  }
  __syncthreads();
}

template <typename T, bool tops>
__global__ void __launch_bounds__(kThreads, 4) k_token_logprobs(LogprobArgs a, int split) {
  constexpr int n = Vec<T>::n;
  __shared__ Shared sh;
  const int row = blockIdx.x / split, rank = blockIdx.x % split;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const T* x0 = (const T*)a.logits + (long long)row * a.stride;
  Row<T> x;
  x.shift = (int)((reinterpret_cast<uintptr_t>(x0) & 15u) / sizeof(T));
  x.base = x0 - x.shift;
  x.vocab = a.vocab;
  const int vectors = x.vectors(), segs = (vectors + 31) / 32;
  const int per = (segs + split - 1) / split;
  const int s0 = min(rank * per, segs), s1 = min(s0 + per, segs);
  const int group = (per + kSegs - 1) / kSegs;   // segments behind one noted maximum
  const int noted = (s1 - s0 + group - 1) / group;
  const float c = a.scale * kLog2e;
  if (tops && group > 1) {
    for (int i = threadIdx.x; i < noted; i += kThreads) sh.seg_max[i] = INT_MIN;
    __syncthreads();
  }

  // ---- one pass ------------------------------------------------------------------------------------------------------
  Sums s = {-3.402823466e38f, 0.f, 0.f};
  for (int g = s0 + warp; g < s1; g += kWarps * kUnroll) {
    uint4 raw[kUnroll];
    bool whole[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int seg = g + u * kWarps, v = seg * 32 + lane;
      whole[u] = seg < s1 && x.whole(v);
      if (whole[u]) raw[u] = x.load(v);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int seg = g + u * kWarps, v = seg * 32 + lane;
      if (seg >= s1) break;
      float y[n];
      if (whole[u]) Vec<T>::unpack(raw[u], y);
      else x.edge(v, y);
      float top = y[0];
#pragma unroll
      for (int e = 1; e < n; ++e) top = fmaxf(top, y[e]);
      if (top > s.m) s.raise(top, c);
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const float d = y[e] - s.m, t = exp2_fast(d * c);
        s.z += t;
        s.zd = fmaf(t, fmaxf(d, -1e30f), s.zd);   // exp(-inf) times -inf is nothing
      }
      if (tops) {
        const int o = __reduce_max_sync(kFull, order_of(top));
        if (lane == 0) {
          if (group == 1) sh.seg_max[seg - s0] = o;
          else atomicMax(&sh.seg_max[(seg - s0) / group], o);
        }
      }
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const Sums o = {__shfl_xor_sync(kFull, s.m, off), __shfl_xor_sync(kFull, s.z, off), __shfl_xor_sync(kFull, s.zd, off)};
    s.join(o, c);
  }
  if (lane == 0) sh.sums[warp] = s;
  __syncthreads();
  s = sh.sums[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s.join(sh.sums[w], c);

  // ---- this CTA's best -------------------------------------------------------------------------------------------------
  if (tops) {
    const int k = a.top_k;
    int part = INT_MIN;
    for (int i = threadIdx.x; i < noted; i += kThreads) part = max(part, sh.seg_max[i]);
    sh.part_max[threadIdx.x] = part;
    if (threadIdx.x == 0) sh.best[0] = 0;
    __syncthreads();
    int above = 0;
    for (int i = 0; i < kThreads; ++i) {
      const int o = sh.part_max[i];
      above += o > part || (o == part && i < threadIdx.x);
    }
    // a bound in key order: (k-th part's maximum, any index)
    if (above == k - 1) sh.best[0] = (unsigned long long)((unsigned)part ^ 0x80000000u) << 32;
    __syncthreads();
    unsigned long long bound = sh.best[0];
    const int nothing = order_of(-INFINITY);
    for (;;) {
      __syncthreads();
      if (threadIdx.x == 0) sh.count = 0;
      __syncthreads();
      const int least = key_order(bound);
      for (int i = warp; i < noted; i += kWarps) {
        if (sh.seg_max[i] < least || sh.seg_max[i] <= nothing) continue;
        for (int seg = s0 + i * group; seg < min(s0 + (i + 1) * group, s1); ++seg) {
          const int v = seg * 32 + lane;
          if (v >= vectors) continue;
          float y[n];
          x.get(v, y);
#pragma unroll
          for (int e = 0; e < n; ++e) {
            const int o = order_of(y[e]);
            if (o < least || !(y[e] > -INFINITY)) continue;
            const unsigned long long key = key_of(o, v * n + e - x.shift);
            if (key >= bound) {
              const int at = atomicAdd(&sh.count, 1);
              if (at < kCandidates) sh.candidates[at] = key;
            }
          }
        }
      }
      __syncthreads();
      const int found = sh.count;
      rank_keys(sh.candidates, min(found, kCandidates), sh.best, k);
      if (found <= kCandidates) break;
      bound = sh.best[k - 1];
    }
  }

  // ---- the row ---------------------------------------------------------------------------------------------------------
  const unsigned long long* best = sh.best;
  if (split > 1) {
    if (threadIdx.x == 0) at_first(sh.all_sums)[rank] = s;
    if (tops && threadIdx.x < ERS_TOP_MAX)
      at_first(sh.all_best)[rank * ERS_TOP_MAX + threadIdx.x] = threadIdx.x < a.top_k ? sh.best[threadIdx.x] : 0;
    cluster_sync();
    if (rank != 0) return;
    s = sh.all_sums[0];
    for (int r = 1; r < split; ++r) s.join(sh.all_sums[r], c);
    if (tops) rank_keys(sh.all_best, split * ERS_TOP_MAX, sh.best, a.top_k);
  }
  const bool none = !(s.z < INFINITY), empty = s.z == 0.f;   // z is at least 1 where anything is left
  const float log_z = logf(s.z);
  if (threadIdx.x == 0) {
    if (a.logprob != nullptr) {
      const int t = a.target[row];
      float lp = 0.f;
      if (t < -1 || t >= a.vocab) {
        report(a.status, ERS_EINVAL);
        lp = NAN;
      } else if (t >= 0) {
        lp = none ? NAN : empty ? -INFINITY : a.scale * (to_f(x0[t]) - s.m) - log_z;
      }
      a.logprob[row] = lp;
    }
    if (a.entropy != nullptr) a.entropy[row] = none ? NAN : empty ? 0.f : log_z - a.scale * s.zd / s.z;
  }
  if (tops && threadIdx.x < a.top_k) {
    const unsigned long long key = best[threadIdx.x];
    const bool gone = none || key == 0;
    const size_t at = (size_t)row * a.top_k + threadIdx.x;
    a.top_id[at] = gone ? -1 : key_index(key);
    a.top_logprob[at] = none ? NAN : gone ? -INFINITY : a.scale * (value_of(key_order(key)) - s.m) - log_z;
  }
}

template <typename T, bool tops>
cudaError_t launch(const LogprobArgs& a, int split, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)a.nrows * (unsigned)split);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_token_logprobs<T, tops>, a, split);
}

}  // namespace

cudaError_t token_logprobs(const LogprobArgs& a, cudaStream_t s) {
  // A row is split while that leaves SMs without a CTA, down to 8 KB a CTA.
  const long long bytes = (long long)a.vocab * (a.io == ERS_DTYPE_BF16 ? 2 : 4);
  int split = 1;
  while (split < kMaxSplit && (long long)a.nrows * split < 304 && bytes / (2 * split) >= 8192) split *= 2;
  if (a.nrows > 0x7fffffff / kMaxSplit) split = 1;
  if (a.io == ERS_DTYPE_BF16)
    return a.top_k > 0 ? launch<__nv_bfloat16, true>(a, split, s) : launch<__nv_bfloat16, false>(a, split, s);
  return a.top_k > 0 ? launch<float, true>(a, split, s) : launch<float, false>(a, split, s);
}

}  // namespace ers
