// Log probabilities of given tokens, entropy and top alternatives (include/ers.h).  Per row, with
// m = max_j x_j, d_j = scale (x_j - m), z = sum_j exp(d_j):
//   logprob = d_target - log z,  entropy = log z - sum_j exp(d_j) d_j / z
//
// One pass over the logits.  A thread keeps a running maximum m and, relative to r = m c (c = scale log2 e), the sums of
// 2^(x c - r) and of that times its exponent, two logits an instruction; threads, and the CTAs of a row's cluster where
// rows are few, are joined at the end.  For the alternatives a thread notes the maximum of every turn (kUnroll vectors) in
// shared memory: the k-th largest of the maxima of 64 disjoint parts is a lower bound of the k-th best logit, so the turns
// that reach it, about 1.2 k of them, are read again by the threads that noted them and what reaches it is ranked.
// Should the candidates overflow, the k-th best of those found is a better bound, and the turns are read once more.  (A
// maximum per warp and segment, the segments then read again by whole warps, cost 130 us where this costs 117.)
//
// x c - r is exact to one rounding while the rounding of r itself, half a unit of |m c|, is a small exponent.  So logits
// below a floor of -kFar / c count as the floor in that pass (-inf times a weight of nothing would be NaN as well), whatever a
// thread's own maximum, and a row whose maximum is not far above the floor, or is above kFar / c, is read once more and
// summed with (x - m) scale in place of x c - r.
//
// What bounds it: 2 (4) bytes a logit from memory; 152 SMs at 6.8 TB/s leave 10.9 issue slots a bf16 logit, of
// which it takes 6.  2048 x 131072 bf16: 88 us (90 % of the measured bandwidth) without alternatives, 111 with 5 and 117 with
// 20 (68 %): the notes, and that a CTA that chooses (reads, counts and ranks in turn) streams nothing meanwhile.  Rows of
// equals, which overflow the candidates, cost twice a plain row's time (515 x 32000 bf16: 26 us against 15).
#include <math.h>
#include <string.h>

#include "ers_common.cuh"
#include "ers_internal.h"
#include "f32x2.cuh"
#include "tc_common.cuh"

namespace ers {
namespace {

constexpr int kWarps = kThreads / 32;
constexpr int kNotes = 32;           // maxima that a thread notes
constexpr int kCandidates = 128;     // (256: the same but for rows of equals, 33 us)
constexpr int kMaxSplit = 8;         // CTAs of a row
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

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

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN stays one
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The largest |x c| of the one pass, and how far a row's maximum has to be above the floor (in exponents: nothing is left of
// the floor then).
constexpr float kFar = 1048576.f, kAbove = 256.f;
constexpr float kMost = 3.4028235e38f, kLowest = -3.3895314e38f;   // the largest float, the lowest bf16 number

template <typename T> struct Vec;   // 16 bytes of logits
template <> struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
  template <int N>
  static __device__ __forceinline__ float top(const uint4 (&r)[N]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(r[i].x), __uint_as_float(r[i].y)), fmaxf(__uint_as_float(r[i].z), __uint_as_float(r[i].w))));
    return m;
  }
  // at least the floor, in pairs
  static __device__ __forceinline__ void raised(const uint4& r, float floor, uint64_t (&x)[2]) {
    x[0] = pair(max_nan(__uint_as_float(r.x), floor), max_nan(__uint_as_float(r.y), floor));
    x[1] = pair(max_nan(__uint_as_float(r.z), floor), max_nan(__uint_as_float(r.w), floor));
  }
  static __device__ __forceinline__ float at(const uint4& r, int e) { return __uint_as_float(e < 2 ? e < 1 ? r.x : r.y : e < 3 ? r.z : r.w); }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
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
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  template <int N>
  static __device__ __forceinline__ float top(const uint4 (&r)[N]) {
    __nv_bfloat162 m = __hmax2(__hmax2(two(r[0].x), two(r[0].y)), __hmax2(two(r[0].z), two(r[0].w)));
#pragma unroll
    for (int i = 1; i < N; ++i)
      m = __hmax2(m, __hmax2(__hmax2(two(r[i].x), two(r[i].y)), __hmax2(two(r[i].z), two(r[i].w))));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void raised(const uint4& r, float floor, uint64_t (&x)[4]) {   // (floor: a bf16 number)
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    const __nv_bfloat162 least = __float2bfloat162_rn(floor);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __hmax2_nan(two(w[i]), least);
      const uint32_t u = *reinterpret_cast<const uint32_t*>(&v);
      x[i] = pair(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
  }
  static __device__ __forceinline__ float at(const uint4& r, int e) {
    const uint32_t w = e < 4 ? e < 2 ? r.x : r.y : e < 6 ? r.z : r.w;
    return __uint_as_float(e % 2 == 0 ? w << 16 : w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {   // of values that are bf16 already
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(x[2 * i]) >> 16 | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A row as 16-byte vectors from the last aligned address at or before its start: element e of vector v is logit
// v * n + e - shift.
template <typename T>
struct Row {
  const T* base;
  int shift, vocab;
  int whole0, whole1;   // vectors [whole0, whole1) lie within the row
  __device__ __forceinline__ Row(const T* x, int vocab_) : vocab(vocab_) {
    shift = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    base = x - shift;
    whole0 = shift == 0 ? 0 : 1;
    whole1 = (int)(((long long)vocab + shift) / Vec<T>::n);
  }
  __device__ __forceinline__ int vectors() const { return (int)(((long long)vocab + shift + Vec<T>::n - 1) / Vec<T>::n); }
  __device__ __forceinline__ bool whole(int v) const { return v >= whole0 && v < whole1; }
  __device__ __forceinline__ uint4 load(int v) const {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(base + (long long)v * Vec<T>::n));
    return r;
  }
  // a vector that the row does not fill: -inf outside
  __device__ __forceinline__ uint4 edge(int v) const {
    float x[Vec<T>::n];
#pragma unroll
    for (int e = 0; e < Vec<T>::n; ++e) {
      const long long j = (long long)v * Vec<T>::n + e - shift;
      x[e] = j >= 0 && j < vocab ? to_f(base[j + shift]) : -INFINITY;
    }
    return Vec<T>::pack(x);
  }
  __device__ __forceinline__ uint4 get(int v) const { return whole(v) ? load(v) : edge(v); }
};

// z = sum 2^(u) and zu = sum 2^(u) u, u = x c - r (or, of the rows that are read again, (x - m) scale log2 e with r = 0)
struct Sums {
  float r, z, zu;
  __device__ __forceinline__ void raise(float to) {
    const float f = exp2_fast(r - to);
    zu = f > 0.f ? f * fmaf(z, r - to, zu) : 0.f;
    z *= f;
    r = to;
  }
  __device__ __forceinline__ void join(const Sums& o) {
    Sums u = o;
    if (u.r > r) raise(u.r);
    else u.raise(r);
    z += u.z;
    zu += u.zu;
  }
  __device__ __forceinline__ Sums across(int off) const {
    return {__shfl_xor_sync(kFull, r, off), __shfl_xor_sync(kFull, z, off), __shfl_xor_sync(kFull, zu, off)};
  }
};

struct Shared {
  Sums sums[kWarps];
  float top[kWarps];
  int part[64];              // maxima of the parts: four threads each
  unsigned long long candidates[kCandidates];
  int count;
  unsigned long long best[ERS_TOP_MAX];
  // of the row's first CTA: what all of them found
  Sums all_sums[kMaxSplit], again[kMaxSplit];
  float all_top[kMaxSplit];   // of every CTA
  unsigned long long all_best[kMaxSplit * ERS_TOP_MAX];
  float notes[kNotes][kThreads];   // of each thread
};

template <typename V>
__device__ __forceinline__ V* at_cta(V* p, int rank) {   // the same object of the cluster's rank-th CTA, which has to be running
  uint64_t r;
  asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
  return reinterpret_cast<V*>(r);
}
template <typename V>
__device__ __forceinline__ V* at_first(V* p) { return at_cta(p, 0); }

// best[0..k), zeros before: the k best of n distinct keys, best first (zeros count as none).  All threads; ends with a barrier.
__device__ __forceinline__ void rank_keys(const unsigned long long* keys, int n, unsigned long long* best, int k) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long mine = keys[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > mine;
    if (rank < k && mine != 0) best[rank] = mine;
  }
  __syncthreads();
}
// The sums of all warps, in the first one's threads.
__device__ __forceinline__ Sums join_warps(const Sums* sums) {
  Sums s = sums[threadIdx.x % kWarps];
#pragma unroll
  for (int off = kWarps / 2; off >= 1; off >>= 1) s.join(s.across(off));
  return s;
}

template <typename T, bool tops>
__global__ void __launch_bounds__(kThreads, 4) k_token_logprobs(LogprobArgs a, int split) {
  constexpr int n = Vec<T>::n;
  // Vectors that a thread has under way while it works on as many (2048 x 131072: 2 take 102 us, 3 92, 4 88; with 20
  // alternatives 3 take 117 and 4 124).
  constexpr int kUnroll = tops ? 3 : 4;
  __shared__ Shared sh;
  const int row = blockIdx.x / split, rank = blockIdx.x % split;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (split > 1) tc::cluster_arrive();   // this CTA runs: waited for before anything is written to another's shared memory
  const T* x0 = (const T*)a.logits + (long long)row * a.stride;
  const Row<T> x(x0, a.vocab);
  const int segs = (x.vectors() + 31) / 32;
  const int per = (segs + split - 1) / split;
  const int s0 = min(rank * per, segs), s1 = min(s0 + per, segs);
  // A thread notes the maximum of each of its turns, or of each `group` turns of a long row.
  constexpr int kTurn = kWarps * kUnroll;        // segments of a turn
  const int group = (s1 - s0 + kTurn * kNotes - 1) / (kTurn * kNotes);
  const float c = a.c, floor = a.floor;

  // ---- one pass ------------------------------------------------------------------------------------------------------
  const float r0 = floor * c;
  float top = -INFINITY;                    // the thread's maximum
  float r = r0;
  uint64_t z2 = 0, zu2 = 0;                 // two zeros each
  const uint64_t c2 = pair(c, c);
  uint4 next[kUnroll];
  int noted = 0, since = 0;                 // the thread's notes, turns in the last one
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int seg = s0 + warp + u * kWarps;
    next[u] = next[0];
    if (seg < s1) next[u] = x.get(seg * 32 + lane);
  }
#pragma unroll 1
  for (int g = s0 + warp; g < s1; g += kTurn) {
    // The vectors of this turn.  Those that the row ends before are the thread's own of an earlier one or of this one, so
    // they change no maximum but at most a note's, which then sends one reader in vain.
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      raw[u] = next[u];
      const int seg = g + (u + kUnroll) * kWarps;
      if (seg < s1) next[u] = x.get(seg * 32 + lane);
    }
    const float t = Vec<T>::top(raw);
    if (tops) {
      if (since == 0) sh.notes[noted++][threadIdx.x] = t;
      else sh.notes[noted - 1][threadIdx.x] = fmaxf(sh.notes[noted - 1][threadIdx.x], t);
      if (++since == group) since = 0;
    }
    if (t > top) {
      top = t;
      const float to = fmaxf(t, floor) * c;
      float za, zb, ua, ub;
      unpair(z2, za, zb);
      unpair(zu2, ua, ub);
      Sums s = {r, za + zb, ua + ub};
      s.raise(to);
      r = to;
      z2 = pair(s.z, 0.f);
      zu2 = pair(s.zu, 0.f);
    }
    const uint64_t r2 = pair(-r, -r);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (g + u * kWarps >= s1) break;
      uint64_t y[n / 2];
      Vec<T>::raised(raw[u], floor, y);
#pragma unroll
      for (int e = 0; e < n / 2; ++e) {
        const uint64_t w = fma2(y[e], c2, r2);
        float wa, wb;
        unpair(w, wa, wb);
        const uint64_t p = pair(exp2_fast(wa), exp2_fast(wb));
        z2 = add2(z2, p);
        zu2 = fma2(p, w, zu2);
      }
    }
  }
  float za, zb, ua, ub;
  unpair(z2, za, zb);
  unpair(zu2, ua, ub);
  Sums s = {r, za + zb, ua + ub};
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    s.join(s.across(off));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    if (tops && off == 2 && lane % 4 == 0) sh.part[threadIdx.x / 4] = order_of(top);
  }
  if (lane == 0) {
    sh.sums[warp] = s;
    sh.top[warp] = top;
  }
  if (tops && threadIdx.x < ERS_TOP_MAX) sh.best[threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  top = sh.top[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sh.top[w]);
  if (warp == 0) s = join_warps(sh.sums);

  // ---- this CTA's best -------------------------------------------------------------------------------------------------
  if (tops) {
    const int k = a.top_k, nothing = order_of(-INFINITY);
    // a bound: the upper 16 bits of the k-th largest of the parts' maxima
    const unsigned upper0 = ((unsigned)sh.part[lane] ^ 0x80000000u) >> 16, upper1 = ((unsigned)sh.part[32 + lane] ^ 0x80000000u) >> 16;
    unsigned least = 0;
#pragma unroll
    for (int b = 15; b >= 0; --b) {
      const unsigned with = least | 1u << b;
      if (__popc(__ballot_sync(kFull, upper0 >= with)) + __popc(__ballot_sync(kFull, upper1 >= with)) >= k) least = with;
    }
    unsigned long long bound = (unsigned long long)least << 48;
    for (;;) {
      const int from = max(key_order(bound), nothing + 1);
      const float least_of = value_of(from);                  // (a NaN reaches nothing)
      unsigned hits = 0;                                      // the thread's notes that reach the bound
#pragma unroll 4
      for (int i = 0; i < noted; ++i) {
        const int o = order_of(sh.notes[i][threadIdx.x]);
        // (among equals of the bound, only what comes before it)
        const int first = ((s0 + i * group * kTurn + warp) * 32 + lane) * n - x.shift;
        if (o >= from && (o > key_order(bound) || (unsigned)max(first, 0) <= (unsigned)key_index(bound))) hits |= 1u << i;
      }
#pragma unroll 1
      while (hits != 0) {
        const int begin = s0 + (__ffs(hits) - 1) * group * kTurn + warp;
        hits &= hits - 1;
#pragma unroll 1
        for (int g = begin; g < min(begin + group * kTurn, s1); g += kTurn) {
          if (*(volatile int*)&sh.count > kCandidates) break;   // there will be another time
          uint4 raw[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u)
            if (g + u * kWarps < s1) raw[u] = x.get((g + u * kWarps) * 32 + lane);
          unsigned which = 0;                                 // of their logits, those that do
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            if (g + u * kWarps >= s1) break;
            float y[n];
            Vec<T>::unpack(raw[u], y);
#pragma unroll
            for (int e = 0; e < n; ++e)
              if (y[e] >= least_of) which |= 1u << (u * n + e);
          }
#pragma unroll 1
          while (which != 0 && *(volatile int*)&sh.count <= kCandidates) {
            const int w = __ffs(which) - 1, e = w % n;
            which &= which - 1;
            uint4 v = raw[0];
#pragma unroll
            for (int u = 1; u < kUnroll; ++u)
              if (w / n == u) v = raw[u];
            const unsigned long long key =
                key_of(order_of(Vec<T>::at(v, e)), ((g + w / n * kWarps) * 32 + lane) * n + e - x.shift);
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
      __syncthreads();
      if (threadIdx.x < ERS_TOP_MAX) sh.best[threadIdx.x] = 0;
      if (threadIdx.x == 0) sh.count = 0;
      __syncthreads();
    }
  }

  // ---- the row ---------------------------------------------------------------------------------------------------------
  if (split > 1) {
    __syncwarp();
    tc::cluster_wait();
    if (threadIdx.x < split) at_cta(sh.all_top, threadIdx.x)[rank] = top;
    if (threadIdx.x == 0) at_first(sh.all_sums)[rank] = s;
    if (tops && threadIdx.x < a.top_k) at_first(sh.all_best)[rank * a.top_k + threadIdx.x] = sh.best[threadIdx.x];
    __syncwarp();
    tc::cluster_sync();
    for (int q = 0; q < split; ++q) top = fmaxf(top, sh.all_top[q]);
  }
  const float most_c = top * c;
  const bool again = fabsf(top) < INFINITY && !(fabsf(most_c) < kFar && most_c - r0 >= kAbove && a.scale * kLog2e <= kMost);
  // (x - m) scale, the difference halved where scale < 1 would bring one that overflows back
  const float half = a.scale < 1.f ? 0.5f : 1.f, by = a.scale / half, half_top = half * top;
  if (again) {
    s = {0.f, 0.f, 0.f};
    for (int v = s0 * 32 + threadIdx.x; v < s1 * 32; v += kThreads * kUnroll) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) raw[u] = x.get(v + u * kThreads);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (v + u * kThreads >= s1 * 32) break;
        float y[n];
        Vec<T>::unpack(raw[u], y);
#pragma unroll
        for (int e = 0; e < n; ++e) {
          const float w = fmaf(y[e], half, -half_top) * by * kLog2e, p = exp2_fast(w);
          s.z += p;
          if (!(p == 0.f)) s.zu = fmaf(p, w, s.zu);
        }
      }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s.join(s.across(off));
    __syncthreads();
    if (lane == 0) sh.sums[warp] = s;
    __syncthreads();
    if (warp == 0) s = join_warps(sh.sums);
    if (split > 1) {
      if (threadIdx.x == 0) at_first(sh.again)[rank] = s;
      __syncwarp();
      tc::cluster_sync();
    }
  }
  if (rank != 0) return;
  if (split > 1) {
    const Sums* all = again ? sh.again : sh.all_sums;
    s = all[0];
    for (int q = 1; q < split; ++q) s.join(all[q]);
    if (tops) {
      __syncthreads();
      if (threadIdx.x < ERS_TOP_MAX) sh.best[threadIdx.x] = 0;
      __syncthreads();
      rank_keys(sh.all_best, split * a.top_k, sh.best, a.top_k);
    }
  }
  if (warp != 0) return;
  const bool none = !(s.z < INFINITY) || top == INFINITY, empty = top == -INFINITY && !none;
  // r is the maximum's x c but for its rounding
  const float log_z = logf(s.z), most = (again ? 0.f : fmaf(top, c, -s.r) * kLn2) - log_z;
  const auto logprob = [&](float v) { return fmaf(fmaf(v, half, -half_top), by, most); };
  if (threadIdx.x == 0) {
    if (a.logprob != nullptr) {
      const int t = a.target[row];
      float lp = 0.f;
      if (t < -1 || t >= a.vocab) {
        report(a.status, ERS_EINVAL);
        lp = NAN;
      } else if (t >= 0) {
        lp = none ? NAN : empty ? -INFINITY : logprob(to_f(x0[t]));
      }
      a.logprob[row] = lp;
    }
    if (a.entropy != nullptr) a.entropy[row] = none ? NAN : empty ? 0.f : log_z - kLn2 * s.zu / s.z;
  }
  if (tops && threadIdx.x < a.top_k) {
    const unsigned long long key = sh.best[threadIdx.x];
    const bool gone = none || key == 0;
    const size_t at = (size_t)row * a.top_k + threadIdx.x;
    a.top_id[at] = gone ? -1 : key_index(key);
    a.top_logprob[at] = none ? NAN : gone ? -INFINITY : logprob(value_of(key_order(key)));
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

cudaError_t token_logprobs(const LogprobArgs& args, cudaStream_t s) {
  LogprobArgs a = args;
  a.c = fminf(a.scale * kLog2e, kMost);
  a.floor = __bfloat162float(__float2bfloat16_rn(fmaxf(-kFar / a.c, kLowest)));
  // A row is split while that leaves SMs without two CTAs, down to 8 KB a CTA.  131072 bf16 logits, 8 alternatives: 1 row 16.2 us
  // whole, 10.1 split; 100 rows by up to 152, 304 and 608 CTAs 15.5, 15.1, 20.3; 200 rows 21.2, 18.7, 23.3; 300 rows
  // 22.4, 23.3, 31.0.  8192 logits: 6.5 by one CTA or two.
  const long long bytes = (long long)a.vocab * (a.io == ERS_DTYPE_BF16 ? 2 : 4);
  int split = 1;
  while (split < kMaxSplit && (long long)a.nrows * split < 304 && bytes / (2 * split) >= 8192) split *= 2;
  if (a.nrows > 0x7fffffff / kMaxSplit) split = 1;
  if (a.io == ERS_DTYPE_BF16)
    return a.top_k > 0 ? launch<__nv_bfloat16, true>(a, split, s) : launch<__nv_bfloat16, false>(a, split, s);
  return a.top_k > 0 ? launch<float, true>(a, split, s) : launch<float, false>(a, split, s);
}

}  // namespace ers
