// Log probabilities of given tokens, entropy and top alternatives (include/ers.h).  Per row, with
// m = max_j x_j, d_j = scale (x_j - m), z = sum_j exp(d_j):
//   logprob = d_target - log z,  entropy = log z - sum_j exp(d_j) d_j / z
#include <math.h>

#include "ers_common.cuh"
#include "ers_internal.h"

namespace ers {
namespace {

// The order of (value, lowest index first) as one whole number: larger is better.  -0 and +0 are equal.
__device__ __forceinline__ unsigned long long order_key(float x, int j) {
  const int b = __float_as_int(x + 0.f);
  const unsigned u = (unsigned)(b ^ ((b >> 31) & 0x7fffffff)) ^ 0x80000000u;
  return ((unsigned long long)u << 32) | (0xffffffffu - (unsigned)j);
}

template <typename V, typename F>
__device__ __forceinline__ V block_reduce(V v, V* scratch, F f) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = f(v, __shfl_xor_sync(kFull, v, off));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = scratch[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v = f(v, scratch[w]);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_token_logprobs(LogprobArgs a) {
  __shared__ float fs[kThreads / 32];
  __shared__ unsigned long long ks[kThreads / 32];
  const auto add = [](float u, float v) { return u + v; };
  const auto top = [](unsigned long long u, unsigned long long v) { return u > v ? u : v; };
  for (int row = blockIdx.x; row < a.nrows; row += gridDim.x) {
    const T* x = (const T*)a.logits + (long long)row * a.stride;
    float m = -INFINITY, odd = 0.f;
    for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
      const float v = to_f(x[j]);
      m = fmaxf(m, v);
      if (!(v < INFINITY)) odd = 1.f;
    }
    m = block_reduce(m, fs, [](float u, float v) { return fmaxf(u, v); });
    const bool none = block_reduce(odd, fs, add) > 0.f;    // a NaN or +inf: no distribution
    const bool empty = m == -INFINITY;
    float z = 0.f, zd = 0.f;
    if (!none && !empty) {
      for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
        const float d = a.scale * (to_f(x[j]) - m), e = expf(d);
        z += e;
        if (e > 0.f) zd = fmaf(e, d, zd);
      }
    }
    z = block_reduce(z, fs, add);
    zd = block_reduce(zd, fs, add);
    const float log_z = logf(z);
    if (threadIdx.x == 0) {
      if (a.logprob != nullptr) {
        const int t = a.target[row];
        float lp = 0.f;
        if (t < -1 || t >= a.vocab) {
          report(a.status, ERS_EINVAL);
          lp = NAN;
        } else if (t >= 0) {
          lp = none ? NAN : empty ? -INFINITY : a.scale * (to_f(x[t]) - m) - log_z;
        }
        a.logprob[row] = lp;
      }
      if (a.entropy != nullptr) a.entropy[row] = none ? NAN : empty ? 0.f : log_z - zd / z;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < a.top_k; ++k) {
      unsigned long long best = 0;
      for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
        const unsigned long long key = order_key(to_f(x[j]), j);
        if (key < last && key > best) best = key;
      }
      best = block_reduce(best, ks, top);
      last = best;
      if (threadIdx.x == 0) {
        const int j = (int)(0xffffffffu - (unsigned)best);
        const float v = best != 0 ? to_f(x[j]) : -INFINITY;
        const bool gone = none || v == -INFINITY;
        a.top_id[(size_t)row * a.top_k + k] = gone ? -1 : j;
        a.top_logprob[(size_t)row * a.top_k + k] = none ? NAN : gone ? -INFINITY : a.scale * (v - m) - log_z;
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t token_logprobs(const LogprobArgs& a, cudaStream_t s) {
  if (a.io == ERS_DTYPE_BF16) k_token_logprobs<__nv_bfloat16><<<a.nrows, kThreads, 0, s>>>(a);
  else k_token_logprobs<float><<<a.nrows, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ers
