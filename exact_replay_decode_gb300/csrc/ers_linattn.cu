// Linear attention with a decay per head (include/ers.h), a = log_decay[h], lambda = exp(a):
//   S_t = lambda S_{t-1} + v_t k_t^T  (S [dv x dk], fp32),  o_t = scale S_t q_t
#include "ers_common.cuh"
#include "ers_internal.h"
#include "linattn.cuh"

namespace ers {
namespace {

// ---- the recurrence, token by token -------------------------------------------------------------------
// A thread owns 16 consecutive k of one state row in registers; dk / 16 neighbouring lanes own a row
// and add up its product with q by a butterfly.  Tokens pass through shared memory kTok at a time.
constexpr int kTok = 16;

template <typename T, int DK>
__global__ void __launch_bounds__(kThreads) k_linattn_steps(LinAttnArgs a) {
  constexpr int W = DK / 16;              // lanes of a row
  constexpr int R = kThreads / W;         // rows of a CTA
  __shared__ float sq[kTok][DK], sk[kTok][DK], sv[kTok][R];
  const int i = blockIdx.x, h = blockIdx.y, g = h / (a.H / a.G);
  LinAttnSeq s;
  if (!linattn_seq(a, i, h, &s)) return;
  const int j = threadIdx.x % W, r = threadIdx.x / W, d = blockIdx.z * R + r;
  const Decay lambda = decay_of(a.log_decay[h]);
  float st[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) st[c] = s.in != nullptr ? s.in[(size_t)d * DK + j * 16 + c] : 0.f;
  for (int t0 = 0; t0 < s.len; t0 += kTok) {
    const int n = s.len - t0 < kTok ? s.len - t0 : kTok;
    __syncthreads();
    for (int e = threadIdx.x; e < n * DK; e += kThreads) {
      const size_t at = ((size_t)(s.t0 + t0 + e / DK) * a.G + g) * DK + e % DK;
      sq[e / DK][e % DK] = to_f(((const T*)a.q)[at]);
      sk[e / DK][e % DK] = to_f(((const T*)a.k)[at]);
    }
    for (int e = threadIdx.x; e < n * R; e += kThreads)
      sv[e / R][e % R] = to_f(((const T*)a.v)[((size_t)(s.t0 + t0 + e / R) * a.H + h) * a.dv + blockIdx.z * R + e % R]);
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float vd = sv[t][r];
      float dot = 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        st[c] = lambda.step(st[c], vd * sk[t][j * 16 + c]);
        dot = fmaf(st[c], sq[t][j * 16 + c], dot);
      }
#pragma unroll
      for (int off = W / 2; off >= 1; off >>= 1) dot += __shfl_xor_sync(kFull, dot, off);
      if (j == 0) ((T*)a.o)[((size_t)(s.t0 + t0 + t) * a.H + h) * a.dv + d] = from_f<T>(a.scale * dot);
    }
  }
#pragma unroll
  for (int c = 0; c < 16; ++c) s.out[(size_t)d * DK + j * 16 + c] = st[c];
}

// ---- one token per sequence ---------------------------------------------------------------------------
template <typename T, int DK>
__global__ void __launch_bounds__(kThreads) k_linattn_decode(LinAttnArgs a) {
  constexpr int W = DK / 4;               // lanes of a row, four k each
  constexpr int R = kThreads / W;
  const int i = blockIdx.x, h = blockIdx.y, g = h / (a.H / a.G);
  LinAttnSeq s;
  if (!linattn_seq(a, i, h, &s)) return;
  const int j = threadIdx.x % W;
  const Decay lambda = decay_of(a.log_decay[h]);
  float kv[4], qv[4];
  load_k<T, 4>((const T*)a.k + ((size_t)i * a.G + g) * DK + 4 * j, kv);
  load_k<T, 4>((const T*)a.q + ((size_t)i * a.G + g) * DK + 4 * j, qv);
  for (int d = threadIdx.x / W; d < a.dv; d += R) {
    const size_t at = ((size_t)i * a.H + h) * a.dv + d;
    const float vd = to_f(((const T*)a.v)[at]);
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s.in != nullptr) st = *reinterpret_cast<const float4*>(s.in + (size_t)d * DK + 4 * j);
    st.x = lambda.step(st.x, vd * kv[0]);
    st.y = lambda.step(st.y, vd * kv[1]);
    st.z = lambda.step(st.z, vd * kv[2]);
    st.w = lambda.step(st.w, vd * kv[3]);
    *reinterpret_cast<float4*>(s.out + (size_t)d * DK + 4 * j) = st;
    float dot = fmaf(st.w, qv[3], fmaf(st.z, qv[2], fmaf(st.y, qv[1], st.x * qv[0])));
#pragma unroll
    for (int off = W / 2; off >= 1; off >>= 1) dot += __shfl_xor_sync(kFull, dot, off);
    if (j == 0) ((T*)a.o)[at] = from_f<T>(a.scale * dot);
  }
}

template <typename T, int DK>
cudaError_t steps(const LinAttnArgs& a, cudaStream_t s) {
  constexpr int R = kThreads / (DK / 16);
  k_linattn_steps<T, DK><<<dim3(a.nseq, a.H, a.dv / R), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t decode(const LinAttnArgs& a, cudaStream_t s) {
  k_linattn_decode<T, DK><<<dim3(a.nseq, a.H), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

bool linattn_supported(int dk, int dv) { return (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

cudaError_t linattn_fwd(const LinAttnArgs& a, cudaStream_t s) {
  if (linattn_tc_supported(a)) return linattn_tc(a, s);
  if (a.io == ERS_DTYPE_BF16)
    return a.dk == 64 ? steps<__nv_bfloat16, 64>(a, s) : steps<__nv_bfloat16, 128>(a, s);
  return a.dk == 64 ? steps<float, 64>(a, s) : steps<float, 128>(a, s);
}

cudaError_t linattn_decode(const LinAttnArgs& a, cudaStream_t s) {
  if (a.io == ERS_DTYPE_BF16)
    return a.dk == 64 ? decode<__nv_bfloat16, 64>(a, s) : decode<__nv_bfloat16, 128>(a, s);
  return a.dk == 64 ? decode<float, 64>(a, s) : decode<float, 128>(a, s);
}

}  // namespace ers
