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
// Each state is read and written once, 128 KB a head of 128 x 128: bandwidth.  A warp takes `rows` state rows at a time, all of
// their loads under way before the first is used, a lane four k of each row; the rows' products with q are added up across
// the lanes by halving: each step exchanges half of what a lane still holds (9 shuffles for 8 rows in place of 40).
// 256 sequences x 64 heads: see the table of cases.
template <typename T, int DK, int rows>
__global__ void __launch_bounds__(kThreads) k_linattn_decode(LinAttnArgs a, int per_cta) {
  constexpr int W = DK / 4;               // lanes of a row, four k each
  constexpr int side = 32 / W;            // rows that a warp's load covers
  const int i = blockIdx.x, h = blockIdx.y, g = h / (a.H / a.G);
  LinAttnSeq s;
  if (!linattn_seq(a, i, h, &s)) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, j = lane % W;
  const int end = min((int)(blockIdx.z + 1) * per_cta, a.dv);
  int d0 = blockIdx.z * per_cta + warp * rows * side;   // a warp's rows d0 + r * side + lane / W
  float4 st[rows];
  auto load = [&]() {
#pragma unroll
    for (int r = 0; r < rows; ++r)
      st[r] = s.in != nullptr ? __ldcs(reinterpret_cast<const float4*>(s.in + (size_t)(d0 + r * side + lane / W) * DK + 4 * j))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  if (d0 < end) load();
  const Decay lambda = decay_of(a.log_decay[h]);
  float kv[4], qv[4];
  load_k<T, 4>((const T*)a.k + ((size_t)i * a.G + g) * DK + 4 * j, kv);
  load_k<T, 4>((const T*)a.q + ((size_t)i * a.G + g) * DK + 4 * j, qv);
  const T* v = (const T*)a.v + ((size_t)i * a.H + h) * a.dv;
  T* o = (T*)a.o + ((size_t)i * a.H + h) * a.dv;
  while (d0 < end) {
    float dot[rows];
#pragma unroll
    for (int r = 0; r < rows; ++r) {
      const int d = d0 + r * side + lane / W;
      const float vd = to_f(v[d]);
      st[r].x = lambda.step(st[r].x, vd * kv[0]);
      st[r].y = lambda.step(st[r].y, vd * kv[1]);
      st[r].z = lambda.step(st[r].z, vd * kv[2]);
      st[r].w = lambda.step(st[r].w, vd * kv[3]);
      __stcs(reinterpret_cast<float4*>(s.out + (size_t)d * DK + 4 * j), st[r]);
      dot[r] = fmaf(st[r].w, qv[3], fmaf(st[r].z, qv[2], fmaf(st[r].y, qv[1], st[r].x * qv[0])));
    }
    const int d1 = d0;
    d0 += kThreads / 32 * rows * side;
    if (d0 < end) load();
    // halving: after the step over `off` a lane holds the rows whose bit is its own
    int row = 0;
    int off = W / 2;
#pragma unroll
    for (int n = rows / 2; n >= 1; n /= 2, off /= 2) {
      const bool upper = (lane & off) != 0;
#pragma unroll
      for (int r = 0; r < n; ++r) {
        const float give = upper ? dot[r] : dot[r + n], keep = upper ? dot[r + n] : dot[r];
        dot[r] = keep + __shfl_xor_sync(kFull, give, off);
      }
      if (upper) row += n;
    }
#pragma unroll
    for (; off >= 1; off /= 2) dot[0] += __shfl_xor_sync(kFull, dot[0], off);
    if (j % (W / rows) == 0) o[d1 + row * side + lane / W] = from_f<T>(a.scale * dot[0]);
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
  // A CTA per head where those fill the SMs; fewer heads are cut up to a batch of rows per warp.
  constexpr int side = 32 / (DK / 4);
  const long long heads = (long long)a.nseq * a.H;
  if (heads >= 608) {
    k_linattn_decode<T, DK, 8><<<dim3(a.nseq, a.H), kThreads, 0, s>>>(a, a.dv);
  } else {
    const int per = kThreads / 32 * 4 * side;
    k_linattn_decode<T, DK, 4><<<dim3(a.nseq, a.H, (a.dv + per - 1) / per), kThreads, 0, s>>>(a, per);
  }
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
