// The gated delta rule over states (include/ers.h), token by token: per head, with a_t = exp(g_t),
//   u_t = beta_t (v_t - a_t S k_t),  S <- a_t S + u_t k_t^T  (S [dv x dk], fp32),  o_t = scale S q_t
// A state row (one d of dv) depends on no other row, so rows are what is shared out.  Eight lanes hold a row, lane j of
// them its elements 4 (j + 8 i) .. + 3: a row's product with k or q is 16 (dk = 64: 8) products a lane and three exchanges.
#include <mutex>

#include "ers_common.cuh"
#include "ers_internal.h"
#include "gdn_rule.cuh"
#include "tc_common.cuh"

namespace ers {
namespace {

constexpr int kRowLanes = 8;                 // lanes of a state row
constexpr int kSide = 32 / kRowLanes;        // rows that a warp holds in one register of its lanes

__device__ __forceinline__ float4 quad(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 quad(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = kRowLanes / 2; off >= 1; off /= 2) v += __shfl_xor_sync(kFull, v, off);
  return v;
}
template <int N>
__device__ __forceinline__ float dot(const float4 (&a)[N], const float4 (&b)[N]) {
  float x = 0.f, y = 0.f, z = 0.f, w = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x = fmaf(a[i].x, b[i].x, x);
    y = fmaf(a[i].y, b[i].y, y);
    z = fmaf(a[i].z, b[i].z, z);
    w = fmaf(a[i].w, b[i].w, w);
  }
  return (x + y) + (z + w);
}
template <int N>
__device__ __forceinline__ void step_row(float4 (&s)[N], const float4 (&k)[N], Decay d, float u) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i].x = d.step(s[i].x, u * k[i].x);
    s[i].y = d.step(s[i].y, u * k[i].y);
    s[i].z = d.step(s[i].z, u * k[i].z);
    s[i].w = d.step(s[i].w, u * k[i].w);
  }
}

// ---- one token per sequence ---------------------------------------------------------------------------
// Each state is read and written once, 128 KB a head of 128 x 128: bandwidth.  A warp takes kSide * sets rows, all of their
// loads under way before the first is used.  The output is taken from the old state, a S q + u (k . q), so that its
// exchanges run beside those of S k.
constexpr int kDecodeRows = kThreads / 32 * kSide;   // rows of a CTA for each set

template <typename T, int DK, int sets>
__global__ void __launch_bounds__(kThreads) k_gdn_decode(const __grid_constant__ DeltaArgs a) {
  constexpr int N = DK / 32;
  const int i = blockIdx.x, h = blockIdx.y, g = h / (a.H / a.G);
  DeltaSeq s;
  if (!delta_seq(a, i, h, &s)) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, j = lane % kRowLanes;
  const int d0 = (blockIdx.z * (kThreads / 32) + warp) * kSide * sets + lane / kRowLanes;   // rows d0 + kSide * r
  float4 st[sets][N];
#pragma unroll
  for (int r = 0; r < sets; ++r)
#pragma unroll
    for (int x = 0; x < N; ++x)
      st[r][x] = s.in != nullptr ? __ldcs(reinterpret_cast<const float4*>(s.in + (size_t)(d0 + kSide * r) * DK + 4 * (j + kRowLanes * x)))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
  const size_t row = (size_t)i * a.H + h;
  const Decay decay = decay_of(a.g[row]);
  const float beta = a.beta[row], whole = decay.hi + decay.lo;
  float4 k[N], q[N];
#pragma unroll
  for (int x = 0; x < N; ++x) {
    const size_t at = ((size_t)i * a.G + g) * DK + 4 * (j + kRowLanes * x);
    k[x] = quad((const T*)a.k + at);
    q[x] = quad((const T*)a.q + at);
  }
  const float kq = row_sum(dot(k, q));
  const T* v = (const T*)a.v + row * a.dv;
  T* o = (T*)a.o + row * a.dv;
#pragma unroll
  for (int r = 0; r < sets; ++r) {
    const int d = d0 + kSide * r;
    const float sk = row_sum(dot(st[r], k)), sq = row_sum(dot(st[r], q));
    const float u = beta * fmaf(-whole, sk, to_f(v[d]));
    step_row(st[r], k, decay, u);
#pragma unroll
    for (int x = 0; x < N; ++x) __stcs(reinterpret_cast<float4*>(s.out + (size_t)d * DK + 4 * (j + kRowLanes * x)), st[r][x]);
    if (j == 0) o[d] = from_f<T>(a.scale * fmaf(whole, sq, u * kq));
  }
}

// ---- prompts, token by token ----------------------------------------------------------------------------
// A CTA keeps kStepRows * rows state rows in registers over the whole sequence; tokens come through shared memory, kTok at a
// time, the next ones under way.  The chain through a token is the product with k, its three exchanges and the update.
constexpr int kStepThreads = 128, kTok = 32;
constexpr int kStepRows = kStepThreads / 32 * kSide;

template <typename T, int DK, int R>
struct StepTiles {
  T q[2][kTok][DK];
  T k[2][kTok][DK];
  T v[2][kTok][R];
  float g[2][kTok], beta[2][kTok];
};

template <typename T, int DK, int rows>
__global__ void __launch_bounds__(kStepThreads) k_gdn_steps(const __grid_constant__ DeltaArgs a) {
  constexpr int N = DK / 32, R = kStepRows * rows;
  using Tiles = StepTiles<T, DK, R>;
  extern __shared__ __align__(16) unsigned char smem[];
  Tiles& tiles = *reinterpret_cast<Tiles*>(smem);
  const int parts = a.dv / R, part = blockIdx.x % parts, unit = blockIdx.x / parts;   // a sequence's CTAs side by side
  const int i = unit / a.H, h = unit % a.H, g = h / (a.H / a.G);
  DeltaSeq s;
  if (!delta_seq(a, i, h, &s)) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, j = lane % kRowLanes;
  const int own = warp * kSide * rows + lane / kRowLanes;   // this lane's rows of the CTA: own + kSide * r
  const int d0 = part * R;
  float4 st[rows][N];
#pragma unroll
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int x = 0; x < N; ++x)
      st[r][x] = s.in != nullptr ? quad(s.in + (size_t)(d0 + own + kSide * r) * DK + 4 * (j + kRowLanes * x))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
  const auto fetch = [&](int t0, int b) {
    constexpr int e = 16 / sizeof(T);                       // elements of a copy
    const int n = min(kTok, s.len - t0);
    for (int x = threadIdx.x; x < n * (DK / e); x += kStepThreads) {
      const int t = x / (DK / e), c = x % (DK / e) * e;
      const size_t at = ((size_t)(s.t0 + t0 + t) * a.G + g) * DK + c;
      tc::cp_async16(&tiles.q[b][t][c], (const T*)a.q + at);
      tc::cp_async16(&tiles.k[b][t][c], (const T*)a.k + at);
    }
    for (int x = threadIdx.x; x < n * (R / e); x += kStepThreads) {
      const int t = x / (R / e), c = x % (R / e) * e;
      tc::cp_async16(&tiles.v[b][t][c], (const T*)a.v + ((size_t)(s.t0 + t0 + t) * a.H + h) * a.dv + d0 + c);
    }
    if (threadIdx.x < n) {
      const size_t at = (size_t)(s.t0 + t0 + threadIdx.x) * a.H + h;
      tiles.g[b][threadIdx.x] = a.g[at];
      tiles.beta[b][threadIdx.x] = a.beta[at];
    }
    static_assert(R % e == 0, "whole copies");
  };
  if (s.len > 0) fetch(0, 0);
  for (int t0 = 0, b = 0; t0 < s.len; t0 += kTok, b ^= 1) {
    tc::cp_async_wait_all();
    __syncthreads();                                        // this tile is there, the other one no longer read
    if (t0 + kTok < s.len) fetch(t0 + kTok, b ^ 1);
    const int n = min(kTok, s.len - t0);
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
      float4 k[N], q[N];
#pragma unroll
      for (int x = 0; x < N; ++x) {
        k[x] = quad(&tiles.k[b][t][4 * (j + kRowLanes * x)]);
        q[x] = quad(&tiles.q[b][t][4 * (j + kRowLanes * x)]);
      }
      const Decay decay = decay_of(tiles.g[b][t]);
      const float beta = tiles.beta[b][t], whole = decay.hi + decay.lo;
      T* o = (T*)a.o + ((size_t)(s.t0 + t0 + t) * a.H + h) * a.dv + d0;
#pragma unroll
      for (int r = 0; r < rows; ++r) {
        const float sk = row_sum(dot(st[r], k));
        step_row(st[r], k, decay, beta * fmaf(-whole, sk, to_f(tiles.v[b][t][own + kSide * r])));
        const float sq = row_sum(dot(st[r], q));
        if (j == 0) o[own + kSide * r] = from_f<T>(a.scale * sq);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int x = 0; x < N; ++x)
      *reinterpret_cast<float4*>(s.out + (size_t)(d0 + own + kSide * r) * DK + 4 * (j + kRowLanes * x)) = st[r][x];
}

template <typename T, int DK, int rows>
cudaError_t launch_steps(const DeltaArgs& a, cudaStream_t s) {
  constexpr int R = kStepRows * rows;
  using Tiles = StepTiles<T, DK, R>;
  const auto kernel = k_gdn_steps<T, DK, rows>;
  if (sizeof(Tiles) > 48 * 1024) {                          // more than a kernel may have without asking: once per device
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Tiles));
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  kernel<<<dim3((unsigned)((long long)a.nseq * a.H * (a.dv / R))), kStepThreads, sizeof(Tiles), s>>>(a);
  return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t steps(const DeltaArgs& a, cudaStream_t s) {
  return launch_steps<T, DK, 2>(a, s);
}

template <typename T, int DK>
cudaError_t decode(const DeltaArgs& a, cudaStream_t s) {
  const dim3 few(a.nseq, a.H, a.dv / kDecodeRows);
  if ((long long)a.nseq * a.H < 608) {
    k_gdn_decode<T, DK, 1><<<few, kThreads, 0, s>>>(a);
  } else if (a.dv == 64) {
    k_gdn_decode<T, DK, 2><<<dim3(a.nseq, a.H), kThreads, 0, s>>>(a);
  } else {
    k_gdn_decode<T, DK, 4><<<dim3(a.nseq, a.H), kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

// bf16 prompts of more tokens than these go by chunks.
constexpr int kFewTokens = 24;
static bool by_chunks(const DeltaArgs& a) { return a.io == ERS_DTYPE_BF16 && a.max_len > kFewTokens; }

cudaError_t gdn_fwd(const DeltaArgs& a, cudaStream_t s) {
  if (by_chunks(a)) return gdn_tc(a, s);
  if (a.io == ERS_DTYPE_BF16) return a.dk == 64 ? steps<__nv_bfloat16, 64>(a, s) : steps<__nv_bfloat16, 128>(a, s);
  return a.dk == 64 ? steps<float, 64>(a, s) : steps<float, 128>(a, s);
}

cudaError_t gdn_decode(const DeltaArgs& a, cudaStream_t s) {
  if (a.io == ERS_DTYPE_BF16) return a.dk == 64 ? decode<__nv_bfloat16, 64>(a, s) : decode<__nv_bfloat16, 128>(a, s);
  return a.dk == 64 ? decode<float, 64>(a, s) : decode<float, 128>(a, s);
}

size_t gdn_fwd_workspace(const DeltaArgs& a) { return by_chunks(a) ? gdn_tc_workspace(a) : 0; }

}  // namespace ers
