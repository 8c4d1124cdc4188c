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
// exchanges run beside those of S k.  256 sequences x 64 heads of 128 x 128: 319 us, the measured bandwidth.
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

// ---- prompts, eight tokens at a time ----------------------------------------------------------------------
// fp32 prompts, and short bf16 ones.  A CTA keeps its state rows in registers over the whole sequence; tokens come through shared
// memory, kTok at a time, the next ones under way.  Of a batch of eight tokens every product with the state is one with the
// state before it, so that their exchanges across lanes run side by side, and the residuals follow from products of keys:
//   y_t = S k_t, z_t = S q_t;   u_t = beta_t (v_t - e^(G_t) y_t) - sum_(s<t) beta_t e^(G_t - G_s) (k_s.k_t) u_s
//   o_t = scale (e^(G_t) z_t + sum_(s<=t) e^(G_t - G_s) (k_s.q_t) u_s),   S <- e^(G_7) S + sum_t e^(G_7 - G_t) u_t k_t^T
// (token by token, with an exchange in the chain of each, 1025 tokens x 16 heads took 400 us in place of 242).  G_t - G_s is summed from the
// gates between: no cancellation.  What a token holds that is not finite reaches nothing before it.
constexpr int kStepThreads = 128, kTok = 32, kBatch = 8;
constexpr int kStepRows = kStepThreads / 32 * kSide;

template <typename T, int DK, int R>
struct StepTiles {
  static constexpr int LD = DK + 16 / sizeof(T);            // rows of tokens start in other banks
  T q[2][kTok][LD];
  T k[2][kTok][LD];
  T v[2][kTok][R];
  alignas(16) float g[2][kTok];
  float beta[2][kTok];
  alignas(16) float kk[kTok][kBatch];                       // beta_t e^(G_t - G_s) k_s.k_t, s < t
  alignas(16) float qk[kTok][kBatch];                       // e^(G_t - G_s) k_s.q_t, s <= t
  float since[kTok], left[kTok];                            // e^(G_t), e^(G_7 - G_t)
  Decay whole[kTok / kBatch];                               // e^(G_7)
};

// Adds up eight values across the eight lanes of a row: lane j gets the total of value j.
__device__ __forceinline__ float totals(float (&v)[kBatch], int j) {
#pragma unroll
  for (int n = 4; n >= 1; n /= 2) {
    const bool upper = (j & n) != 0;
#pragma unroll
    for (int r = 0; r < n; ++r) {
      const float give = upper ? v[r] : v[r + n], keep = upper ? v[r + n] : v[r];
      v[r] = keep + __shfl_xor_sync(kFull, give, n);
    }
  }
  return v[0];
}
__device__ __forceinline__ void axpy(float4& a, float f, float4 x) {
  a.x = fmaf(f, x.x, a.x);
  a.y = fmaf(f, x.y, a.y);
  a.z = fmaf(f, x.z, a.z);
  a.w = fmaf(f, x.w, a.w);
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

template <typename T, int DK, int rows>
__global__ void __launch_bounds__(kStepThreads) k_gdn_steps(const __grid_constant__ DeltaArgs a) {
  constexpr int N = DK / 32, R = kStepRows * rows;
  using Tiles = StepTiles<T, DK, R>;
  extern __shared__ __align__(16) unsigned char smem[];
  Tiles& tiles = *reinterpret_cast<Tiles*>(smem);
  const int parts = a.dv / R, part = blockIdx.x % parts, unit = blockIdx.x / parts;   // a sequence's CTAs side by side
  const int i = unit / a.H, h = unit % a.H, g = h / (a.H / a.G);
  // Beside the chunks of a call's longer sequences the grid may run while theirs does; it ends no sooner.
  const auto done = [&] {
    if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  DeltaSeq s;
  if (!delta_seq(a, i, h, &s)) return done();
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
    const int n = min(kTok, s.len - t0), all = (n + kBatch - 1) / kBatch * kBatch;   // zeros in the rest of the last batch
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int x = threadIdx.x; x < all * (DK / e); x += kStepThreads) {
      const int t = x / (DK / e), c = x % (DK / e) * e;
      if (t < n) {
        const size_t at = ((size_t)(s.t0 + t0 + t) * a.G + g) * DK + c;
        tc::cp_async16(&tiles.q[b][t][c], (const T*)a.q + at);
        tc::cp_async16(&tiles.k[b][t][c], (const T*)a.k + at);
      } else {
        *reinterpret_cast<uint4*>(&tiles.q[b][t][c]) = zero;
        *reinterpret_cast<uint4*>(&tiles.k[b][t][c]) = zero;
      }
    }
    for (int x = threadIdx.x; x < all * (R / e); x += kStepThreads) {
      const int t = x / (R / e), c = x % (R / e) * e;
      if (t < n) tc::cp_async16(&tiles.v[b][t][c], (const T*)a.v + ((size_t)(s.t0 + t0 + t) * a.H + h) * a.dv + d0 + c);
      else *reinterpret_cast<uint4*>(&tiles.v[b][t][c]) = zero;
    }
    if (threadIdx.x < all) {
      const size_t at = (size_t)(s.t0 + t0 + threadIdx.x) * a.H + h;
      tiles.g[b][threadIdx.x] = threadIdx.x < n ? a.g[at] : 0.f;
      tiles.beta[b][threadIdx.x] = threadIdx.x < n ? a.beta[at] : 0.f;
    }
    static_assert(R % e == 0, "whole copies");
  };
  if (s.len > 0) fetch(0, 0);
  for (int t0 = 0, b = 0; t0 < s.len; t0 += kTok, b ^= 1) {
    tc::cp_async_wait_all();
    __syncthreads();                                        // this tile is there, the other one no longer read
    if (t0 + kTok < s.len) fetch(t0 + kTok, b ^ 1);
    const int n = min(kTok, s.len - t0);
    // products of the tile's keys and queries: two lanes for each pair of a batch, the batches' side by side
    const int pair = threadIdx.x / 2, t = pair / kBatch, u = pair % kBatch, half = threadIdx.x % 2;
    float kk[kTok / kBatch] = {}, qk[kTok / kBatch] = {};
    if (u <= t) {
#pragma unroll 2
      for (int x = 4 * half; x < DK; x += 8)
#pragma unroll
        for (int m = 0; m < kTok / kBatch; ++m) {
          if (m * kBatch >= n) break;
          const float4 ku = quad(&tiles.k[b][m * kBatch + u][x]);
          kk[m] = dot4(ku, quad(&tiles.k[b][m * kBatch + t][x]), kk[m]);
          qk[m] = dot4(ku, quad(&tiles.q[b][m * kBatch + t][x]), qk[m]);
        }
    }
#pragma unroll
    for (int m = 0; m < kTok / kBatch; ++m) {
      if (m * kBatch >= n) break;
      kk[m] += __shfl_xor_sync(kFull, kk[m], 1);
      qk[m] += __shfl_xor_sync(kFull, qk[m], 1);
      const float4 g0 = quad(&tiles.g[b][m * kBatch]), g1 = quad(&tiles.g[b][m * kBatch + 4]);
      const float gate[kBatch] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
      const auto sum = [&](int from, int to) {              // of gates, no others in between
        float v = 0.f;
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
          if (x >= from && x <= to) v += gate[x];
        return v;
      };
      if (half == 0) {
        const float f = u <= t ? expf(sum(u + 1, t)) : 0.f;
        tiles.kk[m * kBatch + t][u] = u < t ? tiles.beta[b][m * kBatch + t] * f * kk[m] : 0.f;
        tiles.qk[m * kBatch + t][u] = u <= t ? f * qk[m] : 0.f;
      } else if (u == 0) {
        const float before = sum(0, t);
        tiles.since[m * kBatch + t] = expf(before);
        tiles.left[m * kBatch + t] = expf(sum(t + 1, kBatch - 1));
        if (t == kBatch - 1) tiles.whole[m] = decay_of(before);
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int t8 = 0; t8 < n; t8 += kBatch) {
      float y[rows][kBatch] = {}, z[rows][kBatch] = {};
#pragma unroll
      for (int x = 0; x < N; ++x)
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
          const float4 k = quad(&tiles.k[b][t8 + t][4 * (j + kRowLanes * x)]), q = quad(&tiles.q[b][t8 + t][4 * (j + kRowLanes * x)]);
#pragma unroll
          for (int r = 0; r < rows; ++r) {
            y[r][t] = dot4(st[r][x], k, y[r][t]);
            z[r][t] = dot4(st[r][x], q, z[r][t]);
          }
        }
      float mine[rows];                                     // z of token j
#pragma unroll
      for (int r = 0; r < rows; ++r) {
        const float all = totals(y[r], j);
        mine[r] = totals(z[r], j);
#pragma unroll
        for (int t = 0; t < kBatch; ++t) y[r][t] = __shfl_sync(kFull, all, (lane & ~(kRowLanes - 1)) | t);
      }
      float (&u)[rows][kBatch] = y;                         // the residuals, in place
#pragma unroll
      for (int t = 0; t < kBatch; ++t) {
        const float beta = tiles.beta[b][t8 + t], since = tiles.since[t8 + t];
        const float4 c0 = quad(&tiles.kk[t8 + t][0]), c1 = quad(&tiles.kk[t8 + t][4]);
        const float c[kBatch] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
        for (int r = 0; r < rows; ++r) {
          float x = beta * fmaf(-since, y[r][t], to_f(tiles.v[b][t8 + t][own + kSide * r]));
#pragma unroll
          for (int e = 0; e < t; ++e) x = fmaf(-c[e], u[r][e], x);
          u[r][t] = x;
        }
      }
      {
        const float4 c0 = quad(&tiles.qk[t8 + j][0]), c1 = quad(&tiles.qk[t8 + j][4]);
        const float c[kBatch] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w}, since = tiles.since[t8 + j];
        T* o = (T*)a.o + ((size_t)(s.t0 + t0 + t8 + j) * a.H + h) * a.dv + d0 + own;
#pragma unroll
        for (int r = 0; r < rows; ++r) {
          float x = since * mine[r];
#pragma unroll
          for (int e = 0; e < kBatch; ++e)
            if (e <= j) x = fmaf(c[e], u[r][e], x);         // (what comes later may be anything)
          if (t8 + j < n) o[kSide * r] = from_f<T>(a.scale * x);
        }
      }
      const Decay whole = tiles.whole[t8 / kBatch];
#pragma unroll
      for (int r = 0; r < rows; ++r)
#pragma unroll
        for (int t = 0; t < kBatch; ++t) u[r][t] *= tiles.left[t8 + t];
#pragma unroll
      for (int x = 0; x < N; ++x) {
#pragma unroll
        for (int r = 0; r < rows; ++r) {
          st[r][x].x = fmaf(whole.hi, st[r][x].x, whole.lo * st[r][x].x);
          st[r][x].y = fmaf(whole.hi, st[r][x].y, whole.lo * st[r][x].y);
          st[r][x].z = fmaf(whole.hi, st[r][x].z, whole.lo * st[r][x].z);
          st[r][x].w = fmaf(whole.hi, st[r][x].w, whole.lo * st[r][x].w);
        }
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
          const float4 k = quad(&tiles.k[b][t8 + t][4 * (j + kRowLanes * x)]);
#pragma unroll
          for (int r = 0; r < rows; ++r) axpy(st[r][x], u[r][t], k);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int x = 0; x < N; ++x)
      *reinterpret_cast<float4*>(s.out + (size_t)(d0 + own + kSide * r) * DK + 4 * (j + kRowLanes * x)) = st[r][x];
  done();
}

// beside: as a programmatic dependent of the stream's last launch
template <typename T, int DK, int rows>
cudaError_t launch_steps(const DeltaArgs& a, bool beside, cudaStream_t s) {
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.nseq * a.H * (a.dv / R)));
  cfg.blockDim = dim3(kStepThreads);
  cfg.dynamicSmemBytes = sizeof(Tiles);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Rows of a lane: one while a CTA of such has an SM for itself, two while two of those fit a SM, four beyond: k and q are read from
// shared memory by every warp, which bounds many CTAs.  By one, two and four, us:
//   fp32, 1024 x 16 heads 254, 287, 571; x 32 352, 290, 623; 4 x 1024 x 64 2448, 1618, 1397; 300 and 1025 x 16 242, 261, 279
//   bf16, 16 x 16 6.2, 7.9, 12.8; 33 x 64 28.2, 18.6, 30.4; 4 x 33 x 32 54.3, 35.7, 31.4
template <typename T, int DK>
cudaError_t steps(const DeltaArgs& a, bool beside, cudaStream_t s) {
  // (of the lengths only the longest and the sum are known: as many sequences as the sum has longest ones count, or the others where
  // the longer ones go by chunks)
  const long long longest = max(a.max_len, 1), n = a.len1 == 0x7fffffff ? (a.ntokens + longest / 2) / longest
                                                                       : a.nseq - (a.ntokens + longest - 1) / longest;
  const long long full = min(max(n, 1LL), (long long)a.nseq);
  const long long ctas = full * a.H * (a.dv / kStepRows);
  return ctas <= 152   ? launch_steps<T, DK, 1>(a, beside, s)
         : ctas <= 608 ? launch_steps<T, DK, 2>(a, beside, s)
                       : launch_steps<T, DK, 4>(a, beside, s);
}

template <typename T, int DK>
cudaError_t decode(const DeltaArgs& a, cudaStream_t s) {
  // a CTA per head where those fill the SMs, else one per 32 rows of its state
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

// bf16 sequences of more tokens than these go by chunks, which take 15 us whatever they hold (32 heads: 24 tokens 10.2 us by the
// recurrence, 33 15.0 and 15.0; 128 heads: 24 tokens 20.1 and 23.0, 33 31.4 and 23.2).  A sequence's own length decides, on the
// device, so that neither its neighbours nor a loose max_len take bits from a short one; where that leaves no short ones (the longest
// length times the sequences is all tokens), one launch is spared.  With all of a call by chunks 2048 tokens and 256 single ones x 64
// heads took 2084 us and 1.5 GB in place of 1185 and 0.7, 97 and 15 single ones x 32 73 us (45); 2048, 777, 513 and 1 x 64 270 (274),
// 2048 and 63 of 20 x 32 334 (396).
static int few_tokens(const DeltaArgs& a) { return (long long)a.nseq * a.H <= 64 ? 32 : 24; }

// The sequences that go by chunks, as a call of their own; false: there are none.
static bool by_chunks(const DeltaArgs& a, DeltaArgs* many) {
  if (a.io != ERS_DTYPE_BF16 || a.max_len <= few_tokens(a)) return false;
  *many = a;
  many->len0 = (long long)a.nseq * a.max_len <= a.ntokens ? 0 : few_tokens(a) + 1;
  many->most = many->len0 == 0 || a.ntokens / many->len0 > a.nseq ? a.nseq : (int)(a.ntokens / many->len0);
  return true;
}

static cudaError_t by_steps(const DeltaArgs& a, bool beside, cudaStream_t s) {
  if (a.io == ERS_DTYPE_BF16)
    return a.dk == 64 ? steps<__nv_bfloat16, 64>(a, beside, s) : steps<__nv_bfloat16, 128>(a, beside, s);
  return a.dk == 64 ? steps<float, 64>(a, beside, s) : steps<float, 128>(a, beside, s);
}
cudaError_t gdn_steps_beside(const DeltaArgs& a, cudaStream_t s) { return by_steps(a, true, s); }

cudaError_t gdn_fwd(const DeltaArgs& a, cudaStream_t s) {
  DeltaArgs many;
  if (!by_chunks(a, &many)) return by_steps(a, false, s);
  DeltaArgs few = a;
  few.len1 = many.len0 - 1;
  return gdn_tc(many, many.len0 > 0 ? &few : nullptr, s);
}

cudaError_t gdn_decode(const DeltaArgs& a, cudaStream_t s) {
  if (a.io == ERS_DTYPE_BF16) return a.dk == 64 ? decode<__nv_bfloat16, 64>(a, s) : decode<__nv_bfloat16, 128>(a, s);
  return a.dk == 64 ? decode<float, 64>(a, s) : decode<float, 128>(a, s);
}

size_t gdn_fwd_workspace(const DeltaArgs& a) {
  DeltaArgs many;
  return by_chunks(a, &many) ? gdn_tc_workspace(many) : 0;
}

}  // namespace ers
