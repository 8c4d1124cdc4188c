// Linear attention with a decay per head (include/ers.h), a = log_decay[h], lambda = exp(a):
//   S_t = lambda S_{t-1} + v_t k_t^T  (S [dv x dk], fp32),  o_t = scale S_t q_t
#include <mutex>
#include <type_traits>

#include "ers_common.cuh"
#include "ers_internal.h"
#include "f32x2.cuh"
#include "linattn.cuh"
#include "tc_common.cuh"

namespace ers {
namespace {

__device__ __forceinline__ float sum_of(uint64_t v) {
  float x, y;
  unpair(v, x, y);
  return x + y;
}
// four consecutive elements as two pairs
__device__ __forceinline__ void load4(const float* p, uint64_t (&v)[2]) {
  const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(p);
  v[0] = u.x;
  v[1] = u.y;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, uint64_t (&v)[2]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  v[0] = pair(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
  v[1] = pair(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// Adds up N values (a power of two) across the W neighbouring lanes that each hold a part of all of them, by halving: each
// step exchanges half of what a lane still holds.  Afterwards v[0 .. max(N / W, 1)) of a lane are the totals of values
// first, first + 1, ... (where N < W several lanes hold the same one).
template <int N, int W>
__device__ __forceinline__ void halve(float (&v)[N], int lane, int* first) {
  int row = 0, off = W / 2;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2) {
    if (off < 1) break;
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int r = 0; r < n; ++r) {
      const float give = upper ? v[r] : v[r + n], keep = upper ? v[r + n] : v[r];
      v[r] = keep + __shfl_xor_sync(kFull, give, off);
    }
    if (upper) row += n;
    off /= 2;
  }
#pragma unroll
  for (; off >= 1; off /= 2) v[0] += __shfl_xor_sync(kFull, v[0], off);
  *first = row;
}

// ---- the recurrence, token by token -------------------------------------------------------------------
// fp32 prompts, and bf16 ones too short for chunks.  A warp owns state rows in registers (W = dk / 4 lanes a row, `rows` rows of
// each lane).  Its products with q are added up for kBatch tokens at once.  Tokens come through shared memory, kTok at a
// time, the next ones under way.
//
// While |a| <= kLevel the state is not decayed token by token but held at the level of the middle of the tile: with
// c = kTok / 2, U_j = lambda^(c-1-j) S_j is U_(j-1) + lambda^(c-1-j) v_j k_j^T, an output lambda^(j+1-c) scale U_j q_j, and the
// next tile starts from lambda^n U.  That is 5 packed instructions a row of a token in place of 9; the factors lie within
// e^(+-c), and U is rounded as S would be.  (Chunks of products would need no fewer on these cores.)
//
// What bounds it: a long prompt of few heads is a chain, 44 ns a token; many heads are reads of k and q from shared memory by every
// warp, and packed FMAs at half rate.  fp32, 128 x 128: 4096 tokens x 16 heads 233 us, 4 x 1024 x 64 547 us.
// bf16, 16 x 24 tokens x 32 heads: 37 us.
constexpr int kStepThreads = 128;
constexpr float kLevel = 1.f;            // (c of 16 at most: factors within 1.2e-7 .. 8.9e6)

template <typename T, int DK, int rows>
struct StepTiles {
  // bf16: most that come here in one tile.  fp32: larger tiles and batches wait less often (4096 tokens x 16 heads by 16 and 16
  // 317 us, by 32 and 32 277, both of two rows); 32 tokens of four rows or 16 of eight at once would not fit the registers.
  static constexpr int kTok = sizeof(T) == 2 ? 24 : 32, kBatch = sizeof(T) == 2 ? 8 : rows == 2 ? 32 : rows == 4 ? 16 : 8;
  static constexpr int R = kStepThreads / 32 * rows * (32 / (DK / 4));   // rows of a CTA
  T q[2][kTok][DK];
  T k[2][kTok][DK];
  T v[2][kTok][R];
  float in[kTok], out[kTok];        // factors of the tile's values and of its outputs
};

template <typename T, int DK, int rows, bool leveled>
__global__ void __launch_bounds__(kStepThreads, sizeof(T) == 2 ? 8 : 1)   // (bf16: 64 x 32 single tokens 42 us, by six a SM 47)
    k_linattn_steps(LinAttnArgs a) {
  constexpr int W = DK / 4, side = 32 / W;                  // rows that a warp holds in one register of its lanes
  using Tiles = StepTiles<T, DK, rows>;
  constexpr int R = Tiles::R, kTok = Tiles::kTok, kBatch = Tiles::kBatch;
  constexpr int N = kBatch * rows, copies = N < W ? W / N : 1;   // lanes that end up with the same product
  extern __shared__ __align__(16) unsigned char smem[];
  Tiles& tiles = *reinterpret_cast<Tiles*>(smem);
  auto& sq = tiles.q;
  auto& sk = tiles.k;
  auto& sv = tiles.v;
  const int parts = a.dv / R, part = blockIdx.x % parts, unit = blockIdx.x / parts;   // a sequence's CTAs side by side
  const int i = unit / a.H, h = unit % a.H, g = h / (a.H / a.G);
  LinAttnSeq s;
  if (!linattn_seq(a, i, h, &s)) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, j = lane % W;
  const int own = warp * rows * side + lane / W;            // this lane's rows of the CTA: own + r * side
  const int d0 = part * R;
  uint64_t st[rows][2];
#pragma unroll
  for (int r = 0; r < rows; ++r) {
    st[r][0] = st[r][1] = 0;
    if (s.in != nullptr) load4(s.in + (size_t)(d0 + own + r * side) * DK + 4 * j, st[r]);
  }
  const auto fetch = [&](int t0, int b) {
    constexpr int e = 16 / sizeof(T);                       // elements of a copy
    const int n = min(kTok, s.len - t0);
    for (int x = threadIdx.x; x < n * (DK / e); x += kStepThreads) {
      const int t = x / (DK / e), c = x % (DK / e) * e;
      const size_t at = ((size_t)(s.t0 + t0 + t) * a.G + g) * DK + c;
      tc::cp_async16(&sq[b][t][c], (const T*)a.q + at);
      tc::cp_async16(&sk[b][t][c], (const T*)a.k + at);
    }
    for (int x = threadIdx.x; x < n * (R / e); x += kStepThreads) {
      const int t = x / (R / e), c = x % (R / e) * e;
      tc::cp_async16(&sv[b][t][c], (const T*)a.v + ((size_t)(s.t0 + t0 + t) * a.H + h) * a.dv + d0 + c);
    }
    static_assert(R % e == 0, "whole copies");
  };
  if (s.len > 0) fetch(0, 0);
  const float a_h = a.log_decay[h];
  const bool level = leveled && fabsf(a_h) <= kLevel;
  Decay lambda = {}, tile_step = {};
  if (level) tile_step = decay_of_tokens(a_h, kTok);
  else lambda = decay_of(a_h);
  if (level && threadIdx.x < kTok) {
    tiles.in[threadIdx.x] = power_of(a_h, kTok / 2 - 1 - (int)threadIdx.x);
    tiles.out[threadIdx.x] = power_of(a_h, (int)threadIdx.x + 1 - kTok / 2);
  }
  const auto times = [&](Decay d) {
    const uint64_t hi = pair(d.hi, d.hi), lo = pair(d.lo, d.lo);
#pragma unroll
    for (int r = 0; r < rows; ++r) {
      st[r][0] = fma2(hi, st[r][0], mul2(lo, st[r][0]));
      st[r][1] = fma2(hi, st[r][1], mul2(lo, st[r][1]));
    }
  };
  const auto walk = [&](auto is_level) {
    const uint64_t hi = pair(lambda.hi, lambda.hi), lo = pair(lambda.lo, lambda.lo);
    for (int t0 = 0, b = 0; t0 < s.len; t0 += kTok, b ^= 1) {
      tc::cp_async_wait_all();
      __syncthreads();                                      // this tile is there, the other one no longer read
      if (t0 + kTok < s.len) fetch(t0 + kTok, b ^ 1);
      const int n = min(kTok, s.len - t0);
      const auto batch = [&](int t, auto whole) {           // whole: no token of it is missing, so no branch either
        float dot[N];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (whole.value || t + u < n) {
            uint64_t k2[2], q2[2];
            load4(&sk[b][t + u][4 * j], k2);
            load4(&sq[b][t + u][4 * j], q2);
#pragma unroll
            for (int r = 0; r < rows; ++r) {
              const float x = to_f(sv[b][t + u][own + r * side]) * (is_level.value ? tiles.in[t + u] : 1.f);
              const uint64_t v2 = pair(x, x);
              if (is_level.value) {
                st[r][0] = fma2(v2, k2[0], st[r][0]);
                st[r][1] = fma2(v2, k2[1], st[r][1]);
              } else {
                st[r][0] = fma2(hi, st[r][0], fma2(lo, st[r][0], mul2(v2, k2[0])));
                st[r][1] = fma2(hi, st[r][1], fma2(lo, st[r][1], mul2(v2, k2[1])));
              }
              dot[u * rows + r] = sum_of(fma2(st[r][1], q2[1], mul2(st[r][0], q2[0])));
            }
          } else {
#pragma unroll
            for (int r = 0; r < rows; ++r) dot[u * rows + r] = 0.f;
          }
        }
        int first;
        halve<N, W>(dot, lane, &first);
#pragma unroll
        for (int e = 0; e < (N > W ? N / W : 1); ++e) {
          const int u = (first + e) / rows, r = (first + e) % rows;
          if ((whole.value || t + u < n) && j % copies == 0)
            ((T*)a.o)[((size_t)(s.t0 + t0 + t + u) * a.H + h) * a.dv + d0 + warp * rows * side + lane / W + r * side] =
                from_f<T>(a.scale * (is_level.value ? tiles.out[t + u] * dot[e] : dot[e]));
        }
      };
      int t = 0;
#pragma unroll 1
      for (; t + kBatch <= n; t += kBatch) batch(t, std::true_type());
      if (t < n) batch(t, std::false_type());
      if (is_level.value) times(n == kTok && t0 + n < s.len ? tile_step : decay_of_tokens(a_h, n - kTok / 2));
    }
  };
  if (leveled && level) {
    if (s.len > 0) times(decay_of_tokens(a_h, kTok / 2));
    walk(std::bool_constant<leveled>());
  } else {
    walk(std::false_type());
  }
#pragma unroll
  for (int r = 0; r < rows; ++r)
    *reinterpret_cast<ulonglong2*>(s.out + (size_t)(d0 + own + r * side) * DK + 4 * j) = make_ulonglong2(st[r][0], st[r][1]);
}

// ---- one token per sequence ---------------------------------------------------------------------------
// Each state is read and written once, 128 KB a head of 128 x 128: bandwidth.  A warp takes `rows` state rows at a time, all of
// their loads under way before the first is used, a lane four k of each row; the rows' products with q are added up across
// the lanes by halving: each step exchanges half of what a lane still holds (9 shuffles for 8 rows in place of 40).
// 256 sequences x 64 heads of 128 x 128: 313 us, 101 % of the measured bandwidth.
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
    int row;
    halve<rows, W>(dot, lane, &row);
    if (j % (W / rows) == 0) o[d1 + row * side + lane / W] = from_f<T>(a.scale * dot[0]);
  }
}

constexpr int kAlone = 116 * 1024;       // bytes of shared memory with which a CTA is the only one of its SM

template <typename T, int DK, int rows, bool leveled>
cudaError_t launch_steps(const LinAttnArgs& a, bool alone, cudaStream_t s) {
  using Tiles = StepTiles<T, DK, rows>;
  static_assert(sizeof(Tiles) <= kAlone, "one size does");
  const auto kernel = k_linattn_steps<T, DK, rows, leveled>;
  const int smem = alone ? kAlone : (int)sizeof(Tiles);
  if (smem > 48 * 1024) {                                   // more than a kernel may have without asking: once per device
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAlone);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  kernel<<<dim3((unsigned)((long long)a.nseq * a.H * (a.dv / Tiles::R))), kStepThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int DK>
cudaError_t steps(const LinAttnArgs& a, cudaStream_t s) {
  // bf16 prompts are short here: four rows a lane, CTAs side by side (8 tokens x 32 heads, 1, 2 and 4 sequences: 4.6, 5.6, 7.6 us;
  // two rows 4.8, 6.0, 9.3, and a CTA per SM 6.3, 10.5, 17.0).
  // Of the shortest the state is decayed each token (64 sequences x 32 heads: 8 tokens 66 us against 71, 12 tokens
  // 94 against 95, 24 154 against 139).
  if (a.io == ERS_DTYPE_BF16)
    return a.max_len > 12 ? launch_steps<__nv_bfloat16, DK, 4, true>(a, false, s) : launch_steps<__nv_bfloat16, DK, 4, false>(a, false, s);
  // fp32 ones: a token takes a CTA of two rows a lane 44 ns and one of four 60, alone on their SM; two CTAs beside each
  // other take 70 and 95, and four of four rows 150.  CTAs may be placed beside others while SMs are idle, so where there
  // is work for one per SM it is held to that.  Of the lengths only the longest and the sum are known: as many
  // sequences as the sum has longest ones count.  1024 tokens, 128 x 128, two rows alone / two / four, us:
  //   x 8 heads   45 /  45 /  61        1024, 300 and 20 x 8      59 / 75 /  62
  //   x 16        88 /  75 /  61        1025 and 300 x 16 (dk 64) 60 / 80 / 103 (four alone: 71)
  //   x 24       138 / 104 /  96
  const long long full = min(max((a.ntokens + a.max_len / 2) / max(a.max_len, 1), 1LL), (long long)a.nseq);
  const long long ctas2 = (long long)a.H * (a.dv / StepTiles<float, DK, 2>::R), ctas4 = ctas2 / 2;
  if (full * ctas2 <= 152 && a.ntokens * ctas2 / 152 <= a.max_len + a.max_len / 4) return launch_steps<float, DK, 2, true>(a, true, s);
  // Many heads are bound by the reads of k and q from shared memory, 79 % of its cycles with four rows, which eight halve (4 x
  // 1024 x 64 heads: 547 us against 595, 40 x 100 x 16 of 64 values: 75 against 82; 2 x 1024 x 64, whose CTAs are not quite a
  // wave and a half: 321 against 305).
  if (a.ntokens * (ctas4 / 2) / 152 >= 5LL * a.max_len) return launch_steps<float, DK, 8, true>(a, false, s);
  return launch_steps<float, DK, 4, true>(a, a.ntokens * ctas4 / 152 <= a.max_len, s);
}

template <typename T, int DK>
cudaError_t decode(const LinAttnArgs& a, cudaStream_t s) {
  // A CTA per head where those fill the SMs (1024 heads: 17.1 us against 18.0, 4096: 81 against 91); fewer heads are cut up to
  // a batch of rows per warp (512: 10.5 against 12.1).
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
  constexpr int kStepLen = 8;
  // Of few tokens the recurrence is done before a chunk is, which takes 10.4 us whatever it holds (32 heads: 7.6 us for 40
  // tokens, 10.0 for 64; 64 heads: 9.6 for 32, 11.2 for 40; 512 heads: 36.8 against 38.0 for 24, 45 against 38 for 32).
  const long long heads = (long long)a.nseq * a.H;
  const int few_tokens = heads <= 32 ? 56 : heads <= 64 ? 32 : 24;
  if (a.max_len > few_tokens && linattn_tc_supported(a)) {
    // A prompt or two among many single tokens: the recurrence takes the short sequences, in a launch of its own (32 heads,
    // 97 tokens and 15 single ones: 21.7 us against 37.9 together, 2048 and 63: 98 against 135, but 97 and three: 13.9 against
    // 10.9; 2048 and 63 of 20 tokens: 193 against 134).
    if (heads > 304 && a.ntokens - a.max_len <= (long long)kStepLen * (a.nseq - 1)) {
      LinAttnArgs few = a, many = a;
      few.len1 = few.max_len = kStepLen;
      many.len0 = kStepLen + 1;
      const cudaError_t e = a.dk == 64 ? steps<64>(few, s) : steps<128>(few, s);
      return e != cudaSuccess ? e : linattn_tc(many, s);
    }
    return linattn_tc(a, s);
  }
  return a.dk == 64 ? steps<64>(a, s) : steps<128>(a, s);
}

cudaError_t linattn_decode(const LinAttnArgs& a, cudaStream_t s) {
  if (a.io == ERS_DTYPE_BF16)
    return a.dk == 64 ? decode<__nv_bfloat16, 64>(a, s) : decode<__nv_bfloat16, 128>(a, s);
  return a.dk == 64 ? decode<float, 64>(a, s) : decode<float, 128>(a, s);
}

}  // namespace ers
