// The gated delta rule over prompts in chunks of 64 tokens, bf16, on the tensor cores.
//
// With G_i the sum of a chunk's log-gates up to token i, S the state before it and C its last token:
//   A_ij = beta_i e^(G_i - G_j) k_i.k_j (j < i),   T = (I + A)^-1,   T' = T diag(beta)
//   W = T' diag(e^G) K,   U0 = T' V,   M_ij = e^(G_i - G_j) q_i.k_j (j <= i)            of the chunk alone
//   U = U0 - W S^T,   O = scale (diag(e^G) Q S^T + M U),   S <- e^(G_C) S + (diag(e^(G_C - G)) U)^T K   through the state
// Differences of G are taken between sums held as two floats, so that no gate, however strong, costs the others bits; every
// exponent is <= 0.  The first line depends on no other chunk: k_gdn_inside forms it for all chunks at once, a CTA for a chunk and
// head, and leaves W, M (as two bf16 terms), U0 (fp32) and the factors in the workspace, with Q and K as padded operand tiles.
// k_gdn_through walks a sequence's chunks, a CTA for 64 or 32 rows of a head's state.
//
// T and M are triangles with zeros as operands, so a row of A21 T11 or of U that overflows makes the rows before it in its chunk NaN as
// well (0 x infinity).  Clearing such rows and telling the outputs apart took 3 to 5 % of every prompt's time for sums that are
// beyond 3e38 either way; what is not finite among the inputs is cleared as they are read and reaches nothing before it.
//
// Precision: q, k and v are exact operands.  T' is taken as three bf16 terms (24 bits); W, S, M, U and the decayed U as
// two (16 bits and more: each is off by at most 2^-17, in the mean 2^-18.7; a third term of all of them would double the products of the
// serial loop).  The state itself is fp32 in registers, one rounded multiply-add a chunk by a factor of two floats (of one, whose
// rounding is the same each time where the gate is, a state over 32768 tokens was 4e-5 off): final states are 2e-6 to
// 5e-6 of their size off (three roundings in quadrature: 6.6e-6 at most), over 97 tokens as over 32768, and what they hold from n
// tokens ago sqrt(n / 64) 2^-24 more.
//
// What bounds it (2048 tokens x 32 heads of 128 x 128: 51 and 55 us).  k_gdn_inside: the dependent phases of a CTA, 21000 cycles
// with two a SM (loads 7400, of two products of 128 x 128 x 64 and the scores' 4200, T 4500, the rest made and stored); barriers
// are most of its stalls.  k_gdn_through: the chain of a chunk, 2900 cycles of 32 state rows (4700 of 64): the state into terms 300,
// W S^T 1300, U into terms 550, K^T U' and the state's step 760.  Where all parts of 32 rows have an SM they are taken
// (2048 x 32 heads 81 to 53 us); more CTAs than SMs would do the same operands' work twice.
#include <mutex>
#include <type_traits>

#include "ers_common.cuh"
#include "ers_internal.h"
#include "gdn_rule.cuh"
#include "tc_common.cuh"
#include "tc_terms.cuh"

namespace ers {
namespace {

using namespace tc;
using bf16 = __nv_bfloat16;

constexpr int kC = 64;                       // tokens of a chunk
constexpr uint32_t kAtom = kC * 128;         // 64 rows of 64 bf16 columns
constexpr float kLeast = -200.f;             // a lower log-gate is e^-200 = 0 in fp32 as well

// The factors of a chunk.
struct Factors {
  float since[kC];                           // e^(G_i)
  float left[kC];                            // e^(G_C - G_i)
  Decay whole;                               // e^(G_C): as two floats, for the state meets it once a chunk
  int bad;                                   // the first token with something that is not finite (kC: none)
  float pad[125];
};
static_assert(sizeof(Factors) == 1024, "whole copies");

// What k_gdn_inside leaves of a chunk: a block for each head, and Q and K for each group.
struct Layout {
  uint32_t w, m, f, u, head;                 // offsets of W (hi, lo), M (hi, lo), factors, U0 [dv / 4, 64, 4]; bytes of a block
  uint32_t group;                            // bytes of Q, then K
  size_t chunk;                              // bytes of a chunk's: heads, then groups
  __host__ __device__ Layout(int H, int G, int dk, int dv) {
    w = 0;
    m = 2 * kC * dk * 2;
    f = m + 2 * kAtom;
    u = f + (uint32_t)sizeof(Factors);
    head = u + kC * dv * 4;
    group = 2 * kC * dk * 2;
    chunk = (size_t)H * head + (size_t)G * group;
  }
};

// The chunks of sequence i, which starts at token t0, are numbers t0 / kC + min(i, t0 / len0) on, if it has len0 tokens or more: from
// one such sequence to the next the minimum grows by one at least, so that as many as there can be lie between their first ones,
// and sequences of fewer tokens take no numbers.
__device__ __forceinline__ int first_number(const DeltaArgs& a, int t0, int i) {
  return t0 / kC + (a.len0 == 0 ? i : min(i, t0 / a.len0));
}
long long chunk_numbers(const DeltaArgs& a) { return a.ntokens / kC + a.most; }

// Whether the sequences' borders ascend within [0, ntokens], all of them: chunks are found by them.  By all threads.
__device__ __forceinline__ bool ascending(const DeltaArgs& a) {
  bool ok = true;
  for (int x = threadIdx.x; x < a.nseq; x += blockDim.x) {
    const int t0 = a.cu[x], t1 = a.cu[x + 1];
    ok &= 0 <= t0 && t0 <= t1 && t1 <= a.ntokens;
  }
  return __syncthreads_and(ok);
}

__device__ __forceinline__ bool not_finite(uint4 v) {
  const auto bad = [](uint32_t u) { return (u & 0x7f800000u) == 0x7f800000u || (u & 0x7f80u) == 0x7f80u; };
  return bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
}

// X fp32 values as N bf16 terms: word j of term n holds values 2 j and 2 j + 1.
template <int N, int X>
__device__ __forceinline__ void terms_of(const float (&v)[X], uint32_t (&t)[N][X / 2]) {
#pragma unroll
  for (int j = 0; j < X / 2; ++j) {
    uint64_t p = pair(v[2 * j], v[2 * j + 1]);
#pragma unroll
    for (int n = 0; n < N; ++n) t[n][j] = n == N - 1 ? round2(p) : take_term(p);
  }
}
// columns x on of a row of an operand tile
template <int W>
__device__ __forceinline__ void row_to(uint8_t* tile, uint32_t rows, uint32_t r, uint32_t x, const uint32_t (&t)[W]) {
#pragma unroll
  for (int j = 0; j < W; j += 4)
    *reinterpret_cast<uint4*>(tile + sw128(rows, r, x + 2 * j)) = make_uint4(t[j], t[j + 1], t[j + 2], t[j + 3]);
}
__device__ __forceinline__ void tmem_values(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32_begin(at, r);
  arrived(r);
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}

__device__ __forceinline__ void tmem_values(uint32_t at, float (&v)[16]) { tmem_ld16(at, v); }
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// ---- inside the chunks ------------------------------------------------------------------------------------------
// Two CTAs per SM: one's exponentials and substitutions under the other's products.  A thread owns a lane of tensor memory (a
// row: of Q K^T and T' V below 64, of K K^T and W from there) and the columns x0 .. + 31 of every 64.
constexpr int kInside = 256, kLd = kC + 4;
constexpr uint32_t kColD = 0, kColT = 128, kInsideCols = 256;

template <int DK, int DV>
struct InsideSmem {
  alignas(1024) uint8_t qk[2 * kC * DK * 2];   // rows 0-63 Q, 64-127 K
  alignas(1024) uint8_t v[kC * DV * 2];
  alignas(1024) uint8_t m[2 * kAtom];          // M hi, lo on their way out (W goes by the place of Q and K)
  alignas(16) float a[kC][kLd];
  alignas(16) float t[kC][kLd];
  alignas(16) float x[32][36];
  alignas(16) float2 sum[kC];                  // of gates up to a token, as two floats, times log2 e
  alignas(16) float beta[kC];
  alignas(16) float since[kC];
  float gate[kC];
  uint64_t bar;
  uint32_t tmem;
  int bad;
};

__device__ __forceinline__ float exp2_of(float x) {   // 2 units in the last place; 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// T's blocks below pairs of diagonal blocks that are done, s x s each: -T22 (A21 T11), 2 x 4 outputs a thread.
template <int s>
__device__ __forceinline__ void join_blocks(float (&a)[kC][kLd], float (&t)[kC][kLd], float (&x)[32][36]) {
  constexpr int pairs = kC / (2 * s), threads = s * s / 8;   // of a pair
  const int p = threadIdx.x / threads, e = threadIdx.x % threads, r = e / (s / 4) * 2, c = e % (s / 4) * 4, b = p * 2 * s;
  float acc[2][4];
  const auto multiply = [&](const float* left, const float* right, int ld) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j / 4][j % 4] = 0.f;
#pragma unroll
    for (int k = 0; k < s; k += 4) {
      const float4 f = *reinterpret_cast<const float4*>(left + k), g = *reinterpret_cast<const float4*>(left + kLd + k);
      const float l[2][4] = {{f.x, f.y, f.z, f.w}, {g.x, g.y, g.z, g.w}};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float4 v = *reinterpret_cast<const float4*>(right + (k + y) * ld);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[j][0] = fmaf(l[j][y], v.x, acc[j][0]);
          acc[j][1] = fmaf(l[j][y], v.y, acc[j][1]);
          acc[j][2] = fmaf(l[j][y], v.z, acc[j][2]);
          acc[j][3] = fmaf(l[j][y], v.w, acc[j][3]);
        }
      }
    }
  };
  if (p < pairs) {
    multiply(&a[b + s + r][b], &t[b][b + c], kLd);
#pragma unroll
    for (int j = 0; j < 2; ++j) *reinterpret_cast<float4*>(&x[p * s + r + j][c]) = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  }
  __syncthreads();
  if (p < pairs) {
    multiply(&t[b + s + r][b + s], &x[p * s][c], 36);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<float4*>(&t[b + s + r + j][b + c]) = make_float4(-acc[j][0], -acc[j][1], -acc[j][2], -acc[j][3]);
  }
  __syncthreads();
}

template <int DK, int DV>
__global__ void __launch_bounds__(kInside, 2) k_gdn_inside(const __grid_constant__ DeltaArgs a) {
  extern __shared__ __align__(1024) uint8_t gdn_smem[];
  InsideSmem<DK, DV>& sm = *reinterpret_cast<InsideSmem<DK, DV>*>(gdn_smem);
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid / 32, 0), lane = tid % 32, rep = a.H / a.G;
  const int number = blockIdx.x / a.H, h = blockIdx.x % a.H, g = h / rep;   // a chunk's heads side by side: their inputs share sectors
  if (a.len0 > 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // short sequences' recurrence
  if (!ascending(a) || (smem_u32(gdn_smem) & 1023u) != 0) return;   // (k_gdn_through reports it)
  int i = 0;
  for (int hi = a.nseq - 1; i < hi;) {         // the last sequence whose chunks start at or before this one
    const int mid = (i + hi + 1) / 2;
    if (first_number(a, a.cu[mid], mid) <= number) i = mid;
    else hi = mid - 1;
  }
  const int s0 = a.cu[i], len = a.cu[i + 1] - s0;
  const long long c0 = (long long)(number - first_number(a, s0, i)) * kC;
  if (len < a.len0 || c0 < 0 || c0 >= len) return;
  const int t0 = s0 + (int)c0, n = min(kC, len - (int)c0);
  const Layout lay(a.H, a.G, DK, DV);
  uint8_t* chunk = static_cast<uint8_t*>(a.ws) + number * lay.chunk;
  uint8_t *mine = chunk + (size_t)h * lay.head, *shared = chunk + (size_t)a.H * lay.head + (size_t)g * lay.group;

  // Tiles, zeros behind the last token and in place of what is not finite; all of a thread's loads under way at once.
  constexpr int kQ = kC * (DK / 8) / kInside, kV = kC * (DV / 8) / kInside;
  uint4 q[kQ], k[kQ], v[kV];
#pragma unroll
  for (int y = 0; y < kQ; ++y) {
    const int e = tid + y * kInside, r = e / (DK / 8), x = e % (DK / 8) * 8;
    q[y] = k[y] = make_uint4(0, 0, 0, 0);
    if (r < n) {
      const size_t from = ((size_t)(t0 + r) * a.G + g) * DK + x;
      q[y] = *reinterpret_cast<const uint4*>((const bf16*)a.q + from);
      k[y] = *reinterpret_cast<const uint4*>((const bf16*)a.k + from);
    }
  }
#pragma unroll
  for (int y = 0; y < kV; ++y) {
    const int e = tid + y * kInside, r = e / (DV / 8), x = e % (DV / 8) * 8;
    v[y] = r < n ? *reinterpret_cast<const uint4*>((const bf16*)a.v + ((size_t)(t0 + r) * a.H + h) * DV + x) : make_uint4(0, 0, 0, 0);
  }
  float gate = 0.f, beta = 0.f;
  if (tid < n) {
    gate = a.g[(size_t)(t0 + tid) * a.H + h];
    beta = a.beta[(size_t)(t0 + tid) * a.H + h];
  }
  if (warp == 0) tmem_alloc(&sm.tmem, kInsideCols);
  if (tid == 32) {
    mbar_init(&sm.bar, 1);
    fence_mbar_init();
    sm.bad = kC;
  }
  __syncthreads();
#pragma unroll
  for (int y = 0; y < kQ; ++y) {
    const int e = tid + y * kInside, r = e / (DK / 8), x = e % (DK / 8) * 8;
    if (not_finite(q[y]) || not_finite(k[y])) {
      atomicMin(&sm.bad, r);
      q[y] = k[y] = make_uint4(0, 0, 0, 0);
    }
    *reinterpret_cast<uint4*>(sm.qk + sw128(2 * kC, r, x)) = q[y];
    *reinterpret_cast<uint4*>(sm.qk + sw128(2 * kC, kC + r, x)) = k[y];
    if (h % rep == 0) {
      *reinterpret_cast<uint4*>(shared + sw128(kC, r, x)) = q[y];
      *reinterpret_cast<uint4*>(shared + kC * DK * 2 + sw128(kC, r, x)) = k[y];
    }
  }
#pragma unroll
  for (int y = 0; y < kV; ++y) {
    const int e = tid + y * kInside, r = e / (DV / 8), x = e % (DV / 8) * 8;
    if (not_finite(v[y])) {
      atomicMin(&sm.bad, r);
      v[y] = make_uint4(0, 0, 0, 0);
    }
    *reinterpret_cast<uint4*>(sm.v + sw128(kC, r, x)) = v[y];
  }
  if (tid < kC) {
    if (!(fabsf(beta) < INFINITY) || !(gate < INFINITY)) atomicMin(&sm.bad, tid);
    sm.gate[tid] = fmaxf(gate, kLeast) * 1.44269504088896340736f;
    sm.beta[tid] = beta;
  }
  fence_async_smem();
  before_sync();
  __syncthreads();
  after_sync();
  const uint32_t tb = __shfl_sync(kFull, sm.tmem, 0), quarter = tb + ((uint32_t)(tid & 96) << 16);
  const bool leader = warp == 0 && elected();
  const uint32_t qk = smem_u32(sm.qk);
  if (leader) {                                // rows 0-63 Q K^T, 64-127 K K^T
#pragma unroll
    for (int k = 0; k < DK / 16; ++k) {
      const uint32_t at = qk + (k >> 2) * 2 * kAtom + (k & 3) * 32;
      mma(tb + kColD, sdesc(at, 16, 1024), sdesc(at + kAtom, 16, 1024), idesc_bf16(128, kC, false, false), k > 0);
    }
    commit(&sm.bar);
  }
  const int used = min(n, sm.bad);             // tokens from a bad one on count as none: beta 0, gate 1
  if (warp == 3) {                             // sums of gates: two tokens a lane
    const auto gate_of = [&](int t) { return t < used ? sm.gate[t] : 0.f; };
    const df g0 = {gate_of(2 * lane), 0.f}, g1 = {gate_of(2 * lane + 1), 0.f};
    df sum = df_add(g0, g1);
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const df o = {__shfl_up_sync(kFull, sum.hi, off), __shfl_up_sync(kFull, sum.lo, off)};
      if (lane >= off) sum = df_add(o, sum);
    }
    df before = {__shfl_up_sync(kFull, sum.hi, 1), __shfl_up_sync(kFull, sum.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const df first = df_add(before, g0), all = {__shfl_sync(kFull, sum.hi, 31), __shfl_sync(kFull, sum.lo, 31)};
    Factors& f = *reinterpret_cast<Factors*>(mine + lay.f);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int t = 2 * lane + x;
      const df s = x == 0 ? first : sum;
      sm.sum[t] = make_float2(s.hi, s.lo);
      if (t >= used) sm.beta[t] = 0.f;
      f.since[t] = sm.since[t] = exp2f(s.hi + s.lo);
      f.left[t] = exp2f(df_diff(all, s));
    }
    if (lane == 0) {
      f.whole = decay_of((all.hi + all.lo) * 0.69314718055994530942f);
      f.bad = sm.bad;
    }
  }
  for (int e = tid; e < kC * kLd / 4; e += kInside) reinterpret_cast<float4*>(sm.t)[e] = make_float4(0, 0, 0, 0);
  __syncthreads();
  bool ok = mbar_wait(&sm.bar, 0, a.status);
  __syncwarp();
  after_sync();
  const int r = tid % kC, x0 = tid / 128 * 32;
  const bool upper = tid % 128 < kC;           // lanes 0-63
  {
    float v[32];
    if (x0 <= (r | 31)) {                      // (a whole warp: beyond the diagonal all is zero)
      tmem_values(quarter + kColD + x0, v);
      const df own = {sm.sum[r].x, sm.sum[r].y};
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float4 o = *reinterpret_cast<const float4*>(&sm.sum[x0 + j]);
        v[j] *= exp2_of(df_diff(own, {o.x, o.y}));
        v[j + 1] *= exp2_of(df_diff(own, {o.z, o.w}));
      }
    }
    const int keep = upper ? r - x0 : r - x0 - 1;   // the last column that is kept: with or without the diagonal
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = j <= keep ? v[j] : 0.f;
    if (upper) {                               // M
      uint32_t t[2][16];
      terms_of<2>(v, t);
      row_to(sm.m, kC, r, x0, t[0]);
      row_to(sm.m + kAtom, kC, r, x0, t[1]);
      fence_async_smem();
    } else {                                   // A
      const float beta = sm.beta[r];
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(&sm.a[r][x0 + j]) = make_float4(beta * v[j], beta * v[j + 1], beta * v[j + 2], beta * v[j + 3]);
    }
    before_sync();
  }
  __syncthreads();
  if (tid == 128) {
    bulk_s2g(mine + lay.m, sm.m, 2 * kAtom);
    bulk_commit();
  }
  // T: blocks of 8 on the diagonal by forward substitution, a column each thread, then pairs of blocks joined.
  if (tid < kC) {
    const int b = tid / 8 * 8, c = tid % 8;
    float x[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float4 f = *reinterpret_cast<const float4*>(&sm.a[b + r][b]), g = *reinterpret_cast<const float4*>(&sm.a[b + r][b + 4]);
      const float l[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
      float acc = 0.f;
#pragma unroll
      for (int y = 0; y < r; ++y) acc = fmaf(l[y], x[y], acc);
      x[r] = r < c ? 0.f : r == c ? 1.f : -acc;
      sm.t[b + r][b + c] = x[r];
    }
  }
  __syncthreads();
  join_blocks<8>(sm.a, sm.t, sm.x);
  join_blocks<16>(sm.a, sm.t, sm.x);
  join_blocks<32>(sm.a, sm.t, sm.x);
  {                                            // rows 0-63 T', 64-127 T' diag(e^G), three terms
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 t = *reinterpret_cast<const float4*>(&sm.t[r][x0 + j]), b = *reinterpret_cast<const float4*>(&sm.beta[x0 + j]);
      float4 f = *reinterpret_cast<const float4*>(&sm.since[x0 + j]);
      if (upper) f = make_float4(1.f, 1.f, 1.f, 1.f);
      v[j] = t.x * b.x * f.x;
      v[j + 1] = t.y * b.y * f.y;
      v[j + 2] = t.z * b.z * f.z;
      v[j + 3] = t.w * b.w * f.w;
    }
    uint32_t t[3][16], c[32];
    terms_of<3>(v, t);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      c[j] = t[0][j];
      c[16 + j] = t[1][j];
    }
    tmem_st32(quarter + kColT + x0, c);        // of 32 columns hi and mid; behind those of all, lo
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      c[j] = t[2][j];
      c[16 + j] = 0;
    }
    tmem_st32(quarter + kColT + 64 + x0, c);
    tmem_wait_st();
    before_sync();
  }
  __syncthreads();
  after_sync();
  // U0 = T' V from rows 0-63, W = (T' diag(e^G)) K from rows 64-127
  const auto product = [&](uint32_t tile, uint32_t lbo, uint32_t N) {
    uint32_t more = 0;
#pragma unroll
    for (int k = 0; k < kC / 16; ++k)
#pragma unroll
      for (int term = 0; term < 3; ++term, more = 1)
        mma_ts(tb + kColD, tb + kColT + k / 2 * 32 + (term < 2 ? 16 * term : 64) + k % 2 * 8, sdesc(tile + k * 2048, lbo, 1024),
               idesc_bf16(128, N, false, true), more);
    commit(&sm.bar);
  };
  if (ok && leader) product(smem_u32(sm.v), kAtom, DV);
  ok = ok && mbar_wait(&sm.bar, 1, a.status);
  __syncwarp();
  after_sync();
  if (upper) {
    float4* u = reinterpret_cast<float4*>(mine + lay.u) + r;
#pragma unroll
    for (int x = x0; x < DV; x += 64) {
      float v[32];
      tmem_values(quarter + kColD + x, v);
#pragma unroll
      for (int j = 0; j < 32; j += 4) u[(x + j) / 4 * kC] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
  }
  before_sync();
  __syncthreads();
  after_sync();
  if (ok && leader) product(qk + kAtom, 2 * kAtom, DK);
  ok = ok && mbar_wait(&sm.bar, 0, a.status);
  __syncwarp();
  after_sync();
  if (!upper) {
#pragma unroll
    for (int x = x0; x < DK; x += 64) {
      float v[32];
      tmem_values(quarter + kColD + x, v);
      uint32_t t[2][16];
      terms_of<2>(v, t);
      row_to(sm.qk, kC, r, x, t[0]);
      row_to(sm.qk + kC * DK * 2, kC, r, x, t[1]);
    }
    fence_async_smem();
  }
  __syncthreads();
  if (tid == 128) {
    bulk_s2g(mine + lay.w, sm.qk, 2 * kC * DK * 2);
    bulk_commit();
    bulk_wait_read();
  }
  if (!ok && tid == 0) {                       // a wait gave up: no MMA may be left in flight
    const uint64_t start = globaltimer();
    while (globaltimer() - start < 2000000) {}
  }
  before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tb, kInsideCols);
}

// ---- through the state ----------------------------------------------------------------------------------------------
// P rows of a head's state a CTA.  Warps 0-7 own the state S^T, thread by thread one k (lane quarter warp % 4) and half of the rows
// (warp / 4); those of quarters 2 and 3 make U, those of 0 and 1 the outputs.  Warp 8 loads, warp 9 issues.
constexpr int kOwners = 256, kLoadThread = 256, kThrough = 320;
// Products with an operand of two terms take both as 2 P columns: the other operand is read once, and the halves are added
// up by those who read them.
template <int P>
struct Cols {
  static constexpr uint32_t one = 0, two = 2 * P, three = 3 * P, out = 5 * P, all = P == 64 ? 512 : 256;
};

// the sums of columns and those P further on
template <int P, int X>
__device__ __forceinline__ void tmem_sums(uint32_t at, float (&v)[X]) {
  float w[X];
  tmem_values(at, v);
  tmem_values(at + P, w);
#pragma unroll
  for (int j = 0; j < X; ++j) v[j] += w[j];
}

struct Hdr {
  uint64_t full[2], empty[2], s_ready, u_ready, u_decayed, u_written, s_done, o_done, o_free;
  uint32_t tmem;
  int dead;                                  // a wait gave up: no further wait waits, no copy or MMA is issued
  int seq, counts[kThrough / 32];            // for chunk_sequence
};

// The n-th of the sequences that have chunks, where not all of them can; -1: there are fewer.  By all threads.
__device__ __forceinline__ int chunk_sequence(const DeltaArgs& a, int n, Hdr& hd) {
  if (a.most == a.nseq) return n;
#pragma unroll 1
  for (int x0 = 0; x0 < a.nseq; x0 += kThrough) {
    const int x = x0 + threadIdx.x;
    const bool is = x < a.nseq && a.cu[x + 1] - a.cu[x] >= a.len0;
    const int count = __syncthreads_count(is);
    if (n >= count) {
      n -= count;
      continue;
    }
    const uint32_t mine = __ballot_sync(kFull, is);
    if (threadIdx.x % 32 == 0) hd.counts[threadIdx.x / 32] = __popc(mine);
    __syncthreads();
    for (int w = 0; w < threadIdx.x / 32; ++w) n -= hd.counts[w];
    if (is && __popc(mine & ((1u << threadIdx.x % 32) - 1)) == n) hd.seq = x;
    __syncthreads();
    return hd.seq;
  }
  return -1;
}

// Shared memory: two stages, S^T as two terms side by side [dk x 2 P], U and the decayed U as two terms each [64 x 2 P].
// A stage: for each 64 columns Q's and W hi's atoms, one A operand of 128 rows; W lo's, as rows 64-127 of one whose other rows are
// whatever lies before; M hi and lo, rows 0-63 of two whose others are what lies behind; K; the factors.
template <int DK, int P>
struct Stage {
  static constexpr uint32_t atoms = DK / 64, wlo = 2 * atoms * kAtom, m = wlo + atoms * kAtom, k = m + 2 * kAtom,
                            f = k + atoms * kAtom, size = f + sizeof(Factors);
  static constexpr uint32_t bytes = size;      // all of it arrives by copies
  static constexpr uint32_t term = P / 32 * kAtom;                 // both terms of U
  static constexpr uint32_t s = 2 * size, u = s + P / 32 * DK * 128, hdr = u + 2 * term, smem = hdr + sizeof(Hdr);
  static_assert(smem <= 227 * 1024 && size % 1024 == 0, "one CTA's shared memory; whole swizzle groups");
};

__device__ __forceinline__ bool wait(Hdr& hd, uint64_t* bar, uint32_t parity, int32_t* status) {
  uint64_t t0 = 0;
#pragma unroll 1
  while (!mbar_try(bar, parity & 1u)) {
    const uint64_t now = globaltimer();
    if (*(volatile int*)&hd.dead != 0) return false;
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      if (status != nullptr) atomicCAS(status, 0, ERS_ETIMEOUT);
      *(volatile int*)&hd.dead = 1;
    }
  }
  return true;
}
__device__ __forceinline__ bool dead(const Hdr& hd) { return *(const volatile int*)&hd.dead != 0; }

template <int DK, int P>
__global__ void __launch_bounds__(kThrough, 1) k_gdn_through(const __grid_constant__ DeltaArgs a) {
  using St = Stage<DK, P>;
  using Col = Cols<P>;
  constexpr int X = P / 2;                     // state rows of a thread
  extern __shared__ __align__(1024) uint8_t gdn_smem[];
  Hdr& hd = *reinterpret_cast<Hdr*>(gdn_smem + St::hdr);
  const int parts = a.dv / P, part = blockIdx.x % parts, unit = blockIdx.x / parts, h = unit % a.H;
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid / 32, 0), lane = tid % 32;
  if (!ascending(a) || (smem_u32(gdn_smem) & 1023u) != 0) {
    if (tid == 0) report(a.status, (smem_u32(gdn_smem) & 1023u) != 0 ? ERS_ECUDA : ERS_EINVAL);
    return;
  }
  DeltaSeq seq;
  const int i = chunk_sequence(a, unit / a.H, hd);
  if (i < 0 || !delta_seq(a, i, h, &seq)) return;
  const int chunks = (seq.len + kC - 1) / kC, d0 = part * P;
  const Layout lay(a.H, a.G, DK, a.dv);
  const uint8_t* first = static_cast<const uint8_t*>(a.ws) + (size_t)first_number(a, seq.t0, i) * lay.chunk;
  const uint8_t *mine = first + (size_t)h * lay.head, *shared = first + (size_t)a.H * lay.head + (size_t)(h / (a.H / a.G)) * lay.group;

  if (warp == 9) tmem_alloc(&hd.tmem, Col::all);
  if (tid == kLoadThread) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&hd.full[b], 1);
      mbar_init(&hd.empty[b], 1 + kOwners);
    }
    mbar_init(&hd.s_ready, kOwners);
    mbar_init(&hd.u_ready, 1);
    mbar_init(&hd.u_decayed, kOwners / 2);
    mbar_init(&hd.u_written, kOwners / 2);
    mbar_init(&hd.s_done, 1);
    mbar_init(&hd.o_done, 1);
    mbar_init(&hd.o_free, kOwners / 2);
    fence_mbar_init();
    hd.dead = 0;
  }
  before_sync();
  __syncthreads();
  after_sync();
  const uint32_t tb = __shfl_sync(kFull, hd.tmem, 0);

  if (warp == 8) {
    // ---- loads -----------------------------------------------------------------------------------------------
    if (lane == 0) {
      for (int c = 0; c < chunks; ++c) {
        const int b = c & 1;
        if (c >= 2) wait(hd, &hd.empty[b], (c >> 1) - 1, a.status);
        if (dead(hd)) break;
        uint8_t* to = gdn_smem + b * St::size;
        const uint8_t *w = mine + c * lay.chunk, *qk = shared + c * lay.chunk;
        uint64_t* bar = &hd.full[b];
        mbar_arrive_expect_tx(bar, St::bytes);
        for (uint32_t x = 0; x < St::atoms; ++x) {
          bulk_g2s(to + 2 * x * kAtom, qk + x * kAtom, kAtom, bar);
          bulk_g2s(to + (2 * x + 1) * kAtom, w + x * kAtom, kAtom, bar);
        }
        bulk_g2s(to + St::wlo, w + St::atoms * kAtom, St::atoms * kAtom, bar);
        bulk_g2s(to + St::m, w + lay.m, 2 * kAtom, bar);
        bulk_g2s(to + St::k, qk + St::atoms * kAtom, St::atoms * kAtom, bar);
        bulk_g2s(to + St::f, w + lay.f, sizeof(Factors), bar);
      }
    }
  } else if (warp == 9) {
    // ---- products --------------------------------------------------------------------------------------------
    constexpr uint32_t id = idesc_bf16(128, P, false, true), id2 = idesc_bf16(128, 2 * P, false, true),
                       id3 = idesc_bf16(128, 2 * P, true, true);
    const bool leader = elected();
    const uint32_t st = smem_u32(gdn_smem + St::s), ut = smem_u32(gdn_smem + St::u);
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const uint32_t base = smem_u32(gdn_smem + (c & 1) * St::size);
      if (!wait(hd, &hd.full[c & 1], c >> 1, a.status) || !wait(hd, &hd.s_ready, c, a.status)) break;
      after_sync();
      if (leader) {
#pragma unroll
        for (int k = 0; k < DK / 16; ++k)      // rows 0-63 Q S^T, 64-127 W S^T
          mma(tb + Col::one, sdesc(base + (k >> 2) * 2 * kAtom + (k & 3) * 32, 16, 1024), sdesc(st + k * 2048, DK * 128, 1024), id2, k > 0);
#pragma unroll
        for (int k = 0; k < DK / 16; ++k)      // rows 64-127
          mma(tb + Col::two, sdesc(base + St::wlo - kAtom + (k >> 2) * kAtom + (k & 3) * 32, 16, 1024),
              sdesc(st + k * 2048, DK * 128, 1024), id, k > 0);
        commit(&hd.u_ready);
      }
      if (!wait(hd, &hd.u_decayed, c, a.status)) break;
      after_sync();
      if (leader) {
#pragma unroll
        for (int k = 0; k < kC / 16; ++k)      // K^T U'
          mma(tb + Col::three, sdesc(base + St::k + k * 2048, kAtom, 1024), sdesc(ut + St::term + k * 2048, kAtom, 1024), id3, k > 0);
        commit(&hd.s_done);
      }
      if (!wait(hd, &hd.u_written, c, a.status) || (c > 0 && !wait(hd, &hd.o_free, c - 1, a.status))) break;
      after_sync();
      if (leader) {
#pragma unroll
        for (int k = 0; k < kC / 16; ++k)      // M hi U
          mma(tb + Col::out, sdesc(base + St::m + k * 32, 16, 1024), sdesc(ut + k * 2048, kAtom, 1024), id2, k > 0);
#pragma unroll
        for (int k = 0; k < kC / 16; ++k)      // M lo U hi
          mma(tb + Col::out, sdesc(base + St::m + kAtom + k * 32, 16, 1024), sdesc(ut + k * 2048, kAtom, 1024), id, 1);
        commit(&hd.o_done);
        commit(&hd.empty[c & 1]);
      }
    }
  } else {
    // ---- the state, U and the outputs ------------------------------------------------------------------------
    const int r = tid % 128, x0 = tid / 128 * X, row = r % kC;   // k of the state; token of U or the outputs
    const bool makes_u = r >= kC, holds = r < DK;
    const uint32_t quarter = tb + ((uint32_t)(r & ~31) << 16);
    float s[X];
#pragma unroll
    for (int j = 0; j < X; ++j) s[j] = holds && seq.in != nullptr ? seq.in[(size_t)(d0 + x0 + j) * DK + r] : 0.f;
    bool poisoned = false;
    float u[X], since = 0.f;                  // U, or the last chunk's Q S^T, and its rows' factors
    int bad = kC;
    bool spoiled = false;
    const auto outputs = [&](int c) {          // of chunk c
      wait(hd, &hd.o_done, c, a.status);
      __syncwarp();
      after_sync();
      float o[X];
      tmem_sums<P>(quarter + Col::out + x0, o);
      before_sync();
      mbar_arrive(&hd.o_free);
      if (row >= seq.len - c * kC || dead(hd)) return;
      bf16* to = (bf16*)a.o + ((size_t)(seq.t0 + c * kC + row) * a.H + h) * a.dv + d0 + x0;
      uint32_t w[X / 2];
#pragma unroll
      for (int j = 0; j < X / 2; ++j)
        w[j] = spoiled ? 0x7fff7fffu : pack_bf16x2(a.scale * fmaf(since, u[2 * j], o[2 * j]), a.scale * fmaf(since, u[2 * j + 1], o[2 * j + 1]));
#pragma unroll
      for (int j = 0; j < X / 2; j += 4) *reinterpret_cast<uint4*>(to + 2 * j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
    };
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      // the state as an operand
      if (holds) {
        uint32_t t[2][X / 2];
        terms_of<2>(s, t);
        row_to(gdn_smem + St::s, DK, r, x0, t[0]);
        row_to(gdn_smem + St::s, DK, r, P + x0, t[1]);
      }
      fence_async_smem();
      before_sync();
      mbar_arrive(&hd.s_ready);
      if (!makes_u && c > 0) outputs(c - 1);
      if (makes_u) {                           // on its way while the product is
        const float4* u0 = reinterpret_cast<const float4*>(mine + c * lay.chunk + lay.u) + (d0 + x0) / 4 * kC + row;
#pragma unroll
        for (int j = 0; j < X; j += 4) {
          const float4 v = u0[j / 4 * kC];
          u[j] = v.x;
          u[j + 1] = v.y;
          u[j + 2] = v.z;
          u[j + 3] = v.w;
        }
      }
      wait(hd, &hd.full[c & 1], c >> 1, a.status);
      const Factors& f = *reinterpret_cast<const Factors*>(gdn_smem + (c & 1) * St::size + St::f);
      const Decay whole = f.whole;
      const float left = f.left[row];
      since = f.since[row];
      bad = f.bad;
      mbar_arrive(&hd.empty[c & 1]);
      spoiled = poisoned || row >= bad;
      poisoned = poisoned || bad < kC;
      wait(hd, &hd.u_ready, c, a.status);
      __syncwarp();
      after_sync();
      if (makes_u) {
        float v[X];
        tmem_sums<P>(quarter + Col::one + x0, v);
#pragma unroll
        for (int j = 0; j < X; ++j) u[j] -= v[j];
        tmem_values(quarter + Col::two + x0, v);
#pragma unroll
        for (int j = 0; j < X; ++j) {
          u[j] -= v[j];
          v[j] = u[j] * left;
        }
        uint32_t t[2][X / 2];                     // first what the state waits for
        terms_of<2>(v, t);
        row_to(gdn_smem + St::u + St::term, kC, row, x0, t[0]);
        row_to(gdn_smem + St::u + St::term, kC, row, P + x0, t[1]);
        fence_async_smem();
        before_sync();
        mbar_arrive(&hd.u_decayed);
        if (c > 0) wait(hd, &hd.o_done, c - 1, a.status);   // U's tiles have been read
        terms_of<2>(u, t);
        row_to(gdn_smem + St::u, kC, row, x0, t[0]);
        row_to(gdn_smem + St::u, kC, row, P + x0, t[1]);
        fence_async_smem();
        mbar_arrive(&hd.u_written);
      } else {
        tmem_sums<P>(quarter + Col::one + x0, u);
        before_sync();
      }
      wait(hd, &hd.s_done, c, a.status);
      __syncwarp();
      after_sync();
      float v[X];
      tmem_sums<P>(quarter + Col::three + x0, v);
#pragma unroll
      for (int j = 0; j < X; ++j) s[j] = whole.step(s[j], v[j]);
      before_sync();
    }
    if (chunks > 0 && !makes_u) outputs(chunks - 1);
    if (holds && !dead(hd)) {
#pragma unroll
      for (int j = 0; j < X; ++j) seq.out[(size_t)(d0 + x0 + j) * DK + r] = poisoned ? __int_as_float(0x7fffffff) : s[j];
    }
  }
  __syncwarp();
  if (tid == kLoadThread && dead(hd)) {        // no copy or MMA may be left in flight: 2 ms are a thousand times what one takes
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000) {}
  }
  before_sync();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tb, Col::all);
}

// ---- host side ---------------------------------------------------------------------------------------------------------
template <typename F>
cudaError_t allow(F kernel, int smem, bool (&done)[64], std::mutex& mu) {   // its shared memory, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  done[dev] = e == cudaSuccess;
  return e;
}

template <int DK, int P>
cudaError_t launch_through(const DeltaArgs& a, cudaStream_t s) {
  static std::mutex mu;
  static bool done[64] = {};
  const cudaError_t e = allow(k_gdn_through<DK, P>, Stage<DK, P>::smem, done, mu);
  if (e != cudaSuccess) return e;
  k_gdn_through<DK, P><<<(unsigned)((long long)a.most * a.H * (a.dv / P)), kThrough, Stage<DK, P>::smem, s>>>(a);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t launch(const DeltaArgs& a, const DeltaArgs* few, cudaStream_t s) {
  static std::mutex mu;
  static bool done[64] = {};
  cudaError_t e = allow(k_gdn_inside<DK, DV>, sizeof(InsideSmem<DK, DV>), done, mu);
  if (e != cudaSuccess) return e;
  k_gdn_inside<DK, DV><<<(unsigned)(chunk_numbers(a) * a.H), kInside, sizeof(InsideSmem<DK, DV>), s>>>(a);
  e = cudaGetLastError();
  if (e == cudaSuccess && few != nullptr) e = gdn_steps_beside(*few, s);
  if (e != cudaSuccess) return e;
  // 32 rows a CTA while every one of those has an SM for itself (2048 x 32 heads: 53 us, by 64 rows 81)
  return (long long)a.most * a.H * (DV / 32) <= 152 ? launch_through<DK, 32>(a, s) : launch_through<DK, 64>(a, s);
}

}  // namespace

size_t gdn_tc_workspace(const DeltaArgs& a) {
  return align256(Layout(a.H, a.G, a.dk, a.dv).chunk * chunk_numbers(a));
}

cudaError_t gdn_tc(const DeltaArgs& a, const DeltaArgs* few, cudaStream_t s) {
  if (a.dk == 64) return a.dv == 64 ? launch<64, 64>(a, few, s) : launch<64, 128>(a, few, s);
  return a.dv == 64 ? launch<128, 64>(a, few, s) : launch<128, 128>(a, few, s);
}

}  // namespace ers
