// Linear attention with a decay per head over prompts, on the tensor cores (bf16 io).
//
// Chunks of 128 tokens; rows i, j of a chunk of n tokens that starts from state H ([dv x dk]), lambda = exp(a):
//   P[i,j] = (q_i . k_j) lambda^(i-j)  [j <= i]
//   O[i]   = scale * (sum_j P[i,j] v_j + lambda^(i+1) H q_i)
//   H'     = lambda^n H + sum_j (lambda^(n-1-j) v_j) k_j^T
// Four contractions of 128 x 128 x 128 (at dk = dv = 128), tcgen05 kind::f16 with fp32 accumulators:
//   S = Q K^T                                    A, B from shared memory (TMA tiles)
//   O = Q H^T, scaled by lambda^(i+1) in place   B = H as bf16 hi + lo (two chains)
//   O += P V                                     A = P as bf16 hi + lo in tensor memory, over S
//   H += V'^T K                                  A = V' = lambda^(n-1-j) v_j as hi + mid + lo in tensor memory
// Operands made from fp32 values are split so that outputs keep 16 significant bits before their one rounding (a single
// bf16 term would cost half as much again as that rounding) and states all 24.  The state stays in tensor memory in
// fp32 from chunk to chunk.
//
// What bounds it: at one CTA per SM a chunk moves 128 KB (2.9 us of an SM's share of the memory), 8 MMA chains of
// 4.2 MFLOP and about 3000 issue slots of operand making per scheduler, in one dependent loop through the state.  So the
// warps are specialised: warp 8 loads and stores tiles (TMA; two buffers for K and V, one for Q), warp 9 issues every MMA, warps 0-3 own the
// rows i (scores, outputs), warps 4-7 the rows of the state (V', H), and the two groups run side by side.
//
// A long sequence of few heads is split over the CTAs of a cluster, each a run of chunks: every CTA but the
// last first forms its run's own end state (K and V only), the cluster turns those into start states through
// distributed shared memory, and then all walk their runs.
#include <math.h>
#include <string.h>

#include <mutex>

#include "linattn.cuh"
#include "tc_common.cuh"
#include "tma_host.h"

namespace ers {
namespace {

using namespace tc;
using bf16 = __nv_bfloat16;

constexpr int kC = 128;                  // tokens of a chunk
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kBlock = 320;
constexpr uint32_t kColS = 0, kColO = 128, kColH = 256, kColV = 384, kVStage = 48, kTmemCols = 512;
constexpr uint32_t kBarState = 1;       // named barrier of warps 4-7

struct Hdr {
  alignas(16) float w[2][kC];        // lambda^(n-1-j), 0 from n on: a full chunk, the last chunk (read 16 bytes at a time)
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full, q_empty;   // tile buffers
  uint64_t s_ready, o2_ready, o_ready, kv_done, v_free[2];    // completed by the tensor core
  uint64_t pv_go, o_free, o_staged, h_ready, v_ready[2];      // by the warpgroups
  uint32_t tmem;
  int dead;                          // a wait gave up: no further wait waits, no copy or MMA is issued
  float step_hi, step_lo;            // lambda^128 as two floats,
  float last_hi, last_lo;            // lambda^n of the sequence's last chunk
  float power[kC + 1];               // lambda^j
  int bad[2][4];                     // a chunk's value columns (by state warp) hold something not finite,
  uint8_t first_bad[2][kC];          // from this token on (128: nowhere)
};

struct Maps {
  CUtensorMap q, k, v, o;
};

template <int DK, int DV>
struct Shape {
  static constexpr uint32_t ktile = kC * DK * 2, vtile = kC * DV * 2;
  static constexpr uint32_t hterm = DV * DK * 2;       // one bf16 term of the state operand
  static constexpr uint32_t smem = 1024 + sizeof(Hdr) + 3 * ktile + 2 * vtile + 2 * hterm;
  static_assert(smem <= 227 * 1024, "one CTA's shared memory");
};

// ---- waits -----------------------------------------------------------------------------------------------
__device__ __forceinline__ void wait(Hdr& hd, uint64_t* bar, uint32_t parity, int32_t* status) {
  if (mbar_try(bar, parity)) return;
  const uint64_t t0 = globaltimer();
  while (!mbar_try(bar, parity)) {
    if (*(volatile int*)&hd.dead != 0) return;
    if (globaltimer() - t0 > kWaitLimitNs) {
      if (status != nullptr) atomicCAS(status, 0, ERS_ETIMEOUT);
      *(volatile int*)&hd.dead = 1;
      return;
    }
  }
}
__device__ __forceinline__ bool dead(const Hdr& hd) { return *(const volatile int*)&hd.dead != 0; }

// ---- PTX that the other engines do not need ------------------------------------------------------------------
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_ld(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void peer_st(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// ---- bf16 terms ------------------------------------------------------------------------------------------------
// (a, b) -> packed bf16 hi terms (a in the low half), leaving the remainders in a and b
__device__ __forceinline__ uint32_t take_term(float& a, float& b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&v);
  a = __fsub_rn(a, __uint_as_float(u << 16));
  b = __fsub_rn(b, __uint_as_float(u & 0xffff0000u));
  return u;
}
__device__ __forceinline__ uint32_t last_term(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A CTA's share of the work.
struct Run {
  int t0, len;         // the sequence's tokens
  int c0, c1;          // this CTA's chunks
  int last_run;        // the rank that ends the sequence
  int per;             // chunks of every run but the last
};

template <int DK, int DV>
struct Cta {
  using Sh = Shape<DK, DV>;
  const LinAttnArgs& a;
  const Maps& maps;
  Hdr& hd;
  uint8_t* tiles;      // K, K, V, V, Q
  uint8_t* hop;        // state operand: hi, then lo; between the two passes the fp32 state itself
  uint32_t tb;
  int h, g;
  Run run;

  // Chunks are numbered m = 0, 1, ... over both passes; number m uses K and V buffer m % 2 for the m / 2th time.
  __device__ __forceinline__ uint8_t* kbuf(int m) const { return tiles + (m & 1) * Sh::ktile; }
  __device__ __forceinline__ uint8_t* vbuf(int m) const { return tiles + 2 * Sh::ktile + (m & 1) * Sh::vtile; }
  __device__ __forceinline__ uint8_t* qbuf() const { return tiles + 2 * Sh::ktile + 2 * Sh::vtile; }
  __device__ __forceinline__ int rows(int c) const { return run.len - c * kC < kC ? run.len - c * kC : kC; }
  __device__ __forceinline__ void wt(uint64_t* bar, uint32_t parity) const { wait(hd, bar, parity & 1u, a.status); }

  // ---- warp 8: tiles in, outputs out ------------------------------------------------------------------------
  __device__ __forceinline__ void load(uint8_t* to, const CUtensorMap* map, int d, int head, int c, uint64_t* bar) const {
    if (dead(hd)) return;
    mbar_arrive_expect_tx(bar, kC * d * 2);
    for (int x = 0; x < d; x += 64) tma_load_3d(to + x / 64 * (kC * 128), map, x, head, run.t0 + c * kC, bar);
  }
  __device__ __forceinline__ void load_k(int m, int c) const {
    if (m >= 2) wt(&hd.k_empty[m & 1], m / 2 - 1);
    load(kbuf(m), &maps.k, DK, g, c, &hd.k_full[m & 1]);
  }
  __device__ __forceinline__ void load_v(int m, int c) const {
    if (m >= 2) wt(&hd.v_empty[m & 1], m / 2 - 1);
    load(vbuf(m), &maps.v, DV, h, c, &hd.v_full[m & 1]);
  }
  __device__ __forceinline__ void load_states() const {
    for (int c = run.c0; c < run.c1; ++c) {
      load_k(c - run.c0, c);
      load_v(c - run.c0, c);
    }
  }
  // In the order in which buffers come free: Q after Q H^T, K after V'^T K, V when the output, which takes its
  // place after P V, has been stored.  (The rows of a short chunk are stored by their owners.)
  __device__ __forceinline__ void load_chunks(int m0) const {
    const int n = run.c1 - run.c0;
    load_k(m0, run.c0);
    load(qbuf(), &maps.q, DK, g, run.c0, &hd.q_full);
    load_v(m0, run.c0);
    if (n > 1) {
      load_k(m0 + 1, run.c0 + 1);
      load_v(m0 + 1, run.c0 + 1);
    }
    for (int i = 0; i < n; ++i) {
      const int c = run.c0 + i;
      if (i + 1 < n) {
        wt(&hd.q_empty, i);
        load(qbuf(), &maps.q, DK, g, c + 1, &hd.q_full);
      }
      if (i + 2 < n) load_k(m0 + i + 2, c + 2);
      wt(&hd.o_staged, i);
      if (!dead(hd) && rows(c) == kC) {
        for (int x = 0; x < DV; x += 64)
          tma_store_3d(&maps.o, vbuf(m0 + i) + x / 64 * (kC * 128), x, h, run.t0 + c * kC);
        bulk_commit();
        bulk_wait_read();
      }
      mbar_arrive(&hd.v_empty[(m0 + i) & 1]);
      if (i + 2 < n) load_v(m0 + i + 2, c + 2);
    }
  }
  // After a wait gave up: no copy or MMA may be left in flight when the CTA ends.
  __device__ __forceinline__ void drain() const {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000) {}   // 2 ms: a thousand times what a tile or an MMA takes
  }

  // ---- warp 9: every MMA --------------------------------------------------------------------------------------
  // one quarter (32 tokens) of H += V'^T K
  __device__ __forceinline__ void state_quarter(uint32_t kt, int quarter, uint32_t stage, bool accumulate) const {
    constexpr uint32_t id = idesc_bf16(128, DK, false, true);
    for (int term = 0; term < 3; ++term)
      for (int ks = 0; ks < 2; ++ks)
        mma_ts(tb + kColH, tb + kColV + stage * kVStage + term * 16 + ks * 8,
               sdesc(kt + (32 * quarter + 16 * ks) * 128, kC * 128, 1024), id, accumulate || term + ks > 0);
  }
  __device__ __forceinline__ void issue_states(int& quarters) const {
    const int n = run.c1 - run.c0;
    for (int m = 0; m < n; ++m) {
      wt(&hd.k_full[m & 1], m / 2);
      after_sync();
      for (int quarter = 0; quarter < 4; ++quarter, ++quarters) {
        wt(&hd.v_ready[quarters & 1], quarters >> 1);
        after_sync();
        if (dead(hd)) return;
        state_quarter(smem_u32(kbuf(m)), quarter, quarters & 1, m > 0 || quarter > 0);
        commit(&hd.v_free[quarters & 1]);
      }
      commit(&hd.k_empty[m & 1]);
      commit(&hd.v_empty[m & 1]);
    }
    commit(&hd.kv_done);
  }
  __device__ __forceinline__ void issue_chunks(int m0, int quarters, bool fresh) const {
    constexpr uint32_t id_s = idesc_bf16(128, kC, false, false), id_h = idesc_bf16(128, DV, false, false),
                       id_v = idesc_bf16(128, DV, false, true);
    const uint32_t qt = smem_u32(qbuf()), ht = smem_u32(hop);
    for (int i = 0; i < run.c1 - run.c0; ++i) {
      const int m = m0 + i;
      const uint32_t kt = smem_u32(kbuf(m)), vt = smem_u32(vbuf(m));
      const bool with_h = !(fresh && i == 0);
      wt(&hd.k_full[m & 1], m / 2);
      wt(&hd.q_full, i);
      after_sync();
      if (dead(hd)) return;
      for (int k = 0; k < DK / 16; ++k) {
        const uint32_t at = (k >> 2) * (kC * 128) + (k & 3) * 32;
        mma(tb + kColS, sdesc(qt + at, 16, 1024), sdesc(kt + at, 16, 1024), id_s, k > 0);
      }
      commit(&hd.s_ready);
      wt(&hd.h_ready, i);
      if (i > 0) wt(&hd.o_free, i - 1);
      after_sync();
      if (dead(hd)) return;
      if (with_h)
        for (int term = 0; term < 2; ++term)
          for (int k = 0; k < DK / 16; ++k)
            mma(tb + kColO, sdesc(qt + (k >> 2) * (kC * 128) + (k & 3) * 32, 16, 1024),
                sdesc(ht + term * Sh::hterm + (k >> 2) * (DV * 128) + (k & 3) * 32, 16, 1024), id_h, term + k > 0);
      commit(&hd.o2_ready);
      commit(&hd.q_empty);
      for (int quarter = 0; quarter < 4; ++quarter, ++quarters) {
        wt(&hd.v_ready[quarters & 1], quarters >> 1);
        after_sync();
        if (dead(hd)) return;
        state_quarter(kt, quarter, quarters & 1, with_h || quarter > 0);
        commit(&hd.v_free[quarters & 1]);
      }
      commit(&hd.kv_done);
      commit(&hd.k_empty[m & 1]);
      wt(&hd.pv_go, i);
      after_sync();
      if (dead(hd)) return;
      for (int k = 0; k < kC / 16; ++k)
        for (int term = 0; term < 2; ++term)
          mma_ts(tb + kColO, tb + kColS + (k >> 2) * 64 + term * 32 + (k & 3) * 8, sdesc(vt + 16 * k * 128, kC * 128, 1024),
                 id_v, with_h || k + term > 0);
      commit(&hd.o_ready);
    }
  }

  // ---- warps 0-3: scores and outputs, a thread per row ----------------------------------------------------------
  __device__ __forceinline__ void outputs(int m0, bool fresh) const {
    const int t = threadIdx.x, warp = t / 32;
    const uint32_t lane0 = tb + ((uint32_t)(32 * warp) << 16);
    float u[16];                                   // lambda^(15-j)
#pragma unroll
    for (int j = 0; j < 16; ++j) u[j] = hd.power[15 - j];
    const float carry = hd.power[t + 1];           // lambda^(t+1)
    for (int c = run.c0; c < run.c1; ++c) {
      const int i = c - run.c0;
      const bool with_h = !(fresh && i == 0);
      wt(&hd.s_ready, i);
      after_sync();
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t hi[32], lo[32];
        float s[64];
        if (64 * half <= 32 * warp + 31) tmem_ld64(lane0 + kColS + 64 * half, s);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int j0 = 64 * half + 16 * b;        // columns [j0, j0 + 16)
          if (j0 + 15 <= 32 * warp) {               // all at or below the diagonal
            const float f = hd.power[t - j0 - 15];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float x = s[16 * b + j] * u[j] * f, y = s[16 * b + j + 1] * u[j + 1] * f;
              hi[8 * b + j / 2] = take_term(x, y);
              lo[8 * b + j / 2] = last_term(x, y);
            }
          } else if (j0 <= 32 * warp + 31) {        // on the diagonal
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float x = j0 + j <= t ? s[16 * b + j] * hd.power[t - j0 - j] : 0.f;
              float y = j0 + j + 1 <= t ? s[16 * b + j + 1] * hd.power[t - j0 - j - 1] : 0.f;
              hi[8 * b + j / 2] = take_term(x, y);
              lo[8 * b + j / 2] = last_term(x, y);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) hi[8 * b + j] = lo[8 * b + j] = 0;
          }
        }
        tmem_st32(lane0 + kColS + 64 * half, hi);
        tmem_st32(lane0 + kColS + 64 * half + 32, lo);
      }
      wt(&hd.o2_ready, i);
      after_sync();
      if (with_h) {
#pragma unroll 1
        for (int x = 0; x < DV; x += 32) {
          float o[32];
          uint32_t r[32];
          tmem_ld32(lane0 + kColO + x, o);
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(o[j] * carry);
          tmem_st32(lane0 + kColO + x, r);
        }
      }
      tmem_wait_st();
      before_sync();
      mbar_arrive(&hd.pv_go);
      wt(&hd.o_ready, i);
      after_sync();
      const int live = rows(c);
      const int* bad4 = hd.bad[i & 1];
      const bool bad = (bad4[0] | bad4[1] | bad4[2] | bad4[3]) != 0;
      uint8_t* stage = vbuf(m0 + i);           // P V is done with it
      bf16* out = (bf16*)a.o + ((size_t)(run.t0 + c * kC + t) * a.H + h) * DV;
#pragma unroll 1
      for (int x = 0; x < DV; x += 32) {
        float o[32];
        tmem_ld32(lane0 + kColO + x, o);
        if (bad) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (t >= hd.first_bad[i & 1][x + j]) o[j] = __int_as_float(0x7fffffff);
        }
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint4 v;
          v.x = last_term(o[j] * a.scale, o[j + 1] * a.scale);
          v.y = last_term(o[j + 2] * a.scale, o[j + 3] * a.scale);
          v.z = last_term(o[j + 4] * a.scale, o[j + 5] * a.scale);
          v.w = last_term(o[j + 6] * a.scale, o[j + 7] * a.scale);
          if (live == kC) *reinterpret_cast<uint4*>(stage + sw128(kC, t, x + j)) = v;
          else if (t < live && !dead(hd)) *reinterpret_cast<uint4*>(out + x + j) = v;
        }
      }
      before_sync();
      mbar_arrive(&hd.o_free);
      fence_async_smem();
      mbar_arrive(&hd.o_staged);
    }
  }

  // ---- warps 4-7: V' and the state, a thread per state row --------------------------------------------------------
  // quarter `quarter` of V' of a chunk: 32 tokens as three terms into tensor memory.  f multiplies the weights.
  // nan collects whether anything was not finite.
  __device__ __forceinline__ void make_quarter(const uint8_t* vt, const float* w, float f, int quarter, int& quarters,
                                               float& nan) const {
    const int d = threadIdx.x - 128;
    if (quarters >= 2) {
      wt(&hd.v_free[quarters & 1], (quarters >> 1) - 1);
      after_sync();
    }
    if (d < DV) {
      uint32_t r[3][16];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const int s = 32 * quarter + j;
        const float4 w4 = *reinterpret_cast<const float4*>(w + s);
        const float ws[4] = {w4.x * f, w4.y * f, w4.z * f, w4.w * f};
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = __bfloat162float(*reinterpret_cast<const bf16*>(vt + sw128(kC, s + e, d)));
          nan = fmaf(v, 0.f, nan);
          x[e] = v * ws[e];
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          r[0][(j + e) / 2] = take_term(x[e], x[e + 1]);
          r[1][(j + e) / 2] = take_term(x[e], x[e + 1]);
          r[2][(j + e) / 2] = last_term(x[e], x[e + 1]);
        }
      }
      const uint32_t at = tb + ((uint32_t)(32 * (d / 32)) << 16) + kColV + (quarters & 1) * kVStage;
      tmem_st16(at, r[0]);
      tmem_st16(at + 16, r[1]);
      tmem_st16(at + 32, r[2]);
      tmem_wait_st();
    }
    before_sync();
    ++quarters;
  }
  __device__ __forceinline__ void quarter_done(int quarters) const { mbar_arrive(&hd.v_ready[(quarters - 1) & 1]); }

  // rows from n on of the chunk's K and V tiles belong to the next sequence (or to nobody): zeros
  __device__ __forceinline__ void clear_tail(int n_rows, uint8_t* kt, uint8_t* vt) const {
    constexpr int parts = (DK + DV) / 8;
    for (int e = threadIdx.x - 128; e < (kC - n_rows) * parts; e += 128) {
      const int r = n_rows + e / parts, x = e % parts * 8;
      uint8_t* at = x < DK ? kt + sw128(kC, r, x) : vt + sw128(kC, r, x - DK);
      *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    named_sync(kBarState, 128);
  }

  // the state before a chunk: its operand terms to shared memory, and lambda^n of it back for the accumulation
  __device__ __forceinline__ void hand_state(float step_hi, float step_lo) const {
    const int d = threadIdx.x - 128;
    if (d < DV) {
      const uint32_t at = tb + ((uint32_t)(32 * (d / 32)) << 16) + kColH;
#pragma unroll 1
      for (int x = 0; x < DK; x += 32) {
        float s[32];
        uint32_t r[32];
        tmem_ld32(at + x, s);
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(fmaf(step_hi, s[j], step_lo * s[j]));
        tmem_st32(at + x, r);
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint4 hi, lo;
          hi.x = take_term(s[j], s[j + 1]);
          hi.y = take_term(s[j + 2], s[j + 3]);
          hi.z = take_term(s[j + 4], s[j + 5]);
          hi.w = take_term(s[j + 6], s[j + 7]);
          lo.x = last_term(s[j], s[j + 1]);
          lo.y = last_term(s[j + 2], s[j + 3]);
          lo.z = last_term(s[j + 4], s[j + 5]);
          lo.w = last_term(s[j + 6], s[j + 7]);
          *reinterpret_cast<uint4*>(hop + sw128(DV, d, x + j)) = hi;
          *reinterpret_cast<uint4*>(hop + Sh::hterm + sw128(DV, d, x + j)) = lo;
        }
      }
      tmem_wait_st();
    }
    fence_async_smem();
    before_sync();
  }

  // first pass: the run's own end state, from nothing
  __device__ __forceinline__ void states_only(int& quarters, float a_h) const {
    float nan = 0.f;
    for (int c = run.c0; c < run.c1; ++c) {
      const int m = c - run.c0;
      wt(&hd.v_full[m & 1], m / 2);
      const float f = c + 1 < run.c1 ? expf(a_h * (float)((run.c1 - 1 - c) * kC)) : 1.f;
      for (int quarter = 0; quarter < 4; ++quarter) {
        make_quarter(vbuf(m), hd.w[0], f, quarter, quarters, nan);
        quarter_done(quarters);
      }
    }
    wt(&hd.kv_done, 0);
    after_sync();
  }

  __device__ __forceinline__ void states(int m0, int quarters, uint32_t kv_phase, bool fresh) const {
    const int d = threadIdx.x - 128, warp = d / 32;
    float nan = 0.f;
    const int c_end = (run.len + kC - 1) / kC;    // of the sequence
    auto prepare = [&](int c, int m) {             // chunk c's tiles have arrived
      wt(&hd.v_full[m & 1], m / 2);
      if (rows(c) < kC) {
        wt(&hd.k_full[m & 1], m / 2);
        clear_tail(rows(c), kbuf(m), vbuf(m));
      }
      nan = 0.f;
    };
    auto weights = [&](int c) -> const float* { return hd.w[c + 1 == c_end ? 1 : 0]; };
    for (int c = run.c0; c < run.c1; ++c) {
      const int i = c - run.c0, m = m0 + i;
      uint8_t* vt = vbuf(m);
      if (i == 0) {
        if (!fresh) hand_state(c + 1 == c_end ? hd.last_hi : hd.step_hi, c + 1 == c_end ? hd.last_lo : hd.step_lo);
        mbar_arrive(&hd.h_ready);
        prepare(c, m);
      }
      for (int quarter = i == 0 ? 0 : 2; quarter < 4; ++quarter) {
        make_quarter(vt, weights(c), 1.f, quarter, quarters, nan);
        if (quarter == 3) settle(vt, i, warp, d, nan);
        quarter_done(quarters);
      }
      if (c + 1 < run.c1) {                        // the next chunk's first half, while the tensor core works
        prepare(c + 1, m + 1);
        for (int quarter = 0; quarter < 2; ++quarter) {
          make_quarter(vbuf(m + 1), weights(c + 1), 1.f, quarter, quarters, nan);
          quarter_done(quarters);
        }
      }
      wt(&hd.kv_done, kv_phase + i);
      after_sync();
      if (c + 1 < run.c1) {
        const bool last = c + 2 == c_end;
        hand_state(last ? hd.last_hi : hd.step_hi, last ? hd.last_lo : hd.step_lo);
        mbar_arrive(&hd.h_ready);
      }
    }
  }
  // Where a value column holds something that is not finite, a masked product with it would spoil the outputs of
  // earlier tokens (0 times infinity).  Such values are taken out of the tile (the state has them), and
  // the outputs of their column from their token on are set when they are stored.
  __device__ __forceinline__ void settle(uint8_t* vt, int i, int warp, int d, float nan) const {
    const bool any = __any_sync(kFull, !(nan == 0.f));
    if (d < DV) {
      int first = kC;
      if (any) {
        for (int s = kC - 1; s >= 0; --s) {
          bf16* at = reinterpret_cast<bf16*>(vt + sw128(kC, s, d));
          if (!isfinite(__bfloat162float(*at))) {
            first = s;
            *at = __float2bfloat16_rn(0.f);
          }
        }
        fence_async_smem();
      }
      hd.first_bad[i & 1][d] = (uint8_t)first;
    }
    if (d % 32 == 0) hd.bad[i & 1][warp] = any;
  }

  // ---- the fp32 state between tensor memory and elsewhere, a thread per row ----------------------------------------
  __device__ __forceinline__ uint32_t cell(int d, int x) const {   // byte offset of floats [x, x + 4) of row d in hop
    return (uint32_t)d * (DK * 4) + (uint32_t)(((x / 4) ^ (d & 7)) * 16);
  }
  __device__ __forceinline__ void state_in(const float* src, bool shared) const {
    const int d = threadIdx.x - 128;
    if (d < DV) {
#pragma unroll 1
      for (int x = 0; x < DK; x += 32) {
        uint32_t r[32];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 v = shared ? *reinterpret_cast<const float4*>(hop + cell(d, x + j))
                                  : *reinterpret_cast<const float4*>(src + (size_t)d * DK + x + j);
          r[j] = __float_as_uint(v.x);
          r[j + 1] = __float_as_uint(v.y);
          r[j + 2] = __float_as_uint(v.z);
          r[j + 3] = __float_as_uint(v.w);
        }
        tmem_st32(tb + ((uint32_t)(32 * (d / 32)) << 16) + kColH + x, r);
      }
      tmem_wait_st();
    }
    named_sync(kBarState, 128);   // hop may be overwritten
  }
  __device__ __forceinline__ void state_out(float* dst, bool shared) const {
    const int d = threadIdx.x - 128;
    if (d >= DV) return;
#pragma unroll 1
    for (int x = 0; x < DK; x += 32) {
      float s[32];
      tmem_ld32(tb + ((uint32_t)(32 * (d / 32)) << 16) + kColH + x, s);
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 v = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        if (shared) *reinterpret_cast<float4*>(hop + cell(d, x + j)) = v;
        else *reinterpret_cast<float4*>(dst + (size_t)d * DK + x + j) = v;
      }
    }
  }

  // Start states from the runs' own end states, in place: this CTA turns DV / split rows of every run's.
  __device__ __forceinline__ void join(const float* init, float a_h, int rank, int split) const {
    const int rows_each = DV / split;
    const float f = expf(a_h * (float)(run.per * kC));
    for (int e = threadIdx.x; e < rows_each * (DK / 4); e += kBlock) {
      const int d = rank * rows_each + e / (DK / 4), x = e % (DK / 4) * 4;
      const uint32_t at = smem_u32(hop) + cell(d, x);
      float4 own[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < run.last_run) own[r] = peer_ld(peer(at, r));
      float4 s = init != nullptr ? *reinterpret_cast<const float4*>(init + (size_t)d * DK + x) : make_float4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r > run.last_run) break;
        peer_st(peer(at, r), s);
        if (r < run.last_run) {
          s.x = fmaf(f, s.x, own[r].x);
          s.y = fmaf(f, s.y, own[r].y);
          s.z = fmaf(f, s.z, own[r].z);
          s.w = fmaf(f, s.w, own[r].w);
        }
      }
    }
  }
};

extern __shared__ uint8_t linattn_smem[];

template <int DK, int DV>
__global__ void __launch_bounds__(kBlock, 1)
    k_linattn_chunks(const __grid_constant__ LinAttnArgs a, const __grid_constant__ Maps maps, int split) {
  using Sh = Shape<DK, DV>;
  const int rank = blockIdx.x % split, unit = blockIdx.x / split;
  const int i = unit / a.H, h = unit % a.H;
  LinAttnSeq seq;
  if (!linattn_seq(a, i, h, &seq)) return;   // the same for every CTA of the cluster
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (seq.len == 0) {
    if (rank == 0)
      for (int e = tid; e < DV * DK; e += kBlock) seq.out[e] = seq.in != nullptr ? seq.in[e] : 0.f;
    return;
  }
  const float a_h = a.log_decay[h];
  const int chunks = (seq.len + kC - 1) / kC;
  Run run;
  run.t0 = seq.t0;
  run.len = seq.len;
  run.per = (chunks + split - 1) / split;
  run.last_run = (chunks - 1) / run.per;
  run.c0 = min(rank * run.per, chunks);
  run.c1 = min(run.c0 + run.per, chunks);

  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(linattn_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* hop = base + 3 * Sh::ktile + 2 * Sh::vtile;
  Hdr& hd = *reinterpret_cast<Hdr*>(hop + 2 * Sh::hterm);
  if (warp == kMmaWarp) tmem_alloc(&hd.tmem, kTmemCols);
  if (tid == 0) {
    uint64_t* by_one[] = {&hd.k_full[0], &hd.k_full[1], &hd.k_empty[0], &hd.k_empty[1], &hd.v_full[0], &hd.v_full[1],
                          &hd.v_empty[0], &hd.v_empty[1], &hd.q_full, &hd.q_empty,
                          &hd.s_ready, &hd.o2_ready, &hd.o_ready, &hd.kv_done, &hd.v_free[0], &hd.v_free[1]};
    for (uint64_t* b : by_one) mbar_init(b, 1);
    uint64_t* by_group[] = {&hd.pv_go, &hd.o_free, &hd.o_staged, &hd.h_ready, &hd.v_ready[0], &hd.v_ready[1]};
    for (uint64_t* b : by_group) mbar_init(b, 128);
    fence_mbar_init();
    hd.dead = 0;
  }
  const int n_last = seq.len - (chunks - 1) * kC;
  if (tid >= 128 && tid < 128 + kC) {
    const int j = tid - 128;
    // lambda^0 = 1 whatever lambda
    hd.power[j] = j == 0 ? 1.f : expf(a_h * (float)j);
    if (j == 0) hd.power[kC] = expf(a_h * (float)kC);
    hd.w[0][j] = j == kC - 1 ? 1.f : expf(a_h * (float)(kC - 1 - j));
    hd.w[1][j] = j >= n_last ? 0.f : j == n_last - 1 ? 1.f : expf(a_h * (float)(n_last - 1 - j));
  } else if (tid == 288 || tid == 256) {           // multiplied once a chunk over the whole sequence: as two floats
    const int n = tid == 288 ? kC : n_last;
    const double e = exp((double)a_h * n);
    const float hi = (float)e, lo = (float)(e - (double)hi);
    (tid == 288 ? hd.step_hi : hd.last_hi) = hi;
    (tid == 288 ? hd.step_lo : hd.last_lo) = lo;
  }
  before_sync();
  __syncthreads();
  after_sync();
  Cta<DK, DV> cta{a, maps, hd, base, hop, hd.tmem, h, h / (a.H / a.G), run};

  // ---- first pass -----------------------------------------------------------------------------------------
  const bool first = run.last_run > 0 && rank < run.last_run;
  int quarters = 0;
  uint32_t kv_phase = 0;
  const int m0 = first ? run.c1 - run.c0 : 0;
  if (first) {
    kv_phase = 1;
    if (warp == kLoadWarp) {
      if (lane == 0) cta.load_states();
    } else if (warp == kMmaWarp) {
      if (lane == 0) cta.issue_states(quarters);
    } else if (warp >= 4) {
      cta.states_only(quarters, a_h);
      cta.state_out(nullptr, true);
    }
    quarters = 4 * (run.c1 - run.c0);
    __syncwarp();
  }
  if (split > 1) {
    before_sync();
    cluster_sync();
    if (run.last_run > 0) cta.join(seq.in, a_h, rank, split);
    cluster_sync();
    after_sync();
  }
  const bool given = run.last_run > 0 ? (rank > 0 || seq.in != nullptr) : seq.in != nullptr;

  // ---- the chunks -------------------------------------------------------------------------------------------
  if (run.c0 < run.c1) {
    if (warp == kLoadWarp) {
      if (lane == 0) cta.load_chunks(m0);
    } else if (warp == kMmaWarp) {
      if (lane == 0) cta.issue_chunks(m0, quarters, !given);
    } else if (warp >= 4) {
      if (given) cta.state_in(seq.in, run.last_run > 0);
      cta.states(m0, quarters, kv_phase, !given);
      if (rank == run.last_run && !dead(hd)) cta.state_out(seq.out, false);
    } else {
      cta.outputs(m0, !given);
    }
  }
  __syncwarp();
  if (warp == kLoadWarp && lane == 0 && dead(hd)) cta.drain();
  before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(hd.tmem, kTmemCols);
}

// ---- host side ---------------------------------------------------------------------------------------------
bool encode(CUtensorMap* m, const void* base, long long T, int heads, int d) {
  const EncodeTiledFn fn = tma_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * heads * 2};
  const cuuint32_t box[3] = {64, 1, kC};
  const cuuint32_t each[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, each,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV>
cudaError_t raise_smem() {
  static std::mutex mu;
  static bool done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(k_linattn_chunks<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<DK, DV>::smem);
  done[dev] = e == cudaSuccess;
  return e;
}

template <int DK, int DV>
cudaError_t launch(const LinAttnArgs& a, const Maps& maps, int split, cudaStream_t s) {
  cudaError_t e = raise_smem<DK, DV>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)((long long)a.nseq * a.H * split));
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = Shape<DK, DV>::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_linattn_chunks<DK, DV>, a, maps, split);
}

}  // namespace

bool linattn_tc_supported(const LinAttnArgs& a) {
  return a.io == ERS_DTYPE_BF16 && a.ntokens > 0 && (long long)a.nseq * a.H <= (0x7fffffff >> 3) &&
         tma_encode_fn() != nullptr;
}

cudaError_t linattn_tc(const LinAttnArgs& a, cudaStream_t s) {
  Maps maps;
  if (!encode(&maps.q, a.q, a.ntokens, a.G, a.dk) || !encode(&maps.k, a.k, a.ntokens, a.G, a.dk) ||
      !encode(&maps.v, a.v, a.ntokens, a.H, a.dv) || !encode(&maps.o, a.o, a.ntokens, a.H, a.dv))
    return cudaErrorInvalidValue;
  // Runs of a sequence: as many as fill the SMs, of two chunks at least.
  const int chunks = (int)((a.max_len + kC - 1) / kC);
  int split = 1;
  while (split < 8 && (long long)a.nseq * a.H * split * 2 <= 152 && chunks >= 4 * split) split *= 2;
  if (a.dk == 64) return a.dv == 64 ? launch<64, 64>(a, maps, split, s) : launch<64, 128>(a, maps, split, s);
  return a.dv == 64 ? launch<128, 64>(a, maps, split, s) : launch<128, 128>(a, maps, split, s);
}

}  // namespace ers
