// Linear attention with a decay per head over prompts, on the tensor cores (bf16 io).
//
// Chunks of 128 tokens; rows i, j of a chunk of n tokens that starts from state H ([dv x dk]), lambda = exp(a):
//   O[i] = scale * (sum_{j <= i} (q_i . k_j) lambda^(i-j) v_j + lambda^(i+1) H q_i)
//   H'   = lambda^n H + sum_j (lambda^(n-1-j) v_j) k_j^T
// Four contractions of 128 x 128 x 128 (at dk = dv = 128), tcgen05 kind::f16 with fp32 accumulators:
//   S = Q K^T            A, B from shared memory (TMA tiles)
//   H += V'^T K          A = V' = lambda^(n-1-j) v_j as bf16 hi + mid + lo in tensor memory
//   O = Q H'^T + P V     B = H' as hi + lo in shared memory, A = P as hi + lo in tensor memory, over S
// The decays of a row are taken out of the products: with P[i,j] = S[i,j] lambda^(63-j) and H' = lambda^64 H the row's output is
// scale lambda^(i-63) O[i], and both products go into one accumulator.  All factors lie within lambda^(+-64), which fp32
// and bf16 hold down to a = -1 (6e+-27; there a state's operand keeps its 16 bits above 3.8e-8 and a score above 1.4e-8, the
// low term of a smaller one being below bf16's range).  Beyond that (kStrong) P carries lambda^(i-j), H' = H, and the
// accumulator is multiplied by lambda^(i+1) between the two products.  (kStrong of 0.5 would hold smaller ones, and costs the
// heads in between: 2048, 777, 513 and 1 x 64 heads 74.1 us against 67.2, 32768 x 32 318 against 307.)
// Operands made from fp32 values are split so that outputs keep 16 significant bits before their one rounding (a single
// bf16 term would cost half as much again as that rounding) and states all 24.  The state stays in tensor memory in
// fp32 from chunk to chunk.  Its 24 additions of a chunk are the tensor core's, which does not round but cuts off: a state that
// forgets little loses some 2^-24 of itself with each (4e-6 over 4096 tokens, 3e-5 to 6e-5 over 32768; chunks added by
// themselves in fp32 would not, but need 128 columns of tensor memory more than there are).
//
// Measured (128 x 128, kernel alone): 97 tokens x 32 heads 9.5 us (13.5 from given states), 2048 x 32 33, 32768 x 32 303 (39 % of
// the measured bandwidth), 4096 x 128 112 (54 %; tensor pipe 49 % busy).
//
// What bounds it: at one CTA per SM a chunk moves 128 KB (2.9 us of an SM's share of the memory), 64 MMAs of 64 cycles
// and some 2500 issue slots of operand making per scheduler, in one dependent loop through the state.  So the warps are
// specialised and run side by side, and the MMAs are ordered S, H, O so that each group's work on one product lies under the
// others: while H accumulates the scores become P and the last chunk's outputs are stored; while O accumulates the state is
// handed on.  Four warps make P and own the outputs (on warps of their own the outputs made every product slower: more
// tensor-memory traffic at once), eight make V' and hand the state on, one loads the tiles (TMA; two
// buffers for K and V, one for Q), one issues every MMA and two help with P.  A chunk takes some 6500 cycles where the
// SM's 64 MMAs of 64 cycles would take 4100: under way with the other traffic of shared memory an MMA takes 75 to 115,
// and 900 cycles pass at hand-overs.
//
// A long sequence of few heads is split over the CTAs of a cluster, each a run of chunks: every CTA but the
// last first forms its run's own end state (K and V only), the cluster turns those into start states through
// distributed shared memory, and then all walk their runs.
#include <math.h>
#include <string.h>

#include <mutex>

#include "f32x2.cuh"
#include "linattn.cuh"
#include "tc_common.cuh"
#include "tc_terms.cuh"
#include "tma_host.h"

namespace ers {
namespace {

using namespace tc;
using bf16 = __nv_bfloat16;

constexpr int kC = 128;                  // tokens of a chunk
// warps 0-3 make P and own the outputs, 4-7 and 8-11 (two sets) the state, 12 loads and 13 issues, 14 and 15 help with P; lane
// quarter: warp % 4.  16 warps: 128 registers each, for with spills every reload would go to L2 (the first-level cache is all
// shared memory).
constexpr int kStateThread = 128, kStateThreads = 256, kControlThread = 384;
constexpr int kLoadWarp = 12, kMmaWarp = 13;
constexpr int kBlock = 512;
constexpr float kStrong = 1.f;
__device__ __forceinline__ bool is_strong(float a) { return !(fabsf(a) <= kStrong); }
constexpr uint32_t kColS = 0, kColO = 128, kColH = 256, kColV = 384, kVStage = 48, kTmemCols = 512;
constexpr uint32_t kBarState = 1, kBarRows = 2, kBarSet = 3 /* and 4, 5 */;   // named barriers of the warps of a kind

struct Hdr {
  alignas(16) float w[2][kC];        // lambda^(n-1-j), 0 from n on: a full chunk, the last chunk (read 16 bytes at a time)
  alignas(16) float power[kC + 4];   // lambda^(63-j) of the columns j; kStrong: lambda^j
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full, q_empty;   // tile buffers
  uint64_t s_ready, qh_done, o_ready, kv_done, v_free[2];               // completed by the tensor core
  uint64_t p_ready, o_scaled, o_free, o_staged, h_scaled, h_ready, v_ready[2];    // by the warps
  uint64_t run_full[3], run_empty[3], run_ready[3], run_free[3];       // the first pass's tiles and V'
  uint32_t tmem;
  int dead;                          // a wait gave up: no further wait waits, no copy or MMA is issued
  float step_hi, step_lo;            // lambda^128 as two floats,
  float last_hi, last_lo;            // lambda^n of the sequence's last chunk
  float mid;                         // lambda^64
  alignas(8) uint8_t bad[2][8];      // a chunk's value columns (by state warp) hold something not finite,
  uint8_t first_bad[2][2][kC];       // from this token of the set's quarters on (128: nowhere)
};

struct Maps {
  CUtensorMap q, k, v, o;
};

template <int DK, int DV>
struct Shape {
  static constexpr uint32_t ktile = kC * DK * 2, vtile = kC * DV * 2;
  static constexpr uint32_t hterm = DV * DK * 2;       // one bf16 term of the state operand
  static constexpr int run_bufs = 2 * hterm >= ktile + vtile ? 3 : 2;   // first pass: a third K and V where the operand will be
  static constexpr uint32_t stage = vtile > ktile ? vtile : 0;   // outputs on their way out: in a K tile where they fit
  static constexpr uint32_t smem = sizeof(Hdr) + 3 * ktile + 2 * vtile + 2 * hterm + stage;
  static_assert(smem <= 227 * 1024, "one CTA's shared memory");
};

// ---- waits -----------------------------------------------------------------------------------------------
// Short, and no function call: a call would bind the registers of every caller.  False: gave up.
__device__ __forceinline__ bool wait(Hdr& hd, uint64_t* bar, uint32_t parity, int32_t* status) {
  uint64_t t0 = 0;
#pragma unroll 1
  while (!mbar_try(bar, parity)) {
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

// ---- PTX that the other engines do not need ------------------------------------------------------------------
// f(x, values) for the 32-column groups x, x + 32, ... of [x0, n)
template <typename F>
__device__ __forceinline__ void tmem_each32(uint32_t at, int n, F f, int x0 = 0) {
#pragma unroll 1
  for (int x = x0; x < n; x += 32) {
    uint32_t r[32];
    tmem_ld32_begin(at + x, r);
    arrived(r);
    f(x, r);
  }
}
// 16 lanes x 16 columns in the layout of ldmatrix: thread t holds, of column group g (4 columns), row t / 4 in r[2g] and
// row t / 4 + 8 in r[2g + 1], column t % 4
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
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

// Row t of 32 output columns, from the tokens first[] (of either set) on not finite.
__device__ __forceinline__ void spoil(uint32_t (&o)[32], const uint8_t* first0, const uint8_t* first1, int t) {
  uint32_t m = 0;
#pragma unroll 1
  for (int j = 0; j < 32; ++j) m |= (uint32_t)(t >= first0[j] || t >= first1[j]) << j;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (m >> j & 1u) o[j] = 0x7fffffff;
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
  float a_h;
  bool strong;
  Run run;

  // A run's chunk m = 0, 1, ... uses K and V buffer m % 2 for the m / 2th time.
  __device__ __forceinline__ uint8_t* kbuf(int m) const { return tiles + (m & 1) * Sh::ktile; }
  __device__ __forceinline__ uint8_t* vbuf(int m) const { return tiles + 2 * Sh::ktile + (m & 1) * Sh::vtile; }
  __device__ __forceinline__ uint8_t* qbuf() const { return tiles + 2 * Sh::ktile + 2 * Sh::vtile; }
  __device__ __forceinline__ uint8_t* run_k(int b) const { return b < 2 ? kbuf(b) : hop; }
  __device__ __forceinline__ uint8_t* run_v(int b) const { return b < 2 ? vbuf(b) : hop + Sh::ktile; }
  __device__ __forceinline__ uint8_t* obuf(int m) const {
    return Sh::stage > 0 ? tiles + 3 * Sh::ktile + 2 * Sh::vtile : kbuf(m);
  }
  __device__ __forceinline__ int rows(int c) const { return run.len - c * kC < kC ? run.len - c * kC : kC; }
  __device__ __forceinline__ bool wt(uint64_t* bar, uint32_t parity) const { return wait(hd, bar, parity & 1u, a.status); }
  // one warp of a kind polls, the others wait for it
  __device__ __forceinline__ void wt_group(int id, uint64_t* bar, uint32_t parity) const {
    if (threadIdx.x % 128 < 32) wt(bar, parity);
    named_sync(id, 128);
    after_sync();
  }
  __device__ __forceinline__ int set() const { return (threadIdx.x - kStateThread) / 128; }
  __device__ __forceinline__ void wt_set(uint64_t* bar, uint32_t parity) const { wt_group(kBarSet + set(), bar, parity); }

  // ---- the loading warp ------------------------------------------------------------------------
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
  // first pass: chunk m's K and V
  __device__ __forceinline__ void load_run(int m) const {
    const int b = m % Sh::run_bufs, use = m / Sh::run_bufs, z = run.t0 + (run.c0 + m) * kC;
    if (use > 0) wt(&hd.run_empty[b], use - 1);
    if (dead(hd)) return;
    uint64_t* bar = &hd.run_full[b];
    mbar_arrive_expect_tx(bar, Sh::ktile + Sh::vtile);
    for (int x = 0; x < DK; x += 64) tma_load_3d(run_k(b) + x / 64 * (kC * 128), &maps.k, x, g, z, bar);
    for (int x = 0; x < DV; x += 64) tma_load_3d(run_v(b) + x / 64 * (kC * 128), &maps.v, x, h, z, bar);
  }
  // the first chunks, which need not wait for anything
  __device__ __forceinline__ void load_run_head() const {
    for (int m = 0; m < Sh::run_bufs && run.c0 + m < run.c1; ++m) load_run(m);
  }
  __device__ __forceinline__ void load_run_rest() const {
    for (int m = Sh::run_bufs; run.c0 + m < run.c1; ++m) load_run(m);
  }
  __device__ __forceinline__ void load_head() const {
    for (int m = 0; m < 2 && run.c0 + m < run.c1; ++m) {
      load_k(m, run.c0 + m);
      if (m == 0) load(qbuf(), &maps.q, DK, g, run.c0, &hd.q_full);
      load_v(m, run.c0 + m);
    }
  }
  // After their head, in the order in which buffers come free: Q after Q H^T, V after P V, and K, long done with then, when the
  // output that takes its place has been stored: it is the tile that is needed last.  (A short chunk's rows are stored by the
  // warps that made them.)
  __device__ __forceinline__ void load_chunks() const {
    const int n = run.c1 - run.c0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int c = run.c0 + i;
      if (i + 1 < n) {
        wt(&hd.q_empty, i);
        load(qbuf(), &maps.q, DK, g, c + 1, &hd.q_full);
      }
      if (i + 2 < n) load_v(i + 2, c + 2);
      wt(&hd.o_staged, i);
      if (!dead(hd) && rows(c) == kC) {
        for (int x = 0; x < DV; x += 64)
          tma_store_3d(&maps.o, obuf(i) + x / 64 * (kC * 128), x, h, run.t0 + c * kC);
        bulk_commit();
        bulk_wait_read();
      }
      mbar_arrive(&hd.k_empty[i & 1]);
      if (i + 2 < n) load_k(i + 2, c + 2);
    }
  }
  // After a wait gave up: no copy or MMA may be left in flight when the CTA ends.
  __device__ __forceinline__ void drain() const {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000) {}   // 2 ms: a thousand times what a tile or an MMA takes
  }

  // ---- the issuing warp: every MMA --------------------------------------------------------------------------------------
  // The whole warp runs the loops (their operands then live in uniform registers), one lane issues.  Descriptors step by
  // constants: 16 columns of a tile are 32 bytes on, in units of 16, and 64 columns an atom of `rows` rows on.
  __device__ __forceinline__ void chain(uint32_t d, uint64_t ad, uint64_t bd, int arows, int brows, int n, uint32_t id,
                                        bool accumulate, bool leader) const {
#pragma unroll 1
    for (int k = 0; k < n; k += 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (leader) mma(d, ad + 2 * j, bd + 2 * j, id, accumulate || k + j > 0);
      ad += (uint64_t)arows * 8;
      bd += (uint64_t)brows * 8;
    }
  }
  // one quarter (32 tokens) of H += V'^T K, V' from columns `at` on
  __device__ __forceinline__ void state_quarter(uint64_t kd, uint32_t at, bool accumulate, bool leader) const {
    constexpr uint32_t id = idesc_bf16(128, DK, false, true);
#pragma unroll 1
    for (int term = 0; term < 3; ++term, at += 16) {
      if (leader) {
        mma_ts(tb + kColH, at, kd, id, accumulate || term > 0);
        mma_ts(tb + kColH, at + 8, kd + 16 * 128 / 16, id, 1);
      }
    }
  }
  __device__ __forceinline__ uint64_t by_token(const uint8_t* tile) const { return sdesc(smem_u32(tile), kC * 128, 1024); }
  // First pass: the quarters one after the other, by three sets of warps in turn; the outputs' columns hold the third stage.
  static __device__ __forceinline__ uint32_t run_stage(int s) { return s == 2 ? kColO : kColV + s * kVStage; }
  __device__ __forceinline__ void issue_states() const {
    const bool leader = elected();
    int s = 0, use = 0;                            // quarter number = 3 use + s
#pragma unroll 1
    for (int m = 0; m < run.c1 - run.c0; ++m) {
      const int b = m % Sh::run_bufs;
      if (!wt(&hd.run_full[b], m / Sh::run_bufs)) return;
      uint64_t kd = by_token(run_k(b));
#pragma unroll 1
      for (int quarter = 0; quarter < 4; ++quarter, kd += 32 * 128 / 16) {
        if (!wt(&hd.run_ready[s], use)) return;
        after_sync();
        state_quarter(kd, tb + run_stage(s), m > 0 || quarter > 0, leader);
        if (leader) commit(&hd.run_free[s]);
        if (++s == 3) s = 0, ++use;
      }
      if (leader) commit(&hd.run_empty[b]);
    }
    if (leader) commit(&hd.kv_done);
  }
  __device__ __forceinline__ void issue_chunks(bool fresh) const {
    constexpr uint32_t id_s = idesc_bf16(128, kC, false, false), id_h = idesc_bf16(128, DV, false, false),
                       id_v = idesc_bf16(128, DV, false, true);
    const uint64_t qd = sdesc(smem_u32(qbuf()), 16, 1024), h_hi = sdesc(smem_u32(hop), 16, 1024);
    const bool leader = elected();
#pragma unroll 1
    for (int i = 0; i < run.c1 - run.c0; ++i) {
      const int m = i;
      const bool with_h = !(fresh && i == 0);
      if (!wt(&hd.k_full[m & 1], m / 2) || !wt(&hd.q_full, i)) return;
      after_sync();
      chain(tb + kColS, qd, sdesc(smem_u32(kbuf(m)), 16, 1024), kC, kC, DK / 16, id_s, false, leader);
      if (leader) commit(&hd.s_ready);
      if (!wt(&hd.h_scaled, i)) return;
      after_sync();
      uint64_t ks = by_token(kbuf(m));
#pragma unroll 1
      for (int quarter = 0; quarter < 4; ++quarter, ks += 32 * 128 / 16) {   // two in each of the stages
        if (!wt(&hd.v_ready[quarter & 1], quarter >> 1)) return;
        after_sync();
        state_quarter(ks, tb + kColV + (quarter & 1) * kVStage, with_h || quarter > 0, leader);
        if (leader) commit(&hd.v_free[quarter & 1]);
      }
      if (leader) commit(&hd.kv_done);
      if ((i > 0 && !wt(&hd.o_free, i - 1)) || !wt(&hd.h_ready, i)) return;
      after_sync();
      if (with_h) {
#pragma unroll 1
        for (int term = 0; term < 2; ++term)
          chain(tb + kColO, qd, h_hi + (Sh::hterm >> 4) * term, kC, DV, DK / 16, id_h, term > 0, leader);
      }
      if (leader) {
        commit(&hd.qh_done);
        commit(&hd.q_empty);
      }
      if ((strong && !wt(&hd.o_scaled, i)) || !wt(&hd.p_ready, i)) return;
      after_sync();
      uint64_t vd = by_token(vbuf(m));
      uint32_t pt = tb + kColS;
#pragma unroll 1
      for (int k = 0; k < kC / 16; k += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j, vd += 16 * 128 / 16, pt += 16) {
          if (leader) {
            mma_ts(tb + kColO, pt, vd, id_v, with_h || k + j > 0);
            mma_ts(tb + kColO, pt + 8, vd, id_v, 1);
          }
        }
      }
      if (leader) {
        commit(&hd.o_ready);
        commit(&hd.v_empty[m & 1]);
      }
    }
  }

  // ---- warps 0-3: P over S, and the outputs, a thread per row ------------------------------------------------------------------
  __device__ __forceinline__ void rows_of_chunks(bool fresh) const {
    uint64_t u[16];                                // lambda^-j
#pragma unroll
    for (int j = 0; j < 16; ++j) u[j] = strong ? 0ull : pair(expf(a_h * (float)(-2 * j)), expf(a_h * (float)(-2 * j - 1)));
    // The triangle gives quarter q of the rows q + 1 blocks of 32 columns: of the third and the fourth, helpers make what is beyond
    // two.
    const int quarter = threadIdx.x / 32 % 4;
    const bool helper = threadIdx.x >= kControlThread;
    const int b0 = helper ? 2 : 0, b1 = !helper && quarter > 1 ? 2 : quarter + 1, zeros = !helper && quarter > 1 ? 2 : 4;
    for (int c = run.c0; c < run.c1; ++c) {
      const int i = c - run.c0;
      if (helper) {
        wt(&hd.s_ready, i);
        after_sync();
      } else {
        wt_group(kBarRows, &hd.s_ready, i);
      }
      scores(u, b0, b1, zeros);
      mbar_arrive(&hd.p_ready);
      if (helper) continue;
      if (strong) {
        wt_group(kBarRows, &hd.qh_done, i);
        if (!(fresh && i == 0)) scale_rows();
        mbar_arrive(&hd.o_scaled);
      }
      wt_group(kBarRows, &hd.o_ready, i);
      // The last chunk's store has read its staged rows: before they are overwritten where one buffer stages every chunk's, else
      // before the loader is told of these (its k_empty arrivals stay one a chunk).
      const auto last_stored = [&] {
        if (i > 0) wt_group(kBarRows, &hd.k_empty[(i - 1) & 1], (i - 1) / 2);
      };
      if (Sh::stage > 0) last_stored();
      outputs(c, obuf(i));
      mbar_arrive(&hd.o_free);
      if (rows(c) < kC) {
        named_sync(kBarRows, kStateThread);
        store_rows(c, obuf(i));
      }
      if (Sh::stage == 0) last_stored();
      mbar_arrive(&hd.o_staged);
    }
  }
  // Columns [16 b, 16 b + 16) of S become the hi terms of P in the first 8 columns of the block and the lo terms in the others.
  // The weights lambda^(63-j) are products of u and one factor per 32 columns: loads from shared memory, which the tensor
  // core's operands keep busy, would cost more than the second multiplication.
  // Blocks of 32 columns: [b0, b1) from S, [b1, zeros) above the diagonal.
  __device__ __forceinline__ void scores(const uint64_t (&u)[16], int b0, int b1, int zeros) const {
    const int t = threadIdx.x % 128, quarter = t / 32;
    const uint32_t at = tb + ((uint32_t)(32 * quarter) << 16) + kColS;
    tmem_each32(at, 32 * b1, [&](int x, uint32_t (&s)[32]) {
      // whole blocks of code for each kind: branches inside would cost more than all of this
      if (strong) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int e = t - x - j;
          s[j] = e >= 0 ? __float_as_uint(__uint_as_float(s[j]) * hd.power[e]) : 0u;
        }
        to_terms(s);
      } else {
        const uint64_t f = both(hd.power[x]);
#pragma unroll
        for (int j = 0; j < 16; ++j) unpair(mul2(mul2(pair(s[2 * j], s[2 * j + 1]), f), u[j]), s[2 * j], s[2 * j + 1]);
        to_terms(s);
        if (x == 32 * quarter) {                   // the diagonal: a mask, for a masked score may be anything
          const int lane = t % 32;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t keep = lane > 2 * j ? 0xffffffffu : lane == 2 * j ? 0xffffu : 0u;
            s[16 * (j / 8) + j % 8] &= keep;
            s[16 * (j / 8) + 8 + j % 8] &= keep;
          }
        }
      }
      tmem_st32(at + x, s);
    }, 32 * b0);
#pragma unroll 1
    for (int x = 32 * b1; x < 32 * zeros; x += 32) {
      const uint32_t zero[32] = {};
      tmem_st32(at + x, zero);
    }
    tmem_wait_st();
    before_sync();
  }
  // 32 scores in place to the terms of P's two blocks of 16
  static __device__ __forceinline__ void to_terms(uint32_t (&s)[32]) {
#pragma unroll
    for (int b = 0; b < 32; b += 16) {
      uint32_t r[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint64_t p = pair(s[b + 2 * j], s[b + 2 * j + 1]);
        r[j] = take_term(p);
        r[8 + j] = round2(p);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) s[b + j] = r[j];
    }
  }

  // kStrong: the state's part of the outputs, times lambda^(i+1)
  __device__ __forceinline__ void scale_rows() const {
    const int t = threadIdx.x;
    const uint32_t at = tb + ((uint32_t)(t & ~31) << 16) + kColO;
    const uint64_t carry = both(hd.power[t + 1]);
    tmem_each32(at, DV, [&](int x, uint32_t (&o)[32]) {
#pragma unroll
      for (int j = 0; j < 32; j += 2) unpair(mul2(pair(o[j], o[j + 1]), carry), o[j], o[j + 1]);
      tmem_st32(at + x, o);
    });
    tmem_wait_st();
    before_sync();
  }
  __device__ __forceinline__ void outputs(int c, uint8_t* stage) const {
    const int t = threadIdx.x, i = c - run.c0;
    const uint32_t at = tb + ((uint32_t)(t & ~31) << 16) + kColO;
    // one after the other: their product may leave the range that the outputs are in
    const uint64_t level = both(strong ? 1.f : expf(a_h * (float)(t - 63))), scale = both(a.scale);
    const auto term = [&](uint32_t x, uint32_t y) { return round2(mul2(mul2(pair(x, y), level), scale)); };
    const bool bad = *reinterpret_cast<const uint64_t*>(hd.bad[i & 1]) != 0;
    tmem_each32(at, DV, [&](int x, uint32_t (&o)[32]) {
      if (bad) spoil(o, hd.first_bad[i & 1][0] + x, hd.first_bad[i & 1][1] + x, t);
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        const uint4 v = make_uint4(term(o[j], o[j + 1]), term(o[j + 2], o[j + 3]), term(o[j + 4], o[j + 5]), term(o[j + 6], o[j + 7]));
        *reinterpret_cast<uint4*>(stage + sw128(kC, t, x + j)) = v;
      }
    });
    before_sync();
    fence_async_smem();
  }

  // a short chunk's rows, whole ones by neighbouring lanes
  __device__ __forceinline__ void store_rows(int c, const uint8_t* stage) const {
    bf16* out = (bf16*)a.o + ((size_t)(run.t0 + c * kC) * a.H + h) * DV;
    if (dead(hd)) return;
#pragma unroll 4
    for (int e = threadIdx.x; e < rows(c) * (DV / 8); e += kStateThread) {
      const int r = e / (DV / 8), x = e % (DV / 8) * 8;
      *reinterpret_cast<uint4*>(out + (size_t)r * a.H * DV + x) = *reinterpret_cast<const uint4*>(stage + sw128(kC, r, x));
    }
  }

  // ---- warps 4-11: V' and the state ------------------------------------------------------------------------------------------------
  // Quarter `quarter` of a chunk's V': 32 tokens as three terms into tensor memory, columns `to` on, 32 rows d per warp.
  // The tile's rows are tokens: ldmatrix turns 8 x 8 blocks of it as tcgen05.st takes them.  between receives NaN where
  // anything was not finite, and waits for the columns to be free: only then, for the terms are made under their last product.
  template <bool scaled, typename F>
  __device__ __forceinline__ void make_quarter(const uint8_t* vt, const float* w, float f, int quarter, uint32_t to, F between) const {
    __nv_bfloat162 nan(0.f, 0.f);
    const int lane = threadIdx.x % 32, row = threadIdx.x % 128 & ~31;
    uint64_t w2[4];                                // the weights of tokens 8 b + 2 (lane % 4) + {0, 1}
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      w2[b] = *reinterpret_cast<const uint64_t*>(w + 32 * quarter + 8 * b + 2 * (lane % 4));
      if (scaled) w2[b] = mul2(w2[b], both(f));
    }
    uint32_t r[2][3][8];
    if (row < DV) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {       // 16 rows
        uint32_t v[2][4];                          // (token group b, rows 0-7), (b, 8-15), (b + 1, 0-7), (b + 1, 8-15)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          ldmatrix_x4_trans(v[b], smem_u32(vt) + sw128(kC, 32 * quarter + 8 * (2 * b + lane / 16) + lane % 8,
                                                       row + 16 * half + 8 * (lane / 8 % 2)));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t u = v[e / 4][e % 4];
          nan = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u), __nv_bfloat162(0.f, 0.f), nan);
          uint64_t x = mul2(pair(u << 16, u & 0xffff0000u), w2[e / 2]);
          r[half][0][e] = take_term(x);
          r[half][1][e] = take_term(x);
          r[half][2][e] = round2(x);
        }
      }
    }
    between(nan);
    if (row < DV) {
      const uint32_t at = tb + ((uint32_t)row << 16) + to;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int term = 0; term < 3; ++term)
          tmem_st_16x128b_x4(at + ((uint32_t)(16 * half) << 16) + 16 * term, r[half][term]);
      tmem_wait_st();
    }
    before_sync();
  }

  // rows from n on of the chunk's K and V tiles belong to the next sequence (or to nobody): zeros
  __device__ __forceinline__ void clear_tail(int n_rows, uint8_t* kt, uint8_t* vt) const {
    constexpr int parts = (DK + DV) / 8;
    for (int e = threadIdx.x - kStateThread; e < (kC - n_rows) * parts; e += kStateThreads) {
      const int r = n_rows + e / parts, x = e % parts * 8;
      uint8_t* at = x < DK ? kt + sw128(kC, r, x) : vt + sw128(kC, r, x - DK);
      *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    named_sync(kBarState, kStateThreads);
  }
  // Where a value column holds something that is not finite, a masked product with it would spoil the outputs of
  // earlier tokens (0 times infinity).  Such values are taken out of the tile (the state has them), and
  // the outputs of their column from their token on are set when they are stored.
  // `first` carries over the set's two quarters of the chunk.
  __device__ __forceinline__ void settle(uint8_t* vt, int i, int quarter, __nv_bfloat162 nan, int& first) const {
    const int lane = threadIdx.x % 32, d = threadIdx.x % 128;
    if (quarter < 2) first = kC;
    if (__any_sync(kFull, !(__low2float(nan) == 0.f && __high2float(nan) == 0.f)) && d < DV) {
#pragma unroll 1
      for (int s = 32 * quarter + 31; s >= 32 * quarter; --s) {
        bf16* at = reinterpret_cast<bf16*>(vt + sw128(kC, s, d));
        if (!isfinite(__bfloat162float(*at))) {
          first = first < s ? first : s;
          *at = __float2bfloat16_rn(0.f);
        }
      }
      fence_async_smem();
    }
    if (quarter >= 2) {
      hd.first_bad[i & 1][set()][d] = (uint8_t)first;
      const bool any = __any_sync(kFull, first < kC);
      if (lane == 0) hd.bad[i & 1][(threadIdx.x - kStateThread) / 32] = any;
    }
  }

  // The state before a chunk, a thread per half row: lambda^n of it goes back at once for the next accumulation; its operand
  // terms go to shared memory when the last chunk's Q H^T (the i-1st) is done with the previous ones.
  __device__ __forceinline__ void hand_state(float step_hi, float step_lo, int i) const {
    const int d = threadIdx.x % 128, x0 = set() * (DK / 2);
    const uint32_t at = tb + ((uint32_t)(d & ~31) << 16) + kColH + x0;
    const uint64_t by_hi = both(step_hi), by_lo = both(step_lo), by_mid = both(strong ? 1.f : hd.mid);
    uint32_t hi[DK / 4], lo[DK / 4];
    if (d < DV) {
#pragma unroll
      for (int x = 0; x < DK / 2; x += 32) {
        uint32_t s[32];
        tmem_ld32_begin(at + x, s);
        arrived(s);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint64_t v = pair(s[2 * j], s[2 * j + 1]);
          uint64_t p = mul2(v, by_mid);
          hi[x / 2 + j] = take_term(p);
          lo[x / 2 + j] = round2(p);
          unpair(fma2(by_hi, v, mul2(by_lo, v)), s[2 * j], s[2 * j + 1]);
        }
        tmem_st32(at + x, s);
      }
      tmem_wait_st();
    }
    before_sync();
    mbar_arrive(&hd.h_scaled);
    if (i > 0) wt_set(&hd.qh_done, i - 1);
    if (d < DV) {
#pragma unroll
      for (int j = 0; j < DK / 4; j += 4) {
        *reinterpret_cast<uint4*>(hop + sw128(DV, d, x0 + 2 * j)) = make_uint4(hi[j], hi[j + 1], hi[j + 2], hi[j + 3]);
        *reinterpret_cast<uint4*>(hop + Sh::hterm + sw128(DV, d, x0 + 2 * j)) = make_uint4(lo[j], lo[j + 1], lo[j + 2], lo[j + 3]);
      }
    }
    fence_async_smem();
    mbar_arrive(&hd.h_ready);
  }

  // First pass, set s of three (warps 4-7, 8-11, 0-3): every third quarter, with weights up to the run's end.
  __device__ __forceinline__ void run_values(int s) const {
    int n = s;                                     // quarter number, of which there are 4 a chunk
    for (int c = run.c0; c < run.c1; ++c) {
      const int m = c - run.c0, b = m % Sh::run_bufs;
      wt_group(kBarSet + s, &hd.run_full[b], m / Sh::run_bufs);
      const float f = c + 1 < run.c1 ? expf(a_h * (float)((run.c1 - 1 - c) * kC)) : 1.f;
#pragma unroll 1
      for (; n < 4 * (m + 1); n += 3) {
        make_quarter<true>(run_v(b), hd.w[0], f, n & 3, run_stage(s), [&](__nv_bfloat162) {
          if (n >= 3) wt_group(kBarSet + s, &hd.run_free[s], n / 3 - 1);
        });
        mbar_arrive(&hd.run_ready[s]);
      }
    }
  }
  __device__ __forceinline__ void states(uint32_t kv_phase, bool fresh) const {
    const int c_end = (run.len + kC - 1) / kC;     // of the sequence
    const int all = 2 * (run.c1 - run.c0);
    int first = kC;
    // Each set's quarters one after the other; the state is handed on before the first, and then halfway through each chunk's:
    // as much of V' as there is room for is made before the state is there.
#pragma unroll 1
    for (int n = 0; n < all; ++n) {
      const int i = n >> 1, quarter = 2 * (n & 1) + set(), c = run.c0 + i, m = i;
      const bool last = c + 1 == c_end;
      if (n == 0 || (i > 0 && quarter >= 2)) {
        if (i > 0) wt_set(&hd.kv_done, kv_phase + i - 1);
        if (i > 0 || !fresh) {
          hand_state(last ? hd.last_hi : hd.step_hi, last ? hd.last_lo : hd.step_lo, i);
        } else {
          mbar_arrive(&hd.h_scaled);
          mbar_arrive(&hd.h_ready);
        }
      }
      if (quarter < 2) {
        wt_set(&hd.v_full[m & 1], m / 2);
        if (rows(c) < kC) {
          wt_set(&hd.k_full[m & 1], m / 2);
          clear_tail(rows(c), kbuf(m), vbuf(m));
        }
      }
      make_quarter<false>(vbuf(m), hd.w[last ? 1 : 0], 1.f, quarter, kColV + set() * kVStage, [&](__nv_bfloat162 nan) {
        settle(vbuf(m), i, quarter, nan, first);
        if (n > 0) wt_set(&hd.v_free[set()], n - 1);
      });
      mbar_arrive(&hd.v_ready[set()]);
    }
    wt_set(&hd.kv_done, kv_phase + run.c1 - run.c0 - 1);
  }

  // ---- the fp32 state between tensor memory and elsewhere, a thread per row ----------------------------------------
  __device__ __forceinline__ uint32_t cell(int d, int x) const {   // byte offset of floats [x, x + 4) of row d in hop
    return (uint32_t)d * (DK * 4) + (uint32_t)(((x / 4) ^ (d & 7)) * 16);
  }
  __device__ __forceinline__ void state_in(const float* src, bool shared) const {
    const int d = threadIdx.x % 128, x0 = set() * (DK / 2);
    if (d < DV) {
#pragma unroll 1
      for (int x = x0; x < x0 + DK / 2; x += 32) {
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
        tmem_st32(tb + ((uint32_t)(d & ~31) << 16) + kColH + x, r);
      }
      tmem_wait_st();
    }
    named_sync(kBarState, kStateThreads);   // hop may be overwritten
  }
  __device__ __forceinline__ void state_out(float* dst, bool shared) const {
    const int d = threadIdx.x % 128, x0 = set() * (DK / 2);
    if (d >= DV) return;
    const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;   // whole sectors
    tmem_each32(tb + ((uint32_t)(d & ~31) << 16) + kColH + x0, DK / 2, [&](int x, uint32_t (&s)[32]) {
      if (!shared && wide) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) st_global_32(dst + (size_t)d * DK + x0 + x + j, s + j);
        return;
      }
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const uint4 v = make_uint4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        if (shared) *reinterpret_cast<uint4*>(hop + cell(d, x0 + x + j)) = v;
        else *reinterpret_cast<uint4*>(dst + (size_t)d * DK + x0 + x + j) = v;
      }
    });
  }

  // Start states from the runs' own end states, in place: this CTA turns DV / split rows of every run's.
  __device__ __forceinline__ void join(const float* init, int rank, int split) const {
    const int rows_each = DV / split;
    const float f = expf(a_h * (float)(run.per * kC));
#pragma unroll 2
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

extern __shared__ __align__(1024) uint8_t linattn_smem[];   // whole 1024-byte swizzle groups

template <int DK, int DV>
__global__ void __launch_bounds__(kBlock, 1)
    k_linattn_chunks(const __grid_constant__ LinAttnArgs a, const __grid_constant__ Maps maps, int split) {
  using Sh = Shape<DK, DV>;
  const int rank = blockIdx.x % split, unit = blockIdx.x / split;
  const int i = unit / a.H, h = unit % a.H;
  const float a_h = a.log_decay[h];
  LinAttnSeq seq;
  if (!linattn_seq(a, i, h, &seq)) return;   // the same for every CTA of the cluster
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid / 32, 0), lane = tid % 32;
  if (seq.len == 0) {
    if (rank == 0)
      for (int e = tid; e < DV * DK; e += kBlock) seq.out[e] = seq.in != nullptr ? seq.in[e] : 0.f;
    return;
  }
  const int chunks = (seq.len + kC - 1) / kC;
  Run run;
  run.t0 = seq.t0;
  run.len = seq.len;
  run.per = (chunks + split - 1) / split;
  run.last_run = (chunks - 1) / run.per;
  run.c0 = min(rank * run.per, chunks);
  run.c1 = min(run.c0 + run.per, chunks);

  uint8_t* base = linattn_smem;
  uint8_t* hop = base + 3 * Sh::ktile + 2 * Sh::vtile + Sh::stage;
  Hdr& hd = *reinterpret_cast<Hdr*>(hop + 2 * Sh::hterm);
  if ((smem_u32(base) & 1023u) != 0) {   // the tiles' swizzle counts on it
    if (tid == 0) report(a.status, ERS_ECUDA);
    return;
  }
  // Of a split sequence, all runs but the last first form their own end states (K and V only); the cluster joins them.
  const bool first = run.last_run > 0 && rank < run.last_run;
  if (warp == kMmaWarp) tmem_alloc(&hd.tmem, kTmemCols);
  if (tid == 32 * kLoadWarp) {
    uint64_t* by_one[] = {&hd.k_full[0], &hd.k_full[1], &hd.k_empty[0], &hd.k_empty[1], &hd.v_full[0], &hd.v_full[1],
                          &hd.v_empty[0], &hd.v_empty[1], &hd.q_full, &hd.q_empty, &hd.s_ready, &hd.qh_done, &hd.o_ready,
                          &hd.kv_done, &hd.v_free[0], &hd.v_free[1], &hd.run_free[0], &hd.run_free[1], &hd.run_free[2],
                          &hd.run_full[0], &hd.run_full[1], &hd.run_full[2], &hd.run_empty[0], &hd.run_empty[1],
                          &hd.run_empty[2]};
    for (uint64_t* b : by_one) mbar_init(b, 1);
    mbar_init(&hd.p_ready, 192);
    uint64_t* by_four[] = {&hd.o_scaled, &hd.o_free, &hd.o_staged, &hd.v_ready[0], &hd.v_ready[1],
                           &hd.run_ready[0], &hd.run_ready[1], &hd.run_ready[2]};
    for (uint64_t* b : by_four) mbar_init(b, 128);
    mbar_init(&hd.h_scaled, 256);
    mbar_init(&hd.h_ready, 256);
    fence_mbar_init();
    hd.dead = 0;
    // the first tiles come while the others set up
    const Cta<DK, DV> loader{a, maps, hd, base, hop, 0, h, h / (a.H / a.G), a_h, false, run};
    if (first) loader.load_run_head();
    else loader.load_head();
  }
  const int n_last = seq.len - (chunks - 1) * kC;
  if (tid >= 128 && tid < 128 + kC) {
    const int j = tid - 128;
    // lambda^0 = 1 whatever lambda
    const bool strong = is_strong(a_h);
    hd.power[j] = strong ? (j == 0 ? 1.f : expf(a_h * (float)j)) : expf(a_h * (float)(63 - j));
    if (j == 0) {
      hd.power[kC] = expf(a_h * (float)kC);   // of the strong ones
      hd.mid = expf(a_h * 64.f);
    }
    hd.w[0][j] = j == kC - 1 ? 1.f : expf(a_h * (float)(kC - 1 - j));
    hd.w[1][j] = j >= n_last ? 0.f : j == n_last - 1 ? 1.f : expf(a_h * (float)(n_last - 1 - j));
  } else if (tid < 2) {                            // multiplied once a chunk over the whole sequence: as two floats
    const Decay e = decay_of(a_h * (float)(tid == 0 ? kC : n_last));
    (tid == 0 ? hd.step_hi : hd.last_hi) = e.hi;
    (tid == 0 ? hd.step_lo : hd.last_lo) = e.lo;
  }
  before_sync();
  __syncthreads();
  after_sync();
  Cta<DK, DV> cta{a, maps, hd, base, hop, __shfl_sync(kFull, hd.tmem, 0), h, h / (a.H / a.G), a_h, is_strong(a_h), run};

  uint32_t kv_phase = 0;
  if (first) {
    kv_phase = 1;
    if (warp == kLoadWarp) {
      if (lane == 0) cta.load_run_rest();
    } else if (warp == kMmaWarp) {
      cta.issue_states();
    } else if (tid < kControlThread) {
      cta.run_values(tid < kStateThread ? 2 : cta.set());
      if (tid >= kStateThread) {
        cta.wt_set(&hd.kv_done, 0);
        cta.state_out(nullptr, true);
      }
    }
    __syncwarp();
  }
  if (split > 1) {
    before_sync();
    cluster_sync();
    if (run.last_run > 0) cta.join(seq.in, rank, split);
    cluster_sync();
    after_sync();
  }
  const bool given = run.last_run > 0 ? (rank > 0 || seq.in != nullptr) : seq.in != nullptr;
  if (run.c0 < run.c1) {
    if (warp == kLoadWarp) {
      if (lane == 0) {
        if (first) cta.load_head();
        cta.load_chunks();
      }
    } else if (warp == kMmaWarp) {
      cta.issue_chunks(!given);
    } else if (tid >= kStateThread && tid < kControlThread) {
      if (given) cta.state_in(seq.in, run.last_run > 0);
      cta.states(kv_phase, !given);
      if (rank == run.last_run && !dead(hd)) cta.state_out(seq.out, false);
    } else {
      cta.rows_of_chunks(!given);
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

constexpr int kSplits = 4;               // 1, 2, 4 and 8 CTAs of a sequence and head

template <int DK, int DV>
cudaLaunchConfig_t config(cudaLaunchAttribute* attr, long long units, int split, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(units * split));
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = Shape<DK, DV>::smem;
  cfg.stream = s;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)split;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// How many clusters of 1, 2, 4 and 8 CTAs the current device runs at once; the first call on it also lets the kernel have its
// shared memory.
template <int DK, int DV>
cudaError_t clusters_at_once(int (&fit)[kSplits]) {
  static std::mutex mu;
  static bool done[64];
  static int known[64][kSplits];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    e = cudaFuncSetAttribute(k_linattn_chunks<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<DK, DV>::smem);
    for (int i = 0; i < kSplits && e == cudaSuccess; ++i) {
      cudaLaunchAttribute attr;
      const cudaLaunchConfig_t cfg = config<DK, DV>(&attr, 1, 1 << i, nullptr);
      e = cudaOccupancyMaxActiveClusters(&known[dev][i], k_linattn_chunks<DK, DV>, &cfg);
    }
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  memcpy(fit, known[dev], sizeof(fit));
  return cudaSuccess;
}

// Over how many CTAs a sequence goes: what takes the least time by a model in quarters of a chunk's time (0.8 us).  A split
// sequence's chunks cost half as much again (the first pass) and a join 6; clusters that do not fit at once wait for
// others, and not all that the SMs would hold fit (of 8 CTAs the GPU's clusters of SMs hold few).  Of the lengths only
// the longest and the sum are known: as many sequences as the sum has longest ones count, the others as short ones, 10
// each, beside them or after them (2 where this launch leaves short ones out).  128 x 128, by 1, 2, 4 and 8 CTAs, us:
//   512 tokens x 32 heads   19.9  21.2   19.8     -     |   2048 x 64   57.1   51.3   64.8  110.8
//   1024 x 32               32.2  30.2   24.4   51.9    |   2048 x 128  62.1  102.7  126.5  199.4
//   2048 x 16               55.8  45.7   31.0   43.7    |   8192 x 8   200.2  142.5   79.4   47.8
//   2048 x 32               56.7  47.0   33.5   64.6    |   8192 x 64  204.7  159.4  169.4  238.6
// 4096 and 30 of 40 tokens x 32 heads: 113, 162; 2048 and three of 1: by 2 47.4, by 4 52.7.
int split_of(const LinAttnArgs& a, const int (&fit)[kSplits]) {
  const long long chunks = (a.max_len + kC - 1) / kC;
  const long long full = min(max((a.ntokens + a.max_len / 2) / max(a.max_len, 1), 1LL), (long long)a.nseq);
  const long long others = (a.nseq - full) * a.H * (a.len0 > 1 ? 2 : 10);
  int best = 0;
  long long least = 0;
  for (int i = 0; i < kSplits && (chunks >> i) >= 1; ++i) {
    if (fit[i] <= 0) break;
    const long long run = (chunks + (1 << i) - 1) >> i, one = i == 0 ? 4 * run : 6 * run + 6;
    const long long waves = (full * a.H + fit[i] - 1) / fit[i];
    const long long cost = max(waves * one, (full * a.H * one + others) / fit[i]);
    if (i == 0 || cost < least) {
      least = cost;
      best = i;
    }
  }
  return 1 << best;
}

template <int DK, int DV>
cudaError_t launch(const LinAttnArgs& a, const Maps& maps, cudaStream_t s) {
  int fit[kSplits];
  const cudaError_t e = clusters_at_once<DK, DV>(fit);
  if (e != cudaSuccess) return e;
  const int split = split_of(a, fit);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config<DK, DV>(&attr, (long long)a.nseq * a.H, split, s);
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
  if (a.dk == 64) return a.dv == 64 ? launch<64, 64>(a, maps, s) : launch<64, 128>(a, maps, s);
  return a.dv == 64 ? launch<128, 64>(a, maps, s) : launch<128, 128>(a, maps, s);
}

}  // namespace ers
