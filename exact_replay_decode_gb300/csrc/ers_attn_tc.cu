// Attention of drafts over a paged cache, bf16, on the tensor cores.
//
// A CTA takes 128 query rows that share a head of keys (drafts x heads of the group; the rest of the tile is zeros) and a run of
// the sequence's past, in tiles of 64 tokens, then the drafts themselves:
//   S = Q K^T   (A, B from shared memory)      P = exp(c S - m), rounded to bf16, over S in tensor memory
//   O += P V    (A from tensor memory)         l += sum P, of the rounded ones: O / l is an average of values
// with c = scale log2 e (P by powers of two) and m a running maximum that moves, and O with it, only when a row's maximum has
// risen by more than 2^8: P then stays below 2^8, which costs no bits.
//
// Four warps own the rows, a thread each (a tile's scores of a row stay in its registers), two load tiles, one issues the MMAs: S
// of the next tile before P V of this one if the tile is there, so that the tensor core works under the exponentials.  Whole
// tiles of pages whose tokens are a multiple of 8 come by TMA, `box` tokens at a time; others, and the last one (zeros behind
// the last token: a page may hold anything there), by 16-byte copies of both warps.  Two CTAs per SM (two stages of 32 KB each at D 128, 256 columns of tensor
// memory) run beside each other: one loads while the other computes.
//
// What bounds it: a tile moves 32 KB (D 128), 0.74 us of an SM's share of the memory, and its exponentials take 512 cycles of each
// scheduler.  64 trees of 16 drafts over 2269 to 4096 tokens x 8 heads: 175 us, 126 of them the bytes' (the 512 CTAs come in
// waves of 304; with a head's sequences side by side in place of a sequence's heads 185); one token over 32768 39 us in 37 parts (20 the bytes'; set-up, a part's first loads and the join are the rest);
// 256 single tokens over 1024 214 us (160).  All loading threads polling in place of one cost 388 us in place of 185: they take
// issue slots from the rows'.
#include <string.h>

#include <mutex>

#include "attn_cache.cuh"
#include "ers_common.cuh"
#include "ers_internal.h"
#include "tc_common.cuh"
#include "tc_terms.cuh"
#include "tma_host.h"

namespace ers {
namespace {

using namespace tc;
using bf16 = __nv_bfloat16;

constexpr int kM = 128, kTokens = 64, kStages = 2;
constexpr int kLoadThread = 128, kLoaders = 64, kIssueThread = 192, kBlock = 224;   // (nine warps would have 96 registers each, and spill)
constexpr uint32_t kColS = 0, kColO = 128, kCols = 256;   // two tiles' scores, the outputs
constexpr float kRise = 8.f;

struct Hdr {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], s_ready[2], p_ready, o_done;
  uint64_t bad;                      // drafts whose values are not finite
  int32_t parent[kMaxDrafts];
  uint32_t tmem;
  int dead;                          // a wait gave up: no further wait waits, no copy or MMA is issued
};

template <int D>
struct Shape {
  static constexpr uint32_t qtile = kM * D * 2, tile = kTokens * D * 2, smem = qtile + kStages * 2 * tile + sizeof(Hdr) + 1024;
  static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs per SM");
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

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {   // without waiting
  uint32_t done;
  asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return done != 0;
}
__device__ __forceinline__ float exp2_of(float x) {   // 2 units in the last place; 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void copy16(void* to, const void* from, bool there) {   // zeros where there is nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Where a bf16 pair is not finite: its exponent is all ones.
__device__ __forceinline__ bool not_finite(uint32_t u) {
  return (u & 0x7f800000u) == 0x7f800000u || (u & 0x7f80u) == 0x7f80u;
}

struct Maps {
  CUtensorMap k, v;
};

// box: tokens of a TMA copy, a divisor of a page's and of a tile's; 0: none
template <int D>
__global__ void __launch_bounds__(kBlock, 2) k_attn_tiles(const __grid_constant__ AttnArgs a, const __grid_constant__ Maps maps, int box) {
  using Sh = Shape<D>;
  extern __shared__ uint8_t attn_smem[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(attn_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* stages = base + Sh::qtile;          // K, V, K, V
  Hdr& hd = *reinterpret_cast<Hdr*>(stages + kStages * 2 * Sh::tile);
  // the heads of a sequence's tokens side by side: their rows lie beside each other
  const int heads = (a.T * (a.H / a.KV) + kM - 1) / kM * a.KV, head = blockIdx.x % heads, run = blockIdx.x / heads;
  const int split = run % a.nsplit, i = run / a.nsplit, kv = head % a.KV, row0 = head / a.KV * kM;
  const int rep = a.H / a.KV, nrows = a.T * rep, tid = threadIdx.x, warp = __shfl_sync(kFull, tid / 32, 0);
  const int row = row0 + tid;                  // of the threads that own rows
  const auto out_row = [&](int r) { return ((size_t)i * a.T + r / rep) * a.H + kv * rep + r % rep; };
  AttnSeq s;
  int32_t err = attn_seq(a, i, &s);
  uint4 q[D / 8];
  if (tid < kM) {
    const bf16* from = (const bf16*)a.q + (row < nrows ? out_row(row) * D : 0);
#pragma unroll
    for (int x = 0; x < D / 8; ++x) q[x] = row < nrows ? *reinterpret_cast<const uint4*>(from + 8 * x) : make_uint4(0, 0, 0, 0);
  }
  if (a.parent != nullptr && tid < a.T) hd.parent[tid] = a.parent[(size_t)i * a.T + tid];
  const bool last = split == a.nsplit - 1;
  const long long begin = (long long)split * a.per;
  const int end = err != ERS_OK ? 0 : last ? s.pos : (int)min((long long)s.pos, begin + a.per);
  const int past = begin < end ? (int)((end - begin + kTokens - 1) / kTokens) : 0, tiles = past + (last ? 1 : 0);
  const int whole = box > 0 && begin < end ? (int)((end - begin) / kTokens) : 0;   // tiles that come by TMA
  // ---- TMA: one thread, the first tiles while the others set up.  Pages are looked up a tile ahead, all at once: one after the
  // other they took longer than the copies.
  constexpr int kBoxes = kTokens / 8;
  const int boxes = box > 0 ? kTokens / box : 0;
  int page[kBoxes];
  bool missing = false;
  const auto look_up = [&](int n) {
#pragma unroll
    for (int x = 0; x < kBoxes; ++x) {
      const int at = (int)begin + n * kTokens + x * box;
      page[x] = n < whole && x < boxes ? s.pages[page_of(a, at)] : -1;
    }
  };
  const auto load = [&](int n, uint8_t* to, const CUtensorMap* map, uint64_t* full) {
    if (dead(hd)) return;
    uint32_t count = 0;
#pragma unroll
    for (int x = 0; x < kBoxes; ++x) count += page[x] >= 0 && page[x] < a.npages;
    missing |= count < (uint32_t)boxes;
    mbar_arrive_expect_tx(full, count * box * D * 2);
#pragma unroll
    for (int x = 0; x < kBoxes; ++x) {
      if (page[x] < 0 || page[x] >= a.npages) continue;
      const int at = (int)begin + n * kTokens + x * box, at_row = page[x] * a.page_tokens + (at - page_of(a, at) * a.page_tokens);
#pragma unroll
      for (int d = 0; d < D; d += 64) tma_load_3d(to + d * kTokens * 2 + x * box * 128, map, d, kv, at_row, full);
    }
  };
  const auto load_tile = [&](int n) {
    const int b = n % kStages;
    uint8_t* kt = stages + b * 2 * Sh::tile;
    if (n >= kStages) wait(hd, &hd.k_empty[b], n / kStages - 1, a.status);   // K's place is free long before V's
    load(n, kt, &maps.k, &hd.k_full[b]);
    if (n >= kStages) wait(hd, &hd.v_empty[b], n / kStages - 1, a.status);
    load(n, kt + Sh::tile, &maps.v, &hd.v_full[b]);
    look_up(n + 1);
  };
  if (tid == kLoadThread) {
    for (int b = 0; b < kStages; ++b) {
      mbar_init(&hd.k_full[b], 1);
      mbar_init(&hd.v_full[b], 1);
      mbar_init(&hd.k_empty[b], 1);
      mbar_init(&hd.v_empty[b], 1);
      mbar_init(&hd.s_ready[b], 1);
    }
    mbar_init(&hd.p_ready, min(kM, (nrows - row0 + 31) / 32 * 32));   // of the warps that have rows
    mbar_init(&hd.o_done, 1);
    fence_mbar_init();
    hd.dead = 0;
    hd.bad = 0;
    look_up(0);
    for (int n = 0; n < kStages && n < whole; ++n) load_tile(n);
  }
  if (warp == kIssueThread / 32) tmem_alloc(&hd.tmem, kCols);
  if (tid < kM) {
#pragma unroll
    for (int x = 0; x < D / 8; ++x) *reinterpret_cast<uint4*>(base + sw128(kM, tid, 8 * x)) = q[x];
    fence_async_smem();
  }
  __syncthreads();
  const int32_t* parent = a.parent != nullptr ? hd.parent : nullptr;
  bool wrong = false;
  if (tid < a.T) path_of(parent, tid, &wrong);
  before_sync();
  const bool bad_tree = __syncthreads_or(wrong);
  after_sync();
  const uint32_t tb = __shfl_sync(kFull, hd.tmem, 0);
  if (bad_tree || err != ERS_OK || tiles == 0) {   // an error, or nothing of the past is this CTA's
    if (tid == 0 && (bad_tree || err != ERS_OK)) report(a.status, err != ERS_OK ? err : ERS_EINVAL);
    if (a.nsplit > 1 && tid < kM && row < nrows)
      reinterpret_cast<float2*>(a.part)[out_row(row) * a.nsplit + split] = make_float2(0.f, bad_tree || err != ERS_OK ? -1.f : 0.f);
    if (tid == kLoadThread)                    // no copy may be left in flight
      for (int n = 0; n < kStages && n < whole; ++n) {
        wait(hd, &hd.k_full[n], 0, a.status);
        wait(hd, &hd.v_full[n], 0, a.status);
      }
    __syncthreads();
    if (warp == kIssueThread / 32) tmem_dealloc(tb, kCols);
    return;
  }

  if (tid >= kIssueThread) {
    // ---- the issuing warp: its lanes go on or leave together, whichever of them a wait lets go (one lane alone: 179 us in place
    // of 175) ------------------------------------------------------------------------------------------------
    constexpr uint32_t id_s = idesc_bf16(kM, kTokens, false, false), id_o = idesc_bf16(kM, D, false, true);
    const bool leader = elected();
    const auto there = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, wait(hd, bar, parity, a.status)) != 0; };
    const auto scores = [&](int n) {
      const int b = n % kStages;
      if (!there(&hd.k_full[b], n / kStages)) return false;
      after_sync();
      fence_async_smem();
      const uint32_t kt = smem_u32(stages + b * 2 * Sh::tile), qt = smem_u32(base);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        if (leader)
          mma(tb + kColS + (n & 1) * kTokens, sdesc(qt + (k >> 2) * kM * 128 + (k & 3) * 32, 16, 1024),
              sdesc(kt + (k >> 2) * kTokens * 128 + (k & 3) * 32, 16, 1024), id_s, k > 0);
      if (leader) {
        commit(&hd.s_ready[n & 1]);
        commit(&hd.k_empty[b]);
      }
      return true;
    };
    bool ok = scores(0);
#pragma unroll 1
    for (int n = 0; ok && n < tiles; ++n) {
      bool ahead = n + 1 < tiles;
      if (ahead && !__all_sync(kFull, mbar_test(&hd.k_full[(n + 1) % kStages], (n + 1) / kStages & 1))) ahead = false;
      if (ahead && !scores(n + 1)) break;
      const int b = n % kStages;
      if (!there(&hd.v_full[b], n / kStages) || !there(&hd.p_ready, n)) break;
      after_sync();
      const uint64_t vd = sdesc(smem_u32(stages + b * 2 * Sh::tile + Sh::tile), kTokens * 128, 1024);
#pragma unroll
      for (int k = 0; k < kTokens / 16; ++k)
        if (leader) mma_ts(tb + kColO, tb + kColS + (n & 1) * kTokens + 8 * k, vd + k * (16 * 128 / 16), id_o, n > 0 || k > 0);
      if (leader) {
        commit(&hd.v_empty[b]);
        commit(&hd.o_done);
      }
      if (!ahead && n + 1 < tiles && !scores(n + 1)) break;
    }
  } else if (tid >= kLoadThread) {
    // ---- the loading warps ------------------------------------------------------------------------------
    const int t = tid - kLoadThread;
    if (t == 0)                                // (one thread polls: warps that do take issue slots from the rows')
      for (int n = kStages; n < whole; ++n) load_tile(n);
    // What is left by all of them, a tile's rows by 8 (D 64) or 16 neighbouring threads.
    constexpr int kPer = D / 8, kStep = kLoaders / kPer, kEach = kTokens / kStep;
    const int c = t % kPer * 8, r0 = t / kPer;
    bool pending = false;                      // copies of the tile before
    const auto arrive = [&](int n) {
      if (!pending) return;
      copies_wait();
      fence_async_smem();
      named_sync(1, kLoaders);
      if (t == 0) {
        mbar_arrive(&hd.k_full[n % kStages]);
        mbar_arrive(&hd.v_full[n % kStages]);
      }
    };
    for (int n = whole; n < tiles; ++n) {
      arrive(n - 1);                           // told before any wait for its stage's turn
      const int b = n % kStages;
      if (t == 0 && n >= kStages) {
        wait(hd, &hd.k_empty[b], n / kStages - 1, a.status);
        wait(hd, &hd.v_empty[b], n / kStages - 1, a.status);
      }
      named_sync(1, kLoaders);
      uint8_t *kt = stages + b * 2 * Sh::tile, *vt = kt + Sh::tile;
      pending = true;
      if (dead(hd)) continue;
      if (n < past) {
        int at_page[kEach];
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
          const int at = (int)begin + n * kTokens + r0 + x * kStep;
          at_page[x] = at < end ? s.pages[page_of(a, at)] : -1;
        }
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
          const int r = r0 + x * kStep, at = (int)begin + n * kTokens + r;
          const bool there = at_page[x] >= 0 && at_page[x] < a.npages;
          missing |= !there && at < end;
          const size_t at_row = there ? (size_t)at_page[x] * a.page_tokens + (at - page_of(a, at) * a.page_tokens) : 0;
          const size_t from = (at_row * a.KV + kv) * D + c;
          copy16(kt + sw128(kTokens, r, c), (const bf16*)a.k_pages + from, there);
          copy16(vt + sw128(kTokens, r, c), (const bf16*)a.v_pages + from, there);
        }
        continue;
      }
      // Drafts: a value that is not finite would reach rows that do not see it as 0 x infinity, so it is left out, and
      // those that see it are made NaN at the end.
      for (int r = r0; r < kTokens; r += kStep) {
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        if (r < a.T) {
          const size_t from = (((size_t)i * a.T + r) * a.KV + kv) * D + c;
          k = *reinterpret_cast<const uint4*>((const bf16*)a.k + from);
          v = *reinterpret_cast<const uint4*>((const bf16*)a.v + from);
          if (not_finite(v.x) || not_finite(v.y) || not_finite(v.z) || not_finite(v.w)) {
            atomicOr(reinterpret_cast<unsigned long long*>(&hd.bad), 1ull << r);
            v = make_uint4(0, 0, 0, 0);
          }
        }
        *reinterpret_cast<uint4*>(kt + sw128(kTokens, r, c)) = k;
        *reinterpret_cast<uint4*>(vt + sw128(kTokens, r, c)) = v;
      }
    }
    arrive(tiles - 1);
    if (missing) report(a.status, ERS_ESLOT);
  } else if (row0 + (tid & ~31) < nrows) {
    // ---- the rows (a warp without any does nothing: what its lanes of P and O hold is read by no one) -------------------------------------------------------------------------------------------
    const float c = a.scale * 1.44269504088896340736f;
    bool unused = false;
    const uint64_t path = row < nrows ? path_of(parent, row / rep, &unused) : 0;
    const uint32_t at = tb + ((uint32_t)(tid & ~31) << 16);
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int n = 0; n < tiles; ++n) {
      wait(hd, &hd.s_ready[n & 1], n >> 1, a.status);
      __syncwarp();
      after_sync();
      const uint32_t sc = at + kColS + (n & 1) * kTokens;
      uint32_t u[2][32];
      tmem_ld32_begin(sc, u[0]);
      tmem_ld32_begin(sc + 32, u[1]);
      arrived(u[0]);
      arrived(u[1]);
      uint64_t seen = path;
      if (n < past) {
        const int count = end - ((int)begin + n * kTokens);
        seen = path == 0 ? 0 : count >= kTokens ? ~0ull : (1ull << count) - 1;
      }
      const bool whole = __all_sync(kFull, seen == ~0ull);
      float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < 64; ++x) u[x / 32][x % 32] = __float_as_uint(__uint_as_float(u[x / 32][x % 32]) * c);
      if (!whole) {
#pragma unroll
        for (int x = 0; x < 64; ++x) u[x / 32][x % 32] = (uint32_t)(seen >> (x & 32)) >> (x & 31) & 1u ? u[x / 32][x % 32] : 0xff800000u;
      }
#pragma unroll
      for (int x = 0; x < 64; ++x) tops[x % 4] = fmaxf(tops[x % 4], __uint_as_float(u[x / 32][x % 32]));
      const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
      // (a row that has seen nothing rises from -inf; one that still sees nothing does not)
      const bool rise = top > m + kRise || (m == -INFINITY && top > m);
      const float next = rise ? top : m, factor = rise ? exp2_of(m - next) : 1.f;   // from -inf: 0
      const float down = next == -INFINITY ? 0.f : next;
      uint32_t p[32];
      float sums[4] = {};
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        p[x] = pack_bf16x2(exp2_of(__uint_as_float(u[x / 16][x % 16 * 2]) - down), exp2_of(__uint_as_float(u[x / 16][x % 16 * 2 + 1]) - down));
        sums[x % 2 * 2] += __uint_as_float(p[x] << 16);
        sums[x % 2 * 2 + 1] += __uint_as_float(p[x] & 0xffff0000u);
      }
      l = fmaf(l, factor, (sums[0] + sums[1]) + (sums[2] + sums[3]));
      m = next;
      if (n > 0) {
        wait(hd, &hd.o_done, n - 1, a.status);
        __syncwarp();
        after_sync();
        if (__any_sync(kFull, rise)) {
#pragma unroll 1
          for (int x = 0; x < D; x += 32) {
            uint32_t o[32];
            tmem_ld32_begin(at + kColO + x, o);
            arrived(o);
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * factor);
            tmem_st32(at + kColO + x, o);
          }
        }
      }
      tmem_st32(sc, p);
      tmem_wait_st();
      before_sync();
      mbar_arrive(&hd.p_ready);
    }
    wait(hd, &hd.o_done, tiles - 1, a.status);
    __syncwarp();
    after_sync();
    const bool spoiled = last && (path & *(volatile uint64_t*)&hd.bad) != 0;
    if (spoiled) l = __int_as_float(0x7fffffff);
    const size_t out = row < nrows ? out_row(row) : 0, part = out * a.nsplit + split, all = (size_t)a.nseq * a.T * a.H * a.nsplit;
    if (row < nrows && a.nsplit > 1) reinterpret_cast<float2*>(a.part)[part] = make_float2(m * 0.69314718055994530942f, l);
    const float f = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
    for (int x = 0; x < D; x += 32) {
      uint32_t o[32];
      __syncwarp();                            // (lanes without a row come from the end of the loop)
      tmem_ld32_begin(at + kColO + x, o);
      arrived(o);
      if (row >= nrows) continue;
      if (a.nsplit > 1) {
        float* to = a.part + part_outputs(all) + part * D + x;
#pragma unroll
        for (int y = 0; y < 32; y += 4) *reinterpret_cast<uint4*>(to + y) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
      } else {
        bf16* to = (bf16*)a.o + out * D + x;
        uint32_t w[16];
#pragma unroll
        for (int y = 0; y < 16; ++y)
          w[y] = l == 0.f ? 0u : pack_bf16x2(__uint_as_float(o[2 * y]) * f, __uint_as_float(o[2 * y + 1]) * f);
#pragma unroll
        for (int y = 0; y < 16; y += 4) *reinterpret_cast<uint4*>(to + 2 * y) = make_uint4(w[y], w[y + 1], w[y + 2], w[y + 3]);
      }
    }
  }
  __syncwarp();
  if (tid == kIssueThread && dead(hd)) {       // no MMA may be left in flight: 2 ms are a thousand times what one takes
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000) {}
  }
  before_sync();
  __syncthreads();
  if (warp == kIssueThread / 32) tmem_dealloc(tb, kCols);
}

bool encode(CUtensorMap* m, const void* base, long long rows, int heads, int d, int box_rows) {
  const EncodeTiledFn fn = tma_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * heads * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
  const cuuint32_t each[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, each,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(k_attn_tiles<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::smem);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  const int tiles = (a.T * (a.H / a.KV) + kM - 1) / kM;
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  int box = kTokens;
  while (a.page_tokens % box != 0) box /= 2;
  const long long rows = (long long)a.npages * a.page_tokens;
  if (box < 8 || rows < box || rows > 0x7fffffff || !encode(&maps.k, a.k_pages, rows, a.KV, D, box) ||
      !encode(&maps.v, a.v_pages, rows, a.KV, D, box))
    box = 0;
  k_attn_tiles<D><<<(unsigned)((long long)a.nseq * a.nsplit * tiles * a.KV), kBlock, Shape<D>::smem, s>>>(a, maps, box);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_tiles(const AttnArgs& a, cudaStream_t s) { return a.D == 64 ? launch<64>(a, s) : launch<128>(a, s); }

}  // namespace ers
