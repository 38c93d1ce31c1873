// Masked attention backward for B200 (sm_100a).
//
// With P = exp(score - lse) over the visible pairs and delta = sum dO o (see
// fa_bwd.h for the row statistics):
//     dV = P^T dO,   dS = P * (dO V^T - delta),   dQ = scale dS K,
//     dK = scale dS^T Q
//
// Two walks, one structure. The query walk (kKeys = false) holds 128 query rows
// and visits their key tiles for dQ, the key walk (kKeys = true) holds 128 keys
// and visits their query tiles for dK and dV. Each recomputes the scores: seven
// products a pair of tiles, but every sum stays in tensor memory and has one
// fixed order: no partial gradients go through L2, no atomics, equal bits on
// every call. Or the key walk writes dS out once and a third kernel
// (fa_bwd_dq_sm100) multiplies it by K: five products and 32 KB written and
// read a pair of tiles. Adding the key tiles' shares of dQ up in L2 instead was
// built and measured: red.add of 64 KB a step runs at about 2.6 TB/s over the
// card, 3,200 cycles a step (causal 2 x 16 x 4096 x 128: 444 us against 394).
//
// The walks are the same chain with the roles of the operands exchanged. A0,
// A1 are held (Q, dO; K, V) and B0, B1 streamed (K, V; Q, dO):
//     S = A0 B0^T, dP = A1 B1^T, acc0 += dS B0 (dQ; dK), acc1 += P B1 (dV)
// The rows of every product are tensor memory lanes, and P and dS go back to
// tensor memory in bf16, over the scores they came from, as the A operand of
// the accumulating products, so that shared memory feeds only their B; the
// query walk also holds A0 and A1 in tensor memory (the key walk at head dim
// 128 has no room left there).
//
// One persistent CTA per SM, 24 warps:
//   warps 0-15   P and dS, four groups of four warps, 32 columns of a tile each
//   warps 16-19  epilogue: accumulators to global memory; query walk: Q and
//                dO of the next item from global to tensor memory
//   warp 20      all products (one lane issues; owns tensor memory)
//   warp 21      TMA loads; claims the items; clears the rows of a streamed
//                tile that belong to the next packed sequence
//   warp 22      idle
//   warp 23      bias gradient: the tile's sums by distance (key walk)
// Order of the products: query walk S(t+1), dQ(t), dP(t+1); key walk dV(i),
// S(i+1), dK(i), dP(i+1), also across items, so that the products of one step
// run while P and dS of the other are computed. They are issued by an elected
// lane of a converged warp, which keeps descriptors in uniform registers: a
// thread of its own took 560 to 1,400 cycles to issue eight products, this 410
// to 520, their execution.
//
// What bounds it. Head dim 128: the card's power limit (1,000 W, about 1.45
// GHz, on anything longer than a few milliseconds; the products' rate is then
// 0.84 of what cuBLAS sustains there), so products and bytes count, not
// cycles: an exponential on the FMA pipe, stores moved to other warps or a
// shorter chain cost or change nothing. Head dim 64: the math warps, whose
// phases (scores to P, dP to dS) follow each other; the issue slots are 56 %
// busy, the MUFU unit 40 %.
// Every mbarrier wait is bounded, as in the forward.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "../../include/fa.h"
#include "fa_bwd.h"
#include "fa_device.h"
#include "fa_tmem_asm.h"

namespace fa {
namespace dev {

// The 128 columns of a tile are shared out over groups of four math warps.
// Four groups against two: more warps hide each other's latencies where the
// math bounds a step (head dim 64: 658 -> 638 us on the bias backward of
// 2 x 16 x 4096 x 64; at 128 the same within 1 %).
constexpr int kGroups = 4, kCols = 128 / kGroups, kMathWarps = 4 * kGroups;
constexpr int kWarpEpi = kMathWarps, kWarpMma = kWarpEpi + 4, kWarpLoad = kWarpMma + 1,
              kWarpSums = kWarpMma + 3;
constexpr int kBwdThreads = 32 * (kMathWarps + 8);
// Register split over the registers of the launch.
constexpr int kBwdRegsLaunch = 65536 / kBwdThreads / 8 * 8;
constexpr int kBwdRegsMath = 88, kBwdRegsEpi = 72, kBwdRegsControl = 56;
static_assert(32 * kMathWarps * kBwdRegsMath + 128 * kBwdRegsEpi + 128 * kBwdRegsControl ==
                  kBwdThreads * kBwdRegsLaunch,
              "register split must equal the launch allocation");
constexpr int kSumRow = kCols + 32;  // bias gradient: diagonals of 32 rows x kCols columns
constexpr int kBwdBiasNone = 0, kBwdBiasAlibi = 1, kBwdBiasRel = 2;
constexpr float kLog2e = 1.4426950408889634f;
// Of 8 pairs of columns, how many take the FMA-pipe exponential. At head dim
// 64 the exponentials bound a step (0: 500, 1: 484, 2: 473 us on 2 x 16 x 4096 x
// 64 without a mask; 584, 573, 566 with the learned bias, whose 4: 30 us more); at
// 128 the power cap does, and the MUFU unit needs less (0: 457, 3: 463 us on a
// causal 2 x 16 x 4096 x 128).
template <int D>
constexpr int kPolyOf8 = D == 64 ? 2 : 0;
template <int D>
constexpr bool kWritesDs = bwd_may_write_ds(D);

// Where a wait gave up (error word bits 8..15), after the forward's sites.
enum BwdSite : uint32_t {
  kBSiteB0Empty = 32, kBSiteB1Empty, kBSiteStatEmpty, kBSiteA0Empty, kBSiteA1Empty, kBSiteFix,
  kBSiteB0Full, kBSiteB1Full, kBSiteStatFull, kBSiteA0Full, kBSiteA1Full, kBSiteSFull, kBSiteSFree,
  kBSitePFull, kBSiteDpFull, kBSiteDsFull, kBSiteAccFull, kBSiteAccFree, kBSiteSumFull,
  kBSiteSumEmpty, kBSiteFarFull, kBSiteFarEmpty, kBSiteDrain, kBSiteSmem, kBSiteIdxFull,
  kBSiteIdxEmpty,
};

template <int D, bool kKeys, bool kRel>
struct BCfg {
  // The key walk sums the bias's gradient.
  static constexpr bool kSums = kKeys && kRel;
  static constexpr int kChunks = D / 64;
  static constexpr uint32_t kChunkBytes = 128u * 128u;
  static constexpr uint32_t kTileBytes = 128u * D * 2u;
  // Ring depths. B0(t) is read first by S(t) and last by acc0(t), a step
  // later; B1(t) by dP(t) (and acc1(t)).
  static constexpr int kN0 = D == 64 || !kKeys ? 4 : (kSums ? 2 : 3);
  static constexpr int kN1 = D == 128 ? 2 : 4;
  static constexpr uint32_t kABytes = kKeys ? 2u * kTileBytes : 0u;
  static constexpr uint32_t kRingBytes = (kN0 + kN1) * kTileBytes;
  static constexpr uint32_t kStatBytes = kKeys ? 2u * 1024u : 0u;
  static constexpr uint32_t kSumBytes = kSums ? 2u * kMathWarps * kSumRow * 4u : 0u;
  static constexpr uint32_t kCtlBytes = 1024u;
  static constexpr uint32_t kSmemBytes = kABytes + kRingBytes + kStatBytes + kSumBytes + kCtlBytes;
  static_assert(kSmemBytes <= 227u * 1024u, "shared memory budget");
  // Tensor memory columns.
  static constexpr uint32_t kColS = 0, kColDP = 128, kColAcc0 = 256, kColAcc1 = 256 + D;
  static constexpr uint32_t kColA0 = 256 + D, kColA1 = 256 + D + D / 2;  // query walk
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kColAcc1 + D <= kTmemCols && kColA1 + D / 2 <= kTmemCols, "tensor memory budget");
};

constexpr int kBwdIdxSlots = 4;

struct BCtl {
  uint64_t b0_full[4], b0_empty[4], b1_full[4], b1_empty[4];
  uint64_t stat_full[2], stat_empty[2];  // key walk: the query tile's row statistics
  uint64_t fix;                          // a tile whose tail the load warp clears
  uint64_t a0_full, a0_empty, a1_full, a1_empty;
  uint64_t s_full, s_free;   // S in tensor memory / read into registers (query walk)
  uint64_t p_full[2];        // half of P's columns in tensor memory (key walk)
  uint64_t dp_full, ds_full;
  uint64_t acc_full[2], acc_free[2];
  uint64_t sum_full[2], sum_empty[2];    // bias gradient: sums by diagonal of one tile
  uint64_t far_full, far_empty;          // ... and of the tiles past the reach
  uint64_t idx_full[kBwdIdxSlots], idx_empty[kBwdIdxSlots];  // claimed items
  int idx_ring[kBwdIdxSlots];
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
  float far[kMathWarps][2];
};
static_assert(sizeof(BCtl) <= 1024, "barrier area");

// (a, b) <- (a, b) * (x, y), two lanes per instruction.
__device__ __forceinline__ void mul_x2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 r, s;\n\t"
      "mov.b64 r, {%0, %1};\n\t"
      "mov.b64 s, {%2, %3};\n\t"
      "mul.rn.f32x2 r, r, s;\n\t"
      "mov.b64 {%0, %1}, r;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

// 2^x for two values on the FMA pipe: x = n + f with n = floor(x) (adding
// 1.5 * 2^23 rounded down leaves n in the low mantissa bits), a polynomial p of
// degree kDeg for 2^f on [0, 1), p(f) = 1 + f r(f), as 2^n + (2^n f) r(f) with the
// float 2^n whose exponent field is n + 127: exact, 0 for x < -126 (a masked
// pair) and NaN for NaN (n added into p's exponent field instead would carry
// NaN into a finite value; that was 465 us against 473 on the case at kPolyOf8).
// Relative error 3.0e-6 (degree 4) and 1.6e-7 (degree 5); coefficients from
// gen_exp2_poly.py.
template <int kDeg>
__device__ __forceinline__ void ex2_floor_x2(float& a, float& b) {
  static_assert(kDeg == 4 || kDeg == 5, "fitted degrees");
  constexpr float kShift = 12582912.0f;  // 1.5 * 2^23
  constexpr float kC[2][6] = {
      {1.0f, 0.69304484f, 0.2412802f, 0.052242473f, 0.013426684f, 0.0f},
      {1.0f, 0.6931513f, 0.24016444f, 0.055799913f, 0.009017031f, 0.00186713f}};
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(a));  // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(b));
  float ta = a, tb = b;
  asm("{\n\t.reg .b64 r, s;\n\t"
      "mov.b64 r, {%0, %1};\n\t"
      "mov.b64 s, {%2, %2};\n\t"
      "add.rm.f32x2 r, r, s;\n\t"
      "mov.b64 {%0, %1}, r;\n\t}"
      : "+f"(ta), "+f"(tb)
      : "f"(kShift));
  float fa = ta, fb = tb;
  add_x2(fa, fb, -kShift, -kShift);                              // n
  fma_x2(fa, fb, pack_f32x2(-1.f, -1.f), pack_f32x2(a, b));      // f = x - n
  const uint64_t f2 = pack_f32x2(fa, fb);
  float pa = kC[kDeg - 4][kDeg], pb = pa;
#pragma unroll
  for (int i = kDeg - 1; i > 0; --i)
    fma_x2(pa, pb, f2, pack_f32x2(kC[kDeg - 4][i], kC[kDeg - 4][i]));
  // 2^n: the low 9 bits of 1.5 * 2^23 are 0, only n is left of t's bits.
  const float na = __int_as_float((__float_as_int(ta) << 23) + 0x3f800000);
  const float nb = __int_as_float((__float_as_int(tb) << 23) + 0x3f800000);
  static_assert(kC[kDeg - 4][0] == 1.0f, "2^n stands for 2^n kC[0]");
  mul_x2(fa, fb, na, nb);
  fma_x2(pa, pb, pack_f32x2(fa, fb), pack_f32x2(na, nb));
  a = pa;
  b = pb;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Items are claimed at run time, in list order (longest first): CTA c starts
// with item c, every later one is the next that no CTA has taken. The load warp
// claims each once the loads of the one before are under way and passes its
// index on through a ring; it ends with one past the list.
template <typename Ctl>
__device__ __forceinline__ int bwd_claim(Ctl* ctl, unsigned int* counter, int k, const WaitCtx& w) {
  const int slot = k % kBwdIdxSlots;
  if (k >= kBwdIdxSlots &&
      !wait_warp(&ctl->idx_empty[slot], ((k / kBwdIdxSlots) - 1) & 1u, w, kBSiteIdxEmpty))
    return 0x7fffffff;
  int idx = blockIdx.x;
  if ((threadIdx.x & 31) == 0) {
    if (k > 0) idx = (int)(gridDim.x + atomicAdd(counter, 1u));  // below items + 2 gridDim.x
    ctl->idx_ring[slot] = idx;
    mbar_arrive(&ctl->idx_full[slot]);
  }
  return __shfl_sync(0xffffffffu, idx, 0);
}

// The CTA's k-th item (whole warps of the other roles); past any list when the
// wait gave up.
template <typename Ctl>
__device__ __forceinline__ int bwd_take(Ctl* ctl, int k, const WaitCtx& w) {
  const int slot = k % kBwdIdxSlots;
  if (!wait_warp(&ctl->idx_full[slot], (k / kBwdIdxSlots) & 1u, w, kBSiteIdxFull))
    return 0x7fffffff;
  const int idx = *reinterpret_cast<volatile int*>(&ctl->idx_ring[slot]);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl->idx_empty[slot]);
  return idx;
}

// Whether the phase with the given parity is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// The CTA's steps in order: tile t of an item that has tiles. The query walk
// goes up its key tiles, the key walk down its query tiles: distances grow
// along both.
struct Step {
  int k;        // next position of the CTA's list
  int t, lo, hi;
  bool valid, first, last;
};

// Moves to the next step, over items without tiles. With `block` false it does
// not wait for items that are not claimed yet: false, and the step is unchanged
// but for what has been passed over.
template <bool kKeys>
__device__ __forceinline__ bool next_step(const BwdItem* items, int n, BCtl* ctl, const WaitCtx& w,
                                          Step& s, bool block) {
  if (s.valid && !s.last) {
    s.t += kKeys ? -1 : 1;
    s.first = false;
    s.last = kKeys ? s.t == s.lo : s.t + 1 == s.hi;
    return true;
  }
  for (;;) {
    if (!block && !__all_sync(0xffffffffu, mbar_test(&ctl->idx_full[s.k % kBwdIdxSlots],
                                                     (s.k / kBwdIdxSlots) & 1u)))
      return false;
    const int idx = bwd_take(ctl, s.k, w);
    if (idx >= n) {
      s.valid = false;
      return true;
    }
    ++s.k;
    const int4 r = __ldg(reinterpret_cast<const int4*>(items + idx) + 1);  // lo, hi, full range
    if (r.y <= r.x) continue;
    s.lo = r.x;
    s.hi = r.y;
    s.t = kKeys ? s.hi - 1 : s.lo;
    s.valid = s.first = true;
    s.last = s.lo + 1 == s.hi;
    return true;
  }
}

// ----------------------------------------------------------------- roles

// TMA loads (a whole warp; lane 0 issues): per step the tile of B0, the row
// statistics (key walk) and the tile of B1; in the key walk the item's K and
// V follow its first tiles, as soon as the previous item has read its own.
template <int D, bool kKeys, bool kRel>
__device__ void bwd_load(const BwdParams& p, BCtl* ctl, uint8_t* sA, uint8_t* sB0, uint8_t* sB1,
                         uint8_t* sStat, const WaitCtx& w) {
  using C = BCfg<D, kKeys, kRel>;
  const int lane = threadIdx.x & 31;
  const BwdItem* items = kKeys ? p.k_items : p.q_items;
  const int n_items = kKeys ? p.n_k : p.n_q;
  const CUtensorMap* tm0 = kKeys ? &p.tm_q : &p.tm_k;
  const CUtensorMap* tm1 = kKeys ? &p.tm_do : &p.tm_v;
  uint32_t n0 = 0, n1 = 0, ns = 0, na0 = 0, na1 = 0, nfix = 0;
  bool ok = true, fixing = false;
  auto tma_tile = [&](uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int row, int h, int bc) {
    mbar_expect_tx(bar, C::kTileBytes);
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c)
      tma_load_4d(dst + c * C::kChunkBytes, tm, bar, c * 64, row, h, bc);
  };
  // One streamed tile of which `rows` rows belong to the sequence. Rows past
  // a packed sequence's end are another sequence's tokens: they are cleared,
  // so that a zero weight times whatever they hold adds nothing.
  auto load_b = [&](uint8_t* ring, uint64_t* full, uint64_t* empty, uint32_t& n, int slots,
                    const CUtensorMap* tm, int row, int rows, int h, int bc, uint32_t site) -> bool {
    const uint32_t st = n % slots;
    if (n >= (uint32_t)slots && !wait_warp(&empty[st], ((n / slots) - 1) & 1u, w, site))
      return false;
    uint8_t* dst = ring + st * C::kTileBytes;
    const bool clear = p.tnd && rows < 128;
    if (lane == 0) tma_tile(dst, tm, clear ? &ctl->fix : &full[st], row, h, bc);
    __syncwarp();
    if (clear) {
      // The copy is complete before anything is written over its rows.
      fixing = true;
      if (!wait_warp(&ctl->fix, nfix & 1u, w, kBSiteFix)) return false;
      fixing = false;
      ++nfix;
      for (int x = rows * 8 + lane; x < 128 * 8; x += 32)
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          st_shared_v4(smem_u32(dst) + c * C::kChunkBytes + x * 16, 0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
    }
    ++n;
    return true;
  };
  for (int k = 0; ok; ++k) {
    const int idx = bwd_claim(ctl, p.claims + (kKeys ? 1 : 0), k, w);
    if (idx == 0x7fffffff) ok = false;
    if (idx >= n_items) break;
    const BwdItem it = items[idx];
    if (it.hi <= it.lo) continue;
    const SeqRec sr = p.seqs[it.b];
    const int bc = p.tnd ? 0 : it.b;
    const int off = kKeys ? sr.q_off : sr.kv_off, len = kKeys ? sr.sq : sr.skv;
    for (int x = 0; x < it.hi - it.lo && ok; ++x) {
      const int t = kKeys ? it.hi - 1 - x : it.lo + x;
      const int row = off + t * 128, rows = min(128, len - t * 128);
      ok = load_b(sB0, ctl->b0_full, ctl->b0_empty, n0, C::kN0, tm0, row, rows, it.h, bc,
                  kBSiteB0Empty);
      if (kKeys && ok && x == 0) {
        ok = na0 == 0 || wait_warp(&ctl->a0_empty, (na0 - 1) & 1u, w, kBSiteA0Empty);
        if (ok && lane == 0)
          tma_tile(sA, &p.tm_k, &ctl->a0_full, sr.kv_off + it.tile * 128, it.h, bc);
        if (ok) ++na0;
      }
      if (kKeys && ok) {
        const uint32_t st = ns & 1u;
        ok = ns < 2 || wait_warp(&ctl->stat_empty[st], ((ns >> 1) - 1) & 1u, w, kBSiteStatEmpty);
        if (ok && lane == 0) {
          mbar_expect_tx(&ctl->stat_full[st], 1024u);
          bulk_load(sStat + st * 1024u, p.stats + ((int64_t)it.stat + t) * 256, 1024u,
                    &ctl->stat_full[st]);
        }
        if (ok) ++ns;
      }
      if (ok)
        ok = load_b(sB1, ctl->b1_full, ctl->b1_empty, n1, C::kN1, tm1, row, rows, it.h, bc,
                    kBSiteB1Empty);
      if (kKeys && ok && x == 0) {
        ok = na1 == 0 || wait_warp(&ctl->a1_empty, (na1 - 1) & 1u, w, kBSiteA1Empty);
        if (ok && lane == 0)
          tma_tile(sA + C::kTileBytes, &p.tm_v, &ctl->a1_full, sr.kv_off + it.tile * 128, it.h, bc);
        if (ok) ++na1;
      }
    }
  }
  if (!ok && lane == 0) {
    // Abort: let every copy this warp started land before the CTA exits.
    if (fixing) wait_bounded(&ctl->fix, nfix & 1u, w, kBSiteDrain, false);
    for (uint32_t r = n0 > (uint32_t)C::kN0 ? n0 - C::kN0 : 0u; r < n0; ++r)
      wait_bounded(&ctl->b0_full[r % C::kN0], (r / C::kN0) & 1u, w, kBSiteDrain, false);
    for (uint32_t r = n1 > (uint32_t)C::kN1 ? n1 - C::kN1 : 0u; r < n1; ++r)
      wait_bounded(&ctl->b1_full[r % C::kN1], (r / C::kN1) & 1u, w, kBSiteDrain, false);
    for (uint32_t r = ns > 2u ? ns - 2u : 0u; r < ns; ++r)
      wait_bounded(&ctl->stat_full[r & 1u], (r >> 1) & 1u, w, kBSiteDrain, false);
    if (na0) wait_bounded(&ctl->a0_full, (na0 - 1) & 1u, w, kBSiteDrain, false);
    if (na1) wait_bounded(&ctl->a1_full, (na1 - 1) & 1u, w, kBSiteDrain, false);
  }
  __syncwarp();
}

// Descriptor of an MN-major operand without swizzle: 8 x 16-byte core matrices,
// groups of 8 K rows lbo apart, blocks of 8 MN elements sbo apart.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return sdesc(addr, lbo, sbo) & ~(7ull << 61);
}

// D[128 x 128] = A B^T, both K-major over the head dim; A in shared memory
// (key walk) or tensor memory.
template <int D, bool kKeys, bool kRel>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t a_tmem, uint64_t a0, uint64_t b0) {
  using C = BCfg<D, kKeys, kRel>;
  constexpr uint32_t idesc = idesc_bf16(128, 128, false);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint64_t off = (uint64_t)(((k >> 2) * C::kChunkBytes + (k & 3) * 32u) >> 4);
    if constexpr (kKeys) mma_ss(d, a0 + off, b0 + off, idesc, k > 0 ? 1u : 0u);
    else mma_ts(d, a_tmem + k * 8u, b0 + off, idesc, k > 0 ? 1u : 0u);
  }
}

// acc[128 x D] += W B over half of W's columns, W (P or dS, bf16) in tensor
// memory: columns kCols * g and on from tensor memory column a + kCols * g.
// Half 0 takes the first half of every group's columns (what each math warp
// stores first), half 1 the others.
template <int D>
__device__ __forceinline__ void issue_acc(uint32_t d, uint32_t a, uint64_t b0, uint32_t accumulate,
                                          int half) {
  constexpr uint32_t idesc = idesc_bf16(128, D, true);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    constexpr int kRun = kCols / 32;  // 16-column steps of a group's half
    const int k = (q / kRun) * (2 * kRun) + half * kRun + q % kRun;  // 16 columns of W, 16 rows of B
    mma_ts(d, a + (16 * k / kCols) * kCols + (16 * k % kCols) / 2, b0 + (uint64_t)(k * (2048u >> 4)), idesc,
           q > 0 ? 1u : accumulate);
  }
}

// All products (a whole warp, so that addresses and descriptors stay in
// uniform registers; one lane issues). The products that overwrite tensor
// memory which an earlier product still reads are issued after it by this
// same thread: products execute in order.
template <int D, bool kKeys, bool kRel>
__device__ void bwd_mma(const BwdParams& p, BCtl* ctl, uint32_t tmem, const uint8_t* sA,
                        const uint8_t* sB0, const uint8_t* sB1, const WaitCtx& w) {
  using C = BCfg<D, kKeys, kRel>;
  const BwdItem* items = kKeys ? p.k_items : p.q_items;
  const int n_items = kKeys ? p.n_k : p.n_q;
  const uint32_t tS = tmem + C::kColS, tDP = tmem + C::kColDP;
  // Descriptors of slot 0: K-major (scores) and MN-major (accumulation).
  const uint64_t dA0 = sdesc(smem_u32(sA), 16u, 1024u);
  const uint64_t dA1 = sdesc(smem_u32(sA) + C::kTileBytes, 16u, 1024u);
  const uint64_t dB0 = sdesc(smem_u32(sB0), 16u, 1024u);
  const uint64_t dB1 = sdesc(smem_u32(sB1), 16u, 1024u);
  const uint64_t dM0 = sdesc(smem_u32(sB0), C::kChunkBytes, 1024u);
  const uint64_t dM1 = sdesc(smem_u32(sB1), C::kChunkBytes, 1024u);
  constexpr uint64_t kSlot = C::kTileBytes >> 4;
  Step cur, nx;
  nx.k = 0;
  nx.valid = false;
  next_step<kKeys>(items, n_items, ctl, w, nx, true);
  uint32_t n = 0;       // step of nx
  uint32_t a0 = 0, a1 = 0;  // held operands awaited
  uint32_t items_done = 0;
  // The operands of the products of step nx are waited for ahead of the
  // products that they follow, so that those waits (about 100 cycles each
  // even when the data is there) do not fall between two products.
  auto operands0 = [&]() -> bool {
    if (nx.first && !wait_warp(&ctl->a0_full, a0++ & 1u, w, kBSiteA0Full)) return false;
    return wait_warp(&ctl->b0_full[n % C::kN0], (n / C::kN0) & 1u, w, kBSiteB0Full);
  };
  auto operands1 = [&]() -> bool {
    if (nx.first && !wait_warp(&ctl->a1_full, a1++ & 1u, w, kBSiteA1Full)) return false;
    return wait_warp(&ctl->b1_full[n % C::kN1], (n / C::kN1) & 1u, w, kBSiteB1Full);
  };
  auto scores = [&]() {
    if (elect_one()) {
      issue_scores<D, kKeys, kRel>(tS, tmem + C::kColA0, dA0, dB0 + (n % C::kN0) * kSlot);
      mma_commit(&ctl->s_full);
      if (nx.last) mma_commit(&ctl->a0_empty);
    }
    __syncwarp();
  };
  auto dprobs = [&]() {
    if (elect_one()) {
      issue_scores<D, kKeys, kRel>(tDP, tmem + C::kColA1, dA1, dB1 + (n % C::kN1) * kSlot);
      mma_commit(&ctl->dp_full);
      if (!kKeys) mma_commit(&ctl->b1_empty[n % C::kN1]);
      if (nx.last) mma_commit(&ctl->a1_empty);
    }
    __syncwarp();
  };
  bool ok = !nx.valid || (operands0() && operands1());
  if (ok && nx.valid) {
    tc_fence_after();
    scores();
    dprobs();
  }
  while (ok && nx.valid) {
    cur = nx;
    const uint32_t c = n;
    // The item behind this one may not be claimed yet (items without tiles in
    // between need every role to pass them, the epilogue among them, which
    // waits for this item's products): then its products come after this one's.
    const bool late = !next_step<kKeys>(items, n_items, ctl, w, nx, false);
    ++n;
    if (!late && nx.valid && !operands0()) break;
    if constexpr (kKeys) {
      // dV in two halves of the queries: the first while the other half's P
      // is computed.
      if (cur.first && items_done > 0 &&
          !wait_warp(&ctl->acc_free[1], (items_done - 1) & 1u, w, kBSiteAccFree))
        break;
      const uint32_t st = c % C::kN1;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!wait_warp(&ctl->p_full[half], c & 1u, w, kBSitePFull)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          issue_acc<D>(tmem + C::kColAcc1, tS, dM1 + st * kSlot,
                       (cur.first && half == 0) ? 0u : 1u, half);
          if (half) {
            mma_commit(&ctl->b1_empty[st]);
            if (cur.last) mma_commit(&ctl->acc_full[1]);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      if (!late && nx.valid) scores();
    } else if (!late && nx.valid) {
      if (!wait_warp(&ctl->s_free, c & 1u, w, kBSiteSFree)) break;
      tc_fence_after();
      scores();
    }
    if (!late && nx.valid && !operands1()) break;
    if (cur.first && items_done > 0 &&
        !wait_warp(&ctl->acc_free[0], (items_done - 1) & 1u, w, kBSiteAccFree))
      break;
    if (!wait_warp(&ctl->ds_full, c & 1u, w, kBSiteDsFull)) break;
    tc_fence_after();
    const uint32_t st = c % C::kN0;
    if (elect_one()) {
      issue_acc<D>(tmem + C::kColAcc0, tDP, dM0 + st * kSlot, cur.first ? 0u : 1u, 0);
      issue_acc<D>(tmem + C::kColAcc0, tDP, dM0 + st * kSlot, 1u, 1);
      mma_commit(&ctl->b0_empty[st]);
      if (cur.last) mma_commit(&ctl->acc_full[0]);
    }
    __syncwarp();
    if (cur.last) ++items_done;
    if (late) {
      next_step<kKeys>(items, n_items, ctl, w, nx, true);
      if (!nx.valid) break;
      if (!operands0() || !operands1()) break;
      if (!kKeys && !wait_warp(&ctl->s_free, c & 1u, w, kBSiteSFree)) break;
      tc_fence_after();
      scores();
    }
    if (nx.valid) dprobs();
  }
  // Wait until every product issued here (and its commits) has finished with
  // tensor and shared memory.
  if (elect_one()) mma_commit(&ctl->drain);
  __syncwarp();
  wait_bounded(&ctl->drain, 0u, w, kBSiteDrain, false);
}

__device__ __forceinline__ void tmem_ld_wait(uint32_t a, uint32_t (&r)[32]) { tmem_ld32_wait(a, r); }
__device__ __forceinline__ void tmem_ld_wait(uint32_t a, uint32_t (&r)[64]) { tmem_ld64_wait(a, r); }
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[8]) { tmem_st8(a, r); }
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[16]) { tmem_st16(a, r); }
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[32]) { tmem_st32(a, r); }

// One bit per column of [0, kCols): inside [lo, hi].
__device__ __forceinline__ void interval_bits(int lo, int hi, uint32_t (&wm)[kCols / 32]) {
#pragma unroll
  for (int wd = 0; wd < kCols / 32; ++wd) {
    const int a = lo - 32 * wd, b = hi - 32 * wd;
    const uint32_t upto = b >= 31 ? 0xffffffffu : (b < 0 ? 0u : (0xffffffffu >> (31 - b)));
    const uint32_t from = a <= 0 ? 0xffffffffu : (a > 31 ? 0u : (0xffffffffu << a));
    wm[wd] = upto & from;
  }
}

// P and dS of one group's columns of every tile, one row per thread. Per
// step: S to registers, P = 2^(scale log2e S + bias - lse log2e) (masked
// entries 0), in the key walk P back in bf16 over S; then dP to registers,
// dS = P (dP - delta) back in bf16 over dP. P is rounded to bf16 only as an
// operand of dV; dS uses the fp32 value. With p.ds the key walk also writes
// dS in bf16 to global memory, for the dQ kernel.
template <int D, bool kKeys, int kBias>
__device__ void bwd_math(const BwdParams& p, BCtl* ctl, uint32_t tmem, const uint8_t* sStat,
                         float* sSum, const WaitCtx& w) {
  constexpr bool kRel = kBias == kBwdBiasRel;
  using C = BCfg<D, kKeys, kRel>;
  constexpr bool kGrad = C::kSums;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wq = warp & 3, g = warp >> 2;
  const int row = wq * 32 + lane;
  const uint32_t lane_bits = (uint32_t)(wq * 32) << 16;
  const uint32_t tS = tmem + lane_bits + C::kColS + kCols * g;
  const uint32_t tDP = tmem + lane_bits + C::kColDP + kCols * g;
  const BwdItem* items = kKeys ? p.k_items : p.q_items;
  const int n_items = kKeys ? p.n_k : p.n_q;
  const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2);
  uint32_t n = 0;      // steps
  uint32_t n_near = 0, n_far = 0;
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const int idx = bwd_take(ctl, k, w);
    if (idx >= n_items) break;
    const BwdItem it = items[idx];
    if (it.hi <= it.lo) continue;
    const SeqRec sr = p.seqs[it.b];
    const int delta = sr.skv - sr.sq;
    const int at = it.tile * 128 + row;  // this thread's query row or key
    const bool stored = at < (kKeys ? sr.skv : sr.sq);
    // Visible columns of this row: keys of a query row, or query rows of a key.
    int v_lo = 1, v_hi = 0;
    if (stored) {
      if constexpr (kKeys) {
        v_lo = at < sr.prefix ? 0 : (int)imin64(imax64(0, (int64_t)at - sr.hi_off), sr.sq);
        v_hi = (int)imax64(imin64(sr.sq - 1, (int64_t)at - sr.lo_off), -1);
      } else {
        v_lo = (int)imin64(imax64(0, row_lo(sr, at)), sr.skv);
        v_hi = (int)imax64(imin64(sr.skv - 1, row_hi(sr, at)), -1);
      }
    }
    // This row's words of the mask, one per 32 columns, m_step apart.
    const uint32_t* mrow = nullptr;
    int64_t m_step = 0;
    if (sr.flags & kSeqDenseMask) {
      m_step = kKeys ? p.m_keys : p.m_rows;
      const int64_t plane = it.b * p.m_sb + it.h * p.m_sh;
      mrow = (kKeys ? p.bits_k : p.bits_q) +
             plane * ((kKeys ? p.m_rows : p.m_keys) / 32) * m_step + at;
    }
    float nl = 0.f, nd = 0.f;
    if constexpr (!kKeys) {
      nl = __ldg(p.stats + (int64_t)it.stat * 256 + row);
      nd = __ldg(p.stats + (int64_t)it.stat * 256 + 128 + row);
    }
    float a2 = 0.f;
    if constexpr (kBias == kBwdBiasAlibi) a2 = __ldg(p.slopes + it.h) * kLog2e;
    const float* ext = nullptr;
    if constexpr (kRel) ext = p.rel.ext + (int64_t)it.h * 4 * p.rel.row;
    float far_lo = 0.f, far_hi = 0.f;

    // Spilled dS: this thread's first 8 columns in the item's tile t = 0.
    __nv_bfloat16* ds_out = nullptr;
    bool ragged = false;
    if (kKeys && kWritesDs<D> && p.ds) {
      ds_out = p.ds + (int64_t)p.spans[it.span].first * (128 * 128) + g * (kCols * 128) + row * 8;
      ragged = (it.tile + 1) * 128 > sr.skv;
    }
    for (int s = 0; s < it.hi - it.lo; ++s, ++n) {
      const int t = kKeys ? it.hi - 1 - s : it.lo + s;
      const bool partial = !(t >= it.full_lo && t < it.full_hi);
      const int c0 = t * 128 + kCols * g;  // this group's first column
      // Distance key - diagonal of the row's column 0; it grows with the
      // column in the query walk and falls with it in the key walk.
      const int rel0 = kKeys ? at - (c0 + delta) : c0 - (at + delta);
      uint32_t wm[kCols / 32];
#pragma unroll
      for (int wd = 0; wd < kCols / 32; ++wd) wm[wd] = 0xffffffffu;
      if (partial) {
        interval_bits(v_lo - c0, v_hi - c0, wm);
        if (mrow != nullptr) {
#pragma unroll
          for (int wd = 0; wd < kCols / 32; ++wd)
            wm[wd] &= ~__ldg(mrow + (c0 / 32 + wd) * m_step);
        }
      }
      const float* st = reinterpret_cast<const float*>(sStat + (n & 1u) * 1024u) + kCols * g;
      if (kKeys && !wait_warp(&ctl->stat_full[n & 1u], (n >> 1) & 1u, w, kBSiteStatFull)) {
        ok = false;
        break;
      }
      if (!wait_warp(&ctl->s_full, n & 1u, w, kBSiteSFull)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float x[kCols];
      {
        uint32_t sv[kCols];
        tmem_ld_wait(tS, sv);
#pragma unroll
        for (int c = 0; c < kCols; ++c) x[c] = __uint_as_float(sv[c]);
      }
      if constexpr (!kKeys) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->s_free);
      }
      // Exponent: scale log2e S + bias - lse log2e.
      // Learned bias: past the reach on one side in the whole tile (one
      // scalar), or a bias per distance.
      float base = 0.f;
      bool near = false;
      if constexpr (kRel) {
        const int top = kKeys ? it.tile * 128 + 127 - (t * 128 + delta)
                              : t * 128 + 127 - (it.tile * 128 + delta);
        near = !(top <= -p.rel.reach || top - 254 >= p.rel.reach);
        if (!near) base = __ldg(top <= -p.rel.reach ? ext : ext + p.rel.row - 1);
      }
      if constexpr (kBias == kBwdBiasAlibi) {
        const float d0 = (float)rel0;
        constexpr float kSign = kKeys ? -1.f : 1.f;
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          float da = d0, db = d0;
          add_x2(da, db, kSign * c, kSign * (c + 1));
          if (p.alibi == FA_ALIBI_SQRT) {
            float ra, rb;
            asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(ra) : "f"(fabsf(da)));
            asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(rb) : "f"(fabsf(db)));
            da = copysignf(ra, da);
            db = copysignf(rb, db);
          }
          const float la = kKeys ? st[c] : nl, lb = kKeys ? st[c + 1] : nl;
          fma_x2(da, db, pack_f32x2(a2, a2), pack_f32x2(la, lb));
          fma_x2(x[c], x[c + 1], scale2, pack_f32x2(da, db));
        }
      } else if (kRel && near) {
        // ext entry of column 0, and the copy in which four consecutive
        // distances of these columns are one aligned 16-byte load.
        const int e0 = rel0 + p.rel.reach + kRelPad;
        const int first = kKeys ? e0 - 3 : e0;
        const float4* src =
            reinterpret_cast<const float4*>(ext + (int64_t)(first & 3) * p.rel.row + (first & ~3));
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          float4 e = __ldg(kKeys ? src - c / 4 : src + c / 4);
          if (kKeys) e = make_float4(e.w, e.z, e.y, e.x);
          if constexpr (kKeys) {
            const float4 l = *reinterpret_cast<const float4*>(st + c);
            add_x2(e.x, e.y, l.x, l.y);
            add_x2(e.z, e.w, l.z, l.w);
          } else {
            add_x2(e.x, e.y, nl, nl);
            add_x2(e.z, e.w, nl, nl);
          }
          fma_x2(x[c], x[c + 1], scale2, pack_f32x2(e.x, e.y));
          fma_x2(x[c + 2], x[c + 3], scale2, pack_f32x2(e.z, e.w));
        }
      } else {
        const uint64_t l2 = pack_f32x2(nl + base, nl + base);
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          if constexpr (kKeys) {
            float4 l = *reinterpret_cast<const float4*>(st + c);
            if constexpr (kRel) {
              add_x2(l.x, l.y, base, base);
              add_x2(l.z, l.w, base, base);
            }
            fma_x2(x[c], x[c + 1], scale2, pack_f32x2(l.x, l.y));
            fma_x2(x[c + 2], x[c + 3], scale2, pack_f32x2(l.z, l.w));
          } else {
            fma_x2(x[c], x[c + 1], scale2, l2);
            fma_x2(x[c + 2], x[c + 3], scale2, l2);
          }
        }
      }
      if (partial) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          x[c] = ((wm[c >> 5] >> (c & 31)) & 1u) ? x[c] : -INFINITY;
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int c = kCols / 2 * half; c < kCols / 2 * (half + 1); c += 2) {
          if (((c >> 1) * kPolyOf8<D>) % 8 < kPolyOf8<D>) {
            ex2_floor_x2<kGrad ? 5 : 4>(x[c], x[c + 1]);
          } else {
            x[c] = ex2(x[c]);
            x[c + 1] = ex2(x[c + 1]);
          }
        }
        if constexpr (kKeys) {
          uint32_t pk[kCols / 4];
#pragma unroll
          for (int c = 0; c < kCols / 4; ++c)
            pk[c] = pack_bf16(x[kCols / 2 * half + 2 * c], x[kCols / 2 * half + 2 * c + 1]);
          tmem_st(tS + kCols / 4 * half, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->p_full[half]);
        }
      }
      if (!wait_warp(&ctl->dp_full, n & 1u, w, kBSiteDpFull)) {
        ok = false;
        break;
      }
      tc_fence_after();
      {
        uint32_t dv[kCols];
        tmem_ld_wait(tDP, dv);
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          float y[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = __uint_as_float(dv[c + q]);
          if constexpr (kKeys) {
            const float4 l = *reinterpret_cast<const float4*>(st + 128 + c);
            add_x2(y[0], y[1], l.x, l.y);
            add_x2(y[2], y[3], l.z, l.w);
          } else {
            add_x2(y[0], y[1], nd, nd);
            add_x2(y[2], y[3], nd, nd);
          }
          mul_x2(x[c], x[c + 1], y[0], y[1]);
          mul_x2(x[c + 2], x[c + 3], y[2], y[3]);
        }
      }
      {
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) pk[c] = pack_bf16(x[2 * c], x[2 * c + 1]);
        tmem_st(tDP, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl->ds_full);
          if (kKeys) mbar_arrive(&ctl->stat_empty[n & 1u]);
        }
        if (kKeys && kWritesDs<D> && ds_out) {
          // Rows past the sequence's end go out as zeros, dQ sums over them.
          if (ragged && !stored) {
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) pk[c] = 0u;
          }
          // 8 columns of a warp's rows are 512 contiguous bytes. (Rows of the
          // whole tile are 32 lines a store, which keep shared memory from the
          // products: key walk 252 us against 234 on a causal 2 x 16 x 4096 x 128.
          // The stores still take 900 of a step's 3,800 cycles; written by the
          // epilogue from tensor memory instead, the call was 3 % slower.)
          __nv_bfloat16* dst = ds_out + (int64_t)t * (128 * 128);
#pragma unroll
          for (int u = 0; u < kCols / 8; ++u)
            st_global_na_v4(dst + u * (8 * 128),
                            make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]));
        }
      }
      if constexpr (kGrad) {
        // (Rows past the sequence's end do not count, whatever they hold.)
        if (near) {
          // Sums by diagonal of this warp's 32 rows x kCols columns: the running
          // sum of a diagonal moves to the next lane with each column, and
          // leaves at lane 31 (entry c) or after the last column.
          const uint32_t buf = n_near & 1u;
          if (n_near >= 2 && !wait_warp(&ctl->sum_empty[buf], ((n_near >> 1) - 1) & 1u, w,
                                        kBSiteSumEmpty)) {
            ok = false;
            break;
          }
          float* out = sSum + (buf * kMathWarps + warp) * kSumRow;
          float s = 0.f;
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const float up = __shfl_up_sync(0xffffffffu, s, 1);
            s = (lane == 0 ? 0.f : up) + (stored ? x[c] : 0.f);
            if (lane == 31) out[c] = s;
          }
          if (lane < 31) out[kCols + 30 - lane] = s;
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->sum_full[buf]);
          ++n_near;
        } else {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            add_x2(acc[0], acc[1], x[c], x[c + 1]);
            add_x2(acc[2], acc[3], x[c + 2], x[c + 3]);
          }
          const float s = (acc[0] + acc[1]) + (acc[2] + acc[3]);
          if (stored) {
            if (rel0 < 0) far_lo += s;
            else far_hi += s;
          }
        }
      }
    }
    if constexpr (kGrad) {
      if (!ok) break;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        far_lo += __shfl_xor_sync(0xffffffffu, far_lo, d);
        far_hi += __shfl_xor_sync(0xffffffffu, far_hi, d);
      }
      if (n_far > 0 && !wait_warp(&ctl->far_empty, (n_far - 1) & 1u, w, kBSiteFarEmpty)) break;
      ++n_far;
      if (lane == 0) {
        ctl->far[warp][0] = far_lo;
        ctl->far[warp][1] = far_hi;
        mbar_arrive(&ctl->far_full);
      }
    }
  }
}

// Bias gradient (one warp, key walk): the item's sums by distance, entry e for
// the distance e - reach - kRelPad, each written once. Diagonal y of a tile
// (y = column - row + 127) gathers entry y - 96 - kCols g + 32 wq of each math
// warp (g, wq). In the order of growing distance, d = 254 - y, the sums
// d >= 128 of a step are d - 128 of the next one (the query tile before) and
// wait for it in registers. Entry 0 and the last take the tiles past the
// reach, which near tiles cannot touch.
__device__ void bwd_sums(const BwdParams& p, BCtl* ctl, const float* sSum, const WaitCtx& w) {
  const int lane = threadIdx.x & 31;
  const int width = rel_width(p.rel.reach);
  uint32_t n_near = 0, n_far = 0;
  for (int k = 0;; ++k) {
    const int idx = bwd_take(ctl, k, w);
    if (idx >= p.n_k) return;
    const BwdItem it = p.k_items[idx];
    float* out = p.rel_part + (int64_t)it.span * width;
    for (int e = lane; e < width; e += 32) out[e] = 0.f;
    __syncwarp();
    if (it.hi <= it.lo) continue;
    const SeqRec sr = p.seqs[it.b];
    const int diag0 = p.rel.reach + kRelPad - 127 - (sr.skv - sr.sq);
    float carry[4] = {0.f, 0.f, 0.f, 0.f};
    int pending = -1;  // entry of carry[0] of lane 0
    for (int t = it.hi - 1; t >= it.lo; --t) {
      const int off = it.tile - t;
      const int top = off * 128 + 127 - (sr.skv - sr.sq);
      if (top <= -p.rel.reach || top - 254 >= p.rel.reach) continue;
      const uint32_t buf = n_near & 1u;
      if (!wait_warp(&ctl->sum_full[buf], (n_near >> 1) & 1u, w, kBSiteSumFull)) return;
      const float* in = sSum + buf * kMathWarps * kSumRow;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int d = q * 32 + lane;
        float lo = carry[q], hi = 0.f;
#pragma unroll
        for (int m = 0; m < kMathWarps; ++m) {
          const int base = 96 + kCols * (m >> 2) - 32 * (m & 3);
          const int x = 254 - d - base, y = 126 - d - base;
          if (x >= 0 && x < kCols + 31) lo += in[m * kSumRow + x];
          if (y >= 0 && y < kCols + 31) hi += in[m * kSumRow + y];
        }
        out[diag0 + off * 128 + d] = lo;
        carry[q] = hi;
      }
      pending = diag0 + (off + 1) * 128;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->sum_empty[buf]);
      ++n_near;
    }
    if (pending >= 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) out[pending + q * 32 + lane] = carry[q];
    }
    if (!wait_warp(&ctl->far_full, n_far & 1u, w, kBSiteFarFull)) return;
    ++n_far;
    __syncwarp();
    if (lane < 2) {
      float s = 0.f;
#pragma unroll
      for (int m = 0; m < kMathWarps; ++m) s += ctl->far[m][lane];
      out[lane ? width - 1 : 0] = s;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->far_empty);
  }
}

// Epilogue (one warpgroup, one row per thread): accumulators, times a factor,
// to bf16 rows in global memory (zeros for items without a tile). In the
// query walk it also brings Q and dO of the next item into tensor memory, a
// row per thread, once the last product of the current item that reads them
// is done.
template <int D, bool kKeys, bool kRel>
__device__ void bwd_epilogue(const BwdParams& p, BCtl* ctl, uint32_t tmem, const WaitCtx& w) {
  using C = BCfg<D, kKeys, kRel>;
  const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int row = wq * 32 + lane;
  const uint32_t lane_bits = (uint32_t)(wq * 32) << 16;
  const BwdItem* items = kKeys ? p.k_items : p.q_items;
  const int n_items = kKeys ? p.n_k : p.n_q;
  const int64_t sb = kKeys ? p.k_sb : p.q_sb, sh = kKeys ? p.k_sh : p.q_sh,
                st = kKeys ? p.k_st : p.q_st;
  uint32_t held = 0;  // items with tiles whose Q and dO are in tensor memory
  uint32_t done = 0;  // items with tiles written out
  auto fetch = [&](const BwdItem& it) -> bool {
    const SeqRec sr = p.seqs[it.b];
    const int i = it.tile * 128 + row;
    const bool stored = i < sr.sq;
    const int64_t off = it.b * sb + it.h * sh + ((int64_t)sr.q_off + (stored ? i : 0)) * st;
#pragma unroll 1
    for (int a = 0; a < 2; ++a) {
      const uint4* src = reinterpret_cast<const uint4*>(
          reinterpret_cast<const __nv_bfloat16*>(a ? p.d_o : p.q) + off);
      uint32_t v[D / 2];
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        const uint4 u = stored ? __ldg(src + x) : make_uint4(0u, 0u, 0u, 0u);
        v[4 * x] = u.x;
        v[4 * x + 1] = u.y;
        v[4 * x + 2] = u.z;
        v[4 * x + 3] = u.w;
      }
      if (held > 0 && !wait_warp(a ? &ctl->a1_empty : &ctl->a0_empty, (held - 1) & 1u, w,
                                 a ? kBSiteA1Empty : kBSiteA0Empty))
        return false;
      tc_fence_after();
      const uint32_t dst = tmem + lane_bits + (a ? C::kColA1 : C::kColA0);
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
        tmem_st32(dst + 32u * x, *reinterpret_cast<const uint32_t(*)[32]>(&v[32 * x]));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a ? &ctl->a1_full : &ctl->a0_full);
    }
    ++held;
    return true;
  };
  auto store_acc = [&](const BwdItem& it, const SeqRec& sr, int which, void* dst, float mul) -> bool {
    const int at = it.tile * 128 + row;
    const bool stored = at < (kKeys ? sr.skv : sr.sq);
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(dst) + it.b * sb + it.h * sh +
                       ((int64_t)(kKeys ? sr.kv_off : sr.q_off) + at) * st;
    const bool v8 = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
    if (!wait_warp(&ctl->acc_full[which], done & 1u, w, kBSiteAccFull)) return false;
    tc_fence_after();
    const uint32_t src = tmem + lane_bits + (which ? C::kColAcc1 : C::kColAcc0);
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t ov[32];
      tmem_ld32_wait(src + ch * 32u, ov);
      uint4 pk[4];
      uint32_t* pw = reinterpret_cast<uint32_t*>(pk);
#pragma unroll
      for (int c = 0; c < 16; ++c)
        pw[c] = pack_bf16(__uint_as_float(ov[2 * c]) * mul, __uint_as_float(ov[2 * c + 1]) * mul);
      if (stored) {
        uint4* q = reinterpret_cast<uint4*>(o + ch * 32);
        if (v8) {
          st_global_na_v8(q, pk[0], pk[1]);
          st_global_na_v8(q + 2, pk[2], pk[3]);
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) st_global_na_v4(q + v, pk[v]);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->acc_free[which]);
    return true;
  };
  // Zeros for an item without a tile, whole rows per group of lanes.
  auto zero = [&](const BwdItem& it, void* dst) {
    constexpr int kLanes = D / 8;
    const SeqRec sr = p.seqs[it.b];
    const int rows = min(128, (kKeys ? sr.skv : sr.sq) - it.tile * 128);
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(dst) + it.b * sb + it.h * sh +
                       ((int64_t)(kKeys ? sr.kv_off : sr.q_off) + it.tile * 128) * st;
#pragma unroll 4
    for (int r = wq * 32 + lane / kLanes; r < min(rows, wq * 32 + 32); r += 32 / kLanes)
      st_global_na_v4(reinterpret_cast<uint4*>(o + (int64_t)r * st) + lane % kLanes,
                      make_uint4(0u, 0u, 0u, 0u));
  };
  // The next item with tiles (those without are dealt with on the way), its
  // operands brought in; past the list at its end, -1 when a wait gave up.
  int k = 0;
  auto next_item = [&]() -> int {
    for (;; ++k) {
      const int idx = bwd_take(ctl, k, w);
      if (idx >= n_items) return idx;
      const BwdItem it = items[idx];
      if (it.hi > it.lo) {
        ++k;
        if (!kKeys && !fetch(it)) return -1;
        return idx;
      }
      zero(it, kKeys ? p.dk : p.dq);
      if (kKeys) zero(it, p.dv);
    }
  };
  for (int cur = next_item(); cur >= 0 && cur < n_items; ++done) {
    const BwdItem it = items[cur];
    const SeqRec sr = p.seqs[it.b];
    if constexpr (kKeys) {
      if (!store_acc(it, sr, 1, p.dv, 1.f)) return;
      if (!store_acc(it, sr, 0, p.dk, p.scale)) return;
      cur = next_item();
    } else {
      const int next = next_item();
      if (next < 0 || !store_acc(it, sr, 0, p.dq, p.scale)) return;
      cur = next;
    }
  }
}

template <int D, bool kKeys, int kBias>
__global__ void __launch_bounds__(kBwdThreads, 1) fa_bwd_sm100(const __grid_constant__ BwdParams p) {
  constexpr bool kRel = kBias == kBwdBiasRel;
  using C = BCfg<D, kKeys, kRel>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sA = smem;
  uint8_t* sB0 = sA + C::kABytes;
  uint8_t* sB1 = sB0 + C::kN0 * C::kTileBytes;
  uint8_t* sStat = sB1 + C::kN1 * C::kTileBytes;
  float* sSum = reinterpret_cast<float*>(sStat + C::kStatBytes);
  auto* ctl = reinterpret_cast<BCtl*>(sStat + C::kStatBytes + C::kSumBytes);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(p.err_word, kErrTimeout | (kBSiteSmem << kErrWhereShift));
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(&ctl->b0_full[s], 1);
      mbar_init(&ctl->b0_empty[s], 1);
      mbar_init(&ctl->b1_full[s], 1);
      mbar_init(&ctl->b1_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->stat_full[s], 1);
      mbar_init(&ctl->stat_empty[s], kMathWarps);
      mbar_init(&ctl->p_full[s], kMathWarps);
      mbar_init(&ctl->acc_full[s], 1);
      mbar_init(&ctl->acc_free[s], 4);
      mbar_init(&ctl->sum_full[s], kMathWarps);
      mbar_init(&ctl->sum_empty[s], 1);
    }
    for (int s = 0; s < kBwdIdxSlots; ++s) {
      mbar_init(&ctl->idx_full[s], 1);
      // math, epilogue and MMA warps, the bias sums
      mbar_init(&ctl->idx_empty[s], kMathWarps + 4 + 1 + (C::kSums ? 1 : 0));
    }
    mbar_init(&ctl->fix, 1);
    mbar_init(&ctl->a0_full, kKeys ? 1 : 4);
    mbar_init(&ctl->a1_full, kKeys ? 1 : 4);
    mbar_init(&ctl->a0_empty, 1);
    mbar_init(&ctl->a1_empty, 1);
    mbar_init(&ctl->s_full, 1);
    mbar_init(&ctl->s_free, kMathWarps);
    mbar_init(&ctl->dp_full, 1);
    mbar_init(&ctl->ds_full, kMathWarps);
    mbar_init(&ctl->far_full, kMathWarps);
    mbar_init(&ctl->far_empty, 1);
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
            smem_u32(&ctl->tmem_base)),
        "r"(C::kTmemCols)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  // What is above ran beside the launch ahead of this one; what is below reads
  // its results, but for the key walk behind a query walk: the two need nothing
  // of each other, and each SM that is free may start on it.
  const bool writes_ds = kWritesDs<D> && p.ds != nullptr;
  if (!kKeys || writes_ds) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const WaitCtx w{&ctl->abort_flag, p.err_word, p.timeout_ns};
  if (warp < kMathWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kBwdRegsMath));
    bwd_math<D, kKeys, kBias>(p, ctl, tmem, sStat, sSum, w);
  } else if (warp < kWarpMma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBwdRegsEpi));
    bwd_epilogue<D, kKeys, kRel>(p, ctl, tmem, w);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBwdRegsControl));
    if (warp == kWarpMma) bwd_mma<D, kKeys, kRel>(p, ctl, tmem, sA, sB0, sB1, w);
    if (warp == kWarpLoad) bwd_load<D, kKeys, kRel>(p, ctl, sA, sB0, sB1, sStat, w);
    if constexpr (C::kSums)
      if (warp == kWarpSums) bwd_sums(p, ctl, sSum, w);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::kTmemCols)
                 : "memory");
  }
  // The key walk may have started beside the query walk: it ends after it,
  // so that what follows in the stream follows both.
  if (kKeys && !writes_ds) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------- dQ from dS
// dQ of two query tiles per item from the dS that the key walk wrote: dQ += dS
// K over the key tiles, dS^T [keys x queries] read MN-major as the A operand.
// One pass over dS from memory (32 KB a tile against 512 cycles of products at
// head dim 128) bounds it; two query tiles share each tile of K, which halves
// what L2 delivers. A ring of 32 KB slots takes K, then the dS of the one or
// two query tiles, of each key tile.
//   warps 0-7 epilogue (four per query tile), 8 products, 9 loads
constexpr int kDqThreads = 320, kDqSlots = 7;
constexpr uint32_t kDqSlotBytes = 128u * 128u * 2u;

template <int D>
struct DCfg {
  static constexpr uint32_t kKBytes = 128u * D * 2u;
  static constexpr uint32_t kSmemBytes = kDqSlots * kDqSlotBytes + 1024u;
  static constexpr uint32_t kTmemCols = 4 * D;  // two query tiles, two items
};

struct DCtl {
  uint64_t full[kDqSlots], empty[kDqSlots], fix;
  uint64_t acc_full[2], acc_free[2];
  uint64_t idx_full[kBwdIdxSlots], idx_empty[kBwdIdxSlots];
  int idx_ring[kBwdIdxSlots];
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
};

// Which of the item's two query tiles key tile n holds dS for (bits 0 and 1),
// and the index of the first one's tile of dS.
__device__ __forceinline__ int held_tiles(const BwdParams& p, const BwdItem& it, int n, int& at) {
  const int4 s = __ldg(reinterpret_cast<const int4*>(p.spans + it.span + n));  // first, lo, hi
  const int i = it.tile * 2;
  at = s.x + i;
  return (i >= s.y && i < s.z ? 1 : 0) | (i + 1 >= s.y && i + 1 < s.z ? 2 : 0);
}

template <int D>
__device__ void dq_load(const BwdParams& p, DCtl* ctl, uint8_t* smem, const WaitCtx& w) {
  using C = DCfg<D>;
  const int lane = threadIdx.x & 31;
  uint32_t n_slot = 0, nfix = 0;
  bool ok = true, fixing = false;
  auto slot_free = [&]() -> bool {
    return n_slot < kDqSlots || wait_warp(&ctl->empty[n_slot % kDqSlots],
                                          ((n_slot / kDqSlots) - 1) & 1u, w, kBSiteB0Empty);
  };
  for (int k = 0; ok; ++k) {
    const int idx = bwd_claim(ctl, p.claims + 2, k, w);
    if (idx == 0x7fffffff) ok = false;
    if (idx >= p.n_g) break;
    const BwdItem it = p.g_items[idx];
    const SeqRec sr = p.seqs[it.b];
    for (int n = it.lo; n < it.hi && ok; ++n) {
      int at;
      const int held = held_tiles(p, it, n, at);
      if (!held) continue;
      if (!slot_free()) {
        ok = false;
        break;
      }
      uint32_t st = n_slot % kDqSlots;
      uint8_t* dst = smem + st * kDqSlotBytes;
      const int rows = min(128, sr.skv - n * 128);
      const bool clear = p.tnd && rows < 128;  // K rows of the next packed sequence
      if (lane == 0) {
        uint64_t* bar = clear ? &ctl->fix : &ctl->full[st];
        mbar_expect_tx(bar, C::kKBytes);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(dst + c * 16384, &p.tm_k, bar, c * 64, sr.kv_off + n * 128, it.h,
                      p.tnd ? 0 : it.b);
      }
      __syncwarp();
      if (clear) {
        fixing = true;
        if (!wait_warp(&ctl->fix, nfix & 1u, w, kBSiteFix)) {
          ok = false;
          break;
        }
        fixing = false;
        ++nfix;
        for (int x = rows * 8 + lane; x < 128 * 8; x += 32)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            st_shared_v4(smem_u32(dst) + c * 16384 + x * 16, 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->full[st]);
      }
      ++n_slot;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (!ok || !((held >> q) & 1)) continue;
        if (!slot_free()) {
          ok = false;
          continue;
        }
        st = n_slot % kDqSlots;
        if (lane == 0) {
          mbar_expect_tx(&ctl->full[st], kDqSlotBytes);
          bulk_load(smem + st * kDqSlotBytes, p.ds + (int64_t)(at + q) * (128 * 128), kDqSlotBytes,
                    &ctl->full[st]);
        }
        __syncwarp();
        ++n_slot;
      }
    }
  }
  if (!ok && lane == 0) {
    if (fixing) wait_bounded(&ctl->fix, nfix & 1u, w, kBSiteDrain, false);
    for (uint32_t r = n_slot > kDqSlots ? n_slot - kDqSlots : 0u; r < n_slot; ++r)
      wait_bounded(&ctl->full[r % kDqSlots], (r / kDqSlots) & 1u, w, kBSiteDrain, false);
  }
  __syncwarp();
}

template <int D>
__device__ void dq_mma(const BwdParams& p, DCtl* ctl, uint32_t tmem, const uint8_t* smem,
                       const WaitCtx& w) {
  constexpr uint32_t idesc = idesc_bf16(128, D, true) | (1u << 15);  // A MN-major too
  // dS: no swizzle, 8-key groups 128 bytes apart, blocks of 8 queries 2048
  // bytes apart. K: as in the walks.
  const uint64_t dA = sdesc_plain(smem_u32(smem), 128u, 2048u);
  const uint64_t dB = sdesc(smem_u32(smem), 16384u, 1024u);
  constexpr uint64_t kSlot = kDqSlotBytes >> 4;
  uint32_t n_slot = 0, items = 0;
  bool ok = true;
  for (int k = 0; ok; ++k, ++items) {
    const int idx = bwd_take(ctl, k, w);
    if (idx >= p.n_g) break;
    const BwdItem it = p.g_items[idx];
    const uint32_t buf = items & 1u;
    if (items >= 2 && !wait_warp(&ctl->acc_free[buf], ((items >> 1) - 1) & 1u, w, kBSiteAccFree))
      break;
    uint32_t started = 0;  // query tiles whose sum has begun
    for (int n = it.lo; n < it.hi && ok; ++n) {
      int at;
      const int held = held_tiles(p, it, n, at);
      if (!held) continue;
      const uint32_t ks = n_slot % kDqSlots;
      if (!wait_warp(&ctl->full[ks], (n_slot / kDqSlots) & 1u, w, kBSiteB0Full)) {
        ok = false;
        break;
      }
      ++n_slot;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (!ok || !((held >> q) & 1)) continue;
        const uint32_t st = n_slot % kDqSlots;
        if (!wait_warp(&ctl->full[st], (n_slot / kDqSlots) & 1u, w, kBSiteB1Full)) {
          ok = false;
          continue;
        }
        ++n_slot;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tmem + (2 * buf + q) * D;
          const uint64_t a = dA + st * kSlot, b = dB + ks * kSlot;
#pragma unroll
          for (int x = 0; x < 8; ++x)  // 16 keys
            mma_ss(d, a + x * (256u >> 4), b + x * (2048u >> 4), idesc,
                   (x > 0 || ((started >> q) & 1u)) ? 1u : 0u);
          mma_commit(&ctl->empty[st]);
          if (q == 1 || !(held & 2)) mma_commit(&ctl->empty[ks]);
        }
        __syncwarp();
      }
      started |= held;
    }
    if (!ok) break;
    if (elect_one()) mma_commit(&ctl->acc_full[buf]);
    __syncwarp();
  }
  if (elect_one()) mma_commit(&ctl->drain);
  __syncwarp();
  wait_bounded(&ctl->drain, 0u, w, kBSiteDrain, false);
}

template <int D>
__device__ void dq_epilogue(const BwdParams& p, DCtl* ctl, uint32_t tmem, const WaitCtx& w) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp >> 2, row = (warp & 3) * 32 + lane;
  const uint32_t lane_bits = (uint32_t)((warp & 3) * 32) << 16;
  const bool v8 = (reinterpret_cast<uintptr_t>(p.dq) & 31u) == 0;
  uint32_t items = 0;
  for (int k = 0;; ++k, ++items) {
    const int idx = bwd_take(ctl, k, w);
    if (idx >= p.n_g) return;
    const BwdItem it = p.g_items[idx];
    const SeqRec sr = p.seqs[it.b];
    const uint32_t buf = items & 1u;
    bool any = false;  // a key tile holds dS of this query tile
    for (int n = it.lo; n < it.hi && !any; ++n) {
      int at;
      any = (held_tiles(p, it, n, at) >> q) & 1;
    }
    const int64_t i = ((int64_t)it.tile * 2 + q) * 128 + row;
    const bool stored = i < sr.sq;
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.dq) + it.b * p.q_sb + it.h * p.q_sh +
                       (sr.q_off + i) * p.q_st;
    if (!wait_warp(&ctl->acc_full[buf], (items >> 1) & 1u, w, kBSiteAccFull)) return;
    tc_fence_after();
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t ov[32];
      tmem_ld32_wait(tmem + lane_bits + (2 * buf + q) * D + ch * 32, ov);
      uint4 pk[4];
      uint32_t* pw = reinterpret_cast<uint32_t*>(pk);
#pragma unroll
      for (int c = 0; c < 16; ++c)
        pw[c] = any ? pack_bf16(__uint_as_float(ov[2 * c]) * p.scale,
                                __uint_as_float(ov[2 * c + 1]) * p.scale)
                    : 0u;
      if (stored) {
        uint4* dst = reinterpret_cast<uint4*>(o + ch * 32);
        if (v8) {
          st_global_na_v8(dst, pk[0], pk[1]);
          st_global_na_v8(dst + 2, pk[2], pk[3]);
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) st_global_na_v4(dst + v, pk[v]);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->acc_free[buf]);
  }
}

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1) fa_bwd_dq_sm100(const __grid_constant__ BwdParams p) {
  using C = DCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  auto* ctl = reinterpret_cast<DCtl*>(smem + kDqSlots * kDqSlotBytes);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(p.err_word, kErrTimeout | (kBSiteSmem << kErrWhereShift));
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kDqSlots; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->acc_full[s], 1);
      mbar_init(&ctl->acc_free[s], 8);
    }
    for (int s = 0; s < kBwdIdxSlots; ++s) {
      mbar_init(&ctl->idx_full[s], 1);
      mbar_init(&ctl->idx_empty[s], 9);  // epilogue and MMA warps
    }
    mbar_init(&ctl->fix, 1);
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
            smem_u32(&ctl->tmem_base)),
        "r"(C::kTmemCols)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  const WaitCtx w{&ctl->abort_flag, p.err_word, p.timeout_ns};
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the key walk's dS
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp < 8) dq_epilogue<D>(p, ctl, tmem, w);
  else if (warp == 8) dq_mma<D>(p, ctl, tmem, smem, w);
  else dq_load<D>(p, ctl, smem, w);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::kTmemCols)
                 : "memory");
  }
}

}  // namespace dev

// ----------------------------------------------------------------- host

// One launch with `threads` x `smem` of a kernel that splits `regs` registers
// per thread; with `early` it may start before the launch ahead of it ends.
template <typename Kernel>
static cudaError_t launch_early(Kernel kern, std::atomic<uint64_t>* configured, const BwdParams& p,
                                int grid, int threads, uint32_t smem, int regs, bool early,
                                cudaStream_t stream, const char** why) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = device < 64 ? 1ull << device : 0ull;  // devices with the attributes set
  if (!(configured->load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    // setmaxnreg redistributes the registers the CTA was launched with; a split
    // larger than that allocation would never be granted.
    if (attr.numRegs < regs) {
      if (why) *why = "kernel compiled with fewer registers than its warpgroup split needs";
      return cudaErrorInvalidConfiguration;
    }
    configured->fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D, bool kKeys, int kBias>
static cudaError_t launch_walk(const BwdParams& p, int num_sms, cudaStream_t stream,
                               const char** why) {
  const int n = kKeys ? p.n_k : p.n_q;
  if (n <= 0) return cudaSuccess;
  static std::atomic<uint64_t> configured{0};
  return launch_early(dev::fa_bwd_sm100<D, kKeys, kBias>, &configured, p, n < num_sms ? n : num_sms,
                      dev::kBwdThreads,
                      dev::BCfg<D, kKeys, kBias == dev::kBwdBiasRel>::kSmemBytes,
                      dev::kBwdRegsLaunch, p.n_q > 0, stream, why);
}

template <int D>
static cudaError_t launch_dq(const BwdParams& p, int num_sms, cudaStream_t stream,
                             const char** why) {
  if (p.n_g <= 0) return cudaSuccess;
  static std::atomic<uint64_t> configured{0};
  return launch_early(dev::fa_bwd_dq_sm100<D>, &configured, p, p.n_g < num_sms ? p.n_g : num_sms,
                      dev::kDqThreads, dev::DCfg<D>::kSmemBytes, 0, true, stream, why);
}

template <int D, int kBias>
static cudaError_t launch_walks(const BwdParams& p, int num_sms, cudaStream_t stream,
                                const char** why) {
  if constexpr (dev::kWritesDs<D>) {
    if (p.ds) {
      const cudaError_t e = launch_walk<D, true, kBias>(p, num_sms, stream, why);
      return e == cudaSuccess ? launch_dq<D>(p, num_sms, stream, why) : e;
    }
  }
  const cudaError_t e = launch_walk<D, false, kBias>(p, num_sms, stream, why);
  return e == cudaSuccess ? launch_walk<D, true, kBias>(p, num_sms, stream, why) : e;
}

cudaError_t launch_bwd(int D, const BwdParams& p, int num_sms, cudaStream_t stream,
                       const char** why) {
  auto pick = [&](auto dim) {
    constexpr int kD = decltype(dim)::value;
    if (p.rel.ext) return launch_walks<kD, dev::kBwdBiasRel>(p, num_sms, stream, why);
    if (p.slopes) return launch_walks<kD, dev::kBwdBiasAlibi>(p, num_sms, stream, why);
    return launch_walks<kD, dev::kBwdBiasNone>(p, num_sms, stream, why);
  };
  return D == 128 ? pick(std::integral_constant<int, 128>{}) : pick(std::integral_constant<int, 64>{});
}

}  // namespace fa
