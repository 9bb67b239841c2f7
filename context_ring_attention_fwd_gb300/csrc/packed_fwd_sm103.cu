// Attention over packed prompts of different lengths with grouped heads, on sm_103a
// tensor cores (tcgen05), bf16.
//
// Row (t, h) - token t of its sequence, query head h - sees the keys of its own sequence
// (up to its own position if causal) of key head h / G:  s = q k / sqrt d,  out = softmax(s) v,
// lse = log sum exp s.  Keys are walked in 128-row tiles with the online-softmax merge
// ("上下文並行（Context Parallelism, CP）", compassingai.com, section 線上 Softmax) as in
// attn_sm103.cu: the CTA's roles, its use of TMEM and the softmax with a lagging reference
// are described there.  What differs is the work: packed query rows and items (packed.cuh),
// tiles that start at a sequence's first token, and rows behind a sequence's last key.
//
// Rows of V behind the sequence's last key may hold anything (the next prompt's values, or
// padding), and 0 times infinity is NaN, so the PV product of a ragged tile ends at the next
// multiple of 16 keys, and the up to 15 rows of V beyond the last key are zeroed in
// shared memory first.  K needs none: its rows are columns of S, which the mask replaces.
//
// Bound by the tensor pipe where sequences are long: 32K tokens of 8/2 heads, 2.2 TFLOP, 1200 us, 95 %
// of the cuBLAS rate (80 % of the pipe's cycles); a run of seconds, at the clock that the power cap
// leaves, 1330 - 1410.  In short ones by what an item costs besides its tiles, about 2.3 us (its
// first S, the drain behind its last P, its rows' way out): 14 prompts of up to 2000 tokens, 32/8
// heads, 109 GFLOP, 97 us, 56 % of the pipe's cycles.  (The next item's first S issued between the
// last two PVs, which the drain would hide, made the MMA warp's loop slower: 110 us there, 1280 for
// the 32K.)  P is rounded to bf16 for its product, as in the ring's forward, which costs about as
// much as the output's own rounding (2.0e-3 to 2.2e-3 against 64 bits, relative in the norm, where
// that alone makes 1.65e-3).
//
// Items that see many keys in a call of few are cut along them (packed_plan.cu): a part leaves its
// (O, m, l) in a slot, and the last to end of a query tile's parts joins them by the online
// merge of cp_lse_merge, in the parts' order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "attn_common.cuh"
#include "attn_softmax.cuh"
#include "internal.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace cpring {
namespace {

constexpr int kBM = kTileRows;
constexpr int kBN = kTileRows;
constexpr int kQTiles = 2;      // packed query tiles per item
constexpr int kStages = 2;      // K/V ring depth
constexpr int kThreads = 384;   // three warpgroups
constexpr int kLaunchRegs = 168;   // registers per thread at launch (checked by the build)
constexpr int kSoftmaxRegs = 200;  // softmax warpgroups after setmaxnreg.inc
constexpr int kControlRegs = 104;  // producer / MMA warpgroup after setmaxnreg.dec
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch's register pool");
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kSoftmaxWarps = 8;
constexpr int kTmemCols = 512;
constexpr float kOverflowGuard = 18446744073709551616.0f;  // 2^64
constexpr float kOverflowGuardLog2 = 64.0f;
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Layout {
  static constexpr int kTileBytes = kBM * D * 2;
  static constexpr int kPanelBytes = kBM * 128;  // 128 rows x 64 columns
  static constexpr int kPanels = D / 64;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kQTiles * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kStageOff = kVOff + kStages * kTileBytes;  // the softmax warps' rows on
  static constexpr int kBarOff = kStageOff + kSoftmaxWarps * kRowStage;  // their way out
  static constexpr int kRingOff = kBarOff + 256;  // the item ring
  static constexpr int kBytes = kRingOff + 256;
  static constexpr int kAlloc = kBytes + 1024;  // room to align the base to 1024 B
};

enum Bar : int {
  kQFull = 0,
  kQEmpty = 1,
  kKFull = 2,     // + stage
  kVFull = 4,     // + stage
  kKEmpty = 6,    // + stage: K tile consumed by both S products
  kVEmpty = 8,    // + stage: V tile consumed by both PV products
  kSFull = 10,    // + tile
  kPReady = 12,   // + tile: the first 64 keys' P of tile t stored
  kPReadyB = 14,  // + tile: the last 64 keys' P of tile t stored (and O rescaled)
  kOBar = 16,     // + tile: every PV of tile t in the item done (once per item)
  kDrain = 18,
  kJoin = 19,     // + tile: its threads have stored a part's state; then: know its rank
  kNumBars = 21
};
constexpr int kTmemSlot = kNumBars * 8;
constexpr int kAbortSlot = kNumBars * 8 + 4;
constexpr int kRankSlot = kNumBars * 8 + 8;  // two
static_assert(kRankSlot + 8 <= 256, "the barriers' shared-memory block");

struct FwdParams {
  int* head;           // the plan's list
  const int4* items;
  const int32_t* offsets;  // or, of a call without a plan, the sequences' offsets
  int n_seqs;
  int T, Hq, Hk, G;
  int tq;              // tokens of a packed tile
  int warp_tokens;     // of a warp's 32 rows; 0: they hold a part of a token
  int causal;
  float scale_log2;    // log2(e) / sqrt(d)
  __nv_bfloat16* out;  // [T, Hq, d]
  float* lse;          // [Hq, T]
  float4* parts;       // [slot][Hk][query tile]: O [d / 4][128] float4, then (m, l) [128]
  int* done;           // [slot][Hk][query tile]
  int* err;
  unsigned long long timeout_ns;
  int fault_drop_k;    // test hook: CTA 0 never loads its first K tile
};

// An item: two packed tiles of one sequence for one key head, the first key tile, and the last
// that each tile sees (before the first: none), of an item in parts the part's own.
struct FwdItem {
  int row0, len, hk;
  int token[kQTiles], tokens[kQTiles], last[kQTiles];
  int first;
  int slot, part, parts[kQTiles];  // the part's slot, its index, and the parts of each tile
};
template <bool kParts>
__device__ __forceinline__ void fwd_item(const FwdParams& p, const PackedEntry& x, FwdItem& it) {
  const int4 e = x.e;
  it.hk = x.hk;
  it.row0 = e.x;
  it.len = e.y;
#pragma unroll
  for (int t = 0; t < kQTiles; ++t) {
    it.token[t] = (e.z * kQTiles + t) * p.tq;
    it.tokens[t] = max(0, min(p.tq, it.len - it.token[t]));
    const int seen = p.causal ? it.token[t] + it.tokens[t] : it.len;
    it.last[t] = it.tokens[t] > 0 ? (seen - 1) / kBN : -1;
    it.parts[t] = 1;
  }
  it.first = it.slot = it.part = 0;
  if (kParts && e.w != 0) {
    const int chunk = p.head[2];
    it.slot = (e.w & 0xffff) - 1;
    it.part = e.w >> 16;
    it.first = it.part * chunk;
#pragma unroll
    for (int t = 0; t < kQTiles; ++t) {
      it.parts[t] = it.last[t] / chunk + 1;
      it.last[t] = min(it.last[t], it.first + chunk - 1);
    }
  }
}

// float4 of a query tile's state in a slot.
template <int D>
constexpr int kPartSize = (D / 4) * kBM + kBM / 2;

// (m, l) of this thread's row in part j of the parts from `first` on (its row's first float4).
template <int D>
__device__ __forceinline__ float2 part_ml(const FwdParams& p, const float4* first, int j,
                                          int row_in_tile) {
  const float4* const base = first - row_in_tile +
                             static_cast<size_t>(j) * p.Hk * kQTiles * kPartSize<D> +
                             (D / 4) * kBM;
  float2 ml;
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];"
               : "=f"(ml.x), "=f"(ml.y)
               : "l"(reinterpret_cast<const float2*>(base) + row_in_tile)
               : "memory");
  return ml;
}
// Columns [32 ch, 32 ch + 32) of the row: the parts' O, each against its own reference, to the
// reference m.  Bound by latency: two parts' loads are under way at a time.
template <int D>
__device__ __forceinline__ void join_parts(const FwdParams& p, const float4* first, int ch,
                                           int parts, float m, int row_in_tile,
                                           uint32_t (&sum)[32]) {
  float s[32];
#pragma unroll
  for (int x = 0; x < 32; ++x) s[x] = 0.f;
  const size_t step = static_cast<size_t>(p.Hk) * kQTiles * kPartSize<D>;
#pragma unroll 1
  for (int j = 0; j < parts; j += 2) {
    float4 f[2][8];
    float w[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const bool there = j + y < parts;
      const float2 ml = there ? part_ml<D>(p, first, j + y, row_in_tile) : make_float2(0.f, 0.f);
      w[y] = ml.y == 0.f ? 0.f : ptx::ex2(ml.x - m);
#pragma unroll
      for (int x = 0; x < 8; ++x)
        f[y][x] = there ? load_cg(first + (j + y) * step + (ch * 8 + x) * kBM)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        s[4 * x] = fmaf(f[y][x].x, w[y], s[4 * x]);
        s[4 * x + 1] = fmaf(f[y][x].y, w[y], s[4 * x + 1]);
        s[4 * x + 2] = fmaf(f[y][x].z, w[y], s[4 * x + 2]);
        s[4 * x + 3] = fmaf(f[y][x].w, w[y], s[4 * x + 3]);
      }
  }
#pragma unroll
  for (int x = 0; x < 32; ++x) sum[x] = __float_as_uint(s[x]);
}

// This thread's 128 scores of the S tile, with columns behind c_hi set to -inf (chunk by
// chunk: one that the whole warp sees whole costs a test).
__device__ __forceinline__ void load_seen(uint32_t tS, int c_hi, uint32_t (&sv)[4][32]) {
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) ptx::tmem_ld32(tS + ch * 32, sv[ch]);
  ptx::tmem_wait_ld();
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) ptx::reg_fence(sv[ch]);
  if (__all_sync(0xffffffffu, c_hi >= kBN - 1)) return;
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const int hi = c_hi - ch * 32;
    if (__all_sync(0xffffffffu, hi >= 31)) continue;
    const uint32_t seen = hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1u;
#pragma unroll
    for (int x = 0; x < 32; ++x)
      if (!(seen >> x & 1u)) sv[ch][x] = __float_as_uint(-INFINITY);
  }
}

// kParts: for calls whose items may be in parts.
template <int D, bool kParts>
__global__ void __launch_bounds__(kThreads, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v,
                      const __grid_constant__ CUtensorMap tmap_o, const FwdParams p) {
  using Lay = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t bars = sbase + Lay::kBarOff;
  auto bar = [&](int idx) -> uint32_t { return bars + 8u * static_cast<uint32_t>(idx); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kBarOff + kTmemSlot);
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(smem + Lay::kBarOff + kAbortSlot);
  const PackedRing ring{
      sbase + Lay::kRingOff,
      reinterpret_cast<volatile int(*)[8]>(smem + Lay::kRingOff + 2 * kRing * 8)};
  volatile int* rank = reinterpret_cast<volatile int*>(smem + Lay::kBarOff + kRankSlot);
  // the ring's index of the item whose Q the producer is loading, for the MMA warp
  volatile int* q_item =
      reinterpret_cast<volatile int*>(smem + Lay::kRingOff + 2 * kRing * 8 + kRing * 32);

  // (by a shuffle: the compiler then knows it, and what follows from it, as the warp's)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ptx::mbar_init(bar(kQFull), 1);
    ptx::mbar_init(bar(kQEmpty), 1);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar(kKFull + s), 1);
      ptx::mbar_init(bar(kVFull + s), 1);
      ptx::mbar_init(bar(kKEmpty + s), 1);
      ptx::mbar_init(bar(kVEmpty + s), 1);
    }
    for (int t = 0; t < kQTiles; ++t) {
      ptx::mbar_init(bar(kSFull + t), 1);
      ptx::mbar_init(bar(kPReady + t), 128);
      ptx::mbar_init(bar(kPReadyB + t), 128);
      ptx::mbar_init(bar(kOBar + t), 1);
      ptx::mbar_init(bar(kJoin + t), 128);
    }
    ptx::mbar_init(bar(kDrain), 1);
    ring.init(kSoftmaxWarps);
    *abort_flag = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  // Without a plan a CTA has one item, which its producer finds while the others set up.
  PackedEntry only{make_int4(0, 0, 0, 0), -1};
  if (p.offsets != nullptr && warp == kProducerWarp) {
    bool bad;
    only = packed_direct(p.offsets, p.n_seqs, p.T, kQTiles * p.tq, p.Hk, blockIdx.x, bad);
    if (bad && lane == 0) atomicOr(p.err, kErrDocOffsets);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  cudaGridDependencySynchronize();  // the plan

  if (warp >= kProducerWarp) {
   ptx::setmaxnreg_dec<kControlRegs>();
   if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tmap_q);
      ptx::tma_prefetch_desc(&tmap_k);
      ptx::tma_prefetch_desc(&tmap_v);
      const uint32_t q_bytes = static_cast<uint32_t>(p.tq * p.G) * 128u * Lay::kPanels;
      const PackedOrder order(p.offsets ? 0 : p.head[0], p.Hk, gridDim.x);
      uint32_t kv_iter = 0, q_iter = 0;
      int ahead = INT_MAX;  // the claim of the CTA's next item
      // Loads started into each stage: the n-th one completes phase n - 1.
      uint32_t k_armed0 = 0, k_armed1 = 0, v_armed0 = 0, v_armed1 = 0;
      bool dropped = false;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int w = k == 0 ? static_cast<int>(blockIdx.x) : ahead;
        const PackedEntry x = p.offsets && k == 0 ? only : order.at(p.items, w);
        if (!ring.put(static_cast<uint32_t>(k), x, abort_flag, p)) { ok = false; break; }
        if (x.hk < 0) break;
        FwdItem it;
        fwd_item<kParts>(p, x, it);
        if (!wait1(bar(kQEmpty), (q_iter & 1u) ^ 1u, abort_flag, p)) { ok = false; break; }
        *q_item = k;  // the MMA warp reads it with this phase of kQFull
        const int tiles = it.tokens[1] > 0 ? 2 : 1;
        ptx::mbar_arrive_expect_tx(bar(kQFull), tiles * q_bytes);
        for (int t = 0; t < tiles; ++t)
#pragma unroll
          for (int pn = 0; pn < Lay::kPanels; ++pn)
            ptx::tma_load_3d(sbase + Lay::kQOff + t * Lay::kTileBytes + pn * Lay::kPanelBytes,
                             &tmap_q, bar(kQFull), pn * 64, it.hk * p.G,
                             it.row0 + (t ? it.token[1] : it.token[0]));
        ++q_iter;
        const int last = max(it.last[0], it.last[1]);
        for (int f = it.first; f <= last; ++f) {
          const uint32_t st = kv_iter % kStages;
          const uint32_t ph = (kv_iter / kStages) & 1u;
          const int row = it.row0 + f * kBN;
          // The next item is claimed when the last loads but one are under way, not before: a CTA
          // at its start would take one that another is free for sooner; and not behind the last,
          // where the answer would be waited for.
          if (f == max(it.first, last - 1) && !p.offsets) ahead = packed_claim(p.head, gridDim.x);
          if (!wait1(bar(kKEmpty + st), ph ^ 1u, abort_flag, p)) { ok = false; break; }
          if (p.fault_drop_k && blockIdx.x == 0 && !dropped) {
            // Test hook: this K tile is never loaded, so the MMA warp's
            // bounded wait for it runs out and the CTA takes its abort path.
            dropped = true;
          } else {
            ptx::mbar_arrive_expect_tx(bar(kKFull + st), Lay::kTileBytes);
#pragma unroll
            for (int pn = 0; pn < Lay::kPanels; ++pn)
              ptx::tma_load_3d(sbase + Lay::kKOff + st * Lay::kTileBytes + pn * Lay::kPanelBytes,
                               &tmap_k, bar(kKFull + st), pn * 64, it.hk, row);
            if (st == 0) ++k_armed0; else ++k_armed1;
          }
          if (!wait1(bar(kVEmpty + st), ph ^ 1u, abort_flag, p)) { ok = false; break; }
          ptx::mbar_arrive_expect_tx(bar(kVFull + st), Lay::kTileBytes);
#pragma unroll
          for (int pn = 0; pn < Lay::kPanels; ++pn)
            ptx::tma_load_3d(sbase + Lay::kVOff + st * Lay::kTileBytes + pn * Lay::kPanelBytes,
                             &tmap_v, bar(kVFull + st), pn * 64, it.hk, row);
          if (st == 0) ++v_armed0; else ++v_armed1;
          ++kv_iter;
        }
      }
      // No more items: tell the MMA warp through the next phase of kQFull.
      if (ok && wait1(bar(kQEmpty), (q_iter & 1u) ^ 1u, abort_flag, p)) {
        *q_item = -1;
        ptx::mbar_arrive(bar(kQFull));
        ++q_iter;
      }
      // Let every copy this thread started land before the CTA can exit.
      if (q_iter > 0) wait1(bar(kQFull), (q_iter - 1) & 1u, abort_flag, p, false);
      if (k_armed0 > 0) wait1(bar(kKFull + 0), (k_armed0 - 1) & 1u, abort_flag, p, false);
      if (k_armed1 > 0) wait1(bar(kKFull + 1), (k_armed1 - 1) & 1u, abort_flag, p, false);
      if (v_armed0 > 0) wait1(bar(kVFull + 0), (v_armed0 - 1) & 1u, abort_flag, p, false);
      if (v_armed1 > 0) wait1(bar(kVFull + 1), (v_armed1 - 1) & 1u, abort_flag, p, false);
    }
   } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // (the whole warp with warp-uniform values; see attn_sm103.cu)
    constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(kBM, kBN, false);
    constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, D, true);
    constexpr int kSteps = kBN / 16;  // of a PV product
    uint32_t kv_iter = 0, q_iter = 0;
    uint32_t p_cnt0 = 0, p_cnt1 = 0;
    bool ok = true;
    const uint64_t d_qk = ptx::smem_desc_sw128(sbase, 16, 1024);
    const uint64_t d_v = ptx::smem_desc_sw128(sbase, Lay::kPanelBytes, 1024);
    // O_t (+)= P_t V over the steps [part * 4, part * 4 + 4): keys 0-63 (part 0) or 64-127 (part
    // 1), whose P the softmax signals separately.  kWhole: all of them; otherwise those below
    // `steps`.  (A test between the products would hold this warp's issue up: with one in every
    // step the kernel took 1769 us instead of 1287 for 32K tokens of 8/2 heads.)
    auto issue_pv = [&](auto whole, int t, uint32_t st, bool first, int part, int steps) {
      const uint64_t dv = d_v + ((Lay::kVOff + st * Lay::kTileBytes) >> 4);
      auto step = [&](int s) {
        ptx::mma_ts_w(tmem_base + 256 + t * D, tmem_base + t * 128 + s * 8,
                      dv + static_cast<uint64_t>((s * 16 * 128) >> 4), kIdescPV,
                      (first && s == 0) ? 0u : 1u);
      };
      if constexpr (decltype(whole)::value) {
#pragma unroll
        for (int s = part * (kSteps / 2); s < (part + 1) * (kSteps / 2); ++s) step(s);
      } else {
#pragma unroll 1
        for (int s = part * (kSteps / 2); s < min(steps, (part + 1) * (kSteps / 2)); ++s) step(s);
      }
    };
    // S_t = Q_t K^T (both K-major, 128-byte swizzled panels; a K step is
    // 32 bytes, four steps per panel).
    auto issue_s = [&](int t, uint32_t st) {
      const uint64_t dq = d_qk + ((Lay::kQOff + t * Lay::kTileBytes) >> 4);
      const uint64_t dk = d_qk + ((Lay::kKOff + st * Lay::kTileBytes) >> 4);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint64_t step =
            static_cast<uint64_t>(((s >> 2) * Lay::kPanelBytes + (s & 3) * 32) >> 4);
        ptx::mma_ss_w(tmem_base + t * 128, dq + step, dk + step, kIdescQK, s > 0 ? 1u : 0u);
      }
      ptx::mma_commit_w(bar(kSFull + t));
    };
    for (;;) {
      if (!wait_warp(bar(kQFull), q_iter & 1u, abort_flag, p)) { ok = false; break; }
      ++q_iter;
      const int k = *q_item;
      if (k < 0) break;
      FwdItem it;
      fwd_item<kParts>(p, ring.read(static_cast<uint32_t>(k)), it);
      ptx::tc_fence_after();
      bool pend0 = false, pend1 = false;    // an S issued whose PV is still owed
      bool first0 = true, first1 = true;    // next PV overwrites O
      uint32_t prev_st = 0, prev_ph = 0;
      bool have_prev = false, prev_v_ready = false;
      const int last = max(it.last[0], it.last[1]);
      // keys of the last tile: fewer than 128 where it is the sequence's last
      const int last_keys = min(kBN, it.len - last * kBN);
      // Owed PV of tile t on the previous K/V stage: wait for V and P, issue.  After the item's
      // last PV of tile t, O_t is final.  kWhole: every key of the tile exists; otherwise V's
      // rows behind the last key are zeroed first.
      auto flush = [&](auto whole, int t, uint32_t& pc, bool& first, bool final) -> bool {
        if (!prev_v_ready) {
          if (!wait_warp(bar(kVFull + prev_st), prev_ph, abort_flag, p)) return false;
          if constexpr (!decltype(whole)::value) {
            zero_rows<Lay::kPanels>(sbase + Lay::kVOff + prev_st * Lay::kTileBytes, last_keys,
                                    (last_keys + 15) / 16 * 16);
            ptx::fence_proxy_async_shared();
            __syncwarp();
          }
          prev_v_ready = true;
        }
        const int steps = (last_keys + 15) / 16;
        if (!wait_warp(bar(kPReady + t), pc & 1u, abort_flag, p)) return false;
        ptx::tc_fence_after();
        issue_pv(whole, t, prev_st, first, 0, steps);
        if (!wait_warp(bar(kPReadyB + t), pc & 1u, abort_flag, p)) return false;
        ++pc;
        ptx::tc_fence_after();
        issue_pv(whole, t, prev_st, false, 1, steps);
        if (final) ptx::mma_commit_w(bar(kOBar + t));
        first = false;
        return true;
      };
      for (int f = it.first; f <= last; ++f) {
        const uint32_t st = kv_iter % kStages;
        const uint32_t ph = (kv_iter / kStages) & 1u;
        if (pend0) {
          if (!flush(std::true_type(), 0, p_cnt0, first0, f - 1 == it.last[0])) {
            ok = false;
            break;
          }
          pend0 = false;
        }
        if (!wait_warp(bar(kKFull + st), ph, abort_flag, p)) { ok = false; break; }
        ptx::tc_fence_after();
        if (f <= it.last[0]) {
          issue_s(0, st);
          pend0 = true;
        }
        if (pend1) {
          if (!flush(std::true_type(), 1, p_cnt1, first1, f - 1 == it.last[1])) {
            ok = false;
            break;
          }
          pend1 = false;
        }
        if (f <= it.last[1]) {
          issue_s(1, st);
          pend1 = true;
        }
        ptx::mma_commit_w(bar(kKEmpty + st));                      // K(f) read by every S
        if (have_prev) ptx::mma_commit_w(bar(kVEmpty + prev_st));  // V(f-1) read by every PV
        prev_st = st;
        prev_ph = ph;
        have_prev = true;
        prev_v_ready = false;
        ++kv_iter;
      }
      if (!ok) break;
      ptx::mma_commit_w(bar(kQEmpty));  // every S of this item has been issued
      if (last_keys == kBN) {
        ok = (!pend0 || flush(std::true_type(), 0, p_cnt0, first0, true)) &&
             (!pend1 || flush(std::true_type(), 1, p_cnt1, first1, true));
      } else {
        ok = (!pend0 || flush(std::false_type(), 0, p_cnt0, first0, true)) &&
             (!pend1 || flush(std::false_type(), 1, p_cnt1, first1, true));
      }
      if (!ok) break;
      if (have_prev) ptx::mma_commit_w(bar(kVEmpty + prev_st));
    }
    // Wait until every MMA this warp issued has finished.
    ptx::mma_commit_w(bar(kDrain));
    wait_warp(bar(kDrain), 0u, abort_flag, p, false);
   }
  } else {
    ptx::setmaxnreg_inc<kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;  // query tile of this warpgroup
    const int wq = warp & 3;  // TMEM lane quarter
    const int row_in_tile = wq * 32 + lane;
    const int row_token = row_in_tile / p.G, row_head = row_in_tile - row_token * p.G;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem_base + lane_off + static_cast<uint32_t>(t * 128);
    const uint32_t tO = tmem_base + lane_off + 256u + static_cast<uint32_t>(t * D);
    const float sc = p.scale_log2;
    uint32_t s_cnt = 0, o_cnt = 0, join_cnt = 0;
    bool ok = true;
    PackedEntry entry;
    ok = ring.get(0, entry, abort_flag, p);
    for (uint32_t k = 0; ok; ++k) {
      entry = PackedRing::uniform(entry);
      if (entry.hk < 0) break;
      FwdItem it;
      fwd_item<kParts>(p, entry, it);
      // this warpgroup's tile (selects keep the item in registers)
      const int tokens = t ? it.tokens[1] : it.tokens[0];
      const int last = t ? it.last[1] : it.last[0];
      const int parts = t ? it.parts[1] : it.parts[0];
      if (tokens == 0 || last < it.first) {
        ok = ring.get(k + 1, entry, abort_flag, p);
        continue;
      }
      const bool row_valid = row_token < tokens;
      const int token = (t ? it.token[1] : it.token[0]) + row_token;
      const int seen = !row_valid ? 0 : p.causal ? token + 1 : it.len;  // keys
      // A row that is not stored has a reference from the start, so that it does not hold
      // its warp to the careful pass; all of its columns are masked.
      float m_used = row_valid ? -INFINITY : 0.f, l_run = 0.f;
      for (int f = it.first; f <= last; ++f) {
        if (!wait_warp(bar(kSFull + t), s_cnt & 1u, abort_flag, p)) { ok = false; break; }
        ++s_cnt;
        ptx::tc_fence_after();
        const int c_hi = seen - f * kBN - 1;
        uint32_t sv[4][32];
        uint32_t pk[2][32];
        float lsum, mx;
        float alpha = 1.f;
        bool rescale_o = false;
        load_seen(tS, c_hi, sv);
        if (f == it.first) {
          // Its row max is the reference; a row that sees none of a part's first tile sees
          // none of the part.  (The rest is the code of every tile, so that a short prompt waits
          // for little code to be fetched.)
          const float m_tile = row_max(sv) * sc;
          if (row_valid) m_used = kParts && m_tile == -INFINITY && it.part > 0 ? 0.f : m_tile;
        }
        {
          // P in two halves of 64 keys against the current reference, each signalled once
          // stored; checked first against the guard (see attn_sm103.cu).
          const float lsum1 = exp_half(sv, 0, sc, m_used, pk);
          const float mx2 = half_max(sv, 1);
          const bool in_range =
              (lsum1 <= kOverflowGuard) & (mx2 * sc <= m_used + kOverflowGuardLog2);
          if (__all_sync(0xffffffffu, in_range)) {
            store_p_half(tS, pk, 0);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(kPReady + t));
            const float lsum2 = exp_half(sv, 1, sc, m_used, pk);
            l_run += lsum1 + lsum2;
            store_p_half(tS, pk, 1);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(kPReadyB + t));
            continue;
          }
          // Rare: a row ran past the guard.  Move its reference to this tile's max; every
          // lane recomputes.
          const float m_tile = row_max(sv) * sc;
          if (!in_range && m_tile > m_used) {
            rescale_o = true;
            alpha = ptx::ex2(m_used - m_tile);
            l_run *= alpha;
            m_used = m_tile;
          }
          exponentials<false, false>(sv, sc, m_used, pk, lsum, mx);
        }
        l_run += lsum;
        ptx::tmem_st32(tS, pk[0]);
        ptx::tmem_st32(tS + 32, pk[1]);
        if (__any_sync(0xffffffffu, rescale_o)) {
          // O_t already holds the sum up to the previous tile: the MMA warp
          // issued that PV before this tile's S, and the commit this warp
          // waited on for S tracks every MMA issued before it.
#pragma unroll
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t ov[32];
            ptx::tmem_ld32(tO + ch * 32, ov);
            ptx::tmem_wait_ld();
            ptx::reg_fence(ov);
#pragma unroll
            for (int x = 0; x < 32; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * alpha);
            ptx::tmem_st32(tO + ch * 32, ov);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(kPReady + t));
        ptx::mbar_arrive(bar(kPReadyB + t));
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if (!ring.get(k + 1, entry, abort_flag, p)) { ok = false; break; }  // while O is formed
      if (!wait_warp(bar(kOBar + t), o_cnt & 1u, abort_flag, p)) { ok = false; break; }
      ++o_cnt;
      ptx::tc_fence_after();
      const float4* first_part = nullptr;
      if (kParts && parts > 1) {
        const size_t at = (static_cast<size_t>(it.slot) * p.Hk + it.hk) * kQTiles + t;
        float4* const to = p.parts + at * kPartSize<D> + row_in_tile;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t ov[32];
          ptx::tmem_ld32(tO + ch * 32, ov);
          ptx::tmem_wait_ld();
          ptx::reg_fence(ov);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            to[(ch * 8 + x) * kBM] =
                make_float4(__uint_as_float(ov[4 * x]), __uint_as_float(ov[4 * x + 1]),
                            __uint_as_float(ov[4 * x + 2]), __uint_as_float(ov[4 * x + 3]));
        }
        reinterpret_cast<float2*>(to - row_in_tile + (D / 4) * kBM)[row_in_tile] =
            make_float2(m_used, l_run);
        __threadfence();
        ptx::mbar_arrive(bar(kJoin + t));
        if (!wait_warp(bar(kJoin + t), join_cnt & 1u, abort_flag, p)) { ok = false; break; }
        ++join_cnt;
        const size_t at0 = (static_cast<size_t>(it.slot - it.part) * p.Hk + it.hk) * kQTiles + t;
        if (row_in_tile == 0) {
          rank[t] = atomicAdd(p.done + at0, 1);
          __threadfence();
        }
        ptx::mbar_arrive(bar(kJoin + t));
        if (!wait_warp(bar(kJoin + t), join_cnt & 1u, abort_flag, p)) { ok = false; break; }
        ++join_cnt;
        if (rank[t] != parts - 1) continue;
        __threadfence();
        first_part = p.parts + at0 * kPartSize<D> + row_in_tile;
        // the row's reference and sum over all parts
        m_used = -INFINITY;
        l_run = 0.f;
        for (int j = 0; j < parts; ++j) {
          const float2 ml = part_ml<D>(p, first_part, j, row_in_tile);
          if (ml.y == 0.f) continue;  // the part saw nothing of the row
          const float big = fmaxf(m_used, ml.x);
          l_run = (m_used == -INFINITY ? 0.f : l_run * ptx::ex2(m_used - big)) +
                  ml.y * ptx::ex2(ml.x - big);
          m_used = big;
        }
      }
      const float inv_l = 1.f / l_run;
      const size_t row = static_cast<size_t>(it.row0) + token;
      const int h = it.hk * p.G + row_head;
      __nv_bfloat16* const dst = row_valid ? p.out + (row * p.Hq + h) * D : nullptr;
      const uint32_t rows = sbase + Lay::kStageOff + warp * kRowStage;
      // Whole tokens of all its rows go out by TMA, which the warp does not wait for.  (Rows
      // written by the lanes held it up for 2700 - 3100 clocks an item.)
      const bool by_tma = p.warp_tokens > 0 && (wq + 1) * p.warp_tokens <= tokens;
#pragma unroll 1
      for (int half = 0; half < D / 64; ++half) {  // 64 columns, 128 bytes of a row
        uint32_t ov[2][32];
        if (kParts && first_part != nullptr) {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch)
            join_parts<D>(p, first_part, half * 2 + ch, parts, m_used, row_in_tile, ov[ch]);
        } else {
          ptx::tmem_ld32(tO + half * 64, ov[0]);
          ptx::tmem_ld32(tO + half * 64 + 32, ov[1]);
          ptx::tmem_wait_ld();
          ptx::reg_fence(ov[0]);
          ptx::reg_fence(ov[1]);
        }
        if (lane == 0) ptx::tma_store_wait_read();  // the stage is free again
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t b[16];
#pragma unroll
          for (int x = 0; x < 16; ++x)
            b[x] = ptx::pack_bf16(__uint_as_float(ov[ch][2 * x]) * inv_l,
                                  __uint_as_float(ov[ch][2 * x + 1]) * inv_l);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            stage_chunk(rows, lane, ch * 4 + x, b[4 * x], b[4 * x + 1], b[4 * x + 2], b[4 * x + 3]);
        }
        if (by_tma) {
          ptx::fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0)
            ptx::tma_store_3d(rows, &tmap_o, half * 64, it.hk * p.G,
                              it.row0 + (t ? it.token[1] : it.token[0]) + wq * p.warp_tokens);
        } else {
          write_rows(rows, dst ? dst + half * 64 : nullptr, lane);
        }
      }
      if (row_valid) p.lse[static_cast<size_t>(h) * p.T + row] = (m_used + log2f(l_run)) * kLn2;
    }
    if (lane == 0) ptx::tma_store_wait();
  }

  // ---------------------------------------------------------------- teardown
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <int D, bool kParts>
cudaError_t launch_packed_fwd(const PackedArgs& a, const FwdParams& p, int grid,
                              cudaStream_t stream) {
  using Lay = Layout<D>;
  static_assert(Lay::kAlloc <= 232448, "shared memory budget");
  const auto kern = packed_fwd_kernel<D, kParts>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), Lay::kAlloc);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv, mo;
  if (!packed_map(&mq, a.q, a.T, a.Hq, D, a.qs[0], a.qs[1], p.G, p.tq) ||
      !packed_map(&mk, a.k, a.T, a.Hk, D, a.ks[0], a.ks[1], 1, kBN) ||
      !packed_map(&mv, a.v, a.T, a.Hk, D, a.vs[0], a.vs[1], 1, kBN) ||
      !packed_map(&mo, p.out, a.T, a.Hq, D, static_cast<long long>(a.Hq) * D, D, p.G,
                  std::max(1, p.warp_tokens)))
    return cudaErrorInvalidValue;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Lay::kAlloc;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = p.offsets ? 0 : 1;
  count_launch(0);
  return cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, mo, p);
}

// A call that may have this many items has enough of them, whatever the lengths, and its
// kernel is the one that knows no parts.
constexpr int kManyItems = 1024;

// Byte offsets of the workspace's parts: the list, and the states of items in parts.
struct Space {
  int slots;  // of a key head
  long long list, done, parts, total;
  Space(int T, int n, int Hk, int d, int tokens) {
    const auto up = [](long long x) { return (x + 255) / 256 * 256; };
    const long long items = packed_items(T, n, tokens);
    const long long most = T <= kBN * kLeastCut || items * Hk >= kManyItems
                               ? 0
                               : items * (T / kBN / kLeastPart + 1);
    slots = packed_slots(most, kMaxFwdParts, Hk);
    list = 0;
    done = up(packed_list_bytes(T, n, tokens) + 16LL * slots);
    parts = done + up(4LL * slots * Hk * kQTiles);
    total = parts + 16LL * slots * Hk * kQTiles * (d == 128 ? kPartSize<128> : kPartSize<64>);
  }
};

}  // namespace

bool packed_strides(const int64_t* given, int H, int d, int64_t (&to)[2]) {
  to[0] = static_cast<int64_t>(H) * d;
  to[1] = d;
  if (!given) return true;
  // a tensor map's strides: multiples of one another, below 2^40 bytes
  to[0] = given[0];
  to[1] = given[1];
  return to[1] > 0 && to[0] > 0 && to[1] % d == 0 && to[0] % to[1] == 0 &&
         to[0] / to[1] >= H && to[0] < (1LL << 38);
}

cp_status check_packed(int T, int n, int Hq, int Hk, int d, int causal) {
  if (T < 1 || n < 1 || n > kMaxPacked || Hq < 1 || Hk < 1 || Hk > 65535 || Hq % Hk != 0 ||
      (causal != 0 && causal != 1))
    return CP_ERR_SHAPE;
  if ((d != 64 && d != 128) || Hq / Hk > kTileRows) return CP_ERR_UNSUPPORTED;
  // items and rows are counted in an int
  const long long rows = static_cast<long long>(T) * Hq;
  if (rows > 0x7fffffff || (static_cast<long long>(T) + n) * Hk >= (1LL << 30)) return CP_ERR_SHAPE;
  return CP_OK;
}

}  // namespace cpring

extern "C" {

int64_t cp_packed_attn_fwd_workspace_bytes(int T, int n_seqs, int Hq, int Hk, int d) {
  if (cpring::check_packed(T, n_seqs, Hq, Hk, d, 0) != CP_OK) return -1;
  return cpring::Space(T, n_seqs, Hk, d, cpring::kQTiles * (cpring::kTileRows / (Hq / Hk))).total;
}

cp_status cp_packed_attn_fwd(const void* q, const int64_t* q_strides, const void* k,
                             const int64_t* k_strides, const void* v, const int64_t* v_strides,
                             const int32_t* seq_offsets, void* out, float* lse, int T, int n_seqs,
                             int Hq, int Hk, int d, int causal, void* workspace,
                             int64_t workspace_bytes, cudaStream_t stream) {
  cpring::TraceRange trace_("cp_packed_attn_fwd");
  using namespace cpring;
  if (!q || !k || !v || !seq_offsets || !out || !lse || !workspace) return CP_ERR_NULL;
  const cp_status st = check_packed(T, n_seqs, Hq, Hk, d, causal);
  if (st != CP_OK) return st;
  PackedArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.T = T; a.Hq = Hq; a.Hk = Hk;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(seq_offsets, 4) || !aligned(workspace, 256) ||
      !packed_strides(q_strides, Hq, d, a.qs) || !packed_strides(k_strides, Hk, d, a.ks) ||
      !packed_strides(v_strides, Hk, d, a.vs))
    return CP_ERR_ALIGN;
  const int G = Hq / Hk, tq = kTileRows / G, tokens = kQTiles * tq;
  const Space sp(T, n_seqs, Hk, d, tokens);
  if (workspace_bytes < sp.total) return CP_ERR_BUFFER;
  if (device_cc() != 103) return CP_ERR_DEVICE;
  // A call whose every item, whatever the lengths, has a CTA to itself and stays whole needs no
  // plan.  (12 prompts of up to 90 tokens, 32/8 heads: 14.0 us a call with one, 10.5 without.)
  const long long most_items = packed_items(T, n_seqs, tokens) * Hk;
  const bool direct = most_items <= sm_count() && sp.slots == 0;
  char* const ws = static_cast<char*>(workspace);
  PackedPlan plan{};
  plan.list[0] = packed_list(ws + sp.list, T, n_seqs, tokens, false, sp.slots);
  plan.list[0].done = reinterpret_cast<int*>(ws + sp.done);
  plan.list[0].n_done = sp.slots * Hk * kQTiles;
  plan.tq = tq; plan.Hk = Hk; plan.grid = sm_count();
  plan.lists = 1;
  plan.offsets = seq_offsets;
  plan.n = n_seqs; plan.T = T; plan.causal = causal;
  plan.n_buckets = packed_buckets(T);
  plan.err = device_error_word();
  if (!plan.err) return CP_ERR_CUDA;
  if (!direct && launch_packed_plan(plan, stream) != cudaSuccess) return CP_ERR_CUDA;
  FwdParams p{};
  p.head = plan.list[0].head; p.items = plan.list[0].items;
  p.offsets = direct ? seq_offsets : nullptr;
  p.n_seqs = n_seqs;
  p.T = T; p.Hq = Hq; p.Hk = Hk; p.G = G; p.tq = tq; p.causal = causal;
  p.warp_tokens = 32 % G == 0 ? 32 / G : 0;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.parts = reinterpret_cast<float4*>(ws + sp.parts);
  p.done = plan.list[0].done;
  p.err = plan.err;
  p.timeout_ns = test_wait_limit_ns();
  p.fault_drop_k = test_fault_drop();
  const int grid = static_cast<int>(std::min<long long>(sm_count(), most_items + sp.slots * Hk));
  auto launch = [&](auto parts) {
    constexpr bool kParts = decltype(parts)::value;
    return d == 128 ? launch_packed_fwd<128, kParts>(a, p, grid, stream)
                    : launch_packed_fwd<64, kParts>(a, p, grid, stream);
  };
  const cudaError_t e = sp.slots > 0 ? launch(std::true_type()) : launch(std::false_type());
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // extern "C"
