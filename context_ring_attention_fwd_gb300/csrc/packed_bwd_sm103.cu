// Gradients of the attention over packed prompts with grouped heads (packed_fwd_sm103.cu), on
// sm_103a tensor cores (tcgen05), bf16.
//
// For L = sum(out * dout), row by row with P = exp(s - lse):
//   D = rowsum(dO * O);  dP = dO V^T;  dS = P * (dP - D);
//   dV = P^T dO;  dK = dS^T Q / sqrt(d);  dQ = dS K / sqrt(d)
// ("上下文並行（Context Parallelism, CP）", compassingai.com, section 反向傳播), the sums of a key
// head's dK and dV running over the G query heads that read it.  Two kernels, with the CTA's
// roles as attn_bwd_sm103.cu describes them:
//   kDKDV  a CTA owns a 128-key tile of one key head and walks the packed query tiles
//          (packed.cuh) that see it: G heads' rows are neighbours in the products' inner
//          dimension, so a shared head's gradients are summed in the accumulators.
//   kDQ    a CTA owns a packed query tile and walks the key tiles it sees.
// No gradient is summed by atomics.  A CTA that has all of a tile stores its gradients.  Key
// tiles of many queries may be cut into parts (packed_plan.cu): each leaves its fp32 sums of dV and
// dK in a slot (1024 d bytes, written and read again), counts itself by an atomic, and the last to
// end adds the tile's slots up in the parts' order.
//
// The seven products of a tile pair (two of them twice) are 7 / 5 of the formulas' operations:
// one kernel for all five would add dQ up over CTAs, by atomics in the order of arrival or through
// memory.  Bound by shared memory beside the tensor pipe: S^T and dP^T read both operands there at
// its full rate (128 bytes a clock), and the copies, dV's and dK's tiles and the constants come on
// top, 2560 clocks a tile pair for 2048 of products in kDKDV.  kDQ's fixed operands are therefore
// in TMEM; kDKDV has no columns left for its.  Measured (16K tokens of 16/4 heads, d = 128, in the
// kernels): kDKDV 1450 us, 67 % of the tensor pipe, kDQ 970, 73 %; with S^T and dP^T in halves of
// 64 queries, two in flight, kDKDV took 1830, and with constants read by generic loads 1570.
// P and dS are rounded to bf16 for their products, as the ring's backward rounds them: 2.5e-3 to
// 3.0e-3 of the gradients against 64 bits (relative in the norm), 1.65e-3 of it the outputs' own.
//
// Rows that are not there (behind a sequence, behind tq G) may hold anything.  Where they are
// summed over - Q and dO in kDKDV, K in kDQ - they are zeroed in shared memory up to the next
// multiple of 16, where the product ends; P and dS of masked pairs are replaced by zeros, not
// multiplied.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "attn_common.cuh"
#include "internal.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace cpring {
namespace {

constexpr int kT = kTileRows;       // rows of every tile
constexpr int kThreads = 384;        // three warpgroups (warps 10, 11 idle)
constexpr int kLaunchRegs = 168;     // registers per thread at launch (checked by the build)
constexpr int kSoftmaxRegs = 200;    // softmax warpgroups after setmaxnreg.inc
constexpr int kControlRegs = 104;    // producer / MMA warpgroup after setmaxnreg.dec
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch's register pool");
constexpr int kSoftmaxThreads = 256;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

// Streamed tiles run in two rings of single-tile slots: X0 (K for kDQ, Q for
// kDKDV) and X1 (V or dO).  A step's K or Q is held until its dQ or dK is done, behind the next
// step's first product, V only until dP and dO until dV, so the first ring is one slot deeper.
template <int D, bool kDKDV>
struct BLayout {
  static constexpr int kTileBytes = kT * D * 2;
  static constexpr int kPanelBytes = kT * 128;   // 128 rows x 64 bf16 columns
  static constexpr int kPanels = D / 64;
  static constexpr int kX0Slots = 3;
  static constexpr int kX1Slots = 2;
  static constexpr int kF0 = 0;                  // fixed tiles
  static constexpr int kF1 = kTileBytes;
  static constexpr int kX0 = 2 * kTileBytes;
  static constexpr int kX1 = kX0 + kX0Slots * kTileBytes;
  // kDKDV: fp32 [128], -lse2 of two tiles, -D
  static constexpr int kVec = kX1 + kX1Slots * kTileBytes;
  static constexpr int kBar = kVec + (kDKDV ? 3 * kT * 4 : 0);
  static constexpr int kRingOff = kBar + 256;  // the item ring
  static constexpr int kBytes = kRingOff + 256;
  static constexpr int kAlloc = kBytes + 1024;
  __host__ __device__ static constexpr int x0(int slot) { return kX0 + slot * kTileBytes; }
  __host__ __device__ static constexpr int x1(int slot) { return kX1 + slot * kTileBytes; }
};

enum BBar : int {
  kFixFull = 0,
  kFixEmpty = 1,   // kDKDV: their last products are done; kDQ: they are in TMEM
  kX0Full = 2,     // + slot (3)
  kX1Full = 5,     // + slot (2)
  kX0Empty = 7,    // + slot (3)
  kX1Empty = 10,   // + slot (2)
  kSFull = 12,     // S of a step is in TMEM
  kDPFull = 13,    // dP
  kPReady = 14,    // kDKDV: + half: P^T of 64 queries written by all softmax threads
  kDSReady = 16,   // + half: dS of 64 streamed rows written
  kSRead = 18,     // kDQ: every softmax thread has read S of the step
  kAccFull = 19,   // the item's accumulators are final
  kVecFull = 20,   // kDKDV: + buffer: per-column lse of a query tile written
  kDFull = 22,     // the same of D
  kFixHeld = 23,   // kDQ: Q and dO of the item are in TMEM
  kDrain = 24,
  kJoin = 25,      // kDKDV: the softmax threads have stored a part's sums; then: know its rank
  kNumBars = 26
};
// TMEM: S, dP, the accumulators from 256 on; of kDQ also the fixed tiles, packed, from here on.
constexpr uint32_t kHeldQ = 384, kHeldG = 448;
constexpr int kTmemSlot = kNumBars * 8;
constexpr int kAbortSlot = kNumBars * 8 + 4;
constexpr int kRankSlot = kNumBars * 8 + 8;

struct BParams {
  int* head;            // the plan's list
  const int4* items;
  int T, n_seqs, Hq, Hk, G;
  int tq;               // tokens of a packed tile
  int causal;
  float scale_log2;     // log2(e) / sqrt(d)
  float scale;          // 1 / sqrt(d)
  const float* lse;     // [Hq, T], natural log
  const float* delta;   // [T, Hq]
  __nv_bfloat16* g0;    // dQ (kDQ) or dV (kDKDV)
  __nv_bfloat16* g1;    // dK (kDKDV)
  long long gs0[2], gs1[2];  // their strides: row, head
  int wide;             // the outputs start at multiples of 32 bytes
  float4* sums;         // kDKDV: [slot][Hk][dV, dK][d / 4][128] of the tiles in parts
  int* done;
  int* err;
  unsigned long long timeout_ns;
  int fault_drop;       // test hook: CTA 0 never loads its first streamed X0 tile
};

// An item: the sequence, the key head, the first token of the fixed tile and its tokens, and
// the streamed tiles [x_lo, x_hi].
struct BItem {
  int row0, len, hk;
  int t0, tokens;
  int x_lo, x_hi;
  int slot, part, parts;  // kDKDV: of a tile in parts, the part's slot, its index, their number
};
template <bool kDKDV>
__device__ __forceinline__ void decode_bitem(const BParams& p, const PackedEntry& x, BItem& it) {
  const int4 e = x.e;
  it.hk = x.hk;
  it.row0 = e.x;
  it.len = e.y;
  const int tile = kDKDV ? kT : p.tq;
  it.t0 = e.z * tile;
  it.tokens = min(tile, it.len - it.t0);
  if (kDKDV) {  // query tiles that see a key of the tile
    it.x_lo = p.causal ? it.t0 / p.tq : 0;
    it.x_hi = (it.len - 1) / p.tq;
    it.slot = (e.w & 0xffff) - 1;
    it.part = 0;
    it.parts = 1;
    if (e.w != 0) {
      const int chunk = p.head[2];
      it.part = e.w >> 16;
      it.parts = (it.x_hi - it.x_lo) / chunk + 1;
      it.x_lo += it.part * chunk;
      it.x_hi = min(it.x_hi, it.x_lo + chunk - 1);
    }
  } else {      // key tiles seen by a row of the tile
    it.x_lo = 0;
    it.x_hi = ((p.causal ? it.t0 + it.tokens : it.len) - 1) / kT;
  }
}

// The columns [lo, hi] of 32 as bits, and 32 columns (fp32, and packed in bf16) with the others
// zeroed: what masked pairs of a query and a key hold is replaced, whatever it is.
__device__ __forceinline__ uint32_t seen_columns(int lo, int hi) {
  const uint32_t below = hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1u;
  return lo <= 0 ? below : lo > 31 ? 0u : below & (0xffffffffu << lo);
}
__device__ __forceinline__ void keep_columns(uint32_t (&v)[32], uint32_t (&pk)[16],
                                             uint32_t columns) {
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!(columns >> x & 1u)) v[x] = 0u;
#pragma unroll
  for (int x = 0; x < 16; ++x)
    pk[x] = ptx::pack_bf16(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1]));
}

// The 32 columns at `at` of `parts` parts, `step` apart, added in their order.  Bound by latency:
// the loads of kAtOnce parts are under way at a time.
__device__ __forceinline__ void sum_parts(uint32_t (&sum)[32], const float4* at, int parts,
                                          size_t step) {
  constexpr int kAtOnce = 6;
#pragma unroll
  for (int c = 0; c < 8; c += 4) {
    float4 s[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) s[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int j = 0; j < parts; j += kAtOnce) {
      float4 f[kAtOnce][4];
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          f[y][x] = j + y < parts ? load_cg(at + (j + y) * step + (c + x) * kT)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < kAtOnce; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[x].x += f[y][x].x;
          s[x].y += f[y][x].y;
          s[x].z += f[y][x].z;
          s[x].w += f[y][x].w;
        }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      sum[4 * (c + x)] = __float_as_uint(s[x].x);
      sum[4 * (c + x) + 1] = __float_as_uint(s[x].y);
      sum[4 * (c + x) + 2] = __float_as_uint(s[x].z);
      sum[4 * (c + x) + 3] = __float_as_uint(s[x].w);
    }
  }
}

// Shared memory by its address: through a pointer that was aligned as an integer these would be
// generic, which take more of the bandwidth that the products' operands need.
__device__ __forceinline__ float4 load_floats(uint32_t at) {
  float4 f;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
               : "r"(at));
  return f;
}
__device__ __forceinline__ void store_float(uint32_t at, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}

// 32 bytes of a row, whole sectors where the outputs lie so.  (Measured, in two halves of 16 /
// whole, us a call: 10 prompts of up to 2000 tokens, 32/8 heads, 288 / 279; 6 of up to 200, 16/4,
// 26.3 / 25.1.  Wider rows by way of shared memory would need some, and there is none left.)
__device__ __forceinline__ void store_32(uint4* to, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int D, bool kDKDV>
__global__ void __launch_bounds__(kThreads, 1)
    packed_bwd_kernel(const __grid_constant__ CUtensorMap tm_f0,
                         const __grid_constant__ CUtensorMap tm_f1,
                         const __grid_constant__ CUtensorMap tm_x0,
                         const __grid_constant__ CUtensorMap tm_x1, const BParams p) {
  using Lay = BLayout<D, kDKDV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t bars = sbase + Lay::kBar;
  auto bar = [&](int idx) -> uint32_t { return bars + 8u * static_cast<uint32_t>(idx); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kBar + kTmemSlot);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Lay::kBar + kAbortSlot);
  volatile int* rank = reinterpret_cast<volatile int*>(smem + Lay::kBar + kRankSlot);
  const PackedRing ring{
      sbase + Lay::kRingOff,
      reinterpret_cast<volatile int(*)[8]>(smem + Lay::kRingOff + 2 * kRing * 8)};
  // the ring's index of the item whose fixed tiles the producer is loading, for the MMA warp
  volatile int* fix_item =
      reinterpret_cast<volatile int*>(smem + Lay::kRingOff + 2 * kRing * 8 + kRing * 32);

  // (by a shuffle: the compiler then knows it, and what follows from it, as the warp's)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ptx::mbar_init(bar(kFixFull), 1);
    ptx::mbar_init(bar(kFixEmpty), kDKDV ? 1 : kSoftmaxThreads + 1);  // and the MMA warp
    for (int s = 0; s < Lay::kX0Slots; ++s) {
      ptx::mbar_init(bar(kX0Full + s), 1);
      ptx::mbar_init(bar(kX0Empty + s), 1);
    }
    for (int s = 0; s < Lay::kX1Slots; ++s) {
      ptx::mbar_init(bar(kX1Full + s), 1);
      ptx::mbar_init(bar(kX1Empty + s), 1);
    }
    ptx::mbar_init(bar(kSFull), 1);
    ptx::mbar_init(bar(kDPFull), 1);
    for (int h = 0; h < 2; ++h) {
      ptx::mbar_init(bar(kPReady + h), kSoftmaxThreads);
      ptx::mbar_init(bar(kDSReady + h), kSoftmaxThreads);
      ptx::mbar_init(bar(kVecFull + h), kT);
    }
    ptx::mbar_init(bar(kDFull), kT);
    ptx::mbar_init(bar(kSRead), kSoftmaxThreads);
    ptx::mbar_init(bar(kFixHeld), kSoftmaxThreads);
    ptx::mbar_init(bar(kAccFull), 1);
    ptx::mbar_init(bar(kJoin), kSoftmaxThreads);
    ptx::mbar_init(bar(kDrain), 1);
    ring.init(kSoftmaxThreads / 32);
    *abort_flag = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  const int packed_rows = p.tq * p.G;
  if (kDKDV && packed_rows < kT) {  // no load ever writes these rows of the streamed tiles
    for (int sl = warp; sl < Lay::kX0Slots + Lay::kX1Slots; sl += kThreads / 32)
      zero_rows<Lay::kPanels>(sbase + Lay::x0(sl), packed_rows, kT);  // (X1 lies behind X0)
    ptx::fence_proxy_async_shared();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  cudaGridDependencySynchronize();  // the plan and D
  const int x_tokens = kDKDV ? p.tq : kT;  // of a streamed tile
  const uint32_t packed_bytes = static_cast<uint32_t>(packed_rows) * 128u * Lay::kPanels;
  const uint32_t fix_bytes = kDKDV ? Lay::kTileBytes : packed_bytes;
  const uint32_t x_bytes = kDKDV ? packed_bytes : Lay::kTileBytes;

  if (warp >= kProducerWarp) {
   // the third warpgroup gives registers away, then splits into its roles
   ptx::setmaxnreg_dec<kControlRegs>();
   if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tm_f0);
      ptx::tma_prefetch_desc(&tm_f1);
      ptx::tma_prefetch_desc(&tm_x0);
      ptx::tma_prefetch_desc(&tm_x1);
      const PackedOrder order(p.head[0], p.Hk, gridDim.x);
      uint32_t x_iter = 0, fix_iter = 0;
      uint32_t armed0[3] = {0u, 0u, 0u}, armed1[2] = {0u, 0u};  // loads started per slot
      int ahead = 0;  // the claim of the CTA's next item
      bool dropped = false;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int w = k == 0 ? static_cast<int>(blockIdx.x) : ahead;
        const PackedEntry entry = order.at(p.items, w);
        if (!ring.put(static_cast<uint32_t>(k), entry, abort_flag, p)) { ok = false; break; }
        if (entry.hk < 0) break;
        BItem it;
        decode_bitem<kDKDV>(p, entry, it);
        const int fix_head = kDKDV ? it.hk : it.hk * p.G, x_head = kDKDV ? it.hk * p.G : it.hk;
        if (!wait1(bar(kFixEmpty), (fix_iter & 1u) ^ 1u, abort_flag, p)) { ok = false; break; }
        *fix_item = k;  // the MMA warp reads it once this phase of kFixFull completes
        ptx::mbar_arrive_expect_tx(bar(kFixFull), 2 * fix_bytes);
        for (int pn = 0; pn < Lay::kPanels; ++pn) {
          ptx::tma_load_3d(sbase + Lay::kF0 + pn * Lay::kPanelBytes, &tm_f0, bar(kFixFull),
                           pn * 64, fix_head, it.row0 + it.t0);
          ptx::tma_load_3d(sbase + Lay::kF1 + pn * Lay::kPanelBytes, &tm_f1, bar(kFixFull),
                           pn * 64, fix_head, it.row0 + it.t0);
        }
        ++fix_iter;
        for (int f = it.x_lo; f <= it.x_hi; ++f) {
          const uint32_t s0 = x_iter % Lay::kX0Slots, ph0 = (x_iter / Lay::kX0Slots) & 1u;
          const uint32_t s1 = x_iter % Lay::kX1Slots, ph1 = (x_iter / Lay::kX1Slots) & 1u;
          const int xs = it.row0 + f * x_tokens;
          if (!wait1(bar(kX0Empty + s0), ph0 ^ 1u, abort_flag, p)) { ok = false; break; }
          if (p.fault_drop && blockIdx.x == 0 && !dropped) {
            // Test hook: this tile is never loaded, so the MMA warp's
            // bounded wait for it runs out and the CTA takes its abort path.
            dropped = true;
          } else {
            ptx::mbar_arrive_expect_tx(bar(kX0Full + s0), x_bytes);
            for (int pn = 0; pn < Lay::kPanels; ++pn)
              ptx::tma_load_3d(sbase + Lay::x0(s0) + pn * Lay::kPanelBytes, &tm_x0,
                               bar(kX0Full + s0), pn * 64, x_head, xs);
            ++armed0[s0];
          }
          if (!wait1(bar(kX1Empty + s1), ph1 ^ 1u, abort_flag, p)) { ok = false; break; }
          ptx::mbar_arrive_expect_tx(bar(kX1Full + s1), x_bytes);
          for (int pn = 0; pn < Lay::kPanels; ++pn)
            ptx::tma_load_3d(sbase + Lay::x1(s1) + pn * Lay::kPanelBytes, &tm_x1,
                             bar(kX1Full + s1), pn * 64, x_head, xs);
          ++armed1[s1];
          ++x_iter;
        }
        // The next item is claimed once this one's loads are under way (see packed_fwd_sm103.cu).
        // Measured for kDKDV, so / when this item starts (us a call): 3000 + 200 + 100 tokens of
        // 32/8 heads 219 / 252, 6000 of 16/2 359 / 374, 8 x 2048 of 32/8 781 / 790, 9000 of 4/4
        // (d = 64) 179 / 186; but 20000 of 1/1 (d = 64) 257 / 237.
        ahead = packed_claim(p.head, gridDim.x);
      }
      // No more items: tell the MMA warp through the next phase of kFixFull.
      if (ok && wait1(bar(kFixEmpty), (fix_iter & 1u) ^ 1u, abort_flag, p)) {
        *fix_item = -1;
        ptx::mbar_arrive(bar(kFixFull));
        ++fix_iter;
      }
      // Let every copy this thread started land before the CTA can exit.
      if (fix_iter > 0) wait1(bar(kFixFull), (fix_iter - 1) & 1u, abort_flag, p, false);
      for (int s = 0; s < Lay::kX0Slots; ++s)
        if (armed0[s] > 0) wait1(bar(kX0Full + s), (armed0[s] - 1) & 1u, abort_flag, p, false);
      for (int s = 0; s < Lay::kX1Slots; ++s)
        if (armed1[s] > 0) wait1(bar(kX1Full + s), (armed1[s] - 1) & 1u, abort_flag, p, false);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs this loop with warp-uniform values; one lane picked
    // by elect.sync issues each MMA and commit (the warp-collective forms in
    // ptx.cuh), and every wait is the warp-uniform one.
    {
      constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kT, kT, false);   // N = streamed rows
      constexpr uint32_t kIdescG = ptx::idesc_bf16_f32(kT, D, true);     // N = d, B MN-major
      const uint64_t d_k = ptx::smem_desc_sw128(sbase, 16, 1024);                // K-major
      const uint64_t d_mn = ptx::smem_desc_sw128(sbase, Lay::kPanelBytes, 1024);  // MN-major
      const uint32_t tS = tmem_base, tdP = tmem_base + 128;
      const uint32_t tA0 = tmem_base + 256, tA1 = tmem_base + 256 + D;
      uint32_t x_iter = 0, fix_iter = 0;
      bool ok = true;
      // d = A B^T over the head dimension.  kDKDV: both tiles K-major in shared memory (a_off its
      // offset); kDQ: A's packed columns in TMEM from a_tmem on.
      auto issue_scores = [&](uint32_t d_tmem, int a_off, uint32_t a_tmem, int b_off) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint64_t step =
              static_cast<uint64_t>(((s >> 2) * Lay::kPanelBytes + (s & 3) * 32) >> 4);
          if constexpr (kDKDV)
            ptx::mma_ss_w(d_tmem, d_k + (a_off >> 4) + step, d_k + (b_off >> 4) + step, kIdescS,
                          s > 0 ? 1u : 0u);
          else
            ptx::mma_ts_w(d_tmem, tmem_base + a_tmem + s * 8u, d_k + (b_off >> 4) + step, kIdescS,
                          s > 0 ? 1u : 0u);
        }
      };
      // acc (+)= A B over 64 streamed rows: A = the two warpgroups' packed pieces (32 columns
      // apart), B = half of the streamed tile, at b_off, read MN-major (rows = K).
      auto issue_half = [&](uint32_t acc, uint32_t a_tmem, int b_off, bool first, int steps) {
        auto step = [&](int s) {
          const uint32_t a_col = static_cast<uint32_t>((s >> 1) * 32 + (s & 1) * 8);
          ptx::mma_ts_w(acc, a_tmem + a_col, d_mn + (b_off >> 4) + static_cast<uint64_t>(s * 128),
                      kIdescG, (first && s == 0) ? 0u : 1u);
        };
        if (steps >= 4) {  // without a test between the products
#pragma unroll
          for (int s = 0; s < 4; ++s) step(s);
        } else {
#pragma unroll 1
          for (int s = 0; s < steps; ++s) step(s);
        }
      };
      uint32_t n = 0, n_two = 0;  // steps issued so far (all items), those of two halves
      for (;;) {
        // The producer publishes each item with its fixed tiles' load (and
        // the end of the work with a plain arrival), so this warp needs no
        // wait beyond the one for those tiles.
        if (!wait_warp(bar(kFixFull), fix_iter & 1u, abort_flag, p)) { ok = false; break; }
        ++fix_iter;
        const int k = *fix_item;
        if (k < 0) break;
        if (!kDKDV) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(kFixEmpty));
          if (!wait_warp(bar(kFixHeld), (fix_iter - 1) & 1u, abort_flag, p)) { ok = false; break; }
        }
        BItem it;
        decode_bitem<kDKDV>(p, ring.read(static_cast<uint32_t>(k)), it);
        ptx::tc_fence_after();
        // rows of the last streamed tile: keys, or tokens times heads
        const int x_left = it.len - it.x_hi * x_tokens;
        const int last_rows = kDKDV ? min(x_left, p.tq) * p.G : min(x_left, kT);
        // (a tile of all tq tokens ends in rows that are zero: the product may run over them)
        const bool ragged = kDKDV ? x_left < p.tq : last_rows < kT;
        const int last_steps = ragged ? (last_rows + 15) / 16 : kT / 16;
        const int last_zero = min(last_steps * 16, kDKDV ? packed_rows : kT);
        // A step's first product S; dV += P^T dO, when P^T is written; dQ += dS K or
        // dK += dS^T Q, when dS is.  S of the next step goes out when S has been read and, where
        // P^T lies in its place, dV is under way; dP of the next step behind dQ or dK, as dS lies
        // in dP's place.  So the softmax forms dS during S (and dV) and the next P during dQ or dK
        // and the next dP.  What is written in halves of 64 streamed rows enters its product so.
        // (Measured for kDQ, 16K tokens of 16/4 heads, in the kernel: 970 us, 73 % of the tensor
        // pipe; dS in a place of its own, so that dP need not wait for dQ, and dO for that in
        // shared memory: 1044.)
        // (The last tile's second half is left out where no row is in it.)
        auto loaded = [&](int full, int at, uint32_t round, bool zero) -> bool {
          if (!wait_warp(bar(full), round & 1u, abort_flag, p)) return false;
          ptx::tc_fence_after();
          if (zero) {
            zero_rows<Lay::kPanels>(sbase + at, last_rows, last_zero);
            ptx::fence_proxy_async_shared();
            __syncwarp();
          }
          return true;
        };
        const bool zero_last = ragged && last_rows < last_zero;
        auto issue_s = [&](uint32_t x, bool last) -> bool {
          const uint32_t s0 = x % Lay::kX0Slots;
          if (!loaded(kX0Full + s0, Lay::x0(s0), x / Lay::kX0Slots, last && zero_last))
            return false;
          issue_scores(tS, Lay::kF0, kHeldQ, Lay::x0(s0));
          ptx::mma_commit_w(bar(kSFull));
          return true;
        };
        auto issue_dp = [&](uint32_t x, bool last) -> bool {
          const uint32_t s1 = x % Lay::kX1Slots;
          if (!loaded(kX1Full + s1, Lay::x1(s1), x / Lay::kX1Slots, kDKDV && last && zero_last))
            return false;
          issue_scores(tdP, Lay::kF1, kHeldG, Lay::x1(s1));
          ptx::mma_commit_w(bar(kDPFull));
          if (!kDKDV) ptx::mma_commit_w(bar(kX1Empty + s1));
          return true;
        };
        if (!kDKDV && n > 0 && !wait_warp(bar(kSRead), (n - 1u) & 1u, abort_flag, p)) {
          ok = false;
          break;
        }
        if (!issue_s(x_iter, it.x_lo == it.x_hi) || !issue_dp(x_iter, it.x_lo == it.x_hi)) {
          ok = false;
          break;
        }
        for (int f = it.x_lo; f <= it.x_hi; ++f) {
          const bool first = f == it.x_lo, last = f == it.x_hi;
          const int steps = last ? last_steps : kT / 16;
          auto issue_g = [&](uint32_t acc, uint32_t a_tmem, int b_off, int ready) -> bool {
            if (!wait_warp(bar(ready), n & 1u, abort_flag, p)) return false;
            ptx::tc_fence_after();
            issue_half(acc, a_tmem, b_off, first, steps);
            if (steps <= 4) return true;
            if (!wait_warp(bar(ready + 1), n_two & 1u, abort_flag, p)) return false;
            ptx::tc_fence_after();
            issue_half(acc, a_tmem + 64u, b_off + 64 * 128, false, steps - 4);
            return true;
          };
          const uint32_t s0 = x_iter % Lay::kX0Slots, s1 = x_iter % Lay::kX1Slots;
          if constexpr (kDKDV) {
            if (last) ptx::mma_commit_w(bar(kFixEmpty));  // every S^T and dP^T is under way
            if (!issue_g(tA0, tS, Lay::x1(s1), kPReady)) { ok = false; break; }
            ptx::mma_commit_w(bar(kX1Empty + s1));
          } else {
            if (!last && !wait_warp(bar(kSRead), n & 1u, abort_flag, p)) { ok = false; break; }
          }
          if (!last && !issue_s(x_iter + 1, f + 1 == it.x_hi)) { ok = false; break; }
          if (!issue_g(kDKDV ? tA1 : tA0, tdP, Lay::x0(s0), kDSReady)) { ok = false; break; }
          ptx::mma_commit_w(bar(kX0Empty + s0));
          if (!last && !issue_dp(x_iter + 1, f + 1 == it.x_hi)) { ok = false; break; }
          ++n;
          if (steps > 4) ++n_two;
          ++x_iter;
        }
        if (!ok) break;
        ptx::mma_commit_w(bar(kAccFull));
      }
      // Wait until every MMA this warp issued has finished.
      ptx::mma_commit_w(bar(kDrain));
      wait_warp(bar(kDrain), 0u, abort_flag, p, false);
    }
   }
  } else {
    ptx::setmaxnreg_inc<kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    const int wg = warp >> 2;        // this warpgroup has 32 columns of each half
    const int wq = warp & 3;         // TMEM lane quarter
    const int row_in_tile = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem_base + lane_off;
    const uint32_t tdP = tS + 128;
    const uint32_t tA0 = tS + 256, tA1 = tS + 256 + D;
    const float sc = p.scale_log2;
    // token and head of a packed tile's row: this thread's in kDQ; in kDKDV that of the column
    // whose constants it loads
    const int packed_row = kDKDV ? static_cast<int>(threadIdx.x) : row_in_tile;
    const int my_token = packed_row / p.G, my_head = packed_row - my_token * p.G;
    uint32_t s_cnt = 0, item_cnt = 0, join_cnt = 0;
    bool ok = true;
    // lse and D as loaded (arithmetic on them would wait for them): kDQ: of this thread's row;
    // kDKDV: of its row of the next streamed tile.  Rows behind that tile's last: P = 2^-inf = 0
    // where the scores are finite.
    float lse_next = 0.f, d_next = 0.f;
    auto load_constants = [&](const BItem& it, int token, bool there, float lse_else) {
      lse_next = lse_else;
      d_next = 0.f;
      if (there) {
        const size_t q = static_cast<size_t>(it.row0) + token;
        const int h = it.hk * p.G + my_head;
        lse_next = __ldg(p.lse + static_cast<size_t>(h) * p.T + q);
        d_next = p.delta[q * p.Hq + h];
      }
    };
    auto load_columns = [&](const BItem& it, int f) {
      const int t = f * x_tokens + my_token;
      load_constants(it, t, threadIdx.x < kT && f <= it.x_hi && my_token < p.tq && t < it.len,
                     INFINITY);
    };
    // kDQ: the k-th item, and what its start waits for: its rows' constants, and Q (by the first
    // warpgroup) and dO (by the second) in TMEM, from where the products take them without
    // reading shared memory again.  Of the item before every product but its last dQ is done.
    PackedEntry entry{make_int4(0, 0, 0, 0), -1};
    auto prepare = [&](uint32_t k) -> bool {
      if (!ring.get(k, entry, abort_flag, p)) return false;
      if (entry.hk < 0) return true;
      BItem it;
      decode_bitem<kDKDV>(p, entry, it);
      load_constants(it, it.t0 + my_token, my_token < it.tokens, 0.f);
      if (!wait_warp(bar(kFixFull), k & 1u, abort_flag, p)) return false;
      const uint32_t row = sbase + (wg ? Lay::kF1 : Lay::kF0) + row_in_tile * 128;
#pragma unroll
      for (int pn = 0; pn < Lay::kPanels; ++pn) {
        uint32_t x[32];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[4 * c]), "=r"(x[4 * c + 1]), "=r"(x[4 * c + 2]),
                         "=r"(x[4 * c + 3])
                       : "r"(row + pn * Lay::kPanelBytes + ((c ^ (row_in_tile & 7)) << 4)));
        ptx::tmem_st32(tS + (wg ? kHeldG : kHeldQ) + pn * 32, x);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(bar(kFixHeld));
      ptx::mbar_arrive(bar(kFixEmpty));
      return true;
    };
    if constexpr (!kDKDV) ok = prepare(0);
    for (uint32_t k = 0; ok; ++k) {
      if constexpr (kDKDV) {
        if (!ring.get(k, entry, abort_flag, p)) { ok = false; break; }
      } else {
        entry = PackedRing::uniform(entry);
      }
      if (entry.hk < 0) break;
      BItem it;
      decode_bitem<kDKDV>(p, entry, it);
      // This thread's row: a key, or a token and a head.  One that is not stored sees
      // everything, so that it does not hold its warp to the masked pass.
      const int row_token = kDKDV ? row_in_tile : my_token;
      const bool row_valid = row_token < it.tokens;
      const int token = it.t0 + row_token;
      const size_t row = static_cast<size_t>(it.row0) + token;
      const int head = kDKDV ? it.hk : it.hk * p.G + my_head;
      const int seen = !row_valid ? INT_MAX / 2 : p.causal ? token + 1 : it.len;  // kDQ: keys
      const int from = kDKDV && row_valid && p.causal ? token : 0;  // kDKDV: the first query
      const float lse2_r = lse_next * kLog2e, d_r = d_next;  // kDQ
      if (kDKDV) load_columns(it, it.x_lo);
      for (int f = it.x_lo; f <= it.x_hi; ++f) {
        const int xs = f * x_tokens;  // first streamed token
        const int tokens = min(x_tokens, it.len - xs);
        // The columns that the row sees.  A packed tile of all its tokens ends in zero rows of Q
        // and dO, which need no mask (their P is 0 by their constant).
        const int c_lo = kDKDV ? max(from - xs, 0) * p.G : 0;
        const int c_hi = kDKDV ? (tokens == x_tokens ? kT : tokens * p.G) - 1 : seen - xs - 1;
        const bool two = kDKDV ? f != it.x_hi || tokens == x_tokens || tokens * p.G > 64
                               : tokens > 64;  // halves
        uint32_t columns[2];
        bool masked[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c0 = 64 * h + 32 * wg;
          masked[h] = __any_sync(0xffffffffu, c_lo > c0 || c_hi < c0 + 31);
          columns[h] = seen_columns(c_lo - c0, c_hi - c0);
        }
        // Per-column constants of a streamed query tile, shared by all rows: warps 0-3 write
        // them, having loaded them a tile ahead.  Nobody still reads the buffers: a thread that
        // has seen S of step n - 1 (this loop's last turn) knows that all have formed P of
        // step n - 2, one that has seen dP of step n that all have formed dS of step n - 1.
        const uint32_t lse_vec = sbase + Lay::kVec + (s_cnt & 1u) * kT * 4;
        const uint32_t d_vec = sbase + Lay::kVec + 2 * kT * 4;
        float d_of_row = 0.f;
        if (kDKDV) {
          d_of_row = -d_next;
          if (threadIdx.x < kT) {
            store_float(lse_vec + threadIdx.x * 4, -lse_next * kLog2e);
            ptx::mbar_arrive(bar(kVecFull + (s_cnt & 1u)));
            load_columns(it, f + 1);
          }
          if (!wait_warp(bar(kVecFull + (s_cnt & 1u)), (s_cnt >> 1) & 1u, abort_flag, p)) {
            ok = false;
            break;
          }
        }
        if (!wait_warp(bar(kSFull), s_cnt & 1u, abort_flag, p)) { ok = false; break; }
        ptx::tc_fence_after();
        uint32_t pv[2][32];  // S, then P, which stays in fp32 for dS
        ptx::tmem_ld32(tS + 32 * wg, pv[0]);
        ptx::tmem_ld32(tS + 32 * wg + 64, pv[1]);
        ptx::tmem_wait_ld();
        ptx::reg_fence(pv[0]);
        ptx::reg_fence(pv[1]);
        if (!kDKDV) {
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar(kSRead));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) break;
          const int c0 = 64 * h + 32 * wg;
          uint32_t pk[16];
#pragma unroll
          for (int x4 = 0; x4 < 8; ++x4) {  // paired fp32
            const float4 nl =
                kDKDV ? load_floats(lse_vec + (c0 + 4 * x4) * 4)
                      : make_float4(-lse2_r, -lse2_r, -lse2_r, -lse2_r);
            const float nla[4] = {nl.x, nl.y, nl.z, nl.w};
#pragma unroll
            for (int hx = 0; hx < 2; ++hx) {
              const int x = 2 * x4 + hx;
              float e0, e1;
              ptx::fma_f32x2(e0, e1, __uint_as_float(pv[h][2 * x]),
                             __uint_as_float(pv[h][2 * x + 1]), sc, sc, nla[2 * hx],
                             nla[2 * hx + 1]);
              e0 = ptx::ex2(e0);
              e1 = ptx::ex2(e1);
              pv[h][2 * x] = __float_as_uint(e0);
              pv[h][2 * x + 1] = __float_as_uint(e1);
              if (kDKDV) pk[x] = ptx::pack_bf16(e0, e1);
            }
          }
          if constexpr (kDKDV) {
            if (masked[h]) keep_columns(pv[h], pk, columns[h]);
            ptx::tmem_st16(tS + c0, pk);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(kPReady + h));
          }
        }
        // dS = P (dP - D)
        if (!wait_warp(bar(kDPFull), s_cnt & 1u, abort_flag, p)) { ok = false; break; }
        ptx::tc_fence_after();
        if (kDKDV && threadIdx.x < kT) {
          store_float(d_vec + threadIdx.x * 4, d_of_row);
          ptx::mbar_arrive(bar(kDFull));
        }
        uint32_t dv[2][32];
        ptx::tmem_ld32(tdP + 32 * wg, dv[0]);
        ptx::tmem_ld32(tdP + 32 * wg + 64, dv[1]);
        if (kDKDV && !wait_warp(bar(kDFull), s_cnt & 1u, abort_flag, p)) { ok = false; break; }
        ptx::tmem_wait_ld();
        ptx::reg_fence(dv[0]);
        ptx::reg_fence(dv[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) break;
          const int c0 = 64 * h + 32 * wg;
          uint32_t pk[16];
#pragma unroll
          for (int x4 = 0; x4 < 8; ++x4) {
            const float4 nd = kDKDV ? load_floats(d_vec + (c0 + 4 * x4) * 4)
                                    : make_float4(-d_r, -d_r, -d_r, -d_r);
            const float nda[4] = {nd.x, nd.y, nd.z, nd.w};
#pragma unroll
            for (int hx = 0; hx < 2; ++hx) {
              const int x = 2 * x4 + hx;
              float g0, g1;
              ptx::fma_f32x2(g0, g1, __uint_as_float(dv[h][2 * x]),
                             __uint_as_float(dv[h][2 * x + 1]), 1.f, 1.f, nda[2 * hx],
                             nda[2 * hx + 1]);
              ptx::fma_f32x2(g0, g1, __uint_as_float(pv[h][2 * x]),
                             __uint_as_float(pv[h][2 * x + 1]), g0, g1, 0.f, 0.f);
              dv[h][2 * x] = __float_as_uint(g0);
              dv[h][2 * x + 1] = __float_as_uint(g1);
              pk[x] = ptx::pack_bf16(g0, g1);
            }
          }
          if (masked[h]) keep_columns(dv[h], pk, columns[h]);
          ptx::tmem_st16(tdP + c0, pk);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar(kDSReady + h));
        }
        ++s_cnt;
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if constexpr (!kDKDV) {  // before the wait, so that the next item's first products start
        if (!prepare(k + 1)) { ok = false; break; }
      }
      if (!wait_warp(bar(kAccFull), item_cnt & 1u, abort_flag, p)) { ok = false; break; }
      ++item_cnt;
      ptx::tc_fence_after();
      // A part of a tile: its sums go to its slot, and the last of the tile's parts to end adds
      // them all up, in the parts' order whoever is last.  A thread reads what threads of its
      // own place wrote.
      const bool in_parts = kDKDV && it.parts > 1;
      const float4* first_part = nullptr;
      if (in_parts) {
        constexpr int kSlot = 2 * (D / 4) * kT;  // float4 of a slot
        float4* const to = p.sums + (static_cast<size_t>(it.slot) * p.Hk + it.hk) * kSlot;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int ch = 0; ch < D / 64; ++ch) {
            const int c0 = wg * (D / 2) + ch * 32;
            uint32_t ov[32];
            ptx::tmem_ld32((a == 0 ? tA0 : tA1) + c0, ov);
            ptx::tmem_wait_ld();
            ptx::reg_fence(ov);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              to[(a * (D / 4) + c0 / 4 + x) * kT + row_in_tile] =
                  make_float4(__uint_as_float(ov[4 * x]), __uint_as_float(ov[4 * x + 1]),
                              __uint_as_float(ov[4 * x + 2]), __uint_as_float(ov[4 * x + 3]));
          }
        __threadfence();
        ptx::mbar_arrive(bar(kJoin));
        if (!wait_warp(bar(kJoin), join_cnt & 1u, abort_flag, p)) { ok = false; break; }
        ++join_cnt;
        if (threadIdx.x == 0) {
          *rank = atomicAdd(p.done + (it.slot - it.part) * p.Hk + it.hk, 1);
          __threadfence();
        }
        ptx::mbar_arrive(bar(kJoin));
        if (!wait_warp(bar(kJoin), join_cnt & 1u, abort_flag, p)) { ok = false; break; }
        ++join_cnt;
        if (*rank != it.parts - 1) continue;
        __threadfence();
        first_part = p.sums + (static_cast<size_t>(it.slot - it.part) * p.Hk + it.hk) * kSlot;
      }
#pragma unroll
      for (int a = 0; a < (kDKDV ? 2 : 1); ++a) {
        const uint32_t tacc = a == 0 ? tA0 : tA1;
        __nv_bfloat16* g = a == 0 ? p.g0 : p.g1;
        const float fac = (kDKDV && a == 0) ? 1.f : p.scale;  // dV unscaled; dK, dQ / sqrt(d)
        const long long(&gs)[2] = a == 0 ? p.gs0 : p.gs1;
        uint4* dst = reinterpret_cast<uint4*>(g + static_cast<long long>(row) * gs[0] + head * gs[1]);
#pragma unroll
        for (int ch = 0; ch < D / 64; ++ch) {
          const int c0 = wg * (D / 2) + ch * 32;
          uint32_t ov[32];
          if (kDKDV && in_parts) {
            sum_parts(ov, first_part + (a * (D / 4) + c0 / 4) * kT + row_in_tile, it.parts,
                      static_cast<size_t>(p.Hk) * 2 * (D / 4) * kT);
          } else {
            ptx::tmem_ld32(tacc + c0, ov);
            ptx::tmem_wait_ld();
            ptx::reg_fence(ov);
          }
          if (row_valid) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t w[8];
#pragma unroll
              for (int y = 0; y < 8; ++y)
                w[y] = ptx::pack_bf16(__uint_as_float(ov[16 * x + 2 * y]) * fac,
                                      __uint_as_float(ov[16 * x + 2 * y + 1]) * fac);
              store_32(dst + c0 / 8 + 2 * x, w, p.wide);
            }
          }
        }
      }
    }
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

template <int D, bool kDKDV>
cudaError_t launch_packed_bwd(const PackedArgs& a, BParams p, const PackedList& list,
                              const void* dout, bool dependent, cudaStream_t stream) {
  using Lay = BLayout<D, kDKDV>;
  static_assert(Lay::kAlloc <= 232448, "shared memory budget");
  static_assert(Lay::kX0Slots <= 3 && Lay::kX1Slots == 2, "barrier slots");
  const auto kern = packed_bwd_kernel<D, kDKDV>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), Lay::kAlloc);
  if (e != cudaSuccess) return e;
  // kDQ: fixed (Q, dO), streamed (K, V); kDKDV: fixed (K, V), streamed (Q, dO)
  CUtensorMap mq, mg, mk, mv;
  if (!packed_map(&mq, a.q, a.T, a.Hq, D, a.qs[0], a.qs[1], p.G, p.tq) ||
      !packed_map(&mg, dout, a.T, a.Hq, D, static_cast<long long>(a.Hq) * D, D, p.G, p.tq) ||
      !packed_map(&mk, a.k, a.T, a.Hk, D, a.ks[0], a.ks[1], 1, kT) ||
      !packed_map(&mv, a.v, a.T, a.Hk, D, a.vs[0], a.vs[1], 1, kT))
    return cudaErrorInvalidValue;
  p.head = list.head;
  p.items = list.items;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(
      sm_count(), (packed_items(a.T, p.n_seqs, list.tokens) + list.slots) * a.Hk)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Lay::kAlloc;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = dependent ? 1 : 0;
  count_launch(0);
  return kDKDV ? cudaLaunchKernelEx(&cfg, kern, mk, mv, mq, mg, p)
               : cudaLaunchKernelEx(&cfg, kern, mq, mg, mk, mv, p);
}

// dK/dV on `stream`, dQ beside it, whose CTAs take the SMs that the last dK/dV items leave idle;
// both after the plan.  (A captured dK/dV waits for the whole plan before it starts.)
template <int D>
cudaError_t launch_packed_pair(const PackedArgs& a, const BParams& dkdv, const BParams& dq,
                               const PackedPlan& plan, const void* dout, cudaStream_t stream) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(stream, &status);
  if (e != cudaSuccess) return e;
  const bool early = status == cudaStreamCaptureStatusNone;
  return launch_beside(
      stream,
      [&](cudaStream_t s) {
        return launch_packed_bwd<D, true>(a, dkdv, plan.list[0], dout, early, s);
      },
      [&](cudaStream_t s) {
        return launch_packed_bwd<D, false>(a, dq, plan.list[1], dout, false, s);
      });
}

// Byte offsets of the workspace's parts: the lists of key tiles (with its parts) and of query
// tiles, D, and the sums of key tiles in parts.
struct Space {
  int slots;  // of a key head
  long long keys, queries, delta, done, sums, total;
  Space(int T, int n, int Hq, int Hk, int d) {
    const int tq = kT / (Hq / Hk);
    // All parts of a call, none shorter than the shortest, and no more than kMaxParts, which the
    // plan keeps to; none where every tile stays whole.
    const long long most = (T - 1) / tq + 1 <= kLeastCut
                               ? 0
                               : packed_items(T, n, kT) * (T / tq / kLeastPart + 1);
    slots = packed_slots(most, kMaxParts, Hk);
    const auto up = [](long long x) { return (x + 255) / 256 * 256; };
    keys = 0;
    queries = up(packed_list_bytes(T, n, kT) + 16LL * slots);
    delta = queries + up(packed_list_bytes(T, n, tq));
    done = delta + up(4LL * T * Hq);
    sums = done + up(4LL * slots * Hk);
    total = sums + 8LL * slots * Hk * kT * d;
  }
};

}  // namespace
}  // namespace cpring

extern "C" {

int64_t cp_packed_attn_bwd_workspace_bytes(int T, int n_seqs, int Hq, int Hk, int d) {
  if (cpring::check_packed(T, n_seqs, Hq, Hk, d, 0) != CP_OK) return -1;
  return cpring::Space(T, n_seqs, Hq, Hk, d).total;
}

cp_status cp_packed_attn_bwd(const void* q, const int64_t* q_strides, const void* k,
                             const int64_t* k_strides, const void* v, const int64_t* v_strides,
                             const void* out, const float* lse, const void* dout,
                             const int32_t* seq_offsets, void* dq, const int64_t* dq_strides,
                             void* dk, const int64_t* dk_strides, void* dv,
                             const int64_t* dv_strides, int T, int n_seqs, int Hq, int Hk, int d,
                             int causal, void* workspace, int64_t workspace_bytes,
                             cudaStream_t stream) {
  cpring::TraceRange trace_("cp_packed_attn_bwd");
  using namespace cpring;
  if (!q || !k || !v || !out || !lse || !dout || !seq_offsets || !dq || !dk || !dv || !workspace)
    return CP_ERR_NULL;
  const cp_status st = check_packed(T, n_seqs, Hq, Hk, d, causal);
  if (st != CP_OK) return st;
  PackedArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.T = T; a.Hq = Hq; a.Hk = Hk;
  int64_t dqs[2], dks[2], dvs[2];
  for (const void* t : {q, k, v, out, dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv)})
    if (!aligned(t, 16)) return CP_ERR_ALIGN;
  if (!aligned(lse, 4) || !aligned(seq_offsets, 4) || !aligned(workspace, 256) ||
      !packed_strides(q_strides, Hq, d, a.qs) || !packed_strides(k_strides, Hk, d, a.ks) ||
      !packed_strides(v_strides, Hk, d, a.vs) || !packed_strides(dq_strides, Hq, d, dqs) ||
      !packed_strides(dk_strides, Hk, d, dks) || !packed_strides(dv_strides, Hk, d, dvs))
    return CP_ERR_ALIGN;
  const int G = Hq / Hk, tq = kTileRows / G;
  const Space sp(T, n_seqs, Hq, Hk, d);
  if (workspace_bytes < sp.total) return CP_ERR_BUFFER;
  if (device_cc() != 103) return CP_ERR_DEVICE;
  char* const ws = static_cast<char*>(workspace);
  PackedPlan plan{};
  plan.list[0] = packed_list(ws + sp.keys, T, n_seqs, kT, true, sp.slots);
  plan.list[0].done = reinterpret_cast<int*>(ws + sp.done);
  plan.list[0].n_done = sp.slots * Hk;
  plan.tq = tq; plan.Hk = Hk; plan.grid = sm_count();
  plan.list[1] = packed_list(ws + sp.queries, T, n_seqs, tq, false);
  plan.lists = 2;
  plan.offsets = seq_offsets;
  plan.n = n_seqs; plan.T = T; plan.causal = causal;
  plan.n_buckets = packed_buckets(T);
  plan.out = out; plan.dout = dout;
  plan.delta = reinterpret_cast<float*>(ws + sp.delta);
  plan.rows = static_cast<long long>(T) * Hq;
  plan.d = d;
  plan.err = device_error_word();
  if (!plan.err) return CP_ERR_CUDA;
  if (launch_packed_plan(plan, stream) != cudaSuccess) return CP_ERR_CUDA;
  BParams p{};
  p.T = T; p.n_seqs = n_seqs; p.Hq = Hq; p.Hk = Hk; p.G = G; p.tq = tq; p.causal = causal;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  p.lse = lse;
  p.delta = plan.delta;
  p.err = plan.err;
  p.timeout_ns = test_wait_limit_ns();
  p.fault_drop = test_fault_drop();
  p.sums = reinterpret_cast<float4*>(ws + sp.sums);
  p.done = plan.list[0].done;
  p.wide = aligned(dk, 32) && aligned(dv, 32);
  BParams pq = p;
  pq.wide = aligned(dq, 32);
  p.g0 = static_cast<__nv_bfloat16*>(dv);
  p.g1 = static_cast<__nv_bfloat16*>(dk);
  pq.g0 = static_cast<__nv_bfloat16*>(dq);
  for (int i = 0; i < 2; ++i) {
    p.gs0[i] = dvs[i];
    p.gs1[i] = dks[i];
    pq.gs0[i] = dqs[i];
  }
  const cudaError_t e = d == 128 ? launch_packed_pair<128>(a, p, pq, plan, dout, stream)
                                 : launch_packed_pair<64>(a, p, pq, plan, dout, stream);
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // extern "C"
