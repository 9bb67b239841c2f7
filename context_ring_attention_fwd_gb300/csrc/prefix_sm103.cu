// The shared prefix of the decode attention on tcgen05: partial states of the
// whole batch's rows over the prefix's keys.
//
// With B n_q G rows per key head, reading K and V once leaves the two
// products, 4 d FLOP per row and key: from about 300 rows on the tensor pipe
// bounds it, HBM below.  An item is 256 rows of one key head (two tiles of 128,
// the TMEM lanes) over the prefix's 128-key tiles; the items' tiles are laid end
// to end and every CTA of one per SM takes an equal stretch, so any number of
// rows and heads fills the GPU.  An item cut between CTAs leaves its parts in
// their slots; the join of paged_decode.cu merges them with the sequences' own
// keys.
//
// Roles (384 threads): two softmax warpgroups, one per row tile, a thread a
// row; in the third, one warp that issues the MMAs and three that load K and V.
//   S_t = Q_t K^T (both in shared memory), P_t back into S's TMEM columns in two
//   halves of 64 keys, O_t += P_t V (P from TMEM), as in the ring forward
//   (attn_sm103.cu); no row max on the way: P is taken against a reference
//   that moves only when a row runs 2^64 (fp16 P: 2^8) past it.
//
// Loading.  Pages whose size is a multiple of 8 come by TMA, one box per page
// (or per largest power of two of rows that divides it) and 128-byte panel;
// the rows of V behind the prefix's end are zeroed, whatever the page holds there.  Other
// page sizes and stride orders that no tensor map describes come by cp.async
// with the swizzle written by address, each thread ordering its finished copies
// before the tensor core's reads with a proxy fence.  (us a call with pages of 64
// and of 60 tokens, by TMA and by cp.async: 64 sequences under a 32K prefix, bf16, 56 and
// 68; 512 rows under 128K, E4M3, 216 and 315.)
//
// P in 16 bits, as the ring forward holds it, while l sums it in fp32.  In bf16 that
// costs as much as the output's own rounding: against 64 bits, relative in the norm,
// 2.3e-3 for 64 sequences under a 32K prefix, where the output's rounding alone makes
// 1.66e-3.  A second product for what the rounding leaves, as the 16-row items of
// paged_decode.cu take, would put 1024 more tensor clocks on a pair of tiles that has
// 2048, in a kernel that the tensor pipe bounds; those items are bound by HBM.
//
// Bound by shared memory and the tensor pipe alike: of a pair of 128 x 128 tiles, the
// products take 2048 clocks, and the operands that they read (A and B of S, V) and the
// copies that fill them 2048 clocks at 128 bytes each; a pair takes about 2900.  512 rows
// x 8 heads under a 128K prefix: 192 us, 1430 TFLOP/s.
//
// E4M3, d = 128, by TMA: K's codes are the operand themselves.  A bf16 q has 8
// significant bits, so it is the sum of two E4M3 values (exactly, but for
// entries 2^-10 below the row's largest, which lose at most 2^-18 of that), and
// S = q_hi K^T + q_lo K^T takes as long as one product in 16 bits.  P would
// lose what lies 2^-18 below its reference in such a pair, so P V runs in fp16:
// two warps widen V's codes on their way from a ring of 16 KB to the operand
// tile, and P is held times 2^7, which leaves it 2^31 of range.  The
// cp.async path widens K and V both and holds Q in fp16, exactly but for entries 2^-28
// below the row's largest: the page size decides which of the two a call gets, and either
// is within the 2^-17 of sum |q k| that a score's fp32 sum may be off by.
//
// Registers: launched at 168 per thread; the third warpgroup drops to 104 and
// the softmax warpgroups rise to 200 (the build checks the launch's count).  A
// fourth warp per scheduler would cap the launch at 128.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "attn_common.cuh"
#include "internal.h"
#include "paged_decode.h"
#include "ptx.cuh"

namespace cpring {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp0 = 9;     // by TMA: this warp loads, the next two widen V's codes
constexpr int kLoadWarps = 3;
constexpr int kLaunchRegs = 168;  // registers per thread at launch (checked by the build)
constexpr int kSoftmaxRegs = 200;
constexpr int kControlRegs = 104;
static_assert(2 * kSoftmaxRegs + kControlRegs <= 3 * kLaunchRegs,
              "the register split fits the launch");
constexpr int kStages = 2;
constexpr int kTmemCols = 512;  // S0 | S1 | O0 | O1

template <int D, bool kE4M3, bool kTma>
struct Lay {
  static constexpr bool kCodesK = kE4M3 && kTma;     // S from E4M3 operands
  static constexpr int kPanel = 128 * 128;           // 128 rows x 128 bytes
  static constexpr int kPanels = D / 64;
  static constexpr int kTile = kPanels * kPanel;     // 128 rows of D 16-bit values
  static constexpr int kKTile = kCodesK ? kPanel : kTile;
  static constexpr int kKStages = kCodesK ? 4 : 2;
  static constexpr int kQ = 0;                       // + row tile (codes: hi, then lo)
  static constexpr int kK = kQ + 2 * kTile;
  static constexpr int kV = kK + kKStages * kKTile;
  static constexpr int kCodes = kV + kStages * kTile;
  static constexpr int kCodeTile = kE4M3 ? 128 * D : 0;
  static constexpr int kBars = kCodes + 2 * kCodeTile;
  static constexpr int kBytes = kBars + 256;
  static constexpr int kAlloc = kBytes + 1024;       // room to align the base to 1024 B
  static_assert(kAlloc <= 232448, "shared memory budget");
  static_assert(!kCodesK || D == 128, "one 128-byte panel of codes");
};

enum Bar : int {
  kQFull = 0,     // + row tile
  kKFull = 2,     // + stage (4)
  kDone = 6,      // + parity of the tile: its S and the P V before it done
  kVFull = 10,    // + stage
  kSFull = 14,    // + row tile
  kPReady = 16,   // + row tile: keys 0-63 of P stored
  kPReadyB = 18,  // + row tile: keys 64-127
  kOFull = 20,    // + row tile: the segment's last P V done
  kCFull = 22,    // + buffer: V's codes landed
  kCEmpty = 24,   // + buffer: widened
  kTail = 26,     // V of the prefix's last tile landed
  kDrain = 27,
  kNumBars = 28
};
constexpr int kTmemSlot = kNumBars * 8;
constexpr int kAbortSlot = kTmemSlot + 4;
constexpr int kBadSlot = kTmemSlot + 8;
static_assert(kBadSlot + 4 <= 256, "the barrier block");

// A CTA's next segment: tiles [t0, t1) of an item.
struct Segment {
  int hk, row0, rows, t0, t1;
  bool whole;
};

template <bool kE4M3>
__device__ __forceinline__ bool segment_at(const DecodeParams& p, unsigned& w, unsigned w_end,
                                           Segment& s) {
  const unsigned n = static_cast<unsigned>(p.prefix_tiles) + kItemCost;
  do {
    if (w >= w_end) return false;
    const unsigned item = w / n;
    const unsigned u0 = w - item * n;
    const unsigned u1 = min(n, u0 + (w_end - w));
    s.t0 = tile_of_unit(u0);
    s.t1 = tile_of_unit(u1);
    int t;
    prefix_item_at<kE4M3>(p, static_cast<int>(item), s.hk, t);
    s.row0 = t * kPrefixRows;
    w += u1 - u0;
  } while (s.t0 >= s.t1);
  s.rows = min(kPrefixRows, p.B * p.R - s.row0);
  s.whole = s.t0 == 0 && s.t1 == p.prefix_tiles;
  return true;
}

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((static_cast<uint32_t>(N) >> 3) << 17) |
         ((static_cast<uint32_t>(M) >> 4) << 24);
}

// Four E4M3 codes to four fp16 values, exactly.
__device__ __forceinline__ void widen(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  lo = half2_of_codes(codes & 0xffffu);
  hi = half2_of_codes(codes >> 16);
}

// Four bf16 values times `up` as E4M3 codes and the codes of what those leave.
// fp16 holds the scaled values, and the differences, exactly.
__device__ __forceinline__ void split4(uint32_t x01, uint32_t x23, float up, uint32_t& hi,
                                       uint32_t& lo) {
  uint32_t z[2], back[2];
  uint16_t h[2], r[2];
  z[0] = pack_f16(__uint_as_float(x01 << 16) * up, __uint_as_float(x01 & 0xffff0000u) * up);
  z[1] = pack_f16(__uint_as_float(x23 << 16) * up, __uint_as_float(x23 & 0xffff0000u) * up);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h[i]) : "r"(z[i]));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back[i]) : "h"(h[i]));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(z[i]) : "r"(back[i]));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r[i]) : "r"(z[i]));
  }
  hi = static_cast<uint32_t>(h[0]) | (static_cast<uint32_t>(h[1]) << 16);
  lo = static_cast<uint32_t>(r[0]) | (static_cast<uint32_t>(r[1]) << 16);
}

// Stores 16 widened codes: chunks 2 c and 2 c + 1 of a row of the operand tile.
// Lanes of a row's second panel write theirs in the other order, so that
// eight lanes meet eight banks.
__device__ __forceinline__ void store_widened(uint32_t tile, int panel, int row, int c,
                                              const uint32_t (&h)[8]) {
  const int c0 = 2 * c;
  const uint32_t line = tile + (c0 >> 3) * panel + row * 128;
  const bool swap = c & 4;
  const uint32_t a0 = line + ((((c0 + swap) & 7) ^ (row & 7)) << 4);
  const uint32_t a1 = line + ((((c0 + !swap) & 7) ^ (row & 7)) << 4);
  ptx::st_shared_v4(a0, swap ? h[4] : h[0], swap ? h[5] : h[1], swap ? h[6] : h[2],
                    swap ? h[7] : h[3]);
  ptx::st_shared_v4(a1, swap ? h[0] : h[4], swap ? h[1] : h[5], swap ? h[2] : h[6],
                    swap ? h[3] : h[7]);
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Largest of the scores of keys 64 * half .. + 63.
__device__ __forceinline__ float half_max(const uint32_t (&sv)[4][32], int half) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    m0 = max3f(m0, __uint_as_float(sv[2 * half][x]), __uint_as_float(sv[2 * half][x + 1]));
    m1 = max3f(m1, __uint_as_float(sv[2 * half + 1][x]), __uint_as_float(sv[2 * half + 1][x + 1]));
  }
  return fmaxf(m0, m1);
}
// P = 2^(s sc - base) of those keys as 16-bit pairs, and its sum.
template <bool kF16>
__device__ __forceinline__ float exp_half(const uint32_t (&sv)[4][32], int half, float sc,
                                          float base, uint32_t (&pk)[32]) {
  uint64_t acc = 0;  // two fp32 sums
#pragma unroll
  for (int cc = 0; cc < 2; ++cc)
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      float e0, e1;
      asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
          "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
          "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
          : "=f"(e0), "=f"(e1)
          : "f"(__uint_as_float(sv[2 * half + cc][2 * x])),
            "f"(__uint_as_float(sv[2 * half + cc][2 * x + 1])), "f"(sc), "f"(-base));
      const float p0 = ptx::ex2(e0), p1 = ptx::ex2(e1);
      asm("{\n\t.reg .b64 rp;\n\tmov.b64 rp, {%1, %2};\n\tadd.rn.f32x2 %0, %0, rp;\n\t}"
          : "+l"(acc)
          : "f"(p0), "f"(p1));
      pk[cc * 16 + x] = kF16 ? pack_f16(p0, p1) : ptx::pack_bf16(p0, p1);
    }
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(acc));
  return lo + hi;
}

// Eight TMEM columns of this lane times alpha.
__device__ __forceinline__ void scale8(uint32_t taddr, float alpha) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
  ptx::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    asm volatile("" : "+r"(r[i]));
    r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
  }
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::
                   "r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
               "r"(r[7])
               : "memory");
}

// How the TMA path finds a tile's rows: boxes of `rows` rows; the tensor maps'
// dimensions are (d, head, token, page), or (d, token, head, page).
struct Boxes {
  int rows, token_first;
};

template <int D, bool kE4M3, bool kTma>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const DecodeParams p, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const Boxes boxes) {
  using L = Lay<D, kE4M3, kTma>;
  constexpr float kShift = kE4M3 ? 7.f : 0.f;           // P is held times 2^kShift
  constexpr float kGuardLog2 = kE4M3 ? 8.f : 64.f;      // P / 2^kShift stays below 2^kGuardLog2
  constexpr float kGuard = kE4M3 ? 32768.f : 18446744073709551616.f;  // 2^(kGuardLog2 + kShift)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBars + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* const abort_flag =
      reinterpret_cast<volatile uint32_t*>(smem + L::kBars + kAbortSlot);
  volatile uint32_t* const bad_flag =
      reinterpret_cast<volatile uint32_t*>(smem + L::kBars + kBadSlot);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBars + kTmemSlot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int t = 0; t < L::kKStages; ++t) {
      ptx::mbar_init(bar(kKFull + t), kTma ? 1 : 32 * kLoadWarps);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(bar(kQFull + t), 128);
      ptx::mbar_init(bar(kVFull + t), !kTma ? 32 * kLoadWarps : kE4M3 ? 64 : 1);
      ptx::mbar_init(bar(kDone + t), 1);
      ptx::mbar_init(bar(kCFull + t), 1);
      ptx::mbar_init(bar(kCEmpty + t), 64);
      ptx::mbar_init(bar(kSFull + t), 1);
      ptx::mbar_init(bar(kPReady + t), 128);
      ptx::mbar_init(bar(kPReadyB + t), 128);
      ptx::mbar_init(bar(kOFull + t), 1);
    }
    ptx::mbar_init(bar(kTail), 1);
    ptx::mbar_init(bar(kDrain), 1);
    *abort_flag = 0u;
    *bad_flag = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  cudaTriggerProgrammaticLaunchCompletion();  // the join's blocks may line up
  const unsigned W = (static_cast<unsigned>(p.prefix_tiles) + kItemCost) *
                     static_cast<unsigned>(p.Hk * p.prefix_row_tiles);
  unsigned w = stretch(blockIdx.x, W, gridDim.x);
  const unsigned w_end = stretch(blockIdx.x + 1, W, gridDim.x);
  // Test hook: the launch's first K tile never comes.
  const bool drop = p.fault_drop_k && blockIdx.x == holder(kItemCost, W, gridDim.x);
  Segment s;

  // The CTA's tile n is done (two barriers in turn: the next tile of the same
  // parity needs what waits for this one).
  auto tile_done = [&](uint32_t n) {
    return wait_warp(bar(kDone + (n & 1u)), (n >> 1) & 1u, abort_flag, p);
  };
  if (warp >= kMmaWarp) ptx::setmaxnreg_dec<kControlRegs>();  // the whole third warpgroup
  if (kTma && warp == kLoadWarp0) {
    // ------------------------------------------------------------ K and V by TMA
    // Lane j brings box j of a tile: its page was looked up a tile earlier.
    const int n_boxes = kPrefixKeys / boxes.rows;
    int page = -1, slot = 0;
    auto look_up = [&](int tile, int t1) {
      const int key = tile * kPrefixKeys + lane * boxes.rows;
      page = -1;
      if (tile < t1 && lane < n_boxes && key < p.P) {
        const int at = key / p.page_size;
        slot = key - at * p.page_size;
        page = __ldg(p.prefix_pages + at);
        if (page < 0 || page >= p.n_pages) {
          page = -1;
          *bad_flag = 1u;
        }
      }
    };
    constexpr int kBoxCols = kE4M3 ? 128 : 64;  // of a panel
    constexpr int kBoxPanels = kE4M3 ? 1 : L::kPanels;
    auto bring = [&](const CUtensorMap* map, int hk, uint32_t dst, uint32_t full) {
      const unsigned have = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0)
        ptx::mbar_arrive_expect_tx(
            full, static_cast<uint32_t>(__popc(have) * boxes.rows * 128 * kBoxPanels));
      __syncwarp();
      if (page >= 0) {
#pragma unroll
        for (int pn = 0; pn < kBoxPanels; ++pn)
          ptx::tma_load_4d(dst + pn * L::kPanel + lane * boxes.rows * 128, map, full,
                           pn * kBoxCols, boxes.token_first ? slot : hk,
                           boxes.token_first ? hk : slot, page);
      }
      __syncwarp();
    };
    uint32_t n = 0, nk = 0, nv = 0, tails = 0;  // tiles; K, V and last tiles under way
    bool ok = true;
    while (ok && segment_at<kE4M3>(p, w, w_end, s)) {
      look_up(s.t0, s.t1);
      for (int f = s.t0; f < s.t1; ++f, ++n) {
        // K of tile n may be overwritten once tile n - kKStages is done, V once
        // tile n - 1 is (its P V comes one tile later): the wait for V of the
        // tile before has covered K's (for codes, the wait for their buffer: the
        // widening warps had waited for tile n - 4).
        const uint32_t ks = n % L::kKStages;
        const uint32_t vs = n & 1u;
        if (!(drop && n == 0)) {
          bring(&map_k, s.hk, sbase + L::kK + ks * L::kKTile, bar(kKFull + ks));
          nk = n + 1;
        }
        if (kE4M3 ? n >= 2 && !wait_warp(bar(kCEmpty + vs), ((n >> 1) - 1) & 1u, abort_flag, p)
                  : n >= 1 && !tile_done(n - 1)) {
          ok = false;
          break;
        }
        const int left = p.P - f * kPrefixKeys;
        if (kE4M3) {
          bring(&map_v, s.hk, sbase + L::kCodes + vs * L::kCodeTile, bar(kCFull + vs));
        } else if (left >= kPrefixKeys) {
          bring(&map_v, s.hk, sbase + L::kV + vs * L::kTile, bar(kVFull + vs));
        } else {
          // The prefix ends in this tile: what its last page holds behind the
          // end, and what no box brought, becomes zeros.
          const uint32_t dst = sbase + L::kV + vs * L::kTile;
          bring(&map_v, s.hk, dst, bar(kTail));
          ++tails;
          if (!wait_warp(bar(kTail), (tails - 1) & 1u, abort_flag, p)) {
            ok = false;
            break;
          }
          for (int x = left * 8 * L::kPanels + lane; x < kPrefixKeys * 8 * L::kPanels; x += 32) {
            const int row = x / (8 * L::kPanels), c = x % (8 * L::kPanels);
            ptx::st_shared_v4(dst + (c >> 3) * L::kPanel + row * 128 + (c & 7) * 16, 0, 0, 0, 0);
          }
          ptx::fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(kVFull + vs));
        }
        nv = n + 1;
        look_up(f + 1, s.t1);
      }
    }
    // Every copy under way lands before the CTA can exit: the last use of
    // each buffer, of which the dropped tile was none.
    for (uint32_t x = 0; x < L::kKStages; ++x) {
      const uint32_t uses = nk > x ? (nk - x + L::kKStages - 1) / L::kKStages : 0u;
      if (uses > 0 && !(drop && x == 0))
        wait_warp(bar(kKFull + x), (uses - 1) & 1u, abort_flag, p, false);
    }
    for (uint32_t x = 0; x < 2; ++x) {
      const uint32_t uses = nv > x ? (nv - x + 1) / 2 : 0u;
      if (uses > 0)
        wait_warp(bar((kE4M3 ? kCFull : kVFull) + x), (uses - 1) & 1u, abort_flag, p, false);
    }
    if (tails > 0) wait_warp(bar(kTail), (tails - 1) & 1u, abort_flag, p, false);
  } else if (kTma && warp > kLoadWarp0) {
    // ------------------------------------------------------------ V's codes to fp16
    if (kE4M3) {
      const int tid = (warp - kLoadWarp0 - 1) * 32 + lane;
      constexpr int kRowChunks = D / 16;
      bool ok = true;
      uint32_t n = 0;
      while (ok && segment_at<kE4M3>(p, w, w_end, s)) {
        for (int f = s.t0; f < s.t1; ++f, ++n) {
          const uint32_t vs = n & 1u;
          if (!wait_warp(bar(kCFull + vs), (n >> 1) & 1u, abort_flag, p) ||
              (n >= 1 && !tile_done(n - 1))) {
            ok = false;
            break;
          }
          const int left = p.P - f * kPrefixKeys;
          const uint32_t src = sbase + L::kCodes + vs * L::kCodeTile;
          const uint32_t dst = sbase + L::kV + vs * L::kTile;
          const int chunk = tid % kRowChunks;
#pragma unroll 8
          for (int i = 0; i < 128 * kRowChunks / 64; ++i) {
            const int row = (i * 64 + tid) / kRowChunks;
            uint32_t u[4], h[8];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                         : "r"(src + (i * 64 + tid) * 16));
#pragma unroll
            for (int e = 0; e < 4; ++e) widen(row < left ? u[e] : 0u, h[2 * e], h[2 * e + 1]);
            store_widened(dst, L::kPanel, row, chunk, h);
          }
          ptx::fence_proxy_async_shared();
          ptx::mbar_arrive(bar(kVFull + vs));
          ptx::mbar_arrive(bar(kCEmpty + vs));
        }
      }
    }
  } else if (!kTma && warp >= kLoadWarp0) {
    // ------------------------------------------------------------ K and V by cp.async
    // One copy of a warp moves kRowsPer rows; the tile's copies are dealt to
    // the three warps in turn.
    const int lw = warp - kLoadWarp0;
    constexpr int kRowChunks = D * (kE4M3 ? 1 : 2) / 16;  // 16-byte chunks of a cached row
    constexpr int kRowsPer = 32 / kRowChunks;
    constexpr int kAll = kPrefixKeys / kRowsPer;          // copies of a tile
    constexpr int kCopies = (kAll + kLoadWarps - 1) / kLoadWarps;
    static_assert(kCopies * kRowsPer <= 64, "two rows' places per lane");
    const int chunk = lane % kRowChunks, sub = lane / kRowChunks;
    bool ok = true;
    // The places of the warp's rows of the next tile to be copied: its q-th
    // row (of copy q / kRowsPer) in lane q % 32.
    int page[2] = {-1, -1}, slot[2] = {0, 0};
    auto look_up = [&](int tile, int t1) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = j * 32 + lane;
        const int row = (lw + kLoadWarps * (q / kRowsPer)) * kRowsPer + q % kRowsPer;
        const int key = tile * kPrefixKeys + row;
        page[j] = -1;
        if (tile < t1 && row < kPrefixKeys && key < p.P) {
          const int at = key / p.page_size;
          slot[j] = key - at * p.page_size;
          page[j] = __ldg(p.prefix_pages + at);
          if (page[j] < 0 || page[j] >= p.n_pages) {
            page[j] = -1;
            *bad_flag = 1u;
          }
        }
      }
    };
    auto copy = [&](int x, int hk, uint32_t dst) {  // the warp's rows of K (0) or V (1)
      long long off[2];
      unsigned held[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        off[j] = page[j] >= 0 ? page[j] * p.cs[x][0] + slot[j] * p.cs[x][1] + hk * p.cs[x][2] : 0;
        held[j] = __ballot_sync(0xffffffffu, page[j] >= 0);
      }
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int q = i * kRowsPer + sub;
        constexpr int kHalf = 32 / kRowsPer;  // copies whose rows' places are the lanes' first
        const long long o = __shfl_sync(0xffffffffu, off[i >= kHalf], q & 31);
        const unsigned have = held[i >= kHalf] >> (q & 31) & 1u;
        const int c = lw + kLoadWarps * i;    // of the tile's copies
        if (c < kAll) {
          const int row = c * kRowsPer + sub;
          const uint32_t at = kE4M3 ? dst + (c * 32 + lane) * 16
                                    : dst + (chunk >> 3) * L::kPanel + row * 128 +
                                          (((chunk & 7) ^ (row & 7)) << 4);
          cp_async16(at, p.cache[x] + o + chunk * 16, have ? 16 : 0);
        }
      }
    };
    // Step n copies K (n even) or V (n odd) of the CTA's tile n / 2, into stage
    // (n / 2) % 2, which V finds free once tile n / 2 - 1 is done and K then has been.
    auto full = [&](unsigned n) { return bar((n & 1 ? kVFull : kKFull) + ((n >> 1) & 1)); };
    auto buffer = [&](unsigned n) {
      return sbase + (n & 1 ? L::kV : L::kK) + ((n >> 1) & 1) * L::kTile;
    };
    auto announce = [&](unsigned n) {
      ptx::fence_proxy_async_shared();
      if (!(drop && n == 0)) ptx::mbar_arrive(full(n));
    };
    if (!kE4M3) {
      unsigned n = 0, told = 0;  // steps copied, steps announced
      while (ok && segment_at<kE4M3>(p, w, w_end, s)) {
        look_up(s.t0, s.t1);
        for (int f = s.t0; ok && f < s.t1; ++f) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const unsigned tile = n >> 1;
            if (x == 1 && tile >= 1 &&
                !__all_sync(0xffffffffu, ptx::mbar_try_wait(bar(kDone + ((tile - 1) & 1)),
                                                            ((tile - 1) >> 1) & 1u))) {
              // The buffer is still in use: announce what is under way first.
              cp_wait<0>();
              for (; told < n; ++told) announce(told);
              if (!tile_done(tile - 1)) {
                ok = false;
                break;
              }
            }
            copy(x, s.hk, buffer(n));
            if (x == 1) look_up(f + 1, s.t1);
            cp_commit();
            ++n;
            if (n - told > 2) {
              cp_wait<2>();
              announce(told++);
            }
          }
        }
      }
      cp_wait<0>();
      if (ok)
        for (; told < n; ++told) announce(told);
    } else {
      // Codes run two steps ahead through their own ring; a thread widens
      // the chunks that it copied itself.
      unsigned w2 = w;           // the copying walk
      Segment c{};
      int cf = 0;
      unsigned copied = 0;
      bool more = segment_at<kE4M3>(p, w2, w_end, c);
      if (more) {
        cf = c.t0;
        look_up(cf, c.t1);
      }
      auto copy_step = [&]() {
        if (more) {
          const int x = copied & 1;
          copy(x, c.hk, sbase + L::kCodes + x * L::kCodeTile);
          ++copied;
          if (x == 1 && ++cf == c.t1) {
            more = segment_at<kE4M3>(p, w2, w_end, c);
            if (more) {
              cf = c.t0;
              look_up(cf, c.t1);
            }
          } else if (x == 1) {
            look_up(cf, c.t1);
          }
        }
        cp_commit();
      };
      copy_step();
      copy_step();
      unsigned n = 0;
      while (ok && segment_at<kE4M3>(p, w, w_end, s)) {
        for (int f = s.t0; ok && f < s.t1; ++f) {
#pragma unroll
          for (int x = 0; x < 2; ++x, ++n) {
            if (x == 1 && n >= 2 && !tile_done((n >> 1) - 1)) {
              ok = false;
              break;
            }
            cp_wait<1>();
            const uint32_t src = sbase + L::kCodes + x * L::kCodeTile + lane * 16;
            const uint32_t dst = buffer(n);
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
              const int c = lw + kLoadWarps * i;
              if (c >= kAll) break;
              const int row = c * kRowsPer + sub;
              uint32_t u[4], h[8];
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                           : "r"(src + c * 32 * 16));
#pragma unroll
              for (int e = 0; e < 4; ++e) widen(u[e], h[2 * e], h[2 * e + 1]);
              store_widened(dst, L::kPanel, row, chunk, h);
            }
            announce(n);
            copy_step();
          }
        }
      }
      cp_wait<0>();
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMAs
    constexpr uint32_t kIdescQK = L::kCodesK ? ptx::idesc_e4m3_f32(128, 128)
                                  : kE4M3    ? idesc_f16_f32(128, 128, false)
                                             : ptx::idesc_bf16_f32(128, 128, false);
    constexpr uint32_t kIdescPV =
        kE4M3 ? idesc_f16_f32(128, D, true) : ptx::idesc_bf16_f32(128, D, true);
    const uint64_t d_qk = ptx::smem_desc_sw128(sbase, 16, 1024);
    const uint64_t d_v = ptx::smem_desc_sw128(sbase, L::kPanel, 1024);
    uint32_t p_cnt[2] = {0, 0};
    uint32_t it = 0, segs0 = 0, segs1 = 0;
    bool ok = true;
    auto issue_s = [&](int t, uint32_t st) {
      const uint64_t dq = d_qk + ((L::kQ + t * L::kTile) >> 4);
      const uint64_t dk = d_qk + ((L::kK + st * L::kKTile) >> 4);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t step = static_cast<uint64_t>(((k >> 2) * L::kPanel + (k & 3) * 32) >> 4);
        if (L::kCodesK)  // k-steps of 32 codes: the low parts' panel follows the high ones'
          ptx::mma_ss_f8_w(tmem + t * 128, dq + step,
                           dk + static_cast<uint64_t>(((k & 3) * 32) >> 4), kIdescQK,
                           k > 0 ? 1u : 0u);
        else
          ptx::mma_ss_w(tmem + t * 128, dq + step, dk + step, kIdescQK, k > 0 ? 1u : 0u);
      }
      ptx::mma_commit_w(bar(kSFull + t));
    };
    while (ok && segment_at<kE4M3>(p, w, w_end, s)) {
      const bool two = s.rows > 128;
      if (!wait_warp(bar(kQFull), segs0++ & 1u, abort_flag, p)) { ok = false; break; }
      if (two && !wait_warp(bar(kQFull + 1), segs1++ & 1u, abort_flag, p)) { ok = false; break; }
      ptx::tc_fence_after();
      uint32_t prev_st = 0, prev_ph = 0;
      // O_t (+)= P_t V of the previous key tile, each half once its P is there.
      auto flush = [&](int t, bool first, bool last) -> bool {
        if (t == 0 && !wait_warp(bar(kVFull + prev_st), prev_ph, abort_flag, p)) return false;
        const uint64_t dv = d_v + ((L::kV + prev_st * L::kTile) >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait_warp(bar((half ? kPReadyB : kPReady) + t), p_cnt[t] & 1u, abort_flag, p))
            return false;
          ptx::tc_fence_after();
#pragma unroll
          for (int k = half * 4; k < half * 4 + 4; ++k)
            ptx::mma_ts_w(tmem + 256 + t * D, tmem + t * 128 + k * 8,
                          dv + static_cast<uint64_t>((k * 16 * 128) >> 4), kIdescPV,
                          (first && k == 0) ? 0u : 1u);
        }
        ++p_cnt[t];
        if (last) ptx::mma_commit_w(bar(kOFull + t));
        return true;
      };
      for (int f = s.t0; f < s.t1; ++f) {
        const uint32_t st = it & 1u, ph = (it >> 1) & 1u;  // V's
        const uint32_t kst = it % L::kKStages, kph = (it / L::kKStages) & 1u;
        if (f > s.t0 && !flush(0, f == s.t0 + 1, false)) { ok = false; break; }
        if (!wait_warp(bar(kKFull + kst), kph, abort_flag, p)) { ok = false; break; }
        ptx::tc_fence_after();
        issue_s(0, kst);
        if (two) {
          if (f > s.t0 && !flush(1, f == s.t0 + 1, false)) { ok = false; break; }
          issue_s(1, kst);
        }
        ptx::mma_commit_w(bar(kDone + st));
        prev_st = st;
        prev_ph = ph;
        ++it;
      }
      if (!ok) break;
      const bool only = s.t1 == s.t0 + 1;
      if (!flush(0, only, true) || (two && !flush(1, only, true))) { ok = false; break; }
    }
    ptx::mma_commit_w(bar(kDrain));
    wait_warp(bar(kDrain), 0u, abort_flag, p, false);
  } else {
    // ------------------------------------------------------------ softmax
    ptx::setmaxnreg_inc<kSoftmaxRegs>();
    const int t = warp >> 2;                    // row tile
    const int row_in_tile = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(t * 128);
    const uint32_t tO = tmem + lane_off + 256u + static_cast<uint32_t>(t * D);
    uint32_t s_cnt = 0, o_cnt = 0;
    bool ok = true;
    unsigned w_seg = w;
    while (segment_at<kE4M3>(p, w, w_end, s)) {
      if (t * 128 >= s.rows) { w_seg = w; continue; }
      float sc = p.scale;
      if (ok) {
        // ---- this warp's 32 rows of Q into the swizzled tile (every MMA on the
        // previous segment's has finished: its last P V was waited for).  D / 8
        // lanes read a row, kPer rows a step; all steps' loads are under way
        // before the first is used.
        constexpr int kRowLanes = D / 8, kPer = 32 / kRowLanes, kSteps = kRowLanes;
        const int c = lane % kRowLanes, sub = lane / kRowLanes;
        uint4 v[kSteps];
        {
          const int r = t * 128 + row_in_tile;  // this lane's own row of the item
          const RowOf row(p, 0, s.hk, s.row0 + min(r, s.rows - 1));
          const unsigned long long mine = reinterpret_cast<unsigned long long>(row.query(p));
          const unsigned there = __ballot_sync(0xffffffffu, r < s.rows);
#pragma unroll
          for (int x = 0; x < kSteps; ++x) {
            const int at = x * kPer + sub;
            const uint4* const src = reinterpret_cast<const uint4*>(
                __shfl_sync(0xffffffffu, mine, at));
            v[x] = (there >> at & 1u) ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
          }
        }
        const float desc = kE4M3 ? __ldg(p.descale[0] + s.hk) : 1.f;
        // Four steps a turn, the later ones moved down behind them: unrolled whole,
        // fetching this code took longer than running it.
#pragma unroll 1
        for (int x0 = 0; x0 < kSteps; x0 += 4) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = (warp & 3) * 32 + (x0 + x) * kPer + sub;  // of the tile
            uint32_t u[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
            float up = 1.f;
            if (kE4M3) {
              // magnitudes order like their bits, two to a comparison
              uint32_t big = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                asm("max.u16x2 %0, %0, %1;" : "+r"(big) : "r"(u[e] & 0x7fff7fffu));
#pragma unroll
              for (int o = 1; o < kRowLanes; o <<= 1)
                asm("max.u16x2 %0, %0, %1;"
                    : "+r"(big)
                    : "r"(__shfl_xor_sync(0xffffffffu, big, o)));
              const float top = __uint_as_float(max(big << 16, big & 0xffff0000u));
              float down;
              fp16_row_scale(top, up, down);
              if (L::kCodesK) {  // to [2^7, 2^8): the pair saturates at 448
                up *= 0x1p-7f;
                down *= 0x1p+7f;
                if (!(top < INFINITY)) down = NAN;  // nor has it an infinity
              }
              // the row's own thread keeps what undoes its scale
              const float its = __shfl_sync(0xffffffffu, down, (lane % kPer) * kRowLanes);
              if (lane / kPer == x0 + x) sc = p.scale * desc * its;
            }
            const uint32_t line = sbase + L::kQ + t * L::kTile + row * 128;
            if (L::kCodesK) {
              uint32_t hi[2], lo[2];
              split4(u[0], u[1], up, hi[0], lo[0]);
              split4(u[2], u[3], up, hi[1], lo[1]);
              const uint32_t at = line + (((c >> 1) ^ (row & 7)) << 4) + (c & 1) * 8;
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(hi[0]), "r"(hi[1])
                           : "memory");
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + L::kPanel), "r"(lo[0]),
                           "r"(lo[1])
                           : "memory");
            } else {
              if (kE4M3) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  u[e] = pack_f16(__uint_as_float(u[e] << 16) * up,
                                  __uint_as_float(u[e] & 0xffff0000u) * up);
              }
              ptx::st_shared_v4(line + (c >> 3) * L::kPanel + (((c & 7) ^ (row & 7)) << 4), u[0],
                                u[1], u[2], u[3]);
            }
          }
#pragma unroll
          for (int x = 0; x + 4 < kSteps; ++x) v[x] = v[x + 4];
        }
        ptx::fence_proxy_async_shared();
        ptx::mbar_arrive(bar(kQFull + t));
      }
      float m = -INFINITY, l = 0.f;
      const int first = s.t0, end = s.t1;
      for (int f = first; ok && f < end; ++f) {
        if (!wait_warp(bar(kSFull + t), s_cnt & 1u, abort_flag, p)) { ok = false; break; }
        ++s_cnt;
        ptx::tc_fence_after();
        uint32_t sv[4][32], pk[32];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) ptx::tmem_ld32(tS + ch * 32, sv[ch]);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) ptx::reg_fence(sv[ch]);
        const int left = p.P - f * kPrefixKeys;  // keys of this tile that exist
        if (left < kPrefixKeys) {
#pragma unroll
          for (int ch = 0; ch < 4; ++ch)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (ch * 32 + x >= left) sv[ch][x] = __float_as_uint(-INFINITY);
        }
        const float ref = m - kShift;
        bool in_range = false;
        if (f > first) {
          // P against the reference so far, its first half stored and signalled
          // before the second is computed, if neither runs past the guard.
          const float l1 = exp_half<kE4M3>(sv, 0, sc, ref, pk);
          in_range = (l1 <= kGuard) & (half_max(sv, 1) * sc <= m + kGuardLog2);
          if (__all_sync(0xffffffffu, in_range)) {
            ptx::tmem_st32(tS, pk);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(kPReady + t));
            l += l1 + exp_half<kE4M3>(sv, 1, sc, ref, pk);
            ptx::tmem_st32(tS + 32, pk);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(kPReadyB + t));
            continue;
          }
        }
        // A segment's first tile, or a row of this warp past the guard: such a
        // row's reference moves to this tile's maximum and O with it; the other
        // rows get what they had above.
        const float top = fmaxf(half_max(sv, 0), half_max(sv, 1)) * sc;
        const bool move = f == first || (!in_range && top > m);
        const float alpha = (f == first || !move) ? 1.f : ptx::ex2(m - top);
        if (move) m = top;
        // A row that has met scores of -inf alone keeps the reference -inf: its state is
        // empty, and no later tile is in range of it, so the first with a score sets it.
        const float base = (m == -INFINITY ? 0.f : m) - kShift;
        l *= alpha;
        if (f > first) {
          // O_t holds the sum up to the previous tile: the MMA warp issued
          // that P V before this tile's S, whose commit was waited for.
          // Eight columns at a time: the scores stay in registers.
#pragma unroll 1
          for (int ch = 0; ch < D / 8; ++ch) scale8(tO + ch * 8, alpha);
        }
        float sum = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          sum += exp_half<kE4M3>(sv, half, sc, base, pk);
          ptx::tmem_st32(tS + 32 * half, pk);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar((half ? kPReadyB : kPReady) + t));
        }
        l += sum;
      }
      // ---- the segment's part: O, its reference and its sum.  Where it goes is
      // worked out again, so that the loop above holds no registers for it.
      asm volatile("" : "+r"(w_seg));
      segment_at<kE4M3>(p, w_seg, w_end, s);
      const int r = t * 128 + row_in_tile;
      const bool valid = r < s.rows;
      if (ok && !wait_warp(bar(kOFull + t), o_cnt & 1u, abort_flag, p)) ok = false;
      ++o_cnt;
      ptx::tc_fence_after();
      const bool nan = !ok || *bad_flag != 0u;  // the part is marked, not left as it was
      long long at;
      float *to, *ml;
      if (s.whole) {
        const RowOf row(p, 0, s.hk, s.row0 + min(r, s.rows - 1));
        at = static_cast<long long>(p.B) * p.n_q * p.Hq + row.index(p);
        to = p.whole_o + at * D;
        ml = p.whole_ml + at * 2;
      } else {
        at = (static_cast<long long>(blockIdx.x) * 2 + (s.t0 == 0 ? 1 : 0)) * kPrefixRows + r;
        to = p.pslot_o + at * D;
        ml = p.pslot_ml + at * 2;
      }
      if (ok) {
        // Through this warp's rows of the Q tile, which nothing reads any more:
        // half a row per round and lane goes in, whole lines come out.
        const float vd = kE4M3 ? __ldg(p.descale[1] + s.hk) : 1.f;
        constexpr int kCols = 32 * L::kPanels;       // columns of a round
        constexpr int kLineChunks = kCols / 4;       // 16-byte chunks of a row's round
        const uint32_t mine = sbase + L::kQ + t * L::kTile + (warp & 3) * 32 * 128;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += kCols) {
#pragma unroll
          for (int pn = 0; pn < L::kPanels; ++pn) {
            uint32_t ov[32];
            ptx::tmem_ld32(tO + c0 + pn * 32, ov);
            ptx::tmem_wait_ld();
            ptx::reg_fence(ov);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              ptx::st_shared_v4(mine + pn * L::kPanel + lane * 128 + ((x ^ (lane & 7)) << 4),
                                __float_as_uint(__uint_as_float(ov[4 * x]) * vd),
                                __float_as_uint(__uint_as_float(ov[4 * x + 1]) * vd),
                                __float_as_uint(__uint_as_float(ov[4 * x + 2]) * vd),
                                __float_as_uint(__uint_as_float(ov[4 * x + 3]) * vd));
          }
          __syncwarp();
          constexpr int kRowsPer = 32 / kLineChunks;
          const int chunk = lane % kLineChunks;
#pragma unroll 4
          for (int i = 0; i < kLineChunks; ++i) {
            const int row = i * kRowsPer + lane / kLineChunks;
            float* const dst = reinterpret_cast<float*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), row));
            uint32_t u[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                         : "r"(mine + (chunk >> 3) * L::kPanel + row * 128 +
                               (((chunk & 7) ^ (row & 7)) << 4)));
            if (t * 128 + (warp & 3) * 32 + row < s.rows)
              *reinterpret_cast<uint4*>(dst + c0 + chunk * 4) = make_uint4(u[0], u[1], u[2], u[3]);
          }
          __syncwarp();
        }
        ptx::tc_fence_before();
      }
      if (valid) *reinterpret_cast<float2*>(ml) = make_float2(m - kShift, nan ? NAN : l);
    }
    if (threadIdx.x == 0 && *bad_flag != 0u) atomicOr(p.err, kErrCache);
  }

  // The join waits for this kernel alone, so this kernel ends after the one
  // before it (the sequences' own keys), next to which it runs.
  if (threadIdx.x == 0) cudaGridDependencySynchronize();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// K or V as (d, head, token, page) or (d, token, head, page), the smaller
// stride first; a box is one panel of `rows` tokens of a head.  False where the
// strides are not multiples of one another in that order.
bool make_page_map(CUtensorMap* m, const DecodeParams& p, int x, int d, bool e4m3, bool swizzled,
                   const Boxes& boxes) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t e = e4m3 ? 1 : 2;
  struct Dim { cuuint64_t n, stride; cuuint32_t box; };
  Dim dim[3] = {{static_cast<cuuint64_t>(p.Hk), static_cast<cuuint64_t>(p.cs[x][2]), 1},
                {static_cast<cuuint64_t>(p.page_size), static_cast<cuuint64_t>(p.cs[x][1]),
                 static_cast<cuuint32_t>(boxes.rows)},
                {static_cast<cuuint64_t>(p.n_pages), static_cast<cuuint64_t>(p.cs[x][0]), 1}};
  if (boxes.token_first) std::swap(dim[0], dim[1]);
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d)}, strides[3], inner = d * e;
  cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / e)};
  for (int i = 0; i < 3; ++i) {
    if (dim[i].n == 1) dim[i].stride = inner;  // never used
    if (dim[i].stride % inner != 0) return false;
    inner = strides[i] = dim[i].stride;
    dims[i + 1] = dim[i].n;
    box[i + 1] = dim[i].box;
  }
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<uint8_t*>(p.cache[x]), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kE4M3, bool kTma>
cudaError_t launch_t(const DecodeParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                     const Boxes& boxes, cudaStream_t stream) {
  using L = Lay<D, kE4M3, kTma>;
  const cudaError_t e = ensure_smem_limit(
      reinterpret_cast<const void*>(&prefix_attn_kernel<D, kE4M3, kTma>), L::kAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.prefix_grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  count_launch(0);
  return cudaLaunchKernelEx(&cfg, prefix_attn_kernel<D, kE4M3, kTma>, p, mk, mv, boxes);
}

}  // namespace

cudaError_t launch_prefix_attn(const DecodeParams& p, int d, bool e4m3, cudaStream_t stream) {
  CUtensorMap mk{}, mv{};
  Boxes boxes{p.page_size & -p.page_size, 0};
  boxes.rows = std::min(boxes.rows, kPrefixKeys);
  // TMA needs boxes of whole 8-row swizzle groups, one order of strides for K and V,
  // and a 128-byte panel of codes.
  const bool hnd = p.page_size > 1 && p.Hk > 1 && p.cs[0][1] < p.cs[0][2];
  boxes.token_first = hnd;
  const bool tma = boxes.rows >= 8 && !(e4m3 && d == 64) &&
                   make_page_map(&mk, p, 0, d, e4m3, true, boxes) &&
                   make_page_map(&mv, p, 1, d, e4m3, !e4m3, boxes);
  if (d == 128) {
    if (e4m3)
      return tma ? launch_t<128, true, true>(p, mk, mv, boxes, stream)
                 : launch_t<128, true, false>(p, mk, mv, boxes, stream);
    return tma ? launch_t<128, false, true>(p, mk, mv, boxes, stream)
               : launch_t<128, false, false>(p, mk, mv, boxes, stream);
  }
  if (e4m3) return launch_t<64, true, false>(p, mk, mv, boxes, stream);
  return tma ? launch_t<64, false, true>(p, mk, mv, boxes, stream)
             : launch_t<64, false, false>(p, mk, mv, boxes, stream);
}

}  // namespace cpring
