// Decode attention over a paged key/value cache for a batch whose sequences
// may share a prefix.
//
// Row (b, i, h) - query i of sequence b, head h - sees the prefix's keys
// [0, P) and its own [P, len - n_q + i].  softmax(q k / sqrt d) v over them is
// built from partial states (O, m, l) over parts of the keys, O = sum
// 2^(s - m) v and l = sum 2^(s - m) with s in units of log2, joined by the
// online-softmax merge ("上下文並行（Context Parallelism, CP）",
// compassingai.com, section 線上 Softmax):
//   M = max m_x,  O = sum 2^(m_x - M) O_x,  l = sum 2^(m_x - M) l_x,
//   out = O / l,  lse = (M + log2 l) ln 2.
//
// paged_decode_kernel.  The n_q * G rows that share a key head (G = Hq / Hk)
// are one item per sequence, in tiles of 16 rows; all of them see the keys
// [P, len - n_q], so an item needs no mask but its end.  (The up to n_q - 1
// later keys, which query i sees i of, are left to the join.)  Items of the
// prefix hold the rows of the whole batch.  Bound by HBM: each key and value
// is read once per item and serves 16 rows, 32 FLOP per byte in bf16, which
// mma.sync delivers several times over, so the work is in keeping loads in
// flight.  A warp owns 16 keys of each 64-key tile, with its own cp.async ring
// and its own running (O, m, l): no two warps meet until the item ends, where
// the four states are joined in shared memory.  cp.async takes any page size,
// page order and stride, and fills what lies behind the last key with zeros.
//
// Split: the items' tiles are laid end to end (prefix, then sequence by
// sequence) and every CTA of a fixed grid takes an equal stretch, so a batch of
// ragged lengths, one long sequence and many short ones all fill the GPU.
// The stretch is found on the device from the lengths, which lets a captured
// graph follow them.  An item inside one stretch is finished by its CTA;
// a cut item leaves its parts in the CTAs' slots (one for a stretch's first
// item, one for its last).
//
// paged_decode4_kernel does the same over a cache in 4 bits, with 32 keys of each 128-key tile
// to a warp (decode_int4.cuh: its products and its bound, which is instructions).  Items are of
// 16 rows as above, and where none has more than 8 the kernel for 8 runs: 58 us instead of 75 a
// call for 32 sequences of up to 16K keys, 205 MB; 164 instead of 229 for 16 of up to 128K,
// 833 MB (5.06 TB/s, 76 % of the copy rate), each with append and join.  The prefix goes through
// its items too, whatever its rows: it has no tcgen05 kernel over 4 bits.
//
// Measured (bf16, d = 128, pages of 16): 32 sequences of up to 16K keys, 728 MB, 112 us
// in the kernel, 96 % of the copy rate; E4M3, 364 MB, 69 us (77 %; the widening of
// codes leaves each warp waiting for its own instructions).
//
// decode_join_kernel joins a row's parts and the later keys of an n_q > 1
// call, in a fixed order.
//
// P in 16 bits.  The matrix instructions take it so, while l sums it in fp32.  Rounded to
// bf16 it would cost as much again as the output's own rounding (against 64 bits, relative
// in the norm: 1.77e-3 for 32 sequences of up to 16K keys, where the output's rounding
// alone makes 1.65e-3), so what the rounding left goes through a second product in bf16:
// the sum holds 15 bits of P (measured: 114.5 / 114.7 us a call with one / both products,
// 91.2 / 91.6 at 128 sequences of up to 3100 keys, 70.1 / 70.8 at d = 64).  Over E4M3
// caches P is fp16 alone: 2^-11 of each term, an eighth of the output's rounding (1.67e-3
// against 1.66e-3).
//
// E4M3 caches: codes are exact in fp16, so both products run as fp16 MMAs.
// Q is scaled per row by a power of two into fp16's range (exact but for
// entries 2^-28 below the row's largest), P by 2^15 so that what fp16 flushes
// is below 2^-39 of the row's largest; the descales go to the softmax scale
// and the output.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "decode_int4.cuh"
#include "internal.h"
#include "paged_decode.h"
#include "ptx.cuh"

namespace cpring {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpKeys = 16;                    // keys of a tile that a warp owns
constexpr int kTileKeys = kWarps * kWarpKeys;    // 64
constexpr int kTileKeys4 = 128;                  // over a cache in 4 bits
constexpr int kRows = 16;                        // rows of an item
constexpr int kCtasPerSm = 3;
constexpr int kMaxGrid = 480;                    // bounds the slots of the workspace
constexpr int kMaxBatch = 4096;
// From this many rows on a warp joins a row, four below.  Measured, one / four (us in
// the kernel): 32 rows of 11 parts 5.3 / 4.4; 2048 rows of 21 parts 9.5 / 11.1;
// 4096 rows of 11 parts and up to three later keys 14.3 / 22.1.
constexpr unsigned kManyRows = 1024;
constexpr int kMaxQueries = 16;
constexpr float kLn2 = 0.69314718055994531f;

// One warp's part of a pipeline stage: 16 rows of K, then 16 of V, as 16-byte
// chunks; chunk c of row r at c ^ (r mod 8) (mod 4 for rows of 64 bytes), so
// that both ldmatrix and the row-wise reads of codes are conflict-free.
template <int D, Held kHeld>
struct Stage {
  static constexpr int kRowBytes = D * (kHeld == Held::kE4M3 ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kBytes = 2 * kWarpKeys * kRowBytes;
  static constexpr int kCount = kBytes >= 8192 ? 2 : 4;
  static constexpr int kRing = kCount * kBytes;  // per warp
  static constexpr int kSwz = kChunks >= 8 ? 7 : 3;
  __device__ static uint32_t at(uint32_t base, int row, int chunk) {
    return base + row * kRowBytes + ((chunk ^ (row & kSwz)) << 4);
  }
};

// Keys of sequence b that all of its queries see behind the prefix; -1 if its
// length is out of range.
__device__ __forceinline__ int common_keys(const DecodeParams& p, int len) {
  if (len == 0) return 0;
  if (len < p.P || len > p.capacity) return -1;
  return max(0, len - (p.n_q - 1) - p.P);
}

// Keys of a tile of the kernel that attends a cache of this form.
__host__ __device__ constexpr int tile_keys_of(Held held) {
  return held == Held::kInt4 ? kTileKeys4 : kTileKeys;
}

// Units of sequence b's items.
template <int kKeys>
__device__ __forceinline__ unsigned own_units(const DecodeParams& p, int b) {
  const int n = common_keys(p, __ldg(p.seq_lens + b));
  return n <= 0 ? 0u
                : (static_cast<unsigned>((n + kKeys - 1) / kKeys) + kItemCost) *
                      static_cast<unsigned>(p.Hk * p.own_tiles_of_rows);
}

// Units of the prefix in this kernel's own list.
__device__ __forceinline__ unsigned prefix_units(const DecodeParams& p) {
  return p.prefix_grid > 0 || p.P == 0
             ? 0u
             : (static_cast<unsigned>(p.prefix_tiles) + kItemCost) *
                   static_cast<unsigned>(p.Hk * p.prefix_row_tiles);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <bool kF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// The sequences' first units in `starts` (every CTA scans the lengths; CTA 0 keeps the
// result for the join); returns the units of all.
template <int kKeys>
__device__ __forceinline__ unsigned lay_out(const DecodeParams& p, unsigned prefix_all,
                                            unsigned* starts, unsigned* scan) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned run = prefix_all;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const unsigned n = b < p.B ? own_units<kKeys>(p, b) : 0u;
    unsigned x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    unsigned base = run;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += scan[w];
      run += scan[w];
    }
    if (b < p.B) {
      starts[b] = base + x - n;
      if (blockIdx.x == 0) p.starts[b] = base + x - n;
    }
    __syncthreads();
  }
  const unsigned W = run;
  if (threadIdx.x == 0) {
    starts[p.B] = W;
    if (blockIdx.x == 0) p.starts[p.B] = W;
  }
  __syncthreads();
  return W;
}

// The item that holds unit w, and the unit's place in it.
struct Item {
  bool prefix;
  int b0, hk, row0, rows, n_keys, base_pos;
  unsigned n_tiles, u0;
  const int32_t* pages;
  __device__ __forceinline__ Item(const DecodeParams& p, const unsigned* starts,
                                  unsigned prefix_all, unsigned w, int tile_keys) {
    if (w < prefix_all) {
      prefix = true;
      n_tiles = p.prefix_tiles;
      const unsigned item = w / (n_tiles + kItemCost);
      u0 = w - item * (n_tiles + kItemCost);
      hk = static_cast<int>(item) / p.prefix_row_tiles;
      row0 = (static_cast<int>(item) - hk * p.prefix_row_tiles) * kRows;
      rows = min(kRows, p.B * p.R - row0);
      b0 = 0;
      n_keys = p.P;
      base_pos = 0;
      pages = p.prefix_pages;
    } else {
      prefix = false;
      int lo = 0, hi = p.B;  // the last b with starts[b] <= w; empty sequences in between skip
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= w) lo = mid; else hi = mid;
      }
      b0 = lo;
      n_keys = common_keys(p, __ldg(p.seq_lens + b0));
      n_tiles = (n_keys + tile_keys - 1) / tile_keys;
      const unsigned local = w - starts[b0];
      const unsigned item = local / (n_tiles + kItemCost);
      u0 = local - item * (n_tiles + kItemCost);
      hk = static_cast<int>(item) / p.own_tiles_of_rows;
      row0 = (static_cast<int>(item) - hk * p.own_tiles_of_rows) * kRows;
      rows = min(kRows, p.R - row0);
      base_pos = p.P;
      pages = p.table + b0 * p.table_stride;
    }
  }
};

// The item's state, or its part of it over the tiles [t0, t1), from the four warps': sums
// [warp][16 rows][kPitch] that share a reference, and (m, l) of each; l is NaN for a bad page.
template <int D>
constexpr int kPitch = D + 8;  // floats; staggers the rows over the banks
template <int D, int kShiftLog2>
__device__ __forceinline__ void write_item(const DecodeParams& p, const Item& it, int t0, int t1,
                                           const float* mo,
                                           const float (&merge_ml)[kWarps][kRows][2], bool any_bad,
                                           float vd) {
  constexpr float kShift = kShiftLog2;  // P was held times 2^kShift
  const bool complete = t0 == 0 && static_cast<unsigned>(t1) == it.n_tiles;
  const bool direct = complete && !it.prefix && p.P == 0 && p.n_q == 1;
  constexpr int kVecs = D / 4;  // 4-column vectors of a row
  for (int x = threadIdx.x; x < it.rows * kVecs; x += kThreads) {
    const int r = x / kVecs, col = (x % kVecs) * 4;
    float big = -INFINITY, l = 0.f;
#pragma unroll
    for (int y = 0; y < kWarps; ++y) big = fmaxf(big, merge_ml[y][r][0]);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int y = 0; y < kWarps; ++y) {
      const float my = merge_ml[y][r][0];
      // an empty state's l is 0, or NaN where its scores were
      l += merge_ml[y][r][1] * (my == -INFINITY ? 1.f : ptx::ex2(my - big));
      const float4 a = *reinterpret_cast<const float4*>(mo + (y * kRows + r) * kPitch<D> + col);
      sum.x += a.x;
      sum.y += a.y;
      sum.z += a.z;
      sum.w += a.w;
    }
    if (any_bad) l = NAN;
    const RowOf row(p, it.b0, it.hk, it.row0 + r);
    if (direct) {
      const float inv = l == 0.f ? 0.f : vd / l;
      uint2 v;
      v.x = ptx::pack_bf16(sum.x * inv, sum.y * inv);
      v.y = ptx::pack_bf16(sum.z * inv, sum.w * inv);
      *reinterpret_cast<uint2*>(p.out + row.index(p) * D + col) = v;
      if (col == 0)
        p.lse[(static_cast<long long>(row.b) * p.Hq + row.h) * p.n_q + row.i] =
            (big - kShift + log2f(l)) * kLn2;
      continue;
    }
    float *to, *ml;
    if (complete) {
      const long long at = (it.prefix ? static_cast<long long>(p.B) * p.n_q * p.Hq : 0) +
                           row.index(p);
      to = p.whole_o + at * D;
      ml = p.whole_ml + at * 2;
    } else {
      const long long at = (static_cast<long long>(blockIdx.x) * 2 + (t0 == 0 ? 1 : 0)) * kRows + r;
      to = p.slot_o + at * D;
      ml = p.slot_ml + at * 2;
    }
    *reinterpret_cast<float4*>(to + col) = make_float4(sum.x * vd, sum.y * vd, sum.z * vd,
                                                       sum.w * vd);
    if (col == 0) *reinterpret_cast<float2*>(ml) = make_float2(big - kShift, l);
  }
}

// What a head's codes are multiplied by (x: 0 K, 1 V).
template <Held kHeld>
__device__ __forceinline__ float head_descale(const DecodeParams& p, int x, int hk) {
  if (kHeld == Held::kBf16 || (kHeld == Held::kInt4 && p.descale[x] == nullptr)) return 1.f;
  return __ldg(p.descale[x] + hk);
}

template <int D, Held kHeld>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_decode_kernel(const DecodeParams p) {
  using St = Stage<D, kHeld>;
  static_assert(kHeld != Held::kInt4, "paged_decode4_kernel's");
  constexpr bool kE4M3 = kHeld == Held::kE4M3;
  constexpr int kK = D / 16;   // k-steps of S = Q K^T
  constexpr int kN = D / 8;    // 8-column tiles of O
  constexpr float kShift = kE4M3 ? 15.f : 0.f;  // P is held times 2^kShift
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned scan[kWarps];
  __shared__ float merge_ml[kWarps][kRows][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, c4 = lane & 3;
  const uint32_t ring = ptx::smem_u32(smem) + warp * St::kRing;

  cudaTriggerProgrammaticLaunchCompletion();  // the next kernel's blocks may line up
  const unsigned prefix_all = prefix_units(p);
  unsigned* const starts = reinterpret_cast<unsigned*>(smem + kWarps * St::kRing);
  const unsigned W = lay_out<kTileKeys>(p, prefix_all, starts, scan);
  const unsigned g = min(gridDim.x, W);
  if (blockIdx.x >= g) return;
  unsigned w = stretch(blockIdx.x, W, g);
  const unsigned w_end = stretch(blockIdx.x + 1, W, g);

  while (w < w_end) {
    const Item it(p, starts, prefix_all, w, kTileKeys);
    const int b0 = it.b0, hk = it.hk, row0 = it.row0, rows = it.rows, n_keys = it.n_keys,
              base_pos = it.base_pos;
    const unsigned n_tiles = it.n_tiles, u0 = it.u0;
    const int32_t* const pages = it.pages;
    const unsigned u1 = min(n_tiles + kItemCost, u0 + (w_end - w));
    const int t0 = tile_of_unit(u0), t1 = tile_of_unit(u1);
    w += u1 - u0;
    if (t0 >= t1) continue;

    // ---- this warp's loads of tile t: 16 keys, whose pages are looked up
    // before (the first tiles' together, later ones' one tile ahead)
    struct Place {
      int page, slot;
    };
    bool bad = false;
    auto look_up = [&](int t) {
      Place at{-1, 0};
      const int key = t * kTileKeys + warp * kWarpKeys + lane;
      if (lane < kWarpKeys && t < t1 && key < n_keys) {
        const int x = (base_pos + key) / p.page_size;
        at.slot = base_pos + key - x * p.page_size;
        at.page = __ldg(pages + x);
      }
      return at;
    };
    auto load = [&](int t, int stage, Place at) {
      if (t < t1) {
        const uint32_t dst = ring + stage * St::kBytes;
        const bool have = at.page >= 0 && at.page < p.n_pages;
        if (!have && lane < kWarpKeys && t * kTileKeys + warp * kWarpKeys + lane < n_keys)
          bad = true;
        long long off[2] = {0, 0};
        if (have) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
            off[x] = at.page * p.cs[x][0] + at.slot * p.cs[x][1] + hk * p.cs[x][2];
        }
        constexpr int kPerStep = 32 / St::kChunks;  // keys per warp-wide access
        const int chunk = lane % St::kChunks;
        const unsigned held = __ballot_sync(0xffffffffu, have);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int i = 0; i < kWarpKeys / kPerStep; ++i) {
            const int key = i * kPerStep + lane / St::kChunks;
            const long long o = __shfl_sync(0xffffffffu, off[x], key);
            cp_async16(St::at(dst + x * (St::kBytes / 2), key, chunk),
                       p.cache[x] + o + chunk * 16, (held >> key & 1u) ? 16 : 0);
          }
        }
      }
      cp_commit();
    };
    Place next;
    {
      Place first[St::kCount];
#pragma unroll
      for (int i = 0; i < St::kCount; ++i) first[i] = look_up(t0 + i);
#pragma unroll
      for (int i = 0; i < St::kCount - 1; ++i) load(t0 + i, i, first[i]);
      next = first[St::kCount - 1];
    }
    // ---- Q fragments: rows quad and quad + 8 of the item
    uint32_t qf[kK][4];
    float sc0 = p.scale, sc1 = p.scale;
    {
      const RowOf r0(p, b0, hk, min(row0 + quad, row0 + rows - 1));
      const RowOf r1(p, b0, hk, min(row0 + quad + 8, row0 + rows - 1));
      const __nv_bfloat16* const q0 = r0.query(p);
      const __nv_bfloat16* const q1 = r1.query(p);
      if (!kE4M3) {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          qf[k][0] = *reinterpret_cast<const uint32_t*>(q0 + k * 16 + c4 * 2);
          qf[k][1] = *reinterpret_cast<const uint32_t*>(q1 + k * 16 + c4 * 2);
          qf[k][2] = *reinterpret_cast<const uint32_t*>(q0 + k * 16 + c4 * 2 + 8);
          qf[k][3] = *reinterpret_cast<const uint32_t*>(q1 + k * 16 + c4 * 2 + 8);
        }
      } else {
        // The order of a dot product's terms is free: lane c4 takes the D / 4
        // neighbouring columns from c4 * D / 4 on, in Q as in the codes of K.
        const float desc = head_descale<kHeld>(p, 0, hk);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint4* const src =
              reinterpret_cast<const uint4*>((x ? q1 : q0) + c4 * (D / 4));
          float z[D / 4];
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint4 v = src[i];
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              z[8 * i + 2 * e] = __uint_as_float(u[e] << 16);
              z[8 * i + 2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
              top = fmaxf(top, fmaxf(fabsf(z[8 * i + 2 * e]), fabsf(z[8 * i + 2 * e + 1])));
            }
          }
          top = quad_max(top);
          float up, down;
          fp16_row_scale(top, up, down);
          (x ? sc1 : sc0) = p.scale * desc * down;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            qf[k][x] = pack_f16(z[4 * k] * up, z[4 * k + 1] * up);
            qf[k][2 + x] = pack_f16(z[4 * k + 2] * up, z[4 * k + 3] * up);
          }
        }
      }
    }
    float o[kN][4];
#pragma unroll
    for (int n = 0; n < kN; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    int stage = 0;
    for (int t = t0; t < t1; ++t) {
      cp_wait<St::kCount - 2>();
      __syncwarp();
      load(t + St::kCount - 1, stage == 0 ? St::kCount - 1 : stage - 1, next);
      next = look_up(t + St::kCount);
      const uint32_t ks = ring + stage * St::kBytes;
      const uint32_t vs = ks + St::kBytes / 2;
      if (++stage == St::kCount) stage = 0;
      // ---- S: two 8-key tiles
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
      if (!kE4M3) {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          uint32_t b[4];
          ldsm4(St::at(ks, (lane >> 4) * 8 + (lane & 7), 2 * k + ((lane >> 3) & 1)), b);
          mma16816<false>(s[0], qf[k], b[0], b[1]);
          mma16816<false>(s[1], qf[k], b[2], b[3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          constexpr int kVecs = D / 64;  // 16-byte vectors of codes per lane and row
#pragma unroll
          for (int x = 0; x < kVecs; ++x) {
            const uint32_t addr = St::at(ks, j * 8 + quad, c4 * kVecs + x);
            uint32_t u[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                         : "r"(addr));
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma16816<true>(s[j], qf[4 * x + e], half2_of_codes(u[e] & 0xffffu),
                             half2_of_codes(u[e] >> 16));
          }
        }
      }
      // ---- mask, running maximum, P
      const int left = n_keys - (t * kTileKeys + warp * kWarpKeys);  // keys of mine that exist
      if (left < kWarpKeys) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j * 8 + c4 * 2 + (e & 1) >= left) s[j][e] = -INFINITY;
      }
      const float x0 = quad_max(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])) * sc0);
      const float x1 = quad_max(fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3])) * sc1);
      if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float a0 = m0 == -INFINITY ? 0.f : ptx::ex2(m0 - n0);
        const float a1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          o[n][0] *= a0;
          o[n][1] *= a0;
          o[n][2] *= a1;
          o[n][3] *= a1;
        }
      }
      const float r0 = (m0 == -INFINITY ? 0.f : m0) - kShift;
      const float r1 = (m1 == -INFINITY ? 0.f : m1) - kShift;
      float pr[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        pr[j][0] = ptx::ex2(fmaf(s[j][0], sc0, -r0));
        pr[j][1] = ptx::ex2(fmaf(s[j][1], sc0, -r0));
        pr[j][2] = ptx::ex2(fmaf(s[j][2], sc1, -r1));
        pr[j][3] = ptx::ex2(fmaf(s[j][3], sc1, -r1));
        l0 += pr[j][0] + pr[j][1];
        l1 += pr[j][2] + pr[j][3];
      }
      uint32_t pf[4];
      uint32_t pe[4];  // bf16: what the upper half of P leaves
      if (kE4M3) {
        pf[0] = pack_f16(pr[0][0], pr[0][1]);
        pf[1] = pack_f16(pr[0][2], pr[0][3]);
        pf[2] = pack_f16(pr[1][0], pr[1][1]);
        pf[3] = pack_f16(pr[1][2], pr[1][3]);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          // The upper halves, and what they leave: never 0 (2^-20 of P at least) nor
          // negative, so that a value of infinity stays one through both products.
          const uint32_t a = __float_as_uint(pr[x >> 1][(x & 1) * 2]) | 8u;
          const uint32_t b = __float_as_uint(pr[x >> 1][(x & 1) * 2 + 1]) | 8u;
          pf[x] = __byte_perm(a, b, 0x7632);
          pe[x] = ptx::pack_bf16(__uint_as_float(a) - __uint_as_float(a & 0xffff0000u),
                                 __uint_as_float(b) - __uint_as_float(b & 0xffff0000u));
        }
      }
      // ---- O += P V
#pragma unroll
      for (int ch = 0; ch < St::kChunks; ch += 2) {
        uint32_t b[4];
        ldsm4_t(St::at(vs, ((lane >> 3) & 1) * 8 + (lane & 7), ch + (lane >> 4)), b);
        if (!kE4M3) {
          mma16816<false>(o[ch], pf, b[0], b[1]);
          mma16816<false>(o[ch + 1], pf, b[2], b[3]);
          mma16816<false>(o[ch], pe, b[0], b[1]);
          mma16816<false>(o[ch + 1], pe, b[2], b[3]);
        } else {
          // A 16-bit element is two neighbouring columns: the even ones make
          // one 8-column tile, the odd ones another.
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t k_lo = __byte_perm(b[2 * x], 0, 0x3120);
            const uint32_t k_hi = __byte_perm(b[2 * x + 1], 0, 0x3120);
            mma16816<true>(o[2 * (ch + x)], pf, half2_of_codes(k_lo & 0xffffu),
                           half2_of_codes(k_hi & 0xffffu));
            mma16816<true>(o[2 * (ch + x) + 1], pf, half2_of_codes(k_lo >> 16),
                           half2_of_codes(k_hi >> 16));
          }
        }
      }
    }
    cp_wait<0>();

    // ---- join the four warps' states; a bad page makes the item's l NaN
    l0 = quad_sum(l0);
    l1 = quad_sum(l1);
    const bool any_bad = __syncthreads_or(bad);  // also: every warp is done with its ring
    if (c4 == 0) {
      merge_ml[warp][quad][0] = m0;
      merge_ml[warp][quad][1] = l0;
      merge_ml[warp][quad + 8][0] = m1;
      merge_ml[warp][quad + 8][1] = l1;
    }
    __syncthreads();
    float* const mo = reinterpret_cast<float*>(smem);
    {
      float big0 = -INFINITY, big1 = -INFINITY;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        big0 = fmaxf(big0, merge_ml[x][quad][0]);
        big1 = fmaxf(big1, merge_ml[x][quad + 8][0]);
      }
      const float f0 = m0 == -INFINITY ? 0.f : ptx::ex2(m0 - big0);
      const float f1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - big1);
      float* const w0 = mo + (warp * kRows + quad) * kPitch<D>;
      float* const w1 = w0 + 8 * kPitch<D>;
      if (!kE4M3) {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          *reinterpret_cast<float2*>(w0 + n * 8 + c4 * 2) = make_float2(o[n][0] * f0, o[n][1] * f0);
          *reinterpret_cast<float2*>(w1 + n * 8 + c4 * 2) = make_float2(o[n][2] * f1, o[n][3] * f1);
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < kN / 2; ++ch) {
          const float(&ev)[4] = o[2 * ch];
          const float(&od)[4] = o[2 * ch + 1];
          *reinterpret_cast<float4*>(w0 + ch * 16 + c4 * 4) =
              make_float4(ev[0] * f0, od[0] * f0, ev[1] * f0, od[1] * f0);
          *reinterpret_cast<float4*>(w1 + ch * 16 + c4 * 4) =
              make_float4(ev[2] * f1, od[2] * f1, ev[3] * f1, od[3] * f1);
        }
      }
    }
    __syncthreads();
    write_item<D, kE4M3 ? 15 : 0>(p, it, t0, t1, mo, merge_ml, any_bad,
                                  kE4M3 ? __ldg(p.descale[1] + hk) : 1.f);
    if (any_bad && threadIdx.x == 0) atomicOr(p.err, kErrCache);
    __syncthreads();  // the ring is free again
  }
}

// Over a cache in 4 bits (decode_int4.cuh): 128-key tiles, 32 keys to a warp, up to kNT x 8
// rows of an item.
template <int D, int kNT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_decode4_kernel(const DecodeParams p) {
  using Core = Int4Core<D, kNT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned scan[kWarps];
  __shared__ float merge_ml[kWarps][kRows][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = ptx::smem_u32(smem) + warp * Core::kRing;

  cudaTriggerProgrammaticLaunchCompletion();  // the next kernel's blocks may line up
  const unsigned prefix_all = prefix_units(p);
  unsigned* const starts = reinterpret_cast<unsigned*>(smem + kWarps * Core::kRing);
  const unsigned W = lay_out<kTileKeys4>(p, prefix_all, starts, scan);
  const unsigned g = min(gridDim.x, W);
  if (blockIdx.x >= g) return;
  unsigned w = stretch(blockIdx.x, W, g);
  const unsigned w_end = stretch(blockIdx.x + 1, W, g);

  while (w < w_end) {
    const Item it(p, starts, prefix_all, w, kTileKeys4);
    const unsigned u1 = min(it.n_tiles + kItemCost, it.u0 + (w_end - w));
    const int t0 = tile_of_unit(it.u0), t1 = tile_of_unit(u1);
    w += u1 - it.u0;
    if (t0 >= t1) continue;

    // ---- this warp's loads of tile t: a key to a lane, whose page is looked up before
    struct Place {
      int page, slot;
    };
    bool bad = false;
    const uint8_t* const head[2] = {p.cache[0] + it.hk * p.cs[0][2],
                                    p.cache[1] + it.hk * p.cs[1][2]};
    const uint8_t* const scale_head[2] = {p.scales[0] + it.hk * p.ss[0][2],
                                          p.scales[1] + it.hk * p.ss[1][2]};
    auto look_up = [&](int t) {
      Place at{-1, 0};
      const int key = t * kTileKeys4 + warp * Core::kKeys + lane;
      if (t < t1 && key < it.n_keys) {
        const int pos = it.base_pos + key;
        const int x = p.page_of(pos);
        at.slot = pos - x * p.page_size;
        at.page = __ldg(it.pages + x);
        if (at.page < 0 || at.page >= p.n_pages) {
          at.page = -1;
          bad = true;
        }
      }
      return at;
    };
    auto load = [&](int t, int stage, Place at) {
      if (t < t1) {
        const uint32_t dst = ring + stage * Core::kBytes;
        const bool have = at.page >= 0;
        const unsigned held = __ballot_sync(0xffffffffu, have);
        // unsigned, so that a product with a stride is two instructions
        const unsigned page = have ? at.page : 0, slot = at.slot;
        constexpr int kPerStep = 32 / Core::kChunks;  // keys per warp-wide access
        const int chunk = lane % Core::kChunks, first = lane / Core::kChunks;
        // K's rows, and V's where their strides are the same (0); or V's (1)
        auto rows = [&](auto which, auto whole) {
          constexpr int kX = decltype(which)::value;
          const unsigned long long mine = page * static_cast<unsigned long long>(p.cs[kX][0]) +
                                          slot * static_cast<unsigned long long>(p.cs[kX][1]);
          const uint8_t* const base = head[kX] + chunk * 16;
#pragma unroll
          for (int i = 0; i < Core::kKeys / kPerStep; ++i) {
            const int key = i * kPerStep + first;
            const unsigned long long o = __shfl_sync(0xffffffffu, mine, key);
            const int bytes = decltype(whole)::value || (held >> key & 1u) ? 16 : 0;
            cp_async16(Core::at(dst + kX * Core::kV, key, chunk), base + o, bytes);
            if (kX == 0 && p.alike)
              cp_async16(Core::at(dst + Core::kV, key, chunk), head[1] + chunk * 16 + o, bytes);
          }
        };
        if (held == 0xffffffffu)
          rows(std::integral_constant<int, 0>(), std::true_type());
        else
          rows(std::integral_constant<int, 0>(), std::false_type());
        if (!p.alike) rows(std::integral_constant<int, 1>(), std::false_type());
#pragma unroll
        for (int x = 0; x < 2; ++x)
          cp_async_small<Core::kScaleBytes>(
              dst + Core::kScales + (x * Core::kKeys + lane) * Core::kScaleBytes,
              scale_head[x] + (page * static_cast<unsigned long long>(p.ss[x][0]) +
                               slot * static_cast<unsigned long long>(p.ss[x][1])),
              have);
      }
      cp_commit();
    };
    Place next;
    {
      Place first[Core::kCount];
#pragma unroll
      for (int i = 0; i < Core::kCount; ++i) first[i] = look_up(t0 + i);
#pragma unroll
      for (int i = 0; i < Core::kCount - 1; ++i) load(t0 + i, i, first[i]);
      next = first[Core::kCount - 1];
    }
    Core core;
    core.load_queries(
        [&](int r) { return RowOf(p, it.b0, it.hk, it.row0 + r).query(p); }, it.rows,
        p.scale * head_descale<Held::kInt4>(p, 0, it.hk), lane);

    int stage = 0;
    for (int t = t0; t < t1; ++t) {
      cp_wait<Core::kCount - 2>();
      __syncwarp();
      load(t + Core::kCount - 1, stage == 0 ? Core::kCount - 1 : stage - 1, next);
      next = look_up(t + Core::kCount);
      core.step(ring + stage * Core::kBytes, it.n_keys - t * kTileKeys4 - warp * Core::kKeys, lane);
      if (++stage == Core::kCount) stage = 0;
    }
    cp_wait<0>();

    // ---- join the four warps' states; a bad page makes the item's l NaN
    core.sum_lanes();
    const bool any_bad = __syncthreads_or(bad);  // also: every warp is done with its ring
    const int r0 = 2 * (lane & 3);
    if (lane < 4) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          merge_ml[warp][8 * nt + r0 + e][0] = core.m(nt, e);
          merge_ml[warp][8 * nt + r0 + e][1] = core.l[nt][e];
        }
    }
    __syncthreads();
    float* const mo = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * nt + r0 + e;
        float big = -INFINITY;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) big = fmaxf(big, merge_ml[x][row][0]);
        const float m = core.m(nt, e), f = m == -INFINITY ? 0.f : ptx::ex2(m - big);
        core.store_row(mo + (warp * kRows + row) * kPitch<D>, nt, e, f, lane);
      }
    __syncthreads();
    write_item<D, static_cast<int>(Core::kShift)>(
        p, it, t0, t1, mo, merge_ml, any_bad,
        Core::kUnit * head_descale<Held::kInt4>(p, 1, it.hk));
    if (any_bad && threadIdx.x == 0) atomicOr(p.err, kErrCache);
    __syncthreads();  // the ring is free again
  }
}

// Where the parts of one row of an item lie: `count` of them, the x-th in
// the slots of CTA c0 + x, or the one in the array of finished items.
struct Parts {
  const float* o;
  const float* ml;
  unsigned c0, count;
  int rows, r;  // a slot's rows; this row
  // n > 0 tiles, the item's first unit of W over g CTAs.
  __device__ void find(unsigned first, unsigned n, unsigned W, unsigned g) {
    c0 = holder(first + kItemCost, W, g);
    count = holder(first + kItemCost + n - 1, W, g) - c0 + 1;
  }
  __device__ long long at(unsigned x) const {
    return rows == 0 ? r : (static_cast<long long>(c0 + x) * 2 + (x == 0 ? 1 : 0)) * rows + r;
  }
};

// A lane's kCols columns of a cached row (in 4 bits: and its row of scales).
template <int kCols, Held kHeld>
__device__ __forceinline__ void load_columns(const uint8_t* row, const uint8_t* scales, int lane,
                                             float (&v)[kCols]) {
  if (kHeld == Held::kInt4) {
    const uint32_t u = kCols == 4 ? __ldg(reinterpret_cast<const unsigned short*>(row) + lane)
                                  : __ldg(row + lane);
    const uint32_t h = half2_of_codes(__ldg(scales + lane * kCols / kBlock));
    const float s = __low2float(*reinterpret_cast<const __half2*>(&h));
#pragma unroll
    for (int x = 0; x < kCols; ++x)
      v[x] = static_cast<float>(static_cast<int>(u >> (4 * x) & 15u) - 8) * s;
  } else if (kHeld == Held::kE4M3) {
    uint32_t u;
    if (kCols == 4)
      u = __ldg(reinterpret_cast<const unsigned*>(row) + lane);
    else
      u = __ldg(reinterpret_cast<const unsigned short*>(row) + lane);
#pragma unroll
    for (int x = 0; x < kCols; x += 2) {
      const uint32_t h = half2_of_codes((u >> (8 * x)) & 0xffffu);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[x] = f.x;
      v[x + 1] = f.y;
    }
  } else {
    uint32_t u[2];
    if (kCols == 4) {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(row) + lane);
      u[0] = t.x, u[1] = t.y;
    } else {
      u[0] = __ldg(reinterpret_cast<const unsigned*>(row) + lane);
    }
#pragma unroll
    for (int x = 0; x < kCols; x += 2) {
      v[x] = __uint_as_float(u[x / 2] << 16);
      v[x + 1] = __uint_as_float(u[x / 2] & 0xffff0000u);
    }
  }
}

// kRowWarps warps join a row: four where rows are few (their parts' loads run side
// by side), one where there are enough rows to fill the GPU.
template <int D, Held kHeld, int kRowWarps>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(const DecodeParams p, unsigned grid) {
  constexpr int kCols = D / 32;  // columns per lane
  __shared__ float part_m[kWarps], part_l[kWarps];
  __shared__ float part_o[kRowWarps > 1 ? kWarps : 1][D];
  const int lane = threadIdx.x & 31;
  const int warp = (threadIdx.x >> 5) % kRowWarps;  // of the row's
  cudaGridDependencySynchronize();
  const int rid = static_cast<int>(blockIdx.x) * (kWarps / kRowWarps) +
                  static_cast<int>(threadIdx.x >> 5) / kRowWarps;  // (b, i, h), below 2^24
  if (rid >= p.B * p.n_q * p.Hq) return;  // whole warps, and only with one to a row
  const int bi = rid / p.Hq, h = rid - bi * p.Hq;
  const int b = bi / p.n_q, i = bi - b * p.n_q;
  const int hk = h / p.G;
  const unsigned W = p.starts[p.B];
  const unsigned first_own = p.starts[b];
  const int len = __ldg(p.seq_lens + b);
  const int common = common_keys(p, len);
  const long long lse_at = (static_cast<long long>(b) * p.Hq + h) * p.n_q + i;
  __nv_bfloat16* const out = p.out + static_cast<long long>(rid) * D;
  if (len == 0 || common < 0) {
    if (warp != 0) return;
    const float v = len == 0 ? 0.f : NAN;
    for (int x = lane; x < D; x += 32) out[x] = __float2bfloat16_rn(v);
    if (lane == 0) {
      p.lse[lse_at] = len == 0 ? -INFINITY : NAN;
      if (common < 0) atomicOr(p.err, kErrCache);
    }
    return;
  }
  const unsigned g = min(grid, W);
  const long long whole = rid, whole_pre = static_cast<long long>(p.B) * p.n_q * p.Hq + rid;
  const int r_own = i * p.G + h % p.G;
  Parts own{p.slot_o, p.slot_ml, 0, 0, kRows, r_own % kRows};
  if (common > 0) {
    constexpr int kKeys = tile_keys_of(kHeld);
    const unsigned n = static_cast<unsigned>((common + kKeys - 1) / kKeys);
    own.find(first_own + (hk * p.own_tiles_of_rows + r_own / kRows) * (n + kItemCost), n, W, g);
    if (own.count == 1) {
      if (p.P == 0 && p.n_q == 1) return;  // written by the item's CTA
      own = Parts{p.whole_o + whole * D, p.whole_ml + whole * 2, 0, 1, 0, 0};
    }
  }
  Parts pre{p.slot_o, p.slot_ml, 0, 0, p.prefix_rows, 0};
  if (p.P > 0) {
    const bool wide = p.prefix_grid > 0;  // prefix_attn_kernel's parts
    const int row = b * p.R + r_own;
    const unsigned n = static_cast<unsigned>(p.prefix_tiles), units = n + kItemCost;
    if (wide) {
      pre.o = p.pslot_o;
      pre.ml = p.pslot_ml;
    }
    pre.r = row % p.prefix_rows;
    const int tile = row / p.prefix_rows;
    const int item = wide ? prefix_item<kHeld == Held::kE4M3>(p, hk, tile)
                          : hk * p.prefix_row_tiles + tile;
    pre.find(item * units, n,
             wide ? units * static_cast<unsigned>(p.Hk * p.prefix_row_tiles) : W,
             wide ? static_cast<unsigned>(p.prefix_grid) : g);
    if (pre.count == 1)
      pre = Parts{p.whole_o + whole_pre * D, p.whole_ml + whole_pre * 2, 0, 1, 0, 0};
  }
  // ---- the parts, dealt to the warps, kBatch of a warp's loaded before the first
  // is used; behind them the keys that this query sees beyond the common ones,
  // each a part with m = its score, l = 1, O = its value
  constexpr int kBatch = 6, kKeys = 4;
  float m = -INFINITY, l = 0.f;
  float o[kCols];
#pragma unroll
  for (int x = 0; x < kCols; ++x) o[x] = 0.f;
  auto fold = [&](const auto& ml, const auto& v, auto count) {
    constexpr int kN = decltype(count)::value;
    float big = m;
#pragma unroll
    for (int k = 0; k < kN; ++k) big = fmaxf(big, ml[k].x);
    const float a = m == -INFINITY ? 0.f : ptx::ex2(m - big);
    l = m == -INFINITY ? l : l * a;  // an empty state's l is 0, or NaN
#pragma unroll
    for (int y = 0; y < kCols; ++y) o[y] *= a;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const bool empty = ml[k].x == -INFINITY;
      const float f = empty ? 0.f : ptx::ex2(ml[k].x - big);
      l += empty ? ml[k].y : ml[k].y * f;
#pragma unroll
      for (int y = 0; y < kCols; ++y) o[y] = fmaf(v[k][y], f, o[y]);
    }
    m = big;
  };
  const int n_own = static_cast<int>(own.count), n_parts = n_own + static_cast<int>(pre.count);
  for (int x0 = warp; x0 < n_parts; x0 += kRowWarps * kBatch) {
    float2 ml[kBatch];
    float v[kBatch][kCols];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int x = x0 + k * kRowWarps;
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int y = 0; y < kCols; ++y) v[k][y] = 0.f;
      if (x < n_parts) {
        const Parts& from = x < n_own ? own : pre;
        const long long at = from.at(x < n_own ? x : x - n_own);
        ml[k] = __ldcg(reinterpret_cast<const float2*>(from.ml + at * 2));
        const float* const src = from.o + at * D + lane * kCols;
        if (kCols == 4) {
          const float4 u = __ldcg(reinterpret_cast<const float4*>(src));
          v[k][0] = u.x, v[k][1] = u.y, v[k][kCols - 2] = u.z, v[k][kCols - 1] = u.w;
        } else {
          const float2 u = __ldcg(reinterpret_cast<const float2*>(src));
          v[k][0] = u.x, v[k][1] = u.y;
        }
      }
    }
    fold(ml, v, std::integral_constant<int, kBatch>());
  }
  const int pos0 = max(len - p.n_q + 1, p.P);
  const int pos1 = len - p.n_q + i;
  bool bad = false;
  if (pos0 <= pos1) {
    float q[kCols];
    load_columns<kCols, Held::kBf16>(
        reinterpret_cast<const uint8_t*>(p.q + b * p.qb + i * p.qs + h * p.qh), nullptr, lane, q);
    const float kd = head_descale<kHeld>(p, 0, hk) * p.scale;
    const float vd = head_descale<kHeld>(p, 1, hk);
    for (int first = pos0 + warp; first <= pos1; first += kRowWarps * kKeys) {
      int page[kKeys], slot[kKeys];
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        const int pos = first + k * kRowWarps;
        page[k] = -1;
        slot[k] = 0;
        if (pos <= pos1) {
          const int at = pos / p.page_size;
          slot[k] = pos - at * p.page_size;
          page[k] = __ldg(p.table + b * p.table_stride + at);
          if (page[k] < 0 || page[k] >= p.n_pages) {
            page[k] = -1;
            bad = true;
          }
        }
      }
      float key[kKeys][kCols], value[kKeys][kCols];
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
#pragma unroll
        for (int y = 0; y < kCols; ++y) key[k][y] = value[k][y] = 0.f;
        if (page[k] >= 0) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
            load_columns<kCols, kHeld>(
                p.cache[x] + page[k] * p.cs[x][0] + slot[k] * p.cs[x][1] + hk * p.cs[x][2],
                p.scales[x] + page[k] * p.ss[x][0] + slot[k] * p.ss[x][1] + hk * p.ss[x][2], lane,
                x ? value[k] : key[k]);
        }
      }
      float2 ml[kKeys];
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        float dot = 0.f;
#pragma unroll
        for (int y = 0; y < kCols; ++y) dot = fmaf(q[y], key[k][y], dot);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        ml[k] = page[k] >= 0 ? make_float2(dot * kd, 1.f) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int y = 0; y < kCols; ++y) value[k][y] *= vd;
      }
      fold(ml, value, std::integral_constant<int, kKeys>());
    }
  }
  if (bad) {
    l = NAN;
    if (lane == 0) atomicOr(p.err, kErrCache);
  }
  if (kRowWarps == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (kCols == 4)
      reinterpret_cast<uint2*>(out)[lane] = make_uint2(
          ptx::pack_bf16(o[0] * inv, o[1] * inv), ptx::pack_bf16(o[kCols - 2] * inv, o[kCols - 1] * inv));
    else
      reinterpret_cast<uint32_t*>(out)[lane] = ptx::pack_bf16(o[0] * inv, o[1] * inv);
    if (lane == 0) p.lse[lse_at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    return;
  }
  if (lane == 0) {
    part_m[warp] = m;
    part_l[warp] = l;
  }
#pragma unroll
  for (int x = 0; x < kCols; ++x) part_o[kRowWarps > 1 ? warp : 0][lane * kCols + x] = o[x];
  __syncthreads();
  float big = -INFINITY;
#pragma unroll
  for (int y = 0; y < kRowWarps; ++y) big = fmaxf(big, part_m[y]);
  float total = 0.f, f[kRowWarps];
#pragma unroll
  for (int y = 0; y < kRowWarps; ++y) {
    f[y] = part_m[y] == -INFINITY ? 0.f : ptx::ex2(part_m[y] - big);
    total += part_m[y] == -INFINITY ? part_l[y] : part_l[y] * f[y];
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  for (int x = threadIdx.x; x < D; x += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int y = 0; y < kRowWarps; ++y) v += part_o[kRowWarps > 1 ? y : 0][x] * f[y];
    out[x] = __float2bfloat16_rn(v * inv);
  }
  if (threadIdx.x == 0) p.lse[lse_at] = total == 0.f ? -INFINITY : (big + log2f(total)) * kLn2;
}

long long align256(long long n) { return (n + 255) / 256 * 256; }

// Test hook (cp_test_set_prefix_path): -1 the rule below, 0 or 1 its answer.
std::atomic<int> g_prefix_path{-1};

// Whether the prefix goes to prefix_attn_kernel.  The 16-row items of
// paged_decode_kernel read the prefix's keys and values once per 16 rows of the
// batch, from L2 but for the first time, as fast as they compute: 0.10 to 0.19 us per
// MB.  prefix_attn_kernel takes about 8 us longer to start and to join (80 MB of such
// reads), and then its time is that of the prefix's own bytes, as many of which by TMA
// weigh 1.4 such reads, by cp.async 2.2 (bf16) or 3.0 (E4M3, which is widened on the
// way; stride orders that no tensor map describes count as TMA here).  Up to 16 rows both
// read the prefix once.  Measured over 16 to 512 rows, 2 and 8 key heads, 2K to 128K
// prefixes and pages of 64 (TMA) and 60 tokens (cp.async), the choice is the faster one or
// within 3.5 us of it (16 rows under 128K, 2 key heads: 45 for 41).  Some points (us a call,
// items / prefix_attn_kernel, 8 key heads, 64 more keys a sequence):
//   bf16, d = 128    32K 41 / 37 at 32 rows; 8K 21 / 22 at 32, 27 / 23 at 64;
//                    2K 20 / 22 at 128, 26 / 25 at 192; cp.async 32K 41 / 45 at 32, 55 / 46 at 48
//   bf16, d = 64     32K 28 / 29 at 32, 34 / 29 at 48; cp.async 34 / 37 at 48, 42 / 37 at 64
//   E4M3, d = 128    32K 33 / 38 at 32, 44 / 39 at 48; 8K 23 / 27 at 64, 36 / 30 at 128;
//                    cp.async 32K 44 / 53 at 48, 54 / 54 at 64; 128K 133 / 150 at 48
//   E4M3, d = 64     32K 37 / 42 at 64, 50 / 43 at 96; 128K 96 / 111 at 48, 140 / 111 at 64
bool wide_prefix(long long rows, int prefix_len, int Hk, int d, int elem_bytes, int page_size) {
  if (prefix_len <= 0) return false;
  const int forced = g_prefix_path.load(std::memory_order_relaxed);
  if (forced >= 0) return forced != 0;
  const bool tma = page_size % 8 == 0 && !(elem_bytes == 1 && d == 64);
  const double once = 2.0 * prefix_len * Hk * d * elem_bytes;
  const double read = static_cast<double>((rows + kRows - 1) / kRows) * once;
  return rows > kRows && read > 80e6 + (tma ? 1.4 : elem_bytes == 2 ? 2.2 : 3.0) * once;
}

// Byte offsets of the workspace's parts.
struct Space {
  long long starts, slot_o, slot_ml, whole_o, whole_ml, pslot_o, pslot_ml, total;
  Space(int B, int n_q, int Hq, int Hk, int d, int prefix_len) {
    const long long rows = static_cast<long long>(B) * n_q * Hq;
    const long long slots = 2LL * kMaxGrid * kRows;
    const long long whole = prefix_len > 0 ? 2 * rows : n_q > 1 ? rows : 0;
    const long long pslots =  // bf16 by TMA takes prefix_attn_kernel wherever another form does
        wide_prefix(rows / Hk, prefix_len, Hk, d, 2, 8) ? 2LL * kMaxPrefixGrid * kPrefixRows : 0;
    starts = 0;
    slot_o = align256(4LL * (B + 1));
    slot_ml = slot_o + align256(slots * d * 4);
    whole_o = slot_ml + align256(slots * 8);
    whole_ml = whole_o + align256(whole * d * 4);
    pslot_o = whole_ml + align256(whole * 8);
    pslot_ml = pslot_o + align256(pslots * d * 4);
    total = pslot_ml + align256(pslots * 8);
  }
};

template <int D, Held kHeld>
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream) {
  void (*kern)(DecodeParams);
  int ring;
  if constexpr (kHeld == Held::kInt4) {
    static_assert(Int4Core<D, 2>::kRing >= kRows * kPitch<D> * 4, "the join fits the ring");
    // 8 rows where no item has more, measured above
    const bool few = p.R <= 8 && (p.P == 0 || p.B * p.R <= 8);
    kern = few ? paged_decode4_kernel<D, 1> : paged_decode4_kernel<D, 2>;
    ring = kWarps * Int4Core<D, 1>::kRing;
  } else {
    static_assert(Stage<D, kHeld>::kRing >= kRows * kPitch<D> * 4, "the join fits the ring");
    kern = paged_decode_kernel<D, kHeld>;
    ring = kWarps * Stage<D, kHeld>::kRing;
  }
  const int smem = ring + 4 * (p.B + 1);
  cudaError_t e =
      ensure_smem_limit(reinterpret_cast<const void*>(kern), ring + 4 * (kMaxBatch + 1));
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(std::min(kMaxGrid, kCtasPerSm * sm_count()));
  kern<<<grid, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch(2);
  if (p.prefix_grid > 0) {
    e = launch_prefix_attn(p, D, kHeld == Held::kE4M3, stream);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const unsigned rows = static_cast<unsigned>(p.B) * p.n_q * p.Hq;
  const bool many = rows >= kManyRows;
  cfg.gridDim = dim3(many ? (rows + kWarps - 1) / kWarps : rows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = many ? cudaLaunchKernelEx(&cfg, decode_join_kernel<D, kHeld, 1>, p, grid)
           : cudaLaunchKernelEx(&cfg, decode_join_kernel<D, kHeld, kWarps>, p, grid);
  count_launch(2);
  return e;
}

bool sizes_ok(int B, int n_q, int Hq, int Hk, int prefix_len) {
  return B >= 1 && B <= kMaxBatch && n_q >= 1 && n_q <= kMaxQueries && Hq >= 1 && Hk >= 1 &&
         Hq % Hk == 0 && prefix_len >= 0 &&
         static_cast<long long>(B) * n_q * Hq <= (1LL << 24);
}

}  // namespace
}  // namespace cpring

extern "C" {

void cp_test_set_prefix_path(int path) {
  cpring::g_prefix_path.store(path < 0 ? -1 : path != 0, std::memory_order_relaxed);
}

int64_t cp_paged_attn_decode_workspace_bytes(int B, int n_q, int Hq, int Hk, int d,
                                             int prefix_len) {
  if (!cpring::sizes_ok(B, n_q, Hq, Hk, prefix_len) || (d != 64 && d != 128)) return -1;
  return cpring::Space(B, n_q, Hq, Hk, d, prefix_len).total;
}

cp_status cp_paged_attn_decode(const cp_paged_cache* cache, const void* q,
                               const int64_t* q_strides, const int32_t* seq_lens,
                               const int32_t* prefix_pages, int prefix_len, void* out, float* lse,
                               int B, int n_q, int Hq, void* workspace, int64_t workspace_bytes,
                               cudaStream_t stream) {
  cpring::TraceRange trace_("cp_paged_attn_decode");
  using namespace cpring;
  if (!q || !seq_lens || !out || !lse || !workspace || (prefix_len > 0 && !prefix_pages))
    return CP_ERR_NULL;
  cp_status st = check_cache(cache);
  if (st != CP_OK) return st;
  const int Hk = cache->Hk, d = cache->d;
  if (!sizes_ok(B, n_q, Hq, Hk, prefix_len)) return CP_ERR_SHAPE;
  const long long capacity = static_cast<long long>(cache->max_pages) * cache->page_size;
  if (prefix_len > capacity) return CP_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(seq_lens, 4) ||
      !aligned(prefix_pages, 4) || !aligned(workspace, 256) || !strides_ok(q_strides, 2))
    return CP_ERR_ALIGN;
  const Space sp(B, n_q, Hq, Hk, d, prefix_len);
  if (workspace_bytes < sp.total) return CP_ERR_BUFFER;
  // the units of a call are counted in 32 bits
  const long long G = Hq / Hk, R = G * n_q;
  const bool wide =  // and never without the space for its parts
      cache->elem_bytes > 0 && sp.pslot_ml > sp.pslot_o &&
      wide_prefix(B * R, prefix_len, Hk, d, cache->elem_bytes, cache->page_size);
  const int prefix_rows = wide ? kPrefixRows : kRows,
            prefix_keys = wide ? kPrefixKeys : tile_keys_of(held_by(cache));
  const long long own_rt = (R + kRows - 1) / kRows;
  const long long prefix_rt = (B * R + prefix_rows - 1) / prefix_rows;
  const long long most_tiles = (capacity + kTileKeys - 1) / kTileKeys;
  const long long prefix_tiles =
      (static_cast<long long>(prefix_len) + prefix_keys - 1) / prefix_keys;
  if (((prefix_tiles + kItemCost) * prefix_rt + (most_tiles + kItemCost) * own_rt * B) * Hk >
      0xffffffffLL)
    return CP_ERR_SHAPE;
  if (device_cc() != 103) return CP_ERR_DEVICE;
  DecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache[0] = static_cast<const uint8_t*>(cache->k);
  p.cache[1] = static_cast<const uint8_t*>(cache->v);
  const Held held = held_by(cache);
  for (int i = 0; i < 3; ++i) {  // in bytes
    const int unit = held == Held::kBf16 ? 2 : 1;
    p.cs[0][i] = cache->k_strides[i] * unit;
    p.cs[1][i] = cache->v_strides[i] * unit;
    if (held != Held::kInt4) continue;
    p.ss[0][i] = cache->k_scale_strides[i];
    p.ss[1][i] = cache->v_scale_strides[i];
  }
  if (held == Held::kInt4) {
    p.scales[0] = static_cast<const uint8_t*>(cache->k_scale);
    p.scales[1] = static_cast<const uint8_t*>(cache->v_scale);
  }
  p.descale[0] = cache->k_descale;
  p.descale[1] = cache->v_descale;
  p.table = cache->page_table;
  p.table_stride = cache->table_stride;
  p.seq_lens = seq_lens;
  p.prefix_pages = prefix_pages;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.err = device_error_word();
  if (!p.err) return CP_ERR_CUDA;
  char* const ws = static_cast<char*>(workspace);
  p.starts = reinterpret_cast<unsigned*>(ws + sp.starts);
  p.slot_o = reinterpret_cast<float*>(ws + sp.slot_o);
  p.slot_ml = reinterpret_cast<float*>(ws + sp.slot_ml);
  p.whole_o = reinterpret_cast<float*>(ws + sp.whole_o);
  p.whole_ml = reinterpret_cast<float*>(ws + sp.whole_ml);
  p.pslot_o = reinterpret_cast<float*>(ws + sp.pslot_o);
  p.pslot_ml = reinterpret_cast<float*>(ws + sp.pslot_ml);
  p.qb = q_strides ? q_strides[0] : static_cast<long long>(n_q) * Hq * d;
  p.qs = q_strides ? q_strides[1] : static_cast<long long>(Hq) * d;
  p.qh = q_strides ? q_strides[2] : d;
  p.scale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
  p.B = B; p.n_q = n_q; p.Hq = Hq; p.Hk = Hk;
  p.G = static_cast<int>(G); p.R = static_cast<int>(R);
  p.own_tiles_of_rows = static_cast<int>(own_rt);
  p.prefix_rows = prefix_rows;
  p.prefix_row_tiles = static_cast<int>(prefix_rt);
  p.P = prefix_len;
  p.prefix_tiles = static_cast<int>(prefix_tiles);
  if (wide)
    p.prefix_grid = static_cast<int>(std::min<long long>(
        std::min(kMaxPrefixGrid, sm_count()), prefix_tiles * prefix_rt * Hk));
  p.timeout_ns = test_wait_limit_ns();
  p.fault_drop_k = test_fault_drop();
  p.n_pages = cache->n_pages;
  p.set_page_size(cache->page_size);
  p.alike = std::equal(p.cs[0], p.cs[0] + 3, p.cs[1]);
  p.capacity = capacity;
  auto launch = [&](auto dim) {
    constexpr int kD = decltype(dim)::value;
    return held == Held::kBf16   ? launch_decode<kD, Held::kBf16>(p, stream)
           : held == Held::kE4M3 ? launch_decode<kD, Held::kE4M3>(p, stream)
                                 : launch_decode<kD, Held::kInt4>(p, stream);
  };
  const cudaError_t e = d == 128 ? launch(std::integral_constant<int, 128>())
                                 : launch(std::integral_constant<int, 64>());
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // extern "C"
