// One warp's part of paged_decode_kernel over a cache in 4 bits: 32 keys of each 128-key
// tile, and kNT x 8 rows of queries.
//
// Bound by instructions: a key of one head is 144 bytes (d = 128) and 256 codes to widen, so
// at the copy rate an SM has 6 cycles for it.  What keeps the count down:
//  - Both products are transposed, S^T = K Q^T and O^T = V^T P^T, with the codes as the
//    16-row operand of m16n8k16 and 8 rows of queries as the other: the 4 to 8 rows that a key
//    head usually has fill it, where they would leave most of a 16-row one empty.
//  - A word's eight codes become four pairs of fp16 with a shift, four logic operations and
//    four fused multiply-adds.  (w & 0x000f000f) | 0x64006400 is 1024 + code in each half and
//    (w & 0x00f000f0) | 0x54005400 is 64 + code of the next four bits, so (x + code) s - (x + 8) s
//    is (code - 8) s, exactly: with s = scale / 16, 4 significant bits, 1032 s and 72 s fit
//    fp16's 11 bits and its range, and so does the result.  (The 16 goes to the softmax scale
//    and to the output.)
//  - The order of a dot product's terms is free, so the codes of K are paired as their
//    bits lie (i with i + 4) and Q's entries are put in that order.  V's come from
//    ldmatrix.trans, which moves 16 bits, four neighbouring columns, of two keys to a lane.
//  - P^T leaves the first product with a key to a lane and enters the second with a row to a
//    lane: movmatrix turns its 8 x 8 pieces.
//  - A row's reference moves only when a score passes it by 2^5 (all but a few of the first tiles
//    of an item go without the maximum's shuffles), and V is read while the softmax waits.
// 660 instructions for 32 keys and 8 rows; issue slots are 66 % used in the long case, where the
// whole call runs at 76 % of the copy rate (paged_decode.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "paged_decode.h"
#include "ptx.cuh"

namespace cpring {
namespace {

// kBytes (4 or 8) to shared memory, or zeros.
template <int kBytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src),
               "r"(there ? kBytes : 0), "n"(kBytes)
               : "memory");
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// What widens codes of one scale (of two, one in each half): s / 16, and -72 and -1032 times it.
struct Widener {
  uint32_t s, m72, m1032;
  __device__ explicit Widener(uint32_t scales) {
    s = mul_f16x2(scales, 0x2c002c00u);      // 1 / 16
    m72 = mul_f16x2(scales, 0xc480c480u);    // -4.5
    m1032 = mul_f16x2(scales, 0xd408d408u);  // -64.5
  }
  // half2 i: the codes i (low half) and i + 4 (high half) of a word.
  // (lop3 is written out: from the expression (x & mask) | exponent the compiler makes two
  // operations, 62 us instead of 54 in the kernel for 32 sequences of up to 16K.)
  __device__ __forceinline__ void operator()(uint32_t w, uint32_t (&v)[4]) const {
    const uint32_t t = w >> 8;
    auto low = [&](uint32_t x) {
      uint32_t r;
      asm("{\n\t.reg .b32 n;\n\tlop3.b32 n, %1, 0x000f000f, %2, 0xea;\n\t"
          "fma.rn.f16x2 %0, n, %3, %4;\n\t}"
          : "=r"(r)
          : "r"(x), "r"(0x64006400u), "r"(s), "r"(m1032));
      return r;
    };
    auto high = [&](uint32_t x) {
      uint32_t r;
      asm("{\n\t.reg .b32 n;\n\tlop3.b32 n, %1, 0x00f000f0, %2, 0xea;\n\t"
          "fma.rn.f16x2 %0, n, %3, %4;\n\t}"
          : "=r"(r)
          : "r"(x), "r"(0x54005400u), "r"(s), "r"(m72));
      return r;
    };
    v[0] = low(w);
    v[1] = high(w);
    v[2] = low(t);
    v[3] = high(t);
  }
};

template <int D, int kNT>
struct Int4Core {
  static constexpr int kKeys = 32;              // of a tile, for this warp
  static constexpr int kRowBytes = D / 2, kScaleBytes = D / kBlock, kChunks = kRowBytes / 16;
  static constexpr int kV = kKeys * kRowBytes;  // of a stage: where V starts
  static constexpr int kScales = 2 * kV;        // K's scales, then V's
  static constexpr int kBytes = kScales + 2 * kKeys * kScaleBytes;
  static constexpr int kCount = D == 128 ? 2 : 4;  // stages
  static constexpr int kRing = kCount * kBytes;
  // P is held times 2^kShift and at most 2^kSlack, so below 2^15 in fp16, which flushes what
  // is 2^-34 of the reference.
  static constexpr float kShift = 10.f, kSlack = 5.f;
  static constexpr float kUnit = 16.f;          // values are held divided by it

  uint32_t q[kNT][D / 16][2];
  float sc[kNT][2];    // of rows 2 c4 and 2 c4 + 1
  float lift[kNT][2];  // kShift less the rows' references (infinity: no key yet)
  float l[kNT][2];
  float o[kNT][D / 16][4];

  // Chunk c of row r at c ^ (r / 2 mod 4), for rows of 32 bytes c ^ (r / 4 mod 2): free of bank
  // conflicts by rows and by columns.
  __device__ static uint32_t at(uint32_t base, int row, int chunk) {
    return base + row * kRowBytes + ((chunk ^ ((row / (8 / kChunks)) & (kChunks - 1))) << 4);
  }

  // The rows row0 .. row0 + rows - 1 of the item (later ones repeat the last).
  template <class Rows>
  __device__ __forceinline__ void load_queries(Rows&& query, int rows, float scale, int lane) {
    const int quad = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const uint4* const src = reinterpret_cast<const uint4*>(
          query(min(8 * nt + quad, rows - 1)) + c4 * (D / 4));
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
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float up, down;
      fp16_row_scale(top, up, down);
      const float mine = scale * kUnit * down;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sc[nt][e] = __shfl_sync(0xffffffffu, mine, (2 * c4 + e) * 4);
        lift[nt][e] = INFINITY;
        l[nt][e] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {  // two steps to a word, whose codes i and i + 4 pair
        const int x = 8 * (k / 2) + 2 * (k % 2);
        q[nt][k][0] = pack_f16(z[x] * up, z[x + 4] * up);
        q[nt][k][1] = pack_f16(z[x + 1] * up, z[x + 5] * up);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][k][e] = 0.f;
      }
    }
  }

  __device__ static void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }

  // A stage's words of K row `row` for lane c4, and what widens them (two blocks at d = 128).
  template <int kWords>
  __device__ static __forceinline__ void load_words(uint32_t addr, uint32_t (&u)[kWords]) {
    if constexpr (kWords == 4)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                   : "r"(addr));
    else
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(u[0]), "=r"(u[1]) : "r"(addr));
  }

  // One tile, of whose keys this warp's first `left` exist.
  __device__ __forceinline__ void step(uint32_t stage, int left, int lane) {
    const int quad = lane >> 2, c4 = lane & 3;
    constexpr int kWords = D / 32;
    // ---- S^T: keys quad and quad + 8 of each 16, rows 2 c4 and 2 c4 + 1
    float s[2][kNT][4];
    uint32_t u[2][2][kWords], two[2][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = mt * 16 + h * 8 + quad;
        load_words<kWords>(D == 128 ? at(stage, row, c4) : at(stage, row, c4 / 2) + c4 % 2 * 8,
                           u[mt][h]);
        const uint32_t from = stage + kScales + row * kScaleBytes;
        if constexpr (D == 128)
          asm volatile("ld.shared.u16 %0, [%1];" : "=r"(two[mt][h]) : "r"(from + 2 * c4));
        else
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(two[mt][h]) : "r"(from + c4));
        two[mt][h] = half2_of_codes(two[mt][h]);
      }
    }
#pragma unroll
    for (int b = 0; b < D / 64; ++b)  // the lane's blocks of 16, two words each
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const Widener w0(__byte_perm(two[mt][0], 0, b ? 0x3232 : 0x1010));
        const Widener w1(__byte_perm(two[mt][1], 0, b ? 0x3232 : 0x1010));
#pragma unroll
        for (int x = 2 * b; x < 2 * b + 2; ++x) {
          uint32_t v0[4], v1[4];
          w0(u[mt][0][x], v0);
          w1(u[mt][1][x], v1);
          const uint32_t a0[4] = {v0[0], v1[0], v0[1], v1[1]}, a1[4] = {v0[2], v1[2], v0[3], v1[3]};
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            mma(s[mt][nt], a0, q[nt][2 * x][0], q[nt][2 * x][1]);
            mma(s[mt][nt], a1, q[nt][2 * x + 1][0], q[nt][2 * x + 1][1]);
          }
        }
      }
    // ---- V of the tile, and the scales of keys 2 c4 and 2 c4 + 1 and of the two 8 further,
    // while the softmax waits for its steps
    constexpr int kHalf = D / 64;
    uint32_t v[2][kHalf][4], r4[2][2][2 * kHalf];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int y = 0; y < 2; ++y)
        load_words<2 * kHalf>(
            stage + kScales + (kKeys + mt * 16 + 8 * y + 2 * c4) * kScaleBytes, r4[mt][y]);
#pragma unroll
      for (int x = 0; x < kHalf; ++x) {
        const uint32_t addr = at(stage + kV, mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7),
                                 2 * x + (lane >> 4));
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[mt][x][0]), "=r"(v[mt][x][1]), "=r"(v[mt][x][2]), "=r"(v[mt][x][3])
                     : "r"(addr));
      }
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (left < kKeys && mt * 16 + (e >> 1) * 8 + quad >= left) s[mt][nt][e] = -INFINITY;
    // ---- P against a reference that moves only when a score passes it by 2^kSlack
    float x[2][kNT][4];  // the exponents
    auto against = [&](const float (&from)[kNT][2]) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[mt][nt][e] = fmaf(s[mt][nt][e], sc[nt][e & 1], from[nt][e & 1]);
    };
    against(lift);
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      float top = lift[nt][0] == INFINITY || lift[nt][1] == INFINITY ? INFINITY : -INFINITY;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, x[mt][nt][e]);
      over |= top > kShift + kSlack;
    }
    if (__any_sync(0xffffffffu, over)) {
      float from[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]),
                          fmaxf(s[1][nt][e], s[1][nt][e + 2])) * sc[nt][e];
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
          const float old = lift[nt][e];
          lift[nt][e] = fminf(old, kShift - y);
          a[e] = old == INFINITY ? 0.f : ptx::ex2(lift[nt][e] - old);
          from[nt][e] = lift[nt][e] == INFINITY ? kShift : lift[nt][e];  // no key yet
          l[nt][e] *= a[e];
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][k][e] *= a[e & 1];
      }
      against(from);
    }
    uint32_t p[2][kNT][2];  // of 16 keys: the first 8, the others
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = ptx::ex2(x[mt][nt][e]);
          l[nt][e & 1] += y[e];
        }
        p[mt][nt][0] = transposed8x8(pack_f16(y[0], y[1]));
        p[mt][nt][1] = transposed8x8(pack_f16(y[2], y[3]));
      }
    // ---- O^T += V^T P^T
    const uint32_t pick = 0x6240u + 0x1111u * (quad >> 2);  // of a chunk's two blocks, this lane's
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int h = 0; h < kHalf; ++h) {
        const uint32_t c0 = __byte_perm(r4[mt][0][h], r4[mt][0][kHalf + h], pick);
        const uint32_t c1 = __byte_perm(r4[mt][1][h], r4[mt][1][kHalf + h], pick);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const Widener w0(half2_of_codes(x ? c0 >> 16 : c0 & 0xffffu));
          const Widener w1(half2_of_codes(x ? c1 >> 16 : c1 & 0xffffu));
          uint32_t lo[4], hi[4];  // column 4 quad + i of the chunk: two keys each
          w0(v[mt][h][2 * x], lo);
          w1(v[mt][h][2 * x + 1], hi);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a[4] = {lo[2 * i], lo[2 * i + 1], hi[2 * i], hi[2 * i + 1]};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma(o[nt][2 * (2 * h + x) + i], a, p[mt][nt][0], p[mt][nt][1]);
          }
        }
      }
  }

  __device__ __forceinline__ float m(int nt, int e) const { return kShift - lift[nt][e]; }

  // The sums of the rows' exponentials over the lanes that share them.
  __device__ __forceinline__ void sum_lanes() {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
  }

  // Row `row` (8 nt + 2 c4 + e) of O times f to `to`.
  __device__ __forceinline__ void store_row(float* to, int nt, int e, float f, int lane) const {
    const int quad = lane >> 2;
#pragma unroll
    for (int ch = 0; ch < kChunks; ++ch)
      *reinterpret_cast<float4*>(to + ch * 32 + quad * 4) =
          make_float4(o[nt][2 * ch][e] * f, o[nt][2 * ch][2 + e] * f, o[nt][2 * ch + 1][e] * f,
                      o[nt][2 * ch + 1][2 + e] * f);
  }
};

}  // namespace
}  // namespace cpring
