// The softmax of the tcgen05 forward kernels, one thread to a row of a 128 x 128
// tile of scores: scores from TMEM with their mask, row maxima, and P = 2^(s sc -
// base) as packed bf16 pairs (or E4M3 quads) with its row sums.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_common.cuh"
#include "ptx.cuh"

// CPRING_PACKED_F32X2 (a tuning switch; the same result up to rounding): fast pass: scale-and-shift
// and row sum with the paired fp32 FMA / ADD (two elements per instruction).
#ifndef CPRING_PACKED_F32X2
#define CPRING_PACKED_F32X2 1
#endif

namespace cpring {
namespace {

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// This thread's 128 scores of the S tile (one TMEM lane), with columns
// outside [c_lo, c_hi] set to -inf.
__device__ __forceinline__ void load_scores(uint32_t tS, int c_lo, int c_hi,
                                            uint32_t (&sv)[4][32]) {
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) ptx::tmem_ld32(tS + ch * 32, sv[ch]);
  ptx::tmem_wait_ld();
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) ptx::reg_fence(sv[ch]);
  if (c_lo > 0 || c_hi < kTileRows - 1) {
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        const int cc = ch * 32 + x;
        if (cc < c_lo || cc > c_hi) sv[ch][x] = __float_as_uint(-INFINITY);
      }
  }
}

__device__ __forceinline__ float row_max(const uint32_t (&sv)[4][32]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int ch = 0; ch < 4; ++ch)
#pragma unroll
    for (int x = 0; x < 32; x += 2)
      m[ch] = max3(m[ch], __uint_as_float(sv[ch][x]), __uint_as_float(sv[ch][x + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Two exponent arguments s * sc - base at once (paired fp32 FMA).
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float sc,
                                     float nb) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(sc), "f"(nb));
}
// acc (two fp32 lanes) += (p0, p1) with one paired add.
__device__ __forceinline__ void add2(uint64_t& acc, float p0, float p1) {
  asm("{\n\t.reg .b64 rp;\n\tmov.b64 rp, {%1, %2};\n\tadd.rn.f32x2 %0, %0, rp;\n\t}"
      : "+l"(acc)
      : "f"(p0), "f"(p1));
}
__device__ __forceinline__ float sum2(uint64_t acc) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(acc));
  return lo + hi;
}

// P = 2^(s * sc - base), its row sum, and the raw row max of the scores.  P is
// packed as bf16 pairs (P[2c] low, P[2c+1] high) into pk[0..1][32], or for
// the FP8 form as E4M3 quads (P[4c] lowest byte) into pk[0][32].
// kPaired (the step kernel, where every tile takes this path): paired fp32
// FMA / ADD.  The fused kernel reaches it only on the first tile of a row or
// a rare redo and keeps scalar arithmetic there, which measured faster for
// its hot loop.
template <bool kFp8 = false, bool kPaired = false>
__device__ __forceinline__ void exponentials(const uint32_t (&sv)[4][32], float sc, float base,
                                             uint32_t (&pk)[2][32], float& lsum, float& mx) {
  float ls[4] = {0.f, 0.f, 0.f, 0.f};
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  if constexpr (kFp8) {
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float s0 = __uint_as_float(sv[ch][4 * x]);
        const float s1 = __uint_as_float(sv[ch][4 * x + 1]);
        const float s2 = __uint_as_float(sv[ch][4 * x + 2]);
        const float s3 = __uint_as_float(sv[ch][4 * x + 3]);
        m[ch] = max3(m[ch], max3(s0, s1, s2), s3);
        const float p0 = ptx::ex2(fmaf(s0, sc, -base));
        const float p1 = ptx::ex2(fmaf(s1, sc, -base));
        const float p2 = ptx::ex2(fmaf(s2, sc, -base));
        const float p3 = ptx::ex2(fmaf(s3, sc, -base));
        ls[ch] += (p0 + p1) + (p2 + p3);
        pk[0][ch * 8 + x] = ptx::pack_e4m3x4(p0, p1, p2, p3);
      }
  } else if (kPaired) {
    // paired fp32 FMA / ADD, two scores per instruction
    uint64_t acc = 0;
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float s0 = __uint_as_float(sv[ch][2 * x]);
        const float s1 = __uint_as_float(sv[ch][2 * x + 1]);
        m[ch] = max3(m[ch], s0, s1);
        float e0, e1;
        fma2(e0, e1, s0, s1, sc, -base);
        const float p0 = ptx::ex2(e0);
        const float p1 = ptx::ex2(e1);
        add2(acc, p0, p1);
        pk[ch >> 1][(ch & 1) * 16 + x] = ptx::pack_bf16(p0, p1);
      }
    ls[0] = sum2(acc);
  } else {
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float s0 = __uint_as_float(sv[ch][2 * x]);
        const float s1 = __uint_as_float(sv[ch][2 * x + 1]);
        m[ch] = max3(m[ch], s0, s1);
        const float p0 = ptx::ex2(fmaf(s0, sc, -base));
        const float p1 = ptx::ex2(fmaf(s1, sc, -base));
        ls[ch] += p0 + p1;
        pk[ch >> 1][(ch & 1) * 16 + x] = ptx::pack_bf16(p0, p1);
      }
  }
  lsum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
  mx = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// P for two 32-column chunks of S against `base`, into pk row `half`.
__device__ __forceinline__ void exp_chunks(const uint32_t (&sv)[4][32], int half, float sc,
                                           float base, uint32_t (&pk)[2][32], uint64_t& acc,
                                           float& ls) {
#pragma unroll
  for (int cc = 0; cc < 2; ++cc) {
    const int ch = 2 * half + cc;
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float s0 = __uint_as_float(sv[ch][2 * x]);
      const float s1 = __uint_as_float(sv[ch][2 * x + 1]);
      float e0, e1;
      if (CPRING_PACKED_F32X2) {
        fma2(e0, e1, s0, s1, sc, -base);
      } else {
        e0 = fmaf(s0, sc, -base);
        e1 = fmaf(s1, sc, -base);
      }
      const float p0 = ptx::ex2(e0);
      const float p1 = ptx::ex2(e1);
      if (CPRING_PACKED_F32X2) {
        add2(acc, p0, p1);
      } else {
        ls += p0 + p1;
      }
      pk[half][cc * 16 + x] = ptx::pack_bf16(p0, p1);
    }
  }
}

// The FP8 form of exp_chunks: P as E4M3 quads into pk[0] (P[4c] lowest byte).
__device__ __forceinline__ void exp_chunks_f8(const uint32_t (&sv)[4][32], int half, float sc,
                                              float base, uint32_t (&pk)[2][32], uint64_t& acc) {
#pragma unroll
  for (int cc = 0; cc < 2; ++cc) {
    const int ch = 2 * half + cc;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      float e0, e1, e2, e3;
      fma2(e0, e1, __uint_as_float(sv[ch][4 * x]), __uint_as_float(sv[ch][4 * x + 1]), sc, -base);
      fma2(e2, e3, __uint_as_float(sv[ch][4 * x + 2]), __uint_as_float(sv[ch][4 * x + 3]), sc, -base);
      const float p0 = ptx::ex2(e0), p1 = ptx::ex2(e1), p2 = ptx::ex2(e2), p3 = ptx::ex2(e3);
      add2(acc, p0, p1);
      add2(acc, p2, p3);
      pk[0][ch * 8 + x] = ptx::pack_e4m3x4(p0, p1, p2, p3);
    }
  }
}

// exp_chunks_f8 with the exponentials in half precision: 2^x for two keys
// per ex2.approx.f16x2, E4M3 from the half pair, and the row sum of each
// 32-key chunk formed in half pairs (at most 32 * 2^8, exact to 11 bits per
// add) before it enters the fp32 sum.  The argument is rounded to half
// precision (10 bits): 2^x then carries a relative error below 2^-8 for
// x >= -8, far inside E4M3's 2^-4 rounding, and keys further below the
// reference give P under E4M3's smallest step either way.  An argument
// above half precision's range gives +inf, which the caller's 2^8 guard
// sends to the fp32 redo.
__device__ __forceinline__ void exp_chunks_f8h(const uint32_t (&sv)[4][32], int half, float sc,
                                               float base, uint32_t (&pk)[2][32], float& ls) {
#pragma unroll
  for (int cc = 0; cc < 2; ++cc) {
    const int ch = 2 * half + cc;
    uint32_t hs = 0;  // two half-precision zeros
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      float e0, e1, e2, e3;
      fma2(e0, e1, __uint_as_float(sv[ch][4 * x]), __uint_as_float(sv[ch][4 * x + 1]), sc, -base);
      fma2(e2, e3, __uint_as_float(sv[ch][4 * x + 2]), __uint_as_float(sv[ch][4 * x + 3]), sc, -base);
      uint32_t h01, h23;
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h01) : "f"(e1), "f"(e0));
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h23) : "f"(e3), "f"(e2));
      asm("ex2.approx.f16x2 %0, %0;" : "+r"(h01));
      asm("ex2.approx.f16x2 %0, %0;" : "+r"(h23));
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(h01));
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(h23));
      pk[0][ch * 8 + x] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
      asm("add.rn.f16x2 %0, %0, %1;" : "+r"(hs) : "r"(h01));
      asm("add.rn.f16x2 %0, %0, %1;" : "+r"(hs) : "r"(h23));
    }
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
        "add.rn.f32.f16 %0, lo, %0;\n\tadd.rn.f32.f16 %0, hi, %0;\n\t}"
        : "+f"(ls)
        : "r"(hs));
  }
}

// Raw max of the scores of chunks 2*half, 2*half+1 (64 keys).
__device__ __forceinline__ float half_max(const uint32_t (&sv)[4][32], int half) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    m0 = max3(m0, __uint_as_float(sv[2 * half][x]), __uint_as_float(sv[2 * half][x + 1]));
    m1 = max3(m1, __uint_as_float(sv[2 * half + 1][x]), __uint_as_float(sv[2 * half + 1][x + 1]));
  }
  return fmaxf(m0, m1);
}

// bf16 P of 64 keys (half 0: keys 0-63, half 1: keys 64-127) against `base`
// into pk[half], and its row sum.
__device__ __forceinline__ float exp_half(const uint32_t (&sv)[4][32], int half, float sc,
                                          float base, uint32_t (&pk)[2][32]) {
  uint64_t acc = 0;  // two fp32 zeros
  float ls = 0.f;
  exp_chunks(sv, half, sc, base, pk, acc, ls);
  return CPRING_PACKED_F32X2 ? sum2(acc) : ls;
}

// Stores one half of the keys' bf16 P (columns 32*half .. +32 of the lane's
// S row).
__device__ __forceinline__ void store_p_half(uint32_t tS, const uint32_t (&pk)[2][32], int half) {
  ptx::tmem_st32(tS + 32u * half, pk[half]);
}

}  // namespace
}  // namespace cpring
