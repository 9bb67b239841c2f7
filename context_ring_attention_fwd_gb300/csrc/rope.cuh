// Device helpers of the kernels that norm and rotate the rows of Q and K
// (norm_rope.cu) and append them to a paged cache (paged_append.cu).
//
// A row is one head's d-vector of one token.  Rotating it by position p means
// that each of its rot / 2 pairs (a_c, b_c) becomes
//   (a cos t - b sin t, b cos t + a sin t),  t = p * inv_freq[c],
// where the pair is (x[c], x[c + rot / 2]), or (x[2 c], x[2 c + 1]) in the
// interleaved form; the entries from rot on stay.
//
// Layout of a row over lanes: a lane owns NP pairs as two 16-byte vectors
// (NP = 8 bf16 or 4 fp32), so a row takes d / (2 NP) lanes and both members
// of a pair sit in one lane: the rotation needs no shuffle in either form,
// and every access is 16 bytes wide.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cpring {
namespace {

template <typename T, int D>
struct RowLayout {
  static constexpr int kPairs = 16 / static_cast<int>(sizeof(T));  // pairs per lane (NP)
  static constexpr int kLanes = D / (2 * kPairs);                  // lanes per row
  static constexpr int kRows = 32 / kLanes;                        // rows per warp
  // Of a lane's NP angles it computes kAngles itself and takes the others
  // from the lanes that hold the same columns of the warp's other rows.
  static constexpr int kAngles = kPairs / kRows;
  static_assert(kAngles >= 1 && kAngles * kRows == kPairs, "angles split over the warp's rows");
};

// Where lane l's two vectors of a row start, and whether they are rotated.
template <int NP>
__device__ __forceinline__ void lane_columns(int l, int rot, bool interleaved, int& lo, int& hi,
                                             bool& turned) {
  const int c0 = l * NP;
  turned = c0 < rot / 2;
  if (turned && !interleaved) {
    lo = c0;
    hi = c0 + rot / 2;
  } else {
    lo = turned ? 2 * c0 : rot + 2 * (c0 - rot / 2);
    hi = lo + NP;
  }
}

// inv_freq / (2 pi) as a 64-bit fraction of a turn, modulo one turn.  With
// inv_freq = m 2^e (m an integer below 2^24) and 1 / (2 pi) = C 2^-66, that is
// m C 2^(e - 2), taken from the 88-bit product by a shift.  Angles are then
// exact integer products modulo a turn: at position p the error is p 2^-64
// turns, so far positions lose nothing to range reduction and no 64-bit
// floating-point arithmetic (2 operations a clock on this GPU) is needed.
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  constexpr uint64_t kInvTwoPi = 0xa2f9836e4e441529ull;  // floor(2^66 / (2 pi))
  const uint32_t bits = __float_as_uint(inv_freq);
  const int ex = static_cast<int>((bits >> 23) & 0xffu);
  const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int right = 152 - (ex ? ex : 1);  // m C 2^(e - 2), e = ex - 150
  const uint64_t hi = __umul64hi(m, kInvTwoPi), lo = m * kInvTwoPi;
  uint64_t f;
  if (right <= 0)
    f = right > -64 ? lo << -right : 0;
  else if (right < 64)
    f = (hi << (64 - right)) | (lo >> right);
  else
    f = right < 128 ? hi >> (right - 64) : 0;
  return (bits >> 31) ? 0ull - f : f;
}

// cos and sin of position * inv_freq, from the fraction of a turn.  The top
// 32 bits of the 64-bit product, read as signed, are the angle in units of
// 2^-31 half turns.
__device__ __forceinline__ void angle_of(int position, uint64_t fraction, float& c, float& s) {
  const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(position)) * fraction;
  sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f, &s, &c);
}

// The fractions of the angles that this lane computes (kAngles of its row
// columns' NP); zero where the columns are not rotated.
template <class Lay>
__device__ __forceinline__ void load_fractions(const float* __restrict__ inv_freq, int l, int g,
                                               bool turned, uint64_t (&f)[Lay::kAngles]) {
#pragma unroll
  for (int j = 0; j < Lay::kAngles; ++j)
    f[j] = turned ? turn_fraction(inv_freq[l * Lay::kPairs + g * Lay::kAngles + j]) : 0ull;
}

// cos / sin of the lane's NP pairs at one position (every lane of the warp
// calls it with the same position).
template <class Lay>
__device__ __forceinline__ void row_angles(int position, const uint64_t (&f)[Lay::kAngles], int l,
                                           float (&c)[Lay::kPairs], float (&s)[Lay::kPairs]) {
  float cj[Lay::kAngles], sj[Lay::kAngles];
#pragma unroll
  for (int j = 0; j < Lay::kAngles; ++j) angle_of(position, f[j], cj[j], sj[j]);
#pragma unroll
  for (int e = 0; e < Lay::kPairs; ++e) {
    const int src = (e / Lay::kAngles) * Lay::kLanes + l;
    c[e] = __shfl_sync(0xffffffffu, cj[e % Lay::kAngles], src);
    s[e] = __shfl_sync(0xffffffffu, sj[e % Lay::kAngles], src);
  }
}

// One 16-byte vector as fp32 values and back (each value rounded to nearest).
__device__ __forceinline__ void unpack(const uint4& v, float (&z)[16], int at, __nv_bfloat16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[at + 2 * i] = __uint_as_float(w[i] << 16);
    z[at + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& v, float (&z)[8], int at, float) {
  z[at] = __uint_as_float(v.x);
  z[at + 1] = __uint_as_float(v.y);
  z[at + 2] = __uint_as_float(v.z);
  z[at + 3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint4 repack(const float (&z)[16], int at, __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(z[at + 2 * i], z[at + 2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 repack(const float (&z)[8], int at, float) {
  return make_uint4(__float_as_uint(z[at]), __float_as_uint(z[at + 1]), __float_as_uint(z[at + 2]),
                    __float_as_uint(z[at + 3]));
}

// Rotate the lane's pairs in place (sign -1 turns back).
template <int NP>
__device__ __forceinline__ void rotate(float (&z)[2 * NP], const float (&c)[NP],
                                       const float (&s)[NP], bool interleaved, float sign) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float a = z[2 * e], b = z[2 * e + 1], t = sign * s[e];
      z[2 * e] = a * c[e] - b * t;
      z[2 * e + 1] = b * c[e] + a * t;
    }
  } else {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float a = z[e], b = z[e + NP], t = sign * s[e];
      z[e] = a * c[e] - b * t;
      z[e + NP] = b * c[e] + a * t;
    }
  }
}

// Sum over the lanes of one row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int N>
__device__ __forceinline__ float sum_squares(const float (&z)[N]) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    a = fmaf(z[i], z[i], a);
    b = fmaf(z[i + 1], z[i + 1], b);
  }
  return a + b;
}

// The lane's columns of an fp32 vector of length d.
template <int NP>
__device__ __forceinline__ void load_columns(const float* __restrict__ w, int lo, int hi,
                                             float (&z)[2 * NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    z[i] = __ldg(w + lo + i);
    z[NP + i] = __ldg(w + hi + i);
  }
}

}  // namespace
}  // namespace cpring
