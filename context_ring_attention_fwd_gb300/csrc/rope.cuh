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
// 32 bits of the 64-bit product are the angle in units of 2^-31 half turns: the
// nearest quarter turn (the top two bits, rounded) is taken off before the rest,
// an eighth of a turn at most, is rounded to fp32.  So the angle is off by 2^-27
// half turns, 2.3e-8, where half a turn rounded whole would be off by 9.4e-8.
__device__ __forceinline__ void angle_of(int position, uint64_t fraction, float& c, float& s) {
  const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(position)) * fraction;
  const uint32_t u = static_cast<uint32_t>(turns >> 32);
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  float sn, cs;
  sincospif(static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * 0x1p-31f, &sn, &cs);
  const bool odd = quarter & 1u;
  c = __uint_as_float(__float_as_uint(odd ? sn : cs) ^ (((quarter + 1u) & 2u) << 30));
  s = __uint_as_float(__float_as_uint(odd ? cs : sn) ^ ((quarter & 2u) << 30));
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

// The arithmetic is on pairs of neighbouring fp32 values, two to an
// instruction (fma / mul / add.rn.f32x2, each value rounded to nearest): these
// kernels issue about as many instructions as the bytes they move leave time for.
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 neg2(f32x2 v) { return v ^ 0x8000000080000000ull; }
__device__ __forceinline__ f32x2 swap2(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack2(hi, lo);
}
__device__ __forceinline__ float sum2(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return lo + hi;
}

// One 16-byte vector as pairs of fp32 values and back (rounded to nearest).
// A lane's two vectors are z[0 .. NP / 2) and z[NP / 2 .. NP).
template <int NP>
__device__ __forceinline__ void unpack(const uint4& v, f32x2 (&z)[NP], int at, __nv_bfloat16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    z[at + i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <int NP>
__device__ __forceinline__ void unpack(const uint4& v, f32x2 (&z)[NP], int at, float) {
  z[at] = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
  z[at + 1] = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <int NP>
__device__ __forceinline__ uint4 repack(const f32x2 (&z)[NP], int at, __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(z[at + i], lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int NP>
__device__ __forceinline__ uint4 repack(const f32x2 (&z)[NP], int at, float) {
  float f[4];
  unpack2(z[at], f[0], f[1]);
  unpack2(z[at + 1], f[2], f[3]);
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}

// cos and sin of the lane's NP angles as the pairs that its entries meet:
// entry pair z[i] turns to own[i] * z[i] + other[i] * partner, where the partner
// is z[i +- NP / 2], or z[i] with its entries exchanged in the interleaved form.
// sign -1 turns back.
template <int NP, bool kInterleaved>
__device__ __forceinline__ void turn_factors(const float (&c)[NP], const float (&s)[NP],
                                             float sign, f32x2 (&own)[NP], f32x2 (&other)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (kInterleaved) {
      own[i] = pack2(c[i], c[i]);
      other[i] = pack2(-sign * s[i], sign * s[i]);
    } else {
      const int e = (2 * i) % NP;
      const float t = i < NP / 2 ? -sign : sign;
      own[i] = pack2(c[e], c[e + 1]);
      other[i] = pack2(t * s[e], t * s[e + 1]);
    }
  }
}
template <int NP, bool kInterleaved>
__device__ __forceinline__ f32x2 partner(const f32x2 (&z)[NP], int i) {
  return kInterleaved ? swap2(z[i]) : z[(i + NP / 2) % NP];
}
// The lane's entries turned.
template <int NP, bool kInterleaved>
__device__ __forceinline__ void turn(f32x2 (&z)[NP], const f32x2 (&own)[NP],
                                     const f32x2 (&other)[NP]) {
  f32x2 y[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    y[i] = fma2(z[i], own[i], mul2(partner<NP, kInterleaved>(z, i), other[i]));
#pragma unroll
  for (int i = 0; i < NP; ++i) z[i] = y[i];
}

// A warp's ring of two stages of kVecs 16-byte vectors per lane.  A lane copies
// what it will read itself, so nothing is ordered but its own copies: the next
// unit of work is under way while one is computed, without registers for it.
template <int kVecs>
struct Ring {
  static constexpr int kBytes = 2 * kVecs * 512;  // per warp
  uint32_t base;
  __device__ uint32_t at(int stage, int v) const { return base + (stage * kVecs + v) * 512; }
  __device__ void copy(int stage, int v, const void* src, bool there) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(stage, v)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
  }
  __device__ uint4 read(int stage, int v) const {
    uint4 u;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "r"(at(stage, v))
                 : "memory");
    return u;
  }
};
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the last committed group have landed.
__device__ __forceinline__ void copies_wait_all_but_last() {
  asm volatile("cp.async.wait_group 1;" ::: "memory");
}

// Sum over the lanes of one row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum over the lane's entries of a * b.
template <int NP>
__device__ __forceinline__ float dot(const f32x2 (&a)[NP], const f32x2 (&b)[NP]) {
  f32x2 x = mul2(a[0], b[0]), y = mul2(a[1], b[1]);
#pragma unroll
  for (int i = 2; i < NP; i += 2) {
    x = fma2(a[i], b[i], x);
    y = fma2(a[i + 1], b[i + 1], y);
  }
  return sum2(x) + sum2(y);
}

// A gain vector laid out for a row's lanes: the block copies it to shared memory
// once (ones where it is null), lanes read their columns as pairs.
__device__ __forceinline__ void stage_gain(float* to, const float* __restrict__ w, int d) {
  for (int i = threadIdx.x; i < d; i += blockDim.x) to[i] = w != nullptr ? __ldg(w + i) : 1.f;
}
template <int NP>
__device__ __forceinline__ void load_gain(const float* w, int lo, int hi, f32x2 (&z)[NP]) {
#pragma unroll
  for (int i = 0; i < NP / 2; i += 2) {
    const float4 a = *reinterpret_cast<const float4*>(w + lo + 2 * i);
    const float4 b = *reinterpret_cast<const float4*>(w + hi + 2 * i);
    z[i] = pack2(a.x, a.y);
    z[i + 1] = pack2(a.z, a.w);
    z[NP / 2 + i] = pack2(b.x, b.y);
    z[NP / 2 + i + 1] = pack2(b.z, b.w);
  }
}

}  // namespace
}  // namespace cpring
