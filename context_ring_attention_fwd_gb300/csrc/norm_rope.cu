// Per-head RMS norm of queries and keys with the position rotation in the
// same pass, and its backward.
//
//   forward   r = (mean x^2 + eps)^(-1/2),  y = R(p) (x r w)
//   backward  g = R(p)^T dy,  u = x r,  dw = sum over rows of g u,
//             dx = r (g w - u mean(g w u))
// R(p) rotates pairs of a row by p * inv_freq (rope.cuh).  Everything between
// the load and the one rounding at the store is fp32; r is recomputed in the
// backward, which reads x anyway, so the forward saves nothing for it.
//
// Bound by HBM (d = 128, in the kernel: bf16, 64K tokens x 32 heads forward 164 us, 97 % of
// the copy rate, 8K x 64 forward 41 us and backward 66 us; fp32, 8K x 32 forward 40 us; a
// whole backward of 2 x 32K x 32 in bf16 249 us, 95 %): a forward moves 2 d elements per
// row, a backward 3 d.  A warp's
// unit of work is kUnroll * (rows per warp) heads of one token; while it works
// on one, the next one's rows are on their way to its ring in shared memory
// (kUnroll x 1 KB, the backward twice that, on top of the unit at hand).  A
// warp takes several units of a token in a row where there are enough, and works
// out the token's angles once for them.  Units of q come first, then those of k,
// so a warp changes its gain (and, in the backward, hands over its sums for the
// gain's gradient) once.
//
// The gain's gradient: each lane sums its columns over its rows in registers,
// the block's warps are added in shared memory, and a second kernel adds the
// blocks' sums in block order: no atomics, so it is the same in every run.  It starts
// when the first one's last block has left (no block lets it line up earlier): 6 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "rope.cuh"

namespace cpring {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 1024;  // most blocks of a backward: sizes its workspace

struct Rows {        // one of q and k
  const void* x;     // read: [B, S, H, d] with the strides below (elements)
  const void* dy;    // backward: read, contiguous
  void* y;           // written: the rows (contiguous) or dx (with the strides below)
  long long xb, xs, xh;
  long long yb, ys, yh;
  const float* w;    // [d] or null: rows are not normed
  int H;
  int chunks;        // units per token
  int per, groups;   // of which `per` in a row are one warp's; groups of them per token
};

struct RopeParams {
  Rows t[2];
  const float* inv_freq;
  const int32_t* positions;  // [B, S], or null: position = index in the sequence
  float* partial;            // backward: [blocks][2][d]
  int S, rot, interleaved;
  int groups_q, groups;  // of q; of both
  float eps;
};

template <typename T, int D, int kUnroll, bool kBwd, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 2)
    qk_norm_rope_kernel(const RopeParams p) {
  using Lay = RowLayout<T, D>;
  constexpr int NP = Lay::kPairs;
  constexpr int kUnitRows = kUnroll * Lay::kRows;
  constexpr int kRowVecs = kBwd ? 4 : 2;  // a lane's vectors of a row: x, and dy
  using R = Ring<kUnroll * kRowVecs>;
  extern __shared__ __align__(16) uint8_t rings[];
  __shared__ float sums[kBwd ? 2 * kWarps * D : 1];
  __shared__ __align__(16) float gain[2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % Lay::kLanes, g = lane / Lay::kLanes;
  const R ring{static_cast<uint32_t>(__cvta_generic_to_shared(rings)) + warp * R::kBytes +
               lane * 16};

  int lo, hi;
  bool turned;
  lane_columns<NP>(l, p.rot, kInterleaved, lo, hi, turned);

  struct Unit {
    int ti, tok, b, s;
    int chunk, end;  // this unit, and the one behind the last of the warp's group
  };
  auto group_at = [&](unsigned u) {
    Unit x;
    x.ti = u >= static_cast<unsigned>(p.groups_q);
    const Rows& t = p.t[x.ti];
    const int local = static_cast<int>(u) - (x.ti ? p.groups_q : 0);
    x.tok = local / t.groups;
    x.chunk = (local - x.tok * t.groups) * t.per;
    x.end = min(x.chunk + t.per, t.chunks);
    x.b = x.tok / p.S;
    x.s = x.tok - x.b * p.S;
    return x;
  };
  auto fetch = [&](const Unit& x, int stage) {
    const Rows& t = p.t[x.ti];
    const T* const xrow = static_cast<const T*>(t.x) + x.b * t.xb + x.s * t.xs;
    const T* const dy = static_cast<const T*>(t.dy) + static_cast<long long>(x.tok) * t.H * D;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = x.chunk * kUnitRows + g + i * Lay::kRows;
      const bool there = h < t.H;
      const T* const src = xrow + (there ? h : 0) * t.xh;
      ring.copy(stage, i * kRowVecs, src + lo, there);
      ring.copy(stage, i * kRowVecs + 1, src + hi, there);
      if (kBwd) {
        const T* const gsrc = dy + static_cast<long long>(there ? h : 0) * D;
        ring.copy(stage, i * kRowVecs + 2, gsrc + lo, there);
        ring.copy(stage, i * kRowVecs + 3, gsrc + hi, there);
      }
    }
  };
  const unsigned stride = gridDim.x * kWarps;  // unsigned: the last step may pass 2^31
  const unsigned groups = static_cast<unsigned>(p.groups);
  unsigned u = blockIdx.x * kWarps + warp;
  const bool any_q = u < static_cast<unsigned>(p.groups_q);  // the warp has work on q
  Unit next{};
  bool more = u < groups;
  if (more) {
    next = group_at(u);
    fetch(next, 0);
  }
  copies_commit();

  uint64_t frac[Lay::kAngles];
  load_fractions<Lay>(p.inv_freq, l, g, turned, frac);
  stage_gain(gain[0], p.t[0].w, D);
  stage_gain(gain[1], p.t[1].w, D);
  __syncthreads();
  f32x2 dw[kBwd ? NP : 1];
#pragma unroll
  for (int i = 0; i < (kBwd ? NP : 1); ++i) dw[i] = 0ull;

  // Hand the sums for tensor `ti`'s gain to the block (its warp's own slot).
  auto flush = [&](int ti) {
#pragma unroll
    for (int i = 0; i < (kBwd ? NP : 1); ++i) {
      float v[2];
      unpack2(dw[i], v[0], v[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = Lay::kLanes; o < 32; o <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
        const int col = i < NP / 2 ? lo + 2 * i + e : hi + 2 * i - NP + e;
        if (g == 0) sums[(ti * kWarps + warp) * D + col] = v[e];
      }
      dw[i] = 0ull;
    }
  };

  int cur = -1;
  bool fresh = true;  // a new group: another token, or another tensor
  // The factors of the token's turn; the forward's carry the gain too:
  // y[i] = own w[i] x[i] + other w[partner] x[partner], times r.
  f32x2 own[NP], other[NP], w[NP];
  for (int stage = 0; more; stage ^= 1) {
    const Unit x = next;
    const bool renew = fresh;
    if (++next.chunk < next.end) {
      fresh = false;
    } else {
      fresh = true;
      more = u + stride < groups && u + stride > u;
      u += stride;
      if (more) next = group_at(u);
    }
    if (more) fetch(next, stage ^ 1);
    copies_commit();
    const Rows& t = p.t[x.ti];
    const long long flat = static_cast<long long>(x.tok) * t.H * D;  // contiguous [B, S, H, d]
    if (renew) {
      if (kBwd && x.ti != cur && cur >= 0) flush(cur);
      cur = x.ti;
      load_gain<NP>(gain[x.ti], lo, hi, w);
      if (p.rot > 0) {
        float c[NP], sn[NP];
        row_angles<Lay>(p.positions ? __ldg(p.positions + x.tok) : x.s, frac, l, c, sn);
        turn_factors<NP, kInterleaved>(c, sn, kBwd ? -1.f : 1.f, own, other);
        if (!kBwd) {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            own[i] = mul2(own[i], w[i]);
            other[i] = mul2(other[i], partner<NP, kInterleaved>(w, i));
          }
        }
      }
    }
    copies_wait_all_but_last();
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = x.chunk * kUnitRows + g + i * Lay::kRows;
      if (h - g >= t.H) break;  // the same for the whole warp
      f32x2 z[NP];
      unpack<NP>(ring.read(stage, i * kRowVecs), z, 0, T());
      unpack<NP>(ring.read(stage, i * kRowVecs + 1), z, NP / 2, T());
      float r = 1.f;
      if (t.w != nullptr)
        r = rsqrtf(row_sum<Lay::kLanes>(dot<NP>(z, z)) * (1.f / D) + p.eps);
      const f32x2 r2 = pack2(r, r);
      if (!kBwd) {
        if (turned) {
          turn<NP, kInterleaved>(z, own, other);
        } else {
#pragma unroll
          for (int e = 0; e < NP; ++e) z[e] = mul2(z[e], w[e]);
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) z[e] = mul2(z[e], r2);
        if (h < t.H) {
          T* const dst = static_cast<T*>(t.y) + flat + static_cast<long long>(h) * D;
          *reinterpret_cast<uint4*>(dst + lo) = repack<NP>(z, 0, T());
          *reinterpret_cast<uint4*>(dst + hi) = repack<NP>(z, NP / 2, T());
        }
      } else {
        f32x2 gr[NP];
        unpack<NP>(ring.read(stage, i * kRowVecs + 2), gr, 0, T());
        unpack<NP>(ring.read(stage, i * kRowVecs + 3), gr, NP / 2, T());
        if (turned) turn<NP, kInterleaved>(gr, own, other);
        if (t.w != nullptr) {
          f32x2 gw[NP];
#pragma unroll
          for (int e = 0; e < NP; ++e) gw[e] = mul2(gr[e], w[e]);
          const float m = row_sum<Lay::kLanes>(dot<NP>(gw, z)) * r * (1.f / D);
          if (h < t.H) {
            const f32x2 m2 = pack2(-m, -m);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
              const f32x2 un = mul2(z[e], r2);
              dw[e] = fma2(gr[e], un, dw[e]);
              gr[e] = mul2(r2, fma2(un, m2, gw[e]));
            }
          }
        }
        if (h < t.H) {
          T* const dst = static_cast<T*>(t.y) + x.b * t.yb + x.s * t.ys + h * t.yh;
          *reinterpret_cast<uint4*>(dst + lo) = repack<NP>(gr, 0, T());
          *reinterpret_cast<uint4*>(dst + hi) = repack<NP>(gr, NP / 2, T());
        }
      }
    }
  }
  if (kBwd) {
    // A warp writes the slots of tensors that it had no unit of as zeros.
    for (int ti = 0; ti < 2; ++ti)
      if (ti != cur && !(ti == 0 && cur == 1 && any_q))
        for (int i = lane; i < D; i += 32) sums[(ti * kWarps + warp) * D + i] = 0.f;
    if (cur >= 0) flush(cur);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      const float* at = sums + (i / D) * kWarps * D + i % D;
      float v = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) v += at[x * D];
      p.partial[static_cast<size_t>(blockIdx.x) * 2 * D + i] = v;
    }
  }
}

// dw[tensor][column] = sum over blocks, 32 columns a block of this kernel,
// 32 threads a column; the order is fixed by the block count alone.  (The sums are
// written while this kernel waits: no __restrict__, which with const would promise that
// they do not change, and let their loads go before the wait.)
__global__ void __launch_bounds__(1024)
    gain_grad_kernel(const float* partial, int blocks, int d, float* dqw, float* dkw) {
  __shared__ float part[32][33];
  cudaGridDependencySynchronize();
  const int col = blockIdx.x * 32 + threadIdx.x;  // of 2 d
  float v = 0.f;
  for (int b = threadIdx.y; b < blocks; b += 32) v += partial[static_cast<size_t>(b) * 2 * d + col];
  part[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0) return;
  v = 0.f;
#pragma unroll
  for (int y = 0; y < 32; ++y) v += part[y][threadIdx.x];
  float* const out = col < d ? dqw : dkw;
  if (out != nullptr) out[col < d ? col : col - d] = v;
}

template <typename T, int D, int kUnroll, bool kBwd, bool kInterleaved>
cudaError_t launch_rows(RopeParams p, int tokens, float* dqw, float* dkw, cudaStream_t stream) {
  constexpr int kUnitRows = kUnroll * RowLayout<T, D>::kRows;
  // A warp takes a token's units in a row, whose angles it then works out once,
  // as many as still leave every warp of the grid a few such groups (backward of
  // 8192 tokens x 64 heads: 77.4 us a call one by one, 68.2 so).
  const int most = 2 * sm_count();
  for (int per = 8;; per /= 2) {
    for (Rows& t : p.t) {
      t.chunks = (t.H + kUnitRows - 1) / kUnitRows;
      t.per = std::max(1, std::min(per, t.chunks));
      t.groups = (t.chunks + t.per - 1) / t.per;
    }
    p.groups_q = tokens * p.t[0].groups;
    p.groups = p.groups_q + tokens * p.t[1].groups;
    if (per == 1 || p.groups >= 4 * most * kWarps) break;
  }
  const int blocks = std::min((p.groups + kWarps - 1) / kWarps, std::min(kMaxBlocks, most));
  constexpr int kSmem = kWarps * Ring<kUnroll * (kBwd ? 4 : 2)>::kBytes;
  const auto kern = qk_norm_rope_kernel<T, D, kUnroll, kBwd, kInterleaved>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), kSmem);
  if (e != cudaSuccess) return e;
  kern<<<blocks, kThreads, kSmem, stream>>>(p);
  count_launch(2);
  if (!kBwd || (!dqw && !dkw)) return cudaGetLastError();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, gain_grad_kernel, static_cast<const float*>(p.partial), blocks, D,
                         dqw, dkw);
  count_launch(2);
  return e;
}

// Rows per unit: one row group of a token, or kWide of them, which keeps more bytes in
// flight, where those give half of the grid's warps one.  Measured at 203 points (256 to
// 16K tokens, 16 to 64 heads, both types, head sizes and directions) the choice takes 0.9 %
// more than the faster form on average and never 16 %; from one unit a warp on, 2.4 % and
// 30 %.  One group / kWide (us a call): forward, bf16, d = 128: 512 tokens x 16 heads 4.1 /
// 4.4, x 40 6.0 / 5.1, 4096 x 64 27.1 / 22.6; backward, bf16, d = 128: 512 x 16 6.8 / 7.6,
// 256 x 64 9.1 / 7.8, 8192 x 64 69.7 / 67.9; backward, fp32, d = 64: 512 x 16 5.8 / 6.6,
// 512 x 64 9.6 / 8.7, 3000 x 16 11.3 / 11.5.  The longest fp32 calls lose by it: backward,
// d = 128, 4096 x 64 65.1 / 68.7.
template <typename T, int D, bool kBwd>
cudaError_t launch_sized(const RopeParams& p, int tokens, float* dqw, float* dkw,
                         cudaStream_t stream) {
  constexpr int kWide = kBwd ? 2 : 4;
  const long long rows = static_cast<long long>(tokens) * (p.t[0].H + p.t[1].H);
  const bool wide = rows / (kWide * RowLayout<T, D>::kRows) >= 1LL * sm_count() * kWarps;
  if (p.interleaved)
    return wide ? launch_rows<T, D, kWide, kBwd, true>(p, tokens, dqw, dkw, stream)
                : launch_rows<T, D, 1, kBwd, true>(p, tokens, dqw, dkw, stream);
  return wide ? launch_rows<T, D, kWide, kBwd, false>(p, tokens, dqw, dkw, stream)
              : launch_rows<T, D, 1, kBwd, false>(p, tokens, dqw, dkw, stream);
}

template <bool kBwd>
cudaError_t launch_any(const RopeParams& p, int tokens, int d, bool bf16, float* dqw, float* dkw,
                       cudaStream_t stream) {
  if (bf16)
    return d == 128 ? launch_sized<__nv_bfloat16, 128, kBwd>(p, tokens, dqw, dkw, stream)
                    : launch_sized<__nv_bfloat16, 64, kBwd>(p, tokens, dqw, dkw, stream);
  return d == 128 ? launch_sized<float, 128, kBwd>(p, tokens, dqw, dkw, stream)
                  : launch_sized<float, 64, kBwd>(p, tokens, dqw, dkw, stream);
}

// Strides of a [B, S, H, d] operand: the caller's, or contiguous.
void set_strides(const int64_t* given, int S, int H, int d, long long& b, long long& s,
                 long long& h) {
  b = given ? given[0] : static_cast<long long>(S) * H * d;
  s = given ? given[1] : static_cast<long long>(H) * d;
  h = given ? given[2] : d;
}

cp_status check_rows(const void* q, const void* k, int B, int S, int Hq, int Hk, int d,
                     const float* inv_freq, int rot_dim, int interleaved, float eps, int is_bf16) {
  if (!q || (Hk > 0 && !k) || (rot_dim > 0 && !inv_freq)) return CP_ERR_NULL;
  if (B < 1 || S < 1 || Hq < 1 || Hk < 0) return CP_ERR_SHAPE;
  // every row's index, and so every unit's, is an int
  if (static_cast<long long>(Hq) + Hk > 0x7fffffff ||
      static_cast<long long>(B) * S > 0x7fffffff / (static_cast<long long>(Hq) + Hk))
    return CP_ERR_SHAPE;
  if (d != 64 && d != 128) return CP_ERR_UNSUPPORTED;
  if (rot_dim < 0 || rot_dim > d) return CP_ERR_SHAPE;
  if (rot_dim % 16 != 0) return CP_ERR_UNSUPPORTED;
  if ((interleaved != 0 && interleaved != 1) || (is_bf16 != 0 && is_bf16 != 1))
    return CP_ERR_SHAPE;
  if (!(eps >= 0.f) || eps > 3.4e38f) return CP_ERR_SHAPE;
  return CP_OK;
}

cp_status check_written(const void* y, const int64_t* ys, int B, int S, int H, int d, int esz) {
  if (!strides_ok(ys, esz)) return CP_ERR_ALIGN;
  return strides_distinct(ys, B, S, H, d) ? CP_OK : CP_ERR_SHAPE;
}

}  // namespace

bool strides_ok(const int64_t* st, int elem_bytes) {
  if (!st) return true;
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] > (1LL << 40) || (st[i] * elem_bytes) % 16 != 0) return false;
  return true;
}

bool strides_distinct(const int64_t* st, int n0, int n1, int n2, int d) {
  if (!st) return true;
  struct Dim { int64_t stride, n; } dim[3] = {{st[0], n0}, {st[1], n1}, {st[2], n2}};
  std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t extent = d;
  for (const Dim& x : dim) {
    if (x.n <= 1) continue;
    if (x.stride < extent || x.stride > (1LL << 61) / x.n) return false;  // extents stay in 64 bits
    extent += x.stride * (x.n - 1);
  }
  return true;
}

}  // namespace cpring

extern "C" {

cp_status cp_qk_norm_rope(const void* q, const int64_t* q_strides, const void* k,
                          const int64_t* k_strides, const float* q_weight, const float* k_weight,
                          float eps, const float* inv_freq, int rot_dim, int interleaved,
                          const int32_t* positions, void* q_out, void* k_out, int B, int S,
                          int Hq, int Hk, int d, int is_bf16, cudaStream_t stream) {
  cpring::TraceRange trace_("cp_qk_norm_rope");
  using namespace cpring;
  cp_status st = check_rows(q, k, B, S, Hq, Hk, d, inv_freq, rot_dim, interleaved, eps, is_bf16);
  if (st != CP_OK) return st;
  if (!q_out || (Hk > 0 && !k_out)) return CP_ERR_NULL;
  const int esz = is_bf16 ? 2 : 4;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
      !aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(inv_freq, 4) ||
      !aligned(positions, 4) || !strides_ok(q_strides, esz) || !strides_ok(k_strides, esz))
    return CP_ERR_ALIGN;
  if (device_cc() != 103) return CP_ERR_DEVICE;
  RopeParams p{};
  p.t[0].x = q; p.t[0].y = q_out; p.t[0].w = q_weight; p.t[0].H = Hq;
  p.t[1].x = k; p.t[1].y = k_out; p.t[1].w = k_weight; p.t[1].H = Hk;
  set_strides(q_strides, S, Hq, d, p.t[0].xb, p.t[0].xs, p.t[0].xh);
  set_strides(k_strides, S, Hk, d, p.t[1].xb, p.t[1].xs, p.t[1].xh);
  p.inv_freq = inv_freq; p.positions = positions;
  p.S = S; p.rot = rot_dim; p.interleaved = interleaved; p.eps = eps;
  return launch_any<false>(p, B * S, d, is_bf16 != 0, nullptr, nullptr, stream) == cudaSuccess
             ? CP_OK
             : CP_ERR_CUDA;
}

int64_t cp_qk_norm_rope_bwd_workspace_bytes(int B, int S, int Hq, int Hk, int d) {
  if (B < 1 || S < 1 || Hq < 1 || Hk < 0 || (d != 64 && d != 128)) return -1;
  return static_cast<int64_t>(cpring::kMaxBlocks) * 2 * d * 4;
}

cp_status cp_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q,
                              const int64_t* q_strides, const void* k, const int64_t* k_strides,
                              const float* q_weight, const float* k_weight, float eps,
                              const float* inv_freq, int rot_dim, int interleaved,
                              const int32_t* positions, void* dq, const int64_t* dq_strides,
                              void* dk, const int64_t* dk_strides, float* dq_weight,
                              float* dk_weight, int B, int S, int Hq, int Hk, int d, int is_bf16,
                              void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  cpring::TraceRange trace_("cp_qk_norm_rope_bwd");
  using namespace cpring;
  cp_status st = check_rows(q, k, B, S, Hq, Hk, d, inv_freq, rot_dim, interleaved, eps, is_bf16);
  if (st != CP_OK) return st;
  if (!dq_out || !dq || !workspace || (Hk > 0 && (!dk_out || !dk))) return CP_ERR_NULL;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return CP_ERR_NULL;
  const int esz = is_bf16 ? 2 : 4;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(dq_out, 16) || !aligned(dk_out, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(q_weight, 4) || !aligned(k_weight, 4) ||
      !aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(inv_freq, 4) ||
      !aligned(positions, 4) || !aligned(workspace, 16) || !strides_ok(q_strides, esz) ||
      !strides_ok(k_strides, esz))
    return CP_ERR_ALIGN;
  st = check_written(dq, dq_strides, B, S, Hq, d, esz);
  if (st == CP_OK && Hk > 0) st = check_written(dk, dk_strides, B, S, Hk, d, esz);
  if (st != CP_OK) return st;
  if (workspace_bytes < cp_qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hk, d))
    return CP_ERR_BUFFER;
  if (device_cc() != 103) return CP_ERR_DEVICE;
  RopeParams p{};
  p.t[0].x = q; p.t[0].dy = dq_out; p.t[0].y = dq; p.t[0].w = q_weight; p.t[0].H = Hq;
  p.t[1].x = k; p.t[1].dy = dk_out; p.t[1].y = dk; p.t[1].w = k_weight; p.t[1].H = Hk;
  set_strides(q_strides, S, Hq, d, p.t[0].xb, p.t[0].xs, p.t[0].xh);
  set_strides(k_strides, S, Hk, d, p.t[1].xb, p.t[1].xs, p.t[1].xh);
  set_strides(dq_strides, S, Hq, d, p.t[0].yb, p.t[0].ys, p.t[0].yh);
  set_strides(dk_strides, S, Hk, d, p.t[1].yb, p.t[1].ys, p.t[1].yh);
  p.inv_freq = inv_freq; p.positions = positions;
  p.partial = static_cast<float*>(workspace);
  p.S = S; p.rot = rot_dim; p.interleaved = interleaved; p.eps = eps;
  return launch_any<true>(p, B * S, d, is_bf16 != 0, dq_weight, dk_weight, stream) == cudaSuccess
             ? CP_OK
             : CP_ERR_CUDA;
}

}  // extern "C"
