// Appending new tokens' keys and values to a paged cache, with the per-head
// norm and the position rotation of K (and of Q, for the attention that
// follows) on the way.
//
// Token s of sequence b has the position p = cache_lens[b] + s and goes to
// slot p % page_size of page page_table[b][p / page_size].  K is normed and
// rotated in fp32 (rope.cuh) and rounded once, to what the cache holds: bf16,
// or the E4M3 code of x / descale[head].
//
// Bound by HBM for prefill chunks and by launch latency for single tokens.  A
// warp's unit is a few heads of one token of q, k or v; rows are 16-byte
// vectors of 8 (d = 128) or 4 lanes, so any page size, head order and page
// stride costs the same.
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

struct NewRows {
  const void* x;
  long long xb, xs, xh;  // strides of [B, S, H, d], elements
  const float* w;        // gain, or null
  int H, chunks;
};

struct AppendParams {
  NewRows t[3];  // q, k, v
  __nv_bfloat16* q_out;
  void* cache[2];            // k, v
  long long cs[2][3];        // their strides: page, token, head
  const float* descale[2];   // [Hk], E4M3 caches
  const int32_t* table;
  const int32_t* cache_lens;
  const int32_t* new_lens;
  const float* inv_freq;
  int* err;
  long long table_stride;
  int n_pages, page_size, max_pages;
  int S, rot, interleaved;
  int units_q, units_qk, units;
  float eps;
};

__device__ __forceinline__ uint2 codes8(const float (&z)[16], int at, float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(r)
        : "f"(__fdiv_rn(z[at + 2 * i + 1], scale)), "f"(__fdiv_rn(z[at + 2 * i], scale)));
    w[i] = r;
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <int D, int kUnroll, bool kE4M3>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendParams p) {
  using T = __nv_bfloat16;
  using Lay = RowLayout<T, D>;
  constexpr int NP = Lay::kPairs;
  constexpr int kUnitRows = kUnroll * Lay::kRows;
  const int lane = threadIdx.x & 31;
  const int l = lane % Lay::kLanes, g = lane / Lay::kLanes;
  int lo, hi;
  bool turned;
  lane_columns<NP>(l, p.rot, p.interleaved != 0, lo, hi, turned);
  uint64_t frac[Lay::kAngles];
  load_fractions<Lay>(p.inv_freq, l, g, turned, frac);
  float w[2 * NP];
  int cur = -1;
  const unsigned stride = gridDim.x * kWarps;  // unsigned: the last step may pass 2^31
  for (unsigned u = blockIdx.x * kWarps + (threadIdx.x >> 5);
       u < static_cast<unsigned>(p.units); u += stride) {
    const int kind = (u >= static_cast<unsigned>(p.units_q)) +
                     (u >= static_cast<unsigned>(p.units_qk));  // 0 q, 1 k, 2 v
    const NewRows& t = p.t[kind];
    const int local =
        static_cast<int>(u) - (kind == 0 ? 0 : kind == 1 ? p.units_q : p.units_qk);
    const int tok = local / t.chunks;
    const int h0 = (local - tok * t.chunks) * kUnitRows + g;
    const int b = tok / p.S, s = tok - b * p.S;
    const int held = __ldg(p.cache_lens + b);
    const int n_new = p.new_lens ? __ldg(p.new_lens + b) : p.S;
    const T* const xrow = static_cast<const T*>(t.x) + b * t.xb + s * t.xs;
    uint4 raw[kUnroll][2];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = h0 + i * Lay::kRows;
      raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (h < t.H) {
        raw[i][0] = *reinterpret_cast<const uint4*>(xrow + h * t.xh + lo);
        raw[i][1] = *reinterpret_cast<const uint4*>(xrow + h * t.xh + hi);
      }
    }
    if (n_new < 0 || n_new > p.S) {
      if (lane == 0 && kind == 1) atomicOr(p.err, kErrCache);
    }
    if (s >= n_new) continue;  // padding behind the sequence's new tokens: nothing is written
    const long long pos = static_cast<long long>(held) + s;
    int page = -1, slot = 0;  // this token's place
    if (kind != 0) {
      if (held >= 0 && pos < static_cast<long long>(p.max_pages) * p.page_size) {
        const int at = static_cast<int>(pos / p.page_size);
        slot = static_cast<int>(pos - static_cast<long long>(at) * p.page_size);
        page = __ldg(p.table + b * p.table_stride + at);
      }
      if (page < 0 || page >= p.n_pages) {  // no place in the cache: the token is not written
        if (lane == 0) atomicOr(p.err, kErrCache);
        continue;
      }
    }
    if (kind != cur) {
      cur = kind;
      if (t.w != nullptr) load_columns<NP>(t.w, lo, hi, w);
    }
    float c[NP], sn[NP];
    if (kind != 2 && p.rot > 0) row_angles<Lay>(static_cast<int>(pos), frac, l, c, sn);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = h0 + i * Lay::kRows;
      if (h - g >= t.H) break;  // the same for the whole warp
      float z[2 * NP];
      unpack(raw[i][0], z, 0, T());
      unpack(raw[i][1], z, NP, T());
      if (kind != 2) {
        if (t.w != nullptr) {
          const float r = rsqrtf(row_sum<Lay::kLanes>(sum_squares(z)) * (1.f / D) + p.eps);
#pragma unroll
          for (int e = 0; e < 2 * NP; ++e) z[e] = z[e] * r * w[e];
        }
        if (turned) rotate<NP>(z, c, sn, p.interleaved != 0, 1.f);
      }
      if (h >= t.H) continue;
      if (kind == 0) {
        T* const dst = p.q_out + (static_cast<long long>(tok) * t.H + h) * D;
        *reinterpret_cast<uint4*>(dst + lo) = repack(z, 0, T());
        *reinterpret_cast<uint4*>(dst + hi) = repack(z, NP, T());
        continue;
      }
      const int w_kv = kind - 1;
      const long long off = page * p.cs[w_kv][0] + slot * p.cs[w_kv][1] + h * p.cs[w_kv][2];
      if (kE4M3) {
        uint8_t* const dst = static_cast<uint8_t*>(p.cache[w_kv]) + off;
        const float scale = __ldg(p.descale[w_kv] + h);
        *reinterpret_cast<uint2*>(dst + lo) = codes8(z, 0, scale);
        *reinterpret_cast<uint2*>(dst + hi) = codes8(z, NP, scale);
      } else {
        T* const dst = static_cast<T*>(p.cache[w_kv]) + off;
        *reinterpret_cast<uint4*>(dst + lo) = repack(z, 0, T());
        *reinterpret_cast<uint4*>(dst + hi) = repack(z, NP, T());
      }
    }
  }
}

template <int D, int kUnroll, bool kE4M3>
cudaError_t launch_append(AppendParams p, int tokens, cudaStream_t stream) {
  constexpr int kUnitRows = kUnroll * RowLayout<__nv_bfloat16, D>::kRows;
  for (NewRows& t : p.t) t.chunks = (t.H + kUnitRows - 1) / kUnitRows;
  p.units_q = tokens * p.t[0].chunks;
  p.units_qk = p.units_q + tokens * p.t[1].chunks;
  p.units = p.units_qk + tokens * p.t[2].chunks;
  const int blocks = std::min((p.units + kWarps - 1) / kWarps, 3 * sm_count());
  paged_append_kernel<D, kUnroll, kE4M3><<<blocks, kThreads, 0, stream>>>(p);
  count_launch(2);
  return cudaGetLastError();
}

// Four row groups of a token per unit once that still fills the grid; one
// otherwise (single tokens: more warps, each with less to wait for).
template <int D, bool kE4M3>
cudaError_t launch_sized(const AppendParams& p, int tokens, cudaStream_t stream) {
  const long long rows = static_cast<long long>(tokens) * (p.t[0].H + 2LL * p.t[1].H);
  if (rows / (4 * RowLayout<__nv_bfloat16, D>::kRows) >= 2LL * sm_count() * kWarps)
    return launch_append<D, 4, kE4M3>(p, tokens, stream);
  return launch_append<D, 1, kE4M3>(p, tokens, stream);
}

void take_strides(const int64_t* given, int S, int H, int d, NewRows& t) {
  t.xb = given ? given[0] : static_cast<long long>(S) * H * d;
  t.xs = given ? given[1] : static_cast<long long>(H) * d;
  t.xh = given ? given[2] : d;
}

}  // namespace

cp_status check_cache(const cp_paged_cache* c) {
  if (!c || !c->k || !c->v || !c->page_table) return CP_ERR_NULL;
  if (c->elem_bytes != 1 && c->elem_bytes != 2) return CP_ERR_UNSUPPORTED;
  if (c->elem_bytes == 1 && (!c->k_descale || !c->v_descale)) return CP_ERR_NULL;
  if (c->d != 64 && c->d != 128) return CP_ERR_UNSUPPORTED;
  if (c->n_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->Hk < 1 || c->Hk > 65535 ||
      c->table_stride < c->max_pages || c->table_stride > (1LL << 31))
    return CP_ERR_SHAPE;
  // positions are int32
  if (static_cast<long long>(c->max_pages) * c->page_size > 0x7fffffffLL) return CP_ERR_SHAPE;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) ||
      !aligned(c->k_descale, 4) || !aligned(c->v_descale, 4) ||
      !strides_ok(c->k_strides, c->elem_bytes) || !strides_ok(c->v_strides, c->elem_bytes))
    return CP_ERR_ALIGN;
  if (!strides_distinct(c->k_strides, c->n_pages, c->page_size, c->Hk, c->d) ||
      !strides_distinct(c->v_strides, c->n_pages, c->page_size, c->Hk, c->d))
    return CP_ERR_SHAPE;
  return CP_OK;
}

}  // namespace cpring

extern "C" cp_status cp_paged_append(const cp_paged_cache* cache, const void* q,
                                     const int64_t* q_strides, const void* k,
                                     const int64_t* k_strides, const void* v,
                                     const int64_t* v_strides, const int32_t* cache_lens,
                                     const int32_t* new_lens, const float* q_weight,
                                     const float* k_weight, float eps, const float* inv_freq,
                                     int rot_dim, int interleaved, void* q_out, int B, int S,
                                     int Hq, cudaStream_t stream) {
  cpring::TraceRange trace_("cp_paged_append");
  using namespace cpring;
  if (!k || !v || !cache_lens || (Hq > 0 && (!q || !q_out)) || (rot_dim > 0 && !inv_freq))
    return CP_ERR_NULL;
  cp_status st = check_cache(cache);
  if (st != CP_OK) return st;
  const int Hk = cache->Hk, d = cache->d;
  if (B < 1 || S < 1 || Hq < 0 || rot_dim < 0 || rot_dim > d) return CP_ERR_SHAPE;
  if (rot_dim % 16 != 0) return CP_ERR_UNSUPPORTED;
  // every row's index, and so every unit's, is an int
  const long long heads = static_cast<long long>(Hq) + 2LL * Hk;
  if (heads > 0x7fffffff || static_cast<long long>(B) * S > 0x7fffffff / heads)
    return CP_ERR_SHAPE;
  if ((interleaved != 0 && interleaved != 1) || !(eps >= 0.f) || eps > 3.4e38f)
    return CP_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(cache_lens, 4) || !aligned(new_lens, 4) || !aligned(q_weight, 4) ||
      !aligned(k_weight, 4) || !aligned(inv_freq, 4) || !strides_ok(q_strides, 2) ||
      !strides_ok(k_strides, 2) || !strides_ok(v_strides, 2))
    return CP_ERR_ALIGN;
  if (device_cc() != 103) return CP_ERR_DEVICE;
  AppendParams p{};
  p.t[0].x = q; p.t[0].w = q_weight; p.t[0].H = Hq;
  p.t[1].x = k; p.t[1].w = k_weight; p.t[1].H = Hk;
  p.t[2].x = v; p.t[2].w = nullptr; p.t[2].H = Hk;
  take_strides(q_strides, S, Hq, d, p.t[0]);
  take_strides(k_strides, S, Hk, d, p.t[1]);
  take_strides(v_strides, S, Hk, d, p.t[2]);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.cache[0] = cache->k; p.cache[1] = cache->v;
  for (int i = 0; i < 3; ++i) {
    p.cs[0][i] = cache->k_strides[i];
    p.cs[1][i] = cache->v_strides[i];
  }
  p.descale[0] = cache->k_descale; p.descale[1] = cache->v_descale;
  p.table = cache->page_table; p.table_stride = cache->table_stride;
  p.cache_lens = cache_lens; p.new_lens = new_lens; p.inv_freq = inv_freq;
  p.err = device_error_word();
  if (!p.err) return CP_ERR_CUDA;
  p.n_pages = cache->n_pages; p.page_size = cache->page_size; p.max_pages = cache->max_pages;
  p.S = S; p.rot = rot_dim; p.interleaved = interleaved; p.eps = eps;
  const bool e4m3 = cache->elem_bytes == 1;
  const cudaError_t e =
      d == 128 ? (e4m3 ? launch_sized<128, true>(p, B * S, stream)
                       : launch_sized<128, false>(p, B * S, stream))
               : (e4m3 ? launch_sized<64, true>(p, B * S, stream)
                       : launch_sized<64, false>(p, B * S, stream));
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}
