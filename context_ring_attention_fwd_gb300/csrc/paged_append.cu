// Appending new tokens' keys and values to a paged cache, with the per-head
// norm and the position rotation of K (and of Q, for the attention that
// follows) on the way.
//
// Token s of sequence b has the position p = cache_lens[b] + s and goes to
// slot p % page_size of page page_table[b][p / page_size].  K is normed and
// rotated in fp32 (rope.cuh) and rounded once, to what the cache holds: bf16,
// or the E4M3 code of x times the reciprocal of descale[head] (in fp32, as
// cp_fp8_quantize multiplies by its inverse scale).
//
// Bound by latency.  Single tokens (64 of them: 4.3 us a call) by the launch; prefill
// chunks (3842 tokens of 32 + 8 + 8 heads: 25.7 us in the kernel to E4M3, 25.0 to bf16,
// half the copy rate) by how much 16 warps an SM, which is what the registers allow, keep
// under way with one unit each ahead: DRAM is 23 % used, the issue slots 40 %.  A
// warp's unit is a few heads of one token of q, k or v; rows are 16-byte
// vectors of 8 (d = 128) or 4 lanes, so any page size, head order and page
// stride costs the same; the next unit's rows are on their way meanwhile
// (norm_rope.cu).
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
  int B, S, rot, interleaved;
  int compact;  // units are laid over the new tokens alone (B <= kMaxScan)
  int tokens;   // B * S
  float eps;
};

// A chunk's padding is left out of the work's layout, so that every warp gets an
// equal share of the tokens that are there: each block sums the lengths once, for
// batches of up to this many rows (a chunk of 8192 rows, half of them padding:
// 27.3 -> 24.2 us a call).  Calls of one token a row, and larger
// batches, walk the padding.
constexpr int kMaxScan = 256;

template <int NP>
__device__ __forceinline__ uint2 codes8(const f32x2 (&z)[NP], int at, f32x2 inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(mul2(z[at + i], inv), lo, hi);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    w[i] = r;
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <int D, int kUnroll, bool kE4M3, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 2) paged_append_kernel(const AppendParams p) {
  using T = __nv_bfloat16;
  using Lay = RowLayout<T, D>;
  constexpr int NP = Lay::kPairs;
  constexpr int kUnitRows = kUnroll * Lay::kRows;
  using R = Ring<kUnroll * 2>;
  extern __shared__ __align__(16) uint8_t rings[];
  __shared__ __align__(16) float gain[2][D];
  __shared__ int starts[kMaxScan + 1];
  __shared__ int warp_sum[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % Lay::kLanes, g = lane / Lay::kLanes;
  const R ring{static_cast<uint32_t>(__cvta_generic_to_shared(rings)) + warp * R::kBytes +
               lane * 16};
  int lo, hi;
  bool turned;
  lane_columns<NP>(l, p.rot, kInterleaved, lo, hi, turned);

  // `tells`: this call reports a length that is out of range (some call of each row's does).
  auto new_len = [&](int b, bool tells) {
    const int n = p.new_lens ? __ldg(p.new_lens + b) : p.S;
    if ((n < 0 || n > p.S) && tells) atomicOr(p.err, kErrCache);
    return max(0, min(n, p.S));
  };
  int tokens = p.tokens;
  if (p.compact) {
    static_assert(kMaxScan == kThreads, "one thread a row");
    const int n = threadIdx.x < p.B ? new_len(threadIdx.x, blockIdx.x == 0) : 0;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = x - n;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    starts[threadIdx.x] = before;
    if (threadIdx.x == kThreads - 1) starts[kMaxScan] = before + n;
    __syncthreads();
    tokens = starts[kMaxScan];
  }
  const unsigned units_q = static_cast<unsigned>(tokens) * p.t[0].chunks;
  const unsigned units_qk = units_q + static_cast<unsigned>(tokens) * p.t[1].chunks;
  const unsigned units = units_qk + static_cast<unsigned>(tokens) * p.t[2].chunks;

  struct Unit {
    int kind, tok, h0;  // 0 q, 1 k, 2 v; token (b, s)
    int b, s;
    int pos, page, slot;  // page -1: no place (or none needed), -2: padding
  };
  auto unit_at = [&](unsigned u) {
    Unit x;
    x.kind = (u >= units_q) + (u >= units_qk);
    const int local = static_cast<int>(u - (x.kind == 0 ? 0u : x.kind == 1 ? units_q : units_qk));
    const int tok = local / p.t[x.kind].chunks;
    x.h0 = (local - tok * p.t[x.kind].chunks) * kUnitRows + g;
    if (p.compact) {
      int a = 0, z = p.B;  // the last row that starts at or before tok
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (starts[mid] <= tok) a = mid; else z = mid;
      }
      x.b = a;
      x.s = tok - starts[a];
    } else {
      x.b = tok / p.S;
      x.s = tok - x.b * p.S;
    }
    x.tok = x.b * p.S + x.s;
    return x;
  };
  // Starts the loads of a unit's rows, and finds its token's place meanwhile.
  auto fetch = [&](Unit& x, int stage) {
    const NewRows& t = p.t[x.kind];
    const int b = x.b, s = x.s;
    const int held = __ldg(p.cache_lens + b);
    x.page = -2;
    // Every row has a unit of its first token's values.
    const bool tells = x.kind == 2 && s == 0 && lane == 0;
    if (!p.compact && s >= new_len(b, tells)) return;  // padding behind the new tokens: not touched
    const T* const xrow = static_cast<const T*>(t.x) + b * t.xb + s * t.xs;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = x.h0 + i * Lay::kRows;
      const bool there = h < t.H;
      const T* const src = xrow + (there ? h : 0) * t.xh;
      ring.copy(stage, 2 * i, src + lo, there);
      ring.copy(stage, 2 * i + 1, src + hi, there);
    }
    const long long pos = static_cast<long long>(held) + s;
    x.pos = static_cast<int>(pos);
    x.page = -1;
    x.slot = 0;
    if (x.kind != 0 && held >= 0 && pos < static_cast<long long>(p.max_pages) * p.page_size) {
      const int at = x.pos / p.page_size;
      x.slot = x.pos - at * p.page_size;
      x.page = __ldg(p.table + b * p.table_stride + at);
      if (x.page < 0 || x.page >= p.n_pages) x.page = -1;
    }
  };
  const unsigned stride = gridDim.x * kWarps;  // unsigned: the last step may pass 2^31
  unsigned u = blockIdx.x * kWarps + warp;
  Unit next{};
  if (u < units) {
    next = unit_at(u);
    fetch(next, 0);
  }
  copies_commit();

  uint64_t frac[Lay::kAngles];
  load_fractions<Lay>(p.inv_freq, l, g, turned, frac);
  stage_gain(gain[0], p.t[0].w, D);
  stage_gain(gain[1], p.t[1].w, D);
  __syncthreads();
  for (int stage = 0; u < units; u += stride, stage ^= 1) {
    const Unit x = next;
    if (u + stride < units && u + stride > u) {
      next = unit_at(u + stride);
      fetch(next, stage ^ 1);
    }
    copies_commit();
    if (x.page == -2) continue;
    if (x.kind != 0 && x.page < 0) {  // no place in the cache: the token is not written
      // Its rows are on their way all the same: they land before the stage is filled
      // again (two copies to one address have no order), or the block ends.
      copies_wait_all_but_last();
      if (lane == 0) atomicOr(p.err, kErrCache);
      continue;
    }
    const NewRows& t = p.t[x.kind];
    f32x2 own[NP], other[NP], w[NP];
    if (x.kind != 2) {  // the gain goes with the turn: see norm_rope.cu
      load_gain<NP>(gain[x.kind], lo, hi, w);
      if (p.rot > 0) {
        float c[NP], sn[NP];
        row_angles<Lay>(x.pos, frac, l, c, sn);
        turn_factors<NP, kInterleaved>(c, sn, 1.f, own, other);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          own[i] = mul2(own[i], w[i]);
          other[i] = mul2(other[i], partner<NP, kInterleaved>(w, i));
        }
      }
    }
    copies_wait_all_but_last();
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = x.h0 + i * Lay::kRows;
      if (h - g >= t.H) break;  // the same for the whole warp
      f32x2 z[NP];
      unpack<NP>(ring.read(stage, 2 * i), z, 0, T());
      unpack<NP>(ring.read(stage, 2 * i + 1), z, NP / 2, T());
      if (x.kind != 2) {
        float r = 1.f;
        if (t.w != nullptr)
          r = rsqrtf(row_sum<Lay::kLanes>(dot<NP>(z, z)) * (1.f / D) + p.eps);
        if (turned) {
          turn<NP, kInterleaved>(z, own, other);
        } else {
#pragma unroll
          for (int e = 0; e < NP; ++e) z[e] = mul2(z[e], w[e]);
        }
        const f32x2 r2 = pack2(r, r);
#pragma unroll
        for (int e = 0; e < NP; ++e) z[e] = mul2(z[e], r2);
      }
      if (h >= t.H) continue;
      if (x.kind == 0) {
        T* const dst = p.q_out + (static_cast<long long>(x.tok) * t.H + h) * D;
        *reinterpret_cast<uint4*>(dst + lo) = repack<NP>(z, 0, T());
        *reinterpret_cast<uint4*>(dst + hi) = repack<NP>(z, NP / 2, T());
        continue;
      }
      const int kv = x.kind - 1;
      const long long off = x.page * p.cs[kv][0] + x.slot * p.cs[kv][1] + h * p.cs[kv][2];
      if (kE4M3) {
        uint8_t* const dst = static_cast<uint8_t*>(p.cache[kv]) + off;
        const float inv = __frcp_rn(__ldg(p.descale[kv] + h));
        *reinterpret_cast<uint2*>(dst + lo) = codes8<NP>(z, 0, pack2(inv, inv));
        *reinterpret_cast<uint2*>(dst + hi) = codes8<NP>(z, NP / 2, pack2(inv, inv));
      } else {
        T* const dst = static_cast<T*>(p.cache[kv]) + off;
        *reinterpret_cast<uint4*>(dst + lo) = repack<NP>(z, 0, T());
        *reinterpret_cast<uint4*>(dst + hi) = repack<NP>(z, NP / 2, T());
      }
    }
  }
}

template <int D, int kUnroll, bool kE4M3, bool kInterleaved>
cudaError_t launch_append(AppendParams p, int tokens, cudaStream_t stream) {
  constexpr int kUnitRows = kUnroll * RowLayout<__nv_bfloat16, D>::kRows;
  for (NewRows& t : p.t) t.chunks = (t.H + kUnitRows - 1) / kUnitRows;
  p.tokens = tokens;
  p.compact = p.new_lens != nullptr && p.S > 1 && p.B <= kMaxScan;
  const int units = tokens * (p.t[0].chunks + p.t[1].chunks + p.t[2].chunks);
  const int blocks = std::min((units + kWarps - 1) / kWarps, 2 * sm_count());
  constexpr int kSmem = kWarps * Ring<kUnroll * 2>::kBytes;
  const auto kern = paged_append_kernel<D, kUnroll, kE4M3, kInterleaved>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), kSmem);
  if (e != cudaSuccess) return e;
  kern<<<blocks, kThreads, kSmem, stream>>>(p);
  count_launch(2);
  return cudaGetLastError();
}

// One row group of a token per unit (more warps, each with less to wait for), or four
// where that gives half of the grid's warps one.  Measured at 208 points (16 to 8192 tokens,
// 12 to 96 heads, both types and head sizes) the choice takes 0.5 % more than the faster form
// on average and never 15 %; from one unit a warp on, 1.7 % and 27 %.  One / four (us a call,
// bf16, d = 128): 64 tokens x 48 heads 4.3 / 5.4, 256 x 48 5.8 / 5.4, 512 x 48 7.7 / 6.2,
// 4096 x 48 32.8 / 23.9, 4096 x 12 13.3 / 13.1; d = 64, 8192 x 12 16.6 / 19.1, where it loses.
template <int D, bool kE4M3>
cudaError_t launch_sized(const AppendParams& p, int tokens, cudaStream_t stream) {
  const long long rows = static_cast<long long>(tokens) * (p.t[0].H + 2LL * p.t[1].H);
  const bool wide =
      rows / (4 * RowLayout<__nv_bfloat16, D>::kRows) >= 1LL * sm_count() * kWarps;
  if (p.interleaved)
    return wide ? launch_append<D, 4, kE4M3, true>(p, tokens, stream)
                : launch_append<D, 1, kE4M3, true>(p, tokens, stream);
  return wide ? launch_append<D, 4, kE4M3, false>(p, tokens, stream)
              : launch_append<D, 1, kE4M3, false>(p, tokens, stream);
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
      (c->table_stride != 0 && c->table_stride < c->max_pages) || c->table_stride > (1LL << 31))
    return CP_ERR_SHAPE;
  // positions, and those up to a tile behind the last, are int32
  if (static_cast<long long>(c->max_pages) * c->page_size > (1LL << 30)) return CP_ERR_SHAPE;
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
  p.B = B; p.S = S; p.rot = rot_dim; p.interleaved = interleaved; p.eps = eps;
  const bool e4m3 = cache->elem_bytes == 1;
  const cudaError_t e =
      d == 128 ? (e4m3 ? launch_sized<128, true>(p, B * S, stream)
                       : launch_sized<128, false>(p, B * S, stream))
               : (e4m3 ? launch_sized<64, true>(p, B * S, stream)
                       : launch_sized<64, false>(p, B * S, stream));
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}
