// What the two kernels of the decode attention (paged_decode.cu,
// prefix_sm103.cu) share: the launch's parameters, the split of work, and copies and
// conversions of cached rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cpring {

struct DecodeParams {
  const __nv_bfloat16* q;
  const uint8_t* cache[2];  // k, v
  long long cs[2][3];       // their strides in bytes: page, token, head
  const float* descale[2];
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* prefix_pages;
  __nv_bfloat16* out;
  float* lse;
  int* err;
  unsigned long long timeout_ns;
  int fault_drop_k;
  // workspace
  unsigned* starts;  // [B + 1] first unit of each sequence's items
  float* slot_o;     // [grid][2][16][d]
  float* slot_ml;    // [grid][2][16][2]
  float* whole_o;    // [2][rows][d]: items finished by one CTA but owed a join (own, prefix)
  float* whole_ml;   // [2][rows][2]
  float* pslot_o;    // [prefix_grid][2][256][d]: the wide prefix items' parts
  float* pslot_ml;   // [prefix_grid][2][256][2]
  long long qb, qs, qh;
  long long table_stride;
  float scale;  // log2(e) / sqrt(d)
  int B, n_q, Hq, Hk, G, R;  // R = n_q * G rows of an item before tiling
  int own_tiles_of_rows;     // 16-row tiles of an own item
  int P;
  // The prefix: items of prefix_rows rows and prefix_tiles key tiles of
  // prefix_keys keys each.  prefix_grid > 0: prefix_attn_kernel runs them on
  // that many CTAs (256 rows, 128 keys); 0: they are the first items of
  // paged_decode_kernel (16 rows, 64 keys).
  int prefix_rows, prefix_row_tiles, prefix_tiles, prefix_grid;
  int n_pages, page_size;
  long long capacity;        // max_pages * page_size
};

// 16 bytes to shared memory, the first `bytes` (0 or 16) of them copied, the rest zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Two E4M3 codes (16 bits) to two fp16 values, exactly.
__device__ __forceinline__ uint32_t half2_of_codes(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Both kernels lay their items end to end in units, kItemCost of them for
// starting and ending an item and one for each of its key tiles, and give every
// CTA c of g an equal stretch of the W units, from c W / g on.  An item's cost
// units come first; the CTA that holds only those has no part of it.
// (Measured: an item's loads of pages and queries, its pipeline's filling and
// its state's writing take about as long as that many tiles.)
constexpr unsigned kItemCost = 3;
__device__ __forceinline__ unsigned stretch(unsigned c, unsigned W, unsigned g) {
  return static_cast<unsigned>(static_cast<unsigned long long>(c) * W / g);
}
// The CTA whose stretch holds unit w.
__device__ __forceinline__ unsigned holder(unsigned w, unsigned W, unsigned g) {
  return static_cast<unsigned>((static_cast<unsigned long long>(w + 1ull) * g - 1) / W);
}
// Tiles [t0, t1) of an item for units [u0, u1) of it.
__device__ __forceinline__ int tile_of_unit(unsigned u) {
  return u > kItemCost ? static_cast<int>(u - kItemCost) : 0;
}

// Row r of an item: its place in q, and its index (b, i, h) in [B, n_q, Hq].
struct RowOf {
  int b, i, h;
  __device__ RowOf(const DecodeParams& p, int b0, int hk, int r) {
    b = b0 + r / p.R;  // own items: r < R, so b = b0; prefix items: b0 = 0
    const int rem = r % p.R;
    i = rem / p.G;
    h = hk * p.G + rem % p.G;
  }
  __device__ long long index(const DecodeParams& p) const {
    return (static_cast<long long>(b) * p.n_q + i) * p.Hq + h;
  }
  __device__ const __nv_bfloat16* query(const DecodeParams& p) const {
    return p.q + b * p.qb + i * p.qs + h * p.qh;
  }
};

// The power of two that brings a row's largest magnitude `top` to [2^14, 2^15)
// (1 for zeros and non-finite rows), and its inverse: a bf16 row so scaled
// keeps every bit in fp16 but for entries 2^-28 below its largest.
__device__ __forceinline__ void fp16_row_scale(float top, float& up, float& down) {
  const int ex = static_cast<int>(__float_as_uint(top) >> 23);
  const int e = (ex == 0 || ex == 255) ? 0 : max(ex - 127 - 14, -112);
  up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  down = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

constexpr int kPrefixRows = 256;  // rows of a prefix_attn_kernel item
constexpr int kPrefixKeys = 128;  // keys of its tiles
constexpr int kMaxPrefixGrid = 160;

// The place of prefix_attn_kernel's item (key head hk, row tile t) among its items.
// bf16: row tiles outermost, so that the tiles of a key head walk the same keys at the
// same time and L2 serves all but the first; E4M3: key heads outermost.  Measured at 512
// rows x 8 heads, key heads / row tiles outermost: bf16 under 64K 102-105 / 96-103 us in
// the kernel, 539 / 270 MB from DRAM; E4M3 under 128K 189-194 / 193-194 us, the whole
// call 220 / 224 us, 539 / 404 MB.
template <bool kE4M3>
__host__ __device__ __forceinline__ int prefix_item(const DecodeParams& p, int hk, int t) {
  return kE4M3 ? hk * p.prefix_row_tiles + t : t * p.Hk + hk;
}
template <bool kE4M3>
__host__ __device__ __forceinline__ void prefix_item_at(const DecodeParams& p, int item, int& hk,
                                                        int& t) {
  const int inner = kE4M3 ? p.prefix_row_tiles : p.Hk;
  const int outer = item / inner, rest = item - outer * inner;
  hk = kE4M3 ? outer : rest;
  t = kE4M3 ? rest : outer;
}

// Launch prefix_attn_kernel over the prefix's items (p.prefix_grid CTAs).
cudaError_t launch_prefix_attn(const DecodeParams& p, int d, bool e4m3, cudaStream_t stream);

}  // namespace cpring
