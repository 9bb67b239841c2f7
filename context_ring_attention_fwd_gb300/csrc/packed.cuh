// What the kernels of the attention over packed prompts share (packed_plan.cu,
// packed_fwd_sm103.cu, packed_bwd_sm103.cu): the list of work items that the plan
// makes of the sequences' lengths, and packed tiles of query rows.
//
// Query rows.  The G = Hq / Hk query heads that read one key head are attended
// together: a 128-row tile holds tq = 128 / G (rounded down) tokens of all of them, row
// r being head r % G of token r / G.  So a key tile is loaded once for G heads, a tile's
// rows span few tokens (less of the causal diagonal is computed in vain), and the
// gradients of a shared key head sum up in the products themselves.  In [T, Hq, d]
// the G heads of a token lie side by side, so a tile is one TMA box of G x tq rows.
// Rows behind tq G, and those of tokens behind a sequence's end, are not stored; where
// they are summed over they are zeroed in shared memory, since what lies there may be
// infinite or NaN.
//
// Items.  The lengths are on the device, so a captured call follows them: the
// plan's kernel lists every sequence's tiles, the most expensive first, and the
// attention's CTAs claim (tile, key head) pairs in that order.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "attn_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace cpring {

constexpr int kCostUnit = 128;  // tokens that an item's cost is counted in
constexpr int kLeastPart = 4;   // streamed tiles of a part of an item
constexpr int kLeastCut = 8;    // items with up to this many stay whole
constexpr int kMaxParts = 512;  // parts of a call over all key heads (the sums' space): the
constexpr int kMaxFwdParts = 320;  // backward's, the forward's

// A list in the caller's workspace.  The attention's kernels, which may start before the plan
// is done and wait for it, read it (and D) with plain loads: a read-only load (__ldg) promises
// that nothing writes during the kernel, and the compiler may move it before the wait.
struct PackedList {
  int* head;        // [0] items of a key head (0 where the offsets are malformed), [1] next claim,
                    // [2] streamed tiles of a part
  int4* items;      // {first row of the sequence, its length, the tile's index, part}
  int* starts;      // [n] items before each sequence (scratch)
  int* buckets;     // [n_buckets] (scratch)
  int tokens;       // of a tile
  int of_keys;      // tiles of keys: their cost is the queries that see them
  // Items are cut along the tiles that they stream (packed_plan.cu) into at most this many parts
  // (of a key head; 0: they are not), each with a slot of fp32 sums; part = 1 + slot + (index <<
  // 16).  The last of an item's parts to end, by `done`, joins them.
  int slots;
  int* done;        // counters of parts that ended, cleared by the plan
  int n_done;
};

struct PackedPlan {
  PackedList list[2];
  int lists;
  const int32_t* offsets;
  int n, T, causal, n_buckets;
  int tq, Hk, grid;  // of the backward's key tiles
  int* err;
  // the backward: delta[row] = sum of out * dout over a row's d entries (rows T * Hq)
  const void* out;
  const void* dout;
  float* delta;
  long long rows;
  int d;
};

// A call's tensors: [T, H, d] with strides (token, head) in elements.
struct PackedArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t qs[2], ks[2], vs[2];
  int T, Hq, Hk;
};

constexpr int kMaxPacked = 1 << 20;  // sequences of a call

// The checks that the forward and the backward share, and a tensor's strides (as given,
// or contiguous; false if a tensor map cannot have them).
cp_status check_packed(int T, int n, int Hq, int Hk, int d, int causal);
bool packed_strides(const int64_t* given, int H, int d, int64_t (&to)[2]);

cudaError_t launch_packed_plan(const PackedPlan& p, cudaStream_t stream);

// Slots of a key head for a call of `most` parts a key head, `parts` over all.  With one or two
// the plan's chunk is all that is streamed, which cuts nothing: none then.
inline int packed_slots(long long most, int parts, int Hk) {
  const long long slots = std::min<long long>(most, (parts + Hk - 1) / Hk);
  return slots < 3 ? 0 : static_cast<int>(slots);
}

// Byte sizes and places of a list of tiles of `tokens` tokens.
inline long long packed_items(int T, int n, int tokens) {
  return static_cast<long long>(T) / tokens + n;
}
inline int packed_buckets(int T) { return T / kCostUnit + 2; }
inline long long packed_list_bytes(int T, int n, int tokens) {
  return 256 + 16 * packed_items(T, n, tokens) + 4LL * n + 4LL * packed_buckets(T);
}
inline PackedList packed_list(char* at, int T, int n, int tokens, bool of_keys, int slots = 0) {
  PackedList l{};
  l.head = reinterpret_cast<int*>(at);
  l.items = reinterpret_cast<int4*>(at + 256);
  l.starts = reinterpret_cast<int*>(at + 256 + 16 * (packed_items(T, n, tokens) + slots));
  l.slots = slots;
  l.buckets = l.starts + n;
  l.tokens = tokens;
  l.of_keys = of_keys;
  return l;
}

namespace {

// One CTA's claims of a list: its first item is its own index, later ones come from the
// list's counter (which the plan clears at every call, so a replayed graph starts afresh).
__device__ __forceinline__ int packed_claim(int* head, int grid) {
  return grid + atomicAdd(head + 1, 1);
}

// The CTA's ring of items, as the list has them and with their key heads: the producer reads
// an item once, ahead of its use, and the other roles from shared memory.  (Each reading the
// list waited for L2 at every item's start.)  Full barriers take the producer's arrival, empty
// ones one of each softmax warp; the MMA warp reads a slot with its item's Q (or fixed tiles),
// before its softmax can be done.
struct PackedEntry {
  int4 e;
  int hk;  // -1: no more items
};
struct PackedRing {
  uint32_t bars;             // shared address: kRing full barriers, then kRing empty ones
  volatile int (*slots)[8];  // e.x .. e.w, hk
  __device__ uint32_t full(uint32_t k) const { return bars + 8u * (k % kRing); }
  __device__ uint32_t empty(uint32_t k) const { return bars + 8u * (kRing + k % kRing); }
  __device__ void init(int readers) const {
    for (int s = 0; s < kRing; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), readers);
    }
  }
  // Producer (one thread): the CTA's k-th item.
  template <class P>
  __device__ bool put(uint32_t k, const PackedEntry& x, volatile uint32_t* abort_flag,
                      const P& p) const {
    if (k >= kRing && !wait1(empty(k), (k / kRing - 1) & 1u, abort_flag, p)) return false;
    volatile int* const to = slots[k % kRing];
    to[0] = x.e.x;
    to[1] = x.e.y;
    to[2] = x.e.z;
    to[3] = x.e.w;
    to[4] = x.hk;
    ptx::mbar_arrive(full(k));
    return true;
  }
  // (Every lane of a warp.  The shuffle tells the compiler that the item is one for the warp, so
  // that the loops over its tiles are the warp's and not each lane's.)
  __device__ static PackedEntry uniform(const PackedEntry& x) {
    auto all = [](int y) { return __shfl_sync(0xffffffffu, y, 0); };
    return PackedEntry{make_int4(all(x.e.x), all(x.e.y), all(x.e.z), all(x.e.w)), all(x.hk)};
  }
  __device__ PackedEntry read(uint32_t k) const {
    const volatile int* const from = slots[k % kRing];
    return uniform(PackedEntry{make_int4(from[0], from[1], from[2], from[3]), from[4]});
  }
  // A softmax warp (every lane): the k-th item; false if the wait gave up.
  template <class P>
  __device__ bool get(uint32_t k, PackedEntry& x, volatile uint32_t* abort_flag,
                      const P& p) const {
    if (!wait_warp(full(k), (k / kRing) & 1u, abort_flag, p)) return false;
    x = read(k);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(empty(k));
    return true;
  }
};
// barriers, slots, the MMA warp's word
constexpr int kPackedRingBytes = 2 * kRing * 8 + kRing * 32 + 16;
static_assert(kPackedRingBytes <= 256, "the item ring's shared-memory block");

// The (tile, key head) pair of item w: groups of `hg` heads, in a group the list's order.
// A long list walks few heads at a time, whose keys then come from L2: the smallest group
// whose items fill the grid once; a short one (under 16 rounds of the grid) is one pool, so
// that its cheapest items come last.
struct PackedOrder {
  int items, heads, group, n;
  __device__ PackedOrder(int items_, int heads_, int grid) : items(items_), heads(heads_) {
    n = items * heads;
    group = heads;
    if (n >= 16LL * grid) group = max(1, min(heads, (grid + items - 1) / items));
  }
  // Item w of the list at `list`, whose key head is -1 behind the last.
  __device__ PackedEntry at(const int4* list, int w) const {
    if (w >= n) return PackedEntry{make_int4(0, 0, 0, 0), -1};
    const int g = w / (group * items), r = w - g * group * items;
    const int in_group = min(group, heads - g * group);
    const int tile = r / in_group;
    return PackedEntry{list[tile], g * group + r - tile * in_group};
  }
};

// Item w of a call of few sequences without a plan: the sequences' tiles in their order, the key
// heads of a tile side by side (every lane of the warp calls it).  Malformed offsets: no item.
__device__ __forceinline__ PackedEntry packed_direct(const int32_t* offsets, int n, int T,
                                                     int tokens, int heads, int w, bool& bad) {
  const int lane = threadIdx.x & 31, tile = w / heads;
  PackedEntry found{make_int4(0, 0, 0, 0), -1};
  bad = false;
  int before = 0;
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    int a = 0, len = 0;
    if (i < n) {
      a = __ldg(offsets + i);
      const int z = __ldg(offsets + i + 1);
      bad |= a < 0 || z < a || z > T;
      len = z - a;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad) return PackedEntry{make_int4(0, 0, 0, 0), -1};
    const int tiles = (len + tokens - 1) / tokens;
    int x = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int start = before + x - tiles;
    const unsigned has = __ballot_sync(0xffffffffu, tile >= start && tile < start + tiles);
    if (has) {
      const int from = __ffs(has) - 1;
      found.e = make_int4(__shfl_sync(0xffffffffu, a, from), __shfl_sync(0xffffffffu, len, from),
                          tile - __shfl_sync(0xffffffffu, start, from), 0);
      found.hk = w - tile * heads;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  return found;
}

// A warp's 32 rows of 128 bytes in shared memory, 16-byte chunk c of row r at c ^ (r mod 8), from
// which rows are written to memory by whole lines: a thread that stores its own row writes half
// sectors of 32 lines at a time.
constexpr int kRowStage = 32 * 128;
__device__ __forceinline__ void stage_chunk(uint32_t base, int row, int chunk, uint32_t a,
                                            uint32_t b, uint32_t c, uint32_t d) {
  ptx::st_shared_v4(base + row * 128 + ((chunk ^ (row & 7)) << 4), a, b, c, d);
}
// `to`: where this lane's row starts (null: it is not written).
__device__ __forceinline__ void write_rows(uint32_t base, __nv_bfloat16* to, int lane) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = i * 4 + lane / 8, chunk = lane % 8;
    const unsigned long long at =
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), row);
    uint4 u;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "r"(base + row * 128 + ((chunk ^ (row & 7)) << 4)));
    if (at != 0) reinterpret_cast<uint4*>(at)[chunk] = u;
  }
  __syncwarp();
}

// What another block wrote during this kernel (past L1).
__device__ __forceinline__ float4 load_cg(const float4* at) {
  float4 f;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
               : "l"(at)
               : "memory");
  return f;
}

// Zeroes the bytes [from, to) of shared memory (multiples of 16) with the lanes of a warp.
__device__ __forceinline__ void zero_shared(uint32_t from, uint32_t to) {
  for (uint32_t at = from + (threadIdx.x & 31) * 16; at < to; at += 512)
    ptx::st_shared_v4(at, 0u, 0u, 0u, 0u);
}
// Rows [first, end) of every 128-byte panel of a 128-row tile (the swizzle moves
// chunks within a row only).
template <int kPanels>
__device__ __forceinline__ void zero_rows(uint32_t tile, int first, int end) {
#pragma unroll
  for (int pn = 0; pn < kPanels; ++pn)
    zero_shared(tile + pn * kTileRows * 128 + first * 128, tile + pn * kTileRows * 128 + end * 128);
}

// [T, H, d] with strides (token, head) in elements as (d, H, T); box = one 128-byte panel x
// `heads` x `tokens`.  Strides as packed_strides_ok accepts them.
bool packed_map(CUtensorMap* m, const void* base, int T, int H, int d, long long ts, long long hs,
                int heads, int tokens) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  if (H == 1) hs = d;        // a dimension of one entry: the stride is never used
  if (T == 1) ts = hs * H;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hs) * 2, static_cast<cuuint64_t>(ts) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace cpring
