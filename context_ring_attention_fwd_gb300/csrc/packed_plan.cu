// The plan of a call over packed prompts: every sequence's tiles in a list, the most
// expensive first.
//
// For the backward the launch's other blocks form D = rowsum(dO * O), which is bound by its
// two reads.
//
// One block per list.  The sequences' tiles are counted and summed, and the tiles are
// sorted by cost (key tiles that a query tile sees, or the reverse) by counting: each
// finds its sequence by bisection of the sums.  Ties keep no order, which decides only
// the CTA that computes an item, never a result.  Bound by the latency of its few passes.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "packed.cuh"

namespace cpring {
namespace {

constexpr int kPlanThreads = 1024;  // or, where one pass of so few is enough:
constexpr int kFewThreads = 256;
constexpr int kWarps = kPlanThreads / 32;
// Vectors of a row that a thread has under way for D.  (126 MB, in the kernel: two 22 us, one 24,
// four 26.)
constexpr int kAtOnce = 2;
constexpr int kSmall = 2048;  // sums and buckets up to this many stay in shared memory

// Exclusive sum over the block; `total` gets the whole.
__device__ __forceinline__ int block_scan(int x, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();  // an earlier call's sums are read
  if (lane == 31) warp_sum[warp] = y;
  __syncthreads();
  int s = lane < blockDim.x / 32 ? warp_sum[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += z;
  }
  total = __shfl_sync(0xffffffffu, s, kWarps - 1);
  const int before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  return y - x + (warp > 0 ? before : 0);
}

__device__ __forceinline__ float block_sum(float x, float* warp_sum) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) x += warp_sum[w];
  return x;
}

// The tiles that an item streams: key tiles that its queries see, or packed query tiles that
// see its keys; and the bucket of part j of `chunk` of them.
__device__ __forceinline__ int streamed_tiles(const PackedPlan& p, const PackedList& l,
                                              const int4& it) {
  if (l.of_keys) return (it.y - 1) / p.tq - (p.causal ? it.z * kTileRows / p.tq : 0) + 1;
  const long long seen = p.causal ? (it.z + 1LL) * l.tokens : it.y;
  return (static_cast<int>(min(seen, static_cast<long long>(it.y))) - 1) / kTileRows + 1;
}
__device__ __forceinline__ int part_bucket(const PackedPlan& p, const PackedList& l,
                                           const int4& it, int j, int chunk) {
  const int tiles = min(chunk, streamed_tiles(p, l, it) - j * chunk);
  const int tokens = tiles * (l.of_keys ? p.tq : kTileRows);
  return max(0, p.n_buckets - 1 - (tokens + kCostUnit - 1) / kCostUnit);
}

// D of rows dealt over `blocks` blocks: 8 entries to a lane, d / 8 lanes to a row.
__device__ __forceinline__ void row_dots(const PackedPlan& p, int block, int blocks) {
  const int shift = p.d == 128 ? 4 : 3, lanes = 1 << shift;
  const long long vecs = p.rows << shift, step = static_cast<long long>(blocks) * blockDim.x;
  const uint4* const out = static_cast<const uint4*>(p.out);
  const uint4* const dout = static_cast<const uint4*>(p.dout);
  const long long end = (vecs + 31) / 32 * 32;  // whole warps
  for (long long x0 = static_cast<long long>(block) * blockDim.x + threadIdx.x; x0 < end;
       x0 += kAtOnce * step) {
    uint4 a[kAtOnce], b[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const long long x = x0 + k * step;
      a[k] = b[k] = make_uint4(0, 0, 0, 0);
      if (x < vecs) {
        a[k] = __ldg(out + x);
        b[k] = __ldg(dout + x);
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const long long x = x0 + k * step;
      const uint32_t u[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
      const uint32_t w[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(w[i] << 16), s);
        s = fmaf(__uint_as_float(u[i] & 0xffff0000u), __uint_as_float(w[i] & 0xffff0000u), s);
      }
      for (int o = lanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (x < vecs && (x & (lanes - 1)) == 0) p.delta[x >> shift] = s;
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PackedPlan p) {
  __shared__ int warp_sum[kWarps], next_slot;
  __shared__ float streamed_sum[kWarps];
  __shared__ int near_starts[kSmall], near_buckets[kSmall];
  cudaTriggerProgrammaticLaunchCompletion();  // the attention's blocks may line up
  if (blockIdx.x >= p.lists) {
    row_dots(p, blockIdx.x - p.lists, gridDim.x - p.lists);
    return;
  }
  const PackedList l = p.list[blockIdx.x];
  int* const starts = p.n <= kSmall ? near_starts : l.starts;
  int* const buckets = p.n_buckets <= kSmall ? near_buckets : l.buckets;
  for (int i = threadIdx.x; i < p.n_buckets; i += blockDim.x) buckets[i] = 0;
  int items = 0;
  float streamed = 0.f;  // tiles that the items of a key head stream, or a little more
  bool bad = false;
  for (int base = 0; base < p.n; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int tiles = 0;
    if (i < p.n) {
      const int a = __ldg(p.offsets + i), z = __ldg(p.offsets + i + 1);
      if (a < 0 || z < a || z > p.T)
        bad = true;
      else
        tiles = (z - a + l.tokens - 1) / l.tokens;
      if (l.slots > 0 && tiles > 0) {
        const float t = tiles, all = (z - a - 1) / (l.of_keys ? p.tq : kTileRows) + 1;
        // Causal: the k-th of the key tiles does not stream the first k kTileRows / tq (rounded
        // down), the k-th of the query tiles streams (k + 1) tokens / kTileRows (rounded up).
        float some = t * all;
        if (p.causal && l.of_keys)
          some -= fmaxf(0.f, t * (t - 1.f) * (0.5f * kTileRows) / p.tq - t);
        else if (p.causal)
          some = fminf(some, t * (t + 1.f) * (0.5f / kTileRows) * l.tokens + t);
        streamed += some;
      }
    }
    int total;
    const int before = block_scan(tiles, warp_sum, total);
    if (i < p.n) starts[i] = items + before;
    items += total;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      l.head[0] = l.head[1] = 0;
      atomicOr(p.err, kErrDocOffsets);
    }
    return;
  }
  // Item x: its sequence's rows, its tile, and the bucket of its cost (0: the largest).
  auto item = [&](int x, int& bucket) {
    int lo = 0, hi = p.n;  // the last sequence that starts at or before x; empty ones are passed
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= x) lo = mid; else hi = mid;
    }
    const int row = __ldg(p.offsets + lo), len = __ldg(p.offsets + lo + 1) - row;
    const int tile = x - starts[lo];
    int cost = len;
    if (p.causal)
      cost = l.of_keys ? len - tile * l.tokens
                       : static_cast<int>(min(static_cast<long long>(len),
                                              (tile + 1LL) * l.tokens));
    bucket = p.n_buckets - 1 - (cost + kCostUnit - 1) / kCostUnit;
    return make_int4(row, len, tile, 0);
  };
  // Items that stream more than a CTA's share of the work are cut, so that a call of few items
  // fills the GPU and ends at one time.  A part costs about 5 streamed tiles besides its own (its
  // start, its sums' way through memory, their addition), so parts are as many as CTAs where
  // the share is small, 1.3 of it, and down to 0.6 of it where it is large; they are no
  // shorter than kLeastPart, and items of up to kLeastCut stay whole.  Measured for the backward's
  // key tiles, whole / cut (us a call): 4096 tokens of 8/1 heads 409 / 130, 8192 of 8/2 622 /
  // 331, 5000 + 2500 of 16/2 720 / 329, 1500 of 2/1 50 / 35; 200 of 16/4 (7 streamed tiles) 25 /
  // 25, which stays whole.
  // Key tiles that are no more than the CTAs are cut down to 0.45 of the share: so / to 0.6, 8192
  // tokens of 8/2 heads 331 / 377, 5000 + 2500 of 16/2 329 / 359.  More of them balance
  // themselves: 9000 of 4/4 (d = 64) 183 / 177, 3000 + 200 + 100 of 32/8 222 / 215, 10 prompts of
  // 32/8 281 / 278.  (Nor does the forward gain: 20000 of 1/1, d = 64, 82 / 78.)
  int chunk = INT_MAX;
  auto parts_of = [&](const int4& it) {
    const int n = streamed_tiles(p, l, it);
    return n <= kLeastCut ? 1 : (n - 1) / chunk + 1;
  };
  if (l.slots > 0) {
    // An item of n > chunk streamed tiles is cut into less than n / chunk + 1 parts, and into at
    // most 2 n / chunk, so there are no more parts than slots with a chunk of at least
    // 1 / (slots - items) of all streamed tiles, or of 2 / slots.
    const float all = 1.001f * block_sum(streamed, streamed_sum);  // (whatever was rounded)
    const float mean = all * p.Hk / p.grid;
    const float down = l.of_keys && static_cast<long long>(items) * p.Hk <= p.grid ? 0.45f : 0.6f;
    const float share = down * mean + fminf((1.3f - down) * mean, 20.f);
    const float least = 2 * items < l.slots ? all / (l.slots - items) : 2.f * all / l.slots;
    chunk = max(kLeastPart, static_cast<int>(fminf(fmaxf(share, least) + 1.f, 1e9f)));
    for (int i = threadIdx.x; i < l.n_done; i += blockDim.x) l.done[i] = 0;
    if (threadIdx.x == 0) l.head[2] = chunk;
  }
  for (int x = threadIdx.x; x < items; x += blockDim.x) {
    int b;
    const int4 it = item(x, b);
    const int n = l.slots > 0 ? parts_of(it) : 1;
    if (n == 1) {
      atomicAdd(buckets + b, 1);
    } else {
      for (int j = 0; j < n; ++j) atomicAdd(buckets + part_bucket(p, l, it, j, chunk), 1);
    }
  }
  __syncthreads();
  int placed = 0;
  for (int base = 0; base < p.n_buckets; base += blockDim.x) {
    const int i = base + threadIdx.x;
    const int x = i < p.n_buckets ? buckets[i] : 0;
    int total;
    const int before = block_scan(x, warp_sum, total);
    if (i < p.n_buckets) buckets[i] = placed + before;
    placed += total;
  }
  if (threadIdx.x == 0) {
    l.head[0] = placed;
    l.head[1] = 0;
    next_slot = 0;
  }
  __syncthreads();
  for (int x = threadIdx.x; x < items; x += blockDim.x) {
    int b;
    int4 it = item(x, b);
    const int n = l.slots > 0 ? parts_of(it) : 1;
    if (n == 1) {
      l.items[atomicAdd(buckets + b, 1)] = it;
      continue;
    }
    const int slot = atomicAdd(&next_slot, n);
    for (int j = 0; j < n; ++j) {
      const int at = atomicAdd(buckets + part_bucket(p, l, it, j, chunk), 1);
      l.items[at] = make_int4(it.x, it.y, it.z, 1 + slot + j + (j << 16));
    }
  }
}

}  // namespace

cudaError_t launch_packed_plan(const PackedPlan& p, cudaStream_t stream) {
  unsigned blocks = p.lists;
  const bool few = p.n <= kFewThreads && p.T / p.list[0].tokens <= kFewThreads;
  const int threads = few ? kFewThreads : kPlanThreads;
  if (p.delta) {
    const long long want = (p.rows * (p.d / 8) + kAtOnce * threads - 1) / (kAtOnce * threads);
    const long long most = (few ? 6LL : 2LL) * sm_count();
    blocks += static_cast<unsigned>(std::min<long long>(want, most));
  }
  packed_plan_kernel<<<blocks, threads, 0, stream>>>(p);
  count_launch(2);
  return cudaGetLastError();
}

}  // namespace cpring
