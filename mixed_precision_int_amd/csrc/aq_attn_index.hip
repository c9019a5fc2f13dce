// Attention over the 4-bit cache: the index of many packed sequences, and the
// choice of the kernel.
//
// A workgroup of the attention kernels finds its sequence by summing the rows and
// lengths of all of them, 64 at a time, which costs each of them more the more there
// are.  Beyond kSearched sequences one workgroup does that for all, into the
// workspace (four sequences a thread, 4096 a turn).

#include "aq_attn.h"

namespace aq {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64, kEach = 4;
constexpr long long kFar = 1LL << 30;  // (sums stop there: offsets that do not increase may give any number)

// Sums over threads 0 .. n of the workgroup; `all` that of all.
template <typename T>
__device__ __forceinline__ T block_sums_to(T x, T *waves, T &all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const T y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // (the sums of the turn before are read)
  if (lane == 63) waves[wave] = x;
  __syncthreads();
  T before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? waves[w] : 0;
    all += waves[w];
  }
  return before + x;
}

__global__ __launch_bounds__(kThreads) void attn_index_kernel(AttnArgs a, int T, int unit) {
  __shared__ long long waves[2][kWaves];
  long long units = 0;
  if (a.splits > 1) {
    for (int b0 = 0; b0 < a.B; b0 += kThreads * kEach)
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        int first, n, len;
        sequence(a, b0 + kEach * (int)threadIdx.x + e, first, n, len);
        units += (long long)ceil_div(n * a.G, T) * ceil_div(len, unit);
      }
    long long all;
    block_sums_to(units, waves[0], all);
    units = all;
  }
  const int per = a.splits > 1 ? units_each((float)units, a.c.heads) : 1 << 30;
  if (threadIdx.x == 0) a.index[0] = per;
  int32_t *items_to = a.index + kIndexHead, *tiles_to = items_to + a.B;
  long long items0 = 0, tiles0 = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads * kEach) {
    const int b = b0 + kEach * (int)threadIdx.x;
    long long items[kEach], tiles[kEach];  // of the thread's sequences, up to each
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      int first, n, len, mine;
      sequence(a, b + e, first, n, len);
      tiles[e] = ceil_div(n * a.G, T);
      items[e] = tiles[e] * ranges_in(len, unit, per, mine);
      if (e) {
        tiles[e] += tiles[e - 1];
        items[e] += items[e - 1];
      }
    }
    long long all_items, all_tiles;
    const long long ib = items0 + block_sums_to(items[kEach - 1], waves[0], all_items) - items[kEach - 1];
    const long long tb = tiles0 + block_sums_to(tiles[kEach - 1], waves[1], all_tiles) - tiles[kEach - 1];
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (b + e < a.B) {
        items_to[b + e] = (int32_t)min(ib + items[e], kFar);
        tiles_to[b + e] = (int32_t)min(tb + tiles[e], kFar);
      }
    items0 += all_items;
    tiles0 += all_tiles;
  }
}

}  // namespace

hipError_t launch_attn_kv4(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
  const bool rows = p.rows <= 16;
  if (a.index) {
    hipLaunchKernelGGL(attn_index_kernel, dim3(1), dim3(kThreads), 0, stream, a, p.rows, rows ? 256 : 8192 / a.c.D);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return rows ? launch_attn_rows(a, p.rows, stream) : launch_attn_tiles(a, stream);
}

}  // namespace aq
