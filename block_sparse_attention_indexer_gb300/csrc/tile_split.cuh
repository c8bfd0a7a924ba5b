// The split of a flat list of (tile, page) steps over a persistent grid, by the units' prefix sums (the
// kernels of 128-row tiles: fp8_tile.cu, prompt_attn.cu).
#pragma once

#include <stdint.h>

namespace msa {

// First step of CTA c of n.
__device__ __forceinline__ int ft_lo(int64_t E, int c, int n) { return static_cast<int>(E * c / n); }

// The last unit u with prefix[u] * G <= x, by a whole warp: 32 places a round.
__device__ __forceinline__ int ft_find(const int32_t* prefix, int units, int groups, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = units;  // it is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool below = at < lo + n && static_cast<int64_t>(prefix[at]) * groups <= x;
    const int k = __popc(__ballot_sync(0xffffffffu, below)) - 1;  // (the first place always is)
    n = min(step, lo + n - (lo + k * step));
    lo += k * step;
  }
  return lo;
}

// A cut at place x of the list, in it: inside a unit that stays whole it goes to the nearer of its ends.  A whole warp
// calls it.
__device__ __forceinline__ int ft_cut_inside(const int32_t* prefix, int units, int G, int x, int whole) {
  const int u = ft_find(prefix, units, G, x), steps = prefix[u + 1] - prefix[u];
  if (steps > whole) return x;
  const int off = (x - prefix[u] * G) % steps;
  return x - off + (2 * off < steps ? 0 : steps);
}

// First step of CTA c of n as it is taken.
__device__ __forceinline__ int ft_cut(const int32_t* prefix, int units, int G, int64_t E, int c, int n, int whole) {
  const int x = ft_lo(E, c, n);
  if (c == 0 || x >= E) return x;
  return ft_cut_inside(prefix, units, G, x, whole);
}

// n / d for 0 <= n < 2^29 and 1 <= d <= 8: with m = ceil(2^32 / d), n m / 2^32 exceeds n / d by less than
// n d / (2^32 d) < 1 / d.
struct FtDiv {
  uint32_t m;
  __device__ __forceinline__ explicit FtDiv(int d) : m(d > 1 ? 0xFFFFFFFFu / static_cast<uint32_t>(d) + 1u : 0u) {}
  __device__ __forceinline__ int operator()(int n) const { return m != 0u ? static_cast<int>(__umulhi(n, m)) : n; }
};

}  // namespace msa
