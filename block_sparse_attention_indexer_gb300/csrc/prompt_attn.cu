// Causal attention of packed bf16 prompts on the tcgen05 tensor cores.
//
// Mathematics: P_j = 2^(e_j - M) with e_j = (q . k_j) softmax_scale log2(e), O = sum P_j v_j, l = sum P_j; lse = ln 2 (M +
// log2 l).  M is an integer (rescaling O and l is exact) that moves only where a P would pass 1, to 2^8 above the largest
// so far, so that most blocks move nothing; rows with an e of 2^27 or more have a way of their own (kPtFused).
// P is rounded to bf16, V's type, as the operand of P V: by 2^-8 of itself at most, whatever its size (bf16 has
// float32's range).  O is divided by the sum of the rounded P: a common part of their errors cancels, and a row's
// error is at most that of rounding its output, on average (with l, a row of one key would be off by P's whole
// rounding).  l adds P before the rounding, for lse.  S, O, l and M are float32.
//
// Work.  A row is a (token, head) of a KV head; a tile is 128 rows, floor(128 / Hg) tokens with their Hg heads, a
// unit two tiles (or one, of a sequence's last tokens) of a sequence and a KV head, so that keys loaded once meet
// 256 rows and the causal border costs half a block of 128 keys for each tile, whatever Hg is.  A unit's cost is
// counted in (tile, 128 keys) steps and kPtUnitCost for its start.  A persistent grid, one CTA an SM, gets the units whole,
// dealt out by falling cost, where that balances (kPtCutSteps); else all units are one flat list that is cut into equal
// ranges (tile_split.cuh), and units that are cut leave partial states, which a second kernel adds.  Two accumulator
// slots work in turn: with two tiles each block of keys is used by slot 0 and slot 1, with one tile the blocks
// alternate between the slots.
//   * S = Q K^T: Q and K by tensor copies in 128-byte swizzle (a Q tile is one box of Hg heads by tokens).
//   * O += P V: P in tensor memory over S (the A operand), V as it lies, as the MN-major B operand.
// TMEM: S of the two slots, then O of the two slots: 4 x 128 columns, all of it.
//
// Warps: 0-3 and 4-7 softmax of slot 0 and 1 (one row per thread, a block's 128 scores in registers), 8-11 write the
// rows of a unit while the next one's softmax runs, and look through the V rows that not every row of a unit sees, 12 makes the
// units known and copies Q and K, 13 issues the products S, 14 P V, 15 copies V.
// What a row does not see cannot reach it: its S is replaced by -inf, and infinities and NaN in V are taken out of the blocks
// that not every row of the unit sees; rows that do see them get them back at the end, times their probability.
// Every wait is bounded; a role that gives up flags MSA_DEVERR_TIMEOUT, leaves its loop and meets
// the others at the end, where TMEM is freed.
//
// What bounds it: a slot's chain (S, softmax, P V of a block, one after another) is about as long as both slots' products,
// and the products run at the power limit's clock: 1.42 to 1.45 ms, 1.52 to 1.55 PFLOP/s, for a prompt of 16K tokens and 32
// heads, 7 % less without any exponential.  Measured on the way there, for that prompt: S by halves of 64 keys, so that a half's
// product runs beside the other's softmax, 1.78 ms against 1.43 (an M 128 x N 64 product takes 390 cycles where half of N 128
// takes 256: its operands fill the shared memory's bandwidth); 64 scores at a time 1.51 against 1.33; one hand-over of P
// for 128 keys 1.41 against 1.35; the exponentials of the second half held back behind the first half's hand-over 1.37.
// Stages of K and V and register shares: 1 to 3 %.  Code that a unit runs once costs its instruction fetches (the
// epilogue, unrolled masks: 1 us and more each), so it is short loops, and the softmax's loop has nothing
// rare inside it; function calls in that branch cost it registers (1.40 -> 1.48 ms).  The compiler's report should show no
// spills for it: changes of the V warps' code that brought 8 to 16 bytes of them cost 2 to 4 %, wherever they were.
// Short units wait for latencies: for 31 prompts of 310 to 2,000 tokens (4,612 units, 357 to 361 us) 2 us of a unit's 12 are
// not its steps, and tensor instructions run 58 % of the time (69 % for one prompt of 8K tokens, 365 us).  Products of 64
// keys where a unit's last block has no more: the same to 2 % slower.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <limits.h>

#include "fp8_device.cuh"
#include "fp8_kernels.h"
#include "fp8_merge.cuh"
#include "msa_device.cuh"
#include "prompt.h"
#include "tile_split.cuh"
#include "umma.cuh"

namespace msa {

constexpr int kPtRows = 128;  // rows per tile
constexpr int kPtThreads = 512;
constexpr int kPtK = 2, kPtV = 3;             // stages of 128 keys
constexpr int kPtItems = 2;                   // units known ahead
constexpr int kPtTile = kPtRows * kDim * 2;   // bytes of a Q tile, and of a stage
constexpr int kPtHalf = kPtTile / 2;          // 64 dims of it
constexpr int kPtPlaceFloats = 2 * kPtRows * (kDim + 2);
constexpr uint32_t kPtO = 256;                // TMEM column of slot 0's O
constexpr float kPtRefSet = 8.f;
// From this size of a row's largest e on, e is rounded to float32 before M is subtracted, and M is the largest e itself.  Below it
// S f - M is one fma, with S f exact, while M comes from the rounded S f: the two differ by up to half a unit in the last
// place, 4 below 2^27 but 256 and more from 2^32 on, where every P would be 0 or the largest infinite.  For such rows
// (e - M) / f takes the place of S, and 0 that of M, so that the others' code stays as it is: with a factor and a reference of their
// own for every row, 31 ragged prompts took 363 us instead of 357.
constexpr float kPtFused = 134217728.f;
constexpr int kPtUnitCost = kPromptUnitCost;
// Cost of a unit up to which it is not cut: a cut costs two partial states and a merge, a cut moved to the end of its
// unit leaves one CTA up to half of the unit more than its share.
constexpr int kPtWhole = 16;
// What cutting costs a call (partial states, the merge of 150 units) in steps: without cuts a CTA may have so much more
// than its share.  One prompt of 1K 31 us cut and 26 whole, of 2K 51 and 39, of 4K 116 and 106, of 8K 368 and 357; 31 of 310
// to 2,000 tokens 380 and 358.  4 chunks on 16K, 120 units for 152 CTAs, are cut (their longest has twice a CTA's share).
constexpr int kPtCutSteps = 14;
// Units (of a KV head) up to which they are put in order for that.
constexpr int kPtSpreadUnits = kPromptSpreadUnits;

// A unit, or the part of it that this CTA has: blocks lo .. hi - 1 of 128 keys (none of a unit whose rows see no key).
struct alignas(16) PtItem {
  int flags;   // kPtEnd: no more units; kPtTwo: two tiles; place of its partial state + 1 from kPtPlace on
  int lo, hi;
  int token0;  // the unit's first query token, in the packed list
  int tokens;  // of the unit
  int pos0;    // the first one's position
  int key0;    // the sequence's first key, in the packed list
  int g;
  // the first of its blocks that some row of the unit does not see whole
  __device__ __forceinline__ int edge() const { return min(max(lo, max(pos0 + 1, 0) / kBlock), hi); }
};
constexpr int kPtEnd = 1, kPtTwo = 2, kPtPlace = 2;

struct PtShared {
  uint64_t k_full[kPtK], k_empty[kPtK], v_empty[kPtV];
  uint64_t v_full[kPtV], v_edge[kPtV], v_ok[kPtV];  // plain blocks by turns; edge blocks by turns: copied, looked through
  uint64_t item_full[kPtItems], item_empty[kPtItems];
  uint64_t s_full[2], p_full[2][2], pv_done[2];     // [slot], [slot][half of the keys], [slot]
  uint64_t q_full[2], q_empty[2];                   // [tile]
  uint64_t fin[2], o_full[2], o_empty[2];           // [slot], a unit's: factors left, products done, O read
  uint64_t other;                                   // slot 1's statistics of a one-tile unit left
  uint64_t drain[2];                                // every product issued has ended (after a wait that gave up)
  uint32_t tmem;
  int special[8][4];                                // the last unit (by turns) in whose V warp 8 + i found something
  PtItem item[kPtItems];
  float factor[2][kPtRows];                         // of the rows of the slots' O
  float other_m[kPtRows], other_l[kPtRows];
};
constexpr size_t kPtSmem = 2 * kPtTile + (kPtK + kPtV) * kPtTile + sizeof(PtShared);
static_assert(kPtSmem <= 232448, "227 KB of shared memory per CTA");

struct PromptMaps {
  CUtensorMap q, k, v;
};

// The bounded waits of msa_device.cuh, kept short
__device__ __forceinline__ bool pt_wait(uint64_t* bar, uint32_t parity) {
  uint32_t i = kSpinLimit;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (--i == 0u) return false;
  return true;
}
__device__ __forceinline__ bool pt_wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, pt_wait(bar, parity)) != 0;
}

// ---------------------------------------------------------------- the plan

// Unit i of a sequence.
struct PtUnit {
  int tokens, pos0, width, pages;  // pages 0: no row has a key
  // its share of the flat list, and the blocks before place y of that
  __device__ __forceinline__ int cost() const { return width * max(pages, 1) + kPtUnitCost; }
  __device__ __forceinline__ int block_at(int64_t y) const {
    return static_cast<int>(max(min(y, static_cast<int64_t>(cost())) - kPtUnitCost, int64_t{0}) / width);
  }
};
__device__ __forceinline__ PtUnit pt_unit(int Lq, int Lk, int i, int tile_tokens) {
  PtUnit t;
  const int first = i * 2 * tile_tokens;
  t.tokens = min(Lq - first, 2 * tile_tokens);
  t.pos0 = Lk - Lq + first;
  t.width = t.tokens > tile_tokens ? 2 : 1;
  const int last = t.pos0 + t.tokens - 1;
  t.pages = last < 0 ? 0 : last / kBlock + 1;
  return t;
}

// Exclusive prefix sum of v over the CTA plus `carry`, which moves on by the sum.
__device__ __forceinline__ int pt_prefix(int v, int& carry, int* warp_sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x / 32;
  int x = v;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  const int w = lane < warps ? warp_sum[lane] : 0;
  const int at = carry + x - v + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  carry += __reduce_add_sync(0xffffffffu, w);
  return at;
}

// The plan by a whole CTA: base[b], b = 0..batch: units of the sequences before b; prefix[u], u = 0..units: cost (per
// KV head) of the units before u; order[r], for at most kPtSpreadUnits: the units by falling cost.  Returns the units (0
// where the offsets are bad, and `flag` reports them), with kPtSpread where the units stay whole: dealt out by falling
// cost, forth and back over the n CTAs (pt_dealt), none of these gets much more than its share.
// The sort goes through the cost's bits from the lowest on and keeps the order of what is equal: where every CTA makes
// the plan for itself, all of them have to find the same one.
constexpr int kPtSpread = 1 << 30;
constexpr int kPtMaxDealt = 128;  // units of a CTA
__device__ __forceinline__ int pt_dealt(int k, int c, int n) { return k & 1 ? (k + 1) * n - 1 - c : k * n + c; }
struct PtPlanSpace {
  int *base, *cost, *sum, *zeros;   // shared: batch + 1, units, 32, 64
  int32_t *prefix, *order, *other;  // order and other (both shared): units
};
__device__ __forceinline__ int pt_plan(const PromptArgs& a, const PtPlanSpace& s, bool flag, int n) {
  const int tid = threadIdx.x, threads = blockDim.x, tt = kPtRows / a.heads_per_group, G = a.groups;
  bool bad = false;
  int units = 0;
  for (int b0 = 0; b0 < a.batch; b0 += threads) {
    const int b = b0 + tid;
    int x = 0;
    if (b < a.batch) {
      const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
      bad |= q0 < 0 || k0 < 0 || q1 < q0 || k1 < k0 || q1 > a.q_tokens || k1 > a.k_tokens;
      x = bad ? 0 : (q1 - q0 + 2 * tt - 1) / (2 * tt);
    }
    const int at = pt_prefix(x, units, s.sum);
    if (b < a.batch) s.base[b] = at;
  }
  if (__syncthreads_or(bad)) {  // nothing is done
    if (flag && tid == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
    return 0;
  }
  if (tid == 0) s.base[a.batch] = units;
  __syncthreads();
  const bool sorted = units <= kPtSpreadUnits && units * G <= (kPtMaxDealt - 1) * n;
  int all = 0, largest = 0;
  for (int u0 = 0; u0 < units; u0 += threads) {
    const int u = u0 + tid;
    int x = 0;
    if (u < units) {
      int b = 0, left = a.batch;  // the last sequence with base <= u
      while (left > 1) {
        const int h = left / 2;
        if (s.base[b + h] <= u) {
          b += h;
          left -= h;
        } else {
          left = h;
        }
      }
      x = pt_unit(a.cu_q[b + 1] - a.cu_q[b], a.cu_k[b + 1] - a.cu_k[b], u - s.base[b], tt).cost();
      if (sorted) s.cost[u] = x;
    }
    largest = max(largest, x);
    const int at = pt_prefix(x, all, s.sum);
    if (u < units) s.prefix[u] = at;
  }
  if (tid == 0) s.prefix[units] = all;
  if (!sorted || units == 0) return units;
  largest = __reduce_max_sync(0xffffffffu, largest);
  __syncthreads();
  if ((tid & 31) == 0) s.sum[tid >> 5] = largest;
  __syncthreads();
  largest = __reduce_max_sync(0xffffffffu, (tid & 31) < threads / 32 ? s.sum[tid & 31] : 0);
  if (largest <= kPtWhole) return units;  // nothing is cut in any case
  const int warp = tid >> 5, lane = tid & 31, warps = threads / 32, groups = (units + 31) / 32, bits = 32 - __clz(largest);
  int32_t *from = nullptr, *to = bits & 1 ? s.order : s.other;  // (the last pass goes to s.order)
  auto unit_at = [&](int bit, int i) { return bit == 0 ? i : from[i]; };
  static_assert(kPtSpreadUnits / 32 <= 64, "two counts a lane");
  for (int bit = 0; bit < bits; ++bit) {
    // units without the bit in largest - cost come first: how many each 32 places have
    for (int w = warp; w < groups; w += warps) {
      const int i = 32 * w + lane;
      const uint32_t zeros = __ballot_sync(0xffffffffu, i < units && !((largest - s.cost[unit_at(bit, i)]) >> bit & 1));
      if (lane == 0) s.zeros[w] = __popc(zeros);
    }
    __syncthreads();
    const int low = lane < groups ? s.zeros[lane] : 0, high = lane + 32 < groups ? s.zeros[lane + 32] : 0;
    const int all_zeros = __reduce_add_sync(0xffffffffu, low + high);
    for (int w = warp; w < groups; w += warps) {
      const int i = 32 * w + lane, u = i < units ? unit_at(bit, i) : 0;
      const bool zero = i < units && !((largest - s.cost[u]) >> bit & 1);
      const int before = __reduce_add_sync(0xffffffffu, (lane < w ? low : 0) + (lane + 32 < w ? high : 0)) +
                         __popc(__ballot_sync(0xffffffffu, zero) & ((1u << lane) - 1));
      if (i < units) to[zero ? before : all_zeros + i - before] = u;
    }
    __syncthreads();
    from = to;
    to = to == s.order ? s.other : s.order;
  }
  int64_t most = 0;  // that a CTA gets
  if (tid < n) {
    const FtDiv by_g(G);
    const int each = (units * G + n - 1) / n;
#pragma unroll 4
    for (int k = 0; k < each; ++k) {
      const int at = pt_dealt(k, tid, n);
      if (at < units * G) most += s.cost[s.order[by_g(at)]];
    }
  }
  const bool much = most > static_cast<int64_t>(all) * G / n + kPtCutSteps;
  return units | (__syncthreads_or(much) ? 0 : kPtSpread);
}

// Sequences and units up to which every CTA of the attention makes the plan for itself (a launch for the plan cost 8 short
// prompts 6.6 us more).  More are planned by a launch before it.
constexpr int kPtOwnBatch = kPtThreads, kPtOwnUnits = 2048;
// Calls without a plan: the units are dealt out whole, as they come, by the producer's warp alone.  For up to so many
// sequences, where no unit can cost more than kPtQuickCost, and for one prompt (lengths as its tokens say) that has a unit
// for every CTA, where none can cost more than kPtQuickOne and what a CTA would get above its share is little.  8 short
// prompts 11.3 -> 8.1 us, one of 512 tokens 15.7 -> 12.9, of 1K 25.5 -> 20.3, of 2K 38.7 -> 33.2, of 3,500 86 -> 81; where
// cuts help most, 100 tokens on 1,500 keys, 24.9 -> 26.0.  With the larger limit for more sequences, 5 of up to 900 tokens took
// 29 us instead of 24.
constexpr int kPtQuickBatch = 64, kPtQuickCost = 32, kPtQuickOne = 64, kPtQuickSteps = 20;
static bool pt_quick(const PromptArgs& a, int64_t largest, int ctas) {
  if (a.batch > kPtQuickBatch) return false;
  if (largest <= kPtQuickCost) return true;
  const int pair = 2 * prompt_tile_tokens(a.heads_per_group), units = (a.q_tokens + pair - 1) / pair * a.groups;
  if (a.batch > 1 || largest > kPtQuickOne || units < ctas) return false;
  const int before = a.k_tokens > a.q_tokens ? a.k_tokens - a.q_tokens : 0, rest = units % ctas;
  const float least = 2.f * ((before + pair + kBlock - 1) / kBlock) + kPtUnitCost;  // cost of the first unit
  const float rise = (largest - least) / units, half = (units / ctas & 1) ? .5f * rise * ctas : 0.f;
  const float more = rest > 0 ? least + .5f * rise * rest - half : 0.f;             // a round begun
  return (more > half ? more : half) <= kPtQuickSteps;
}

// The same in shared memory, by every CTA of the attention.
struct PtOwnPlan {
  int cost[kPtOwnUnits], base[kPtOwnBatch + 1], sum[32], zeros[64];
  int32_t prefix[kPtOwnUnits + 1], order[kPtOwnUnits], other[kPtOwnUnits];
};
__device__ __noinline__ int pt_own_plan(const PromptArgs& a, PtOwnPlan& s) {
  return pt_plan(a, PtPlanSpace{s.base, s.cost, s.sum, s.zeros, s.prefix, s.order, s.other}, blockIdx.x == 0, gridDim.x);
}

constexpr int kPtPlanThreads = 1024;
__global__ void __launch_bounds__(kPtPlanThreads) prompt_plan_kernel(const PromptArgs a, int ctas) {
  __shared__ int s_base[2048 + 1], s_sum[32], s_zeros[64], s_cost[kPtSpreadUnits];
  __shared__ int32_t s_order[kPtSpreadUnits], s_other[kPtSpreadUnits];
  grid_dependency_wait();
  grid_dependents_launch();
  const int units = pt_plan(a, PtPlanSpace{s_base, s_cost, s_sum, s_zeros, a.prefix, s_order, s_other}, true, ctas);
  if (threadIdx.x == 0) a.plan[0] = units;
  for (int b = threadIdx.x; units > 0 && b <= a.batch; b += kPtPlanThreads) a.base[b] = s_base[b];
  for (int u = threadIdx.x; (units & kPtSpread) && u < (units & (kPtSpread - 1)); u += kPtPlanThreads) a.order[u] = s_order[u];
}

// The unit inside which a CTA's range starts (id -1: it starts with one), for the merge.
struct alignas(16) PtCut {
  int id, lo, hi;  // of the unit, with its KV head; blocks before the CTA's part of it, and at its end
  int token0, tokens, g, pad[2];
};

// ---------------------------------------------------------------- bf16 forms

// A box of a tensor of rank 3 (x: dims, y: heads, z: tokens)
__device__ __forceinline__ void tma_box(void* dst, const void* map, int x, int y, int z, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// The warpgroup's registers from here on: a multiple of 8 a thread.  The four shares are 2 x 192 + 2 x 64, what the
// 512 threads were launched with (128).
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 1 / x to one unit in the last place, for x from 2^-126 to 2^126
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// a += the low half of w, b += the high half
__device__ __forceinline__ void add_bf16x2(float& a, float& b, uint32_t w) {
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n add.rn.f32.bf16 %0, lo, %0;\n add.rn.f32.bf16 %1, hi, %1;\n}"
      : "+f"(a), "+f"(b)
      : "r"(w));
}

// Lane q of four has piece i of lane i's afterwards where it had its own piece i: w[i] of lane q <-> w[q] of lane i
__device__ __forceinline__ void turn_pair(uint4& a, uint4& b, int bit) {  // (the lanes without the bit send b, the others a)
  const bool odd = threadIdx.x & bit;
  const uint4 give = odd ? a : b;
  uint4 got;
  got.x = __shfl_xor_sync(0xffffffffu, give.x, bit);
  got.y = __shfl_xor_sync(0xffffffffu, give.y, bit);
  got.z = __shfl_xor_sync(0xffffffffu, give.z, bit);
  got.w = __shfl_xor_sync(0xffffffffu, give.w, bit);
  if (odd)
    a = got;
  else
    b = got;
}
__device__ __forceinline__ void turn_quad(uint4 (&w)[4]) {
  turn_pair(w[0], w[1], 1);
  turn_pair(w[2], w[3], 1);
  turn_pair(w[0], w[2], 2);
  turn_pair(w[1], w[3], 2);
}

// The top bits of the halves of w that are infinities or NaN (exponent all ones; no half's sum carries)
__device__ __forceinline__ uint32_t bf16_special(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// What was taken out of V comes back to the rows that see its key: the infinities and NaN of the unit's keys that not
// every row sees, times the row's probability (an infinity is NaN where that is 0, as it is in a product), added to the
// row's outputs or its partial state by the threads that wrote these.  flags: the unit's, the top bit set in every other unit,
// by which the rows' M are found.  (More registers in here are spills in the caller: what is only needed for a value that
// comes back is computed from the arguments there.)
__device__ __noinline__ void pt_put_back(const PromptArgs& a, int flags, int lo, int hi, int token0, int tokens, int pos0,
                                         int key0, int g) {
#pragma unroll 1
  for (int pr = threadIdx.x & 127; pr < 2 * kPtRows; pr += 128) {
    const int Hg = a.heads_per_group, tt = kPtRows / Hg, row = (pr & (kPtRows - 1)) / Hg, h = (pr & (kPtRows - 1)) - row * Hg;
    const int t = row + (pr >= kPtRows ? tt : 0);
    if (row >= tt || t >= tokens) continue;
#pragma unroll 1
    for (int j = max(pos0 + 1, lo * kBlock); j <= min(pos0 + t, hi * kBlock - 1); ++j) {
      float p = -1.f;  // the row's probability of the key, once it is asked for
#pragma unroll 1
      for (int d = 0; d < kDim; ++d) {
        float y = __uint_as_float(static_cast<uint32_t>(a.v[(key0 + j) * a.v_stride + g * kDim + d]) << 16);
        if (fabsf(y) < INFINITY) continue;
        const int head = g * a.heads_per_group + h;
        if (p == -1.f) {
          const uint16_t *q = a.q + (token0 + t) * a.q_stride + head * kDim, *k = a.k + (key0 + j) * a.k_stride + g * kDim;
          float z = 0.f;
#pragma unroll 1
          for (int i = 0; i < kDim; ++i, ++q, ++k)
            z += __uint_as_float(static_cast<uint32_t>(*q) << 16) * __uint_as_float(static_cast<uint32_t>(*k) << 16);
          const float m = *static_cast<const volatile float*>(a.row_max + (2 * blockIdx.x + (flags < 0 ? 0 : 1)) * (2 * kPtRows) + pr);
          const float f = finite_factor(a.scale_log2);
          p = m == -INFINITY ? 0.f : ex2(fabsf(m) < kPtFused ? fmaf(z, f, -m) : __fmul_rn(z, f) - m);
        }
        y *= p;
        const int place = ((flags & 0x7FFFFFFF) >> kPtPlace) - 1;
        if (place < 0) {
          volatile uint16_t* dst = a.out + ((token0 + t) * static_cast<int64_t>(a.groups * a.heads_per_group) + head) * kDim + d;
          *dst = static_cast<uint16_t>(pack_bf16x2(__uint_as_float(static_cast<uint32_t>(*dst) << 16) + y, 0.f));
        } else {
          volatile float* dst = a.partial + (2 * static_cast<int64_t>(blockIdx.x) + place) * kPtPlaceFloats + (d / 4) * (8 * kPtRows) +
                                4 * pr + (d & 3);
          *dst += y;
        }
      }
    }
  }
}

// ---------------------------------------------------------------- the kernel

// kQuick: a call without a plan.  A kernel of its own, so that its code is not in the way of the longer calls (in one
// kernel they took 4 % more).
template <bool kQuick>
__global__ void __launch_bounds__(kPtThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptArgs a,
                                                                    const __grid_constant__ PromptMaps maps, int own_plan) {
  extern __shared__ __align__(1024) uint8_t q_tile[];
  uint8_t* k_ring = q_tile + 2 * kPtTile;
  uint8_t* v_ring = k_ring + kPtK * kPtTile;
  PtShared* sh = reinterpret_cast<PtShared*>(v_ring + kPtV * kPtTile);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hg = a.heads_per_group, G = a.groups, H = G * Hg, tt = kPtRows / Hg;

  if (tid == 0) {
    for (int i = 0; i < kPtK; ++i) {
      mbar_init(&sh->k_full[i], 1);
      mbar_init(&sh->k_empty[i], 1);
    }
    for (int i = 0; i < kPtV; ++i) {
      mbar_init(&sh->v_full[i], 1);
      mbar_init(&sh->v_edge[i], 1);
      mbar_init(&sh->v_ok[i], 4);
      mbar_init(&sh->v_empty[i], 1);
    }
    for (int i = 0; i < kPtItems; ++i) {
      mbar_init(&sh->item_full[i], 1);
      mbar_init(&sh->item_empty[i], 15);  // eight softmax warps, four of V, two issuers, the loader of V
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->s_full[i], 1);
      for (int h = 0; h < 2; ++h) mbar_init(&sh->p_full[i][h], 4);
      mbar_init(&sh->pv_done[i], 1);
      mbar_init(&sh->q_full[i], 1);
      mbar_init(&sh->q_empty[i], 1);
      mbar_init(&sh->fin[i], 4);
      mbar_init(&sh->o_full[i], 1);
      mbar_init(&sh->o_empty[i], 4);
      mbar_init(&sh->drain[i], 1);
    }
    mbar_init(&sh->other, 4);
    fence_mbar_init();
  }
  if (tid < 32) sh->special[tid >> 2][tid & 3] = -1;
  // rows of a tile behind its tokens (Hg does not divide 128): no copy writes them
  if (tt * Hg < kPtRows && tid < 2 * (kPtRows - tt * Hg) * 16) {
    const int i = tid / 16, t = i & 1, r = tt * Hg + (i >> 1), c = tid & 15;
    *reinterpret_cast<uint4*>(q_tile + t * kPtTile + (c >> 3) * kPtHalf + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == 12 && lane < 3) {
    const CUtensorMap* m = lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh->tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  grid_dependency_wait();
  grid_dependents_launch();
  // the plan, in what will be the stages of K
  PtOwnPlan& own = *reinterpret_cast<PtOwnPlan*>(k_ring);
  int units = 0;
  if (!kQuick && own_plan) {
    units = pt_own_plan(a, own);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  bool failed = false;

  // The next record, for a whole warp; `n` counts records.
  auto take_item = [&](int n, PtItem& it) -> bool {
    if (!pt_wait_warp(&sh->item_full[n % kPtItems], (n / kPtItems) & 1)) return false;
    it = sh->item[n % kPtItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->item_empty[n % kPtItems]);
    return true;
  };

  if (warp < 8) {
    registers_up<192>();
    // ---- softmax of slot `slot`: row r of its tile
    const int slot = warp >> 2, r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + slot * 128 + lane_base, tO = tmem + kPtO + slot * 128 + lane_base;
    const float f = finite_factor(a.scale_log2);
    const int my_token = r / Hg, my_head = r - my_token * Hg;
    int done = 0, live = 0;                        // steps of this slot, units with keys so far
    bool shared_par = false;
    float M = -INFINITY, l = 0.f, l_bf16 = 0.f;    // (l_bf16: of P as it is multiplied)
    float fused = -INFINITY;                       // M, but -inf in rows whose e is rounded first (kPtFused)
    int pos = 0;

    for (int n = 0;; ++n) {
      PtItem it;
      if (!take_item(n, it)) {
        failed = true;
        break;
      }
      if (it.flags & kPtEnd) break;
      if (it.lo >= it.hi) continue;
      const bool two = it.flags & kPtTwo;
      M = fused = -INFINITY;
      l = l_bf16 = 0.f;
      pos = it.pos0 + min(min(my_token, tt - 1) + (two && slot ? tt : 0), it.tokens - 1);
      // with one tile the blocks alternate between the slots
      const int step = two ? 1 : 2, first = it.lo + (two ? 0 : slot);
      const int tile0 = it.pos0 + (two && slot ? tt : 0);  // position of the tile's first row
#pragma unroll 1
      for (int p = first; p < it.hi; p += step) {
        if (!pt_wait_warp(&sh->s_full[slot], done & 1)) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (__builtin_expect(p * kBlock + kBlock - 1 > tile0, 0)) {
          // some row of the tile must not see one of these keys: -inf over its scores, where they lie (a short loop: code that
          // a unit runs once costs its instruction fetches)
          const int vis = pos - p * kBlock + 1;  // visible columns
#pragma unroll 1
          for (int c = max(__reduce_min_sync(0xffffffffu, vis), 0) >> 5; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32(tS + 32 * c, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = 32 * c + j < vis ? x[j] : 0xff800000u;
            tmem_st16(tS + 32 * c, x);
            tmem_st16(tS + 32 * c + 16, x + 16);
          }
          tmem_wait_st();
        }
        uint32_t v[2][64];
        float mx, mx1;
        tmem_ld64_max(tS, v[0], mx);
        tmem_ld64_max(tS + 64, v[1], mx1);
        tmem_wait_ld(v[0]);
        tmem_wait_ld(v[1]);
        asm volatile("" : "+f"(mx), "+f"(mx1));
        mx = fmaxf(mx, mx1);
        mx *= f;
        if (__builtin_expect(__any_sync(0xffffffffu, mx > fused), 0)) {
          float alpha = 1.f;
          if (mx > M) {
            const bool large = !(fabsf(mx) < kPtFused);
            const float mn = large ? mx : ceilf(mx) + kPtRefSet;
            alpha = ex2(M - mn);
            M = mn;
            fused = large ? -INFINITY : mn;
            l *= alpha;
            l_bf16 *= alpha;
          }
          if (p > first) {  // O as the products so far leave it, rescaled
            if (!pt_wait_warp(&sh->pv_done[slot], (done - 1) & 1)) {
              failed = true;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t y[16];
              tmem_ld16(tO + 16 * c, y);
              tmem_wait_ld(y);
#pragma unroll
              for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * alpha);
              tmem_st16(tO + 16 * c, y);
            }
          }
          if (__builtin_expect(__any_sync(0xffffffffu, fused != M), 0)) {  // in those rows (e - M) / f in the place of S
            float rf;
            asm("rcp.approx.f32 %0, %1;" : "=f"(rf) : "f"(f));  // (f may be above 2^126)
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t x[16];
              tmem_ld16(tS + 16 * c, x);
              tmem_wait_ld(x);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float e = __fmul_rn(__uint_as_float(x[j]), f);
                x[j] = fused != M ? __float_as_uint((e - M) * rf) : x[j];
              }
              tmem_st16(tS + 16 * c, x);
            }
            tmem_wait_st();
            tmem_ld64(tS, v[0]);
            tmem_ld64(tS + 64, v[1]);
            tmem_wait_ld(v[0]);
            tmem_wait_ld(v[1]);
          }
        }
        // P goes over the first 32 columns of each half of S
        const float c0 = fused == -INFINITY ? 0.f : -fused;
        const float2 ff = make_float2(f, f), cc = make_float2(c0, c0);
        float2 sum = make_float2(0.f, 0.f);
        float sum_bf16[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int k = 32 * i + 2 * j;
              const float2 x = fma2(make_float2(__uint_as_float(v[h][k]), __uint_as_float(v[h][k + 1])), ff, cc);
              const float2 y = make_float2(ex2(x.x), ex2(x.y));
              sum = add2(sum, y);
              pk[j] = pack_bf16x2(y.x, y.y);
              add_bf16x2(sum_bf16[2 * (j & 1)], sum_bf16[2 * (j & 1) + 1], pk[j]);
            }
            tmem_st16(tS + 64 * h + 16 * i, pk);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->p_full[slot][h]);
        }
        ++done;
        l += sum.x + sum.y;
        l_bf16 += (sum_bf16[0] + sum_bf16[1]) + (sum_bf16[2] + sum_bf16[3]);
      }
      // what is left to the V warps, who write the rows: the factors of O.  They have read the last unit's.
      if (failed || (live > 0 && !pt_wait_warp(&sh->o_empty[slot], (live - 1) & 1))) {
        failed = true;
        break;
      }
      ++live;
      // O is put right by the ratio of the sums of P before and after its rounding
      float fa = l_bf16 != 0.f ? l * rcp(l_bf16) : 1.f;
      if (!two) {  // slot 0 adds both slots' states
        if (slot == 1) {
          sh->other_m[r] = M;
          sh->other_l[r] = l;
          sh->factor[1][r] = fa;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh->other);
            mbar_arrive(&sh->fin[1]);
          }
          continue;
        }
        if (!pt_wait_warp(&sh->other, shared_par)) {
          failed = true;
          break;
        }
        shared_par = !shared_par;
      }
      const int place = kQuick ? -1 : (it.flags >> kPtPlace) - 1;
      float fb = 0.f;
      if (!two) {
        const float mo = sh->other_m[r], lo = sh->other_l[r];
        const float mn = fmaxf(M, mo);
        const float wa = mn == -INFINITY ? 1.f : ex2(M - mn), wb = mn == -INFINITY ? 1.f : ex2(mo - mn);
        fa *= wa;
        fb = wb * sh->factor[1][r];
        l = l * wa + lo * wb;
        M = mn;
      }
      const float inv = place >= 0 ? 1.f : l != 0.f ? rcp(l) : 0.f;  // (NaN counts as a sum)
      sh->factor[slot][r] = fa * inv;
      if (!two) sh->factor[1][r] = fb * inv;
      const int t = my_token + (two && slot ? tt : 0);               // token of the unit
      const int pr = r + (two && slot ? kPtRows : 0);                // row of the unit
      a.row_max[(2 * blockIdx.x + (live & 1)) * (2 * kPtRows) + pr] = M;
      if (my_token < tt && t < it.tokens) {
        if (place >= 0) {
          float* part = a.partial + (2 * static_cast<int64_t>(blockIdx.x) + place) * kPtPlaceFloats + 2 * kPtRows * kDim;
          part[pr] = M;
          part[2 * kPtRows + pr] = l;
        } else if (a.lse != nullptr) {
          a.lse[static_cast<int64_t>(it.token0 + t) * H + it.g * Hg + my_head] = fp8_lse(M, l);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->fin[slot]);
    }
  } else if (warp < 12) {
    registers_down<64>();
    // ---- V: infinities and NaN out of the rows that not every row of the unit sees
    // and the rows of a unit when its products are done
    const int ct = tid - 256, my_token = ct / Hg, my_head = ct - my_token * Hg;
    int blocks = 0, edges = 0, full0 = 0, full1 = 0;  // blocks, edge blocks, units with products in slot 0 and 1
    // Unit n of those with keys: row ct of both tiles.
    auto write = [&](int n, const PtItem& it) -> bool {
      const bool two = it.flags & kPtTwo, both = !two && it.lo + 1 < it.hi;  // (one tile: slot 1 has blocks as well)
      const int place = kQuick ? -1 : (it.flags >> kPtPlace) - 1;
      float* part = a.partial + (2 * static_cast<int64_t>(blockIdx.x) + max(place, 0)) * kPtPlaceFloats;
      const uint32_t tO = tmem + kPtO + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      // with one tile slot 0 has the sum's factors, and all is done with it
      if (!pt_wait_warp(&sh->fin[0], n & 1) || !pt_wait_warp(&sh->o_full[0], full0 & 1)) return false;
      ++full0;
      if (!two && !pt_wait_warp(&sh->fin[1], n & 1)) return false;
      if (both && !pt_wait_warp(&sh->o_full[1], full1 & 1)) return false;
      if (both) ++full1;
#pragma unroll 1
      for (int s = 0; s < (two ? 2 : 1); ++s) {
        if (s == 1) {
          if (!pt_wait_warp(&sh->fin[1], n & 1) || !pt_wait_warp(&sh->o_full[1], full1 & 1)) return false;
          ++full1;
        }
        tc_fence_after();
        float fa = sh->factor[s][ct]; const float fb = sh->factor[1][ct];
        const bool valid = my_token < tt && my_token + s * tt < it.tokens;
        if (both) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t x[16], y[16];
            tmem_ld16(tO + 16 * c, x);
            tmem_ld16(tO + 128 + 16 * c, y);
            tmem_wait_ld(x);
            tmem_wait_ld(y);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(fmaf(__uint_as_float(y[i]), fb, __uint_as_float(x[i]) * fa));
            tmem_st16(tO + 16 * c, x);
          }
          tmem_wait_st();
          fa = 1.f;
        }
        if (place < 0) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32(tO + s * 128 + 32 * c, x);
            tmem_wait_ld(x);
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t* p = reinterpret_cast<uint32_t*>(&w[j]);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                p[i] = pack_bf16x2(__uint_as_float(x[8 * j + 2 * i]) * fa, __uint_as_float(x[8 * j + 2 * i + 1]) * fa);
            }
            turn_quad(w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int to = __shfl_sync(0xffffffffu, valid ? my_token * H + my_head : -1, (lane & ~3) + i);
              if (to >= 0)
                *reinterpret_cast<uint4*>(a.out + ((static_cast<int64_t>(it.token0) + s * tt) * H + it.g * Hg + to) * kDim + 32 * c +
                                          8 * (lane & 3)) = w[i];
            }
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t x[16];
            tmem_ld16(tO + s * 128 + 16 * c, x);
            tmem_wait_ld(x);
            float4* to = reinterpret_cast<float4*>(part) + 4 * c * (2 * kPtRows) + ct + s * kPtRows;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (valid) to[j * 2 * kPtRows] = make_float4(__uint_as_float(x[4 * j]) * fa, __uint_as_float(x[4 * j + 1]) * fa, __uint_as_float(x[4 * j + 2]) * fa, __uint_as_float(x[4 * j + 3]) * fa);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh->o_empty[s]);
          if (!two) mbar_arrive(&sh->o_empty[1]);
        }
      }
      // what the other V warps found in the unit's V: they have been through its last edge block
      if (edges > 0 && !pt_wait_warp(&sh->v_ok[(edges - 1) % kPtV], ((edges - 1) / kPtV) & 1)) return false;
      const int* sp = sh->special[n & 7];
      if (sp[0] == n || sp[1] == n || sp[2] == n || sp[3] == n)
        pt_put_back(a, it.flags | (n & 1 ? INT_MIN : 0), it.lo, it.hi, it.token0, it.tokens, it.pos0, it.key0, it.g);
      return true;
    };
    PtItem before{};  // the last unit with keys, not written yet
    int live = 0;     // units with keys so far
    for (int n = 0; !failed; ++n) {
      PtItem it;
      if (!take_item(n, it)) {
        failed = true;
        break;
      }
      if (!(it.flags & kPtEnd) && it.lo >= it.hi) {  // no row has a key
        for (int t = my_token; my_token < tt && t < it.tokens; t += tt) {
          const int64_t row = static_cast<int64_t>(it.token0 + t) * H + it.g * Hg + my_head;
          for (int c = 0; c < kDim / 8; ++c) reinterpret_cast<uint4*>(a.out + row * kDim)[c] = make_uint4(0, 0, 0, 0);
          if (a.lse != nullptr) a.lse[row] = -INFINITY;
        }
        continue;
      }
      // A short unit's V is looked through before the last unit's rows are written, so that its products find it done (64 prompts
      // of up to 100 tokens 34 -> 30 us).  In longer units the V of blocks from the kPtV-th on may lie in stages that only
      // products behind that writing make free.
#pragma unroll 1
      for (int p = it.edge(), state = it.hi - it.lo <= kPtV ? 1 : 0; ; ++p, ++edges) {
        // state 0: the last unit's rows are to be written now; 1: behind this unit's blocks; 2: they are written
        if (state == 0 || p >= it.hi) {
          if (state < 2 && live > 0 && !write(live - 1, before)) {
            failed = true;
            break;
          }
          state = 2;
          if (p >= it.hi) break;
        }
        const int vs = (blocks + p - it.lo) % kPtV;
        if (!pt_wait_warp(&sh->v_edge[edges % kPtV], (edges / kPtV) & 1)) {
          failed = true;
          break;
        }
        const int r0 = max(it.pos0 + 1 - p * kBlock, 0);  // first row to look at
        uint8_t* stage = v_ring + vs * kPtTile + (ct & 7) * 16;
        uint32_t any = 0u;
#pragma unroll 2
        for (int r = (r0 & ~15) + (ct >> 3); r < kBlock; r += 16) {
          const uint4 x = lds128(stage + r * 128), y = lds128(stage + kPtHalf + r * 128);
          const uint32_t s = bf16_special(x.x) | bf16_special(x.y) | bf16_special(x.z) | bf16_special(x.w) | bf16_special(y.x) |
                             bf16_special(y.y) | bf16_special(y.z) | bf16_special(y.w);
          any |= r >= r0 ? s : 0u;
        }
        if (any != 0u) {
          sh->special[live & 7][warp - 8] = live;
          auto clear = [](uint32_t w) {
            const uint32_t s = bf16_special(w);
            return w & ~(s | (s - (s >> 15)));  // (whole halves: the top bit and the 15 below it)
          };
#pragma unroll 1
          for (int r = (r0 & ~15) + (ct >> 3); r < kBlock; r += 16) {
            if (r < r0) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint8_t* at = stage + half * kPtHalf + r * 128;
              const uint4 x = lds128(at);
              *reinterpret_cast<uint4*>(at) = make_uint4(clear(x.x), clear(x.y), clear(x.z), clear(x.w));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->v_ok[edges % kPtV]);
      }
      if (failed || (it.flags & kPtEnd)) break;
      blocks += it.hi - it.lo;
      before = it;
      ++live;
    }
  } else {
   registers_down<64>();
   if (warp == 12) {
    // ---- producer: units and the copies of Q and K
    int base0 = 0, base1 = 0;  // kQuick: units of the sequences before sequence lane and 32 + lane
    if (kQuick) {
      bool bad = false;
      int x[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int s = 32 * j + lane;
        x[j] = 0;
        if (s < a.batch) {
          const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
          bad |= q0 < 0 || k0 < 0 || q1 < q0 || k1 < k0 || q1 > a.q_tokens || k1 > a.k_tokens;
          x[j] = (q1 - q0 + 2 * tt - 1) / (2 * tt);
        }
      }
      base0 = x[0], base1 = x[1];
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int y0 = __shfl_up_sync(0xffffffffu, base0, s), y1 = __shfl_up_sync(0xffffffffu, base1, s);
        if (lane >= s) base0 += y0, base1 += y1;
      }
      const int all0 = __shfl_sync(0xffffffffu, base0, 31);
      units = all0 + __shfl_sync(0xffffffffu, base1, 31);
      base0 -= x[0];
      base1 += all0 - x[1];
      if (__any_sync(0xffffffffu, bad)) {  // nothing is done
        if (blockIdx.x == 0 && lane == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
        units = 0;
      }
    } else if (!own_plan) {
      units = a.plan[0];
    }
    const int* base = own_plan ? own.base : a.base;
    const int32_t *prefix = own_plan ? own.prefix : a.prefix, *order = own_plan ? own.order : a.order;
    const bool spread = !kQuick && units & kPtSpread;
    if (!kQuick) units &= kPtSpread - 1;
    int x0 = 0, x1 = 0, u = 0, b = 0, i = 0, dealt = 0;  // dealt: units of this CTA where they stay whole
    int64_t E = 0, first = 0;                            // all cost, cost before unit u
    int2* mine = a.dealt + blockIdx.x * kPtMaxDealt;
    if (spread) {  // (looked up before the copies of K go over the plan)
      const FtDiv by_g(G);
      const int all = units * G, whole = all / gridDim.x;
      dealt = whole + (pt_dealt(whole, blockIdx.x, gridDim.x) < all ? 1 : 0);
      for (int k = lane; k < dealt; k += 32) {
        const int at = pt_dealt(k, blockIdx.x, gridDim.x), unit = order[by_g(at)];
        int s = 0, left = a.batch;  // the last sequence with base <= unit
        while (left > 1) {
          const int h = left / 2;
          if (base[s + h] <= unit) {
            s += h;
            left -= h;
          } else {
            left = h;
          }
        }
        mine[k] = make_int2(s | (at - by_g(at) * G) << 16, unit - base[s]);
      }
    } else if (!kQuick && units > 0) {
      E = static_cast<int64_t>(prefix[units]) * G;
      const int n = gridDim.x, share = static_cast<int>(E) / n, rest = static_cast<int>(E) - share * n;
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        x0 = x1;
        const int c = blockIdx.x + k;  // (E c / n in 32 bits)
        x1 = share * c + rest * c / n;
        if (c > 0 && x1 < E) x1 = ft_cut_inside(prefix, units, G, x1, kPtWhole);
      }
      u = ft_find(prefix, units, G, static_cast<int>(min(static_cast<int64_t>(x0), E - 1)));
      b = ft_find(base, a.batch, 1, u);
      i = u - base[b];
      first = static_cast<int64_t>(prefix[u]) * G;
    }
    __syncwarp();  // (lane 0's copies go over the plan that all lanes have read, and all read what others left in `mine`)
    const uint64_t keep = l2_evict_normal_policy(), once = l2_evict_first_policy();
    const uint32_t q_bytes = static_cast<uint32_t>(tt) * Hg * 256;
    int n = 0, blocks = 0, tiles0 = 0, tiles1 = 0;  // units, blocks, units that used tile 0 and tile 1
    auto record = [&](const PtItem& it) -> bool {
      if (n >= kPtItems && !pt_wait_warp(&sh->item_empty[n % kPtItems], (n / kPtItems - 1) & 1)) return false;
      if (lane == 0) {
        sh->item[n % kPtItems] = it;
        mbar_arrive(&sh->item_full[n % kPtItems]);
      }
      ++n;
      return true;
    };
    PtCut cut{-1, 0, 0, 0, 0, 0, {0, 0}};
    // kQuick: a prompt's units cost more and more, so the last ones come first; the CTAs that start first get the units of
    // one round, or the second units of more
    const int c = units * G > static_cast<int>(gridDim.x) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    for (int k = 0; !failed && (kQuick ? pt_dealt(k, c, gridDim.x) < units * G
                                       : spread ? k < dealt : units > 0 && first <= x1); ++k) {  // unit i of sequence b
      int g = 0, g_end = G;
      if (kQuick) {
        const int at = units * G - 1 - pt_dealt(k, c, gridDim.x), unit = FtDiv(G)(at);
        b = __popc(__ballot_sync(0xffffffffu, base0 <= unit)) - 1;
        if (b == 31) b += __popc(__ballot_sync(0xffffffffu, base1 <= unit));
        i = unit - __shfl_sync(0xffffffffu, b < 32 ? base0 : base1, b & 31);
        g = at - unit * G;
        g_end = g + 1;
      } else if (spread) {
        const int2 x = __ldcg(mine + k);
        b = x.x & 0xFFFF;
        g = x.x >> 16;
        g_end = g + 1;
        i = x.y;
      }
      const int q0 = a.cu_q[b], key0 = a.cu_k[b], Lq = a.cu_q[b + 1] - q0;
      const PtUnit t = pt_unit(Lq, a.cu_k[b + 1] - key0, i, tt);
      const int pages = max(t.pages, 1), cost = t.cost(), token0 = q0 + i * 2 * tt;
#pragma unroll 1
      for (; g < g_end && !failed; ++g) {
        int lo = 0, hi = pages;
        if (!kQuick && !spread) {
          const int64_t u0 = first + static_cast<int64_t>(g) * cost;
          if (u0 + cost <= x0) continue;
          lo = t.block_at(x0 - u0), hi = t.block_at(x1 - u0);
          if (u0 < x0 && x0 < E) cut = PtCut{u * G + g, lo, hi, token0, t.tokens, g, {0, 0}};
          if (u0 >= x1) break;
          if (lo >= hi) continue;
        }
        const int place = lo == 0 && hi == pages ? -1 : lo == 0 ? 1 : 0;
        if (!record(PtItem{(t.width == 2 ? kPtTwo : 0) | (place + 1) << kPtPlace, lo, t.pages > 0 ? hi : lo, token0, t.tokens,
                           t.pos0, key0, g})) {
          failed = true;
          break;
        }
        if (t.pages == 0) continue;
#pragma unroll 1
        for (int k = 0; k < t.width && !failed; ++k) {  // the unit's queries
          int& used = k ? tiles1 : tiles0;
          if (used > 0 && !pt_wait_warp(&sh->q_empty[k], (used - 1) & 1)) {
            failed = true;
            break;
          }
          ++used;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sh->q_full[k], q_bytes);
            tma_box(q_tile + k * kPtTile, &maps.q, 0, g * Hg, token0 + k * tt, &sh->q_full[k], once);
            tma_box(q_tile + k * kPtTile + kPtHalf, &maps.q, 64, g * Hg, token0 + k * tt, &sh->q_full[k], once);
          }
        }
#pragma unroll 1
        for (int p = lo; p < hi && !failed; ++p) {
          const int ks = blocks % kPtK;
          if (blocks >= kPtK && !pt_wait_warp(&sh->k_empty[ks], (blocks / kPtK - 1) & 1)) {
            failed = true;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&sh->k_full[ks], kPtTile);
            tma_box(k_ring + ks * kPtTile, &maps.k, 0, g, key0 + p * kBlock, &sh->k_full[ks], keep);
            tma_box(k_ring + ks * kPtTile + kPtHalf, &maps.k, 64, g, key0 + p * kBlock, &sh->k_full[ks], keep);
          }
          ++blocks;
        }
      }
      if (kQuick || spread) continue;
      // the next unit: of this sequence, or the first one of the next sequence that has any
      first += static_cast<int64_t>(cost) * G;
      if (++u >= units) break;
      if (++i * 2 * tt >= Lq) {
        i = 0;
        do ++b;
        while (a.cu_q[b + 1] == a.cu_q[b]);
      }
    }
    if (!kQuick && lane == 0) a.cuts[blockIdx.x] = cut;
    if (!failed) failed = !record(PtItem{kPtEnd, 0, 0, 0, 0, 0, 0, 0});
    if (failed) {
      // wait (bounded) for the copies still in flight
#pragma unroll 1
      for (int k = max(0, blocks - kPtK); k < blocks; ++k) pt_wait(&sh->k_full[k % kPtK], (k / kPtK) & 1);
      if (tiles0 > 0) pt_wait(&sh->q_full[0], (tiles0 - 1) & 1);
      if (tiles1 > 0) pt_wait(&sh->q_full[1], (tiles1 - 1) & 1);
    }
   } else if (warp == 15) {
    // ---- the copies of V
    const uint64_t keep = l2_evict_normal_policy();
    int blocks = 0, plain = 0, edges = 0;
    for (int uc = 0; !failed; ++uc) {
      PtItem it;
      if (!take_item(uc, it)) {
        failed = true;
        break;
      }
      if (it.flags & kPtEnd) break;
      const int edge = it.edge();
#pragma unroll 1
      for (int p = it.lo; p < it.hi; ++p) {
        const int vs = blocks % kPtV;
        if (blocks >= kPtV && !pt_wait_warp(&sh->v_empty[vs], (blocks / kPtV - 1) & 1)) {
          failed = true;
          break;
        }
        if (lane == 0) {
          fence_proxy_async_smem();  // the V warps' stores to the stage are before the copy
          uint64_t* bar = p < edge ? &sh->v_full[plain % kPtV] : &sh->v_edge[edges % kPtV];
          mbar_arrive_expect_tx(bar, kPtTile);
          tma_box(v_ring + vs * kPtTile, &maps.v, 0, it.g, it.key0 + p * kBlock, bar, keep);
          tma_box(v_ring + vs * kPtTile + kPtHalf, &maps.v, 64, it.g, it.key0 + p * kBlock, bar, keep);
        }
        ++blocks;
        p < edge ? ++plain : ++edges;
      }
    }
    if (failed) {  // wait (bounded) for the copies still in flight
#pragma unroll 1
      for (int k = max(0, plain - kPtV); k < plain; ++k) pt_wait(&sh->v_full[k % kPtV], (k / kPtV) & 1);
#pragma unroll 1
      for (int k = max(0, edges - kPtV); k < edges; ++k) pt_wait(&sh->v_edge[k % kPtV], (k / kPtV) & 1);
    }
   } else {
    // ---- product issuers: warp 13 S, warp 14 P V.  Two warps, because issuing blocks while the tensor
    // pipe is full: each waits for its operands while the other's products run.
    const bool scores = warp == 13;
    if (elect_one()) {
      constexpr uint32_t kBf16 = 1u << 7 | 1u << 10;  // A and B
      const uint32_t id_s = umma_idesc_f16(kPtRows, kBlock) | kBf16;
      const uint32_t id_o = umma_idesc_f16(kPtRows, kDim) | kBf16 | 1u << 16;  // B MN-major
      const uint32_t qb = smem_u32(q_tile), kb = smem_u32(k_ring), vb = smem_u32(v_ring);
      int blocks = 0, done0 = 0, done1 = 0;             // blocks, steps of the slots so far
      int plain = 0, edges = 0;                         // blocks of the two kinds in the units before
      int live = 0;                                     // units with keys before
      int tiles1 = 0, tiles0 = 0;                       // units that used tile 1 and tile 0
      bool bad = false;
      for (int n = 0; !bad; ++n) {
        if (!pt_wait(&sh->item_full[n % kPtItems], (n / kPtItems) & 1)) {
          bad = true;
          break;
        }
        const PtItem it = sh->item[n % kPtItems];
        mbar_arrive(&sh->item_empty[n % kPtItems]);
        if (it.flags & kPtEnd) break;
        if (it.lo >= it.hi) continue;
        const int width = it.flags & kPtTwo ? 2 : 1, edge = it.edge();
        ++tiles0;
        if (width == 2) ++tiles1;
        bool read0 = live == 0, read1 = live == 0;  // the last unit's O of slot 0 and 1 is known to be read
#pragma unroll 1
        for (int p = it.lo; p < it.hi && !bad; ++p, ++blocks) {
          const int ks = blocks % kPtK, vs = blocks % kPtV;
          const int k = p < edge ? plain + p - it.lo : edges + p - edge;
          if (scores ? !pt_wait(&sh->k_full[ks], (blocks / kPtK) & 1)
                     : !pt_wait(p < edge ? &sh->v_full[k % kPtV] : &sh->v_ok[k % kPtV], (k / kPtV) & 1)) {
            bad = true;
            break;
          }
  #pragma unroll 1
        for (int i = 0; i < width && !bad; ++i) {
            const int s = width == 2 ? i : (p - it.lo) & 1;
            const int d = s ? done1 : done0;
            const bool last = i == width - 1;
            if (scores) {
              // S overwrites the slot's P: it waits until that has been multiplied
              if ((p == it.lo && !pt_wait(&sh->q_full[i], ((i ? tiles1 : tiles0) - 1) & 1)) ||
                  (d > 0 && !pt_wait(&sh->pv_done[s], (d - 1) & 1))) {
                bad = true;
                break;
              }
              tc_fence_after();
              const uint64_t qd = umma_desc(qb + i * kPtTile), kd = umma_desc(kb + ks * kPtTile);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {  // 16 dims a step
                const uint32_t off = (kk >> 2) * kPtHalf + 32 * (kk & 3);
                umma_f16(tmem + s * 128, qd + (off >> 4), kd + (off >> 4), id_s, kk > 0 ? 1u : 0u);
              }
              umma_commit(&sh->s_full[s]);
              if (p == it.hi - 1) umma_commit(&sh->q_empty[i]);
              if (last) umma_commit(&sh->k_empty[ks]);
            } else {
              const bool first = p < it.lo + 2 && (width == 2 ? p == it.lo : true);  // of the slot in this unit
              const bool final = width == 2 ? p == it.hi - 1 : p >= it.hi - 2;
              // a slot's O is overwritten when the last unit's has been read; both are asked for before the unit's last
              // product, so that no phase of o_empty is missed
              const bool end = last && p == it.hi - 1;
              if ((first && s == 0 || end) && !read0) read0 = pt_wait(&sh->o_empty[0], (live - 1) & 1), bad |= !read0;
              if ((first && s == 1 || end) && !read1) read1 = pt_wait(&sh->o_empty[1], (live - 1) & 1), bad |= !read1;
              if (bad) break;
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {  // 64 keys: the products of the first half run beside the softmax of the second
                if (!pt_wait(&sh->p_full[s][h], d & 1)) {
                  bad = true;
                  break;
                }
                tc_fence_after();
                const uint64_t vd = umma_desc_mn(vb + vs * kPtTile + h * 64 * 128, kPtHalf);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // 16 keys: 8 TMEM columns of P, two 8-row groups of V
                  umma_f16_tmem_a(tmem + kPtO + s * 128, tmem + s * 128 + h * 64 + 8 * kk, vd + ((kk * 2048) >> 4), id_o,
                                  !first || h > 0 || kk > 0 ? 1u : 0u);
                if (h == 1) umma_commit(&sh->pv_done[s]);
                if (final && h == 1) umma_commit(&sh->o_full[s]);
                if (last && h == 1) umma_commit(&sh->v_empty[vs]);
              }
            }
            s ? ++done1 : ++done0;
          }
        }
        plain += edge - it.lo;
        edges += it.hi - edge;
        ++live;
      }
      if (bad) {  // the products still running end before TMEM is freed
        flag_error(a.err, MSA_DEVERR_TIMEOUT);
        umma_commit(&sh->drain[scores]);
        pt_wait(&sh->drain[scores], 0);
      }
    }
    __syncwarp();
   }
  }
  if (failed && lane == 0) flag_error(a.err, MSA_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------- units cut by range boundaries

// The partial states that their CTAs left, added.  blockIdx.x: the unit, by its place among those that are cut or, where as
// many units can be cut as there are CTAs, by the first CTA that starts inside it (the others' blocks find nothing to do).
// blockIdx.y: the row (kSplit, for many parts a unit: fp8_merge.cuh) or every gridDim.y-th group of 16 of the unit's
// `rows`.  A thread has four dims of a row, without kSplit of two rows, whose loads of two parts go out together (40 MB of
// states, 151 cuts, take 10 us; a row at a time they took 18).
template <bool kSplit>
__global__ void __launch_bounds__(kFp8MergeThreads, kSplit ? 1 : 4) prompt_merge_kernel(const PromptArgs a, int ctas, int rows) {
  __shared__ Fp8MergeShared sh;
  grid_dependency_wait();
  grid_dependents_launch();
  const int G = a.groups, Hg = a.heads_per_group, tt = kPtRows / Hg, lane = threadIdx.x & 31;
  int c = blockIdx.x + 1;
  if (static_cast<int>(gridDim.x) < ctas - 1) {  // (every warp)
    int ids[kFp8MaxCtas / 32];
#pragma unroll
    for (int i = 0; i < kFp8MaxCtas / 32; ++i) ids[i] = 32 * i + lane < ctas ? a.cuts[32 * i + lane].id : -1;
    int before = 0, last = -1;
    c = -1;
#pragma unroll
    for (int i = 0; i < kFp8MaxCtas / 32; ++i) {
      const int up = __shfl_up_sync(0xffffffffu, ids[i], 1);
      const bool starts = ids[i] >= 0 && ids[i] != (lane == 0 ? last : up);
      const unsigned m = __ballot_sync(0xffffffffu, starts);
      const bool it = starts && before + __popc(m & ((1u << lane) - 1u)) == static_cast<int>(blockIdx.x);
      const unsigned mine = __ballot_sync(0xffffffffu, it);
      if (mine != 0) c = 32 * i + __ffs(mine) - 1;
      before += __popc(m);
      last = __shfl_sync(0xffffffffu, ids[i], 31);
    }
    if (c < 0) return;
  }
  // every warp: the CTA before and those from c on, a lane each
  const PtCut none{-1, 0, 0, 0, 0, 0, {0, 0}};
  PtCut x = c - 1 + lane < ctas ? a.cuts[c - 1 + lane] : none;
  const int id = __shfl_sync(0xffffffffu, x.id, 1), lo = __shfl_sync(0xffffffffu, x.lo, 1);
  const int token0 = __shfl_sync(0xffffffffu, x.token0, 1), tokens = __shfl_sync(0xffffffffu, x.tokens, 1);
  const int g = __shfl_sync(0xffffffffu, x.g, 1);
  if (id < 0 || __shfl_sync(0xffffffffu, x.id, 0) == id) return;
  if (threadIdx.x < 32) {  // the CTAs with blocks of the unit, in order
    int n = lo > 0;
    if (lane == 0) {
      if (lo > 0) sh.list[0] = 2 * (c - 1) + 1;
      x = none;
    }
    for (int c0 = c - 1;;) {
      const bool some = x.id == id && x.lo < x.hi;
      const unsigned m = __ballot_sync(0xffffffffu, some);
      if (some) sh.list[n + __popc(m & ((1u << lane) - 1u))] = 2 * (c0 + lane) + (x.lo == 0 ? 1 : 0);
      n += __popc(m);
      const int last = __shfl_sync(0xffffffffu, x.id, 31);
      if (last != id) break;
      c0 += 32;
      x = c0 + lane < ctas ? a.cuts[c0 + lane] : none;
    }
    if (lane == 0) sh.n = n;
  }
  __syncthreads();
  const int n = sh.n;
  if (n < 2) return;  // one CTA's: written by it
  const FtDiv by_hg(Hg);
  // a row's place among the outputs' rows, -1 where it is none of the unit's
  const int64_t hr0 = static_cast<int64_t>(token0) * G * Hg + g * Hg;
  auto place = [&](int row) -> int {
    const int r = row & (kPtRows - 1), token = by_hg(r), all = token + (row >= kPtRows ? tt : 0);
    return token < tt && all < tokens ? all * G * Hg + r - token * Hg : -1;
  };
  auto write = [&](int at, int chunk, const float4& o, float M, float l) {
    const float inv = l != 0.f ? rcp(l) : 0.f;
    reinterpret_cast<uint2*>(a.out + (hr0 + at) * kDim)[chunk] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (chunk == 0 && a.lse != nullptr) a.lse[hr0 + at] = fp8_lse(M, l);
  };
  if (kSplit) {
    const int pr = blockIdx.y;
    const int at = place(pr);
    if (at < 0) return;
    float4 o;
    float M, l;
    fp8_merge_row<true>(a.partial, 2 * kPtRows, pr, lane * 2 * kPtRows + pr, sh, o, M, l);
    if (threadIdx.x < 32) write(at, lane, o, M, l);
    return;
  }
  // states lie by chunks of four dims: eight rows of a chunk are one 128-byte line
  constexpr int kRows = 2, kParts = 2;
  const int chunk = threadIdx.x >> 3;
#pragma unroll 1
  for (int r = 8 * kRows * blockIdx.y; r < rows; r += 8 * kRows * gridDim.y) {
  const int row0 = r + (threadIdx.x & 7);
  float M[kRows], l[kRows];
  float4 o[kRows];
  int at[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    at[i] = place(row0 + 8 * i);
    M[i] = -INFINITY;
    l[i] = 0.f;
    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int k0 = 0; k0 < n; k0 += kParts) {
    float ms[kRows][kParts], ls[kRows][kParts];
    float4 os[kRows][kParts];
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const float* part = a.partial + static_cast<int64_t>(sh.list[min(k0 + k, n - 1)]) * kPtPlaceFloats;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const bool in = k0 + k < n && at[i] >= 0;
        ms[i][k] = in ? __ldcg(part + 2 * kPtRows * kDim + row0 + 8 * i) : -INFINITY;
        ls[i][k] = in ? __ldcg(part + 2 * kPtRows * (kDim + 1) + row0 + 8 * i) : 0.f;
        os[i][k] = in ? __ldcg(reinterpret_cast<const float4*>(part) + chunk * 2 * kPtRows + row0 + 8 * i)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float mb = M[i];
#pragma unroll
      for (int k = 0; k < kParts; ++k) mb = fmaxf(mb, ms[i][k]);
      // (no key so far: the sums hold zeros, or NaN)
      const float f = mb == -INFINITY ? 1.f : ex2(M[i] - mb);
      l[i] *= f;
      o[i] = make_float4(o[i].x * f, o[i].y * f, o[i].z * f, o[i].w * f);
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const float w = mb == -INFINITY ? 1.f : ex2(ms[i][k] - mb);
        l[i] += w * ls[i][k];
        o[i].x += w * os[i][k].x;
        o[i].y += w * os[i][k].y;
        o[i].z += w * os[i][k].z;
        o[i].w += w * os[i][k].w;
      }
      M[i] = mb;
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (at[i] >= 0) write(at[i], chunk, o[i], M[i], l[i]);
  }
}

// ---------------------------------------------------------------- launch

size_t prompt_dealt_bytes() { return kFp8MaxCtas * kPtMaxDealt * sizeof(int2); }
size_t prompt_cut_bytes() { return kFp8MaxCtas * sizeof(PtCut); }
size_t prompt_row_max_bytes() { return static_cast<size_t>(kFp8MaxCtas) * 4 * kPtRows * sizeof(float); }
size_t prompt_partial_bytes() { return static_cast<size_t>(2) * kFp8MaxCtas * kPtPlaceFloats * sizeof(float); }

static cudaError_t prompt_maps(const PromptArgs& a, PromptMaps* maps) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint32_t tt = static_cast<cuuint32_t>(prompt_tile_tokens(a.heads_per_group));
  const struct {
    CUtensorMap* map;
    const uint16_t* data;
    int64_t stride;
    int heads, tokens;
    cuuint32_t box_heads, box_tokens;
  } x[3] = {{&maps->q, a.q, a.q_stride, a.groups * a.heads_per_group, a.q_tokens, static_cast<cuuint32_t>(a.heads_per_group), tt},
            {&maps->k, a.k, a.k_stride, a.groups, a.k_tokens, 1, kBlock},
            {&maps->v, a.v, a.v_stride, a.groups, a.k_tokens, 1, kBlock}};
  for (const auto& t : x) {
    // (without keys nothing is copied: any address)
    const void* data = t.tokens > 0 ? t.data : a.q;
    const cuuint64_t dims[3] = {kDim, static_cast<cuuint64_t>(t.heads), static_cast<cuuint64_t>(t.tokens > 0 ? t.tokens : 1)};
    const cuuint64_t strides[2] = {kDim * 2, static_cast<cuuint64_t>(t.stride) * 2};
    const cuuint32_t box[3] = {64, t.box_heads, t.box_tokens}, estr[3] = {1, 1, 1};
    const CUresult r = encode(t.map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(data), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

cudaError_t launch_prompt_attn(const PromptArgs& a, int num_sms, cudaStream_t s) {
  PromptMaps maps;
  cudaError_t e = prompt_maps(a, &maps);
  if (e != cudaSuccess) return e;
  const int ctas = num_sms < kFp8MaxCtas ? num_sms : kFp8MaxCtas;
  const int64_t most = prompt_max_units(a.q_tokens, a.batch, a.heads_per_group), units = most * a.groups;
  const int64_t largest = 2 * ((static_cast<int64_t>(a.k_tokens) + kBlock - 1) / kBlock) + kPtUnitCost;  // cost of a unit
  const bool quick = pt_quick(a, largest, ctas);
  const int own_plan = a.batch <= kPtOwnBatch && most <= kPtOwnUnits ? 1 : 0;
  const auto kernel = quick ? prompt_attn_kernel<true> : prompt_attn_kernel<false>;
  if ((e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), kPtSmem)) != cudaSuccess) return e;
  if (!quick && !own_plan && (e = launch_dependent(prompt_plan_kernel, dim3(1), kPtPlanThreads, 0, s, a, ctas)) != cudaSuccess)
    return e;
  if ((e = launch_dependent(kernel, dim3(ctas), kPtThreads, kPtSmem, s, a, maps, own_plan)) != cudaSuccess) return e;
  if (ctas == 1 || quick || largest <= kPtWhole) return cudaSuccess;  // nothing can be cut
  // Units that may be cut (many: by CTA, which needs no search), and the rows of the largest: blocks that find nothing to
  // do are most of the time of a merge of few units (one token on 16K keys 57 us with 151 x 256 blocks, 23 with 4 x 32).
  const int cut = static_cast<int>(units < ctas / 2 ? units : ctas - 1), tt = prompt_tile_tokens(a.heads_per_group);
  const int rows = a.q_tokens <= tt ? static_cast<int>(a.q_tokens) * a.heads_per_group : 2 * kPtRows;
  if (ctas / units >= kFp8MergeSplitParts)
    return launch_dependent(prompt_merge_kernel<true>, dim3(cut, rows), kFp8MergeThreads, 0, s, a, ctas, rows);
  int y = 4 * num_sms / cut;  // one wave (588 tokens on 10K, 24 units: 45 -> 41 us)
  y = y < 1 ? 1 : y > (rows + 15) / 16 ? (rows + 15) / 16 : y;
  return launch_dependent(prompt_merge_kernel<false>, dim3(cut, y), kFp8MergeThreads, 0, s, a, ctas, rows);
}

}  // namespace msa
