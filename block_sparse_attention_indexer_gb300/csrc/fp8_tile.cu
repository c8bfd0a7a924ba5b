// Dense attention over the FP8 page cache for more than 16 query rows per (sequence, group):
// draft tokens and prompt chunks, on the tcgen05 tensor cores.
//
// Mathematics: as fp8_stream.cu has it, P_j = 2^(e_j - M) with e_j = z_j log2(e) + b (2^b the page's V scale)
// and an integer reference M that keeps P inside fp16's range (kFtRefSet below).
//
// Work.  A unit is 256 query rows (token, head) of a (sequence, group), as two tiles of 128, or the
// at most 128 rows of a last one, as one tile.  A unit's products are counted in (tile, page) steps;
// the units of the call, in order, are one flat list of steps that a persistent grid (one CTA an SM)
// cuts into equal ranges by the units' prefix sums (causal units differ in length), short units
// staying whole (ft_cut).  Two accumulator slots work in turn: with two tiles each page is used by
// slot 0 (tile 0) and slot 1 (tile 1), so a page is loaded and its V converted once for 256 rows;
// with one tile the pages alternate between the slots and the two states are added at the end.
//   * S = Q K^T: kind::f8f6f4, E4M3 from the page as it is (a tensor copy lands the 128-byte key rows
//     in the operand's 128-byte swizzle), exact products, float32 sums.  bf16 queries are split into
//     two parts, q = 2^k (hi + lo) with the row's largest value in [2^7, 2^8): hi is q 2^-k rounded to
//     E4M3, and the rest is at most 8 units of bf16's last place, which E5M2's three significant bits hold
//     exactly for values of at least 2^-6 (2^-13 of the largest); below, it is rounded by at most 2^-14.
//   * O += P V: kind::f16, P in fp16 written over S in tensor memory (the A operand), V converted
//     exactly to fp16 as the MN-major B operand (keys as K rows, as the page has them: no transpose).
// TMEM: S of the two slots, then O of the two slots: 4 x 128 columns, all of it.
//
// Warps: 0-3 and 4-7 softmax of slot 0 and 1 (one row per thread, 64 scores at a time in registers), 8-11
// load Q and convert V, 12 resolves pages and issues the copies, 13 issues S, 14 issues P V.  Two issuers,
// because an issue blocks while the tensor queue is full: each waits for its operands while the other's products
// run (one warp for both: 4.12 ms against 3.41).  An issuer is one elected lane, waits included (3.41 -> 3.06 ms).
// P goes over in halves of 64 keys, so that the first half's product runs beside the second half's softmax.
// Queries lie twice (but two tiles of bf16 rows), so that the next unit's are loaded beside this one's pages.
// Every wait is bounded; a role that gives up flags MSA_DEVERR_TIMEOUT, leaves its loop and meets
// the others at the end, where TMEM is freed.
//
// Measured: 4,096 tokens on 64K, 32 heads of E4M3 queries, 2.74 ms = 1.65 PFLOP/s of the products: a slot's chain (S,
// softmax, P V, rescale) is longer than the other slot's products.  8 draft tokens of 4 sequences of 512K:
// 306 us = 5.0 TB/s of pages; the same chain, the pages' stream alone would take 230.
// More stages of K, raw V or fp16 V, polling waits, S in halves of 64 keys and register shares between the warps
// changed nothing or lost.  Registers spilled in the softmax's steps cost 10 % and more, so what they do not need
// is kept in shared memory or made again where a unit ends.  Short contexts (a few pages a unit) wait for
// latencies: lengths, table, scales, queries, first pages, then a unit's rows written before the next begin.
#include <cuda_bf16.h>

#include "fp8_device.cuh"
#include "fp8_kernels.h"
#include "fp8_merge.cuh"
#include "msa_device.cuh"
#include "tile_split.cuh"
#include "umma.cuh"

namespace msa {

constexpr int kFtRows = 128;                 // rows per tile
constexpr int kFtThreads = 480;
constexpr int kFtK = 3, kFtRaw = 2, kFtV = 2;  // stages: K pages, raw V pages, V as fp16
constexpr int kFtItems = 8;                  // page records in flight
constexpr int kFtVBytes = kBlock * kDim * 2;
constexpr int kFtPlaceFloats = 2 * kFtRows * (kDim + 2);  // a partial state of 256 rows
constexpr uint32_t kFtO = 256;               // TMEM column of slot 0's O

struct alignas(16) FtItem {
  int unit;       // index into the plan's units; -1: no more items
  int g;
  int block;      // -1: a unit (or a part of one) with no page
  int place;      // partial-state place of a cut unit; -1: the whole unit is this CTA's
  float k_scale;  // 2^a
  float v_exp;    // b
  int seq;        // sequence
  int flags;      // kFtEdge ...
};
// Flags of a record: some row of the sequence must not see all of the page; some row of slot s's tile must not
// see all of its half h (bit kFtHide + 2 s + h); the unit has two tiles; the page's V scale is more than 2^kFtRefSlack
// below that of an earlier page of the unit.
constexpr int kFtEdge = 1, kFtTwo = 2, kFtHide = 2, kFtLow = 64;

// The reference's rule (fp8_device.cuh has what it must hold): it goes up where a P would pass 2^kFp8RefMax, and down
// only at pages marked kFtLow, where the row's sum so far at the page's scale is below 2^kFtRefMin.  So that sum is at
// least 2^4 wherever P is rounded, and 2^6 where the row's pages have one scale: 2^-29 and 2^-31 of the row's sum.  A
// first place four higher, as the streaming form has it, moves more references early: a prompt chunk took 2.77 ms
// instead of 2.69.  The mark and the way down cost 1 to 2 % (4 x 128K with 8 draft tokens 121.8 -> 124.5 us); asking
// every page 5 %.
constexpr float kFtRefSet = 7.f, kFtRefMin = 4.f, kFtRefSlack = 2.f;

struct FtShared {
  uint64_t k_full[kFtK], k_empty[kFtK], raw_full[kFtRaw], raw_empty[kFtRaw], v_full[kFtV], v_empty[kFtV];
  uint64_t item_full[kFtItems], item_empty[kFtItems];
  uint64_t s_full[2], p_full[2][2], pv_done[2][2];  // [slot], [slot][half of the page's keys]
  uint64_t q_full[2], fin[2];   // Q of a unit loaded; a unit written (by the unit's parity on this CTA)
  uint64_t other;               // slot 1's statistics of a one-tile unit left
  uint64_t drain[2];             // every product issued has ended (after a wait that gave up)
  uint32_t tmem;
  int nan_any[2];
  FtItem item[kFtItems];
  float q_fac[2][2 * kFtRows];  // the power of two taken out of each row (bf16)
  float other_m[kFtRows], other_l[kFtRows];
  int32_t prefix[1024 + 1];     // the units' prefix sums, where the CTA makes them itself
  float2 ref[2 * kFtRows];      // of a row whose reference is to go down (M is -inf meanwhile): the old one, and the
                                // row's sum at the page's scale (log2)
  int pos[2 * kFtRows];         // positions of the rows of the slots' tiles: read by the thread that wrote it
  int nan_key[2][kDim];         // first key of the unit's edge pages with a NaN code in V, per dim
};

constexpr int kFtQHalf = 2 * kFtRows * 128;   // two tiles of E4M3 rows
constexpr size_t kFtQ = 2 * kFtQHalf;         // bf16: the parts hi and lo; E4M3: this unit's and the next one's
constexpr size_t kFtSmem = 1024 + kFtQ + kFtK * kFp8PageBytes + kFtRaw * kFp8PageBytes + kFtV * kFtVBytes + sizeof(FtShared);
static_assert(kFtSmem <= 232448, "227 KB of shared memory per CTA");

// ---------------------------------------------------------------- the plan

// Tiles of 256 rows per (sequence, group), and of one of them: first row, rows, steps per page, pages.
struct FtUnit {
  int b, row0, rows, width, pages;
  bool live;
};
__device__ __forceinline__ FtUnit ft_unit(const Fp8AttnArgs& a, int u, int per_seq) {
  FtUnit t;
  t.b = u / per_seq;
  t.row0 = (u - t.b * per_seq) * 2 * kFtRows;
  const int all = a.q_len * a.heads_per_group;
  t.rows = min(all - t.row0, 2 * kFtRows);
  t.width = t.rows > kFtRows ? 2 : 1;
  const int L = a.seq_lens[t.b];
  t.live = length_ok(a, L);
  t.pages = t.live ? (L - a.q_len + (t.row0 + t.rows - 1) / a.heads_per_group) / kBlock + 1 : 1;
  return t;
}

// out[u]: steps (per group) of the units before u, u = 0..units; every thread of the CTA (a whole number of
// warps, at most 32) calls it.  `flag`: report bad lengths.
__device__ __forceinline__ void ft_prefix(const Fp8AttnArgs& a, int per_seq, int32_t* out, int* warp_sum, bool flag) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  const int units = a.batch * per_seq;
  int base = 0;
  for (int u0 = 0; u0 < units; u0 += threads) {
    const int u = u0 + tid;
    int v = 0;
    if (u < units) {
      const FtUnit t = ft_unit(a, u, per_seq);
      v = t.width * t.pages;
      if (flag && t.row0 == 0 && !t.live && a.seq_lens[t.b] != 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
    }
    int x = v;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, s);
      if (lane >= s) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    const int w = lane < threads / 32 ? warp_sum[lane] : 0;
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    if (u < units) out[u] = base + x - v + before;
    base += __reduce_add_sync(0xffffffffu, w);
    __syncthreads();
  }
  if (tid == 0) out[units] = base;
}

// Units up to which every CTA of the attention sums for itself (as many as a CTA sums in three rounds: 32.6 ->
// 31.6 us for one prompt of 512, 58.3 -> 58.1 for 23 short sequences); more are summed by a launch before it, which
// is then little beside the units' own time.
constexpr int kFtOwnUnits = 1024;

constexpr int kFtPlanThreads = 1024;
__global__ void __launch_bounds__(kFtPlanThreads) fp8_tile_plan_kernel(const Fp8AttnArgs a, int per_seq) {
  __shared__ int s_warp[32];
  grid_dependency_wait();
  grid_dependents_launch();
  ft_prefix(a, per_seq, a.block_prefix, s_warp, true);
}

// ---------------------------------------------------------------- tcgen05 forms used here only

// kind::f8f6f4, both operands in shared memory
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

// 16 bytes (or, with bytes = 0, as many zeros) global -> shared by this thread's own queue
__device__ __forceinline__ void cp_async16(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Four floats as E5M2 codes, the first in the low byte
__device__ __forceinline__ uint32_t f32x4_to_e5m2x4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n"
      " .reg .b16 lo, hi;\n"
      " cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n"
      " cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n"
      "}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

// Output dim of accumulator column n: the upper 64 dims' 16-byte chunks are stored in swapped
// pairs (the converters' shared stores are then free of bank conflicts).  Of column group n / 8:
__device__ __forceinline__ int ft_dim8(int group) { return group < 8 ? group : group ^ 1; }

// A lane's 16 bf16 dims of a row (eight lanes hold the row) as the E4M3 and E5M2 parts hi + lo = q 2^-k;
// returns 2^k, which puts the row's largest value into [2^7, 2^8) (below that for rows of at most 2^-119, whose
// 2^-k float32 would not hold).  A row with an infinity becomes NaN.
__device__ __forceinline__ float ft_split_bf16(const uint4& a, const uint4& b, uint4& hi, uint4& lo) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float v[16], m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    m = fmaxf(m, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
  }
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  const int k = min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127 - 7, -126), 120);
  const float inv = m < INFINITY ? exp2_int(-k) : NAN;
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = v[4 * i + j] * inv;
    h[i] = f32x4_to_e4m3x4(x[0], x[1], x[2], x[3]);
    uint32_t p0, p1;
    e4m3x4_to_f16x4(h[i], p0, p1);
    const float2 p = f16x2_to_float2(p0), q = f16x2_to_float2(p1);
    l[i] = f32x4_to_e5m2x4(x[0] - p.x, x[1] - p.y, x[2] - q.x, x[3] - q.y);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  return exp2_int(k);
}

// A row's factor f, at least 2^-86: times any page's 2^a it is then a normal number (-inf, a hidden key's score,
// times it stays -inf), and a score, at most 2^25, times 2^-86 2^40 is below 2^-20, whatever smaller f it had.
__device__ __forceinline__ float ft_factor(float f) {
  return __uint_as_float(max(__float_as_uint(f), static_cast<uint32_t>(127 - 86) << 23));
}

// ---------------------------------------------------------------- the kernel

__global__ void __launch_bounds__(kFtThreads, 1)
    fp8_tile_kernel(const Fp8AttnArgs a, const __grid_constant__ Fp8Maps maps, int per_seq, int whole) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* q_tile = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* k_ring = q_tile + kFtQ;
  uint8_t* raw_ring = k_ring + kFtK * kFp8PageBytes;
  uint8_t* v_ring = raw_ring + kFtRaw * kFp8PageBytes;
  FtShared* sh = reinterpret_cast<FtShared*>(v_ring + kFtV * kFtVBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = a.q_len, Hg = a.heads_per_group, G = a.groups;

  if (tid == 0) {
    for (int i = 0; i < kFtK; ++i) {
      mbar_init(&sh->k_full[i], 1);
      mbar_init(&sh->k_empty[i], 1);
    }
    for (int i = 0; i < kFtRaw; ++i) {
      mbar_init(&sh->raw_full[i], 1);
      mbar_init(&sh->raw_empty[i], 4);
    }
    for (int i = 0; i < kFtV; ++i) {
      mbar_init(&sh->v_full[i], 4);
      mbar_init(&sh->v_empty[i], 1);
    }
    for (int i = 0; i < kFtItems; ++i) {
      mbar_init(&sh->item_full[i], 1);
      mbar_init(&sh->item_empty[i], 14);  // eight softmax warps, four converters, two issuers
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->s_full[i], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sh->p_full[i][h], 4);
        mbar_init(&sh->pv_done[i][h], 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->q_full[i], 4);
      mbar_init(&sh->fin[i], 9);  // eight softmax warps, the issuer of S
    }
    mbar_init(&sh->drain[0], 1);
    mbar_init(&sh->drain[1], 1);
    mbar_init(&sh->other, 4);
    fence_mbar_init();
  }
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh->tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  grid_dependency_wait();
  grid_dependents_launch();
  const int units = a.batch * per_seq;
  const int32_t* prefix = a.block_prefix;
  if (units <= kFtOwnUnits) {
    ft_prefix(a, per_seq, sh->prefix, sh->nan_key[0], blockIdx.x == 0);
    prefix = sh->prefix;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (units <= kFtOwnUnits && blockIdx.x == 0)  // for the merge
    for (int u = tid; u <= units; u += kFtThreads) a.block_prefix[u] = sh->prefix[u];
  const uint32_t tmem = sh->tmem;
  // Two units' queries fit by turns, but for two tiles of bf16 rows: where the odd units' lie
  const bool q_by_turns = !a.q_bf16 || T * Hg <= kFtRows;
  const int q_turn = !q_by_turns ? 0 : a.q_bf16 ? kFtRows * 128 : kFtQHalf;
  bool failed = false;

  // The next page record, for a whole warp; `n` counts records.
  const FtDiv by_hg(Hg);
  auto take_item = [&](int n, FtItem& it) -> bool {
    if (!mbar_wait_warp(&sh->item_full[n % kFtItems], (n / kFtItems) & 1)) return false;
    it = sh->item[n % kFtItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->item_empty[n % kFtItems]);
    return true;
  };

  if (warp < 8) {
    // ---- softmax of slot `slot`: row r of its tile
    const int slot = warp >> 2, r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + slot * 128 + lane_base, tO = tmem + kFtO + slot * 128 + lane_base;
    // What the steps need stays in registers, the rest is made again where a unit ends.  Steps of this slot and of
    // the other one so far, pages, units before this one:
    int unit = -1, g = 0, done = 0, done_o = 0, valid_pages = 0, uc = -1;
    // bits: steps of this slot, of the other one in the unit; slot of a one-tile unit's next page; parity of the
    // one-tile units so far; two tiles; place + 1 (two bits)
    constexpr int kMine = 1, kOther = 2, kTurn = 4, kShared = 8, kTwo = 16, kPlace = 32;
    int st = 0;
    float M = -INFINITY, l = 0.f, q_fac = ft_factor(a.scale_log2);
    const int row_of_slot = r + ((warp >> 2) << 7);

    // writes the unit's rows (or its partial state)
    auto finish = [&]() -> bool {
      const bool mine = st & kMine;
      if (M == -INFINITY) M = sh->ref[row_of_slot].x;  // (a way down that no key followed)
      if (mine && !mbar_wait_warp(&sh->pv_done[slot][1], (done - 1) & 1)) return false;
      const int place = st / kPlace - 1, b = unit / per_seq, row0 = (unit - b * per_seq) * 2 * kFtRows;
      const int row = row0 + (st & kTwo ? row_of_slot : r), row_end = min(row0 + 2 * kFtRows, T * Hg);
      if (!(st & kTwo)) {
        if (slot == 1) {
          sh->other_m[r] = M;
          sh->other_l[r] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->other);
          return true;
        }
        if (!mbar_wait_warp(&sh->other, (st & kShared) != 0)) return false;
        if (st & kOther && !mbar_wait_warp(&sh->pv_done[1][1], (done_o - 1) & 1)) return false;
      }
      tc_fence_after();
      // state of the row = fa * own O + fb * the other slot's O
      float fa = mine ? 1.f : 0.f, fb = 0.f;
      const bool both = (st & (kTwo | kOther)) == kOther;
      if (both) {
        const float mo = sh->other_m[r], lo = sh->other_l[r];
        const float mn = fmaxf(M, mo);
        fa = mn == -INFINITY ? 1.f : ex2(M - mn);
        fb = mn == -INFINITY ? 1.f : ex2(mo - mn);
        l = l * fa + lo * fb;
        M = mn;
      }
      const bool valid = row < row_end;
      const bool any = l != 0.f;  // (NaN counts as any)
      const float inv = any ? 1.f / l : 0.f;
      const float out_f = place < 0 ? inv : 1.f;
      const int64_t token = static_cast<int64_t>(b) * T + by_hg(row);
      const int64_t hr = token * G * Hg + g * Hg + (row - by_hg(row) * Hg);
      const int pr = row - row0;  // row of the partial state
      float* part = place < 0 ? nullptr
                              : a.partial + (2 * static_cast<int64_t>(blockIdx.x) + place) * kFtPlaceFloats;
      const bool poison = sh->nan_any[uc & 1] != 0;
      const int pos = sh->pos[row_of_slot];
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {  // 16 columns = dims of two groups of 8
        uint32_t x[16];
        float v[16];
        if (mine) {
          tmem_ld16(tO + 16 * c, x);
          tmem_wait_ld(x);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = mine ? __uint_as_float(x[i]) * fa : 0.f;
        if (both) {
          tmem_ld16(tO + 128 + 16 * c, x);
          tmem_wait_ld(x);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(x[i]) * fb;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (poison && pos >= sh->nan_key[uc & 1][8 * ft_dim8(2 * c + (i >> 3)) + (i & 7)]) v[i] = NAN;
          v[i] *= out_f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!valid) break;
          const int d = 8 * ft_dim8(2 * c + i);
          if (place < 0) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
              w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(a.out + hr * kDim + d) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
            // four dims of all rows together: the lanes of a store are neighbouring rows
            float4* dst = reinterpret_cast<float4*>(part) + (d / 4) * (2 * kFtRows) + pr;
            dst[0] = make_float4(v[8 * i], v[8 * i + 1], v[8 * i + 2], v[8 * i + 3]);
            dst[2 * kFtRows] = make_float4(v[8 * i + 4], v[8 * i + 5], v[8 * i + 6], v[8 * i + 7]);
          }
        }
        __syncwarp();
      }
      if (valid) {
        if (place < 0) {
          if (a.lse != nullptr) a.lse[hr] = fp8_lse(M, l);
          if (a.weight_out != nullptr)
            a.row_stat[(static_cast<int64_t>(b) * G + g) * T * Hg + row] = make_float2(any ? M : 0.f, inv);
        } else {
          part[2 * kFtRows * kDim + pr] = M;
          part[2 * kFtRows * (kDim + 1) + pr] = l;
        }
      }
      tc_fence_before();
      return true;
    };

    for (int n = 0;; ++n) {
      FtItem it;
      if (!take_item(n, it)) {
        failed = true;
        break;
      }
      if (it.unit < 0 || it.unit != unit || it.g != g) {
        if (unit >= 0) {
          if (!finish()) {
            failed = true;
            break;
          }
          if (!(st & kTwo)) st ^= kShared;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->fin[uc & 1]);
        }
        const bool shared_o = unit >= 0 && !(st & kTwo);
        unit = it.unit;
        g = it.g;
        if (unit < 0) break;
        ++uc;
        // slot 0 reads slot 1's O and statistics of a one-tile unit: slot 1 goes on when it has
        if (slot == 1 && shared_o && !mbar_wait_warp(&sh->fin[(uc - 1) & 1], ((uc - 1) >> 1) & 1)) {
          failed = true;
          break;
        }
        st = (st & kShared) | (it.flags & kFtTwo ? kTwo : 0) | (it.place + 1) * kPlace;
        const int row = (unit - it.seq * per_seq) * 2 * kFtRows + (st & kTwo ? row_of_slot : r);
        sh->pos[row_of_slot] = a.seq_lens[it.seq] - T + by_hg(min(row, T * Hg - 1));
        M = -INFINITY;
        sh->ref[row_of_slot] = make_float2(M, M);
        l = 0.f;
        if (!mbar_wait_warp(&sh->q_full[uc & 1], (uc >> 1) & 1)) {
          failed = true;
          break;
        }
        if (a.q_bf16) q_fac = ft_factor(a.scale_log2 * sh->q_fac[uc & 1][st & kTwo ? row_of_slot : r]);
      }
      if (it.block < 0) continue;
      // the page's V stage, and whether its step is this slot's
      const int vstage = valid_pages % kFtV, vphase = (valid_pages / kFtV) & 1;
      ++valid_pages;
      if (!(st & kTwo)) {
        st ^= kTurn;
        if ((st & kTurn) == (slot ? kTurn : 0)) {  // (toggled already)
          ++done_o;
          st |= kOther;
          continue;
        }
      }
      if (it.flags & kFtLow) {  // (a row sets its reference aside here; it goes down with the row's next score)
        const float t = M + __log2f(l) + it.v_exp;
        if (t < M + kFtRefMin) {
          sh->ref[row_of_slot] = make_float2(M, t);
          M = -INFINITY;
        }
      }
      // the converters' NaN marks of a page that some row of the sequence does not see whole are read
      // when the unit is written: seeing the page's stage full orders them before that (the stage
      // is not used again before this step's P)
      if (!mbar_wait_warp(&sh->s_full[slot], done & 1) ||
          (it.flags & kFtEdge && !mbar_wait_warp(&sh->v_full[vstage], vphase))) {
        failed = true;
        break;
      }
      tc_fence_after();
      // positive, so that -inf times it stays -inf
      const float f = finite_factor(it.k_scale * q_fac);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const uint32_t tH = tS + 64 * h;
        uint32_t v[64];
        float mx;
        tmem_ld64_max(tH, v, mx);
        tmem_wait_ld(v);
        asm volatile("" : "+f"(mx));
        if (it.flags >> (kFtHide + 2 * slot + h) & 1) {
          // some row of the tile must not see one of these keys: -inf over its scores, and the maximum again
          const int vis = sh->pos[row_of_slot] - it.block * kBlock - 64 * h + 1;  // visible columns
          mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            v[j] = j < vis ? v[j] : 0xff800000u;
            mx = fmaxf(mx, __uint_as_float(v[j]));
          }
        }
        mx = fmaf(mx, f, it.v_exp);
        if (__any_sync(0xffffffffu, mx > M + kFp8RefMax)) {
          float alpha = 1.f;
          if (mx > M + kFp8RefMax) {
            if (M == -INFINITY) {  // the row's first key, or the reference goes down
              const float2 ref = sh->ref[row_of_slot];
              M = ref.x;
              mx = fmaxf(mx, ref.y);
            }
            const float mn = ceilf(mx) - kFtRefSet;
            alpha = ex2(M - mn);
            M = mn;
            l *= alpha;
            sum.x *= alpha;
            sum.y *= alpha;
          }
          if (st & kMine || h > 0) {  // O as the products issued so far leave it, rescaled
            if (!mbar_wait_warp(&sh->pv_done[slot][h ^ 1], (h ? done : done - 1) & 1)) {
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
        }
        // P goes over the first 32 columns of S
        const float c0 = it.v_exp - (M == -INFINITY ? 0.f : M);
        const float2 ff = make_float2(f, f), cc = make_float2(c0, c0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int k = 32 * i + 2 * j;
            const float2 e = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), ff, cc);
            const float2 p = make_float2(ex2(e.x), ex2(e.y));
            sum = add2(sum, p);
            pk[j] = pack_f16x2(p.x, p.y);
          }
          tmem_st16(tH + 16 * i, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p_full[slot][h]);
      }
      if (failed) break;
      ++done;
      st |= kMine;
      if (st & kTwo) ++done_o;
      const float total = sum.x + sum.y;
      l = fmaf(total, ex2(-it.v_exp), l);
      if (a.weight_out != nullptr) {
        const int row = (unit - it.seq * per_seq) * 2 * kFtRows + (st & kTwo ? row_of_slot : r);
        if (row < T * Hg)
          a.share[((static_cast<int64_t>(it.seq) * G + g) * a.max_blocks + it.block) * T * Hg + row] =
              make_float2(total, (M == -INFINITY ? 0.f : M) - it.v_exp);
      }
    }
  } else {
    if (warp < 12) {
      // ---- Q tiles, V conversion
      const int ct = tid - 256;
      int unit = -1, g = 0, page = 0, uc = -1;
      FtUnit t{};
      int L = 0;
      for (int n = 0; !failed; ++n) {
        FtItem it;
        if (!take_item(n, it)) {
          failed = true;
          break;
        }
        if (it.unit < 0 || it.unit != unit || it.g != g) {
          unit = it.unit;
          g = it.g;
          if (unit < 0) break;
          ++uc;
          // the unit that used this one's half of Q (bf16: both halves), factors and NaN marks is written
          const int back = a.q_bf16 && !q_by_turns ? 1 : 2;
          if (uc >= back && !mbar_wait_warp(&sh->fin[(uc - back) & 1], ((uc - back) >> 1) & 1)) {
            failed = true;
            break;
          }
          t = ft_unit(a, unit, per_seq);
          L = a.seq_lens[t.b];
          sh->nan_key[uc & 1][ct] = INT32_MAX;
          if (ct == 0) sh->nan_any[uc & 1] = 0;
          uint8_t* q_half = q_tile + (uc & 1) * q_turn;
          const int c = ct & 7;  // dims 16 c .. 16 c + 15 of rows ct / 8, + 16, ...
          // Rows behind the unit's are zeros.  bf16 rows are copied as they are first, their first 64 dims into
          // the place of the row's hi part and the others into that of its lo part, and split there.
          const int rows = t.width * kFtRows;
          const int64_t at0 = static_cast<int64_t>(t.b) * T * a.q_stride + g * Hg * kDim;
#pragma unroll 2
          for (int rr = ct >> 3; rr < rows; rr += 16) {
            const int row = t.row0 + rr, token = by_hg(row);
            const int64_t at = rr < t.rows ? at0 + token * a.q_stride + (row - token * Hg) * kDim : 0;
            const uint32_t bytes = rr < t.rows ? 16u : 0u;
            uint8_t* tile = q_half + (rr >> 7) * (kFtRows * 128);
            if (a.q_bf16) {
              const uint8_t* src = static_cast<const uint8_t*>(a.q) + 2 * at + 32 * c;
              uint8_t* raw = tile + (c >> 2) * kFtQHalf + (rr & 127) * 128 + (c & 3) * 32;
              cp_async16(raw, src, bytes);
              cp_async16(raw + 16, src + 16, bytes);
            } else {
              cp_async16(tile + sw128(rr & 127, c), static_cast<const uint8_t*>(a.q) + at + 16 * c, bytes);
            }
          }
          cp_async_wait_all();
          if (a.q_bf16) {
#pragma unroll 1
            for (int rr = ct >> 3; rr < rows; rr += 16) {
              uint8_t* tile = q_half + (rr >> 7) * (kFtRows * 128);
              const uint8_t* raw = tile + (c >> 2) * kFtQHalf + (rr & 127) * 128 + (c & 3) * 32;
              uint4 hi, lo;
              const float fac = ft_split_bf16(lds128(raw), lds128(raw + 16), hi, lo);
              __syncwarp();  // the lanes of a row have read it
              uint8_t* dst = tile + sw128(rr & 127, c);
              *reinterpret_cast<uint4*>(dst) = hi;
              *reinterpret_cast<uint4*>(dst + kFtQHalf) = lo;
              if (c == 0) sh->q_fac[uc & 1][rr] = fac;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->q_full[uc & 1]);
          // every converter has reset its marks before any page sets one
          if (!mbar_wait_warp(&sh->q_full[uc & 1], (uc >> 1) & 1)) {
            failed = true;
            break;
          }
        }
        if (it.block < 0) continue;
        const int rs = page % kFtRaw, vs = page % kFtV;
        if (!mbar_wait_warp(&sh->raw_full[rs], (page / kFtRaw) & 1)) {
          failed = true;
          break;
        }
        // all of the page's loads first: the raw stage is free again before the fp16 stage is waited for
        const uint8_t* src = raw_ring + rs * kFp8PageBytes;
        const int c = ct & 7;
        uint4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = lds128(src + page_chunk(16 * i + (ct >> 3), c));
        if (it.block * kBlock + kBlock - 1 > L - T) {  // hidden from some row of the sequence
          uint32_t any = 0u;
#pragma unroll
          for (int i = 0; i < 8; ++i) any |= e4m3_nans(u[i].x) | e4m3_nans(u[i].y) | e4m3_nans(u[i].z) | e4m3_nans(u[i].w);
          if (any != 0u) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              const int r = 16 * i + (ct >> 3), key = it.block * kBlock + r;
              const uint4 x = lds128(src + page_chunk(r, c));
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t nan = e4m3_nans(w[j]);
                if (nan == 0u || key >= L) continue;
                sh->nan_any[uc & 1] = 1;
#pragma unroll 1
                for (int q = 0; q < 4; ++q)
                  if (nan >> (8 * q + 7) & 1u) atomicMin(&sh->nan_key[uc & 1][16 * c + 4 * j + q], key);
              }
            }
            auto clear = [](uint32_t& w) { w &= ~whole_bytes(e4m3_nans(w)); };
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              clear(u[i].x);
              clear(u[i].y);
              clear(u[i].z);
              clear(u[i].w);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->raw_empty[rs]);
        if (page >= kFtV && !mbar_wait_warp(&sh->v_empty[vs], (page / kFtV - 1) & 1)) {
          failed = true;
          break;
        }
        uint8_t* dst = v_ring + vs * kFtVBytes;
        const int h0 = c < 4 ? 2 * c : 2 * (c & 3) + 1;  // chunk of the first 8 dims within its half
        uint8_t* half = dst + (c < 4 ? 0 : kFtVBytes / 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 16 * i + (ct >> 3);
          uint32_t x[8];
          e4m3x4_to_f16x4(u[i].x, x[0], x[1]);
          e4m3x4_to_f16x4(u[i].y, x[2], x[3]);
          e4m3x4_to_f16x4(u[i].z, x[4], x[5]);
          e4m3x4_to_f16x4(u[i].w, x[6], x[7]);
          *reinterpret_cast<uint4*>(half + sw128(r, h0)) = make_uint4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<uint4*>(half + sw128(r, h0 ^ 1)) = make_uint4(x[4], x[5], x[6], x[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->v_full[vs]);
        ++page;
      }
    } else if (warp == 12) {
      // ---- producer: page records and copies
      const int64_t E = static_cast<int64_t>(prefix[units]) * G;
      int x0 = 0, x1 = 0;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        x0 = x1;
        x1 = ft_cut(prefix, units, G, E, blockIdx.x + i, gridDim.x, whole);
      }
      // every sequence's tiles read its pages again: keep them in L2, unless one tile has them all
      const uint64_t policy = per_seq > 1 ? l2_evict_normal_policy() : l2_evict_first_policy();
      int n = 0, page_n = 0;
      auto record = [&](const FtItem& it) -> bool {
        if (n >= kFtItems && !mbar_wait_warp(&sh->item_empty[n % kFtItems], (n / kFtItems - 1) & 1)) return false;
        if (lane == 0) {
          sh->item[n % kFtItems] = it;
          mbar_arrive(&sh->item_full[n % kFtItems]);
        }
        ++n;
        return true;
      };
      int u = x0 < x1 ? ft_find(prefix, units, G, x0) : units;
      for (; u < units && !failed; ++u) {
        const int64_t first = static_cast<int64_t>(prefix[u]) * G;
        if (first >= x1) break;
        const FtUnit t = ft_unit(a, u, per_seq);
        const int steps = t.width * t.pages, two = t.width == 2 ? kFtTwo : 0;
        // positions of the sequence's first token and of the first row of each slot's tile
        const int pos0 = t.live ? a.seq_lens[t.b] - T : 0, pos1 = pos0 + t.row0 / Hg;
        const int pos2 = two ? pos0 + (t.row0 + kFtRows) / Hg : pos1;
        for (int g = 0; g < G && !failed; ++g) {
          const int64_t u0 = first + static_cast<int64_t>(g) * steps;
          if (u0 >= x1) break;
          const int lo = static_cast<int>(max(x0 - u0, int64_t{0}) / t.width);
          const int hi = min(static_cast<int>((x1 - u0) / t.width), t.pages);
          if (lo >= hi) continue;
          const int place = lo == 0 && hi == t.pages ? -1 : lo == 0 ? 1 : 0;
          FtItem it{u, g, -1, place, 0.f, 0.f, t.b, two};
          bool any = false;
          float top_exp = -INFINITY;  // largest V scale of the unit's pages so far
          for (int p0 = lo; p0 < hi && !failed; p0 += 32) {
            const int p = p0 + lane;
            int row = -1;
            float ks = 0.f, ve = 0.f;
            if (p < hi && t.live) {
              const int pg = a.block_table[static_cast<int64_t>(t.b) * a.max_blocks + p];
              if (pg >= 0 && pg < a.num_pages) {
                const int ph = pg * G + g;
                const int kb = a.k_scale[ph], vb = a.v_scale[ph];
                if (e8m0_ok(kb) && e8m0_ok(vb)) {
                  row = ph * kBlock;
                  ks = exp2_int(kb - kE8m0One);
                  ve = static_cast<float>(vb - kE8m0One);
                } else {
                  flag_error(a.err, MSA_DEVERR_BAD_SCALE);
                }
              } else {
                flag_error(a.err, MSA_DEVERR_BAD_PAGE);
              }
              if (row < 0 && a.weight_out != nullptr) {  // a skipped page collects nothing
                float2* share = a.share + ((static_cast<int64_t>(t.b) * G + g) * a.max_blocks + p) * T * Hg + t.row0;
                for (int i = 0; i < t.rows; ++i) share[i] = make_float2(0.f, 0.f);
              }
            }
            const int count = min(hi - p0, 32);
            for (int j = 0; j < count && !failed; ++j) {
              const int y = __shfl_sync(0xffffffffu, row, j);
              it.k_scale = __shfl_sync(0xffffffffu, ks, j);
              it.v_exp = __shfl_sync(0xffffffffu, ve, j);
              if (y < 0) continue;
              any = true;
              it.block = p0 + j;
              const int half = it.block * kBlock + 63, last = half + 64;  // last keys of the page's halves
              it.flags = two | (last > pos0 ? kFtEdge : 0) | (half > pos1 ? 1 : 0) << kFtHide |
                         (last > pos1 ? 2 : 0) << kFtHide | (half > pos2 ? 4 : 0) << kFtHide |
                         (last > pos2 ? 8 : 0) << kFtHide | (it.v_exp < top_exp - kFtRefSlack ? kFtLow : 0);
              top_exp = fmaxf(top_exp, it.v_exp);
              const int ksl = page_n % kFtK, rsl = page_n % kFtRaw;
              if (!record(it) || (page_n >= kFtK && !mbar_wait_warp(&sh->k_empty[ksl], (page_n / kFtK - 1) & 1)) ||
                  (page_n >= kFtRaw && !mbar_wait_warp(&sh->raw_empty[rsl], (page_n / kFtRaw - 1) & 1))) {
                failed = true;
                break;
              }
              if (lane == 0) {
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(&sh->k_full[ksl], kFp8PageBytes);
                tma_page(k_ring + ksl * kFp8PageBytes, &maps.k, y, &sh->k_full[ksl], policy);
                mbar_arrive_expect_tx(&sh->raw_full[rsl], kFp8PageBytes);
                tma_page(raw_ring + rsl * kFp8PageBytes, &maps.v, y, &sh->raw_full[rsl], policy);
              }
              ++page_n;
            }
          }
          if (!any && !failed) {
            it.block = -1;
            failed = !record(it);
          }
        }
      }
      if (!failed) failed = !record(FtItem{-1, 0, -1, -1, 0.f, 0.f, 0, 0});
      if (failed) {
        // wait (bounded) for the copies still in flight
        for (int k = max(0, page_n - kFtK); k < page_n; ++k) mbar_wait(&sh->k_full[k % kFtK], (k / kFtK) & 1);
        for (int k = max(0, page_n - kFtRaw); k < page_n; ++k) mbar_wait(&sh->raw_full[k % kFtRaw], (k / kFtRaw) & 1);
      }
    } else if (warp == 13 || warp == 14) {
      // ---- product issuers: warp 13 S, warp 14 P V.  Two warps, because issuing blocks while the tensor
      // pipe is full: each waits for its operands while the other's products run.
      const bool scores = warp == 13;
      if (elect_one()) {
        const uint32_t id_s = umma_idesc_f16(kFtRows, kBlock);             // (E4M3 has format code 0 too)
        const uint32_t id_lo = id_s | (1u << 7);                           // A is E5M2
        const uint32_t id_o = umma_idesc_f16(kFtRows, kDim) | (1u << 16);  // B MN-major
        const uint32_t qb = smem_u32(q_tile), kb = smem_u32(k_ring), vb = smem_u32(v_ring);
        int unit = -1, g = 0, width = 1, pages = 0, page = 0, uc = -1;
        int done0 = 0, done1 = 0, start0 = 0, start1 = 0;  // steps of the slots so far, and at the unit's start
        bool bad = false;
        for (int n = 0; !bad; ++n) {
          if (!mbar_wait(&sh->item_full[n % kFtItems], (n / kFtItems) & 1)) {
            bad = true;
            break;
          }
          const int it_unit = sh->item[n % kFtItems].unit, it_g = sh->item[n % kFtItems].g;
          const bool empty = sh->item[n % kFtItems].block < 0;
          mbar_arrive(&sh->item_empty[n % kFtItems]);
          if (it_unit < 0 || it_unit != unit || it_g != g) {
            if (scores && unit >= 0) mbar_arrive(&sh->fin[uc & 1]);
            unit = it_unit;
            g = it_g;
            if (unit < 0) break;
            width = ft_unit(a, unit, per_seq).width;
            pages = 0;
            start0 = done0;
            start1 = done1;
            ++uc;
            if (scores && !mbar_wait(&sh->q_full[uc & 1], (uc >> 1) & 1)) {
              bad = true;
              break;
            }
          }
          if (empty) continue;
          const int ks = page % kFtK, vs = page % kFtV;
          if (scores ? !mbar_wait(&sh->k_full[ks], (page / kFtK) & 1) : !mbar_wait(&sh->v_full[vs], (page / kFtV) & 1)) {
            bad = true;
            break;
          }
          for (int i = 0; i < width && !bad; ++i) {
            const int s = width == 2 ? i : pages & 1;
            const int d = s ? done1 : done0;
            const bool last = i == width - 1;
            if (scores) {
              // S overwrites the slot's P: it waits until that has been multiplied
              if (d > 0 && !mbar_wait(&sh->pv_done[s][1], (d - 1) & 1)) {
                bad = true;
                break;
              }
              tc_fence_after();
              const uint64_t qd = umma_desc(qb + (uc & 1) * q_turn + (width == 2 ? s : 0) * (kFtRows * 128));
              const uint64_t kd = umma_desc(kb + ks * kFp8PageBytes);
              for (int part = 0; part < (a.q_bf16 ? 2 : 1); ++part)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // 32 dims a step
                  umma_f8(tmem + s * 128, qd + ((part * kFtQHalf + 32 * kk) >> 4), kd + ((32 * kk) >> 4),
                          part > 0 ? id_lo : id_s, part > 0 || kk > 0 ? 1u : 0u);
              umma_commit(&sh->s_full[s]);
              if (last) umma_commit(&sh->k_empty[ks]);
            } else {
              for (int h = 0; h < 2; ++h) {  // 64 keys: the products of the first half run beside the softmax of the second
                if (!mbar_wait(&sh->p_full[s][h], d & 1)) {
                  bad = true;
                  break;
                }
                tc_fence_after();
                const bool add = h > 0 || d > (s ? start1 : start0);
                const uint64_t vd = umma_desc_mn(vb + vs * kFtVBytes + h * 64 * 128, kFtVBytes / 2);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // 16 keys: 8 TMEM columns of P, two 8-row groups of V
                  umma_f16_tmem_a(tmem + kFtO + s * 128, tmem + s * 128 + h * 64 + 8 * kk,
                                  vd + ((kk * 2048) >> 4), id_o, add || kk > 0 ? 1u : 0u);
                umma_commit(&sh->pv_done[s][h]);
                if (last && h == 1) umma_commit(&sh->v_empty[vs]);
              }
            }
            s ? ++done1 : ++done0;
          }
          ++pages;
          ++page;
        }
        if (bad) {  // the products still running end before TMEM is freed
          flag_error(a.err, MSA_DEVERR_TIMEOUT);
          umma_commit(&sh->drain[scores]);
          mbar_wait(&sh->drain[scores], 0);
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

// Units cut by range boundaries: the partial states that their CTAs left, added (fp8_merge.cuh).
// blockIdx.x is the unit (by_unit) or the boundary whose unit the CTA takes if it is the unit's first
// cut, whichever is fewer; blockIdx.y the row (kSplit) or eight of them.
template <bool kSplit>
__global__ void __launch_bounds__(kFp8MergeThreads)
    fp8_tile_merge_kernel(const Fp8AttnArgs a, int per_seq, int ctas, int by_unit, int whole) {
  __shared__ Fp8MergeShared sh;
  grid_dependency_wait();
  grid_dependents_launch();
  const int units = a.batch * per_seq, G = a.groups, Hg = a.heads_per_group, T = a.q_len;
  const int64_t E = static_cast<int64_t>(a.block_prefix[units]) * G;
  const int x = blockIdx.x;
  int u = x / G, xb = 0;
  if (!by_unit) {
    xb = ft_lo(E, x + 1, ctas);
    if (xb >= E) return;
    u = ft_find(a.block_prefix, units, G, xb);
  }
  if (a.block_prefix[u + 1] - a.block_prefix[u] <= whole) return;  // not cut
  const FtUnit t = ft_unit(a, u, per_seq);
  const int steps = t.width * t.pages;
  const int64_t first = static_cast<int64_t>(a.block_prefix[u]) * G;
  const int g = by_unit ? x - u * G : static_cast<int>((xb - first) / steps);
  const int64_t u0 = first + static_cast<int64_t>(g) * steps;
  if (!by_unit) {
    const int xa = ft_lo(E, x, ctas);
    if ((xb - u0) / t.width == 0 || (xa > u0 && (xa - u0) / t.width > 0)) return;  // no page before it, or not the first
  }
  if (threadIdx.x < 32) {  // the CTAs with pages of the unit, in order
    int n = 0;
    for (int c0 = by_unit ? static_cast<int>(((u0 + 1) * ctas - 1) / E) : x; c0 < ctas && ft_lo(E, c0, ctas) < u0 + steps;
         c0 += 32) {
      const int c = c0 + threadIdx.x;
      const int64_t a0 = ft_lo(E, c, ctas) - u0, a1 = ft_lo(E, c + 1, ctas) - u0;
      const int lo = static_cast<int>(max(a0, int64_t{0}) / t.width);
      const int hi = static_cast<int>(min(a1 / t.width, static_cast<int64_t>(t.pages)));
      const bool some = c < ctas && a0 < steps && lo < hi;
      const unsigned m = __ballot_sync(0xffffffffu, some);
      if (some) sh.list[n + __popc(m & ((1u << threadIdx.x) - 1u))] = 2 * c + (lo == 0 ? 1 : 0);
      n += __popc(m);
    }
    if (threadIdx.x == 0) sh.n = n;
  }
  __syncthreads();
  if (sh.n < 2) return;  // one CTA's: written by it
  // states lie by chunks of four dims: without kSplit a CTA's eight rows of a chunk are one 128-byte line
  const int pr = kSplit ? blockIdx.y : blockIdx.y * 8 + (threadIdx.x & 7);
  const int chunk = kSplit ? threadIdx.x & 31 : threadIdx.x >> 3;
  if (pr >= t.rows) return;
  float4 o;
  float M, l;
  fp8_merge_row<kSplit>(a.partial, 2 * kFtRows, pr, chunk * 2 * kFtRows + pr, sh, o, M, l);
  if (kSplit && threadIdx.x >= 32) return;
  const int row = t.row0 + pr;
  fp8_write_row(a, (static_cast<int64_t>(t.b) * T + row / Hg) * G * Hg + g * Hg + row % Hg,
                (static_cast<int64_t>(t.b) * G + g) * T * Hg + row, chunk, o, M, l);
}

int fp8_tile_units_per_seq(int64_t rows) { return static_cast<int>((rows + 2 * kFtRows - 1) / (2 * kFtRows)); }

size_t fp8_tile_partial_bytes() { return static_cast<size_t>(2) * kFp8MaxCtas * kFtPlaceFloats * sizeof(float); }

// Steps of a unit up to which it is not cut (ft_cut).  A cut costs two partial states and a merge, about as
// much as kFtCutSteps steps; not cutting leaves CTAs idle: of `all` units (with groups) on n CTAs some take
// ceil(all / n), so that a unit of S steps costs idle * S / n more than its share.  46 sequences of 144 rows and up to 6
// pages take 60 us whole and 76 cut, one prompt of 2,048 tokens 162 and 197, 23 sequences of 75 rows 28 and 44; 12
// sequences of 64 rows and up to 16 pages (48 units) 29 whole and 24 cut.  Above 64 steps a unit is cut in any case,
// so that the long sequences of a ragged batch do not wait for a CTA of their own.
static int ft_whole(const Fp8AttnArgs& a, int per_seq, int n) {
  constexpr int kFtWhole = 64, kFtCutSteps[2] = {6, 11};  // one tile of rows, two
  const int64_t all = static_cast<int64_t>(a.batch) * per_seq * a.groups, idle = n - 1 - (all - 1) % n;
  const int64_t most = static_cast<int64_t>(kFtCutSteps[a.q_len * a.heads_per_group > kFtRows]) * n;
  return idle * kFtWhole <= most ? kFtWhole : static_cast<int>(most / idle);
}

cudaError_t launch_fp8_tile(const Fp8AttnArgs& a, int num_sms, cudaStream_t s) {
  Fp8Maps maps;
  cudaError_t e = fp8_page_maps(a, &maps);
  if (e != cudaSuccess) return e;
  const int per_seq = fp8_tile_units_per_seq(static_cast<int64_t>(a.q_len) * a.heads_per_group);
  const int ctas = num_sms < kFp8MaxCtas ? num_sms : kFp8MaxCtas;
  const int whole = ft_whole(a, per_seq, ctas);
  if ((e = ensure_dynamic_smem(reinterpret_cast<const void*>(fp8_tile_kernel), kFtSmem)) != cudaSuccess) return e;
  if (static_cast<int64_t>(a.batch) * per_seq > kFtOwnUnits &&
      (e = launch_dependent(fp8_tile_plan_kernel, dim3(1), kFtPlanThreads, 0, s, a, per_seq)) != cudaSuccess)
    return e;
  if ((e = launch_dependent(fp8_tile_kernel, dim3(ctas), kFtThreads, kFtSmem, s, a, maps, per_seq, whole)) != cudaSuccess)
    return e;
  const int rows = a.q_len * a.heads_per_group < 2 * kFtRows ? a.q_len * a.heads_per_group : 2 * kFtRows;
  if (ctas == 1 || static_cast<int64_t>(a.max_blocks) * (rows > kFtRows ? 2 : 1) <= whole) return cudaSuccess;  // no cut
  const int64_t units = static_cast<int64_t>(a.batch) * per_seq * a.groups;
  const int by_unit = units < ctas - 1 ? 1 : 0;
  const unsigned grid = by_unit ? static_cast<unsigned>(units) : static_cast<unsigned>(ctas - 1);
  return ctas / units >= kFp8MergeSplitParts
             ? launch_dependent(fp8_tile_merge_kernel<true>, dim3(grid, rows), kFp8MergeThreads, 0, s, a, per_seq,
                                ctas, by_unit, whole)
             : launch_dependent(fp8_tile_merge_kernel<false>, dim3(grid, (rows + 7) / 8), kFp8MergeThreads, 0, s, a, per_seq,
                                ctas, by_unit, whole);
}

}  // namespace msa
