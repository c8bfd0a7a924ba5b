// Attention over the FP8 page cache for few query rows: decode steps (dense, at most 16 rows
// (token, head) of a group) and selections (the at most 8 heads of a group per token).
//
// Mathematics.  For row r and key j of a page with scales 2^a (K) and 2^b (V) the kernel works in
// the log2 domain on e_j = z_j log2(e) + b, the size of the key's term of the output sum:
//   P_j = 2^(e_j - M) in fp16,  O = sum P_j code(v_j),  l = sum over pages of 2^-b sum P_j,
// out = O / l, lse = ln 2 (M + log2 l).  So the V scale costs no multiply per element.  M is an
// integer that keeps P inside fp16's range and moves rarely (kFsRefSet below): P is rounded by 2^-11
// of itself, or by 2^-33 of the row's sum where it is small beside that.  Rescaling and differences
// of M's (shares of the blocks, merges) are exact.  Sums are float32.
//
// Work.  A unit is the rows that share a page list; the (unit, page) pairs of the call are one
// flat list, cut into equal ranges, one for each of the teams of a persistent grid (one CTA an
// SM), short units staying whole (fs_cut).  A team is a producer warp and four consuming warps: the producer resolves 32 entries at a
// time (table -> page -> scales) and streams K and V pages (16 KB each) through a ring of slots
// with tensor copies that land the 128-byte rows swizzled; consumer w takes keys 32w..32w+31 of
// every page: S^T = K Q^T on mma.sync (keys as M, 8 or 16 rows as N; a lane's 16 bytes of a key
// are four k-steps' worth of its fragment, the dims permuted alike in Q), the online softmax, and
// O^T += V^T P^T (pairs of keys byte-interleaved by two permutes per 8 codes, P transposed by
// movmatrix).  E4M3 -> fp16 is exact, so only P is rounded.  With the swizzle every 8-lane phase
// of the 16-byte shared loads touches 8 different bank groups, for K and for V.  At the end of a
// unit the four warps' states are added through shared memory in two steps; a unit that the split
// cut leaves partial states, which fp8_stream_merge_kernel adds.
//
// Bound by the page stream (256 B per token and KV head, read once): 64 sequences of up to 128K 705 us =
// 6.8 TB/s; 8 of up to 32K 39 us with their weights (24 at the stream's rate: start, merge and weights are the rest);
// one token of one sequence of 4,096 11 us, all of it latency.
#include <cuda_bf16.h>

#include "fp8_device.cuh"
#include "fp8_kernels.h"
#include "fp8_merge.cuh"
#include "msa_device.cuh"

namespace msa {

constexpr int kFsWarps = 4;       // consuming warps per team
constexpr int kFsMeta = 4;        // item records (more items than the ring can hold)
constexpr int kFsMaxBatch = 2048; // host bound on the batch
// The reference's rule (fp8_device.cuh has what it must hold).  t is the larger of the page's largest e and the row's
// largest z so far at the page's scale: M moves to ceil(t) - kFsRefSet when t leaves M + kFsRefMin .. M + kFp8RefMax.
// With equal scales t only grows: M moves up only.
constexpr float kFsRefSet = 11.f, kFsRefMin = 8.f;

// NT n-tiles of 8 rows.  Teams and ring slots per team are what fits 227 KB with the merge areas.
template <int NT>
struct FsShape {
  static constexpr int kTeams = NT == 1 ? 3 : 2;
  static constexpr int kSlots = 4;
  static constexpr int kThreads = kTeams * (kFsWarps + 1) * 32;
  static constexpr int kRows = 8 * NT;
  static constexpr int kMergeFloats = NT * 8 * 4 * 32 + 2 * kRows;  // fragments, M, l
  static constexpr int kSlotFloats = kRows * (kDim + 2);             // a partial state
};

struct FsItem {
  int unit;       // -1: no more items
  int place;      // block (dense) or selection slot (sparse)
  int block;      // logical block
  int page;       // -1: nothing to attend to in this range of the unit
  int pos;        // position of the unit's first query token
  float k_scale;  // 2^a
  float v_exp;    // b
};

template <int NT>
struct FsTeam {
  uint64_t full[FsShape<NT>::kSlots], empty[FsShape<NT>::kSlots];
  uint64_t pair;    // warps 2 and 3 wrote their states
  uint64_t last;    // warp 1 wrote its sum
  uint64_t freed;   // warp 0 has read both areas
  FsItem item[kFsMeta];
};

template <int NT>
struct FsShared {
  FsTeam<NT> team[FsShape<NT>::kTeams];
  alignas(16) float merge[FsShape<NT>::kTeams][2][FsShape<NT>::kMergeFloats];
  uint4 q[NT == 1 ? 1 : FsShape<NT>::kTeams * kFsWarps * 8][NT == 1 ? 1 : 32];  // two n-tiles: each warp's B fragments
  int prefix[kFsMaxBatch + 1];
  int chunk[kFsMaxBatch / 32];
};

template <int NT>
constexpr size_t fs_smem_bytes() {
  return 1024 + static_cast<size_t>(FsShape<NT>::kTeams) * FsShape<NT>::kSlots * kFp8PageBytes + sizeof(FsShared<NT>);
}
static_assert(fs_smem_bytes<1>() <= 232448 && fs_smem_bytes<2>() <= 232448, "227 KB of shared memory per CTA");

// Range of team c of n over E entries, and the team that holds entry x.
__device__ __forceinline__ int fs_lo(int64_t E, int c, int n) { return static_cast<int>(E * c / n); }
__device__ __forceinline__ int fs_owner(int64_t E, int64_t x, int n) { return static_cast<int>(((x + 1) * n - 1) / E); }

// Entries of a sequence per group: its blocks; one (with nothing in it) for a padding row, so that
// some team writes the row.
__device__ __forceinline__ int fs_blocks(const Fp8AttnArgs& a, int L) {
  return length_ok(a, L) ? (L + kBlock - 1) / kBlock : 1;
}

// prefix[b] = entries (per group) of the sequences before b, b = 0..batch; every thread calls it.
__device__ __forceinline__ void fs_prefix(const Fp8AttnArgs& a, int* prefix, int* chunk) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = (a.batch + 31) / 32;
  for (int c = warp; c < chunks; c += warps) {
    const int b = 32 * c + lane;
    int v = b < a.batch ? fs_blocks(a, a.seq_lens[b]) : 0;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, s);
      if (lane >= s) v += y;
    }
    if (b < a.batch) prefix[b + 1] = v;
    if (lane == 31) chunk[c] = v;
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
  if (chunks > 1) {
    if (warp == 0) {
      int before = 0;
      for (int c0 = 0; c0 < chunks; c0 += 32) {
        const int own = c0 + lane < chunks ? chunk[c0 + lane] : 0;
        int v = own;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, v, s);
          if (lane >= s) v += y;
        }
        if (c0 + lane < chunks) chunk[c0 + lane] = before + v - own;
        before += __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) prefix[b + 1] += chunk[b >> 5];
    __syncthreads();
  }
}

// The unit and place of entry x: dense units (b, g) hold their sequence's blocks, sparse units
// (b, t, g) 16 places.
struct FsEntry {
  int unit, b, place;
};
__device__ __forceinline__ FsEntry fs_entry(const Fp8AttnArgs& a, const int* prefix, int x) {
  FsEntry e;
  if (a.selection != nullptr) {
    e.unit = x / kTopK;
    e.place = x % kTopK;
    e.b = static_cast<int>(static_cast<unsigned>(e.unit) / static_cast<unsigned>(a.groups * a.q_len));
    return e;
  }
  int lo = 0, hi = a.batch;  // the last b with prefix[b] * G <= x
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(prefix[mid]) * a.groups <= x) lo = mid;
    else hi = mid;
  }
  const int off = x - prefix[lo] * a.groups, nb = prefix[lo + 1] - prefix[lo];
  const int g = off / nb;
  e.b = lo;
  e.unit = lo * a.groups + g;
  e.place = off - g * nb;
  return e;
}

// First entry of team c of n as it is taken: a cut inside a unit of at most `whole` pages goes to the nearer of the
// unit's ends (fs_whole).
__device__ __forceinline__ int fs_cut(const Fp8AttnArgs& a, const int* prefix, int64_t E, int c, int n, int whole) {
  const int x = fs_lo(E, c, n);
  if (whole == 0 || c == 0 || x >= E) return x;
  const FsEntry e = fs_entry(a, prefix, x);
  const int pages = a.selection != nullptr ? kTopK : prefix[e.b + 1] - prefix[e.b];
  if (pages > whole) return x;
  return x - e.place + (2 * e.place < pages ? 0 : pages);
}

// Eight query rows of a unit, from r0, as B fragments (f16), and each row's factor: softmax_scale * log2(e) times the
// power of two taken out of it (bf16).
__device__ __forceinline__ void fs_load_q(const Fp8AttnArgs& a, int unit, int rows, int r0, int gq, int t4,
                                          uint32_t (&bq)[8][2], float (&fac)[2]) {
  const bool sparse = a.selection != nullptr;
  const int Hg = a.heads_per_group;
  const int g = unit % a.groups, bt = unit / a.groups;  // dense: bt = b
  const int r = r0 + gq;
  float f = 1.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) bq[i][0] = bq[i][1] = 0u;
  uint4 v[4] = {};  // 32 bf16 dims
  if (r < rows) {
    const int64_t token = sparse ? bt : static_cast<int64_t>(bt) * a.q_len + r / Hg;
    const int64_t at = token * a.q_stride + (g * Hg + r % Hg) * kDim + 32 * t4;
    if (!a.q_bf16) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + at);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 u = src[h];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) e4m3x4_to_f16x4(w[i], bq[4 * h + i][0], bq[4 * h + i][1]);
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = src[i];
    }
  }
  if (a.q_bf16) {
    // the row times 2^-k, its largest value in [2^14, 2^15): the 8 significant bits of a bf16 value
    // stay exact in f16 down to 2^-31 of that
    float m = 0.f;
    if (r < rows) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
      }
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // (at 112 the largest bf16 value becomes 2^16 - 2^8, which f16 holds)
    const int k = min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127 - 14, -126), 112);
    f = exp2_int(k);
    const float inv = m < INFINITY ? exp2_int(-k) : NAN;  // (a row with an infinity gives NaN: its elements are)
    if (r < rows) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w0 = i & 1 ? v[i >> 1].z : v[i >> 1].x, w1 = i & 1 ? v[i >> 1].w : v[i >> 1].y;
        bq[i][0] = pack_f16x2(__uint_as_float(w0 << 16) * inv, __uint_as_float(w0 & 0xFFFF0000u) * inv);
        bq[i][1] = pack_f16x2(__uint_as_float(w1 << 16) * inv, __uint_as_float(w1 & 0xFFFF0000u) * inv);
      }
    }
  }
  // softmax_scale before the page's 2^a: a large and a small one of the three then meet.  At least 2^-100: times 2^a it
  // is not 0 (-inf, a hidden key's score, stays -inf), and a score, at most 2^32, times 2^-100 2^40 is below 2^-20.
  f = __uint_as_float(max(__float_as_uint(f * a.scale_log2), static_cast<uint32_t>(127 - 100) << 23));
  // accumulator columns of this lane: rows r0 + 2 t4, + 1
  fac[0] = __shfl_sync(0xffffffffu, f, 8 * t4);
  fac[1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
}

template <int NT>
__global__ void __launch_bounds__(FsShape<NT>::kThreads, 1)
    fp8_stream_kernel(const Fp8AttnArgs a, const __grid_constant__ Fp8Maps maps, int whole) {
  using S = FsShape<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);  // the swizzle counts from 1 KB
  uint8_t* slots = base;
  FsShared<NT>* sh = reinterpret_cast<FsShared<NT>*>(base + S::kTeams * S::kSlots * kFp8PageBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, t4 = lane & 3;
  const bool sparse = a.selection != nullptr;
  const int T = a.q_len, Hg = a.heads_per_group;
  const int rows = sparse ? Hg : T * Hg;

  if (tid < S::kTeams) {
    FsTeam<NT>* tm = &sh->team[tid];
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&tm->full[i], 2);  // the copy (its bytes too), the item's record
      mbar_init(&tm->empty[i], kFsWarps);
    }
    mbar_init(&tm->pair, 2);
    mbar_init(&tm->last, 1);
    mbar_init(&tm->freed, 1);
  }
  fence_mbar_init();
  grid_dependency_wait();
  grid_dependents_launch();
  if (!sparse) {
    fs_prefix(a, sh->prefix, sh->chunk);
    if (blockIdx.x == 0) {
      for (int b = tid; b <= a.batch; b += S::kThreads) a.block_prefix[b] = sh->prefix[b];
      for (int b = tid; b < a.batch; b += S::kThreads)
        if (a.seq_lens[b] != 0 && !length_ok(a, a.seq_lens[b])) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
    }
  }
  __syncthreads();
  const int team = warp < S::kTeams * kFsWarps ? warp / kFsWarps : warp - S::kTeams * kFsWarps;
  const int tt = blockIdx.x * S::kTeams + team, teams = gridDim.x * S::kTeams;
  const int64_t E = sparse ? static_cast<int64_t>(a.batch) * T * a.groups * kTopK
                           : static_cast<int64_t>(sh->prefix[a.batch]) * a.groups;
  const int cut = fs_cut(a, sh->prefix, E, tt + (lane & 1), teams, whole);  // both at once
  const int x0 = __shfl_sync(0xffffffffu, cut, 0), x1 = __shfl_sync(0xffffffffu, cut, 1);
  uint8_t* my_slots = slots + team * S::kSlots * kFp8PageBytes;
  FsTeam<NT>* tm = &sh->team[team];

  if (warp >= S::kTeams * kFsWarps) {
    // ---- producer
    const uint64_t policy = sparse && T > 1 ? l2_evict_normal_policy() : l2_evict_first_policy();
    int copied = 0, items = 0;  // items whose copies are issued, whose records are written
    bool ok = true;
    // Slots 2 i, 2 i + 1 of the ring hold item i's K and V.  A slot is full when its copy and the item's
    // record are there, so that the first copies can start before the pages' scales are known.
    auto copy = [&](int page, int row) {
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int use = 2 * copied + kv, slot = use % S::kSlots;
        if (use >= S::kSlots && !mbar_wait_warp(&tm->empty[slot], (use / S::kSlots - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if (page >= 0) {
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&tm->full[slot], kFp8PageBytes);
            tma_page(my_slots + slot * kFp8PageBytes, kv ? &maps.v : &maps.k, row, &tm->full[slot], policy);
          } else {
            mbar_arrive(&tm->full[slot]);
          }
        }
      }
      ++copied;
    };
    auto record = [&](const FsItem& it) {
      if (lane == 0) {
        tm->item[items % kFsMeta] = it;
        mbar_arrive(&tm->full[2 * items % S::kSlots]);
        mbar_arrive(&tm->full[(2 * items + 1) % S::kSlots]);
      }
      ++items;
    };
    auto send = [&](const FsItem& it, int row) {
      if (copied == items) copy(it.page, row);
      if (ok) record(it);
    };
    int open = -1;      // the unit that the last item belongs to
    bool sent = false;  // whether it has an item
    for (int xb = x0; xb < x1 && ok; xb += 32) {
      const int x = xb + lane;
      FsItem it{-1, 0, -1, -1, 0, 0.f, 0.f};
      int ph = -1;
      if (x < x1) {
        const FsEntry en = fs_entry(a, sh->prefix, x);
        it.unit = en.unit;
        it.place = en.place;
        const int L = a.seq_lens[en.b];
        const int n = sparse ? a.selection[x] : en.place;
        // (the table entry is read before the length is known; its place in the table is in range)
        const int page = a.block_table[static_cast<int64_t>(en.b) * a.max_blocks + (n >= 0 && n < a.max_blocks ? n : 0)];
        const bool live = length_ok(a, L);
        if (sparse && !live && L != 0 && en.place == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
        it.pos = L - T + (sparse ? (en.unit / a.groups) % T : 0);
        if (live && n >= 0 && n <= (sparse ? it.pos : L - 1) / kBlock) {
          it.block = n;
          if (page >= 0 && page < a.num_pages) {
            it.page = page;
            ph = page * a.groups + en.unit % a.groups;
          } else {
            flag_error(a.err, MSA_DEVERR_BAD_PAGE);
          }
        }
      }
      const int count = min(x1 - xb, 32);
      const int ks = ph >= 0 ? a.k_scale[ph] : kE8m0One, vs = ph >= 0 ? a.v_scale[ph] : kE8m0One;
      if (xb == x0) {  // the first pages' copies, while the scales are on their way
        const unsigned have = __ballot_sync(0xffffffffu, ph >= 0);
        const int j0 = __ffs(have) - 1;
        // (only where the first item sent is this page: no marker of an empty unit comes before it)
        const int u0 = __shfl_sync(0xffffffffu, it.unit, 0), uj = __shfl_sync(0xffffffffu, it.unit, max(j0, 0));
        if (j0 >= 0 && uj == u0) copy(0, __shfl_sync(0xffffffffu, ph, j0) * kBlock);
      }
      if (it.page >= 0 && !(e8m0_ok(ks) && e8m0_ok(vs))) {
        flag_error(a.err, MSA_DEVERR_BAD_SCALE);
        it.page = -1;
      }
      it.k_scale = exp2_int(ks - kE8m0One);
      it.v_exp = static_cast<float>(vs - kE8m0One);
      if (it.block >= 0 && it.page < 0 && a.weight_out != nullptr) {  // a skipped page collects nothing
        float2* share = a.share + (static_cast<int64_t>(it.unit) * (sparse ? kTopK : a.max_blocks) + it.place) *
                                      kFp8StreamParts * rows;
        for (int i = 0; i < kFp8StreamParts * rows; ++i) share[i] = make_float2(0.f, 0.f);
      }
      for (int j = 0; j < count && ok; ++j) {
        FsItem s;
        s.unit = __shfl_sync(0xffffffffu, it.unit, j);
        s.place = __shfl_sync(0xffffffffu, it.place, j);
        s.block = __shfl_sync(0xffffffffu, it.block, j);
        s.page = __shfl_sync(0xffffffffu, it.page, j);
        s.pos = __shfl_sync(0xffffffffu, it.pos, j);
        s.k_scale = __shfl_sync(0xffffffffu, it.k_scale, j);
        s.v_exp = __shfl_sync(0xffffffffu, it.v_exp, j);
        const int pj = __shfl_sync(0xffffffffu, ph, j);
        if (s.unit != open) {
          if (open >= 0 && !sent) send(FsItem{open, 0, -1, -1, 0, 0.f, 0.f}, 0);
          open = s.unit;
          sent = false;
        }
        // (a page with a bad scale whose copy is on its way goes as an item without a page)
        if (ok && (s.page >= 0 || (pj >= 0 && copied > items))) {
          send(s, pj * kBlock);
          sent = true;
        }
      }
    }
    if (ok && open >= 0 && !sent) send(FsItem{open, 0, -1, -1, 0, 0.f, 0.f}, 0);
    if (ok) send(FsItem{-1, 0, -1, -1, 0, 0.f, 0.f}, 0);
    if (!ok) {
      if (lane == 0) flag_error(a.err, MSA_DEVERR_TIMEOUT);
      // wait (bounded) for the copies still in flight before leaving
      for (int use = max(0, 2 * copied - S::kSlots); use < 2 * copied; ++use)
        mbar_wait(&tm->full[use % S::kSlots], (use / S::kSlots) & 1);
    }
    return;
  }

  // ---- consumers: warp wt of the team, keys 32 wt .. 32 wt + 31 of every page
  const int wt = warp % kFsWarps;
  uint32_t bq[8][2];  // the queries' fragments, of one n-tile
  float fac[NT][2], m_run[NT][2], l_run[NT][2];
  float z_top[NT][2];  // largest z of the row's keys so far, times log2(e)
  float o[NT][8][4];
  int pos[NT][2];  // positions of this lane's accumulator columns
  int unit = -1, units_done = 0, pos_min = 0;
  const int first_unit = x0 < x1 ? fs_entry(a, sh->prefix, x0).unit : -1;
  auto* my_q = sh->q + (NT == 1 ? 0 : 8 * warp);
  auto load_q = [&](int u) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      fs_load_q(a, u, rows, 8 * nt, gq, t4, bq, fac[nt]);
      if constexpr (NT == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) reinterpret_cast<uint2*>(&my_q[i][lane])[nt] = make_uint2(bq[i][0], bq[i][1]);
      }
    }
    __syncwarp();
  };
  if (first_unit >= 0) load_q(first_unit);  // while the first pages come
  bool failed = false;

  // Adds the state in a merge area to this warp's.  An area has O's fragments, four floats a lane, then M and l
  // of the rows.
  auto absorb = [&](const float* area) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float fa[2], fb[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * t4 + e;
        const float mo = area[NT * 1024 + r], lo = area[NT * 1024 + S::kRows + r];
        const float mn = fmaxf(m_run[nt][e], mo);
        fa[e] = mn == -INFINITY ? 1.f : ex2(m_run[nt][e] - mn);
        fb[e] = mn == -INFINITY ? 1.f : ex2(mo - mn);
        m_run[nt][e] = mn;
        l_run[nt][e] = l_run[nt][e] * fa[e] + lo * fb[e];
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        const float4 v = reinterpret_cast<const float4*>(area)[(nt * 8 + mt) * 32 + lane];
        o[nt][mt][0] = o[nt][mt][0] * fa[0] + v.x * fb[0];
        o[nt][mt][1] = o[nt][mt][1] * fa[1] + v.y * fb[1];
        o[nt][mt][2] = o[nt][mt][2] * fa[0] + v.z * fb[0];
        o[nt][mt][3] = o[nt][mt][3] * fa[1] + v.w * fb[1];
      }
    }
    __syncwarp();
  };
  auto leave = [&](float* area) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
        reinterpret_cast<float4*>(area)[(nt * 8 + mt) * 32 + lane] =
            make_float4(o[nt][mt][0], o[nt][mt][1], o[nt][mt][2], o[nt][mt][3]);
      if (gq == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          area[NT * 1024 + 8 * nt + 2 * t4 + e] = m_run[nt][e];
          area[NT * 1024 + S::kRows + 8 * nt + 2 * t4 + e] = l_run[nt][e];
        }
      }
    }
    __syncwarp();
  };

  // The unit's state: warps 2 and 3 hand theirs to 0 and 1, warp 1 hands the sum to 0, which writes.
  auto finalize = [&]() -> bool {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l_run[nt][e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        l_run[nt][e] = v;
      }
    const uint32_t parity = units_done & 1;
    if (wt >= 2 && units_done > 0 && !mbar_wait_warp(&tm->freed, parity ^ 1)) return false;
#pragma unroll 1
    for (int k = wt; k < 2; ++k) {  // warp 0: of warps 2 and 1; warp 1: of warp 3
      if (!mbar_wait_warp(k == wt ? &tm->pair : &tm->last, parity)) return false;
      absorb(sh->merge[team][k]);
    }
    if (wt != 0) {
      leave(sh->merge[team][wt & 1]);
      if (lane == 0) mbar_arrive(wt == 1 ? &tm->last : &tm->pair);
      return true;
    }
    if (lane == 0) mbar_arrive(&tm->freed);
    // whole, or cut by a range boundary?
    int64_t u0, u1;
    if (sparse) {
      u0 = static_cast<int64_t>(unit) * kTopK;
      u1 = u0 + kTopK;
    } else {
      const int b = unit / a.groups, nb = sh->prefix[b + 1] - sh->prefix[b];
      u0 = static_cast<int64_t>(sh->prefix[b]) * a.groups + static_cast<int64_t>(unit % a.groups) * nb;
      u1 = u0 + nb;
    }
    const bool whole = u0 >= x0 && u1 <= x1;
    float* part = a.partial + (2 * static_cast<int64_t>(tt) + (x0 > u0 ? 0 : 1)) * S::kSlotFloats;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * t4 + e;
        if (r >= rows) continue;
        const float m = m_run[nt][e], l = l_run[nt][e];
        if (whole) {
          const bool any = l != 0.f;  // (NaN counts as any)
          const float inv = any ? 1.f / l : 0.f;
          const int64_t token = sparse ? unit / a.groups : static_cast<int64_t>(unit / a.groups) * T + r / Hg;
          const int64_t hr = token * a.groups * Hg + unit % a.groups * Hg + r % Hg;
          uint32_t w[8];
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(o[nt][mt][e] * inv, o[nt][mt][2 + e] * inv);
            w[mt] = *reinterpret_cast<const uint32_t*>(&h);
          }
          uint4* dst = reinterpret_cast<uint4*>(a.out + hr * kDim + 16 * gq);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
          if (gq == 0) {
            if (a.lse != nullptr) a.lse[hr] = fp8_lse(m, l);
            if (a.weight_out != nullptr) a.row_stat[static_cast<int64_t>(unit) * rows + r] = make_float2(any ? m : 0.f, inv);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(part + r * kDim + 16 * gq);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_float4(o[nt][2 * i][e], o[nt][2 * i][2 + e], o[nt][2 * i + 1][e], o[nt][2 * i + 1][2 + e]);
          if (gq == 0) {
            part[S::kRows * kDim + r] = m;
            part[S::kRows * (kDim + 1) + r] = l;
          }
        }
      }
    return true;
  };

  for (int item = 0;; ++item) {
    const int ku = 2 * item, kslot = ku % S::kSlots, vu = ku + 1, vslot = vu % S::kSlots;
    if (!mbar_wait_warp(&tm->full[kslot], (ku / S::kSlots) & 1)) {
      failed = true;
      break;
    }
    const FsItem it = tm->item[item % kFsMeta];
    if (it.unit != unit) {
      if (unit >= 0) {
        if (!finalize()) {
          failed = true;
          break;
        }
        ++units_done;
      }
      unit = it.unit;
      if (unit >= 0) {
        if (unit != first_unit) load_q(unit);
        pos_min = it.pos;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            m_run[nt][e] = z_top[nt][e] = -INFINITY;
            l_run[nt][e] = 0.f;
            pos[nt][e] = sparse ? pos_min : pos_min + min((8 * nt + 2 * t4 + e) / Hg, T - 1);
          }
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
        }
      }
    }
    if (it.page < 0) {
      if (unit < 0) break;  // (the end: nothing waits for these slots)
      if (!mbar_wait_warp(&tm->full[vslot], (vu / S::kSlots) & 1)) {
        failed = true;
        break;
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&tm->empty[kslot]);
        mbar_arrive(&tm->empty[vslot]);
      }
      continue;
    }
    const uint8_t* kd = my_slots + kslot * kFp8PageBytes;
    const uint8_t* vd = my_slots + vslot * kFp8PageBytes;
    const int key0 = it.block * kBlock + 32 * wt;  // this warp's first key
    // keys that some row must not see, or that do not exist
    const bool edge = it.block * kBlock + kBlock - 1 > pos_min;

    // ---- S^T = K Q^T
    float s[2][NT][4];
#pragma unroll
    for (int mq = 0; mq < 2; ++mq)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[mq][nt][0] = s[mq][nt][1] = s[mq][nt][2] = s[mq][nt][3] = 0.f;
    if constexpr (NT == 1) {
#pragma unroll
      for (int mq = 0; mq < 2; ++mq) {
        const int r = 32 * wt + 16 * mq + gq;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 u0 = lds128(kd + page_chunk(r, 2 * t4 + h)), u1 = lds128(kd + page_chunk(r + 8, 2 * t4 + h));
          const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(w0[i], a0, a2);
            e4m3x4_to_f16x4(w1[i], a1, a3);
            mma_f16_16816(s[mq][0], a0, a1, a2, a3, bq[4 * h + i][0], bq[4 * h + i][1]);
          }
        }
      }
    } else {
      // the queries' fragments from shared memory, each for both groups of 16 keys: as registers they would
      // not fit beside O
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 u[2][2];
#pragma unroll
        for (int mq = 0; mq < 2; ++mq)
#pragma unroll
          for (int e = 0; e < 2; ++e) u[mq][e] = lds128(kd + page_chunk(32 * wt + 16 * mq + gq + 8 * e, 2 * t4 + h));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 q = lds128(&my_q[4 * h + i][lane]);
#pragma unroll
          for (int mq = 0; mq < 2; ++mq) {
            const uint32_t w0[4] = {u[mq][0].x, u[mq][0].y, u[mq][0].z, u[mq][0].w};
            const uint32_t w1[4] = {u[mq][1].x, u[mq][1].y, u[mq][1].z, u[mq][1].w};
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(w0[i], a0, a2);
            e4m3x4_to_f16x4(w1[i], a1, a3);
            mma_f16_16816(s[mq][0], a0, a1, a2, a3, q.x, q.y);
            mma_f16_16816(s[mq][NT - 1], a0, a1, a2, a3, q.z, q.w);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&tm->empty[kslot]);

    // ---- online softmax on e = s * f + b (the difference with M is taken in one rounding: b and M may be large)
    bool move = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = finite_factor(it.k_scale * fac[nt][e]);
        float m = -INFINITY;
#pragma unroll
        for (int mq = 0; mq < 2; ++mq)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float& z = s[mq][nt][2 * half + e];
            if (edge && key0 + 16 * mq + 8 * half + gq > pos[nt][e]) z = -INFINITY;
            m = fmaxf(m, z);
          }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        m = fmaf(m, f, it.v_exp);  // (f is positive)
        z_top[nt][e] = fmaxf(z_top[nt][e], m - it.v_exp);
        top[nt][e] = z_top[nt][e] + it.v_exp;  // >= m
        move |= top[nt][e] > m_run[nt][e] + kFp8RefMax || top[nt][e] < m_run[nt][e] + kFsRefMin;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (top[nt][e] > m_run[nt][e] + kFp8RefMax || top[nt][e] < m_run[nt][e] + kFsRefMin) {
            const float mn = ceilf(top[nt][e]) - kFsRefSet, alpha = ex2(m_run[nt][e] - mn);
            m_run[nt][e] = mn;
            l_run[nt][e] *= alpha;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              o[nt][mt][e] *= alpha;
              o[nt][mt][2 + e] *= alpha;
            }
          }
    }
    uint32_t pb[2][NT][2];
    const float inv_v = ex2(-it.v_exp);  // (an integer: exact)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float sum[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = finite_factor(it.k_scale * fac[nt][e]);
        const float c0 = it.v_exp - (m_run[nt][e] == -INFINITY ? 0.f : m_run[nt][e]);
        sum[e] = 0.f;
#pragma unroll
        for (int mq = 0; mq < 2; ++mq)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float& z = s[mq][nt][2 * half + e];
            z = ex2(fmaf(z, f, c0));
            sum[e] += z;
          }
        l_run[nt][e] = fmaf(sum[e], inv_v, l_run[nt][e]);
      }
      if (a.weight_out != nullptr) {
        const int64_t place = static_cast<int64_t>(unit) * (sparse ? kTopK : a.max_blocks) + it.place;
        float2* share = a.share + (place * kFp8StreamParts + wt) * rows;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = sum[e];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          const int r = 8 * nt + 2 * t4 + e;
          if (gq == 0 && r < rows)
            share[r] = make_float2(v, (m_run[nt][e] == -INFINITY ? 0.f : m_run[nt][e]) - it.v_exp);
        }
      }
#pragma unroll
      for (int mq = 0; mq < 2; ++mq) {
        pb[mq][nt][0] = movmatrix_trans(pack_f16x2(s[mq][nt][0], s[mq][nt][1]));
        pb[mq][nt][1] = movmatrix_trans(pack_f16x2(s[mq][nt][2], s[mq][nt][3]));
      }
    }

    // ---- O^T += V^T P^T
    if (!mbar_wait_warp(&tm->full[vslot], (vu / S::kSlots) & 1)) {
      failed = true;
      break;
    }
#pragma unroll
    for (int mq = 0; mq < 2; ++mq) {
      const int r = 32 * wt + 16 * mq + 2 * t4;  // rows r, r + 1, r + 8, r + 9
      uint32_t w[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int rj = r + (j & 1) + 8 * (j >> 1);
        const uint4 u = lds128(vd + page_chunk(rj, gq));
        w[j][0] = u.x;
        w[j][1] = u.y;
        w[j][2] = u.z;
        w[j][3] = u.w;
      }
      if (edge) {
        // NaN codes: zero in the product (a hidden key's probability is 0, and 0 * NaN is not), and NaN in
        // the rows that see their key
        uint32_t dims[4];  // of key j: bit i, dim 16 gq + i
        bool found = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dims[j] = 0u;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t nan = __vcmpeq4(w[j][i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
            w[j][i] &= ~nan;
            dims[j] |= (((nan & 0x08040201u) * 0x01010101u) >> 24) << (4 * i);
          }
          found |= dims[j] != 0u;
        }
        if (__any_sync(0xffffffffu, found)) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            for (int c = 0; c < 4; ++c) {
              const uint32_t d = __shfl_sync(0xffffffffu, dims[j], (lane & ~3) | c);
              const int key = key0 + 16 * mq + 2 * c + (j & 1) + 8 * (j >> 1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (key <= pos[nt][e]) {
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                      if (d >> (2 * mt) & 1u) o[nt][mt][e] = NAN;
                      if (d >> (2 * mt + 1) & 1u) o[nt][mt][2 + e] = NAN;
                    }
                  }
            }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // bytes (key r, key r + 1) of dims 16 gq + 4 i and + 1, then + 2 and + 3
        uint32_t a0, a1, a2, a3;
        e4m3x4_to_f16x4(__byte_perm(w[0][i], w[1][i], 0x5140), a0, a1);
        e4m3x4_to_f16x4(__byte_perm(w[2][i], w[3][i], 0x5140), a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][2 * i], a0, a1, a2, a3, pb[mq][nt][0], pb[mq][nt][1]);
        e4m3x4_to_f16x4(__byte_perm(w[0][i], w[1][i], 0x7362), a0, a1);
        e4m3x4_to_f16x4(__byte_perm(w[2][i], w[3][i], 0x7362), a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][2 * i + 1], a0, a1, a2, a3, pb[mq][nt][0], pb[mq][nt][1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&tm->empty[vslot]);
  }
  if (failed && lane == 0) flag_error(a.err, MSA_DEVERR_TIMEOUT);
}

// Units cut by range boundaries: the partial states that their teams left, added (fp8_merge.cuh).
// blockIdx.x is the unit (by_unit) or the boundary whose unit the CTA takes if it is the unit's
// first, whichever is fewer; blockIdx.y the row (kSplit) or eight of them.
template <int NT, bool kSplit>
__global__ void __launch_bounds__(kFp8MergeThreads)
    fp8_stream_merge_kernel(const Fp8AttnArgs a, int teams, int by_unit, int whole) {
  __shared__ Fp8MergeShared sh;
  grid_dependency_wait();
  grid_dependents_launch();
  const bool sparse = a.selection != nullptr;
  const int64_t E = sparse ? static_cast<int64_t>(a.batch) * a.q_len * a.groups * kTopK
                           : static_cast<int64_t>(a.block_prefix[a.batch]) * a.groups;
  int unit = blockIdx.x;
  if (!by_unit) {
    const int xb = fs_lo(E, blockIdx.x + 1, teams);
    if (xb >= E) return;
    unit = fs_entry(a, a.block_prefix, xb).unit;
  }
  int64_t u0, u1;
  if (sparse) {
    u0 = static_cast<int64_t>(unit) * kTopK;
    u1 = u0 + kTopK;
  } else {
    const int b = unit / a.groups, p = a.block_prefix[b], nb = a.block_prefix[b + 1] - p;
    u0 = static_cast<int64_t>(p) * a.groups + static_cast<int64_t>(unit % a.groups) * nb;
    u1 = u0 + nb;
  }
  if (u1 - u0 <= whole) return;  // not cut
  const int ca = fs_owner(E, u0, teams), cb = fs_owner(E, u1 - 1, teams);
  if (ca == cb || (!by_unit && static_cast<int>(blockIdx.x) != ca)) return;  // whole, or another boundary's
  if (threadIdx.x < 32) {  // the teams ca .. cb with a range, in order
    int n = 0;
    for (int c0 = ca; c0 <= cb; c0 += 32) {
      const int c = c0 + threadIdx.x;
      const int lo = fs_lo(E, c, teams);
      const bool some = c <= cb && lo < fs_lo(E, c + 1, teams);
      const unsigned m = __ballot_sync(0xffffffffu, some);
      // the state is in the team's first place if its range begins inside the unit
      if (some) sh.list[n + __popc(m & ((1u << threadIdx.x) - 1u))] = 2 * c + (lo > u0 ? 0 : 1);
      n += __popc(m);
    }
    if (threadIdx.x == 0) sh.n = n;
  }
  __syncthreads();
  const int Hg = a.heads_per_group, rows = sparse ? Hg : a.q_len * Hg;
  const int r = kSplit ? blockIdx.y : blockIdx.y * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  float4 o;
  float M, l;
  const int chunk = threadIdx.x & 31;
  fp8_merge_row<kSplit>(a.partial, FsShape<NT>::kRows, r, r * 32 + chunk, sh, o, M, l);
  if (kSplit && threadIdx.x >= 32) return;
  const int64_t token = sparse ? unit / a.groups : static_cast<int64_t>(unit / a.groups) * a.q_len + r / Hg;
  fp8_write_row(a, token * a.groups * Hg + unit % a.groups * Hg + r % Hg, static_cast<int64_t>(unit) * rows + r, chunk, o,
                M, l);
}

size_t fp8_stream_partial_bytes() {
  const size_t one = static_cast<size_t>(FsShape<1>::kTeams) * FsShape<1>::kSlotFloats;
  const size_t two = static_cast<size_t>(FsShape<2>::kTeams) * FsShape<2>::kSlotFloats;
  return 2 * kFp8MaxCtas * (one > two ? one : two) * sizeof(float);
}

// Pages of a unit up to which it is not cut: a cut costs a merge, about as much as kFsCutPages pages; not cutting
// leaves teams idle, as `all` units on n teams give some ceil(all / n), which for a unit of S pages is idle * S / n
// more than its share.  200 sequences of up to 500 tokens, 4 groups: 29 us whole and 34 cut, with two new tokens (16
// rows) 54 and 63.
static int fs_whole(int64_t all, int n) {
  constexpr int kFsWhole = 32, kFsCutPages = 3;
  const int64_t idle = n - 1 - (all - 1) % n, most = kFsCutPages * static_cast<int64_t>(n);
  const int whole = idle * kFsWhole <= most ? kFsWhole : static_cast<int>(most / idle);
  return whole > kFsCutPages ? whole : 0;
}

template <int NT>
static cudaError_t launch_stream(const Fp8AttnArgs& a, int num_sms, cudaStream_t s) {
  Fp8Maps maps;
  cudaError_t e = fp8_page_maps(a, &maps);
  if (e != cudaSuccess) return e;
  const size_t smem = fs_smem_bytes<NT>();
  if ((e = ensure_dynamic_smem(reinterpret_cast<const void*>(fp8_stream_kernel<NT>), smem)) != cudaSuccess) return e;
  const int ctas = num_sms < kFp8MaxCtas ? num_sms : kFp8MaxCtas, teams = ctas * FsShape<NT>::kTeams;
  const bool sparse = a.selection != nullptr;
  const int64_t units = static_cast<int64_t>(a.batch) * a.groups * (sparse ? a.q_len : 1);
  // (tables of much longer sequences: no search for units to leave whole)
  const int limit = fs_whole(units, teams), whole = (sparse ? kTopK : a.max_blocks) <= 2 * limit ? limit : 0;
  if ((e = launch_dependent(fp8_stream_kernel<NT>, dim3(ctas), FsShape<NT>::kThreads, smem, s, a, maps, whole)) !=
      cudaSuccess)
    return e;
  if ((sparse ? kTopK : a.max_blocks) <= whole) return cudaSuccess;  // no unit is cut
  const int rows = sparse ? a.heads_per_group : a.q_len * a.heads_per_group;
  const int by_unit = units < teams - 1 ? 1 : 0;
  const unsigned grid = by_unit ? static_cast<unsigned>(units) : static_cast<unsigned>(teams - 1);
  return teams / units >= kFp8MergeSplitParts
             ? launch_dependent(fp8_stream_merge_kernel<NT, true>, dim3(grid, rows), kFp8MergeThreads, 0, s, a,
                                teams, by_unit, whole)
             : launch_dependent(fp8_stream_merge_kernel<NT, false>, dim3(grid, (rows + 7) / 8), kFp8MergeThreads, 0, s, a,
                                teams, by_unit, whole);
}

cudaError_t launch_fp8_stream(const Fp8AttnArgs& a, int num_sms, cudaStream_t s) {
  // 9 to 16 rows as two n-tiles: 64 sequences of 32K with 16 rows take 194 us, with 128-row tiles 254 (200 of 500
  // tokens 62 and 71)
  const int rows = a.selection != nullptr ? a.heads_per_group : a.q_len * a.heads_per_group;
  return rows <= 8 ? launch_stream<1>(a, num_sms, s) : launch_stream<2>(a, num_sms, s);
}

}  // namespace msa
