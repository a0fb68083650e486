// The attention weight each key of packed prompts got, on the tensor cores.
//
//   w[g, u] = sum over the listed heads h of KV head g and the observed rows t
//             that attend u of exp(scale q[t,h].k[u,g] - lse[h,t]);
// observed are the last n_obs rows of each sequence. With n_obs at least the
// length that is the sum over the whole attention matrix's columns; nothing of
// that matrix leaves the chip.
//
// The scores are formed transposed: 128 keys of one sequence and KV head are
// the rows of S^T = K Q^T (M128 N128 K128), the queries its columns. So a
// thread owns one key (a TMEM lane), its sum stays in registers, and the only
// exchange is the columns' -lse, read as broadcasts from shared memory. One
// exponential per pair against 256 flops makes it bound by the exponential unit
// (16 a clock and SM: 1024 clocks a tile against about 512 for the products).
//
// Two kernels; which one runs depends on n_obs and the group alone:
//   * few observed rows (those of all the group's heads fit 512 columns): a
//     CTA keeps the queries of a (sequence, KV head) in shared memory and
//     streams key tiles past them, one unit of 128 keys after another; the
//     warpgroups share every tile by columns. The last 64 rows of 4 prompts
//     (40462 tokens, 8 heads a KV head): 46 us, and 119 us by the other kernel,
//     which reads the queries again for every 128 keys;
//   * many: a CTA owns 128 keys and streams the query tiles of every head of
//     the group past them. A cluster of 1 to 8 CTAs shares one set of keys when
//     there are few: each takes every n-th query tile, and the sums are added over
//     distributed shared memory in the order of the ranks, so no result
//     depends on timing.
//
// Warp roles of both (640 threads): warp 0 TMA producer, warp 1 TMEM owner and
// MMA issuer, and four warpgroups that sum, with a 128-column score buffer
// each. (Every row of 6 prompts, 24657 tokens, 32 heads: 930 us with two
// warpgroups of two buffers each, 695 us with four, 685 us with 16 columns on
// their way to registers while 16 are added.)
#include <cooperative_groups.h>
#include <stddef.h>
#include <type_traits>

#include "attn_packed_common.cuh"
#include "paged.cuh"
#include "sm100.cuh"

namespace rtp {
using namespace sm100;
namespace cg = cooperative_groups;

namespace {

constexpr int kGroups = 4;                           // warpgroups that sum, with a score buffer each
constexpr int kThreads = 128 * (1 + kGroups);
constexpr int kTile = 128;
constexpr int kRing = 5;
constexpr int kBufs = kGroups;
constexpr uint32_t kStage = 32768;
constexpr uint32_t kRingOff = kStage;                // behind the K tile
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxCluster = 8;
constexpr int kStatusTimeout = 4;

struct WeightParams {
  const int32_t* cu;
  const float* lse;                                  // [n_heads, T]
  float* w;                                          // [Hkv, T]
  int S, T, window, n_obs, n_ag;
  float scale_log2;
  uint8_t head[kMaxHeads], lse_row[kMaxHeads];       // listed heads, sorted by KV head
  uint8_t ag_kv[kMaxHeads], ag_start[kMaxHeads], ag_n[kMaxHeads];
};

struct Shared {
  uint64_t k_full, full[kRing], empty[kRing], s_full[kBufs], s_empty[kBufs], fin;
  uint32_t tmem_base;
  int abort;
  __align__(16) float neg_lse[4 * kGroups][kTile];   // [warp][column], log2 domain; read 16 bytes at a time
  float sum[kGroups][kTile];                         // per warpgroup, read by the cluster
};
static_assert(offsetof(Shared, neg_lse) % 16 == 0, "16-byte reads");
constexpr size_t kSmemBytes = 1024 + kRingOff + kRing * kStage + sizeof(Shared);

// Adds exp2(s * scale + neg_lse) over 16 columns of scores; where kCut those
// outside [c_lo, c_hi) are left out.
template <bool kCut>
__device__ __forceinline__ void add_chunk(const uint32_t (&v)[16], const float* neg_lse, uint64_t sc2, int c_lo,
                                          int c_hi, uint64_t& acc0, uint64_t& acc1) {
  const ulonglong2* nl2 = reinterpret_cast<const ulonglong2*>(neg_lse);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const ulonglong2 l = nl2[c];
    float e[4];
    f2_split(f2_fma(f2(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1])), sc2, l.x), e[0], e[1]);
    f2_split(f2_fma(f2(__uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3])), sc2, l.y), e[2], e[3]);
    if (kCut) {
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (4 * c + y < c_lo || 4 * c + y >= c_hi) e[y] = -INFINITY;
    }
    acc0 = f2_add(acc0, f2(ex2(e[0]), ex2(e[1])));
    acc1 = f2_add(acc1, f2(ex2(e[2]), ex2(e[3])));
  }
}
__device__ __forceinline__ float sum_pairs(uint64_t acc0, uint64_t acc1) {
  float s0, s1, s2, s3;
  f2_split(acc0, s0, s1);
  f2_split(acc1, s2, s3);
  return (s0 + s1) + (s2 + s3);
}

// The same over the first `cols` columns of a tile, 16 of them on their way
// while 16 are added; `release` is called when the last are in registers.
template <bool kCut, class Release>
__device__ __forceinline__ float sum_tile(uint32_t tmem, const float* neg_lse, uint64_t sc2, int cols, int c_lo,
                                          int c_hi, Release release) {
  uint64_t acc0 = 0, acc1 = 0;                       // pairs of +0
  const int chunks = kCut ? (cols + 31) / 32 : 4;
  uint32_t v[2][16];
  tmem_ld16(tmem, v[0]);
#pragma unroll
  for (int c4 = 0; c4 < 4; ++c4) {
    if (kCut && c4 >= chunks) break;
    tc_wait_ld();
    tmem_ld16(tmem + c4 * 32u + 16u, v[1]);
    add_chunk<kCut>(v[0], neg_lse + c4 * 32, sc2, c_lo - c4 * 32, c_hi - c4 * 32, acc0, acc1);
    tc_wait_ld();
    if (c4 + 1 < chunks) tmem_ld16(tmem + c4 * 32u + 32u, v[0]);
    else release();
    add_chunk<kCut>(v[1], neg_lse + c4 * 32 + 16, sc2, c_lo - c4 * 32 - 16, c_hi - c4 * 32 - 16, acc0, acc1);
  }
  return sum_pairs(acc0, acc1);
}

// Tile x of a unit's list: every query tile of the first head, of the next, ..
struct Spot {
  int head, tile;
  __device__ __forceinline__ Spot(int x, int n_q) : head(n_q > 0 ? x / n_q : 0), tile(n_q > 0 ? x % n_q : 0) {}
  __device__ __forceinline__ void skip(int by, int n_q) {
    tile += by;
    while (tile >= n_q) {
      tile -= n_q;
      ++head;
    }
  }
};

// The 128 threads of summing warpgroup wg meet.
__device__ __forceinline__ void group_sync(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(wg + 1) : "memory"); }

// -lse in the log2 domain; a row that attended nothing weighs nothing.
__device__ __forceinline__ float neg_log2(float l) {
  return l == -INFINITY ? -INFINITY : l * -1.4426950408889634f;
}

}  // namespace

// ---------------------------------------------------------------------------
// Many observed rows
// ---------------------------------------------------------------------------
template <bool F16>
__global__ void __launch_bounds__(kThreads, 1)
key_weights_kernel(const __grid_constant__ WeightParams p, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmK, int* status) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  Shared& sh = *reinterpret_cast<Shared*>(smem + kRingOff + kRing * kStage);
  volatile int* abort_flag = &sh.abort;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), n_ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = blockIdx.x / n_ranks;
  const int a = unit % p.n_ag, g = p.ag_kv[a];
  int c0, n, k0;
  // a wait runs out seconds after its block began, long after this
  if (blockIdx.x == 0 && tid == 0) *status = 0;
  if (!packed_tile<kTile>(p.cu, p.S, p.T, unit / p.n_ag, &c0, &n, &k0)) return;   // the whole cluster alike

  // query rows that attend a key of the tile: [q_lo, q_hi), in tiles of 128 from q_lo
  const int obs0 = n - min(n, p.n_obs);
  const int q_lo = max(k0, obs0);
  const int q_hi = min(n, min(k0 + kTile, n) - 1 + p.window);
  const int n_q = q_hi > q_lo ? (q_hi - q_lo + kTile - 1) / kTile : 0;
  const int n_all = n_q * p.ag_n[a];                 // tiles of every head
  const int n_x = n_all > rank ? (n_all - rank + n_ranks - 1) / n_ranks : 0;   // this CTA's: rank, rank + n_ranks, ...

  if (tid == 0) {
    mbar_init(smem_u32(&sh.k_full), 1);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    for (int s = 0; s < kBufs; ++s) {
      mbar_init(smem_u32(&sh.s_full[s]), 1);
      mbar_init(smem_u32(&sh.s_empty[s]), 4);
    }
    mbar_init(smem_u32(&sh.fin), 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && n_x > 0) {
      tma_prefetch(&tmQ);
      tma_prefetch(&tmK);
      const uint32_t kbar = smem_u32(&sh.k_full);
      mbar_arrive_expect_tx(kbar, kStage);
      tma_load_4d(sb, &tmK, kbar, 0, g, c0 + k0, 0);
      tma_load_4d(sb + 16384, &tmK, kbar, 64, g, c0 + k0, 0);
      int issued = 0;
      Spot at(rank, n_q);
      for (int i = 0; i < n_x; ++i, at.skip(n_ranks, n_q)) {
        const int s = i % kRing;
        if (i >= kRing && !mbar_wait(smem_u32(&sh.empty[s]), (i / kRing - 1) & 1, abort_flag)) break;
        const int h = p.head[p.ag_start[a] + at.head], row = c0 + q_lo + at.tile * kTile;
        const uint32_t dst = sb + kRingOff + s * kStage, bar = smem_u32(&sh.full[s]);
        mbar_arrive_expect_tx(bar, kStage);
        tma_load_4d(dst, &tmQ, bar, 0, h, row, 0);
        tma_load_4d(dst + 16384, &tmQ, bar, 64, h, row, 0);
        issued = i + 1;
      }
      {
        const long long t0 = clock64();
        while (!mbar_try_wait(smem_u32(&sh.fin), 0) && !*abort_flag && clock64() - t0 < kWaitLimitCycles) {
        }
      }
      if (*abort_flag) {
        wait_short(kbar, 0);
        for (int i = max(0, issued - kRing); i < issued; ++i) wait_short(smem_u32(&sh.full[i % kRing]), (i / kRing) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (n_x > 0) {
      const uint32_t on = elect_one();
      const uint64_t k_desc = desc_k_major(sb), q_desc = desc_k_major(sb + kRingOff);
      bool ok = mbar_wait(smem_u32(&sh.k_full), 0, abort_flag);
      for (int i = 0; ok && i < n_x; ++i) {
        const int s = i % kRing, buf = i % kBufs;
        ok = mbar_wait(smem_u32(&sh.full[s]), (i / kRing) & 1, abort_flag) &&
             (i < kBufs || mbar_wait(smem_u32(&sh.s_empty[buf]), (i / kBufs - 1) & 1, abort_flag));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        issue_qk<F16>(on, tmem + buf * 128u, k_desc, q_desc + (uint64_t)s * (kStage >> 4));
        commit_if(on, smem_u32(&sh.s_full[buf]));
        commit_if(on, smem_u32(&sh.empty[s]));
      }
      commit_if(on, smem_u32(&sh.fin));
      wait_short(smem_u32(&sh.fin), 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums
    const int wg = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;            // key within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int u = k0 + r;
    const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
    // Each warp keeps its own copy of a tile's -lse (log2 domain), fetched one
    // tile ahead: lane l holds columns l, l + 32, .. A row that attended nothing
    // weighs nothing.
    float* nl = sh.neg_lse[warp - 4];
    float next[4];
    auto fetch = [&](const Spot& at) {
      const float* from = p.lse + (int64_t)p.lse_row[p.ag_start[a] + at.head] * p.T + c0;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int row = q_lo + at.tile * kTile + y * 32 + lane;
        next[y] = neg_log2(row < n ? __ldg(from + row) : -INFINITY);
      }
    };
    float total = 0.f;
    Spot at(rank + wg * n_ranks, n_q);
    if (n_x > wg) fetch(at);
    for (int i = wg; i < n_x; i += kGroups) {
      const int buf = wg;
      __syncwarp();
#pragma unroll
      for (int y = 0; y < 4; ++y) nl[y * 32 + lane] = next[y];
      __syncwarp();
      const int q0 = q_lo + at.tile * kTile;
      at.skip(kGroups * n_ranks, n_q);
      if (i + kGroups < n_x) fetch(at);
      const bool w = mbar_spin(smem_u32(&sh.s_full[buf]), (i / kBufs) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, w)) break;
      tc_fence_after();
      // some pair of the tile is masked: a query before the tile's last key or past
      // the end, or a key out of a query's window (all observed: q0 >= q_lo)
      const bool cut = q0 < k0 + kTile - 1 || q0 + kTile > q_hi || q0 + kTile - 1 - k0 >= p.window;
      const int cols = min(kTile, q_hi - q0), c_lo = u - q0;
      const int c_hi = min(n, u + p.window) - q0;    // columns [c_lo, c_hi)
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.s_empty[buf]));
      };
      const uint32_t from = tmem + lane_off + buf * 128u;
      // two copies: with the mask as selects every tile would pay for it
      total += cut ? sum_tile<true>(from, nl, sc2, cols, c_lo, c_hi, release)
                   : sum_tile<false>(from, nl, sc2, kTile, 0, kTile, release);
    }
    sh.sum[wg][r] = total;
  }

  // ---- the sums of the warpgroups and ranks, in order; teardown
  tc_fence_before();
  if (n_ranks > 1) cluster.sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && sh.abort) atomicExch(status, kStatusTimeout);
  if (rank == 0 && tid < kTile && k0 + tid < n) {
    float w = 0.f;
    for (int r = 0; r < n_ranks; ++r) {
      const float* s = n_ranks > 1 ? cluster.map_shared_rank(&sh.sum[0][0], r) : &sh.sum[0][0];
      for (int y = 0; y < kGroups; ++y) w += s[y * kTile + tid];
    }
    p.w[(int64_t)g * p.T + c0 + k0 + tid] = w;
  }
  if (n_ranks > 1) cluster.sync();                   // no CTA leaves while its sums may be read
}

// ---------------------------------------------------------------------------
// Few observed rows
// ---------------------------------------------------------------------------
namespace {
constexpr int kHalf = 64;                            // query rows of one head side by side in a tile
constexpr int kMaxHalves = 8;                        // 512 columns: 128 KB of queries
constexpr int kKeyRing = 2;
constexpr uint32_t kKeyOff = kMaxHalves / 2 * kStage;

struct FewShared {
  uint64_t q_full[kMaxHalves / 2], q_empty, full[kKeyRing], empty[kKeyRing], s_full[kBufs], s_empty[kBufs], fin;
  uint32_t tmem_base;
  int abort;
  // of warpgroup w: columns 32 w .. 32 w + 31 of every tile, log2 domain; read 16 bytes at a time
  __align__(16) float neg_lse[kGroups][kMaxHalves / 2 * 32];
  float part[2][kGroups][kTile];                     // sums of a unit (units alternate)
};
static_assert(offsetof(FewShared, neg_lse) % 16 == 0, "16-byte reads");
constexpr size_t kFewSmemBytes = 1024 + kKeyOff + kKeyRing * kStage + sizeof(FewShared);

// A unit: 128 keys of one sequence and KV head against its observed rows.
struct Unit {
  int c0, n, k0, a;                                  // sequence, its first key here, listed KV head
  int obs0, per_head, halves, tiles;                 // first observed row; half tiles of one head and of all; tiles
  bool there, work;                                  // there are such keys; some observed row attends one
};
__device__ __forceinline__ Unit unit_at(const WeightParams& p, int x, int n_numbers) {
  Unit u;
  u.a = x / n_numbers;
  u.there = packed_tile<kTile>(p.cu, p.S, p.T, x - u.a * n_numbers, &u.c0, &u.n, &u.k0);
  const int rows = min(u.n, p.n_obs);
  u.obs0 = u.n - rows;
  u.per_head = (rows + kHalf - 1) / kHalf;
  u.halves = u.per_head * p.ag_n[u.a];
  u.tiles = (u.halves + 1) / 2;
  u.work = u.there && min(u.k0 + kTile, u.n) - 1 + p.window > u.obs0;
  return u;
}
// The unit behind u (number x): most often the next keys of the same sequence.
__device__ __forceinline__ void next_unit(const WeightParams& p, int x, int n_numbers, Unit& u) {
  if (u.there && u.k0 + kTile < u.n) {
    u.k0 += kTile;
    u.work = min(u.k0 + kTile, u.n) - 1 + p.window > u.obs0;
  } else {
    u = unit_at(p, x, n_numbers);
  }
}
}  // namespace

template <bool F16>
__global__ void __launch_bounds__(kThreads, 1)
key_weights_few_kernel(const __grid_constant__ WeightParams p, int n_numbers, int per_cta, int more,
                       const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, int* status) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  FewShared& sh = *reinterpret_cast<FewShared*>(smem + kKeyOff + kKeyRing * kStage);
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // units x0 .. x1 - 1, numbered KV head by KV head, so that neighbours mostly
  // share their queries
  const int b = blockIdx.x, x0 = b * per_cta + min(b, more), x1 = x0 + per_cta + (b < more);
  // a wait runs out seconds after its block began, long after this
  if (blockIdx.x == 0 && tid == 0) *status = 0;

  if (tid == 0) {
    for (int t = 0; t < kMaxHalves / 2; ++t) mbar_init(smem_u32(&sh.q_full[t]), 1);
    mbar_init(smem_u32(&sh.q_empty), 1);
    for (int s = 0; s < kKeyRing; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    for (int s = 0; s < kBufs; ++s) {
      mbar_init(smem_u32(&sh.s_full[s]), 1);
      mbar_init(smem_u32(&sh.s_empty[s]), 4 * kGroups);
    }
    mbar_init(smem_u32(&sh.fin), 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;                       // every column is allocated, so the address is 0

  // Every role walks the same units: m counts those with work, set the changes
  // of queries.
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch(&tmQ);
      tma_prefetch(&tmK);
    }
    int m = 0, set = 0, c0 = -1, a = -1;
    Unit u = {};
    for (int x = x0; x < x1; ++x) {
      next_unit(p, x, n_numbers, u);
      if (!u.work) continue;
      const int s = m % kKeyRing;
      if (m >= kKeyRing) mbar_pass(smem_u32(&sh.empty[s]), (m / kKeyRing - 1) & 1, abort_flag);
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      if (lane == 0) {
        const uint32_t dst = sb + kKeyOff + s * kStage, bar = smem_u32(&sh.full[s]);
        const int g = p.ag_kv[u.a], row = u.c0 + u.k0;
        mbar_arrive_expect_tx(bar, kStage);
        tma_load_4d(dst, &tmK, bar, 0, g, row, 0);
        tma_load_4d(dst + 16384, &tmK, bar, 64, g, row, 0);
      }
      ++m;
      if (u.c0 != c0 || u.a != a) {
        if (set > 0) mbar_pass(smem_u32(&sh.q_empty), (set - 1) & 1, abort_flag);
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        if (lane == 0) {
          const int start = p.ag_start[u.a];
          for (int f = 0, j = 0, part = 0; f < u.halves; ++f) {
            const uint32_t bar = smem_u32(&sh.q_full[f >> 1]), dst = sb + (f >> 1) * kStage + (f & 1) * 8192u;
            const int h = p.head[start + j], row = u.c0 + u.obs0 + part * kHalf;
            if (!(f & 1)) mbar_arrive_expect_tx(bar, f + 1 < u.halves ? kStage : kStage / 2);
            tma_load_4d(dst, &tmQ, bar, 0, h, row, 0);
            tma_load_4d(dst + 16384, &tmQ, bar, 64, h, row, 0);
            if (++part == u.per_head) { part = 0; ++j; }
          }
          for (int t = u.tiles; t < kMaxHalves / 2; ++t) mbar_arrive(smem_u32(&sh.q_full[t]));   // nothing there
        }
        c0 = u.c0;
        a = u.a;
        ++set;
      }
    }
    if (lane == 0) {
      const long long t0 = clock64();
      while (!mbar_try_wait(smem_u32(&sh.fin), 0) && !*abort_flag && clock64() - t0 < kWaitLimitCycles) {
      }
      if (*abort_flag) {
        for (int t = 0; t < kMaxHalves / 2; ++t)
          if (set > 0) wait_short(smem_u32(&sh.q_full[t]), (set - 1) & 1);
        for (int i = max(0, m - kKeyRing); i < m; ++i)
          wait_short(smem_u32(&sh.full[i % kKeyRing]), (i / kKeyRing) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t on = elect_one();
    const uint64_t k_desc = desc_k_major(sb + kKeyOff), q_desc = desc_k_major(sb);
    int m = 0, set = 0, c0 = -1, a = -1;
    int i = 0;                                       // tiles
    bool fresh = false;                              // queries that no product has read yet
    Unit u = {};
    for (int x = x0; x < x1; ++x) {
      next_unit(p, x, n_numbers, u);
      if (!u.work) continue;
      if (u.c0 != c0 || u.a != a) {
        if (set > 0) commit_if(on, smem_u32(&sh.q_empty));     // the old queries' products are done
        c0 = u.c0;
        a = u.a;
        ++set;
        fresh = true;
      }
      const int s = m % kKeyRing;
      mbar_pass(smem_u32(&sh.full[s]), (m / kKeyRing) & 1, abort_flag);
      const uint64_t k_d = k_desc + (uint64_t)s * (kStage >> 4);
      for (int t = 0; t < u.tiles; ++t, ++i) {
        const int buf = i % kBufs;
        if (i >= kBufs) mbar_pass(smem_u32(&sh.s_empty[buf]), (i / kBufs - 1) & 1, abort_flag);
        if (fresh) mbar_pass(smem_u32(&sh.q_full[t]), (set - 1) & 1, abort_flag);
        tc_fence_after();
        const uint64_t q_d = q_desc + (uint64_t)t * (kStage >> 4);
        if (2 * t + 1 < u.halves) issue_qk<F16>(on, tmem + buf * 128u, k_d, q_d);
        else issue_qk<F16, 64>(on, tmem + buf * 128u, k_d, q_d);
        commit_if(on, smem_u32(&sh.s_full[buf]));
      }
      commit_if(on, smem_u32(&sh.empty[s]));
      fresh = false;
      ++m;
    }
    commit_if(on, smem_u32(&sh.fin));
    wait_short(smem_u32(&sh.fin), 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums
    const int wg = (warp - 4) >> 2;                  // takes columns 32 wg .. 32 wg + 31 of every tile
    const int r = (warp & 3) * 32 + lane;            // key within the tile = TMEM lane
    const uint32_t from = ((uint32_t)((warp & 3) * 32) << 16) + wg * 32u;
    const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
    float* nl = sh.neg_lse[wg];
    int m = 0, c0 = -1, a = -1, i = 0;
    bool ok = true;              // after a wait that ran out a warp still meets the others at every barrier
    Unit u = {};
    for (int x = x0; x < x1; ++x) {
      next_unit(p, x, n_numbers, u);
      if (!u.there) continue;
      const int key = u.k0 + r;
      if (!u.work) {                                 // nothing attends these keys
        if (wg == 0 && key < u.n) p.w[(int64_t)p.ag_kv[u.a] * p.T + u.c0 + key] = 0.f;
        continue;
      }
      if (u.c0 != c0 || u.a != a) {
        c0 = u.c0;
        a = u.a;
        // thread r: column 32 wg + r % 32 of tile r / 32
        const int f = r / 32 * 2 + (wg >> 1), row = u.obs0 + f % u.per_head * kHalf + (wg & 1) * 32 + r % 32;
        const float l = f < u.halves && row < u.n
                            ? __ldg(p.lse + (int64_t)p.lse_row[p.ag_start[a] + f / u.per_head] * p.T + c0 + row)
                            : -INFINITY;
        group_sync(wg);                              // every warp is done with the old ones
        nl[r] = neg_log2(l);
        group_sync(wg);
      }
      uint64_t acc0 = 0, acc1 = 0;                   // pairs of +0
      // Queries q0 .. q0 + 31 are this warpgroup's columns of a tile (at: of its
      // head's rows). 16 columns are on their way while 16 are added.
      int at = (wg >> 1) * kHalf;
      const int per_head = u.per_head * kHalf;
      auto mine = [&](int t) {                       // some column is an observed row
        while (at >= per_head) at -= per_head;
        return 2 * t + (wg >> 1) < u.halves && u.obs0 + at + (wg & 1) * 32 < u.n;
      };
      auto ready = [&](int x) {
        const bool w = ok && mbar_spin(smem_u32(&sh.s_full[x % kBufs]), (x / kBufs) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, w);
        tc_fence_after();
      };
      uint32_t v[2][16];
      bool here = u.tiles > 0 && mine(0);
      ready(i);
      if (here) tmem_ld16(tmem + from + i % kBufs * 128u, v[0]);
      for (int t = 0; t < u.tiles; ++t, ++i) {
        const int q0 = u.obs0 + at + (wg & 1) * 32;
        const bool cut = q0 < u.k0 + kTile - 1 || q0 + 32 > u.n || q0 + 31 - u.k0 >= p.window;
        const int c_hi = min(u.n, key + p.window) - q0;
        const bool now = here;
        // two copies: with the mask as selects every tile would pay for it
        auto add = [&](int half) {
          if (cut) add_chunk<true>(v[half], nl + t * 32 + half * 16, sc2, key - q0 - half * 16, c_hi - half * 16, acc0, acc1);
          else add_chunk<false>(v[half], nl + t * 32 + half * 16, sc2, 0, 16, acc0, acc1);
        };
        tc_wait_ld();
        if (now) {
          tmem_ld16(tmem + from + i % kBufs * 128u + 16u, v[1]);
          add(0);
        }
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.s_empty[i % kBufs]));
        if (t + 1 < u.tiles) {
          at += 2 * kHalf;
          here = mine(t + 1);
          ready(i + 1);
          if (here) tmem_ld16(tmem + from + (i + 1) % kBufs * 128u, v[0]);
        }
        if (now) add(1);
      }
      // the warpgroups' sums, added in their order by each in turn
      float(*part)[kTile] = sh.part[m & 1];
      part[wg][r] = sum_pairs(acc0, acc1);
      asm volatile("bar.sync 5, %0;" ::"n"(128 * kGroups) : "memory");
      if (ok && m % kGroups == wg && key < u.n) {
        float total = 0.f;
#pragma unroll
        for (int y = 0; y < kGroups; ++y) total += part[y][r];
        p.w[(int64_t)p.ag_kv[u.a] * p.T + u.c0 + key] = total;
      }
      ++m;
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && sh.abort) atomicExch(status, kStatusTimeout);
}

template <bool F16>
static cudaError_t launch_typed(const WeightParams& p, int64_t units, int ranks, const CUtensorMap& tq,
                                const CUtensorMap& tk, int* status, cudaStream_t stream) {
  cudaError_t e =
      cudaFuncSetAttribute(key_weights_kernel<F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_weights_kernel<F16>, p, tq, tk, status);
}

cudaError_t launch_key_weights(const Tensor4& q, const Tensor4& k, bool f16, int T, int Hq, int Hkv,
                               const int32_t* heads, int n_heads, const int32_t* cu, int S, const float* lse,
                               int n_obs, int window, float scale, float* weights, int* status, cudaStream_t stream) {
  CUtensorMap tq, tk;
  if (!make_tmap_bnhd(&tk, k.p, 1, T, Hkv, 0, k.sn, k.sh, kTile)) return cudaErrorInvalidValue;
  WeightParams p;
  p.cu = cu; p.lse = lse; p.w = weights;
  p.S = S; p.T = T; p.window = window < T ? window : T; p.n_obs = n_obs;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.n_ag = 0;
  const int G = Hq / Hkv;
  int m = 0;
  for (int g = 0; g < Hkv; ++g) {
    const int start = m;
    for (int j = 0; j < n_heads; ++j)
      if (heads[j] / G == g) {
        p.head[m] = (uint8_t)heads[j];
        p.lse_row[m++] = (uint8_t)j;
      }
    if (m == start) continue;
    p.ag_kv[p.n_ag] = (uint8_t)g;
    p.ag_start[p.n_ag] = (uint8_t)start;
    p.ag_n[p.n_ag++] = (uint8_t)(m - start);
  }
  const int64_t n_numbers = (int64_t)T / kTile + S, units = n_numbers * p.n_ag;
  int most = 0;                                      // listed heads of a KV head
  for (int a = 0; a < p.n_ag; ++a) most = p.ag_n[a] > most ? p.ag_n[a] : most;
  const int rows = n_obs < T ? n_obs : T;
  if ((int64_t)most * ((rows + kHalf - 1) / kHalf) <= kMaxHalves) {
    if (!make_tmap_bnhd(&tq, q.p, 1, T, Hq, 0, q.sn, q.sh, kHalf)) return cudaErrorInvalidValue;
    auto kernel = f16 ? key_weights_few_kernel<true> : key_weights_few_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSmemBytes);
    if (e != cudaSuccess) return e;
    const int n_units = (int)units, grid = n_units < 148 ? n_units : 148;   // (fits: checked with the arguments)
    kernel<<<grid, kThreads, kFewSmemBytes, stream>>>(p, (int)n_numbers, n_units / grid, n_units % grid, tq, tk, status);
    return cudaGetLastError();
  }
  if (!make_tmap_bnhd(&tq, q.p, 1, T, Hq, 0, q.sn, q.sh, kTile)) return cudaErrorInvalidValue;
  // few keys: up to eight CTAs share each tile, until about two per SM exist
  int ranks = 1;
  while (ranks < kMaxCluster && units * ranks * 2 <= 296) ranks *= 2;
  return f16 ? launch_typed<true>(p, units, ranks, tq, tk, status, stream)
             : launch_typed<false>(p, units, ranks, tq, tk, status, stream);
}

}  // namespace rtp
