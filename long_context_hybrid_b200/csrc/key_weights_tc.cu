// The attention weight each key of packed prompts got, on the tensor cores.
//
//   w[g, u] = sum over the listed heads h of KV head g and the observed rows t
//             that attend u of exp(scale q[t,h].k[u,g] - lse[h,t]);
// observed are the last n_obs rows of each sequence. With n_obs at least the
// length that is the sum over the whole attention matrix's columns; nothing of
// that matrix leaves the chip.
//
// The scores are formed transposed: a CTA owns 128 keys of one sequence and
// KV head as the rows of S^T = K Q^T (M128 N128 K128), and streams the query
// tiles of every head of the group past them. So a thread owns one key (a
// TMEM lane), its sum stays in registers, and the only exchange is the
// columns' -lse, read as broadcasts from shared memory. One exponential per
// pair against 256 flops makes it bound by the exponential unit (16 a clock
// and SM: 1024 clocks a tile against about 512 for the products).
//
// A cluster of 1 to 8 CTAs shares one set of keys when there are few: each
// takes every n-th query tile, and the sums are added over distributed shared
// memory in the order of the ranks, so no result depends on timing.
//
// Warp roles (384 threads): warp 0 TMA producer (K once, then Q tiles through
// a ring of five), warp 1 TMEM owner and MMA issuer (four 128-column score
// buffers), warps 4-7 and 8-11 two warpgroups that take the tiles in turn.
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

constexpr int kThreads = 384;
constexpr int kTile = 128;
constexpr int kRing = 5;
constexpr int kBufs = 4;
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
  __align__(16) float neg_lse[8][kTile];             // [warp][column], log2 domain; read 16 bytes at a time
  float sum[2][kTile];                               // per warpgroup, read by the cluster
};
static_assert(offsetof(Shared, neg_lse) % 16 == 0, "16-byte reads");
constexpr size_t kSmemBytes = 1024 + kRingOff + kRing * kStage + sizeof(Shared);

}  // namespace

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
  if (!packed_tile(p.cu, p.S, p.T, kTile, unit / p.n_ag, &c0, &n, &k0)) return;   // the whole cluster alike

  // query rows that attend a key of the tile: [q_lo, q_hi), in tiles of 128
  const int obs0 = n - min(n, p.n_obs);
  const int q_lo = max(k0, obs0);
  const int64_t reach = (int64_t)min(k0 + kTile, n) - 1 + p.window;
  const int q_hi = reach < n ? (int)reach : n;
  const int t_lo = q_lo / kTile;
  const int n_q = q_hi > q_lo ? (q_hi - 1) / kTile + 1 - t_lo : 0;
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
      for (int i = 0; i < n_x; ++i) {
        const int s = i % kRing;
        if (i >= kRing && !mbar_wait(smem_u32(&sh.empty[s]), (i / kRing - 1) & 1, abort_flag)) break;
        const int x = rank + i * n_ranks;
        const int h = p.head[p.ag_start[a] + x / n_q], row = c0 + (t_lo + x % n_q) * kTile;
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
    auto fetch = [&](int i) {
      const int x = rank + i * n_ranks;
      const int hh = x / n_q, row0 = (t_lo + x - hh * n_q) * kTile;
      const float* from = p.lse + (int64_t)p.lse_row[p.ag_start[a] + hh] * p.T + c0;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int row = row0 + y * 32 + lane;
        const float l = row < n ? __ldg(from + row) : -INFINITY;
        next[y] = l == -INFINITY ? -INFINITY : l * -1.4426950408889634f;
      }
    };
    float total = 0.f;
    if (n_x > wg) fetch(wg);
    for (int i = wg; i < n_x; i += 2) {
      const int buf = i % kBufs;
      __syncwarp();
#pragma unroll
      for (int y = 0; y < 4; ++y) nl[y * 32 + lane] = next[y];
      __syncwarp();
      if (i + 2 < n_x) fetch(i + 2);
      const int x = rank + i * n_ranks;
      const int q0 = (t_lo + x % n_q) * kTile;
      const bool w = mbar_wait(smem_u32(&sh.s_full[buf]), (i / kBufs) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, w)) break;
      tc_fence_after();
      // some pair of the tile is masked: a query before the tile's last key, not
      // observed or past the end, or a key out of a query's window
      const bool cut = q0 < k0 + kTile - 1 || q0 < obs0 || q0 + kTile > n ||
                       (int64_t)q0 + kTile - 1 - k0 >= p.window;
      const int c_lo = max(u, obs0) - q0;
      const int c_hi = (int)min((int64_t)(n - q0), (int64_t)u + p.window - q0);   // columns [c_lo, c_hi)
      uint64_t acc0 = 0, acc1 = 0;                   // pairs of +0
      auto add_tile = [&](auto is_cut) {
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
          uint32_t v[32];
          tmem_ld32(tmem + lane_off + buf * 128u + c4 * 32u, v);
          tc_wait_ld();
          if (c4 == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.s_empty[buf]));
          }
          const ulonglong2* nl2 = reinterpret_cast<const ulonglong2*>(nl + c4 * 32);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const ulonglong2 l = nl2[c];
            float e[4];
            f2_split(f2_fma(f2(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1])), sc2, l.x), e[0], e[1]);
            f2_split(f2_fma(f2(__uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3])), sc2, l.y), e[2], e[3]);
            if constexpr (decltype(is_cut)::value) {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int col = c4 * 32 + 4 * c + y;
                if (col < c_lo || col >= c_hi) e[y] = -INFINITY;
              }
            }
            acc0 = f2_add(acc0, f2(ex2(e[0]), ex2(e[1])));
            acc1 = f2_add(acc1, f2(ex2(e[2]), ex2(e[3])));
          }
        }
      };
      // two copies: with the mask as selects every tile would pay for it
      if (cut) add_tile(std::true_type{});
      else add_tile(std::false_type{});
      float s0, s1, s2, s3;
      f2_split(acc0, s0, s1);
      f2_split(acc1, s2, s3);
      total += (s0 + s1) + (s2 + s3);
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
      w += s[tid] + s[kTile + tid];
    }
    p.w[(int64_t)g * p.T + c0 + k0 + tid] = w;
  }
  if (n_ranks > 1) cluster.sync();                   // no CTA leaves while its sums may be read
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
  if (!make_tmap_bnhd(&tq, q.p, 1, T, Hq, 0, q.sn, q.sh, kTile) ||
      !make_tmap_bnhd(&tk, k.p, 1, T, Hkv, 0, k.sn, k.sh, kTile))
    return cudaErrorInvalidValue;
  WeightParams p;
  p.cu = cu; p.lse = lse; p.w = weights;
  p.S = S; p.T = T; p.window = window; p.n_obs = n_obs;
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
  const int64_t units = ((int64_t)T / kTile + S) * p.n_ag;
  // few keys: up to eight CTAs share each tile, until about two per SM exist
  int ranks = 1;
  while (ranks < kMaxCluster && units * ranks * 2 <= 296) ranks *= 2;
  return f16 ? launch_typed<true>(p, units, ranks, tq, tk, status, stream)
             : launch_typed<false>(p, units, ranks, tq, tk, status, stream);
}

}  // namespace rtp
