// Causal attention of packed prompts on the 5th-generation tensor cores
// (tcgen05 + TMEM + TMA): sequences of any lengths one behind the other, each
// head over its whole prefix or its last `window` keys.
//
//   o[t] = sum_u p_u v_u,  p_u = exp(scale q[t].k[u] - lse[t]),
//   u in t's sequence, u <= t, t - u < window.
//
// A unit of work is 256 consecutive query rows of one sequence and head, or 128
// where rows have few keys (Cfg below), against tiles of 128 keys aligned to the
// sequence's start. The lengths stay on the device: the grid covers every tile
// number that any lengths could need, a block is one number of one head, and its
// sequence is found by a search of the offsets; numbers run downwards, so that
// within a sequence the rows with most keys start first. A CTA that has issued
// its unit's copies asks for a block of the grid that has not started
// (clusterlaunchcontrol) and goes on with its work, so the next unit's search,
// copies and first scores run under the last tiles and the output of the one
// before, and nothing is kept in memory between calls. (One unit a CTA: 700 us
// against 610 for 16 prompts of 64 to 8190 tokens, 32 heads, window 1024; 74
// against 51 for 64 x 128 tokens, 32 heads.)
//
// One prompt of 32768 tokens, 32 heads: 7.3 to 7.9 ms, 1.11 to 1.2 PFLOP/s, at
// about 1.6 GHz under the power limit. Bound by the chain of a unit: scores,
// softmax, product, about 3300 clocks a key tile for both query tiles, of which
// the exponentials are 2048 and the products 2048; 4230 with a window of 1024,
// where 40% of the key tiles are cut by a mask and a unit has few of them.
//
// Warp roles (384 threads; of 256 with one query tile):
//   warp 0     producer: finds units, hands them to the other warps through two
//              slots, and issues the TMA copies: Q tiles, then K and V tiles (32
//              KB each, 128-byte swizzle) through a ring of two key tiles;
//   warp 1     TMEM owner and MMA issuer: S_t = Q_t K^T (M128 N128 K128) and
//              O_t += P_t V (P from TMEM, where it takes the place of S; V
//              MN-major) in the order PV0 QK0' PV1 QK1', so that one query
//              tile's products run under the other's softmax. The product with
//              a tile's first 64 keys starts while the softmax works on the
//              other 64. A query tile takes only the key tiles that it attends;
//   warps 2, 3 V guard: in key tiles that a mask cuts, rows behind the sequence's
//              end and non-finite values are zeroed before the product (there
//              P is 0, and 0 * NaN would reach rows that do not attend the
//              key); the epilogue puts non-finite values back into the rows
//              that do attend them;
//   warps 4-11 softmax, one warpgroup per query tile, one row per thread:
//              running maximum in the log2 domain with lazy rescaling of O (only
//              when the maximum grows by more than 8, so P stays below 2^8, within the
//              range of both 16-bit types), row sum in fp32 from the
//              unrounded exponentials, P rounded to the input type over S in TMEM.
// Every wait on an mbarrier is bounded, as in the other tensor-core kernels; a
// cluster's barriers are reached on every path.
#include <cstddef>
#include <type_traits>

#include "attn_packed_common.cuh"
#include "paged.cuh"
#include "sm100.cuh"

namespace rtp {
using namespace sm100;

namespace {

constexpr int kKeyTile = 128;
constexpr uint32_t kStage = 32768;                   // one K or V tile: [D half][128 rows][128 B]
// A CTA of NQ query tiles. Two: one CTA an SM, each key tile read once for both.
// One, with a ring of one key tile: two CTAs an SM, so that one computes while
// the other begins or ends, for units of few keys. Measured, us with two tiles
// and with one: 48 prompts of 16 tokens, 8 heads 18, 13; 32 heads 55, 34; 64 x 128
// tokens 72, 52; 64 x 200 123, 113; 32 x 256 67, 62; 16 x 500 82, 76; 8 x 1000 101,
// 101; a prompt of 4000 among 60 of 20 189, 170; windows over 32768 tokens, 8
// heads: 64 keys 74, 73; 256 96, 88; 512 119, 119; 1024 170, 183; over 4096 tokens,
// 4 heads: 64 14, 11; 512 20, 18; 1024 24, 26.
template <int NQ>
struct Cfg {
  static constexpr int kThreads = 128 + 128 * NQ;
  static constexpr int kTileRows = 128 * NQ;         // query rows of a CTA
  static constexpr int kRing = 2 * NQ;               // even stages hold K, odd ones V
  static constexpr uint32_t kRingOff = NQ * kStage;  // behind the Q tiles
  static constexpr uint32_t kTmemCols = 256 * NQ;    // tile t: S at 256 t, O at 256 t + 128
  static constexpr int kOutCols = 32 * NQ;           // columns of O that a softmax warp lays out at once
  static constexpr uint32_t kOutOff = kRingOff + kRing * kStage;
  static constexpr uint32_t kOutWarp = 32 * kOutCols * 2;
  static constexpr uint32_t kBarsOff = kOutOff + 4 * NQ * kOutWarp;
};
constexpr int kFewKeys = 512;                        // of a row: its window, or the prompts' mean length
constexpr int kSMs = 148;
constexpr int kMaxMisses = 256;
constexpr int kStatusTimeout = 4;
// Few units: the CTAs of a cluster split the key tiles of one. At the end each
// query tile's partials (64 KB and a maximum and sum a row) go to the CTA whose
// rank is the tile's number, over distributed shared memory, into the space of
// the query tiles and the ring.
constexpr int kMaxRanks = 3;
constexpr uint32_t kPartial = 65536;
constexpr uint32_t kMergedSumsOff = (kMaxRanks - 1) * kPartial;       // float2 [rank slot][row]
struct PackedParams {
  void* o; int64_t o_sn, o_sh;
  const void* v; int64_t v_sn, v_sh;                 // for the epilogue's non-finite values
  const int32_t* cu;
  float* lse;                                        // [n_heads, T] or NULL
  int S, T, G, window, n_heads;
  int ranks;                                         // CTAs that share a unit's keys (a cluster): 1 to kMaxRanks
  int64_t n_numbers;                                 // tile numbers: floor(T / rows of a CTA) + S
  float scale_log2;
  uint8_t head[kMaxHeads];
};

// A unit of work: query rows row0 .. of a sequence [c0, c0 + n) and head h, the
// jh-th listed one, of KV head g.
struct __align__(8) Place {
  int c0, n, row0, jh, h, g;                         // n < 0: no more units
};
// What it takes from the keys: tiles kt_lo .. kt_lo + n_tiles - 1 (of 128 keys);
// query tile t takes those of [first[t], last[t]), counted from kt_lo.
template <int NQ>
struct Unit : Place {
  int first[NQ], last[NQ], kt_lo, n_tiles, kt_all, n_all;
  __device__ __forceinline__ Unit(const Place& at, int window, int ranks, int rank) : Place(at) {
    kt_lo = kt_all = max(0, row0 - window + 1) / kKeyTile;
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      const int r = row0 + t * 128;
      const bool any = r < n;
      first[t] = any ? max(0, r - window + 1) / kKeyTile - kt_lo : 0;
      last[t] = any ? min(n - 1, r + 127) / kKeyTile + 1 - kt_lo : 0;
    }
    n_tiles = n_all = max(last[0], last[NQ - 1]);
    if (ranks > 1) {                                 // this rank's part of them
      const int lo = rank * n_all / ranks, hi = (rank + 1) * n_all / ranks;
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        first[t] = min(max(first[t], lo), hi) - lo;
        last[t] = max(min(max(last[t], lo), hi) - lo, first[t]);
      }
      kt_lo += lo;
      n_tiles = hi - lo;
    }
  }
  // whether some row of the unit does not attend some key of a tile
  __device__ __forceinline__ bool masked(int kt, int window) const {
    const int k0 = kt * kKeyTile, row_last = min(n - 1, row0 + 128 * NQ - 1);
    return k0 + kKeyTile - 1 > row0 || k0 <= row_last - window;
  }
};

template <int NQ>
struct Bars {
  static constexpr int kRing = Cfg<NQ>::kRing;
  uint4 next;                                        // the answer to a request for another block's work
  uint64_t next_full, unit_full[2], unit_free[2];
  uint64_t q_full[NQ], q_free[NQ], full[kRing], empty[kRing], v_ok[kRing];
  uint64_t s_full[NQ], p_full[NQ][2], o_full[NQ], fin;   // p_full[query tile][64-key half]
  Place unit[2];                                     // units take turns
  int poison[2];                                     // the guard met a non-finite value of the unit's keys
  uint32_t tmem_base;
  int found;                                         // the CTA's own block had work; set before the roles part
  int abort;
};

template <int NQ>
constexpr size_t kSmemBytes = 1024 + Cfg<NQ>::kBarsOff + sizeof(Bars<NQ>);

// The first two warps meet: one has made the barriers, the other found its unit.
__device__ __forceinline__ void barriers_ready() { asm volatile("bar.sync 1, 64;" ::: "memory"); }

// Asks for a block of the grid that has not started, to do its work here: 16
// bytes come to `to` and complete on `bar`.
__device__ __forceinline__ void ask_for_block(uint32_t to, uint32_t bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to),
               "r"(bar)
               : "memory");
}
// The block's number, or -1 where there was none left.
__device__ __forceinline__ int block_given(uint32_t at) {
  int x;
  asm volatile(
      "{\n\t.reg .b128 answer;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 answer, [%1];\n\t"
      "mov.b32 %0, -1;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, answer;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, answer;\n\t}"
      : "=r"(x)
      : "r"(at)
      : "memory");
  fence_proxy_async_smem();                          // read before the next answer is written
  return x;
}

// The n lowest bits, of any n.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Halves of a pair whose exponent is all ones, as bits 15 and 31.
template <bool F16>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) {
  return F16 ? ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u : ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

}  // namespace

template <bool F16, int NQ>
__global__ void __launch_bounds__(Cfg<NQ>::kThreads, NQ == 2 ? 1 : 2)
attn_packed_kernel(const __grid_constant__ PackedParams p, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, int* status) {
  using C = Cfg<NQ>;
  constexpr int kRing = C::kRing;
  constexpr uint32_t kRingOff = C::kRingOff;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  Bars<NQ>& bars = *reinterpret_cast<Bars<NQ>*>(smem + C::kBarsOff);
  volatile int* abort_flag = &bars.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ranks = NQ == 2 ? p.ranks : 1, rank = blockIdx.x % ranks;
  const int window = p.window;

  // producer's state: the unit at hand, its items issued, all items and Q tiles issued
  Place at = {};
  int r = 0, items = 0, n_q[NQ] = {};
  bool have = false;
  // the place of a block's work; false where its tile number is none (the whole warp, all ranks alike)
  auto find = [&](int unit) {
    // a wait runs out seconds after its block began, long after this
    if (unit == 0 && rank == 0 && lane == 0) *status = 0;
    at.jh = unit % p.n_heads;
    at.h = p.head[at.jh];
    at.g = at.h / p.G;
    return packed_tile<C::kTileRows>(p.cu, p.S, p.T, p.n_numbers - 1 - unit / p.n_heads, &at.c0, &at.n, &at.row0);
  };
  auto copy_q = [&](const Unit<NQ>& u, int t) {
    const uint32_t bar = smem_u32(&bars.q_full[t]);
    mbar_arrive_expect_tx(bar, kStage);
    tma_load_4d(sb + t * kStage, &tmQ, bar, 0, u.h, u.c0 + u.row0 + t * 128, 0);
    tma_load_4d(sb + t * kStage + 16384, &tmQ, bar, 64, u.h, u.c0 + u.row0 + t * 128, 0);
    ++n_q[t];
  };
  auto copy_kv = [&](const Unit<NQ>& u) {            // item 2j of a unit is K of its tile j, 2j + 1 V
    const int s = items % kRing;
    const uint32_t dst = sb + kRingOff + s * kStage, bar = smem_u32(&bars.full[s]);
    const CUtensorMap* map = (r & 1) ? &tmV : &tmK;
    const int key = u.c0 + (u.kt_lo + (r >> 1)) * kKeyTile;
    mbar_arrive_expect_tx(bar, kStage);
    tma_load_4d(dst, map, bar, 0, u.g, key, 0);
    tma_load_4d(dst + 16384, map, bar, 64, u.g, key, 0);
    ++r, ++items;
  };
  // the same once the space is free
  auto load_q = [&](const Unit<NQ>& u, int t) {
    if (u.last[t] <= u.first[t]) return true;
    if (n_q[t] > 0 && !mbar_wait(smem_u32(&bars.q_free[t]), (n_q[t] - 1) & 1, abort_flag)) return false;
    copy_q(u, t);
    return true;
  };
  auto load_kv = [&](const Unit<NQ>& u) {
    if (items >= kRing && !mbar_wait(smem_u32(&bars.empty[items % kRing]), (items / kRing - 1) & 1, abort_flag))
      return false;
    copy_kv(u);
    return true;
  };
  if (warp == 1) {
    // every barrier by a lane of its own
    using B = Bars<NQ>;
    constexpr int kFirst = offsetof(B, next_full) / 8, kLast = offsetof(B, fin) / 8;
    static_assert(kLast - kFirst < 32, "a lane each");
    const int x = kFirst + lane;
    auto of = [&](size_t offset, int count) { return x >= (int)(offset / 8) && x < (int)(offset / 8) + count; };
    if (x <= kLast)
      mbar_init(smem_u32(&bars) + x * 8, of(offsetof(B, unit_free), 2) ? 3 + 4 * NQ
                                         : of(offsetof(B, v_ok), kRing) ? 2
                                         : of(offsetof(B, p_full), 2 * NQ) ? 4 : 1);
    if (lane == 0) {
      bars.abort = 0;
      bars.poison[0] = bars.poison[1] = 0;
    }
    fence_mbar_init();
    barriers_ready();
    tmem_alloc(smem_u32(&bars.tmem_base), C::kTmemCols);
    tmem_relinquish();
  } else if (warp == 0) {
    have = find(blockIdx.x / ranks);
    barriers_ready();
    if (lane == 0) {
      bars.found = have;
      if (have) {
        // the first copies need nothing else: on their way under the rest of the prologue
        const Unit<NQ> u(at, window, ranks, rank);
        if (u.last[0] > u.first[0]) copy_q(u, 0);
        if (u.n_tiles > 0) copy_kv(u);
        if (NQ == 2 && u.last[NQ - 1] > u.first[NQ - 1]) copy_q(u, NQ - 1);
        while (r < min(kRing, 2 * u.n_tiles)) copy_kv(u);
        bars.unit[0] = at;
        mbar_arrive(smem_u32(&bars.unit_full[0]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // with every column allocated the address is 0, known without a load
  const uint32_t tmem = NQ == 2 ? 0u : bars.tmem_base;
  const bool meets = ranks > 1 && bars.found;        // the cluster joins its parts
  // the m-th unit; false at the end or after a wait that ran out (the whole warp)
  auto take = [&](int m, Place& place) {
    const bool w = mbar_spin(smem_u32(&bars.unit_full[m & 1]), (m >> 1) & 1, abort_flag);
    if (!__all_sync(0xffffffffu, w)) return false;
    place = bars.unit[m & 1];
    return place.n >= 0;
  };
  auto release = [&](int m) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.unit_free[m & 1]));
  };
  // A softmax thread holds its row of 128 scores: 128 * (56 + 2 * 224) registers
  // of the launch's 384 * 168, or 128 * (56 + 200) of its 256 * 128.
  if (warp < 4) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
   if (warp == 0) {
    // ------------------------------------------------------------ producer
    // Where clusters do not split units, a CTA goes on with the work of blocks
    // that have not started: its next unit's copies and first scores run under
    // the last tiles and the output of the one before.
    bool fine = true;
    int asked = 0, told = 0, misses = 0, m = have ? 1 : 0;   // m units handed out
    auto ask = [&] {
      ask_for_block(smem_u32(&bars.next), smem_u32(&bars.next_full));
      ++asked;
    };
    while (true) {
      if (have && lane == 0) {
        const Unit<NQ> u(at, window, ranks, rank);
        while (fine && r < 2 * u.n_tiles) {
          // late, so that whoever is done first takes what is left
          if (ranks == 1 && asked == told && r >= 2 * u.n_tiles - kRing) ask();
          fine = load_kv(u);
        }
        if (fine && ranks == 1 && asked == told) ask();
      }
      int unit = -1;
      if (ranks == 1) {
        if (lane == 0 && fine) {
          if (asked == told) ask();
          fine = mbar_wait(smem_u32(&bars.next_full), told & 1, abort_flag);
          if (fine) {
            ++told;
            unit = block_given(smem_u32(&bars.next));
          }
        }
        unit = __shfl_sync(0xffffffffu, unit, 0);
      }
      have = unit >= 0 && find(unit);
      // No such tile: the next one. Not for ever, as the others wait with a
      // bound; the blocks that are left start by themselves.
      if (unit >= 0 && !have && ++misses < kMaxMisses) continue;
      misses = 0;
      if (lane == 0 && fine) {
        // into the slot of the unit before the last
        if (m > 1) fine = mbar_wait(smem_u32(&bars.unit_free[m & 1]), ((m >> 1) - 1) & 1, abort_flag);
        if (fine) {
          if (!have) at.n = -1;
          bars.unit[m & 1] = at;
          bars.poison[m & 1] = 0;
          mbar_arrive(smem_u32(&bars.unit_full[m & 1]));
          if (have) {
            const Unit<NQ> u(at, window, ranks, rank);
            r = 0;
            fine = load_q(u, 0) && load_kv(u) && (NQ == 1 || load_q(u, NQ - 1));
          }
        }
      }
      if (!have) break;
      ++m;
    }
    if (lane == 0) {
      // The MMA side ends every path by committing `fin`; after an abort the
      // copies that nobody consumed are waited for, with a short bound.
      const long long t0 = clock64();
      while (!mbar_try_wait(smem_u32(&bars.fin), 0) && !*abort_flag && clock64() - t0 < kWaitLimitCycles) {
      }
      if (*abort_flag) {
        if (asked > told) wait_short(smem_u32(&bars.next_full), told & 1);
        for (int t = 0; t < NQ; ++t)
          if (n_q[t] > 0) wait_short(smem_u32(&bars.q_full[t]), (n_q[t] - 1) & 1);
        for (int x = max(0, items - kRing); x < items; ++x)
          wait_short(smem_u32(&bars.full[x % kRing]), (x / kRing) & 1);
      }
    }
   } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t on = elect_one();
    const uint64_t q_desc = desc_k_major(sb), k_desc = desc_k_major(sb + kRingOff),
                   v_desc = desc_mn_major(sb + kRingOff);
    // stage and turn of the K item of the next scores and of the V item of the next product
    int k_st = 0, k_turn = 0, v_st = 1, v_turn = 0;
    int q_turn[NQ] = {}, p_turn[NQ] = {};
    auto next_k = [&] {
      commit_if(on, smem_u32(&bars.empty[k_st]));
      k_st += 2;
      if (k_st >= kRing) { k_st -= kRing; ++k_turn; }
    };
    Place place;
    for (int m = 0; take(m, place); ++m) {
      release(m);
      const Unit<NQ> u(place, window, ranks, rank);
      const int n_tiles = u.n_tiles;
      // scores of query tile t with key tile j, whose K is in stage st
      auto scores = [&](int t, int j, int st) {
        tc_fence_after();
        issue_qk<F16>(on, tmem + t * 256u, q_desc + t * (kStage >> 4), k_desc + (uint64_t)st * (kStage >> 4));
        commit_if(on, smem_u32(&bars.s_full[t]));
        if (j + 1 == u.last[t]) commit_if(on, smem_u32(&bars.q_free[t]));
      };
      // each tile's first scores (the second's first key tile may be number 1)
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        if (u.last[t] > u.first[t]) {
          int st = k_st + 2 * u.first[t], turn = k_turn;
          if (st >= kRing) { st -= kRing; ++turn; }
          mbar_pass(smem_u32(&bars.q_full[t]), q_turn[t]++ & 1, abort_flag);
          mbar_pass(smem_u32(&bars.full[st]), turn & 1, abort_flag);
          scores(t, u.first[t], st);
        }
      }
      if (n_tiles > 0) next_k();
      for (int j = 0; j < n_tiles; ++j) {
        const uint64_t v_d = v_desc + (uint64_t)v_st * (kStage >> 4);
        // v_ok of every tile, so that the guard never falls a ring behind
        mbar_pass(smem_u32(&bars.full[v_st]), v_turn & 1, abort_flag);
        mbar_pass(smem_u32(&bars.v_ok[v_st]), v_turn & 1, abort_flag);
        if (NQ == 2 && j + 1 < n_tiles) mbar_pass(smem_u32(&bars.full[k_st]), k_turn & 1, abort_flag);
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          if (j >= u.first[t] && j < u.last[t]) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              mbar_pass(smem_u32(&bars.p_full[t][half]), p_turn[t] & 1, abort_flag);
              tc_fence_after();
              issue_pv<F16>(on, tmem + t * 256u + 128u, tmem + t * 256u + half * 32u, v_d, half, half || j > u.first[t]);
            }
            ++p_turn[t];
            if (j + 1 == u.last[t]) commit_if(on, smem_u32(&bars.o_full[t]));
          }
          if (j + 1 > u.first[t] && j + 1 < u.last[t]) {
            // a ring of one key tile: K of the next one follows this one's product
            if (NQ == 1) mbar_pass(smem_u32(&bars.full[k_st]), k_turn & 1, abort_flag);
            scores(t, j + 1, k_st);
          }
        }
        commit_if(on, smem_u32(&bars.empty[v_st]));
        v_st += 2;
        if (v_st >= kRing) { v_st -= kRing; ++v_turn; }
        if (j + 1 < n_tiles) next_k();
      }
    }
    commit_if(on, smem_u32(&bars.fin));
    wait_short(smem_u32(&bars.fin), 0);
    __syncwarp();
   } else {
    // ------------------------------------------------------------ V guard
    const int gt = tid - 64;
    bool w = true;
    Place place;
    for (int m = 0, item = 1; w && take(m, place); ++m) {
      release(m);
      const Unit<NQ> u(place, window, ranks, rank);
      for (int j = 0; j < u.n_tiles; ++j, item += 2) {
        const int s = item % kRing;
        w = mbar_spin(smem_u32(&bars.full[s]), (item / kRing) & 1, abort_flag);
        w = __all_sync(0xffffffffu, w);
        if (!w) break;
        if (u.masked(u.kt_lo + j, window)) {
          uint4* tile = reinterpret_cast<uint4*>(smem + kRingOff + s * kStage);
          const int there = u.n - (u.kt_lo + j) * kKeyTile;   // rows of the tile that are keys of the sequence
          bool met = false;
#pragma unroll 8
          for (int x = gt; x < (int)(kStage / 16); x += 64) {
            uint4 d = tile[x];
            const uint32_t a = nonfinite_bits<F16>(d.x), b = nonfinite_bits<F16>(d.y), c = nonfinite_bits<F16>(d.z),
                           e = nonfinite_bits<F16>(d.w);
            if (a | b | c | e) {
              met = met || ((x >> 3) & 127) < there;
              d.x &= ~((a >> 15) * 0xffffu); d.y &= ~((b >> 15) * 0xffffu);
              d.z &= ~((c >> 15) * 0xffffu); d.w &= ~((e >> 15) * 0xffffu);
              tile[x] = d;
            }
          }
          if (met) bars.poison[m & 1] = 1;
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(smem_u32(&bars.v_ok[s]));
      }
    }
   }
   if (meets) {                                      // as the softmax warps below
    cluster_meet();
    cluster_meet();
   }
  } else {
    if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ------------------------------------------------------------ softmax
    const int t = NQ == 2 ? (warp - 4) >> 2 : 0;    // query tile of this warpgroup
    const int r = (warp & 3) * 32 + lane;           // row within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = p.scale_log2;
    const uint32_t s_addr = tmem + lane_off + t * 256u, o_addr = s_addr + 128u;
    const uint64_t sc2 = f2(sl2, sl2);
    uint32_t s_turn = 0, o_turn = 0;
    bool ok = true;
    Place place;
    for (int m = 0; ok && take(m, place); ++m) {
    int i, j0, j1, kt_lo;
    {
      const Unit<NQ> u(place, window, ranks, rank);
      i = u.row0 + t * 128 + r;                     // row within the sequence
      j0 = u.first[t], j1 = u.last[t], kt_lo = u.kt_lo;
    }
    float m_run = -INFINITY;
    uint64_t sum = 0;                               // the row's sum, even and odd keys
    for (int j = j0; j < j1; ++j) {
      const bool w = mbar_spin(smem_u32(&bars.s_full[t]), s_turn++ & 1, abort_flag);
      if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
      tc_fence_after();
      const int key0 = (kt_lo + j) * kKeyTile;
      auto tile = [&](auto is_cut) {
        constexpr bool kCut = decltype(is_cut)::value;
        uint32_t v[128];
        tmem_ld32(s_addr, v);
        tmem_ld32(s_addr + 32u, v + 32);
        tc_wait_ld();
        tmem_ld32(s_addr + 64u, v + 64);             // under the first half's maximum
        tmem_ld32(s_addr + 96u, v + 96);
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half) tc_wait_ld();
          if (kCut) {
#pragma unroll
            for (int x = half * 2; x < half * 2 + 2; ++x) {
              // the keys of these 32 that the row attends, as bits
              const uint32_t in = low_bits(i + 1 - key0 - x * 32) & ~low_bits(i - window + 1 - key0 - x * 32);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(in >> c & 1u)) v[x * 32 + c] = __float_as_uint(-INFINITY);
            }
          }
#pragma unroll
          for (int c = half * 64; c < half * 64 + 64; c += 2)
            top[(c >> 1) & 3] =
                max3f(top[(c >> 1) & 3], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
        }
        const float m_cand = max3f(max3f(top[0], top[1], top[2]), top[3], top[3]) * sl2;
        const bool need = m_cand > m_run + 8.f;
        const float f = need ? ex2(m_run - m_cand) : 1.f;     // 0 while nothing was attended yet
        if (need) m_run = m_cand;
        const bool rescale = __any_sync(0xffffffffu, need) && j > j0;
        sum = f2_mul(sum, f2(f, f));
        const float base = (m_run == -INFINITY) ? 0.f : m_run;
        const uint64_t nb2 = f2(-base, -base);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int at = half * 64 + 2 * c;
            const uint64_t x = f2_fma(f2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), sc2, nb2);
            float x0, x1;
            f2_split(x, x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            sum = f2_add(sum, f2(p0, p1));
            pk[c] = Elem16<F16>::pack(p0, p1);
          }
          tmem_st32(s_addr + half * 32u, pk);
          if (half == 0 && rescale) {
            // S(j) was committed behind PV(j - 1), so O is complete up to it
#pragma unroll 1
            for (int c8 = 0; c8 < 8; ++c8) {
              uint32_t o[16];
              tmem_ld16(o_addr + c8 * 16u, o);
              tc_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
              tmem_st16(o_addr + c8 * 16u, o);
            }
          }
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[t][half]));
        }
      };
      // two copies: with the mask as selects every tile would pay for it
      const bool cut = __any_sync(0xffffffffu, key0 + kKeyTile - 1 > i || key0 <= i - window);
      if (cut) tile(std::true_type{});
      else tile(std::false_type{});
    }
    float l_run;
    {
      float s0, s1;
      f2_split(sum, s0, s1);
      l_run = s0 + s1;
    }
    // read again: nothing of it stays in registers through the loop
    const Unit<NQ> u(bars.unit[m & 1], window, ranks, rank);
    const int c0 = u.c0, n = u.n, row0 = u.row0;
    // Scales the row's sum of P V, of this CTA and (kMerged) the other ranks'
    // partials in their order, and writes it and its lse.
    using T16 = typename Elem16<F16>::T;
    auto write_out = [&](auto merged, bool poison) {
      constexpr bool kMerged = decltype(merged)::value;
      float m_all = m_run, l_all = l_run, f_own = 1.f, f_other[kMaxRanks - 1];
      const float2* sums = reinterpret_cast<const float2*>(smem + kMergedSumsOff);
      if (kMerged) {
#pragma unroll
        for (int x = 0; x < kMaxRanks - 1; ++x)
          if (x < ranks - 1) m_all = fmaxf(m_all, sums[x * 128 + r].x);
        f_own = l_run == 0.f ? 0.f : ex2(m_run - m_all);
        l_all = l_run * f_own;
#pragma unroll
        for (int x = 0; x < kMaxRanks - 1; ++x) {
          const float2 y = x < ranks - 1 ? sums[x * 128 + r] : make_float2(0.f, 0.f);
          f_other[x] = y.y == 0.f ? 0.f : ex2(y.x - m_all);
          l_all += y.y == 0.f ? 0.f : y.y * f_other[x];
        }
      }
      // a row whose every score was -inf is zero
      const float inv = l_all == 0.f ? 0.f : 1.f / l_all;
      // Rows go out through shared memory (this warp's 32 rows), so that a store
      // covers whole 64 or 128 bytes of some rows and not 16 bytes of 32 (6500
      // against 2500 clocks); 16-byte pieces XOR-swizzled by the row.
      constexpr int kPieces = C::kOutCols / 8, kRowsAt = 32 / kPieces;
      unsigned char* rows = smem + C::kOutOff + (warp - 4) * C::kOutWarp;
      auto piece = [&](int row, int x) -> uint4* {
        const int swizzle = kPieces == 8 ? row & 7 : (row >> 1) & 3;
        return reinterpret_cast<uint4*>(rows + row * (C::kOutCols * 2) + ((x ^ swizzle) << 4));
      };
      const int i0 = row0 + t * 128 + (warp & 3) * 32;
      const int h = u.h, g = u.g;
      T16* out = static_cast<T16*>(p.o) + (int64_t)(c0 + i0) * p.o_sn + (int64_t)h * p.o_sh + (lane % kPieces) * 8;
#pragma unroll 1
      for (int c4 = 0; c4 < 4; ++c4) {
        uint32_t o[32];
        tmem_ld32(o_addr + c4 * 32u, o);
        tc_wait_ld();
        if (kMerged) {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = l_run == 0.f ? 0u : __float_as_uint(__uint_as_float(o[c]) * f_own);
#pragma unroll
          for (int x = 0; x < kMaxRanks - 1; ++x) {
            if (x >= ranks - 1 || f_other[x] == 0.f) continue;       // nothing was written there
            const float4* part = reinterpret_cast<const float4*>(smem + x * kPartial) + c4 * 8 * 128 + r;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 y = part[c * 128];
              o[4 * c] = __float_as_uint(__uint_as_float(o[4 * c]) + f_other[x] * y.x);
              o[4 * c + 1] = __float_as_uint(__uint_as_float(o[4 * c + 1]) + f_other[x] * y.y);
              o[4 * c + 2] = __float_as_uint(__uint_as_float(o[4 * c + 2]) + f_other[x] * y.z);
              o[4 * c + 3] = __float_as_uint(__uint_as_float(o[4 * c + 3]) + f_other[x] * y.w);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv);
        if (poison && i < n) {
          // what the guards took out, back into this row if it attends the key
          for (int kt = u.kt_all; kt < u.kt_all + u.n_all; ++kt) {
            if (!u.masked(kt, window)) continue;
            const int k0 = kt * kKeyTile;
            for (int u = max(k0, i - window + 1); u <= min(i, k0 + kKeyTile - 1); ++u) {
              const uint4* vrow = reinterpret_cast<const uint4*>(
                  static_cast<const T16*>(p.v) + (int64_t)(c0 + u) * p.v_sn + (int64_t)g * p.v_sh + c4 * 32);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint4 d = __ldg(vrow + x);
                const uint32_t wd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const uint32_t bad = nonfinite_bits<F16>(wd[y]);
                  const int at = x * 8 + y * 2;
                  if (bad & 0x8000u) o[at] = __float_as_uint(__uint_as_float(o[at]) + Elem16<F16>::lo(wd[y]));
                  if (bad & 0x80000000u)
                    o[at + 1] = __float_as_uint(__uint_as_float(o[at + 1]) + Elem16<F16>::hi(wd[y]));
                }
              }
            }
          }
        }
#pragma unroll
        for (int v4 = 0; v4 < 4; ++v4) {
          uint4 w4;
          w4.x = Elem16<F16>::pack(__uint_as_float(o[v4 * 8 + 0]), __uint_as_float(o[v4 * 8 + 1]));
          w4.y = Elem16<F16>::pack(__uint_as_float(o[v4 * 8 + 2]), __uint_as_float(o[v4 * 8 + 3]));
          w4.z = Elem16<F16>::pack(__uint_as_float(o[v4 * 8 + 4]), __uint_as_float(o[v4 * 8 + 5]));
          w4.w = Elem16<F16>::pack(__uint_as_float(o[v4 * 8 + 6]), __uint_as_float(o[v4 * 8 + 7]));
          *piece(lane, c4 % (kPieces / 4) * 4 + v4) = w4;
        }
        if (c4 % (kPieces / 4) != kPieces / 4 - 1) continue;
        __syncwarp();
        T16* at16 = out + (c4 / (kPieces / 4)) * C::kOutCols;
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
          const int rr = x * kRowsAt + lane / kPieces;
          const uint4 w4 = *piece(rr, lane % kPieces);
          if (i0 + rr < n) *reinterpret_cast<uint4*>(at16 + rr * p.o_sn) = w4;
        }
        __syncwarp();
      }
      if (p.lse && i < n)
        p.lse[(int64_t)u.jh * p.T + c0 + i] = l_all == 0.f ? -INFINITY : (m_all + log2f(l_all)) * 0.69314718055994531f;
    };

    const bool here = j1 > j0;                       // this CTA has a part of the tile
    if (here) {
      const bool w = ok && mbar_spin(smem_u32(&bars.o_full[t]), o_turn++ & 1, abort_flag);
      ok = __all_sync(0xffffffffu, w && !*abort_flag);
      tc_fence_after();
    }
    volatile int* poison = &bars.poison[m & 1];
    if (ranks == 1) {
      if (here && ok) write_out(std::false_type{}, *poison != 0);
    } else if constexpr (NQ == 2) {
      cluster_meet();                                // nobody's query tiles and ring are in use any more
      if (rank != t && ok && row0 + t * 128 < n) {
        const uint32_t slot = rank < t ? rank : rank - 1;
        const uint32_t to = remote_smem(sb, t);
        remote_st2(to + kMergedSumsOff + (slot * 128 + r) * 8u, m_run, l_run);
        if (*poison) remote_st1(remote_smem(smem_u32(&bars.poison[0]), t), 1);
        if (here) {
#pragma unroll 1
          for (int c4 = 0; c4 < 4; ++c4) {
            uint32_t o[32];
            tmem_ld32(o_addr + c4 * 32u, o);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 8; ++c)
              remote_st4(to + slot * kPartial + ((c4 * 8 + c) * 128 + r) * 16u, o[4 * c], o[4 * c + 1], o[4 * c + 2],
                         o[4 * c + 3]);
          }
        }
      }
      cluster_meet();
      if (rank == t && ok && row0 + t * 128 < n) write_out(std::true_type{}, *poison != 0);
    }
    release(m);
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (tid == 0 && bars.abort) atomicExch(status, kStatusTimeout);
}

template <bool F16, int NQ>
static cudaError_t launch_typed(const PackedParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                                const CUtensorMap& tv, int* status, cudaStream_t stream) {
  auto kernel = attn_packed_kernel<F16, NQ>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<NQ>);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.n_numbers * p.n_heads * p.ranks));
  cfg.blockDim = dim3(Cfg<NQ>::kThreads);
  cfg.dynamicSmemBytes = kSmemBytes<NQ>;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.ranks > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p, tq, tk, tv, status);
}

// How many CTAs share a unit's keys, from what the host knows: the units and
// the mean length. In key tiles' time: alone the call takes as long as its
// longest unit or its share of all, `work`, whichever is more; split by r the
// longest unit shrinks, but handing the parts over costs about 2 and every CTA
// about 4 (2 alone) for its beginning and end. Three only while all CTAs run
// at once. Measured, alone against by 2 (by 3): one prompt of 8192 tokens, 4 heads
// 122 against 75 us (98); 4096, 8 heads 65, 51; 2048, 8 heads 37, 26 (34); 2048, 16
// heads 38, 38; 1024, 32 heads 24, 32; 100 tokens, 8 heads 8, 11.
static int choose_ranks(int64_t units, int mean_len, int window) {
  const bool cut = window < mean_len;
  const double longest = ((cut ? (double)window + Cfg<2>::kTileRows : mean_len) + kKeyTile - 1) / kKeyTile;
  const double work = (double)units * (cut ? longest : (longest + 1) / 2) / kSMs;
  int best = 1;
  double least = 0;
  for (int r = 1; r <= kMaxRanks; ++r) {
    if (r > 2 && units * r > kSMs) break;
    const double alone = longest / r + (r > 1 ? 2 : 0), share = work + (double)units * r * (r > 1 ? 4 : 2) / kSMs;
    const double time = alone > share ? alone : share;
    if (r == 1 || time < 0.9 * least) {
      best = r;
      least = time;
    }
  }
  return best;
}

cudaError_t launch_attn_packed(const Tensor4& q, const Tensor4& k, const Tensor4& v, void* o, int64_t o_sn,
                               int64_t o_sh, bool f16, int T, int Hq, int Hkv, const int32_t* heads, int n_heads,
                               const int32_t* cu, int S, int window, float scale, float* lse, int* status,
                               cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  if (!make_tmap_bnhd(&tq, q.p, 1, T, Hq, 0, q.sn, q.sh, 128) ||
      !make_tmap_bnhd(&tk, k.p, 1, T, Hkv, 0, k.sn, k.sh, kKeyTile) ||
      !make_tmap_bnhd(&tv, v.p, 1, T, Hkv, 0, v.sn, v.sh, kKeyTile))
    return cudaErrorInvalidValue;
  PackedParams p;
  p.o = o; p.o_sn = o_sn; p.o_sh = o_sh;
  p.v = v.p; p.v_sn = v.sn; p.v_sh = v.sh;
  p.cu = cu; p.lse = lse;
  p.S = S; p.T = T; p.G = Hq / Hkv; p.window = min(window, T); p.n_heads = n_heads;
  const bool small = min(T / S, window) <= kFewKeys;
  p.n_numbers = (int64_t)T / (small ? Cfg<1>::kTileRows : Cfg<2>::kTileRows) + S;
  p.ranks = small ? 1 : choose_ranks(p.n_numbers * n_heads, T / S, window);
  p.scale_log2 = scale * 1.4426950408889634f;
  for (int j = 0; j < n_heads; ++j) p.head[j] = (uint8_t)heads[j];
  if (small)
    return f16 ? launch_typed<true, 1>(p, tq, tk, tv, status, stream)
               : launch_typed<false, 1>(p, tq, tk, tv, status, stream);
  return f16 ? launch_typed<true, 2>(p, tq, tk, tv, status, stream)
             : launch_typed<false, 2>(p, tq, tk, tv, status, stream);
}

}  // namespace rtp
