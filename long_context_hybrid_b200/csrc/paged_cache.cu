// The paged cache: filling it and shrinking it.
//
// rtp_paged_append copies packed K/V rows (and weights) to their slots, 1 KB
// moved per token and KV head. Bound by the rounds of a CTA, which wait for one
// another (26477 tokens of 4 heads: 24.6 us, of HBM's time 16.7). A CTA takes up to 32
// consecutive tokens: one warp finds their sequences, pages and rows (a lane
// each), then the warps copy whole rows in 16-byte pieces.
//
// rtp_cache_evict keeps, per KV head, the first `sink` tokens, the last
// `recent` and the budget - sink - recent others of largest accumulated
// weight, and moves them to the front in order. Two kernels:
//   * selection, one thread-block cluster per (sequence, KV head): every CTA
//     holds the order-preserving keys of a contiguous slice of the candidates
//     in shared memory (read once through the page table); the threshold key is
//     found by four radix passes of 8 bits whose histograms are summed over
//     distributed shared memory; the CTAs then exchange their counts and write
//     their slice of the ascending list. Nothing depends on the order of
//     atomics: counts are integers and ties go to the lower slot. (Passes of 11
//     bits are fewer, but every CTA then reads 64 KB of its neighbours'
//     histograms a pass: 22 against 16 us for 8 x 4 rows of 5000 to 32768);
//   * the move, bound by HBM: 512 bytes of K and V read and written per kept
//     token and KV head (the same rows cut to 8192 each, 249 MB both ways: 41 us,
//     6.1 TB/s). In place it is a chain, a step of 128 rows after another: 221 us.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace rtp {
namespace cg = cooperative_groups;

namespace {

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
// 26477 tokens of 4 heads: 24.6 us; with 16 rows, 256 threads 32.8
constexpr int kAppendThreads = 128;
constexpr int kAppendTokens = 32;              // most tokens of one CTA: a lane each
constexpr int kAppendAhead = 4;                // rows a warp keeps in flight
static_assert(kAppendTokens <= 32, "a lane finds a token's slot");

struct AppendParams {
  PagedView c;
  const char* k; int64_t k_sn, k_sh;           // byte strides
  const char* v; int64_t v_sn, v_sh;
  const float* w; int64_t w_sh;                // NULL: the new tokens' weights are 0
  const int32_t* cu; const int32_t* pos;
  int S, T, per_cta;
};

__global__ void __launch_bounds__(kAppendThreads)
paged_append_kernel(const AppendParams p) {
  __shared__ int s_page[kAppendTokens], s_row[kAppendTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * p.per_cta;
  const int n = min(p.per_cta, p.T - t0);
  if (warp == 0) {
    // the sequence of the first token, then every lane goes on to its own
    int i = max(0, warp_last_le([&](int x) -> int64_t { return __ldg(p.cu + x); }, p.S + 1, t0));
    const int t = t0 + lane;
    while (i < p.S && __ldg(p.cu + i + 1) <= t) ++i;
    int page = -1, row = 0;
    if (lane < n && i < p.S && __ldg(p.cu + i) <= t) {
      const int64_t slot = (int64_t)__ldg(p.pos + i) + t - __ldg(p.cu + i);
      if (slot >= 0 && slot < p.c.capacity) {
        page = page_of(p.c, i, slot);
        row = (int)(slot & ((1 << p.c.page_shift) - 1));
      }
    }
    if (lane < n) {
      s_page[lane] = page;
      s_row[lane] = row;
    }
  }
  __syncthreads();
  // a warp moves whole rows: lanes 0..15 the K row, 16..31 the V row of one
  // token and head; kAppendAhead rows' loads are in flight at once
  const int c = (lane & 15) * 16;
  const char* from = lane < 16 ? p.k + c : p.v + c;
  const int64_t from_n = lane < 16 ? p.k_sn : p.v_sn, from_h = lane < 16 ? p.k_sh : p.v_sh;
  char* to = lane < 16 ? p.c.k + c : p.c.v + c;
  const int64_t to_p = lane < 16 ? p.c.k_sp : p.c.v_sp, to_n = lane < 16 ? p.c.k_sn : p.c.v_sn,
                to_h = lane < 16 ? p.c.k_sh : p.c.v_sh;
  const int rows = n * p.c.Hkv;
  for (int x0 = warp; x0 < rows; x0 += kAppendAhead * (kAppendThreads / 32)) {
    uint4 d[kAppendAhead];
    char* at[kAppendAhead];
#pragma unroll
    for (int y = 0; y < kAppendAhead; ++y) {
      const int x = x0 + y * (kAppendThreads / 32);
      at[y] = nullptr;
      if (x < rows) {
        const int j = x / p.c.Hkv, h = x - j * p.c.Hkv;
        if (s_page[j] >= 0) {
          at[y] = to + s_page[j] * to_p + s_row[j] * to_n + h * to_h;
          d[y] = __ldg(reinterpret_cast<const uint4*>(from + (int64_t)(t0 + j) * from_n + h * from_h));
        }
      }
    }
#pragma unroll
    for (int y = 0; y < kAppendAhead; ++y)
      if (at[y]) *reinterpret_cast<uint4*>(at[y]) = d[y];
  }
  if (p.c.w) {
    for (int x = threadIdx.x; x < n * p.c.Hkv; x += kAppendThreads) {
      const int h = x / n, j = x - h * n;
      if (s_page[j] >= 0)
        p.c.w[(((int64_t)s_page[j] * p.c.Hkv + h) << p.c.page_shift) + s_row[j]] =
            p.w ? __ldg(p.w + h * p.w_sh + t0 + j) : 0.f;
    }
  }
}

// ---------------------------------------------------------------------------
// Eviction: selection
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxCluster = 8;
constexpr int kSelKeys = 40960;                // keys a CTA keeps in shared memory (160 KB)
constexpr int kBins = 256;
constexpr int kCopies = 8;                     // of a CTA's histogram: weights share few exponents

struct EvictParams {
  PagedView src, dst;
  const int32_t* lens;
  int B, max_len, budget, sink, recent;
  int32_t* idx;                                // [B, Hkv, budget]
  int32_t* new_lens;                           // [B]
};

struct SelectSmem {
  uint32_t copies[kCopies][kBins];             // lane l counts in copy l % kCopies
  uint32_t hist[2][kBins];                     // their sums (passes alternate), read by the cluster
  int warp_sum[kBins / 32];
  int above, equal;                            // this CTA's keys above / at the threshold, read by its cluster
  int digit, before;
  int warp_above[kSelWarps], warp_equal[kSelWarps];
};

// Inclusive prefix sum over the warp.
__device__ __forceinline__ int warp_scan(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Sums the cluster's histograms (thread t < 256: bin 255 - t, so that sums run
// from the top bin down) and finds the digit that holds the `left`-th key.
// Every rank's count is loaded at once: a round trip to another CTA's shared
// memory takes as long as one to L2. The whole block calls it.
__device__ __forceinline__ void find_digit(cg::cluster_group& cluster, SelectSmem& sm, const uint32_t* hist,
                                           int n_ranks, int left) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bin = kBins - 1 - tid;
  int count = 0, incl = 0;
  if (tid < kBins) {
    uint32_t c[kSelMaxCluster];                          // past the last rank, its again
#pragma unroll
    for (int r = 0; r < kSelMaxCluster; ++r)
      c[r] = cluster.map_shared_rank(const_cast<uint32_t*>(hist), min(r, n_ranks - 1))[bin];
#pragma unroll
    for (int r = 0; r < kSelMaxCluster; ++r) count += r < n_ranks ? (int)c[r] : 0;
    incl = warp_scan(count);
    if (lane == 31) sm.warp_sum[warp] = incl;
  }
  __syncthreads();
  if (tid < kBins) {
    int before = lane < warp ? sm.warp_sum[lane] : 0;    // warp < 8
    before = __reduce_add_sync(0xffffffffu, before) + incl - count;
    if (before < left && before + count >= left) {
      sm.digit = bin;
      sm.before = before;
    }
  }
  __syncthreads();
}

// Order-preserving key of a weight; NaN ranks above every number.
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0xffffffffu : f2key(w); }

__global__ void __launch_bounds__(kSelThreads, 2)
evict_select_kernel(const EvictParams p, int n_keys) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SelectSmem& sm = *reinterpret_cast<SelectSmem*>(smem_raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem_raw + sizeof(SelectSmem));
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), n_ranks = (int)cluster.num_blocks();
  const int row = blockIdx.x / n_ranks;
  const int b = row / p.src.Hkv, g = row - b * p.src.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = seq_len(p.lens, b, p.max_len);
  const int keep = min(len, p.budget);
  int32_t* out = p.idx + (int64_t)row * p.budget;
  if (g == 0 && rank == 0 && tid == 0) p.new_lens[b] = keep;
  // the parts that need no selection, spread over the cluster
  const int step = n_ranks * kSelThreads;
  for (int j = keep + rank * kSelThreads + tid; j < p.budget; j += step) out[j] = -1;
  if (len <= p.budget) {                       // the same for the whole cluster
    for (int j = rank * kSelThreads + tid; j < len; j += step) out[j] = j;
    return;
  }
  const int need = p.budget - p.sink - p.recent;
  for (int j = rank * kSelThreads + tid; j < p.sink; j += step) out[j] = j;
  for (int j = rank * kSelThreads + tid; j < p.recent; j += step) out[p.sink + need + j] = len - p.recent + j;
  if (need == 0) return;

  // this CTA's slice of the candidates [sink, len - recent)
  const int n_cand = len - p.recent - p.sink;
  const int per = (n_cand + n_ranks - 1) / n_ranks;
  const int c0 = min(n_cand, rank * per), n = min(n_cand, c0 + per) - c0;
  const int first = p.sink + c0;               // slot of the slice's key 0
  // keys i, i + step, .. below end of the slice, from the pages. Every load is
  // unconditional (clamped to the last key, or to page 0) and none is used
  // before all of its kind are under way: under a condition the compiler
  // waits for them one by one (measured: 6 us for eight instead of 2).
  constexpr int kAhead = 8;
  const int row_mask = (1 << p.src.page_shift) - 1;
  const int32_t* table = p.src.table + (int64_t)b * p.src.table_stride;
  auto load_keys = [&](int i, int step_, int end, uint32_t (&x)[kAhead]) {
    int page[kAhead];
    float w[kAhead];
#pragma unroll
    for (int y = 0; y < kAhead; ++y) page[y] = __ldg(table + ((first + min(i + y * step_, end - 1)) >> p.src.page_shift));
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int64_t from = (unsigned)page[y] < (unsigned)p.src.num_pages ? page[y] : 0;
      w[y] = p.src.w[((from * p.src.Hkv + g) << p.src.page_shift) + ((first + min(i + y * step_, end - 1)) & row_mask)];
    }
#pragma unroll
    for (int y = 0; y < kAhead; ++y)           // a token that is not there ranks last
      x[y] = (unsigned)page[y] < (unsigned)p.src.num_pages ? weight_key(w[y]) : 0u;
  };
  const int n_smem = min(n, n_keys);
  for (int i = tid; i < n_smem; i += kAhead * kSelThreads) {
    uint32_t x[kAhead];
    load_keys(i, kSelThreads, n_smem, x);
#pragma unroll
    for (int y = 0; y < kAhead; ++y)
      if (i + y * kSelThreads < n_smem) keys[i + y * kSelThreads] = x[y];
  }
  // f(i, key) for i = from, from + stride, .. below end: from shared memory, and
  // what did not fit there from the pages again
  auto each_key = [&](int from, int stride, int end, auto f) {
    const int near = min(end, n_smem);
    int i = from;
    for (; i < near; i += kAhead * stride) {
      uint32_t x[kAhead];
#pragma unroll
      for (int y = 0; y < kAhead; ++y) x[y] = keys[min(i + y * stride, near - 1)];
#pragma unroll
      for (int y = 0; y < kAhead; ++y)
        if (i + y * stride < near) f(i + y * stride, x[y]);
    }
    if (end > n_smem) {
      i = from + (max(0, n_smem - from) + stride - 1) / stride * stride;
      for (; i < end; i += kAhead * stride) {
        uint32_t x[kAhead];
        load_keys(i, stride, end, x);
#pragma unroll
        for (int y = 0; y < kAhead; ++y)
          if (i + y * stride < end) f(i + y * stride, x[y]);
      }
    }
  };

  uint32_t prefix = 0, mask = 0;
  int left = need;                             // still to take among the keys matching the prefix
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    uint32_t* hist = sm.hist[(shift >> 3) & 1];          // the other one may still be read by the cluster
    for (int x = tid; x < kCopies * kBins; x += kSelThreads) (&sm.copies[0][0])[x] = 0;
    __syncthreads();
    uint32_t* mine = sm.copies[lane % kCopies];
    each_key(tid, kSelThreads, n, [&](int, uint32_t x) {
      if ((x & mask) == prefix) atomicAdd(&mine[(x >> shift) & (kBins - 1)], 1u);
    });
    __syncthreads();
    if (tid < kBins) {
      uint32_t c = 0;
#pragma unroll
      for (int y = 0; y < kCopies; ++y) c += sm.copies[y][tid];
      hist[tid] = c;
    }
    cluster.sync();
    find_digit(cluster, sm, hist, n_ranks, left);
    left -= sm.before;
    prefix |= (uint32_t)sm.digit << shift;
    mask |= 255u << shift;
  }
  // every key above `prefix` is taken, and the `left` lowest slots equal to it

  // counts of this CTA, warp by warp (warp w owns a contiguous part)
  const int per_w = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int w0 = min(n, warp * per_w), w1 = min(n, w0 + per_w);
  int above = 0, equal = 0;
  each_key(w0 + lane, 32, w1, [&](int, uint32_t x) {
    above += x > prefix;
    equal += x == prefix;
  });
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) { sm.warp_above[warp] = above; sm.warp_equal[warp] = equal; }
  __syncthreads();
  const int wa = lane < kSelWarps ? sm.warp_above[lane] : 0, we = lane < kSelWarps ? sm.warp_equal[lane] : 0;
  if (warp == 0) {
    const int a = __reduce_add_sync(0xffffffffu, wa), e = __reduce_add_sync(0xffffffffu, we);
    if (lane == 0) { sm.above = a; sm.equal = e; }
  }
  cluster.sync();
  // taken before this warp's part, over the cluster: lane r looks at rank r and warp r
  int a0 = lane < warp ? wa : 0, e0 = lane < warp ? we : 0;
  if (lane < rank) {
    a0 += *cluster.map_shared_rank(&sm.above, lane);
    e0 += *cluster.map_shared_rank(&sm.equal, lane);
  }
  a0 = __reduce_add_sync(0xffffffffu, a0);
  e0 = __reduce_add_sync(0xffffffffu, e0);
  const unsigned below = (1u << lane) - 1u;
  for (int i0 = w0; i0 < w1; i0 += kAhead * 32) {
    uint32_t x[kAhead];
    const int i = i0 + lane;
    if (min(w1, i0 + kAhead * 32) <= n_smem) {
#pragma unroll
      for (int y = 0; y < kAhead; ++y) x[y] = keys[min(i + y * 32, w1 - 1)];
    } else {
      load_keys(i, 32, w1, x);
    }
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const bool in = i + y * 32 < w1;
      const unsigned ab = __ballot_sync(0xffffffffu, in && x[y] > prefix);
      const unsigned eq = __ballot_sync(0xffffffffu, in && x[y] == prefix);
      const int ea = e0 + __popc(eq & below);
      const bool take = ((ab >> lane) & 1u) || (((eq >> lane) & 1u) && ea < left);
      if (take) out[p.sink + a0 + __popc(ab & below) + min(ea, left)] = first + i + y * 32;
      a0 += __popc(ab);
      e0 += __popc(eq);
    }
  }
  cluster.sync();                              // no CTA leaves while its counts may be read
}

// ---------------------------------------------------------------------------
// Eviction: the move
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 128;

// Out of place: a warp moves whole rows (lanes 0..15 the K row, 16..31 the V
// row), kMoveRows of them with all loads in flight.
constexpr int kMoveRows = 8;
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const EvictParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.y;
  const int b = row / p.src.Hkv, g = row - b * p.src.Hkv;
  pdl_wait();                                  // the lists come from the selection
  const int keep = min(seq_len(p.lens, b, p.max_len), p.budget);
  const int j0 = (blockIdx.x * (kMoveThreads / 32) + warp) * kMoveRows;
  if (j0 >= keep) return;
  const int32_t* idx = p.idx + (int64_t)row * p.budget;
  // lane r < kMoveRows resolves row j0 + r
  int sp = -1, so = 0, dp = -1, dof = 0;
  if (lane < kMoveRows && j0 + lane < keep) {
    const int s = idx[j0 + lane], d = j0 + lane;
    sp = page_of(p.src, b, s);
    so = s & ((1 << p.src.page_shift) - 1);
    dp = d < p.dst.capacity ? page_of(p.dst, b, d) : -1;
    dof = d & ((1 << p.dst.page_shift) - 1);
  }
  const bool is_v = lane >= 16;
  const char* sbase = is_v ? p.src.v : p.src.k;
  char* dbase = is_v ? p.dst.v : p.dst.k;
  const int64_t s_sp = is_v ? p.src.v_sp : p.src.k_sp, s_sn = is_v ? p.src.v_sn : p.src.k_sn;
  const int64_t d_sp = is_v ? p.dst.v_sp : p.dst.k_sp, d_sn = is_v ? p.dst.v_sn : p.dst.k_sn;
  sbase += g * (is_v ? p.src.v_sh : p.src.k_sh) + (lane & 15) * 16;
  dbase += g * (is_v ? p.dst.v_sh : p.dst.k_sh) + (lane & 15) * 16;
  uint4 d[kMoveRows];
#pragma unroll
  for (int r = 0; r < kMoveRows; ++r) {
    const int page = __shfl_sync(0xffffffffu, sp, r), off = __shfl_sync(0xffffffffu, so, r);
    d[r] = make_uint4(0u, 0u, 0u, 0u);
    if (page >= 0) d[r] = *reinterpret_cast<const uint4*>(sbase + page * s_sp + off * s_sn);
  }
#pragma unroll
  for (int r = 0; r < kMoveRows; ++r) {
    const int from = __shfl_sync(0xffffffffu, sp, r);
    const int page = __shfl_sync(0xffffffffu, dp, r), off = __shfl_sync(0xffffffffu, dof, r);
    if (from >= 0 && page >= 0) *reinterpret_cast<uint4*>(dbase + page * d_sp + off * d_sn) = d[r];
  }
  if (sp >= 0 && dp >= 0)
    p.dst.w[(((int64_t)dp * p.dst.Hkv + g) << p.dst.page_shift) + dof] =
        p.src.w[(((int64_t)sp * p.src.Hkv + g) << p.src.page_shift) + so];
}

// In place: slot j takes the row of slot idx[j] >= j of the same pages. One
// CTA owns a 64-byte column of the rows of one (sequence, KV head) and goes
// through them in order, a block of rows at a time: it reads the block's
// sources, waits for all its threads, and writes. A row that is overwritten
// (slot below the block's end) was the source of this or an earlier block
// only, so every source is read before it is lost. The columns are independent;
// the last "column" holds the weights.
constexpr int kColBytes = 64;
constexpr int kCols = 2 * (RTP_D * 2 / kColBytes);       // of K, then of V
constexpr int kInRows = 4;                               // rows per thread and block
__global__ void __launch_bounds__(kMoveThreads)
evict_move_inplace_kernel(const EvictParams p) {
  const int tid = threadIdx.x;
  const int row = blockIdx.y, col = blockIdx.x;
  const int b = row / p.src.Hkv, g = row - b * p.src.Hkv;
  pdl_wait();
  const int len = seq_len(p.lens, b, p.max_len);
  if (len <= p.budget) return;                           // every token stays where it is
  const int keep = p.budget;
  const int32_t* idx = p.idx + (int64_t)row * p.budget;
  const int smask = (1 << p.src.page_shift) - 1;
  if (col == kCols) {
    auto at = [&](int slot) -> float* {
      const int page = page_of(p.src, b, slot);
      return page < 0 ? nullptr : p.src.w + (((int64_t)page * p.src.Hkv + g) << p.src.page_shift) + (slot & smask);
    };
    constexpr int kRows = kMoveThreads * kInRows;
    for (int j0 = 0; j0 < keep; j0 += kRows) {
      float x[kInRows];
      float* to[kInRows];
#pragma unroll
      for (int r = 0; r < kInRows; ++r) {
        const int j = j0 + r * kMoveThreads + tid;
        const float* from = j < keep ? at(idx[j]) : nullptr;
        to[r] = from ? at(j) : nullptr;
        x[r] = from ? *from : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kInRows; ++r)
        if (to[r]) *to[r] = x[r];
      __syncthreads();
    }
    return;
  }
  const bool is_v = col >= kCols / 2;
  char* base = (is_v ? p.src.v : p.src.k) + g * (is_v ? p.src.v_sh : p.src.k_sh) +
               (col % (kCols / 2)) * kColBytes + (tid & 3) * 16;
  const int64_t s_sp = is_v ? p.src.v_sp : p.src.k_sp, s_sn = is_v ? p.src.v_sn : p.src.k_sn;
  auto at = [&](int slot) -> uint4* {
    const int page = page_of(p.src, b, slot);
    return page < 0 ? nullptr : reinterpret_cast<uint4*>(base + page * s_sp + (slot & smask) * s_sn);
  };
  constexpr int kLanes = kMoveThreads / 4;               // rows side by side
  constexpr int kRows = kLanes * kInRows;
  for (int j0 = 0; j0 < keep; j0 += kRows) {
    uint4 x[kInRows];
    uint4* to[kInRows];
#pragma unroll
    for (int r = 0; r < kInRows; ++r) {
      const int j = j0 + r * kLanes + (tid >> 2);
      const uint4* from = j < keep ? at(idx[j]) : nullptr;
      to[r] = from ? at(j) : nullptr;
      x[r] = from ? *from : make_uint4(0u, 0u, 0u, 0u);
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kInRows; ++r)
      if (to[r]) *to[r] = x[r];
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedView& c, const void* k, int64_t k_sn, int64_t k_sh, const void* v,
                                int64_t v_sn, int64_t v_sh, const float* w, const int32_t* cu, const int32_t* pos,
                                int S, int T, cudaStream_t stream) {
  AppendParams p;
  p.c = c;
  p.k = static_cast<const char*>(k); p.k_sn = k_sn * 2; p.k_sh = k_sh * 2;
  p.v = static_cast<const char*>(v); p.v_sn = v_sn * 2; p.v_sh = v_sh * 2;
  p.w = w; p.w_sh = T;
  p.cu = cu; p.pos = pos; p.S = S; p.T = T;
  // few tokens spread over the SMs; many share a CTA and its search
  p.per_cta = T / 148 < 1 ? 1 : (T / 148 < kAppendTokens ? T / 148 : kAppendTokens);
  paged_append_kernel<<<(T + p.per_cta - 1) / p.per_cta, kAppendThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const PagedView& src, const PagedView& dst, bool in_place, int B,
                               const int32_t* lens, int max_len, int budget, int sink, int recent, int32_t* idx,
                               int32_t* new_lens, cudaStream_t stream) {
  EvictParams p;
  p.src = src; p.dst = dst;
  p.lens = lens; p.B = B; p.max_len = max_len; p.budget = budget; p.sink = sink; p.recent = recent;
  p.idx = idx; p.new_lens = new_lens;
  const int rows = B * src.Hkv;
  // A cluster per row: as many CTAs as give each at least 2048 keys, while
  // the grid stays within about two per SM (or until the keys fit on chip).
  const int64_t most = max_len > sink + recent ? max_len - sink - recent : 1;
  int ranks = 1;
  while (ranks < kSelMaxCluster &&
         ((most > (int64_t)ranks * 2048 && rows * ranks * 2 <= 296) || most > (int64_t)ranks * kSelKeys))
    ranks *= 2;
  int64_t n_keys = (most + ranks - 1) / ranks;
  if (n_keys > kSelKeys) n_keys = kSelKeys;
  const size_t smem = sizeof(SelectSmem) + (size_t)n_keys * 4;
  // The limit is the function's, not the launch's: always the most that any call
  // takes, so that a call in another host thread cannot lower it in between.
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(sizeof(SelectSmem) + kSelKeys * 4));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * ranks));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, (int)n_keys);
  if (e != cudaSuccess) return e;
  const int keep = budget < max_len ? budget : max_len;
  if (in_place) {
    e = launch_pdl(evict_move_inplace_kernel, dim3(kCols + 1, rows), dim3(kMoveThreads), 0, stream, p);
  } else {
    const int per_cta = (kMoveThreads / 32) * kMoveRows;
    e = launch_pdl(evict_move_kernel, dim3((keep + per_cta - 1) / per_cta, rows), dim3(kMoveThreads), 0, stream, p);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace rtp
