// The paged cache: filling it and shrinking it.
//
// rtp_paged_append copies packed K/V rows (and weights) to their slots; it
// moves 1 KB per token and KV head and is bound by HBM. A CTA takes a few
// consecutive tokens: one warp per token finds its sequence, page and row,
// then all threads copy 16-byte pieces.
//
// rtp_cache_evict keeps, per KV head, the first `sink` tokens, the last
// `recent` and the budget - sink - recent others of largest accumulated
// weight, and moves them to the front in order. Two kernels:
//   * selection, one thread-block cluster per (sequence, KV head): every CTA
//     holds the order-preserving keys of a contiguous slice of the candidates
//     in shared memory (read once through the page table); the threshold key is
//     found by three radix passes (11, 11, 10 bits) whose histograms are summed
//     over distributed shared memory; the CTAs then exchange their counts and
//     write their slice of the ascending list. Nothing depends on the order of
//     atomics: counts are integers and ties go to the lower slot;
//   * the move, bound by HBM: 512 bytes of K and V read and written per kept
//     token and KV head.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace rtp {
namespace cg = cooperative_groups;

namespace {

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;               // most tokens of one CTA: one per warp

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
  if (warp < n) {
    const int t = t0 + warp;
    const int i = warp_find_seq(p.cu, p.S, t);
    if (lane == 0) {
      int page = -1, row = 0;
      if (i >= 0) {
        const int64_t slot = (int64_t)__ldg(p.pos + i) + t - __ldg(p.cu + i);
        if (slot >= 0 && slot < p.c.capacity) {
          page = page_of(p.c, i, slot);
          row = (int)(slot & ((1 << p.c.page_shift) - 1));
        }
      }
      s_page[warp] = page;
      s_row[warp] = row;
    }
  }
  __syncthreads();
  const int per_token = p.c.Hkv * 32;          // 16-byte pieces of a token's K and V rows
  for (int x = threadIdx.x; x < n * per_token; x += kAppendThreads) {
    const int j = x / per_token, y = x - j * per_token;
    const int page = s_page[j];
    if (page < 0) continue;
    const int h = y >> 5, c = y & 31;          // lanes 0..15: the K row, 16..31: the V row
    const int64_t t = t0 + j, row = s_row[j];
    if (c < 16) {
      const uint4 d = __ldg(reinterpret_cast<const uint4*>(p.k + t * p.k_sn + h * p.k_sh) + c);
      *(reinterpret_cast<uint4*>(p.c.k + page * p.c.k_sp + row * p.c.k_sn + h * p.c.k_sh) + c) = d;
    } else {
      const uint4 d = __ldg(reinterpret_cast<const uint4*>(p.v + t * p.v_sn + h * p.v_sh) + (c - 16));
      *(reinterpret_cast<uint4*>(p.c.v + page * p.c.v_sp + row * p.c.v_sn + h * p.c.v_sh) + (c - 16)) = d;
    }
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
constexpr int kBins = 2048;

struct EvictParams {
  PagedView src, dst;
  const int32_t* lens;
  int B, max_len, budget, sink, recent;
  int32_t* idx;                                // [B, Hkv, budget]
  int32_t* new_lens;                           // [B]
};

struct SelectSmem {
  uint32_t hist[kBins];                        // this CTA's counts, read by its cluster
  uint32_t sum[kBins];                         // the cluster's
  BlockScanSmem<kSelThreads> scan;
  int above, equal;                            // this CTA's keys above / at the threshold
  int digit, before;
  int warp_above[kSelWarps], warp_equal[kSelWarps];
};

// Order-preserving key of a weight; NaN ranks above every number.
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0xffffffffu : f2key(w); }

__global__ void __launch_bounds__(kSelThreads, 1)
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
  auto load_key = [&](int i) -> uint32_t {
    const int slot = first + i;
    const int page = page_of(p.src, b, slot);
    if (page < 0) return 0u;                   // a token that is not there ranks last
    return weight_key(p.src.w[(((int64_t)page * p.src.Hkv + g) << p.src.page_shift) +
                              (slot & ((1 << p.src.page_shift) - 1))]);
  };
  const int n_smem = min(n, n_keys);
  constexpr int kAhead = 8;                    // loads a thread keeps in flight
  for (int i0 = tid; i0 < n_smem; i0 += kAhead * kSelThreads) {
    uint32_t x[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * kSelThreads;
      x[a] = i < n_smem ? load_key(i) : 0u;
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * kSelThreads;
      if (i < n_smem) keys[i] = x[a];
    }
  }
  auto key = [&](int i) -> uint32_t { return i < n_smem ? keys[i] : load_key(i); };

  uint32_t prefix = 0, mask = 0;
  int left = need;                             // still to take among the keys matching the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bins = pass == 2 ? 1024 : 2048;
    for (int x = tid; x < bins; x += kSelThreads) sm.hist[x] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t x = key(i);
      if ((x & mask) == prefix) atomicAdd(&sm.hist[(x >> shift) & (bins - 1)], 1u);
    }
    cluster.sync();
    // thread t owns the bins bins - 1 - t * per_t ... walking downwards
    const int per_t = bins / kSelThreads;
    int local = 0;
    for (int q = 0; q < per_t; ++q) {
      const int x = bins - 1 - (tid * per_t + q);
      uint32_t s = 0;
      for (int r = 0; r < n_ranks; ++r) s += cluster.map_shared_rank(sm.hist, r)[x];
      sm.sum[x] = s;
      local += (int)s;
    }
    int total;
    const int before = block_exclusive_scan<kSelThreads>(local, total, sm.scan);
    if (before < left && before + local >= left) {
      int run = before;
      for (int q = 0; q < per_t; ++q) {
        const int x = bins - 1 - (tid * per_t + q);
        const int s = (int)sm.sum[x];
        if (run + s >= left) { sm.digit = x; sm.before = run; break; }
        run += s;
      }
    }
    cluster.sync();                            // the digit is set, and every CTA has read the histograms
    left -= sm.before;
    prefix |= (uint32_t)sm.digit << shift;
    mask |= (uint32_t)(bins - 1) << shift;
  }
  // every key above `prefix` is taken, and the `left` lowest slots equal to it

  // counts of this CTA, warp by warp (warp w owns a contiguous part)
  const int per_w = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int w0 = min(n, warp * per_w), w1 = min(n, w0 + per_w);
  int above = 0, equal = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t x = key(i);
    above += x > prefix;
    equal += x == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) { sm.warp_above[warp] = above; sm.warp_equal[warp] = equal; }
  __syncthreads();
  if (tid == 0) {
    int a = 0, e = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      const int xa = sm.warp_above[w], xe = sm.warp_equal[w];
      sm.warp_above[w] = a; sm.warp_equal[w] = e;
      a += xa; e += xe;
    }
    sm.above = a; sm.equal = e;
  }
  cluster.sync();
  int a0 = sm.warp_above[warp], e0 = sm.warp_equal[warp];   // before this warp's part, over the cluster
  for (int r = 0; r < rank; ++r) {
    a0 += *cluster.map_shared_rank(&sm.above, r);
    e0 += *cluster.map_shared_rank(&sm.equal, r);
  }
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t x = i < w1 ? key(i) : 0u;
    const unsigned ab = __ballot_sync(0xffffffffu, i < w1 && x > prefix);
    const unsigned eq = __ballot_sync(0xffffffffu, i < w1 && x == prefix);
    const unsigned below = (1u << lane) - 1u;
    const int ea = e0 + __popc(eq & below);
    const bool take = ((ab >> lane) & 1u) || (((eq >> lane) & 1u) && ea < left);
    if (take) out[p.sink + a0 + __popc(ab & below) + min(ea, left)] = first + i;
    a0 += __popc(ab);
    e0 += __popc(eq);
  }
  cluster.sync();                              // no CTA leaves while its counts may be read
}

// ---------------------------------------------------------------------------
// Eviction: the move
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;

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
  // few tokens: one per CTA, so that they spread over the SMs
  p.per_cta = T >= 8 * 148 ? kAppendTokens : 1;
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
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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
