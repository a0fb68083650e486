// One new token per sequence over a paged cache, split over the cache's
// length and joined.
//
// Sequence b attends the slots {0 .. sink-1} U {len-window .. len-1}, each
// once, every head over the same set:
//   o = sum_u p_u v_u,  p_u = exp(scale q.k_u - lse),  lse = ln sum_u exp(scale q.k_u).
// The work is bound by HBM: 512 bytes of K and V per attended token and KV
// head, read once for all the query heads of the group.
//
//   * The attended slots of a (sequence, KV head) are a segment of 64-key
//     chunks; the segments of the whole batch form one list that the CTAs (two
//     per SM) cut into equal runs, so that sequences of any mix of lengths
//     load every SM alike. A segment counts kSegCost units more than it has
//     chunks (in front of them): beginning and ending one costs about as much
//     as streaming that many. The lengths stay on the device: each CTA finds
//     its run with a scan over them.
//   * Each of a CTA's four warps owns 16 keys of every chunk: it resolves
//     their pages one chunk ahead of the copies, copies the rows with 16-byte
//     cp.async two chunks ahead into a private three-stage ring (zero-filled
//     where no key is: values there cannot reach a product), and computes
//     S = Q K^T and O += P V with mma.sync (fp32 accumulate; the heads of the
//     group are the rows of the 16-row tile) under an online softmax. P is
//     rounded to the cache's 16-bit type for the second product; the sum of
//     the softmax takes it unrounded.
//   * At the end of a segment the four warps join through shared memory. A
//     segment that lies within one run is finished there; otherwise the CTA
//     leaves one partial (a run has at most two: its first and its last
//     segment), and a second kernel joins the partials of each cut segment.
//   * Short batches (each segment a few chunks a CTA) take one kernel: the
//     CTAs of a cluster share a segment and join over distributed shared
//     memory, each writing every n-th row.
//   * With weights, the first kernel also stores the scaled scores (fp32, 4
//     bytes against 512 / G per key and head) and a third kernel adds
//     exp(score - lse) over the heads of a group, in a fixed order.
//
// Measured: 8 sequences of 131072 tokens, 32/4 heads, 332 us (6.5 TB/s, all of
// what HBM gives a copy); 32 of 1 to 16385 tokens with weights, 55 us: 41 here
// (start, ragged ends and score stores are on top of 27 of HBM), 2 the join, 9
// the weights; one of 4099 tokens, window 1024, 8 us of the GPU's time.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace rtp {
namespace cg = cooperative_groups;

namespace {
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kChunk = 64;                    // keys per chunk
constexpr int kKeys = kChunk / kWarps;        // keys per warp and chunk
constexpr int kStages = 3;
// 32 sequences of 1 to 16385 tokens (32 / 4 heads), weights and all: 55 us with 2,
// 3 or 4; 80 where beginnings do not count
constexpr int kSegCost = 3;
constexpr int kRowBytes = RTP_D * 2;
constexpr int kSlab = kKeys * kRowBytes;      // one warp's K (or V) rows of one chunk
constexpr int kMaxRanks = 8;                  // CTAs of a cluster that share a segment
constexpr int kGroup = 16;                    // query heads per KV head: rows of the tile
constexpr int kPart = 4 + RTP_D;              // m, l, 2 pad, o[128]
constexpr size_t kHeaderBytes = 256;          // status word

struct DecodeParams {
  PagedView c;
  const char* q; int64_t q_sb, q_sh;          // byte strides
  char* o; int64_t o_sb, o_sh;
  const int32_t* lens;
  int B, max_len, window, sink;
  float scale_log2;
  int n_heads, n_ag, rows;                    // listed heads, KV heads with one, most rows of one
  int ranks;                                  // CTAs that share a segment; 0: the batch's list is cut into runs
  float* part;                                // [2 * CTAs, rows, kPart]
  float* lse;                                 // caller's [B, n_heads] (natural log) or NULL
  float* lse2;                                // [B, n_heads], log2 domain (with weights)
  float* logits;                              // [B, n_heads, att_cap] (with weights) or NULL
  float* w_out;
  int64_t att_cap;                            // most attended slots of a sequence, a multiple of kChunk
  int* status;
  uint8_t head[kMaxHeads];                    // query heads, sorted by KV head
  uint8_t out_row[kMaxHeads];                 // position of each in the caller's list
  uint8_t ag_kv[kMaxHeads], ag_start[kMaxHeads], ag_n[kMaxHeads];
};

struct Smem {
  unsigned char ring[kWarps][kStages][2][kSlab];
  float join[2][kGroup][kPart];
  BlockScanSmem<kThreads> scan;
  unsigned ok[kWarps][kStages];               // which of the 16 keys are there
  int64_t place[2];                           // a Place
};

// The attended slots of one sequence: `sink` from the front, then lo .. len-1.
struct Span {
  int len, lo, sink, n;
};
__device__ __forceinline__ Span span_of(const DecodeParams& p, int b) {
  Span s;
  s.len = seq_len(p.lens, b, p.max_len);
  s.lo = s.len > p.window ? s.len - p.window : 0;
  s.sink = min(p.sink, s.lo);
  s.n = s.sink + s.len - s.lo;
  return s;
}
__device__ __forceinline__ int chunks_of(const DecodeParams& p, int b) {
  return (span_of(p, b).n + kChunk - 1) / kChunk;
}
__device__ __forceinline__ int units_of(int chunks) { return chunks > 0 ? chunks + kSegCost : 0; }

// Run c of a list of n units cut for n_ctas CTAs (n_ctas <= n).
__device__ __forceinline__ int64_t run_start(int c, int64_t n, int n_ctas) { return (int64_t)c * n / n_ctas; }
__device__ __forceinline__ int cta_of(int64_t x, int64_t n, int n_ctas) {
  return (int)(((x + 1) * n_ctas - 1) / n);
}

// Where unit x of the list lies: the sequence, its chunks, and the list's
// units before it.
struct Place {
  int64_t before;
  int b, nc;
};

// The scan over the lengths by a block of NT threads: thread i holds sequence
// i of the batch's last NT sequences (all of it, for most batches). Work
// says what a sequence holds: chunks(p, b) pieces of work, units(chunks) units.
template <int NT, class Work>
struct LenScan {
  int64_t total;                              // units of the whole batch, per KV head
  int nc, ex;                                 // this thread's chunks, and the units before it in its block
  __device__ LenScan(const DecodeParams& p, BlockScanSmem<NT>& scan) {
    total = 0;
    for (int b0 = 0; b0 < p.B; b0 += NT) {
      const int b = b0 + threadIdx.x;
      int tot;
      nc = b < p.B ? Work::chunks(p, b) : 0;
      ex = block_exclusive_scan<NT>(Work::units(nc), tot, scan);
      total += tot;
    }
  }
  // Finds the sequence that holds unit x (x < n_ag * total); `at` is shared.
  __device__ void locate(const DecodeParams& p, int64_t x, BlockScanSmem<NT>& scan, Place* at) {
    int64_t before = 0;
    for (int b0 = 0; b0 < p.B; b0 += NT) {
      const int b = b0 + threadIdx.x;
      int tot = 0;
      if (p.B > NT) {                         // otherwise the first scan still stands
        nc = b < p.B ? Work::chunks(p, b) : 0;
        ex = block_exclusive_scan<NT>(Work::units(nc), tot, scan);
      }
      const int64_t first = (before + ex) * p.n_ag;
      if (nc > 0 && first <= x && x < first + (int64_t)Work::units(nc) * p.n_ag) {
        at->b = b;
        at->nc = nc;
        at->before = first;
      }
      before += tot;
      if (before * p.n_ag > x) break;
    }
    __syncthreads();
  }
};

struct AttendedChunks {
  static __device__ __forceinline__ int chunks(const DecodeParams& p, int b) { return chunks_of(p, b); }
  static __device__ __forceinline__ int units(int chunks) { return units_of(chunks); }
};
using ChunkScan = LenScan<kThreads, AttendedChunks>;

// Walks the chunks of a run: sequence-major, then KV head, then chunk.
struct Cursor {
  int64_t unit;                               // of the current chunk; INT64_MAX past the last
  int b, a, local, nc;
  Span s;
  __device__ Cursor() {}
  __device__ Cursor(const DecodeParams& p, const Place& at, int64_t x) {
    b = at.b;
    nc = at.nc;
    s = span_of(p, b);
    const int64_t into = x - at.before;
    a = (int)(into / units_of(nc));
    const int rem = (int)(into - (int64_t)a * units_of(nc));
    local = rem > kSegCost ? rem - kSegCost : 0;
    unit = rem > kSegCost ? x : x + (kSegCost - rem);
  }
  // chunks [lo, ..) of segment (b, a), a unit each
  __device__ Cursor(const DecodeParams& p, int b_, int a_, int lo) : unit(lo), b(b_), a(a_), local(lo) {
    nc = chunks_of(p, b);
    s = span_of(p, b);
  }
  __device__ void next(const DecodeParams& p) {
    ++unit;
    if (++local < nc) return;
    local = 0;
    unit += kSegCost;
    if (++a < p.n_ag) return;
    a = 0;
    do {
      if (++b >= p.B) { unit = INT64_MAX; return; }
      nc = chunks_of(p, b);
    } while (nc == 0);
    s = span_of(p, b);
  }
  // slot of key e of the segment, -1 past its end
  __device__ int slot(int e) const { return e >= s.n ? -1 : (e < s.sink ? e : s.lo + e - s.sink); }
};

__device__ __forceinline__ void ldsm_x4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <bool F16>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// Byte offset of 16-byte piece c of row r in a slab: XOR-swizzled, so that
// the eight rows of an ldmatrix read hit distinct banks.
__device__ __forceinline__ uint32_t slab_off(int r, int c) {
  return (uint32_t)(r * kRowBytes + ((c ^ (r & 7)) << 4));
}

// 2^(a - b) with an empty side (-inf) weighing nothing.
__device__ __forceinline__ float weight2(float a, float b) { return a == -INFINITY ? 0.f : exp2f(a - b); }

// Writes row `j` (sorted head) of sequence b: o / l, and the log-sum-exps.
// l == 0: nothing was attended (or every score was -inf): the row is zero.
template <bool F16>
__device__ __forceinline__ void write_row(const DecodeParams& p, int b, int j, float m, float l, float4 o, int lane) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 w;
  w.x = Elem16<F16>::pack(o.x * inv, o.y * inv);
  w.y = Elem16<F16>::pack(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.o + b * p.o_sb + (int64_t)p.head[j] * p.o_sh + lane * 8) = w;
  if (lane == 0) {
    const float x = l == 0.f ? -INFINITY : m + log2f(l);
    if (p.lse2) p.lse2[(int64_t)b * p.n_heads + j] = x;
    if (p.lse) p.lse[(int64_t)b * p.n_heads + p.out_row[j]] = x * 0.69314718055994531f;
  }
}
}  // namespace

template <bool F16>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
paged_decode_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  pdl_wait();
  pdl_trigger();                              // the join may launch; it waits for this grid
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  if (blockIdx.x == 0 && tid == 0) *p.status = 0;
  int64_t x1;                                 // end of this CTA's chunks, in units
  Cursor cur;                                 // chunk being computed
  if (p.ranks > 0) {
    const int seg = blockIdx.x / p.ranks, rank = blockIdx.x - seg * p.ranks;
    const int b = seg / p.n_ag, a = seg - b * p.n_ag;
    const int nc = chunks_of(p, b);
    if (nc == 0) {                            // nothing to attend (the same for the whole cluster)
      for (int r = rank * kWarps + warp; r < p.ag_n[a]; r += p.ranks * kWarps)
        write_row<F16>(p, b, p.ag_start[a] + r, 0.f, 0.f, make_float4(0, 0, 0, 0), lane);
      return;
    }
    cur = Cursor(p, b, a, rank * nc / p.ranks);
    x1 = (rank + 1) * nc / p.ranks;
  } else {
    ChunkScan lens(p, sm.scan);
    const int64_t n_list = lens.total * p.n_ag;
    const int n_ctas = (int)(n_list < gridDim.x ? n_list : gridDim.x);
    // sequences that attend nothing
    for (int x = blockIdx.x * kWarps + warp; x < p.B * p.n_heads; x += gridDim.x * kWarps) {
      const int b = x / p.n_heads;
      if (chunks_of(p, b) == 0) write_row<F16>(p, b, x - b * p.n_heads, 0.f, 0.f, make_float4(0, 0, 0, 0), lane);
    }
    if ((int)blockIdx.x >= n_ctas) return;
    const int64_t x0 = run_start(blockIdx.x, n_list, n_ctas);
    x1 = run_start(blockIdx.x + 1, n_list, n_ctas);
    Place& place = *reinterpret_cast<Place*>(sm.place);
    lens.locate(p, x0, sm.scan, &place);
    cur = Cursor(p, place, x0);
    if (cur.unit >= x1) return;
  }

  // this warp's ring and its copies of a chunk into stage st
  const uint32_t ring = su32(sm.ring[warp]);
  Cursor icur = cur;                          // next chunk to copy
  const int my_key = warp * kKeys + (lane & (kKeys - 1));
  const int row_mask = (1 << p.c.page_shift) - 1;
  auto fetch = [&](int& slot) -> int {        // lane r < kKeys: page of key r of the next chunk
    slot = icur.slot(icur.local * kChunk + my_key);
    return slot < 0 ? -1 : page_of(p.c, icur.b, slot);
  };
  int slot = -1, page = icur.unit < x1 ? fetch(slot) : -1;
  auto issue = [&](int t) {
    if (icur.unit < x1) {
      const int st = t % kStages;
      const int g = p.ag_kv[icur.a];
      if (icur.local == 0 || t == 0) {        // a segment begins: its query rows on their way to L1
        const int r = lane >> 1;
        if (r < p.ag_n[icur.a])
          asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + icur.b * p.q_sb +
                                                        (int64_t)p.head[p.ag_start[icur.a] + r] * p.q_sh +
                                                        (lane & 1) * 128));
      }
      const int64_t r64 = slot < 0 ? 0 : slot & row_mask, pg = page < 0 ? 0 : page;
      const char* krow = p.c.k + pg * p.c.k_sp + r64 * p.c.k_sn + g * p.c.k_sh;
      const char* vrow = p.c.v + pg * p.c.v_sp + r64 * p.c.v_sn + g * p.c.v_sh;
      const unsigned ok = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0) sm.ok[warp][st] = ok & 0xffffu;
      const uint32_t kdst = ring + (uint32_t)(st * 2) * kSlab, vdst = kdst + kSlab;
      const int c = lane & 15;
#pragma unroll
      for (int i = 0; i < kKeys / 2; ++i) {
        const int r = 2 * i + (lane >> 4);
        const char* ks = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(krow), r));
        const char* vs = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(vrow), r));
        const bool there = (ok >> r) & 1u;
        cp_async16(kdst + slab_off(r, c), ks + c * 16, there);
        cp_async16(vdst + slab_off(r, c), vs + c * 16, there);
      }
      icur.next(p);
      if (icur.unit < x1) page = fetch(slot);
    }
    cp_async_commit();                        // one group per chunk, empty past the run
  };

  uint32_t qa[8][4];
  float o[16][4];
#pragma unroll
  for (int nt = 0; nt < 16; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
  float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
  int seg_local = 0;                          // first chunk of this CTA's piece of the segment
  bool first_piece = true, fresh = true;

  // Joins the warps' rows of a finished piece through shared memory and
  // writes the piece out, a row at a time. Up to eight rows: the four warps'
  // partials fit side by side; more: warps 2, 3 go into 0, 1 first.
  float* const join = &sm.join[0][0][0];
  auto put = [&](float* to) {                 // rows 0..7, and 8..15 behind them where the group has them
    if (tq == 0) { to[gq * kPart] = m_a; to[gq * kPart + 1] = l_a; }
#pragma unroll
    for (int nt = 0; nt < 16; ++nt)
      *reinterpret_cast<float2*>(to + gq * kPart + 4 + nt * 8 + 2 * tq) = make_float2(o[nt][0], o[nt][1]);
    if (p.rows <= 8) return;
    if (tq == 0) { to[(gq + 8) * kPart] = m_b; to[(gq + 8) * kPart + 1] = l_b; }
#pragma unroll
    for (int nt = 0; nt < 16; ++nt)
      *reinterpret_cast<float2*>(to + (gq + 8) * kPart + 4 + nt * 8 + 2 * tq) = make_float2(o[nt][2], o[nt][3]);
  };
  auto add = [&](const float* from) {
    const float* fa_ = from + gq * kPart;
    const float* fb_ = from + (gq + 8) * kPart;
    const float xa = fa_[0], xb = fb_[0];
    const float na = fmaxf(m_a, xa), nb = fmaxf(m_b, xb);
    const float fa = weight2(m_a, na), fb = weight2(m_b, nb), ga = weight2(xa, na), gb = weight2(xb, nb);
    l_a = l_a * fa + fa_[1] * ga;
    l_b = l_b * fb + fb_[1] * gb;
    m_a = na; m_b = nb;
#pragma unroll
    for (int nt = 0; nt < 16; ++nt) {
      const int col = 4 + nt * 8 + 2 * tq;
      const float2 x = *reinterpret_cast<const float2*>(fa_ + col);
      const float2 y = *reinterpret_cast<const float2*>(fb_ + col);
      o[nt][0] = o[nt][0] * fa + x.x * ga; o[nt][1] = o[nt][1] * fa + x.y * ga;
      o[nt][2] = o[nt][2] * fb + y.x * gb; o[nt][3] = o[nt][3] * fb + y.y * gb;
    }
  };
  // Leaves the warps' partials in shared memory: `parts` of them, `part_rows`
  // rows apart.
  const int parts = p.rows <= 8 ? kWarps : 2, part_rows = p.rows <= 8 ? 8 : kGroup;
  auto gather = [&]() {
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
    if (p.rows <= 8) {
      put(join + warp * 8 * kPart);
    } else {
      if (warp >= 2) put(join + (warp - 2) * kGroup * kPart);
      __syncthreads();
      if (warp < 2) {
        add(join + warp * kGroup * kPart);
        __syncwarp();
        put(join + warp * kGroup * kPart);
      }
    }
    __syncthreads();
  };
  // Row r of them, joined.
  auto joined = [&](int r, float& m, float& l) -> float4 {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    m = -INFINITY;
    l = 0.f;
    for (int w = 0; w < parts; ++w) m = fmaxf(m, join[(w * part_rows + r) * kPart]);
    for (int w = 0; w < parts; ++w) {
      const float* from = join + (w * part_rows + r) * kPart;
      const float f = weight2(from[0], m);
      const float4 y = *reinterpret_cast<const float4*>(from + 4 + lane * 4);
      l += f * from[1];
      x.x += f * y.x; x.y += f * y.y; x.z += f * y.z; x.w += f * y.w;
    }
    return x;
  };
  auto finish = [&](bool whole) {
    gather();
    const int n = p.ag_n[cur.a], j0 = p.ag_start[cur.a];
    float* part = p.part + ((int64_t)blockIdx.x * 2 + (first_piece ? 0 : 1)) * p.rows * kPart;
    for (int r = warp; r < n; r += kWarps) {
      float m, l;
      const float4 x = joined(r, m, l);
      if (whole) {
        write_row<F16>(p, cur.b, j0 + r, m, l, x, lane);
      } else {
        float* to = part + r * kPart;
        if (lane == 0) { to[0] = m; to[1] = l; }
        *reinterpret_cast<float4*>(to + 4 + lane * 4) = x;
      }
    }
    __syncthreads();                          // the buffer is free for the next piece
  };

#pragma unroll
  for (int t = 0; t < kStages - 1; ++t) issue(t);
  for (int t = 0; cur.unit < x1; ++t, cur.next(p)) {
    issue(t + kStages - 1);
    if (fresh) {
      fresh = false;
      seg_local = cur.local;
      // query fragments (A operand, 16 x 128): row r is head ag_start + r
      const int n = p.ag_n[cur.a], j0 = p.ag_start[cur.a];
      const char* qb = p.q + cur.b * p.q_sb;
      const uint32_t* qra = reinterpret_cast<const uint32_t*>(qb + (int64_t)p.head[gq < n ? j0 + gq : j0] * p.q_sh);
      const uint32_t* qrb =
          reinterpret_cast<const uint32_t*>(qb + (int64_t)p.head[gq + 8 < n ? j0 + gq + 8 : j0] * p.q_sh);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int c = kk * 8 + tq;            // in pairs of elements
        qa[kk][0] = gq < n ? __ldg(qra + c) : 0u;
        qa[kk][1] = gq + 8 < n ? __ldg(qrb + c) : 0u;
        qa[kk][2] = gq < n ? __ldg(qra + c + 4) : 0u;
        qa[kk][3] = gq + 8 < n ? __ldg(qrb + c + 4) : 0u;
      }
      m_a = m_b = -INFINITY;
      l_a = l_b = 0.f;
#pragma unroll
      for (int nt = 0; nt < 16; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
    }
    cp_async_wait<kStages - 1>();             // chunk t has landed (this lane's copies)
    __syncwarp();                             // ... and every lane's
    const int st = t % kStages;
    const uint32_t kbase = ring + (uint32_t)(st * 2) * kSlab, vbase = kbase + kSlab;
    // S = Q K^T (16 rows x this warp's 16 keys)
    float sacc[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sacc[nt][e] = 0.f;
    {
      const int m = lane >> 3;
      const int key = 8 * (m >> 1) + (lane & 7);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t bf[4];
        ldsm_x4(bf, kbase + slab_off(key, kk * 2 + (m & 1)));
        mma16816<F16>(sacc[0], qa[kk], bf[0], bf[1]);
        mma16816<F16>(sacc[1], qa[kk], bf[2], bf[3]);
      }
    }
    // scale, mask, online softmax (rows gq and gq + 8)
    const unsigned ok = sm.ok[warp][st];
    float mx_a = -INFINITY, mx_b = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool there = (ok >> (nt * 8 + 2 * tq + e)) & 1u;
        sacc[nt][e] = there ? sacc[nt][e] * p.scale_log2 : -INFINITY;
        sacc[nt][2 + e] = there ? sacc[nt][2 + e] * p.scale_log2 : -INFINITY;
        mx_a = fmaxf(mx_a, sacc[nt][e]);
        mx_b = fmaxf(mx_b, sacc[nt][2 + e]);
      }
    if (p.logits) {
      const int n = p.ag_n[cur.a], j0 = p.ag_start[cur.a];
      float* at = p.logits + ((int64_t)cur.b * p.n_heads + j0) * p.att_cap + cur.local * kChunk + warp * kKeys;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        if (gq < n)
          *reinterpret_cast<float2*>(at + gq * p.att_cap + nt * 8 + 2 * tq) = make_float2(sacc[nt][0], sacc[nt][1]);
        if (gq + 8 < n)
          *reinterpret_cast<float2*>(at + (gq + 8) * p.att_cap + nt * 8 + 2 * tq) =
              make_float2(sacc[nt][2], sacc[nt][3]);
      }
    }
    mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
    mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2));
    mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
    mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2));
    if (mx_a > m_a || mx_b > m_b) {           // the running max only moves up: rescale O and l when it does
      const float na = fmaxf(m_a, mx_a), nb = fmaxf(m_b, mx_b);
      const float ra = weight2(m_a, na), rb = weight2(m_b, nb);
      m_a = na; m_b = nb;
      l_a *= ra; l_b *= rb;
#pragma unroll
      for (int nt = 0; nt < 16; ++nt) {
        o[nt][0] *= ra; o[nt][1] *= ra;
        o[nt][2] *= rb; o[nt][3] *= rb;
      }
    }
    const float base_a = m_a == -INFINITY ? 0.f : m_a, base_b = m_b == -INFINITY ? 0.f : m_b;
    uint32_t pa[4];                           // A fragment of P (16 rows x 16 keys)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const float e0 = exp2f(sacc[nt][0] - base_a), e1 = exp2f(sacc[nt][1] - base_a);
      const float e2 = exp2f(sacc[nt][2] - base_b), e3 = exp2f(sacc[nt][3] - base_b);
      l_a += e0 + e1;
      l_b += e2 + e3;
      pa[nt * 2 + 0] = Elem16<F16>::pack(e0, e1);
      pa[nt * 2 + 1] = Elem16<F16>::pack(e2, e3);
    }
    // O += P V (16 rows x 128 dims)
    {
      const int m = lane >> 3;
      const int key = 8 * (m & 1) + (lane & 7);
#pragma unroll
      for (int np = 0; np < 8; ++np) {
        uint32_t bf[4];
        ldsm_x4_t(bf, vbase + slab_off(key, 2 * np + (m >> 1)));
        mma16816<F16>(o[2 * np], pa, bf[0], bf[1]);
        mma16816<F16>(o[2 * np + 1], pa, bf[2], bf[3]);
      }
    }
    __syncwarp();                             // stage st is free for chunk t + kStages
    const bool seg_end = cur.local + 1 == cur.nc;
    if (p.ranks == 0 && (seg_end || cur.unit + 1 == x1)) {
      finish(seg_end && seg_local == 0);
      first_piece = false;
      fresh = true;
    }
  }
  cp_async_wait<0>();
  if (p.ranks == 0) return;

  // the cluster's CTAs hold a part of the segment each
  const int seg = blockIdx.x / p.ranks, rank = blockIdx.x - seg * p.ranks;
  const int b = seg / p.n_ag, a = seg - b * p.n_ag, n = p.ag_n[a], j0 = p.ag_start[a];
  gather();
  if (p.ranks == 1) {
    for (int r = warp; r < n; r += kWarps) {
      float m, l;
      const float4 x = joined(r, m, l);
      write_row<F16>(p, b, j0 + r, m, l, x, lane);
    }
    return;
  }
  for (int r = warp; r < n; r += kWarps) {    // this CTA's sums, in the place of the first partial
    float m, l;
    const float4 x = joined(r, m, l);
    __syncwarp();
    float* to = join + r * kPart;
    if (lane == 0) { to[0] = m; to[1] = l; }
    *reinterpret_cast<float4*>(to + 4 + lane * 4) = x;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int r = rank + warp * p.ranks; r < n; r += p.ranks * kWarps) {
    float ms[kMaxRanks], ls[kMaxRanks];
    float4 os[kMaxRanks];
#pragma unroll
    for (int y = 0; y < kMaxRanks; ++y) {     // past the last rank, its again
      const float* from = cluster.map_shared_rank(join, min(y, p.ranks - 1)) + r * kPart;
      ms[y] = from[0];
      ls[y] = from[1];
      os[y] = *reinterpret_cast<const float4*>(from + 4 + lane * 4);
    }
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int y = 0; y < kMaxRanks; ++y) m = fmaxf(m, ms[y]);
#pragma unroll
    for (int y = 0; y < kMaxRanks; ++y) {
      if (y >= p.ranks) break;
      const float f = weight2(ms[y], m);
      l += f * ls[y];
      x.x += f * os[y].x; x.y += f * os[y].y; x.z += f * os[y].z; x.w += f * os[y].w;
    }
    write_row<F16>(p, b, j0 + r, m, l, x, lane);
  }
  cluster.sync();                             // no CTA leaves while its sums may be read
}

// Joins the partials of the segments that the runs cut: CTA (c, r) looks at
// the boundary before run c; if that is the first one inside its segment, it
// sums the pieces of row r in the order of the runs.
template <bool F16>
__global__ void __launch_bounds__(kThreads)
paged_join_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ BlockScanSmem<kThreads> scan;
  __shared__ Place place;
  __shared__ float wm[kWarps], wl[kWarps];
  __shared__ float4 wo[kWarps][32];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // which pieces to join depends on the lengths alone, which were complete
  // before the first kernel let this one start; the pieces are awaited below
  ChunkScan lens(p, scan);
  const int64_t n_list = lens.total * p.n_ag;
  const int n_ctas = (int)(n_list < gridDim.x ? n_list : gridDim.x);
  const int c = blockIdx.x, r = blockIdx.y;
  int b = 0, a = 0, n = 0, slot0 = 0;          // sequence, listed KV head, pieces, first piece
  if (c > 0 && c < n_ctas) {
    const int64_t x = run_start(c, n_list, n_ctas);
    lens.locate(p, x, scan, &place);
    b = place.b;
    const int units = units_of(place.nc);
    a = (int)((x - place.before) / units);
    const int64_t u0 = place.before + (int64_t)a * units, s0 = u0 + kSegCost;   // chunks at [s0, s0 + nc)
    const int64_t x_prev = run_start(c - 1, n_list, n_ctas);
    // piece i comes from run c - 1 + i; the first is that run's last piece
    // unless nothing lies before the segment in it
    if (x > s0 && x_prev <= s0 && r < p.ag_n[a]) n = cta_of(s0 + place.nc - 1, n_list, n_ctas) - (c - 1) + 1;
    slot0 = (c - 1) * 2 + (x_prev >= u0 ? 0 : 1);
  }
  pdl_wait();                                 // every block: the next kernel relies on it
  if (n == 0) return;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 8;
  for (int i0 = warp; i0 < n; i0 += kWarps * kBatch) {
    float ms[kBatch], ls[kBatch];
    float4 os[kBatch];
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const int i = i0 + s * kWarps;
      ms[s] = -INFINITY; ls[s] = 0.f; os[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const int slot = i == 0 ? slot0 : (c - 1 + i) * 2;
        const float* part = p.part + ((int64_t)slot * p.rows + r) * kPart;
        ms[s] = part[0]; ls[s] = part[1];
        os[s] = *reinterpret_cast<const float4*>(part + 4 + lane * 4);
      }
    }
    float top = M;
#pragma unroll
    for (int s = 0; s < kBatch; ++s) top = fmaxf(top, ms[s]);
    const float f = weight2(M, top);
    L *= f; acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const float wt = weight2(ms[s], top);
      L += wt * ls[s];                        // NaN comes through, whatever its weight
      acc.x += wt * os[s].x; acc.y += wt * os[s].y; acc.z += wt * os[s].z; acc.w += wt * os[s].w;
    }
    M = top;
  }
  if (lane == 0) { wm[warp] = M; wl[warp] = L; }
  wo[warp][lane] = acc;
  __syncthreads();
  if (warp != 0) return;
  const float top = fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3]));
  L = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = weight2(wm[w], top);
    L += f * wl[w];
    const float4 v = wo[w][lane];
    acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
  }
  write_row<F16>(p, b, p.ag_start[a] + r, top, L, acc, lane);
}

// w_out = w + sum over the group's listed heads of exp(score - lse), for
// every slot of the sequence that is in a page. Bound by L2 and HBM: 8 bytes
// of weights and 4 bytes of score per listed head a slot. The batch's blocks of
// 256 slots form a list cut into equal runs, as above.
namespace {
constexpr int kWeightThreads = 256;
// all at once; 32 sequences of 1 to 16385 tokens, the whole call: 55 us, with
// 148 * 3 57, with 148 * 5 and 148 * 8 58
constexpr int kWeightCtas = 148 * 4;
struct SlotBlocks {
  static __device__ __forceinline__ int chunks(const DecodeParams& p, int b) {
    return (int)(((int64_t)seq_len(p.lens, b, p.max_len) + kWeightThreads - 1) / kWeightThreads);
  }
  static __device__ __forceinline__ int units(int chunks) { return chunks; }
};
}  // namespace
__global__ void __launch_bounds__(kWeightThreads)
paged_weights_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ BlockScanSmem<kWeightThreads> scan;
  __shared__ Place place;
  // Lengths, tables and the old weights are complete before this call's first
  // kernel lets the next one start; only scores and lse come from this call.
  LenScan<kWeightThreads, SlotBlocks> lens(p, scan);
  const int64_t n_list = lens.total * p.n_ag;
  const int n_ctas = (int)(n_list < gridDim.x ? n_list : gridDim.x);
  if ((int)blockIdx.x >= n_ctas) {
    pdl_wait();
    return;
  }
  const int64_t x0 = run_start(blockIdx.x, n_list, n_ctas), x1 = run_start(blockIdx.x + 1, n_list, n_ctas);
  lens.locate(p, x0, scan, &place);
  int b = place.b, nc = place.nc, a = (int)((x0 - place.before) / nc);
  int block = (int)((x0 - place.before) - (int64_t)a * nc);
  for (int64_t x = x0; x < x1; ++x) {
    const Span s = span_of(p, b);
    const int u = block * kWeightThreads + threadIdx.x;
    const int page = u < s.len ? page_of(p.c, b, u) : -1;
    const int g = p.ag_kv[a], n = p.ag_n[a], j0 = p.ag_start[a];
    const int64_t w = (((int64_t)max(page, 0) * p.c.Hkv + g) << p.c.page_shift) + (u & ((1 << p.c.page_shift) - 1));
    const float before = p.c.w[w];            // of page 0 where there is none: loads stay unconditional
    if (x == x0) pdl_wait();
    const int e = u < s.sink ? u : (u >= s.lo ? u - s.lo + s.sink : -1);
    const float* at = p.logits + ((int64_t)b * p.n_heads + j0) * p.att_cap + max(min(e, s.n - 1), 0);
    const float* lse2 = p.lse2 + (int64_t)b * p.n_heads + j0;
    float sum = 0.f;
    constexpr int kAhead = 8;                 // scores a thread keeps in flight
    for (int r0 = 0; r0 < n; r0 += kAhead) {
      float x_[kAhead], l_[kAhead];
#pragma unroll
      for (int r = 0; r < kAhead; ++r) {
        x_[r] = at[min(r0 + r, n - 1) * p.att_cap];
        l_[r] = lse2[min(r0 + r, n - 1)];
      }
#pragma unroll
      for (int r = 0; r < kAhead; ++r) sum += r0 + r >= n || l_[r] == -INFINITY ? 0.f : exp2f(x_[r] - l_[r]);
    }
    if (page >= 0) p.w_out[w] = before + (e >= 0 ? sum : 0.f);
    if (++block == nc && x + 1 < x1) {
      block = 0;
      if (++a == p.n_ag) {
        a = 0;
        do nc = SlotBlocks::chunks(p, ++b); while (nc == 0);
      }
    }
  }
}

namespace {
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
int64_t attended_cap(int max_len, int window, int sink) {
  const int64_t n = max_len <= window ? max_len : (int64_t)window + (sink < max_len - window ? sink : max_len - window);
  return (n + kChunk - 1) / kChunk * kChunk;
}
constexpr int kMaxCtas = 148 * kCtasPerSm;     // partials are sized for this many
}  // namespace

// LenScan adds up the units of a block's sequences in an int. (The slot blocks of
// the weights kernel are fewer: 256 sequences of at most 2^22.)
bool paged_decode_countable(int B, int max_len, int window, int sink) {
  const int64_t units = attended_cap(max_len, window, sink) / kChunk + kSegCost;
  return (B < kThreads ? B : kThreads) * units <= INT32_MAX;
}

size_t paged_decode_ws_bytes(int B, int max_len, int n_heads, int window, int sink, bool weights) {
  const int rows = n_heads < kGroup ? n_heads : kGroup;
  size_t n = kHeaderBytes + up256((size_t)2 * kMaxCtas * rows * kPart * sizeof(float));
  if (weights)
    n += up256((size_t)B * n_heads * sizeof(float)) +
         (size_t)B * n_heads * attended_cap(max_len, window, sink) * sizeof(float);
  return n;
}

// CTAs that share a segment, or 0 for runs over the whole list: where a
// segment of the longest length is at most six chunks a CTA and all CTAs run at
// once, the second kernel's launch and start (about 3 us) are more than what an
// even cut saves.
static int choose_ranks(int64_t segments, int64_t chunks) {
  int ranks = 1;
  while (ranks < kMaxRanks && chunks > ranks * 2 && segments * ranks * 2 <= kMaxCtas) ranks *= 2;
  return segments * ranks <= kMaxCtas && chunks <= ranks * 6 ? ranks : 0;
}

template <bool F16>
static cudaError_t launch_typed(const DecodeParams& p, int grid, cudaStream_t stream) {
  const size_t smem = sizeof(Smem);
  cudaError_t e =
      cudaFuncSetAttribute(paged_decode_kernel<F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (p.ranks <= 1) {
    e = launch_pdl(paged_decode_kernel<F16>, dim3(grid), dim3(kThreads), smem, stream, p);
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<F16>, p);
  }
  if (e != cudaSuccess || p.ranks > 0) return e;
  return launch_pdl(paged_join_kernel<F16>, dim3(grid, p.rows), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_paged_decode(const PagedView& c, const void* q, int64_t q_sb, int64_t q_sh, void* o, int64_t o_sb,
                                int64_t o_sh, bool f16, int B, int G, const int32_t* heads, int n_heads,
                                const int32_t* lens, int max_len, int window, int sink, float scale, float* lse,
                                float* w_out, void* ws, cudaStream_t stream) {
  DecodeParams p;
  p.c = c;
  p.q = static_cast<const char*>(q); p.q_sb = q_sb * 2; p.q_sh = q_sh * 2;
  p.o = static_cast<char*>(o); p.o_sb = o_sb * 2; p.o_sh = o_sh * 2;
  p.lens = lens; p.B = B; p.max_len = max_len; p.window = window; p.sink = sink;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.n_heads = n_heads;
  // the listed heads, KV head by KV head
  p.n_ag = 0; p.rows = 0;
  int n = 0;
  for (int g = 0; g < c.Hkv; ++g) {
    const int start = n;
    for (int j = 0; j < n_heads; ++j)
      if (heads[j] / G == g) {
        p.head[n] = (uint8_t)heads[j];
        p.out_row[n++] = (uint8_t)j;
      }
    if (n == start) continue;
    p.ag_kv[p.n_ag] = (uint8_t)g;
    p.ag_start[p.n_ag] = (uint8_t)start;
    p.ag_n[p.n_ag] = (uint8_t)(n - start);
    ++p.n_ag;
    if (n - start > p.rows) p.rows = n - start;
  }
  if (p.rows > kGroup) return cudaErrorInvalidValue;
  p.lse = lse;
  p.w_out = w_out;
  p.att_cap = attended_cap(max_len, window, sink);
  char* base = static_cast<char*>(ws);
  p.status = reinterpret_cast<int*>(base);
  p.part = reinterpret_cast<float*>(base + kHeaderBytes);
  p.lse2 = nullptr;
  p.logits = nullptr;
  if (w_out) {
    const int most_rows = n_heads < kGroup ? n_heads : kGroup;
    char* at = base + kHeaderBytes + up256((size_t)2 * kMaxCtas * most_rows * kPart * sizeof(float));
    p.lse2 = reinterpret_cast<float*>(at);
    p.logits = reinterpret_cast<float*>(at + up256((size_t)B * n_heads * sizeof(float)));
  }
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t segments = (int64_t)B * p.n_ag;
  p.ranks = choose_ranks(segments, p.att_cap / kChunk);
  int64_t grid = segments * (p.ranks > 0 ? p.ranks : p.att_cap / kChunk);
  const int most = sms * kCtasPerSm < kMaxCtas ? sms * kCtasPerSm : kMaxCtas;
  if (p.ranks == 0 && grid > most) grid = most;
  e = f16 ? launch_typed<true>(p, (int)grid, stream) : launch_typed<false>(p, (int)grid, stream);
  if (e != cudaSuccess) return e;
  if (w_out) {
    const int64_t blocks = ((int64_t)max_len + kWeightThreads - 1) / kWeightThreads * p.n_ag * B;
    e = launch_pdl(paged_weights_kernel, dim3((unsigned)(blocks < kWeightCtas ? blocks : kWeightCtas)),
                   dim3(kWeightThreads), 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace rtp
