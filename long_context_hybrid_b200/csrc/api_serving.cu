// C ABI of the serving calls (packed prompts, paged cache): argument
// validation on the host, then dispatch. See include/rtp.h for the contract.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rtp.h"
#include "api_check.h"
#include "rtp_common.cuh"
#include "rtp_internal.h"

using namespace rtp;

namespace {

constexpr int64_t kMaxRows = 1 << 30;

// A softmax scale that stays finite in the log2 domain.
bool scale_ok(float s) { return s > 0.f && s < 1e38f; }

bool dtype_ok(rtp_dtype d) { return d == RTP_BF16 || d == RTP_F16; }

// Element strides of a dimension of n rows: a multiple of 8, and rows do not
// overlap (a dimension of one row is never stepped over).
bool step_ok(int64_t s, int64_t n) { return n <= 1 || (s % 8 == 0 && s >= RTP_D); }
bool packed_strides_ok(rtp_strides s, int64_t rows, int heads) { return step_ok(s.n, rows) && step_ok(s.h, heads); }

// Strides of single-row dimensions are the caller's accident: replaced by
// what the tensor maps accept.
Tensor4 packed_tensor(const void* p, rtp_strides s, int64_t rows, int heads) {
  return Tensor4{p, 0, rows > 1 ? s.n : (int64_t)heads * RTP_D, heads > 1 ? s.h : RTP_D};
}

// Checks a paged cache and makes the kernels' view of it.
rtp_status make_view(const rtp_paged_cache* c, PagedView* view) {
  if (!c || !c->k || !c->v || !c->table) return RTP_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->Hkv < 1) return RTP_ERR_INVALID_ARG;
  if (c->table_stride < c->max_pages) return RTP_ERR_INVALID_ARG;
  if (c->Hkv > kMaxHeads) return RTP_ERR_UNSUPPORTED;
  if ((c->page_size & (c->page_size - 1)) != 0 || c->page_size > 65536) return RTP_ERR_UNSUPPORTED;
  const int64_t capacity = (int64_t)c->max_pages * c->page_size;
  if (capacity > kMaxRows) return RTP_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v)) return RTP_ERR_INVALID_ARG;
  for (const rtp_strides* s : {&c->ks, &c->vs})
    if (!step_ok(s->b, c->num_pages) || !step_ok(s->n, c->page_size) || !step_ok(s->h, c->Hkv))
      return RTP_ERR_INVALID_ARG;
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  view->k = static_cast<char*>(c->k);
  view->k_sp = c->ks.b * 2; view->k_sn = c->ks.n * 2; view->k_sh = c->ks.h * 2;
  view->v = static_cast<char*>(c->v);
  view->v_sp = c->vs.b * 2; view->v_sn = c->vs.n * 2; view->v_sh = c->vs.h * 2;
  view->w = c->weights;
  view->table = c->table;
  view->table_stride = c->table_stride;
  view->capacity = capacity;
  view->num_pages = c->num_pages;
  view->page_shift = shift;
  view->Hkv = c->Hkv;
  return RTP_OK;
}

bool same_strides(rtp_strides a, rtp_strides b) { return a.b == b.b && a.n == b.n && a.h == b.h; }

}  // namespace

extern "C" {

size_t rtp_workspace_size_attn_packed(void) { return kStatusBytes; }

rtp_status rtp_attn_packed(const void* q, rtp_strides qs, const void* k, rtp_strides ks, const void* v,
                           rtp_strides vs, void* o, rtp_strides os, rtp_dtype dtype, int T, int Hq, int Hkv,
                           const int32_t* heads, int n_heads, const int32_t* cu_seqlens, int S, int window,
                           float scale, float* lse, void* ws, size_t ws_bytes, rtp_stream_t stream) {
  if (T < 0 || S < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !cu_seqlens) return RTP_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || window < 1 || !scale_ok(scale)) return RTP_ERR_INVALID_ARG;
  rtp_status st = check_heads(heads, n_heads, Hq);
  if (st != RTP_OK) return st;
  if (Hq > 256 || T > kMaxRows || S > kMaxRows) return RTP_ERR_UNSUPPORTED;
  if (((int64_t)T / 128 + S) * n_heads > INT32_MAX) return RTP_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < kStatusBytes || !aligned256(ws)) return RTP_ERR_WORKSPACE;
  if (T > 0) {
    if (!q || !k || !v || !o) return RTP_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return RTP_ERR_INVALID_ARG;
    if (!packed_strides_ok(qs, T, Hq) || !packed_strides_ok(ks, T, Hkv) || !packed_strides_ok(vs, T, Hkv) ||
        !packed_strides_ok(os, T, Hq))
      return RTP_ERR_INVALID_ARG;
  }
  if ((st = check_device()) != RTP_OK) return st;
  if (T == 0)
    return from_cuda(cudaMemsetAsync(ws, 0, sizeof(int), (cudaStream_t)stream));
  const Tensor4 to = packed_tensor(o, os, T, Hq);
  return from_cuda(launch_attn_packed(packed_tensor(q, qs, T, Hq), packed_tensor(k, ks, T, Hkv),
                                      packed_tensor(v, vs, T, Hkv), o, to.sn, to.sh, dtype == RTP_F16, T, Hq, Hkv,
                                      heads, n_heads, cu_seqlens, S, window, scale, lse, static_cast<int*>(ws),
                                      (cudaStream_t)stream));
}

size_t rtp_workspace_size_attn_key_weights(void) { return kStatusBytes; }

rtp_status rtp_attn_key_weights(const void* q, rtp_strides qs, const void* k, rtp_strides ks, rtp_dtype dtype, int T,
                                int Hq, int Hkv, const int32_t* heads, int n_heads, const int32_t* cu_seqlens, int S,
                                const float* lse, int n_obs, int window, float scale, float* weights, void* ws,
                                size_t ws_bytes, rtp_stream_t stream) {
  if (T < 0 || S < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !cu_seqlens) return RTP_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || window < 1 || n_obs < 1 || !scale_ok(scale)) return RTP_ERR_INVALID_ARG;
  rtp_status st = check_heads(heads, n_heads, Hq);
  if (st != RTP_OK) return st;
  if (Hq > 256 || T > kMaxRows || S > kMaxRows) return RTP_ERR_UNSUPPORTED;
  if (((int64_t)T / 128 + S) * n_heads > INT32_MAX) return RTP_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < kStatusBytes || !aligned256(ws)) return RTP_ERR_WORKSPACE;
  if (T > 0) {
    if (!q || !k || !lse || !weights || !aligned16(q) || !aligned16(k)) return RTP_ERR_INVALID_ARG;
    if (!packed_strides_ok(qs, T, Hq) || !packed_strides_ok(ks, T, Hkv)) return RTP_ERR_INVALID_ARG;
  }
  if ((st = check_device()) != RTP_OK) return st;
  if (T == 0)
    return from_cuda(cudaMemsetAsync(ws, 0, sizeof(int), (cudaStream_t)stream));
  return from_cuda(launch_key_weights(packed_tensor(q, qs, T, Hq), packed_tensor(k, ks, T, Hkv), dtype == RTP_F16, T,
                                      Hq, Hkv, heads, n_heads, cu_seqlens, S, lse, n_obs, window, scale, weights,
                                      static_cast<int*>(ws), (cudaStream_t)stream));
}

rtp_status rtp_paged_append(const rtp_paged_cache* cache, const void* k, rtp_strides ks, const void* v,
                            rtp_strides vs, const float* weights, int T, const int32_t* cu_seqlens, int S,
                            const int32_t* pos, rtp_stream_t stream) {
  PagedView view;
  rtp_status st = make_view(cache, &view);
  if (st != RTP_OK) return st;
  if (T < 0 || S < 1 || !cu_seqlens || !pos) return RTP_ERR_INVALID_ARG;
  if (weights && !cache->weights) return RTP_ERR_INVALID_ARG;
  if (T > kMaxRows || S > kMaxRows) return RTP_ERR_UNSUPPORTED;
  if (T > 0) {
    if (!k || !v || !aligned16(k) || !aligned16(v)) return RTP_ERR_INVALID_ARG;
    if (!packed_strides_ok(ks, T, view.Hkv) || !packed_strides_ok(vs, T, view.Hkv)) return RTP_ERR_INVALID_ARG;
  }
  if ((st = check_device()) != RTP_OK) return st;
  if (T == 0) return RTP_OK;
  const Tensor4 tk = packed_tensor(k, ks, T, view.Hkv), tv = packed_tensor(v, vs, T, view.Hkv);
  return from_cuda(launch_paged_append(view, k, tk.sn, tk.sh, v, tv.sn, tv.sh, weights, cu_seqlens, pos, S, T,
                                       (cudaStream_t)stream));
}

size_t rtp_workspace_size_paged_attn_decode(int B, int max_len, int n_heads, int window, int sink,
                                            int with_weights) {
  if (B < 1 || max_len < 1 || n_heads < 1 || window < 1 || sink < 0) return kStatusBytes;
  return paged_decode_ws_bytes(B, max_len, n_heads, window, sink, with_weights != 0);
}

rtp_status rtp_paged_attn_decode(const void* q, rtp_strides qs, const rtp_paged_cache* cache, const int32_t* lens,
                                 int max_len, void* o, rtp_strides os, rtp_dtype dtype, int B, int Hq,
                                 const int32_t* heads, int n_heads, int window, int sink, float scale, float* lse,
                                 float* weights_out, void* ws, size_t ws_bytes, rtp_stream_t stream) {
  PagedView view;
  rtp_status st = make_view(cache, &view);
  if (st != RTP_OK) return st;
  if (!q || !o || !lens || !dtype_ok(dtype)) return RTP_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hq % view.Hkv != 0 || max_len < 1 || max_len > view.capacity) return RTP_ERR_INVALID_ARG;
  if (window < 1 || sink < 0 || !scale_ok(scale)) return RTP_ERR_INVALID_ARG;
  if (weights_out && !cache->weights) return RTP_ERR_INVALID_ARG;
  if ((st = check_heads(heads, n_heads, Hq)) != RTP_OK) return st;
  if (Hq > 256 || Hq / view.Hkv > 16 || B > 65535) return RTP_ERR_UNSUPPORTED;
  if (!paged_decode_countable(B, max_len, window, sink)) return RTP_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(o)) return RTP_ERR_INVALID_ARG;
  if (!step_ok(qs.b, B) || !step_ok(qs.h, Hq) || !step_ok(os.b, B) || !step_ok(os.h, Hq)) return RTP_ERR_INVALID_ARG;
  const size_t need = paged_decode_ws_bytes(B, max_len, n_heads, window, sink, weights_out != nullptr);
  if (!ws || ws_bytes < need || !aligned256(ws)) return RTP_ERR_WORKSPACE;
  if ((st = check_device()) != RTP_OK) return st;
  return from_cuda(launch_paged_decode(view, q, qs.b, qs.h, o, os.b, os.h, dtype == RTP_F16, B, Hq / view.Hkv, heads,
                                       n_heads, lens, max_len, window, sink, scale, lse, weights_out, ws,
                                       (cudaStream_t)stream));
}

rtp_status rtp_cache_evict(const rtp_paged_cache* src, const rtp_paged_cache* dst, int B, const int32_t* lens,
                           int max_len, int budget, int sink, int recent, int32_t* idx, int32_t* new_lens,
                           rtp_stream_t stream) {
  PagedView from, to;
  rtp_status st = make_view(src, &from);
  if (st != RTP_OK || (st = make_view(dst, &to)) != RTP_OK) return st;
  if (!src->weights || !dst->weights || !lens || !idx || !new_lens || new_lens == lens) return RTP_ERR_INVALID_ARG;
  if (from.Hkv != to.Hkv || B < 1 || max_len < 1 || max_len > from.capacity) return RTP_ERR_INVALID_ARG;
  if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget) return RTP_ERR_INVALID_ARG;
  const int keep = budget < max_len ? budget : max_len;
  if (to.capacity < keep) return RTP_ERR_INVALID_ARG;
  // in place: the same pages through the same table; or pages of its own
  const bool same_k = src->k == dst->k, same_v = src->v == dst->v, same_w = src->weights == dst->weights;
  const bool same_table = src->table == dst->table && src->table_stride == dst->table_stride;
  const bool in_place = same_k && same_v && same_w && same_table;
  if (in_place && (!same_strides(src->ks, dst->ks) || !same_strides(src->vs, dst->vs) ||
                   src->page_size != dst->page_size || src->num_pages != dst->num_pages))
    return RTP_ERR_INVALID_ARG;
  if (!in_place && same_table && (same_k || same_v || same_w)) return RTP_ERR_INVALID_ARG;
  if ((int64_t)B * from.Hkv > 65535) return RTP_ERR_UNSUPPORTED;
  if ((st = check_device()) != RTP_OK) return st;
  return from_cuda(launch_cache_evict(from, to, in_place, B, lens, max_len, budget, sink, recent, idx, new_lens,
                                      (cudaStream_t)stream));
}

}  // extern "C"
