// C ABI of the head norm and rotation and of the paged cache (declared in include/dsa.h):
// argument checks, and the decode pipelines over a paged cache.  As everywhere, every check
// happens on the host before anything is enqueued.
#include <algorithm>

#include "common.cuh"

namespace dsa_host {

static bool rope_args_ok(const double* inv_freq, int rotary_dim, int d) {
  if (!inv_freq) return rotary_dim == 0;
  return rotary_dim > 0 && rotary_dim <= d;
}
static bool rows_ok(const void* x, int64_t stride, int64_t heads, int d) {
  return x && aligned16(x) && stride >= heads * d && stride % 8 == 0 && stride <= 0x7FFFFFFFLL;
}
static bool head_dim_supported(int d) { return d == 32 || d == 64 || d == 128; }
static bool page_size_supported(int page_size) {
  return page_size >= 16 && page_size <= 1024 && (page_size & (page_size - 1)) == 0;
}
static int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

static dsa::HeadSeg head_seg(const void* x, int64_t x_stride, const void* weight, const double* inv_freq, int rotary,
                             int interleaved, int heads, int d, void* y, int64_t y_stride) {
  dsa::HeadSeg s{};
  s.x = static_cast<const uint16_t*>(x);
  s.x_stride = (int)x_stride;
  s.y = static_cast<uint16_t*>(y);
  s.y_stride = y_stride;
  s.g = static_cast<const uint16_t*>(weight);
  s.inv_freq = inv_freq;
  s.rotary = rotary;
  s.interleaved = interleaved != 0;
  s.heads = heads;
  s.D = d;
  return s;
}

// Checks shared by the norm-and-rotation calls, in the documented order.
static int norm_rope_args_status(const void* Q, int64_t q_stride, const void* K, int64_t k_stride, const void* q_weight,
                                 const void* k_weight, float eps, const double* inv_freq, int rotary_dim,
                                 const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int batch, int64_t total_q, int Hq, int Hk, int d) {
  if (total_q < 0 || batch < 1 || d < 1 || Hq < 1 || Hk < 0 || (Hk == 0) != (K == nullptr)) return DSA_ERR_INVALID_ARG;
  if (!rows_ok(Q, q_stride, Hq, d) || (K && !rows_ok(K, k_stride, Hk, d))) return DSA_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return DSA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !rope_args_ok(inv_freq, rotary_dim, d)) return DSA_ERR_INVALID_ARG;
  if ((!cu_seqlens_q && batch != 1) || (seqlens_k && !cu_seqlens_q)) return DSA_ERR_INVALID_ARG;
  if (!head_dim_supported(d) || rotary_dim % 16 != 0) return DSA_ERR_UNSUPPORTED;
  if (total_q > 0x7FFFFFFFLL / std::max(Hq, Hk)) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

static dsa::TokenMap token_map(const int32_t* positions, const int32_t* cu, const int32_t* lens, int batch, int64_t T) {
  dsa::TokenMap tk{};
  tk.positions = positions;
  tk.cu = cu;
  tk.lens = lens;
  tk.batch = batch;
  tk.T = (int)T;
  return tk;
}

// (6b) and (6c).  zero_outside: rows of tokens outside the sequences are written as zeros.
static int norm_rope_call(const void* Q, int64_t q_stride, const void* K, int64_t k_stride, const void* q_weight,
                          const void* k_weight, float eps, const double* inv_freq, int rotary_dim, int interleaved,
                          const int32_t* positions, const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int batch,
                          int64_t total_q, int Hq, int Hk, int d, void* Q_out, int64_t q_out_stride, void* K_out,
                          int64_t k_out_stride, bool zero_outside, void* stream) {
  const int st = norm_rope_args_status(Q, q_stride, K, k_stride, q_weight, k_weight, eps, inv_freq, rotary_dim,
                                       cu_seqlens_q, seqlens_k, batch, total_q, Hq, Hk, d);
  if (st == DSA_ERR_INVALID_ARG) return st;
  if (!rows_ok(Q_out, q_out_stride, Hq, d) || (K && !rows_ok(K_out, k_out_stride, Hk, d))) return DSA_ERR_INVALID_ARG;
  if (st != DSA_OK) return st;
  if (total_q == 0) return DSA_OK;
  dsa::HeadRowsParams p{};
  p.eps = eps;
  p.zero_outside = zero_outside && cu_seqlens_q;
  p.tk = token_map(positions, cu_seqlens_q, seqlens_k, batch, total_q);
  // K's few heads per token cost more per row: they go first
  if (K) p.seg[p.nseg++] = head_seg(K, k_stride, k_weight, inv_freq, rotary_dim, interleaved, Hk, d, K_out, k_out_stride);
  p.seg[p.nseg++] = head_seg(Q, q_stride, q_weight, inv_freq, rotary_dim, interleaved, Hq, d, Q_out, q_out_stride);
  return head_rows_fwd_launch(p, static_cast<cudaStream_t>(stream));
}

static int norm_rope_bwd_call(const void* Q, int64_t q_stride, const void* K, int64_t k_stride, const void* dQ_out,
                              int64_t dq_out_stride, const void* dK_out, int64_t dk_out_stride, const void* q_weight,
                              const void* k_weight, float eps, const double* inv_freq, int rotary_dim,
                              int interleaved, const int32_t* positions, const int32_t* cu_seqlens_q,
                              const int32_t* seqlens_k, int batch, int64_t total_q, int Hq, int Hk, int d, void* dQ,
                              int64_t dq_stride, void* dK, int64_t dk_stride, float* dq_weight, float* dk_weight,
                              void* workspace, size_t workspace_bytes, bool zero_outside, void* stream) {
  const int st = norm_rope_args_status(Q, q_stride, K, k_stride, q_weight, k_weight, eps, inv_freq, rotary_dim,
                                       cu_seqlens_q, seqlens_k, batch, total_q, Hq, Hk, d);
  if (st == DSA_ERR_INVALID_ARG) return st;
  if (!rows_ok(dQ_out, dq_out_stride, Hq, d) || (K && !rows_ok(dK_out, dk_out_stride, Hk, d)) ||
      !rows_ok(dQ, dq_stride, Hq, d) || (K && !rows_ok(dK, dk_stride, Hk, d)))
    return DSA_ERR_INVALID_ARG;
  if ((q_weight && !dq_weight) || (K && k_weight && !dk_weight)) return DSA_ERR_INVALID_ARG;
  if (st != DSA_OK) return st;
  const bool norms = q_weight || (K && k_weight);
  if (norms && total_q > 0 &&
      (!workspace || !aligned16(workspace) ||
       workspace_bytes < norm_rope_bwd_ws_bytes(total_q, Hq, K ? Hk : 0, d)))
    return DSA_ERR_WORKSPACE;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (total_q == 0) {  // the sums over no rows
    if (q_weight)
      if (const cudaError_t e = cudaMemsetAsync(dq_weight, 0, (size_t)d * 4, s); e != cudaSuccess) return cuda_fail(e);
    if (K && k_weight)
      if (const cudaError_t e = cudaMemsetAsync(dk_weight, 0, (size_t)d * 4, s); e != cudaSuccess) return cuda_fail(e);
    return DSA_OK;
  }
  dsa::HeadRowsParams p{};
  p.eps = eps;
  p.zero_outside = zero_outside && cu_seqlens_q;
  p.tk = token_map(positions, cu_seqlens_q, seqlens_k, batch, total_q);
  float* dg[2] = {dq_weight, dk_weight};
  p.seg[0] = head_seg(Q, q_stride, q_weight, inv_freq, rotary_dim, interleaved, Hq, d, dQ, dq_stride);
  p.seg[0].dy = static_cast<const uint16_t*>(dQ_out);
  p.seg[0].dy_stride = (int)dq_out_stride;
  p.nseg = 1;
  if (K) {
    p.seg[1] = head_seg(K, k_stride, k_weight, inv_freq, rotary_dim, interleaved, Hk, d, dK, dk_stride);
    p.seg[1].dy = static_cast<const uint16_t*>(dK_out);
    p.seg[1].dy_stride = (int)dk_out_stride;
    p.nseg = 2;
  }
  return head_rows_bwd_launch(p, static_cast<float*>(workspace), dg, s);
}

// Checks of a paged cache's description, in the documented order (a cache may be absent).
static int paged_args_status(const int32_t* table, int max_pages, const int32_t* lens, int batch, int num_pages,
                             int page_size) {
  if (!table || !lens || batch < 1 || max_pages < 1 || num_pages < 1 || page_size < 1)
    return DSA_ERR_INVALID_ARG;
  if (!page_size_supported(page_size) || (int64_t)num_pages * page_size > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}
static bool pool_ok(const void* cache, int64_t page_stride, int64_t page_elems) {
  return cache && aligned16(cache) && page_stride >= page_elems && page_stride % 8 == 0;
}

static int append_args_status(const void* K, int64_t k_stride, const void* V, int64_t v_stride, const void* k_idx,
                              int64_t ki_stride, const void* k_weight, const void* k_idx_weight, float eps,
                              const double* inv_freq, int rotary_dim, const double* idx_inv_freq, int idx_rotary_dim,
                              const int32_t* cu_seqlens_q, int64_t total_q, int Hkv, int d,
                              int d_I, const void* k_cache, int64_t k_page_stride, const void* v_cache,
                              int64_t v_page_stride, const void* ki_cache, int64_t ki_page_stride,
                              const int32_t* table, int max_pages, const int32_t* lens, int batch, int num_pages,
                              int page_size) {
  if (total_q < 0 || !cu_seqlens_q || Hkv < 1 || d < 1 || d_I < 0) return DSA_ERR_INVALID_ARG;
  const int st = paged_args_status(table, max_pages, lens, batch, num_pages, page_size);
  if (st == DSA_ERR_INVALID_ARG) return st;
  if (!rows_ok(K, k_stride, Hkv, d) || !rows_ok(V, v_stride, Hkv, d)) return DSA_ERR_INVALID_ARG;
  if ((k_idx == nullptr) != (d_I == 0) || (k_idx && !rows_ok(k_idx, ki_stride, 1, d_I))) return DSA_ERR_INVALID_ARG;
  const int64_t page_kv = (int64_t)page_size * Hkv * d, page_ki = (int64_t)page_size * d_I;
  if (!pool_ok(k_cache, k_page_stride, page_kv) || !pool_ok(v_cache, v_page_stride, page_kv)) return DSA_ERR_INVALID_ARG;
  if (k_idx && !pool_ok(ki_cache, ki_page_stride, page_ki)) return DSA_ERR_INVALID_ARG;
  if (!aligned16(k_weight) || !aligned16(k_idx_weight) || !(eps >= 0.f))
    return DSA_ERR_INVALID_ARG;
  if (!rope_args_ok(inv_freq, rotary_dim, d) || !rope_args_ok(idx_inv_freq, idx_rotary_dim, d_I))
    return DSA_ERR_INVALID_ARG;
  if (st != DSA_OK) return st;
  if (!head_dim_supported(d) || (k_idx && !head_dim_supported(d_I)) || rotary_dim % 16 != 0 || idx_rotary_dim % 16 != 0)
    return DSA_ERR_UNSUPPORTED;
  if (total_q > 0x7FFFFFFFLL / Hkv) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

// The rows that go into the pages: K and k_idx normed and rotated, V as it is.
static void paged_segs(dsa::HeadRowsParams& p, const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                       const void* k_idx, int64_t ki_stride, const void* k_weight, const void* k_idx_weight,
                       const double* inv_freq, int rotary, int interleaved, const double* idx_inv_freq, int idx_rotary,
                       int idx_interleaved, int Hkv, int d, int d_I, void* k_cache, int64_t k_page_stride,
                       void* v_cache, int64_t v_page_stride, void* ki_cache, int64_t ki_page_stride,
                       const int32_t* table, int max_pages, int num_pages, int page_size) {
  const int first = p.nseg;
  // the rows that cost most go first, the plain copies fill up behind them
  if (k_idx)
    p.seg[p.nseg++] = head_seg(k_idx, ki_stride, k_idx_weight, idx_inv_freq, idx_rotary, idx_interleaved, 1, d_I,
                               ki_cache, ki_page_stride);
  p.seg[p.nseg++] = head_seg(K, k_stride, k_weight, inv_freq, rotary, interleaved, Hkv, d, k_cache, k_page_stride);
  p.seg[p.nseg++] = head_seg(V, v_stride, nullptr, nullptr, 0, 0, Hkv, d, v_cache, v_page_stride);
  for (int i = first; i < p.nseg; ++i) p.seg[i].paged = 1;
  p.tk.table = table;
  p.tk.table_width = max_pages;
  p.tk.page_shift = log2_of(page_size);
  p.tk.num_pages = num_pages;
}

static int index_paged_args_status(const void* q_idx, const void* k_cache, int64_t page_stride, const void* w,
                                   const int32_t* table, int max_pages, const int32_t* lens, int batch, int num_pages,
                                   int page_size, int max_seqlen_k, int H_I, int d_I) {
  const int st = paged_args_status(table, max_pages, lens, batch, num_pages, page_size);
  if (st == DSA_ERR_INVALID_ARG) return st;
  if (!q_idx || !w || !aligned16(q_idx) || !aligned16(w) || max_seqlen_k < 0 || H_I < 1 || d_I < 1)
    return DSA_ERR_INVALID_ARG;
  if (!pool_ok(k_cache, page_stride, (int64_t)page_size * d_I)) return DSA_ERR_INVALID_ARG;
  if (st != DSA_OK) return st;
  if (!index_shape_supported(H_I, d_I) || (int64_t)batch * H_I > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  if (max_seqlen_k > 0x7FFFFFFF - 1024) return DSA_ERR_UNSUPPORTED;  // positions a few tiles past the end stay ints
  return DSA_OK;
}

static int index_paged_call(const void* q_idx, const void* k_cache, int64_t page_stride, const void* w,
                            const int32_t* table, int max_pages, const int32_t* lens, int batch, int num_pages,
                            int page_size, int max_seqlen_k, int H_I, int d_I, float* scores, int64_t ld, int* cu_q,
                            int* cu_k, cudaStream_t stream) {
  const int st = index_paged_args_status(q_idx, k_cache, page_stride, w, table, max_pages, lens, batch, num_pages,
                                         page_size, max_seqlen_k, H_I, d_I);
  if (st == DSA_ERR_INVALID_ARG) return st;
  if (!scores || !aligned16(scores) || ld < max_seqlen_k || ld < 1 || ld % 4 != 0) return DSA_ERR_INVALID_ARG;
  if (st != DSA_OK) return st;
  dsa::IndexPagedParams p{};
  p.w = static_cast<const uint16_t*>(w);
  p.lens = lens;
  p.table = table;
  p.batch = batch;
  p.table_width = max_pages;
  p.page_shift = log2_of(page_size);
  p.num_pages = num_pages;
  p.max_len = max_seqlen_k;
  p.scores = scores;
  p.ld = ld;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  return index_paged_launch(q_idx, k_cache, page_stride, p, H_I, d_I, stream);
}

static int sparse_attn_paged_args_status(const void* Q, const void* k_cache, int64_t k_page_stride, const void* v_cache,
                                         int64_t v_page_stride, const int32_t* indices, const int32_t* table,
                                         int max_pages, const int32_t* lens, int batch, int num_pages, int page_size,
                                         int Hq, int Hkv, int d, int k, float scale, const void* O) {
  const int st = paged_args_status(table, max_pages, lens, batch, num_pages, page_size);
  if (st == DSA_ERR_INVALID_ARG) return st;
  if (!Q || !indices || !O || !aligned16(Q) || !aligned16(O)) return DSA_ERR_INVALID_ARG;
  if (Hq < 1 || Hkv < 1 || d < 1 || k < 1 || !(scale > 0.f)) return DSA_ERR_INVALID_ARG;
  const int64_t page_kv = (int64_t)page_size * Hkv * d;
  if (!pool_ok(k_cache, k_page_stride, page_kv) || !pool_ok(v_cache, v_page_stride, page_kv)) return DSA_ERR_INVALID_ARG;
  if (st != DSA_OK) return st;
  if (!attn_shape_supported(Hq, Hkv, d) || k % 16 != 0 || k > 4096) return DSA_ERR_UNSUPPORTED;
  if (page_kv > 0x7FFFFFFFLL || (int64_t)batch * Hkv > 0x7FFFFFFFLL / 8) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

static int sparse_attn_paged_call(const void* Q, const void* k_cache, int64_t k_page_stride, const void* v_cache,
                                  int64_t v_page_stride, const int32_t* indices, const int32_t* table, int max_pages,
                                  const int32_t* lens, int batch, int num_pages, int page_size, int Hq, int Hkv, int d,
                                  int k, float scale, void* O, float* lse, cudaStream_t stream) {
  if (const int st = sparse_attn_paged_args_status(Q, k_cache, k_page_stride, v_cache, v_page_stride, indices, table,
                                                   max_pages, lens, batch, num_pages, page_size, Hq, Hkv, d, k, scale,
                                                   O);
      st != DSA_OK)
    return st;
  dsa::SAPagedParams p{};
  p.Q = static_cast<const uint16_t*>(Q);
  p.K = static_cast<const uint16_t*>(k_cache);
  p.V = static_cast<const uint16_t*>(v_cache);
  p.k_page_stride = k_page_stride;
  p.v_page_stride = v_page_stride;
  p.indices = indices;
  p.table = table;
  p.lens = lens;
  p.table_width = max_pages;
  p.page_shift = log2_of(page_size);
  p.num_pages = num_pages;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.k = k;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.O = static_cast<uint16_t*>(O);
  p.lse = lse;
  return sparse_attn_paged_launch(p, batch, d, stream);
}

// Scratch of the paged decode: the offsets that the top-k reads, the scores, its workspace.
struct DecodePagedWs {
  size_t cu_k, scores, topk, topk_bytes, bytes;
  int64_t ld;
};
static DecodePagedWs decode_paged_ws(int batch, int max_seqlen_k) {
  DecodePagedWs w;
  w.ld = (int64_t)round_up((size_t)std::max(max_seqlen_k, 1), 4);
  w.cu_k = round_up((size_t)(batch + 1) * sizeof(int), 256);
  w.scores = 2 * w.cu_k;
  w.topk = w.scores + round_up((size_t)batch * w.ld * sizeof(float), 256);
  w.topk_bytes = topk_ws_bytes(batch, w.ld);
  w.bytes = w.topk + round_up(w.topk_bytes, 256);
  return w;
}

static int decode_paged_args_status(const void* q_idx, const void* w, const void* Q, const void* k_cache,
                                    int64_t k_page_stride, const void* v_cache, int64_t v_page_stride,
                                    const void* ki_cache, int64_t ki_page_stride, const int32_t* table, int max_pages,
                                    const int32_t* lens, int batch, int num_pages, int page_size, int max_seqlen_k,
                                    int Hq, int Hkv, int d, int H_I, int d_I, int k, float scale,
                                    const int32_t* indices, const void* O) {
  const int a = index_paged_args_status(q_idx, ki_cache, ki_page_stride, w, table, max_pages, lens, batch, num_pages,
                                        page_size, max_seqlen_k, H_I, d_I);
  const int b = sparse_attn_paged_args_status(Q, k_cache, k_page_stride, v_cache, v_page_stride, indices, table,
                                              max_pages, lens, batch, num_pages, page_size, Hq, Hkv, d, k, scale, O);
  if (a == DSA_ERR_INVALID_ARG || b == DSA_ERR_INVALID_ARG) return DSA_ERR_INVALID_ARG;
  if (a != DSA_OK) return a;
  if (b != DSA_OK) return b;
  // the top-k's int32 offsets of the lengths
  return (int64_t)batch * max_seqlen_k > 0x7FFFFFFFLL ? DSA_ERR_UNSUPPORTED : DSA_OK;
}

static int decode_paged_run(const void* q_idx, const void* w, const void* Q, const void* k_cache, int64_t k_page_stride,
                            const void* v_cache, int64_t v_page_stride, const void* ki_cache, int64_t ki_page_stride,
                            const int32_t* table, int max_pages, const int32_t* lens, int batch, int num_pages,
                            int page_size, int max_seqlen_k, int Hq, int Hkv, int d, int H_I, int d_I, int k,
                            float scale, int32_t* indices, void* O, float* lse, void* workspace,
                            cudaStream_t stream) {
  const DecodePagedWs L = decode_paged_ws(batch, max_seqlen_k);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int* cu_q = reinterpret_cast<int*>(ws);
  int* cu_k = reinterpret_cast<int*>(ws + L.cu_k);
  float* scores = reinterpret_cast<float*>(ws + L.scores);
  int st = index_paged_call(q_idx, ki_cache, ki_page_stride, w, table, max_pages, lens, batch, num_pages, page_size,
                            max_seqlen_k, H_I, d_I, scores, L.ld, cu_q, cu_k, stream);
  if (st != DSA_OK) return st;
  st = topk_launch(scores, L.ld, cu_q, cu_k, batch, 0, batch, k, indices, (int)L.ld, L.topk_bytes ? ws + L.topk : nullptr,
                   L.topk_bytes, stream);
  if (st != DSA_OK) return st;
  return sparse_attn_paged_call(Q, k_cache, k_page_stride, v_cache, v_page_stride, indices, table, max_pages, lens,
                                batch, num_pages, page_size, Hq, Hkv, d, k, scale, O, lse, stream);
}

}  // namespace dsa_host

using namespace dsa_host;

extern "C" {

DSA_API int dsa_norm_rope(const void* Q, int64_t q_stride, const void* K, int64_t k_stride, const void* q_weight,
                          const void* k_weight, float eps, const double* inv_freq, int rotary_dim, int interleaved,
                          const int32_t* positions, const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int batch,
                          int64_t total_q, int Hq, int Hk, int d, void* Q_out, int64_t q_out_stride, void* K_out,
                          int64_t k_out_stride, void* stream) {
  return norm_rope_call(Q, q_stride, K, k_stride, q_weight, k_weight, eps, inv_freq, rotary_dim, interleaved, positions,
                        cu_seqlens_q, seqlens_k, batch, total_q, Hq, Hk, d, Q_out, q_out_stride, K_out, k_out_stride, false,
                        stream);
}

DSA_API int dsa_norm_rope_zeroed(const void* Q, int64_t q_stride, const void* K, int64_t k_stride, const void* q_weight,
                                 const void* k_weight, float eps, const double* inv_freq, int rotary_dim, int interleaved,
                                 const int32_t* positions, const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int batch,
                                 int64_t total_q, int Hq, int Hk, int d, void* Q_out, int64_t q_out_stride, void* K_out,
                                 int64_t k_out_stride, void* stream) {
  return norm_rope_call(Q, q_stride, K, k_stride, q_weight, k_weight, eps, inv_freq, rotary_dim, interleaved, positions,
                        cu_seqlens_q, seqlens_k, batch, total_q, Hq, Hk, d, Q_out, q_out_stride, K_out, k_out_stride, true,
                        stream);
}

DSA_API size_t dsa_norm_rope_bwd_workspace_size(int64_t total_q, int Hq, int Hk, int d) {
  if (total_q < 0 || Hq < 1 || Hk < 0 || !head_dim_supported(d)) return 0;
  return norm_rope_bwd_ws_bytes(total_q, Hq, Hk, d);
}

DSA_API int dsa_norm_rope_bwd(const void* Q, int64_t q_stride, const void* K, int64_t k_stride, const void* dQ_out,
                              int64_t dq_out_stride, const void* dK_out, int64_t dk_out_stride, const void* q_weight,
                              const void* k_weight, float eps, const double* inv_freq, int rotary_dim,
                              int interleaved, const int32_t* positions, const int32_t* cu_seqlens_q,
                              const int32_t* seqlens_k, int batch, int64_t total_q, int Hq, int Hk, int d, void* dQ,
                              int64_t dq_stride, void* dK, int64_t dk_stride, float* dq_weight, float* dk_weight,
                              void* workspace, size_t workspace_bytes, void* stream) {
  return norm_rope_bwd_call(Q, q_stride, K, k_stride, dQ_out, dq_out_stride, dK_out, dk_out_stride, q_weight, k_weight,
                            eps, inv_freq, rotary_dim, interleaved, positions, cu_seqlens_q, seqlens_k, batch, total_q,
                            Hq, Hk, d, dQ, dq_stride, dK, dk_stride, dq_weight, dk_weight, workspace, workspace_bytes,
                            false, stream);
}

DSA_API int dsa_norm_rope_bwd_zeroed(const void* Q, int64_t q_stride, const void* K, int64_t k_stride, const void* dQ_out,
                                     int64_t dq_out_stride, const void* dK_out, int64_t dk_out_stride, const void* q_weight,
                                     const void* k_weight, float eps, const double* inv_freq, int rotary_dim,
                                     int interleaved, const int32_t* positions, const int32_t* cu_seqlens_q,
                                     const int32_t* seqlens_k, int batch, int64_t total_q, int Hq, int Hk, int d, void* dQ,
                                     int64_t dq_stride, void* dK, int64_t dk_stride, float* dq_weight, float* dk_weight,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  return norm_rope_bwd_call(Q, q_stride, K, k_stride, dQ_out, dq_out_stride, dK_out, dk_out_stride, q_weight, k_weight,
                            eps, inv_freq, rotary_dim, interleaved, positions, cu_seqlens_q, seqlens_k, batch, total_q,
                            Hq, Hk, d, dQ, dq_stride, dK, dk_stride, dq_weight, dk_weight, workspace, workspace_bytes,
                            true, stream);
}

DSA_API int dsa_cache_append(const void* K, int64_t k_stride, const void* V, int64_t v_stride, const void* k_idx,
                             int64_t k_idx_stride, const void* k_weight, const void* k_idx_weight, float eps,
                             const double* inv_freq, int rotary_dim, int interleaved, const double* idx_inv_freq,
                             int idx_rotary_dim, int idx_interleaved, const int32_t* positions,
                             const int32_t* cu_seqlens_q, int64_t total_q, int Hkv, int d, int d_I, void* k_cache,
                             int64_t k_page_stride, void* v_cache, int64_t v_page_stride, void* k_idx_cache,
                             int64_t k_idx_page_stride, const int32_t* block_table, int max_pages,
                             const int32_t* seqlens_k, int batch, int num_pages, int page_size, void* stream) {
  if (const int st = append_args_status(K, k_stride, V, v_stride, k_idx, k_idx_stride, k_weight, k_idx_weight, eps,
                                        inv_freq, rotary_dim, idx_inv_freq, idx_rotary_dim, cu_seqlens_q, total_q,
                                        Hkv, d, d_I, k_cache, k_page_stride, v_cache, v_page_stride,
                                        k_idx_cache, k_idx_page_stride, block_table, max_pages, seqlens_k, batch,
                                        num_pages, page_size);
      st != DSA_OK)
    return st;
  if (total_q == 0) return DSA_OK;
  dsa::HeadRowsParams p{};
  p.eps = eps;
  p.tk = token_map(positions, cu_seqlens_q, seqlens_k, batch, total_q);
  paged_segs(p, K, k_stride, V, v_stride, k_idx, k_idx_stride, k_weight, k_idx_weight, inv_freq, rotary_dim, interleaved,
             idx_inv_freq, idx_rotary_dim, idx_interleaved, Hkv, d, d_I, k_cache, k_page_stride, v_cache, v_page_stride,
             k_idx_cache, k_idx_page_stride, block_table, max_pages, num_pages, page_size);
  return head_rows_fwd_launch(p, static_cast<cudaStream_t>(stream));
}

DSA_API int dsa_index_paged(const void* q_idx, const void* k_idx_cache, int64_t k_idx_page_stride, const void* w,
                            const int32_t* block_table, int max_pages, const int32_t* seqlens_k, int batch,
                            int num_pages, int page_size, int max_seqlen_k, int H_I, int d_I, float* scores,
                            int64_t ld_scores, void* stream) {
  return index_paged_call(q_idx, k_idx_cache, k_idx_page_stride, w, block_table, max_pages, seqlens_k, batch, num_pages,
                          page_size, max_seqlen_k, H_I, d_I, scores, ld_scores, nullptr, nullptr,
                          static_cast<cudaStream_t>(stream));
}

DSA_API int dsa_sparse_attn_decode_paged(const void* Q, const void* k_cache, int64_t k_page_stride,
                                         const void* v_cache, int64_t v_page_stride, const int32_t* indices,
                                         const int32_t* block_table, int max_pages, const int32_t* seqlens_k,
                                         int batch, int num_pages, int page_size, int Hq, int Hkv, int d, int k,
                                         float scale, void* O, float* lse, void* stream) {
  return sparse_attn_paged_call(Q, k_cache, k_page_stride, v_cache, v_page_stride, indices, block_table, max_pages,
                                seqlens_k, batch, num_pages, page_size, Hq, Hkv, d, k, scale, O, lse,
                                static_cast<cudaStream_t>(stream));
}

DSA_API size_t dsa_decode_paged_workspace_size(int batch, int max_seqlen_k) {
  if (batch < 1 || max_seqlen_k < 0) return 0;
  return decode_paged_ws(batch, max_seqlen_k).bytes;
}

DSA_API int dsa_decode_paged(const void* q_idx, const void* w, const void* Q, const void* k_cache,
                             int64_t k_page_stride, const void* v_cache, int64_t v_page_stride,
                             const void* k_idx_cache, int64_t k_idx_page_stride, const int32_t* block_table,
                             int max_pages, const int32_t* seqlens_k, int batch, int num_pages, int page_size,
                             int max_seqlen_k, int Hq, int Hkv, int d, int H_I, int d_I, int k, float scale,
                             int32_t* indices, void* O, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (const int st = decode_paged_args_status(q_idx, w, Q, k_cache, k_page_stride, v_cache, v_page_stride, k_idx_cache,
                                              k_idx_page_stride, block_table, max_pages, seqlens_k, batch, num_pages,
                                              page_size, max_seqlen_k, Hq, Hkv, d, H_I, d_I, k, scale, indices, O);
      st != DSA_OK)
    return st;
  if (!workspace || !aligned16(workspace) || workspace_bytes < dsa_decode_paged_workspace_size(batch, max_seqlen_k))
    return DSA_ERR_WORKSPACE;
  return decode_paged_run(q_idx, w, Q, k_cache, k_page_stride, v_cache, v_page_stride, k_idx_cache, k_idx_page_stride,
                          block_table, max_pages, seqlens_k, batch, num_pages, page_size, max_seqlen_k, Hq, Hkv, d, H_I,
                          d_I, k, scale, indices, O, lse, workspace, static_cast<cudaStream_t>(stream));
}

DSA_API size_t dsa_decode_step_paged_workspace_size(int batch, int max_seqlen_k, int Hq, int d, int H_I, int d_I) {
  if (batch < 1 || max_seqlen_k < 0 || Hq < 1 || d < 1 || H_I < 1 || d_I < 1) return 0;
  return round_up((size_t)batch * Hq * d * 2, 256) + round_up((size_t)batch * H_I * d_I * 2, 256) +
         dsa_decode_paged_workspace_size(batch, max_seqlen_k);
}

DSA_API int dsa_decode_step_paged(const void* q_idx, int64_t q_idx_stride, const void* w, const void* Q,
                                  int64_t q_stride, const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                                  const void* k_idx, int64_t k_idx_stride, const void* q_weight, const void* k_weight,
                                  const void* q_idx_weight, const void* k_idx_weight, float eps,
                                  const double* inv_freq, int rotary_dim, int interleaved,
                                  const double* idx_inv_freq, int idx_rotary_dim, int idx_interleaved,
                                  const int32_t* positions, void* k_cache, int64_t k_page_stride, void* v_cache,
                                  int64_t v_page_stride, void* k_idx_cache, int64_t k_idx_page_stride,
                                  const int32_t* block_table, int max_pages, const int32_t* seqlens_k, int batch,
                                  int num_pages, int page_size, int max_seqlen_k, int Hq, int Hkv, int d, int H_I,
                                  int d_I, int k, float scale, int32_t* indices, void* O, float* lse,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  // the token map needs no offsets: token b is the one new token of sequence b
  int st = append_args_status(K, k_stride, V, v_stride, k_idx, k_idx_stride, k_weight, k_idx_weight, eps, inv_freq,
                              rotary_dim, idx_inv_freq, idx_rotary_dim, seqlens_k, batch, Hkv, d, d_I,
                              k_cache, k_page_stride, v_cache, v_page_stride, k_idx_cache, k_idx_page_stride,
                              block_table, max_pages, seqlens_k, batch, num_pages, page_size);
  if (st == DSA_ERR_INVALID_ARG) return st;
  if (!k_idx || Hq < 1 || H_I < 1 || !rows_ok(Q, q_stride, Hq, d) || !rows_ok(q_idx, q_idx_stride, H_I, d_I) ||
      !aligned16(q_weight) || !aligned16(q_idx_weight))
    return DSA_ERR_INVALID_ARG;
  const int st2 = decode_paged_args_status(q_idx, w, Q, k_cache, k_page_stride, v_cache, v_page_stride, k_idx_cache,
                                           k_idx_page_stride, block_table, max_pages, seqlens_k, batch, num_pages,
                                           page_size, max_seqlen_k, Hq, Hkv, d, H_I, d_I, k, scale, indices, O);
  if (st2 == DSA_ERR_INVALID_ARG) return st2;
  if (st != DSA_OK) return st;
  if (st2 != DSA_OK) return st2;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < dsa_decode_step_paged_workspace_size(batch, max_seqlen_k, Hq, d, H_I, d_I))
    return DSA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  void* q_out = ws;
  ws += round_up((size_t)batch * Hq * d * 2, 256);
  void* qi_out = ws;
  ws += round_up((size_t)batch * H_I * d_I * 2, 256);
  dsa::HeadRowsParams p{};
  p.eps = eps;
  p.tk = token_map(positions, nullptr, seqlens_k, batch, batch);
  p.seg[p.nseg++] = head_seg(Q, q_stride, q_weight, inv_freq, rotary_dim, interleaved, Hq, d, q_out, (int64_t)Hq * d);
  p.seg[p.nseg++] = head_seg(q_idx, q_idx_stride, q_idx_weight, idx_inv_freq, idx_rotary_dim, idx_interleaved, H_I, d_I,
                             qi_out, (int64_t)H_I * d_I);
  paged_segs(p, K, k_stride, V, v_stride, k_idx, k_idx_stride, k_weight, k_idx_weight, inv_freq, rotary_dim, interleaved,
             idx_inv_freq, idx_rotary_dim, idx_interleaved, Hkv, d, d_I, k_cache, k_page_stride, v_cache, v_page_stride,
             k_idx_cache, k_idx_page_stride, block_table, max_pages, num_pages, page_size);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (st = head_rows_fwd_launch(p, s); st != DSA_OK) return st;
  return decode_paged_run(qi_out, w, q_out, k_cache, k_page_stride, v_cache, v_page_stride, k_idx_cache,
                          k_idx_page_stride, block_table, max_pages, seqlens_k, batch, num_pages, page_size,
                          max_seqlen_k, Hq, Hkv, d, H_I, d_I, k, scale, indices, O, lse, ws, s);
}

}  // extern "C"
