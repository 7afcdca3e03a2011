// The extern "C" entry points of bsa_seq.h: host-side validation of every
// argument (nothing is launched on error) and the launches on the caller's
// stream.
#include <climits>
#include <cmath>
#include <cstring>

#include "seq_internal.cuh"

namespace {

using bsa::SeqGeo;

#define SEQ_TRY(x)               \
  do {                           \
    bsa_status _s = (x);         \
    if (_s != BSA_OK) return _s; \
  } while (0)

struct Range {
  explicit Range(const char* name) {
    bsa::clear_error();
    bsa::range_push(name);
  }
  ~Range() { bsa::range_pop(); }
};
#define SEQ_RANGE() Range seq_range_(__func__)

template <typename... A>
bsa_status fail(bsa_status st, const char* fmt, A... a) {
  return bsa::set_error(st, fmt, a...);
}

bsa_status make_geo(const bsa_seq_problem* p, SeqGeo* g) {
  if (!p) return fail(BSA_ERR_INVALID_ARG, "problem is NULL");
  if (p->head_dim != 64 && p->head_dim != 128)
    return fail(BSA_ERR_UNSUPPORTED, "head_dim %d: only 64 and 128 are supported", p->head_dim);
  if (p->kv_heads < 1 || p->heads < 1 || p->heads > 65535)
    return fail(BSA_ERR_SHAPE, "heads (%d) must lie in 1..65535 and kv_heads (%d) be >= 1",
                p->heads, p->kv_heads);
  if (p->heads % p->kv_heads)
    return fail(BSA_ERR_SHAPE, "kv_heads %d does not divide heads %d", p->kv_heads, p->heads);
  if (p->dtype != BSA_DTYPE_BF16 && p->dtype != BSA_DTYPE_FP16)
    return fail(BSA_ERR_INVALID_ARG, "dtype %d is not a bsa_dtype", p->dtype);
  if (p->causal != 0 && p->causal != 1)
    return fail(BSA_ERR_INVALID_ARG, "causal must be 0 or 1, not %d", p->causal);
  if (!(std::isfinite(p->softmax_scale) && p->softmax_scale > 0.f))
    return fail(BSA_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  g->heads = p->heads;
  g->kv_heads = p->kv_heads;
  g->group = p->heads / p->kv_heads;
  g->d = p->head_dim;
  g->fp16 = p->dtype == BSA_DTYPE_FP16;
  g->causal = p->causal != 0;
  g->scale = p->softmax_scale;
  return BSA_OK;
}

bsa_status check_ptr(const void* p, const char* name, unsigned align = 16) {
  if (!p) return fail(BSA_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return fail(BSA_ERR_INVALID_ARG, "%s is not %u-byte aligned", name, align);
  return BSA_OK;
}

// A [rows, heads, d] tensor.  The stride of an axis of extent 1 is replaced
// by the contiguous one; `own` (outputs): rows and heads must not overlap.
bsa_status check_rows(bsa::Rows* r, const void* p, int64_t sn, int64_t sh, int64_t rows, int heads,
                      int d, bool own, const char* name) {
  SEQ_TRY(check_ptr(p, name));
  if (heads == 1) sh = d;
  if (rows <= 1) sn = int64_t(heads) * d;
  if (sn < 0 || sh < 0 || (sn % 8) || (sh % 8))
    return fail(BSA_ERR_INVALID_ARG, "%s strides must be non-negative multiples of 8 elements",
                name);
  if (own && (sn < d || sh < d))
    return fail(BSA_ERR_INVALID_ARG, "%s is written: its strides must be at least head_dim", name);
  r->p = const_cast<void*>(p);
  r->sn = sn;
  r->sh = sh;
  return BSA_OK;
}

bsa_status check_cache(bsa::PagedCache* c, const SeqGeo& g, const void* k, const void* v,
                       int32_t n_pages, int32_t page_size, int64_t sp, int64_t st, int64_t sh,
                       const int32_t* table, int64_t table_stride, int32_t table_width,
                       int32_t n_seqs) {
  SEQ_TRY(check_ptr(k, "k_cache"));
  SEQ_TRY(check_ptr(v, "v_cache"));
  SEQ_TRY(check_ptr(table, "block_table", 4));
  if (n_pages < 1 || page_size < 1)
    return fail(BSA_ERR_SHAPE, "n_pages (%d) and page_size (%d) must be >= 1", n_pages, page_size);
  if (table_width < 1 || (n_seqs > 1 && table_stride < table_width))
    return fail(BSA_ERR_SHAPE, "block_table: width %d, row stride %lld", table_width,
                (long long)table_stride);
  if (n_pages == 1) sp = 0;
  if (page_size == 1) st = 0;
  if (g.kv_heads == 1) sh = 0;
  if (sp < 0 || st < 0 || sh < 0 || (sp % 8) || (st % 8) || (sh % 8) ||
      (n_pages > 1 && sp < g.d) || (page_size > 1 && st < g.d) || (g.kv_heads > 1 && sh < g.d))
    return fail(BSA_ERR_INVALID_ARG,
                "cache strides must be multiples of 8 elements and at least head_dim");
  c->k = const_cast<void*>(k);
  c->v = const_cast<void*>(v);
  c->sp = sp;
  c->st = st;
  c->sh = sh;
  c->n_pages = n_pages;
  c->page_size = page_size;
  c->table = table;
  c->table_stride = table_stride;
  c->table_width = table_width;
  return BSA_OK;
}

bsa_status check_counts(int32_t n_seqs, int64_t rows, const char* what) {
  if (n_seqs < 0 || n_seqs > (1 << 24))
    return fail(BSA_ERR_SHAPE, "n_seqs %d outside 0..2^24", n_seqs);
  if (rows < 0 || rows > INT32_MAX)
    return fail(BSA_ERR_SHAPE, "%s %lld outside 0..2^31-1", what, (long long)rows);
  return BSA_OK;
}

// one CTA per 128-row tile and head at most
bsa_status check_grid(int64_t rows, int32_t n_seqs, int heads) {
  if ((rows / 128 + (n_seqs < rows ? n_seqs : rows)) * heads > INT32_MAX)
    return fail(BSA_ERR_SHAPE, "too many (tile, head) pairs for one call");
  return BSA_OK;
}

bsa_status check_status(const int32_t* p) {
  if (p && (reinterpret_cast<uintptr_t>(p) & 3u))
    return fail(BSA_ERR_INVALID_ARG, "dev_status is not 4-byte aligned");
  return BSA_OK;
}

// a tensor read by TMA boxes: broadcast views have no tensor map
bsa_status check_tma_rows(bsa::Rows* r, const SeqGeo& g, const void* p, int64_t sn, int64_t sh,
                          int64_t rows, int heads, const char* name) {
  SEQ_TRY(check_rows(r, p, sn, sh, rows, heads, g.d, false, name));
  if (r->sn == 0 || r->sh == 0)
    return fail(BSA_ERR_INVALID_ARG, "%s: strides of 0 (broadcast views) are not supported", name);
  return BSA_OK;
}

// its map of 128-row boxes (zeros for an empty tensor, which is not read)
bsa_status rows_map(CUtensorMap* m, const SeqGeo& g, const bsa::Rows& r, int64_t rows, int heads) {
  std::memset(m, 0, sizeof(*m));
  return rows ? bsa::make_rows_map(m, r.p, rows, heads, g.d, r.sn, r.sh, 128, g.fp16) : BSA_OK;
}

bsa_status done(cudaError_t e, const char* what) {
  return e == cudaSuccess ? BSA_OK : bsa::cuda_error(e, what);
}

}  // namespace

extern "C" {

bsa_status bsa_kv_append(const bsa_seq_problem* prob, int32_t n_seqs, int64_t n_tokens,
                         const void* k, int64_t k_stride_n, int64_t k_stride_h, const void* v,
                         int64_t v_stride_n, int64_t v_stride_h, void* k_cache, void* v_cache,
                         int32_t n_pages, int32_t page_size, int64_t stride_page,
                         int64_t stride_token, int64_t stride_head, const int32_t* block_table,
                         int64_t table_stride, int32_t table_width, const int32_t* cu_new,
                         const int32_t* seq_lens, const float* rope, int32_t rope_n,
                         int32_t rot_dim, int32_t interleaved, const int32_t* rope_rows,
                         const void* q, int64_t q_stride_n, int64_t q_stride_h, void* q_out,
                         int64_t qo_stride_n, int64_t qo_stride_h, void* k_out,
                         int64_t ko_stride_n, int64_t ko_stride_h, int32_t* dev_status,
                         void* stream) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  SEQ_TRY(check_counts(n_seqs, n_tokens, "n_tokens"));
  if (n_tokens == 0 || n_seqs == 0) return BSA_OK;
  bsa::AppendIO io{};
  bsa::PagedCache c{};
  SEQ_TRY(check_rows(&io.k, k, k_stride_n, k_stride_h, n_tokens, g.kv_heads, g.d, false, "k"));
  SEQ_TRY(check_rows(&io.v, v, v_stride_n, v_stride_h, n_tokens, g.kv_heads, g.d, false, "v"));
  SEQ_TRY(check_cache(&c, g, k_cache, v_cache, n_pages, page_size, stride_page, stride_token,
                      stride_head, block_table, table_stride, table_width, n_seqs));
  SEQ_TRY(check_ptr(cu_new, "cu_new", 4));
  SEQ_TRY(check_ptr(seq_lens, "seq_lens", 4));
  if (rope) {
    SEQ_TRY(check_ptr(rope, "rope"));
    if (rope_n < 1) return fail(BSA_ERR_SHAPE, "rope_n must be >= 1");
    if (rot_dim < 16 || rot_dim > g.d || rot_dim % 16)
      return fail(BSA_ERR_SHAPE, "rot_dim %d must be a multiple of 16 up to head_dim", rot_dim);
    if (rope_rows) SEQ_TRY(check_ptr(rope_rows, "rope_rows", 4));
  }
  if (!q != !q_out) return fail(BSA_ERR_INVALID_ARG, "give q and q_out, or neither");
  if (q) {
    SEQ_TRY(check_rows(&io.q, q, q_stride_n, q_stride_h, n_tokens, g.heads, g.d, false, "q"));
    SEQ_TRY(check_rows(&io.q_out, q_out, qo_stride_n, qo_stride_h, n_tokens, g.heads, g.d, true,
                       "q_out"));
  }
  if (k_out)
    SEQ_TRY(check_rows(&io.k_out, k_out, ko_stride_n, ko_stride_h, n_tokens, g.kv_heads, g.d, true,
                       "k_out"));
  SEQ_TRY(check_status(dev_status));
  SEQ_TRY(bsa::require_device());
  SEQ_TRY(bsa::resolve_status(&dev_status));
  io.cu = cu_new;
  io.lens = seq_lens;
  io.rope = rope;
  io.rope_rows = rope_rows;
  io.rope_n = rope_n;
  io.rot = rope ? rot_dim : 0;
  io.interleaved = interleaved != 0;
  io.n_seqs = n_seqs;
  io.n_tokens = n_tokens;
  io.status = dev_status;
  return done(bsa::launch_kv_append(g, c, io, static_cast<cudaStream_t>(stream)),
              "bsa_kv_append launch");
}

bsa_status bsa_packed_attn_fwd(const bsa_seq_problem* prob, int32_t n_seqs, int64_t total_q,
                               int64_t total_k, const void* q, int64_t q_stride_n,
                               int64_t q_stride_h, const void* k, int64_t k_stride_n,
                               int64_t k_stride_h, const void* v, int64_t v_stride_n,
                               int64_t v_stride_h, const int32_t* cu_q, const int32_t* cu_k,
                               void* o, int64_t o_stride_n, int64_t o_stride_h, float* lse,
                               int32_t* dev_status, void* stream) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  SEQ_TRY(check_counts(n_seqs, total_q, "total_q"));
  SEQ_TRY(check_counts(n_seqs, total_k, "total_k"));
  if (total_q == 0 || n_seqs == 0) return BSA_OK;
  SEQ_TRY(check_grid(total_q, n_seqs, g.heads));
  bsa::PackedIO io{};
  bsa::Rows rq, rk{}, rv{};
  SEQ_TRY(check_ptr(cu_q, "cu_q", 4));
  SEQ_TRY(check_ptr(cu_k, "cu_k", 4));
  SEQ_TRY(check_rows(&io.o, o, o_stride_n, o_stride_h, total_q, g.heads, g.d, true, "o"));
  if (lse) SEQ_TRY(check_ptr(lse, "lse", 4));
  SEQ_TRY(check_status(dev_status));
  SEQ_TRY(check_tma_rows(&rq, g, q, q_stride_n, q_stride_h, total_q, g.heads, "q"));
  if (total_k > 0) {  // else no row sees a key
    SEQ_TRY(check_tma_rows(&rk, g, k, k_stride_n, k_stride_h, total_k, g.kv_heads, "k"));
    SEQ_TRY(check_tma_rows(&rv, g, v, v_stride_n, v_stride_h, total_k, g.kv_heads, "v"));
  }
  SEQ_TRY(bsa::require_device());
  CUtensorMap maps[3];
  SEQ_TRY(rows_map(&maps[0], g, rq, total_q, g.heads));
  SEQ_TRY(rows_map(&maps[1], g, rk, total_k, g.kv_heads));
  SEQ_TRY(rows_map(&maps[2], g, rv, total_k, g.kv_heads));
  SEQ_TRY(bsa::resolve_status(&dev_status));
  io.cu_q = cu_q;
  io.cu_k = cu_k;
  io.n_seqs = n_seqs;
  io.total_q = total_q;
  io.total_k = total_k;
  io.lse = lse;
  io.status = dev_status;
  io.stall = bsa::stall_enabled();
  return done(bsa::launch_packed_fwd(g, maps, io, static_cast<cudaStream_t>(stream)),
              "bsa_packed_attn_fwd launch");
}

bsa_status bsa_query_packed_bwd_workspace(const bsa_seq_problem* prob, int32_t n_seqs,
                                          int64_t total_q, size_t* bytes) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  SEQ_TRY(check_counts(n_seqs, total_q, "total_q"));
  if (!bytes) return fail(BSA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = bsa::packed_bwd_workspace_bytes(g, total_q, n_seqs);
  return BSA_OK;
}

bsa_status bsa_packed_attn_bwd(const bsa_seq_problem* prob, int32_t n_seqs, int64_t total_q,
                               int64_t total_k, const void* q, int64_t q_stride_n,
                               int64_t q_stride_h, const void* k, int64_t k_stride_n,
                               int64_t k_stride_h, const void* v, int64_t v_stride_n,
                               int64_t v_stride_h, const void* o, int64_t o_stride_n,
                               int64_t o_stride_h, const void* dout, int64_t do_stride_n,
                               int64_t do_stride_h, const float* lse, const int32_t* cu_q,
                               const int32_t* cu_k, void* dq, int64_t dq_stride_n,
                               int64_t dq_stride_h, void* dk, int64_t dk_stride_n,
                               int64_t dk_stride_h, void* dv, int64_t dv_stride_n,
                               int64_t dv_stride_h, void* workspace, size_t ws_bytes,
                               int32_t* dev_status, void* stream) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  SEQ_TRY(check_counts(n_seqs, total_q, "total_q"));
  SEQ_TRY(check_counts(n_seqs, total_k, "total_k"));
  if (n_seqs == 0 || (total_q == 0 && total_k == 0)) return BSA_OK;
  SEQ_TRY(check_grid(total_q, n_seqs, g.heads));
  SEQ_TRY(check_grid(total_k, n_seqs, g.kv_heads));
  bsa::PackedBwdIO io{};
  bsa::Rows rq{}, rk{};
  SEQ_TRY(check_ptr(cu_q, "cu_q", 4));
  SEQ_TRY(check_ptr(cu_k, "cu_k", 4));
  if (total_q > 0) {
    SEQ_TRY(check_tma_rows(&rq, g, q, q_stride_n, q_stride_h, total_q, g.heads, "q"));
    SEQ_TRY(check_rows(&io.o, o, o_stride_n, o_stride_h, total_q, g.heads, g.d, false, "o"));
    SEQ_TRY(check_tma_rows(&io.dout, g, dout, do_stride_n, do_stride_h, total_q, g.heads, "dout"));
    SEQ_TRY(check_ptr(lse, "lse", 4));
    SEQ_TRY(check_rows(&io.dq, dq, dq_stride_n, dq_stride_h, total_q, g.heads, g.d, true, "dq"));
  }
  if (total_k > 0) {
    SEQ_TRY(check_tma_rows(&rk, g, k, k_stride_n, k_stride_h, total_k, g.kv_heads, "k"));
    SEQ_TRY(check_tma_rows(&io.v, g, v, v_stride_n, v_stride_h, total_k, g.kv_heads, "v"));
    SEQ_TRY(check_rows(&io.dk, dk, dk_stride_n, dk_stride_h, total_k, g.kv_heads, g.d, true, "dk"));
    SEQ_TRY(check_rows(&io.dv, dv, dv_stride_n, dv_stride_h, total_k, g.kv_heads, g.d, true, "dv"));
  }
  SEQ_TRY(check_ptr(workspace, "workspace"));
  if (ws_bytes < bsa::packed_bwd_workspace_bytes(g, total_q, n_seqs))
    return fail(BSA_ERR_WORKSPACE, "workspace of %zu bytes; %zu are needed", ws_bytes,
                bsa::packed_bwd_workspace_bytes(g, total_q, n_seqs));
  SEQ_TRY(check_status(dev_status));
  SEQ_TRY(bsa::require_device());
  CUtensorMap maps[4];
  SEQ_TRY(rows_map(&maps[0], g, rq, total_q, g.heads));
  SEQ_TRY(rows_map(&maps[1], g, rk, total_k, g.kv_heads));
  SEQ_TRY(rows_map(&maps[2], g, io.v, total_k, g.kv_heads));
  SEQ_TRY(rows_map(&maps[3], g, io.dout, total_q, g.heads));
  SEQ_TRY(bsa::resolve_status(&dev_status));
  io.cu_q = cu_q;
  io.cu_k = cu_k;
  io.n_seqs = n_seqs;
  io.total_q = total_q;
  io.total_k = total_k;
  io.lse = lse;
  io.status = dev_status;
  io.stall = bsa::stall_enabled();
  bsa::packed_bwd_workspace_split(g, &io, workspace);
  return done(bsa::launch_packed_bwd(g, maps, io, static_cast<cudaStream_t>(stream)),
              "bsa_packed_attn_bwd launch");
}

bsa_status bsa_query_decode_workspace(const bsa_seq_problem* prob, size_t* bytes) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  if (!bytes) return fail(BSA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = bsa::decode_workspace_bytes(g);
  return BSA_OK;
}

bsa_status bsa_paged_attn_decode(const bsa_seq_problem* prob, int32_t n_seqs, const void* q,
                                 int64_t q_stride_n, int64_t q_stride_h, const void* k_cache,
                                 const void* v_cache, int32_t n_pages, int32_t page_size,
                                 int64_t stride_page, int64_t stride_token, int64_t stride_head,
                                 const int32_t* block_table, int64_t table_stride,
                                 int32_t table_width, const int32_t* seq_lens, void* o,
                                 int64_t o_stride_n, int64_t o_stride_h, void* workspace,
                                 size_t ws_bytes, int32_t* dev_status, void* stream) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  SEQ_TRY(check_counts(n_seqs, n_seqs, "n_seqs"));
  if (int64_t(n_seqs) * g.heads > INT32_MAX)
    return fail(BSA_ERR_SHAPE, "n_seqs * heads must be <= 2^31-1");
  if (n_seqs == 0) return BSA_OK;
  bsa::DecodeIO io{};
  bsa::PagedCache c{};
  SEQ_TRY(check_rows(&io.q, q, q_stride_n, q_stride_h, n_seqs, g.heads, g.d, false, "q"));
  SEQ_TRY(check_cache(&c, g, k_cache, v_cache, n_pages, page_size, stride_page, stride_token,
                      stride_head, block_table, table_stride, table_width, n_seqs));
  SEQ_TRY(check_ptr(seq_lens, "seq_lens", 4));
  SEQ_TRY(check_rows(&io.o, o, o_stride_n, o_stride_h, n_seqs, g.heads, g.d, true, "o"));
  SEQ_TRY(check_ptr(workspace, "workspace"));
  if (ws_bytes < bsa::decode_workspace_bytes(g))
    return fail(BSA_ERR_WORKSPACE, "workspace of %zu bytes; %zu are needed", ws_bytes,
                bsa::decode_workspace_bytes(g));
  SEQ_TRY(check_status(dev_status));
  SEQ_TRY(bsa::require_device());
  SEQ_TRY(bsa::resolve_status(&dev_status));
  io.lens = seq_lens;
  io.n_seqs = n_seqs;
  io.workspace = workspace;
  io.status = dev_status;
  return done(bsa::launch_paged_decode(g, c, io, static_cast<cudaStream_t>(stream)),
              "bsa_paged_attn_decode launch");
}

}  // extern "C"
