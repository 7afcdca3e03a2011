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
bsa_status check_rows(bsa::Rows* r, const bsa_rows& in, int64_t rows, int heads, int d, bool own,
                      const char* name) {
  void* p = in.data;
  int64_t sn = in.stride_n, sh = in.stride_h;
  SEQ_TRY(check_ptr(p, name));
  if (heads == 1) sh = d;
  if (rows <= 1) sn = int64_t(heads) * d;
  if (sn < 0 || sh < 0 || (sn % 8) || (sh % 8))
    return fail(BSA_ERR_INVALID_ARG, "%s strides must be non-negative multiples of 8 elements",
                name);
  if (own && (sn < d || sh < d))
    return fail(BSA_ERR_INVALID_ARG, "%s is written: its strides must be at least head_dim", name);
  r->p = p;
  r->sn = sn;
  r->sh = sh;
  return BSA_OK;
}

bsa_status check_cache(bsa::PagedCache* c, const SeqGeo& g, const bsa_paged_cache& in,
                       int64_t n_seqs) {
  SEQ_TRY(check_ptr(in.k, "k_cache"));
  SEQ_TRY(check_ptr(in.v, "v_cache"));
  SEQ_TRY(check_ptr(in.block_table, "block_table", 4));
  if (in.n_pages < 1 || in.page_size < 1 || in.n_pages > INT32_MAX || in.page_size > INT32_MAX)
    return fail(BSA_ERR_SHAPE, "n_pages (%lld) and page_size (%lld) must lie in 1..2^31-1",
                (long long)in.n_pages, (long long)in.page_size);
  if (in.table_width < 1 || in.table_width > INT32_MAX ||
      (n_seqs > 1 && in.table_stride < in.table_width))
    return fail(BSA_ERR_SHAPE, "block_table: width %lld, row stride %lld",
                (long long)in.table_width, (long long)in.table_stride);
  const int64_t sp = in.n_pages == 1 ? 0 : in.stride_page;
  const int64_t st = in.page_size == 1 ? 0 : in.stride_token;
  const int64_t sh = g.kv_heads == 1 ? 0 : in.stride_head;
  if (sp < 0 || st < 0 || sh < 0 || (sp % 8) || (st % 8) || (sh % 8) ||
      (in.n_pages > 1 && sp < g.d) || (in.page_size > 1 && st < g.d) ||
      (g.kv_heads > 1 && sh < g.d))
    return fail(BSA_ERR_INVALID_ARG,
                "cache strides must be multiples of 8 elements and at least head_dim");
  c->k = in.k;
  c->v = in.v;
  c->sp = sp;
  c->st = st;
  c->sh = sh;
  c->n_pages = int(in.n_pages);
  c->page_size = int(in.page_size);
  c->table = in.block_table;
  c->table_stride = in.table_stride;
  c->table_width = int(in.table_width);
  return BSA_OK;
}

bsa_status check_counts(int64_t n_seqs, int64_t rows, const char* what) {
  if (n_seqs < 0 || n_seqs > (1 << 24))
    return fail(BSA_ERR_SHAPE, "n_seqs %lld outside 0..2^24", (long long)n_seqs);
  if (rows < 0 || rows > INT32_MAX)
    return fail(BSA_ERR_SHAPE, "%s %lld outside 0..2^31-1", what, (long long)rows);
  return BSA_OK;
}

// one CTA per 128-row tile and head at most; row counts that sums of two of
// them stay within 32 bits
bsa_status check_grid(int64_t rows, int64_t n_seqs, int heads) {
  if (bsa::tile_places(rows, n_seqs, 128) * heads > INT32_MAX / 2)
    return fail(BSA_ERR_SHAPE, "too many (tile, head) pairs for one call");
  if (rows > (int64_t(1) << 30))
    return fail(BSA_ERR_SHAPE, "%lld rows; at most 2^30 in one call", (long long)rows);
  return BSA_OK;
}

bsa_status check_status(const int32_t* p) {
  if (p && (reinterpret_cast<uintptr_t>(p) & 3u))
    return fail(BSA_ERR_INVALID_ARG, "dev_status is not 4-byte aligned");
  return BSA_OK;
}

// a tensor read by TMA boxes: broadcast views have no tensor map
bsa_status check_tma_rows(bsa::Rows* r, const SeqGeo& g, const bsa_rows& in, int64_t rows,
                          int heads, const char* name) {
  SEQ_TRY(check_rows(r, in, rows, heads, g.d, false, name));
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

bsa_status bsa_packed_attn_fwd(const bsa_seq_problem* prob, const bsa_packed_args* a,
                               int32_t* dev_status, void* stream) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  if (!a) return fail(BSA_ERR_INVALID_ARG, "args is NULL");
  const int64_t tq = a->total_q, tk = a->total_k;
  SEQ_TRY(check_counts(a->n_seqs, tq, "total_q"));
  SEQ_TRY(check_counts(a->n_seqs, tk, "total_k"));
  if (tq == 0 || a->n_seqs == 0) return BSA_OK;
  SEQ_TRY(check_grid(tq, a->n_seqs, g.heads));
  SEQ_TRY(check_grid(tk, a->n_seqs, 1));
  bsa::PackedIO io{};
  bsa::Rows rq, rk{}, rv{};
  SEQ_TRY(check_ptr(a->cu_q, "cu_q", 4));
  SEQ_TRY(check_ptr(a->cu_k, "cu_k", 4));
  SEQ_TRY(check_rows(&io.o, a->o, tq, g.heads, g.d, true, "o"));
  if (a->lse) SEQ_TRY(check_ptr(a->lse, "lse", 4));
  SEQ_TRY(check_status(dev_status));
  SEQ_TRY(check_tma_rows(&rq, g, a->q, tq, g.heads, "q"));
  if (tk > 0) {  // else no row sees a key
    SEQ_TRY(check_tma_rows(&rk, g, a->k, tk, g.kv_heads, "k"));
    SEQ_TRY(check_tma_rows(&rv, g, a->v, tk, g.kv_heads, "v"));
  }
  SEQ_TRY(bsa::require_device());
  CUtensorMap maps[3];
  SEQ_TRY(rows_map(&maps[0], g, rq, tq, g.heads));
  SEQ_TRY(rows_map(&maps[1], g, rk, tk, g.kv_heads));
  SEQ_TRY(rows_map(&maps[2], g, rv, tk, g.kv_heads));
  SEQ_TRY(bsa::resolve_status(&dev_status));
  io.cu_q = a->cu_q;
  io.cu_k = a->cu_k;
  io.n_seqs = int(a->n_seqs);
  io.total_q = tq;
  io.total_k = tk;
  io.lse = a->lse;
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

bsa_status bsa_packed_attn_bwd(const bsa_seq_problem* prob, const bsa_packed_args* a,
                               int32_t* dev_status, void* stream) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  if (!a) return fail(BSA_ERR_INVALID_ARG, "args is NULL");
  const int64_t tq = a->total_q, tk = a->total_k;
  SEQ_TRY(check_counts(a->n_seqs, tq, "total_q"));
  SEQ_TRY(check_counts(a->n_seqs, tk, "total_k"));
  if (a->n_seqs == 0 || (tq == 0 && tk == 0)) return BSA_OK;
  SEQ_TRY(check_grid(tq, a->n_seqs, g.heads));
  SEQ_TRY(check_grid(tk, a->n_seqs, g.kv_heads));
  bsa::PackedBwdIO io{};
  bsa::Rows rq{}, rk{};
  SEQ_TRY(check_ptr(a->cu_q, "cu_q", 4));
  SEQ_TRY(check_ptr(a->cu_k, "cu_k", 4));
  if (tq > 0) {
    SEQ_TRY(check_tma_rows(&rq, g, a->q, tq, g.heads, "q"));
    SEQ_TRY(check_rows(&io.o, a->o, tq, g.heads, g.d, false, "o"));
    SEQ_TRY(check_tma_rows(&io.dout, g, a->dout, tq, g.heads, "dout"));
    SEQ_TRY(check_ptr(a->lse, "lse", 4));
    SEQ_TRY(check_rows(&io.dq, a->dq, tq, g.heads, g.d, true, "dq"));
  }
  if (tk > 0) {
    SEQ_TRY(check_tma_rows(&rk, g, a->k, tk, g.kv_heads, "k"));
    SEQ_TRY(check_tma_rows(&io.v, g, a->v, tk, g.kv_heads, "v"));
    SEQ_TRY(check_rows(&io.dk, a->dk, tk, g.kv_heads, g.d, true, "dk"));
    SEQ_TRY(check_rows(&io.dv, a->dv, tk, g.kv_heads, g.d, true, "dv"));
  }
  SEQ_TRY(check_ptr(a->workspace, "workspace"));
  if (a->ws_bytes < bsa::packed_bwd_workspace_bytes(g, tq, a->n_seqs))
    return fail(BSA_ERR_WORKSPACE, "workspace of %zu bytes; %zu are needed", a->ws_bytes,
                bsa::packed_bwd_workspace_bytes(g, tq, a->n_seqs));
  SEQ_TRY(check_status(dev_status));
  SEQ_TRY(bsa::require_device());
  CUtensorMap maps[4];
  SEQ_TRY(rows_map(&maps[0], g, rq, tq, g.heads));
  SEQ_TRY(rows_map(&maps[1], g, rk, tk, g.kv_heads));
  SEQ_TRY(rows_map(&maps[2], g, io.v, tk, g.kv_heads));
  SEQ_TRY(rows_map(&maps[3], g, io.dout, tq, g.heads));
  SEQ_TRY(bsa::resolve_status(&dev_status));
  io.cu_q = a->cu_q;
  io.cu_k = a->cu_k;
  io.n_seqs = int(a->n_seqs);
  io.total_q = tq;
  io.total_k = tk;
  io.lse = a->lse;
  io.status = dev_status;
  io.stall = bsa::stall_enabled();
  bsa::packed_bwd_workspace_split(g, &io, a->workspace);
  return done(bsa::launch_packed_bwd(g, maps, io, static_cast<cudaStream_t>(stream)),
              "bsa_packed_attn_bwd launch");
}

bsa_status bsa_kv_append(const bsa_seq_problem* prob, const bsa_append_args* a,
                         int32_t* dev_status, void* stream) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  if (!a) return fail(BSA_ERR_INVALID_ARG, "args is NULL");
  const int64_t n = a->n_tokens;
  SEQ_TRY(check_counts(a->n_seqs, n, "n_tokens"));
  if (n == 0 || a->n_seqs == 0) return BSA_OK;
  bsa::AppendIO io{};
  bsa::PagedCache c{};
  SEQ_TRY(check_rows(&io.k, a->k, n, g.kv_heads, g.d, false, "k"));
  SEQ_TRY(check_rows(&io.v, a->v, n, g.kv_heads, g.d, false, "v"));
  SEQ_TRY(check_cache(&c, g, a->cache, a->n_seqs));
  SEQ_TRY(check_ptr(a->cu_new, "cu_new", 4));
  SEQ_TRY(check_ptr(a->seq_lens, "seq_lens", 4));
  if (a->rope) {
    SEQ_TRY(check_ptr(a->rope, "rope"));
    if (a->rope_n < 1 || a->rope_n > INT32_MAX)
      return fail(BSA_ERR_SHAPE, "rope_n must lie in 1..2^31-1");
    if (a->rot_dim < 16 || a->rot_dim > g.d || a->rot_dim % 16)
      return fail(BSA_ERR_SHAPE, "rot_dim %lld must be a multiple of 16 up to head_dim",
                  (long long)a->rot_dim);
    if (a->rope_rows) SEQ_TRY(check_ptr(a->rope_rows, "rope_rows", 4));
  }
  if (!a->q.data != !a->q_out.data)
    return fail(BSA_ERR_INVALID_ARG, "give q and q_out, or neither");
  if (a->q.data) {
    SEQ_TRY(check_rows(&io.q, a->q, n, g.heads, g.d, false, "q"));
    SEQ_TRY(check_rows(&io.q_out, a->q_out, n, g.heads, g.d, true, "q_out"));
  }
  if (a->k_out.data) SEQ_TRY(check_rows(&io.k_out, a->k_out, n, g.kv_heads, g.d, true, "k_out"));
  SEQ_TRY(check_status(dev_status));
  SEQ_TRY(bsa::require_device());
  SEQ_TRY(bsa::resolve_status(&dev_status));
  io.cu = a->cu_new;
  io.lens = a->seq_lens;
  io.rope = a->rope;
  io.rope_rows = a->rope ? a->rope_rows : nullptr;
  io.rope_n = int(a->rope_n);
  io.rot = a->rope ? int(a->rot_dim) : 0;
  io.interleaved = a->interleaved != 0;
  io.n_seqs = int(a->n_seqs);
  io.n_tokens = n;
  io.status = dev_status;
  return done(bsa::launch_kv_append(g, c, io, static_cast<cudaStream_t>(stream)),
              "bsa_kv_append launch");
}

bsa_status bsa_query_decode_workspace(const bsa_seq_problem* prob, size_t* bytes) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  if (!bytes) return fail(BSA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = bsa::decode_workspace_bytes(g);
  return BSA_OK;
}

bsa_status bsa_paged_attn_decode(const bsa_seq_problem* prob, const bsa_decode_args* a,
                                 int32_t* dev_status, void* stream) {
  SEQ_RANGE();
  SeqGeo g;
  SEQ_TRY(make_geo(prob, &g));
  if (!a) return fail(BSA_ERR_INVALID_ARG, "args is NULL");
  const int64_t n = a->n_seqs;
  SEQ_TRY(check_counts(n, n, "n_seqs"));
  if (n * g.heads > INT32_MAX)
    return fail(BSA_ERR_SHAPE, "n_seqs * heads must be <= 2^31-1");
  if (n == 0) return BSA_OK;
  bsa::DecodeIO io{};
  bsa::PagedCache c{};
  SEQ_TRY(check_rows(&io.q, a->q, n, g.heads, g.d, false, "q"));
  SEQ_TRY(check_cache(&c, g, a->cache, n));
  SEQ_TRY(check_ptr(a->seq_lens, "seq_lens", 4));
  SEQ_TRY(check_rows(&io.o, a->o, n, g.heads, g.d, true, "o"));
  SEQ_TRY(check_ptr(a->workspace, "workspace"));
  if (a->ws_bytes < bsa::decode_workspace_bytes(g))
    return fail(BSA_ERR_WORKSPACE, "workspace of %zu bytes; %zu are needed", a->ws_bytes,
                bsa::decode_workspace_bytes(g));
  SEQ_TRY(check_status(dev_status));
  SEQ_TRY(bsa::require_device());
  SEQ_TRY(bsa::resolve_status(&dev_status));
  io.lens = a->seq_lens;
  io.n_seqs = int(n);
  io.workspace = a->workspace;
  io.status = dev_status;
  return done(bsa::launch_paged_decode(g, c, io, static_cast<cudaStream_t>(stream)),
              "bsa_paged_attn_decode launch");
}

}  // extern "C"
