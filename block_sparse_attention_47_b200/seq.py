"""Attention over token sequences: packed prompts and a paged key-value cache.

The part of the binding over include/bsa_seq.h, for what a model runs next
to its block-sparse video attention: conditioning encoders and causal
generation over packed sequences of different lengths, and serving one token
at a time from a cache.  As in the rest of the binding every function only
marshals arguments; all work runs in the library's CUDA kernels.

Tensors are torch tensors on one GPU, bf16 or fp16 (`SeqProblem`'s dtype),
shaped [rows, heads, head_dim] with head_dim contiguous and the other
strides multiples of 8 elements; offsets, lengths and block tables are
int32.  Calls run on that GPU, on its current stream unless `stream` is
given, whatever device is current.
"""
import ctypes
import math

import torch

from . import _check, lib as _base_lib

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class SeqProblem(ctypes.Structure):
    """Mirror of bsa_seq_problem."""
    _fields_ = [("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("softmax_scale", ctypes.c_float)]

    @classmethod
    def make(cls, heads, kv_heads=None, head_dim=128, dtype=torch.bfloat16, causal=True,
             softmax_scale=None):
        if dtype not in _DTYPES:
            raise ValueError("dtype is torch.bfloat16 or torch.float16, not %s" % dtype)
        p = cls()
        p.heads, p.head_dim = heads, head_dim
        p.kv_heads = heads if kv_heads is None else kv_heads
        p.dtype = _DTYPES[dtype]
        p.causal = 1 if causal else 0
        p.softmax_scale = ((1.0 / math.sqrt(head_dim)) if head_dim > 0 else 0.0) \
            if softmax_scale is None else softmax_scale
        return p

    @property
    def torch_dtype(self):
        return torch.float16 if self.dtype == 1 else torch.bfloat16


_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
_PROB = ctypes.POINTER(SeqProblem)
_ROWS = [_P, _I64, _I64]
_CACHE = [_P, _P, _I32, _I32, _I64, _I64, _I64, _P, _I64, _I32]
_SIGS = {
    "bsa_packed_attn_fwd": [_PROB, _I32, _I64, _I64, *_ROWS, *_ROWS, *_ROWS, _P, _P, *_ROWS, _P,
                            _P, _P],
    "bsa_query_packed_bwd_workspace": [_PROB, _I32, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "bsa_packed_attn_bwd": [_PROB, _I32, _I64, _I64, *_ROWS, *_ROWS, *_ROWS, *_ROWS, *_ROWS, _P,
                            _P, _P, *_ROWS, *_ROWS, *_ROWS, _P, ctypes.c_size_t, _P, _P],
    "bsa_kv_append": [_PROB, _I32, _I64, *_ROWS, *_ROWS, *_CACHE, _P, _P, _P, _I32, _I32, _I32, _P,
                      *_ROWS, *_ROWS, *_ROWS, _P, _P],
    "bsa_query_decode_workspace": [_PROB, ctypes.POINTER(ctypes.c_size_t)],
    "bsa_paged_attn_decode": [_PROB, _I32, *_ROWS, *_CACHE, _P, *_ROWS, _P, ctypes.c_size_t, _P,
                              _P],
}
_FNS = {}


def _fn(name):
    f = _FNS.get(name)
    if f is None:
        f = getattr(_base_lib(), name)
        f.restype, f.argtypes = ctypes.c_int, _SIGS[name]
        _FNS[name] = f
    return f


# ---- argument checks ----------------------------------------------------------
_NO_ROWS = (None, 0, 0)


def _rows(prob, t, rows, heads, dev, name):
    """(pointer, row stride, head stride) of a [rows, heads, head_dim] tensor."""
    if t.device != dev or t.dtype != prob.torch_dtype:
        raise ValueError("%s must be %s on %s" % (name, prob.torch_dtype, dev))
    if t.dim() != 3 or t.shape[0] != rows or t.shape[1] != heads or t.shape[2] != prob.head_dim:
        raise ValueError("%s must be [%d, %d, %d], not %s" % (name, rows, heads, prob.head_dim,
                                                              tuple(t.shape)))
    sn, sh, sd = t.stride()
    if sd != 1:
        raise ValueError("%s: head_dim must be contiguous" % name)
    return t.data_ptr(), sn, sh


def _ints(t, n, dev, name):
    """Pointer of a contiguous int32 vector of n entries."""
    if t.device != dev or t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n or \
            not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 vector of %d on %s" % (name, n, dev))
    return t.data_ptr()


def _cache_args(prob, k_cache, v_cache, table, n_seqs, dev):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or \
            k_cache.stride() != v_cache.stride() or k_cache.shape[2] != prob.kv_heads or \
            k_cache.shape[3] != prob.head_dim or k_cache.stride(3) != 1:
        raise ValueError("k_cache and v_cache are [n_pages, page_size, kv_heads, head_dim] with "
                         "the same strides and head_dim contiguous")
    if k_cache.device != dev or v_cache.device != dev or k_cache.dtype != prob.torch_dtype or \
            v_cache.dtype != prob.torch_dtype:
        raise ValueError("k_cache and v_cache must be %s on %s" % (prob.torch_dtype, dev))
    if table.device != dev or table.dtype != torch.int32 or table.dim() != 2 or \
            table.shape[0] != n_seqs or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("block_table must be int32 [%d, width] on %s with contiguous rows"
                         % (n_seqs, dev))
    sp, st, sh, _ = k_cache.stride()
    return (k_cache.data_ptr(), v_cache.data_ptr(), k_cache.shape[0], k_cache.shape[1], sp, st, sh,
            table.data_ptr(), table.stride(0), table.shape[1])


def _device(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.device


def _status_ptr(t, dev):
    if t is None:
        return None
    if t.device != dev or t.dtype != torch.int32 or t.numel() < 1:
        raise ValueError("dev_status must be an int32 tensor on %s" % dev)
    return t.data_ptr()


def _call(name, dev, stream, *args):
    """The entry point on `dev` and `stream` (its current one by default)."""
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError("stream belongs to %s, the tensors to %s" % (stream.device, dev))
    f = _fn(name)
    if torch.cuda.current_device() == dev.index:
        _check(f(*args, stream.cuda_stream))
    else:
        with torch.cuda.device(dev):
            _check(f(*args, stream.cuda_stream))


def _workspace(t, dev):
    if t.device != dev or not t.is_contiguous():
        raise ValueError("workspace must be contiguous on %s" % dev)
    return t.data_ptr(), t.numel() * t.element_size()


def _lse_ptr(prob, t, rows, dev):
    if t.device != dev or t.dtype != torch.float32 or tuple(t.shape) != (prob.heads, rows) or \
            not t.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [%d, %d] on %s" % (prob.heads, rows, dev))
    return t.data_ptr()


# ---- entry points ----------------------------------------------------------------
def packed_attn_fwd(prob, q, k, v, cu_q, cu_k, out, lse=None, dev_status=None, stream=None):
    """Attention over packed sequences (bsa_packed_attn_fwd): q and out
    [total_q, heads, head_dim], k and v [total_k, kv_heads, head_dim], cu_q
    and cu_k [n_seqs + 1] row offsets.  prob.causal aligns the last query
    with the last key.  lse, float32 [heads, total_q], receives the rows'
    log-sum-exp (exp2 domain) for packed_attn_bwd."""
    dev = _device(q, "q")
    tq, tk, n_seqs = q.shape[0], k.shape[0], cu_q.shape[0] - 1
    _call("bsa_packed_attn_fwd", dev, stream, ctypes.byref(prob), n_seqs, tq, tk,
          *_rows(prob, q, tq, prob.heads, dev, "q"), *_rows(prob, k, tk, prob.kv_heads, dev, "k"),
          *_rows(prob, v, tk, prob.kv_heads, dev, "v"), _ints(cu_q, n_seqs + 1, dev, "cu_q"),
          _ints(cu_k, n_seqs + 1, dev, "cu_k"), *_rows(prob, out, tq, prob.heads, dev, "out"),
          None if lse is None else _lse_ptr(prob, lse, tq, dev), _status_ptr(dev_status, dev))


def packed_bwd_workspace_bytes(prob, total_q, n_seqs):
    n = ctypes.c_size_t(0)
    _check(_fn("bsa_query_packed_bwd_workspace")(ctypes.byref(prob), n_seqs, total_q,
                                                 ctypes.byref(n)))
    return int(n.value)


def packed_attn_bwd(prob, q, k, v, out, dout, lse, cu_q, cu_k, dq, dk, dv, workspace,
                    dev_status=None, stream=None):
    """Gradients dq, dk, dv of packed_attn_fwd from its out and lse and the
    gradient dout of out (bsa_packed_attn_bwd).  workspace: at least
    packed_bwd_workspace_bytes(prob, total_q, n_seqs), one per call that may
    overlap."""
    dev = _device(q, "q")
    tq, tk, n_seqs = q.shape[0], k.shape[0], cu_q.shape[0] - 1
    H, K = prob.heads, prob.kv_heads
    _call("bsa_packed_attn_bwd", dev, stream, ctypes.byref(prob), n_seqs, tq, tk,
          *_rows(prob, q, tq, H, dev, "q"), *_rows(prob, k, tk, K, dev, "k"),
          *_rows(prob, v, tk, K, dev, "v"), *_rows(prob, out, tq, H, dev, "out"),
          *_rows(prob, dout, tq, H, dev, "dout"), _lse_ptr(prob, lse, tq, dev),
          _ints(cu_q, n_seqs + 1, dev, "cu_q"), _ints(cu_k, n_seqs + 1, dev, "cu_k"),
          *_rows(prob, dq, tq, H, dev, "dq"), *_rows(prob, dk, tk, K, dev, "dk"),
          *_rows(prob, dv, tk, K, dev, "dv"), *_workspace(workspace, dev),
          _status_ptr(dev_status, dev))


def kv_append(prob, k, v, k_cache, v_cache, block_table, cu_new, seq_lens, rope=None,
              interleaved=False, rope_rows=None, q=None, q_out=None, k_out=None, dev_status=None,
              stream=None):
    """Write new keys and values into the paged cache, keys (and queries)
    rotated on the way (bsa_kv_append).  k and v are packed [tokens,
    kv_heads, head_dim]; cu_new [n_seqs + 1] their offsets; seq_lens the
    sequences' lengths including them.  rope is a float32 [rows, rot_dim]
    table of cos | sin halves, read at the token's position or at
    rope_rows[token]."""
    dev = _device(k, "k")
    n, n_seqs = k.shape[0], seq_lens.shape[0]
    rope_ptr, rope_n, rot, rr = None, 0, 0, None
    if rope is not None:
        if rope.device != dev or rope.dtype != torch.float32 or rope.dim() != 2 or \
                not rope.is_contiguous():
            raise ValueError("rope must be a contiguous float32 [rows, rot_dim] on %s" % dev)
        rope_ptr, rope_n, rot = rope.data_ptr(), rope.shape[0], rope.shape[1]
        if rope_rows is not None:
            rr = _ints(rope_rows, n, dev, "rope_rows")
    if (q is None) != (q_out is None):
        raise ValueError("give q and q_out, or neither")
    K = prob.kv_heads
    _call("bsa_kv_append", dev, stream, ctypes.byref(prob), n_seqs, n,
          *_rows(prob, k, n, K, dev, "k"), *_rows(prob, v, n, K, dev, "v"),
          *_cache_args(prob, k_cache, v_cache, block_table, n_seqs, dev),
          _ints(cu_new, n_seqs + 1, dev, "cu_new"), _ints(seq_lens, n_seqs, dev, "seq_lens"),
          rope_ptr, rope_n, rot, 1 if interleaved else 0, rr,
          *(_NO_ROWS if q is None else _rows(prob, q, n, prob.heads, dev, "q")),
          *(_NO_ROWS if q is None else _rows(prob, q_out, n, prob.heads, dev, "q_out")),
          *(_NO_ROWS if k_out is None else _rows(prob, k_out, n, K, dev, "k_out")),
          _status_ptr(dev_status, dev))


def decode_workspace_bytes(prob):
    n = ctypes.c_size_t(0)
    _check(_fn("bsa_query_decode_workspace")(ctypes.byref(prob), ctypes.byref(n)))
    return int(n.value)


def paged_attn_decode(prob, q, k_cache, v_cache, block_table, seq_lens, out, workspace,
                      dev_status=None, stream=None):
    """Attention of one new token per sequence, q [n_seqs, heads, head_dim],
    over the paged cache (bsa_paged_attn_decode).  workspace: at least
    decode_workspace_bytes(prob), one per call that may overlap."""
    dev = _device(q, "q")
    n = q.shape[0]
    _call("bsa_paged_attn_decode", dev, stream, ctypes.byref(prob), n,
          *_rows(prob, q, n, prob.heads, dev, "q"),
          *_cache_args(prob, k_cache, v_cache, block_table, n, dev),
          _ints(seq_lens, n, dev, "seq_lens"), *_rows(prob, out, n, prob.heads, dev, "out"),
          *_workspace(workspace, dev), _status_ptr(dev_status, dev))


__all__ = ["SeqProblem", "packed_attn_fwd", "packed_bwd_workspace_bytes",
           "packed_attn_bwd", "kv_append", "decode_workspace_bytes", "paged_attn_decode"]
