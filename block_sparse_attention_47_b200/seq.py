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

    prob = SeqProblem.make(heads=32, kv_heads=8, head_dim=128)
    layer = PagedAttention(prob, n_pages=4096, page_size=16, max_seqs=64, max_pages_per_seq=64)
    layer.block_table.copy_(pages)                      # which pages each sequence has
    out = layer.prompt(q, k, v, cu, rope=table)         # caches the prompts, attends causally
    out = layer.step(q1, k1, v1, rope=table)            # one new token per sequence
"""
import ctypes
import math
import struct

import torch

from . import BSAError, _check, lib as _base_lib

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
# the argument structs travel as packed 8-byte fields: converting one pointer
# costs a fraction of converting twenty to forty separate arguments
_CALL = [_PROB, ctypes.c_char_p, _P, _P]
_SIGS = {
    "bsa_packed_attn_fwd": _CALL,
    "bsa_query_packed_bwd_workspace": [_PROB, _I32, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "bsa_packed_attn_bwd": _CALL,
    "bsa_kv_append": _CALL,
    "bsa_query_decode_workspace": [_PROB, ctypes.POINTER(ctypes.c_size_t)],
    "bsa_paged_attn_decode": _CALL,
}
_PACKED = struct.Struct("=32q")   # bsa_packed_args
_APPEND = struct.Struct("=34q")   # bsa_append_args
_DECODE = struct.Struct("=20q")   # bsa_decode_args
_FNS = {}


def _fn(name):
    f = _FNS.get(name)
    if f is None:
        f = getattr(_base_lib(), name)
        f.restype, f.argtypes = ctypes.c_int, _SIGS[name]
        _FNS[name] = f
    return f


# ---- argument checks ----------------------------------------------------------
_NO_ROWS = (0, 0, 0)


def _rows(t, shape, dtype, dev, name):
    """(pointer, row stride, head stride) of a [rows, heads, head_dim] tensor."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError("%s must be %s %s on cuda:%d, not %s %s on %s"
                         % (name, dtype, list(shape), dev, t.dtype, list(t.shape), t.device))
    sn, sh, sd = t.stride()
    if sd != 1:
        raise ValueError("%s: head_dim must be contiguous" % name)
    return t.data_ptr(), sn, sh


def _ints(t, n, dev, name):
    """Pointer of a contiguous int32 vector of n entries."""
    if t.dtype is not torch.int32 or t.shape != (n,) or t.get_device() != dev or \
            not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 vector of %d on cuda:%d" % (name, n, dev))
    return t.data_ptr()


def _cache(k_cache, v_cache, table, kv_heads, d, dtype, n_seqs, dev):
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or v_cache.stride() != strides or \
            shape[2] != kv_heads or shape[3] != d or strides[3] != 1:
        raise ValueError("k_cache and v_cache are [n_pages, page_size, kv_heads, head_dim] with "
                         "the same strides and head_dim contiguous")
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype or \
            k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise ValueError("k_cache and v_cache must be %s on cuda:%d" % (dtype, dev))
    wide = table.shape
    if table.dtype is not torch.int32 or len(wide) != 2 or wide[0] != n_seqs or \
            table.get_device() != dev or (wide[1] > 1 and table.stride(1) != 1):
        raise ValueError("block_table must be int32 [%d, width] on cuda:%d with contiguous rows"
                         % (n_seqs, dev))
    return (k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1], strides[2], shape[0],
            shape[1], table.data_ptr(), table.stride(0), wide[1])


def _device(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.get_device()


def _shape3(t, name):
    if t.dim() != 3:
        raise ValueError("%s must be [rows, heads, head_dim]" % name)
    return t.shape[0]


def _offsets(t, name):
    if t.dim() != 1 or t.shape[0] < 1:
        raise ValueError("%s holds n_seqs + 1 offsets" % name)
    return t.shape[0] - 1


def _status_ptr(t, dev):
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError("dev_status must be an int32 tensor on cuda:%d" % dev)
    return t.data_ptr()


def _workspace(t, dev):
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be contiguous on cuda:%d" % dev)
    return t.data_ptr(), t.numel() * t.element_size()


def _lse_ptr(heads, t, rows, dev):
    if t.dtype is not torch.float32 or t.shape != (heads, rows) or t.get_device() != dev or \
            not t.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [%d, %d] on cuda:%d" % (heads, rows, dev))
    return t.data_ptr()


# the current stream's handle without a Stream object (1.1 us of a 10 us call)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call(name, dev, stream, prob, args, dev_status):
    """The entry point on device `dev` and `stream` (its current one by default)."""
    if stream is None:
        stream = _current_stream(dev)
    elif stream.device_index != dev:
        raise ValueError("stream belongs to cuda:%d, the tensors to cuda:%d"
                         % (stream.device_index, dev))
    else:
        stream = stream.cuda_stream
    f, st = _fn(name), _status_ptr(dev_status, dev)
    if torch.cuda.current_device() == dev:
        rc = f(prob, args, st, stream)
    else:
        with torch.cuda.device(dev):
            rc = f(prob, args, st, stream)
    if rc:
        _check(rc)


def _query(name, *args):
    n = ctypes.c_size_t(0)
    _check(_fn(name)(*args, ctypes.byref(n)))
    return int(n.value)


# ---- entry points ----------------------------------------------------------------
def packed_attn_fwd(prob, q, k, v, cu_q, cu_k, out, lse=None, dev_status=None, stream=None):
    """Attention over packed sequences (bsa_packed_attn_fwd): q and out
    [total_q, heads, head_dim], k and v [total_k, kv_heads, head_dim], cu_q
    and cu_k [n_seqs + 1] row offsets.  prob.causal aligns the last query
    with the last key.  lse, float32 [heads, total_q], receives the rows'
    log-sum-exp (exp2 domain) for packed_attn_bwd."""
    dev, dt, H, d = _device(q, "q"), prob.torch_dtype, prob.heads, prob.head_dim
    tq, tk, n = _shape3(q, "q"), _shape3(k, "k"), _offsets(cu_q, "cu_q")
    qs, ks = (tq, H, d), (tk, prob.kv_heads, d)
    args = _PACKED.pack(
        n, tq, tk, *_rows(q, qs, dt, dev, "q"), *_rows(k, ks, dt, dev, "k"),
        *_rows(v, ks, dt, dev, "v"), *_rows(out, qs, dt, dev, "out"),
        _ints(cu_q, n + 1, dev, "cu_q"), _ints(cu_k, n + 1, dev, "cu_k"),
        0 if lse is None else _lse_ptr(H, lse, tq, dev), *_NO_ROWS, *_NO_ROWS, *_NO_ROWS,
        *_NO_ROWS, 0, 0)
    _call("bsa_packed_attn_fwd", dev, stream, prob, args, dev_status)


def packed_bwd_workspace_bytes(prob, total_q, n_seqs):
    return _query("bsa_query_packed_bwd_workspace", prob, n_seqs, total_q)


def packed_attn_bwd(prob, q, k, v, out, dout, lse, cu_q, cu_k, dq, dk, dv, workspace,
                    dev_status=None, stream=None):
    """Gradients dq, dk, dv of packed_attn_fwd from its out and lse and the
    gradient dout of out (bsa_packed_attn_bwd).  workspace: at least
    packed_bwd_workspace_bytes(prob, total_q, n_seqs), one per call that may
    overlap."""
    dev, dt, H, d = _device(q, "q"), prob.torch_dtype, prob.heads, prob.head_dim
    tq, tk, n = _shape3(q, "q"), _shape3(k, "k"), _offsets(cu_q, "cu_q")
    qs, ks = (tq, H, d), (tk, prob.kv_heads, d)
    args = _PACKED.pack(
        n, tq, tk, *_rows(q, qs, dt, dev, "q"), *_rows(k, ks, dt, dev, "k"),
        *_rows(v, ks, dt, dev, "v"), *_rows(out, qs, dt, dev, "out"),
        _ints(cu_q, n + 1, dev, "cu_q"), _ints(cu_k, n + 1, dev, "cu_k"),
        _lse_ptr(H, lse, tq, dev), *_rows(dout, qs, dt, dev, "dout"),
        *_rows(dq, qs, dt, dev, "dq"), *_rows(dk, ks, dt, dev, "dk"),
        *_rows(dv, ks, dt, dev, "dv"), *_workspace(workspace, dev))
    _call("bsa_packed_attn_bwd", dev, stream, prob, args, dev_status)


def kv_append(prob, k, v, k_cache, v_cache, block_table, cu_new, seq_lens, rope=None,
              interleaved=False, rope_rows=None, q=None, q_out=None, k_out=None, dev_status=None,
              stream=None):
    """Write new keys and values into the paged cache, keys (and queries)
    rotated on the way (bsa_kv_append).  k and v are packed [tokens,
    kv_heads, head_dim]; cu_new [n_seqs + 1] their offsets; seq_lens the
    sequences' lengths including them.  rope is a float32 [rows, rot_dim]
    table of cos | sin halves, read at the token's position or at
    rope_rows[token]."""
    dev, dt, K, d = _device(k, "k"), prob.torch_dtype, prob.kv_heads, prob.head_dim
    n, n_seqs = _shape3(k, "k"), _offsets(cu_new, "cu_new")
    rope_ptr, rope_n, rot, rr = 0, 0, 0, 0
    if rope is not None:
        if rope.dtype is not torch.float32 or rope.dim() != 2 or rope.get_device() != dev or \
                not rope.is_contiguous():
            raise ValueError("rope must be a contiguous float32 [rows, rot_dim] on cuda:%d" % dev)
        rope_ptr, (rope_n, rot) = rope.data_ptr(), rope.shape
        if rope_rows is not None:
            rr = _ints(rope_rows, n, dev, "rope_rows")
    if (q is None) != (q_out is None):
        raise ValueError("give q and q_out, or neither")
    ks, qs = (n, K, d), (n, prob.heads, d)
    args = _APPEND.pack(
        n_seqs, n, *_rows(k, ks, dt, dev, "k"), *_rows(v, ks, dt, dev, "v"),
        *_cache(k_cache, v_cache, block_table, K, d, dt, n_seqs, dev),
        _ints(cu_new, n_seqs + 1, dev, "cu_new"), _ints(seq_lens, n_seqs, dev, "seq_lens"),
        rope_ptr, rope_n, rot, 1 if interleaved else 0, rr,
        *(_NO_ROWS if q is None else _rows(q, qs, dt, dev, "q")),
        *(_NO_ROWS if q is None else _rows(q_out, qs, dt, dev, "q_out")),
        *(_NO_ROWS if k_out is None else _rows(k_out, ks, dt, dev, "k_out")))
    _call("bsa_kv_append", dev, stream, prob, args, dev_status)


def decode_workspace_bytes(prob):
    return _query("bsa_query_decode_workspace", prob)


def paged_attn_decode(prob, q, k_cache, v_cache, block_table, seq_lens, out, workspace,
                      dev_status=None, stream=None):
    """Attention of one new token per sequence, q [n_seqs, heads, head_dim],
    over the paged cache (bsa_paged_attn_decode).  workspace: at least
    decode_workspace_bytes(prob), one per call that may overlap."""
    dev, dt, d = _device(q, "q"), prob.torch_dtype, prob.head_dim
    n = _shape3(q, "q")
    qs = (n, prob.heads, d)
    args = _DECODE.pack(
        n, *_rows(q, qs, dt, dev, "q"),
        *_cache(k_cache, v_cache, block_table, prob.kv_heads, d, dt, n, dev),
        _ints(seq_lens, n, dev, "seq_lens"), *_rows(out, qs, dt, dev, "out"),
        *_workspace(workspace, dev))
    _call("bsa_paged_attn_decode", dev, stream, prob, args, dev_status)


class PagedAttention:
    """One attention layer's paged cache with its buffers, allocated once:
    the pages, the block table and lengths of up to max_seqs sequences, the
    decode workspace and a status word.  Pages are handed out by the caller:
    write page numbers into `block_table` (int32 [max_seqs,
    max_pages_per_seq]) before tokens reach them.  It starts at -1, which is
    no page: a token that reaches such an entry is reported through the status
    word (check_status) and written nowhere.

    `seq_lens` holds the cached tokens of each sequence; prompt() and step()
    add the new tokens to it.  Rows of a padded batch, behind the last
    sequence's, are not set in what the calls return.  prompt() runs on every sequence of the cache in
    order, one without new tokens having length 0 in cu; step() on the first
    ones, as many as it gets tokens."""

    def __init__(self, prob, n_pages, page_size, max_seqs, max_pages_per_seq, device="cuda"):
        self.prob = prob
        dev, dt = torch.device(device), prob.torch_dtype
        shape = (n_pages, page_size, prob.kv_heads, prob.head_dim)
        self.k_cache = torch.empty(shape, dtype=dt, device=dev)
        self.v_cache = torch.empty(shape, dtype=dt, device=dev)
        self.block_table = torch.full((max_seqs, max_pages_per_seq), -1, dtype=torch.int32, device=dev)
        self.seq_lens = torch.zeros(max_seqs, dtype=torch.int32, device=dev)
        self.workspace = torch.empty(decode_workspace_bytes(prob), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._step_cu = torch.arange(max_seqs + 1, dtype=torch.int32, device=dev)

    def _add(self, lens, new, q, k, v, cu, table, rope, interleaved, rope_rows, k_out=None,
             attend=None):
        """Append `new` tokens and attend to them: the rotated q, or what
        `attend` makes of it.  Whatever is refused, the lengths are taken back
        (slots behind them may hold anything)."""
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        lens += new
        try:
            kv_append(self.prob, k, v, self.k_cache, self.v_cache, table, cu, lens, rope=rope,
                      interleaved=interleaved, rope_rows=rope_rows, q=q, q_out=q_out, k_out=k_out,
                      dev_status=self.status)
            return q_out if attend is None else attend(q_out)
        except Exception:
            lens -= new
            raise

    def _new(self, cu):
        _ints(cu, self.seq_lens.shape[0] + 1, self.seq_lens.get_device(), "cu")
        return cu[1:] - cu[:-1]

    def append(self, q, k, v, cu, rope=None, interleaved=False, rope_rows=None, k_out=None):
        """Add packed tokens to the sequences; returns the rotated q.  A call
        that is refused leaves the lengths as they were, here and below."""
        return self._add(self.seq_lens, self._new(cu), q, k, v, cu, self.block_table, rope,
                         interleaved, rope_rows, k_out)

    def prompt(self, q, k, v, cu, rope=None, interleaved=False, rope_rows=None):
        """Whole prompts of sequences that were empty: cache their keys and
        values and return their causal attention (as prob.causal says).  New
        tokens of a sequence that holds some are cached, too, but their
        attention lacks the earlier ones: that is reported as INVALID_ARG
        through the status word (check_status), the output being meaningless."""
        new = self._new(cu)
        # the host does not know the lengths: 1 (INVALID_ARG) where a sequence has both
        both = torch.minimum(new, self.seq_lens).amax().clamp_(0, 1)
        k_rot = torch.empty_like(k, memory_format=torch.contiguous_format)

        def attend(q_rot):
            out = torch.empty_like(q_rot)
            packed_attn_fwd(self.prob, q_rot, k_rot, v, cu, cu, out, dev_status=self.status)
            torch.maximum(self.status, both, out=self.status)
            return out

        return self._add(self.seq_lens, new, q, k, v, cu, self.block_table, rope,
                         interleaved, rope_rows, k_rot, attend)

    def step(self, q, k, v, rope=None, interleaved=False, rope_rows=None):
        """One new token for each of the first n sequences, q [n, heads,
        head_dim], n up to max_seqs: cache it and return its attention over its
        sequence.  The sequences behind them rest; what is served changes
        places by its block_table row and its length."""
        n = _shape3(q, "q")
        if n > self.seq_lens.shape[0]:
            raise ValueError("%d tokens for %d sequences" % (n, self.seq_lens.shape[0]))
        lens, table = self.seq_lens[:n], self.block_table[:n]

        def attend(q_rot):
            out = torch.empty_like(q_rot)
            paged_attn_decode(self.prob, q_rot, self.k_cache, self.v_cache, table, lens, out,
                              self.workspace, dev_status=self.status)
            return out

        return self._add(lens, 1, q, k, v, self._step_cu[:n + 1], table, rope, interleaved,
                         rope_rows, attend=attend)

    def check_status(self):
        v = int(self.status.item())
        if v:
            raise BSAError(v, "device-side error reported by a sequence kernel")


__all__ = ["SeqProblem", "PagedAttention", "packed_attn_fwd", "packed_bwd_workspace_bytes", "packed_attn_bwd",
           "kv_append", "decode_workspace_bytes", "paged_attn_decode"]
