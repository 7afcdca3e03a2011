"""Host-side checks of the token-sequence entry points that need no GPU: the
library exports what include/bsa_seq.h declares, the header is strict C99,
and invalid arguments are refused before any launch."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import block_sparse_attention_47_b200 as bsa
from block_sparse_attention_47_b200 import seq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_sparse_attention_47_b200 import build
    build.build()
    return bsa.lib()


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "bsa_seq.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(bsa_[a-z_0-9]+)\s*\(", text))
    assert names == set(seq._SIGS), "binding and header disagree"
    for n in names:
        assert hasattr(bsa.lib(), n), n


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_header_is_strict_c99(tmp_path):
    src = tmp_path / "client.c"
    src.write_text('#include "bsa_seq.h"\n'
                   "int main(void) { bsa_seq_problem p = {8, 2, 96, BSA_DTYPE_FP16, 1, 0.1f};\n"
                   "  if (sizeof(bsa_packed_args) != %d || sizeof(bsa_append_args) != %d ||\n"
                   "      sizeof(bsa_decode_args) != %d) return 2;\n"
                   "  size_t n; return bsa_query_decode_workspace(&p, &n) == BSA_ERR_UNSUPPORTED "
                   "? 0 : 1; }\n" % (seq._PACKED.size, seq._APPEND.size, seq._DECODE.size))
    exe = tmp_path / "client"
    libdir = os.path.dirname(bsa.LIB_PATH)
    cc = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror",
                         "-I", os.path.join(ROOT, "include"), str(src), "-L", libdir, "-lbsa",
                         "-Wl,-rpath," + libdir, "-o", str(exe)], capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


def prob(**kw):
    d = dict(heads=8, kv_heads=2, head_dim=64)
    d.update(kw)
    return bsa.SeqProblem.make(**d)


@pytest.mark.parametrize("field,value,status", [
    ("head_dim", 96, UNSUPPORTED), ("head_dim", 0, UNSUPPORTED), ("heads", 0, SHAPE),
    ("kv_heads", 0, SHAPE), ("kv_heads", 3, SHAPE), ("heads", 65536, SHAPE), ("dtype", 2, INVALID),
    ("causal", 2, INVALID), ("softmax_scale", 0.0, INVALID),
    ("softmax_scale", float("nan"), INVALID)])
def test_invalid_problems_are_refused(field, value, status):
    p = prob()
    setattr(p, field, value)
    with pytest.raises(bsa.BSAError) as e:
        bsa.decode_workspace_bytes(p)
    assert e.value.status == status


def test_dtype_of_the_problem():
    with pytest.raises(ValueError):
        prob(dtype=torch.float32)
    assert prob(dtype=torch.float16).torch_dtype == torch.float16


def call(name, layout, a):
    """The entry point with the dict's values as its argument struct."""
    p, st, stream = a.pop("prob"), a.pop("status"), a.pop("stream")
    return seq._fn(name)(p, layout.pack(*(0 if x is None else x for x in a.values())), st, stream)


def decode_args(**kw):
    """Arguments of bsa_paged_attn_decode that pass every host check."""
    a = dict(prob=ctypes.byref(prob()), n_seqs=2, q=16, q_sn=512, q_sh=64, k=16, v=16,
             sp=2048, st=128, sh=64, n_pages=4, page_size=16, table=16, table_stride=4, table_width=4,
             lens=16,
             o=16, o_sn=512, o_sh=64, ws=16, ws_bytes=1 << 30, status=None, stream=None)
    a.update(kw)
    return a


DECODE_BAD = [
    (dict(prob=None), INVALID, b"problem"), (dict(n_seqs=-1), SHAPE, b"n_seqs"),
    (dict(n_seqs=1 << 25), SHAPE, b"n_seqs"), (dict(q=None), INVALID, b"q is NULL"),
    (dict(q=24), INVALID, b"aligned"), (dict(q_sh=60), INVALID, b"strides"),
    (dict(q_sn=-512), INVALID, b"strides"), (dict(k=None), INVALID, b"k_cache"),
    (dict(v=8), INVALID, b"v_cache"), (dict(n_pages=0), SHAPE, b"n_pages"),
    (dict(page_size=0), SHAPE, b"page_size"), (dict(sp=2052), INVALID, b"cache strides"),
    (dict(st=8), INVALID, b"cache strides"), (dict(sh=0), INVALID, b"cache strides"),
    (dict(table=None), INVALID, b"block_table"), (dict(table=18), INVALID, b"block_table"),
    (dict(table_width=0), SHAPE, b"block_table"), (dict(table_stride=3), SHAPE, b"block_table"),
    (dict(lens=None), INVALID, b"seq_lens"), (dict(o=None), INVALID, b"o is NULL"),
    (dict(o_sh=0), INVALID, b"o is written"), (dict(ws=None), INVALID, b"workspace"),
    (dict(ws_bytes=16), WORKSPACE, b"workspace"), (dict(status=2), INVALID, b"dev_status"),
]


@pytest.mark.parametrize("kw,status,word", DECODE_BAD, ids=[str(k) for k, _, _ in DECODE_BAD])
def test_decode_refuses(kw, status, word):
    rc = call("bsa_paged_attn_decode", seq._DECODE, decode_args(**kw))
    assert rc == status, (rc, bsa.lib().bsa_last_error())
    assert word in bsa.lib().bsa_last_error()


def test_empty_batches_need_no_device():
    assert call("bsa_packed_attn_fwd", seq._PACKED, fwd_args(tq=0)) == 0
    assert call("bsa_paged_attn_decode", seq._DECODE, decode_args(n_seqs=0)) == 0
    assert call("bsa_kv_append", seq._APPEND, append_args(n=0)) == 0


def append_args(**kw):
    a = dict(prob=ctypes.byref(prob()), n_seqs=2, n=5, k=16, k_sn=128, k_sh=64, v=16, v_sn=128,
             v_sh=64, kc=16, vc=16, sp=2048, st=128, sh=64, n_pages=4, page_size=16, table=16,
             table_stride=4, table_width=4, cu=16, lens=16, rope=16, rope_n=100, rot=64,
             interleaved=0, rope_rows=None, q=16, q_sn=512, q_sh=64, qo=16, qo_sn=512, qo_sh=64,
             ko=16, ko_sn=128, ko_sh=64, status=None, stream=None)
    a.update(kw)
    return a


APPEND_BAD = [
    (dict(n=-1), SHAPE, b"n_tokens"), (dict(n=1 << 31), SHAPE, b"n_tokens"),
    (dict(k=None), INVALID, b"k is NULL"), (dict(v=4), INVALID, b"v is not"),
    (dict(k_sn=4), INVALID, b"k strides"), (dict(kc=None), INVALID, b"k_cache"),
    (dict(cu=None), INVALID, b"cu_new"), (dict(cu=2), INVALID, b"cu_new"),
    (dict(lens=6), INVALID, b"seq_lens"), (dict(rope=8), INVALID, b"rope"),
    (dict(rope_n=0), SHAPE, b"rope_n"), (dict(rot=24), SHAPE, b"rot_dim"),
    (dict(rot=80), SHAPE, b"rot_dim"), (dict(rot=0), SHAPE, b"rot_dim"),
    (dict(rope_rows=3), INVALID, b"rope_rows"), (dict(q=None), INVALID, b"q and q_out"),
    (dict(qo=None), INVALID, b"q and q_out"), (dict(qo_sn=0), INVALID, b"q_out is written"),
    (dict(ko=8), INVALID, b"k_out"), (dict(ko_sh=0), INVALID, b"k_out is written"),
    (dict(status=1), INVALID, b"dev_status"),
]


@pytest.mark.parametrize("kw,status,word", APPEND_BAD, ids=[str(k) for k, _, _ in APPEND_BAD])
def test_append_refuses(kw, status, word):
    rc = call("bsa_kv_append", seq._APPEND, append_args(**kw))
    assert rc == status, (rc, bsa.lib().bsa_last_error())
    assert word in bsa.lib().bsa_last_error()


def fwd_args(**kw):
    a = dict(prob=ctypes.byref(prob()), n_seqs=2, tq=100, tk=100, q=16, q_sn=512, q_sh=64, k=16,
             k_sn=128, k_sh=64, v=16, v_sn=128, v_sh=64, o=16, o_sn=512, o_sh=64, cu_q=16, cu_k=16,
             lse=None, **{"rest%d" % i: 0 for i in range(14)}, status=None, stream=None)
    a.update(kw)
    return a


FWD_BAD = [
    (dict(n_seqs=-1), SHAPE, b"n_seqs"), (dict(tq=-1), SHAPE, b"total_q"),
    (dict(tk=1 << 31), SHAPE, b"total_k"), (dict(tq=(1 << 31) - 1, n_seqs=1 << 24, prob="wide"), SHAPE, b"pairs"),
    (dict(q=None), INVALID, b"q is NULL"), (dict(q=18), INVALID, b"aligned"),
    (dict(q_sn=516), INVALID, b"q strides"), (dict(k_sh=0), INVALID, b"broadcast"),
    (dict(v_sn=0), INVALID, b"broadcast"), (dict(cu_q=None), INVALID, b"cu_q"),
    (dict(cu_k=2), INVALID, b"cu_k"), (dict(o=None), INVALID, b"o is NULL"),
    (dict(o_sn=0), INVALID, b"o is written"), (dict(lse=2), INVALID, b"lse"),
    (dict(status=1), INVALID, b"dev_status"),
]


@pytest.mark.parametrize("kw,status,word", FWD_BAD, ids=[str(k) for k, _, _ in FWD_BAD])
def test_packed_fwd_refuses(kw, status, word):
    kw = dict(kw)
    if kw.get("prob") == "wide":
        kw["prob"] = ctypes.byref(prob(heads=4096, kv_heads=2))
    rc = call("bsa_packed_attn_fwd", seq._PACKED, fwd_args(**kw))
    assert rc == status, (rc, bsa.lib().bsa_last_error())
    assert word in bsa.lib().bsa_last_error()


def test_binding_refuses_host_tensors():
    t = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        bsa.paged_attn_decode(prob(), t, None, None, None, i, t, None)
    with pytest.raises(ValueError, match="CUDA"):
        bsa.kv_append(prob(), t, t, None, None, None, i, i)


# ---- the gradient oracle ------------------------------------------------------------
@pytest.mark.parametrize("lq,lk,causal", [(7, 7, True), (5, 9, True), (9, 5, True), (6, 4, False)])
def test_gradient_oracle_agrees_with_differences(lq, lk, causal):
    from seq_helpers import attention64, grads64, limits
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(n, 16, generator=g, dtype=torch.float64) for n in (lq, lk, lk, lq))
    lim, scale, h = limits(lq, lk, causal), 0.3, 1e-5
    (dq, dk, dv), _ = grads64(q, k, v, do, lim, scale, torch.bfloat16)

    def loss(a, b, c):
        return float((attention64(a, b, c, lim, scale)[0] * do).sum())

    for i, (x, dx) in enumerate(((q, dq), (k, dk), (v, dv))):
        for _ in range(4):
            way = torch.randn(x.shape, generator=g, dtype=torch.float64)
            up, down = [q, k, v], [q, k, v]
            up[i], down[i] = x + h * way, x - h * way
            num = (loss(*up) - loss(*down)) / (2 * h)
            assert abs(num - float((dx * way).sum())) <= 1e-7 * (1 + abs(num))


def bwd_args(**kw):
    a = dict(prob=ctypes.byref(prob()), n_seqs=2, tq=100, tk=100, q=16, q_sn=512, q_sh=64, k=16,
             k_sn=128, k_sh=64, v=16, v_sn=128, v_sh=64, o=16, o_sn=512, o_sh=64, cu_q=16,
             cu_k=16, lse=16, do=16, do_sn=512, do_sh=64, dq=16, dq_sn=512, dq_sh=64, dk=16, dk_sn=128,
             dk_sh=64, dv=16, dv_sn=128, dv_sh=64, ws=16, ws_bytes=1 << 30, status=None, stream=None)
    a.update(kw)
    return a


BWD_BAD = [
    (dict(n_seqs=-1), SHAPE, b"n_seqs"), (dict(tq=1 << 31), SHAPE, b"total_q"),
    (dict(tk=-1), SHAPE, b"total_k"), (dict(q=None), INVALID, b"q is NULL"),
    (dict(k_sn=0), INVALID, b"broadcast"), (dict(v=17), INVALID, b"v is not"),
    (dict(o=None), INVALID, b"o is NULL"), (dict(do_sh=0), INVALID, b"dout"),
    (dict(do=4), INVALID, b"dout"), (dict(lse=None), INVALID, b"lse"), (dict(cu_q=1), INVALID, b"cu_q"),
    (dict(cu_k=None), INVALID, b"cu_k"), (dict(dq=None), INVALID, b"dq"), (dict(dk_sh=8), INVALID, b"dk"),
    (dict(dv_sn=0), INVALID, b"dv"), (dict(ws=None), INVALID, b"workspace"),
    (dict(ws=8), INVALID, b"workspace"), (dict(ws_bytes=100), WORKSPACE, b"workspace"),
    (dict(status=3), INVALID, b"dev_status"),
]


@pytest.mark.parametrize("kw,status,word", BWD_BAD, ids=[str(k) for k, _, _ in BWD_BAD])
def test_packed_bwd_refuses(kw, status, word):
    rc = call("bsa_packed_attn_bwd", seq._PACKED, bwd_args(**kw))
    assert rc == status, (rc, bsa.lib().bsa_last_error())
    assert word in bsa.lib().bsa_last_error()


def test_args_are_required():
    for n in ("bsa_packed_attn_fwd", "bsa_packed_attn_bwd", "bsa_kv_append", "bsa_paged_attn_decode"):
        assert seq._fn(n)(ctypes.byref(prob()), None, None, None) == INVALID
        assert b"args" in bsa.lib().bsa_last_error()


def test_bwd_workspace():
    """Two floats per head and row of every 128-row tile there can be."""
    for tq, n in ((0, 0), (1, 1), (1000, 3), (127, 127)):
        assert bsa.packed_bwd_workspace_bytes(prob(), tq, n) == 4 * (2 * 8 * 128 * (tq // 128 + n + 1) + 2 * 2)
    assert call("bsa_packed_attn_bwd", seq._PACKED, bwd_args(tq=0, tk=0)) == 0


def test_a_refused_append_leaves_the_lengths():
    at = bsa.PagedAttention(prob_of(), n_pages=4, page_size=16, max_seqs=3, max_pages_per_seq=2, device="cpu")
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        at.step(x, x, x)
    with pytest.raises(ValueError, match="cu must be"):
        at.prompt(x, x, x, torch.tensor([0, 3], dtype=torch.int32))
    assert at.seq_lens.tolist() == [0, 0, 0]


def prob_of():
    return bsa.SeqProblem.make(2, 2, 64)


def test_rows_of_a_packed_call_are_limited():
    rc = call("bsa_packed_attn_bwd", seq._PACKED, bwd_args(tk=(1 << 30) + 1, n_seqs=1))
    assert rc == SHAPE and b"2^30" in bsa.lib().bsa_last_error()


def test_bwd_fp16_workspace_has_the_norms_of_every_sequence():
    for n in (1, 3, 1000):
        rows = 128 * (500 // 128 + n + 1)
        assert bsa.packed_bwd_workspace_bytes(prob(dtype=torch.float16), 500, n) == \
            4 * (2 * 8 * rows + 2 * 2 * n)


def test_the_build_checks_the_registers_of_a_split():
    from block_sparse_attention_47_b200 import build
    line = ("ptxas info    : Compiling entry function '_Z%s' for 'sm_100a'\n"
            "    0 bytes stack frame\nptxas info    : Used %d registers, used 1 barriers\n")
    good = line % ("17packed_fwd_kernelIfE", 168) + line % ("5other", 30)
    build.check_registers(good)
    for bad in (good + line % ("17packed_fwd_kernelIhE", 160), line % ("5other", 168), ""):
        with pytest.raises(RuntimeError, match="registers"):
            build.check_registers(bad)
