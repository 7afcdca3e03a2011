"""Attention over packed sequences on the GPU against 64-bit oracles with
derived bounds."""
import math

import pytest
import torch

import block_sparse_attention_47_b200 as bsa
from seq_helpers import (assert_within, attention64, cu_of, grads64, limits, output_bound,
                         rounded_bound)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def inputs(lq, lk, H, K, d, dt, seed=11, gain=2.0, tail=2):
    """q, k, v as slices of wider tensors; the rows behind the last sequence
    are NaN."""
    gen = torch.Generator().manual_seed(seed)
    wide_q = torch.randn(sum(lq) + tail, H + 1, d, generator=gen) * gain
    wide_kv = torch.randn(sum(lk) + tail, 2 * K, d, generator=gen)
    wide_q[sum(lq):], wide_kv[sum(lk):] = math.nan, math.nan
    wide_q, wide_kv = wide_q.to(dt).cuda(), wide_kv.to(dt).cuda()
    return wide_q[:, :H], wide_kv[:, :K], wide_kv[:, K:]


def check_fwd(q, k, v, lq, lk, causal, out, lse, scale):
    H, K = q.shape[1], k.shape[1]
    q0 = k0 = 0
    for a, b in zip(lq, lk):
        lim = limits(a, b, causal)
        for h in range(H):
            kk, vv = k[k0:k0 + b, h // (H // K)], v[k0:k0 + b, h // (H // K)]
            o, lse2, p, g = attention64(q[q0:q0 + a, h], kk, vv, lim, scale)
            what = "%d x %d, head %d" % (a, b, h)
            assert_within(out[q0:q0 + a, h], o, output_bound(o, p, vv, g, q.dtype), what)
            if lse is not None and a:
                got, want = lse[h, q0:q0 + a].double().cpu(), lse2.cpu()
                none = lim == 0
                assert bool((got[none] == -math.inf).all())
                # the scores' error, the exponentials' (4e-6 on a quarter of
                # them) and a few fp32 roundings of values up to |lse|
                tol = (g + 4e-6) / math.log(2.0) + 2.0 ** -22 * (1 + want[~none].abs())
                assert bool(((got - want)[~none].abs() <= tol).all()), what
        q0, k0 = q0 + a, k0 + b


FWD = [
    # lens_q, lens_k, heads, kv, d, dtype, causal
    ([1], [1], 1, 1, 64, BF, True),
    ([1], [1], 2, 1, 128, FP, False),
    ([37], [37], 2, 2, 64, FP, True),
    ([127, 128, 129], [127, 128, 129], 4, 2, 128, BF, True),
    ([255, 256, 257, 1], [255, 256, 257, 1], 3, 1, 64, BF, True),
    ([0, 300, 0, 5, 0], [0, 300, 7, 5, 0], 6, 2, 128, FP, True),
    ([64, 511, 3], [640, 700, 130], 8, 1, 64, BF, True),       # the last part of longer texts
    ([300, 129, 40], [100, 1, 0], 4, 4, 128, BF, True),         # rows that see nothing
    ([300, 40, 9], [77, 0, 513], 3, 3, 128, FP, False),         # cross attention
    ([1500], [1500], 2, 1, 128, BF, True),
    ([1000, 700], [1000, 700], 5, 5, 64, FP, False),
    ([5] * 70 + [200], [5] * 70 + [200], 4, 4, 64, BF, True),    # more sequences than a warp
    ([2, 129] * 40, [129, 2] * 40, 2, 1, 128, FP, True),
    ([0] * 30 + [3, 700, 0, 257] + [0] * 30, [9] * 31 + [600, 5, 300] + [1] * 30, 3, 1, 64, BF, True),
    ([20] * 1100, [20] * 1100, 1, 1, 64, BF, True),
    ([0] * 33, [5] * 33, 2, 2, 64, BF, True),
]


# few query tiles and many keys: the key axis is shared by a cluster
FWD += [
    ([1], [5000], 8, 1, 128, BF, True),
    ([64, 1, 200], [4096, 3000, 129], 4, 2, 64, FP, True),
    ([256, 130], [2600, 700], 3, 1, 128, BF, True),
    ([130], [6001], 6, 2, 128, FP, False),
    ([5, 0, 300], [1030, 0, 40], 2, 1, 64, BF, True),   # a text with no key for its first rows
    ([700], [2000], 1, 1, 64, BF, True),
    ([512], [2100], 16, 16, 64, BF, True),              # four and two CTAs a tile
    ([1000], [1100], 16, 16, 64, FP, True),
]


@pytest.mark.parametrize("case", FWD, ids=[str(i) for i in range(len(FWD))])
def test_fwd(cuda_ok, case):
    lq, lk, H, K, d, dt, causal = case
    q, k, v = inputs(lq, lk, H, K, d, dt)
    prob = bsa.SeqProblem.make(H, K, d, dt, causal=causal)
    wide = torch.full((q.shape[0], H + 1, d + 8), 5.0, dtype=dt, device="cuda")
    out, st = wide[:, :H, :d], status_word()
    lse = torch.full((H, q.shape[0]), 5.0, device="cuda")
    bsa.packed_attn_fwd(prob, q, k, v, cu_of(lq), cu_of(lk), out, lse, dev_status=st)
    assert int(st) == 0
    check_fwd(q, k, v, lq, lk, causal, out, lse, 1 / math.sqrt(d))
    # what no sequence owns is as it was
    n = sum(lq)
    assert bool((wide[n:] == 5.0).all()) and bool((lse[:, n:] == 5.0).all())
    assert bool((wide[:, H] == 5.0).all()) and bool((wide[:, :, d:] == 5.0).all())
    again = torch.empty_like(out)
    bsa.packed_attn_fwd(prob, q, k, v, cu_of(lq), cu_of(lk), again)
    assert torch.equal(again[:n], out[:n])


def test_fwd_large_and_growing_scores(cuda_ok):
    """Row maxima that grow from key tile to key tile force the rescale."""
    lens = [900]
    q, k, v = inputs(lens, lens, 2, 1, 128, BF, gain=8.0)
    k = k * torch.linspace(0.1, 4.0, k.shape[0], device="cuda", dtype=BF)[:, None, None]
    prob = bsa.SeqProblem.make(2, 1, 128)
    out, lse = torch.empty_like(q), torch.empty(2, q.shape[0], device="cuda")
    bsa.packed_attn_fwd(prob, q, k, v, cu_of(lens), cu_of(lens), out, lse)
    check_fwd(q, k, v, lens, lens, True, out, lse, 1 / math.sqrt(128))


def test_fwd_one_dead_value_stays_where_it_is(cuda_ok):
    """A NaN in one sequence reaches no other one."""
    lens = [200, 130, 64]
    q, k, v = inputs(lens, lens, 2, 2, 64, BF)
    prob = bsa.SeqProblem.make(2, 2, 64)
    a, b = torch.empty_like(q), torch.empty_like(q)
    bsa.packed_attn_fwd(prob, q, k, v, cu_of(lens), cu_of(lens), a)
    for t in (q, k, v):
        t[200:330] = math.nan
    bsa.packed_attn_fwd(prob, q, k, v, cu_of(lens), cu_of(lens), b)
    for s in (slice(0, 200), slice(330, 394)):
        assert torch.equal(a[s], b[s])
    assert bool(b[200:330].isnan().all())


def test_fwd_long_sequence_sampled(cuda_ok):
    """A long walk: sampled rows against the oracle."""
    n, H, K, d = 20000, 2, 1, 128
    q, k, v = inputs([n], [n], H, K, d, BF, tail=0)
    prob = bsa.SeqProblem.make(H, K, d)
    out, lse = torch.empty_like(q), torch.empty(H, n, device="cuda")
    bsa.packed_attn_fwd(prob, q, k, v, cu_of([n]), cu_of([n]), out, lse)
    rows = torch.tensor([0, 1, 127, 128, 9999, 10000, 15487, n - 129, n - 1])
    for h in range(H):
        o, lse2, p, g = attention64(q[rows.cuda(), h], k[:, 0], v[:, 0], rows + 1, 1 / math.sqrt(d))
        assert_within(out[rows.cuda(), h], o, output_bound(o, p, v[:, 0], g, BF))
        assert bool(((lse[h, rows.cuda()].double() - lse2).abs() <= 2e-3).all())


def test_rows_in_front_of_the_first_offset(cuda_ok):
    """Offsets that begin behind row 0: the rows in front are not a sequence's."""
    q, k, v = inputs([5, 200, 130], [9, 200, 130], 4, 2, 64, FP, tail=3)
    for t, n in ((q, 5), (k, 9), (v, 9)):
        t[:n] = math.nan
    dout = torch.randn(q.shape, device="cuda").half()
    dout[:5], dout[335:] = math.nan, math.nan
    cq = torch.tensor([5, 205, 335], dtype=torch.int32, device="cuda")
    ck = torch.tensor([9, 209, 339], dtype=torch.int32, device="cuda")
    prob, st = bsa.SeqProblem.make(4, 2, 64, FP), status_word()
    out, lse = torch.full_like(q, 5.0), torch.full((4, q.shape[0]), 5.0, device="cuda")
    bsa.packed_attn_fwd(prob, q, k, v, cq, ck, out, lse, dev_status=st)
    assert int(st) == 0
    check_fwd(q[5:335], k[9:339], v[9:339], [200, 130], [200, 130], True, out[5:335], None, 1 / 8)
    assert bool((out[:5] == 5.0).all()) and bool((out[335:] == 5.0).all())
    assert bool((lse[:, :5] == 5.0).all()) and bool((lse[:, 335:] == 5.0).all())
    dq, dk, dv, bufs = backward(prob, q, k, v, dout, cq, ck)
    check_bwd(q[5:335], k[9:339], v[9:339], dout[5:335], [200, 130], [200, 130], True, dq[5:335],
              dk[9:339], dv[9:339], 1 / 8)
    for x, a, b in ((bufs[0], 5, 335), (bufs[1], 9, 339), (bufs[2], 9, 339)):
        assert bool((x[:a] == 5.0).all()) and bool((x[b:] == 5.0).all())


def test_no_keys_and_no_queries(cuda_ok):
    """Tensors without a row: the outputs that exist are 0."""
    prob = bsa.SeqProblem.make(4, 2, 128)
    some, none = torch.randn(70, 4, 128, device="cuda").bfloat16(), torch.empty(0, 4, 128, dtype=BF, device="cuda")
    kv, no_kv = torch.randn(70, 2, 128, device="cuda").bfloat16(), torch.empty(0, 2, 128, dtype=BF, device="cuda")
    full, empty = cu_of([30, 40]), cu_of([0, 0])
    for q, k, cq, ck in ((some, no_kv, full, empty), (none, kv, empty, full), (none, no_kv, empty, empty)):
        out, lse, st = torch.full_like(q, 5.0), torch.full((4, q.shape[0]), 5.0, device="cuda"), status_word()
        bsa.packed_attn_fwd(prob, q, k, k, cq, ck, out, lse, dev_status=st)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
        grads = [torch.full_like(t, 5.0) for t in (q, k, k)]
        ws = torch.empty(bsa.packed_bwd_workspace_bytes(prob, q.shape[0], 2), dtype=torch.uint8, device="cuda")
        bsa.packed_attn_bwd(prob, q, k, k, out, q, lse, cq, ck, *grads, ws, dev_status=st)
        assert all(bool((x == 0).all()) for x in grads) and int(st) == 0


def test_fwd_timeout_path_of_a_cluster(cuda_ok):
    """The same where a cluster shares the keys."""
    q, k, v = inputs([64], [3000], 4, 2, 64, BF, tail=0)
    prob, st = bsa.SeqProblem.make(4, 2, 64), status_word()
    out, cq, ck = torch.empty_like(q), cu_of([64]), cu_of([3000])
    bsa.debug_stall_pv(True)
    try:
        bsa.packed_attn_fwd(prob, q, k, v, cq, ck, out, dev_status=st)
        torch.cuda.synchronize()
    finally:
        bsa.debug_stall_pv(False)
    assert int(st) == 6
    bsa.packed_attn_fwd(prob, q, k, v, cq, ck, out)
    check_fwd(q, k, v, [64], [3000], True, out, None, 1 / 8)


def test_fwd_reports_bad_offsets(cuda_ok):
    """Offsets that descend or leave the tensor: reported, read as empty; the
    other sequences are right."""
    lens = [100, 50, 70]
    q, k, v = inputs(lens, lens, 4, 2, 64, BF, tail=0)
    prob = bsa.SeqProblem.make(4, 2, 64)
    for bad_q, bad_k in (([0, 100, 150, 221], None), ([0, 100, 90, 90], None), (None, [0, 100, 150, 9999]),
                         ([-5, 100, 150, 220], None)):
        cq, ck = cu_of(lens), cu_of(lens)
        if bad_q:
            cq = torch.tensor(bad_q, dtype=torch.int32, device="cuda")
        if bad_k:
            ck = torch.tensor(bad_k, dtype=torch.int32, device="cuda")
        out, st = torch.full_like(q, 5.0), status_word()
        bsa.packed_attn_fwd(prob, q, k, v, cq, ck, out, dev_status=st)
        assert int(st) == 1
        good = slice(100, 150) if (bad_q or [0, 0, 150])[2] == 150 else slice(0, 100)
        b = 1 if good.start else 0
        n = lens[b]
        check_fwd(q[good], k[good], v[good], [n], [n], True, out[good], None, 1 / 8)


def test_fwd_reports_bad_offsets_among_many(cuda_ok):
    """Among many sequences, found by a search, a bad one is reported."""
    lens = [7, 0, 3, 150] * 10
    q, k, v = inputs(lens, lens, 2, 2, 64, BF, tail=0)
    prob, good = bsa.SeqProblem.make(2, 2, 64), cu_of(lens)
    for at, value in ((17, 10_000_000), (25, 0), (1, -5), (40, q.shape[0] + 1)):
        cu, st = good.clone(), status_word()
        cu[at] = value
        out = torch.full_like(q, 3.0)
        bsa.packed_attn_fwd(prob, q, k, v, cu, cu, out, dev_status=st)
        assert int(st) == 1
    out, st = torch.full_like(q, 3.0), status_word()
    bsa.packed_attn_fwd(prob, q, k, v, good, good, out, dev_status=st)
    assert int(st) == 0
    check_fwd(q, k, v, lens, lens, True, out, None, 1 / 8)


def test_fwd_captured_and_replayed(cuda_ok):
    lens = [130, 257]
    q, k, v = inputs(lens, lens, 4, 2, 128, FP, tail=0)
    prob = bsa.SeqProblem.make(4, 2, 128, FP)
    out, cu = torch.empty_like(q), cu_of(lens)
    bsa.packed_attn_fwd(prob, q, k, v, cu, cu, out)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsa.packed_attn_fwd(prob, q, k, v, cu, cu, out)
    out.zero_()
    g.replay()
    assert torch.equal(out, want)
    cu.copy_(torch.tensor([0, 300, 387], dtype=torch.int32))
    g.replay()
    check_fwd(q, k, v, [300, 87], [300, 87], True, out, None, 1 / math.sqrt(128))


def test_fwd_timeout_path(cuda_ok):
    """With the products held back the waits run out, the status says so and
    the next call is right."""
    lens = [300]
    q, k, v = inputs(lens, lens, 2, 1, 64, BF, tail=0)
    prob, st = bsa.SeqProblem.make(2, 1, 64), status_word()
    out, cu = torch.empty_like(q), cu_of(lens)
    bsa.debug_stall_pv(True)
    try:
        bsa.packed_attn_fwd(prob, q, k, v, cu, cu, out, dev_status=st)
        torch.cuda.synchronize()
    finally:
        bsa.debug_stall_pv(False)
    assert int(st) == 6
    bsa.packed_attn_fwd(prob, q, k, v, cu, cu, out)
    check_fwd(q, k, v, lens, lens, True, out, None, 1 / 8)


def test_fwd_binding_refuses(cuda_ok):
    lens = [40]
    q, k, v = inputs(lens, lens, 4, 2, 64, BF, tail=0)
    prob, cu = bsa.SeqProblem.make(4, 2, 64), cu_of(lens)
    out, lse = torch.empty_like(q), torch.empty(4, 40, device="cuda")
    ok = [prob, q, k, v, cu, cu, out, lse]
    for i, bad in [(1, q.float()), (1, q[:, :3]), (2, k.cpu()), (2, k[..., ::2]), (3, v[:39]),
                   (4, cu.long()), (5, cu[:1]), (6, out.half()), (6, out[:, :2]), (7, lse.double()),
                   (7, lse[:3])]:
        a = list(ok)
        a[i] = bad
        with pytest.raises(ValueError):
            bsa.packed_attn_fwd(*a)
    a = list(ok)
    a[2] = k[:, :1].expand(40, 2, 64)  # a broadcast view
    with pytest.raises(bsa.BSAError, match="broadcast"):
        bsa.packed_attn_fwd(*a)
    bsa.packed_attn_fwd(*ok)


# ---- backward --------------------------------------------------------------------------
def check_bwd(q, k, v, dout, lq, lk, causal, dq, dk, dv, scale):
    H, K, dt = q.shape[1], k.shape[1], q.dtype
    G = H // K
    q0 = k0 = 0
    do_n, v_n = dout[:sum(lq)].double(), v[:sum(lk)].double()
    for a, b in zip(lq, lk):
        lim = limits(a, b, causal)
        for kv in range(K):
            want_k = want_v = e_k = e_v = 0
            for h in range(kv * G, (kv + 1) * G):
                top = 2 * float(do_n[:, kv * G:(kv + 1) * G].norm(dim=-1).max() * v_n[:, kv].norm(dim=-1).max()) if sum(lk) and sum(lq) else None
                (x, y, z), (e, f, g) = grads64(q[q0:q0 + a, h], k[k0:k0 + b, kv], v[k0:k0 + b, kv],
                                               dout[q0:q0 + a, h], lim, scale, dt, top)
                assert_within(dq[q0:q0 + a, h], x, rounded_bound(x, e, dt), "dq %d x %d head %d" % (a, b, h))
                want_k, want_v, e_k, e_v = want_k + y, want_v + z, e_k + f, e_v + g
            what = "%d x %d kv head %d" % (a, b, kv)
            assert_within(dk[k0:k0 + b, kv], want_k, rounded_bound(want_k, e_k, dt), "dk " + what)
            assert_within(dv[k0:k0 + b, kv], want_v, rounded_bound(want_v, e_v, dt), "dv " + what)
        q0, k0 = q0 + a, k0 + b


def backward(prob, q, k, v, dout, cq, ck, wide=8):
    """Forward and backward into gradients that are slices of wider buffers,
    with a workspace of NaN."""
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[1], q.shape[0], device="cuda")
    st = status_word()
    bsa.packed_attn_fwd(prob, q, k, v, cq, ck, out, lse, dev_status=st)
    bufs = [torch.full((t.shape[0], t.shape[1] + 1, t.shape[2] + wide), 5.0, dtype=t.dtype, device="cuda")
            for t in (q, k, v)]
    dq, dk, dv = (x[:, :-1, :q.shape[2]] for x in bufs)
    ws = torch.full((bsa.packed_bwd_workspace_bytes(prob, q.shape[0], cq.shape[0] - 1),), 255,
                    dtype=torch.uint8, device="cuda")
    bsa.packed_attn_bwd(prob, q, k, v, out, dout, lse, cq, ck, dq, dk, dv, ws, dev_status=st)
    assert int(st) == 0
    return dq, dk, dv, bufs


BWD = [
    # lens_q, lens_k, heads, kv, d, dtype, causal, scale of dout
    ([1], [1], 1, 1, 64, BF, True, 1.0),
    ([64, 100, 3], [64, 100, 3], 8, 2, 64, FP, True, 1.0),
    ([127, 128, 129], [127, 128, 129], 4, 2, 128, BF, True, 1.0),
    ([0, 300, 0, 5, 0], [0, 300, 7, 5, 0], 6, 2, 128, FP, True, 1e-4),
    ([64, 511, 3], [640, 700, 130], 4, 1, 64, BF, True, 1.0),
    ([300, 129, 40], [100, 1, 0], 4, 4, 128, BF, True, 1.0),
    ([300, 40, 9], [77, 0, 513], 3, 3, 128, FP, False, 500.0),
    ([700], [700], 3, 1, 128, BF, True, 1.0),
    ([500, 257], [500, 257], 2, 2, 64, BF, False, 1.0),
    ([5] * 40 + [200], [5] * 40 + [200], 2, 1, 64, FP, True, 1.0),
    ([2, 4, 1], [2, 4, 9], 6, 3, 64, BF, True, 1.0),            # rows of a few keys: dS cancels
    ([1100, 1024], [1100, 1024], 2, 1, 64, BF, True, 1.0),      # around where D changes its form
    ([300], [1300], 2, 2, 128, FP, False, 1.0),
    ([200, 77, 300], [200, 77, 300], 20, 20, 64, BF, True, 1.0),  # a CTA per key tile
    ([130, 257], [130, 300], 44, 22, 128, FP, False, 1.0),
    ([0] * 30 + [3, 700, 0, 257] + [0] * 30, [9] * 31 + [600, 5, 300] + [1] * 30, 3, 1, 64, BF, True, 1.0),
    ([20, 3] * 550, [20, 3] * 550, 1, 1, 64, FP, True, 1.0),
    ([1100], [1100], 8, 1, 128, BF, True, 1.0),                  # several CTAs per key tile
    ([1000, 130], [900, 140], 8, 1, 64, FP, True, 1.0),
]


@pytest.mark.parametrize("case", BWD, ids=[str(i) for i in range(len(BWD))])
def test_bwd(cuda_ok, case):
    lq, lk, H, K, d, dt, causal, gain = case
    q, k, v = inputs(lq, lk, H, K, d, dt)
    gen = torch.Generator().manual_seed(12)
    dout = (torch.randn(q.shape[0], H + 2, d, generator=gen) * gain).to(dt)
    dout[sum(lq):] = math.nan
    dout = dout.cuda()[:, 1:H + 1]
    prob = bsa.SeqProblem.make(H, K, d, dt, causal=causal)
    cq, ck = cu_of(lq), cu_of(lk)
    dq, dk, dv, bufs = backward(prob, q, k, v, dout, cq, ck)
    check_bwd(q, k, v, dout, lq, lk, causal, dq, dk, dv, 1 / math.sqrt(d))
    for x, n in zip(bufs, (sum(lq), sum(lk), sum(lk))):
        assert bool((x[n:] == 5.0).all()) and bool((x[:, -1] == 5.0).all()) and bool((x[:, :, d:] == 5.0).all())
    again = backward(prob, q, k, v, dout, cq, ck, wide=0)
    for x, y, n in zip((dq, dk, dv), again, (sum(lq), sum(lk), sum(lk))):
        assert torch.equal(x[:n], y[:n])


def test_bwd_one_dead_value_stays_where_it_is(cuda_ok):
    lens = [200, 130, 64]
    q, k, v = inputs(lens, lens, 2, 1, 64, BF, tail=0)
    dout = torch.randn(q.shape, device="cuda").bfloat16()
    prob, cu = bsa.SeqProblem.make(2, 1, 64), cu_of(lens)
    a = backward(prob, q, k, v, dout, cu, cu)
    for t in (q, k, v, dout):
        t[200:330] = math.nan
    b = backward(prob, q, k, v, dout, cu, cu)
    for x, y in zip(a[:3], b[:3]):
        for s in (slice(0, 200), slice(330, 394)):
            assert torch.equal(x[s], y[s])
        assert bool(y[200:330].isnan().all())


def test_bwd_captured_and_replayed(cuda_ok):
    lens = [130, 257]
    q, k, v = inputs(lens, lens, 4, 2, 64, FP, tail=0)
    dout = torch.randn(q.shape, device="cuda").half()
    prob, cu = bsa.SeqProblem.make(4, 2, 64, FP), cu_of(lens)
    want = backward(prob, q, k, v, dout, cu, cu)
    out, lse = torch.empty_like(q), torch.empty(4, q.shape[0], device="cuda")
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    ws = torch.empty(bsa.packed_bwd_workspace_bytes(prob, q.shape[0], 2), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsa.packed_attn_fwd(prob, q, k, v, cu, cu, out, lse)
        bsa.packed_attn_bwd(prob, q, k, v, out, dout, lse, cu, cu, *grads, ws)
    for _ in range(2):
        g.replay()
        for x, y in zip(grads, want):
            assert torch.equal(x, y)
            x.zero_()


@pytest.mark.parametrize("heads", [(2, 1), (32, 32)])  # key tiles shared by CTAs or not
def test_bwd_timeout_path(cuda_ok, heads):
    lens = [300]
    q, k, v = inputs(lens, lens, *heads, 64, BF, tail=0)
    dout = torch.randn(q.shape, device="cuda").bfloat16()
    prob, cu, st = bsa.SeqProblem.make(*heads, 64), cu_of(lens), status_word()
    want = backward(prob, q, k, v, dout, cu, cu)
    out, lse = torch.empty_like(q), torch.empty(heads[0], 300, device="cuda")
    bsa.packed_attn_fwd(prob, q, k, v, cu, cu, out, lse)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    ws = torch.empty(bsa.packed_bwd_workspace_bytes(prob, 300, 1), dtype=torch.uint8, device="cuda")
    bsa.debug_stall_pv(True)
    try:
        bsa.packed_attn_bwd(prob, q, k, v, out, dout, lse, cu, cu, *grads, ws, dev_status=st)
        torch.cuda.synchronize()
    finally:
        bsa.debug_stall_pv(False)
    assert int(st) == 6
    bsa.packed_attn_bwd(prob, q, k, v, out, dout, lse, cu, cu, *grads, ws)
    for x, y in zip(grads, want):
        assert torch.equal(x, y)


def test_bwd_binding_refuses(cuda_ok):
    lens = [40]
    q, k, v = inputs(lens, lens, 4, 2, 64, BF, tail=0)
    prob, cu = bsa.SeqProblem.make(4, 2, 64), cu_of(lens)
    out, lse = torch.empty_like(q), torch.empty(4, 40, device="cuda")
    bsa.packed_attn_fwd(prob, q, k, v, cu, cu, out, lse)
    ws = torch.empty(bsa.packed_bwd_workspace_bytes(prob, 40, 1), dtype=torch.uint8, device="cuda")
    ok = [prob, q, k, v, out, q.clone(), lse, cu, cu, torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), ws]
    for i, bad in [(1, q.cpu()), (2, k.half()), (3, v[:, :1]), (4, out[:3]), (5, q.float()), (6, lse[:, :3]),
                   (7, cu.long()), (8, cu[:1]), (9, k), (10, q), (11, v.cpu()), (12, ws.cpu())]:
        a = list(ok)
        a[i] = bad
        with pytest.raises(ValueError):
            bsa.packed_attn_bwd(*a)
    with pytest.raises(bsa.BSAError):
        bsa.packed_attn_bwd(*ok[:-1], ws[:64])
    a = list(ok)
    a[5] = q[:1].expand_as(q)  # the gradient of a sum: a broadcast view
    with pytest.raises(bsa.BSAError, match="broadcast"):
        bsa.packed_attn_bwd(*a)
    bsa.packed_attn_bwd(*ok)


# fp16 scales dS by a power of two; it has to come from the sequence's own rows
@pytest.mark.parametrize("H,K,d", [(2, 1, 64), (4, 2, 128), (20, 20, 64)])
@pytest.mark.parametrize("many", [False, True])
def test_bwd_fp16_beside_a_large_neighbour(cuda_ok, H, K, d, many):
    """Rows of sequence 0 grow by 2^15 in dO and V together: the gradients of
    the others stay bit for bit, within bounds from their own maxima."""
    lens = [300, 200, 64] + ([3] * 40 if many else [])
    q, k, v = inputs(lens, lens, H, K, d, FP, tail=0)
    gen = torch.Generator().manual_seed(21)
    dout = torch.randn(q.shape, generator=gen)
    v, dout = v.clone(), dout.cuda()
    v[300:] *= 2.0 ** -4
    dout[300:] *= 2.0 ** -6
    dout = dout.half()
    prob, cu = bsa.SeqProblem.make(H, K, d, FP), cu_of(lens)
    a = backward(prob, q, k, v, dout, cu, cu)
    v[:300] *= 2.0 ** 6
    dout[:300] *= 2.0 ** 9
    b = backward(prob, q, k, v, dout, cu, cu)
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x[300:], y[300:])
    at = 300
    for n in lens[1:4]:
        s = slice(at, at + n)
        check_bwd(q[s], k[s], v[s], dout[s], [n], [n], True, *(x[s] for x in b[:3]), 1 / math.sqrt(d))
        at += n


@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_bwd_fp16_one_dead_value_stays_where_it_is(cuda_ok, value):
    lens = [200, 130, 64]
    q, k, v = inputs(lens, lens, 2, 1, 64, FP, tail=0)
    v, dout = v.clone(), torch.randn(q.shape, device="cuda").half()
    v[:200] *= 2.0 ** -7
    dout[:200] *= 2.0 ** -7
    prob, cu = bsa.SeqProblem.make(2, 1, 64, FP), cu_of(lens)
    a = backward(prob, q, k, v, dout, cu, cu)
    dout[230, 0, 5] = value
    b = backward(prob, q, k, v, dout, cu, cu)
    for x, y in zip(a[:3], b[:3]):
        for s in (slice(0, 200), slice(330, 394)):
            assert torch.equal(x[s], y[s])
    assert not bool(b[0][230, 0].isfinite().any())


# a cluster's size comes from the lengths' sums: batches on both sides of every step
SPLIT = [
    ([1] * 30, [128] * 30, 8, 2, 64, BF),          # many walks of a step: none
    ([250] * 8, [250] * 8, 4, 2, 128, FP),
    ([1] * 16, [4000] * 16, 8, 2, 64, BF),         # twos, two waves of fours
    ([1] * 8, [4000] * 8, 8, 2, 128, FP),          # fours
    ([7, 130, 1], [600, 500, 700], 4, 2, 64, BF),  # eights
    ([1, 1, 1, 300], [9, 20, 300, 300], 2, 2, 128, BF),
    ([200, 1], [3000, 4000], 8, 8, 64, FP),
    ([40] * 5, [2000, 3, 0, 900, 129], 2, 1, 128, BF),
]


@pytest.mark.parametrize("case", SPLIT, ids=[str(i) for i in range(len(SPLIT))])
def test_fwd_shared_walks_of_several_sequences(cuda_ok, case):
    lq, lk, H, K, d, dt = case
    q, k, v = inputs(lq, lk, H, K, d, dt)
    prob, st = bsa.SeqProblem.make(H, K, d, dt), status_word()
    out, lse = torch.full_like(q, 5.0), torch.full((H, q.shape[0]), 5.0, device="cuda")
    bsa.packed_attn_fwd(prob, q, k, v, cu_of(lq), cu_of(lk), out, lse, dev_status=st)
    assert int(st) == 0
    check_fwd(q, k, v, lq, lk, True, out, lse, 1 / math.sqrt(d))
    n = sum(lq)
    assert bool((out[n:] == 5.0).all()) and bool((lse[:, n:] == 5.0).all())
