"""The paged cache on the GPU: appending with rotation and the attention of
one new token, against 64-bit oracles with derived bounds."""
import math

import pytest
import torch

import block_sparse_attention_47_b200 as bsa
from seq_helpers import (HALF, TINY, assert_within, attention64, cu_of, make_pages, output_bound,
                         rope_table)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def new_cache(n_pages, page, kv, d, dtype, layout, fill=float("nan")):
    """k and v views [n_pages, page, kv, d] of token- or head-major storage."""
    if layout == "head":
        mk = lambda: torch.full((n_pages, kv, page, d), fill, dtype=dtype, device="cuda").transpose(1, 2)  # noqa: E731
        return mk(), mk()
    if layout == "fused":  # K and V of a page side by side
        both = torch.full((n_pages, page, 2, kv, d), fill, dtype=dtype, device="cuda")
        return both[:, :, 0], both[:, :, 1]
    return (torch.full((n_pages, page, kv, d), fill, dtype=dtype, device="cuda"),
            torch.full((n_pages, page, kv, d), fill, dtype=dtype, device="cuda"))


# ---- append ------------------------------------------------------------------
def turn64(x, rope, rows, rot, interleaved):
    y = x.double().clone()
    if rope is None:
        return y, torch.zeros_like(y)
    half, i = rot // 2, torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    cs = rope.double()[rows]
    c, s = cs[:, None, :half], cs[:, None, half:]
    x1, x2 = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
    # two fp32 products and a sum, then one rounding to the element type
    bound = torch.zeros_like(y)
    bound[..., a] = bound[..., b] = (x1.abs() + x2.abs()) * 2.0 ** -22
    bound[..., a] += HALF[x.dtype] * y[..., a].abs() + TINY[x.dtype]
    bound[..., b] += HALF[x.dtype] * y[..., b].abs() + TINY[x.dtype]
    return y, bound


APPEND = [
    # new, past, heads, kv, d, dtype, page, rot, interleaved, layout, dense, rows
    ([1], [0], 1, 1, 64, BF, 1, 64, False, "token", True, False),
    ([1, 1, 1], [0, 15, 16], 8, 2, 128, BF, 16, 128, False, "token", False, False),
    ([5, 0, 33, 1], [3, 7, 0, 129], 6, 3, 64, FP, 5, 32, True, "head", True, False),
    ([700, 1, 129], [0, 100, 31], 24, 8, 128, FP, 64, 64, True, "fused", True, True),
    ([257, 64], [1, 2], 4, 4, 128, BF, 16, 16, False, "head", True, False),
    ([1] * 70, list(range(70)), 16, 2, 64, BF, 32, 0, False, "token", False, False),
    ([0, 0, 2100, 0], [4, 0, 60, 9], 3, 1, 128, BF, 7, 96, False, "token", True, True),
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
def test_append(cuda_ok, case):
    new, past, H, K, d, dt, page, rot, inter, layout, dense, by_row = case
    gen = torch.Generator().manual_seed(7)
    lens = [a + b for a, b in zip(new, past)]
    n, tail = sum(new), 3  # rows behind the last sequence: not to be touched
    table, n_pages = make_pages(lens, page, gen)
    kc, vc = new_cache(n_pages, page, K, d, dt, layout, fill=7.0)
    kc0, vc0 = kc.clone(), vc.clone()
    fused = torch.randn(n + tail, H + 2 * K, d, generator=gen).to(dt).cuda()
    q, k, v = fused[:, :H], fused[:, H:H + K], fused[:, H + K:]
    rows = torch.randint(0, 50, (n + tail,), generator=gen, dtype=torch.int32).cuda() if by_row else None
    rope = rope_table(max(max(lens), 50), rot) if rot else None
    q_out = torch.full((n + tail, H, d), 5.0, dtype=dt, device="cuda")
    k_out = torch.full((n + tail, K, d), 5.0, dtype=dt, device="cuda") if dense else None
    st = status_word()
    bsa.kv_append(bsa.SeqProblem.make(H, K, d, dt), k, v, kc, vc, table, cu_of(new),
                  torch.tensor(lens, dtype=torch.int32, device="cuda"), rope=rope,
                  interleaved=inter, rope_rows=rows, q=q, q_out=q_out, k_out=k_out, dev_status=st)
    assert int(st) == 0
    pos = torch.cat([torch.arange(p, p + a) for a, p in zip(new, past)]).cuda()
    at = rows[:n].long() if by_row else pos
    seq = torch.cat([torch.full((a,), b, dtype=torch.long) for b, a in enumerate(new)]).cuda()
    pg, tok = table[seq, pos // page].long(), pos % page
    for name, got, src in (("q", q_out, q), ("k_out", k_out, k)):
        if got is None:
            continue
        want, bound = turn64(src[:n], rope, at, rot, inter)
        assert_within(got[:n], want, bound, name)
        assert bool((got[n:] == 5.0).all()), "rows behind the last sequence changed"
    want, bound = turn64(k[:n], rope, at, rot, inter)
    assert_within(kc[pg, tok], want, bound, "k_cache")
    assert torch.equal(vc[pg, tok], v[:n])
    # everything else is as it was
    kc0[pg, tok], vc0[pg, tok] = kc[pg, tok], vc[pg, tok]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


def test_append_in_place(cuda_ok):
    gen = torch.Generator().manual_seed(1)
    p = bsa.SeqProblem.make(8, 2, 128)
    q, k = torch.randn(40, 8, 128, generator=gen).bfloat16().cuda(), torch.randn(40, 2, 128, generator=gen).bfloat16().cuda()
    rope, cu = rope_table(64, 128), cu_of([40])
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    table, n_pages = make_pages([40], 16, gen)
    kc, vc = new_cache(n_pages, 16, 2, 128, BF, "token", 0.0)
    a, b = torch.empty_like(q), torch.empty_like(k)
    bsa.kv_append(p, k, k, kc, vc, table, cu, lens, rope=rope, q=q, q_out=a, k_out=b)
    bsa.kv_append(p, k, k.clone(), kc, vc, table, cu, lens, rope=rope, q=q, q_out=q, k_out=k)
    assert torch.equal(a, q) and torch.equal(b, k)


@pytest.mark.parametrize("what", ["page", "negative_page", "position", "rope", "rope_row", "table"])
def test_append_reports_what_the_host_cannot_see(cuda_ok, what):
    """The bad token's outputs are left alone; the others are written."""
    p = bsa.SeqProblem.make(4, 2, 64)
    kc, vc = new_cache(4, 16, 2, 64, BF, "token", 7.0)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    lens, cu = [20, 5], cu_of([1, 1])
    rope, rows = rope_table(64, 64), None
    if what == "page":
        table[0, 1] = 4
    elif what == "negative_page":
        table[0, 1] = -1
    elif what == "position":
        lens[0] = 0
    elif what == "rope":
        rope = rope_table(10, 64)
    elif what == "rope_row":
        rows = torch.tensor([-1, 3], dtype=torch.int32, device="cuda")
    else:
        lens[0] = 33
    x = torch.ones(2, 4, 64, dtype=BF, device="cuda")
    q_out, k_out, st = torch.full_like(x, 5.0), torch.full_like(x[:, :2], 5.0), status_word()
    bsa.kv_append(p, x[:, :2], x[:, :2], kc, vc, table, cu,
                  torch.tensor(lens, dtype=torch.int32, device="cuda"), rope=rope, rope_rows=rows,
                  q=x, q_out=q_out, k_out=k_out, dev_status=st)
    assert int(st) == 1
    assert bool((q_out[0] == 5.0).all()) and bool((k_out[0] == 5.0).all())
    assert not bool((q_out[1] == 5.0).any())
    assert bool((vc[2, 4] == 1.0).all())
    vc[2, 4] = 7.0
    assert bool((vc == 7.0).all())


# ---- decode --------------------------------------------------------------------
def check_decode(q, kc, vc, table, lens, out, scale):
    B, H, d = q.shape
    K, page = kc.shape[2], kc.shape[1]
    G = H // K
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((out[b] == 0).all())
            continue
        rows = table[b, :-(-n // page)].long()
        for h in range(K):
            k = kc[rows][:, :, h].reshape(-1, d)[:n]
            v = vc[rows][:, :, h].reshape(-1, d)[:n]
            qh = q[b, h * G:(h + 1) * G]
            o, _, p, g = attention64(qh, k, v, torch.full((G,), n), scale)
            assert_within(out[b, h * G:(h + 1) * G], o, output_bound(o, p, v, g, q.dtype),
                          "sequence %d, kv head %d" % (b, h))


def decode_case(lens, H, K, d, dt, page, layout, seed=3, spare=3, gain=2.0):
    gen = torch.Generator().manual_seed(seed)
    table, n_pages = make_pages(lens, page, gen, spare)
    kc, vc = new_cache(n_pages, page, K, d, dt, layout)  # NaN wherever nothing is cached
    for b, n in enumerate(lens):
        if n:
            pos = torch.arange(n)
            pg, tok = table.cpu()[b, pos // page].long().cuda(), (pos % page).cuda()
            kc[pg, tok] = torch.randn(n, K, d, generator=gen).to(dt).cuda()
            vc[pg, tok] = torch.randn(n, K, d, generator=gen).to(dt).cuda()
    q = (torch.randn(len(lens), H, d, generator=gen) * gain).to(dt).cuda()
    return q, kc, vc, table


DECODE = [
    # lens, heads, kv, d, dtype, page, layout
    ([1], 1, 1, 64, BF, 16, "token"),
    ([31, 32, 33], 8, 2, 128, FP, 16, "token"),
    ([0, 5, 0, 64, 0], 6, 2, 64, BF, 5, "head"),
    ([129, 1, 4097, 700], 32, 8, 128, BF, 64, "head"),
    ([20011], 3, 1, 128, BF, 7, "token"),
    ([9000, 3], 16, 1, 64, FP, 32, "fused"),
    ([600, 77], 17, 1, 128, FP, 1, "token"),
    ([333], 40, 1, 64, BF, 128, "token"),
    ([(37 * i) % 300 for i in range(200)], 4, 4, 64, FP, 16, "token"),
    ([(997 * i) % 2000 for i in range(24)], 24, 8, 128, BF, 16, "fused"),
]


@pytest.mark.parametrize("case", DECODE, ids=[str(i) for i in range(len(DECODE))])
def test_decode(cuda_ok, case):
    lens, H, K, d, dt, page, layout = case
    q, kc, vc, table = decode_case(lens, H, K, d, dt, page, layout)
    prob = bsa.SeqProblem.make(H, K, d, dt)
    wide = torch.full((len(lens), H + 1, d + 8), 5.0, dtype=dt, device="cuda")
    out = wide[:, :H, :d]
    # a workspace of NaN: nothing in it may be read before it is written
    ws = torch.full((bsa.decode_workspace_bytes(prob),), 255, dtype=torch.uint8, device="cuda")
    ln, st = torch.tensor(lens, dtype=torch.int32, device="cuda"), status_word()
    bsa.paged_attn_decode(prob, q, kc, vc, table, ln, out, ws, dev_status=st)
    assert int(st) == 0
    check_decode(q, kc, vc, table, lens, out, 1 / math.sqrt(d))
    assert bool((wide[:, H] == 5.0).all()) and bool((wide[:, :, d:] == 5.0).all())
    first = out.clone()
    for _ in range(3):
        bsa.paged_attn_decode(prob, q, kc, vc, table, ln, out, ws)
        assert torch.equal(first, out)


def test_decode_large_scores(cuda_ok):
    """Scores in the hundreds: the running maximum has to carry them."""
    q, kc, vc, table = decode_case([700, 2500], 8, 2, 128, BF, 16, "token", gain=60.0)
    prob = bsa.SeqProblem.make(8, 2, 128)
    out, ws = torch.empty_like(q), torch.empty(bsa.decode_workspace_bytes(prob), dtype=torch.uint8, device="cuda")
    bsa.paged_attn_decode(prob, q, kc, vc, table, torch.tensor([700, 2500], dtype=torch.int32, device="cuda"), out, ws)
    check_decode(q, kc, vc, table, [700, 2500], out, 1 / math.sqrt(128))


def test_decode_offsets_beyond_32_bits(cuda_ok):
    """A cache of over 2^31 elements, the sequence in its last pages."""
    K, d, page = 8, 128, 64
    n_pages = (1 << 31) // (K * d * page) + 40
    kc = torch.zeros((n_pages, page, K, d), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    gen = torch.Generator().manual_seed(5)
    n = 1000
    table = torch.arange(n_pages - 1, n_pages - 17, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    for c in (kc, vc):
        c[n_pages - 16:] = torch.randn(16, page, K, d, generator=gen).to(BF).cuda()
    q = torch.randn(1, 16, d, generator=gen).to(BF).cuda()
    prob = bsa.SeqProblem.make(16, K, d)
    out, ws = torch.empty_like(q), torch.empty(bsa.decode_workspace_bytes(prob), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    bsa.paged_attn_decode(prob, q, kc, vc, table, lens, out, ws)
    check_decode(q, kc, vc, table, [n], out, 1 / math.sqrt(d))
    # and the append reaches them
    k = torch.randn(1, K, d, generator=gen).to(BF).cuda()
    bsa.kv_append(prob, k, k, kc, vc, table, cu_of([1]), lens)
    assert torch.equal(kc[table[0, 999 // page].long(), 999 % page], k[0])
    assert torch.equal(vc[table[0, 999 // page].long(), 999 % page], k[0])


@pytest.mark.parametrize("what", ["page", "length", "negative"])
def test_decode_reports_bad_pages_and_lengths(cuda_ok, what):
    """The bad sequence's output is meaningless, the other one's is right."""
    q, kc, vc, table = decode_case([300, 200], 8, 2, 64, BF, 16, "token")
    prob, st = bsa.SeqProblem.make(8, 2, 64), status_word()
    given = [300, 200]
    if what == "page":
        table[0, 3] = kc.shape[0]
    else:
        given[0] = 10 ** 9 if what == "length" else -4
        table[0] = table[0].clamp(max=kc.shape[0] - 1)
    out, ws = torch.empty_like(q), torch.empty(bsa.decode_workspace_bytes(prob), dtype=torch.uint8, device="cuda")
    bsa.paged_attn_decode(prob, q, kc, vc, table, torch.tensor(given, dtype=torch.int32, device="cuda"), out, ws, dev_status=st)
    assert int(st) == 1
    check_decode(q[1:], kc, vc, table[1:], [200], out[1:], 1 / 8)
    # without a word of the caller's the library's own receives it
    bsa.take_default_status()
    bsa.paged_attn_decode(prob, q, kc, vc, table, torch.tensor(given, dtype=torch.int32, device="cuda"), out, ws)
    assert bsa.take_default_status() == 1


def test_decode_captured_and_replayed_with_other_lengths(cuda_ok):
    lens = [257, 40, 1100]
    q, kc, vc, table = decode_case(lens, 8, 2, 128, FP, 16, "token")
    prob = bsa.SeqProblem.make(8, 2, 128, FP)
    out, ws = torch.empty_like(q), torch.empty(bsa.decode_workspace_bytes(prob), dtype=torch.uint8, device="cuda")
    ln = torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        bsa.paged_attn_decode(prob, q, kc, vc, table, ln, out, ws)
    for now in ([3, 40, 1000], [257, 1, 1100], [1, 33, 8]):
        ln.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check_decode(q, kc, vc, table, now, out, 1 / math.sqrt(128))


def test_decode_on_two_streams_at_once(cuda_ok):
    lens = [1500, 900]
    q, kc, vc, table = decode_case(lens, 8, 2, 128, BF, 16, "token")
    prob = bsa.SeqProblem.make(8, 2, 128)
    n = bsa.decode_workspace_bytes(prob)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    runs = [(torch.cuda.Stream(), torch.empty_like(q), torch.empty(n, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, out, ws in runs:
            bsa.paged_attn_decode(prob, q, kc, vc, table, ln, out, ws, stream=s)
    torch.cuda.synchronize()
    for _, out, _ in runs:
        check_decode(q, kc, vc, table, lens, out, 1 / math.sqrt(128))


def test_binding_refuses(cuda_ok):
    p = bsa.SeqProblem.make(8, 2, 64)
    q, kc, vc, table = decode_case([20, 7], 8, 2, 64, BF, 16, "token")
    ln = torch.tensor([20, 7], dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(q), torch.empty(bsa.decode_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    ok = [p, q, kc, vc, table, ln, out, ws]
    for i, bad in [(1, q.half()), (1, q[:, :4]), (1, q.cpu()), (2, kc.half()), (3, vc[:1]),
                   (2, kc[..., :32]), (4, table.long()), (4, table[:1]), (5, ln.long()), (5, ln.cpu()),
                   (6, out.float()), (6, out[:1]), (7, ws.cpu())]:
        a = list(ok)
        a[i] = bad
        with pytest.raises(ValueError):
            bsa.paged_attn_decode(*a)
    with pytest.raises(bsa.BSAError):
        bsa.paged_attn_decode(*ok[:-1], ws[:100])
    with pytest.raises(ValueError):
        bsa.paged_attn_decode(*ok, dev_status=torch.zeros(1, device="cuda"))
    bsa.paged_attn_decode(*ok)


@pytest.mark.parametrize("n,H,K,d,dt", [(5000, 4, 4, 64, BF), (3001, 34, 2, 64, FP), (300000, 1, 1, 64, BF)])
def test_decode_many_sequences(cuda_ok, n, H, K, d, dt):
    """Thousands of caches, some empty, some shared by several CTAs."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    lens = torch.randint(0, 60, (n,), generator=gen, device="cuda", dtype=torch.int32)
    lens[::7] = 0
    lens[n // 2] = 4000
    page, pages, width = 16, 4096, 250
    kc, vc = (torch.randn(pages, page, K, d, generator=gen, device="cuda").to(dt) for _ in range(2))
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    reach = torch.arange(width, device="cuda")[None] < ((lens + page - 1) // page)[:, None]
    table[reach] = torch.randint(0, pages, (int(reach.sum()),), generator=gen, device="cuda", dtype=torch.int32)
    q = torch.randn(n, H, d, generator=gen, device="cuda").to(dt)
    prob, out, st = bsa.SeqProblem.make(H, K, d, dt), torch.full_like(q, 5.0), status_word()
    ws = torch.full((bsa.decode_workspace_bytes(prob),), 255, dtype=torch.uint8, device="cuda")
    bsa.paged_attn_decode(prob, q, kc, vc, table, lens, out, ws, dev_status=st)
    assert int(st) == 0
    assert bool((out[lens == 0] == 0).all())
    at = torch.cat([torch.tensor([0, 1, 2, n // 2 - 1, n // 2, n // 2 + 1, n - 1]),
                    torch.randint(0, n, (50,), generator=torch.Generator().manual_seed(7))]).cuda()
    check_decode(q[at], kc, vc, table[at], lens[at].tolist(), out[at], 1 / math.sqrt(d))
    again = torch.empty_like(out)
    bsa.paged_attn_decode(prob, q, kc, vc, table, lens, again, ws)
    assert torch.equal(again, out)
