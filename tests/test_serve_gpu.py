"""The sequence operators as a serving or training program uses them: prompts
into the cache, then tokens one by one, against one 64-bit pass over the whole
text; the steps captured once and replayed; and a training step's gradients
against differences of its own forward."""
import math

import pytest
import torch

import block_sparse_attention_47_b200 as bsa
from seq_helpers import HALF, assert_within, attention64, cu_of, output_bound, rope_table

pytestmark = pytest.mark.gpu


def turned(x, rope, pos):
    """The rotation in 64 bits, rounded as the cache rounds it."""
    half = rope.shape[1] // 2
    c, s = rope.double()[pos][:, None, :half], rope.double()[pos][:, None, half:]
    y = x.double().clone()
    a, b = y[..., :half].clone(), y[..., half:2 * half].clone()
    y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


def layer(prob, n_seqs, page=16, pages_each=40, seed=0):
    n_pages = n_seqs * pages_each + 5
    at = bsa.PagedAttention(prob, n_pages, page, n_seqs, pages_each)
    at.k_cache.fill_(math.nan)
    at.v_cache.fill_(math.nan)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))
    at.block_table.copy_(order[:n_seqs * pages_each].reshape(n_seqs, pages_each).int())
    return at


def check_text(text, outs, prompts, rope, scale):
    """outs[b]: attention outputs of every token of sequence b, in order."""
    for b, (q, k, v) in enumerate(text):
        n, H, K = outs[b].shape[0], q.shape[1], k.shape[1]
        pos = torch.arange(n, device=q.device)
        qr, kr = turned(q[:n], rope, pos), turned(k[:n], rope, pos)
        # the rotated operands are themselves rounded: half a step of each of
        # q and k moves a score by up to 2 u scale sum |q_c k_c|
        u = HALF[q.dtype]
        for h in range(H):
            kk, vv = kr[:, h // (H // K)], v[:n, h // (H // K)]
            o, _, p, g = attention64(qr[:, h], kk, vv, pos.cpu() + 1, scale)
            g = g + 2.02 * u * scale * float((qr[:, h].abs() @ kk.abs().t()).max())
            assert_within(outs[b][:, h], o, output_bound(o, p, vv, g, q.dtype), "sequence %d head %d" % (b, h))


@pytest.mark.parametrize("H,K,d,dt", [(8, 2, 128, torch.bfloat16), (6, 6, 64, torch.float16)])
def test_prompts_then_tokens(cuda_ok, H, K, d, dt):
    prompts, steps = [130, 1, 300], 20
    gen = torch.Generator().manual_seed(4)
    text = [tuple(torch.randn(n + steps, x, d, generator=gen).to(dt).cuda() for x in (H, K, K)) for n in prompts]
    prob = bsa.SeqProblem.make(H, K, d, dt)
    at, rope = layer(prob, len(prompts)), rope_table(512, d)
    cu = cu_of(prompts)
    first = [torch.cat([t[i][:n] for t, n in zip(text, prompts)]) for i in range(3)]
    out = at.prompt(*first, cu, rope=rope)
    outs = [[o] for o in out.split(prompts)]
    # the generation step is captured once and replayed
    q1, k1, v1 = (torch.empty(len(prompts), x, d, dtype=dt, device="cuda") for x in (H, K, K))

    def feed(i):
        for src, dst in zip(range(3), (q1, k1, v1)):
            dst.copy_(torch.stack([t[src][n + i] for t, n in zip(text, prompts)]))

    feed(0)
    outs = [o + [s[None].clone()] for o, s in zip(outs, at.step(q1, k1, v1, rope=rope))]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one = at.step(q1, k1, v1, rope=rope)
    for i in range(1, steps):
        feed(i)
        g.replay()
        outs = [o + [s[None].clone()] for o, s in zip(outs, one)]
    at.check_status()
    assert at.seq_lens.tolist() == [n + steps for n in prompts]
    check_text(text, [torch.cat(o) for o in outs], prompts, rope, 1 / math.sqrt(d))


def test_pages_run_out(cuda_ok):
    """Tokens behind a sequence's last page are refused through the status."""
    prob = bsa.SeqProblem.make(2, 2, 64)
    at = layer(prob, 1, page=4, pages_each=2)
    x = torch.randn(8, 2, 64, device="cuda").bfloat16()
    at.prompt(x, x, x, cu_of([8]))
    at.check_status()
    at.step(x[:1], x[:1], x[:1])
    with pytest.raises(bsa.BSAError, match="INVALID_ARG"):
        at.check_status()


def test_other_stream(cuda_ok):
    """Calls on a stream that is not the current one."""
    prob = bsa.SeqProblem.make(4, 2, 128)
    q = torch.randn(500, 4, 128, device="cuda").bfloat16()
    k, v = (torch.randn(500, 2, 128, device="cuda").bfloat16() for _ in range(2))
    cu, want, got = cu_of([200, 300]), torch.empty_like(q), torch.empty_like(q)
    bsa.packed_attn_fwd(prob, q, k, v, cu, cu, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    bsa.packed_attn_fwd(prob, q, k, v, cu, cu, got, stream=s)
    s.synchronize()
    assert torch.equal(want, got)


def test_gradients_against_differences(cuda_ok):
    """sum(w * out) of the forward itself, in fp16, moved along a direction:
    the central difference against the gradients' inner product.  A difference
    of two rounded sums is off by at most 2 u sum |w out| / (2 h), and the
    third-order term is removed by halving h (Richardson)."""
    lens, H, K, d, dt = [70, 129], 4, 2, 64, torch.float16
    gen = torch.Generator().manual_seed(9)
    q, k, v, w = (torch.randn(sum(lens), x, d, generator=gen).to(dt).cuda() for x in (H, K, K, H))
    prob, cu = bsa.SeqProblem.make(H, K, d, dt), cu_of(lens)
    out, lse = torch.empty_like(q), torch.empty(H, sum(lens), device="cuda")
    bsa.packed_attn_fwd(prob, q, k, v, cu, cu, out, lse)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    ws = torch.empty(bsa.packed_bwd_workspace_bytes(prob, sum(lens), 2), dtype=torch.uint8, device="cuda")
    bsa.packed_attn_bwd(prob, q, k, v, out, w, lse, cu, cu, *grads, ws)

    def loss(a, b, c):
        o = torch.empty_like(q)
        bsa.packed_attn_fwd(prob, a, b, c, cu, cu, o)
        return float((o.double() * w.double()).sum())

    u = HALF[dt]
    for i, gr in enumerate(grads):
        base = [q, k, v]
        # a direction along the gradient: its inner product is far above the noise
        way = gr.double() / gr.double().norm() * 8.0
        ds, moved = [], []
        for h in (0.5, 0.25):
            up, down = [list(base) for _ in range(2)]
            up[i], down[i] = (base[i].double() + h * way).to(dt), (base[i].double() - h * way).to(dt)
            ds.append((loss(*up) - loss(*down)) / (2 * h))
            # the step actually taken, after rounding the moved operand
            moved.append(float((gr.double() * (up[i].double() - down[i].double())).sum()) / (2 * h))
        exact = float((gr.double() * way).sum())
        # outputs are rounded independently: the noise of a sum of n products
        # w o with errors up to 2 u |o| is within 4 sqrt(n) of its rms terms
        n = q.numel()
        noise = 4 * math.sqrt(n) * 2 * u * float((w.double() * out.double()).pow(2).mean().sqrt()) / (2 * 0.25)
        slack = abs(ds[0] - ds[1]) + noise + 4 * u * abs(exact) + max(abs(m - exact) for m in moved)
        assert abs(ds[1] - moved[1]) <= slack, (i, ds, moved, slack)
        assert slack <= 0.2 * abs(exact), (i, slack, exact)


def test_pages_that_nobody_assigned(cuda_ok):
    """A row of the table that nobody filled and a sequence's next page that is
    not there yet name no page: their tokens are reported, page 0 (another
    sequence's) stays as it was and the sequences beside them are right."""
    prob = bsa.SeqProblem.make(4, 2, 64)
    at = bsa.PagedAttention(prob, 8, 4, 3, 4)
    at.k_cache.zero_()
    at.v_cache.zero_()
    at.block_table[0, 0] = 0  # 3 tokens and the next: one page
    at.block_table[1, 0] = 5  # 4 tokens: the next one needs a page it does not have
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(7, x, 64, generator=gen).bfloat16().cuda() for x in (4, 2, 2))
    at.prompt(q, k, v, cu_of([3, 4, 0]))
    at.check_status()
    before = [at.k_cache.clone(), at.v_cache.clone()]
    q1, k1, v1 = (torch.randn(3, x, 64, generator=gen).bfloat16().cuda() for x in (4, 2, 2))
    out = at.step(q1, k1, v1)
    with pytest.raises(bsa.BSAError, match="INVALID_ARG"):
        at.check_status()
    for c, b, new in ((at.k_cache, before[0], k1), (at.v_cache, before[1], v1)):
        b[0, 3] = new[0]
        assert torch.equal(c, b)
    for h in range(4):
        kk, vv = (torch.cat([t[:3, h // 2], n[:1, h // 2]]) for t, n in ((k, k1), (v, v1)))
        o, _, p, g = attention64(q1[:1, h], kk, vv, torch.tensor([4]), 1 / 8)
        assert_within(out[:1, h], o, output_bound(o, p, vv, g, torch.bfloat16))


def test_a_refused_call_leaves_the_lengths(cuda_ok):
    """Whatever part of a call is refused, the lengths are as before it, and
    the corrected call writes where the refused one did."""
    prob = bsa.SeqProblem.make(4, 2, 64)
    at, other = layer(prob, 2, page=4), layer(prob, 2, page=4)
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(9, x, 64, generator=gen).bfloat16().cuda() for x in (4, 2, 2))
    cu = cu_of([5, 4])
    for bad in (v[:, :1].expand(9, 2, 64), v[:1].expand(9, 2, 64)):  # appended as they are, but not attended to
        with pytest.raises(bsa.BSAError, match="broadcast"):
            at.prompt(q, k, bad, cu)
        assert at.seq_lens.tolist() == [0, 0]
    assert torch.equal(at.prompt(q, k, v, cu), other.prompt(q, k, v, cu))
    for bad in ((q[:3], k[:3], v[:3]), (q[:2], k[:3], v[:3]), (q[:2, :2], k[:2], v[:2])):
        with pytest.raises(ValueError):
            at.step(*bad)
        assert at.seq_lens.tolist() == [5, 4]
    assert torch.equal(at.step(q[:2], k[:2], v[:2]), other.step(q[:2], k[:2], v[:2]))
    at.check_status()
    assert at.seq_lens.tolist() == [6, 5]


def test_the_first_sequences_take_a_step(cuda_ok):
    """A layer made for more sequences than there are: those behind the rows
    rest, with tokens or without."""
    prob, n = bsa.SeqProblem.make(4, 2, 64), 64
    at, small = layer(prob, 5, page=4), layer(prob, 2, page=4)
    small.block_table.copy_(at.block_table[:2])
    small.k_cache, small.v_cache = torch.zeros_like(at.k_cache), torch.zeros_like(at.v_cache)
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(12, x, n, generator=gen).bfloat16().cuda() for x in (4, 2, 2))
    at.prompt(q, k, v, cu_of([5, 4, 0, 3, 0]))
    small.prompt(q[:9], k[:9], v[:9], cu_of([5, 4]))
    cache = at.k_cache.clone()
    for i in range(3):
        x = (q[i:i + 2], k[i:i + 2], v[i:i + 2])
        assert torch.equal(at.step(*x), small.step(*x))
    assert at.seq_lens.tolist() == [8, 7, 0, 3, 0]
    assert at.step(q[:0], k[:0], v[:0]).shape == (0, 4, 64)
    at.check_status()
    third = at.block_table[3].long()
    assert torch.equal(at.k_cache[third].nan_to_num(7.0), cache[third].nan_to_num(7.0))


def test_a_second_prompt_is_reported(cuda_ok):
    """prompt() attends to its own tokens only: on a sequence that holds some
    already it says so; sequences without new tokens may hold any."""
    prob = bsa.SeqProblem.make(4, 2, 64)
    at = layer(prob, 3, page=4)
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(9, x, 64, generator=gen).bfloat16().cuda() for x in (4, 2, 2))
    at.prompt(q[:5], k[:5], v[:5], cu_of([5, 0, 0]))
    at.prompt(q[:4], k[:4], v[:4], cu_of([0, 4, 0]))  # the first rests
    at.check_status()
    assert at.seq_lens.tolist() == [5, 4, 0]
    at.prompt(q[:3], k[:3], v[:3], cu_of([0, 1, 2]))
    with pytest.raises(bsa.BSAError, match="INVALID_ARG"):
        at.check_status()
