"""64-bit oracles and error bounds of the token-sequence operators.

Rounding to a type with `torch.finfo(t).eps` is off by at most half a step,
u = eps / 2 relative to the value.  An attention output is sum_j p_j v_j with
p rounded to the element type before the product and the result rounded once
more, so its error is at most

    u (sum_j p_j |v_j| + |o|) + 2 g sum_j p_j |v_j|

where g bounds the relative error of a probability before its rounding: a
score is a sum of d fp32 products, off by at most d 2^-24 scale sum_c |q_c k_c|
(in the exponent, so relative in p), and the exponential, the scaling and the
running rescale add a few 2^-22.  Normalising by the fp32 sum doubles g.
"""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}  # smallest step near 0


def limits(lq, lk, causal):
    """Keys each row sees."""
    i = torch.arange(lq)
    return (i + 1 + lk - lq).clamp(0, lk) if causal else torch.full((lq,), lk)


def attention64(q, k, v, lim, scale):
    """One head in float64: o, log2-sum-exp2, p and the scores' error bound g."""
    q, k, v = q.double(), k.double(), v.double()
    z = (q @ k.t()) * scale
    seen = torch.arange(k.shape[0], device=q.device)[None] < lim.to(q.device)[:, None]
    z = z.masked_fill(~seen, -math.inf)
    none = ~seen.any(dim=1)
    m = z.amax(dim=1, keepdim=True) if k.shape[0] else z.new_zeros(q.shape[0], 1)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(z - m)
    s = e.sum(dim=1, keepdim=True)
    p = torch.where(none[:, None], torch.zeros_like(e), e / s.clamp(min=1e-300))
    lse2 = (m[:, 0] + torch.log(s[:, 0])) / math.log(2.0)
    g = 0.0
    if k.shape[0] and q.shape[0]:
        g = q.shape[1] * 2.0 ** -24 * scale * float((q.abs() @ k.abs().t()).max())
    return p @ v, lse2, p, g + 8 * 2.0 ** -22


def output_bound(o, p, v, g, dtype):
    pv = p @ v.double().abs()
    return HALF[dtype] * (pv + o.abs()) * 1.01 + 2 * g * pv + TINY[dtype]


def assert_within(got, want, bound, what=""):
    err = (got.double().cpu() - want.cpu()).abs()
    bound = bound.cpu()
    bad = ~(err <= bound)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g against %.3g" % (
        what, int(bad.sum()), bad.numel(), float(err[bad].max()),
        float(bound[bad][err[bad].argmax()]))


def cu_of(lens, device="cuda"):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=device)


def make_pages(lens, page, gen, spare=3, device="cuda"):
    """A shuffled block table (unused entries hold a page outside the cache)
    and the number of pages."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), 1 << 30, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.to(device), total


def rope_table(rows, rot, device="cuda"):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * inv[None]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().to(device)


def grads64(q, k, v, dout, lim, scale, dtype, factor_bound=None):
    """One head in float64: (dq, dk, dv) and their error bounds.

    The kernels recompute p from the rounded row statistics and round p and dS
    to the element type (half a step u):
        e_p  <= p gp,  gp = 2 g + 6e-6 + 2^-22 (1 + |lse2|)
        e_dS <= |dS| (u + gp) + p (e_dP + e_D),  e_dP <= d 2^-24 |dO| |V|
    D is sum_j p_j dP_j in fp32 for rows of up to 1,024 keys,
        e_D <= sum_j p_j (gp |dP_j| + e_dP_j) + n 2^-24 sum_j p_j |dP_j|,
    and rowsum(dO * O) of the forward's rounded output beyond,
        e_D <= |dO| (bound of O) + d 2^-24 |dO| |O|,
    and the products add n fp32 roundings and the final half step.  In fp16
    p and dS are scaled to 2^13 and at most 2^15, so that a value below fp16's
    normal range adds at most 2^-25 of that scale."""
    u, n = HALF[dtype], max(q.shape[0], k.shape[0])
    o, lse2, p, g = attention64(q, k, v, lim, scale)
    q, k, v, do = q.double(), k.double(), v.double(), dout.double()
    d = q.shape[1]
    dp = do @ v.t()
    row = (do * o).sum(dim=1, keepdim=True)
    ds = p * (dp - row)
    dq, dk, dv = scale * ds @ k, scale * ds.t() @ q, p.t() @ do
    finite = torch.where(torch.isinf(lse2), torch.zeros_like(lse2), lse2)
    gp = 2 * g + 6e-6 + 2.0 ** -22 * (1 + finite.abs())[:, None]
    e_dp = d * 2.0 ** -24 * (do.abs() @ v.abs().t())
    if k.shape[0] <= 1024:
        e_d = (p * (gp * dp.abs() + e_dp) + n * 2.0 ** -24 * p * dp.abs()).sum(dim=1, keepdim=True)
    else:
        e_o = output_bound(o, p, v, g, dtype)
        e_d = (do.abs() * e_o).sum(dim=1, keepdim=True) + d * 2.0 ** -24 * (do * o).abs().sum(dim=1, keepdim=True)
    e_ds = ds.abs() * (u + gp) + p * (e_dp + e_d)
    e_p = p * (u + gp)
    if dtype == torch.float16:
        e_p = e_p + 2.0 ** -25 * 2.0 ** -13
        if factor_bound:  # 2 max|dO| max|V| sits between 2^14 and 2^15
            e_ds = e_ds + 2.0 ** -25 * factor_bound * 2.0 ** -14
    acc = 1.01 + n * 2.0 ** -23
    e_q = scale * (e_ds @ k.abs()) * acc + n * 2.0 ** -23 * scale * (ds.abs() @ k.abs())
    e_k = scale * (e_ds.t() @ q.abs()) * acc + n * 2.0 ** -23 * scale * (ds.abs().t() @ q.abs())
    e_v = (e_p.t() @ do.abs()) * acc + n * 2.0 ** -23 * (p.t() @ do.abs())
    return (dq, dk, dv), (e_q, e_k, e_v)


def rounded_bound(x, e, dtype):
    """The bound of a stored gradient: its sums' error and the last rounding."""
    return e + HALF[dtype] * (x.abs() + e) + TINY[dtype]
