"""Measured cases of the packed-sequence and paged-cache attention operators.

Four kinds of case:
  fwd     attention over packed sequences (causal, or full as in cross
          attention), grouped heads
  grad    that forward with its row statistics, then its backward
  append  new keys and values into a paged cache, rotated on the way, and the
          new queries rotated
  decode  one new token per sequence over the paged cache

Each runs either in a plain form (elementary torch operations in 32 bits,
rounded once) or, with `own` set, through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _package():
    import block_sparse_attention_47_b200 as bsa
    return bsa


# ---- cases -----------------------------------------------------------------
# lens_q / lens_k: comma-separated lengths of the packed sequences.  append:
# lens_q are the new tokens, lens_k the lengths after them.  decode: lens_k
# are the cached lengths.

def listed():
    return [
        # one short caption through a small conditioning encoder: latency
        dict(name="prompt_short", kind="fwd", heads=8, kv_heads=8, d=64, dtype="bf16", causal=True,
             lens_q="37", lens_k="37"),
        # a batch of conditioning prompts of very different lengths, grouped heads
        dict(name="prompt_ragged", kind="fwd", heads=32, kv_heads=8, d=128, dtype="bf16",
             causal=True, lens_q="1,17,128,129,640,1000,2048,4096",
             lens_k="1,17,128,129,640,1000,2048,4096"),
        # one long prompt (a whole clip's tokens in causal order)
        dict(name="prompt_long", kind="fwd", heads=16, kv_heads=2, d=128, dtype="fp16",
             causal=True, lens_q="16384", lens_k="16384"),
        # video tokens of two clips attending to their text prefixes
        dict(name="cross_text", kind="fwd", heads=24, kv_heads=24, d=128, dtype="bf16",
             causal=False, lens_q="8064,5003", lens_k="512,77"),
        # the next piece of three prompts whose first tokens were seen before
        dict(name="prompt_next", kind="fwd", heads=16, kv_heads=2, d=64, dtype="fp16", causal=True,
             lens_q="256,511,64", lens_k="5000,511,2113"),
        # a training step's attention on a handful of short sequences
        dict(name="train_short", kind="grad", heads=8, kv_heads=2, d=64, dtype="fp16", causal=True,
             lens_q="64,100,3", lens_k="64,100,3"),
        # a packed training batch, three query heads to a key head
        dict(name="train_ragged", kind="grad", heads=24, kv_heads=8, d=128, dtype="bf16",
             causal=True, lens_q="4096,2048,1111,300", lens_k="4096,2048,1111,300"),
        # one generation step's append of a served batch
        dict(name="append_step", kind="append", heads=32, kv_heads=8, d=128, dtype="bf16",
             page=16, rot=128, interleaved=False, dense_k=False,
             lens_q=",".join(["1"] * 32),
             lens_k=",".join(str(1 + (i * 977) % 4096) for i in range(32))),
        # prompts written into the cache, with the dense rotated keys kept for
        # the prompt's own attention
        dict(name="append_prompt", kind="append", heads=24, kv_heads=8, d=128, dtype="fp16",
             page=64, rot=64, interleaved=True, dense_k=True,
             lens_q="12000,1,0,4097,8191,333", lens_k="12000,700,5,4097,9215,333"),
        # one sequence, short cache: latency
        dict(name="decode_one", kind="decode", heads=8, kv_heads=2, d=64, dtype="fp16", page=16,
             lens_k="300"),
        # a served batch of ragged lengths
        dict(name="decode_batch", kind="decode", heads=32, kv_heads=8, d=128, dtype="bf16",
             page=16, lens_k=",".join(str(1 + (i * i * 1931 + 613 * i) % 8192) for i in range(64))),
        # few sequences, very long caches: the split over the length
        dict(name="decode_long", kind="decode", heads=24, kv_heads=8, d=128, dtype="bf16",
             page=64, lens_k="131072,130001,65537,99991"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "grad", "append", "decode", "decode"])
    d = rng.choice([64, 128])
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8])
    heads = min(kv * group, 32) // kv * kv
    case = dict(kind=kind, heads=heads, kv_heads=kv, d=d, dtype=rng.choice(["bf16", "fp16"]))
    if kind in ("fwd", "grad"):
        n = rng.randint(1, 6)
        # the plain form pads to the longest: heads * n * longest^2 is bounded
        top = int(min(8192 if kind == "fwd" else 4096, math.sqrt((3.0e9 if kind == "fwd" else 1.2e9) / (heads * n))))
        lq = [_log_int(rng, 1, top) for _ in range(n)]
        causal = rng.random() < 0.75
        if rng.random() < 0.5:
            lk = list(lq)
        else:
            lk = [_log_int(rng, 1, top) for _ in range(n)]
        if n > 1 and rng.random() < 0.4:
            lq[rng.randrange(n)] = 0
        case.update(causal=causal, lens_q=",".join(map(str, lq)), lens_k=",".join(map(str, lk)))
    elif kind == "append":
        n = rng.randint(1, 48)
        step = rng.random() < 0.4
        new = [1 if step else _log_int(rng, 1, 1200) - 1 for _ in range(n)]
        if sum(new) == 0:
            new[0] = 5
        past = [_log_int(rng, 1, 4096) - 1 for _ in range(n)]
        case.update(page=rng.choice([1, 5, 16, 32, 64, 128]), rot=rng.choice([0, 32, d]),
                    interleaved=rng.random() < 0.5, dense_k=rng.random() < 0.5,
                    lens_q=",".join(map(str, new)),
                    lens_k=",".join(str(a + b) for a, b in zip(new, past)))
    else:
        n = _log_int(rng, 1, 64)
        top = int(min(131072, 4.0e8 / (n * kv * d)))
        lens = [_log_int(rng, 1, top) for _ in range(n)]
        if n > 2 and rng.random() < 0.3:
            lens[rng.randrange(n)] = 0
        case.update(page=rng.choice([5, 16, 32, 64, 128]), lens_k=",".join(map(str, lens)))
    return case


def _lens(text):
    return [int(x) for x in text.split(",")]


def _limits(lq, lk, causal):
    """Visible keys summed over the rows of one sequence."""
    if not causal:
        return lq * lk
    first = lk - lq + 1  # keys of row 0 (may be <= 0)
    if first >= 1:
        return (first + lk) * lq // 2
    return lk * (lk + 1) // 2


def work(case):
    H, K, d = case["heads"], case["kv_heads"], case["d"]
    lk = _lens(case["lens_k"])
    if case["kind"] in ("fwd", "grad"):
        lq = _lens(case["lens_q"])
        pairs = sum(_limits(a, b, case["causal"]) for a, b in zip(lq, lk))
        tq, tk = sum(lq), sum(lk)
        if case["kind"] == "fwd":
            return {"bytes": 2 * d * (2 * tq * H + 2 * tk * K), "flops": 4 * d * H * pairs}
        # q, k, v, dO read; o, dq, dk, dv and the row statistics written
        return {"bytes": 2 * d * (4 * tq * H + 4 * tk * K) + 4 * tq * H,
                "flops": 14 * d * H * pairs}
    if case["kind"] == "append":
        t = sum(_lens(case["lens_q"]))
        rows = t * (2 * H + 4 * K + (K if case["dense_k"] else 0))
        return {"bytes": rows * d * 2 + t * case["rot"] * 4, "flops": 3 * t * (H + K) * case["rot"]}
    n = len(lk)
    return {"bytes": 2 * d * (2 * sum(lk) * K + 2 * n * H), "flops": 4 * d * H * sum(lk)}


# ---- inputs ----------------------------------------------------------------

def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)


def _randn(gen, shape, dtype, gain=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=gen)
    return x.mul_(gain) if gain != 1.0 else x


def _pages(gen, lens, page):
    """Block table over a shuffled pool with a few pages to spare; unused
    entries hold -1."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    width = max(1, max(need))
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _rope_table(rows, rot):
    """cos | sin of position * 10000^(-2i/rot), angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    ang = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    H, K, d, dt = case["heads"], case["kv_heads"], case["d"], DTYPES[case["dtype"]]
    lk = _lens(case["lens_k"])
    s = dict(case=case, scale=1.0 / math.sqrt(d))
    if case["kind"] in ("fwd", "grad"):
        lq = _lens(case["lens_q"])
        # scores of standard deviation 2, as trained heads have them
        s.update(q=_randn(gen, (sum(lq), H, d), dt, 2.0), k=_randn(gen, (sum(lk), K, d), dt),
                 v=_randn(gen, (sum(lk), K, d), dt), cu_q=_cu(lq), cu_k=_cu(lk),
                 max_q=max(lq), max_k=max(lk))
        if case["kind"] == "grad":
            s["dout"] = _randn(gen, (sum(lq), H, d), dt)
    elif case["kind"] == "append":
        lq = _lens(case["lens_q"])
        table, n_pages = _pages(gen, lk, case["page"])
        s.update(q=_randn(gen, (sum(lq), H, d), dt), k=_randn(gen, (sum(lq), K, d), dt),
                 v=_randn(gen, (sum(lq), K, d), dt), cu_q=_cu(lq), table=table,
                 lens=torch.tensor(lk, dtype=torch.int32, device=DEV),
                 k_cache=_randn(gen, (n_pages, case["page"], K, d), dt),
                 v_cache=_randn(gen, (n_pages, case["page"], K, d), dt),
                 rope=_rope_table(max(lk), case["rot"]) if case["rot"] else None)
    else:
        table, n_pages = _pages(gen, lk, case["page"])
        s.update(q=_randn(gen, (len(lk), H, d), dt, 2.0), table=table,
                 lens=torch.tensor(lk, dtype=torch.int32, device=DEV),
                 k_cache=_randn(gen, (n_pages, case["page"], K, d), dt),
                 v_cache=_randn(gen, (n_pages, case["page"], K, d), dt), max_k=max(lk))
    if own:
        # the handle and the buffers that a program allocates once
        bsa = _package()
        prob = bsa.SeqProblem.make(heads=H, kv_heads=K, head_dim=d, dtype=dt,
                                   causal=case.get("causal", True), softmax_scale=s["scale"])
        s["prob"] = prob
        s["out"] = torch.empty_like(s["q"])
        if case["kind"] == "grad":
            s["lse"] = torch.empty((H, s["q"].shape[0]), dtype=torch.float32, device=DEV)
            s["grads"] = [torch.empty_like(s[n]) for n in ("q", "k", "v")]
            s["work"] = torch.empty(bsa.packed_bwd_workspace_bytes(prob, s["q"].shape[0], len(lk)),
                                    dtype=torch.uint8, device=DEV)
        elif case["kind"] == "append" and case["dense_k"]:
            s["k_out"] = torch.empty_like(s["k"])
        elif case["kind"] == "decode":
            s["work"] = torch.empty(bsa.decode_workspace_bytes(prob), dtype=torch.uint8,
                                    device=DEV)
    return s


# ---- one pass --------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"fwd": _plain_fwd, "grad": _plain_grad, "append": _plain_append,
            "decode": _plain_decode}[s["case"]["kind"]](s)


def _run_own(s):
    bsa, c, prob = _package(), s["case"], s["prob"]
    if c["kind"] == "fwd":
        bsa.packed_attn_fwd(prob, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"])
        return {"o": s["out"]}
    if c["kind"] == "grad":
        dq, dk, dv = s["grads"]
        bsa.packed_attn_fwd(prob, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], s["lse"])
        bsa.packed_attn_bwd(prob, s["q"], s["k"], s["v"], s["out"], s["dout"], s["lse"], s["cu_q"],
                            s["cu_k"], dq, dk, dv, s["work"])
        return {"o": s["out"], "lse": s["lse"], "dq": dq, "dk": dk, "dv": dv}
    if c["kind"] == "append":
        bsa.kv_append(prob, s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu_q"],
                      s["lens"], rope=s["rope"], interleaved=c["interleaved"], q=s["q"],
                      q_out=s["out"], k_out=s.get("k_out"))
        out = {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if c["dense_k"]:
            out["k"] = s["k_out"]
        return out
    bsa.paged_attn_decode(prob, s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                          s["out"], s["work"])
    return {"o": s["out"]}


def _padded(x, cu, longest):
    """[T, h, d] packed -> [B, h, longest, d] fp32, zero behind each length."""
    lens = (cu[1:] - cu[:-1]).long()
    at = torch.arange(longest, device=x.device)
    live = at[None, :] < lens[:, None]
    rows = (cu[:-1].long()[:, None] + at[None, :]).clamp_(max=max(x.shape[0] - 1, 0))
    y = x[rows].float() * live[:, :, None, None]
    return y.transpose(1, 2), live, rows


def _scores(s):
    """Masked scores [B, kv_heads, group, Lq, Lk] and what they came from."""
    c = s["case"]
    H, K = c["heads"], c["kv_heads"]
    q, live_q, rows_q = _padded(s["q"], s["cu_q"], s["max_q"])
    k, live_k, rows_k = _padded(s["k"], s["cu_k"], s["max_k"])
    v, _, _ = _padded(s["v"], s["cu_k"], s["max_k"])
    B = q.shape[0]
    q = q.reshape(B, K, H // K, q.shape[2], q.shape[3])
    seen = live_q[:, :, None] & live_k[:, None, :]
    if c["causal"]:
        lq = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
        lk = (s["cu_k"][1:] - s["cu_k"][:-1]).long()
        i = torch.arange(s["max_q"], device=q.device)
        j = torch.arange(s["max_k"], device=q.device)
        seen &= j[None, None, :] <= i[None, :, None] + (lk - lq)[:, None, None]
    seen = seen[:, None, None]
    sc = torch.matmul(q * s["scale"], k[:, :, None].transpose(-1, -2))
    sc.masked_fill_(~seen, float("-inf"))
    return sc, seen, q, k, v, (live_q, rows_q), (live_k, rows_k)


def _softmax(sc):
    """In place: the scores become probabilities; rows without any key 0."""
    m = sc.amax(dim=-1, keepdim=True)
    sc.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    total = sc.sum(dim=-1, keepdim=True)
    sc.div_(total.clamp(min=1e-37))
    return sc, m, total


def _packed(x, live):
    """[B, K, group, L, d] -> [T, K * group, d] of the live rows."""
    B, K, G, L, d = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(B, L, K * G, d)[live]


def _plain_fwd(s):
    sc, _, _, _, v, (live_q, _), _ = _scores(s)
    p, _, _ = _softmax(sc)
    return {"o": _packed(torch.matmul(p, v[:, :, None]), live_q).to(s["q"].dtype)}


def _plain_grad(s):
    dt = s["q"].dtype
    sc, _, q, k, v, (live_q, _), (live_k, _) = _scores(s)
    p, m, total = _softmax(sc)
    lse = (m + total.log()) * (1.0 / math.log(2.0))
    o = torch.matmul(p, v[:, :, None])
    do, _, _ = _padded(s["dout"], s["cu_q"], s["max_q"])
    do = do.reshape(q.shape)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(dim=2, keepdim=True)
    ds = torch.matmul(do, v[:, :, None].transpose(-1, -2))
    ds.sub_((do * o).sum(dim=-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k[:, :, None])
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(dim=2, keepdim=True)
    return {"o": _packed(o, live_q).to(dt), "lse": _packed(lse, live_q)[..., 0].t().contiguous(),
            "dq": _packed(dq, live_q).to(dt), "dk": _packed(dk, live_k).to(dt),
            "dv": _packed(dv, live_k).to(dt)}


def _rotated(x, rope, rows, rot, interleaved):
    if not rot:
        return x
    half = rot // 2
    cs = rope[rows]
    cos, sin = cs[:, None, :half], cs[:, None, half:]
    y = x.float()
    r, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, rest], dim=-1).to(x.dtype)


def _plain_append(s):
    c = s["case"]
    new = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    t = torch.arange(s["k"].shape[0], device=s["k"].device)
    b = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    pos = (s["lens"].long() - new)[b] + t - s["cu_q"].long()[b]
    slot = s["table"].long()[b, pos // c["page"]] * c["page"] + pos % c["page"]
    k = _rotated(s["k"], s["rope"], pos, c["rot"], c["interleaved"])
    q = _rotated(s["q"], s["rope"], pos, c["rot"], c["interleaved"])
    s["k_cache"].flatten(0, 1)[slot] = k
    s["v_cache"].flatten(0, 1)[slot] = s["v"]
    out = {"q": q if c["rot"] else q.clone(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["dense_k"]:
        out["k"] = k if c["rot"] else k.clone()
    return out


def _plain_decode(s):
    c = s["case"]
    H, K, d = c["heads"], c["kv_heads"], c["d"]
    B = s["q"].shape[0]
    table = s["table"].long().clamp(min=0)
    seen = torch.arange(table.shape[1] * c["page"], device=table.device)[None] < s["lens"][:, None]
    k = s["k_cache"][table].flatten(1, 2).transpose(1, 2).float()  # [B, K, L, d]
    q = s["q"].float().reshape(B, K, H // K, d) * s["scale"]
    sc = torch.matmul(q, k.transpose(-1, -2))
    del k
    sc.masked_fill_(~seen[:, None, None], float("-inf"))
    p, _, _ = _softmax(sc)
    v = s["v_cache"][table].flatten(1, 2).transpose(1, 2).float()
    return {"o": torch.matmul(p, v).reshape(B, H, d).to(s["q"].dtype)}


# ---- the definition in 64 bits ----------------------------------------------

def _exact_rows(q, k, v, lim, scale):
    """One head in float64: o, natural log-sum-exp and probabilities."""
    j = torch.arange(k.shape[0], device=q.device)
    z = (q @ k.t()) * scale
    z = torch.where(j[None, :] < lim[:, None], z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, dim=1)
    p = torch.where(lim[:, None] > 0, torch.exp(z - lse[:, None]), torch.zeros_like(z))
    return p @ v, lse, p


def _exact_attention(case, s):
    H, K = case["heads"], case["kv_heads"]
    lq, lk = _lens(case["lens_q"]), _lens(case["lens_k"])
    f64 = dict(dtype=torch.float64, device=s["q"].device)
    o = torch.zeros(s["q"].shape, **f64)
    grad = case["kind"] == "grad"
    if grad:
        lse2 = torch.zeros((H, s["q"].shape[0]), **f64)
        dq, dk, dv = torch.zeros_like(o), torch.zeros(s["k"].shape, **f64), torch.zeros(s["k"].shape, **f64)
    q0 = k0 = 0
    for a, b in zip(lq, lk):
        i = torch.arange(a, device=o.device)
        lim = torch.full((a,), b, device=o.device)
        if case["causal"]:
            lim = (i + 1 + b - a).clamp(0, b)
        for h in range(H):
            g = h // (H // K)
            q = s["q"][q0:q0 + a, h].double()
            k, v = s["k"][k0:k0 + b, g].double(), s["v"][k0:k0 + b, g].double()
            if a == 0:
                continue
            oh, lse, p = _exact_rows(q, k, v, lim, s["scale"])
            o[q0:q0 + a, h] = oh
            if grad:
                lse2[h, q0:q0 + a] = lse / math.log(2.0)
                do = s["dout"][q0:q0 + a, h].double()
                dv[k0:k0 + b, g] += p.t() @ do
                dp = do @ v.t()
                dz = p * (dp - (p * dp).sum(dim=1, keepdim=True))
                dq[q0:q0 + a, h] = dz @ k * s["scale"]
                dk[k0:k0 + b, g] += dz.t() @ q * s["scale"]
        q0, k0 = q0 + a, k0 + b
    return {"o": o, "lse": lse2, "dq": dq, "dk": dk, "dv": dv} if grad else {"o": o}


def _exact_turn(x, rope, rows, rot, interleaved):
    y = x.double()
    if not rot:
        return y
    half = rot // 2
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    cs = rope.double()[rows]
    z = torch.complex(y[..., first], y[..., second]) * torch.complex(cs[:, None, :half], cs[:, None, half:])
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_append(case, s):
    lq, lk = _lens(case["lens_q"]), _lens(case["lens_k"])
    pos = torch.cat([torch.arange(n - a, n, device=s["k"].device) for a, n in zip(lq, lk)])
    args = (s["rope"], pos, case["rot"], case["interleaved"])
    k, q = _exact_turn(s["k"], *args), _exact_turn(s["q"], *args)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    table, t = s["table"].tolist(), 0
    for b, (a, n) in enumerate(zip(lq, lk)):
        at = torch.arange(n - a, n, device=k.device)
        page = torch.tensor([table[b][x // case["page"]] for x in range(n - a, n)],
                            dtype=torch.long, device=k.device)
        kc[page, at % case["page"]] = k[t:t + a]
        vc[page, at % case["page"]] = s["v"][t:t + a].double()
        t += a
    out = {"q": q, "k_cache": kc, "v_cache": vc}
    if case["dense_k"]:
        out["k"] = k
    return out


def _exact_decode(case, s):
    H, K, page = case["heads"], case["kv_heads"], case["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(_lens(case["lens_k"])):
        if n == 0:
            continue
        rows = s["table"][b, :-(-n // page)].long()
        for g in range(K):
            k = s["k_cache"][rows][:, :, g].reshape(-1, case["d"])[:n].double()
            v = s["v_cache"][rows][:, :, g].reshape(-1, case["d"])[:n].double()
            h = slice(g * (H // K), (g + 1) * (H // K))
            q = s["q"][b, h].double()
            lim = torch.full((q.shape[0],), n, device=q.device)
            o[b, h] = _exact_rows(q, k, v, lim, s["scale"])[0]
    return {"o": o}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("fwd", "grad"):
        return _exact_attention(case, s)
    if case["kind"] == "append":
        return _exact_append(case, s)
    return _exact_decode(case, s)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(4)]:
        w = work(c)
        print("%-16s %10.3f MB %12.3f GFLOP" % (c.get("name", c["kind"]), w["bytes"] / 1e6, w["flops"] / 1e9))
