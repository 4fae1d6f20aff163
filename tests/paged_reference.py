"""Plain 64-bit forms of the paged-cache operators, and paged caches to run
them on (test infrastructure only)."""

import math

import torch

INF = float("inf")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Cache:
    """A paged cache with random rows, as a server would leave it: pages in
    random places of the pool, unused table entries that are no pages, and NaN
    in every slot past a sequence's last key.  layout: "nhd" pages (token, head,
    d); "hnd" pages (head, token, d); "joint" keys and values in one buffer."""

    def __init__(self, lens, hkv, d, page, dtype, seed, layout="nhd", poison=True, device="cuda", spare=2, table_pad=1,
                 v_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g, dtype=torch.int64).tolist()
        width = max(1, max(need)) + table_pad
        table = torch.full((B, width), -7, dtype=torch.int32)
        table[:, -1] = 1 << 30
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.lens, self.page, self.hkv, self.d, self.dtype = list(lens), page, hkv, d, dtype
        k = torch.randn(self.n_pages, page, hkv, d, generator=g).to(dtype)
        v = (torch.randn(self.n_pages, page, hkv, d, generator=g) * v_scale).to(dtype)
        if poison:
            live = torch.zeros(self.n_pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                j = torch.arange(n)
                live[table[b, j // page].long(), j % page] = True
            k[~live] = float("nan")
            v[~live] = float("nan")
        k, v = k.to(device), v.to(device)
        if layout == "hnd":
            k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
        elif layout == "joint":
            both = torch.stack((k, v), dim=1)
            k, v = both[:, 0], both[:, 1]
        self.k, self.v = k, v
        self.table = table.to(device)
        self.seqlens = torch.tensor(lens, dtype=torch.int32, device=device)

    def args(self):
        return self.k, self.v, self.table, self.seqlens

    def rows(self, pages, b, n=None):
        """(n, Hkv, d) history of sequence b."""
        j = torch.arange(self.lens[b] if n is None else n, device=pages.device)
        return pages[self.table[b, j // self.page].long(), j % self.page]


def cu_of(lens, device="cuda"):
    t = [0]
    for n in lens:
        t.append(t[-1] + n)
    return torch.tensor(t, dtype=torch.int32, device=device)


def attention(q, k, v, causal, scale):
    """One sequence in 64 bits: q (m, Hq, d), k, v (n, Hkv, d).  Returns O (m,
    Hq, d), lse (Hq, m), and per output the sums that its tolerance needs:
    sum p |v| / l and sum |v| / l (l relative to the row's maximum)."""
    m, hq, d = q.shape
    n, hkv = k.shape[0], k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    o = torch.zeros(m, hq, d, dtype=torch.float64, device=q.device)
    a, t = torch.zeros_like(o), torch.zeros_like(o)
    lse = torch.full((hq, m), -INF, dtype=torch.float64, device=q.device)
    if n == 0 or m == 0:
        return o, lse, a, t
    hidden = torch.ones(m, n, dtype=torch.bool, device=q.device).triu(n - m + 1) if causal else \
        torch.zeros(m, n, dtype=torch.bool, device=q.device)
    for h in range(hq):
        s = (q[:, h] @ k[:, h // (hq // hkv)].t()) * scale
        s = s.masked_fill(hidden, -INF)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -INF, torch.zeros_like(top), top)
        p = (s - top).exp()
        l = p.sum(-1, keepdim=True)
        seen = l[:, 0] > 0
        lse[h] = torch.where(seen, l[:, 0].log() + top[:, 0], torch.full_like(l[:, 0], -INF))
        l = torch.where(l > 0, l, torch.ones_like(l))
        vv = v[:, h // (hq // hkv)]
        o[:, h], a[:, h] = (p @ vv) / l, (p @ vv.abs()) / l
        t[:, h] = ((~hidden).double() @ vv.abs()) / l
    return o, lse, a, t


def score_error(q, k, scale):
    """Bound of the error of one score: a dot product of exact 16-bit products
    accumulated in fp32 (d terms, each addition off by at most 2^-23 of the sum
    of magnitudes, tensor cores may truncate), and its scaling."""
    if q.numel() == 0 or k.numel() == 0:
        return 0.0
    big = float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) * scale
    return (q.shape[-1] + 8) * 2.0 ** -23 * big


def check_attention(o, lse, q, cache, cu_lens, causal, scale):
    """Every element of o and lse against the 64-bit form.  The bar of o: the
    rounding of each weight to 16 bits (half a step of sum p |v|; in fp16 below
    2^-14 a weight is off by up to 2^-25 of the row's maximum), of o itself, and
    the fp32 scores, exponentials and sums."""
    u = half_step(q.dtype)
    at = 0
    assert torch.isfinite(o.float()).all()
    for b, m in enumerate(cu_lens):
        k, v = cache.rows(cache.k, b), cache.rows(cache.v, b)
        qb = q[at:at + m]
        ref, rl, a, t = attention(qb, k, v, causal, scale)
        ds = score_error(qb, k, scale) + 2.0 ** -18
        bar = u * (a + ref.abs()) * 1.01 + 2 * ds * a + 1e-30
        bar = bar + (2.0 ** -25 * t + 2.0 ** -25 if q.dtype == torch.float16 else 0.0)
        err = (o[at:at + m].double() - ref).abs()
        assert bool((err <= bar).all()), (b, float((err / bar).max()))
        got = lse[:, at:at + m].double()
        assert torch.equal(got == -INF, rl == -INF), b
        fin = rl != -INF
        if fin.any():
            e = (got - rl)[fin].abs()
            assert bool((e <= ds + 2.0 ** -20 + rl[fin].abs() * 2.0 ** -22).all()), (b, float(e.max()))
        gone = (rl == -INF).t()
        assert bool((o[at:at + m][gone] == 0).all())
        at += m


def key_weights(q, k, lse, causal, scale):
    """One sequence in 64 bits: (Hkv, n) sums of exp(score - lse)."""
    m, hq, _ = q.shape
    n, hkv = k.shape[0], k.shape[1]
    w = torch.zeros(hkv, n, dtype=torch.float64, device=q.device)
    hidden = torch.ones(m, n, dtype=torch.bool, device=q.device).triu(n - m + 1) if causal else \
        torch.zeros(m, n, dtype=torch.bool, device=q.device)
    for h in range(hq):
        g = h // (hq // hkv)
        s = (q[:, h].double() @ k[:, g].double().t()) * scale - lse[h].double()[:, None]
        s = s.masked_fill(hidden | (lse[h] == -INF)[:, None], -INF)
        w[g] += s.exp().sum(0)
    return w


def turn(x, pos, freqs, amplitude, interleaved, sign=1.0):
    """Rotary embedding in 64 bits: x (rows, H, d), pos (rows)."""
    y = x.double().clone()
    half = freqs.numel()
    p = torch.arange(half, device=x.device)
    i1, i2 = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
    a = pos.double().to(x.device)[:, None] * freqs.to(x.device)[None]
    c, s = a.cos()[:, None] * amplitude, a.sin()[:, None] * amplitude * sign
    x1, x2 = y[..., i1].clone(), y[..., i2].clone()
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x1 * s + x2 * c
    return y


def check_turn(y, x, pos, freqs, amplitude, interleaved, sign=1.0):
    """Bar: half a step of the result, and of the rotation (angle off by up to
    2^-24 pi from its 32-bit fraction, sine and cosine and two products in
    fp32: 2^-20 in all) the pair's norm; in fp16 2^-25 for subnormal results."""
    ref = turn(x, pos, freqs, amplitude, interleaved, sign)
    half = freqs.numel()
    p = torch.arange(half, device=x.device)
    i1, i2 = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
    norm = torch.zeros_like(ref)
    norm[..., i1] = norm[..., i2] = torch.hypot(x.double()[..., i1], x.double()[..., i2]) * abs(amplitude)
    bar = half_step(x.dtype) * ref.abs() * 1.001 + 2.0 ** -20 * norm
    if x.dtype == torch.float16:
        bar = bar + 2.0 ** -25
    err = (y.double() - ref).abs()
    assert bool((err <= bar).all()), float((err / bar.clamp(min=1e-30)).max())
    assert torch.equal(y[..., 2 * half:], x[..., 2 * half:])


def evict(weights, n, budget, recent):
    """Kept indices of one (sequence, head) row of weights (host list)."""
    if n <= budget:
        return list(range(n))
    cand = n - recent
    big = [INF if x != x else x for x in weights[:cand]]
    nan = [x != x for x in weights[:cand]]
    order = sorted(range(cand), key=lambda j: (not nan[j], -big[j], j))
    return sorted(order[: budget - recent]) + list(range(cand, n))
