"""Plain 64-bit forms of the operators over caches of 8-bit floating point, and
such caches to run them on (test infrastructure only)."""

import math

import torch

from .paged_reference import INF, cu_of, half_step, score_error, turn   # noqa: F401

E4M3 = torch.float8_e4m3fn


def quantise(x):
    """(e4m3 values, scales) of x's rows, in fp32: what the cache's definition says."""
    x = x.float()
    top = x.abs().amax(-1)
    # (by a tensor: a division by a number is a product with its reciprocal on the GPU)
    scale = (top / torch.full_like(top, 448.0)).clamp(min=2.0 ** -126)
    bad = ~torch.isfinite(x).all(-1)
    v = (x / scale[..., None]).clamp(-448.0, 448.0)
    v = torch.where(bad[..., None], torch.zeros_like(v), v).to(E4M3)
    return v, torch.where(bad, torch.full_like(scale, math.nan), scale)


class Cache8:
    """A paged cache of e4m3 rows, as a server would leave it: pages in random places
    of the pool, unused table entries that are no pages, and NaN (values and scales)
    in every slot past a sequence's last key.  layout: "nhd" pages (token, head, d);
    "hnd" pages (head, token, d), scales too; "joint" keys and values in one buffer."""

    def __init__(self, lens, hkv, d, page, seed, layout="nhd", poison=True, device="cuda", spare=2, table_pad=1,
                 spread=1.0):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g, dtype=torch.int64).tolist()
        table = torch.full((B, max(1, max(need)) + table_pad), -7, dtype=torch.int32)
        table[:, -1] = 1 << 30
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.lens, self.page, self.hkv, self.d = list(lens), page, hkv, d
        shape = (self.n_pages, page, hkv, d)
        # rows of different sizes: the values' scales differ by up to `spread` octaves each way
        (k, ks), (v, vs) = (quantise(torch.randn(shape, generator=g) * size) for size in
                            (1.0, 2.0 ** ((torch.rand(shape[:3], generator=g) * 2 - 1) * spread)[..., None]))
        if poison:
            live = torch.zeros(self.n_pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                j = torch.arange(n)
                live[table[b, j // page].long(), j % page] = True
            for t in (k, v):
                t.view(torch.uint8)[~live] = 0x7f
            for t in (ks, vs):
                t[~live] = math.nan
        k, v, ks, vs = (t.to(device) for t in (k, v, ks, vs))
        if layout == "hnd":
            k, v, ks, vs = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v, ks, vs))
        elif layout == "joint":
            both, scales = torch.stack((k.view(torch.uint8), v.view(torch.uint8)), dim=1), torch.stack((ks, vs), dim=1)
            k, v, ks, vs = both[:, 0].view(E4M3), both[:, 1].view(E4M3), scales[:, 0], scales[:, 1]
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        self.table = table.to(device)
        self.seqlens = torch.tensor(lens, dtype=torch.int32, device=device)

    def args(self):
        return self.k, self.v, self.ks, self.vs, self.table, self.seqlens

    def places(self, b, n=None, first=0):
        j = torch.arange(first, self.lens[b] if n is None else first + n, device=self.table.device)
        return self.table[b, j // self.page].long(), j % self.page

    def rows(self, b, which):
        """(values, scales) of sequence b's history, (n, Hkv, d) fp32 and (n, Hkv)."""
        at = self.places(b)
        pages, scales = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        return pages.view(torch.uint8)[at].view(E4M3).float(), scales[at]

    def snapshot(self):
        return [t.clone() for t in (self.k.view(torch.uint8), self.v.view(torch.uint8), self.ks, self.vs)]


def bits_of(mask):
    """Python ints below 2^64 as an int64 tensor's entries."""
    return [m - (1 << 64) if m >> 63 else m for m in mask]


def random_trees(lens, seed):
    """Ancestors of each token and itself, as ints: parents drawn at random."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for n in lens:
        mask = []
        for i in range(n):
            up = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            mask.append((mask[up] if up >= 0 else 0) | 1 << i)
        rows += mask
    return rows


def attention(q, k, ks, v, vs, mask, scale):
    """One sequence in 64 bits: q (T, Hq, d), k and v e4m3 values (n, Hkv, d) with
    scales (n, Hkv), mask T ints or None (a chain).  Returns O, lse (Hq, T), and
    per output the sums that its tolerance needs: sum p |v| / l, and with l relative
    to the row's maximum, max vs sum |v| / l over what it sees (v unscaled)."""
    T, hq, d = q.shape
    n, hkv = k.shape[0], k.shape[1]
    dev = q.device
    o = torch.zeros(T, hq, d, dtype=torch.float64, device=dev)
    a, t = torch.zeros_like(o), torch.zeros_like(o)
    lse = torch.full((hq, T), -INF, dtype=torch.float64, device=dev)
    if n == 0 or T == 0:
        return o, lse, a, t
    place = torch.arange(n) - (n - T)
    rows = []
    for i in range(T):
        m = mask[i] if mask is not None else (2 << i) - 1
        tree = torch.tensor([bool(m >> x & 1) for x in range(T)])
        rows.append(torch.where(place < 0, torch.ones(n, dtype=torch.bool), tree[place.clamp(min=0)]))
    seen = torch.stack(rows).to(dev)
    q = q.double()
    for h in range(hq):
        g = h // (hq // hkv)
        kk, vv = k[:, g].double() * ks[:, g].double()[:, None], v[:, g].double() * vs[:, g].double()[:, None]
        s = (q[:, h] @ kk.t() * scale).masked_fill(~seen, -INF)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -INF, torch.zeros_like(top), top)
        p = (s - top).exp()
        l = p.sum(-1, keepdim=True)
        some = l[:, 0] > 0
        lse[h] = torch.where(some, l[:, 0].log() + top[:, 0], torch.full_like(l[:, 0], -INF))
        l = torch.where(l > 0, l, torch.ones_like(l))
        # (0 times a NaN that is not seen is no part of the sum)
        def dot(w, x):
            return torch.stack([(w[i][seen[i]][:, None] * x[seen[i]]).sum(0) for i in range(T)])
        o[:, h], a[:, h] = dot(p, vv) / l, dot(p, vv.abs()) / l
        big = torch.where(seen, vs[:, g].double()[None].expand(T, n), torch.zeros(1, dtype=torch.float64, device=dev)).amax(-1, True)
        t[:, h] = big * dot(torch.ones_like(p), v[:, g].double().abs()) / l
    return o, lse, a, t


def check_attention(o, lse, q, cache, lens, masks, scale):
    """Every element of o and lse against the 64-bit form.  The bar of o:
    * its own rounding, half a step of |o| (fp16: 2^-25 where it is subnormal);
    * a weight, times its value's scale over the largest, rounded to fp16 (2^-11 of
      it; held times 2^7 relative to a maximum that may lag by 2^8 and a scale
      reference of up to 4 times the largest, an absolute 2^-25 2^-7 4 = 2^-30);
    * the scores: exact products summed in fp32 (score_error), and the query held as
      a sum of e4m3 values down to 2^-10 where its largest is at least 224, so off by
      2^-17.8 of that: sqrt(d) 2^-17.8 max |q| |k| scale in a score;
    * exponentials, sums and the scales' products in fp32: 2^-18."""
    u = half_step(q.dtype)
    at = 0
    assert torch.isfinite(o.float()).all()
    for b, T in enumerate(lens):
        (k, ks), (v, vs) = cache.rows(b, "k"), cache.rows(b, "v")
        qb = q[at:at + T]
        ref, rl, a, t = attention(qb, k, ks, v, vs, masks[at:at + T] if masks is not None else None, scale)
        kk = k * ks[..., None]
        ds = 2.0 ** -18
        if k.numel() and T:
            ds += score_error(qb, kk, scale)
            ds += math.sqrt(q.shape[-1]) * 2.0 ** -17.8 * float(qb.abs().max()) * float(kk.double().norm(dim=-1).max()) * scale
        bar = u * ref.abs() * 1.01 + (2.0 ** -11 + 2 * ds) * 1.01 * a + 2.0 ** -30 * t + 1e-30
        if q.dtype == torch.float16:
            bar = bar + 2.0 ** -25
        err = (o[at:at + T].double() - ref).abs()
        assert bool((err <= bar).all()), (b, float((err / bar).max()))
        got = lse[:, at:at + T].double()
        assert torch.equal(got == -INF, rl == -INF), b
        fin = rl != -INF
        if fin.any():
            e = (got - rl)[fin].abs()
            assert bool((e <= ds + 2.0 ** -20 + rl[fin].abs() * 2.0 ** -22).all()), (b, float(e.max()))
        assert bool((o[at:at + T][(rl == -INF).t()] == 0).all())
        at += T


def half_step8(y):
    """Half a step of the e4m3 value nearest y (|y| <= 448)."""
    _, e = torch.frexp(y.abs().clamp(min=2.0 ** -6))
    return torch.ldexp(torch.ones_like(y), e - 5)
