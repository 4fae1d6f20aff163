"""Cases of two families of operators around the paged caches: the norm of each
head of the new queries and keys with their rotary embedding over one or several
axes of positions (forward and backward), and caches of 8-bit floating point
(new tokens quantised as they are written to the pages, keys and values read
back, and attention of single tokens or of trees of drafted tokens over them).

``run`` computes a case in its plain form (elementary torch operations in 32
bits, angles in 64), or, where ``own`` is set, through the package's entry
points.  ``exact`` gives the definition in 64 bits.
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
TOP = 448.0            # the largest e4m3 value
LEAST = 2.0 ** -126    # the smallest scale of a row


def listed():
    return [
        # a decoding step's queries and keys: 32 sequences, one token each, far positions
        dict(name="norm_decode_b32", op="norm", dtype="bf16", tokens=32, hq=32, hkv=8, d=128, rot=128, axes=1, far=131072,
             interleaved=False),
        # a prompt with pictures: positions of time, height and width, heads of 128
        dict(name="norm_prompt_8192_3axes", op="norm", dtype="bf16", tokens=8192, hq=32, hkv=8, d=128, rot=128, axes=3,
             far=8192, interleaved=False),
        # gradients of a training batch of 2 x 8192 tokens
        dict(name="norm_bwd_16384", op="norm_bwd", dtype="bf16", tokens=16384, hq=32, hkv=8, d=128, rot=128, axes=1,
             far=8192, interleaved=False),
        # gradients of a short odd batch, heads of 64 of which half is rotated, two axes, neighbouring pairs
        dict(name="norm_bwd_1537_d64", op="norm_bwd", dtype="fp16", tokens=1537, hq=16, hkv=16, d=64, rot=32, axes=2,
             far=64, interleaved=True),
        # a decoding step's append: one token per sequence behind caches of up to 4096 tokens
        dict(name="append_decode_b32", op="append", dtype="bf16", B=32, hq=32, hkv=8, d=128, page=16, q_lo=1, q_hi=1,
             k_lo=2048, k_hi=4096, rot=128, interleaved=False, lens=1),
        # a prompt chunk's append: ragged chunks of several requests
        dict(name="append_chunks_b8", op="append", dtype="bf16", B=8, hq=32, hkv=8, d=128, page=32, q_lo=200,
             q_hi=2048, k_lo=2048, k_hi=8192, rot=128, interleaved=False, lens=2),
        # one short cache read back, heads of 64
        dict(name="read_b1_777_d64", op="read", dtype="fp16", B=1, hkv=5, d=64, page=16, k_lo=777, k_hi=777, lens=3),
        # what the cache holds of several requests, read back for the next chunks of their prompts
        dict(name="read_b8_16384", op="read", dtype="bf16", B=8, hkv=8, d=128, page=64, k_lo=6000, k_hi=16384, lens=4),
        # a decoding step of a batch, ragged caches, small pages
        dict(name="decode_b32_4096", op="decode", dtype="bf16", B=32, hq=32, hkv=8, d=128, page=16, q_lo=1, q_hi=1,
             k_lo=3000, k_hi=4097, lens=5),
        # a decoding step of one long request
        dict(name="decode_b1_131072", op="decode", dtype="fp16", B=1, hq=32, hkv=8, d=128, page=64, q_lo=1, q_hi=1,
             k_lo=131072, k_hi=131072, lens=6),
        # small trees of drafted tokens, one size per request, heads of 64
        dict(name="tree_b16_t12_d64", op="tree", dtype="bf16", B=16, hq=16, hkv=4, d=64, page=32, q_lo=3, q_hi=12,
             k_lo=1000, k_hi=8192, lens=7),
        # trees of 64 drafted tokens over long contexts
        dict(name="tree_b8_t64_16384", op="tree", dtype="bf16", B=8, hq=32, hkv=8, d=128, page=64, q_lo=64, q_hi=64,
             k_lo=9000, k_hi=16384, lens=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "append", "read", "decode", "decode", "tree", "tree"))
    d = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 4, 5, 8))
    group = rng.choice((1, 2, 3, 4, 6, 8))
    c = dict(op=op, dtype=rng.choice(("bf16", "fp16")), d=d, hkv=hkv)
    if op in ("norm", "norm_bwd"):
        c.update(tokens=_log(rng, 1, 16384), hq=min(32, hkv * group), rot=rng.choice((d, d // 2)), axes=rng.choice((1, 2, 3, 4)),
                 far=_log(rng, 64, 1 << 20), interleaved=rng.random() < 0.5)
        return c
    c.update(B=_log(rng, 1, 32), page=rng.choice((16, 32, 64, 128)), lens=rng.randrange(1 << 20))
    if op == "read":
        hi = _log(rng, 16, 131072 // c["B"])
        c.update(k_lo=max(1, int(hi * rng.uniform(0.1, 1.0))), k_hi=hi)
        return c
    c["hq"] = hkv * group
    if op == "append":
        q_hi = _log(rng, 1, max(1, 8192 // c["B"]))
        c.update(q_lo=max(1, q_hi // 3), q_hi=q_hi, k_lo=q_hi, k_hi=max(q_hi, _log(rng, 32, 8192)), rot=rng.choice((d, d // 2)),
                 interleaved=rng.random() < 0.5)
        return c
    hi = _log(rng, 64, 131072 // c["B"])
    q_hi = 1 if op == "decode" else _log(rng, 2, 64)
    # queries x keys x heads bounded by the largest listed tree
    hi = max(64, min(hi, 8 * 64 * 32 * 16384 // (c["B"] * q_hi * c["hq"])))
    c.update(q_lo=1 if op == "decode" else max(1, int(q_hi * rng.uniform(0.2, 1.0))), q_hi=q_hi,
             k_lo=max(q_hi, int(hi * rng.uniform(0.1, 1.0))), k_hi=hi)
    return c


def _lengths(c):
    """(queries, keys) of each sequence: the case's own, the same for every seed."""
    r = random.Random(c["lens"])
    k = [r.randint(c["k_lo"], c["k_hi"]) for _ in range(c["B"])]
    k[0] = c["k_hi"]
    q = [min(n, r.randint(c["q_lo"], c["q_hi"])) for n in k] if "q_lo" in c else list(k)
    return q, k


def _axes(c):
    """The axis of each pair: equal runs of pairs, the last the longest; with one axis, none is given."""
    pairs = c["rot"] // 2
    return [min(p // (pairs // c["axes"]), c["axes"] - 1) for p in range(pairs)]


def _cu(lens, dev):
    t = [0]
    for n in lens:
        t.append(t[-1] + n)
    return torch.tensor(t, dtype=torch.int32, device=dev)


def _pool(c, k, g, dev):
    """Pages of the sequences, scattered over a pool, as a server's allocator leaves them; unused table entries are -1."""
    need = [-(-n // c["page"]) for n in k]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((c["B"], max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _trees(lens, seed):
    """Ancestors of each drafted token, itself among them, as bits: tree after tree, parents drawn from the seed."""
    r, rows = random.Random(seed), []
    for n in lens:
        mask = []
        for i in range(n):
            up = r.randrange(-1, i) if i else -1
            mask.append((mask[up] if up >= 0 else 0) | 1 << i)
        rows += mask
    return [m - (1 << 64) if m >> 63 else m for m in rows]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    c, dt = case, DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    s = dict(c=c)
    if "rot" in c:
        s["freqs"] = 10000.0 ** (-2.0 * torch.arange(c["rot"] // 2, dtype=torch.float64) / c["rot"])
        s["freqs_dev"] = s["freqs"].to(dev)
    if c["op"] in ("norm", "norm_bwd"):
        n, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
        # the slices of one fused projection's output
        qkv = (normal(n, hq + 2 * hkv, d) * 1.5).to(dt)
        s["q"], s["k"], _ = qkv.split((hq, hkv, hkv), dim=1)
        s["wq"], s["wk"] = (1.0 + 0.2 * normal(d)).to(dt), (1.0 + 0.2 * normal(d)).to(dt)
        s["positions"] = torch.randint(0, c["far"], (c["axes"], n), generator=g, device=dev, dtype=torch.int32)
        s["axes"] = _axes(c) if c["axes"] > 1 else None
        s["axes_dev"] = torch.tensor(_axes(c), device=dev)
        if c["op"] == "norm_bwd":
            s["dq"], s["dk"] = normal(n, hq, d).to(dt), normal(n, hkv, d).to(dt)
        return s
    q_len, k_len = _lengths(c)
    s["seqlens"] = torch.tensor(k_len, dtype=torch.int32, device=dev)
    s["max_q"], s["max_k"] = max(q_len), max(k_len)
    s["cu"] = _cu(q_len, dev)
    s["total"] = sum(q_len)
    s["table"], n_pages = _pool(c, k_len, g, dev)
    for name in ("k", "v"):
        s[name + "_pages"], s[name + "_scales"] = _quantised(normal(n_pages, c["page"], c["hkv"], c["d"]))
    if c["op"] == "append":
        qkv = normal(s["total"], c["hq"] + 2 * c["hkv"], c["d"]).to(dt)
        s["q"], s["k"], s["v"] = qkv.split((c["hq"], c["hkv"], c["hkv"]), dim=1)
    elif c["op"] != "read":
        s["q"] = normal(s["total"], c["hq"], c["d"]).to(dt)
        if c["op"] == "tree":
            s["mask"] = torch.tensor(_trees(q_len, seed), dtype=torch.int64, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _quantised(x):
    """e4m3 values and one scale for each row of features, of x in 32 bits."""
    scale = (x.abs().amax(-1) / TOP).clamp(min=LEAST)
    return (x / scale[..., None]).clamp(-TOP, TOP).to(E4M3), scale


def _pairs(x, rot, interleaved):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def _turn(x, cos, sin, rot, interleaved):
    """x in 32 bits with its pairs turned; cos and sin (tokens, rot / 2)."""
    cos, sin = cos[:, None, :], sin[:, None, :]
    x1, x2 = _pairs(x, rot, interleaved)
    y1, y2 = x1 * cos - x2 * sin, x1 * sin + x2 * cos
    turned = torch.stack((y1, y2), dim=-1).flatten(-2) if interleaved else torch.cat((y1, y2), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _angles(s):
    """cos and sin in 32 bits, (tokens, rot / 2), of the positions that the pairs' axes give."""
    angle = s["positions"][s["axes_dev"]].double().t() * s["freqs_dev"]
    return angle.cos().float(), angle.sin().float()


def _norm(s):
    c = s["c"]
    cos, sin = _angles(s)

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        return _turn(y, cos, sin, c["rot"], c["interleaved"]).to(w.dtype)

    return dict(q=one(s["q"], s["wq"]), k=one(s["k"], s["wk"]))


def _norm_bwd(s):
    c = s["c"]
    cos, sin = _angles(s)

    def one(dy, x, w):
        x = x.float()
        g = _turn(dy.float(), cos, -sin, c["rot"], c["interleaved"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        z = x * r
        gw = g * w.float()
        dx = r * (gw - z * (gw * z).mean(-1, keepdim=True))
        return dx.to(w.dtype), (g * z).sum(1).double().sum(0).to(w.dtype)

    dq, dwq = one(s["dq"], s["q"], s["wq"])
    dk, dwk = one(s["dk"], s["k"], s["wk"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _rows_of(cu, total):
    """(sequence, index in it) of each packed row."""
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return b, t - cu[b].long()


def _append(s):
    c = s["c"]
    b, i = _rows_of(s["cu"], s["total"])
    key = i + s["seqlens"][b].long() - (s["cu"][b + 1] - s["cu"][b]).long()
    angle = key.double()[:, None] * s["freqs_dev"]
    cos, sin = angle.cos().float(), angle.sin().float()
    page, slot = s["table"][b, key // c["page"]].long(), key % c["page"]
    k8, ks = _quantised(_turn(s["k"].float(), cos, sin, c["rot"], c["interleaved"]))
    v8, vs = _quantised(s["v"].float())
    # (bytes: 8-bit types have no indexed assignment of their own)
    s["k_pages"].view(torch.uint8)[page, slot] = k8.view(torch.uint8)
    s["v_pages"].view(torch.uint8)[page, slot] = v8.view(torch.uint8)
    s["k_scales"][page, slot] = ks
    s["v_scales"][page, slot] = vs
    q = _turn(s["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    return dict(q=q, **{n: s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales")})


def _read(s):
    c, dt = s["c"], DT[s["c"]["dtype"]]
    b, j = _rows_of(s["cu"], s["total"])
    page, slot = s["table"][b, j // c["page"]].long(), j % c["page"]

    def one(name):
        values = s[name + "_pages"].view(torch.uint8)[page, slot].view(E4M3).float()
        return (values * s[name + "_scales"][page, slot][..., None]).to(dt)

    return dict(k=one("k"), v=one("v"))


def _gathered(s, name):
    """Keys or values of every sequence, (B, max_k, Hkv, d), in 32 bits."""
    t = s["table"].clamp(min=0).long()
    values = s[name + "_pages"].view(torch.uint8)[t].view(E4M3).float() * s[name + "_scales"][t][..., None]
    return values.flatten(1, 2)[:, :s["max_k"]]


def _tree(s):
    c, cu, n = s["c"], s["cu"].long(), s["seqlens"].long()
    dev, B, hkv, total = cu.device, c["B"], c["hkv"], s["total"]
    group = c["hq"] // hkv
    i = torch.arange(s["max_q"], device=dev)
    j = torch.arange(s["max_k"], device=dev)
    q_len = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp(max=total - 1)
    q = s["q"][row].float().view(B, -1, hkv, group, c["d"]).permute(0, 2, 3, 1, 4)
    scores = q.reshape(B, hkv, -1, c["d"]) @ _gathered(s, "k").permute(0, 2, 3, 1)
    scores = scores.view(B, hkv, group, s["max_q"], s["max_k"])
    scores *= 1.0 / math.sqrt(c["d"])
    # the key's place among the drafted tokens; before them lies the context, which every token sees
    place = j - (n - q_len)[:, None]                                       # (B, max_k)
    bits = s["mask"][row] if "mask" in s else torch.ones_like(row)         # (B, max_q)
    in_tree = (bits[:, :, None] >> place.clamp(0, 63)[:, None]) & 1 == 1
    seen = torch.where(place[:, None] < 0, torch.ones_like(in_tree), in_tree) & (j < n[:, None])[:, None]
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    b, at = _rows_of(s["cu"], total)
    lse = (l.log() + top)[..., 0].flatten(1, 2).permute(0, 2, 1)[b, at].t().contiguous()
    o = (p.flatten(2, 3) @ _gathered(s, "v").permute(0, 2, 1, 3)).view(*p.shape[:-1], c["d"]) / l.clamp(min=1e-38)
    return dict(o=o.flatten(1, 2).permute(0, 2, 1, 3)[b, at].to(s["q"].dtype), lse=lse)


def run(state):
    s = state
    c = s["c"]
    if own:
        from tiled_attention_attn_gb300 import attn
        if c["op"] == "norm":
            q, k = attn.qk_norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["freqs"], s["positions"], axes=s["axes"],
                                       eps=1e-6, interleaved=c["interleaved"])
            return dict(q=q, k=k)
        if c["op"] == "norm_bwd":
            dq, dk, dwq, dwk = attn.qk_norm_rotary_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["freqs"],
                                                       s["positions"], axes=s["axes"], eps=1e-6,
                                                       interleaved=c["interleaved"])
            return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
        cache = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"], s["seqlens"])
        if c["op"] == "append":
            q = attn.cache_append_fp8(s["k"], s["v"], *cache, s["cu"], q=s["q"], freqs=s["freqs"],
                                      interleaved=c["interleaved"])
            return dict(q=q, **{n: s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales")})
        if c["op"] == "read":
            k, v = attn.cache_read_fp8(*cache, s["cu"], s["total"], DT[c["dtype"]])
            return dict(k=k, v=v)
        if c["op"] == "decode":
            o, lse = attn.attn_decode_fp8(s["q"], *cache)
        else:
            o, lse = attn.attn_tree_fp8(s["q"], *cache, s["cu"], tree_mask=s["mask"], max_tokens=s["max_q"])
        return dict(o=o, lse=lse)
    return dict(norm=_norm, norm_bwd=_norm_bwd, append=_append, read=_read, decode=_tree, tree=_tree)[c["op"]](s)


def work(case):
    c = case
    if c["op"] in ("norm", "norm_bwd"):
        n = c["tokens"] * (c["hq"] + c["hkv"]) * c["d"]
        if c["op"] == "norm":
            return dict(bytes=4 * n + c["tokens"] * c["axes"] * 4 + 4 * c["d"], flops=7 * n)
        return dict(bytes=6 * n + c["tokens"] * c["axes"] * 4 + 8 * c["d"], flops=13 * n)
    q, k = _lengths(c)
    row = c["hkv"] * (c["d"] + 4)                                  # one token's keys (or values) with their scales
    if c["op"] == "read":
        return dict(bytes=sum(k) * 2 * (row + c["hkv"] * c["d"] * 2), flops=sum(k) * 2 * c["hkv"] * c["d"])
    new = sum(q)
    if c["op"] == "append":
        return dict(bytes=new * (c["hq"] * c["d"] * 4 + 2 * c["hkv"] * c["d"] * 2 + 2 * row),
                    flops=new * ((c["hq"] + c["hkv"]) * c["rot"] * 3 + 4 * c["hkv"] * c["d"]))
    pairs = sum(a * b for a, b in zip(q, k)) * c["hq"]
    masks = new * 8 if c["op"] == "tree" else 0
    return dict(bytes=new * c["hq"] * (c["d"] * 4 + 4) + sum(k) * 2 * row + masks, flops=4 * pairs * c["d"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _turned64(x, angle, c, sign=1.0):
    """x (tokens, heads, d) with pair p of token t turned by sign * angle[t, p], as complex numbers."""
    z = x.double().clone()
    half = c["rot"] // 2
    p = torch.arange(half, device=x.device)
    first, second = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + half)
    e = torch.polar(torch.ones_like(angle), sign * angle)[:, None, :]
    w = torch.complex(z[..., first], z[..., second]) * e
    z[..., first], z[..., second] = w.real, w.imag
    return z


def _rounded64(x):
    """e4m3 values (as float64) and scales of x's rows: the nearest multiple of the value's step, ties to even."""
    scale = (x.abs().amax(-1) / TOP).clamp(min=LEAST)
    y = (x / scale[..., None]).clamp(-TOP, TOP)
    _, e = torch.frexp(y)                                          # |y| = m 2^e, m in [1/2, 1)
    step = torch.ldexp(torch.ones_like(y), (e - 4).clamp(min=-9))  # 3 bits behind the leading one; 2^-9 at the least
    return torch.round(y / step) * step, scale


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] in ("norm", "norm_bwd"):
        pos = torch.stack([s["positions"][a] for a in _axes(c)], 1).double()
        angle = pos * s["freqs"].to(pos.device)
        out = {}
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            x, w = s[name].double(), w.double()
            size = ((x ** 2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt()
            if c["op"] == "norm":
                out[name] = _turned64(x / size * w, angle, c)
                continue
            g = _turned64(s["d" + name], angle, c, -1.0)
            # y = w x / size: the direct term, and what x changes in size (d size / d x = x / (d size))
            out["d" + name] = g * w / size - x * (g * w * x).sum(-1, keepdim=True) / (c["d"] * size ** 3)
            out["dw" + name] = (g * x / size).sum((0, 1))
        return out
    q_len, k_len = _lengths(c)
    dev, P = s["table"].device, c["page"]
    if c["op"] == "append":
        pages = {n: s[n + "_pages"].double() for n in ("k", "v")}
        scales = {n: s[n + "_scales"].double() for n in ("k", "v")}
        qs, at = [], 0
        for b, (m, n) in enumerate(zip(q_len, k_len)):
            pos = torch.arange(n - m, n, device=dev)
            page, slot = s["table"][b, pos // P].long(), pos % P
            angle = torch.outer(pos.double(), s["freqs"].to(dev))
            qs.append(_turned64(s["q"][at:at + m], angle, c))
            for name, x in (("k", _turned64(s["k"][at:at + m], angle, c)), ("v", s["v"][at:at + m].double())):
                pages[name][page, slot], scales[name][page, slot] = _rounded64(x)
            at += m
        return dict(q=torch.cat(qs), k_pages=pages["k"], v_pages=pages["v"], k_scales=scales["k"], v_scales=scales["v"])

    def history(name, b, n):
        t = s["table"][b, : -(-n // P)].long()
        values = s[name + "_pages"].view(torch.uint8)[t].view(E4M3).double() * s[name + "_scales"][t].double()[..., None]
        return values.reshape(-1, c["hkv"], c["d"])[:n]

    if c["op"] == "read":
        return {name: torch.cat([history(name, b, n) for b, n in enumerate(k_len)]) for name in ("k", "v")}
    group, at, outs, lses = c["hq"] // c["hkv"], 0, [], []
    for b, (m, n) in enumerate(zip(q_len, k_len)):
        kk, vv = history("k", b, n), history("v", b, n)
        seen = torch.ones(m, n, dtype=torch.bool, device=dev)
        if c["op"] == "tree":
            for i, word in enumerate(s["mask"][at:at + m].tolist()):
                seen[i, n - m:] = torch.tensor([bool(word >> t & 1) for t in range(m)], device=dev)
        o, l = [], []
        for h in range(c["hq"]):
            x = s["q"][at:at + m, h].double() @ kk[:, h // group].t() / math.sqrt(c["d"])
            x = x.masked_fill(~seen, float("-inf"))
            l.append(x.logsumexp(-1))
            o.append((x - l[-1][:, None]).exp() @ vv[:, h // group])
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(l))
        at += m
    return dict(o=torch.cat(outs), lse=torch.cat(lses, 1))
