"""Cases of the paged-cache operators: scaled rotary embedding and its gradient,
the append of new tokens to the pages, attention of a chunk or of single tokens
over the pages, the accumulated attention weight of each cached key, and
eviction by that weight.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, angles in 64), or, where ``own`` is set, through the package's entry
points.  ``exact`` gives the definition in 64 bits.
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # rotary of the new queries of a decoding step: 32 sequences, one token each, far positions
        dict(name="rotary_decode_b32", op="rotary", dtype="bf16", tokens=32, heads=32, d=128, rot=128, interleaved=False,
             inverse=False, scaling="yarn", factor=32.0, original=4096, far=131072),
        # gradient of the rotary embedding of a training batch's queries, rotary on half of the head
        dict(name="rotary_bwd_b2_l8192", op="rotary", dtype="fp16", tokens=16384, heads=32, d=128, rot=64,
             interleaved=True, inverse=True, scaling="ntk", factor=8.0, original=4096, far=32768),
        # a decoding step's append: one token per sequence behind caches of up to 4096 tokens
        dict(name="append_decode_b32", op="append", dtype="bf16", B=32, hq=32, hkv=8, d=128, page=16, q_lo=1, q_hi=1,
             k_lo=2048, k_hi=4096, rot=128, interleaved=False, scaling="linear", factor=4.0, original=4096, lens=1),
        # a prompt chunk's append: ragged chunks of several requests
        dict(name="append_chunks_b8", op="append", dtype="bf16", B=8, hq=32, hkv=8, d=128, page=32, q_lo=200,
             q_hi=2048, k_lo=2048, k_hi=8192, rot=128, interleaved=False, scaling="yarn", factor=8.0, original=4096,
             lens=2),
        # a mixed batch: decoding requests (one token) beside prompt chunks
        dict(name="chunk_ragged_b8", op="chunk", dtype="fp16", B=8, hq=16, hkv=4, d=128, page=32, q_lo=1, q_hi=512,
             k_lo=600, k_hi=8192, lens=3),
        # one long prompt's next chunk over what the cache holds of it
        dict(name="chunk_2048_over_16384", op="chunk", dtype="bf16", B=1, hq=32, hkv=8, d=128, page=64, q_lo=2048,
             q_hi=2048, k_lo=16384, k_hi=16384, lens=4),
        # a decoding step of a batch, ragged caches, small pages
        dict(name="decode_b32_4096", op="decode", dtype="bf16", B=32, hq=32, hkv=8, d=128, page=16, q_lo=1, q_hi=1,
             k_lo=3000, k_hi=4097, lens=5),
        # a decoding step of one long request
        dict(name="decode_b1_131072", op="decode", dtype="bf16", B=1, hq=32, hkv=8, d=128, page=64, q_lo=1, q_hi=1,
             k_lo=131072, k_hi=131072, lens=6),
        # the weights a decoding step adds, as eviction policies accumulate them
        dict(name="weights_decode_b32", op="weights", dtype="bf16", B=32, hq=32, hkv=8, d=128, page=16, q_lo=1, q_hi=1,
             k_lo=3000, k_hi=4097, decay=1.0, lens=7),
        # the weights of a whole prompt's queries over its own keys, head_dim 64
        dict(name="weights_prompt_4096", op="weights", dtype="fp16", B=2, hq=16, hkv=16, d=64, page=32, q_lo=3500,
             q_hi=4096, k_lo=4096, k_hi=4096, decay=0.5, lens=8),
        # a batch cut back to its budget between decoding steps
        dict(name="evict_b32_4096", op="evict", dtype="bf16", B=32, hkv=8, d=128, page=16, k_lo=1500, k_hi=4096,
             budget=2048, recent=256, lens=9),
        # one long prompt cut to a small cache
        dict(name="evict_b1_131072", op="evict", dtype="bf16", B=1, hkv=8, d=128, page=64, k_lo=131072, k_hi=131072,
             budget=8192, recent=1024, lens=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "append", "chunk", "chunk", "decode", "decode", "weights", "weights", "evict"))
    c = dict(op=op, dtype=rng.choice(("bf16", "fp16")))
    d = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 4, 5, 8))
    group = rng.choice((1, 2, 3, 4, 6, 8))
    scale = dict(interleaved=rng.random() < 0.5, scaling=rng.choice(("none", "linear", "ntk", "yarn")),
                 factor=rng.choice((2.0, 4.0, 8.0, 32.0)), original=rng.choice((2048, 4096, 8192)))
    c["lens"] = rng.randrange(1 << 20)
    if op == "rotary":
        c.update(tokens=_log(rng, 1, 16384), heads=rng.choice((1, 3, 8, 16, 32)), d=d, rot=rng.choice((d, d // 2, d - 16)),
                 inverse=rng.random() < 0.5, far=_log(rng, 1024, 1 << 20), **scale)
        return c
    c.update(B=_log(rng, 1, 32), hkv=hkv, d=d, page=rng.choice((16, 32, 64, 128)))
    if op == "evict":
        hi = _log(rng, 64, min(131072, 131072 // c["B"]))
        budget = max(2, int(hi * rng.uniform(0.1, 0.9)))
        c.update(k_lo=max(1, int(hi * rng.uniform(0.2, 1.0))), k_hi=hi, budget=budget,
                 recent=rng.choice((0, 1, budget // 8, budget // 2)))
        return c
    c["hq"] = hkv * group
    if op == "append":
        q_hi = _log(rng, 1, max(1, 8192 // c["B"]))
        c.update(q_lo=max(1, q_hi // 3), q_hi=q_hi, k_lo=q_hi, k_hi=max(q_hi, _log(rng, 32, 8192)), rot=d, **scale)
        return c
    if op == "decode":
        hi = _log(rng, 16, 131072 // c["B"])
        c.update(q_lo=1, q_hi=1, k_lo=max(1, int(hi * rng.uniform(0.1, 1.0))), k_hi=hi)
        return c
    # chunk, weights: queries x keys x heads bounded by the largest listed chunk
    k_hi = _log(rng, 16, 16384)
    most = max(1, min(k_hi, 2048 * 16384 * 32 // (k_hi * c["B"] * c["hq"])))
    q_hi = _log(rng, 1, min(4096, most))
    c.update(q_lo=max(1, q_hi // 4), q_hi=q_hi, k_lo=max(q_hi, int(k_hi * rng.uniform(0.3, 1.0))), k_hi=k_hi)
    if op == "weights":
        c["decay"] = rng.choice((0.0, 0.5, 1.0))
    return c


def _lengths(c):
    """(queries, keys) of each sequence: the case's own, the same for every seed."""
    r = random.Random(c["lens"])
    k = [r.randint(c["k_lo"], c["k_hi"]) for _ in range(c["B"])]
    k[0] = c["k_hi"]
    q = [min(n, r.randint(c["q_lo"], c["q_hi"])) for n in k] if "q_lo" in c else [0] * c["B"]
    return q, k


def _frequencies(c):
    """Radians per position of each pair, and the amplitude, in 64 bits: the base 10000 spectrum f_i = base^(-2i/rot),
    scaled for contexts longer than `original` by `factor`."""
    rot, base, s = c["rot"], 10000.0, c["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        return f / s, 1.0
    if c["scaling"] == "ntk":
        return (base * s ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    if c["scaling"] == "yarn":
        # pairs that turn more than 32 times within the original context keep f, those below one turn take f / s
        lo = max(math.floor(rot * math.log(c["original"] / (32.0 * 2 * math.pi)) / (2 * math.log(base))), 0)
        hi = min(math.ceil(rot * math.log(c["original"] / (1.0 * 2 * math.pi)) / (2 * math.log(base))), rot // 2 - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f * (1.0 - ramp) + f / s * ramp, 0.1 * math.log(s) + 1.0
    return f, 1.0


def _cu(lens, dev):
    t = [0]
    for n in lens:
        t.append(t[-1] + n)
    return torch.tensor(t, dtype=torch.int32, device=dev)


def _pool(c, k, g, dev, extra=0):
    """Pages of the sequences, scattered over a pool, as a server's allocator leaves them; unused table entries are -1."""
    need = [-(-n // c["page"]) for n in k]
    total = sum(need) + extra + 3
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((c["B"], max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:], total


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    c, dt = case, DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    s = dict(c=c)
    if c["op"] == "rotary":
        s["x"] = normal(c["tokens"], c["heads"], c["d"])
        s["positions"] = torch.randint(0, c["far"], (c["tokens"],), generator=g, device=dev, dtype=torch.int32)
        s["freqs"], s["amplitude"] = _frequencies(c)
        s["freqs_dev"] = s["freqs"].to(dev)
        return s
    q_len, k_len = _lengths(c)
    s["seqlens"] = torch.tensor(k_len, dtype=torch.int32, device=dev)
    s["max_q"], s["max_k"] = max(q_len), max(k_len)
    if c["op"] == "evict":
        kept = [min(n, c["budget"]) for n in k_len]
        need = sum(-(-n // c["page"]) for n in kept)
        s["table"], free, n_pages = _pool(c, k_len, g, dev, extra=need)
        s["dst"] = torch.full((c["B"], max(-(-n // c["page"]) for n in kept)), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(kept):
            m = -(-n // c["page"])
            s["dst"][b, :m] = free[at:at + m]
            at += m
        s["k_pages"] = normal(n_pages, c["page"], c["hkv"], c["d"])
        s["v_pages"] = normal(n_pages, c["page"], c["hkv"], c["d"])
        # heavy-tailed sums of softmax weights, a share of them equal (keys that no query has looked at: 0)
        w = torch.rand(c["B"], c["hkv"], s["table"].shape[1] * c["page"], generator=g, device=dev) ** 6
        w = torch.where(w < 0.05, (w * 200).floor() / 200, w * 8)
        s["weights"] = w.contiguous()
        return s
    s["cu"] = _cu(q_len, dev)
    total = sum(q_len)
    s["table"], _, n_pages = _pool(c, k_len, g, dev)
    shape = (n_pages, c["page"], c["hkv"], c["d"])
    s["k_pages"], s["v_pages"] = normal(*shape), normal(*shape)
    if c["op"] == "append":
        # the slices of one fused projection's output
        qkv = normal(total, c["hq"] + 2 * c["hkv"], c["d"])
        s["q"], s["k"], s["v"] = qkv.split((c["hq"], c["hkv"], c["hkv"]), dim=1)
        s["freqs"], s["amplitude"] = _frequencies(c)
        s["freqs_dev"] = s["freqs"].to(dev)
        return s
    s["q"] = normal(total, c["hq"], c["d"])
    if c["op"] == "weights":
        # what the forward of these queries returned
        s["lse"] = _attention(s, want_o=False)[1]
        s["weights"] = torch.rand(c["B"], c["hkv"], s["table"].shape[1] * c["page"], generator=g, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rotate(x, positions, freqs, amplitude, rot, interleaved, inverse):
    angle = positions.double()[:, None] * freqs[None, :]
    cos = (angle.cos() * amplitude).float()[:, None, :]
    sin = (angle.sin() * (-amplitude if inverse else amplitude)).float()[:, None, :]
    y = x.float()
    if interleaved:
        x1, x2 = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((x1 * cos - x2 * sin, x1 * sin + x2 * cos), dim=-1).flatten(-2)
    else:
        x1, x2 = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((x1 * cos - x2 * sin, x1 * sin + x2 * cos), dim=-1)
    return torch.cat((turned, y[..., rot:]), dim=-1).to(x.dtype)


def _rows_of(cu, seqlens, total):
    """(sequence, key index) of each packed new token: the last tokens of its sequence."""
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return b, t - cu[b].long() + seqlens[b].long() - (cu[b + 1] - cu[b]).long()


def _gathered(pages, table, max_k):
    return pages[table.clamp(min=0).long()].flatten(1, 2)[:, :max_k].float()


def _padded(s):
    """Scaled scores (B, Hkv, G, max_q, max_k) in 32 bits, -inf where masked, and the packed row of each padded query."""
    c, cu, n = s["c"], s["cu"].long(), s["seqlens"].long()
    dev, B, hkv = cu.device, c["B"], c["hkv"]
    group = c["hq"] // hkv
    i = torch.arange(s["max_q"], device=dev)
    j = torch.arange(s["max_k"], device=dev)
    q_len = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, -1, hkv, group, c["d"]).permute(0, 2, 3, 1, 4)
    k = _gathered(s["k_pages"], s["table"], s["max_k"]).permute(0, 2, 3, 1)
    scores = (q.reshape(B, hkv, -1, c["d"]) @ k).view(B, hkv, group, s["max_q"], s["max_k"])
    scores *= 1.0 / math.sqrt(c["d"])
    seen = (j <= i[:, None] + (n - q_len)[:, None, None]) & (i[:, None] < q_len[:, None, None])
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    b, _ = _rows_of(s["cu"], s["seqlens"], s["q"].shape[0])
    return scores, b, torch.arange(s["q"].shape[0], device=dev) - cu[b]


def _attention(s, want_o=True):
    c = s["c"]
    scores, b, i = _padded(s)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top)[..., 0]                            # (B, Hkv, G, max_q)
    lse = lse.flatten(1, 2).permute(0, 2, 1)[b, i].t().contiguous()
    if not want_o:
        return None, lse
    v = _gathered(s["v_pages"], s["table"], s["max_k"]).permute(0, 2, 1, 3)
    o = (p.flatten(2, 3) @ v).view(*p.shape[:-1], c["d"]) / total.clamp(min=1e-38)
    o = o.flatten(1, 2).permute(0, 2, 1, 3)[b, i]
    return o.to(s["q"].dtype), lse


def _key_weights(s):
    c = s["c"]
    scores, _, _ = _padded(s)
    i = torch.arange(s["max_q"], device=scores.device)
    row = (s["cu"][:-1, None].long() + i).clamp(max=s["q"].shape[0] - 1)
    lse = s["lse"][:, row].view(c["hkv"], -1, c["B"], s["max_q"]).permute(2, 0, 1, 3)
    added = scores.sub_(lse[..., None]).exp_().sum((2, 3))        # (B, Hkv, max_k)
    w = s["weights"][..., :s["max_k"]]
    live = (torch.arange(s["max_k"], device=w.device) < s["seqlens"][:, None])[:, None]
    old = w * c["decay"] if c["decay"] else torch.zeros_like(w)
    w.copy_(torch.where(live, old + added, w))
    return s["weights"]


def _evict(s):
    c, n = s["c"], s["seqlens"].long()
    dev, B, hkv, P, budget = n.device, c["B"], c["hkv"], c["page"], c["budget"]
    w = s["weights"][..., :s["max_k"]]
    j = torch.arange(s["max_k"], device=dev)
    live, old = j < n[:, None], j < (n - c["recent"])[:, None]
    # the recent keys rank first, then by weight, the lower index first among equals; what is past the end last
    key = torch.where((live & ~old)[:, None], torch.full_like(w, float("inf")), w)
    key = torch.where(live[:, None], key, torch.full_like(w, float("-inf")))
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    new_len = n.clamp(max=budget)
    slot = torch.arange(order.shape[-1], device=dev)
    rank = torch.where(slot < new_len[:, None, None], order, torch.full_like(order, s["max_k"]))
    kept = rank.sort(dim=-1).values                              # back in the order of the cache
    valid = (slot < new_len[:, None, None]).expand_as(kept)
    b = torch.arange(B, device=dev)[:, None, None].expand_as(kept)[valid]
    h = torch.arange(hkv, device=dev)[:, None].expand_as(kept)[valid]
    src, dst = kept[valid], slot.expand_as(kept)[valid]
    moved = s["weights"][b, h, src]
    out = {}
    for name in ("k_pages", "v_pages"):
        pages = s[name]
        rows = pages[s["table"][b, src // P].long(), src % P, h]
        pages[s["dst"][b, dst // P].long(), dst % P, h] = rows
        out[name] = pages
    weights = torch.zeros(B, hkv, budget, device=dev)
    weights[b, h, dst] = moved
    full = torch.full((B, hkv, budget), -1, dtype=torch.int32, device=dev)
    full[..., :kept.shape[-1]] = torch.where(valid, kept, torch.full_like(kept, -1)).to(torch.int32)
    return dict(kept=full, seqlens=new_len.to(torch.int32), weights=weights, **out)


def run(state):
    s = state
    c = s["c"]
    if own:
        from tiled_attention_attn_gb300 import attn
        if c["op"] == "rotary":
            return dict(y=attn.rotary_scaled(s["x"], s["freqs"], s["amplitude"], interleaved=c["interleaved"],
                                             positions=s["positions"], inverse=c["inverse"]))
        if c["op"] == "append":
            q = attn.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"], s["cu"],
                                  q=s["q"], freqs=s["freqs"], amplitude=s["amplitude"], interleaved=c["interleaved"])
            return dict(q=q, k_pages=s["k_pages"], v_pages=s["v_pages"])
        if c["op"] == "chunk":
            o, lse = attn.attn_fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"], s["cu"], causal=True)
            return dict(o=o, lse=lse)
        if c["op"] == "decode":
            o, lse = attn.attn_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"])
            return dict(o=o, lse=lse)
        if c["op"] == "weights":
            return dict(weights=attn.key_weights(s["q"], s["k_pages"], s["lse"], s["table"], s["seqlens"], s["cu"],
                                                 causal=True, decay=c["decay"], weights=s["weights"]))
        kept, seqlens, weights = attn.cache_evict(s["weights"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"],
                                                  c["budget"], recent=c["recent"], dst_page_table=s["dst"])
        return dict(kept=kept, seqlens=seqlens, weights=weights, k_pages=s["k_pages"], v_pages=s["v_pages"])
    if c["op"] == "rotary":
        return dict(y=_rotate(s["x"], s["positions"], s["freqs_dev"], s["amplitude"], c["rot"], c["interleaved"],
                              c["inverse"]))
    if c["op"] == "append":
        b, key = _rows_of(s["cu"], s["seqlens"], s["k"].shape[0])
        turn = (key, s["freqs_dev"], s["amplitude"], c["rot"], c["interleaved"], False)
        page, slot = s["table"][b, key // c["page"]].long(), key % c["page"]
        s["k_pages"][page, slot] = _rotate(s["k"], *turn)
        s["v_pages"][page, slot] = s["v"]
        return dict(q=_rotate(s["q"], *turn), k_pages=s["k_pages"], v_pages=s["v_pages"])
    if c["op"] in ("chunk", "decode"):
        o, lse = _attention(s)
        return dict(o=o, lse=lse)
    if c["op"] == "weights":
        return dict(weights=_key_weights(s))
    return _evict(s)


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["tokens"] * c["heads"]
        return dict(bytes=n * c["d"] * 4 + c["tokens"] * 4, flops=n * c["rot"] * 3)
    q, k = _lengths(c)
    row = c["hkv"] * c["d"] * 2                                   # one token's keys (or values)
    if c["op"] == "evict":
        kept = sum(min(a, c["budget"]) for a in k)
        return dict(bytes=sum(k) * c["hkv"] * 4 + kept * (4 * row + 8 * c["hkv"]), flops=sum(k) * c["hkv"])
    new = sum(q)
    if c["op"] == "append":
        return dict(bytes=new * (c["hq"] * c["d"] * 4 + 4 * row), flops=new * (c["hq"] + c["hkv"]) * c["rot"] * 3)
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, k)) * c["hq"]
    io = new * c["hq"] * (c["d"] * 2 + 4)
    if c["op"] == "weights":
        return dict(bytes=io + sum(k) * (row + c["hkv"] * (8 if c["decay"] else 4)), flops=2 * pairs * c["d"])
    return dict(bytes=io + new * c["hq"] * c["d"] * 2 + sum(k) * 2 * row, flops=4 * pairs * c["d"])


# ---------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------

def _turned64(x, pos, c, freqs, amplitude, sign):
    z = x.double()
    half = c["rot"] // 2
    p = torch.arange(half, device=x.device)
    first, second = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + half)
    e = torch.polar(torch.full((pos.numel(), half), float(amplitude), dtype=torch.float64, device=x.device),
                    sign * torch.outer(pos.double(), freqs.to(x.device)))
    w = torch.complex(z[..., first], z[..., second]) * e[:, None, :]
    z[..., first], z[..., second] = w.real, w.imag
    return z


def _history(pages, table_row, n):
    return pages[table_row[: -(-n // pages.shape[1])].long()].reshape(-1, *pages.shape[2:])[:n]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rotary":
        return dict(y=_turned64(s["x"], s["positions"], c, s["freqs"], s["amplitude"], -1.0 if c["inverse"] else 1.0))
    q_len, k_len = _lengths(c)
    if c["op"] == "evict":
        kept = torch.full((c["B"], c["hkv"], c["budget"]), -1, dtype=torch.int32)
        weights = torch.zeros(c["B"], c["hkv"], c["budget"], dtype=torch.float64)
        w = s["weights"].cpu().double()
        for b, n in enumerate(k_len):
            m = min(n, c["budget"])
            tail = min(c["recent"], m)
            for h in range(c["hkv"]):
                if n <= c["budget"]:
                    keep = torch.arange(n)
                else:
                    rank = sorted(range(n - tail), key=lambda a, v=w[b, h].tolist(): (-v[a], a))[: m - tail]
                    keep = torch.tensor(sorted(rank) + list(range(n - tail, n)), dtype=torch.long)
                kept[b, h, :m] = keep.int()
                weights[b, h, :m] = w[b, h, keep]
        return dict(kept=kept, seqlens=torch.tensor([min(n, c["budget"]) for n in k_len], dtype=torch.int32),
                    weights=weights, k_pages=None, v_pages=None)
    at = 0
    if c["op"] == "append":
        kp, vp, qs = s["k_pages"].double(), s["v_pages"].double(), []
        for b, (m, n) in enumerate(zip(q_len, k_len)):
            pos = torch.arange(n - m, n, device=kp.device)
            page, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
            qs.append(_turned64(s["q"][at:at + m], pos, c, s["freqs"], s["amplitude"], 1.0))
            kp[page, slot] = _turned64(s["k"][at:at + m], pos, c, s["freqs"], s["amplitude"], 1.0)
            vp[page, slot] = s["v"][at:at + m].double()
            at += m
        return dict(q=torch.cat(qs), k_pages=kp, v_pages=vp)
    group = c["hq"] // c["hkv"]
    outs, lses = [], []
    weights = s["weights"].double() if c["op"] == "weights" else None
    for b, (m, n) in enumerate(zip(q_len, k_len)):
        kk = _history(s["k_pages"], s["table"][b], n)
        vv = _history(s["v_pages"], s["table"][b], n)
        hidden = torch.ones(m, n, dtype=torch.bool, device=kk.device).triu(n - m + 1)
        o, l = [], []
        for h in range(c["hq"]):
            x = s["q"][at:at + m, h].double() @ kk[:, h // group].double().t() / math.sqrt(c["d"])
            x = x.masked_fill(hidden, float("-inf"))
            if weights is not None:
                if h % group == 0:
                    weights[b, h // group, :n] *= c["decay"]
                weights[b, h // group, :n] += (x - s["lse"][h, at:at + m].double()[:, None]).exp().sum(0)
                continue
            l.append(x.logsumexp(-1))
            o.append((x - l[-1][:, None]).exp() @ vv[:, h // group].double())
        at += m
        if weights is None:
            outs.append(torch.stack(o, 1))
            lses.append(torch.stack(l))
    if weights is not None:
        return dict(weights=weights)
    return dict(o=torch.cat(outs), lse=torch.cat(lses, 1))
