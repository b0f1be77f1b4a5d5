"""Cases of the paged 8-bit cache's positions and scores: rotary positions, the append that rotates its keys on the way
into the pages, and attention over the pages with capped scores, distance biases, prefix and document masks.

Rotation: pair p of a row (channels p and pairs + p, or 2 p and 2 p + 1) turns by position[axis(p)] * frequency[p]; cos and
sin come from a table that a program makes once. The cache: E4M3 codes [1, n_pages, kv_heads, page, d], one power-of-two
scale per page and head, block tables. Scores of a row at position t and a key at j:
cap * tanh(q.k / sqrt(d) / cap) - slope[head] * |t - j|, over the keys that the masks leave.
"""
import math
import random

import torch

own = False

E_MIN, E_MAX = -60, 60


# ---------------------------------------------------------------- cases

def _attn(name, **kw):
    c = dict(name=name, op="attn", batch=1, q_heads=8, kv_heads=8, d=128, page=64, kv=1000, q=1, ragged=False, causal=True,
             window=0, softcap=0.0, alibi=False, prefix=False, docs=0, heat=1.0)
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of a small batch, queries and keys: nothing but latency
        dict(name="rope_decode", op="rope", layout="packed", batch=1, rows=64, q_heads=32, kv_heads=8, d=128, pairs=64,
             axes=1, interleaved=False, positions=131072, inverse=False),
        # one chunk of a video stream (3 x 30 x 52 tokens), time, height and width
        dict(name="rope_video_chunk", op="rope", layout="window", batch=1, rows=4680, q_heads=24, kv_heads=24, d=128,
             pairs=64, axes=3, interleaved=True, positions=1024, inverse=False),
        # one new token of every sequence of a serving batch, its queries beside it
        dict(name="append_decode", op="append", batch=128, q_heads=32, kv_heads=8, d=128, page=64, kv=2048, new=1,
             ragged=True, pairs=64, axes=1, interleaved=False, positions=16384),
        # a whole chunk of a video stream, all heads
        dict(name="append_video_chunk", op="append", batch=1, q_heads=24, kv_heads=24, d=128, page=64, kv=23400, new=4680,
             ragged=False, pairs=64, axes=3, interleaved=True, positions=1024),
        # prompts with images in them, half of each head rotated
        dict(name="append_prompts", op="append", batch=8, q_heads=32, kv_heads=4, d=128, page=32, kv=6000, new=2500,
             ragged=True, pairs=32, axes=3, interleaved=False, positions=8192),
        # one sequence just after its start, capped scores: latency again
        _attn("attn_cap_small", q_heads=24, kv_heads=24, page=16, kv=333, softcap=30.0, heat=4.0),
        # a serving batch of mixed lengths, a distance bias of each head
        _attn("attn_bias_ragged", batch=64, q_heads=32, kv_heads=8, kv=8192, ragged=True, alibi=True),
        # few sequences with a very long context, capped scores
        _attn("attn_cap_long", batch=4, q_heads=40, kv_heads=8, page=128, kv=100001, softcap=50.0),
        # several proposed tokens of each sequence, narrow heads, sliding window, documents in one sequence
        _attn("attn_verify_docs", batch=16, q_heads=32, kv_heads=4, d=64, page=32, kv=12000, q=5, ragged=True, window=4096,
              softcap=30.0, docs=3),
        # one chunk of a video stream over its window and itself, capped scores, no mask
        _attn("attn_cap_chunk_24h", q_heads=24, kv_heads=24, kv=23400, q=4680, causal=False, softcap=50.0),
        # prompts whose image or instruction in front sees itself whole, hot capped scores
        _attn("attn_prefix_ragged", batch=4, q_heads=32, kv_heads=8, page=32, kv=8192, q=2048, ragged=True, softcap=20.0,
              prefix=True, heat=6.0),
        # documents packed into one long row, a distance bias of each head
        _attn("attn_docs_bias", q_heads=32, kv_heads=8, page=128, kv=8000, q=8000, alibi=True, docs=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 12])
    op = rng.choice(["rope", "rope", "append", "append", "decode", "decode", "verify", "chunk"])
    axes, interleaved = rng.choice([1, 1, 2, 3]), rng.random() < 0.5
    pairs = rng.choice([d // 2, d // 2, d // 4, d // 2 - 8])
    positions = _log(rng, 600, 131072)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "rope":
        layout = rng.choice(["packed", "window"])
        batch = 1 if layout == "packed" else rng.randint(1, 3)
        heads = kv_heads * (group if layout == "packed" else 1)
        rows = _log(rng, 1, max(2, int(2.8e7 / ((heads + kv_heads) * d * batch))))
        return dict(op="rope", layout=layout, batch=batch, rows=rows, q_heads=heads, kv_heads=kv_heads, d=d, pairs=pairs,
                    axes=axes, interleaved=interleaved, positions=positions, inverse=rng.random() < 0.2)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        batch = _log(rng, 1, 200)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, max(2, int(1.4e7 / (batch * kv_heads * d))))
        group = min(group, max(1, int(2.8e7 / (batch * new * kv_heads * d))))
        kv = new + _log(rng, 1, 4000)
        return dict(op="append", batch=batch, q_heads=group * kv_heads, kv_heads=kv_heads, d=d, page=page, kv=kv, new=new,
                    ragged=rng.random() < 0.7, pairs=pairs, axes=axes, interleaved=interleaved,
                    positions=max(positions, kv))
    q = {"decode": 1, "verify": rng.randint(2, 9), "chunk": _log(rng, 16, 2500)}[op]
    batch = _log(rng, 1, {"decode": 96, "verify": 24, "chunk": 4}[op])
    top = min({"decode": 60000, "verify": 24000, "chunk": 16000}[op], int(2e9 / (batch * kv_heads * d)))
    if op == "chunk":   # pairs of the largest listed case at most
        top = min(top, int(1.6e9 / (batch * kv_heads * group * q)))
    q = min(q, max(1, top))
    kv = max(q, _log(rng, 1, max(1, top)))
    softcap = rng.choice([0.0, 0.0, 15.0, 30.0, 50.0])
    docs = rng.randint(1, 6) if rng.random() < 0.3 else 0
    prefix = rng.random() < 0.3
    alibi = rng.random() < 0.4 or not (softcap or docs or prefix)
    c = _attn("", batch=batch, q_heads=group * kv_heads, kv_heads=kv_heads, d=d, page=page, kv=kv, q=q,
              ragged=rng.random() < 0.7, causal=rng.random() < 0.8, window=_log(rng, 1, 8192) if rng.random() < 0.25 else 0,
              softcap=softcap, alibi=alibi, prefix=prefix, docs=docs, heat=rng.choice([1.0, 1.0, 3.0, 6.0]))
    del c["name"]
    return c


def _rng(case, salt):
    return random.Random("%s %s" % (salt, sorted((k, v) for k, v in case.items() if k != "name")))


def _lens(case):
    """(kv_lens, new or query tokens) of a case, the same whatever the seed of its inputs."""
    rng = _rng(case, "lens")
    ragged, more = case["ragged"], case["batch"] - 1
    kv = [case["kv"]] + [max(1, int(case["kv"] * rng.random() ** 1.5)) if ragged else case["kv"] for _ in range(more)]
    top = case["q"] if case["op"] == "attn" else case["new"]
    n = [top] + [rng.randint(1, top) if ragged and top > 8 else top for _ in range(more)]
    return [max(a, b) for a, b in zip(kv, n)], n


def _prefix(case):
    """Tokens at the front of each sequence that all its rows see; none in some of them."""
    rng = _rng(case, "prefix")
    return [0 if rng.random() < 0.2 else int(length * rng.random()) for length in _lens(case)[0]]


def _ranges(case):
    """[first, end) of the keys that each row may see: its document; the last rows of some sequences are padding."""
    rng = _rng(case, "docs")
    rows = []
    for b, (length, n) in enumerate(zip(*_lens(case))):
        cuts = [0] + sorted(rng.randint(0, length) for _ in range(case["docs"] - 1)) + [length]
        pad = n // 16 if b % 2 else 0
        at = 0
        for t in range(length - n, length):
            while cuts[at + 1] <= t:
                at += 1
            rows.append((0, 0) if t >= length - pad else (cuts[at], cuts[at + 1]))
    return rows


def _visible(case):
    """[first, end) that each row of each sequence sees, by sequence (a mask leaves one run of keys)."""
    kv, n = _lens(case)
    pre = _prefix(case) if case["prefix"] else [0] * len(kv)
    ranges = _ranges(case) if case["docs"] else None
    at = 0
    for length, rows, p in zip(kv, n, pre):
        out = []
        for i in range(rows):
            t = length - rows + i
            hi = min(length, max(t + 1, p)) if case["causal"] else length
            lo = max(0, t - case["window"] + 1) if case["window"] else 0
            if ranges:
                lo, hi = max(lo, ranges[at + i][0]), min(hi, ranges[at + i][1])
            out.append((lo, max(lo, hi)))
        at += rows
        yield out


# ---------------------------------------------------------------- the formats

def _axis_of(case):
    """Pairs of each axis, and the axis of each pair."""
    pairs, axes = case["pairs"], case["axes"]
    sections = [pairs // axes + (pairs % axes if a == 0 else 0) for a in range(axes)]
    return sections, [a for a, n in enumerate(sections) for _ in range(n)]


def _frequencies(case):
    """10000^(-i / n): a ladder of its own for each axis where pairs are interleaved, one ladder over all pairs otherwise."""
    sections, _ = _axis_of(case)
    if not case["interleaved"]:
        sections = [case["pairs"]]
    return [10000.0 ** (-i / n) for n in sections for i in range(n)]


def _positions(case, rows, base, gen, dev):
    """[rows, axes] of a video (frames of 30 x 52) or of text with images in it; [rows] of text."""
    top = case["positions"]
    if case["axes"] == 1:
        return None if base is not None else torch.randint(0, top, (rows,), generator=gen, device=dev, dtype=torch.int32)
    i = torch.arange(rows, device=dev) + int(torch.randint(0, 1560, (1,), generator=gen, device=dev))
    grid = [i // 1560 + torch.randint(0, 64, (1,), generator=gen, device=dev), i % 1560 // 52, i % 52]
    return torch.stack([(g % top).int() for g in grid[:case["axes"]]], 1).contiguous()


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, within [E_MIN, E_MAX], of fp32 values."""
    m, e = torch.frexp(amax)                                  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _pow2(e, dtype=torch.float32):
    """2^e, exactly, from the bits of the exponent."""
    if dtype == torch.float64:
        return ((e.long() + 1023) << 52).view(torch.float64)
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(x, e):
    return (x * _pow2(-e)).clamp(-448, 448).to(torch.float8_e4m3fn)


def _pool(shape, gen, dev):
    """A filled pool: values with a mean and a few strong channels for K, page by page scales of its own for V."""
    layers, n_pages, heads, page, d = shape
    codes, scales = [], []
    for kind in "kv":
        c = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
        s = torch.empty(shape[:3], dtype=torch.bfloat16, device=dev)
        lift = torch.randn(heads, 1, d, generator=gen, device=dev) * 0.5
        gain = torch.where(torch.rand(heads, 1, d, generator=gen, device=dev) < 0.03, 4.0, 1.0)
        for p0 in range(0, n_pages, 512):
            x = torch.randn(min(512, n_pages - p0), heads, page, d, generator=gen, device=dev)
            if kind == "k":
                x = x * gain + lift
            else:
                x = x * torch.exp(torch.randn(x.shape[0], heads, 1, 1, generator=gen, device=dev))
            x = x.bfloat16().float()
            e = _exponent(x.abs().amax(dim=(2, 3)))
            c[0, p0:p0 + 512] = _codes(x, e[:, :, None, None])
            s[0, p0:p0 + 512] = _pow2(e).bfloat16()
        codes.append(c)
        scales.append(s)
    return codes + scales


def _table(n_pages_of, n_pages, gen, dev):
    ids = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    need = torch.tensor(n_pages_of, device=dev)
    first = need.cumsum(0) - need
    at = torch.arange(max(n_pages_of), device=dev)
    t = ids[(first[:, None] + at).clamp(max=n_pages - 1)]
    return torch.where(at < need[:, None], t, -1).to(torch.int32).contiguous()


def _values(gen, dev, *shape):
    """Rows of uneven size, as projections give them."""
    x = torch.randn(*shape, generator=gen, device=dev)
    return (x * torch.exp(torch.randn(*shape[:-2], 1, 1, generator=gen, device=dev) * 0.3)).bfloat16()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, heads, d = case["op"], case["kv_heads"], case["d"]
    s = dict(case=dict(case), op=op)
    if op != "attn":
        angle = torch.arange(case["positions"], device=dev)[:, None] * torch.tensor(_frequencies(case), dtype=torch.float64, device=dev)
        s["cos_sin"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        s["sections"], of = _axis_of(case)
        s["axis"] = torch.tensor(of, device=dev)
    if op == "rope":
        lead = (case["rows"],) if case["layout"] == "packed" else (case["batch"],)
        shape = (lambda h: lead + (h, d)) if case["layout"] == "packed" else (lambda h: lead + (h, case["rows"], d))
        s["q"], s["k"] = _values(gen, dev, *shape(case["q_heads"])), _values(gen, dev, *shape(heads))
        s["positions"] = _positions(case, case["rows"], None, gen, dev)
    else:
        kv, n = _lens(case)
        used = [-(-x // case["page"]) for x in kv]
        s["lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        # one token of every sequence needs no offsets
        s["offsets"] = None if max(n) == 1 else torch.tensor([0] + n, device=dev).cumsum(0).to(torch.int32)
        s["max_n"], total = max(n), sum(n)
        s["table"] = _table(used, sum(used) + 3, gen, dev)
        s["kc"], s["vc"], s["ks"], s["vs"] = _pool((1, sum(used) + 3, heads, case["page"], d), gen, dev)
        s["q"] = _values(gen, dev, total, case["q_heads"], d) if op == "append" else (
            torch.randn(total, case["q_heads"], d, generator=gen, device=dev) * case["heat"]).bfloat16()
    if op == "append":
        s["k"], s["v"] = _values(gen, dev, total, heads, d), _values(gen, dev, total, heads, d)
        s["positions"] = _positions(case, total, s["lens"], gen, dev)
    if op == "attn":
        hq = case["q_heads"]
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=dev) if case["alibi"] else None
        s["prefix"] = torch.tensor(_prefix(case), dtype=torch.int32, device=dev) if case["prefix"] else None
        s["ranges"] = torch.tensor(_ranges(case), dtype=torch.int32, device=dev) if case["docs"] else None
    if own:
        from quantized_kv_cache_quantize_gb300 import kvq
        s["kvq"] = kvq
        if op != "attn":
            s["rope"] = kvq.RopeTable(s["cos_sin"], s["sections"], case["interleaved"])
        if op != "rope":
            s["cache"] = kvq.PagedCache(s["kc"], s["vc"], s["ks"], s["vs"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"rope": _rope, "append": _append, "attn": _attention}[s["op"]](s)


def _rotated(s, x, positions):
    """x [..., heads, d] in 32 bits, rotated by positions [..., axes] (broadcast over what x has in front)."""
    pairs = s["case"]["pairs"]
    at = positions.long()[..., s["axis"]]                                             # [..., pairs]
    cs = s["cos_sin"][at, torch.arange(pairs, device=x.device)]
    c, w = cs[..., 0].unsqueeze(-2), cs[..., 1].unsqueeze(-2)                          # over the heads
    x = x.float()
    x0, x1 = (x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]) if s["case"]["interleaved"] else (x[..., :pairs], x[..., pairs:2 * pairs])
    if s["case"].get("inverse"):
        w = -w
    y0, y1 = x0 * c - x1 * w, x1 * c + x0 * w
    y = torch.stack([y0, y1], -1).flatten(-2) if s["case"]["interleaved"] else torch.cat([y0, y1], -1)
    return torch.cat([y, x[..., 2 * pairs:]], -1)


def _rope(s):
    if own:
        q, k = s["kvq"].rope(s["rope"], s["q"], s["positions"], k=s["k"], inverse=s["case"]["inverse"])
        return {"q": q, "k": k}
    pos = s["positions"].view(s["case"]["rows"], -1)
    if s["case"]["layout"] == "packed":
        return {n: _rotated(s, s[n], pos).bfloat16() for n in "qk"}
    return {n: _rotated(s, s[n].transpose(1, 2), pos).transpose(1, 2).bfloat16().contiguous() for n in "qk"}


def _spots(s):
    """Sequence, position of each packed row; first position of each sequence's rows; rows of each sequence."""
    dev, total, batch = s["q"].device, s["q"].shape[0], s["table"].shape[0]
    off = torch.arange(batch + 1, device=dev) if s["offsets"] is None else s["offsets"].long()
    n = off[1:] - off[:-1]
    seq = torch.repeat_interleave(torch.arange(batch, device=dev), n, output_size=total)
    begin = s["lens"].long() - n
    return seq, begin[seq] + torch.arange(total, device=dev) - off[seq], begin, n, off


def _append(s):
    if own:
        q = s["kvq"].pages_append_rope(s["cache"], s["rope"], s["k"], s["v"], s["table"], s["lens"], s["offsets"],
                                       positions=s["positions"], q=s["q"])
        return {"q": q, "k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    page, dev = s["case"]["page"], s["k"].device
    total, heads, d = s["k"].shape
    seq, pos, begin, n, off = _spots(s)
    turn = pos[:, None] if s["positions"] is None else s["positions"]
    slot, line = s["table"].long()[seq, pos // page], pos % page                     # each row's page, and its place there
    first = (pos // page) * page >= begin[seq]                                       # its page holds no earlier token
    n_pages = s["kc"].shape[1]
    fresh = torch.zeros(n_pages, dtype=torch.bool, device=dev).index_fill_(0, slot[first], True)
    old = torch.arange(page, device=dev)
    start = torch.full((n_pages,), page, device=dev).scatter_reduce_(0, slot, line, "amin")
    rows = {"k": _rotated(s, s["k"], turn), "v": s["v"].float()}
    for codes, scale, new in ((s["kc"][0], s["ks"][0], rows["k"]), (s["vc"][0], s["vs"][0], rows["v"])):
        codes = codes.view(torch.uint8)
        amax = torch.zeros(n_pages, heads, device=dev)
        amax.scatter_reduce_(0, slot[:, None].expand(-1, heads), new.abs().amax(-1), "amax")
        had = torch.frexp(scale.float())[1] - 1
        e = _exponent(amax)
        e = torch.where(fresh[:, None], e, torch.maximum(e, had))
        # earlier tokens of the pages written to (the first page of each sequence at most)
        part = torch.where(first | (pos != begin[seq]), -1, slot)[off[:-1].clamp(max=total - 1)]
        part = torch.where((n > 0) & (part >= 0), part, n_pages)                     # [B]; n_pages: nothing there
        at = part.clamp(max=n_pages - 1)
        kept = _codes(codes[at].view(torch.float8_e4m3fn).float(), (e - had)[at][..., None, None]).view(torch.uint8)
        kept = torch.where((old < start[at][:, None])[:, None, :, None], kept, codes[at])
        codes[at[part < n_pages]] = kept[part < n_pages]
        codes[slot, :, line] = _codes(new, e[slot][..., None]).view(torch.uint8)
        scale[slot] = _pow2(e[slot]).bfloat16()
    return {"q": _rotated(s, s["q"], turn).bfloat16(), "k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}


def _attention(s):
    c = s["case"]
    if own:
        out, lse = s["kvq"].paged_attention(s["cache"], s["q"], s["table"], s["lens"], s["offsets"], max_q=s["max_n"],
                                            causal=c["causal"], window=c["window"], with_lse=True, softcap=c["softcap"],
                                            slopes=s["slopes"], prefix=s["prefix"], ranges=s["ranges"])
        return {"out": out, "lse": lse}
    q, page, dev = s["q"], c["page"], s["q"].device
    total, hq, d = q.shape
    batch, width = s["table"].shape
    hkv = c["kv_heads"]
    group = hq // hkv
    seq, _, begin, n, off = _spots(s)
    lens = s["lens"].long()
    step = torch.arange(s["max_n"], device=dev)
    row = (off[:-1, None] + step).clamp(max=total - 1)                               # [B, max_n]
    qp = q[row].float().view(batch, -1, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    pos = begin[:, None] + step                                                      # [B, max_n]
    key = torch.arange(width * page, device=dev)
    seen = (key < lens[:, None])[:, None, :] & (step < n[:, None])[:, :, None]       # [B, max_n, keys]
    if c["causal"]:
        upto = key <= pos[:, :, None]
        if s["prefix"] is not None:
            upto = upto | (key < s["prefix"][:, None, None])
        seen = seen & upto
    if c["window"]:
        seen = seen & (key > pos[:, :, None] - c["window"])
    if s["ranges"] is not None:
        of = s["ranges"][row]
        seen = seen & (key >= of[..., :1]) & (key < of[..., 1:])
    ids = s["table"].long().clamp(min=0)

    def rows(codes, scale):
        x = codes[0].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()         # [B, width, Hkv, page, d]
        x = x * scale[0][ids].float()[..., None, None]
        x = x.transpose(1, 2).reshape(batch, hkv, width * page, d)
        return torch.where((key < lens[:, None])[:, None, :, None], x, 0.0)

    x = torch.matmul(qp, rows(s["kc"], s["ks"]).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    x = x.view(batch, hkv, group, s["max_n"], -1)
    if c["softcap"]:
        x = torch.tanh(x * (1.0 / c["softcap"])) * c["softcap"]
    if s["slopes"] is not None:
        far = (pos[:, :, None] - key).abs().float()
        x = x - s["slopes"].view(hkv, group, 1, 1) * far[:, None, None]
    x = torch.where(seen[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    base = torch.where(top > -math.inf, top, 0.0)
    x = torch.exp(x - base)
    tot = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(batch, hkv, group * s["max_n"], -1), rows(s["vc"], s["vs"])).view(batch, hkv, group, -1, d)
    out = out / torch.where(tot > 0, tot, 1.0)
    lse = base + torch.log(tot)
    at = torch.arange(total, device=dev) - off[seq]
    return {"out": out[seq, :, :, at].reshape(total, hq, d).bfloat16(), "lse": lse[seq, :, :, at].reshape(total, hq)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    heads, hq, d = case["kv_heads"], case["q_heads"], case["d"]
    if case["op"] == "attn":
        rows = sum(_lens(case)[1])
        keys = pairs = 0
        for seen in _visible(case):
            some = [r for r in seen if r[1] > r[0]]
            pairs += sum(b - a for a, b in some)
            keys += max(b for _, b in some) - min(a for a, _ in some) if some else 0
        cache = 2 * heads * (keys * d + 2 * (keys // case["page"])) + 4 * (keys // case["page"])
        asked = 4 * hq * case["alibi"] + 4 * case["batch"] * case["prefix"] + 8 * rows * (case["docs"] > 0)
        return {"bytes": cache + rows * hq * (4 * d + 4) + asked, "flops": 4 * pairs * hq * d}
    rows = case["rows"] * case["batch"] if case["op"] == "rope" else sum(_lens(case)[1])
    # entries of the table that the rows name: a row each, or those of a video's frames, lines and columns
    entries = min(case["positions"], rows) if case["axes"] == 1 else min(case["positions"], rows // 1560 + 30 + 52)
    turns = 8 * case["pairs"] * entries + 4 * case["axes"] * rows
    if case["op"] == "rope":
        return {"bytes": 4 * rows * (hq + heads) * d + turns, "flops": 6 * rows * (hq + heads) * case["pairs"]}
    pages = rows // case["page"] + case["batch"]
    return {"bytes": rows * d * (4 * hq + 6 * heads) + 4 * heads * pages + 8 * case["batch"] + turns,
            "flops": 6 * rows * (hq + heads) * case["pairs"] + 4 * rows * heads * d}


# ---------------------------------------------------------------- from the definition, in 64 bits

def _exact_codes(x, e):
    """Nearest E4M3 value (ties to even) of x / 2^e, in 64 bits: 3 bits behind the point, steps of 2^-9 at the least."""
    x = x * _pow2(-e, torch.float64)
    b = (torch.frexp(x)[1] - 4).clamp(min=-9)
    return (torch.round(x * _pow2(-b, torch.float64)) * _pow2(b, torch.float64)).clamp(-448, 448)


def _exact_exponent(amax):
    if amax == 0:
        return E_MIN
    e = math.ceil(math.log2(amax / 448.0)) - 2
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return max(E_MIN, min(E_MAX, e))


def _turned(case, x, pos):
    """x [rows, heads, d] times the rotations' complex numbers, the angles from the positions [rows, axes]."""
    p = case["pairs"]
    z = x[..., :2 * p].double()
    z = torch.view_as_complex(z.unflatten(-1, (p, 2)).contiguous()) if case["interleaved"] else torch.complex(z[..., :p].contiguous(), z[..., p:].contiguous())
    freq = torch.tensor(_frequencies(case), dtype=torch.float64, device=x.device)
    angle = pos.double()[:, _axis_of(case)[1]] * freq * (-1.0 if case.get("inverse") else 1.0)
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
    y = torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., 2 * p:].double()], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        pos = s["positions"].view(case["rows"], -1)
        if case["layout"] == "packed":
            return {n: _turned(case, s[n], pos) for n in "qk"}
        return {n: torch.stack([_turned(case, x.transpose(0, 1), pos).transpose(0, 1) for x in s[n]]) for n in "qk"}
    kc, vc, ks, vs = (s[k] for k in ("kc", "vc", "ks", "vs"))
    kv, n = _lens(case)
    page, heads, d = case["page"], case["kv_heads"], case["d"]
    table = s["table"].tolist()
    if case["op"] == "append":
        pos = s["positions"]
        if pos is None:
            pos = torch.cat([torch.arange(a - b, a, device=kc.device) for a, b in zip(kv, n)])[:, None]
        turned = _turned(case, s["k"], pos)
        new = [t.double() for t in (kc, vc, ks, vs)]
        at = 0
        for b, (length, rows) in enumerate(zip(kv, n)):
            start, p = length - rows, (length - rows) // page
            while p * page < length:
                lo, hi, slot = max(start, p * page), min(length, (p + 1) * page), table[b][p]
                for codes, scale, x in ((new[0], new[2], turned), (new[1], new[3], s["v"].double())):
                    x = x[at + lo - start:at + hi - start]
                    es = [_exact_exponent(a) for a in x.abs().amax(dim=(0, 2)).tolist()]
                    if lo > p * page:
                        had = [int(round(math.log2(v))) for v in scale[0, slot].tolist()]
                        es = [max(a, b_) for a, b_ in zip(es, had)]
                        up = torch.tensor([a - b_ for a, b_ in zip(es, had)], device=x.device)[:, None, None]
                        codes[0, slot, :, :lo - p * page] = _exact_codes(codes[0, slot, :, :lo - p * page], up)
                    e = torch.tensor(es, device=x.device)
                    codes[0, slot, :, lo - p * page:hi - p * page] = _exact_codes(x.transpose(0, 1), e[:, None, None])
                    scale[0, slot] = _pow2(e, torch.float64)
                p += 1
            at += rows
        return dict(q=_turned(case, s["q"], pos), **dict(zip(("k", "v", "k_scale", "v_scale"), new)))
    hq = case["q_heads"]
    out = torch.zeros(sum(n), hq, d, dtype=torch.float64, device=kc.device)
    lse = torch.full((sum(n), hq), -math.inf, dtype=torch.float64, device=kc.device)
    at = 0
    for b, seen in enumerate(_visible(case)):
        length, rows = kv[b], n[b]
        ids = torch.tensor(table[b][:-(-length // page)], device=kc.device)
        k, v = ((c[0].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * x[0][ids].double()[..., None, None]).transpose(0, 1).reshape(heads, -1, d)[:, :length]
                for c, x in ((kc, ks), (vc, vs)))
        j = torch.arange(length, device=kc.device)
        run_of = torch.tensor(seen, device=kc.device)
        for r0 in range(0, rows, 512):
            r1 = min(rows, r0 + 512)
            t = torch.arange(length - rows + r0, length - rows + r1, device=kc.device)[:, None]
            hide = (j < run_of[r0:r1, :1]) | (j >= run_of[r0:r1, 1:])
            for h in range(heads):
                g = slice(h * (hq // heads), (h + 1) * (hq // heads))
                x = s["q"][at + r0:at + r1, g].double().transpose(0, 1) @ k[h].T / math.sqrt(d)
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if case["alibi"]:
                    x = x - s["slopes"][g].double()[:, None, None] * (t - j).abs()
                x = x.masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, -1, keepdim=True)
                out[at + r0:at + r1, g] = (torch.exp(x - torch.where(z > -math.inf, z, 0.0)) @ v[h]).transpose(0, 1)
                lse[at + r0:at + r1, g] = z[..., 0].T
        at += rows
    return {"out": out, "lse": lse}
