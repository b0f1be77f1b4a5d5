"""Cases of the paged 8-bit cache's operators: appending tokens, attention over the pages, copying and compacting pages.

A cache of ``layers`` x ``n_pages`` pages holds K and V as E4M3 codes [layers, n_pages, kv_heads, page, d] with one
power-of-two scale per page and head (bf16 [layers, n_pages, kv_heads]); a block table (int32 [batch, width], -1 where a row
has no page) gives each sequence its pages.

The exponent of a scale is the smallest e with max|x| <= 448 * 2^e, held within [-60, 60]; a code is e4m3(x / 2^e).
"""
import math
import random

import torch

own = False

E_MIN, E_MAX = -60, 60


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one sequence just after its start, a head per cache head: nothing but latency
        dict(name="attn_decode_small", op="attn", batch=1, q_heads=24, kv_heads=24, d=128, page=16, kv=333, q=1,
             ragged=False, causal=True, window=0),
        # a serving batch of mixed lengths, one new token each, grouped heads
        dict(name="attn_decode_ragged", op="attn", batch=64, q_heads=32, kv_heads=8, d=128, page=64, kv=8192, q=1,
             ragged=True, causal=True, window=0),
        # few sequences with a very long context
        dict(name="attn_decode_long", op="attn", batch=4, q_heads=40, kv_heads=8, d=128, page=128, kv=100001, q=1,
             ragged=False, causal=True, window=0),
        # several proposed tokens of each sequence checked at once, narrow heads, a sliding window
        dict(name="attn_verify_window", op="attn", batch=16, q_heads=32, kv_heads=4, d=64, page=32, kv=12000, q=5,
             ragged=True, causal=True, window=4096),
        # one chunk of a video stream (3 x 30 x 52 tokens) over its window and itself, no mask
        dict(name="attn_chunk_24h", op="attn", batch=1, q_heads=24, kv_heads=24, d=128, page=64, kv=23400, q=4680,
             ragged=False, causal=False, window=0),
        # prompts of several sequences, partly cached already, in one ragged batch
        dict(name="attn_prefill_ragged", op="attn", batch=4, q_heads=32, kv_heads=8, d=128, page=32, kv=8192, q=2048,
             ragged=True, causal=True, window=0),
        # one new token of every sequence of a serving batch
        dict(name="append_decode", op="append", batch=128, kv_heads=8, d=128, page=64, kv=2048, new=1, ragged=True),
        # a whole chunk of a video stream, all heads
        dict(name="append_chunk_24h", op="append", batch=1, kv_heads=24, d=128, page=64, kv=23400, new=4680,
             ragged=False),
        # the last pages of a few forked sequences
        dict(name="copy_fork_tails", op="copy", layers=4, n_pages=96, kv_heads=8, d=128, page=16, pairs=8),
        # a prefix of long contexts copied out, every layer
        dict(name="copy_prefix", op="copy", layers=24, n_pages=640, kv_heads=8, d=128, page=64, pairs=300),
        # a small pool after one of its sequences ended
        dict(name="compact_small", op="compact", layers=2, n_pages=200, kv_heads=4, d=64, page=32, batch=7, live=0.5),
        # a serving pool, half of its pages free, all layers
        dict(name="compact_pool", op="compact", layers=8, n_pages=2000, kv_heads=8, d=128, page=64, batch=40, live=0.55),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 12])
    op = rng.choice(["decode", "decode", "verify", "chunk", "append", "append", "copy", "compact"])
    if op in ("decode", "verify", "chunk"):
        q = {"decode": 1, "verify": rng.randint(2, 9), "chunk": _log(rng, 16, 3000)}[op]
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        batch = _log(rng, 1, {"decode": 96, "verify": 24, "chunk": 4}[op])
        top = min({"decode": 60000, "verify": 24000, "chunk": 16000}[op], int(2e9 / (batch * kv_heads * d)))
        if op == "chunk":   # pairs of the largest listed case at most
            top = min(top, int(2.4e9 / (batch * kv_heads * group * q)))
        q = min(q, max(1, top))
        kv = max(q, _log(rng, 1, max(1, top)))
        return dict(op="attn", batch=batch, q_heads=group * kv_heads, kv_heads=kv_heads, d=d, page=page, kv=kv, q=q,
                    ragged=rng.random() < 0.7, causal=rng.random() < 0.8,
                    window=_log(rng, 1, 8192) if rng.random() < 0.25 else 0)
    if op == "append":
        batch = _log(rng, 1, 200)
        new = 1 if rng.random() < 0.5 else _log(rng, 1, max(2, int(4e7 / (batch * kv_heads * d))))
        return dict(op="append", batch=batch, kv_heads=kv_heads, d=d, page=page, kv=new + _log(rng, 1, 4000), new=new,
                    ragged=rng.random() < 0.7)
    layers = _log(rng, 1, 24)
    page_bytes = layers * kv_heads * page * d * 2
    n_pages = _log(rng, 24, max(30, min(6000, int(2e9 / page_bytes))))
    if op == "copy":
        return dict(op="copy", layers=layers, n_pages=n_pages, kv_heads=kv_heads, d=d, page=page,
                    pairs=_log(rng, 1, n_pages // 2))
    return dict(op="compact", layers=layers, n_pages=n_pages, kv_heads=kv_heads, d=d, page=page, batch=_log(rng, 1, 64),
                live=round(rng.uniform(0.1, 0.95), 3))


def _rng(case, salt):
    return random.Random("%s %s" % (salt, sorted((k, v) for k, v in case.items() if k != "name")))


def _spread(case, rng, top):
    """Lengths of a batch: all `top`, or for a ragged batch spread below it, the first at the top."""
    n = case["batch"]
    return [top] + [max(1, int(top * rng.random() ** 1.5)) if case["ragged"] else top for _ in range(n - 1)]


def _lens(case):
    """(kv_lens, new or query tokens) of a case, the same whatever the seed of its inputs."""
    rng = _rng(case, "lens")
    kv, top = _spread(case, rng, case["kv"]), case["q"] if case["op"] == "attn" else case["new"]
    n = [top] + [rng.randint(1, top) if case["ragged"] and top > 8 else top for _ in range(case["batch"] - 1)]
    if case["op"] == "append" or top > 8:
        kv = [max(a, b) for a, b in zip(kv, n)]
    return kv, n


def _pages(kv, page):
    return [-(-x // page) for x in kv]


# ---------------------------------------------------------------- the format

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
        for i in range(layers):
            for p0 in range(0, n_pages, 512):
                x = torch.randn(min(512, n_pages - p0), heads, page, d, generator=gen, device=dev)
                if kind == "k":
                    x = x * gain + lift
                else:
                    x = x * torch.exp(torch.randn(x.shape[0], heads, 1, 1, generator=gen, device=dev))
                x = x.bfloat16().float()
                e = _exponent(x.abs().amax(dim=(2, 3)))
                c[i, p0:p0 + 512] = _codes(x, e[:, :, None, None])
                s[i, p0:p0 + 512] = _pow2(e).bfloat16()
        codes.append(c)
        scales.append(s)
    return codes + scales


def _table(n_pages_of, n_pages, gen, dev, width=None):
    width = width or max(n_pages_of)
    ids = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    need = torch.tensor(n_pages_of, device=dev)
    first = need.cumsum(0) - need
    at = torch.arange(width, device=dev)
    t = ids[(first[:, None] + at).clamp(max=n_pages - 1)]
    return torch.where(at < need[:, None], t, -1).to(torch.int32).contiguous()


def _offsets(n, dev):
    return torch.tensor([0] + n, device=dev).cumsum(0).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, heads, d, page = case["op"], case["kv_heads"], case["d"], case["page"]
    s = dict(case=dict(case), op=op)
    if op in ("attn", "append"):
        kv, n = _lens(case)
        used = _pages(kv, page)
        n_pages = sum(used) + 3
        s["lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        # one token of every sequence needs no offsets
        s["offsets"] = None if max(n) == 1 else _offsets(n, dev)
        s["max_n"] = max(n)
        s["table"] = _table(used, n_pages, gen, dev)
        s["kc"], s["vc"], s["ks"], s["vs"] = _pool((1, n_pages, heads, page, d), gen, dev)
        total = sum(n)
        if op == "attn":
            s["q"] = torch.randn(total, case["q_heads"], d, generator=gen, device=dev).bfloat16()
        else:
            s["k"] = (torch.randn(total, heads, d, generator=gen, device=dev)
                      * torch.exp(torch.randn(total, 1, 1, generator=gen, device=dev) * 0.3)).bfloat16()
            s["v"] = torch.randn(total, heads, d, generator=gen, device=dev).bfloat16()
    else:
        n_pages = case["n_pages"]
        s["kc"], s["vc"], s["ks"], s["vs"] = _pool((case["layers"], n_pages, heads, page, d), gen, dev)
        order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32).cpu()
        if op == "copy":
            s["src"], s["dst"] = order[:case["pairs"]].clone(), order[n_pages // 2:n_pages // 2 + case["pairs"]].clone()
            s["src_dev"], s["dst_dev"] = s["src"].to(dev), s["dst"].to(dev)
        else:
            s["table"] = _live_table(case, order).to(dev)
    if own:
        from quantized_kv_cache_quantize_gb300 import kvq
        s["kvq"] = kvq
        s["cache"] = kvq.PagedCache(s["kc"], s["vc"], s["ks"], s["vs"])
    return s


def _live_table(case, order):
    """Rows of uneven lengths over a share of the pages, in no order; the first pages of row 0 shared by every third row."""
    rng = _rng(case, "rows")
    live = max(1, int(case["n_pages"] * case["live"]))
    cuts = sorted(rng.randint(0, live) for _ in range(case["batch"] - 1))
    of = [b - a for a, b in zip([0] + cuts, cuts + [live])]
    width = max(of) + 2
    t = torch.full((case["batch"], width), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(of):
        t[r, :n] = order[at:at + n]
        at += n
    shared = min(of[0], 4)
    for r in range(3, case["batch"], 3):
        t[r, :min(shared, of[r])] = t[0, :min(shared, of[r])]
    return t


# ---------------------------------------------------------------- one pass

def run(s):
    return {"attn": _attn, "append": _append, "copy": _copy, "compact": _compact}[s["op"]](s)


def _attn(s):
    c = s["case"]
    if own:
        out, lse = s["kvq"].paged_attention(s["cache"], s["q"], s["table"], s["lens"], s["offsets"], max_q=s["max_n"],
                                            causal=c["causal"], window=c["window"], with_lse=True)
        return {"out": out, "lse": lse}
    q, page, dev = s["q"], c["page"], s["q"].device
    total, hq, d = q.shape
    batch, width = s["table"].shape
    hkv = c["kv_heads"]
    group = hq // hkv
    lens = s["lens"].long()
    off = torch.arange(batch + 1, device=dev) if s["offsets"] is None else s["offsets"].long()
    n = off[1:] - off[:-1]
    step = torch.arange(s["max_n"], device=dev)
    row = (off[:-1, None] + step).clamp(max=total - 1)                               # [B, max_n]
    qp = q[row].float().view(batch, -1, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    pos = lens[:, None] - n[:, None] + step                                          # [B, max_n]
    key = torch.arange(width * page, device=dev)
    seen = (key < lens[:, None])[:, None, :] & (step < n[:, None])[:, :, None]
    if c["causal"]:
        seen = seen & (key <= pos[:, :, None])
    if c["window"]:
        seen = seen & (key > pos[:, :, None] - c["window"])
    ids = s["table"].long().clamp(min=0)

    def rows(codes, scale):
        x = codes[0].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()         # [B, width, Hkv, page, d]
        x = x * scale[0][ids].float()[..., None, None]
        x = x.transpose(1, 2).reshape(batch, hkv, width * page, d)
        return torch.where((key < lens[:, None])[:, None, :, None], x, 0.0)

    seen = seen[:, None, None].expand(batch, 1, group, -1, -1).reshape(batch, 1, group * s["max_n"], -1)
    x = torch.matmul(qp, rows(s["kc"], s["ks"]).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    base = torch.where(top > -math.inf, top, 0.0)
    x = torch.exp(x - base)
    tot = x.sum(-1, keepdim=True)
    out = torch.matmul(x, rows(s["vc"], s["vs"])) / torch.where(tot > 0, tot, 1.0)
    lse = base + torch.log(tot)
    back = torch.repeat_interleave(torch.arange(batch, device=dev), n, output_size=total)
    at = torch.arange(total, device=dev) - off[back]
    out = out.view(batch, hkv, group, -1, d)[back, :, :, at].reshape(total, hq, d).bfloat16()
    return {"out": out, "lse": lse.view(batch, hkv, group, -1)[back, :, :, at].reshape(total, hq)}


def _append(s):
    if own:
        s["kvq"].pages_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["offsets"])
        return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    c, dev = s["case"], s["k"].device
    page, batch = c["page"], s["table"].shape[0]
    total, heads, d = s["k"].shape
    lens = s["lens"].long()
    off = torch.arange(batch + 1, device=dev) if s["offsets"] is None else s["offsets"].long()
    n = off[1:] - off[:-1]
    seq = torch.repeat_interleave(torch.arange(batch, device=dev), n, output_size=total)
    pos = (lens - n)[seq] + torch.arange(total, device=dev) - off[seq]               # where each new token goes
    slot, line = s["table"].long()[seq, pos // page], pos % page                     # its page, and its place there
    first = (pos // page) * page >= (lens - n)[seq]                                  # its page holds no earlier token
    n_pages = s["kc"].shape[1]
    fresh = torch.zeros(n_pages, dtype=torch.bool, device=dev).index_fill_(0, slot[first], True)
    old = torch.arange(page, device=dev)
    begin = torch.full((n_pages,), page, device=dev).scatter_reduce_(0, slot, line, "amin")
    for codes, scale, new in ((s["kc"][0], s["ks"][0], s["k"].float()), (s["vc"][0], s["vs"][0], s["v"].float())):
        codes = codes.view(torch.uint8)
        amax = torch.zeros(n_pages, heads, device=dev)
        amax.scatter_reduce_(0, slot[:, None].expand(-1, heads), new.abs().amax(-1), "amax")
        had = torch.frexp(scale.float())[1] - 1
        e = _exponent(amax)
        e = torch.where(fresh[:, None], e, torch.maximum(e, had))
        # earlier tokens of the pages written to (the first page of each sequence at most)
        part = torch.where(first | (pos != (lens - n)[seq]), -1, slot)
        part = part[(off[:-1]).clamp(max=total - 1)]
        part = torch.where((n > 0) & (part >= 0), part, n_pages)                     # [B]; n_pages: nothing there
        at = part.clamp(max=n_pages - 1)
        kept = _codes(codes[at].view(torch.float8_e4m3fn).float(), (e - had)[at][..., None, None]).view(torch.uint8)
        kept = torch.where((old < begin[at][:, None])[:, None, :, None], kept, codes[at])
        codes[at[part < n_pages]] = kept[part < n_pages]
        codes[slot, :, line] = _codes(new, e[slot][..., None]).view(torch.uint8)
        scale[slot] = _pow2(e[slot]).bfloat16()
    return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}


def _copy(s):
    if own:
        s["kvq"].pages_copy(s["cache"], s["src"], s["dst"])
    else:
        src, dst = s["src_dev"].long(), s["dst_dev"].long()
        for t in (s["kc"].view(torch.uint8), s["vc"].view(torch.uint8), s["ks"], s["vs"]):
            t[:, dst] = t[:, src]
    return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}


def _compact(s):
    if own:
        table, n_live = s["kvq"].pages_compact(s["cache"], s["table"])
    else:
        t = s["table"].long()
        n_pages = s["kc"].shape[1]
        ids = torch.arange(n_pages, device=t.device)
        live = torch.zeros(n_pages + 1, dtype=torch.bool, device=t.device)
        live = live.index_fill_(0, torch.where(t >= 0, t, n_pages).reshape(-1), True)[:n_pages]
        n_live = live.sum().to(torch.int32).reshape(1)
        src, dst = ids[live & (ids >= n_live)], ids[~live & (ids < n_live)]
        to = ids.clone()
        to[src] = dst
        table = torch.where(t >= 0, to[t.clamp(min=0)], t).to(torch.int32)
        for x in (s["kc"].view(torch.uint8), s["vc"].view(torch.uint8), s["ks"], s["vs"]):
            x[:, dst] = x[:, src]
    return {"table": table, "n_live": n_live, "k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}


# ---------------------------------------------------------------- what a pass cannot do without

def _pairs(case):
    """(keys read, query-key pairs) summed over the sequences, of one head."""
    keys = pairs = 0
    kv, n = _lens(case)
    for length, rows in zip(kv, n):
        t0 = length - rows
        lo_first = max(0, t0 - case["window"] + 1) if case["window"] else 0
        keys += length - lo_first
        for t in (t0, length - 1) if rows > 1 else (t0,):
            hi = min(length, t + 1) if case["causal"] else length
            lo = max(0, t - case["window"] + 1) if case["window"] else 0
            pairs += max(0, hi - lo) * (rows / 2 if rows > 1 else 1)
    return keys, pairs


def work(case):
    heads, d, page = case["kv_heads"], case["d"], case["page"]
    if case["op"] == "attn":
        keys, pairs = _pairs(case)
        rows = sum(_lens(case)[1]) * case["q_heads"]
        cache = 2 * heads * (keys * d + 2 * keys // page) + 4 * (keys // page)
        return {"bytes": cache + rows * (4 * d + 4), "flops": 4 * pairs * case["q_heads"] * d}
    if case["op"] == "append":
        n = sum(_lens(case)[1])
        return {"bytes": 2 * n * heads * d * 3 + 8 * case["batch"] + 2 * heads * 2 * (n // page + case["batch"]), "flops": 4 * n * heads * d}
    page_bytes = 2 * case["layers"] * heads * (page * d + 2)
    if case["op"] == "copy":
        return {"bytes": 2 * case["pairs"] * page_bytes, "flops": 0}
    live = max(1, int(case["n_pages"] * case["live"]))
    moves = live * (case["n_pages"] - live) / case["n_pages"]          # on average
    return {"bytes": 2 * moves * page_bytes + 8 * live, "flops": 0}


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


def exact(case, seed):
    s = prepare(case, seed)
    kc, vc, ks, vs = (s[k] for k in ("kc", "vc", "ks", "vs"))
    if case["op"] == "copy":
        new = [t.double() for t in (kc, vc, ks, vs)]
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            for t in new:
                t[:, b] = t[:, a]
        return dict(zip(("k", "v", "k_scale", "v_scale"), new))
    if case["op"] == "compact":
        rows = s["table"].tolist()
        live = sorted({x for r in rows for x in r if x >= 0})
        n, held = len(live), set(live)
        to = dict(zip([x for x in live if x >= n], [x for x in range(n) if x not in held]))
        new = [t.double() for t in (kc, vc, ks, vs)]
        for a, b in to.items():
            for t in new:
                t[:, b] = t[:, a]
        return dict(table=None, n_live=None, **dict(zip(("k", "v", "k_scale", "v_scale"), new)))
    kv, n = _lens(case)
    page, heads, d = case["page"], case["kv_heads"], case["d"]
    table = s["table"].tolist()
    if case["op"] == "append":
        new = [t.double() for t in (kc, vc, ks, vs)]
        at = 0
        for b, (length, rows) in enumerate(zip(kv, n)):
            start, p = length - rows, (length - rows) // page
            while p * page < length:
                lo, hi, slot = max(start, p * page), min(length, (p + 1) * page), table[b][p]
                for codes, scale, x in ((new[0], new[2], s["k"]), (new[1], new[3], s["v"])):
                    x = x[at + lo - start:at + hi - start].double()
                    amax = x.abs().amax(dim=(0, 2)).tolist()
                    es = [_exact_exponent(a) for a in amax]
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
        return dict(zip(("k", "v", "k_scale", "v_scale"), new))
    hq = case["q_heads"]
    out = torch.zeros(sum(n), hq, d, dtype=torch.float64, device=kc.device)
    lse = torch.full((sum(n), hq), -math.inf, dtype=torch.float64, device=kc.device)
    at = 0
    for b, (length, rows) in enumerate(zip(kv, n)):
        ids = torch.tensor(table[b][:-(-length // page)], device=kc.device)
        k, v = ((c[0].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * x[0][ids].double()[..., None, None]).transpose(0, 1).reshape(heads, -1, d)[:, :length]
                for c, x in ((kc, ks), (vc, vs)))
        j = torch.arange(length, device=kc.device)
        for r0 in range(0, rows, 512):
            r1 = min(rows, r0 + 512)
            t = torch.arange(length - rows + r0, length - rows + r1, device=kc.device)[:, None]
            hide = (j > t if case["causal"] else j < 0) | (j <= t - case["window"] if case["window"] else j < 0)
            for h in range(heads):
                g = slice(h * (hq // heads), (h + 1) * (hq // heads))
                x = s["q"][at + r0:at + r1, g].double().transpose(0, 1) @ k[h].T / math.sqrt(d)
                x = x.masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, -1, keepdim=True)
                out[at + r0:at + r1, g] = (torch.exp(x - torch.where(z > -math.inf, z, 0.0)) @ v[h]).transpose(0, 1)
                lse[at + r0:at + r1, g] = z[..., 0].T
        at += rows
    return {"out": out, "lse": lse}
