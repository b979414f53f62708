"""Workloads of the paged-cache operators: append with rotation, decode
attention over the pages, page selection and attention over selected pages.

With ``own`` false ``run`` computes an operator from elementary torch
operations in FP32 (the page scores, which decide an order, in FP64); with
``own`` true it makes the calls of ``quantized_cross_loop_gb300.kvq``.
"""

from __future__ import annotations

import math
import random

import torch

own = False

D = 128  # channels of a head, as everywhere in the library
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


def listed():
    return [
        # one decode step of a serving batch: one new token per request, K rotated into its page, q rotated with it
        dict(name="append_step", op="append", B=64, lo=512, T=2047, H=8, Hq=32, ps=64, cache="bf16", act="bf16",
             rows=1, rotary=128, inter=False, bounds=True, pad=0, heads_first=False, empty=False),
        # the smallest step: one request, one token
        dict(name="append_one", op="append", B=1, lo=256, T=256, H=8, Hq=32, ps=64, cache="bf16", act="bf16",
             rows=1, rotary=128, inter=False, bounds=True, pad=0, heads_first=False, empty=False),
        # prefill of four long prompts in one call
        dict(name="append_prompts", op="append", B=4, lo=0, T=0, H=8, Hq=64, ps=64, cache="bf16", act="bf16",
             rows=8192, rotary=128, inter=False, bounds=True, pad=0, heads_first=False, empty=False),
        # chunks of odd sizes into an 8-bit cache of small pages, interleaved pairs on half of the channels, padded rows
        dict(name="append_chunks_e4m3", op="append", B=9, lo=1, T=777, H=8, Hq=32, ps=16, cache="e4m3", act="bf16",
             rows=613, rotary=64, inter=True, bounds=True, pad=37, heads_first=True, empty=False),
        # one short request: latency
        dict(name="attn_one", op="attn", B=1, lo=256, T=256, H=8, Hq=32, ps=64, cache="bf16", act="bf16",
             heads_first=False, empty=False),
        # a wide batch of medium requests, odd length
        dict(name="attn_batch", op="attn", B=512, lo=1000, T=1000, H=8, Hq=32, ps=64, cache="bf16", act="bf16",
             heads_first=False, empty=False),
        # few long requests, eight query heads a KV head, small pages
        dict(name="attn_long", op="attn", B=4, lo=32768, T=32768, H=8, Hq=64, ps=16, cache="fp16", act="fp16",
             heads_first=True, empty=False),
        # a ragged batch over an 8-bit cache
        dict(name="attn_ragged_e4m3", op="attn", B=64, lo=512, T=16383, H=8, Hq=32, ps=64, cache="e4m3", act="bf16",
             heads_first=False, empty=True),
        # page selection of a batch
        dict(name="select_batch", op="select", B=32, lo=4096, T=4096, H=8, Hq=32, ps=16, cache="bf16", act="bf16",
             nsel=33, nfirst=1, nlast=2, empty=False),
        # page selection of long requests
        dict(name="select_long", op="select", B=4, lo=30001, T=131071, H=8, Hq=64, ps=16, cache="bf16", act="bf16",
             nsel=256, nfirst=1, nlast=4, empty=False),
        # attention over the pages selected in a ragged batch
        dict(name="sparse_ragged", op="sparse", B=64, lo=512, T=16383, H=8, Hq=32, ps=64, cache="bf16", act="bf16",
             nsel=16, heads_first=False, empty=False),
        # attention over selected small pages of long requests
        dict(name="sparse_long", op="sparse", B=4, lo=30001, T=65535, H=8, Hq=64, ps=16, cache="bf16", act="bf16",
             nsel=255, heads_first=True, empty=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "select", "sparse"])
    H = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 8, 8, 12, 16] if H < 8 else [1, 2, 3, 4, 5, 8])
    cache = rng.choice(["bf16", "bf16", "fp16", "e4m3"])
    act = cache if cache != "e4m3" else rng.choice(["bf16", "fp16"])
    ps = rng.choice([8, 16, 24, 32, 48, 64, 64, 128])
    case = dict(op=op, H=H, Hq=H * g, ps=ps, cache=cache, act=act, empty=rng.random() < 0.3)
    if op == "append":
        rows = _log(rng, 1, 4000)
        B = max(1, min(_log(rng, 1, 256), 16000 // rows))
        T = _log(rng, 1, 1500)
        rotary = rng.choice([0, 32, 64, 96, 128, 128])
        case.update(B=B, lo=rng.choice([0, T // 2, T]), T=T, rows=rows, rotary=rotary, inter=rng.random() < 0.3,
                    bounds=rng.random() < 0.7, pad=rng.choice([0, 0, 1, 50]), heads_first=rng.random() < 0.4)
        return case
    T = _log(rng, 1, 100000) if op != "select" else _log(rng, 200, 200000)
    T += 1 - T % 2 if rng.random() < 0.7 else 0
    B = max(1, min(_log(rng, 1, 400), (250000 if op != "select" else 500000) // T))
    lo = rng.choice([T, max(1, T // 8), 1])
    case.update(B=B, lo=lo, T=T)
    if op != "select":
        case.update(heads_first=rng.random() < 0.4)
    if op != "attn":
        nsel = _log(rng, 4, 300)
        case.update(nsel=nsel)
    if op == "select":
        case.update(nfirst=rng.choice([0, 1, 2]), nlast=rng.choice([0, 1, 2]))
    return case


# ------------------------------------------------------------------ sizes of a case (from its fields alone)


def _lengths(c):
    """Tokens of each request: T for lo == T, else spread over lo..T by their logarithm; `empty`: every fifth has none."""
    rng = random.Random(c["B"] * 1000003 + c["T"] * 31 + c["lo"])
    n = [c["T"] if c["lo"] == c["T"] else min(c["T"], max(c["lo"], _log(rng, c["lo"] + 1, c["T"] + 1) - 1))
         for _ in range(c["B"])]
    return [0 if c["empty"] and b % 5 == 3 else t for b, t in enumerate(n)]


def _new_rows(c):
    """Rows that an append brings for each request: one each in a decode step, else between a half and all of `rows`."""
    if c["rows"] == 1:
        return [1] * c["B"]
    rng = random.Random(c["B"] * 7919 + c["rows"])
    n = [c["rows"] if c["B"] == 4 else rng.randint(max(1, c["rows"] // 2), c["rows"]) for _ in range(c["B"])]
    return [0 if c["empty"] and b % 5 == 3 else r for b, r in enumerate(n)]


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    c = case
    cb = 1 if c["cache"] == "e4m3" else 2
    H, Hq, ps = c["H"], c["Hq"], c["ps"]
    lens = _lengths(c)
    if c["op"] == "append":
        rows = _new_rows(c)
        n = sum(rows)
        touched = sum(_cdiv(s + r, ps) - s // ps for s, r in zip(lens, rows) if r)
        partial = sum(1 for s, r in zip(lens, rows) if r and s % ps)
        by = n * H * D * 2 * (2 + cb) + n * Hq * D * 4 + n * c["rotary"] * 4
        by += (touched + partial) * H * 2 * D * cb if c["bounds"] else 0
        return {"bytes": by, "flops": 3 * n * (H + Hq) * c["rotary"]}
    if c["op"] == "select":
        pages = sum(_cdiv(t, ps) for t in lens)
        return {"bytes": pages * H * 2 * D * cb + c["B"] * (Hq * D * 2 + H * c["nsel"] * 4), "flops": pages * H * 4 * D}
    if c["op"] == "sparse":
        tokens = sum(min(t, c["nsel"] * ps - (-t) % ps) for t in lens)
    else:
        tokens = sum(lens)
    by = tokens * H * D * 2 * cb + c["B"] * Hq * D * 6 + (c["B"] * H * c["nsel"] * 4 if c["op"] == "sparse" else 0)
    return {"bytes": by, "flops": 4 * tokens * Hq * D}


# ------------------------------------------------------------------ inputs


def _pool(g, c, n_pages):
    """A K or V pool [n_pages][page][H][D] of the cache's type: normal values around a mean of each page (so that pages
    differ in what a query finds there); head-major in memory where the case says so."""
    H, ps = c["H"], c["ps"]
    dt = DTYPES[c["cache"]]
    out = torch.empty((n_pages, H, ps, D) if c.get("heads_first") else (n_pages, ps, H, D), dtype=dt, device="cuda")
    for a in range(0, n_pages, 4096):
        e = min(n_pages, a + 4096)
        mean = torch.randn((e - a, 1, H, D), generator=g, device="cuda") * 0.5
        x = torch.randn((e - a, ps, H, D), generator=g, device="cuda") + mean
        if c["cache"] == "e4m3":
            x = x * 16
        out[a:e] = (x.transpose(1, 2) if c.get("heads_first") else x).to(dt)
    return out.transpose(1, 2) if c.get("heads_first") else out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, Hq, ps = c["B"], c["H"], c["Hq"], c["ps"]
    act = DTYPES[c["act"]]
    lens = _lengths(c)
    rows = _new_rows(c) if c["op"] == "append" else [0] * B
    pages = [_cdiv(t + r, ps) for t, r in zip(lens, rows)]
    used = sum(pages)
    n_pages = used + 3  # some pages belong to nobody
    width = max(1, max(pages))
    # a table of shuffled pages, as a long-running server has it; entries behind a request's last page are not looked at
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + pages, device="cuda").cumsum(0)[:-1]
    at = first[:, None] + torch.arange(width, device="cuda")[None]
    live = torch.arange(width, device="cuda")[None] < torch.tensor(pages, device="cuda")[:, None]
    table = torch.where(live, perm[at.clamp(max=n_pages - 1)], torch.full_like(perm[:1], -1)).contiguous()
    s = dict(case=c, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    s["k_scale"] = s["v_scale"] = None
    if c["cache"] == "e4m3":
        s["k_scale"] = 0.05 + 0.02 * torch.rand(H, generator=g, device="cuda")
        s["v_scale"] = 0.05 + 0.02 * torch.rand(H, generator=g, device="cuda")
    if c["op"] == "select":
        # the key bounds of the pages, from keys around each page's mean: min and max of ps normal values
        mid = torch.randn((n_pages, H, D), generator=g, device="cuda") * 0.5
        w = math.sqrt(2 * math.log(ps + 1))
        lo = mid - w * (0.7 + 0.6 * torch.rand((n_pages, H, D), generator=g, device="cuda"))
        hi = mid + w * (0.7 + 0.6 * torch.rand((n_pages, H, D), generator=g, device="cuda"))
        f = 16 if c["cache"] == "e4m3" else 1
        s["bounds"] = (torch.stack([lo, hi], 2) * f).to(DTYPES[c["cache"]])
        s["k"] = s["v"] = None
    else:
        s["k"], s["v"] = _pool(g, c, n_pages), _pool(g, c, n_pages)
        s["bounds"] = None
    q = torch.randn((B, Hq, D), generator=g, device="cuda")
    s["q"] = q.to(act)
    if c["op"] == "append":
        n = sum(rows) + c["pad"]
        s["offsets"] = None if c["rows"] == 1 and not c["pad"] else torch.tensor(
            [0] + rows, device="cuda").cumsum(0).to(torch.int32)
        s["n_live"] = sum(rows)
        # one projection's output: q | k | v side by side in a row, the operators get views of it
        qkv = torch.randn((n, (Hq + 2 * H) * D), generator=g, device="cuda").to(act).view(n, Hq + 2 * H, D)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["q_out"] = torch.zeros((n, Hq, D), dtype=act, device="cuda")
        R = c["rotary"]
        s["rope"] = None
        if R:
            pos = torch.arange(max(1, max(t + r for t, r in zip(lens, rows))), dtype=torch.float64, device="cuda")
            freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
            ang = pos[:, None] * freq[None]
            s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        if c["bounds"]:  # of the keys that are there; a page's place behind the request's last token holds nothing yet
            fill = torch.zeros(n_pages, dtype=torch.long, device="cuda")
            full = (torch.tensor(lens, device="cuda")[:, None] - torch.arange(width, device="cuda")[None] * ps).clamp(0, ps)
            fill[table.long().clamp(min=0)[live]] = full[live]
            k = s["k"].float()
            there = (torch.arange(ps, device="cuda")[None] < fill[:, None])[:, :, None, None]
            lo = torch.where(there, k, torch.full_like(k, 448.0)).amin(1)
            hi = torch.where(there, k, torch.full_like(k, -448.0)).amax(1)
            s["bounds"] = torch.stack([lo, hi], 2).to(DTYPES[c["cache"]])
            del k, lo, hi
    if c["op"] == "sparse":
        s["sel"] = _random_selection(g, c, lens)
    if own:
        from quantized_cross_loop_gb300 import kvq

        s["cache"] = kvq.PagedCache(page_size=ps, n_heads=H, k=s["k"], v=s["v"], key_bounds=s["bounds"],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"])
        s["workspace"] = None if c["op"] == "append" else torch.empty(
            s["cache"].workspace_bytes(B, Hq, width), dtype=torch.uint8, device="cuda")
    return s


def _random_selection(g, c, lens):
    """Per request and KV head: the last page and random others, ascending, -1 behind them."""
    B, H, n = c["B"], c["H"], c["nsel"]
    pages = torch.tensor([_cdiv(t, c["ps"]) for t in lens], device="cuda")
    width = max(int(pages.max()), n)
    key = torch.rand((B, H, width), generator=g, device="cuda")
    i = torch.arange(width, device="cuda")
    key = torch.where(i == pages[:, None, None] - 1, torch.full_like(key, 2.0), key)
    key = torch.where(i < pages[:, None, None], key, torch.full_like(key, -1.0))
    top = key.topk(n, dim=2)
    at = torch.where(top.values >= 0, top.indices, torch.full_like(top.indices, 1 << 30)).sort(2).values
    return torch.where(at < (1 << 30), at, torch.full_like(at, -1)).to(torch.int32).contiguous()


# ------------------------------------------------------------------ one pass


def run(state):
    s = state
    c = s["case"]
    if own:
        from quantized_cross_loop_gb300 import kvq

        if c["op"] == "append":
            kvq.kvq_paged_append(s["cache"], s["table"], s["lens"], s["k_new"], s["v_new"], offsets=s["offsets"],
                                 q=s["q"], q_out=s["q_out"], rope=s["rope"], interleaved=c["inter"])
            return _written(s)
        if c["op"] == "attn":
            lse = torch.empty((c["B"], c["Hq"]), device="cuda")
            out = kvq.kvq_paged_decode_attn(s["cache"], s["table"], s["lens"], s["q"], lse=lse,
                                            workspace=s["workspace"])
            return {"out": out, "lse": lse}
        if c["op"] == "select":
            return {"sel": kvq.kvq_paged_select(s["cache"], s["table"], s["lens"], s["q"], c["nsel"],
                                                n_first=c["nfirst"], n_last=c["nlast"], workspace=s["workspace"])}
        lse = torch.empty((c["B"], c["Hq"]), device="cuda")
        out = kvq.kvq_paged_sparse_attn(s["cache"], s["table"], s["lens"], s["q"], s["sel"], lse=lse,
                                        workspace=s["workspace"])
        return {"out": out, "lse": lse}
    if c["op"] == "append":
        _plain_append(s)
        return _written(s)
    if c["op"] == "select":
        return {"sel": _plain_select(s)}
    out, lse = _plain_attention(s)
    return {"out": out, "lse": lse}


def _written(s):
    """What an append writes: the pools, the key bounds, the rotated queries (all of them the caller's own buffers)."""
    r = {"k": s["k"], "v": s["v"], "q": s["q_out"]}
    if s["bounds"] is not None:
        r["bounds"] = s["bounds"]
    return r


# ------------------------------------------------------------------ the plain forms


def _plain_rotate(x, s, pos):
    c = s["case"]
    R = c["rotary"]
    x = x.float()
    if not R:
        return x
    cs = s["rope"][pos]
    cos, sin = cs[:, None, :R // 2], cs[:, None, R // 2:]
    y = x.clone()
    if c["inter"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2], y[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_append(s):
    c = s["case"]
    ps, n = c["ps"], s["n_live"]
    row = torch.arange(n, device="cuda")
    if s["offsets"] is None:
        req, pos = row, s["lens"].long()
    else:
        off = s["offsets"].long()
        req = torch.searchsorted(off[1:], row, right=True)
        pos = s["lens"].long()[req] + row - off[req]
    page, slot = s["table"].long()[req, pos // ps], pos % ps
    k, v = _plain_rotate(s["k_new"][:n], s, pos), s["v_new"][:n].float()
    s["q_out"][:n] = _plain_rotate(s["q"][:n], s, pos).to(s["q_out"].dtype)
    if s["k_scale"] is not None:
        k = (k / s["k_scale"][None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"][None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    k = k.to(s["k"].dtype)
    s["k"].view(_bits(k))[page, slot] = k.view(_bits(k))
    v = v.to(s["v"].dtype)
    s["v"].view(_bits(v))[page, slot] = v.view(_bits(v))
    if s["bounds"] is not None:
        # bounds that were there count for pages that held tokens before; the new keys join them
        fresh = torch.zeros(s["k"].shape[0], dtype=torch.bool, device="cuda")
        fresh[page[slot == 0]] = True
        b = s["bounds"].float()
        lo = torch.where(fresh[:, None, None], torch.full_like(b[:, :, 0], math.inf), b[:, :, 0])
        hi = torch.where(fresh[:, None, None], torch.full_like(b[:, :, 1], -math.inf), b[:, :, 1])
        at = page[:, None, None].expand(-1, c["H"], D)
        lo = lo.scatter_reduce(0, at, k.float(), "amin")
        hi = hi.scatter_reduce(0, at, k.float(), "amax")
        new = torch.stack([lo, hi], 2).to(s["bounds"].dtype)
        s["bounds"].view(_bits(new)).copy_(new.view(_bits(new)))


def _bits(t):
    return torch.uint8 if t.element_size() == 1 else torch.int16


def _plain_attention(s):
    c = s["case"]
    B, H, Hq, ps = c["B"], c["H"], c["Hq"], c["ps"]
    P = s["table"].shape[1]
    if c["op"] == "sparse":  # [B, H, selected pages]: the tokens of each
        page = s["sel"].long()
        pos = page[..., None] * ps + torch.arange(ps, device="cuda")
        live = (page[..., None] >= 0) & (pos < s["lens"].long()[:, None, None, None])
        phys = torch.gather(s["table"].long(), 1, page.clamp(0, P - 1).reshape(B, -1)).view(B, H, -1).clamp(min=0)
        head = torch.arange(H, device="cuda")[None, :, None]
        k, v = (x.view(_bits(x)).transpose(1, 2)[phys, head].view(x.dtype).float().flatten(2, 3) for x in (s["k"], s["v"]))
        live = live.flatten(2, 3)
    else:
        phys = s["table"].long().clamp(min=0)
        k, v = (x.view(_bits(x))[phys].view(x.dtype).float().flatten(1, 2).transpose(1, 2) for x in (s["k"], s["v"]))
        live = (torch.arange(P * ps, device="cuda")[None] < s["lens"].long()[:, None])[:, None]
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][None, :, None, None], v * s["v_scale"][None, :, None, None]
    q = s["q"].float().view(B, H, Hq // H, D)
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = torch.where(live[:, :, None], x, torch.full_like(x, -math.inf))
    v = torch.where(live[..., None], v, torch.zeros_like(v))
    m = x.amax(3, keepdim=True)
    p = (x - torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp()
    l = p.sum(3, keepdim=True)
    out = (p @ v) / torch.where(l == 0, torch.ones_like(l), l)
    lse = torch.where(l == 0, torch.full_like(l, -math.inf), m + l.log())
    return out.reshape(B, Hq, D), lse.reshape(B, Hq)


def _plain_select(s):
    c = s["case"]
    B, H, Hq, ps, n = c["B"], c["H"], c["Hq"], c["ps"], c["nsel"]
    q = s["q"].double().view(B, H, Hq // H, D)
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    pages = (s["lens"].long() + ps - 1) // ps
    i = torch.arange(s["table"].shape[1], device="cuda")
    b = s["bounds"].view(_bits(s["bounds"]))[s["table"].long().clamp(min=0)].view(s["bounds"].dtype).double()
    score = (b[:, :, :, 1] * up[:, None]).sum(3) + (b[:, :, :, 0] * down[:, None]).sum(3)  # [B, P, H]
    must = (i < c["nfirst"]) | (i >= pages[:, None] - c["nlast"])
    score = torch.where(must[..., None], torch.full_like(score, math.inf), score)
    live = (i < pages[:, None])[..., None]
    order = torch.where(live, score, torch.full_like(score, -math.inf)).transpose(1, 2)
    top = order.sort(dim=2, descending=True, stable=True).indices[..., :n]
    top = torch.where(top < pages[:, None, None], top, torch.full_like(top, 1 << 30)).sort(2).values
    sel = torch.full((B, H, n), -1, dtype=torch.int32, device="cuda")
    sel[..., :top.shape[2]] = torch.where(top < (1 << 30), top, torch.full_like(top, -1)).to(torch.int32)
    return sel


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    c = case
    if c["op"] == "select":
        return None  # whole numbers: the order of the scores, which run() takes in 64 bits already
    s = prepare(c, seed)
    lens = _lengths(c)
    if c["op"] == "append":
        return _exact_append(s, lens)
    return _exact_attention(s, lens)


def _exact_append(s, lens):
    c = s["case"]
    ps, R, H = c["ps"], c["rotary"], c["H"]
    k, v, q = s["k"].double(), s["v"].double(), s["q_out"].double()
    bounds = None if s["bounds"] is None else s["bounds"].double()
    # the table holds the angles' cosines and sines in 32 bits: they are inputs
    row = 0
    for b, n in enumerate(_new_rows(c)):
        for at in range(lens[b] // ps, _cdiv(lens[b] + n, ps) if n else 0):  # the pages that get tokens
            a, e = max(lens[b], at * ps), min(lens[b] + n, (at + 1) * ps)
            r = slice(row + a - lens[b], row + e - lens[b])
            kn, qn, vn = s["k_new"][r].double(), s["q"][r].double(), s["v_new"][r].double()
            if R:
                z = torch.complex(*s["rope"][a:e].double().unsqueeze(1).chunk(2, dim=2))
                for x in (kn, qn):
                    if c["inter"]:
                        w = torch.complex(x[..., :R].unflatten(2, (R // 2, 2))[..., 0].contiguous(),
                                          x[..., :R].unflatten(2, (R // 2, 2))[..., 1].contiguous()) * z
                        x[..., :R] = torch.view_as_real(w).flatten(2)
                    else:
                        w = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * z
                        x[..., :R] = torch.cat([w.real, w.imag], 2)
            if s["k_scale"] is not None:
                kn = (kn / s["k_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
                vn = (vn / s["v_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            page = int(s["table"][b, at])
            k[page, a - at * ps:e - at * ps], v[page, a - at * ps:e - at * ps], q[r] = kn, vn, qn
            if bounds is not None:
                lo, hi = kn.amin(0), kn.amax(0)
                if a > at * ps:
                    lo, hi = torch.minimum(lo, bounds[page, :, 0]), torch.maximum(hi, bounds[page, :, 1])
                bounds[page, :, 0], bounds[page, :, 1] = lo, hi
        row += n
    return {"k": k, "v": v, "q": q, "bounds": bounds} if bounds is not None else {"k": k, "v": v, "q": q}


def _exact_attention(s, lens):
    c = s["case"]
    H, Hq, ps = c["H"], c["Hq"], c["ps"]
    g = Hq // H
    out = torch.zeros((c["B"], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    kb, vb = s["k"].view(_bits(s["k"])), s["v"].view(_bits(s["v"]))
    chosen = s["sel"].tolist() if c["op"] == "sparse" else None
    for b, T in enumerate(lens):
        if T == 0:
            continue
        table = s["table"][b].long()
        for h in range(H):
            if chosen is None:
                t = torch.arange(T, device="cuda")
            else:
                p = torch.tensor([x for x in chosen[b][h] if x >= 0], device="cuda")
                t = (p[:, None] * ps + torch.arange(ps, device="cuda")).flatten()
                t = t[t < T]
            page, slot = table[t // ps], t % ps
            k = kb[page, slot, h].view(s["k"].dtype).double()
            v = vb[page, slot, h].view(s["v"].dtype).double()
            if s["k_scale"] is not None:
                k, v = k * float(s["k_scale"][h]), v * float(s["v_scale"][h])
            x = s["q"][b, h * g:(h + 1) * g].double() @ k.T / math.sqrt(D)
            out[b, h * g:(h + 1) * g] = torch.softmax(x, 1) @ v
            lse[b, h * g:(h + 1) * g] = torch.logsumexp(x, 1)
    return {"out": out, "lse": lse}
