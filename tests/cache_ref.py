"""Plain 64-bit references of the operators on a paged cache, written token by
token from their definitions, and the inputs that their tests share."""
import math

import torch

from layer_ref import DTYPES, offsets

DEV = "cuda:0"


def pool(pages, page, heads, d, dtype, order, gen):
    """A cache of random values; order: what a page holds together."""
    r = lambda *s: torch.randn(s, generator=gen).to(dtype)
    if order == "token":
        return r(pages, page, heads, d)
    if order == "head":
        return r(pages, heads, page, d).transpose(1, 2)
    if order == "pair":  # the first half of each page's two
        return r(pages, 2, page, heads, d)[:, 0]
    raise ValueError(order)


def second(cache, order, gen):
    """The values' cache beside the keys'."""
    if order == "pair":
        both = cache._base.view(cache.shape[0], 2, *cache.shape[1:])
        return both[:, 1]
    t = torch.randn(cache.shape, generator=gen).to(cache.dtype)
    return t if order == "token" else t.transpose(1, 2).contiguous().transpose(1, 2)


def on_gpu(k, v, order):
    """The caches on the GPU in the same order in memory."""
    if order == "pair":
        both = torch.stack([k, v], 1).to(DEV)
        return both[:, 0], both[:, 1]
    if order == "token":
        return k.to(DEV), None if v is None else v.to(DEV)
    to = lambda t: t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    return to(k), None if v is None else to(v)


def tables(used, shared, page, gen, spare=2, room=1):
    """(page_table, prefix_pages, pages): used[n] and shared pages at random places."""
    pages = sum(used) + shared + spare
    order = torch.randperm(pages, generator=gen).int()
    table = torch.full((len(used), max(used) + room), -1, dtype=torch.int32)
    at = 0
    for n, u in enumerate(used):
        table[n, :u] = order[at: at + u]
        at += u
    return table, order[at: at + shared].contiguous(), pages


def new_places(table, lens, new, page):
    """[(token, session, page or -1, slot)] of every new token."""
    out, t = [], 0
    most = table.shape[1] * page
    for s, n in enumerate(new):
        length = max(0, min(int(lens[s]), most))
        for i in range(n):
            p = length - n + i
            out.append((t, s, int(table[s, p // page]) if p >= 0 else -1, p % page))
            t += 1
    return out


def rotate_ref(x, table, pos, off, inter):
    """x [T, H, d] in 64 bits."""
    rot = table.shape[1]
    half = rot // 2
    i = torch.arange(half)
    a, b = (off + 2 * i, off + 2 * i + 1) if inter else (off + i, off + i + half)
    row = table[pos.long().clamp(0, table.shape[0] - 1)].unsqueeze(1)
    cos, sin = row[..., :half], row[..., half:]
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def held(cache, pages_of, length, page):
    """Tokens 0 .. length of a list of pages, in 64 bits, and which of them have a page."""
    H, d = cache.shape[2:]
    rows = torch.zeros(length, H, d, dtype=torch.float64)
    ok = torch.zeros(length, dtype=torch.bool)
    for j in range(length):
        p = int(pages_of[j // page])
        if 0 <= p < cache.shape[0]:
            rows[j], ok[j] = cache[p, j % page].double(), True
    return rows, ok


def attention_ref(q, k_cache, v_cache, table, lens, prefix_pages, prefix_len, new, scale, dv):
    """(out, lse, weight): weight = sum_j p_j |v_j|, what the bounds scale with."""
    T, Hq, d = q.shape
    H, page = k_cache.shape[2], k_cache.shape[1]
    G = Hq // H
    vals = k_cache[..., :dv] if v_cache is None else v_cache
    out = torch.zeros(T, Hq, dv, dtype=torch.float64)
    wgt, lse = out.clone(), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    P = 0
    if prefix_pages is not None:
        P = max(0, min(int(prefix_len), len(prefix_pages) * page))
    kp, okp = held(k_cache, prefix_pages, P, page)
    vp, _ = held(vals, prefix_pages, P, page)
    t = 0
    for s, n in enumerate(new):
        L = max(0, min(int(lens[s]), table.shape[1] * page))
        ko, oko = held(k_cache, table[s], L, page)
        vo, _ = held(vals, table[s], L, page)
        for i in range(n):
            own = max(0, L - n + i + 1)
            k, v = torch.cat([kp, ko[:own]]), torch.cat([vp, vo[:own]])
            ok = torch.cat([okp, oko[:own]])
            k, v = k[ok], v[ok]
            if len(k):
                z = (k.repeat_interleave(G, 1) * q[t].double()).sum(-1) * scale
                lse[t] = torch.logsumexp(z, 0)
                p = torch.exp(z - lse[t])[..., None]
                out[t] = (p * v.repeat_interleave(G, 1)).sum(0)
                wgt[t] = (p * v.abs().repeat_interleave(G, 1)).sum(0)
            t += 1
    return out, lse, wgt


def attention_inputs(case, seed=0):
    """case: dict(new, lens, prefix, page, hq, h, d, dtype, order, packed, pad); host tensors."""
    g = torch.Generator().manual_seed(seed)
    dt, d, page = DTYPES[case["dtype"]], case["d"], case["page"]
    used = [max(0, -(-n // page)) for n in case["lens"]]
    shared = -(-case["prefix"] // page)
    table, prefix, pages = tables(used, shared, page, g, room=case.get("room", 1))
    k = pool(pages, page, case["h"], d, dt, case["order"], g)
    v = None if d == 576 else second(k, case["order"], g)
    T, pad = sum(case["new"]), case.get("pad", 0)
    wide = torch.randn(T, case["hq"] * d + pad, generator=g).to(dt)
    if pad:
        wide[:, case["hq"] * d:] = float("nan")
    return dict(q=wide, k=k, v=v, table=table, lens=torch.tensor(case["lens"], dtype=torch.int32),
                prefix_pages=prefix if case["prefix"] else None,
                prefix_len=torch.tensor([case["prefix"]], dtype=torch.int32) if case["prefix"] else None,
                cu=offsets(case["new"]) if case["packed"] else None)


def heads_of(wide, hq, d):
    return wide[:, : hq * d].unflatten(1, (hq, d))


def d_v(case):
    return 512 if case["d"] == 576 else case["d"]


def attend(kda, x, case, **kw):
    """The public call on the GPU."""
    to = lambda t: None if t is None else t.to(DEV)
    k, v = on_gpu(x["k"], x["v"], case["order"])
    return kda.prefix_attention(heads_of(to(x["q"]), case["hq"], case["d"]), k, v, to(x["table"]),
                                to(x["lens"]), to(x["prefix_pages"]), to(x["prefix_len"]),
                                to(x["cu"]), output_lse=True, **kw)


def reference(x, case, scale=None):
    return attention_ref(heads_of(x["q"], case["hq"], case["d"]), x["k"], x["v"], x["table"],
                         x["lens"], x["prefix_pages"], x["prefix_len"], case["new"],
                         case["d"] ** -0.5 if scale is None else scale, d_v(case))
