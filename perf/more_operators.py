"""Cases and plain forms of attention and its cache: attention over whole prompts
of packed sequences, attention of one new token over a paged cache, the write of
new keys and values into the pages (with the rotary embedding, and as e4m3 where
the cache is), and the pages themselves: forked, reserved, freed and compacted.

Each operator has a plain form in elementary torch operations and the calls a
program makes of this package; `own` chooses between the two.

A cache of one layer is [pages, kv heads, page, dim]; row r of a table lists the
pages of sequence r in order, and refs counts the sequences that hold a page.
8-bit caches are e4m3 with one fp32 scale for each head of each token, max(m,
1e-30) / 448 for a largest magnitude of m.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 1e-30


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a handful of short prompts that arrive together: the smallest call, all latency
        {"name": "prefill-short-61", "op": "prefill", "seqs": 5, "tokens": 61, "past": 0, "heads": 16, "kv_heads": 16,
         "dim": 64, "dtype": "f16", "causal": True, "mix": 1},
        # an ordinary batch of prompts of different lengths, packed
        {"name": "prefill-packed-4099", "op": "prefill", "seqs": 11, "tokens": 4099, "past": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "causal": True, "mix": 2},
        # the next chunk of a long prompt, behind the keys of the chunks before it, wide heads
        {"name": "prefill-chunk-1021", "op": "prefill", "seqs": 1, "tokens": 1021, "past": 7170, "heads": 16,
         "kv_heads": 2, "dim": 256, "dtype": "bf16", "causal": True, "mix": 3},
        # the longest prompt the block is run at
        {"name": "prefill-long-16384", "op": "prefill", "seqs": 1, "tokens": 16384, "past": 0, "heads": 16,
         "kv_heads": 4, "dim": 128, "dtype": "bf16", "causal": True, "mix": 4},
        # one user at the start of an answer: latency
        {"name": "decode-short-1", "op": "decode", "seqs": 1, "longest": 77, "heads": 16, "kv_heads": 2, "dim": 256,
         "dtype": "bf16", "cache": "same", "page": 16, "mix": 5},
        # one user with a long document: a single sequence has to fill the card
        {"name": "decode-long-1", "op": "decode", "seqs": 1, "longest": 131072, "heads": 32, "kv_heads": 4, "dim": 128,
         "dtype": "bf16", "cache": "same", "page": 64, "mix": 6},
        # a serving batch of ragged lengths
        {"name": "decode-batch-64", "op": "decode", "seqs": 64, "longest": 8192, "heads": 32, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "cache": "same", "page": 64, "mix": 7},
        # a large serving batch over an 8-bit cache
        {"name": "decode-e4m3-256", "op": "decode", "seqs": 256, "longest": 3001, "heads": 32, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "cache": "e4m3", "page": 32, "mix": 8},
        # one token of every sequence of a serving batch into an 8-bit cache
        {"name": "append-decode-64", "op": "append", "seqs": 64, "tokens": 64, "past": 1000, "heads": 32,
         "kv_heads": 8, "dim": 128, "rotary": 128, "interleaved": False, "dtype": "bf16", "cache": "e4m3", "page": 64,
         "prompt": False, "mix": 9},
        # the keys and values of packed prompts, half of each head rotated
        {"name": "append-prompts-16381", "op": "append", "seqs": 9, "tokens": 16381, "past": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "rotary": 64, "interleaved": False, "dtype": "bf16", "cache": "same", "page": 64,
         "prompt": True, "mix": 10},
        # eight answers each to eight prompts: the samples fork from their prompt, get room, and end
        {"name": "pages-fork-64", "op": "pages", "action": "fork", "rows": 64, "parents": 8, "longest": 1500,
         "layers": 8, "kv_heads": 8, "dim": 128, "page": 64, "mix": 11},
        # a cache after many requests have come and gone, packed to its low pages
        {"name": "pages-compact-1024", "op": "pages", "action": "compact", "rows": 96, "parents": 0, "longest": 900,
         "layers": 8, "kv_heads": 8, "dim": 128, "page": 32, "mix": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "decode", "append", "pages"])
    dim = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    mix = rng.randrange(1 << 30)
    while True:
        kv_heads, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 4, 5, 8, 16])
        if kv_heads * group <= 64:
            break
    heads = kv_heads * group
    if op == "prefill":
        while True:
            tokens = _log_int(rng, 1, 16384)
            case = {"op": op, "seqs": _log_int(rng, 1, min(tokens, 64)), "tokens": tokens,
                    "past": rng.choice([0, 0, _log_int(rng, 1, 8192)]), "heads": heads, "kv_heads": kv_heads,
                    "dim": dim, "dtype": dtype, "causal": rng.random() < 0.8, "mix": mix}
            if work(case)["flops"] <= work(listed()[3])["flops"]:
                return case
    if op == "decode":
        cache = rng.choice(["same", "same", "e4m3"])
        while True:
            seqs, longest = _log_int(rng, 1, 256), _log_int(rng, 1, 131072)
            if seqs * longest * kv_heads * dim <= 64 * 8192 * 8 * 128:
                return {"op": op, "seqs": seqs, "longest": longest, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                        "dtype": dtype, "cache": cache, "page": rng.choice([16, 32, 64, 128]), "mix": mix}
    if op == "append":
        prompt = rng.random() < 0.5
        while True:
            seqs = _log_int(rng, 1, 64)
            tokens = max(seqs, _log_int(rng, 1, 16384)) if prompt else seqs
            past = rng.choice([0, _log_int(rng, 1, 1000)])
            if (tokens * (heads + 2 * kv_heads) + 2 * seqs * past * kv_heads) * dim <= 16384 * 48 * 128:
                return {"op": op, "seqs": seqs, "tokens": tokens, "past": past, "heads": heads, "kv_heads": kv_heads,
                        "dim": dim, "rotary": rng.choice([dim, dim, dim // 2, dim // 4]),
                        "interleaved": rng.random() < 0.3, "dtype": dtype,
                        "cache": rng.choice(["same", "e4m3"]), "page": rng.choice([16, 32, 64, 128]),
                        "prompt": prompt, "mix": mix}
    action, page = rng.choice(["fork", "compact"]), rng.choice([16, 32, 64])
    while True:
        rows, longest, layers = _log_int(rng, 4, 96), _log_int(rng, 1, 1500), rng.choice([1, 2, 4, 8])
        kv_heads = rng.choice([1, 2, 4, 8])
        if rows * (longest + 2 * page) * layers * kv_heads * dim <= 96 * 964 * 8 * 8 * 128:
            return {"op": op, "action": action, "rows": rows,
                    "parents": _log_int(rng, 1, rows // 2) if action == "fork" else 0, "longest": longest,
                    "layers": layers, "kv_heads": kv_heads, "dim": dim, "page": page, "mix": mix}


_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _split(mix, parts, total, least):
    """total as so many whole numbers of at least `least`, of quite different sizes."""
    r = random.Random(mix)
    weights = [math.exp(r.gauss(0.0, 0.8)) for _ in range(parts)]
    free, whole = total - least * parts, sum(weights)
    out = [least + int(free * w / whole) for w in weights]
    out[0] += total - sum(out)
    return out


def _prompt_lengths(case):
    """Queries and keys of every sequence."""
    new = _split(case["mix"], case["seqs"], case["tokens"], 1)
    past = _split(case["mix"] + 1, case["seqs"], case["past"], 0)
    return new, [n + p for n, p in zip(new, past)]


def _cache_lengths(case):
    """Cached tokens of every sequence; one is the longest."""
    r = random.Random(case["mix"])
    lens = [1 + int(case["longest"] * r.random()) for _ in range(case["seqs"])]
    lens = [min(n, case["longest"]) for n in lens]
    lens[-1] = case["longest"]
    return lens


def _append_lengths(case):
    """New and earlier tokens of every sequence."""
    r = random.Random(case["mix"] + 1)
    return (_split(case["mix"], case["seqs"], case["tokens"], 1),
            [r.randint(0, case["past"]) for _ in range(case["seqs"])])


def _row_lengths(case):
    """Cached tokens of every row of a table of pages: fork: the parents', then none;
    compact: 0 where the request has ended."""
    r = random.Random(case["mix"])
    if case["action"] == "fork":
        return [r.randint(1, case["longest"]) for _ in range(case["parents"])] + \
            [0] * (case["rows"] - case["parents"])
    return [r.randint(1, case["longest"]) if r.random() < 0.5 else 0 for _ in range(case["rows"])]


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case)
    {"prefill": _prepare_prefill, "decode": _prepare_decode, "append": _prepare_append,
     "pages": _prepare_pages}[case["op"]](case, seed, gen, dev, s)
    return s


def _queries(gen, shape, dev):
    return 1.5 * torch.randn(shape, generator=gen, device=dev)


def _keys(gen, shape, dev):
    """Keys as a model has them: a few channels far from zero, whatever the token."""
    k = torch.randn(shape, generator=gen, device=dev)
    hot = torch.randint(0, shape[-1], (max(1, shape[-1] // 32),), generator=gen, device=dev)
    k[..., hot] += 3.0
    return k


def _int32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _prepare_prefill(case, seed, gen, dev, s):
    """q, k and v as a projection leaves them: slices of one matrix's rows."""
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    new, keys = _prompt_lengths(case)
    dt = _DTYPES[case["dtype"]]
    if case["past"]:
        s["q"] = _queries(gen, (sum(new), H, D), dev).to(dt)
        kv = torch.empty((sum(keys), 2 * Hk, D), dtype=dt, device=dev)
        k, v = kv[:, :Hk], kv[:, Hk:]
    else:
        qkv = torch.empty((sum(new), H + 2 * Hk, D), dtype=dt, device=dev)
        s["q"], k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        s["q"].copy_(_queries(gen, (sum(new), H, D), dev))
    k.copy_(_keys(gen, (sum(keys), Hk, D), dev))
    v.copy_(torch.randn((sum(keys), Hk, D), generator=gen, device=dev))
    s["k"], s["v"] = k, v
    s["new"], s["keys"] = new, keys
    s["starts"] = _int32([sum(new[:i]) for i in range(len(new) + 1)], dev)
    s["k_starts"] = _int32([sum(keys[:i]) for i in range(len(keys) + 1)], dev)


def _tables(lens, page, width, n_pages, seed, dev):
    """Pages of every sequence, in no order; -1 behind the last."""
    free = list(range(n_pages))
    random.Random(seed).shuffle(free)
    rows = []
    for n in lens:
        need = -(-n // page)
        rows.append(free[:need] + [-1] * (width - need))
        free = free[need:]
    return _int32(rows, dev)


def _cache(gen, shape, dt, e4m3, keys, dev):
    """Pages that hold earlier tokens, and their scales."""
    x = _keys(gen, shape, dev) if keys else torch.randn(shape, generator=gen, device=dev)
    if not e4m3:
        return x.to(dt), None
    return _to_e4m3(x)


def _to_e4m3(x):
    m = x.abs().amax(dim=-1).clamp(min=AMAX_FLOOR)
    return (x * (E4M3_MAX / m)[..., None]).to(torch.float8_e4m3fn), m / E4M3_MAX


def _prepare_decode(case, seed, gen, dev, s):
    B, H, Hk, D, P = case["seqs"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens = _cache_lengths(case)
    width = -(-case["longest"] // P)
    n_pages = sum(-(-n // P) for n in lens) + 3
    dt = _DTYPES[case["dtype"]]
    s["q"] = _queries(gen, (B, H, D), dev).to(dt)
    shape, e4m3 = (n_pages, Hk, P, D), case["cache"] == "e4m3"
    s["k_cache"], s["k_scales"] = _cache(gen, shape, dt, e4m3, True, dev)
    s["v_cache"], s["v_scales"] = _cache(gen, shape, dt, e4m3, False, dev)
    s["tables"] = _tables(lens, P, width, n_pages, seed, dev)
    s["lengths"] = _int32(lens, dev)


def _prepare_append(case, seed, gen, dev, s):
    H, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    new, past = _append_lengths(case)
    T = sum(new)
    dt = _DTYPES[case["dtype"]]
    qkv = torch.empty((T, H + 2 * Hk, D), dtype=dt, device=dev)
    s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    s["q"].copy_(_queries(gen, (T, H, D), dev))
    s["k"].copy_(_keys(gen, (T, Hk, D), dev))
    s["v"].copy_(torch.randn((T, Hk, D), generator=gen, device=dev))
    s["rows"] = _int32([r for r, n in enumerate(new) for _ in range(n)], dev)
    s["positions"] = _int32([p + i for n, p in zip(new, past) for i in range(n)], dev)
    lens = [n + p for n, p in zip(new, past)]
    n_pages = sum(-(-n // P) for n in lens) + 2
    s["tables"] = _tables(lens, P, max(-(-n // P) for n in lens), n_pages, seed, dev)
    shape, e4m3 = (n_pages, Hk, P, D), case["cache"] == "e4m3"
    s["k_cache"], s["k_scales"] = _cache(gen, shape, dt, e4m3, True, dev)
    s["v_cache"], s["v_scales"] = _cache(gen, shape, dt, e4m3, False, dev)
    half = case["rotary"] // 2
    s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(dev)


def _prepare_pages(case, seed, gen, dev, s):
    P, R = case["page"], case["rows"]
    lens = _row_lengths(case)
    need = [-(-n // P) for n in lens]
    r = random.Random(seed)
    if case["action"] == "fork":
        # every child gets a page for its part of the prompt's last one and up to two for what it will write
        grow = [0] * case["parents"] + [r.randint(1, P) for _ in range(R - case["parents"])]
        n_pages = sum(need) + 2 * (R - case["parents"]) + 3
        s["grow"] = _int32(grow, dev)
        s["parent_rows"] = _int32([-1] * case["parents"] + [r.randrange(case["parents"])
                                                        for _ in range(R - case["parents"])], dev)
        s["drop"] = _int32([0] * case["parents"] + [1] * (R - case["parents"]), dev)
        width = max(need) + 2
    else:
        n_pages = 2 * sum(need) + 8
        width = max(need + [1])
    tables = _tables(lens, P, width, n_pages, seed, dev)
    refs = [0] * n_pages
    for row, n in zip(tables.tolist(), need):
        for p in row[:n]:
            refs[p] = 1
    s["refs"] = _int32(refs, dev)
    s["lengths"] = _int32(lens, dev)
    s["tables"] = tables
    if case["action"] == "compact":
        s["new_tables"], s["new_refs"] = torch.empty_like(tables), torch.empty_like(s["refs"])
    shape = (case["layers"], n_pages, case["kv_heads"], P, case["dim"])
    s["pools"] = [torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16) for _ in range(2)]


# ------------------------------------------------------------------ the plain forms
def _plain_prefill(s):
    H, Hk, D = s["heads"], s["kv_heads"], s["dim"]
    G, scale = H // Hk, 1.0 / math.sqrt(s["dim"])
    y = torch.empty((sum(s["new"]), H, D), dtype=s["q"].dtype, device=s["q"].device)
    q0 = k0 = 0
    for n, m in zip(s["new"], s["keys"]):
        k = s["k"][k0:k0 + m].float().permute(1, 2, 0).contiguous()
        v = s["v"][k0:k0 + m].float().transpose(0, 1).contiguous()
        step = max(1, (1 << 28) // (H * m))
        for a in range(0, n, step):
            b = min(n, a + step)
            q = s["q"][q0 + a:q0 + b].float().view(b - a, Hk, G, D).transpose(0, 1).reshape(Hk, (b - a) * G, D)
            x = (torch.matmul(q, k) * scale).view(Hk, b - a, G, m)
            if s["causal"]:
                last = torch.arange(a, b, device=x.device)[:, None, None] + (m - n)
                x = torch.where(torch.arange(m, device=x.device) <= last, x, torch.full_like(x, float("-inf")))
            p = torch.exp(x - x.amax(dim=3, keepdim=True))
            p = (p / p.sum(dim=3, keepdim=True)).view(Hk, (b - a) * G, m)
            part = torch.matmul(p, v).view(Hk, b - a, G, D).transpose(0, 1)
            y[q0 + a:q0 + b] = part.reshape(b - a, H, D).to(y.dtype)
        q0, k0 = q0 + n, k0 + m
    return y


def _gathered(cache, scales, tables):
    """[sequences, kv heads, width x page, dim] in fp32."""
    b, w = tables.shape
    _, Hk, P, D = cache.shape
    at = tables.clamp(min=0).long().reshape(-1)
    x = cache.view(torch.uint8)[at].view(cache.dtype).float() if scales is not None else cache[at].float()
    if scales is not None:
        x = x * scales[at][..., None]
    return x.view(b, w, Hk, P, D).permute(0, 2, 1, 3, 4).reshape(b, Hk, w * P, D)


def _plain_decode(s):
    B, H, Hk, D, P = s["seqs"], s["heads"], s["kv_heads"], s["dim"], s["page"]
    room = s["tables"].shape[1] * P
    y = torch.empty((B, H, D), dtype=s["q"].dtype, device=s["q"].device)
    step = max(1, (1 << 27) // (room * Hk * D))
    for a in range(0, B, step):
        b = min(B, a + step)
        k = _gathered(s["k_cache"], s["k_scales"], s["tables"][a:b])
        v = _gathered(s["v_cache"], s["v_scales"], s["tables"][a:b])
        there = (torch.arange(room, device=k.device) < s["lengths"][a:b, None])[:, None]
        q = s["q"][a:b].float().view(b - a, Hk, H // Hk, D)
        x = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(D)
        x = torch.where(there[:, :, None], x, torch.full_like(x, float("-inf")))
        p = torch.exp(x - x.amax(dim=3, keepdim=True))
        p = p / p.sum(dim=3, keepdim=True)
        v = torch.where(there[..., None], v, torch.zeros_like(v))
        y[a:b] = torch.matmul(p, v).view(b - a, H, D).to(y.dtype)
    return y


def _plain_rotate(x, cos, sin, interleaved):
    """fp32 [tokens, heads, dim] with its first 2 cos.shape[1] channels rotated in pairs."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _plain_append(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _plain_rotate(s["q"].float(), cos, sin, s["interleaved"])
    k = _plain_rotate(s["k"].float(), cos, sin, s["interleaved"])
    P = s["page"]
    page = s["tables"][s["rows"].long(), (s["positions"] // P).long()].long()
    off = (s["positions"] % P).long()
    out = {"q": q.to(s["q"].dtype)}
    if s["prompt"]:
        out["k"] = k.to(s["k"].dtype)
    for name, x in (("k", k), ("v", s["v"].float())):
        cache, scales = s[name + "_cache"], s[name + "_scales"]
        if scales is None:
            cache[page, :, off] = x.to(cache.dtype)
        else:
            codes, scale = _to_e4m3(x)
            cache.view(torch.uint8)[page, :, off] = codes.view(torch.uint8)
            scales[page, :, off] = scale
            out[name + "_scales"] = scales
        out[name + "_cache"] = cache
    return out


def _free_pages(refs, count):
    """The lowest free pages, one for each place of a running count (0 where there is none)."""
    free = torch.nonzero(refs == 0)[:, 0]
    at = (count - 1).clamp(min=0, max=max(free.numel() - 1, 0)).long()
    return free[at], count <= free.numel()


def _plain_fork(s):
    """Children take over their parent's full pages and get a copy of the last, partly filled one; then rows get
    room for more tokens; then rows end."""
    P, tables, lengths, refs = s["page"], s["tables"], s["lengths"], s["refs"]
    R, W = tables.shape
    rows, cols = torch.arange(R, device=refs.device), torch.arange(W, device=refs.device)
    parent = s["parent_rows"].long()
    asked = parent >= 0
    ok = asked & (lengths == 0) & (parent[parent.clamp(min=0)] < 0)
    parent = parent.clamp(min=0)
    n = torch.where(ok, lengths[parent], torch.zeros_like(lengths))
    partly = ok & (n % P != 0)
    page, there = _free_pages(refs, torch.cumsum(partly.int(), 0))
    made = ok & (there | ~partly)
    forked = torch.where(made, partly.int(), torch.where(ok, -2, torch.where(asked, -1, 0)).int())
    held = made[:, None] & (cols < -(-n // P)[:, None])
    copied = held & partly[:, None] & (cols == (n // P)[:, None])
    taken = torch.where(copied, page[:, None].int(), tables[parent])
    tables.copy_(torch.where(held, taken, tables))
    refs.index_add_(0, tables[held].long(), torch.ones_like(tables[held]))
    lengths.copy_(torch.where(made, n, lengths))
    both = made & partly
    src, dst = tables[parent[both], (n // P)[both].long()].long(), page[both]
    for pool in s["pools"]:
        pool[:, dst] = pool[:, src]

    grow = s["grow"]
    have, want = -(-lengths // P), -(-(lengths + grow) // P)
    ok = (grow >= 0) & (want <= W)
    need = torch.where(ok, want - have, torch.zeros_like(want))
    upto = torch.cumsum(need, 0)
    slot = upto[:, None] - need[:, None] + (cols - have[:, None]) + 1
    page, there = _free_pages(refs, slot)
    served = ok & ((upto <= (refs == 0).sum()) | (need == 0))
    fresh = served[:, None] & (cols >= have[:, None]) & (cols < want[:, None])
    tables.copy_(torch.where(fresh, page.int(), tables))
    refs.index_add_(0, tables[fresh].long(), torch.ones_like(tables[fresh]))
    lengths.copy_(torch.where(served, lengths + grow, lengths))
    grown = torch.where(served, need, torch.where(ok, -2, -1)).int()

    gone = (s["drop"] != 0)[:, None] & (cols < -(-lengths // P)[:, None])
    refs.index_add_(0, tables[gone].long(), -torch.ones_like(tables[gone]))
    lengths.copy_(torch.where(s["drop"] != 0, torch.zeros_like(lengths), lengths))
    return {"forked": forked, "grown": grown, "tables": tables, "lengths": lengths, "refs": refs,
            "k_pool": s["pools"][0], "v_pool": s["pools"][1]}


def _plain_compact(s):
    """Pages in use move to the free ones among the lowest, in rising order."""
    P, tables, refs = s["page"], s["tables"], s["refs"]
    used = refs > 0
    live = used.sum()
    at = torch.arange(refs.numel(), device=refs.device)
    src, dst = torch.nonzero(used & (at >= live))[:, 0], torch.nonzero(~used & (at < live))[:, 0]
    for pool in s["pools"]:
        pool[:, dst] = pool[:, src]
    to = at.clone()
    to[src] = dst
    held = torch.arange(tables.shape[1], device=refs.device) < -(-s["lengths"] // P)[:, None]
    s["new_tables"].copy_(torch.where(held, to[tables.clamp(min=0).long()].int(), tables))
    s["new_refs"].copy_(refs)
    s["new_refs"][dst] = refs[src]
    s["new_refs"][src] = 0
    return {"tables": s["new_tables"], "refs": s["new_refs"], "live": live.int().view(1), "k_pool": s["pools"][0],
            "v_pool": s["pools"][1]}


def run(state):
    s, op = state, state["op"]
    if own:
        import ternary_quantized_moe_amd as tq
        if op == "prefill":
            return {"y": tq.attention_prefill(s["q"], s["k"], s["v"], s["starts"], s["k_starts"],
                                              causal=s["causal"])}
        if op == "decode":
            return {"y": tq.attention_decode(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lengths"],
                                             k_scales=s["k_scales"], v_scales=s["v_scales"])}
        if op == "append":
            out = tq.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["tables"], s["rows"], s["positions"],
                               k_scales=s["k_scales"], v_scales=s["v_scales"], q=s["q"], inv_freq=s["inv_freq"],
                               interleaved=s["interleaved"], rotated_k=s["prompt"])
            out.update({n: s[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales") if s[n] is not None})
            return out
        if s["action"] == "fork":
            forked = tq.kv_fork(s["tables"], s["lengths"], s["refs"], s["parent_rows"], s["page"], s["pools"])
            grown = tq.kv_reserve(s["tables"], s["lengths"], s["refs"], s["grow"], s["page"])
            tq.kv_free(s["tables"], s["lengths"], s["refs"], s["drop"], s["page"])
            return {"forked": forked, "grown": grown, "tables": s["tables"], "lengths": s["lengths"],
                    "refs": s["refs"], "k_pool": s["pools"][0], "v_pool": s["pools"][1]}
        tables, refs, live = tq.kv_compact(s["tables"], s["lengths"], s["refs"], s["page"], s["pools"],
                                           new_tables=s["new_tables"], new_refs=s["new_refs"])
        return {"tables": tables, "refs": refs, "live": live, "k_pool": s["pools"][0], "v_pool": s["pools"][1]}
    if op == "prefill":
        return {"y": _plain_prefill(s)}
    if op == "decode":
        return {"y": _plain_decode(s)}
    if op == "append":
        return _plain_append(s)
    return _plain_fork(s) if s["action"] == "fork" else _plain_compact(s)


# ------------------------------------------------------------------ the work
def work(case):
    op = case["op"]
    if op == "pages":
        # the pages that move are read and written; tables, lengths and counts are read and written once
        P, lens = case["page"], _row_lengths(case)
        if case["action"] == "fork":
            r = [n for n in lens if n % P]
            moved = (case["rows"] - case["parents"]) * len(r) / max(1, case["parents"])
        else:
            moved = sum(-(-n // P) for n in lens) / 2
        page = 2 * 2 * case["layers"] * P * case["kv_heads"] * case["dim"]
        return {"bytes": int(2 * moved * page) + 16 * case["rows"] + 8 * sum(-(-n // P) for n in lens), "flops": 0}
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    if op == "prefill":
        new, keys = _prompt_lengths(case)
        pairs = sum(n * m - (n * (n - 1) // 2 if case["causal"] else 0) for n, m in zip(new, keys))
        return {"bytes": 2 * D * (2 * H * sum(new) + 2 * Hk * sum(keys)), "flops": 4 * D * H * pairs}
    size = 2 if case["cache"] == "same" else 1 + 4 / D
    if op == "decode":
        total = sum(_cache_lengths(case))
        return {"bytes": int(2 * total * Hk * D * size) + 4 * case["seqs"] * H * D, "flops": 4 * D * H * total}
    T = case["tokens"]
    return {"bytes": int(T * D * (4 * H + (6 if case["prompt"] else 4) * Hk + 2 * Hk * size)),
            "flops": 3 * T * (H + Hk) * case["rotary"]}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """What run() returns, in 64 bits and not rounded (8-bit values: what they round, the value over its scale)."""
    s = prepare(case, seed)
    return {"prefill": _exact_prefill, "decode": _exact_decode, "append": _exact_append,
            "pages": _exact_pages}[case["op"]](s)


def _attend(q, k, v, hidden):
    """One head in 64 bits; hidden marks the pairs that are not seen."""
    logits = torch.mm(q, k.t().contiguous()) * (q.shape[1] ** -0.5)
    if hidden is not None:
        logits.masked_fill_(hidden, -math.inf)
    return torch.mm(torch.softmax(logits, 1), v)


def _exact_prefill(s):
    H, G = s["heads"], s["heads"] // s["kv_heads"]
    out, starts, k_starts = [], s["starts"].tolist(), s["k_starts"].tolist()
    for i in range(s["seqs"]):
        q = s["q"][starts[i]:starts[i + 1]].double()
        k, v = (s[x][k_starts[i]:k_starts[i + 1]].double() for x in ("k", "v"))
        heads = []
        for h in range(H):
            parts = []
            for a in range(0, q.shape[0], 4096):
                part = q[a:a + 4096, h]
                hidden = None
                if s["causal"]:
                    at = torch.arange(a, a + part.shape[0], device=q.device) + k.shape[0] - q.shape[0]
                    hidden = torch.arange(k.shape[0], device=q.device)[None] > at[:, None]
                parts.append(_attend(part, k[:, h // G].contiguous(), v[:, h // G].contiguous(), hidden))
            heads.append(torch.cat(parts))
        out.append(torch.stack(heads, 1))
    return {"y": torch.cat(out)}


def _values(cache, scales):
    x = cache.double()
    return x if scales is None else x * scales.double()[..., None]


def _exact_decode(s):
    H, G, out = s["heads"], s["heads"] // s["kv_heads"], []
    for b, n in enumerate(s["lengths"].tolist()):
        at = s["tables"][b, : -(-n // s["page"])].long()
        k, v = (_values(s[x + "_cache"].view(torch.uint8)[at].view(s[x + "_cache"].dtype),
                        None if s[x + "_scales"] is None else s[x + "_scales"][at]) for x in ("k", "v"))
        k, v = (x.transpose(0, 1).reshape(s["kv_heads"], -1, s["dim"])[:, :n] for x in (k, v))
        out.append(torch.cat([_attend(s["q"][b, h * G:(h + 1) * G].double(), k[h], v[h], None)
                              for h in range(s["kv_heads"])]))
    return {"y": torch.stack(out)}


def _exact_append(s):
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                       s["positions"].double()[:, None] * s["inv_freq"].double()[None])[:, None]
    half, out, new = s["rotary"] // 2, {}, {"v": s["v"].double()}
    for name in ("q", "k"):
        x = s[name].double()
        first, second = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if s["interleaved"] else \
            (x[..., :half], x[..., half:2 * half])
        z = torch.complex(first.contiguous(), second.contiguous()) * turn
        x = x.clone()
        if s["interleaved"]:
            x[..., 0:2 * half:2], x[..., 1:2 * half:2] = z.real, z.imag
        else:
            x[..., :half], x[..., half:2 * half] = z.real, z.imag
        new[name] = x
    out["q"] = new["q"]
    if s["prompt"]:
        out["k"] = new["k"]
    P = s["page"]
    where = [s["tables"][r, p // P].long() * P + p % P for r, p in ((s["rows"].long(), s["positions"].long()),)][0]
    for name in ("k", "v"):
        cache, scales, x = s[name + "_cache"].double(), s[name + "_scales"], new[name]
        n, Hk, _, D = cache.shape
        flat = cache.transpose(1, 2).reshape(n * P, Hk, D)
        if scales is not None:
            big = x.abs().max(dim=2).values
            unit = torch.where(big < AMAX_FLOOR, torch.full_like(big, AMAX_FLOOR), big) / E4M3_MAX
            x = x / unit[..., None]
            all_units = scales.double().transpose(1, 2).reshape(n * P, Hk)
            all_units[where] = unit
            out[name + "_scales"] = all_units.view(n, P, Hk).transpose(1, 2).contiguous()
        flat[where] = x
        out[name + "_cache"] = flat.view(n, P, Hk, D).transpose(1, 2).contiguous()
    return out


def _exact_pages(s):
    """Pages by a loop over rows and a list of free pages; what the pools hold is copied, so it is exact as it is."""
    P, R = s["page"], s["rows"]
    tables, lengths, refs = (s[x].tolist() for x in ("tables", "lengths", "refs"))
    count = lambda n: -(-n // P)

    def result(values):
        return torch.tensor(values, dtype=torch.int32)
    if s["action"] == "compact":
        live = sum(1 for n in refs if n)
        holes = [p for p in range(live) if not refs[p]]
        moves = dict(zip([p for p in range(live, len(refs)) if refs[p]], holes))
        for row, n in zip(tables, lengths):
            row[:count(n)] = [moves.get(p, p) for p in row[:count(n)]]
        for p, to in moves.items():
            refs[to], refs[p] = refs[p], 0
            for pool in s["pools"]:
                pool[:, to] = pool[:, p]
        return {"tables": result(tables), "refs": result(refs), "live": result([live]), "k_pool": s["pools"][0],
                "v_pool": s["pools"][1]}
    parents = s["parent_rows"].tolist()
    free, forked, grown = [p for p, n in enumerate(refs) if not n], [0] * R, [0] * R
    for r in range(R):
        if parents[r] < 0:
            continue
        n = lengths[parents[r]]
        row = tables[parents[r]][:count(n)]
        if n % P:
            to = free.pop(0)
            for pool in s["pools"]:
                pool[:, to] = pool[:, row[-1]]
            row[-1], forked[r] = to, 1
        for p in row:
            refs[p] += 1
        tables[r][:len(row)], lengths[r] = row, n
    for r, more in enumerate(s["grow"].tolist()):
        a, b = count(lengths[r]), count(lengths[r] + more)
        for c in range(a, b):
            tables[r][c] = free.pop(0)
            refs[tables[r][c]] += 1
        lengths[r], grown[r] = lengths[r] + more, b - a
    for r, gone in enumerate(s["drop"].tolist()):
        if gone:
            for p in tables[r][:count(lengths[r])]:
                refs[p] -= 1
            lengths[r] = 0
    return {"forked": result(forked), "grown": result(grown), "tables": result(tables), "lengths": result(lengths),
            "refs": result(refs), "k_pool": s["pools"][0], "v_pool": s["pools"][1]}
