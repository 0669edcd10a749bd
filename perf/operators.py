"""Cases and plain forms of the operators between a residual stream and the
next token: the 8-bit quantizer with one scale per block of 128, the RMS norm
that adds the residual and can write 8 bits, the block-scaled 8-bit product and
the sampler.

Each operator has a plain form in elementary torch operations and the calls a
program makes of this package; `own` chooses between the two.  8-bit values are
e4m3 (largest value 448); the scale of a block whose largest magnitude is m is
max(m, 1e-30) / 448.
"""
import math

import numpy as np
import torch

own = False

GROUP = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-30
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode batch's attention output on its way into the output projection
        {"name": "quantize-rows-64", "op": "quantize", "rows": 64, "cols": 4096, "block_rows": 1, "dtype": "bf16"},
        # an output head quantized once when a model is loaded
        {"name": "quantize-head", "op": "quantize", "rows": 50304, "cols": 2048, "block_rows": 128, "dtype": "bf16"},
        # one token between two sub-layers: the smallest call, all latency
        {"name": "norm-decode-1", "op": "norm", "tokens": 1, "d": 2048, "residual": True, "bf16": False, "fp8": True},
        # a ragged batch that feeds the routed experts (bf16) and an 8-bit projection at once
        {"name": "norm-both-333", "op": "norm", "tokens": 333, "d": 4096, "residual": True, "bf16": True, "fp8": True},
        # the longest prefill the block is run at
        {"name": "norm-prefill-16384", "op": "norm", "tokens": 16384, "d": 2048, "residual": True, "bf16": False,
         "fp8": True},
        # one token through the output head: the weights are the traffic
        {"name": "linear-head-1", "op": "linear", "m": 1, "n": 50304, "k": 2048, "out": "f32"},
        # a decode batch through an attention projection
        {"name": "linear-decode-32", "op": "linear", "m": 32, "n": 4096, "k": 2048, "out": "bf16"},
        # a chunk of a prompt, neither side a multiple of a tile
        {"name": "linear-ragged-333", "op": "linear", "m": 333, "n": 2561, "k": 4096, "out": "bf16"},
        # a prefill through a dense feed-forward projection
        {"name": "linear-prefill-4096", "op": "linear", "m": 4096, "n": 8192, "k": 4096, "out": "bf16"},
        # one user, the usual filters
        {"name": "sample-1", "op": "sample", "batch": 1, "vocab": 50304, "pad": 0, "dtype": "f32", "filters": "usual"},
        # a serving batch in which every request has settings of its own
        {"name": "sample-mixed-64", "op": "sample", "batch": 64, "vocab": 131072, "pad": 0, "dtype": "f32",
         "filters": "mixed"},
        # bf16 logits of an odd vocabulary in padded rows, cut by probability mass alone
        {"name": "sample-topp-257", "op": "sample", "batch": 257, "vocab": 49157, "pad": 3, "dtype": "bf16",
         "filters": "top_p"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "linear", "linear", "sample"])
    if op == "quantize":
        cols = GROUP * _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, min(65536, 50304 * 2048 // cols))
        return {"op": op, "rows": rows, "cols": cols, "block_rows": rng.choice([1, 128]),
                "dtype": rng.choice(["bf16", "f16"])}
    if op == "norm":
        d = GROUP * _log_int(rng, 1, 64)
        fp8 = rng.random() < 0.7
        return {"op": op, "tokens": _log_int(rng, 1, min(16384, 16384 * 2048 // d)), "d": d,
                "residual": rng.random() < 0.7, "bf16": (not fp8) or rng.random() < 0.3, "fp8": fp8}
    if op == "linear":
        while True:
            m, n, k = _log_int(rng, 1, 4096), _log_int(rng, 64, 50304), GROUP * _log_int(rng, 1, 64)
            if m * n * k <= 4096 * 8192 * 4096 and n * k <= 50304 * 2048 and m * n <= 4096 * 8192:
                return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "f32"])}
    vocab = _log_int(rng, 1000, 200000)
    return {"op": op, "batch": _log_int(rng, 1, min(512, 64 * 131072 // vocab)), "vocab": vocab,
            "pad": rng.choice([0, 0, 1, 7]), "dtype": rng.choice(["f32", "bf16", "f16"]),
            "filters": rng.choice(["usual", "mixed", "top_p", "none"])}


_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the inputs
def _activations(gen, rows, cols, dev):
    """Hidden states as a model has them: unit scale, rows of different size, a few channels 20 times larger."""
    x = torch.randn((rows, cols), generator=gen, device=dev)
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device=dev))
    hot = torch.randint(0, cols, (max(1, cols // 256),), generator=gen, device=dev)
    x[:, hot] *= 20.0
    return x


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        rows, cols, br = case["rows"], case["cols"], case["block_rows"]
        x = _activations(gen, rows, cols, dev) if br == 1 else torch.randn((rows, cols), generator=gen,
                                                                           device=dev) / math.sqrt(cols)
        s["x"] = x.to(_DTYPES[case["dtype"]])
    elif op == "norm":
        T, d = case["tokens"], case["d"]
        s["x"] = _activations(gen, T, d, dev).bfloat16()
        s["residual"] = (4.0 * _activations(gen, T, d, dev)).bfloat16() if case["residual"] else None
        s["weight"] = 1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["a_scales"] = _quantize(_activations(gen, m, k, dev), 1)
        w = torch.randn((n, k), generator=gen, device=dev) / math.sqrt(k)
        s["w"], s["w_scales"] = _quantize(w, GROUP)
        s["y"] = torch.empty((m, n), dtype=_DTYPES[case["out"]], device=dev)
    else:
        _prepare_sample(case, gen, dev, s)
    return s


def _prepare_sample(case, gen, dev, s):
    B, V, ld = case["batch"], case["vocab"], case["vocab"] + case["pad"]
    spread = 1.5 + 2.0 * torch.rand((B, 1), generator=gen, device=dev)
    logits = torch.randn((B, ld), generator=gen, device=dev) * spread
    likely = torch.randint(0, V, (B, 8), generator=gen, device=dev)
    logits.scatter_add_(1, likely, 6.0 * torch.rand((B, 8), generator=gen, device=dev))
    banned = torch.randint(0, V, (B, 16), generator=gen, device=dev)
    logits.scatter_(1, banned, float("-inf"))
    s["logits"] = logits.to(_DTYPES[case["dtype"]])[:, :V]

    def one_of(values, dtype):
        table = torch.tensor(values, dtype=dtype, device=dev)
        return table[torch.randint(0, len(values), (B,), generator=gen, device=dev)].contiguous()

    f = case["filters"]
    s["temperature"] = one_of([0.0, 0.6, 0.8, 1.0, 1.0, 1.3] if f == "mixed" else [1.0] if f == "none" else [0.8, 1.0],
                              torch.float32)
    s["top_k"] = one_of([0, 0, 1, 20, 50, 500] if f == "mixed" else [50] if f == "usual" else [0], torch.int32)
    s["top_p"] = one_of([1.0, 1.0, 0.95, 0.8] if f == "mixed" else [0.9, 0.95] if f in ("usual", "top_p") else [1.0],
                        torch.float32)
    s["min_p"] = one_of([0.0, 0.0, 0.05] if f == "mixed" else [0.0], torch.float32)
    s["u"] = torch.rand(B, generator=gen, device=dev)


# ------------------------------------------------------------------ the plain forms
def _block_amax(x, block_rows):
    """Largest magnitude of every block of block_rows rows and 128 columns, [ceil(rows / block_rows), cols / 128]."""
    rows, cols = x.shape
    pad = -rows % block_rows
    if pad:
        x = torch.cat([x, x.new_zeros((pad, cols))])
    return x.abs().view(-1, block_rows, cols // GROUP, GROUP).amax(dim=(1, 3))


def _spread(s, block_rows, rows):
    """One value per block -> one value per element."""
    return s.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(GROUP, 1)


def _quantize(x, block_rows):
    """fp32 -> e4m3 and its scales."""
    a = _block_amax(x, block_rows).clamp(min=AMAX_FLOOR)
    q = (x * _spread(E4M3_MAX / a, block_rows, x.shape[0])).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), a / E4M3_MAX


def _plain_norm(s):
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["sum"] = h.bfloat16()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["weight"]
    if s["bf16"]:
        out["y"] = y.bfloat16()
    if s["fp8"]:
        out["q"], out["scales"] = _quantize(y, 1)
    return out


def _plain_linear(s):
    m, n = s["m"], s["n"]
    a = s["a"].float() * _spread(s["a_scales"], 1, m)
    w = s["w"].float() * _spread(s["w_scales"], GROUP, n)
    return torch.matmul(a, w.t()).to(s["y"].dtype)


def _plain_sample(s):
    x = s["logits"].double() + 0.0
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x)
    B, V = x.shape
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    top = x[:, :1]
    t = s["temperature"].double()[:, None]
    greedy = ~(t > 0)
    w = torch.where(x == top, torch.ones_like(x), torch.exp((x - top) / torch.where(greedy, torch.ones_like(t), t)))
    at = torch.arange(V, device=x.device)[None]
    k = s["top_k"].long()[:, None]
    k = torch.where((k <= 0) | (k > V), torch.full_like(k, V), k)
    keep = at < torch.where(greedy, torch.ones_like(k), k)
    w = torch.where(keep, w, torch.zeros_like(w))
    p = s["top_p"].double()[:, None]
    c = torch.cumsum(w, 1)
    before = torch.cat([torch.zeros_like(top), c[:, :-1]], 1)
    keep = keep & ((before < p * c[:, -1:]) | ~(p < 1) | (at == 0))
    mp = s["min_p"].double()[:, None]
    keep = keep & ((w >= mp) | ~(mp > 0) | (x == top))
    w = torch.where(keep, w, torch.zeros_like(w))
    c = torch.cumsum(w, 1)
    total = c[:, -1:]
    place = (c <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    place = torch.minimum(place, (w > 0).sum(1, keepdim=True) - 1).clamp(min=0)
    none = (top == float("-inf"))[:, 0]
    tokens = torch.where(none, torch.full_like(place[:, 0], -1), order.gather(1, place)[:, 0])
    probs = torch.where(none, torch.zeros_like(total[:, 0]), (w.gather(1, place) / total)[:, 0])
    return {"tokens": tokens.to(torch.int32), "probs": probs.float()}


def run(state):
    s, op = state, state["op"]
    if own:
        import ternary_quantized_moe_amd as tq
        if op == "quantize":
            q, scales = tq.fp8_quantize(s["x"], s["block_rows"])
            return {"q": q, "scales": scales}
        if op == "norm":
            return tq.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], bf16=s["bf16"], fp8=s["fp8"])
        if op == "linear":
            return {"y": tq.fp8_linear(s["a"], s["a_scales"], s["w"], s["w_scales"], y=s["y"])}
        tokens, probs = tq.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                  top_p=s["top_p"], min_p=s["min_p"])
        return {"tokens": tokens, "probs": probs}
    if op == "quantize":
        q, scales = _quantize(s["x"].float(), s["block_rows"])
        return {"q": q, "scales": scales}
    if op == "norm":
        return _plain_norm(s)
    if op == "linear":
        return {"y": _plain_linear(s)}
    return _plain_sample(s)


# ------------------------------------------------------------------ the work
def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        blocks = -(-case["rows"] // case["block_rows"]) * (case["cols"] // GROUP)
        return {"bytes": 3 * n + 4 * blocks, "flops": 3 * n}
    if op == "norm":
        T, d = case["tokens"], case["d"]
        per = 2 + (4 if case["residual"] else 0) + (2 if case["bf16"] else 0) + (1 + 4 / GROUP if case["fp8"] else 0)
        return {"bytes": T * d * per + 4 * d, "flops": 8 * T * d}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        out = 4 if case["out"] == "f32" else 2
        scales = 4 * (m + -(-n // GROUP)) * (k // GROUP)
        return {"bytes": m * k + n * k + scales + out * m * n, "flops": 2 * m * n * k}
    B, V = case["batch"], case["vocab"]
    return {"bytes": B * V * (4 if case["dtype"] == "f32" else 2) + 28 * B, "flops": 4 * B * V}


# ------------------------------------------------------------------ in 64 bits
def _exact_scales(x, block_rows):
    """Scale of every element's block, and the scales themselves, by a loop over the row blocks."""
    rows, cols = x.shape
    groups = x.abs().reshape(rows, cols // GROUP, GROUP).max(dim=2).values
    if block_rows > 1:
        groups = torch.stack([g.max(dim=0).values for g in torch.split(groups, block_rows)])
    scales = torch.where(groups < AMAX_FLOOR, torch.full_like(groups, AMAX_FLOOR), groups) / E4M3_MAX
    of_row = torch.div(torch.arange(rows, device=x.device), block_rows, rounding_mode="floor")
    return scales[of_row][:, :, None].expand(rows, cols // GROUP, GROUP).reshape(rows, cols), scales


def exact(case, seed):
    """What run() returns, in 64 bits and not rounded (8-bit values: what they round, the value over its scale)."""
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        x = s["x"].double()
        per, scales = _exact_scales(x, case["block_rows"])
        return {"q": x / per, "scales": scales}
    if op == "norm":
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            h = h + s["residual"].double()
            out["sum"] = h
        size = torch.sqrt(torch.sum(h ** 2, 1) / case["d"] + EPS)
        y = s["weight"].double()[None, :] * (h / size[:, None])
        if case["bf16"]:
            out["y"] = y
        if case["fp8"]:
            per, out["scales"] = _exact_scales(y, 1)
            out["q"] = y / per
        return out
    if op == "linear":
        y = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device=s["a"].device)
        rows = torch.arange(case["n"], device=y.device) // GROUP
        for g in range(case["k"] // GROUP):
            at = slice(g * GROUP, (g + 1) * GROUP)
            part = torch.mm(s["a"][:, at].double(), s["w"][:, at].double().t().contiguous())
            y += part * s["a_scales"][:, g].double()[:, None] * s["w_scales"][rows, g].double()[None, :]
        return {"y": y}
    return _exact_sample(s)


def _exact_sample(s):
    logits = s["logits"].double().cpu().numpy()
    host = {k: s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "u")}
    tokens, probs = [], []
    for b, row in enumerate(logits):
        row = np.where(np.isnan(row), -np.inf, row)
        if row.max() == -np.inf:
            tokens.append(-1)
            probs.append(0.0)
            continue
        order = np.argsort(-row, kind="stable")
        t, k = float(host["temperature"][b]), int(host["top_k"][b])
        if not t > 0:
            tokens.append(int(order[0]))
            probs.append(1.0)
            continue
        if 0 < k < len(order):
            order = order[:k]
        z = row[order]
        w = np.where(z == z[0], 1.0, np.exp((z - z[0]) / t))
        p, floor = float(host["top_p"][b]), float(host["min_p"][b])
        if p < 1:
            n = max(1, int(np.searchsorted(np.cumsum(w), p * np.sum(w), side="left")) + 1)
            w = w[:n]
        if floor > 0:
            w = w[w >= min(floor, 1.0)]
        c = np.cumsum(w)
        i = int(np.searchsorted(c, float(host["u"][b]) * c[-1], side="right"))
        i = min(i, int(np.count_nonzero(w > 0)) - 1)
        tokens.append(int(order[i]))
        probs.append(float(w[i] / c[-1]))
    return {"tokens": np.array(tokens, dtype=np.int32), "probs": np.array(probs)}
