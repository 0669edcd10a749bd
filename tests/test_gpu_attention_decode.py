"""GPU parity of attention of one token over a paged cache against the float64 oracle.

The tolerance is that of attention over prompts (tests/test_gpu_attention.py), with two
additions: workers' and waves' shares of a sequence are scaled and added in fp32, each
share by an exponential that is off by d + 2 e, twice: 4 (d + 2 e) A in place of 2 (d + 2
e) A; and of an e4m3 cache the score is multiplied by the key's scale and the weight by
the value's, 2 e S and 2 e A.
"""
import numpy as np
import pytest

from oracle import attention
from test_gpu_attention import BF16, E, F16, host, ints, lse_tolerance, say, tq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Case:
    """Sequences of these lengths over shuffled pages; what no sequence uses is NaN."""

    def __init__(self, tq, seed, lens, H, Hk, D, P, dtype=BF16, e4m3=False, spare=3, width=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        need = [-(-n // P) for n in lens]
        self.n_pages = sum(need) + spare
        self.tq, self.lens, self.P, self.D, self.dtype, self.e4m3 = tq, lens, P, D, dtype, e4m3
        width = max(need + [1]) if width is None else width
        order = np.random.default_rng(seed).permutation(self.n_pages).tolist()
        table = np.random.default_rng(seed + 1).integers(-5, self.n_pages + 5, (len(lens), width))
        for row, n in zip(table, need):
            row[:n] = [order.pop() for _ in range(n)]
        self.table_host = table
        self.tables, self.lengths = ints(table.tolist()).view(len(lens), width), ints(lens)
        self.q = (1.5 * r(len(lens), H, D)).to(dtype)
        shape = (self.n_pages, Hk, P, D)
        self.k, self.v = r(*shape), r(*shape)
        self.scales = {}
        if e4m3:
            for name in ("k", "v"):
                x = getattr(self, name)
                m = x.abs().amax(-1)
                setattr(self, name, (x * (448 / m)[..., None]).to(torch.float8_e4m3fn))
                self.scales[name + "_scales"] = m / 448
        else:
            self.k, self.v = self.k.to(dtype), self.v.to(dtype)
        used = torch.zeros((self.n_pages, P), dtype=torch.bool)
        for row, n in zip(table, lens):
            for i in range(n):
                used[row[i // P], i % P] = True
        hide = (~used).cuda()[:, None].expand(self.n_pages, Hk, P)
        for x in (self.k, self.v):
            x.view(torch.uint8 if e4m3 else torch.int16)[hide] = 0x7F if e4m3 else 0x7FFF
        for s in self.scales.values():
            s[hide] = float("nan")

    def run(self, **kw):
        return self.tq.attention_decode(self.q, self.k, self.v, self.tables, self.lengths, **self.scales, **kw)

    def cached(self, name, b):
        n, x = self.lens[b], getattr(self, name)
        at = torch.from_numpy(self.table_host[b, : -(-n // self.P)]).cuda()
        y = x.view(torch.uint8)[at].view(x.dtype).double()
        if self.e4m3:
            y = y * self.scales[name + "_scales"][at].double()[..., None]
        return y.transpose(1, 2).flatten(0, 1)[:n].cpu().numpy()

    def oracle(self, scale=None, rows=None):
        q, out = host(self.q), []
        for b in range(len(self.lens)) if rows is None else rows:
            out.append(attention.attend(q[b:b + 1], self.cached("k", b), self.cached("v", b), [self.lens[b] - 1],
                                        self.D ** -0.5 if scale is None else scale))
        return {x: np.concatenate([r[x] for r in out]) for x in out[0]}

    def check(self, y, lse=None, rows=None, scale=None):
        want, n = self.oracle(scale, rows), max(self.lens)
        got = host(y) if rows is None else host(y)[rows]
        u = 2.0 ** -8 if self.dtype == BF16 else 2.0 ** -11
        d = (2 * self.D + 7) * E * want["score"][..., None]
        tol = u * want["size"] + u * np.abs(want["y"]) + (4 * d + 10 * E + 4 * n * E) * want["size"]
        if self.dtype == F16:
            tol = tol + 2.0 ** -25 * (n * 8 + 1)
        bad = ~(np.abs(got - want["y"]) <= 1.01 * tol)
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want["y"][bad][:5], tol[bad][:5])
        if lse is not None:
            lse = host(lse) if rows is None else host(lse)[rows]
            none = want["lse"] == -np.inf
            assert np.all(lse[none] == -np.inf)
            with np.errstate(invalid="ignore"):
                assert np.all((np.abs(lse - want["lse"]) <= 2 * lse_tolerance(want, self.D, n)) | none)


LENS = {"one": [1], "ends": [0, 1, 31, 32, 33, 0, 127, 128, 129], "ragged": [700, 3, 64, 255, 256, 257, 12, 511]}


@pytest.mark.parametrize("name", list(LENS))
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,dtype", [(64, BF16), (64, F16), (128, BF16), (128, F16), (256, BF16), (256, F16)])
def test_lengths(tq, D, dtype, e4m3, name):
    say(f"decode {LENS[name]} dim {D} {dtype} e4m3 {e4m3}")
    c = Case(tq, 1, LENS[name], 8, 2, D, 16, dtype, e4m3)
    lse = torch.empty((len(c.lens), 8), device="cuda")
    c.check(c.run(lse=lse), lse)


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 6), (5, 1), (16, 1), (17, 1), (40, 1), (14, 2), (64, 4)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_head_layouts(tq, H, Hk, e4m3):
    say(f"decode heads {H} of {Hk} e4m3 {e4m3}")
    c = Case(tq, 2, [130, 1, 77], H, Hk, 64, 32, BF16, e4m3)
    c.check(c.run())


@pytest.mark.parametrize("H,Hk", [(256, 256), (4096, 1), (4096, 4096)])
def test_as_many_groups_as_workers(tq, H, Hk):
    """One worker for each group of heads: no shares, no workspace."""
    say(f"decode heads {H} of {Hk}")
    assert tq.lib().moe_attention_decode_workspace_bytes(3, H, Hk, 64) == 0
    c = Case(tq, 22, [130, 0, 77], H, Hk, 64, 32, BF16)
    c.check(c.run())


@pytest.mark.parametrize("P", [1, 2, 8, 64, 512, 4096])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_of_any_size(tq, P, e4m3):
    say(f"decode pages of {P} e4m3 {e4m3}")
    c = Case(tq, 3, [300, 5, 64], 4, 2, 128, P, BF16, e4m3)
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 256])
def test_one_long_sequence(tq, D):
    """Shared among as many workers as there are, with tables wider than it."""
    say(f"decode long, dim {D}")
    c = Case(tq, 4, [20011], 4, 1, D, 64, BF16, width=500)
    lse = torch.empty((1, 4), device="cuda")
    c.check(c.run(lse=lse), lse)


def test_many_sequences(tq):
    """More sequences than threads of a block, none and few tokens, two long ones."""
    lens = [(i * 37) % 90 for i in range(600)]
    lens[300], lens[599] = 3000, 2000
    say("decode 600 sequences")
    c = Case(tq, 5, lens, 2, 1, 256, 16, BF16)
    rows = [0, 1, 2, 255, 256, 257, 299, 300, 301, 598, 599] + list(range(90, 120))
    c.check(c.run(), rows=rows)
    again = Case(tq, 5, lens, 2, 1, 64, 16, F16, True)
    again.check(again.run(), rows=rows)


def test_the_largest_batch(tq):
    """65535 sequences of one token or none; of one, y is the value (tests/test_gpu_attention.py)."""
    say("decode 65535 sequences")
    n = 65535
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    q = torch.randn((n, 2, 64), generator=g, device="cuda").to(BF16)
    k, v = (torch.randn((n, 1, 1, 64), generator=g, device="cuda").to(BF16) for _ in range(2))
    tables = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    lengths = (torch.arange(n, device="cuda") % 3 != 1).to(torch.int32)
    y = tq.attention_decode(q, k, v, tables, lengths)
    want = v[tables[:, 0].long(), :, 0].expand(n, 2, 64) * lengths[:, None, None].to(BF16)
    assert torch.equal(y, want)


def test_the_batch_changes_last_bits_only(tq):
    say("decode in other batches")
    c = Case(tq, 6, [900, 40, 1300, 7], 8, 2, 128, 32)
    y = c.run()
    assert torch.equal(y, c.run())
    for b in range(4):
        alone = c.tq.attention_decode(c.q[b:b + 1], c.k, c.v, c.tables[b:b + 1], c.lengths[b:b + 1])
        c.check(torch.cat([y[:b], alone, y[b + 1:]]))


def test_lengths_outside_the_table(tq):
    """Longer than the table's room, negative, and a table without columns."""
    say("odd lengths")
    c = Case(tq, 7, [64, 64, 0, 10], 4, 2, 64, 16)
    assert c.tables.shape[1] == 4
    want = c.run()
    c.lengths.copy_(ints([1 << 30, 64, -7, 10]))
    assert torch.equal(c.run(), want) and torch.all(want[2] == 0)
    none = c.tables[:, :0].contiguous()
    lse = torch.empty((4, 4), device="cuda")
    y = c.tq.attention_decode(c.q, c.k, c.v, none, c.lengths, lse=lse)
    assert torch.all(y == 0) and torch.all(lse == float("-inf"))


def test_pages_that_are_none(tq):
    """Their sequence's results are NaN, others are not touched."""
    say("bad pages")
    c = Case(tq, 8, [300, 80, 90, 2000], 4, 2, 128, 16)
    want = c.run()
    c.tables[0, 18], c.tables[2, 0], c.tables[3, 100] = c.n_pages, -1, 1 << 30
    y = c.run()
    assert torch.isnan(y[0]).all() and torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    assert torch.equal(y[1], want[1])


def test_infinities(tq):
    """Infinite values give infinities of their sign where the last tile is cut short, keys of
    -inf score have no weight, NaN stays in its sequence."""
    say("decode infinities")
    c = Case(tq, 9, [70, 70, 70], 2, 2, 64, 64, spare=0)
    c.q.copy_(c.q.abs() + 0.1)
    c.k.clamp_(min=-0.5, max=0.5)
    page = c.table_host
    c.v[page[0, 1], 0, 5, 7] = float("inf")          # token 69, the last one
    c.v[page[0, 0], 0, 5, 8] = float("-inf")
    c.k[page[1, 0], :, :64] = float("-inf")
    c.k[page[2, 1], 1, 3] = float("nan")
    y = host(c.run())
    want = c.oracle()
    assert y[0, 0, 7] == np.inf and y[0, 0, 8] == -np.inf and np.isfinite(y[0, 0, 9:]).all()
    assert np.all(np.abs(y[1] - want["y"][1]) <= 2.0 ** -7 * (want["size"][1] + np.abs(want["y"][1])))
    assert np.isnan(y[2, 1]).all() and np.isfinite(y[2, 0]).all()


def test_all_scores_of_minus_infinity(tq):
    say("decode, no weight at all")
    c = Case(tq, 10, [40, 700], 2, 1, 64, 16)
    c.q.copy_(c.q.abs() + 0.1)
    c.k.fill_(float("-inf"))
    lse = torch.empty((2, 2), device="cuda")
    y = c.run(lse=lse)
    assert torch.all(y == 0) and torch.all(lse == float("-inf"))


@pytest.mark.parametrize("e4m3", [False, True])
def test_moving_maximum(tq, e4m3):
    say(f"decode moving maximum e4m3 {e4m3}")
    c = Case(tq, 11, [1500, 1000], 2, 1, 64, 32, BF16, e4m3)
    c.q[:, 0, 0], c.q[:, 1, 0] = 60.0, -60.0
    c.check(c.run())
    c.check(c.run(scale=2.0), scale=2.0)


def test_strided_queries_and_stream(tq):
    say("decode strided, stream")
    c = Case(tq, 12, [100, 300], 4, 2, 128, 16)
    want = c.run()
    wide = torch.zeros((2, 7, 136), dtype=BF16, device="cuda")
    part = wide[:, 2:6, :128]
    part.copy_(c.q)
    c.q = part
    assert torch.equal(c.run(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = c.run(stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_offsets_past_32_bits(tq):
    """Pages more than 4 GiB into the cache."""
    say("far pages")
    D, P, Hk, n = 128, 64, 8, 40000
    k = torch.empty((n, Hk, P, D), dtype=BF16, device="cuda")
    v = torch.empty((n, Hk, P, D), dtype=BF16, device="cuda")
    c = Case(tq, 13, [150], 16, Hk, D, P, spare=0)
    far = [39999, 20000, 36000]
    for at, p in zip(far, c.table_host[0]):
        k[at], v[at] = c.k[int(p)], c.v[int(p)]
    y = tq.attention_decode(c.q, k, v, ints([far]), c.lengths)
    assert torch.equal(y, c.run())


@pytest.mark.parametrize("e4m3", [False, True])
def test_the_longest_length(tq, e4m3):
    """2^31 - 1 tokens, one page over and over, keys that weigh alike.  Every share's sums of
    weights and of integers are exact in fp32 (below 2^24); joining 256 of them rounds 263
    times at most, each sum by 2^-24 of sum_j |v_j| < 2^31: y is off by 264 2^-24 < 2^-15 and
    its rounding, lse by as much and its own."""
    say("2^31 - 1 tokens", e4m3)
    D, P, n = 64, 4096, (1 << 31) - 1
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    v = torch.randint(-1, 2, (1, 1, P, D), generator=g, device="cuda").float()
    v[..., : D // 2] = v[..., : D // 2].abs()
    k = torch.randn((1, 1, P, D), generator=g, device="cuda")
    cache = torch.float8_e4m3fn if e4m3 else BF16
    scales = {x: torch.ones((1, 1, P), device="cuda") for x in ("k_scales", "v_scales")} if e4m3 else {}
    lse = torch.empty((1, 2), device="cuda")
    y = tq.attention_decode(torch.zeros((1, 2, D), dtype=BF16, device="cuda"), k.to(cache), v.to(cache),
                            torch.zeros((1, (n + 1) // P), dtype=torch.int32, device="cuda"), ints([n]), lse=lse, **scales)
    v = host(v)[0, 0]
    want = (v.sum(0) * ((n + 1) // P) - v[-1]) / n
    assert np.all(np.abs(host(y)[0] - want) <= 2.0 ** -15 + 2.0 ** -8 * np.abs(want))
    assert np.all(np.abs(host(lse) - np.log(n)) <= 2.0 ** -15 + 2.0 ** -24 * 4 * np.log(n))


def test_two_graphs_share_a_workspace(tq):
    say("decode graphs")
    a, b = Case(tq, 14, [900, 31, 500], 8, 2, 128, 32), Case(tq, 15, [3000], 8, 2, 128, 32)
    need = tq.lib().moe_attention_decode_workspace_bytes(3, 8, 2, 128)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    ys = [torch.empty_like(x.q) for x in (a, b)]
    graphs = []
    for x, y in zip((a, b), ys):
        x.run(y=y, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(y=y, workspace=ws)
        graphs.append(g)
    for i in range(4):
        a.lengths.copy_(ints([900 - 100 * i, i, 500]))
        b.lengths.copy_(ints([3000 - 999 * i]))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, y in zip((a, b), ys):
            assert torch.equal(y, x.run())


def test_refusals(tq):
    say("decode refusals")
    c = Case(tq, 16, [20, 30], 4, 2, 64, 16)
    e = Case(tq, 16, [20, 30], 4, 2, 64, 16, e4m3=True)
    good = dict(q=c.q, k_cache=c.k, v_cache=c.v, tables=c.tables, lengths=c.lengths)
    for bad in (dict(q=c.q.half()), dict(k_cache=c.k[:, :1].contiguous()), dict(v_cache=c.v[:-1]), dict(k_cache=c.k[0]),
                dict(tables=c.tables[:1]), dict(tables=c.tables.long()), dict(lengths=c.lengths[:1]),
                dict(lengths=c.lengths.cpu()), dict(k_cache=e.k, v_cache=e.v), dict(k_scales=e.scales["k_scales"]),
                dict(scale=-1.0), dict(y=c.q[:1].contiguous()), dict(workspace=torch.empty(300, dtype=torch.uint8, device="cuda")),
                dict(q=c.q[..., :32].contiguous()), dict(k_cache=c.k.transpose(0, 1))):
        with pytest.raises(tq.MoeError):
            tq.attention_decode(**{**good, **bad})
    with pytest.raises(tq.MoeError, match="overlap"):
        tq.attention_decode(**good, y=c.q)
