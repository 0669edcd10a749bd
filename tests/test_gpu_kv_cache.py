"""GPU parity of the cache's write and its pages against the float64 oracle.

Turned values, e = 2^-24 the fp32 half step: the angle in turns is a product of two fp64
roundings, at most 2^31 2^-53 and far below; its fraction in fp32 is at most 1/2 and off
by 2^-26, doubled by a factor of two exactly, so the angle is off by pi 2^-25; sine and cosine
are within 4 e of theirs beyond that; two products and a sum add 3 e of the magnitudes.  With
|a| + |b| = m: 16 e m; the output's rounding adds half a step, u |y|, and below fp16's normal
numbers 2^-25.  e4m3: a scale is off by 16 e m / 448 and 2 e of itself; a code's value over its scale is off by
half a step, 2^-4 of itself or 2^-10 for the smallest, and 448 times (32 e m / the block's largest + 4 e).
"""
import numpy as np
import pytest

from oracle import attention
from test_gpu_attention import BF16, E, F16, host, ints, say, tq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Append:
    def __init__(self, seed, rows, positions, H, Hk, D, P, rotary, dtype=BF16, e4m3=False, width=None, scale=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        n, R = len(rows), max(rows) + 1
        self.width = max(positions) // P + 1 if width is None else width
        self.n_pages = R * self.width + 2
        self.P, self.D, self.rotary, self.dtype, self.e4m3 = P, D, rotary, dtype, e4m3
        self.x = (scale * r(n, H + 2 * Hk, D)).to(dtype)
        self.q, self.k, self.v = self.x[:, :H], self.x[:, H:H + Hk], self.x[:, H + Hk:]
        order = np.random.default_rng(seed).permutation(self.n_pages)[:R * self.width]
        self.tables = ints(order.tolist()).view(R, self.width)
        self.rows, self.positions = ints(rows), ints(positions)
        kind = torch.float8_e4m3fn if e4m3 else dtype
        self.k_cache = torch.full((self.n_pages, Hk, P, D), 3.0, device="cuda").to(kind)
        self.v_cache = self.k_cache.clone()
        self.scales = {}
        if e4m3:
            self.scales = {x: torch.full((self.n_pages, Hk, P), 5.0, device="cuda") for x in ("k_scales", "v_scales")}
        self.inv_freq = (1e4 ** (-torch.arange(rotary // 2, dtype=torch.float64) / max(rotary // 2, 1))).float().cuda()

    def run(self, tq, **kw):
        if self.rotary:
            kw.setdefault("q", self.q)
            kw.setdefault("inv_freq", self.inv_freq)
        return tq.kv_append(self.k, self.v, self.k_cache, self.v_cache, self.tables, self.rows, self.positions,
                            **self.scales, **kw)

    def slots(self):
        t, r, p = self.tables.cpu().numpy(), self.rows.cpu().numpy(), self.positions.cpu().numpy()
        return t[r, p // self.P], p % self.P

    def check(self, out, interleaved=False):
        u, low = (2.0 ** -8, 0.0) if self.dtype == BF16 else (2.0 ** -11, 2.0 ** -25)
        pos, f, half = self.positions.cpu().numpy(), host(self.inv_freq), self.rotary // 2

        def turned(x):
            y = attention.rotate(host(x), pos, f, interleaved)
            m = np.zeros_like(y)
            pair = np.sqrt(2 * (y[..., 0:2 * half:2] ** 2 + y[..., 1:2 * half:2] ** 2)) if interleaved else \
                np.sqrt(2 * (y[..., :half] ** 2 + y[..., half:2 * half] ** 2))     # at least |a| + |b|
            if interleaved:
                m[..., 0:2 * half:2] = m[..., 1:2 * half:2] = pair
            else:
                m[..., :half] = m[..., half:2 * half] = pair
            return y, 16 * E * m

        def near(got, want, tol):
            bad = ~(np.abs(host(got) - want) <= 1.01 * tol)
            assert not bad.any(), (np.argwhere(bad)[:5], host(got)[bad][:5], want[bad][:5], tol[bad][:5])
        k, k_err = turned(self.k)
        if "q" in out:
            q, err = turned(self.q)
            near(out["q"], q, err + u * np.abs(q) + low)
        if "k" in out:
            near(out["k"], k, k_err + u * np.abs(k) + low)
        page, off = self.slots()
        for name, y, err in (("k", k, k_err), ("v", host(self.v), 0 * host(self.v))):
            cache = host(getattr(self, name + "_cache"))
            got = cache[page, :, off]
            if self.e4m3:
                s = host(self.scales[name + "_scales"])
                m = np.maximum(np.abs(y).max(-1), 1e-30)
                assert np.all(np.abs(s[page, :, off] - m / 448) <= err.max(-1) / 448 + 2.01 * E * m / 448)
                want = y / (m / 448)[..., None]
                tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 448 * (2 * err.max(-1) / m + 4 * E)[..., None]
                assert np.all(np.abs(got - want) <= 1.07 * tol)
                s[page, :, off] = 5.0
                assert np.all(s == 5.0)
            else:
                assert np.all(np.abs(got - y) <= 1.01 * (err + u * np.abs(y) + low))
            cache[page, :, off] = 3.0
            assert np.all(cache == 3.0), "places of no token stay as they were"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,rotary,dtype", [(64, 64, BF16), (64, 16, F16), (128, 128, F16), (128, 64, BF16),
                                            (256, 256, BF16), (256, 96, F16)])
def test_append(tq, D, rotary, dtype, e4m3, interleaved):
    say(f"append dim {D} rotary {rotary} {dtype} e4m3 {e4m3} interleaved {interleaved}")
    rows = [0] * 20 + [2] * 7 + [1]
    positions = list(range(13, 33)) + list(range(7)) + [60]
    a = Append(1, rows, positions, 6, 2, D, 16, rotary, dtype, e4m3)
    a.check(a.run(tq, interleaved=interleaved, rotated_k=True), interleaved)


@pytest.mark.parametrize("H,Hk,P", [(1, 1, 1), (3, 3, 2), (10, 5, 64), (64, 4, 4096)])
def test_append_layouts(tq, H, Hk, P):
    say(f"append heads {H} of {Hk}, pages of {P}")
    a = Append(2, [0, 0, 1, 3], [0, 1, 5, 130], H, Hk, 128, P, 128)
    a.check(a.run(tq))


def test_append_without_rotation(tq):
    """The cache takes the bits, and e4m3 the quantizer's codes and scales."""
    say("append plain")
    a = Append(3, [0] * 40, list(range(40)), 4, 4, 128, 16, 0)
    assert a.run(tq) == {}
    page, off = a.slots()
    page, off = torch.from_numpy(page).cuda(), torch.from_numpy(off).cuda()
    assert torch.equal(a.k_cache[page, :, off], a.k) and torch.equal(a.v_cache[page, :, off], a.v)
    b = Append(3, [0] * 40, list(range(40)), 4, 4, 128, 16, 0, e4m3=True)
    b.run(tq)
    for name in ("k", "v"):
        codes, scales = tq.fp8_quantize(getattr(b, name).reshape(160, 128), 1)
        assert torch.equal(getattr(b, name + "_cache").view(torch.uint8)[page, :, off].flatten(), codes.view(torch.uint8).flatten())
        assert torch.equal(b.scales[name + "_scales"][page, :, off].flatten(), scales.flatten())


def test_more_tokens_than_one_dimension(tq):
    """2^20 + 3 tokens of 257 sequences, a block each."""
    say("append 2^20 + 3 tokens")
    n, P = (1 << 20) + 3, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    k, v = (torch.randn((n, 1, 64), generator=g, device="cuda").to(BF16) for _ in range(2))
    k_cache, v_cache = (torch.zeros((257, 1, P, 64), dtype=BF16, device="cuda") for _ in range(2))
    token = torch.arange(n, device="cuda")
    tables = torch.randperm(257, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    rows, positions = (token // P).to(torch.int32), (token % P).to(torch.int32)
    tq.kv_append(k, v, k_cache, v_cache, tables, rows, positions)
    page = tables[rows.long(), 0].long()
    assert torch.equal(k_cache[page, 0, positions.long()], k[:, 0])
    assert torch.equal(v_cache[page, 0, positions.long()], v[:, 0])
    assert not k_cache[tables[256, 0].long(), 0, 3:].any()


def test_far_positions(tq):
    say("far positions")
    a = Append(4, [0, 0, 0], [1, (1 << 20) - 1, 999983], 2, 1, 64, 4096, 64, F16)
    a.check(a.run(tq))
    a.positions.copy_(ints([0, 1 << 20, (1 << 31) - 1]))     # past the table: turned or not, the cache keeps out
    before = a.k_cache.clone()
    out = a.run(tq)
    assert torch.equal(out["q"][0], a.q[0]) and torch.isnan(out["q"][1:]).all()
    before[a.tables[0, 0].item(), :, 0] = a.k[0]
    assert torch.equal(a.k_cache, before)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(tq, D, interleaved):
    say(f"append in place, dim {D}")
    a = Append(5, [0] * 50, list(range(50)), 8, 4, D, 16, D // 2, F16)
    want = a.run(tq, rotated_k=True, interleaved=interleaved)
    cache = a.k_cache.clone()
    out = a.run(tq, q_out=a.q, k_out=a.k, interleaved=interleaved)
    assert out["q"] is a.q and torch.equal(a.q, want["q"]) and torch.equal(a.k, want["k"])
    assert torch.equal(a.k_cache, cache)


def test_padding_and_places_that_are_none(tq):
    say("append padding")
    a = Append(6, [0, 1, 1, 0, 1], [3, 4, 5, 6, 7], 4, 2, 64, 4, 32)
    table = a.tables.cpu().tolist()
    a.rows.copy_(ints([-1, 1, 9, 0, 1]))
    a.positions.copy_(ints([3, 4, 5, -1, 6]))
    a.tables[1, 1] = a.n_pages                               # tokens 1 and 4: a page that is none
    q_out = torch.full((5, 4, 64), 9.0, dtype=BF16, device="cuda")
    k_out = torch.full((5, 2, 64), 9.0, dtype=BF16, device="cuda")
    a.run(tq, q_out=q_out, k_out=k_out)
    assert torch.all(q_out[0] == 9) and torch.all(k_out[0] == 9)
    assert torch.isnan(q_out[1:]).all() and torch.isnan(k_out[1:]).all()
    assert torch.all(a.k_cache == 3) and torch.all(a.v_cache == 3)
    a.tables.copy_(ints(table))
    a.run(tq, q_out=q_out, k_out=k_out)
    assert torch.isfinite(q_out[[1, 4]].float()).all() and torch.isnan(q_out[2:4]).all()


def test_nan_and_infinities_stay_in_their_head(tq):
    say("append NaN")
    a = Append(7, [0, 0, 0], [0, 1, 2], 2, 2, 64, 4, 64, e4m3=True)
    a.v[1, 0, 5] = float("nan")
    a.v[2, 1, 6] = float("inf")
    a.run(tq)
    s = a.scales["v_scales"][a.tables[0, 0]]
    assert torch.isnan(s[0, 1]) and torch.isinf(s[1, 2]) and torch.isfinite(s[1, :2]).all() and torch.isfinite(s[0, [0, 2]]).all()


def test_append_refusals(tq):
    say("append refusals")
    a = Append(8, [0, 0], [0, 1], 4, 2, 64, 4, 32)
    for bad in (dict(q=a.q[:1]), dict(q=a.q.half()), dict(q_out=a.k), dict(k_out=a.v), dict(k_out=a.q[:, :2]),
                dict(inv_freq=None), dict(inv_freq=a.inv_freq[:3]), dict(q=None, q_out=a.q),
                dict(inv_freq=torch.ones(40, device="cuda")), dict(inv_freq=a.inv_freq.double()), dict(q_out=a.q[:, :2]),
                dict(q_out=a.k_cache[0].view(2, 2, -1)[..., :64])):
        with pytest.raises(tq.MoeError):
            a.run(tq, **bad)
    with pytest.raises(tq.MoeError):
        tq.kv_append(a.k, a.v, a.k_cache, a.v_cache[:1], a.tables, a.rows, a.positions)
    with pytest.raises(tq.MoeError):
        tq.kv_append(a.k, a.v, a.k_cache, a.v_cache, a.tables, a.rows.long(), a.positions)
    with pytest.raises(tq.MoeError):
        tq.kv_append(a.k, a.v, a.k_cache, a.v_cache, a.tables, a.rows, a.positions, k_scales=a.inv_freq)


# ------------------------------------------------------------------ pages
class Pages:
    """The same cache on the GPU and in the oracle; page contents are numbered."""

    def __init__(self, tq, rows, width, n, page, pools=((3, 5), (2, 1))):
        self.tq, self.page = tq, page
        data = [np.arange(planes * n * page * per).reshape(planes, n, page, per) % 100003 for planes, per in pools]
        self.model = attention.Pages([[-1] * width for _ in range(rows)], [0] * rows, [0] * n, page, data)
        self.tables = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.lengths, self.refs = ints([0] * rows), ints([0] * n)
        self.pools = [torch.from_numpy(x).to(torch.int32).cuda() for x in data]

    def state(self):
        return self.tables, self.lengths, self.refs

    def reserve(self, grow):
        got = self.tq.kv_reserve(*self.state(), ints(grow), self.page)
        assert got.tolist() == self.model.reserve(grow)
        self.same()

    def fork(self, parents):
        got = self.tq.kv_fork(*self.state(), ints(parents), self.page, self.pools)
        assert got.tolist() == self.model.fork(parents)
        self.same()

    def free(self, drop):
        self.tq.kv_free(*self.state(), ints(drop), self.page)
        self.model.free(drop)
        self.same()

    def compact(self, in_place):
        kw = dict(new_tables=self.tables, new_refs=self.refs) if in_place else {}
        tables, refs, live = self.tq.kv_compact(*self.state(), self.page, self.pools, **kw)
        assert live.tolist() == [self.model.compact()]
        self.tables, self.refs = tables, refs
        self.same()

    def same(self):
        assert self.tables.tolist() == self.model.tables
        assert self.lengths.tolist() == self.model.lengths
        assert self.refs.tolist() == self.model.refs
        for a, b in zip(self.pools, self.model.pools):
            assert np.array_equal(a.cpu().numpy(), b)


def test_pages_one_by_one(tq):
    say("pages")
    p = Pages(tq, 6, 5, 20, 4)
    p.reserve([5, 0, 4, 21, -1, 0])
    p.fork([-1, 0, -1, 2, 1, 0])
    p.free([1, 0, 1, 0, 0, 0])
    p.compact(False)
    p.reserve([0, 3, 0, 9, 0, 1])
    p.free([0, 1, 0, 0, 0, 1])
    p.compact(True)
    p.compact(True)


@pytest.mark.parametrize("seed", range(6))
def test_pages_at_random(tq, seed):
    """Calls in any order, with too few pages now and then."""
    r = np.random.default_rng(seed)
    rows, width, page = int(r.integers(1, 40)), int(r.integers(1, 12)), int(2 ** r.integers(0, 6))
    n = int(r.integers(1, rows * width + 2))
    say(f"pages at random: {rows} rows of {width}, {n} pages of {page}")
    p = Pages(tq, rows, width, n, page)
    for step in range(25):
        what = r.integers(0, 4)
        if what == 0:
            p.reserve([int(x) for x in r.integers(-1, 2 * page * width // 3 + 2, rows) * (r.random(rows) < 0.4)])
        elif what == 1:
            p.fork([int(x) for x in np.where(r.random(rows) < 0.4, r.integers(0, rows + 1, rows), -1)])
        elif what == 2:
            p.free([int(x) for x in r.random(rows) < 0.3])
        else:
            p.compact(bool(step % 2))


def test_many_rows_and_pages(tq):
    """More than one step of the plan over rows and pages, and rows with many pages."""
    say("pages: many")
    rows, width, n, page = 2500, 40, 50000, 2
    p = Pages(tq, rows, width, n, page, pools=((1, 1),))
    r = np.random.default_rng(0)
    p.reserve([int(x) for x in r.integers(0, 2 * width, rows) * (r.random(rows) < 0.5)])
    p.fork([int(x) for x in np.where(np.array(p.model.lengths) == 0, r.integers(-1, rows, rows), -1)])
    p.free([int(x) for x in r.random(rows) < 0.5])
    p.compact(False)
    p.reserve([3] * rows)


def test_copy_pages(tq):
    """Every plane of every pool, wide and narrow pages; pairs that are none are passed over."""
    say("copy pages")
    for shape in ((2, 30, 4, 16, 64), (1, 30, 3, 7), (5, 30, 1)):
        a = torch.arange(int(np.prod(shape)), device="cuda", dtype=torch.int32).view(shape)
        b = a.clone().to(torch.bfloat16).expand(*shape).contiguous() if len(shape) == 5 else a.clone()
        want = [x.clone() for x in (a, b)]
        src, dst = [3, 0, 29, -1, 5, 30], [4, 28, 1, 7, -2, 8]
        for x in want:
            for s, d in zip(src[:3], dst[:3]):
                x[:, d] = x[:, s]
        tq.kv_copy_pages([a, b], ints(src), ints(dst))
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    tq.kv_copy_pages([a], ints([]), ints([]))
    tq.kv_copy_pages([], ints([1]), ints([2]))


def test_pages_past_32_bits(tq):
    say("pages past 4 GiB")
    pool = torch.empty((1, 3000, 1 << 20), dtype=torch.int16, device="cuda")     # 6 GiB
    pool[0, 2999] = 5
    pool[0, 7] = 6
    tq.kv_copy_pages([pool], ints([2999, 7]), ints([0, 2500]))
    assert torch.all(pool[0, 0] == 5) and torch.all(pool[0, 2500] == 6)


def test_pages_captured(tq):
    """Reserve, fork, free and compact in a HIP graph that is replayed with other requests."""
    say("pages graph")
    p = Pages(tq, 8, 6, 40, 4)
    grow, parents, drop = ints([0] * 8), ints([-1] * 8), ints([0] * 8)
    ws = torch.empty(tq.lib().moe_kv_pages_workspace_bytes(8, 40) + 256, dtype=torch.uint8, device="cuda")
    status, forked, live = ints([0] * 8), ints([0] * 8), ints([0])

    def step():
        tq.kv_reserve(*p.state(), grow, 4, status=status, workspace=ws)
        tq.kv_fork(*p.state(), parents, 4, p.pools, status=forked, workspace=ws)
        tq.kv_free(*p.state(), drop, 4)
        tq.kv_compact(*p.state(), 4, p.pools, new_tables=p.tables, new_refs=p.refs, live=live, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    r = np.random.default_rng(3)
    for _ in range(5):
        asks = ([int(x) for x in r.integers(0, 9, 8)], [int(x) for x in r.integers(-1, 8, 8)],
                [int(x) for x in r.random(8) < 0.3])
        for t, a in zip((grow, parents, drop), asks):
            t.copy_(ints(a))
        graph.replay()
        torch.cuda.synchronize()
        assert status.tolist() == p.model.reserve(asks[0]) and forked.tolist() == p.model.fork(asks[1])
        p.model.free(asks[2])
        assert live.tolist() == [p.model.compact()]
        p.same()


def test_pages_refusals(tq):
    say("pages refusals")
    p = Pages(tq, 4, 3, 10, 4)
    t, l, f = p.state()
    one = ints([0] * 4)
    for call in (lambda: tq.kv_reserve(t.long(), l, f, one, 4), lambda: tq.kv_reserve(t, l[:3], f, one, 4),
                 lambda: tq.kv_reserve(t, l, f, one[:2], 4), lambda: tq.kv_reserve(t, l, f, one, 3),
                 lambda: tq.kv_reserve(t, l, f, l, 4, status=l), lambda: tq.kv_reserve(t, l, f, one, 0),
                 lambda: tq.kv_fork(t, l, f, one, 4, [p.pools[0][:, :9]]),
                 lambda: tq.kv_fork(t, l, f, one, 4, [p.pools[0].transpose(0, 1)]),
                 lambda: tq.kv_fork(t, l, f, one, 4, [p.pools[0], p.pools[0]]), lambda: tq.kv_fork(t, l, f, one, 4, p.pools * 5),
                 lambda: tq.kv_free(t, l, f, one.cpu(), 4), lambda: tq.kv_free(t, l, f, l, 4),
                 lambda: tq.kv_compact(t, l, f, 4, p.pools, new_refs=l), lambda: tq.kv_compact(t, l, f, 4, [p.pools[0].cpu()]),
                 lambda: tq.kv_copy_pages(p.pools, one, one[:2]), lambda: tq.kv_copy_pages(p.pools, one.float(), one),
                 lambda: tq.kv_reserve(t, l, f, one, 4, workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(tq.MoeError):
            call()
    p.same()
