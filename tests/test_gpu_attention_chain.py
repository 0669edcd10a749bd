"""Attention and its cache together, as a program uses them: 8-bit projections -> rotary
embedding and pages -> attention over the prompts -> the branch on its output; then single
tokens over the pages, with sequences that fork, grow, end and are packed together, eagerly,
into a HIP graph and on a side stream."""
import numpy as np
import pytest

from oracle import attention
from test_gpu_attention import BF16, check, host, ints, say, starts_of, tolerance, tq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Layer:
    """One attention layer and a cache for `rows` sequences."""

    def __init__(self, tq, rows, width, n_pages, page, d=256, H=8, Hk=2, D=64, e4m3=False, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.tq, self.H, self.Hk, self.D, self.d, self.page, self.e4m3 = tq, H, Hk, D, d, page, e4m3
        self.norm = 1 + 0.1 * self.r(d)
        self.w, self.w_scales = tq.fp8_quantize((self.r((H + 2 * Hk) * D, d) / d ** 0.5).bfloat16(), 128)
        self.a, self.b = (self.r(128, H * D) / 30).half(), (self.r(H * D, 128) / 30).half()
        self.inv_freq = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
        kind = torch.float8_e4m3fn if e4m3 else BF16
        self.k = torch.zeros((1, n_pages, Hk, page, D), device="cuda").to(kind)
        self.v = self.k.clone()
        self.pools, self.scales = [self.k, self.v], {}
        if e4m3:
            s = torch.zeros((2, 1, n_pages, Hk, page), device="cuda")
            self.scales = {"k_scales": s[0, 0], "v_scales": s[1, 0]}
            self.pools += [s[0], s[1]]
        self.tables = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.lengths, self.refs = ints([0] * rows), ints([0] * n_pages)

    def state(self):
        return self.tables, self.lengths, self.refs

    def project(self, x, rows, positions, stream=None):
        """q, k, v of hidden states x, turned in place and put into the cache."""
        tq, H, Hk, D = self.tq, self.H, self.Hk, self.D
        n = tq.rms_norm(x, self.norm, 1e-6, bf16=False, fp8=True, stream=stream)
        qkv = tq.fp8_linear(n["q"], n["scales"], self.w, self.w_scales, stream=stream).view(-1, H + 2 * Hk, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        tq.kv_append(k, v, self.k[0], self.v[0], self.tables, rows, positions, **self.scales, q=q, inv_freq=self.inv_freq,
                     q_out=q, k_out=k, stream=stream)
        return q, k, v

    def decode(self, q, stream=None, **kw):
        return self.tq.attention_decode(q, self.k[0], self.v[0], self.tables, self.lengths, **self.scales, stream=stream, **kw)

    def cached(self, name, row):
        """A row's cached values as they stand in the pages, in fp64."""
        n = self.lengths[row].item()
        at = self.tables[row, : -(-n // self.page)].long()
        x = getattr(self, name)[0]
        y = x.view(torch.uint8)[at].view(x.dtype).double()
        if self.e4m3:
            y = y * self.scales[name + "_scales"][at].double()[..., None]
        return y.transpose(1, 2).flatten(0, 1)[:n].cpu().numpy()

    def check_decode(self, q, y, rows):
        q, y = host(q), host(y)
        for r in rows:
            k, v = self.cached("k", r), self.cached("v", r)
            want = attention.attend(q[r:r + 1], k, v, [len(k) - 1], self.D ** -0.5)
            tol = 2 * tolerance(want, BF16, self.D, len(k), 8.0)   # shares joined and scales of e4m3: below the second half
            assert np.all(np.abs(y[r] - want["y"][0]) <= tol[0]), r


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompts_then_tokens(tq, e4m3):
    say(f"layer, e4m3 {e4m3}")
    lens = [70, 1, 0, 200, 33]
    layer = Layer(tq, 8, 20, 60, 16, e4m3=e4m3)
    assert tq.kv_reserve(*layer.state(), ints(lens + [0] * 3), 16).tolist() == [5, 1, 0, 13, 3, 0, 0, 0]
    rows = ints([r for r, n in enumerate(lens) for _ in range(n)])
    positions = ints([i for n in lens for i in range(n)])
    q, k, v = layer.project(layer.r(sum(lens), layer.d).bfloat16(), rows, positions)
    y = tq.attention_prefill(q, k, v, starts_of(lens))
    at, parts = 0, []
    for r, n in enumerate(lens):
        parts.append(attention.attend(host(q)[at:at + n], host(k)[at:at + n], host(v)[at:at + n], np.arange(n), layer.D ** -0.5))
        if n and not e4m3:
            assert np.array_equal(layer.cached("k", r), host(k)[at:at + n]) and np.array_equal(layer.cached("v", r), host(v)[at:at + n])
        at += n
    check(y, None, {x: np.concatenate([p[x] for p in parts]) for x in parts[0]}, BF16, layer.D, 200, 8.0)
    flat = y.view(sum(lens), -1)
    out = tq.lowrank_apply(flat, flat, layer.a, layer.b, 128)
    assert out.shape == flat.shape and torch.isfinite(out.float()).all()

    # each prompt's last token again, over the pages: what the prompt gave it
    ends = (starts_of(lens)[1:] - 1).long()
    again = layer.decode(torch.cat([q[ends], q[:3]]).contiguous())
    layer.check_decode(torch.cat([q[ends], q[:3]]), again, [0, 1, 3, 4])
    assert torch.all(again[2] == 0) and torch.all(again[5:] == 0)

    # row 0 forks twice, row 3 once; the copies go their own ways
    assert tq.kv_fork(*layer.state(), ints([-1, -1, -1, -1, -1, 0, 0, 3]), 16, layer.pools).tolist() == [0] * 5 + [1, 1, 1]
    before = [layer.cached("v", r) for r in range(8)]
    assert all(np.array_equal(before[0], before[r]) for r in (5, 6)) and np.array_equal(before[3], before[7])
    alive = [0, 1, 3, 4, 5, 6, 7]
    for step in range(20):
        grow = ints([int(r in alive) for r in range(8)])
        where = layer.lengths.clone()
        assert (tq.kv_reserve(*layer.state(), grow, 16) >= 0).all()
        one = torch.where(grow > 0, torch.arange(8, device="cuda", dtype=torch.int32), -1).int()
        q1, _, _ = layer.project(layer.r(8, layer.d).bfloat16(), one, where)
        y1 = layer.decode(q1)
        if step in (0, 1, 10, 19):
            layer.check_decode(q1, y1, alive)
            for r in alive:                          # what was there is still there, in the copies too
                assert np.array_equal(layer.cached("v", r)[:len(before[r])], before[r])
        if step == 9:                                # some end, the others' pages move together
            tq.kv_free(*layer.state(), ints([0, 1, 0, 0, 0, 1, 0, 0]), 16)
            alive = [0, 3, 4, 6, 7]
            old = layer.decode(q1)
            layer.tables, layer.refs, live = tq.kv_compact(*layer.state(), 16, layer.pools)
            assert live.item() == int((layer.refs > 0).sum()) and (layer.refs[live.item():] == 0).all()
            assert torch.equal(layer.decode(q1), old)
    # no page is lost: each is held as often as it is counted
    held = torch.zeros_like(layer.refs)
    for r, n in enumerate(layer.lengths.tolist()):
        for p in layer.tables[r, : -(-n // 16)].tolist():
            held[p] += 1
    assert torch.equal(held, layer.refs)


def test_a_prompt_in_chunks(tq):
    """Chunks of a prompt behind the keys so far give what the whole prompt gives."""
    say("chunks")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q = torch.randn((300, 8, 128), generator=g, device="cuda").bfloat16()
    k, v = (torch.randn((300, 2, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    want = attention.attend(host(q), host(k), host(v), np.arange(300), 128 ** -0.5)
    parts = []
    for a, b in ((0, 100), (100, 101), (101, 300)):
        parts.append(tq.attention_prefill(q[a:b], k[:b], v[:b], ints([0, b - a]), ints([0, b])))
    check(torch.cat(parts), None, want, BF16, 128, 300, 8.0)


def test_two_parts_join_by_their_logarithms(tq):
    """Attention over a shared prefix and over the rest, weighted by the softmax sums, is attention over both."""
    say("join by lse")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    q = torch.randn((50, 4, 64), generator=g, device="cuda").bfloat16()
    k, v = (torch.randn((250, 4, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    lse = [torch.empty((50, 4), device="cuda") for _ in range(2)]
    a = tq.attention_prefill(q, k[:200], v[:200], ints([0, 50]), ints([0, 200]), causal=False, lse=lse[0])
    b = tq.attention_prefill(q, k[200:], v[200:], ints([0, 50]), lse=lse[1])
    w = torch.softmax(torch.stack(lse).double(), 0)[..., None]
    both = w[0] * a.double() + w[1] * b.double()
    want = attention.attend(host(q), host(k), host(v), np.arange(50) + 200, 0.125)
    tol = 2 * tolerance(want, BF16, 64, 250, 8.0) + 2.0 ** -8 * np.abs(host(w[0] * a.double().abs() + w[1] * b.double().abs()))
    assert np.all(np.abs(host(both) - want["y"]) <= tol)


def test_a_step_captured_and_replayed(tq):
    """Room, projections, append and attention of one token in a graph, replayed while the sequences grow, with eager
    work between; and the same on a side stream."""
    say("captured step")
    lens = [40, 3, 90, 15]
    layer, other = (Layer(tq, 4, 12, 40, 16) for _ in range(2))
    rows, positions = ints([r for r, n in enumerate(lens) for _ in range(n)]), ints([i for n in lens for i in range(n)])
    x0 = layer.r(sum(lens), layer.d).bfloat16()
    for one in (layer, other):
        tq.kv_reserve(*one.state(), ints(lens), 16)
        one.project(x0, rows, positions)
    x, y = torch.zeros((4, layer.d), dtype=BF16, device="cuda"), torch.zeros((4, 8, 64), dtype=BF16, device="cuda")
    every, where = ints([0, 1, 2, 3]), ints([0] * 4)
    grow, none = ints([1] * 4), ints([0] * 4)
    status = ints([0] * 4)

    def step(one, grow, x, y):
        where.copy_(one.lengths)
        tq.kv_reserve(*one.state(), grow, 16, status=status)
        q, _, _ = one.project(x, every, where)
        one.decode(q, y=y)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                    # warm up without growing
        where.copy_(layer.lengths)
        tq.kv_reserve(*layer.state(), none, 16, status=status)
        layer.decode(torch.zeros((4, 8, 64), dtype=BF16, device="cuda"), y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(layer, grow, x, y)
    for i in range(40):
        x.copy_(other.r(4, layer.d))
        graph.replay()
        want = torch.empty_like(y)
        if i % 2:
            step(other, grow, x, want)
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step(other, grow, x, want)
            torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(layer.lengths, other.lengths) and torch.equal(layer.tables, other.tables), i
    assert layer.lengths.tolist() == [n + 40 for n in lens]
