"""The operators together, as a program uses them: block output and residual ->
norm in 8 bits -> output head -> sampler, on a side stream, into a HIP graph, and
behind the MoE block and the draft head."""
import sys

import numpy as np
import pytest

from layer_fixtures import Layer
from oracle import fp8, sampler

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_quantized_moe_amd as tq
    tq.lib()
    return tq


class Head:
    def __init__(self, tq, T, d, V, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.tq = tq
        self.weight = 1 + 0.1 * r(d)
        self.w, self.w_scales = tq.fp8_quantize((r(V, d) / d ** 0.5).bfloat16(), 128)
        self.residual = (2 * r(T, d)).bfloat16()
        self.x = r(T, d).bfloat16()
        self.u = torch.rand(T, generator=g, device="cuda")
        self.top_p = torch.full((T,), 0.9, device="cuda")
        self.temperature = torch.full((T,), 0.7, device="cuda")

    def step(self, stream=None):
        tq = self.tq
        n = tq.rms_norm(self.x, self.weight, 1e-6, residual=self.residual, bf16=False, fp8=True, stream=stream)
        logits = tq.fp8_linear(n["q"], n["scales"], self.w, self.w_scales, out_dtype=torch.float32, stream=stream)
        tokens, probs = tq.sample(logits, self.u, temperature=self.temperature, top_p=self.top_p, stream=stream)
        return n["sum"], n["q"], n["scales"], logits, tokens, probs


def equal(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("T,d,V", [(1, 2048, 5003), (33, 512, 1000), (300, 256, 4096)])
def test_the_chain_against_the_oracle(tq, T, d, V):
    say(f"chain {T} x {d} -> {V}")
    h = Head(tq, T, d, V)
    s, q, scales, logits, tokens, probs = h.step()
    y, mag = fp8.linear(q.cpu().view(torch.uint8).numpy(), scales.cpu().numpy(), h.w.cpu().view(torch.uint8).numpy(),
                        h.w_scales.cpu().numpy())
    tol = (2 * 128 + 4 + d // 128) * 2.0 ** -24 * mag
    assert np.all(np.abs(logits.cpu().double().numpy() - y) <= tol)
    for t in range(0, T, max(1, T // 20)):
        token, prob, margin = sampler.sample_row(logits[t].cpu().double().numpy(), float(h.u[t]), float(np.float32(0.7)),
                                                 0, float(np.float32(0.9)))
        assert margin < 1e-9 or int(tokens[t]) == token


def test_side_stream(tq):
    h = Head(tq, 20, 1024, 3000)
    want = h.step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = h.step()
    torch.cuda.current_stream().wait_stream(st)
    assert equal(got, want)
    st.wait_stream(torch.cuda.current_stream())
    got = h.step(stream=st)
    torch.cuda.synchronize()
    assert equal(got, want)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_graph_replays(tq, T):
    """Captured once, replayed on new inputs with eager work between: the same bits as eager calls."""
    h = Head(tq, T, 512, 2500)
    h.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = h.step()
    for i in range(4):
        new = Head(tq, T, 512, 2500, seed=10 + i)
        for k in ("x", "residual", "u"):
            getattr(h, k).copy_(getattr(new, k))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert equal(got, h.step())
        torch.cuda.synchronize()


def test_given_stream_keeps_what_the_call_made(tq):
    """A workspace of a call on another stream is nobody's until that stream is done with it."""
    logits, u = torch.randn((4, 50000), device="cuda"), torch.rand(4, device="cuda")
    want = tq.sample(logits, u)
    n = tq.lib().moe_sample_workspace_bytes(4, 50000) + 256
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    first = torch.empty(n, dtype=torch.uint8, device="cuda")
    place = first.data_ptr()
    del first                                             # the call's workspace will be here
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)                     # some 10 ms of work before the call's
    got = tq.sample(logits, u, stream=st)
    later = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert later.data_ptr() != place
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_graphs_and_two_streams(tq):
    """Two captured steps with inputs of their own, replayed side by side."""
    heads = [Head(tq, 24, 512, 4000, seed=s) for s in (1, 2)]
    want = [h.step() for h in heads]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for h in heads:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(h.step())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in heads]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert equal(o, w)


def test_behind_the_block_and_the_draft_head(tq):
    """Norm of the residual stream -> MoE block -> draft head -> output head -> token."""
    L = Layer("olmoe")
    c = L.cfg
    T, d = 8, c.d_model
    dev = L.tensors(L.gen.tokens(T, 1))
    ones = torch.ones(d, device="cuda")
    n = tq.rms_norm(dev["x"], ones, 1e-6)
    y = tq.forward(n["y"], dev["router"], dev["delta"], L.device(), dev["a"], dev["b"], c.top_k)
    out = tq.rms_norm(y, ones, 1e-6, residual=dev["x"], bf16=True, fp8=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    draft = tq.draft_head(out["y"], dev["x"], (r(256, 2 * d) / d).half(), None, (r(d, 256) / 16).half(), None)
    m = tq.rms_norm(draft, ones, 1e-6, bf16=False, fp8=True)
    w, sw = tq.fp8_quantize((r(3000, d) / d ** 0.5).bfloat16(), 128)
    for f in (out, m):
        logits = tq.fp8_linear(f["q"], f["scales"], w, sw, out_dtype=torch.float32)
        assert bool(torch.isfinite(logits).all())
        u = torch.rand(T, generator=g, device="cuda")
        tokens, probs = tq.sample(logits, u)
        for t in range(T):
            token, prob, margin = sampler.sample_row(logits[t].cpu().double().numpy(), float(u[t]))
            assert margin < 1e-9 or int(tokens[t]) == token


def test_a_stream_of_another_device_is_refused(tq):
    from types import SimpleNamespace
    st = SimpleNamespace(device=torch.device("cuda", torch.cuda.current_device() + 1), cuda_stream=0)
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    q, s = tq.fp8_quantize(x, 1)
    for call in (lambda: tq.fp8_quantize(x, 1, stream=st), lambda: tq.rms_norm(x, torch.ones(256, device="cuda"), 1e-6, stream=st),
                 lambda: tq.fp8_linear(q, s, q, s[:1].contiguous(), stream=st),
                 lambda: tq.sample(torch.zeros((2, 8), device="cuda"), torch.zeros(2, device="cuda"), stream=st)):
        with pytest.raises(tq.MoeError) as e:
            call()
        assert e.value.code == -1 and "stream" in str(e.value)
