"""GPU parity of attention of one fp16 token over e4m3 caches whose scales lie anywhere in fp32.

The tolerance is that of tests/test_gpu_attention_decode.py but for fp16's smallest numbers.  A
weight times its value's scale is rounded to fp16, held so that the largest so far is 2^7 or more.
Below 2^-14 it is off by 2^-25 instead of half a step of itself, which is 2^-32 of the largest:
with R the largest of these over the sum of the weights, each met by a code of at most 448,
2^-32 448 n R (and 2^-65 448 n, since products below 2^-33 count as that and the sum of the weights
is 1 or more); and y, rounded once, by 2^-25.  Bringing a product to that range costs a
multiplication and an exponential whose argument is below 48 (34 e), and every move of the
largest, by 2^8 or more and so no more than 20 times, 3 e: 100 e A together, A = sum p |v|.
"""
import numpy as np
import pytest

from oracle import attention
from test_gpu_attention import E, F16, host, ints, lse_tolerance, say, tq  # noqa: F401
from test_gpu_attention_decode import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -11


def close(got, want, D, n, small):
    """small: the bound on what fp16's smallest numbers cost."""
    d = (2 * D + 7) * E * want["score"][..., None]
    tol = U * want["size"] + U * np.abs(want["y"]) + (4 * d + (110 + 4 * n) * E) * want["size"] + small + 2.0 ** -25
    bad = ~(np.abs(got - want["y"]) <= 1.01 * tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want["y"][bad][:5], tol[bad][:5])


def close_lse(lse, want, D, n):
    assert np.all(np.abs(host(lse) - want["lse"]) <= 2 * lse_tolerance(want, D, n))


def largest_share(c, b):
    """Of sequence b and every head: the largest weight times its value's scale, over the sum of the
    weights."""
    q, k, n = host(c.q)[b], c.cached("k", b), c.lens[b]
    H, G = q.shape[0], q.shape[0] // k.shape[1]
    at = torch.from_numpy(c.table_host[b, : -(-n // c.P)]).cuda()
    vs = c.scales["v_scales"][at].double().transpose(1, 2).flatten(0, 1)[:n].cpu().numpy()
    out = np.empty((H, 1))
    for h in range(H):
        s = c.D ** -0.5 * (k[:, h // G] * q[h]).sum(1)
        p = np.exp(s - s.max())
        out[h] = (p * vs[:, h // G]).max() / p.sum()
    return out


def check(c, y, lse=None):
    want = c.oracle()
    got = host(y)
    for b, n in enumerate(c.lens):
        if n == 0:
            continue
        one = {x: want[x][b:b + 1] for x in want}
        close(got[b:b + 1], one, c.D, n, 448 * n * (2.0 ** -32 * largest_share(c, b) + 2.0 ** -65))
        if lse is not None:
            close_lse(lse[b:b + 1], one, c.D, n)


@pytest.mark.parametrize("factor", [1e-6, 1e-5, 1e-4, 1e-3, 1e-2, 0.1, 100.0, 5000.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_of_any_size(tq, D, factor):
    """One token, a few, many, and sequences that several workers share."""
    say(f"e4m3 values of {factor}, dim {D}")
    c = Case(tq, 31, [1, 0, 77, 700, 3000], 4, 2, D, 16, F16, True)
    c.scales["v_scales"].mul_(factor)
    lse = torch.empty((len(c.lens), 4), device="cuda")
    check(c, c.run(lse=lse), lse)


@pytest.mark.parametrize("low,high", [(-6, 2), (-9, -3), (-4, 4)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_that_differ_from_token_to_token(tq, D, low, high):
    say(f"e4m3 values of 1e{low} to 1e{high}, dim {D}")
    c = Case(tq, 32, [5, 300, 2500], 6, 2, D, 32, F16, True)
    s = c.scales["v_scales"]
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    s.mul_(10.0 ** (low + (high - low) * torch.rand(s.shape, generator=g, device="cuda")))
    check(c, c.run())


def test_strong_keys_with_values_of_zero(tq):
    """A row of zeros has the smallest scale there is; it may have nearly all of the weight."""
    say("e4m3 zeros with the weight")
    c = Case(tq, 33, [200, 600, 1500], 4, 2, 64, 16, F16, True)
    c.q.copy_(c.q.abs() + 0.1)
    c.k.view(torch.uint8)[:] = 0                         # weak keys score 0
    c.scales["v_scales"].mul_(0.01)
    for b, n in enumerate(c.lens):
        for i in (0, 70, n - 1):
            page, place = int(c.table_host[b, i // 16]), i % 16
            c.k.view(torch.uint8)[page, :, place] = 0x38     # 1
            c.scales["k_scales"][page, :, place] = 0.8 + 0.1 * (i % 3)
            c.v.view(torch.uint8)[page, :, place] = 0
            c.scales["v_scales"][page, :, place] = 1e-30 / 448
    lse = torch.empty((3, 4), device="cuda")
    check(c, c.run(lse=lse), lse)


def test_large_scales_behind_a_rising_maximum(tq):
    """Scores that rise by just under the 2^8 that the maximum may lag, scales of 2^10 beside small
    codes: the results are within fp16, and so is all that leads there."""
    n, P, B, D = 768, 64, 256, 64
    say("e4m3 scales of 1024")
    k = torch.zeros((n, 1, D), device="cuda")
    k[256:, 0, 0] = 5.5                                  # 2^7.93 of the weight of the first 256
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    v = torch.randint(-1, 3, (n, 1, D), generator=g, device="cuda").float()
    q = torch.zeros((1, 1, D), device="cuda")
    q[..., 0] = 1.0
    pages = [x.view(n // P, P, 1, D).transpose(1, 2).contiguous().to(torch.float8_e4m3fn) for x in (k, v)]
    ks = torch.ones((n // P, 1, P), device="cuda")
    tables = torch.arange(n // P, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    y = tq.attention_decode(q.to(F16).expand(B, 1, D).contiguous(), *pages, tables, ints([n] * B), k_scales=ks,
                            v_scales=1024 * ks, scale=1.0)
    want = attention.attend(host(q), host(k), 1024 * host(v), [n - 1], 1.0)
    for b in (0, 255):
        close(host(y)[b:b + 1], want, D, n, 448 * n * 2.0 ** -32 * 1024)


def test_scales_in_a_graph_and_shared_workspaces(tq):
    """Replays over other scales give what a call on them gives."""
    say("e4m3 scales in a graph")
    c = Case(tq, 34, [900, 31, 0, 2000], 8, 2, 128, 32, F16, True)
    need = tq.lib().moe_attention_decode_workspace_bytes(4, 8, 2, 128)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(c.q)
    c.run(y=y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(y=y, workspace=ws)
    for factor in (1e-4, 1e3, 1e-5):
        c.scales["v_scales"].mul_(factor)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        check(c, y)
        assert torch.equal(y, c.run())
