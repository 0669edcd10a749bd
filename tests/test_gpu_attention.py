"""GPU parity of attention over whole prompts against the float64 oracle.

Tolerance, u the half step of the 16-bit type (bf16 2^-8, fp16 2^-11), e = 2^-24 the
fp32 half step.  With A = sum p |v|:
  * every weight is rounded once to the type: u A; y once: u |y|;
  * a score is a sum of head_dim exact products in fp32, each addition off by at most
    2 e of the magnitudes summed (the matrix core's adder may cut), and is scaled by c =
    scale log2 e (3 e) and subtracted (2 e of the larger operand): the exponent is off by
    d = (2 head_dim + 5) e S with S the largest scale sum |q k|, and its exponential, with
    the instruction's own 2 e, by d + 2 e; weight and sum each carry that: 2 (d + 2 e) A;
  * the sum of n weights and the products' sums over n keys: each addition 2 e: 4 n e A;
  * fp16 below its smallest normal number is off by 2^-25 instead: of n weights, which are
    relative to a sum of at least 1 (the largest weight is 1 or more): 2^-25 n max |v|, and
    of y 2^-25.
The logarithm of the sum is off by d + 4 n e, its own steps by 8 e of its terms.
"""
import sys

import numpy as np
import pytest

from oracle import attention

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24
BF16, F16 = torch.bfloat16, torch.float16


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_quantized_moe_amd as tq
    tq.lib()
    return tq


def host(t):
    return t.detach().cpu().to(torch.float64).numpy()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def starts_of(lens, first=0):
    return ints(np.concatenate([[first], first + np.cumsum(lens)]).tolist())


def tolerance(r, dtype, D, n, vmax):
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -11
    d = (2 * D + 5) * E * r["score"][..., None]
    tol = u * r["size"] + u * np.abs(r["y"]) + (2 * d + 4 * E + 4 * n * E) * r["size"]
    if dtype == F16:
        tol = tol + 2.0 ** -25 * (n * vmax + 1)
    return 1.01 * tol


def lse_tolerance(r, D, n):
    big = np.where(np.isfinite(r["lse"]), np.abs(r["lse"]), 0)
    return 1.01 * ((2 * D + 5) * E * r["score"] + 4 * n * E + 8 * E * (big + r["score"] + np.log(n + 1) + 1))


def inputs(seed, lens, k_lens, H, Hk, D, dtype, spread=1.5):
    """q, k, v as slices of one matrix where the lengths agree."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    n, m = sum(lens), sum(k_lens)
    if lens == k_lens:
        x = r(n, H + 2 * Hk, D).to(dtype)
        x[:, :H] *= spread
        return x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    kv = r(m, 2 * Hk, D).to(dtype)
    return (spread * r(n, H, D)).to(dtype), kv[:, :Hk], kv[:, Hk:]


def oracle_of(q, k, v, lens, k_lens, causal, scale):
    q, k, v = host(q), host(k), host(v)
    out, a, b = [], 0, 0
    for n, m in zip(lens, k_lens):
        last = np.arange(n) + m - n if causal else np.full(n, m - 1)
        out.append(attention.attend(q[a:a + n], k[b:b + m], v[b:b + m], last, scale))
        a, b = a + n, b + m
    return {x: np.concatenate([r[x] for r in out]) for x in out[0]}


def check(got, lse, want, dtype, D, n, vmax):
    got = host(got)
    tol = tolerance(want, dtype, D, n, vmax)
    bad = ~(np.abs(got - want["y"]) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want["y"][bad][:5], tol[bad][:5])
    if lse is not None:
        lse = host(lse)
        none = want["lse"] == -np.inf
        assert np.all(lse[none] == -np.inf)
        with np.errstate(invalid="ignore"):
            assert np.all((np.abs(lse - want["lse"]) <= lse_tolerance(want, D, n)) | none)


LENS = {"one": [1], "empty": [0, 1, 2, 0, 33, 0], "tile-ends": [31, 32, 33, 63, 64, 65], "block-ends": [127, 128, 129],
        "long": [517]}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", list(LENS))
@pytest.mark.parametrize("D,dtype", [(64, BF16), (64, F16), (128, BF16), (128, F16), (256, BF16), (256, F16)])
def test_prompts(tq, D, dtype, name, causal):
    lens, H, Hk = LENS[name], 4, 2
    say(f"prompts {lens} dim {D} {dtype} causal {causal}")
    q, k, v = inputs(1, lens, lens, H, Hk, D, dtype)
    lse = torch.empty((sum(lens), H), device="cuda")
    y = tq.attention_prefill(q, k, v, starts_of(lens), causal=causal, lse=lse)
    want = oracle_of(q, k, v, lens, lens, causal, D ** -0.5)
    check(y, lse, want, dtype, D, max(lens), float(v.abs().max()))


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (5, 1), (16, 1), (14, 2), (24, 8)])
def test_head_layouts(tq, H, Hk):
    say(f"heads {H} of {Hk}")
    lens = [70, 3]
    q, k, v = inputs(2, lens, lens, H, Hk, 64, BF16)
    y = tq.attention_prefill(q, k, v, starts_of(lens))
    check(y, None, oracle_of(q, k, v, lens, lens, True, 0.125), BF16, 64, 70, float(v.abs().max()))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_before_and_missing(tq, D, causal):
    """Chunks behind earlier keys; more queries than keys (the first see none); no keys."""
    lens, k_lens = [5, 40, 130, 7, 1, 200], [133, 40, 3, 0, 300, 71]
    say(f"lengths {lens} over {k_lens} dim {D} causal {causal}")
    q, k, v = inputs(3, lens, k_lens, 4, 2, D, BF16)
    lse = torch.empty((sum(lens), 4), device="cuda")
    y = tq.attention_prefill(q, k, v, starts_of(lens), starts_of(k_lens), causal=causal, lse=lse)
    want = oracle_of(q, k, v, lens, k_lens, causal, D ** -0.5)
    check(y, lse, want, BF16, D, max(k_lens), float(v.abs().max()))
    none = torch.from_numpy(want["lse"] == -np.inf).cuda()
    assert none.any() and torch.all(y[none] == 0)


@pytest.mark.parametrize("lens,k_lens", [([3], [5000]), ([33, 1, 0, 64], [3000, 1100, 500, 40]), ([200], [2100])])
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16), (256, BF16)])
def test_few_queries_share_many_keys(tq, D, dtype, lens, k_lens):
    """Several blocks have the keys of a tile of queries; the workspace holds rubbish before."""
    H, Hk = 4, 1
    say(f"shared keys {lens} over {k_lens} dim {D}")
    need = tq.lib().moe_attention_prefill_workspace_bytes(sum(lens), sum(k_lens), len(lens), H, Hk, D)
    assert need > 0
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    q, k, v = inputs(20, lens, k_lens, H, Hk, D, dtype)
    for causal in (True, False):
        lse = torch.empty((sum(lens), H), device="cuda")
        y = tq.attention_prefill(q, k, v, starts_of(lens), starts_of(k_lens), causal=causal, lse=lse, workspace=ws)
        want = oracle_of(q, k, v, lens, k_lens, causal, D ** -0.5)
        want["size"] = 2 * want["size"]           # the shares are scaled and added once more
        check(y, lse, want, dtype, D, max(k_lens), float(v.abs().max()))
        assert torch.equal(y, tq.attention_prefill(q, k, v, starts_of(lens), starts_of(k_lens), causal=causal))


def test_shared_keys_with_hidden_and_seen_infinities(tq):
    say("shared keys, infinities")
    q, k, v = (x.clone() for x in inputs(21, [40], [4000], 4, 2, 64, BF16, spread=0.1))
    v[3970:, 0], v[3999, 1] = float("nan"), float("inf")   # the last 30 keys: query 10 is the first to see one
    v[100, 1, 5], v[3900, 1, 6] = float("inf"), float("-inf")
    y = tq.attention_prefill(q, k, v, ints([0, 40]), ints([0, 4000]))
    assert torch.isfinite(y[:10, :2]).all() and torch.isnan(y[10:, :2]).all()
    assert torch.isfinite(y[:39, 2:, 7:]).all() and torch.all(y[39, 2:, 7:] == float("inf"))
    assert torch.all(y[:39, 2:, 5] == float("inf")) and torch.all(y[:39, 2:, 6] == float("-inf"))
    assert torch.isnan(y[39, 2:, 6]).all()


def test_graphs_share_a_workspace(tq):
    say("graphs share a workspace")
    a, b = inputs(22, [40], [3000], 4, 2, 64, BF16), inputs(23, [9], [5000], 4, 2, 64, BF16)
    starts = [(ints([0, 40]), ints([0, 3000])), (ints([0, 9]), ints([0, 5000]))]
    need = max(tq.lib().moe_attention_prefill_workspace_bytes(n, m, 1, 4, 2, 64) for n, m in ((40, 3000), (9, 5000)))
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    ys, graphs = [torch.empty((n, 4, 64), dtype=BF16, device="cuda") for n in (40, 9)], []
    for x, s, y in zip((a, b), starts, ys):
        tq.attention_prefill(*x, *s, y=y, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.attention_prefill(*x, *s, y=y, workspace=ws)
        graphs.append(g)
    for i in range(3):
        for x in (a, b):
            x[0].mul_(1 + 0.25 * i)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, s, y in zip((a, b), starts, ys):
            assert torch.equal(y, tq.attention_prefill(*x, *s))


def test_many_sequences(tq):
    """More sequences than lanes of a wave, most of them tiny or empty."""
    lens = [(7 * i) % 5 for i in range(300)]
    lens[211] = 150
    say("300 sequences")
    q, k, v = inputs(4, lens, lens, 2, 1, 64, BF16)
    y = tq.attention_prefill(q, k, v, starts_of(lens))
    check(y, None, oracle_of(q, k, v, lens, lens, True, 0.125), BF16, 64, 150, float(v.abs().max()))


@pytest.mark.parametrize("H,Hk", [(4096, 1), (4096, 4096)])
def test_most_heads(tq, H, Hk):
    say(f"{H} heads of {Hk}")
    lens = [40, 1, 3]
    q, k, v = inputs(22, lens, lens, H, Hk, 64, BF16)
    check(tq.attention_prefill(q, k, v, starts_of(lens)), None, oracle_of(q, k, v, lens, lens, True, 0.125), BF16, 64, 40,
          float(v.abs().max()))


def test_more_blocks_than_one_dimension(tq):
    """20000 sequences of one token and 64 heads of their own: 1.3 M blocks.  The one weight is off
    from 1 by the score's roundings, far below half a step of bf16, so y is v."""
    say("20000 sequences of one token")
    q, k, v = inputs(21, [20000], [20000], 64, 64, 64, BF16)
    y = tq.attention_prefill(q, k, v, torch.arange(20001, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, v)


def test_packing_does_not_matter(tq):
    lens = [129, 64, 1, 300]
    say("packed against alone")
    q, k, v = inputs(5, lens, lens, 4, 4, 128, BF16)
    y = tq.attention_prefill(q, k, v, starts_of(lens))
    at = 0
    for n in lens:
        alone = tq.attention_prefill(q[at:at + n], k[at:at + n], v[at:at + n], ints([0, n]))
        assert torch.equal(alone, y[at:at + n])
        at += n
    assert torch.equal(y, tq.attention_prefill(q.contiguous(), k.contiguous(), v.contiguous(), starts_of(lens)))


def test_tokens_outside_every_sequence_stay(tq):
    say("tokens outside")
    q, k, v = inputs(6, [100], [100], 2, 2, 64, BF16)
    y = torch.full((100, 2, 64), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((100, 2), 7.0, device="cuda")
    tq.attention_prefill(q, k, v, ints([10, 40, 40, 90]), y=y, lse=lse)
    for part in (slice(0, 10), slice(90, 100)):
        assert torch.all(y[part] == 7) and torch.all(lse[part] == 7)
    want = oracle_of(q[10:90], k[10:90], v[10:90], [30, 0, 50], [30, 0, 50], True, 0.125)
    check(y[10:90], lse[10:90], want, BF16, 64, 50, float(v.abs().max()))


def test_starts_outside_the_tokens(tq):
    """Ends beyond the tokens are taken as the last token's, falling starts as empty sequences."""
    say("odd starts")
    q, k, v = inputs(7, [100], [100], 2, 2, 64, BF16)
    y = torch.zeros((100, 2, 64), dtype=BF16, device="cuda")
    tq.attention_prefill(q, k, v, ints([-5, 60, 50, 1 << 30]), y=y)
    want = oracle_of(q[:50], k[:50], v[:50], [50], [50], True, 0.125)
    check(y[:50], None, want, BF16, 64, 100, float(v.abs().max()))


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16), (256, BF16)])
def test_hidden_values_do_not_reach(tq, D, dtype):
    """Keys and values of NaN and infinities after a query, and in another sequence."""
    say(f"hidden NaN, dim {D}")
    lens = [150, 90, 40]
    q, k, v = (x.clone() for x in inputs(8, lens, lens, 2, 1, D, dtype))
    nan, inf = float("nan"), float("inf")
    k[100], v[101], v[117, 0, 3], v[130, 0, 5], k[120, 0, 0] = nan, nan, inf, -inf, inf
    k[160:200], v[160:200] = nan, nan            # inside the second sequence
    v[279] = -inf                                # the last token of all
    y = tq.attention_prefill(q, k, v, starts_of(lens))
    want = oracle_of(q, k, v, lens, lens, True, D ** -0.5)
    clean = torch.ones(280, dtype=torch.bool)
    clean[100:150] = clean[160:240] = clean[279] = False
    got = host(y)
    tol = tolerance(want, dtype, D, 150, 8.0)[clean.numpy()]
    assert np.all(np.abs(got[clean.numpy()] - want["y"][clean.numpy()]) <= tol)
    assert torch.isnan(y[100:150]).all() and torch.isnan(y[160:240]).all()
    assert torch.all(y[279] == -inf)


@pytest.mark.parametrize("causal", [True, False])
def test_seen_infinities(tq, causal):
    """Infinite values that are seen give infinities of their sign, both signs NaN, channel by channel."""
    say(f"seen infinities, causal {causal}")
    q, k, v = (x.clone() for x in inputs(9, [77], [77], 2, 2, 64, BF16, spread=0.1))
    v[20, 0, 1], v[30, 0, 2], v[40, 0, 2], v[50, 0, 3] = float("inf"), float("inf"), float("-inf"), float("-inf")
    y = host(tq.attention_prefill(q, k, v, ints([0, 77]), causal=causal))
    want = oracle_of(q, k, v, [77], [77], causal, 0.125)
    fine = np.isfinite(want["y"])
    assert np.array_equal(np.nan_to_num(want["y"][~fine], nan=7.0), np.nan_to_num(y[~fine], nan=7.0))
    tol = tolerance({x: np.nan_to_num(want[x], posinf=0.0, neginf=0.0) for x in want}, BF16, 64, 77, 8.0)
    assert np.all(np.abs(y - want["y"])[fine] <= tol[fine])


def test_scores_of_minus_infinity(tq):
    """A key whose score is -inf has no weight; a query with no other gets zeros."""
    say("scores of -inf")
    q, k, v = (x.clone() for x in inputs(10, [80], [80], 1, 1, 64, BF16))
    q[:] = q.abs() + 0.1
    k[:10] = k[3] = float("-inf")
    k[60] = float("-inf")
    lse = torch.empty((80, 1), device="cuda")
    y = tq.attention_prefill(q, k, v, ints([0, 80]), lse=lse)
    assert torch.all(y[:10] == 0) and torch.all(lse[:10] == float("-inf"))
    want = attention.attend(host(q)[10:], np.delete(host(k)[10:], 50, 0), np.delete(host(v)[10:], 50, 0),
                            np.arange(70) - (np.arange(70) >= 50), 0.125)
    check(y[10:], lse[10:], want, BF16, 64, 80, 8.0)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_moving_maximum(tq, dtype):
    """Scores that rise and fall by hundreds over the keys, and far below zero throughout."""
    say(f"moving maximum {dtype}")
    n = 400
    q, k, v = (x.clone() for x in inputs(11, [n], [n], 2, 2, 64, dtype))
    q[..., 0], q[:, 1, 0] = 10.0, -10.0
    k[..., 0] = torch.linspace(-30, 30, n, device="cuda")[:, None].to(dtype)
    k[200:220, :, 0] = 35.0
    for shift in (0.0, -60.0):
        k[..., 1] = shift
        q[..., 1] = 20.0
        lse = torch.empty((n, 2), device="cuda")
        y = tq.attention_prefill(q, k, v, ints([0, n]), lse=lse)
        check(y, lse, oracle_of(q, k, v, [n], [n], True, 0.125), dtype, 64, n, float(v.abs().max()))


def test_scale_is_the_callers(tq):
    say("scale")
    q, k, v = inputs(12, [90], [90], 2, 2, 128, BF16)
    for scale in (1e-3, 0.7):
        y = tq.attention_prefill(q, k, v, ints([0, 90]), scale=scale)
        check(y, None, oracle_of(q, k, v, [90], [90], True, scale), BF16, 128, 90, float(v.abs().max()))


def test_a_row_of_nan_stays_its_own(tq):
    say("NaN query")
    q, k, v = (x.clone() for x in inputs(13, [70], [70], 2, 2, 64, BF16))
    y = tq.attention_prefill(q, k, v, ints([0, 70]))
    q[33, 1] = float("nan")
    z = tq.attention_prefill(q, k, v, ints([0, 70]))
    assert torch.isnan(z[33, 1]).all()
    y[33, 1] = z[33, 1] = 0
    assert torch.equal(y, z)


def test_offsets_past_32_bits(tq):
    """Keys and values more than 4 GiB apart."""
    say("far keys")
    n, stride = 400, 1 << 23                      # 16 MiB from token to token
    far = torch.empty((n, stride), dtype=BF16, device="cuda")
    q, k, v = inputs(14, [n], [n], 2, 2, 64, BF16)
    kf, vf = far[:, :128].view(n, 2, 64), far[:, 256:384].view(n, 2, 64)
    kf.copy_(k)
    vf.copy_(v)
    y = tq.attention_prefill(q, kf, vf, ints([0, n]))
    assert torch.equal(y, tq.attention_prefill(q, k, v, ints([0, n])))


def test_given_buffers_and_stream(tq):
    say("stream")
    lens = [200, 33]
    q, k, v = inputs(15, lens, lens, 4, 2, 128, F16)
    s = starts_of(lens)
    want = tq.attention_prefill(q, k, v, s)
    side, y = torch.cuda.Stream(), torch.empty_like(want)
    side.wait_stream(torch.cuda.current_stream())
    assert tq.attention_prefill(q, k, v, s, y=y, stream=side) is y
    again = tq.attention_prefill(q, k, v, s, stream=side)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(again, want)


def test_captured(tq):
    """In a HIP graph, with inputs that change between the replays."""
    say("graph")
    lens = [100, 29]
    q, k, v = (x.clone() for x in inputs(16, lens, lens, 4, 2, 128, BF16))
    s = starts_of(lens)
    y = torch.empty((129, 4, 128), dtype=BF16, device="cuda")
    tq.attention_prefill(q, k, v, s, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.attention_prefill(q, k, v, s, y=y)
    for i, cut in enumerate((100, 1, 128, 64)):
        s.copy_(ints([0, cut, 129]))
        q.mul_(1 + 0.1 * i)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tq.attention_prefill(q, k, v, s))


def test_refusals(tq):
    say("refusals")
    q, k, v = inputs(17, [10], [10], 4, 2, 64, BF16)
    s = ints([0, 10])
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(v=v[:9]), dict(k=k[..., :32]), dict(k=k[:, :1]),
                dict(starts=s.long()), dict(starts=s.cpu()), dict(k_starts=ints([0, 5, 10])), dict(scale=0.0),
                dict(scale=float("nan")), dict(q=q.cpu()), dict(y=torch.empty((10, 4, 64), device="cuda")),
                dict(q=q[..., ::2].repeat(1, 1, 2)[..., ::2]), dict(lse=torch.empty((4, 10), device="cuda")),
                dict(y=q.contiguous()[:, :2].contiguous())):
        args = dict(q=q, k=k, v=v, starts=s, k_starts=None, scale=None)
        args.update(bad)
        with pytest.raises(tq.MoeError):
            tq.attention_prefill(**args)
    whole = torch.empty((10, 4, 64), dtype=BF16, device="cuda")
    with pytest.raises(tq.MoeError, match="overlaps"):
        tq.attention_prefill(whole, k, v, s, y=whole)
    assert tq.attention_prefill(q[:0], k, v, ints([0, 0])).shape == (0, 4, 64)
    assert tq.attention_prefill(q, k, v, ints([0])).shape == (10, 4, 64)
