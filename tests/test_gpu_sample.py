"""GPU parity of the sampler against the float64 oracle, through the binding.

Tokens are equal wherever the oracle's decisions are further than 1e-9 of the
mass from going the other way: the kernel's weights are integers in units of
2^-35 of their bin's largest, off by one unit, so a weight and a sum of weights is
good to e^(1/16) 2^-35, 3e-11 of itself; the oracle's own sums are good to 1e-12.  Probabilities are
fp32: half a step, 2^-24, and the same 1e-9.
"""
import sys

import numpy as np
import pytest

from oracle import sampler

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


NAMES = ("temperature", "top_k", "top_p", "min_p")
OFF = {"temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0}


def run(tq, logits, u, **settings):
    """The kernel on a numpy or torch matrix; settings are lists or None."""
    dev = {k: None if settings.get(k) is None else
           torch.tensor(settings[k], dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda")
           for k in NAMES}
    tokens, probs = tq.sample(logits, torch.tensor(u, dtype=torch.float32, device="cuda"), **dev)
    return tokens.cpu().numpy(), probs.cpu().numpy().astype(np.float64)


def check(tq, logits, u, least=0.9, **settings):
    """Every row against the oracle; at least this share of the rows must be decided."""
    tokens, probs = run(tq, logits, u, **settings)
    rows = logits.cpu().to(torch.float64).numpy()
    decided = 0
    for b in range(len(rows)):
        s = {k: OFF[k] if settings.get(k) is None else settings[k][b] for k in NAMES}
        for k in ("temperature", "top_p", "min_p"):
            s[k] = float(np.float32(s[k]))
        token, prob, margin = sampler.sample_row(rows[b], float(np.float32(u[b])), **s)
        if margin > 1e-9:
            decided += 1
            assert tokens[b] == token, (b, s, u[b], margin)
            assert abs(probs[b] - prob) <= (2.0 ** -24 + 1e-9) * prob
    assert decided >= least * len(rows)


def logits_of(B, V, seed, dtype=torch.float32, spread=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((B, V), generator=g, device="cuda") * spread).to(dtype)


SETTINGS = [dict(), dict(top_k=20), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=0.6, top_k=50, top_p=0.95),
            dict(temperature=1.5, top_p=0.5, min_p=0.01), dict(top_k=1), dict(temperature=0.0), dict(top_k=700),
            dict(temperature=0.1), dict(top_p=0.01), dict(top_k=5, top_p=0.99, min_p=0.3), dict(temperature=30.0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1, 2, 63, 1000, 4097, 50257])
def test_every_setting(tq, V, dtype):
    B = len(SETTINGS)
    say(f"sample {B} x {V} {dtype}")
    rng = np.random.default_rng(V)
    logits = logits_of(B, V, V, dtype)
    settings = {k: [s.get(k, OFF[k]) for s in SETTINGS] for k in NAMES}
    for _ in range(3):
        check(tq, logits, rng.random(B), **settings)


@pytest.mark.parametrize("B,V", [(1, 131072), (3, 200000), (40, 3000), (300, 700)])
def test_batches(tq, B, V):
    rng = np.random.default_rng(B)
    logits = logits_of(B, V, B)
    say(f"sample {B} x {V}")
    pick = [SETTINGS[i % len(SETTINGS)] for i in range(B)]
    check(tq, logits, rng.random(B), **{k: [s.get(k, OFF[k]) for s in pick] for k in NAMES})


@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.3, 10.0, 100.0])
def test_flat_and_peaked(tq, spread):
    """From all logits equal (every decision is a count) to one token with all the mass."""
    V = 30000
    settings = dict(temperature=[1.0] * 6, top_k=[0, 7, 0, 0, 3000, 0], top_p=[1.0, 1.0, 0.3, 0.9, 0.5, 1.0],
                    min_p=[0.0, 0.0, 0.0, 0.0, 0.0, 0.9])
    check(tq, logits_of(6, V, 1, spread=spread), np.random.default_rng(2).random(6), **settings)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_full_borders(tq, dtype):
    """A long vocabulary so even that every border lies among thousands of near-equal logits."""
    V = 180001
    settings = dict(temperature=[1.3] * 7, top_k=[0, 0, 60000, 0, 90000, 0, 170000], top_p=[0.5, 1.0, 1.0, 0.99, 0.7, 0.2, 1.0],
                    min_p=[0.0, 0.0, 0.0, 0.3, 0.2, 0.0, 0.5])
    check(tq, logits_of(7, V, 3, dtype, spread=1.0), np.random.default_rng(5).random(7), **settings)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [70001, 300001])
def test_borders_anywhere(tq, V, dtype):
    """More and fewer chunks than a row's block keeps bounds of; borders near logits of zero and of powers of two."""
    logits = logits_of(8, V, 9, dtype, spread=1.0)
    logits[4:] = (logits[4:] * 0.05 + torch.tensor([[-0.0], [2.0], [-4.0], [0.25]], device="cuda")).to(dtype)
    settings = dict(temperature=[1.0, 0.5, 0.7, 2.0, 0.05, 0.01, 1.0, 0.02], top_k=[0, 5000, 0, 0, 0, 30000, 60000, 0],
                    top_p=[0.6, 1.0, 0.9, 0.5, 0.5, 0.9, 0.3, 0.8], min_p=[0.0, 0.001, 0.02, 0.1, 0.0, 0.05, 0.9, 0.4])
    check(tq, logits, np.random.default_rng(8).random(8), **settings)


def test_temperatures(tq):
    V, t = 9000, [1e-38, 1e-30, 1e-6, 1e-5, 1e-2, 300.0, 1e30, 3e38, float("inf")]
    for settings in (dict(), dict(top_k=[700] * 9), dict(top_p=[0.7] * 9), dict(min_p=[0.5] * 9, top_k=[8000] * 9)):
        check(tq, logits_of(9, V, 12), np.random.default_rng(3).random(9), temperature=t, **settings)


def test_ties_take_the_lowest_index(tq):
    V = 5000
    logits = torch.zeros((5, V), device="cuda")
    logits[:, 1::7] = -0.0                               # -0 is +0
    logits[1, 100:200] = 2.0
    tokens, probs = run(tq, logits, [0.5, 0.505, 0.5, 0.5, 0.999], top_k=[10, 40, 1, 0, 0],
                        temperature=[1.0, 1.0, 1.0, 0.0, 1.0], top_p=[1.0, 1.0, 1.0, 1.0, 0.25])
    assert tokens.tolist() == [5, 120, 0, 0, int(0.999 * 1250)]
    assert np.allclose(probs, [0.1, 1 / 40, 1.0, 1.0, 1 / 1250])
    few = torch.tensor([[1.0, 3.0, 3.0, 1.0, 3.0, 3.0]], device="cuda").repeat(4, 1)
    tokens, _ = run(tq, few, [0.0, 0.49, 0.5, 0.99], top_k=[2] * 4)
    assert tokens.tolist() == [1, 1, 2, 2]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_masked_rows(tq, dtype):
    inf, V = float("inf"), 3000
    logits = logits_of(9, V, 5, dtype)
    logits[0] = -inf                                      # nothing left
    logits[1] = float("nan")
    logits[2] = -inf
    logits[2, 2999] = -5.0                                # one left
    logits[3] = torch.finfo(dtype).min                    # a mask of the type's lowest value, everywhere
    logits[4] = torch.finfo(dtype).min
    logits[4, 17] = 1.0
    logits[5, ::2] = float("nan")
    logits[6, [10, 400]] = inf
    logits[7, 1:] = -inf
    logits[8, :2500] = -inf
    u = [0.3, 0.3, 0.9, 0.5, 0.7, 0.4, 0.6, 0.2, 0.8]
    for settings in (dict(), dict(top_k=[5] * 9), dict(top_p=[0.5] * 9), dict(min_p=[0.2] * 9), dict(temperature=[0.0] * 9)):
        tokens, probs = run(tq, logits, u, **settings)
        assert tokens[:3].tolist() == [-1, -1, 2999] and probs[:3].tolist() == [0.0, 0.0, 1.0]
        assert tokens[4] == 17 and tokens[7] == 0
        assert tokens[6] == (10 if "temperature" in settings or "top_p" in settings else 400)
        assert probs[6] == (1.0 if "temperature" in settings or "top_p" in settings else 0.5)
    check(tq, logits, u)
    check(tq, logits, u, top_k=[3000] * 9, top_p=[0.9] * 9)


def test_u_and_settings_at_their_ends(tq):
    nan, inf = float("nan"), float("inf")
    logits = torch.log(torch.tensor([[0.5, 0.1, 0.4]], device="cuda")).repeat(8, 1)
    u = [0.0, 1.0, 2.0, -1.0, nan, 0.9999999, 0.55, 0.95]
    tokens, _ = run(tq, logits, u)
    assert tokens.tolist() == [0, 1, 1, 0, 0, 1, 2, 1]
    u = [0.95] * 8
    assert run(tq, logits, u, top_k=[-5, 0, 3, 4, 2**31 - 1, -2**31, 2, 1])[0].tolist() == [1, 1, 1, 1, 1, 1, 2, 0]
    assert run(tq, logits, u, top_p=[1.0, 2.0, nan, 0.0, -1.0, inf, 0.4, 0.6])[0].tolist() == [1, 1, 1, 0, 0, 1, 0, 2]
    assert run(tq, logits, u, min_p=[0.0, -1.0, nan, 1.0, 2.0, inf, 0.5, 0.9])[0].tolist() == [1, 1, 1, 0, 0, 0, 2, 0]
    assert run(tq, logits, u, temperature=[0.0, -1.0, nan, 1e-30, 1.0, 1e30, 1.0, 1.0])[0].tolist() == [0, 0, 0, 0, 1, 1, 1, 1]


def test_padded_rows_and_given_outputs(tq):
    V = 777
    buf = torch.full((6, V + 5), 1000.0, device="cuda")
    buf[:, 2:2 + V] = logits_of(6, V, 8)
    view = buf[:, 2:2 + V]
    u = torch.linspace(0.1, 0.9, 6, device="cuda")
    want = tq.sample(view.contiguous(), u)
    tokens = torch.full((10,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((10,), -7.0, device="cuda")
    tq.sample(view, u, tokens=tokens[2:8], probs=probs[2:8])
    assert torch.equal(tokens[2:8], want[0]) and torch.equal(probs[2:8], want[1])
    assert bool((tokens[[0, 1, 8, 9]] == -7).all()) and bool((probs[[0, 1, 8, 9]] == -7).all())
    one = tq.sample(view[3:4], u[3:4])
    assert one[0][0] == want[0][3]


def test_rows_do_not_depend_on_the_batch(tq):
    """The decisions are integer sums: a row's token is the same alone and in a batch."""
    B, V = 70, 9000
    logits, u = logits_of(B, V, 11), torch.rand(B, device="cuda")
    p = torch.full((B,), 0.93, device="cuda")
    all_t, _ = tq.sample(logits, u, top_p=p)
    for b in (0, 13, 69):
        t, _ = tq.sample(logits[b:b + 1], u[b:b + 1], top_p=p[b:b + 1])
        assert t[0] == all_t[b]


def test_long_vocabulary_and_far_rows(tq):
    """The largest vocabulary, and a row stride that passes 32 bits of bytes."""
    V = 1 << 21
    logits = logits_of(2, V, 3, torch.bfloat16)
    check(tq, logits, [0.3, 0.9], least=0.5, top_p=[0.9, 1.0])
    far = torch.zeros((3, (1 << 30) + 8), dtype=torch.bfloat16, device="cuda")
    far[:, :100] = logits_of(3, 100, 4, torch.bfloat16)
    check(tq, far[:, :100], [0.3, 0.6, 0.9])
    del far
    torch.cuda.empty_cache()


def test_empty_batch(tq):
    tokens, probs = tq.sample(torch.empty((0, 100), device="cuda"), torch.empty(0, device="cuda"))
    assert tokens.shape == (0,) and probs.shape == (0,)


def test_binding_refusals(tq):
    x, u = torch.zeros((2, 100), device="cuda"), torch.zeros(2, device="cuda")

    def code(f):
        with pytest.raises(tq.MoeError) as e:
            f()
        return e.value.code
    assert code(lambda: tq.sample(x.double(), u)) == -2
    assert code(lambda: tq.sample(x, u[:1])) == -3
    assert code(lambda: tq.sample(x.t(), torch.zeros(100, device="cuda"))) == -1
    assert code(lambda: tq.sample(x, u, top_k=u)) == -2
    assert code(lambda: tq.sample(x, u, temperature=u.cpu())) == -1
    assert code(lambda: tq.sample(x, u, tokens=torch.zeros(2, dtype=torch.int64, device="cuda"))) == -2
    assert code(lambda: tq.sample(torch.zeros((1, 0), device="cuda"), u[:1])) == -3
