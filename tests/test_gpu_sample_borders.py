"""GPU parity of the sampler where a row's decisions lie at the ends of its bins,
against the float64 oracle, through the binding.

Tokens are equal wherever the oracle's decisions are further than 1e-9 of the
mass from going the other way, and probabilities agree to half an fp32 step,
2^-24, and the same 1e-9: a weight is good to 4e-11 of itself, and so is every
sum of weights.
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


OFF = {"temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0}


def check(tq, logits, u, least=0.9, margin=1e-9, **settings):
    """Every row of a float32 matrix against the oracle, with one setting each for all rows or a list of them; at
    least this share of the rows must be decided by more than the margin."""
    rows = np.asarray(logits, np.float32)
    B = len(rows)
    u = np.broadcast_to(np.asarray(u, np.float32), B)
    per = {k: np.broadcast_to(np.asarray(settings.get(k, OFF[k]), np.int32 if k == "top_k" else np.float32), B)
           for k in OFF}
    dev = {k: torch.tensor(v.copy(), device="cuda") for k, v in per.items()}
    tokens, probs = tq.sample(torch.tensor(rows, device="cuda"), torch.tensor(u.copy(), device="cuda"), **dev)
    tokens, probs = tokens.cpu().numpy(), probs.cpu().numpy().astype(np.float64)
    decided = 0
    for b in range(B):
        s = {k: v[b].item() for k, v in per.items()}
        token, prob, m = sampler.sample_row(rows[b], float(u[b]), **s)
        if m > margin:
            decided += 1
            if u[b] >= 1 and tokens[b] != token:
                # The last token with mass: one lighter than 2^-43 of the largest weight may count as having
                # none, so the answer may be any from the last heavier token on.
                down = (rows[b].max().astype(np.float64) - rows[b]) / s["temperature"]
                reach = np.where(down > 43 * np.log(2), -np.inf, rows[b])
                near = sampler.sample_row(reach, float(u[b]), **s)[0]
                got = rows[b, tokens[b]].item()
                assert rows[b, token] <= got <= rows[b, near], (b, s, u[b])
                prob *= np.exp((got - rows[b, token].item()) / s["temperature"])
            else:
                assert tokens[b] == token, (b, s, u[b], m)
            assert abs(probs[b] - prob) <= (2.0 ** -24 + 1e-9) * prob, (b, s, u[b])
    assert decided >= least * B


def test_top_k_beyond_the_tokens_with_mass(tq):
    """A count that no bin reaches, and a border by mass right behind it."""
    rng = np.random.default_rng(1)
    B, V = 256, 3000
    masked = np.full((B, V), -np.inf, np.float32)
    for b in range(B):
        at = rng.choice(V, 20, replace=False)
        masked[b, at] = rng.normal(size=20) * 3
    spread = (rng.normal(size=(B, V)) * 30).astype(np.float32)
    for settings in (dict(), dict(top_p=0.9), dict(min_p=0.05), dict(top_p=0.95, min_p=0.01), dict(temperature=0.3)):
        say("top-k beyond the mass", settings)
        check(tq, masked, rng.random(B), top_k=50, **settings)
        check(tq, spread, rng.random(B), top_k=700, **settings)


def gapped_rows(seed, B, V):
    """Rows whose bins of 1 / 16 nat have gaps: peaked ones of 50 tokens and up, and few likely tokens over a flat rest."""
    rng = np.random.default_rng(seed)
    rows = np.full((B, V), -np.inf)
    for b in range(B):
        if b % 2:
            n = int(rng.integers(50, V))
            rows[b, :n] = rng.normal(size=n) * rng.uniform(1, 6)
        else:
            rows[b, :V - 8] = -3.05
            rows[b, V - 8:] = rng.uniform(-2, 0, 8)
        rng.shuffle(rows[b])
    return rows.astype(np.float32)


@pytest.mark.parametrize("seed", [11, 12])  # rows 145, 425 and 501 of the second: a fp64 scan's sum of an empty bin
@pytest.mark.parametrize("u", [1.0, 2.0, float("inf"), 0.0, 0.9999999])  # lies above that of the bin before it
def test_borders_where_a_bin_is_empty(tq, u, seed):
    """u of 1 or more behind a min-p border that keeps nothing of its bin."""
    say("borders beside empty bins, u", u)
    rows = gapped_rows(seed, 600, 2000)
    check(tq, rows, u, min_p=0.05)
    check(tq, rows[:200], u, min_p=0.03, top_p=0.9)
    # 1.2e-7 of the mass before its end many steps are shorter than the margin (the oracle alone says how many)
    check(tq, rows[:200], u, least=0.75 if 0.9 < u < 1 else 0.9)


def test_last_token_with_mass(tq):
    """A tail too light to show in the row's sum still ends with its last token."""
    rng = np.random.default_rng(4)
    rows = np.concatenate([rng.uniform(-0.01, 0, (4, 20000)), -rng.uniform(25, 30, (4, 30))], axis=1)
    rows = rng.permuted(rows, axis=1).astype(np.float32)
    check(tq, rows, [1.0, 1.5, 3.0, float("inf")])
    check(tq, rows, 1.0, top_k=20010)


def test_rows_across_the_end_of_the_grid(tq):
    """Rows whose l / T lies around -2^18 and 2^18, where bins of 1 / 16 nat end to be numbered: their chunks lie on
    both sides of it."""
    V, step = 6000, 0.03125
    row = np.full(V, -262144.0 - step, np.float32)
    row[0] = -262144.0
    check(tq, row[None].repeat(3, 0), [0.9, 0.3, 0.0])
    rng = np.random.default_rng(6)
    for sign in (-1, 1):
        say("around the end of the grid", sign)
        top = sign * 262144.0 + np.arange(-40, 41, 4)[:, None]
        rows = top - step * rng.integers(0, 900, (len(top), V)) * rng.random((len(top), V)) ** 3 // step * step
        rows = rows.astype(np.float32)
        assert np.all(np.abs(rows / step) < 2 ** 24)
        for settings in (dict(), dict(top_p=0.8), dict(top_k=4000, min_p=0.01)):
            check(tq, rows, rng.random(len(top)), **settings)
        small = (rows * 2.0 ** -17).astype(np.float32)                      # the same at a temperature of 2^-17
        check(tq, small, rng.random(len(top)), temperature=2.0 ** -17, top_p=0.95)


@pytest.mark.parametrize("temperature", [1.0, 0.7, 1e-7])  # the last off the grid
def test_equal_logits_are_counted(tq, temperature):
    """Tokens of equal weight: u and top-p on the border between two of them are exact."""
    rng = np.random.default_rng(8)
    B, V = 400, 4096
    rows, share = np.full((B, V), -np.inf, np.float32), np.empty(B, np.float32)
    for b in range(B):
        parts = 1 << int(rng.integers(1, 6))
        n = parts * int(rng.integers(1, 1 + (V if b % 4 == 0 else 128) // parts))
        rows[b, rng.choice(V, n, replace=False)] = rng.normal() * 5
        share[b] = rng.integers(1, parts) / parts                          # n share is a whole number
    say("equal logits", temperature)
    check(tq, rows, share, least=1.0, temperature=temperature)
    check(tq, rows, np.float32(0.999999), least=1.0, temperature=temperature, top_p=share)
    check(tq, rows, rng.random(B), least=1.0, temperature=temperature, top_p=share, top_k=V // 2)


def outside_its_bin(l, t):
    """How far l / T lies outside the bin of 1 / 16 nat that a product in fp32 puts it into, in bins."""
    y = float(l) * 16 / float(t) - float(np.floor(np.float32(l) * np.float32(16 / float(t))))
    return max(-y, y - 1)


@pytest.mark.parametrize("far", [1e3, 2.0 ** 17, 2.0 ** 18 - 33])
def test_weights_of_far_logits(tq, far):
    """Rows of two logits whose l / T is `far` and a little more, each at the edge of its bin: u is put 1.6e-10 to
    3e-10 of the mass from the border between two tokens.  Two weights good to 4e-11 move it by 8e-11 at most."""
    rng = np.random.default_rng(int(far))
    V, per_row = 50000, 16
    say("far logits", far)
    rows, us, ts, want = [], [], [], []
    for sign in (-1, 1, -1, 1, -1, 1, -1, 1):
        tries = []
        for _ in range(2000):
            t = np.float32(rng.uniform(0.01, 3))
            hi = np.float32(sign * far * t * rng.uniform(0.97, 0.999))
            lo = np.float32(hi - t * rng.uniform(0.3, 1.5))
            tries.append((max(outside_its_bin(hi, t), outside_its_bin(lo, t)), t, hi, lo))
        _, t, hi, lo = max(tries)
        assert lo < hi and abs(float(lo) / float(t)) < 2 ** 18 - 32
        n0 = V // 4
        r = np.exp((float(lo) - float(hi)) / float(t))
        total = n0 + (V - n0) * r
        u = rng.permutation(1 << 24) / 2.0 ** 24
        u = u[u * total > n0 + 0.3 * (V - n0) * r]
        place = (u * total - n0) / r                                       # the answer is n0 + floor(place)
        off = np.abs(place - np.round(place)) * r / total
        u, place = (v[(off > 1.6e-10) & (off < 3e-10)][:per_row] for v in (u, place))
        assert len(u) == per_row
        for x, i in zip(u, place):
            rows.append(np.where(np.arange(V) < n0, hi, lo))
            us.append(x)
            ts.append(t)
            want.append(n0 + int(np.floor(i)))
    dev = [torch.tensor(np.array(v, np.float32), device="cuda") for v in (rows, us, ts)]
    tokens, _ = tq.sample(dev[0], dev[1], temperature=dev[2])
    assert tokens.tolist() == want


def test_rows_off_the_grid(tq):
    """|l / T| of 3 million nats, logits an fp32 step or a few apart, 0.24 nats each: weights there are good to 2^-43 of
    the largest, so 3000 of them to 3.4e-10 of the mass together."""
    rng = np.random.default_rng(14)
    B, V = 24, 3000
    k = rng.integers(0, 200, (B, V))
    k[:, rng.integers(0, V, 20)] = 0
    for sign in (1, -1):
        rows = (sign * 3.0 - 2.0 ** -22 * k).astype(np.float32)
        for settings in (dict(), dict(top_k=300), dict(top_p=0.9), dict(min_p=0.1), dict(top_k=1500, top_p=0.7, min_p=0.2)):
            say("off the grid", sign, settings)
            check(tq, rows, rng.random(B), temperature=1e-6, **settings)
            check(tq, rows, [0.0, 1.0, 7.0] * 8, temperature=1e-6, **settings)


@pytest.mark.parametrize("dtype,bits", [(torch.float32, 0x7F800001), (torch.bfloat16, 0x7F81), (torch.float16, 0x7C01)])
def test_signalling_nans_count_as_minus_infinity(tq, dtype, bits):
    ints = torch.int32 if dtype == torch.float32 else torch.int16
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    logits = (torch.randn((8, 5000), generator=g, device="cuda") * 3).to(dtype)
    at = torch.rand((8, 5000), generator=g, device="cuda") < 0.3
    at[0], at[1, 1:], at[1, 0] = True, True, False
    u = torch.rand(8, generator=g, device="cuda")
    want = tq.sample(logits.masked_fill(at, float("-inf")), u, top_p=torch.full((8,), 0.8, device="cuda"))
    for b in (bits, bits - (1 << 32 if dtype == torch.float32 else 1 << 16) + (1 << 31 if dtype == torch.float32 else 1 << 15)):
        got = tq.sample(logits.view(ints).masked_fill(at, b).view(dtype), u, top_p=torch.full((8,), 0.8, device="cuda"))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert int(want[0][0]) == -1 and int(want[0][1]) == 0
