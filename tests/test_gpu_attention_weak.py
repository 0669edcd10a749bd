"""GPU parity of attention in fp16 with many weak keys beside a strong one.

The tolerance is that of tests/test_gpu_attention.py but for fp16's smallest numbers.  Weights are
rounded to fp16, held so that the largest so far is 2^7 or more.  Below 2^-14 one is off by 2^-25
instead of half a step of itself, which is 2^-32 of the largest; of n weights, whose sum is the
largest or more, 2^-32 n max |v|; and y, rounded once, by 2^-25.
"""
import numpy as np
import pytest

from test_gpu_attention import E, F16, host, ints, lse_tolerance, oracle_of, say, tq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -11


def close(got, want, D, n, small):
    """small: the bound on what fp16's smallest numbers cost."""
    d = (2 * D + 7) * E * want["score"][..., None]
    tol = U * want["size"] + U * np.abs(want["y"]) + (4 * d + (10 + 4 * n) * E) * want["size"] + small + 2.0 ** -25
    bad = ~(np.abs(got - want["y"]) <= 1.01 * tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want["y"][bad][:5], tol[bad][:5])


def close_lse(lse, want, D, n):
    assert np.all(np.abs(host(lse) - want["lse"]) <= 2 * lse_tolerance(want, D, n))


def weak_and_strong(n, D, bits):
    """One query; key 0 weighs 2^bits times as much as any other and has a value of zero."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n + D)
    q, k = torch.zeros((1, 1, D), device="cuda"), torch.zeros((n, 1, D), device="cuda")
    q[..., 0], k[0, 0, 0] = 4.0, bits * np.log(2) / 4
    v = 100.0 * torch.randint(1, 8, (n, 1, D), generator=g, device="cuda")
    v[..., ::3] *= -1
    v[0] = 0
    return q.to(F16), k.to(F16), v.to(F16)


@pytest.mark.parametrize("bits", [14.0, 21.5, 25.5])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts_keep_weak_keys(tq, D, bits):
    """Of prompts whose keys one block walks over, and of some that several blocks share."""
    for n in (1000, 5000):
        say(f"weak keys: prompt, {n} keys, dim {D}, 2^-{bits}")
        q, k, v = weak_and_strong(n, D, bits)
        lse = torch.empty((1, 1), device="cuda")
        y = tq.attention_prefill(q, k, v, ints([0, 1]), ints([0, n]), scale=1.0, lse=lse)
        want = oracle_of(q, k, v, [1], [n], True, 1.0)
        close(host(y), want, D, n, 2.0 ** -32 * n * float(v.abs().max()))
        close_lse(lse, want, D, n)


@pytest.mark.parametrize("bits", [14.0, 21.5, 25.5])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_single_tokens_keep_weak_keys(tq, D, bits):
    """256 sequences of the same pages, so that one worker goes through one from end to end."""
    n, P, B = 1024, 64, 256
    say(f"weak keys: single tokens, dim {D}, 2^-{bits}")
    q, k, v = weak_and_strong(n, D, bits)
    pages = [x.view(n // P, P, 1, D).transpose(1, 2).contiguous() for x in (k, v)]
    tables = torch.arange(n // P, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    lse = torch.empty((B, 1), device="cuda")
    y = tq.attention_decode(q.expand(B, 1, D).contiguous(), *pages, tables, ints([n] * B), scale=1.0, lse=lse)
    want = oracle_of(q, k, v, [1], [n], True, 1.0)
    for b in (0, 100, 255):
        close(host(y)[b:b + 1], want, D, n, 2.0 ** -32 * n * float(v.abs().max()))
        close_lse(lse[b:b + 1], want, D, n)
