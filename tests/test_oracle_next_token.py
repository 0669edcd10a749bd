"""Pins of the oracle of the e4m3 quantizer, the norm, the product and the
sampler (CPU)."""
import numpy as np
import pytest

from oracle import fp8, sampler

torch = pytest.importorskip("torch")


def test_e4m3_table_matches_torch():
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(fp8.decode(codes.numpy()), want, equal_nan=True)


def test_encode_is_nearest_even():
    v = fp8.VALUES[:127]
    mid = (v[1:] + v[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(fp8.encode(mid), even)
    assert np.array_equal(fp8.encode(-v[1:]), np.arange(1, 127) + 128)
    x = np.random.default_rng(0).normal(scale=100, size=10000).clip(-448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(x), want)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_keeps_the_largest_value_and_half_a_step(block_rows):
    x = np.random.default_rng(1).normal(size=(200, 256)).astype(np.float32)
    codes, scales = fp8.quantize(x, block_rows)
    s = fp8.spread(scales.astype(np.float64), block_rows, 200)
    v = fp8.decode(codes) * s
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) * (1 + 2.0 ** -20))
    assert np.all(np.isclose(fp8.block_amax(v, block_rows), fp8.block_amax(x, block_rows), rtol=1e-6))


def test_norm_has_unit_mean_square_and_ignores_scale():
    x = np.random.default_rng(2).normal(size=(3, 256))
    _, y = fp8.rms_norm(x, None, np.ones(256), 0.0)
    assert np.allclose(np.mean(y * y, axis=1), 1.0)
    _, y2 = fp8.rms_norm(5 * x, None, np.ones(256), 0.0)
    assert np.allclose(y, y2)
    h, _ = fp8.rms_norm(x, -x, np.ones(256), 1e-6)
    assert np.all(h == 0)


def test_linear_by_a_loop():
    rng = np.random.default_rng(3)
    a, w = rng.integers(0, 127, (3, 256)), rng.integers(0, 127, (130, 256))
    sa, sw = rng.random((3, 2)), rng.random((2, 2))
    y, _ = fp8.linear(a, sa, w, sw)
    for t, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
        want = sum(fp8.VALUES[a[t, k]] * sa[t, k // 128] * fp8.VALUES[w[n, k]] * sw[n // 128, k // 128]
                   for k in range(256))
        assert np.isclose(y[t, n], want, rtol=1e-12)


def test_sampler_frequencies_follow_the_weights():
    logits = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    us = (np.arange(1000) + 0.5) / 1000
    got = np.bincount([sampler.sample_row(logits, u)[0] for u in us], minlength=4) / 1000
    assert np.allclose(got, [0.1, 0.4, 0.2, 0.3], atol=1e-3)
    got = np.bincount([sampler.sample_row(logits, u, top_k=2)[0] for u in us], minlength=4) / 1000
    assert np.allclose(got, [0, 4 / 7, 0, 3 / 7], atol=1e-3)
    got = np.bincount([sampler.sample_row(logits, u, top_p=0.75)[0] for u in us], minlength=4) / 1000
    assert np.allclose(got, [0, 4 / 9, 2 / 9, 3 / 9], atol=1e-3)
    got = np.bincount([sampler.sample_row(logits, u, min_p=0.6)[0] for u in us], minlength=4) / 1000
    assert np.allclose(got, [0, 4 / 7, 0, 3 / 7], atol=1e-3)
    got = np.bincount([sampler.sample_row(logits, u, temperature=0.5)[0] for u in us], minlength=4) / 1000
    assert np.allclose(got, np.array([1, 16, 4, 9]) / 30, atol=1e-3)


def test_sampler_special_rows():
    inf = np.inf
    assert sampler.sample_row(np.array([-inf, -inf]), 0.5)[:2] == (-1, 0.0)
    assert sampler.sample_row(np.array([np.nan, -3.0]), 0.5)[:2] == (1, 1.0)
    assert sampler.sample_row(np.array([0.0, inf, inf]), 0.6)[:2] == (2, 0.5)
    assert sampler.sample_row(np.array([2.0, 2.0, 2.0]), 0.0, temperature=0.0)[0] == 0
    assert sampler.sample_row(np.zeros(4), 0.5, top_p=0.5)[0] == 1
    assert sampler.sample_row(np.zeros(4), 0.75, top_k=2)[0] == 1
