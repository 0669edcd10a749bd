"""The oracle of attention, the rotary embedding and the pages against what their
definitions imply (CPU)."""
import numpy as np
import pytest

from oracle import attention


def draw(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_attention_is_a_mean_of_the_seen_values():
    q, k, v = draw(0, 6, 4, 8), draw(1, 9, 2, 8), draw(2, 9, 2, 8)
    r = attention.attend(q, k, v, np.arange(6) + 3, 0.3)
    x = 0.3 * np.einsum("ihd,jhd->ihj", q, np.repeat(k, 2, 1))
    x = np.where(np.arange(9)[None, None, :] > np.arange(6)[:, None, None] + 3, -np.inf, x)
    p = np.exp(x)
    assert np.allclose(r["y"], np.einsum("ihj,jhd->ihd", p / p.sum(2, keepdims=True), np.repeat(v, 2, 1)), atol=1e-13)
    assert np.allclose(r["lse"], np.log(p.sum(2)), atol=1e-13)
    one = attention.attend(q, k, np.ones_like(v), np.full(6, 8), 0.3)
    assert np.allclose(one["y"], 1) and np.allclose(one["size"], 1)


def test_attention_ends():
    q, k, v = draw(0, 3, 1, 4), draw(1, 5, 1, 4), draw(2, 5, 1, 4)
    r = attention.attend(q, k, v, [-1, 0, 4], 1.0)
    assert np.all(r["y"][0] == 0) and r["lse"][0, 0] == -np.inf
    assert np.allclose(r["y"][1, 0], v[0, 0])
    hidden = v.copy()
    hidden[1:] = np.nan
    assert np.array_equal(attention.attend(q, k, hidden, [-1, 0, 0], 1.0)["y"][1], r["y"][1])
    low = np.full_like(k, -np.inf)
    z = attention.attend(np.abs(q), low, v, [4, 4, 4], 1.0)
    assert np.all(z["y"] == 0) and np.all(z["lse"] == -np.inf)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_sizes_and_sees_differences_alone(interleaved):
    x, f = draw(3, 5, 2, 16), 10.0 ** -np.arange(4)
    r = attention.rotate(x, [0, 1, 7, 100, 5], f, interleaved)
    assert np.array_equal(r[0], x[0]) and np.array_equal(r[..., 8:], x[..., 8:])
    assert np.allclose((r ** 2).sum(-1), (x ** 2).sum(-1))
    a, b = x[:1], x[1:2]
    dots = [(attention.rotate(a, [p], f, interleaved) * attention.rotate(b, [p + 3], f, interleaved)).sum()
            for p in (0, 11, 1000)]
    assert np.allclose(dots, dots[0])


def new_pages(rows=6, width=5, n=20, page=4):
    pool = np.arange(2 * n * page, dtype=np.float64).reshape(2, n, page)
    return attention.Pages([[-1] * width for _ in range(rows)], [0] * rows, [0] * n, page, [pool])


def content(p, r):
    n = p.lengths[r]
    return [p.pools[0][:, p.tables[r][i // p.page], i % p.page].tolist() for i in range(n)]


def test_pages_are_lent_shared_and_returned():
    p = new_pages()
    assert p.reserve([5, 0, 4, 21, -1, 0]) == [2, 0, 1, -1, -1, 0]
    assert p.tables[0][:2] == [0, 1] and p.tables[2][0] == 2 and p.lengths == [5, 0, 4, 0, 0, 0]
    assert p.fork([-1, 0, -1, 2, 1, 0]) == [0, 1, 0, 0, -1, 1]
    assert p.tables[1][:2] == [0, 3] and p.tables[5][:2] == [0, 4] and p.tables[3][:1] == [2]
    assert p.refs[:5] == [3, 1, 2, 1, 1]
    assert content(p, 1) == content(p, 0) == content(p, 5) and content(p, 3) == content(p, 2)
    p.free([1, 0, 1, 0, 0, 0])
    assert p.refs[:5] == [2, 0, 1, 1, 1] and p.lengths[:3] == [0, 5, 0]
    before = [content(p, r) for r in range(6)]
    assert p.compact() == 4 and p.refs == [2, 1, 1, 1] + [0] * 16
    assert p.tables[5][:2] == [0, 1] and [content(p, r) for r in range(6)] == before


def test_pages_run_out():
    p = new_pages(rows=4, n=3)
    assert p.reserve([4, 8, 4, 0]) == [1, 2, -2, 0]
    assert p.lengths == [4, 8, 0, 0] and p.refs == [1, 1, 1]
    assert p.fork([-1, -1, 0, 1]) == [0, 0, 0, 0] and p.refs == [2, 2, 2]
