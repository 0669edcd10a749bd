"""GPU parity of the e4m3 quantizer, the residual RMS norm and the block-scaled
product against the float64 oracle, through the binding.

Tolerances, u = 2^-24 the fp32 half step:
  * quantizer: bit for bit;
  * norm: h takes one addition; the mean adds at most 8 x 4 squares in a thread,
    6 exchanges and 16 waves, all positive, so it is within (32 + 6 + 16 + 3) u
    and its root within half that; root, reciprocal and two products add 5 u:
    under 64 u = 2^-18.  A bf16 output adds half a step, 2^-8, an e4m3 code half
    a step, 2^-4 of its value or 2^-10 of the scale for the smallest;
  * product: the products of a group are exact and their 128 additions each lose
    at most a whole fp32 step, 2 u, of the group's sum of magnitudes; the scale
    product and its multiplication add 2 u and each group's addition u of all
    magnitudes: (2 * 128 + 2 + groups) u sum |a w|, then the output's half step.
    A bf16 output takes the matrix cores' 8-bit instruction, which cuts eight
    neighbouring products at 2^-13 of the largest of them, at most 2^-13 of it from
    each of the other seven: 7 * 2^-13 sum over the eights of max |a w| more.
"""
import sys

import numpy as np
import pytest

from oracle import fp8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_quantized_moe_amd as tq
    tq.lib()
    return tq


def randn(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def host(t):
    return t.detach().cpu().to(torch.float64).numpy()


def codes(t):
    return t.cpu().view(torch.uint8).numpy()


def near(got, want, tol):
    """|got - want| <= tol, element by element."""
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{bad.sum()} values off, first at {tuple(np.argwhere(bad)[0])}: "
                           f"{got[bad][0]} for {want[bad][0]}")


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(1, 128), (7, 384), (128, 256), (129, 2048), (300, 1152)])
def test_quantize_exact(tq, rows, cols, dtype, block_rows):
    say(f"fp8 quantize {rows} x {cols} {dtype} blocks of {block_rows}")
    x = randn(rows, rows, cols).to(dtype)
    x[:, 5] *= 30
    q, s = tq.fp8_quantize(x, block_rows)
    want_q, want_s = fp8.quantize(x.float().cpu().numpy(), block_rows)
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(codes(q), want_q)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_blocks(tq, block_rows):
    x = randn(3, 3 * block_rows, 512).bfloat16()
    r = block_rows
    x[:r, :128] = 0                                  # zeros
    x[:r, 128:256] = 1e-38                           # below the floor
    x[r:2 * r, 0] = float("nan")
    x[r:2 * r, 128] = float("inf")
    x[r:2 * r, 256:384] *= 1e30
    x[2 * r:, 0] = -448
    q, s = tq.fp8_quantize(x, block_rows)
    v, s = q.cpu().float().numpy(), s.cpu().numpy()
    assert np.all(v[:r, :256] == 0) and np.all(s[0, :2] == np.float32(1e-30) / np.float32(448))
    assert np.isnan(s[1, 0]) and np.isnan(v[r:2 * r, :128]).all()
    assert np.isinf(s[1, 1]) and np.isnan(v[r:2 * r, 128]).all() and np.all(v[r:2 * r, 129:256] == 0)
    keep = x.clone()
    keep[r:2 * r, :256] = 0
    want_q, want_s = fp8.quantize(keep.float().cpu().numpy(), block_rows)
    assert np.array_equal(s[:, 2:], want_s[:, 2:]) and np.array_equal(codes(q)[:, 256:], want_q[:, 256:])
    assert np.array_equal(codes(q)[2 * r:], want_q[2 * r:])


def test_quantize_writes_only_its_rows(tq):
    x = randn(4, 130, 256).bfloat16()
    q = torch.full((140, 256), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((6, 2), -1.0, device="cuda")
    tq.fp8_quantize(x, 128, q=q[5:135], scales=s[2:4])
    assert bool((q[:5] == 0x55).all()) and bool((q[135:] == 0x55).all())
    assert bool((s[:2] == -1).all()) and bool((s[4:] == -1).all())
    want_q, want_s = fp8.quantize(x.float().cpu().numpy(), 128)
    assert np.array_equal(q[5:135].cpu().numpy(), want_q) and np.array_equal(s[2:4].cpu().numpy(), want_s)


# ------------------------------------------------------------------ norm
def check_norm(out, x, residual, w, eps):
    h, y = fp8.rms_norm(host(x), None if residual is None else host(residual), host(w), eps)
    if "sum" in out:
        near(host(out["sum"]), h, (2.0 ** -8 + U) * np.abs(h))
    tol = 64 * U * np.abs(y)
    if "y" in out:
        near(host(out["y"]), y, tol * 2 + 2.0 ** -8 * np.abs(y) + 2.0 ** -134)
    if "q" in out:
        s = host(out["scales"])
        m = np.maximum(fp8.block_amax(y, 1), 1e-30) / 448
        near(s, m, 66 * U * m)
        per = fp8.spread(s, 1, y.shape[0])
        near(host(out["q"].float()) * per, y, np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * per) * (1 + 2.0 ** -16) + tol)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,d", [(1, 128), (3, 384), (1, 2048), (33, 2048), (5, 4096), (2, 8320), (2, 32768), (700, 640)])
def test_norm(tq, T, d, residual):
    say(f"rms norm {T} x {d} residual {residual}")
    x = (randn(d, T, d) * torch.exp(3 * randn(1, T, 1))).bfloat16()
    r = (4 * randn(d + 1, T, d)).bfloat16() if residual else None
    w = 1 + 0.3 * randn(2, d)
    for bf16, f8 in ((True, False), (False, True), (True, True)):
        out = tq.rms_norm(x, w, EPS, residual=r, bf16=bf16, fp8=f8)
        assert set(out) == ({"sum"} if residual else set()) | ({"y"} if bf16 else set()) | ({"q", "scales"} if f8 else set())
        check_norm(out, x, r, w, EPS)


def test_norm_in_place(tq):
    T, d = 9, 2048
    x, r, w = randn(1, T, d).bfloat16(), randn(2, T, d).bfloat16(), 1 + 0.1 * randn(3, d)
    want = tq.rms_norm(x, w, EPS, residual=r, bf16=True, fp8=True)
    for s, y in ((0, 1), (1, 0), (0, None), (None, 0)):
        a = [x.clone(), r.clone()]
        out = tq.rms_norm(a[0], w, EPS, residual=a[1], bf16=True, fp8=True, sum=None if s is None else a[s],
                          y=None if y is None else a[y])
        for k in want:
            assert torch.equal(out[k].view(torch.uint8), want[k].view(torch.uint8)), (s, y, k)


def test_norm_special_rows(tq):
    d = 512
    x = randn(5, 6, d).bfloat16()
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 7] = float("inf")
    x[3] *= 1e30                        # the mean square overflows: finite values give 0
    x[4] *= 1e-30
    w = torch.ones(d, device="cuda")
    out = tq.rms_norm(x, w, EPS, bf16=True, fp8=True)
    y, v, s = host(out["y"]), host(out["q"].float()), host(out["scales"])
    assert np.all(y[0] == 0) and np.all(v[0] == 0)
    assert np.isnan(y[1]).all() and np.isnan(v[1]).all() and np.isnan(s[1]).all()
    assert np.isnan(y[2, 7]) and np.all(np.delete(y[2], 7) == 0) and np.isnan(s[2, 0]) and np.all(v[2, 128:] == 0)
    assert np.all(y[3] == 0)
    check_norm({k: t[4:] for k, t in out.items()}, x[4:], None, w, EPS)


# ------------------------------------------------------------------ product
def operands(tq, m, n, k, seed=0):
    a = randn(seed, m, k) * torch.exp(randn(seed + 1, m, 1))
    a[:, :: max(1, k // 7)] *= 20
    w = randn(seed + 2, n, k) / k ** 0.5
    return (*tq.fp8_quantize(a.bfloat16(), 1), *tq.fp8_quantize(w.bfloat16(), 128))


def largest_of_eights(a, sa, w, sw):
    """Sum over eights of neighbouring k of max |a w|, scaled."""
    def scaled(c, s, rows):
        per = s.repeat_interleave(rows, 0)[:c.shape[0]].repeat_interleave(128, 1)
        return (c.float().abs() * per).view(c.shape[0], -1, 8)
    x, v = scaled(a, sa, 1), scaled(w, sw, 128)
    out = torch.zeros((x.shape[0], v.shape[0]), dtype=torch.float64, device="cuda")
    for g in range(x.shape[1]):
        out += (x[:, None, g] * v[None, :, g]).amax(2)
    return out.cpu().numpy()


def check_linear(y, a, sa, w, sw):
    want, mag = fp8.linear(codes(a), host(sa), codes(w), host(sw))
    tol = (2 * 128 + 2 + a.shape[1] // 128) * U * mag
    half = U
    if y.dtype == torch.bfloat16:
        half = 2.0 ** -8
        tol = tol + 7 * 2.0 ** -13 * largest_of_eights(a, sa, w, sw)
    near(host(y), want, tol + half * (np.abs(want) + tol))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 1000, 2048), (2, 129, 384), (15, 257, 512), (16, 64, 128), (17, 300, 1024),
                                   (31, 2048, 256), (33, 513, 640), (64, 384, 2048), (65, 127, 896), (100, 1025, 512),
                                   (128, 128, 128), (129, 259, 1280), (200, 2561, 256), (256, 256, 4096),
                                   (333, 515, 1152), (515, 640, 384), (1030, 1100, 256), (257, 4100, 128)])
def test_linear(tq, m, n, k, dtype):
    say(f"fp8 linear {m} x {n} x {k} {dtype}")
    ops = operands(tq, m, n, k, seed=m + n)
    check_linear(tq.fp8_linear(*ops, out_dtype=dtype), *ops)


# sizes at which each tile shape and the split kernel are taken, with ragged edges on every side and an
# odd number of groups
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(3500, 3601, 384), (1800, 1701, 640), (2500, 2203, 128), (700, 2402, 1152),
                                   (60, 34001, 256), (1030, 1101, 896), (20, 25003, 384), (3, 25000, 640), (30, 13001, 1152),
                                   (1, 13000, 256), (40, 4101, 1152), (10, 8301, 2176), (5, 100, 2304)])
def test_linear_every_shape(tq, m, n, k, dtype):
    say(f"fp8 linear {m} x {n} x {k} {dtype}")
    ops = operands(tq, m, n, k, seed=m + n)
    check_linear(tq.fp8_linear(*ops, out_dtype=dtype), *ops)


def test_linear_past_32_bits(tq):
    """An output of more than 2^31 values, and a w of more than 2^32 bytes: rows at the far end."""
    say("fp8 linear past 32 bits")
    a, sa, w, sw = operands(tq, 70001, 33000, 128)
    y = tq.fp8_linear(a, sa, w, sw)
    far = [0, 40000, 65535, 69999, 70000]
    check_linear(y[far], a.view(torch.uint8)[far].view(a.dtype), sa[far], w, sw)
    del y
    n, k = 36000, 1024 * 128
    w = torch.randint(0, 100, (n, k), dtype=torch.uint8, device="cuda")
    sw = torch.rand((-(-n // 128), k // 128), device="cuda")
    a, sa = tq.fp8_quantize(randn(1, 3, k).bfloat16(), 1)
    y = tq.fp8_linear(a, sa, w, sw, out_dtype=torch.float32)
    check_linear(y[:, 281 * 128:], a, sa, w[281 * 128:].view(a.dtype), sw[281:])
    del w
    torch.cuda.empty_cache()


def test_norm_and_quantize_past_32_bits(tq):
    T, d = 1_100_000, 2048
    say("norm and quantizer past 32 bits")
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 100_000):
        x[i:i + 100_000] = randn(i, min(100_000, T - i), d).bfloat16()
    w = 1 + 0.1 * randn(1, d)
    far = [0, 600_000, 1_048_576, T - 1]
    out = tq.rms_norm(x, w, EPS, bf16=True, fp8=True)
    check_norm({k: t[far] if t.dtype != torch.float8_e4m3fn else t.view(torch.uint8)[far].view(t.dtype)
                for k, t in out.items()}, x[far], None, w, EPS)
    del out
    for rows in (1, 128):
        q, s = tq.fp8_quantize(x, rows)
        lo = 1_099_900 // 128 * 128
        want_q, want_s = fp8.quantize(x[lo:].float().cpu().numpy(), rows)
        assert np.array_equal(q.view(torch.uint8)[lo:].cpu().numpy(), want_q)
        assert np.array_equal(s[lo // rows:].cpu().numpy(), want_s)
        del q
    torch.cuda.empty_cache()


def test_norm_and_quantize_of_many_rows(tq):
    """More blocks than one dimension of a launch holds: the last rows are those of a small call."""
    for rows, fn in (((1 << 26) + 3, "norm"), ((1 << 28) + 5, "rows"), ((1 << 28) + 5, "tiles")):
        say("many rows", fn, rows)
        x = torch.zeros((rows, 128), dtype=torch.bfloat16, device="cuda")
        last = rows // 128 * 128                              # whole blocks of 128 rows before
        x[last:] = torch.randn((rows - last, 128), device="cuda").bfloat16()
        if fn == "norm":
            weight = torch.ones(128, device="cuda")
            got, want = (tq.rms_norm(v, weight, 1e-6, bf16=False, fp8=True) for v in (x, x[last:].clone()))
            got, want = (got["q"], got["scales"]), (want["q"], want["scales"])
        else:
            got, want = (tq.fp8_quantize(v, 1 if fn == "rows" else 128) for v in (x, x[last:].clone()))
        assert torch.equal(got[0][last:].view(torch.uint8), want[0].view(torch.uint8))
        assert torch.equal(got[1][-want[1].shape[0]:], want[1])
        assert not bool(got[0][last - 128:last].view(torch.uint8).any())
        del x, got, want
        torch.cuda.empty_cache()


def test_linear_long_k(tq):
    ops = operands(tq, 5, 130, 128 * 150)
    check_linear(tq.fp8_linear(*ops, out_dtype=torch.float32), *ops)


@pytest.mark.parametrize("m", [1, 33, 300])
def test_linear_padded_output_keeps_its_padding(tq, m):
    ops = operands(tq, m, 301, 512, seed=9)
    want = tq.fp8_linear(*ops)
    for ld, first in ((301, 0), (303, 1), (320, 8)):
        buf = torch.full((m + 2, ld + first), 7.0, dtype=torch.bfloat16, device="cuda")
        y = buf[1:-1, first:first + 301]
        tq.fp8_linear(*ops, y=y)
        assert torch.equal(y, want)
        buf[1:-1, first:first + 301] = 7.0
        assert bool((buf == 7.0).all())


@pytest.mark.parametrize("m,n", [(40, 260), (700, 2402)])
def test_linear_nan_stays_in_its_row_and_column(tq, m, n):
    a, sa, w, sw = operands(tq, m, n, 256)
    base = tq.fp8_linear(a, sa, w, sw, out_dtype=torch.float32)
    a2, w2 = a.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    a2[3, 100] = 0x7F
    w2[129, 7] = 0xFF
    y = tq.fp8_linear(a2, sa, w2, sw, out_dtype=torch.float32)
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[:, 129]).all())
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[3] = False
    keep[:, 129] = False
    assert torch.equal(y[keep], base[keep])


def test_linear_rows_do_not_depend_on_their_neighbours(tq):
    """A token's result is the same bits wherever it stands in a batch of one size."""
    a, sa, w, sw = operands(tq, 48, 200, 512)
    y = tq.fp8_linear(a, sa, w, sw)
    at = torch.randperm(48, device="cuda")
    y2 = tq.fp8_linear(a.view(torch.uint8)[at], sa[at], w, sw)
    assert torch.equal(y[at], y2)


def test_empty_calls(tq):
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    q, s = tq.fp8_quantize(x, 128)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    assert tq.rms_norm(x, torch.ones(256, device="cuda"), EPS)["y"].shape == (0, 256)
    w, sw = tq.fp8_quantize(randn(0, 64, 256).bfloat16(), 128)
    assert tq.fp8_linear(q, torch.empty((0, 2), device="cuda"), w, sw).shape == (0, 64)


# ------------------------------------------------------------------ refusals that need a device tensor
def test_binding_refusals(tq):
    x = randn(0, 4, 256).bfloat16()
    q, s = tq.fp8_quantize(x, 1)
    w, sw = tq.fp8_quantize(x, 128)
    one = torch.ones(256, device="cuda")

    def code(f):
        with pytest.raises(tq.MoeError) as e:
            f()
        return e.value.code
    assert code(lambda: tq.fp8_quantize(x, 64)) == -1
    assert code(lambda: tq.fp8_quantize(x, 0)) == -1
    assert code(lambda: tq.fp8_quantize(x[:, :200].contiguous(), 1)) == -3
    assert code(lambda: tq.fp8_quantize(x.t(), 1)) == -1
    assert code(lambda: tq.fp8_quantize(x.float(), 1)) == -2
    assert code(lambda: tq.rms_norm(x, one[:128], EPS)) == -3
    assert code(lambda: tq.rms_norm(x, one.bfloat16(), EPS)) == -2
    assert code(lambda: tq.rms_norm(x, one.cpu(), EPS)) == -1
    assert code(lambda: tq.rms_norm(x, one, EPS, residual=x[:2])) == -3
    assert code(lambda: tq.rms_norm(x, one, EPS, bf16=False)) == -1
    assert code(lambda: tq.rms_norm(x, one, EPS, q=q)) == -1
    assert code(lambda: tq.rms_norm(x, one, EPS, bf16=False, fp8=True, y=x)) == -1
    assert code(lambda: tq.rms_norm(x, one, EPS, sum=x)) == -1
    assert code(lambda: tq.fp8_linear(q, s, w[:, :128].contiguous(), sw)) == -3
    assert code(lambda: tq.fp8_linear(q, s[:2], w, sw)) == -3
    assert code(lambda: tq.fp8_linear(q, s, w, s)) == -3
    assert code(lambda: tq.fp8_linear(q, s, w, sw, out_dtype=torch.float16)) == -2
    assert code(lambda: tq.fp8_linear(q, s, w, sw, y=torch.empty((4, 4), device="cuda").t())) == -1
    assert code(lambda: tq.fp8_linear(q, s, w, sw, y=torch.empty((4, 4), device="cuda"),
                                      out_dtype=torch.bfloat16)) == -2
