"""Refusals of the e4m3 quantizer, the RMS norm, the block-scaled product and the
sampler: every check happens on the host, before any launch (CPU)."""
import pytest

import ternary_quantized_moe_amd as tq

torch = pytest.importorskip("torch")

ARG, FORMAT, SHAPE, SPACE = -1, -2, -3, -6
BF16, F16, F32 = 0, 1, 2
BIG = 1 << 40


def test_quantize_refusals():
    L = tq.lib()

    def rc(type=BF16, x=0x100000, rows=4, cols=256, br=1, q=0x200000, s=0x300000):
        return L.moe_fp8_quantize(type, x, rows, cols, br, q, s, None)
    assert rc(type=F32) == FORMAT and rc(type=7) == FORMAT
    assert rc(br=64) == ARG and rc(br=0) == ARG
    assert rc(cols=200) == SHAPE and rc(cols=0) == SHAPE and rc(rows=-1) == SHAPE
    assert rc(rows=1 << 50) == SHAPE
    assert rc(x=None) == ARG and rc(q=None) == ARG and rc(s=None) == ARG
    assert rc(x=0x100008) == ARG and rc(q=0x200004) == ARG and rc(s=0x300002) == ARG
    assert rc(q=0x100000 + 2 * 4 * 256 - 16) == ARG and "overlap" in L.moe_last_error().decode()
    assert rc(s=0x200000) == ARG and rc(s=0x100010) == ARG
    assert rc(rows=0) == 0


def test_norm_refusals():
    L = tq.lib()

    def rc(x=0x100000, res=0x200000, T=4, d=256, w=0x300000, eps=1e-6, sum=0x400000, y=0x500000, q=0x600000,
           s=0x700000):
        return L.moe_rms_norm(x, res, T, d, w, eps, sum, y, q, s, None)
    assert rc(d=200) == SHAPE and rc(d=0) == SHAPE and rc(d=32768 + 128) == SHAPE
    assert rc(T=-1) == SHAPE and rc(T=1 << 31) == SHAPE
    assert rc(eps=-1.0) == ARG and rc(eps=float("nan")) == ARG and rc(eps=float("inf")) == ARG
    assert rc(y=None, q=None, s=None) == ARG and rc(s=None) == ARG and rc(q=None) == ARG
    assert rc(res=None) == ARG                                            # sum without a residual
    assert rc(x=None) == ARG and rc(w=None) == ARG
    for k in ("x", "res", "w", "sum", "y", "q"):
        assert rc(**{k: 0x800008}) == ARG
    assert rc(s=0x700002) == ARG
    assert rc(sum=0x100010) == ARG and rc(y=0x200000 + 16) == ARG         # part of an input
    assert rc(sum=0x500000) == ARG and rc(q=0x500000) == ARG and rc(s=0x600000) == ARG
    assert rc(q=0x100000) == ARG and rc(y=0x300000) == ARG
    assert rc(T=0) == 0


def test_linear_refusals():
    L = tq.lib()

    def rc(a=0x100000, sa=0x200000, m=4, w=0x300000, sw=0x400000, n=300, k=256, type=BF16, y=0x500000, ldy=300):
        return L.moe_fp8_linear(a, sa, m, w, sw, n, k, type, y, ldy, None)
    assert rc(type=F16) == FORMAT
    assert rc(k=100) == SHAPE and rc(k=0) == SHAPE and rc(m=-1) == SHAPE and rc(n=-1) == SHAPE
    assert rc(m=1 << 31) == SHAPE and rc(ldy=299) == SHAPE and rc(ldy=1 << 62) == SHAPE
    assert rc(k=(1 << 22) + 128) == SHAPE and rc(m=1 << 21, n=1 << 20, ldy=1 << 20) == SHAPE
    for k in ("a", "sa", "w", "sw", "y"):
        assert rc(**{k: None}) == ARG
    assert rc(a=0x100008) == ARG and rc(w=0x300008) == ARG and rc(sa=0x200002) == ARG
    assert rc(y=0x500001) == ARG and rc(type=F32, y=0x500002) == ARG
    assert rc(y=0x100000) == ARG and rc(y=0x200000) == ARG and rc(y=0x300100) == ARG and rc(y=0x400004) == ARG
    assert rc(m=0) == 0 and rc(n=0, ldy=0) == 0


def test_linear_sizes_of_one_launch():
    """What would be 2^32 threads or more is refused before the launch."""
    L = tq.lib()

    def rc(m, n):
        return L.moe_fp8_linear(0x1000000, 0x2000000, m, 0x3000000, 0x4000000, n, 128, BF16, 0x5000000, n, None)
    assert rc((1 << 29) + 1, 1) == SHAPE and rc(1, (1 << 29) + 1) == SHAPE
    assert rc(1 << 19, (1 << 18) + 1) == SHAPE


def test_sample_refusals():
    L = tq.lib()

    def rc(type=F32, logits=0x100000, b=2, v=1000, ld=1000, t=None, k=None, p=None, mp=None, u=0x200000,
           tokens=0x300000, probs=None, ws=0x400000, ws_bytes=BIG):
        return L.moe_sample(type, logits, b, v, ld, t, k, p, mp, u, tokens, probs, ws, ws_bytes, None)
    assert rc(type=3) == FORMAT
    assert rc(v=0) == SHAPE and rc(v=(1 << 21) + 1, ld=1 << 22) == SHAPE
    assert rc(b=-1) == SHAPE and rc(b=(1 << 22) + 1) == SHAPE and rc(ld=999) == SHAPE
    assert rc(logits=None) == ARG and rc(u=None) == ARG and rc(tokens=None) == ARG
    assert rc(ws=0x400010) == ARG
    for k in ("logits", "t", "k", "p", "mp", "u", "tokens", "probs"):
        assert rc(**{k: 0x500002}) == ARG
    assert rc(type=BF16, logits=0x500001) == ARG
    assert rc(b=0) == 0
    assert L.moe_sample_workspace_bytes(-1, 100) == -1 and L.moe_sample_workspace_bytes(1, 0) == -1
    assert L.moe_sample_workspace_bytes(1, 1 << 22) == -1 and L.moe_sample_workspace_bytes(0, 100) >= 0


def test_sample_overlaps_are_refused():
    L = tq.lib()
    places = dict(logits=0x100000, t=0x200000, k=0x210000, p=0x220000, mp=0x230000, u=0x240000, tokens=0x300000,
                  probs=0x310000, ws=0x400000)

    def rc(**at):
        a = {**places, **at}
        return L.moe_sample(F32, a["logits"], 2, 1000, 1200, a["t"], a["k"], a["p"], a["mp"], a["u"], a["tokens"],
                            a["probs"], a["ws"], 1 << 20, None)
    inputs = [places[k] for k in ("logits", "t", "k", "p", "mp", "u")]
    for out in ("tokens", "probs", "ws"):
        for at in inputs:
            assert rc(**{out: at}) == ARG and "overlap" in L.moe_last_error().decode()
    assert rc(probs=places["tokens"] + 4) == ARG and rc(tokens=places["ws"] + 256) == ARG
    assert rc(tokens=places["logits"] + 4 * (1200 + 999)) == ARG


def test_host_tensors_are_refused():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    w = torch.ones(128)
    calls = [lambda: tq.fp8_quantize(x, 1), lambda: tq.rms_norm(x, w, 1e-6),
             lambda: tq.fp8_linear(x.to(torch.float8_e4m3fn), torch.ones(2, 1), x.to(torch.float8_e4m3fn),
                                   torch.ones(1, 1)),
             lambda: tq.sample(torch.zeros(2, 8), torch.zeros(2))]
    for call in calls:
        with pytest.raises(tq.MoeError) as e:
            call()
        assert e.value.code == ARG
