"""The residual RMS norm at the ends of its range (GPU): eps of 0, rows of zeros
and the smallest values."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ternary_quantized_moe_amd as tq
    tq.lib()
    return tq


def test_eps_of_zero(tq):
    d = 512
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn((6, d), generator=g, device="cuda")
    x[1] = 0
    x[2] *= 1e-15                                     # squares of some 1e-30: normal numbers
    x[3] = 1e-38
    x = x.bfloat16()
    w = torch.ones(d, device="cuda")
    y = tq.rms_norm(x, w, 0.0)["y"]
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isinf(y[3]).all())
    keep = [0, 2, 4, 5]
    h = x[keep].double()
    want = h / h.square().mean(1, keepdim=True).sqrt()
    # 64 fp32 half steps before the rounding to bf16, whose half step is 2^-8 of the value
    assert bool(((y[keep].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -17) * want.abs()).all())
    zero = tq.rms_norm(x, w, 1e-6)["y"]
    assert bool((zero[1] == 0).all()) and not bool(torch.isnan(zero).any())
