"""The sums of the block-scaled product where the largest products of eight
neighbours cancel (GPU): exact to fp32, and to bf16 within the documented cut of
7 2^-13 of an eight's largest product."""
import numpy as np
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


# sizes that the split kernel and tiles of 64 x 32 to 256 x 256 take
@pytest.mark.parametrize("m,n", [(3, 200), (16, 4100), (40, 12500), (300, 4100), (3500, 3601)])
def test_products_that_cancel(tq, m, n):
    K, rng = 256, np.random.default_rng(m)
    a, w = np.full((m, K), 4.0, np.float32), np.full((n, K), 4.0, np.float32)
    big = 8 * rng.integers(0, K // 8, 4)[:, None] + np.stack([rng.permutation(8)[:2] for _ in range(4)])
    big = big[np.unique(big[:, 0] // 8, return_index=True)[1]]           # two places in some of the eights
    a[:, big], w[:, big[:, 0]], w[:, big[:, 1]] = 448.0, 448.0, -448.0
    a[1::2, big] = 224.0
    want = 16.0 * (K - 2 * len(big))                                     # every product is whole, fp32 holds the sums
    a, w = (torch.from_numpy(v).cuda().to(torch.float8_e4m3fn) for v in (a, w))
    sa, sw = torch.ones((m, K // 128), device="cuda"), torch.ones((-(-n // 128), K // 128), device="cuda")
    y = tq.fp8_linear(a, sa, w, sw, out_dtype=torch.float32)
    assert bool((y == want).all())
    y = tq.fp8_linear(a, sa, w, sw).float()
    lost = 7 * 2.0 ** -13 * 448.0 ** 2 * len(big)                        # the other eights' products are equal: none is cut
    assert bool(((y - want).abs() <= lost + 2.0 ** -8 * (want + lost)).all())
