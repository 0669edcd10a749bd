"""What the binding makes of the pools of a cache (CPU)."""
import pytest

from ternary_quantized_moe_amd import binding

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("layers,pages", [(8, 1), (1, 8), (1, 1), (3, 4)])
def test_pages_of_pools(layers, pages):
    """Also where one page or one layer leaves a stride without meaning."""
    x = torch.zeros((layers, pages, 2, 4, 16), dtype=torch.bfloat16)
    turned = torch.zeros((pages, layers, 2, 4, 16), dtype=torch.bfloat16).transpose(0, 1)
    for p in (x, turned) if turned.is_contiguous() else (x,):
        c, n = binding._pools([p], -1, pages)
        assert n == 1 and c[0].base == p.data_ptr()
        assert (c[0].planes, c[0].page_bytes) == (layers, 2 * 4 * 16 * 2)
