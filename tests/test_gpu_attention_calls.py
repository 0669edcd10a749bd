"""Calls of attention and its cache at the ends of what they take."""
import pytest

from test_gpu_attention import BF16, ints, say, tq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_compact_without_rows(tq):
    """Pages that no row of the table holds move all the same."""
    say("compact, no rows")
    refs = ints([0, 2, 0, 0, 1, 1, 0])
    pool = torch.arange(2 * 7 * 12, device="cuda", dtype=torch.int32).view(2, 7, 12)
    want = pool.clone()
    want[:, 0], want[:, 2] = pool[:, 4], pool[:, 5]
    tables, lengths = torch.empty((0, 5), dtype=torch.int32, device="cuda"), ints([])
    side = torch.cuda.Stream()
    for i, stream in enumerate((None, side)):
        x = pool.clone()
        side.wait_stream(torch.cuda.current_stream())
        new_tables, new_refs, live = tq.kv_compact(tables, lengths, refs, 4, [x], stream=stream)
        side.synchronize()
        assert new_tables.shape == (0, 5)
        assert live.tolist() == [3] and new_refs.tolist() == [1, 2, 1, 0, 0, 0, 0] and torch.equal(x, want)
    x = pool.clone()
    need = tq.lib().moe_kv_pages_workspace_bytes(0, 7)
    space = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    space = space[-space.data_ptr() % 256:][:need]
    tq.kv_compact(tables, lengths, refs, 4, [x], new_tables=tables, new_refs=refs, live=live, workspace=space)
    assert live.tolist() == [3] and refs.tolist() == [1, 2, 1, 0, 0, 0, 0] and torch.equal(x, want)
    with pytest.raises(tq.MoeError):
        tq.kv_compact(tables[:, :0], lengths, refs, 4, [x])
    with pytest.raises(tq.MoeError):
        tq.kv_compact(tables, lengths, refs, 4, [x], new_tables=ints([[1] * 5]))
