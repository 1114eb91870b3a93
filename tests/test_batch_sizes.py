"""CPU: sizes that the ragged-batch calls take, answered before anything touches a GPU."""
import pytest

from quantized_paged_kv_q4_b200 import build, kvattn
from test_batch import batch, desc


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kvattn.lib()


@pytest.mark.parametrize("kw", [dict(max_rows=5), dict(max_rows=131072), dict(max_rows=400_000_000),
                                dict(max_rows=2 ** 31 - 1), dict(max_rows=1, n_seqs=1 << 13, max_blocks=(1 << 12) + 1)])
def test_no_workspace_for_a_batch_that_decode_refuses(lib, kw):
    d = desc()  # 6 query heads per KV head
    assert lib.kvattn_decode_batch_workspace_size(d, batch(**kw)) == 0
    assert 0 < lib.kvattn_decode_batch_workspace_size(d, batch(max_rows=4)) < 1 << 30
    assert 0 < lib.kvattn_decode_batch_workspace_size(d, batch(max_rows=1, n_seqs=1 << 13, max_blocks=1 << 12)) < 1 << 30


def test_a_batch_without_rows_is_fine_whatever_its_table(lib):
    assert lib.kvattn_decode_batch(desc(), batch(n_rows=0, n_seqs=1 << 13, max_blocks=(1 << 12) + 1), None, None, None, 0,
                                   None, None, None, 0, None) == kvattn.OK


def test_counts_that_do_not_fit_are_refused(monkeypatch):
    """A window of 2^32 + 5 is not a window of 5."""
    import torch

    b = batch()
    b.heads, b.device = 4, 0
    for window in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="window"):
            kvattn.kvattn_decode_batch(desc(), b, None, None, None, None, window=window)
    monkeypatch.setattr(kvattn, "_on", lambda x, what, device: x.data_ptr())
    monkeypatch.setattr(kvattn._Torch, "current_device", lambda: 0)
    monkeypatch.setattr(kvattn._Torch, "int32", torch.int32)
    row, pos, table = (torch.zeros(s, dtype=torch.int32) for s in ((3,), (2,), (2, 4, 5)))
    assert kvattn.make_batch(row, pos, table, 10, 2 ** 31 - 1).max_rows == 2 ** 31 - 1
    with pytest.raises(ValueError, match="max_rows"):
        kvattn.make_batch(row, pos, table, 10, 2 ** 32 + 1)
