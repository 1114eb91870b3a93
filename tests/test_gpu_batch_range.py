"""GPU: the ragged-batch decode where its numbers and its work get uneven: rings that fill over a page's
end, more units than the grid has places."""
import numpy as np
import pytest

from helpers_batch import BatchCache
from test_gpu_batch import check_decode, run_decode

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- the shares of the work
@pytest.mark.parametrize("name", ["float32", "bfloat16"])
def test_ring_fills_over_a_pages_end(kv_gpu, name):
    """Every sequence's window starts at another tile of a page, so that the first copies of a warp run
    from one page into the next; the same bits every time."""
    lens = [(128 * 3 + 16 * j + 5, 1) for j in range(8)] * 4
    c = BatchCache(lens, 2, 6, "q8_0", "q4_0", 61)
    first = run_decode(kv_gpu, c, name, window=170)
    check_decode(c, name, *first, window=170)
    for _ in range(20):
        again = run_decode(kv_gpu, c, name, window=170)
        assert np.array_equal(first[1], again[1]) and np.array_equal(first[2], again[2])
