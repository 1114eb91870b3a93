"""GPU: the ragged-batch decode where its numbers and its work get uneven: rings that fill over a page's
end, more units than the grid has places."""
import numpy as np
import pytest

from helpers_batch import EPS, PAIRS, BatchCache
from oracle import layout as olay
from oracle import quant as oq
from test_gpu_batch import check_decode, rounded, run_decode

pytestmark = pytest.mark.gpu
TYPES = ["float32", "float16", "bfloat16"]


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


# ------------------------------------------------------------------------- tiny blocks
@pytest.mark.parametrize("k_fmt,v_fmt", [("q4_0", "q4_0"), ("q5_0", "q4_1"), ("q8_0", "q8_0"), ("q5_1", "q4_0")])
def test_blocks_whose_reciprocal_scale_overflows(kv_gpu, k_fmt, v_fmt):
    """A block near 1e-40 has a scale that fp16 holds as zero and fp32 cannot invert.  Its values read as
    zero, its codes stay its own (every other block reads as if the tiny one were zero), and the
    ragged-batch writer's bytes, a whole tile or a part, are the single-sequence writer's."""
    import torch

    kv = kv_gpu
    rng = np.random.default_rng(62)
    for rows in (16, 5):
        x = rng.standard_normal((rows, 1, 256)).astype(np.float32)
        tiny = (rng.standard_normal((rows, 32)) * 1e-40).astype(np.float32)
        tiny[:, 0] = np.abs(tiny).max(1) * 1.01  # the largest is positive: a negative scale
        tiny[:, 5:7] = -tiny[:, :1] / 2
        clean = x.copy()
        for i in range(rows):
            x[i, 0, 32 * (i % 8):32 * (i % 8) + 32], clean[i, 0, 32 * (i % 8):32 * (i % 8) + 32] = tiny[i], 0
        got = {}
        for what, data in (("tiny", x), ("clean", clean)):
            c = BatchCache([(0, rows)], 1, 1, k_fmt, v_fmt, 63, written="before", fill=0).on_gpu(kv)
            t = torch.from_numpy(data).cuda()
            kv.kvattn_append_batch(c.desc, c.batch, t, t)
            back = [torch.zeros((rows, 1, 256), device="cuda") for _ in range(2)]
            kv.kvattn_read_batch(c.desc, c.batch, *back)
            got[what] = [b.cpu().numpy() for b in back]
            k2, v2 = torch.zeros_like(c.k_pool), torch.zeros_like(c.v_pool)
            d2 = kv.make_desc(1, 1, k2, v2, c.n_phys, k_fmt=k_fmt, v_fmt=v_fmt)
            kv.kvattn_quantize_append(d2, t, t, rows, 0, c.t_table[0].contiguous(), c.blocks)
            assert torch.equal(k2, c.k_pool) and torch.equal(v2, c.v_pool), what
        for a, b in zip(got["tiny"], got["clean"]):
            assert np.array_equal(a, b)
    assert kv.kvattn_device_error() == 0
