"""CPU: argument checks of the ragged-batch calls (made before anything touches a GPU), and the
tests' own page writer against the oracle's page encoder."""
import ctypes

import numpy as np
import pytest

from helpers_batch import PAIRS, put_tokens
from oracle import layout as olay
from oracle import quant as oq
from quantized_paged_kv_q4_b200 import build, kvattn


@pytest.fixture(scope="module")
def lib():
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses passed here are not memory: only where no device can be initialised")
    build.build()
    return kvattn.lib()


def desc(**kw):
    base = dict(n_kv_heads=4, n_q_heads=24, k_pool=16 * 1000, v_pool=16 * 5000, n_pages=64)
    base.update(kw)
    return kvattn.make_desc(**base)


def batch(**kw):
    base = dict(row_start=64, pos_start=64, page_table=64, n_rows=10, n_seqs=3, max_rows=4, max_blocks=9, reserved=0)
    base.update(kw)
    return kvattn.kvattn_batch(**base)


def rows(heads, **kw):
    base = dict(data=4096, row_stride=heads * 256, head_stride=256, dtype=kvattn.BF16, reserved=0)
    base.update(kw)
    return kvattn.kvattn_rows(**base)


def calls(lib, d, b, kv=None, kv2=None, q=None, out=None, lse=64, ws=256, ws_bytes=1 << 40, window=0):
    """Status of each of the three calls for these arguments."""
    k, v = kv or rows(4), kv2 or rows(4)
    q, out = q or rows(24), out or rows(24)
    return {"append": lib.kvattn_append_batch(d, b, k, v, None), "read": lib.kvattn_read_batch(d, b, k, v, None),
            "decode": lib.kvattn_decode_batch(d, b, q, None, None, window, out, lse, ws, ws_bytes, None)}


INVALID, FORMAT, SHAPE = kvattn.ERR_INVALID_ARG, kvattn.ERR_UNSUPPORTED_FORMAT, kvattn.ERR_UNSUPPORTED_SHAPE


def test_good_arguments_reach_the_device_check(lib):
    # no device here was initialised: everything before that check has passed
    for st in calls(lib, desc(), batch()).values():
        assert st in (kvattn.ERR_NOT_INITIALIZED, kvattn.ERR_CUDA)


@pytest.mark.parametrize("kw", [dict(n_seqs=-1), dict(n_rows=-1), dict(n_rows=2 ** 31), dict(max_rows=-1),
                                dict(max_blocks=-1), dict(max_blocks=2 ** 24 + 1), dict(reserved=1),
                                dict(row_start=None), dict(pos_start=None), dict(page_table=None)])
def test_bad_batches(lib, kw):
    assert set(calls(lib, desc(), batch(**kw)).values()) == {INVALID}
    assert lib.kvattn_decode_batch_workspace_size(desc(), batch(**kw)) == 0


def test_too_many_units(lib):
    good = (kvattn.ERR_NOT_INITIALIZED, kvattn.ERR_CUDA)
    assert all(st in good for st in calls(lib, desc(), batch(n_seqs=1 << 25, max_blocks=1)).values())
    assert set(calls(lib, desc(), batch(n_seqs=(1 << 25) + 1, max_blocks=1)).values()) == {SHAPE}


def test_null_arguments(lib):
    b, d, k = batch(), desc(), rows(4)
    assert lib.kvattn_append_batch(None, b, k, k, None) == INVALID
    assert lib.kvattn_append_batch(d, None, k, k, None) == INVALID
    assert lib.kvattn_append_batch(d, b, None, k, None) == INVALID
    assert lib.kvattn_append_batch(d, b, k, None, None) == INVALID
    assert lib.kvattn_read_batch(d, b, None, None, None) == kvattn.OK  # nothing asked for
    assert lib.kvattn_decode_batch(d, b, None, None, None, 0, rows(24), 64, 256, 1 << 40, None) == INVALID
    assert lib.kvattn_decode_batch(d, b, rows(24), None, None, 0, None, 64, 256, 1 << 40, None) == INVALID


@pytest.mark.parametrize("kw,want", [(dict(data=None), INVALID), (dict(data=4104), INVALID), (dict(reserved=3), INVALID),
                                     (dict(dtype=3), FORMAT), (dict(dtype=-1), FORMAT),
                                     (dict(row_stride=4 * 256 + 4), INVALID), (dict(head_stride=257), INVALID),
                                     (dict(row_stride=-1024), INVALID), (dict(row_stride=1 << 60), INVALID)])
def test_bad_rows(lib, kw, want):
    got = calls(lib, desc(), batch(), kv=rows(4, **kw), q=rows(24, **kw))
    assert set(got.values()) == {want}
    got = calls(lib, desc(), batch(), kv2=rows(4, **kw), out=rows(24, **kw))
    assert set(got.values()) == {want}


def test_mixed_types_are_refused(lib):
    got = calls(lib, desc(), batch(), kv=rows(4, dtype=kvattn.F32), q=rows(24, dtype=kvattn.F16))
    assert set(got.values()) == {FORMAT}


@pytest.mark.parametrize("heads,kw,ok", [
    (4, dict(row_stride=0), False),                          # every row in the same place
    (4, dict(head_stride=0), False),
    (4, dict(row_stride=256), False),                        # rows inside another row's heads
    (4, dict(row_stride=2048), True),                        # a slice of a wider array
    (4, dict(row_stride=256, head_stride=2560), True),       # head-major
    (4, dict(row_stride=256, head_stride=2552), False),      # head-major, a row too short
])
def test_outputs_may_not_overlap_themselves(lib, heads, kw, ok):
    good = (kvattn.ERR_NOT_INITIALIZED, kvattn.ERR_CUDA)
    d, b = desc(), batch()
    st = lib.kvattn_read_batch(d, b, rows(heads, **kw), None, None)
    assert (st in good) if ok else st == INVALID
    # the same strides are fine for an input
    assert lib.kvattn_append_batch(d, b, rows(heads, **kw), rows(heads), None) in good
    d1 = desc(n_kv_heads=1, n_q_heads=4)
    st = lib.kvattn_decode_batch(d1, b, rows(4, **kw), None, None, 0, rows(heads, **kw), 64, 256, 1 << 40, None)
    assert (st in good) if ok else st == INVALID


def test_strides_of_single_rows_and_heads_are_not_looked_at(lib):
    d = desc(n_kv_heads=1, n_q_heads=1)
    good = (kvattn.ERR_NOT_INITIALIZED, kvattn.ERR_CUDA)
    r = rows(1, row_stride=-5, head_stride=3)
    got = calls(lib, d, batch(n_rows=1), kv=r, kv2=r, q=r, out=r)
    assert all(st in good for st in got.values())


def test_decode_refusals(lib):
    d, b = desc(), batch()
    assert calls(lib, d, b, window=-1)["decode"] == INVALID
    assert calls(lib, d, b, lse=None)["decode"] == INVALID
    assert calls(lib, d, b, ws=None)["decode"] == INVALID
    assert calls(lib, d, b, ws=128)["decode"] == INVALID
    need = lib.kvattn_decode_batch_workspace_size(d, b)
    assert need > 0
    assert calls(lib, d, b, ws_bytes=need - 1)["decode"] == kvattn.ERR_WORKSPACE_TOO_SMALL
    assert calls(lib, d, batch(max_rows=5))["decode"] == SHAPE       # 6 query heads x 5 rows > 24
    assert calls(lib, desc(n_kv_heads=1, n_q_heads=25), batch(max_rows=1))["decode"] == SHAPE
    # the line of tiles is counted in 32 bits: n_seqs x H_kv x max_blocks <= 2^27
    assert calls(lib, d, batch(n_seqs=1 << 13, max_blocks=1 << 12, max_rows=1))["decode"] in (
        kvattn.ERR_NOT_INITIALIZED, kvattn.ERR_CUDA)
    assert calls(lib, d, batch(n_seqs=1 << 13, max_blocks=(1 << 12) + 1, max_rows=1))["decode"] == SHAPE
    for kf, vf in (("q5_0", "q4_0"), ("q8_0", "q4_1")):
        assert set(calls(lib, desc(k_fmt=kf, v_fmt=vf), b).values()) == {FORMAT}


def test_empty_batches_are_fine_without_a_device(lib):
    for kw in (dict(n_seqs=0, row_start=None, pos_start=None, page_table=None), dict(n_rows=0), dict(max_rows=0)):
        assert set(calls(lib, desc(), batch(**kw)).values()) == {kvattn.OK}


def test_binding_checks_tensors():
    import torch

    x = torch.zeros((3, 4, 256))
    with pytest.raises(ValueError, match="CUDA"):
        kvattn.make_rows(x, 3, 4, 0)
    fake = type("T", (), {"shape": (3, 4, 256), "dtype": torch.float64, "device": "cuda:1",
                          "get_device": lambda s: 1, "stride": lambda s: (1024, 256, 1)})
    with pytest.raises(ValueError, match="current device"):
        kvattn.make_rows(fake(), 3, 4, 0)
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        kvattn.make_rows(fake(), 3, 4, 1)
    with pytest.raises(ValueError, match="shape"):
        kvattn.make_rows(fake(), 3, 5, 1)
    fake.dtype, fake.stride = torch.float32, lambda s: (1024, 1, 4)
    with pytest.raises(ValueError, match="contiguous"):
        kvattn.make_rows(fake(), 3, 4, 1)
    with pytest.raises(ValueError, match="n_seqs"):
        kvattn.make_batch(x, x, x[0], 1, 1)
    i = torch.zeros((3, 4), dtype=torch.int32)
    for bad, match in ((i.long(), "int32"), (i[:2], "int32"), (i, "CUDA")):
        with pytest.raises(ValueError, match=match):
            kvattn._i32(bad, "n_pages", 0, (3, 4))
    assert kvattn._i32(None, "n_pages", 0, (3, 4)) is None
    b = batch()
    b.heads, b.device = 3, 0
    with pytest.raises(ValueError, match="KV heads"):
        kvattn.kvattn_read_batch(desc(), b)


@pytest.mark.parametrize("role,fmt", sorted({("k", k) for k, _ in PAIRS} | {("v", v) for _, v in PAIRS}))
def test_page_writer_of_these_tests(role, fmt):
    """Tokens put into a page one by one give the oracle's page, and leave other slots alone."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((128, 256)).astype(np.float32)
    page = rng.integers(0, 256, olay.page_bytes(role, fmt)).astype(np.uint8)
    got = page.copy()
    for t in rng.permutation(128):
        got = put_tokens(got, role, fmt, x[t:t + 1], t)
    codes, d = oq.quantize(x, fmt)
    assert np.array_equal(got, np.asarray(olay.encode_page(role, fmt, codes, d)).view(np.uint8).reshape(-1))
    once = put_tokens(page, role, fmt, x[5:6], 40)
    share = (once != page).mean()
    assert 0 < share <= 1 / 64
    assert ctypes.sizeof(kvattn.kvattn_batch) == 48 and ctypes.sizeof(kvattn.kvattn_rows) == 32
