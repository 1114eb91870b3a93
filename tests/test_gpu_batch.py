"""GPU: the ragged-batch calls (append, read back, attention) against the oracle, at the lengths,
types, strides and masks where they can go wrong."""
import numpy as np
import pytest

from oracle import quant as oq
from helpers_batch import PAIRS, BatchCache, attend_rows, check_attention, put_tokens, tdtype

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]
# (tokens before, rows): empty sequences, single tokens, page and tile borders on every side
EDGES = [(0, 1), (0, 0), (15, 1), (16, 1), (127, 1), (128, 3), (126, 4), (0, 4), (333, 2), (0, 0), (1000, 4), (2047, 1)]


def rounded(x, name):
    """x rounded to the type, as fp32 numpy and as a CUDA tensor."""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x)).to(tdtype(name))
    return t.float().numpy(), t.cuda()


def padded_rows(x, name, extra, value, layout="dense"):
    """A token array with `extra` rows behind the last sequence, in one of three layouts."""
    import torch

    n, H, D = x.shape
    if layout == "dense":
        t = torch.full((n + extra, H, D), value, dtype=tdtype(name), device="cuda")
    elif layout == "fused":    # a slice of a wider projection
        t = torch.full((n + extra, H + 3, D), value, dtype=tdtype(name), device="cuda")[:, 2:2 + H]
    else:                      # head-major
        t = torch.full((H, n + extra + 1, D), value, dtype=tdtype(name), device="cuda")[:, :n + extra].transpose(0, 1)
    t[:n] = torch.from_numpy(x).to(t)
    return t


# ------------------------------------------------------------------------------- append
@pytest.mark.parametrize("k_fmt,v_fmt", PAIRS)
@pytest.mark.parametrize("name", TYPES)
def test_append_writes_the_oracles_bytes(kv_gpu, k_fmt, v_fmt, name):
    c = BatchCache([(0, 1), (5, 0), (15, 3), (120, 20), (0, 150), (255, 1), (7, 41), (112, 16)], 2, 3, k_fmt, v_fmt, 11,
                   written="before")
    layout = {"float32": "dense", "float16": "fused", "bfloat16": "heads"}[name]
    kx, vx = (rounded(c.rows_of(w), name)[0] for w in ("k", "v"))
    k, v = (padded_rows(x, name, 3, 9.0, layout) for x in (kx, vx))
    c.on_gpu(kv_gpu, n_rows=c.total + 3)
    kv_gpu.kvattn_append_batch(c.desc, c.batch, k, v)
    assert kv_gpu.kvattn_device_error() == 0
    want_k, want_v = c.k_bytes.copy(), c.v_bytes.copy()
    for s, (ctx, rows) in enumerate(c.lens):
        for h in range(c.H):
            for i in range(rows):
                page, slot, r = c.table[s, h, (ctx + i) // 128], (ctx + i) % 128, c.row_start[s] + i
                want_k[page] = put_tokens(want_k[page], "k", k_fmt, kx[r:r + 1, h], slot)
                want_v[page] = put_tokens(want_v[page], "v", v_fmt, vx[r:r + 1, h], slot)
    assert np.array_equal(c.k_pool.cpu().numpy(), want_k)
    assert np.array_equal(c.v_pool.cpu().numpy(), want_v)


def positive_zeros(page, fmt):
    """The page with -0 minima as +0.  Row 8 of the test below holds zeros of both signs; which of them
    a minimum over the block returns is not defined (numpy's own answer depends on its vector
    width), and q * d + -0 equals q * d + 0 for every code."""
    if fmt in ("q5_1", "q4_1"):
        page = page.copy()
        low = page[-2048:].view(np.uint16)
        low[low == 0x8000] = 0
    return page


def test_append_zero_and_extreme_rows(kv_gpu):
    """Zero blocks, single loud elements, ties of sign, values near the top of fp16's range."""
    import torch

    for k_fmt, v_fmt in PAIRS:
        c = BatchCache([(0, 40)], 1, 1, k_fmt, v_fmt, 3, written="before", fill=0)
        x = np.random.default_rng(4).standard_normal((40, 1, 256)).astype(np.float32)
        x[0] = 0
        x[1, 0, 5] = 4000.0
        x[2, 0, ::2], x[2, 0, 1::2] = 1.5, -1.5
        x[3] = 0.25
        x[4:8] *= 3e4 / np.abs(x[4:8]).max()
        x[8] = -x[8] * 0
        x[16:32] *= 1e-3
        c.on_gpu(kv_gpu)
        t = torch.from_numpy(x).cuda()
        kv_gpu.kvattn_append_batch(c.desc, c.batch, t, t)
        page = c.table[0, 0, 0]
        for pool, role, fmt, old in ((c.k_pool, "k", k_fmt, c.k_bytes), (c.v_pool, "v", v_fmt, c.v_bytes)):
            got, want = pool.cpu().numpy()[page], put_tokens(old[page], role, fmt, x[:, 0], 0)
            assert np.array_equal(positive_zeros(got, fmt), positive_zeros(want, fmt)), (role, fmt)
    assert kv_gpu.kvattn_device_error() == 0


# --------------------------------------------------------------------------------- read
@pytest.mark.parametrize("k_fmt,v_fmt", PAIRS)
@pytest.mark.parametrize("name", TYPES)
def test_read_gives_the_held_values(kv_gpu, k_fmt, v_fmt, name):
    import torch

    c = BatchCache([(0, 1), (5, 0), (15, 3), (120, 20), (0, 150), (255, 1), (7, 41), (112, 16), (0, 300)], 2, 3, k_fmt,
                   v_fmt, 12)
    layout = {"float32": "heads", "float16": "dense", "bfloat16": "fused"}[name]
    zeros = np.full((c.total, 2, 256), 5.0, np.float32)
    k, v = (padded_rows(zeros, name, 2, 5.0, layout) for _ in range(2))
    c.on_gpu(kv_gpu, n_rows=c.total + 2)
    kv_gpu.kvattn_read_batch(c.desc, c.batch, k, v)
    assert kv_gpu.kvattn_device_error() == 0
    for which, got in (("k", k), ("v", v)):
        fmt = k_fmt if which == "k" else v_fmt
        x = c.rows_of(which)
        # the value rounded to fp32 and then to the type, as documented
        want = torch.from_numpy(oq.dequantize(*oq.quantize(x, fmt), fmt)).float().to(tdtype(name))
        assert torch.equal(got[:c.total].cpu(), want), which
        assert (got[c.total:] == 5.0).all(), "rows of no sequence were written"
    # one side alone leaves the other as it was
    k2 = torch.zeros((c.total + 2, 2, 256), dtype=tdtype(name), device="cuda")
    kv_gpu.kvattn_read_batch(c.desc, c.batch, k=k2)
    assert torch.equal(k2[:c.total], k[:c.total])
    kv_gpu.kvattn_read_batch(c.desc, c.batch, v=k2)
    assert torch.equal(k2[:c.total], v[:c.total])


# ------------------------------------------------------------------------------- decode
def run_decode(kv, c, name, seed=0, window=0, extra=2, layout="dense", lists=None, q_scale=1.0, ws=None):
    import torch

    rng = np.random.default_rng(seed)
    Hq = c.H * c.group
    qx = rounded(rng.standard_normal((c.total, Hq, 256)).astype(np.float32) * q_scale, name)[0]
    c.on_gpu(kv, n_rows=c.total + extra)
    q = padded_rows(qx, name, extra, 0.5, layout)
    out = padded_rows(np.full_like(qx, 3.0), name, extra, 3.0, layout)
    lse = torch.full((c.total + extra, Hq), 4.0, device="cuda")
    kw = {}
    if lists is not None:
        c.t_table.copy_(torch.from_numpy(lists["table"]))
        kw = {"page_logical": None if lists["logical"] is None else torch.from_numpy(lists["logical"]).cuda(),
              "n_pages": None if lists["n"] is None else torch.from_numpy(lists["n"]).cuda()}
    if ws is None:
        ws = torch.empty(kv.kvattn_decode_batch_workspace_size(c.desc, c.batch), dtype=torch.uint8, device="cuda")
        ws.fill_(0xFF)
    kv.kvattn_decode_batch(c.desc, c.batch, q, out, lse, ws, window=window, **kw)
    assert kv.kvattn_device_error() == 0
    assert (out[c.total:] == 3.0).all() and (lse[c.total:] == 4.0).all(), "rows of no sequence were written"
    return qx, out[:c.total].float().cpu().numpy(), lse[:c.total].cpu().numpy()


def check_decode(c, name, qx, out, lse, window=0, listed=None):
    for s, (ctx, rows) in enumerate(c.lens):
        pos = np.arange(ctx + rows)
        for i in range(rows):
            r = c.row_start[s] + i
            seen = pos <= ctx + i
            if window:
                seen &= pos > ctx + i - window
            for h in range(c.H):
                ok = seen if listed is None else seen & np.isin(pos // 128, listed(s, h))
                rows_q = qx[r, h * c.group:(h + 1) * c.group]
                ref = attend_rows(rows_q, c.held(s, h, "k"), c.held(s, h, "v"),
                                  np.broadcast_to(ok, (c.group, ok.size)), *c.codes(s, h))
                check_attention(out[r, h * c.group:(h + 1) * c.group], lse[r, h * c.group:(h + 1) * c.group], *ref,
                                int(ok.sum()), name)


@pytest.mark.parametrize("k_fmt,v_fmt", PAIRS)
@pytest.mark.parametrize("name", TYPES)
def test_decode_edges(kv_gpu, k_fmt, v_fmt, name):
    c = BatchCache(EDGES, 2, 3, k_fmt, v_fmt, 21)
    check_decode(c, name, *run_decode(kv_gpu, c, name, layout={"float32": "fused", "float16": "heads"}.get(name, "dense")))


@pytest.mark.parametrize("H,group,rows", [(1, 1, 1), (1, 6, 4), (4, 6, 1), (3, 8, 3), (2, 24, 1), (2, 2, 8), (1, 5, 2),
                                          (1, 1, 24), (5, 7, 1)])
@pytest.mark.parametrize("name", ["float32", "bfloat16"])
def test_decode_head_layouts(kv_gpu, H, group, rows, name):
    lens = [(100, rows), (0, 1), (700, max(1, rows - 1)), (1, rows)]
    c = BatchCache(lens, H, group, "q8_0", "q4_0", 22)
    check_decode(c, name, *run_decode(kv_gpu, c, name, seed=3))


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 128, 129, 1000, 100000])
@pytest.mark.parametrize("name", ["float32", "bfloat16"])
def test_decode_window(kv_gpu, window, name):
    c = BatchCache([(0, 1), (127, 3), (500, 4), (1300, 2), (128, 1), (15, 2)], 2, 6, "q4_0", "q4_0", 23)
    # pages the window has left behind may be gone: their entries are never read
    for s, (ctx, _) in enumerate(c.lens):
        c.table[s, :, :max(0, ctx + 1 - window) // 128] = -3
    check_decode(c, name, *run_decode(kv_gpu, c, name, window=window), window=window)


@pytest.mark.parametrize("name", ["float32", "float16", "bfloat16"])
def test_decode_selected_pages(kv_gpu, name):
    """Lists in any order, a head with no page at all, blocks past the sequence's end."""
    c = BatchCache([(900, 4), (300, 1), (2000, 2)], 2, 4, "q8_0", "q4_0", 24)
    rng = np.random.default_rng(5)
    logical = np.full((3, 2, c.blocks), -9, np.int32)
    table = np.full_like(logical, -9)
    n = np.zeros((3, 2), np.int32)
    chosen = {}
    for s, (ctx, rows) in enumerate(c.lens):
        nb = (ctx + rows + 127) // 128
        for h in range(2):
            take = 0 if (s, h) == (1, 1) else rng.integers(1, nb + 1)
            pick = rng.permutation(nb)[:take]
            chosen[s, h] = pick
            n[s, h], logical[s, h, :take], table[s, h, :take] = take, pick, c.table[s, h, pick]
    got = run_decode(kv_gpu, c, name, lists={"table": table, "logical": logical, "n": n})
    check_decode(c, name, *got, listed=lambda s, h: chosen[s, h])
    assert np.isneginf(got[2][4, 4:]).all() and (got[1][4, 4:] == 0).all()
    # n_pages alone: a prefix of the blocks
    short = np.minimum(n + 1, 3).astype(np.int32)
    got = run_decode(kv_gpu, c, name, lists={"table": c.table, "logical": None, "n": short})
    check_decode(c, name, *got, listed=lambda s, h: np.arange(short[s, h]))


def test_decode_window_over_selected_pages(kv_gpu):
    c = BatchCache([(900, 4), (2000, 2)], 1, 6, "q8_0", "q8_0", 25)
    logical = np.stack([np.concatenate([np.arange(c.blocks - 1)[::-1], [0]])[None] for _ in c.lens]).astype(np.int32)
    n = np.array([[8], [16]], np.int32)
    for s in range(2):
        nb = (sum(c.lens[s]) + 127) // 128
        logical[s, 0, :n[s, 0]] = np.arange(nb)[::-1][:n[s, 0]]
    table = np.take_along_axis(c.table, logical.astype(np.int64), 2)
    got = run_decode(kv_gpu, c, "bfloat16", window=300, lists={"table": table, "logical": logical, "n": n})
    check_decode(c, "bfloat16", *got, window=300)


@pytest.mark.parametrize("n_seqs", [1, 33, 200])
@pytest.mark.parametrize("name", ["bfloat16", "float32"])
def test_decode_many_sequences(kv_gpu, n_seqs, name):
    rng = np.random.default_rng(n_seqs)
    lens = [(int(rng.integers(0, 300)), int(rng.integers(0, 3))) for _ in range(n_seqs)]
    lens[0] = (6000, 1)
    c = BatchCache(lens, 1, 6, "q4_0", "q4_0", 26)
    check_decode(c, name, *run_decode(kv_gpu, c, name))


def test_decode_same_result_every_time_and_in_any_place(kv_gpu):
    """The same call twice gives the same bits, whatever the workspace held."""
    import torch

    c = BatchCache([(3000, 4), (10, 1), (777, 2)], 4, 6, "q8_0", "q4_0", 27)
    a = run_decode(kv_gpu, c, "float32", seed=9)
    ws = torch.randint(0, 255, (kv_gpu.kvattn_decode_batch_workspace_size(c.desc, c.batch),), dtype=torch.uint8,
                       device="cuda")
    for _ in range(3):
        b = run_decode(kv_gpu, c, "float32", seed=9, ws=ws)
        assert np.array_equal(a[1], b[1]) and np.array_equal(a[2], b[2])


@pytest.mark.parametrize("k_fmt,v_fmt", PAIRS)
def test_decode_large_and_small_values(kv_gpu, k_fmt, v_fmt):
    """Values up to the top of fp16's range, and a thousandth: P times the scale stays finite in f16."""
    for scale in (6e4, 1e-3):
        c = BatchCache([(200, 2), (0, 1)], 1, 4, k_fmt, v_fmt, 28)
        for s in range(2):
            c.v[s] *= scale / np.abs(c.v[s]).max()
            for b in range((len(c.v[s]) + 127) // 128):
                page = c.table[s, 0, b]
                c.v_bytes[page] = put_tokens(c.v_bytes[page], "v", v_fmt, c.v[s][128 * b:128 * b + 128, 0], 0)
        for name in ("float32", "bfloat16"):
            qx, out, lse = run_decode(kv_gpu, c, name)
            assert np.isfinite(out).all()
            check_decode(c, name, qx, out, lse)


def test_decode_peaked_scores(kv_gpu):
    """Scores that span hundreds: one key takes all of the weight, and the running maximum moves often."""
    c = BatchCache([(1500, 2)], 1, 6, "q8_0", "q8_0", 29)
    c.k[0] *= np.linspace(0.05, 4, 1502)[:, None, None].astype(np.float32)
    for b in range(12):
        page = c.table[0, 0, b]
        c.k_bytes[page] = put_tokens(c.k_bytes[page], "k", "q8_0", c.k[0][128 * b:128 * b + 128, 0], 0)
    for name in TYPES:
        check_decode(c, name, *run_decode(kv_gpu, c, name, q_scale=8.0))


def test_decode_in_place_and_on_few_sms(kv_gpu):
    """out may be q's array; a descriptor's SM budget sizes the grid (other splits, the same answer)."""
    import torch

    for lens, group in (([(2000, 1), (3, 1), (700, 1)], 6), ([(2000, 4), (3, 2), (700, 3)], 6)):
        c = BatchCache(lens, 2, group, "q8_0", "q4_0", 51).on_gpu(kv_gpu)
        for budget in (0, 3, 40):
            c.desc.sm_budget = budget
            qx, q = rounded(np.random.default_rng(1).standard_normal((c.total, 2 * group, 256)).astype(np.float32), "float32")
            lse = torch.zeros((c.total, 2 * group), device="cuda")
            ws = torch.empty(kv_gpu.kvattn_decode_batch_workspace_size(c.desc, c.batch), dtype=torch.uint8, device="cuda")
            kv_gpu.kvattn_decode_batch(c.desc, c.batch, q, q, lse, ws)
            check_decode(c, "float32", qx, q.cpu().numpy(), lse.cpu().numpy())
    assert kv_gpu.kvattn_device_error() == 0


def test_decode_nan_and_inf_queries_stay_in_their_row(kv_gpu):
    import torch

    for lens in ([(40, 1), (3000, 1)], [(40, 2), (3000, 3)]):
        for name in TYPES:
            c = BatchCache(lens, 1, 6, "q8_0", "q4_0", 52).on_gpu(kv_gpu)
            qx, q = rounded(np.random.default_rng(2).standard_normal((c.total, 6, 256)).astype(np.float32), name)
            bad = [(0, 2, 7, float("nan")), (c.total - 1, 5, 250, float("inf"))]
            for r, h, ch, x in bad:
                q[r, h, ch] = x
            out, lse = torch.zeros_like(q), torch.zeros((c.total, 6), device="cuda")
            ws = torch.empty(kv_gpu.kvattn_decode_batch_workspace_size(c.desc, c.batch), dtype=torch.uint8, device="cuda")
            kv_gpu.kvattn_decode_batch(c.desc, c.batch, q, out, lse, ws)
            o, l = out.float().cpu().numpy(), lse.cpu().numpy()
            for r, h, _, _ in bad:
                assert np.isnan(o[r, h]).all() and np.isnan(l[r, h])
                # the row's own place aside, the answer is that of the clean queries
                o[r, h], l[r, h] = 0, 0
            assert np.isfinite(o).all() and np.isfinite(l).all()
            out2, lse2 = torch.zeros_like(q), torch.zeros_like(lse)
            kv_gpu.kvattn_decode_batch(c.desc, c.batch, torch.from_numpy(qx).to(q), out2, lse2, ws)
            o2, l2 = out2.float().cpu().numpy(), lse2.cpu().numpy()
            for r, h, _, _ in bad:
                o2[r, h], l2[r, h] = 0, 0
            assert np.array_equal(o, o2) and np.array_equal(l, l2)
    assert kv_gpu.kvattn_device_error() == 0


def test_two_streams_and_two_graphs(kv_gpu):
    """Calls on two streams at once with a workspace each; two captured graphs that share one workspace,
    replayed in turn; lengths that change between replays."""
    import torch

    kv = kv_gpu
    a = BatchCache([(900, 1), (50, 1), (4000, 1)], 2, 6, "q8_0", "q4_0", 53).on_gpu(kv)
    b = BatchCache([(300, 4), (1200, 2)], 2, 6, "q4_0", "q4_0", 54).on_gpu(kv)
    sets = []
    for c, name, seed in ((a, "bfloat16", 1), (b, "float32", 2)):
        qx, q = rounded(np.random.default_rng(seed).standard_normal((c.total, 12, 256)).astype(np.float32), name)
        size = kv.kvattn_decode_batch_workspace_size(c.desc, c.batch)
        sets.append([c, name, qx, q, torch.zeros_like(q), torch.zeros((c.total, 12), device="cuda"), size])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    own_ws = [torch.empty(s[6], dtype=torch.uint8, device="cuda") for s in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws, st in zip(sets, own_ws, streams):
            kv.kvattn_decode_batch(s[0].desc, s[0].batch, s[3], s[4], s[5], ws, stream=st)
    torch.cuda.synchronize()
    for c, name, qx, _, out, lse, _ in sets:
        check_decode(c, name, qx, out.float().cpu().numpy(), lse.cpu().numpy())
    shared = torch.empty(max(s[6] for s in sets), dtype=torch.uint8, device="cuda")
    graphs = []
    for c, _, _, q, out, lse, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv.kvattn_decode_batch(c.desc, c.batch, q, out, lse, shared)
        graphs.append(g)
    for _ in range(3):
        for s in sets:
            s[4].zero_()
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, name, qx, _, out, lse, _ in sets:
        check_decode(c, name, qx, out.float().cpu().numpy(), lse.cpu().numpy())
    # the first graph again, with its sequences cut short
    a.t_pos.copy_(torch.tensor([100, 0, 2500], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    a.lens = [(100, 1), (0, 1), (2500, 1)]
    for s in range(3):
        a.k[s], a.v[s] = a.k[s][:sum(a.lens[s])], a.v[s][:sum(a.lens[s])]
    check_decode(a, "bfloat16", sets[0][2], sets[0][4].float().cpu().numpy(), sets[0][5].cpu().numpy())
    assert kv.kvattn_device_error() == 0


@pytest.mark.parametrize("group,rows", [(6, 1), (6, 3)])
def test_decode_long_and_short_together(kv_gpu, group, rows):
    """One long sequence among many single tokens: stretches that hold many units, units of many parts."""
    lens = [(0, 1)] * 60 + [(9000, rows)] + [(0, 0)] * 40 + [(int(i), 1) for i in range(37)]
    c = BatchCache(lens, 1, group, "q8_0", "q4_0", 55)
    check_decode(c, "bfloat16", *run_decode(kv_gpu, c, "bfloat16"))


# ------------------------------------------------------------------------- device checks
def test_bad_sequences_and_pages_are_left_out(kv_gpu):
    import torch

    kv = kv_gpu
    good = BatchCache([(40, 2), (200, 1), (0, 3)], 2, 6, "q8_0", "q4_0", 31)
    name = "float32"
    want = run_decode(kv, good, name)
    for what in ("rows", "order", "range", "pos", "blocks", "negative"):
        good.on_gpu(kv)
        row, pos = good.row_start.copy(), good.pos_start.copy()
        if what == "rows":
            good.batch.max_rows = 2        # the third sequence has three
        if what == "order":
            # the third sequence descends, and the second, by the same entry, has rows 2 .. 4: each is
            # checked by itself, so the second is answered
            row[2], row[3] = 5, 3
        if what == "range":
            row[3] = 100
        if what == "pos":
            pos[2] = -1
        if what == "blocks":
            pos[2] = 128 * good.blocks - 2
        if what == "negative":
            pos[2] = 2 ** 31 - 2
        good.t_row.copy_(torch.from_numpy(row))
        good.t_pos.copy_(torch.from_numpy(pos))
        q = torch.from_numpy(want[0]).cuda()
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        ws = torch.empty(kv.kvattn_decode_batch_workspace_size(good.desc, good.batch), dtype=torch.uint8, device="cuda")
        kv.kvattn_decode_batch(good.desc, good.batch, q, out, lse, ws)
        assert kv.kvattn_device_error() == kv.ERR_INVALID_ARG, what
        n, left = (2, 5) if what == "order" else (3, 3)
        assert (out[left:] == 7).all() and (lse[left:] == 7).all(), what
        assert np.array_equal(out[:n].cpu().numpy(), want[1][:n]), what
        k = torch.full((6, 2, 256), 7.0, device="cuda")
        kv.kvattn_read_batch(good.desc, good.batch, k, k.clone())
        assert kv.kvattn_device_error() == kv.ERR_INVALID_ARG, what
        assert (k[left:] == 7).all() and (k[:n] != 7).any()
        before = good.k_pool.clone()
        kv.kvattn_append_batch(good.desc, good.batch, k, k)
        assert kv.kvattn_device_error() == kv.ERR_INVALID_ARG, what
        keep = [p for p in range(good.n_phys) if p not in set(good.table[:2].ravel())]
        assert torch.equal(good.k_pool[keep], before[keep])


def test_bad_page_ids_are_skipped(kv_gpu):
    import torch

    kv = kv_gpu
    c = BatchCache([(300, 2), (40, 1)], 1, 6, "q8_0", "q4_0", 32).on_gpu(kv)
    table = c.table.copy()
    table[0, 0, 1] = c.n_phys
    table[1, 0, 0] = -2
    c.t_table.copy_(torch.from_numpy(table))
    q = torch.randn((3, 6, 256), device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((3, 6), 7.0, device="cuda")
    ws = torch.empty(kv.kvattn_decode_batch_workspace_size(c.desc, c.batch), dtype=torch.uint8, device="cuda")
    kv.kvattn_decode_batch(c.desc, c.batch, q, out, lse, ws)
    assert kv.kvattn_device_error() == kv.ERR_BAD_PAGE
    check_decode(BatchCacheView(c, 1), "float32", q.cpu().numpy(), out.cpu().numpy(), lse.cpu().numpy(),
                 listed=lambda s, h: np.array([0, 2]))
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    k = torch.full((3, 1, 256), 7.0, device="cuda")
    kv.kvattn_read_batch(c.desc, c.batch, k, k.clone())
    assert kv.kvattn_device_error() == kv.ERR_BAD_PAGE
    assert (k[2] == 0).all() and (k[:2] != 0).any()
    before = c.k_pool.clone()
    kv.kvattn_append_batch(c.desc, c.batch, k, k)
    assert kv.kvattn_device_error() == kv.ERR_BAD_PAGE
    changed = (c.k_pool != before).any(1).nonzero().ravel().cpu().tolist()
    assert set(changed) <= set(c.table[0, 0, 2:3])


class BatchCacheView:
    """The first n sequences of a cache."""

    def __init__(self, c, n):
        self.__dict__.update(c.__dict__)
        self.lens = c.lens[:n]
        self.held, self.codes = c.held, c.codes


def test_empty_calls(kv_gpu):
    import torch

    kv = kv_gpu
    c = BatchCache([(0, 0), (300, 0)], 1, 6, "q8_0", "q4_0", 33).on_gpu(kv)
    x = torch.zeros((0, 1, 256), device="cuda")
    kv.kvattn_append_batch(c.desc, c.batch, x, x)
    kv.kvattn_read_batch(c.desc, c.batch, x, x)
    ws = torch.empty(kv.kvattn_decode_batch_workspace_size(c.desc, c.batch), dtype=torch.uint8, device="cuda")
    kv.kvattn_decode_batch(c.desc, c.batch, torch.zeros((0, 6, 256), device="cuda"),
                           torch.zeros((0, 6, 256), device="cuda"), torch.zeros((0, 6), device="cuda"), ws)
    none = kv.make_batch(torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                         torch.zeros((0, 1, 4), dtype=torch.int32, device="cuda"), 5, 1)
    y = torch.full((5, 1, 256), 2.0, device="cuda")
    kv.kvattn_append_batch(c.desc, none, y, y)
    kv.kvattn_read_batch(c.desc, none, y, y.clone())
    assert (y == 2).all()
    assert kv.kvattn_device_error() == 0


# ------------------------------------------------------- the calls together, as they are used
@pytest.mark.parametrize("name", TYPES)
def test_serving_steps(kv_gpu, name):
    """Prompts are appended, then several steps append and attend, on a stream of their own and as a
    captured graph; every step agrees with the single-sequence calls and with the oracle, and the
    cache reads back what it holds."""
    import torch

    kv = kv_gpu
    prompts, steps, H, group = [70, 1, 300], 4, 2, 6
    c = BatchCache([(p, steps) for p in prompts], H, group, "q8_0", "q4_0", 41, written="before", fill=0)
    for s in range(3):  # what the typed rows hold
        c.k[s], c.v[s] = rounded(c.k[s], name)[0], rounded(c.v[s], name)[0]
    c.k_bytes[:], c.v_bytes[:] = 0, 0
    c.on_gpu(kv)
    dt = tdtype(name)
    S = len(prompts)
    # the prompts, in one call
    row = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32, device="cuda")
    zero = torch.zeros(S, dtype=torch.int32, device="cuda")
    first = kv.make_batch(row, zero, c.t_table, sum(prompts), max(prompts))
    kp, vp = (torch.from_numpy(np.concatenate([x[s][:prompts[s]] for s in range(S)])).to(dt).cuda() for x in (c.k, c.v))
    kv.kvattn_append_batch(c.desc, first, kp, vp)
    # then one token of every sequence a step
    row1 = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    pos = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    step = kv.make_batch(row1, pos, c.t_table, S, 1)
    qkv = torch.zeros((S, H * group + 2 * H, 256), dtype=dt, device="cuda")
    q, k, v = qkv[:, :H * group], qkv[:, H * group:H * group + H], qkv[:, H * group + H:]
    out, lse = torch.zeros((S, H * group, 256), dtype=dt, device="cuda"), torch.zeros((S, H * group), device="cuda")
    ws = torch.empty(kv.kvattn_decode_batch_workspace_size(c.desc, step), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(6)

    def one_step():
        kv.kvattn_append_batch(c.desc, step, k, v)
        kv.kvattn_decode_batch(c.desc, step, q, out, lse, ws)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for i in range(steps):
        qx = rng.standard_normal((S, H * group, 256)).astype(np.float32)
        qx, q_new = rounded(qx, name)
        q.copy_(q_new)
        for s in range(S):
            k[s] = torch.from_numpy(c.k[s][prompts[s] + i]).to(dt)
            v[s] = torch.from_numpy(c.v[s][prompts[s] + i]).to(dt)
        torch.cuda.synchronize()
        if i == 0:
            with torch.cuda.stream(side):
                one_step()
            side.synchronize()
        elif i == 1:
            with torch.cuda.graph(graph):
                one_step()
            graph.replay()
        else:
            graph.replay()
        torch.cuda.synchronize()
        o, l = out.float().cpu().numpy(), lse.cpu().numpy()
        for s in range(S):
            n = prompts[s] + i + 1
            for h in range(H):
                kh = oq.dequantize(*oq.quantize(c.k[s][:n, h], "q8_0"), "q8_0")
                vh = oq.dequantize(*oq.quantize(c.v[s][:n, h], "q4_0"), "q4_0")
                ref = attend_rows(qx[s, h * group:(h + 1) * group], kh, vh, np.ones((group, n), bool),
                                  *(x[:n] for x in c.codes(s, h)))
                check_attention(o[s, h * group:(h + 1) * group], l[s, h * group:(h + 1) * group], *ref, n, name)
        pos += 1
    # the bytes are those of the single-sequence writer
    k2, v2 = torch.zeros_like(c.k_pool), torch.zeros_like(c.v_pool)
    d2 = kv.make_desc(H, H * group, k2, v2, c.n_phys)
    for s in range(S):
        kv.kvattn_quantize_append(d2, torch.from_numpy(c.k[s]).cuda(), torch.from_numpy(c.v[s]).cuda(),
                                  prompts[s] + steps, 0, c.t_table[s].contiguous(), c.blocks)
    assert torch.equal(k2, c.k_pool) and torch.equal(v2, c.v_pool)
    # the whole history of every sequence, read back
    lens = [p + steps for p in prompts]
    row = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    whole = kv.make_batch(row, zero, c.t_table, sum(lens), max(lens))
    kr = torch.zeros((sum(lens), H, 256), dtype=dt, device="cuda")
    vr = torch.zeros_like(kr)
    kv.kvattn_read_batch(c.desc, whole, kr, vr)
    at = 0
    for s in range(S):
        for got, x, fmt in ((kr, c.k[s], "q8_0"), (vr, c.v[s], "q4_0")):
            want = torch.from_numpy(oq.dequantize(*oq.quantize(x, fmt), fmt)).float().to(dt)
            assert torch.equal(got[at:at + lens[s]].cpu(), want)
        at += lens[s]
    assert kv.kvattn_device_error() == 0


def test_offsets_past_32_bits(kv_gpu):
    """Pages at byte offsets above 2^32 of a large pool, and rows at element offsets above 2^31 of a
    strided array."""
    import torch

    kv = kv_gpu
    stride = 34816 * 64                     # a wide page stride puts few pages far apart
    n = (5 << 30) // stride
    pool = torch.zeros(n * stride, dtype=torch.uint8, device="cuda")
    vpool = torch.zeros((n, 18432), dtype=torch.uint8, device="cuda")
    d = kv.make_desc(1, 6, pool, vpool, n, k_page_stride=stride)
    table = torch.tensor([[[n - 1, 0, n - 2]]], dtype=torch.int32, device="cuda")
    assert (n - 2) * stride > 2 ** 32
    row = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    wide = (1 << 31) // 3 + 8 - ((1 << 31) // 3) % 8
    big = torch.zeros(3 * wide + 256, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (4, 1, 256), (wide, 256, 1))
    x.copy_(torch.randn((4, 1, 256), device="cuda"))
    assert 3 * wide > 2 ** 31
    pos = torch.tensor([254], dtype=torch.int32, device="cuda")
    b = kv.make_batch(row, pos, table, 4, 4)
    kv.kvattn_append_batch(d, b, x, x)
    back, vback = torch.zeros((4, 1, 256), device="cuda"), torch.zeros((4, 1, 256), device="cuda")
    kv.kvattn_read_batch(d, b, back, vback)
    for got, fmt in ((back, "q8_0"), (vback, "q4_0")):
        want = oq.dequantize(*oq.quantize(x.float().cpu().numpy(), fmt), fmt)
        assert np.array_equal(got.cpu().numpy(), want.astype(np.float32))
    q = torch.randn((4, 6, 256), device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((4, 6), device="cuda")
    ws = torch.empty(kv.kvattn_decode_batch_workspace_size(d, b), dtype=torch.uint8, device="cuda")
    kv.kvattn_decode_batch(d, b, q, out, lse, ws, window=2)
    for i in range(4):
        lo = max(0, i - 1)
        # a row's window reaches the row before it; position 253, before the first, holds zeros
        keys = np.concatenate([np.zeros((1 if i == 0 else 0, 256)), back[lo:i + 1, 0].cpu().numpy()])
        vals = np.concatenate([np.zeros((1 if i == 0 else 0, 256)), vback[lo:i + 1, 0].cpu().numpy()])
        ref = attend_rows(q[i].cpu().numpy(), keys, vals, np.ones((6, 2), bool), np.full((2, 256), 8),
                          np.abs(vals).max(1, keepdims=True) / 8)
        check_attention(out[i].cpu().numpy(), lse[i].cpu().numpy(), *ref, 2, "float32")
    assert kv.kvattn_device_error() == 0
