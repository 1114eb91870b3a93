"""GPU: the ragged-batch decode where its numbers and its work get uneven: dominant keys, tiny and huge values,
values that are not finite, long stretches, rings that fill over a page's end, more units than the grid has
places, and lists that the selection fills."""
import numpy as np
import pytest

from helpers_batch import EPS, PAIRS, BatchCache
from oracle import layout as olay
from oracle import quant as oq
from test_gpu_batch import check_decode, rounded, run_decode

pytestmark = pytest.mark.gpu
TYPES = ["float32", "float16", "bfloat16"]


# --------------------------------------------------- what the header states, with no floor of its own
def exact_rows(q, k, v):
    """Attention of rows q [n][256] over keys k and values v [T][256], float64, with what the bound needs:
    (o, lse, p [n][T], sum_c |q k| / 16 at its largest, [n])."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    s = q @ k.T / 16.0
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    tot = p.sum(1, keepdims=True)
    big = np.array([(np.abs(a) @ np.abs(k).T).max() for a in q]) / 16.0
    return p / tot @ v, (m + np.log(tot))[:, 0], p / tot, big


def half_step(x, dtype):
    least = {"float32": -126, "float16": -14, "bfloat16": -126}[dtype]
    return np.exp2(np.maximum(np.floor(np.log2(np.maximum(x, 1e-300))), least)) * EPS[dtype]


def check_range(out, lse, ref, v, codes, scales, dtype, tiles):
    """The bounds of the header, by arithmetic.
    Scores: products of a query held to 22 bits (fp32; 16-bit queries are exact here), accumulated in fp32
    by 4 MMAs in each of 8 blocks: 2^-18 of sum |q k| / 16 = big, and 2^-21 for the exponential, in the
    numerator and in the sum.
    P and P x scale: 2^-22 each in two f16 parts; the parts end 2^-37 below the row's largest P times the larger
    of 1 and the largest scale (P), and 2^-36 below the largest P times the largest scale (the product).
    Accumulation: one step per MMA, two MMAs per tile of 16 keys, in a group's share of `tiles`: each
    step cuts at most 2^-23 of the sum so far, twice what a rounding would; a merge adds a few.
    (fp32 outputs add every tile's two MMAs by themselves: within the same bound.)
    The store rounds once, by half a step of the value's own binade."""
    o_ref, lse_ref, p, big = ref
    dmax = float(np.abs(scales).max())
    top = p.max(1, keepdims=True)
    mass = np.abs(v) + codes * scales  # what is added: codes times scales, and minima
    pv = p @ mass
    floor = top * (2.0 ** -37 * max(1.0, dmax) * mass.sum(0) + 2.0 ** -36 * max(dmax, 2.0 ** -16) * codes.sum(0))
    ew = 2.0 ** -18 * big + 2.0 ** -21
    tol = (2 * ew + 2.0 ** -20 + (2 * tiles + 64) * 2.0 ** -23)[:, None] * pv + floor
    tol = tol + half_step(np.abs(o_ref) + tol, dtype)
    gone = ~np.isfinite(lse_ref)  # rows that see a key which fp16 does not hold: nothing is said of them
    if gone.any():
        return tol
    err = np.abs(np.asarray(out, np.float64) - o_ref)
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert (err <= tol).all(), (worst, err[worst], tol[worst], o_ref[worst])
    ltol = ew + (2 * tiles + 64) * 2.0 ** -23 + np.abs(lse_ref) * 2.0 ** -22
    assert (np.abs(lse - lse_ref) <= ltol).all(), np.abs(lse - lse_ref).max()
    return tol


class History:
    """One KV head's T tokens in oracle-encoded pages, which any number of sequences share."""

    def __init__(self, kv, group, k_fmt, v_fmt, k, v, poison=()):
        """poison: (token, block, 0 or 1 for the value's scale or minimum, what to put there)."""
        import torch

        T = k.shape[0]
        self.T, self.group, self.v_fmt, n = T, group, v_fmt, (T + 127) // 128
        pools, self.held, quantized = [], [], []
        for role, fmt, x in (("k", k_fmt, k), ("v", v_fmt, v)):
            codes, d = oq.quantize(x, fmt)
            if role == "v":
                for token, block, which, what in poison:
                    d[(token, block) + ((which,) if d.ndim == 3 else ())] = what
            quantized.append((codes, d))
            self.held.append(oq.dequantize(codes, d, fmt))
            pad = lambda a: np.concatenate([a, np.zeros((n * 128 - T,) + a.shape[1:], a.dtype)])  # noqa: E731
            codes, d = pad(codes), pad(d)
            pages = [np.asarray(olay.encode_page(role, fmt, codes[128 * b:128 * b + 128], d[128 * b:128 * b + 128]))
                     .view(np.uint8).reshape(-1) for b in range(n)]
            pools.append(torch.from_numpy(np.stack(pages)).cuda())
        codes, d = quantized[1]
        d = np.abs((d if d.ndim == 2 else d[..., 0]).astype(np.float64))
        self.codes = np.abs(codes.astype(np.int64) - (8 if v_fmt == "q4_0" else 0)).reshape(-1, 256)
        self.scales = np.repeat(d, 32, axis=-1)
        self.pools, self.n = pools, n
        self.table = torch.arange(n, dtype=torch.int32, device="cuda")[None, None]
        self.desc = kv.make_desc(1, group, *pools, n, k_fmt=k_fmt, v_fmt=v_fmt)

    def exact(self, q):
        return exact_rows(q, *self.held)

    def check(self, out, lse, ref, dtype):
        return check_range(out, lse, ref, self.held[1], self.codes, self.scales, dtype, self.n * 8)

    def decode(self, kv, name, n_seqs, budget, q):
        """The newest token of n_seqs sequences, queries q [1][group][256] each, on `budget` SMs."""
        return self.batch(kv, name, np.repeat(q, n_seqs, 0), [self.T - 1] * n_seqs, [1] * n_seqs, budget=budget)

    def batch(self, kv, name, q, pos, rows, window=0, budget=0, listed=False):
        """Sequences of rows[s] tokens from position pos[s] on, queries q [sum of rows][group][256]."""
        import torch

        self.desc.sm_budget = budget
        S = len(pos)
        row = torch.from_numpy(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).cuda()
        start = torch.tensor(pos, dtype=torch.int32, device="cuda")
        table = self.table.expand(S, 1, self.n).contiguous()
        batch = kv.make_batch(row, start, table, int(sum(rows)), max(rows))
        qt = torch.from_numpy(np.ascontiguousarray(q)).to(getattr(torch, name)).cuda()
        out, lse = torch.zeros_like(qt), torch.zeros(qt.shape[:2], device="cuda")
        ws = torch.empty(kv.kvattn_decode_batch_workspace_size(self.desc, batch), dtype=torch.uint8, device="cuda")
        kw = {"page_logical": table, "n_pages": torch.full((S, 1), self.n, dtype=torch.int32, device="cuda")} if listed else {}
        kv.kvattn_decode_batch(self.desc, batch, qt, out, lse, ws, window=window, **kw)
        assert kv.kvattn_device_error() == 0
        return out.float().cpu().numpy(), lse.cpu().numpy()


def history(rng, T, spread, mean, logit, q_scale, group):
    """Keys and queries with N(0, q_scale) scores, key 0 `logit` above them with a value near zero."""
    sign = np.where(rng.random(256) < 0.5, -1.0, 1.0).astype(np.float32)
    k = rng.standard_normal((T, 256)).astype(np.float32)
    v = (rng.standard_normal((T, 256)) * spread + mean).astype(np.float32)
    q = (rng.standard_normal((1, group, 256)) * q_scale).astype(np.float32)
    if logit:
        k[0] = sign
        v[0] *= 1e-3
        q = q + (logit / 16 - q @ sign / 256)[..., None] * sign  # q . k0 / 16 = logit
    return k, v, q.astype(np.float32)


@pytest.mark.parametrize("v_fmt,spread,mean", [("q8_0", 0.1, 0.05), ("q4_0", 0.03, 0.01), ("q8_0", 1e-3, 4e-4),
                                               ("q4_1", 1.0, 0.5), ("q4_1", 1e-2, 5e-3)])
@pytest.mark.parametrize("logit", [0, 8, 12, 16])
@pytest.mark.parametrize("group", [6, 20])
def test_values_behind_a_dominant_key(kv_gpu, v_fmt, spread, mean, logit, group):
    """An attention sink in position 0: the other keys' weights are far below 1 and their small values
    make the answer.  The history in one warp group's stretch, and cut into many; the answers agree with each
    other as with the definition."""
    k_fmt = "q5_0" if v_fmt == "q4_1" else "q8_0"
    k, v, q = history(np.random.default_rng(int(logit * 10 + group)), 4096, spread, mean, logit,
                      2.0 if logit == 0 else 1.0, group)
    c = History(kv_gpu, group, k_fmt, v_fmt, k, v)
    for name in TYPES:
        qx = rounded(q, name)[0]
        ref = c.exact(qx[0])
        for n_seqs, budget in ((1, 0), (26, 1)):
            out, lse = c.decode(kv_gpu, name, n_seqs, budget, qx)
            for s in range(n_seqs):
                tol = c.check(out[s], lse[s], ref, name)
            if name == "float32":  # zeros, or answers 1 % off, would not pass
                assert (np.median(np.abs(ref[0]) / tol) > 100) or logit > 12


@pytest.mark.parametrize("k_fmt,v_fmt", PAIRS)
@pytest.mark.parametrize("amplitude", [1e-3, 1.0, 100.0, 6e4, 4e5])
def test_amplitudes_of_values(kv_gpu, k_fmt, v_fmt, amplitude):
    """Values from a thousandth to the top of what the formats hold."""
    rng = np.random.default_rng(7)
    for T, group in ((700, 4), (333, 12)):
        k, v, q = history(rng, T, 1.0, 0.3, 0, 1.5, group)
        # the largest scale stays below fp16's largest number: 8 (Q4_0), 127 (Q8_0) and 15 (Q4_1) codes a side
        v *= min(amplitude, {"q4_0": 8, "q8_0": 127, "q4_1": 1}[v_fmt] * 65000) / np.abs(v).max()
        c = History(kv_gpu, group, k_fmt, v_fmt, k, v)
        for name in ("float32", "bfloat16"):
            qx = rounded(q, name)[0]
            ref = c.exact(qx[0])
            out, lse = c.decode(kv_gpu, name, 3, 1, qx)
            for s in range(3):
                c.check(out[s], lse[s], ref, name)


@pytest.mark.parametrize("group", [4, 16])
def test_scales_that_grow_and_shrink(kv_gpu, group):
    """Loud and quiet stretches of values in turn, in one group's stretch: the sums follow the loudest."""
    rng = np.random.default_rng(8)
    T = 2048
    k, v, q = history(rng, T, 1.0, 0.2, 0, 1.0, group)
    v *= np.repeat(10.0 ** np.array([-4, 0, 2, -2, 4, -5, 1, 3]), T // 8)[:, None].astype(np.float32)
    for v_fmt in ("q8_0", "q4_0"):
        c = History(kv_gpu, group, "q8_0", v_fmt, k, v)
        for name in ("float32", "bfloat16"):
            qx = rounded(q, name)[0]
            ref = c.exact(qx[0])
            out, lse = c.decode(kv_gpu, name, 14, 1, qx)
            for s in range(14):
                c.check(out[s], lse[s], ref, name)


@pytest.mark.parametrize("n_q", [1, 4])
@pytest.mark.parametrize("logit", [0, 8, 12])
def test_single_sequence_decode_behind_a_dominant_key(kv_gpu, n_q, logit):
    """The single-sequence call has the same arithmetic, on one SM's stretch and on all."""
    import torch

    kv = kv_gpu
    rng = np.random.default_rng(9)
    T, group = 4096, 6
    k, v, q = history(rng, T, 0.1, 0.05, logit, 1.0, group)
    q = np.repeat(q, n_q, 0)
    for v_fmt in ("q8_0", "q4_0"):
        c = History(kv, group, "q8_0", v_fmt, k, v)
        ref = c.exact(q[0])
        for budget in (0, 1):
            c.desc.sm_budget = budget
            out, lse = torch.zeros((n_q, group, 256), device="cuda"), torch.zeros((n_q, group), device="cuda")
            pos = torch.full((n_q,), T - 1, dtype=torch.int32, device="cuda")
            size = kv.kvattn_decode_workspace_size(c.desc, n_q, c.n)
            ws = torch.zeros(max(size, 256), dtype=torch.uint8, device="cuda")
            kv.kvattn_decode(c.desc, torch.from_numpy(q).cuda(), n_q, pos, c.table[0], None, None, c.n, out, lse, ws,
                             size)
            for i in range(n_q):
                c.check(out[i].cpu().numpy(), lse[i].cpu().numpy(), ref, "float32")


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
@pytest.mark.parametrize("group", [6, 20])
def test_outputs_of_16_bits_are_rounded_once(kv_gpu, name, group):
    """What the kernel holds before the store is as exact as for fp32: the output is the definition's nearest
    value, but where that lies within the header's bound of a border between two.  How many are not: an
    error of 2^-20 of the sum of p |v| crosses a border with a chance of 2 x error / step."""
    import torch

    for k_fmt, v_fmt in PAIRS:
        k, v, q = history(np.random.default_rng(15), 700, 1.0, 0.1, 0, 1.0, group)
        c = History(kv_gpu, group, k_fmt, v_fmt, k, v)
        qx = rounded(q, name)[0]
        ref = c.exact(qx[0])
        nearest = torch.from_numpy(ref[0]).to(getattr(torch, name)).float().numpy()
        chance = 2.0 ** -20 * (ref[2] @ (np.abs(c.held[1]) + c.codes * c.scales)) / half_step(np.abs(ref[0]), name)
        allowed = np.minimum(chance, 1).sum()
        out, lse = c.decode(kv_gpu, name, 3, 1, qx)
        for s in range(3):
            c.check(out[s], lse[s], ref, name)
            assert (out[s] != nearest).sum() <= allowed + 5 * allowed ** 0.5 + 5, (k_fmt, v_fmt)


@pytest.mark.parametrize("name,spread", [("float16", 2.0 ** 28), ("bfloat16", 2.0 ** 24), ("float32", 2.0 ** 12)])
@pytest.mark.parametrize("k_fmt,v_fmt", [("q8_0", "q4_0"), ("q5_1", "q8_0"), ("q4_0", "q4_0")])
def test_queries_with_one_loud_channel(kv_gpu, name, spread, k_fmt, v_fmt):
    """A channel of the query `spread` times the others, where every key is zero: the others make the scores."""
    rng = np.random.default_rng(10)
    T = 300
    for group in (3, 12):
        k, v, q = history(rng, T, 1.0, 0.0, 0, 1.0, group)
        k[:, 32:64] = 0
        q = np.sign(q) * np.clip(np.abs(q), 0.25, 3)
        q[..., 40] = 2.0
        # fp16: from the bottom of the type to its top; the keys make up for the small queries
        low = 2.0 ** -14 if name == "float16" else 1.0
        q = (q * low).astype(np.float32)
        q[..., 40] *= spread
        for keys in (k / low, np.clip(k, -3, 3) / low):  # (with Q5_1 some of the first are past fp16's range)
            c = History(kv_gpu, group, k_fmt, v_fmt, keys.astype(np.float32), v)
            assert (c.held[0][:, 40] == 0).all()
            qx = rounded(q, name)[0]
            ref = c.exact(qx[0])
            out, lse = c.decode(kv_gpu, name, 2, 0, qx)
            for s in range(2):
                c.check(out[s], lse[s], ref, name)


@pytest.mark.parametrize("group", [4, 20])
def test_long_stretches_do_not_drift(kv_gpu, group):
    """2,048 tiles in one group's stretch, values of mostly one sign.  A sum that is cut in every step is low by up
    to 4,096 x 2^-23 of it (one unit in the last place of 24 bits a step).  Rounded tile by tile the errors are
    independent: sqrt(2,048 / 3) steps of 2^-24 / sqrt(3) = 9e-7 of the sum, a quarter of the bound.
    fp16: what the store rounds has no sign (the answers spread over ten steps around 1 and more): over 256 x group
    values the mean error is within 5 x half a step / sqrt(3 x 256 x group) and that bound.
    bf16 sums may be cut.  Their answers lie within a step or two of 1, where the steps above are twice those
    below, so that the roundings' mean says nothing: every value by itself is within half a step and the cuts."""
    k, v, q = history(np.random.default_rng(11), 32768, 0.5, 1.0, 0, 1.0, group)
    c = History(kv_gpu, group, "q4_0", "q8_0", k, v)
    for name in TYPES:
        qx = rounded(q, name)[0]
        ref = c.exact(qx[0])
        out, lse = c.decode(kv_gpu, name, 12, 1, qx)
        if name == "float32":
            err = np.linalg.norm((out - ref[0]).reshape(12, -1), axis=1) / np.linalg.norm(ref[0])
            assert err.max() < 2.0 ** -18, err
        elif name == "float16":
            drift = np.abs(((out - ref[0]) / ref[0]).reshape(12, -1).mean(1))
            assert drift.max() < 5 * EPS[name] / (3 * 256 * group) ** 0.5 + 2.0 ** -18, drift
        else:
            for s in range(12):
                c.check(out[s], lse[s], ref, name)


# ------------------------------------------------------------------ what is not finite
@pytest.mark.parametrize("v_fmt", ["q4_0", "q8_0", "q4_1"])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("group", [2, 6])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(kv_gpu, v_fmt, what, group):
    """A value scale (or minimum) that is not finite: the rows that see its key get channels of its block that
    are not finite, however small the key's weight is, and every other row and channel is exact."""
    rng = np.random.default_rng(12)
    rows, window, first = 3, 40, 300  # row i sees positions first + i - 39 .. first + i
    T = first + rows
    k, v, q = history(rng, T, 1.0, 0.2, 0, 1.0, group)
    sign = np.where(rng.random(256) < 0.5, -1.0, 1.0).astype(np.float32)
    k[first - 20] = -8 * sign  # far below every other key
    q = (np.repeat(q, rows, 0) + sign / 4).astype(np.float32)
    # the token before every window (its tile is read), one that only row 0 sees, the last row's own, and
    # one of almost no weight that all rows see
    for tokens in ([first - 40], [first - 39], [first + 2], [first - 20], [first - 40, first - 38, first + 1]):
        for which in (0, 1) if v_fmt == "q4_1" else (0,):
            c = History(kv_gpu, group, "q5_0" if v_fmt == "q4_1" else "q8_0", v_fmt, k, v,
                        [(x, 3, which, what) for x in tokens])
            clean = History(kv_gpu, group, "q5_0" if v_fmt == "q4_1" else "q8_0", v_fmt, k, v)
            for name in ("float32", "bfloat16"):
                qx = rounded(q, name)[0]
                out, lse = c.batch(kv_gpu, name, qx, [first], [rows], window=window)
                for i in range(rows):
                    low, last = first + i - window + 1, first + i
                    sl = slice(low, last + 1)
                    vd = clean.held[1][sl].copy()
                    poisoned = any(low <= x <= last for x in tokens)
                    ref = exact_rows(qx[i], c.held[0][sl], vd)
                    o = out[i].copy()
                    if poisoned:
                        assert not np.isfinite(o[:, 96:128]).any(), (tokens, i)
                        o[:, 96:128] = ref[0][:, 96:128]
                    check_range(o, lse[i], ref, vd, clean.codes[sl], clean.scales[sl], name, 4)


def test_stale_slots_do_not_move_the_powers_of_two(kv_gpu):
    """Slots past the sequence's end hold the largest scales there are: the answer is the same bits."""
    k, v, q = history(np.random.default_rng(13), 128, 0.1, 0.05, 10, 1.0, 6)
    tokens = 69
    for v_fmt in ("q4_0", "q8_0", "q4_1"):
        k_fmt = "q5_0" if v_fmt == "q4_1" else "q8_0"
        got = []
        for loud in (0, 1):
            x = v.copy()
            x[tokens:] *= 6e5 if loud and v_fmt != "q4_1" else 5e4 if loud else 1
            x[tokens:] = np.clip(x[tokens:], -5e5, 5e5)
            c = History(kv_gpu, 6, k_fmt, v_fmt, k, x)
            got.append([c.batch(kv_gpu, name, rounded(q, name)[0], [tokens - 1], [1]) for name in ("float32", "bfloat16")])
        for a, b in zip(*got):
            assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


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


@pytest.mark.parametrize("group,rows", [(6, 1), (6, 4), (2, 2)])
@pytest.mark.parametrize("how", ["whole", "window", "listed"])
def test_more_units_than_places(kv_gpu, group, rows, how):
    """A full server: 2,500 sequences, several to a thread of the plan and more than the grid has warp groups."""
    rng = np.random.default_rng(14)
    T = 420
    k, v, q = history(rng, T, 1.0, 0.1, 0, 1.0, group)
    c = History(kv_gpu, group, "q8_0", "q4_0", k, v)
    S, window = 2500, 100 if how == "window" else 0
    kinds = [(int(a), int(b)) for a, b in zip(rng.integers(0, T - rows, 12), rng.integers(0, rows + 1, 12))]
    kinds[0], kinds[1], kinds[2] = (0, 1), (T - rows, rows), (5, 0)
    pick = rng.integers(0, 12, S)
    n_rows = [kinds[i][1] for i in pick]
    for name in ("float32", "bfloat16"):
        per_kind = rounded(rng.standard_normal((12, rows, group, 256)).astype(np.float32), name)[0]
        qx = np.concatenate([per_kind[i, :n] for i, n in zip(pick, n_rows)])
        out, lse = c.batch(kv_gpu, name, qx, [kinds[i][0] for i in pick], n_rows, window=window, listed=how == "listed")
        starts = np.concatenate([[0], np.cumsum(n_rows)])
        for i, (pos, n) in enumerate(kinds):
            which = np.nonzero(pick == i)[0]
            for j in range(n):
                low = max(0, pos + j - window + 1) if window else 0
                sl = slice(low, pos + j + 1)
                ref = exact_rows(per_kind[i, j], c.held[0][sl], c.held[1][sl])
                for s in which[:40]:
                    r = starts[s] + j
                    check_range(out[r], lse[r], ref, c.held[1][sl], c.codes[sl], c.scales[sl], name, 27)
                # sequences that are alike get answers that differ by their cuts alone
                assert np.abs(out[starts[which] + j] - out[starts[which[0]] + j]).max() <= (1e-5 if name == "float32" else 0.02)


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


# ------------------------------------------------------------------- selection, then attention
@pytest.mark.parametrize("name", ["float32", "bfloat16"])
def test_selected_blocks_of_sequences_of_different_lengths(kv_gpu, name):
    """Summaries and a selection per sequence, each into its own rows of the lists, and one attention call."""
    import torch

    kv = kv_gpu
    H, group, budget, recent, cap = 2, 6, 3, 1, 6
    c = BatchCache([(1500, 2), (700, 1), (300, 3)], H, group, "q8_0", "q4_0", 64).on_gpu(kv)
    rng = np.random.default_rng(16)
    qx = rounded(rng.standard_normal((c.total, H * group, 256)).astype(np.float32), name)[0]
    q = torch.from_numpy(qx).to(getattr(torch, name)).cuda()
    logical, phys = (torch.full((3, H, cap), -5, dtype=torch.int32, device="cuda") for _ in range(2))
    n = torch.zeros((3, H), dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.kvattn_select_workspace_size(H, c.blocks), dtype=torch.uint8, device="cuda")
    for s, (ctx, rows) in enumerate(c.lens):
        full, total = (ctx + rows) // 128, (ctx + rows + 127) // 128
        summaries = torch.zeros((H, c.blocks, 256), device="cuda")
        table = c.t_table[s].contiguous()
        kv.kvattn_block_summaries(c.desc, table, H, c.blocks, 0, full, summaries)
        ask = q[int(c.row_start[s])].float().view(H, group, 256).contiguous()
        kv.kvattn_select_blocks(summaries, ask, H, group, c.blocks, full, total, budget, recent, table, logical[s],
                                phys[s], n[s], cap, ws, ws.nbytes)
    batch = kv.make_batch(c.t_row, c.t_pos, phys, c.total, c.max_rows)
    out, lse = torch.zeros_like(q), torch.zeros((c.total, H * group), device="cuda")
    dws = torch.empty(kv.kvattn_decode_batch_workspace_size(c.desc, batch), dtype=torch.uint8, device="cuda")
    kv.kvattn_decode_batch(c.desc, batch, q, out, lse, dws, page_logical=logical, n_pages=n)
    assert kv.kvattn_device_error() == 0
    log, counts = logical.cpu().numpy(), n.cpu().numpy()
    assert (counts == np.array([[5], [5], [3]])).all()  # budget, the recent block and the tail; 300 + 3 tokens: all
    check_decode(c, name, qx, out.float().cpu().numpy(), lse.cpu().numpy(), listed=lambda s, h: log[s, h, :counts[s, h]])


# ----------------------------------------------------------------- inputs that are not finite
@pytest.mark.parametrize("k_fmt,v_fmt", PAIRS)
def test_inputs_that_are_not_finite_are_written_as_by_the_single_sequence_call(kv_gpu, k_fmt, v_fmt):
    """NaN and infinities, alone and together, in some blocks: the same bytes from both writers, and every other
    block's are those of clean rows."""
    import torch

    kv = kv_gpu
    rng = np.random.default_rng(17)
    for rows in (16, 5):
        x = rng.standard_normal((rows, 1, 256)).astype(np.float32)
        clean = x.copy()
        for i in range(rows):
            block = 32 * (i % 8)
            for j, what in enumerate((np.nan, np.inf, -np.inf)):
                if (i + 1) >> j & 1:
                    x[i, 0, block + rng.choice(32, 2, replace=False)] = what
            clean[i, 0, block:block + 32] = 0
        back = {}
        for what, data in (("odd", x), ("clean", clean)):
            c = BatchCache([(0, rows)], 1, 1, k_fmt, v_fmt, 63, written="before", fill=0).on_gpu(kv)
            t = torch.from_numpy(data).cuda()
            kv.kvattn_append_batch(c.desc, c.batch, t, t)
            k2, v2 = torch.zeros_like(c.k_pool), torch.zeros_like(c.v_pool)
            d2 = kv.make_desc(1, 1, k2, v2, c.n_phys, k_fmt=k_fmt, v_fmt=v_fmt)
            kv.kvattn_quantize_append(d2, t, t, rows, 0, c.t_table[0].contiguous(), c.blocks)
            assert torch.equal(k2, c.k_pool) and torch.equal(v2, c.v_pool), what
            back[what] = [torch.zeros((rows, 1, 256), device="cuda") for _ in range(2)]
            kv.kvattn_read_batch(c.desc, c.batch, *back[what])
        for a, b in zip(back["odd"], back["clean"]):
            for i in range(rows):
                keep = np.ones(256, bool)
                keep[32 * (i % 8):32 * (i % 8) + 32] = False
                assert np.array_equal(a.cpu().numpy()[i, 0, keep], b.cpu().numpy()[i, 0, keep])
    assert kv.kvattn_device_error() == 0
