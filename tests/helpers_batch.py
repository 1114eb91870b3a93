"""Shared helpers of the ragged-batch tests: a cache of several sequences built from the oracle's
page encoder, the oracle's answers, and error bounds.  Imported by tests only."""
from __future__ import annotations

import numpy as np

from oracle import layout as olay
from oracle import quant as oq

PAIRS = [("q8_0", "q4_0"), ("q8_0", "q8_0"), ("q4_0", "q4_0"), ("q4_0", "q8_0"), ("q5_1", "q4_0"), ("q5_1", "q8_0"),
         ("q5_0", "q4_1")]
EPS = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}  # half a step, relative


def tdtype(name):
    import torch

    return getattr(torch, name)


class BatchCache:
    """`lens` = [(tokens before the call, rows of the call)] per sequence.  K and V of every token are
    drawn N(0, 1) with loud channels; `fill` is the byte of every slot no token was written to
    (0xFF: scales and minima are NaN there).  written: how many of a sequence's tokens sit in its
    pages already (default: all, the call's own included)."""

    def __init__(self, lens, H, group, k_fmt, v_fmt, seed, fill=0xFF, written="all", extra_blocks=1, extra_pages=3):
        import torch

        rng = np.random.default_rng(seed)
        self.lens, self.H, self.group, self.k_fmt, self.v_fmt = lens, H, group, k_fmt, v_fmt
        self.S = len(lens)
        self.blocks = max([(c + r + 127) // 128 for c, r in lens] + [1]) + extra_blocks
        n_used = [H * ((c + r + 127) // 128) for c, r in lens]
        self.n_phys = sum(n_used) + extra_pages
        perm = rng.permutation(self.n_phys).astype(np.int32)
        self.table = np.full((self.S, H, self.blocks), -7, np.int32)  # entries no token needs
        self.k, self.v = [], []
        loud = np.where(rng.random(256) < 0.02, 8.0, 1.0).astype(np.float32)
        kp = np.full((self.n_phys, olay.page_bytes("k", k_fmt)), fill, np.uint8)
        vp = np.full((self.n_phys, olay.page_bytes("v", v_fmt)), fill, np.uint8)
        at = 0
        for s, (c, r) in enumerate(lens):
            T, nb = c + r, (c + r + 127) // 128
            self.table[s, :, :nb] = perm[at:at + H * nb].reshape(H, nb)
            at += H * nb
            self.k.append((rng.standard_normal((T, H, 256)) * loud).astype(np.float32))
            self.v.append((rng.standard_normal((T, H, 256)) * loud).astype(np.float32))
            held = T if written == "all" else c
            for h in range(H):
                for b in range((held + 127) // 128):
                    n = min(128, held - 128 * b)
                    page = self.table[s, h, b]
                    kp[page] = put_tokens(kp[page], "k", k_fmt, self.k[s][128 * b:128 * b + n, h], 0)
                    vp[page] = put_tokens(vp[page], "v", v_fmt, self.v[s][128 * b:128 * b + n, h], 0)
        self.k_bytes, self.v_bytes = kp, vp
        self.row_start = np.concatenate([[0], np.cumsum([r for _, r in lens])]).astype(np.int32)
        self.total = int(self.row_start[-1])
        self.pos_start = np.array([c for c, _ in lens], np.int32)
        self.max_rows = max([r for _, r in lens] + [1])
        self.torch = torch

    def on_gpu(self, kv, n_rows=None, **desc):
        torch = self.torch
        self.k_pool = torch.from_numpy(self.k_bytes).cuda()
        self.v_pool = torch.from_numpy(self.v_bytes).cuda()
        self.t_row, self.t_pos, self.t_table = (torch.from_numpy(x).cuda()
                                                for x in (self.row_start, self.pos_start, self.table))
        self.desc = kv.make_desc(self.H, self.H * self.group, self.k_pool, self.v_pool, self.n_phys,
                                 k_fmt=self.k_fmt, v_fmt=self.v_fmt, **desc)
        self.batch = kv.make_batch(self.t_row, self.t_pos, self.t_table, self.total if n_rows is None else n_rows,
                                   self.max_rows)
        return self

    def rows_of(self, which):
        """The call's own rows of K or V: [total][H][256]."""
        x = self.k if which == "k" else self.v
        return np.concatenate([a[c:c + r] for a, (c, r) in zip(x, self.lens)] + [np.zeros((0, self.H, 256), np.float32)])

    def held(self, s, h, which):
        fmt, x = (self.k_fmt, self.k) if which == "k" else (self.v_fmt, self.v)
        return oq.dequantize(*oq.quantize(x[s][:, h], fmt), fmt)

    def codes(self, s, h):
        """|code| (the whole number that multiplies the block's scale) and |scale| of the sequence's values."""
        q, d = oq.quantize(self.v[s][:, h], self.v_fmt)
        d = np.abs((d if d.ndim == 2 else d[..., 0]).astype(np.float64))
        return (np.abs(q.astype(np.int64) - (8 if self.v_fmt == "q4_0" else 0)).reshape(-1, 256),
                np.repeat(d, 32, axis=-1))


def put_tokens(page, role, fmt, x, slot):
    """The page bytes after tokens x [n][256] were encoded into slots slot, slot + 1, ..."""
    n = x.shape[0]
    codes, d = oq.quantize(np.ascontiguousarray(x, np.float32), fmt)
    full_c = np.zeros((128,) + codes.shape[1:], codes.dtype)
    full_d = np.zeros((128,) + d.shape[1:], d.dtype)
    full_c[slot:slot + n], full_d[slot:slot + n] = codes, d
    new = np.asarray(olay.encode_page(role, fmt, full_c, full_d)).view(np.uint8).reshape(-1)
    # which bits belong to the written slots: those that all-ones codes and scales set
    top = {"q8_0": 127, "q4_0": 15, "q4_1": 15, "q5_0": 31, "q5_1": 31}[fmt]
    mask_c, mask_d = np.zeros_like(full_c), np.zeros_like(full_d)
    mask_c[slot:slot + n] = top
    mask_d.view(np.uint16)[slot:slot + n] = 0xFFFF
    base_c = np.full_like(full_c, -128) if fmt == "q8_0" else np.zeros_like(full_c)
    if fmt == "q8_0":
        base_c[slot:slot + n] = 127  # offset-binary byte 255
        mask_c = base_c
    mask = np.asarray(olay.encode_page(role, fmt, mask_c, mask_d)).view(np.uint8).reshape(-1)
    return (page & ~mask) | (new & mask)


def attend_rows(q, k, v, seen, codes, scales):
    """Exact attention of rows q [n][256] over keys k, v [T][256] where seen [n][T], float64: (o, lse,
    sum p max(|v|, |code x scale|), max_t sum_c |q k| / 16, the sum that f16's smallest step can add,
    below).  codes, scales [T][256]: |code| and |scale| of every value.

    P enters the MMAs relative to the running maximum, which is within 2^2 of the row's own, so the
    largest P is >= 1 and the sum of P is >= 1 / max p with p normalised.  Its f16 parts, and those of
    P x scale, end at f16's subnormal step 2^-24: a key's P is off by up to 2^-25 and its product by up to
    2 x 2^-25 (a high and a low part), whatever their size, times |v| and |code|."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    s = np.where(seen, q @ k.T / 16.0, -np.inf)
    big = np.abs(q) @ np.abs(k).T / 16.0
    m = np.max(s, axis=1, initial=-np.inf)
    live = np.isfinite(m)
    p = np.where(seen, np.exp(s - np.where(live, m, 0)[:, None]), 0)
    tot = p.sum(1)
    safe = np.where(live, tot, 1)
    p = p / safe[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(live, m + np.log(safe), -np.inf)
    v = np.where(seen.any(0)[:, None], v, 0)
    floor = (seen @ np.abs(codes) * 2.0 ** -24 + seen @ np.abs(v) * 2.0 ** -25) * p.max(1, initial=0)[:, None]
    return p @ v, lse, p @ np.maximum(np.abs(v), codes * scales), np.max(np.where(seen, big, 0), axis=1, initial=0), floor


def check_attention(o, lse, o_ref, lse_ref, pv, big, floor, n_keys, dtype):
    """Bounds by arithmetic.  A score is a sum of 256 products of a query held to 22 bits (error <=
    2^-22 of sum |q k| / 16 = big) accumulated in fp32 over 8 blocks of 4 MMAs, each step within
    2^-24 of the running sum (< 2^-19 big with the scaling); the exponential adds 2^-21 relative,
    so a weight is off by ew = 2^-18 big + 2^-21 relative, in the numerator and in the sum.  The
    output accumulates one MMA step per 16 keys and a merge, each 2^-24 of the sum of p times what is
    added: code x scale, and a minimum where the format has one, each at most 2 pv, with pv = sum p
    max(|v|, |code x scale|).  bf16 outputs take P (2^-12 of p |v|), and P times the value's scale (2^-12
    of p |code x scale|), rounded to f16: 2^-11 pv.  f16's smallest step adds `floor` (attend_rows).  The
    store rounds once."""
    ew = 2.0 ** -18 * big + 2.0 ** -21
    acc = 4 * (n_keys / 16 + 64) * 2.0 ** -24
    tol = (2 * ew + acc + (2.0 ** -11 if dtype == "bfloat16" else 2.0 ** -20))[:, None] * pv + floor
    tol = tol + EPS[dtype] * (np.abs(o_ref) + tol) + 1e-30
    # f16 has no more than its smallest subnormal step below 2^-14
    tol = tol + (2.0 ** -25 if dtype == "float16" else 0)
    err = np.abs(np.asarray(o, np.float64) - o_ref)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), (worst, err[worst], tol[worst], o_ref[worst])
    assert np.array_equal(np.isneginf(lse), np.isneginf(lse_ref))
    fin = np.isfinite(lse_ref)
    ltol = ew + np.abs(np.where(fin, lse_ref, 0)) * 2.0 ** -22 + acc
    assert (np.abs(lse[fin] - lse_ref[fin]) <= ltol[fin]).all(), np.abs(lse[fin] - lse_ref[fin]).max()
