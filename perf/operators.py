"""The operators of a ragged batch of sequences that share one quantized paged cache:

* ``append``: the new tokens of every sequence are quantized into the sequence's pages, and the
  values the cache then holds for them are read back;
* ``read``: the values the cache holds for a range of tokens of every sequence;
* ``attend``: the attention of the newest tokens of every sequence (one token, or a few drafted
  ones to verify) over its pages, in whole, over a sliding window, or over selected pages.

A case is a batch: ``seqs`` sequences, each with ``ctx`` tokens that came before the call and
``rows`` tokens that the call is about, both drawn per sequence from the case alone (``mix``).
The cache is the framework's: pages of 128 tokens of one KV head with 256 channels, a shuffled
page table, block formats of 32 channels with fp16 scales, each page in the byte order that
include/kvattn.h documents."""
import math
import random

import torch

own = False

PAGE, DIM, BLK = 128, 256, 32
NB = DIM // BLK
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PAIRS = ("q8_0/q4_0", "q4_0/q4_0", "q8_0/q8_0", "q5_0/q4_1", "q5_1/q4_0", "q4_0/q8_0", "q5_1/q8_0")
BITS = {"q8_0": 34, "q4_0": 18, "q5_0": 22, "q5_1": 24, "q4_1": 20}  # bytes per block of 32
HALF = {"q4_0": 8, "q5_0": 16}       # codes around an offset: value (q - half) d
TOP = {"q4_1": 15, "q5_1": 31}       # codes above a minimum: value q d + m


# ------------------------------------------------------------------------------- the cases
def _case(name, op, fmt, typ, seqs, rows, ctx, kv=4, group=6, window=0, pick=0, mix=1):
    return ({"name": name} if name else {}) | {
        "op": op, "fmt": fmt, "type": typ, "seqs": seqs, "rows_lo": rows[0], "rows_hi": rows[1], "ctx_lo": ctx[0],
        "ctx_hi": ctx[1], "kv": kv, "group": group, "window": window, "pick": pick, "mix": mix}


def listed():
    return [
        # one short conversation on a model with one KV head: what a single call costs
        _case("attend 1 x 4096", "attend", "q8_0/q4_0", "f32", 1, (1, 1), (4095, 4095), kv=1),
        # a server's decode step: many conversations of very different lengths
        _case("attend 32 ragged", "attend", "q4_0/q4_0", "bf16", 32, (1, 1), (17, 16384), mix=2),
        # a verify step with three drafted tokens
        _case("attend 8 verify", "attend", "q8_0/q4_0", "bf16", 8, (4, 4), (4001, 32768), mix=3),
        # the largest: eight long documents side by side
        _case("attend 8 x 131072", "attend", "q8_0/q4_0", "bf16", 8, (1, 1), (131071, 131071), mix=4),
        # a layer with a sliding window
        _case("attend 48 window", "attend", "q5_0/q4_1", "f16", 48, (1, 2), (100, 20000), window=1024, mix=5),
        # pages picked by a retrieval query out of long histories
        _case("attend 2 picked", "attend", "q8_0/q4_0", "f32", 2, (4, 4), (262140, 262140), pick=384, mix=6),
        # the tokens of one decode step
        _case("append 64 x 1", "append", "q8_0/q4_0", "bf16", 64, (1, 1), (17, 16384), mix=7),
        # prompts of several users, in one chunk
        _case("append 6 prompts", "append", "q4_0/q4_0", "bf16", 6, (100, 4000), (0, 9000), mix=8),
        # a prompt from fp32 projections into the format pair with the most parts
        _case("append f32 chunk", "append", "q5_0/q4_1", "f32", 2, (500, 2048), (0, 1000), mix=9),
        # the last few tokens of every sequence
        _case("read 16 x few", "read", "q8_0/q4_0", "bf16", 16, (1, 8), (17, 16384), mix=10),
        # a long history that goes to a kernel that takes 16-bit keys and values
        _case("read 131072", "read", "q8_0/q4_0", "bf16", 1, (131072, 131072), (0, 0), mix=11),
        # ragged histories, as fp32, from an 8-bit cache
        _case("read ragged", "read", "q5_1/q8_0", "f32", 12, (33, 6000), (0, 500), mix=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "append", "read"))
    fmt, typ = rng.choice(PAIRS), rng.choice(("f32", "f16", "bf16", "bf16"))
    kv = rng.choice((1, 2, 4, 8))
    mix = rng.randrange(1, 1 << 30)
    if op == "attend":
        group = rng.randint(1, 8)
        rows = rng.randint(1, min(4, 24 // group))
        hi = _log_int(rng, 64, 131072)
        seqs = min(_log_int(rng, 1, 64), max(1, (8 * 131072 * 4) // (hi * kv)))
        window = rng.choice((0, 0, 0, _log_int(rng, 1, hi)))
        pick = _log_int(rng, 1, max(1, hi // 256)) if not window and rng.random() < 0.25 else 0
        return _case(None, op, fmt, typ, seqs, (1, rows), (_log_int(rng, 1, hi), hi), kv, group, window, pick, mix)
    hi = _log_int(rng, 1, 16384 if op == "append" else 65536)
    seqs = min(_log_int(rng, 1, 64), max(1, (65536 if op == "append" else 131072) * 4 // (hi * kv)))
    lo = _log_int(rng, 1, hi)
    return _case(None, op, fmt, typ, seqs, (lo, hi), (0, rng.randint(0, 5000)), kv, 6, 0, 0, mix)


def _lengths(case):
    """Per sequence: the tokens before the call, and the tokens of the call."""
    rng = random.Random(case["mix"])
    lo, hi = case["ctx_lo"], case["ctx_hi"]
    ctx = [_log_int(rng, max(lo, 1), max(hi, 1)) if hi else 0 for _ in range(case["seqs"])]
    rows = [_log_int(rng, case["rows_lo"], case["rows_hi"]) for _ in range(case["seqs"])]
    return ctx, rows


def work(case):
    kf, vf = case["fmt"].split("/")
    ctx, rows = _lengths(case)
    total, size = sum(rows), 4 if case["type"] == "f32" else 2
    token = case["kv"] * NB * (BITS[kf] + BITS[vf])
    values = 2 * total * case["kv"] * DIM * size
    if case["op"] == "read":
        return {"bytes": total * token + values, "flops": 2 * total * case["kv"] * DIM}
    if case["op"] == "append":  # the tokens in, the pages written and read, the values out
        return {"bytes": 2 * values + 2 * total * token, "flops": 8 * total * case["kv"] * DIM}
    keys = pairs = 0
    for c, r in zip(ctx, rows):
        seen = min(c + r, case["window"] + r - 1) if case["window"] else c + r
        if case["pick"]:
            seen = min(seen, case["pick"] * PAGE)
        keys, pairs = keys + seen, pairs + seen * r
    heads = case["kv"] * case["group"]
    return {"bytes": keys * token + total * heads * (2 * DIM * size + 4), "flops": 4 * DIM * heads * pairs}


# ------------------------------------------------ the formats, in elementary operations
def _step(x):
    """One rounding to 32 bits of what was computed in 64."""
    return x.to(torch.float32).double()


def _encode(x, fmt):
    """fp32 [..., 256] -> codes [..., 8, 32] and scales and minima [..., 8] as fp16 (no minimum: 0). Every
    step that decides a code is rounded to 32 bits, from 64: the steps are what the format fixes."""
    x = x.reshape(*x.shape[:-1], NB, BLK).double()
    low = torch.zeros_like(x[..., 0])
    if fmt == "q8_0":
        d = _step(x.abs().amax(-1) / 127)
    elif fmt in HALF:
        big = x.abs().argmax(-1, keepdim=True)  # the first of equals
        d = _step(x.gather(-1, big)[..., 0] / -HALF[fmt])
    else:
        low = x.amin(-1)
        d = _step(_step(x.amax(-1) - low) / TOP[fmt])
    inv = torch.where(d == 0, 0.0, _step(1 / torch.where(d == 0, 1.0, d)))
    y = _step(_step(x - low[..., None]) * inv[..., None])
    if fmt == "q8_0":
        q = (y.sign() * (y.abs() + 0.5).floor()).clamp(-127, 127)
    elif fmt in HALF:
        q = _step(y + (HALF[fmt] + 0.5)).floor().clamp(max=2 * HALF[fmt] - 1)
    else:
        q = _step(y + 0.5).floor().clamp(max=TOP[fmt])
    return q.to(torch.int16), d.to(torch.float32).half(), low.to(torch.float32).half()


def _decode(q, d, m, fmt):
    """Codes [..., 8, 32] and scales -> fp32 values [..., 256]."""
    x = (q.float() - HALF.get(fmt, 0)) * d.float()[..., None]
    if fmt in TOP:
        x = x + m.float()[..., None]
    return x.flatten(-2)


def _pages(q, d, m, fmt, key):
    """Codes [n, 128, 8, 32] and scales [n, 128, 8] -> page bytes [n, bytes], in the documented order."""
    n = q.shape[0]
    if fmt == "q8_0":
        q = (q + 128).to(torch.uint8)
        if key:    # token (G, H, R), channel (P, j / 8, T, j % 8)
            codes = q.view(n, 8, 2, 8, 4, 2, 4, 8).permute(0, 1, 4, 2, 3, 6, 5, 7)
        else:      # token (G, w % 2, T, y % 2), channel (b, w / 2, y / 2, R)
            codes = q.view(n, 8, 2, 4, 2, 8, 2, 2, 8).permute(0, 1, 5, 8, 3, 6, 2, 7, 4)
        parts = [codes.reshape(n, -1)]
    else:
        nib = (q & 15).to(torch.uint8)
        if key:    # token (G, H, R), channel (Q, c, T, i): i = 2 u + v at bit 4 u + 16 v
            nib = nib.view(n, 8, 2, 8, 2, 4, 4, 2, 2, 2).permute(0, 1, 4, 2, 3, 6, 5, 9, 7, 8)
            codes = nib[..., 0] | (nib[..., 1] << 4)
        else:      # token (G, w % 2, T, y / 2), channel (C, w / 2, y % 2, nibble, R)
            nib = nib.view(n, 8, 2, 4, 2, 4, 2, 2, 2, 8).permute(0, 1, 5, 9, 3, 6, 2, 4, 7, 8)
            codes = nib[..., 0] | (nib[..., 1] << 4)
        parts = [codes.reshape(n, -1)]
        if fmt in ("q5_0", "q5_1"):  # bit 4 of channel (c, i = 2 u + v) at bit 16 v + 4 c + u
            top = (q >> 4).to(torch.int64).view(n, 8, 2, 8, 2, 4, 4, 4, 2).permute(0, 1, 4, 2, 3, 6, 8, 5, 7)
            word = (top.reshape(n, -1, 32) << torch.arange(32, device=q.device)).sum(-1)
            parts.append(torch.stack([(word >> s) & 255 for s in (0, 8, 16, 24)], -1).to(torch.uint8).reshape(n, -1))
    for s in (d, m) if fmt in TOP else (d,):
        if key:
            s = s.reshape(n, 8, 2, 8, 8).permute(0, 1, 3, 2, 4)
        else:
            s = s.reshape(n, 8, 2, 4, 2, 8).permute(0, 1, 3, 5, 2, 4)
        parts.append(s.reshape(n, -1).contiguous().view(torch.uint8))
    return torch.cat(parts, 1)


def _unpages(pages, fmt, key):
    """Page bytes [n, bytes] -> codes [n, 128, 8, 32], scales and minima [n, 128, 8]."""
    n, at = pages.shape[0], 128 * DIM // (1 if fmt == "q8_0" else 2)
    codes = pages[:, :at]
    if fmt == "q8_0":
        if key:
            q = codes.reshape(n, 8, 4, 2, 8, 4, 2, 8).permute(0, 1, 3, 4, 2, 6, 5, 7)
        else:
            q = codes.reshape(n, 8, 8, 8, 4, 2, 2, 2, 2).permute(0, 1, 6, 4, 8, 2, 5, 7, 3)
        q = q.reshape(n, PAGE, NB, BLK).to(torch.int16) - 128
    else:
        nib = torch.stack((codes & 15, codes >> 4), -1)
        if key:
            q = nib.view(n, 8, 2, 2, 8, 4, 4, 2, 2, 2).permute(0, 1, 3, 4, 2, 6, 5, 8, 9, 7)
        else:
            q = nib.view(n, 8, 4, 8, 4, 2, 2, 2, 2, 2).permute(0, 1, 6, 4, 7, 2, 5, 8, 9, 3)
        q = q.reshape(n, PAGE, NB, BLK).to(torch.int16)
        if fmt in ("q5_0", "q5_1"):
            b = pages[:, at:at + 4096].reshape(n, -1, 4, 1)
            top = ((b >> torch.arange(8, device=b.device, dtype=torch.uint8)) & 1).view(n, 8, 2, 2, 8, 4, 2, 4, 4)
            q = q | (top.permute(0, 1, 3, 4, 2, 7, 5, 8, 6).reshape(n, PAGE, NB, BLK).to(torch.int16) << 4)
            at += 4096
    scales = []
    for _ in range(2 if fmt in TOP else 1):
        s = pages[:, at:at + 2048].contiguous().view(torch.float16)
        if key:
            s = s.view(n, 8, 8, 2, 8).permute(0, 1, 3, 2, 4)
        else:
            s = s.view(n, 8, 4, 8, 2, 2).permute(0, 1, 4, 2, 5, 3)
        scales.append(s.reshape(n, PAGE, NB))
        at += 2048
    return q, scales[0], scales[1] if fmt in TOP else torch.zeros_like(scales[0])


# -------------------------------------------------------------------- inputs of a program
def _normal(shape, gen, loud):
    """N(0, 1) with one channel in a hundred eight times as large."""
    return torch.randn(shape, generator=gen, device="cuda") * loud


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed * 7919 + case["mix"])
    kf, vf = case["fmt"].split("/")
    H, Hq, typ = case["kv"], case["kv"] * case["group"], TYPES[case["type"]]
    ctx, rows = _lengths(case)
    S, total = case["seqs"], sum(rows)
    blocks = max((c + r + PAGE - 1) // PAGE for c, r in zip(ctx, rows))
    used = torch.tensor([(c + r + PAGE - 1) // PAGE for c, r in zip(ctx, rows)], device="cuda")
    here = (torch.arange(blocks, device="cuda") < used[:, None])[:, None].expand(S, H, blocks)
    n_pages = int(here.sum())
    table = torch.full((S, H, blocks), -1, dtype=torch.int32, device="cuda")
    table[here] = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    loud = 1 + 7 * (torch.rand(DIM, generator=gen, device="cuda") < 0.01)
    pools = []
    for fmt, key in ((kf, True), (vf, False)):
        pool = torch.zeros((n_pages, PAGE * NB * BITS[fmt]), dtype=torch.uint8, device="cuda")
        for at in range(0, n_pages if case["op"] != "append" else 0, 4096):
            n = min(4096, n_pages - at)
            pool[at:at + n] = _pages(*_encode(_normal((n, PAGE, DIM), gen, loud), fmt), fmt, key)
        pools.append(pool)
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    # the projection's output: queries, keys and values of a token side by side
    qkv = _normal((total, Hq + 2 * H, DIM), gen, loud if case["op"] == "append" else 1).to(typ)
    state = {"case": dict(case), "k_pool": pools[0], "v_pool": pools[1], "n_pages": n_pages, "table": table,
             "row_start": torch.tensor(start, dtype=torch.int32, device="cuda"),
             "pos_start": torch.tensor(ctx, dtype=torch.int32, device="cuda"),
             "total": total, "max_rows": max(rows), "logical": None, "listed": None}
    if case["op"] == "attend":
        state["q"] = qkv[:, :Hq]
        state["out"] = torch.zeros((total, Hq, DIM), dtype=typ, device="cuda")
        state["lse"] = torch.zeros((total, Hq), device="cuda")
    else:
        if case["op"] == "append":
            state["k"], state["v"] = qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        state["k_out"] = torch.zeros((total, H, DIM), dtype=typ, device="cuda")
        state["v_out"] = torch.zeros((total, H, DIM), dtype=typ, device="cuda")
    if case["pick"]:
        # every KV head has its own pages, in ascending order, the newest one among them
        mark = torch.rand((S, H, blocks), generator=gen, device="cuda").masked_fill(~here, -1)
        mark.scatter_(2, (used - 1)[:, None, None].expand(S, H, 1), 2.0)
        cap = min(case["pick"], blocks)
        got = mark.topk(cap, 2)
        state["listed"] = (got.values >= 0).sum(2).to(torch.int32)
        order = got.indices.masked_fill(got.values < 0, blocks).sort(2).values
        state["logical"] = order.to(torch.int32)
        state["table"] = table.gather(2, order.clamp(max=blocks - 1)).masked_fill(order == blocks, -1).contiguous()
    return state


# ------------------------------------------------------------------------ the plain forms
def _places(state):
    """Of every row of the call: its sequence, its position, and its pages' numbers by KV head."""
    start, rows = state["row_start"].long(), torch.arange(state["total"], device="cuda")
    seq = torch.searchsorted(start[1:].contiguous(), rows, right=True)
    pos = state["pos_start"].long()[seq] + rows - start[seq]
    return seq, pos, state["table"].long()[seq, :, pos // PAGE]


def _values(state, fmt, key, pages):
    """fp32 values [..., 128, 256] of the pages listed."""
    pool = state["k_pool" if key else "v_pool"]
    x = _decode(*_unpages(pool[pages.reshape(-1)], fmt, key), fmt)
    return x.view(*pages.shape, PAGE, DIM)


def _plain_read(state):
    kf, vf = state["case"]["fmt"].split("/")
    seq, pos, pages = _places(state)
    used, where = torch.unique(pages, return_inverse=True)
    slot = (pos % PAGE)[:, None].expand_as(pages)
    for name, fmt, key in (("k_out", kf, True), ("v_out", vf, False)):
        state[name].copy_(_values(state, fmt, key, used)[where, slot])
    return {"k": state["k_out"], "v": state["v_out"]}


def _plain_append(state):
    kf, vf = state["case"]["fmt"].split("/")
    seq, pos, pages = _places(state)
    used, where = torch.unique(pages, return_inverse=True)
    slot = (pos % PAGE)[:, None].expand_as(pages)
    for name, fmt, key in (("k", kf, True), ("v", vf, False)):
        pool = state[name + "_pool"]
        held = _unpages(pool[used], fmt, key)
        for old, new in zip(held, _encode(state[name].float(), fmt)):
            old[where, slot] = new
        pool[used] = _pages(*held, fmt, key)
    return _plain_read(state)


def _plain_attend(state):
    case = state["case"]
    kf, vf = case["fmt"].split("/")
    S, H, g, R, window = case["seqs"], case["kv"], case["group"], state["max_rows"], case["window"]
    start, first = state["row_start"].long(), state["pos_start"].long()
    count = start[1:] - start[:-1]
    r = torch.arange(R, device="cuda")
    row = (start[:-1, None] + r).clamp(max=state["total"] - 1)                    # [S, R]
    pos = first[:, None] + r
    table = state["table"].long()
    if case["pick"]:
        logical = state["logical"].long()                                        # [S, H, n]
        there = torch.arange(logical.shape[2], device="cuda") < state["listed"][..., None]
    else:
        n = table.shape[2]
        low = torch.zeros_like(first)
        if window:  # only the pages that the window reaches
            low = (first - (window - 1)).clamp(min=0) // PAGE
            n = min(n, (window + R - 2) // PAGE + 2)
        logical = (low[:, None] + torch.arange(n, device="cuda"))[:, None].expand(S, H, n)
        there = logical * PAGE < (first + count)[:, None, None]
        table = table.gather(2, logical.clamp(max=table.shape[2] - 1))
    pages = table.clamp(min=0)
    keys = _values(state, kf, True, pages).flatten(2, 3)                          # [S, H, n * 128, 256]
    q = state["q"].float()[row].view(S, R, H, g, DIM).permute(0, 2, 1, 3, 4).reshape(S, H, R * g, DIM)
    s = (q @ keys.transpose(2, 3) / 16).view(S, H, R, g, -1)
    del keys
    at = (logical[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(2)   # [S, H, n * 128]
    seen = there.repeat_interleave(PAGE, 2)[:, :, None] & (at[:, :, None] <= pos[:, None, :, None])
    if window:
        seen = seen & (at[:, :, None] > pos[:, None, :, None] - window)
    s = s.masked_fill(~seen[:, :, :, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    values = _values(state, vf, False, pages).flatten(2, 3)
    values = values.masked_fill(~seen.any(2)[..., None], 0)
    o = (p.view(S, H, R * g, -1) @ values).view(S, H, R, g, DIM) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    live = r < count[:, None]
    state["out"][row[live]] = o.permute(0, 2, 1, 3, 4)[live].flatten(1, 2).to(state["out"].dtype)
    state["lse"][row[live]] = lse.permute(0, 2, 1, 3)[live].flatten(1, 2)
    return {"out": state["out"], "lse": state["lse"]}


# ------------------------------------------------------------------------ the framework's
def _own(state):
    """The calls of a program that keeps its descriptors and its workspace from step to step."""
    from quantized_paged_kv_q4_b200 import kvattn as kv

    case = state["case"]
    if "desc" not in state:
        kv.kvattn_init(torch.cuda.current_device())
        kf, vf = case["fmt"].split("/")
        state["desc"] = kv.make_desc(case["kv"], case["kv"] * case["group"], state["k_pool"], state["v_pool"],
                                     state["n_pages"], k_fmt=kf, v_fmt=vf)
        state["batch"] = kv.make_batch(state["row_start"], state["pos_start"], state["table"], state["total"],
                                       state["max_rows"])
        if case["op"] == "attend":
            size = kv.kvattn_decode_batch_workspace_size(state["desc"], state["batch"])
            state["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    desc, batch = state["desc"], state["batch"]
    if case["op"] == "attend":
        kv.kvattn_decode_batch(desc, batch, state["q"], state["out"], state["lse"], state["ws"],
                               page_logical=state["logical"], n_pages=state["listed"], window=case["window"])
        return {"out": state["out"], "lse": state["lse"]}
    if case["op"] == "append":
        kv.kvattn_append_batch(desc, batch, state["k"], state["v"])
    kv.kvattn_read_batch(desc, batch, state["k_out"], state["v_out"])
    return {"k": state["k_out"], "v": state["v_out"]}


def run(state):
    if own:
        return _own(state)
    return {"read": _plain_read, "append": _plain_append, "attend": _plain_attend}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definition in 64 bits
def _byte_of(fmt, key, tok, c):
    """Where the code of token `tok` and channel `c` sits in its page (byte, shift), by the documented formulas,
    and where its fifth bit, its scale and its minimum do."""
    G, b = tok // 16, c // 32
    if key:
        H, R, T = tok % 16 // 8, tok % 8, c % 32 // 8
        scale = ((G * 8 + R) * 2 + H) * 8 + b
        Q, i = b // 4, c % 8
        line = (((G * 2 + Q) * 2 + H) * 8 + R) * 4 + T
        if fmt == "q8_0":
            return ((((G * 4 + c // 64) * 2 + H) * 8 + R) * 4 + T) * 16 + c % 64 // 32 * 8 + i, None, None, 32768 + 2 * scale, None
        bit = 4 * (i // 2) + 16 * (i % 2)
        fifth = 16 * (i % 2) + 4 * (b % 4) + i // 2
        at = {"q4_0": (16384, 0), "q5_0": (20480, 0), "q5_1": (20480, 22528)}[fmt]
        return (4 * (line * 4 + b % 4) + bit // 8, bit % 8, (16384 + 4 * line + fifth // 8, fifth % 8) if at[0] > 16384 else None,
                at[0] + 2 * scale, at[1] + 2 * scale if at[1] else None)
    T, hi, odd = tok % 8 // 2, tok % 16 // 8, tok % 2
    scale = ((G * 4 + T) * 8 + b) * 4 + odd + 2 * hi
    x = c % 32
    if fmt == "q8_0":
        return (((G * 8 + b) * 8 + x % 8) * 4 + T) * 16 + 4 * (2 * (x // 16) + hi) + 2 * (x // 8 % 2) + odd, None, None, 32768 + 2 * scale, None
    byte = (((G * 4 + b // 2) * 8 + x % 8) * 4 + T) * 16 + 4 * (2 * (b % 2) + hi) + 2 * odd + x // 16
    return byte, x // 8 % 2 * 4, None, 16384 + 2 * scale, 18432 + 2 * scale if fmt == "q4_1" else None


def _held(pool, pages, slots, fmt, key):
    """float64 values [n, 256] of slot slots[i] of page pages[i]."""
    c = torch.arange(DIM, device="cuda")
    code, shift, fifth, scale, low = _byte_of(fmt, key, slots[:, None], c[None])
    page = pages[:, None]
    half = lambda at: pool.view(torch.float16)[page, at // 2].double()  # noqa: E731
    q = pool[page, code].long()
    if fmt == "q8_0":
        return (q - 128).double() * half(scale)
    q = (q >> shift) & 15
    if fifth is not None:
        q = q + 16 * ((pool[page, fifth[0]].long() >> fifth[1]) & 1)
    x = (q - {"q4_0": 8, "q5_0": 16}.get(fmt, 0)).double() * half(scale)
    return x if low is None else x + half(low)


def _quantized(x, fmt):
    """float64 values that the format holds for fp32 rows [n, 256], block by block from its rules: codes by fp32 steps."""
    f = lambda y: y.float().double()  # noqa: E731
    b = x.double().view(-1, BLK)
    if fmt in ("q4_1", "q5_1"):
        n = 15.0 if fmt == "q4_1" else 31.0
        lo, hi = b.min(1, True).values, b.max(1, True).values
        d = f(f(hi - lo) / n)
        r = torch.where(d > 0, f(d.reciprocal()), 0.0)
        q = torch.minimum(f(f(f(b - lo) * r) + 0.5).floor(), torch.full_like(d, n))
        return (q * d.float().half().double() + lo.float().half().double()).view(-1, DIM)
    if fmt == "q8_0":
        d = f(b.abs().max(1, True).values / 127.0)
        r = torch.where(d > 0, f(d.reciprocal()), 0.0)
        y = f(b * r)
        q = torch.where(y < 0, -(0.5 - y).floor(), (0.5 + y).floor()).clamp(-127, 127)
        return (q * d.float().half().double()).view(-1, DIM)
    h = 8.0 if fmt == "q4_0" else 16.0
    size, where = b.abs(), torch.arange(BLK, device=b.device)
    first = torch.where(size == size.max(1, True).values, where, BLK).min(1, True).values
    d = f(b.gather(1, first) / -h)
    r = torch.where(d != 0, f(d.reciprocal()), 0.0)
    q = torch.minimum(f(f(b * r) + (h + 0.5)).floor(), torch.full_like(d, 2 * h - 1))
    return ((q - h) * d.float().half().double()).view(-1, DIM)


def exact(case, seed):
    s = prepare(case, seed)
    kf, vf = case["fmt"].split("/")
    H, g = case["kv"], case["group"]
    ctx, rows = _lengths(case)
    if case["op"] == "append":
        return {"k": _quantized(s["k"].reshape(-1, DIM), kf).view(-1, H, DIM),
                "v": _quantized(s["v"].reshape(-1, DIM), vf).view(-1, H, DIM)}
    table = s["table"].long()
    if case["op"] == "read":
        answer = {}
        for name, fmt, key in (("k", kf, True), ("v", vf, False)):
            got = []
            for i, (c, r) in enumerate(zip(ctx, rows)):
                pos = torch.arange(c, c + r, device="cuda")
                one = [torch.cat([_held(s[name + "_pool"], table[i, h, p // PAGE], p % PAGE, fmt, key) for p in pos.split(8192)])
                       for h in range(H)]
                got.append(torch.stack(one, 1))
            answer[name] = torch.cat(got)
        return answer
    out = torch.zeros((s["total"], H * g, DIM), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total"], H * g), dtype=torch.float64, device="cuda")
    at = 0
    for i, (c, r) in enumerate(zip(ctx, rows)):
        for h in range(H):
            if case["pick"]:
                n = int(s["listed"][i, h])
                pages, first = table[i, h, :n], s["logical"][i, h, :n].long() * PAGE
                pos = (first[:, None] + torch.arange(PAGE, device="cuda")).flatten()
                page = pages.repeat_interleave(PAGE)
                page, pos = page[pos < c + r], pos[pos < c + r]
            else:
                pos = torch.arange(max(0, c + 1 - case["window"]) if case["window"] else 0, c + r, device="cuda")
                page = table[i, h, pos // PAGE]
            k = torch.cat([_held(s["k_pool"], a, b % PAGE, kf, True) for a, b in zip(page.split(8192), pos.split(8192))])
            v = torch.cat([_held(s["v_pool"], a, b % PAGE, vf, False) for a, b in zip(page.split(8192), pos.split(8192))])
            for j in range(r):
                ok = pos <= c + j
                if case["window"]:
                    ok &= pos > c + j - case["window"]
                x = s["q"][at + j, h * g:(h + 1) * g].double() @ k[ok].T / 16
                lse[at + j, h * g:(h + 1) * g] = x.logsumexp(1)
                out[at + j, h * g:(h + 1) * g] = x.softmax(1) @ v[ok]
        at += r
    return {"out": out, "lse": lse}
