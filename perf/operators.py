"""What is measured of the KV cache kept in 8 bits in the page pool.

Three operators, named by a case's ``op``:

* ``append``: q and k of the new tokens are rotated by their positions, k and v are stored as 8-bit codes in the
  sequences' blocks (one range for each block of tokens and kv head, old codes re-coded where the range grows), and
  the blocks that were touched are read back as values: ``run`` returns the rotated q and those values;
* ``attend``: attention of a step's rows (one token a sequence, whole prompts, or both) over the cached blocks;
* ``read``: the cached values of whole sequences, as they are when a sequence moves to another cache or to the host.

A case's sequences: ``seqs`` of ``ctx_lo..ctx_hi`` cached tokens with ``rows_lo..rows_hi`` new ones, and ``more``
further ones of ``more_lo..more_hi`` cached tokens with one new token each.  The lengths follow from ``lengths``
alone, the data from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
DTYPES = {"f16": torch.float16, "f32": torch.float32}


def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="f16", code="int8", heads=32, kv_heads=32, dim=128, page=8192, rot=128,
             pairs="halves", seqs=0, ctx_lo=0, ctx_hi=0, rows_lo=1, rows_hi=1, more=0, more_lo=0, more_hi=0,
             window=0, lengths=1)
    assert set(kw) <= set(c)
    return {**c, **kw}


def listed():
    gqa = dict(heads=64, kv_heads=8, page=16384)       # 8192 wide: 64 query heads on 8 kv heads
    return [
        # one user's next token: what a launch costs
        _case("append_one", "append", seqs=1, ctx_lo=700, ctx_hi=700, **gqa),
        # a decode batch of 256 requests at the 4096-wide shape; blocks partly filled, ranges that grow
        _case("append_decode", "append", seqs=256, ctx_lo=1, ctx_hi=900),
        # 32 prompts of 64 to 512 tokens, e4m3 codes
        _case("append_prefill", "append", code="fp8", seqs=32, rows_lo=64, rows_hi=512),
        # a long prompt arriving in one piece, on a context that ends inside a block; rotation of half the head
        _case("append_long", "append", seqs=1, ctx_lo=1001, ctx_hi=1001, rows_lo=16384, rows_hi=16384, rot=64,
              pairs="neighbours", **gqa),
        # one user's next token over a short context: latency
        _case("attend_one", "attend", seqs=1, ctx_lo=777, ctx_hi=777, **gqa),
        # fp32, heads of 64: the parity type
        _case("attend_f32", "attend", dtype="f32", heads=16, kv_heads=16, dim=64, rot=64, page=4096, seqs=16,
              ctx_lo=1, ctx_hi=700),
        # the decode batch of 256 requests, each at its own length
        _case("attend_decode", "attend", seqs=256, ctx_lo=300, ctx_hi=2000),
        # few long conversations: the split over the tokens carries it; e4m3 codes
        _case("attend_long", "attend", code="fp8", seqs=12, ctx_lo=12000, ctx_hi=33000, **gqa),
        # 32 fresh prompts of 64 to 512 tokens
        _case("attend_prefill", "attend", seqs=32, rows_lo=64, rows_hi=512),
        # the next piece of a long prompt
        _case("attend_chunk", "attend", seqs=1, ctx_lo=6001, ctx_hi=6001, rows_lo=2048, rows_hi=2048, **gqa),
        # prompts of 256 tokens beside 384 decode requests at the 5120-wide shape, with a sliding window; e4m3 codes
        _case("attend_mixed", "attend", code="fp8", heads=40, kv_heads=40, page=10240, seqs=8, rows_lo=256,
              rows_hi=256, more=384, more_lo=100, more_hi=1000, window=512),
        # sequences leaving for the host
        _case("read_whole", "read", seqs=8, ctx_lo=500, ctx_hi=4000, **gqa),
    ]


def _lengths(case):
    """(cached, new) tokens of each sequence."""
    rng = random.Random(case["lengths"])
    some = [(rng.randint(case["ctx_lo"], case["ctx_hi"]), rng.randint(case["rows_lo"], case["rows_hi"]))
            for _ in range(case["seqs"])]
    return some + [(rng.randint(case["more_lo"], case["more_hi"]), 1) for _ in range(case["more"])]


def _block(case):
    """Tokens of a block: what a page holds of one head's keys and values, in whole groups of 32."""
    return case["page"] // (2 * case["dim"]) // 32 * 32


def _seen(c, r, window):
    """(query, key) pairs of r rows after c cached tokens."""
    short = min(r, max(0, window - c)) if window else r      # rows that see every token before them
    return short * c + short * (short + 1) // 2 + (r - short) * window


def _keys(c, r, window):
    """Cached tokens that some row of the sequence sees."""
    return c + r if not window else c + r - max(0, c + 1 - window)


def work(case):
    e = 2 if case["dtype"] == "f16" else 4
    h, hk, d, bt = case["heads"], case["kv_heads"], case["dim"], _block(case)
    lens = _lengths(case)
    rows = sum(r for _, r in lens)
    if case["op"] == "attend":
        keys = sum(_keys(c, r, case["window"]) for c, r in lens)
        return {"bytes": 2 * rows * h * d * e + keys * hk * d * 2 + keys * hk * 12 // bt,
                "flops": 4 * d * h * sum(_seen(c, r, case["window"]) for c, r in lens)}
    if case["op"] == "read":
        n = sum(c + r for c, r in lens)
        return {"bytes": n * hk * d * 2 * (1 + e), "flops": 2 * n * hk * d}
    touched = sum(c % bt + r for c, r in lens)
    # q in and out, k and v in, their codes out; the touched blocks' codes in and their values out
    return {"bytes": 2 * rows * h * d * e + 2 * rows * hk * d * (e + 1) + 2 * touched * hk * d * (1 + e),
            "flops": rows * (h + 2 * hk) * d * 6 + 2 * touched * hk * d}


def _cost(case):
    w = work(case)
    return w["bytes"] / 4e12 + w["flops"] / (4e14 if case["dtype"] == "f16" else 4e13)


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    limit = max(_cost(c) for c in listed())
    while True:
        dim, rot = rng.choice([(64, 64), (128, 128), (128, 128), (128, 64), (256, 256), (256, 32), (64, 0)])
        kv_heads = rng.choice([1, 2, 3, 4, 8, 16, 32, 40])
        heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16])
        tokens = rng.choice([32, 32, 64, 96, 128])
        c = _case("", rng.choice(["append", "attend", "attend", "attend", "read"]), heads=heads, kv_heads=kv_heads,
                  dtype=rng.choice(["f16", "f16", "f16", "f32"]), code=rng.choice(["int8", "fp8"]), dim=dim, rot=rot,
                  pairs=rng.choice(["halves", "neighbours"]), page=2 * dim * tokens + rng.choice([0, 0, 64, 1024]),
                  lengths=rng.randrange(1 << 30))
        del c["name"]
        kind = rng.choice(["decode", "decode", "prompts", "chunk", "mixed"])
        ctx = log(1, 33000) if kind != "prompts" else 0
        c.update(ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, seqs=log(1, 256 if kind == "decode" else 32))
        if kind != "decode":
            hi = log(2, 4000)
            c.update(rows_lo=rng.randint(1, hi), rows_hi=hi)
        if kind == "mixed":
            hi = log(1, 2000)
            c.update(more=log(1, 256), more_lo=rng.randint(0, hi), more_hi=hi)
        if rng.random() < 0.25:
            c["window"] = log(1, 4000)
        if heads <= 128 and c["page"] <= 32768 and _cost(c) <= limit and _padded(c) <= 2e9:
            return c


def _padded(case):
    """Scores of the plain form, which pads the sequences of a group to the longest."""
    lens = _lengths(case)
    parts = [[x for x in lens if x[1] > 1], [x for x in lens if x[1] <= 1]]
    cells = [len(p) * max(r for _, r in p) * max(c + r for c, r in p) * case["heads"] for p in parts if p]
    cache = [len(p) * max(c + r for c, r in p) * case["kv_heads"] * case["dim"] for p in parts if p]
    return max(cells + cache)


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _tables(case, n_pos):
    """cos and sin of every position's angles, from 64 bits, as fp32 [n_pos, rot]: the cosines, then the sines."""
    half = case["rot"] // 2
    if not half:
        return None
    inv = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    ang = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _qkv(case, g, n):
    """One fused projection's output for n tokens: rows of heads + 2 kv_heads heads.  Some channels of k are several
    times larger than others, as in trained models."""
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    x = torch.randn((n, h + 2 * hk, d), generator=g, device=DEV, dtype=torch.float32)
    x[:, h:h + hk] *= torch.exp(0.6 * torch.randn((hk, d), generator=g, device=DEV))
    return x.to(DTYPES[case["dtype"]])


def _inputs(case, seed):
    """(k and v of the cached tokens [sum ctx, 2 kv_heads, dim], q, k, v of the new ones [rows, heads + 2 kv_heads, dim])"""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    lens = _lengths(case)
    h = case["heads"]
    past = _qkv({**case, "heads": 0}, g, max(1, sum(c for c, _ in lens)))
    return past, _qkv(case, g, max(1, sum(r for _, r in lens))), h


def _long(x):
    return torch.tensor(x, device=DEV, dtype=torch.long)


def _touched(case, starts, counts, tables):
    """Index tensors of an append of counts[i] tokens at position starts[i] of sequence i: for every block touched, its
    pages, the new token of each slot, which slots are new, which hold older tokens, and whether the block is begun."""
    bt = _block(case)
    blocks, seq, tok0 = [], [], []
    at = 0
    for i, (s, n) in enumerate(zip(starts, counts)):
        for b in range(s // bt, -(-(s + n) // bt) if n else s // bt):
            blocks.append(b), seq.append(i), tok0.append(at + b * bt - s)
        at += n
    start, count = _long(starts), _long(counts)
    blocks, seq, tok0 = _long(blocks), _long(seq), _long(tok0)
    slot = torch.arange(bt, device=DEV)
    pos = blocks[:, None] * bt + slot
    new = (pos >= start[seq][:, None]) & (pos < (start + count)[seq][:, None])
    tok = torch.where(new, tok0[:, None] + slot, 0)
    return {"pages": tables[seq, blocks], "tok": tok, "new": new, "old": pos < start[seq][:, None],
            "begun": blocks * bt < start[seq], "pos": torch.cat([_long(range(s, s + n)) for s, n in zip(starts, counts)])}


def _rows_of(case, starts, counts, tables):
    """Pages [rows, kv_heads] and slot [rows] of the tokens starts[i] .. starts[i] + counts[i] of each sequence."""
    bt = _block(case)
    pos = torch.cat([_long(range(s, s + n)) for s, n in zip(starts, counts)])
    seq = torch.repeat_interleave(torch.arange(len(counts), device=DEV), _long(counts))
    return {"pages": tables[seq, pos // bt], "slot": (pos % bt)[:, None]}


def _group(case, lens, which, tables):
    """Padded index tensors of the sequences `which`: a step's rows, their positions and their blocks."""
    bt = _block(case)
    first = [sum(r for _, r in lens[:i]) for i in range(len(lens))]
    most = max(lens[i][1] for i in which)
    blocks = max(-(-(lens[i][0] + lens[i][1]) // bt) for i in which)
    row = torch.arange(most, device=DEV)
    r, c, f = _long([lens[i][1] for i in which]), _long([lens[i][0] for i in which]), _long([first[i] for i in which])
    valid = row < r[:, None]
    return {"rows": torch.where(valid, f[:, None] + row, 0), "pos": c[:, None] + row, "pages": tables[_long(which), :blocks],
            "from": torch.nonzero(valid.reshape(-1))[:, 0],
            "to": (f[:, None] + row).reshape(-1)[torch.nonzero(valid.reshape(-1))[:, 0]]}


def prepare(case, seed):
    past, new, h = _inputs(case, seed)
    hk, d, bt = case["kv_heads"], case["dim"], _block(case)
    lens = _lengths(case)
    ctx, rows = [c for c, _ in lens], [r for _, r in lens]
    cos_sin = _tables(case, max(c + r for c, r in lens))
    st = {"case": case, "q": new[:, :h], "k": new[:, h:h + hk], "v": new[:, h + hk:], "cos_sin": cos_sin,
          "scale": 1.0 / math.sqrt(d)}
    blocks = [-(-(c + r) // bt) for c, r in lens]
    pages = sum(blocks) * hk
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 5))
    # what is read back: the touched blocks after an append, everything for a read
    back = [0 if case["op"] == "read" else c // bt * bt for c in ctx]
    if own:
        return _prepare_own(st, past, order, ctx, rows, back)
    tables = torch.zeros((len(lens), max(blocks), hk), dtype=torch.long)
    at = 0
    for i, b in enumerate(blocks):
        tables[i, :b] = order[at:at + b * hk].reshape(b, hk)
        at += b * hk
    tables = tables.to(DEV)
    st["codes"] = torch.zeros((pages, 2, bt, d), dtype=torch.uint8, device=DEV)
    st["range"] = torch.zeros((pages, 2), dtype=torch.float32, device=DEV)
    # the cached tokens, some sequences at a time
    at, i = 0, 0
    while i < len(lens):
        j, n = i, 0
        while j < len(lens) and (j == i or n + ctx[j] <= 65536):
            n, j = n + ctx[j], j + 1
        if n:
            part = _touched(case, [0] * (j - i), ctx[i:j], tables[i:j])
            _append(st, past[at:at + n, :hk], past[at:at + n, hk:], part)
        at, i = at + n, j
    st["part"] = _touched(case, ctx, rows, tables)
    if case["op"] != "append":
        _append(st, st["k"], st["v"], st["part"])
    st["q"] = _rotated(st, st["q"], st["part"]["pos"]).to(new.dtype) if case["op"] == "attend" else st["q"]
    st["read"] = _rows_of(case, back, [c + r - b for (c, r), b in zip(lens, back)], tables)
    parts = [[i for i, r in enumerate(rows) if r > 1], [i for i, r in enumerate(rows) if r <= 1]]
    st["groups"] = [_group(case, lens, p, tables) for p in parts if p]
    return st


def _prepare_own(st, past, order, ctx, rows, back):
    """The pool, the cache and the steps that a server keeps: the cached tokens arrive in a step of their own."""
    from rank_gemm_page_amd import slora as S
    case = st["case"]
    h, hk, d, dt = case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    stream = torch.cuda.current_stream()
    elems = case["page"] // dt.itemsize
    n_pages = order.numel()
    mem = torch.empty((n_pages, elems), dtype=dt, device=DEV)
    pool = S.slora_pool_create(S.SLORA_F16 if dt == torch.float16 else S.SLORA_F32, elems, elems, 1, 1, 1, [mem],
                               [n_pages], [order.numpy()])
    desc = dict(cls=0, code=S.SLORA_KV_INT8 if case["code"] == "int8" else S.SLORA_KV_FP8, n_layers=1, n_heads=h,
                n_kv_heads=hk, head_dim=d, block_tokens=_block(case), max_seqs=len(ctx),
                max_tokens=max(c + r for c, r in zip(ctx, rows)), rot_dim=case["rot"],
                rot_pairs=S.SLORA_KV_HALVES if case["pairs"] == "halves" else S.SLORA_KV_NEIGHBOURS)
    dev = torch.empty(S.slora_kv_device_bytes(pool, **desc), dtype=torch.uint8, device=DEV)
    kv = S.slora_kv_create(pool, dev, dev.numel(), **desc)
    st.update(S=S, pool=pool, kv=kv, keep=_Handles(S, pool, kv, [mem, dev]))

    def step(counts, reread=False):
        s = S.slora_kv_build_step(kv, list(range(len(counts))), counts, reread)
        st["keep"].steps.append(s)
        info = S.slora_kv_step_get_info(s)
        meta = torch.empty(max(16, info["meta_bytes"]), dtype=torch.uint8, device=DEV)
        st["keep"].memory.append(meta)
        S.slora_kv_step_upload(s, meta, meta.numel(), stream)
        return s, info

    if sum(ctx):
        s, _ = step(ctx)
        S.slora_kv_append(kv, s, 0, past[:, :hk], past[:, hk:], cos_sin=st["cos_sin"], stream=stream)
    st["step"], info = step(rows)
    if case["op"] != "append":
        q = torch.empty_like(st["q"], memory_format=torch.contiguous_format)
        S.slora_kv_append(kv, st["step"], 0, st["k"], st["v"], st["q"], q, cos_sin=st["cos_sin"], stream=stream)
        st["q"] = q
    counts = [c + r - b for c, r, b in zip(ctx, rows, back)]
    if case["op"] != "attend":
        st["reread"], _ = step(counts, True)
        st["k_out"] = torch.empty((sum(counts), hk, d), dtype=dt, device=DEV)
        st["v_out"] = torch.empty_like(st["k_out"])
    st["out"] = torch.empty((st["q"].shape[0], h, d), dtype=dt, device=DEV)
    st["workspace"] = torch.empty(max(16, info["workspace_bytes"]), dtype=torch.uint8, device=DEV)
    return st


class _Handles:
    """The handles of one state, released with it."""

    def __init__(self, S, pool, kv, memory):
        self.S, self.pool, self.kv, self.memory, self.steps = S, pool, kv, memory, []

    def __del__(self):
        torch.cuda.synchronize()
        for s in self.steps:
            self.S.slora_kv_step_destroy(s)
        self.S.slora_kv_destroy(self.kv)
        self.S.slora_pool_destroy(self.pool)


# ---- the plain forms ---------------------------------------------------------------------------------------------------

def _rotated(st, x, pos):
    """x [rows, heads, dim] rotated by the rows' positions, in 64 bits."""
    rot = st["case"]["rot"]
    x = x.double()
    if not rot:
        return x
    cs = st["cos_sin"][pos].double()[:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    y = x.clone()
    if st["case"]["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def _limit(st):
    return 127.0 if st["case"]["code"] == "int8" else 448.0


def _rounded(st, x):
    """The codes (as bytes) of scaled values x (64 bits): the nearest, ties to even."""
    if st["case"]["code"] == "int8":
        return x.round().to(torch.int8).view(torch.uint8)
    return x.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _worth(st, codes):
    """What code bytes stand for, before the block's scale, in fp32."""
    return codes.view(torch.int8 if st["case"]["code"] == "int8" else torch.float8_e4m3fn).float()


def _store(st, which, x, part):
    """x [rows, kv_heads, dim] (64 bits) into the touched blocks, as keys (which = 0) or values (1)."""
    pages, new, old = part["pages"], part["new"][:, None, :, None], part["old"][:, None, :, None]
    limit = torch.tensor(_limit(st), dtype=torch.float64, device=x.device)
    x = torch.where(new, x[part["tok"]].permute(0, 2, 1, 3), 0.0)
    held = torch.where(part["begun"][:, None], st["range"][pages, which], 0.0)
    grown = torch.maximum(held, x.abs().amax((2, 3)).float())
    inv = torch.where(grown > 0, limit / grown.double(), 0.0)[..., None, None]
    codes = st["codes"][pages, which]
    ratio = torch.where(grown > 0, held.double() / grown.double(), 0.0)[..., None, None]
    codes = torch.where(old, _rounded(st, _worth(st, codes).nan_to_num().double() * ratio), codes)
    st["codes"][pages, which] = torch.where(new, _rounded(st, x * inv), codes)
    st["range"][pages, which] = grown


def _append(st, k, v, part):
    _store(st, 0, _rotated(st, k, part["pos"]), part)
    _store(st, 1, v.double(), part)


def _read(st, which, at):
    step = (st["range"][:, which] / _limit(st))[at["pages"]][..., None]
    return _worth(st, st["codes"][at["pages"], which, at["slot"]]) * step


def _cached(st, which, pages):
    """Keys or values of padded sequences, [seqs, kv_heads, tokens, dim] in fp32."""
    step = (st["range"][:, which] / _limit(st))[pages][..., None, None]
    x = (_worth(st, st["codes"][pages, which]).nan_to_num() * step.nan_to_num()).permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _attend(st, group):
    case = st["case"]
    hk, d, g = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    n, r = group["rows"].shape
    q = st["q"].float()[group["rows"]].reshape(n, r, hk, g, d).permute(0, 2, 1, 3, 4).reshape(n, hk, r * g, d)
    s = torch.matmul(q, _cached(st, 0, group["pages"]).transpose(2, 3)) * st["scale"]
    key, pos = torch.arange(s.shape[-1], device=s.device), group["pos"][:, :, None]
    hidden = (key > pos) | (key <= pos - case["window"]) if case["window"] else key > pos
    s = s.view(n, hk, r, g, -1).masked_fill_(hidden[:, None, :, None], float("-inf")).view(n, hk, r * g, -1)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p, _cached(st, 1, group["pages"])) / p.sum(-1, keepdim=True)
    return o.view(n, hk, r, g, d).permute(0, 2, 1, 3, 4).reshape(n * r, hk * g, d)[group["from"]]


def run(st):
    op = st["case"]["op"]
    if own:
        S, kv = st["S"], st["kv"]
        stream = torch.cuda.current_stream()
        if op == "attend":
            S.slora_kv_attend(kv, st["step"], 0, st["q"], st["out"], st["scale"], st["case"]["window"], st["workspace"],
                              st["workspace"].numel(), stream)
            return st["out"]
        if op == "append":
            S.slora_kv_append(kv, st["step"], 0, st["k"], st["v"], st["q"], st["out"], cos_sin=st["cos_sin"], stream=stream)
        S.slora_kv_read(kv, st["reread"], 0, st["k_out"], st["v_out"], stream)
        values = {"k": st["k_out"], "v": st["v_out"]}
        return values if op == "read" else {"q": st["out"], **values}
    dt = st["k"].dtype
    if op == "attend":
        o = torch.cat([_attend(st, g) for g in st["groups"]])
        return torch.empty_like(o, dtype=dt).index_copy_(0, torch.cat([g["to"] for g in st["groups"]]), o.to(dt))
    if op == "append":
        _append(st, st["k"], st["v"], st["part"])
    values = {"k": _read(st, 0, st["read"]).to(dt), "v": _read(st, 1, st["read"]).to(dt)}
    return values if op == "read" else {"q": _rotated(st, st["q"], st["part"]["pos"]).to(dt), **values}


# ---- 64 bits, from the definitions -------------------------------------------------------------------------------------

def _turned(case, cos_sin, x, first):
    """One sequence's x [tokens, heads, dim] at positions first, first + 1, ...: each pair times its rotation, as a
    product of complex numbers."""
    half, x = case["rot"] // 2, x.double()
    if not half:
        return x
    cs = cos_sin[first:first + x.shape[0], None].double()
    turn = torch.complex(cs[..., :half], cs[..., half:])
    head, tail = x[..., :2 * half], x[..., 2 * half:]
    z = head.unflatten(-1, (2, half)).transpose(-1, -2) if case["pairs"] == "halves" else head.unflatten(-1, (half, 2))
    z = torch.view_as_real(torch.complex(z[..., 0], z[..., 1]) * turn)
    z = z.transpose(-1, -2) if case["pairs"] == "halves" else z
    return torch.cat([z.flatten(-2), tail], -1)


def _codes_of(case, x):
    return x.round() if case["code"] == "int8" else x.float().to(torch.float8_e4m3fn).double()


def _held(case, past, new):
    """What one sequence's cache holds of x after `past` [tokens, kv_heads, dim] and then `new` were appended."""
    top, bt = 127.0 if case["code"] == "int8" else 448.0, _block(case)
    both = torch.cat([past, new])
    pad = -both.shape[0] % bt
    blocks = torch.nn.functional.pad(both, (0, 0, 0, 0, 0, pad)).unflatten(0, (-1, bt))     # [blocks, bt, heads, dim]
    late = (torch.arange(blocks.shape[0] * bt, device=DEV) >= past.shape[0]).view(-1, bt, 1, 1)
    peak = lambda y: y.abs().amax((1, 3), keepdim=True).float().double()  # noqa: E731
    before, after = peak(blocks.masked_fill(late, 0.0)), peak(blocks)
    safe = lambda y: torch.where(y > 0, y, 1.0)  # noqa: E731
    early = _codes_of(case, blocks * (top / safe(before)))
    early = torch.where(before < after, _codes_of(case, early * (before / safe(after))), early)
    codes = torch.where(late, _codes_of(case, blocks * (top / safe(after))), early)
    return (codes * after / top).flatten(0, 1)[:both.shape[0]]


def exact(case, seed):
    past, new, h = _inputs(case, seed)
    hk, bt = case["kv_heads"], _block(case)
    lens = _lengths(case)
    cos_sin = _tables(case, max(c + r for c, r in lens))
    qs, ks, vs, at, row = [], [], [], 0, 0
    for c, r in lens:
        p, x = past[at:at + c], new[row:row + r]
        q = _turned(case, cos_sin, x[:, :h], c)
        k = _held(case, _turned(case, cos_sin, p[:, :hk], 0), _turned(case, cos_sin, x[:, h:h + hk], c))
        v = _held(case, p[:, hk:].double(), x[:, h + hk:].double())
        if case["op"] == "attend":
            # the rows of q reach the attention rounded to the pool's type
            q = q.to(new.dtype).double().unflatten(1, (hk, -1)).permute(1, 2, 0, 3)          # [kv_heads, group, rows, dim]
            pos = torch.arange(c, c + r, device=DEV)[:, None]
            key = torch.arange(c + r, device=DEV)
            seen = (key <= pos) & (key > pos - case["window"]) if case["window"] else key <= pos
            o = []
            for a in range(hk):
                s = (q[a] @ k[:, a].T / math.sqrt(case["dim"])).masked_fill(~seen, -math.inf)
                o.append(torch.softmax(s, -1) @ v[:, a].contiguous())
            qs.append(torch.stack(o).permute(2, 0, 1, 3).flatten(1, 2))
        else:
            b = 0 if case["op"] == "read" else c // bt * bt
            qs.append(q), ks.append(k[b:]), vs.append(v[b:])
        at, row = at + c, row + r
    if case["op"] == "attend":
        return torch.cat(qs)
    values = {"k": torch.cat(ks), "v": torch.cat(vs)}
    return values if case["op"] == "read" else {"q": torch.cat(qs), **values}
