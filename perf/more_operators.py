"""What is measured of the KV cache's operators for models with normed heads, far positions and long conversations.

Four operators, named by a case's ``op``:

* ``rotary``: the table of cosines and sines that append rotates by, for positions ``first .. first + positions - 1``,
  with the frequencies as they are or scaled for contexts longer than the trained one;
* ``norm``: q and k of the new tokens are normed head by head, rotated by their positions, k and v are stored as 8-bit
  codes in the sequences' blocks and the blocks that were touched are read back as values: ``run`` returns q and those;
* ``sinks``: attention of a step's rows over a window of cached tokens and the first ``sinks`` ones;
* ``take``: sequences that hold given runs of other sequences' tokens (all of them: a fork; the first few and the last
  ones, or scattered ones: a shortened copy), in every layer, read back as values: a fork from the block on that it does
  not share, the others from their start.

A case's sequences: ``seqs`` of ``ctx_lo..ctx_hi`` cached tokens with ``rows_lo..rows_hi`` new ones.  The lengths and the
runs that are taken follow from ``lengths`` alone, the data from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
DTYPES = {"f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="f16", code="int8", heads=32, kv_heads=32, dim=128, page=8192, rot=0,
             pairs="halves", layers=1, seqs=0, ctx_lo=0, ctx_hi=0, rows_lo=0, rows_hi=0, window=0, sinks=0,
             per_head=False, take="", copies=1, run=0, gap=0, positions=0, first=0, scaling="none", base=10000.0,
             factor=1.0, trained=4096, lengths=1)
    assert set(kw) <= set(c)
    return {**c, **kw}


def listed():
    gqa = dict(heads=64, kv_heads=8, page=16384)       # 8192 wide: 64 query heads on 8 kv heads
    some = dict(heads=32, kv_heads=8)                  # 4096 wide, 32 query heads on 8 kv heads
    return [
        # a model's table for the context it was trained on, at start-up
        _case("rotary_short", "rotary", rot=128, positions=4096),
        # the table of a context 32 times the trained one, scaled by bands of wavelengths
        _case("rotary_long", "rotary", rot=128, positions=131072, scaling="bands", base=500000.0, factor=32.0),
        # one user's next token: what a launch costs; the parity type
        _case("norm_one", "norm", dtype="f32", rot=128, seqs=1, ctx_lo=700, ctx_hi=700, rows_lo=1, rows_hi=1, **gqa),
        # a decode batch of 256 requests at the 4096-wide shape; weights of each head its own
        _case("norm_decode", "norm", rot=128, seqs=256, ctx_lo=1, ctx_hi=900, rows_lo=1, rows_hi=1, per_head=True),
        # 32 prompts of 64 to 512 tokens, e4m3 codes; half of each head is rotated
        _case("norm_prefill", "norm", code="fp8", rot=64, pairs="neighbours", seqs=32, rows_lo=64, rows_hi=512),
        # one user's next token late in a conversation
        _case("sinks_one", "sinks", seqs=1, ctx_lo=20000, ctx_hi=20000, rows_lo=1, rows_hi=1, window=4096, sinks=4,
              **gqa),
        # a decode batch of long conversations
        _case("sinks_decode", "sinks", code="fp8", seqs=64, ctx_lo=1500, ctx_hi=6000, rows_lo=1, rows_hi=1,
              window=1024, sinks=4, **some),
        # the next piece of a long prompt
        _case("sinks_chunk", "sinks", seqs=1, ctx_lo=6001, ctx_hi=6001, rows_lo=2048, rows_hi=2048, window=2048,
              sinks=64, **gqa),
        # a second answer to one short conversation: latency; the parity type
        _case("fork_one", "take", dtype="f32", heads=16, kv_heads=16, dim=64, page=4096, layers=4, seqs=1,
              ctx_lo=777, ctx_hi=777, take="fork"),
        # eight answers to each of eight prompts
        _case("fork_many", "take", layers=8, seqs=8, ctx_lo=500, ctx_hi=4000, take="fork", copies=8, **some),
        # a conversation that keeps its first tokens and its last half, which ends inside blocks; e4m3 codes
        _case("keep_recent", "take", code="fp8", layers=4, seqs=1, ctx_lo=32001, ctx_hi=32001, take="recent",
              window=16003, sinks=4, **gqa),
        # conversations that keep the tokens that mattered, in short runs
        _case("keep_scattered", "take", layers=2, seqs=16, ctx_lo=1000, ctx_hi=4000, take="runs", run=3, gap=3, **some),
    ]


# ---- sizes -------------------------------------------------------------------------------------------------------------

def _lengths(case):
    """(cached, new) tokens of each sequence."""
    rng = random.Random(case["lengths"])
    return [(rng.randint(case["ctx_lo"], case["ctx_hi"]), rng.randint(case["rows_lo"], case["rows_hi"]))
            for _ in range(case["seqs"])]


def _block(case):
    """Tokens of a block: what a page holds of one head's keys and values, in whole groups of 32."""
    return case["page"] // (2 * case["dim"]) // 32 * 32


def _taken(case):
    """Of each sequence that is made: (source, its runs of tokens as an array of first and last + 1)."""
    rng = random.Random(case["lengths"] + 1)
    out = []
    for i, (n, _) in enumerate(_lengths(case)):
        for _ in range(case["copies"]):
            if case["take"] == "fork":
                runs = [(0, n)]
            elif case["take"] == "recent":
                late = max(case["sinks"], n - case["window"])
                runs = [(0, min(n, case["sinks"])), (min(n, late), n)]
            else:
                runs, at = [], 0
                while at < n:
                    end = min(n, at + rng.randint(1, 2 * case["run"] - 1))
                    runs.append((at, end))
                    at = end + rng.randint(1, 2 * case["gap"] - 1)
            out.append((i, np.array([r for r in runs if r[1] > r[0]] or [(0, 1)], dtype=np.int64)))
    return out


def _back(case):
    """(tokens, first token that is read back) of each sequence that is made."""
    bt = _block(case)
    counts = [int((r[:, 1] - r[:, 0]).sum()) for _, r in _taken(case)]
    return [(n, (n - 1) // bt * bt if case["take"] == "fork" else 0) for n in counts]


def _seen(c, r, window, sinks):
    """(query, key) pairs of r rows after c cached tokens."""
    total = 0
    for p in range(c, c + r):
        lo = max(0, p - window + 1)
        total += p + 1 - lo + min(sinks, lo)
    return total


def work(case):
    e = 2 if case["dtype"] == "f16" else 4
    h, hk, d, bt = case["heads"], case["kv_heads"], case["dim"], _block(case)
    if case["op"] == "rotary":
        return {"bytes": 4 * case["positions"] * case["rot"], "flops": 4 * case["positions"] * case["rot"]}
    lens = _lengths(case)
    if case["op"] == "take":
        # the tokens' codes in and, where they are not shared, out; codes in and values out of what is read back; the
        # page table's entries in and out
        n = sum(n for n, _ in _back(case))
        tail = sum(n - b for n, b in _back(case))
        moved = sum(n % bt for n, _ in _back(case)) if case["take"] == "fork" else n
        return {"bytes": case["layers"] * hk * (2 * d * (2 * moved + tail * (1 + e)) + 8 * -(-n // bt)),
                "flops": case["layers"] * hk * 2 * d * (moved + tail)}
    rows = sum(r for _, r in lens)
    if case["op"] == "sinks":
        w, s = case["window"], case["sinks"]
        keys = sum(c + r - max(0, c + 1 - w) + min(s, max(0, c + 1 - w)) for c, r in lens)
        return {"bytes": 2 * rows * h * d * e + keys * hk * d * 2 + keys * hk * 12 // bt,
                "flops": 4 * d * h * sum(_seen(c, r, w, s) for c, r in lens)}
    touched = sum(c % bt + r for c, r in lens)
    # q in and out, k and v in, their codes out; the touched blocks' codes in and their values out
    return {"bytes": 2 * rows * h * d * e + 2 * rows * hk * d * (e + 1) + 2 * touched * hk * d * (1 + e),
            "flops": rows * (h + hk) * d * 10 + rows * hk * d * 2 + 2 * touched * hk * d}


def _cost(case):
    w = work(case)
    return w["bytes"] / 4e12 + w["flops"] / (4e14 if case["dtype"] == "f16" else 4e13)


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    limits = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("rotary", "norm", "sinks", "take")}
    while True:
        op = rng.choice(["rotary", "norm", "norm", "sinks", "sinks", "take", "take"])
        dim, rot = rng.choice([(64, 64), (128, 128), (128, 128), (128, 64), (256, 256), (256, 32), (64, 0)])
        kv_heads = rng.choice([1, 2, 3, 4, 8, 16, 32, 40])
        heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16])
        tokens = rng.choice([32, 32, 64, 96, 128])
        c = _case("", op, heads=heads, kv_heads=kv_heads, dtype=rng.choice(["f16", "f16", "f16", "f32"]),
                  code=rng.choice(["int8", "fp8"]), dim=dim, pairs=rng.choice(["halves", "neighbours"]),
                  page=2 * dim * tokens + rng.choice([0, 0, 64, 1024]), lengths=rng.randrange(1 << 30))
        del c["name"]
        if op == "rotary":
            c.update(rot=rng.choice([16, 32, 64, 96, 128, 256]), positions=log(1000, 131072),
                     first=rng.choice([0, 0, log(1, 1000000)]), base=rng.choice([10000.0, 500000.0, 1000000.0]),
                     scaling=rng.choice(["none", "linear", "base", "bands", "ramp"]),
                     factor=rng.choice([1.0, 2.5, 4.0, 8.0, 32.0]), trained=rng.choice([2048, 4096, 8192]))
        else:
            many = rng.random() < 0.5
            ctx = log(1, 4000 if many else 20000)
            c.update(seqs=log(1, 256 if many else 16), ctx_lo=rng.randint(0, ctx), ctx_hi=ctx)
            hi = 1 if many else log(2, 2000)
            c.update(rows_lo=rng.randint(1, hi), rows_hi=hi)
        if op == "norm":
            c.update(rot=rot, per_head=rng.random() < 0.3)
        if op == "sinks":
            c.update(window=log(1, 8000), sinks=rng.choice([0, 1, 4, 4, 33, log(1, 1000)]))
        if op == "take":
            c.update(rows_lo=0, rows_hi=0, ctx_lo=max(1, c["ctx_lo"]), take=rng.choice(["fork", "recent", "runs"]),
                     layers=rng.choice([1, 2, 4]), run=log(1, 300), gap=log(1, 300), window=log(1, 20000),
                     sinks=rng.choice([0, 4, 64, 100]), copies=rng.choice([1, 1, 2, 5]))
        if heads > 128 or c["page"] > 32768 or _cost(c) > limits[op] or _plain_size(c) > 4e8:
            continue
        return c


def _plain_size(case):
    """The most elements that a tensor of the plain form or of the inputs holds."""
    hk, d = case["kv_heads"], case["dim"]
    lens = _lengths(case)
    cached = sum(c + r + _block(case) for c, r in lens) * hk * d * 2 * case["layers"]
    if case["op"] == "take":
        cached = max(cached, sum(n + _block(case) for n, _ in _back(case)) * hk * d * case["layers"])
    if case["op"] == "sinks":
        for c, r in lens:
            cached = max(cached, r * case["heads"] * (min(c + r, case["window"] + r) + case["sinks"]))
    return cached


# ---- inputs ------------------------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 29)
    return g


def _drawn(case, g, n, heads):
    """n tokens of q (kv heads 0) beside k and v, [n, heads + 2 kv_heads, dim], one projection's output.  Some channels
    of k are several times larger than others, as in trained models."""
    hk, d = case["kv_heads"], case["dim"]
    x = torch.randn((n, heads + 2 * hk, d), generator=g, device=DEV, dtype=torch.float32)
    x[:, heads:heads + hk] *= torch.exp(0.6 * torch.randn((hk, d), generator=g, device=DEV))
    return x.to(DTYPES[case["dtype"]])


def _inputs(case, seed):
    """(k and v of the cached tokens by layer, each [sum ctx, 2 kv_heads, dim]; q, k and v of the new ones [rows, heads +
    2 kv_heads, dim]; the norms' weights of q and of k)"""
    g = _generator(seed)
    lens = _lengths(case)
    past = [_drawn(case, g, sum(c for c, _ in lens), 0) for _ in range(case["layers"])]
    new = _drawn(case, g, sum(r for _, r in lens), case["heads"])
    weights = []
    for h in (case["heads"], case["kv_heads"]):
        shape = (h, case["dim"]) if case["per_head"] else (case["dim"],)
        w = 1.0 + 0.3 * torch.randn(shape, generator=g, device=DEV)
        weights.append(w.to(DTYPES[case["dtype"]]))
    return past, new, weights


def _long(x):
    return torch.tensor(x, device=DEV, dtype=torch.long)


def _angles(case, n):
    """fp32 [n, rot] for the append cases: cosines, then sines."""
    half = case["rot"] // 2
    if not half:
        return None
    inv = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    ang = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def prepare(case, seed):
    if case["op"] == "rotary":
        # what a table is made for: the seed moves the first position, as where a server lengthens its table
        st = {"case": case, "first": case["first"] + seed % 1009}
        if own:
            _cache_own(st, {**case, "dim": 256, "page": 16384}, 1, seed, max_seqs=1, max_tokens=32)
        return st
    past, new, weights = _inputs(case, seed)
    h, hk = case["heads"], case["kv_heads"]
    st = {"case": case, "q": new[:, :h], "k": new[:, h:h + hk], "v": new[:, h + hk:], "weights": weights,
          "cos_sin": _angles(case, max(c + r for c, r in _lengths(case))), "scale": 1.0 / math.sqrt(case["dim"])}
    return _prepare_own(st, past, seed) if own else _prepare_plain(st, past)


# ---- the framework's operators -----------------------------------------------------------------------------------------

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


def _cache_own(st, case, n_pages, seed, **desc):
    from rank_gemm_page_amd import slora as S
    dt = DTYPES[case["dtype"]]
    elems = case["page"] // dt.itemsize
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed + 5)).to(torch.int32)
    mem = torch.empty((n_pages, elems), dtype=dt, device=DEV)
    pool = S.slora_pool_create(S.SLORA_F16 if dt == torch.float16 else S.SLORA_F32, elems, elems, 1, 1, 1, [mem],
                               [n_pages], [order.numpy()])
    desc = dict(cls=0, code=S.SLORA_KV_INT8 if case["code"] == "int8" else S.SLORA_KV_FP8, n_layers=case["layers"],
                n_heads=case["heads"], n_kv_heads=case["kv_heads"], head_dim=case["dim"], block_tokens=_block(case),
                rot_dim=case["rot"], rot_pairs=S.SLORA_KV_HALVES if case["pairs"] == "halves" else S.SLORA_KV_NEIGHBOURS,
                **desc)
    dev = torch.empty(S.slora_kv_device_bytes(pool, **desc), dtype=torch.uint8, device=DEV)
    kv = S.slora_kv_create(pool, dev, dev.numel(), **desc)
    st.update(S=S, kv=kv, keep=_Handles(S, pool, kv, [mem, dev]))
    return S, kv


def _step(st, seqs, counts, reread=False, **window):
    S, kv = st["S"], st["kv"]
    s = S.slora_kv_build_step(kv, seqs, counts, reread, **window)
    st["keep"].steps.append(s)
    info = S.slora_kv_step_get_info(s)
    meta = torch.empty(max(16, info["meta_bytes"]), dtype=torch.uint8, device=DEV)
    st["keep"].memory.append(meta)
    S.slora_kv_step_upload(s, meta, meta.numel(), torch.cuda.current_stream())
    return s, info


def _prepare_own(st, past, seed):
    """The pool, the cache and the steps that a server keeps: the cached tokens arrive in a step of their own."""
    case = st["case"]
    hk, d, bt, dt = case["kv_heads"], case["dim"], _block(case), DTYPES[case["dtype"]]
    lens = _lengths(case)
    ctx, rows = [c for c, _ in lens], [r for _, r in lens]
    blocks = sum(-(-(c + r) // bt) for c, r in lens)
    made = _back(case) if case["op"] == "take" else []
    S, kv = _cache_own(st, case, (blocks + sum(-(-n // bt) for n, _ in made)) * hk * case["layers"],
                       seed, max_seqs=len(lens) + len(made), max_tokens=max(c + r for c, r in lens))
    if case["op"] == "sinks":                          # the rows are cached too: all tokens arrive together
        past = [torch.cat([_joined(lens, past[0][:, :hk], st["k"]), _joined(lens, past[0][:, hk:], st["v"])], 1)]
        ctx = [c + r for c, r in lens]
    if sum(ctx):
        s, _ = _step(st, list(range(len(lens))), ctx)
        for layer, x in enumerate(past):
            S.slora_kv_append(kv, s, layer, x[:, :hk], x[:, hk:], cos_sin=st["cos_sin"],
                              stream=torch.cuda.current_stream())
    if case["op"] == "take":
        st["src"] = [i for i, _ in _taken(case)]
        st["dst"] = [len(lens) + i for i in range(len(made))]
        st["runs"] = [r for _, r in _taken(case)]
        st["counts"] = [n - b for n, b in made]
        st["meta"] = torch.empty(S.slora_kv_take_bytes(kv, st["dst"], st["src"], st["runs"]), dtype=torch.uint8,
                                 device=DEV)
        st["k_out"] = torch.empty((case["layers"], sum(st["counts"]), hk, d), dtype=dt, device=DEV)
        st["v_out"] = torch.empty_like(st["k_out"])
        _take_own(st)                                  # how much metadata the read back takes
        return st
    if case["op"] == "sinks":
        st["step"], info = _step(st, list(range(len(lens))), rows, True, window=case["window"], sinks=case["sinks"])
        st["workspace"] = torch.empty(max(16, info["workspace_bytes"]), dtype=torch.uint8, device=DEV)
    else:
        st["step"], _ = _step(st, list(range(len(lens))), rows)
        S.slora_kv_append_norm(kv, st["step"], 0, st["k"], st["v"], q_weight=st["weights"][0], k_weight=st["weights"][1],
                               eps=EPS, per_head=case["per_head"], cos_sin=st["cos_sin"],
                               stream=torch.cuda.current_stream())
        counts = [c % bt + r for c, r in lens]
        st["reread"], _ = _step(st, list(range(len(lens))), counts, True)
        st["k_out"] = torch.empty((sum(counts), hk, d), dtype=dt, device=DEV)
        st["v_out"] = torch.empty_like(st["k_out"])
    st["out"] = torch.empty((st["q"].shape[0], case["heads"], d), dtype=dt, device=DEV)
    return st


def _take_own(st):
    S, kv, stream = st["S"], st["kv"], torch.cuda.current_stream()
    for i in st["dst"]:
        S.slora_kv_drop(kv, i)
    S.slora_kv_take(kv, st["dst"], st["src"], st["runs"], st["meta"], st["meta"].numel(), stream)
    step = S.slora_kv_build_step(kv, st["dst"], st["counts"], True)
    info = S.slora_kv_step_get_info(step)
    if "read_meta" not in st or st["read_meta"].numel() < info["meta_bytes"]:
        st["read_meta"] = torch.empty(max(16, info["meta_bytes"]), dtype=torch.uint8, device=DEV)
    S.slora_kv_step_upload(step, st["read_meta"], st["read_meta"].numel(), stream)
    for layer in range(st["case"]["layers"]):
        S.slora_kv_read(kv, step, layer, st["k_out"][layer], st["v_out"][layer], stream)
    S.slora_kv_step_destroy(step)
    return {"k": st["k_out"], "v": st["v_out"]}


def _run_own(st):
    case, S, kv, stream = st["case"], st["S"], st["kv"], torch.cuda.current_stream()
    if case["op"] == "take":
        return _take_own(st)
    if case["op"] == "rotary":
        table = torch.empty((case["positions"], case["rot"]), dtype=torch.float32, device=DEV)
        S.slora_kv_rotary_table(kv, table, st["first"], stream=stream, **_scaling(case))
        return table
    if case["op"] == "sinks":
        S.slora_kv_attend_sinks(kv, st["step"], 0, st["q"], st["out"], st["scale"], case["window"], case["sinks"],
                                st["workspace"], st["workspace"].numel(), stream)
        return st["out"]
    S.slora_kv_append_norm(kv, st["step"], 0, st["k"], st["v"], st["q"], st["out"], st["weights"][0], st["weights"][1],
                           EPS, case["per_head"], cos_sin=st["cos_sin"], stream=stream)
    S.slora_kv_read(kv, st["reread"], 0, st["k_out"], st["v_out"], stream)
    return {"q": st["out"], "k": st["k_out"], "v": st["v_out"]}


def _scaling(case):
    """The arguments that say how a case's frequencies are scaled."""
    return dict(base=case["base"], scaling=case["scaling"], factor=case["factor"], trained=case["trained"],
                **({"low": 1.0, "high": 4.0} if case["scaling"] == "bands" else {}),
                **({"low": 1.0, "high": 32.0, "amplitude": _amplitude(case)} if case["scaling"] == "ramp" else {}))


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0


# ---- the plain forms ---------------------------------------------------------------------------------------------------
# A cache is one array of blocks, those of a sequence one after another: codes [layers, blocks, block, kv_heads, dim] and
# ranges [layers, blocks, kv_heads], of keys (0) and values (1).

def _limit(case):
    return 127.0 if case["code"] == "int8" else 448.0


def _rounded(case, x):
    """The codes (as bytes) of scaled values x (64 bits): the nearest, ties to even."""
    if case["code"] == "int8":
        return x.round().to(torch.int8).view(torch.uint8)
    return x.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _worth(case, codes):
    """What code bytes stand for, before the block's scale, in fp32."""
    return codes.view(torch.int8 if case["code"] == "int8" else torch.float8_e4m3fn).float()


def _ratio(a, b):
    """a / b in 64 bits, 0 where b is (a tensor's division, so that both are numbers of the GPU)."""
    return torch.where(b > 0, torch.as_tensor(a, dtype=torch.float64, device=b.device) / b.double(), 0.0)


def _stored(case, x, step=1024):
    """(codes, ranges) of whole blocks x [blocks, block, kv_heads, dim]."""
    codes = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    ranges = x.abs().amax((1, 3)).float()
    for i in range(0, x.shape[0], step):
        inv = _ratio(_limit(case), ranges[i:i + step])[:, None, :, None]
        codes[i:i + step] = _rounded(case, x[i:i + step].double() * inv)
    return codes, ranges


def _prepare_plain(st, past):
    case = st["case"]
    hk, d, bt = case["kv_heads"], case["dim"], _block(case)
    lens = _lengths(case)
    whole = [c if case["op"] != "sinks" else c + r for c, r in lens]       # attention: the new tokens are cached too
    first, at = [], 0
    for (c, r) in lens:
        first.append(at)
        at += -(-(c + r) // bt)
    st["first"] = first
    # the cached tokens' places among all blocks' slots
    place = torch.cat([_long(range(f * bt, f * bt + n)) for f, n in zip(first, whole)])
    st["codes"], st["range"] = [], []
    for which in (0, 1):
        codes = torch.zeros((case["layers"], at, bt, hk, d), dtype=torch.uint8, device=DEV)
        ranges = torch.zeros((case["layers"], at, hk), dtype=torch.float32, device=DEV)
        for layer, p in enumerate(past):
            x = p[:, which * hk:(which + 1) * hk]
            if case["op"] == "sinks":
                x = _joined(lens, x, st["v" if which else "k"])
            if which == 0 and case["op"] == "norm" and case["rot"]:
                pos = torch.cat([_long(range(c)) for c, _ in lens])
                x = _rotated(case, st["cos_sin"], x, pos)
            full = torch.zeros((at * bt, hk, d), dtype=x.dtype, device=DEV)
            full[place] = x
            codes[layer], ranges[layer] = _stored(case, full.view(at, bt, hk, d))
        st["codes"].append(codes), st["range"].append(ranges)
    if case["op"] == "norm":
        st["part"] = _touched(case, lens, first)
    if case["op"] == "sinks":
        st["groups"] = _groups(case, lens, first)
    if case["op"] == "take":
        _prepare_take(st, lens, first)
    return st


def _joined(lens, old, new):
    """Each sequence's cached tokens and then its new ones."""
    out, a, b = [], 0, 0
    for c, r in lens:
        out += [old[a:a + c], new[b:b + r]]
        a, b = a + c, b + r
    return torch.cat(out)


def _rotated(case, cos_sin, x, pos):
    """x [rows, heads, dim] rotated by the rows' positions, in 64 bits."""
    rot = case["rot"]
    x = x.double()
    if not rot:
        return x
    cs = cos_sin[pos].double()[:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    y = x.clone()
    if case["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def _normed(x, weight):
    """Each head over the root of its mean square, times the weights, in 64 bits."""
    x = x.double()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()


def _touched(case, lens, first):
    """Index tensors of the append: the blocks it touches, the new token of each of their slots, which slots are new,
    which hold older tokens, and what is read back of them."""
    bt = _block(case)
    blocks, tok0, start, end = [], [], [], []
    row = 0
    for f, (c, r) in zip(first, lens):
        for b in range(c // bt, -(-(c + r) // bt)):
            blocks.append(f + b), tok0.append(row - (c - b * bt)), start.append(c - b * bt), end.append(c + r - b * bt)
        row += r
    slot = torch.arange(bt, device=DEV)
    tok = _long(tok0)[:, None] + slot
    new = (slot >= _long(start)[:, None]) & (slot < _long(end)[:, None])
    used = (slot < _long(end)[:, None]).reshape(-1)
    return {"blocks": _long(blocks), "tok": torch.where(new, tok, 0), "new": new, "old": slot < _long(start)[:, None],
            "begun": _long(start) > 0, "pos": torch.cat([_long(range(c, c + r)) for c, r in lens]),
            "back": torch.nonzero(used)[:, 0]}


def _norm(st):
    case, part = st["case"], st["part"]
    dt = st["k"].dtype
    pos = part["pos"]
    q = _rotated(case, st["cos_sin"], _normed(st["q"], st["weights"][0]), pos).to(dt)
    out = {"q": q}
    for which, x in ((0, _rotated(case, st["cos_sin"], _normed(st["k"], st["weights"][1]), pos)), (1, st["v"].double())):
        new, old = part["new"][:, :, None, None], part["old"][:, :, None, None]
        x = torch.where(new, x[part["tok"]], 0.0)                              # [blocks, block, kv_heads, dim]
        codes, ranges = st["codes"][which][0], st["range"][which][0]
        held = torch.where(part["begun"][:, None], ranges[part["blocks"]], 0.0)
        grown = torch.maximum(held, x.abs().amax((1, 3)).float())
        was = codes[part["blocks"]]
        again = _rounded(case, _worth(case, was).double() * _ratio(held.double(), grown)[:, None, :, None])
        now = torch.where(new, _rounded(case, x * _ratio(_limit(case), grown)[:, None, :, None]),
                          torch.where(old, again, was))
        codes[part["blocks"]] = now
        ranges[part["blocks"]] = grown
        y = _worth(case, now) * (grown / _limit(case))[:, None, :, None]
        out["kv"[which]] = y.flatten(0, 1)[part["back"]].to(dt)
    return out


def _groups(case, lens, first):
    """Sequences of like sizes, padded: the rows of each, their positions, and the places of the cached tokens that some
    row of it sees, with their positions (-1: none)."""
    bt, w, s = _block(case), case["window"], case["sinks"]
    row0 = np.concatenate([[0], np.cumsum([r for _, r in lens])])
    order = sorted((i for i in range(len(lens)) if lens[i][1]), key=lambda i: (lens[i][1], lens[i][0]))
    out, at = [], 0
    while at < len(order):
        # as many as keep the padded scores and keys small
        end, keys, rows = at, 0, 0
        while end < len(order):
            c, r = lens[order[end]]
            k, n = max(keys, c + r - max(0, c + 1 - w) + min(s, max(0, c + 1 - w))), max(rows, r)
            size = (end - at + 1) * k * max(n * case["heads"], case["kv_heads"] * case["dim"])
            if end > at and size > 3e8:
                break
            end, keys, rows = end + 1, k, n
        pos = np.full((end - at, rows), -1, dtype=np.int64)
        row = np.zeros((end - at, rows), dtype=np.int64)
        key = np.full((end - at, keys), -1, dtype=np.int64)
        place = np.zeros((end - at, keys), dtype=np.int64)
        for a, i in enumerate(order[at:end]):
            c, r = lens[i]
            lo = max(0, c + 1 - w)
            seen = np.concatenate([np.arange(min(s, lo)), np.arange(lo, c + r)])
            pos[a, :r], row[a, :r] = np.arange(c, c + r), row0[i] + np.arange(r)
            key[a, :seen.size], place[a, :seen.size] = seen, first[i] * bt + seen
        valid = torch.from_numpy(pos >= 0).to(DEV).reshape(-1)
        g = {k: torch.from_numpy(v).to(DEV) for k, v in (("pos", pos), ("row", row), ("key", key), ("place", place))}
        g["from"] = torch.nonzero(valid)[:, 0]
        g["to"] = g["row"].reshape(-1)[g["from"]]
        out.append(g)
        at = end
    return out


def _visible(st, which, group):
    """Keys or values of a group's tokens, [seqs, kv_heads, tokens, dim] in fp32."""
    case = st["case"]
    codes = st["codes"][which][0].flatten(0, 1)[group["place"]]
    unit = (st["range"][which][0] / _limit(case))[group["place"] // _block(case)]
    return (_worth(case, codes) * unit[..., None]).permute(0, 2, 1, 3).contiguous()


def _sinks(st):
    case = st["case"]
    hk, d, g = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    out = torch.empty((st["q"].shape[0], case["heads"], d), dtype=st["q"].dtype, device=DEV)
    for group in st["groups"]:
        n, r = group["row"].shape
        q = st["q"][group["row"]].float().reshape(n, r, hk, g, d).permute(0, 2, 1, 3, 4).reshape(n, hk, r * g, d)
        s = torch.matmul(q.contiguous(), _visible(st, 0, group).transpose(2, 3).contiguous()) * st["scale"]
        key, pos = group["key"][:, None], group["pos"][:, :, None]
        seen = (key >= 0) & (key <= pos) & ((key > pos - case["window"]) | (key < case["sinks"]))
        s = s.view(n, hk, r, g, -1).masked_fill_(~seen[:, None, :, None], float("-inf")).view(n, hk, r * g, -1)
        p = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-3e38))
        o = torch.matmul(p, _visible(st, 1, group)) / p.sum(-1, keepdim=True)
        o = o.view(n, hk, r, g, d).permute(0, 2, 1, 3, 4).reshape(n * r, hk * g, d)
        out[group["to"]] = o[group["from"]].to(out.dtype)
    return out


def _prepare_take(st, lens, first):
    """Places of the tokens that each made sequence holds, its slots among its own whole blocks, and what is read back."""
    case = st["case"]
    bt = _block(case)
    place, slot, back, at = [], [], [], 0
    for (i, runs), (n, b) in zip(_taken(case), _back(case)):
        tokens = np.concatenate([np.arange(a, e) for a, e in runs])
        place.append(first[i] * bt + tokens)
        slot.append(at * bt + np.arange(n))
        back.append(at * bt + np.arange(b, n))
        at += -(-n // bt)
    st["place"], st["slot"], st["back"] = (torch.from_numpy(np.concatenate(x)).to(DEV) for x in (place, slot, back))
    st["blocks"] = at


def _take(st):
    case = st["case"]
    hk, d, bt = case["kv_heads"], case["dim"], _block(case)
    place, slot, nb = st["place"], st["slot"], st["blocks"]
    dt = DTYPES[case["dtype"]]
    out = {}
    for which in (0, 1):
        y = torch.empty((case["layers"], st["back"].numel(), hk, d), dtype=dt, device=DEV)
        for layer in range(case["layers"]):
            codes = st["codes"][which][layer].flatten(0, 1)[place]             # [tokens, kv_heads, dim]
            held = st["range"][which][layer][place // bt]                      # [tokens, kv_heads]
            every = torch.zeros((nb * bt, hk), dtype=torch.float32, device=DEV)
            every[slot] = held
            ranges = every.view(nb, bt, hk).amax(1)
            ratio = _ratio(held.double(), ranges[slot // bt])[..., None]
            made = torch.zeros((nb * bt, hk, d), dtype=torch.uint8, device=DEV)
            made[slot] = _rounded(case, _worth(case, codes).double() * ratio)
            back = st["back"]
            y[layer] = (_worth(case, made[back]) * (ranges / _limit(case))[back // bt][..., None]).to(dt)
        out["kv"[which]] = y
    return out


def _frequencies(case):
    """The angle of pair i by which a position turns it, in 64 bits."""
    half, rot = case["rot"] // 2, case["rot"]
    base, factor, trained = case["base"], case["factor"], case["trained"]
    i = torch.arange(half, device=DEV, dtype=torch.float64)
    if case["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2))
    theta = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        return theta / factor
    if case["scaling"] == "bands":
        turns = trained * theta / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return theta * keep + theta / factor * (1.0 - keep)
    if case["scaling"] == "ramp":
        pair = lambda turns: rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        part = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return theta / factor * part + theta * (1.0 - part)
    return theta


def _rotary(st):
    case = st["case"]
    pos = torch.arange(st["first"], st["first"] + case["positions"], device=DEV, dtype=torch.float64)
    ang = pos[:, None] * _frequencies(case)
    a = _amplitude(case)
    return torch.cat([(ang.cos() * a).float(), (ang.sin() * a).float()], 1)


def run(st):
    if own:
        return _run_own(st)
    return {"rotary": _rotary, "norm": _norm, "sinks": _sinks, "take": _take}[st["case"]["op"]](st)


# ---- 64 bits, from the definitions -------------------------------------------------------------------------------------

def _codes_of(case, x):
    return x.round() if case["code"] == "int8" else x.float().to(torch.float8_e4m3fn).double()


def _blocks_of(case, x):
    """[tokens, kv_heads, dim] as whole blocks [blocks, block, kv_heads, dim], the last one filled with zeros."""
    bt = _block(case)
    return torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -x.shape[0] % bt)).unflatten(0, (-1, bt))


def _peaks(x):
    return x.abs().amax((1, 3), keepdim=True).float().double()


def _over(a, b):
    return a / torch.where(b > 0, b, 1.0)


def _top(case):
    return torch.tensor(127.0 if case["code"] == "int8" else 448.0, dtype=torch.float64, device=DEV)


def _held(case, x):
    """(codes, ranges) of one sequence's tokens x that were appended together."""
    blocks = _blocks_of(case, x.double())
    peak = _peaks(blocks)
    return _codes_of(case, blocks * _over(_top(case), peak)), peak


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


def _unit(x, weight):
    x = x.double()
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()


def exact(case, seed):
    if case["op"] == "rotary":
        return _exact_rotary(case, seed)
    past, new, weights = _inputs(case, seed)
    lens = _lengths(case)
    h, hk, bt = case["heads"], case["kv_heads"], _block(case)
    ends = np.cumsum([c for c, _ in lens]).tolist()
    tokens = lambda x, i: x[ends[i] - lens[i][0]:ends[i]]  # noqa: E731
    if case["op"] == "take":
        out = {"k": [], "v": []}
        for layer in range(case["layers"]):
            for which in (0, 1):
                held = {}
                rows = []
                for (i, runs), (n, b) in zip(_taken(case), _back(case)):
                    if i not in held:
                        held = {i: _held(case, tokens(past[layer], i)[:, which * hk:(which + 1) * hk])}
                    codes, peak = held[i]
                    at = torch.cat([torch.arange(a, e, device=DEV) for a, e in runs.tolist()])
                    c, old = _blocks_of(case, codes.flatten(0, 1)[at]), _blocks_of(case, peak[at // bt, 0])
                    now = old.amax(1, keepdim=True)
                    rows.append((_codes_of(case, c * _over(old, now)) * now / _top(case)).flatten(0, 1)[b:n])
                out["kv"[which]].append(torch.cat(rows))
        return {k: torch.stack(v) for k, v in out.items()}
    cos_sin = _angles(case, max(c + r for c, r in lens))
    qs, ks, vs, row = [], [], [], 0
    for i, (c, r) in enumerate(lens):
        p, x = tokens(past[0], i), new[row:row + r]
        row += r
        if case["op"] == "norm":
            qs.append(_turned(case, cos_sin, _unit(x[:, :h], weights[0]), c))
            old_k, new_k = _turned(case, cos_sin, p[:, :hk], 0), _turned(case, cos_sin, _unit(x[:, h:h + hk], weights[1]), c)
            for to, old, late in ((ks, old_k, new_k), (vs, p[:, hk:].double(), x[:, h + hk:].double())):
                both = _blocks_of(case, torch.cat([old, late]))
                after = (torch.arange(both.shape[0] * bt, device=DEV) >= c).view(-1, bt, 1, 1)
                before, now = _peaks(both.masked_fill(after, 0.0)), _peaks(both)
                early = _codes_of(case, both * _over(_top(case), before))
                early = torch.where(before < now, _codes_of(case, early * _over(before, now)), early)
                codes = torch.where(after, _codes_of(case, both * _over(_top(case), now)), early)
                to.append((codes * now / _top(case)).flatten(0, 1)[c // bt * bt:c + r])
            continue
        both = [torch.cat([p[:, a * hk:(a + 1) * hk], x[:, h + a * hk:h + (a + 1) * hk]]) for a in (0, 1)]
        k, v = ((codes * peak / _top(case)).flatten(0, 1)[:c + r] for codes, peak in (_held(case, y) for y in both))
        lo, few = max(0, c + 1 - case["window"]), case["sinks"]
        key = torch.cat([torch.arange(min(few, lo), device=DEV), torch.arange(lo, c + r, device=DEV)])
        pos = torch.arange(c, c + r, device=DEV)[:, None]
        seen = (key <= pos) & ((pos - key < case["window"]) | (key < few))
        q = x[:, :h].double().unflatten(1, (hk, -1)).permute(1, 2, 0, 3)       # [kv_heads, group, rows, dim]
        o = []
        for a in range(hk):
            s = (q[a] @ k[key, a].T.contiguous() / math.sqrt(case["dim"])).masked_fill(~seen, -math.inf)
            o.append(torch.softmax(s, -1) @ v[key, a].contiguous())
        qs.append(torch.stack(o).permute(2, 0, 1, 3).flatten(1, 2))
    if case["op"] == "sinks":
        return torch.cat(qs)
    return {"q": torch.cat(qs), "k": torch.cat(ks), "v": torch.cat(vs)}


def _exact_rotary(case, seed):
    """Longer than 64 bits where the machine has it: frequencies from logarithms, each pair by itself."""
    rot, wide = case["rot"], np.longdouble
    tau = 8 * np.arctan(wide(1))
    base, factor = wide(case["base"]), wide(case["factor"])
    pos = np.arange(case["positions"], dtype=np.int64).astype(wide) + case["first"] + seed % 1009
    out = np.empty((case["positions"], rot))
    for i in range(rot // 2):
        if case["scaling"] == "base":
            f = np.exp(-2 * i * (np.log(base) / rot + np.log(factor) / (rot - 2)))
        else:
            f = np.exp(-2 * i * np.log(base) / rot)
        if case["scaling"] == "linear":
            f = f / factor
        if case["scaling"] in ("bands", "ramp"):
            if case["scaling"] == "bands":
                slow = 1 - min(max((case["trained"] * f / tau - 1) / 3, wide(0)), wide(1))
            else:
                edge = [rot * np.log(case["trained"] / (tau * t)) / (2 * np.log(base)) for t in (32, 1)]
                lo, hi = max(np.floor(edge[0]), 0), min(np.ceil(edge[1]), rot - 1)
                slow = min(max((i - lo) / max(hi - lo, wide(0.001)), wide(0)), wide(1))
            f = f * (1 - slow + slow / factor)
        a = np.remainder(pos * f, tau).astype(np.float64)
        out[:, i], out[:, rot // 2 + i] = np.cos(a), np.sin(a)
    return torch.from_numpy(out * (0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0))
