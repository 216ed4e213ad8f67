"""Sequences made of other sequences' tokens on the GPU against the 64-bit model."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kv_oracle as O  # noqa: E402
from rank_gemm_page_amd import slora as S  # noqa: E402
from tests.kv_more import MoreCase  # noqa: E402

pytestmark = pytest.mark.gpu

CODES = [S.SLORA_KV_INT8, S.SLORA_KV_FP8]


@pytest.fixture(autouse=True)
def _gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.lib()
    print(f"[gpu] {request.node.name}", flush=True)


def refused(status, fn, *a, **kw):
    with pytest.raises(S.SloraError) as e:
        fn(*a, **kw)
    assert e.value.status == status, e.value
    return str(e.value)


KINDS = [("f16", 0, 64, 96), ("f16", 1, 128, 32), ("f16", 0, 256, 32), ("f32", 1, 64, 32), ("f32", 0, 128, 64)]


@pytest.mark.parametrize("dtype,code,dim,block", KINDS)
@pytest.mark.parametrize("length", [1, 31, 32, 96, 97, 210])
def test_fork_shares_whole_blocks(dtype, code, dim, block, length):
    """Two forks of one sequence: whole blocks are shared, the last one is a copy; each then goes its own way."""
    with MoreCase(torch, dtype, code, 4, 2, dim, block, n_layers=2, max_tokens=320) as c:
        c.grow([0, 3], [length, 40])
        before = c.free()
        c.take([(1, 0, None), (2, 0, [(0, length)])])
        whole = length // block
        assert before - c.free() == 2 * 4 * (length % block > 0)
        for i in (1, 2):
            assert (c.pages(i)[:whole] == c.pages(0)[:whole]).all()
            assert not np.intersect1d(c.pages(i)[whole:], c.pages(0)).size
        c.check_all([0, 1, 2, 3])
        c.grow([0, 1, 2], [1, 70, 1], 3.0, attend=(0, 0))
        c.grow([2, 0], [33, 2], 0.5, attend=(20, 3))
        c.check_all([0, 1, 2, 3])
        c.drop(0)                                              # the shared blocks stay for the others
        c.grow([3], [100])                                     # and what was freed is written to
        c.check_all([1, 2, 3])
        for i in (1, 2, 3):
            c.drop(i)
        assert c.free() == c.mem.shape[0]


RANGES = {
    "first and last": [(0, 4), (101, 230)],
    "inside blocks": [(5, 9), (33, 34), (60, 131), (200, 201)],
    "whole blocks": [(0, 96), (192, 230)],
    "shifted by whole groups": [(32, 64), (128, 224)],
    "joined": [(0, 50), (50, 50), (50, 96), (96, 230)],
    "begin": [(0, 100)],
    "end of a block": [(0, 192)],
    "one": [(229, 230)],
    "none": [(7, 7)],
    "no ranges": [],
    "every third": [(i, i + 1) for i in range(0, 230, 3)],
    "all but one": [(0, 100), (101, 230)],
    "threes": [(i, min(i + 3, 230)) for i in range(1, 230, 4)],
}


@pytest.mark.parametrize("dtype,code,dim,block", KINDS)
@pytest.mark.parametrize("name", RANGES)
def test_ranges(dtype, code, dim, block, name):
    """Into an empty sequence and in place, with block ranges of different sizes; then tokens follow, at the positions
    behind the last one that was taken."""
    with MoreCase(torch, dtype, code, 4, 2, dim, block, n_layers=2, max_tokens=320, positions=600) as c:
        for gain, n in ((1.0, 50), (20.0, 40), (0.3, 60), (2.0, 80)):
            c.grow([0, 1], [n, 5], gain)
        before = c.free()
        c.take([(3, 0, RANGES[name])])
        c.check_all([0, 1, 3])
        c.take([(0, 0, RANGES[name])])
        c.check_all([0, 1, 3])
        c.grow([3, 0, 1], [1, 40, 1], attend=(30, 5))
        c.grow([0, 1, 3], [1, 1, 65], attend=(0, 0))
        c.check_all([0, 1, 3])
        c.drop(3)
        c.drop(0)
        assert c.free() - before == 4 * -(-230 // block) - 4 * (len(c.pages(1)) - -(-20 // block))


def test_positions_follow_the_tokens():
    """Left out in the middle, then taken back to before the gap: the next token's position is behind the last one's."""
    with MoreCase(torch, "f16", 0, 4, 2, 64, 32, max_tokens=200, positions=700) as c:
        c.grow([0], [150])
        c.take([(0, 0, [(0, 10), (90, 150)])])
        assert S.slora_kv_length(c.kv, 0) == 70 and S.slora_kv_position(c.kv, 0) == 150
        c.grow([0], [7], attend=(0, 0))
        c.take([(1, 0, [(0, 40)]), (2, 0, [(0, 10)]), (3, 0, [(0, 11), (60, 77)])])
        assert [S.slora_kv_position(c.kv, i) for i in range(4)] == [157, 120, 10, 157]
        c.grow([0, 1, 2, 3], [3, 40, 1, 30], attend=(0, 0))
        c.take([(2, 2, [])])
        assert S.slora_kv_position(c.kv, 2) == 0
        for _ in range(3):                                     # a conversation far longer than the cache
            c.grow([0, 2], [100, 5], attend=(64, 4))
            n = S.slora_kv_length(c.kv, 0)
            c.take([(0, 0, [(0, 4), (n - 64, n)])])
        assert S.slora_kv_position(c.kv, 0) == 460 and S.slora_kv_length(c.kv, 0) == 68
        c.check_all([0, 1, 2, 3])
        # a table of angles that ends before the next position
        st, _, _ = c.step([0], [1])
        x = torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda:0")
        assert "position" in refused(S.SLORA_E_INVAL, S.slora_kv_append, c.kv, st, 0, x, x, cos_sin=c.cos_sin[:460])
        S.slora_kv_append(c.kv, st, 0, x, x, cos_sin=c.cos_sin[:461], stream=torch.cuda.current_stream())


def test_whole_blocks_move_nothing():
    """Ranges at multiples of the block: pages change their places only, over more entries than a wave writes at once."""
    with MoreCase(torch, "f16", 1, 2, 2, 64, 32, n_layers=2, max_seqs=2, max_tokens=6000) as c:
        c.grow([0, 1], [5990, 1])
        was, before = c.pages(0), c.free()
        c.take([(0, 0, [(0, 32), (96, 3200), (3264, 5990)])])
        now = c.pages(0)
        assert (now == np.concatenate([was[:1], was[3:100], was[102:]])).all() and c.free() - before == 4 * 4
        c.check_all([0, 1])
        c.take([(0, 0, [(1, 2), (64, 5000)])])                 # shifts everything: all blocks are written anew
        assert not np.intersect1d(c.pages(0), now).size
        c.check_all([0, 1])
        c.grow([0], [1], attend=(0, 0))


def test_taking_tokens_back_touches_no_memory():
    """A shorter end, in place: no metadata, no launch, the pages stay; not so where the last block is shared."""
    with MoreCase(torch, "f16", 0, 4, 2, 64, 32, n_layers=2, max_tokens=200) as c:
        c.grow([0], [100])
        was, before = c.pages(0), c.free()
        assert S.slora_kv_take_bytes(c.kv, [0], [0], [[(0, 70)]]) == 16
        S.slora_kv_take(c.kv, [0], [0], [[(0, 70)]])
        c.model.take([(0, 0, [(0, 70)])])
        assert (c.pages(0) == was[:3]).all() and c.free() - before == 4
        c.grow([0], [3], 9.0, attend=(0, 0))
        c.check_all([0])
        c.take([(1, 0, [(0, 64)])])
        assert (c.pages(1) == was[:2]).all()
        assert "dev_meta" in refused(S.SLORA_E_INVAL, S.slora_kv_take, c.kv, [0], [0], [[(0, 40)]])
        c.take([(0, 0, [(0, 40)])])
        assert (c.pages(0)[0] == was[0]).all() and not np.intersect1d(c.pages(0)[1], was[1]).size
        c.grow([0, 1], [1, 1], 5.0, attend=(0, 0))
        c.check_all([0, 1])


def test_shared_blocks_take_no_more_appends():
    with MoreCase(torch, "f16", 0, 4, 2, 64, 32, max_tokens=200) as c:
        st = c.grow([0], [64])
        x = torch.zeros((64, 2, 64), dtype=torch.float16, device="cuda:0")
        again = lambda: S.slora_kv_append(c.kv, st, 0, x, x, cos_sin=c.cos_sin,  # noqa: E731
                                          stream=torch.cuda.current_stream())
        c.take([(1, 0, [(0, 32)])])
        assert "shares" in refused(S.SLORA_E_INVAL, again)
        c.check_all([0, 1])
        # attention of the older step goes on: its sequence is as it was
        q = torch.randn((64, 4, 64), device="cuda:0").half()
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda:0")
        c.check_sinks(c.attend_sinks(st, q, ws, 0.1, 0, 0), q, [0], [64], [0], 0.1, 0, 0)
        c.drop(1)
        again()                                                # nobody shares it any longer
        c.model.drop(0)
        c.model.append(0, 0, np.zeros((64, 2, 64)), np.zeros((64, 2, 64)))
        c.check_all([0])


def test_refusals_change_nothing():
    with MoreCase(torch, "f16", 0, 4, 2, 64, 32, n_layers=2, max_seqs=5, max_tokens=96, extra_pages=-24) as c:
        st = c.grow([0, 1], [70, 33])                          # 5 blocks of 4 pages; 16 pages are left
        assert c.free() == 16
        grown, _, _ = c.step([1], [1])
        x = torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda:0")
        S.slora_kv_append(c.kv, grown, 0, x, x, cos_sin=c.cos_sin, stream=torch.cuda.current_stream())
        meta = torch.empty(4096, dtype=torch.uint8, device="cuda:0")
        take = lambda *a: S.slora_kv_take(c.kv, *a, meta, 4096, torch.cuda.current_stream())  # noqa: E731
        inval = S.SLORA_E_INVAL
        for dst, src, ranges in (
                ([5], [0], [None]), ([-1], [0], [None]), ([2], [5], [None]), ([2], [-1], [None]), ([2, 2], [0, 0], [None] * 2),
                ([1], [0], [None]), ([0, 2], [0, 0], [None] * 2), ([2, 0], [0, 0], [None, [(0, 5)]]),
                ([2, 3], [0, 2], [None] * 2), ([2], [0], [[(0, 71)]]), ([2], [0], [[(-1, 5)]]), ([2], [0], [[(5, 4)]]),
                ([2], [0], [[(0, 5), (4, 6)]]), ([2], [0], [[(5, 6), (0, 1)]]), ([2], [0], [[(1 << 40, 1 << 41)]])):
            refused(inval, take, dst, src, ranges)
            refused(inval, S.slora_kv_take_bytes, c.kv, dst, src, ranges)
        assert "every layer" in refused(inval, take, [2], [1], [None])         # its last token is in layer 0 only
        for bad in (([2], [0], [[(0, 5)]], 0, 4096), ([2], [0], [[(0, 5)]], meta[8:], 4000)):
            refused(inval, S.slora_kv_take, c.kv, *bad)
        need = S.slora_kv_take_bytes(c.kv, [2], [0], [[(0, 5)]])
        refused(S.SLORA_E_NOMEM, S.slora_kv_take, c.kv, [2], [0], [[(0, 5)]], meta, need - 1)
        with pytest.raises(ValueError):
            S.slora_kv_take(c.kv, [2], [0], [[(0, 5)]], meta[:16], 17)
        with pytest.raises(ValueError):
            S.slora_kv_take(c.kv, [2], [0], [None, None], meta, 4096)
        many = [[(1, 66)], [(1, 40)]]                          # 3 and 2 blocks: 20 pages
        assert "free pages" in refused(S.SLORA_E_NOMEM, take, [2, 3], [0, 0], many)
        assert c.free() == 16 and [S.slora_kv_length(c.kv, i) for i in range(5)] == [70, 34, 0, 0, 0]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                y = x + 1
                assert "captured" in refused(inval, take, [2], [0], [[(1, 5)]])
        graph.replay()
        torch.cuda.synchronize()
        assert (y == 1).all()
        c.take([(2, 0, [(1, 66)]), (3, 1, [(0, 33)])])         # what fits is taken
        assert c.free() == 0
        c.model.drop(1)                                        # (its half-appended token is not the model's)
        c.check_all([0, 2, 3])
        # the sequences that the call made stand anew: older steps are stale, those of their sources are not
        empty, _, _ = c.step([4], [0])
        c.take([(4, 0, [(0, 64)])])
        refused(S.SLORA_E_STALE, S.slora_kv_read, c.kv, empty, 0, x, x)
        c.take([(0, 0, [(0, 65)])])
        rows = torch.zeros((103, 2, 64), dtype=torch.float16, device="cuda:0")
        refused(S.SLORA_E_STALE, S.slora_kv_read, c.kv, st, 0, rows, rows)
        c.check_all([0, 2, 3, 4])


@pytest.mark.parametrize("dtype,code", [("f16", 0), ("f16", 1), ("f32", 0), ("f32", 1)])
def test_ranges_of_nan_zero_and_far_sizes(dtype, code):
    """Blocks that read as NaN, blocks of zeros and ranges thousands of times apart, joined in one block."""
    with MoreCase(torch, dtype, code, 2, 2, 64, 32, max_tokens=400) as c:
        for n, gain in enumerate((1.0, 0.0, 3e3, 1e-4, 0.0, 50.0)):
            v = (c.draw(32, 2).astype(np.float32) * gain).astype(c.np_dtype)
            k = (c.draw(32, 2).astype(np.float32) * gain).astype(c.np_dtype)
            if n == 3:
                k[5, 0, 7], v[9, 1, 3] = np.inf, np.nan        # keys of head 0, values of head 1
            c.append([0], [32], k=k, v=v)
        for i, ranges in ((1, [(3, 20), (40, 50), (70, 75)]), (2, [(32, 40), (130, 140)]), (3, [(90, 110), (150, 180)])):
            c.take([(i, 0, ranges)])
        c.check_all([0, 1, 2, 3])
        c.grow([1, 2, 3], [30, 2, 1], 2.0)
        c.check_all([1, 2, 3])


def test_fp32_subnormal_ranges():
    """Ranges below the smallest normal number, coded again beside one another."""
    with MoreCase(torch, "f32", 0, 2, 2, 64, 32, max_tokens=200) as c:
        for gain in (1e-43, 3e-39, 1e-41):
            c.append([0], [32], k=(c.draw(32, 2).astype(np.float64) * gain).astype(np.float32),
                     v=(c.draw(32, 2).astype(np.float64) * gain).astype(np.float32))
        c.take([(1, 0, [(0, 10), (64, 90)]), (2, 0, [(20, 50)])])
        for what in (0, 1):
            for i in (1, 2):
                assert np.isfinite(c.model.values(i, 0, what)).all()
        c.check_all([0, 1, 2])


@pytest.mark.parametrize("dim,tokens", [(128, 224), (64, 448), (256, 96)])
@pytest.mark.parametrize("code", CODES)
def test_blocks_of_more_tokens_than_a_workgroup(dim, tokens, code):
    """A pool of two classes with the blocks in the larger pages, whose tokens are found some at a time."""
    n = 80
    mem = [torch.full((n, 1024), 255, dtype=torch.uint8, device="cuda:0"),
           torch.full((n, 57344), 255, dtype=torch.uint8, device="cuda:0")]
    pool = S.slora_pool_create(S.SLORA_F16, 512, 28672, 1, 1, 1, mem, [n, n])
    desc = dict(cls=1, code=code, n_layers=1, n_heads=4, n_kv_heads=2, head_dim=dim,
                block_tokens=0 if dim != 256 else 96, max_seqs=4, max_tokens=1000, rot_dim=0)
    dev = torch.empty(S.slora_kv_device_bytes(pool, **desc), dtype=torch.uint8, device="cuda:0")
    kv = S.slora_kv_create(pool, dev, dev.numel(), **desc)
    model, rng, steps, keep = O.KvModel(code, 4, 2, dim, tokens), np.random.default_rng(1), [], []
    stream = torch.cuda.current_stream()

    def step(seqs, counts, reread):
        st = S.slora_kv_build_step(kv, seqs, counts, reread)
        steps.append(st)
        keep.append(torch.empty(max(16, S.slora_kv_step_get_info(st)["meta_bytes"]), dtype=torch.uint8, device="cuda:0"))
        S.slora_kv_step_upload(st, keep[-1], keep[-1].numel(), stream)
        return st

    try:
        for count, gain in ((500, 1.0), (450, 5.0)):
            k, v = ((rng.standard_normal((count, 2, dim)) * gain).astype(np.float16) for _ in range(2))
            S.slora_kv_append(kv, step([1], [count], False), 0, *(torch.from_numpy(x).to("cuda:0") for x in (k, v)),
                              stream=stream)
            model.append(1, 0, k, v)
        made = ([0, 2, 3], [1, 1, 1], [[(3, 901)], [(i, i + 2) for i in range(0, 950, 3)], [(0, 940)]])
        keep.append(torch.empty(S.slora_kv_take_bytes(kv, *made), dtype=torch.uint8, device="cuda:0"))
        S.slora_kv_take(kv, *made, keep[-1], keep[-1].numel(), stream)
        model.take(list(zip(*made)))
        for i in range(4):
            n = model.length(i)
            assert n == S.slora_kv_length(kv, i)
            x = [torch.zeros((n, 2, dim), dtype=torch.float16, device="cuda:0") for _ in range(2)]
            S.slora_kv_read(kv, step([i], [n], True), 0, *x, stream)
            for what in (0, 1):
                # a rounding of code * range to fp32 and one to fp16; a code's neighbours are further away
                value = model.values(i, 0, what)
                assert (np.abs(x[what].cpu().numpy() - value) <= 2.0 ** -10.9 * np.abs(value) + 2.0 ** -25).all()
    finally:
        torch.cuda.synchronize()
        for st in steps:
            S.slora_kv_step_destroy(st)
        S.slora_kv_destroy(kv)
        S.slora_pool_destroy(pool)


def test_steps_of_more_metadata_than_a_kernel_uploads():
    """270000 tokens at once (1.1 MB of metadata, by the copy engine) and in pieces (by a kernel): the same values."""
    rows, rng = 270000, torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn((rows, 1, 64), generator=rng, device="cuda:0").half() for _ in range(2))
    last = []
    for pieces in ([rows], [131072, 131072, rows - 262144]):
        with MoreCase(torch, "f16", 0, 1, 1, 64, 256, rot=0, max_seqs=1, max_tokens=rows) as c:
            at = 0
            for n in pieces:
                st, info, _ = c.step([0], [n])
                assert (info["meta_bytes"] > 1 << 20) == (n == rows)
                S.slora_kv_append(c.kv, st, 0, k[at:at + n], v[at:at + n], stream=torch.cuda.current_stream())
                at += n
            st, _, _ = c.step([0], [5000], True)
            x = [torch.zeros((5000, 1, 64), dtype=torch.float16, device="cuda:0") for _ in range(2)]
            S.slora_kv_read(c.kv, st, 0, *x, torch.cuda.current_stream())
            last.append(torch.stack(x))
    assert torch.equal(last[0], last[1])
    assert (last[0][0] - k[-5000:]).abs().max() < 0.03         # half a code of ranges up to 6


def test_another_stream_and_many_at_once():
    """Forks on a stream of their own, ordered by events; a prompt with eight answers beside a shortened sequence."""
    with MoreCase(torch, "f16", 0, 4, 2, 128, 32, n_layers=3, max_seqs=12, max_tokens=300) as c:
        c.grow([0, 9], [170, 130])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        c.take([(i, 0, None) for i in range(1, 9)] + [(9, 9, [(0, 3), (50, 130)]), (10, 0, [(10, 75)])], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        c.grow(list(range(11)), [1] * 11, attend=(0, 0))
        c.grow(list(range(11)), [1 + i for i in range(11)], attend=(50, 4))
        c.check_all(range(11))
        c.take([(i, i, [(0, 100 - 9 * i)]) for i in range(9)])
        c.check_all(range(11))
        c.grow(list(range(11)), [2] * 11, 4.0, attend=(0, 0))
        c.check_all(range(11))
        for i in range(11):
            c.drop(i)
        assert c.free() == c.mem.shape[0]


@pytest.mark.parametrize("seed", range(6))
def test_random_life(seed):
    """Sequences grow, fork, lose tokens and end in any order; pages are counted after every step."""
    rng = np.random.default_rng(seed)
    dtype, code, dim, block = KINDS[seed % len(KINDS)]
    with MoreCase(torch, dtype, code, 4, 2, dim, block, n_layers=2, max_seqs=6, max_tokens=260, positions=6000,
                  seed=seed, extra_pages=-20) as c:
        total = c.mem.shape[0]
        for _ in range(30):
            lens = [c.model.length(i) for i in range(6)]
            live, empty = [i for i in range(6) if lens[i]], [i for i in range(6) if not lens[i]]
            kind = rng.choice(["grow", "grow", "fork", "keep", "back", "drop"])
            try:
                if kind == "grow" or not live:
                    seqs = [int(i) for i in rng.permutation(6)[:rng.integers(1, 5)]]
                    c.grow(seqs, [int(min(260 - lens[i], rng.integers(0, 80))) for i in seqs],
                           float(2.0 ** rng.integers(-3, 4)), attend=(int(rng.integers(0, 90)), int(rng.integers(0, 40))))
                elif kind == "fork" and empty:
                    made = []
                    for d in empty[:rng.integers(1, 4)]:
                        s = int(rng.choice(live))
                        cut = np.unique(rng.integers(0, lens[s] + 1, rng.choice([2, 2, 6])))
                        made.append((d, s, None if rng.random() < 0.4 else
                                     [(int(a), int(b)) for a, b in zip(cut[:-1:2], cut[1::2])]))
                    c.take(made)
                elif kind in ("keep", "back"):
                    s = int(rng.choice(live))
                    cut = np.unique(rng.integers(0, lens[s] + 1, 4))
                    c.take([(s, s, [(0, int(cut[0]))] if kind == "back" else
                             [(int(a), int(b)) for a, b in zip(cut[:-1:2], cut[1::2])])])
                else:
                    c.drop(int(rng.choice(live)))
            except S.SloraError as e:
                assert e.status == S.SLORA_E_NOMEM, e
                c.drop(int(rng.choice(live)))
            assert [S.slora_kv_length(c.kv, i) for i in range(6)] == [c.model.length(i) for i in range(6)]
            held = [c.pages(i) for i in range(6)]
            alive = np.unique(np.concatenate([h.reshape(-1) for h in held]))
            assert c.free() == total - alive.size
            for i in range(6):
                n = c.model.length(i)
                mine = held[i][n // block:].reshape(-1)        # a block that is not full is nobody else's
                others = np.concatenate([held[j].reshape(-1) for j in range(6) if j != i])
                assert not np.intersect1d(mine, others).size
        c.check_all(range(6))


def test_the_model_takes_tokens_as_the_definition_says():
    """The model against a small case by hand: two blocks of ranges 127 and 254 join in one."""
    m = O.KvModel(O.INT8, 1, 1, 64, 32)
    x = np.zeros((64, 1, 64))
    x[:32, 0, 0], x[32:, 0, 0] = 127.0, 254.0
    x[1, 0, 1], x[40, 0, 1] = 3.0, -7.0
    m.append(0, 0, x, x)
    m.take([(1, 0, [(0, 3), (40, 42)])])
    assert m.range[1, 0, 0].tolist() == [[254.0]] and m.position(1) == 42 and m.length(1) == 5
    # 127 of 254 is the code 63.5, held as 64; 3 is 1.5, held as 2; -7 is -3.5, which was held as -4
    assert m.codes[1, 0, 0][:, 0, :2].tolist() == [[64, 0], [64, 2], [64, 0], [127, -4], [127, 0]]
    m.take([(0, 0, [(0, 32)])])
    assert m.range[0, 0, 1].tolist() == [[127.0]] and m.position(0) == 32
