"""The 8-bit paged KV cache on the GPU against its 64-bit model."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kv_oracle as O  # noqa: E402
from rank_gemm_page_amd import slora as S  # noqa: E402
from tests.kv_case import KvCase  # noqa: E402

pytestmark = pytest.mark.gpu

CODES = [S.SLORA_KV_INT8, S.SLORA_KV_FP8]


@pytest.fixture(autouse=True)
def _gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.lib()
    print(f"[gpu] {request.node.name}", flush=True)


@pytest.mark.parametrize("dtype,code,dim,rot,pairs", [
    ("f16", 0, 64, 64, 0), ("f16", 1, 64, 32, 1), ("f16", 0, 128, 128, 1), ("f16", 1, 128, 128, 0),
    ("f16", 0, 256, 64, 0), ("f16", 1, 256, 256, 1), ("f32", 0, 64, 64, 1), ("f32", 1, 128, 0, 0),
    ("f32", 0, 256, 256, 0), ("f32", 1, 64, 16, 0)])
@pytest.mark.parametrize("block,slack", [(32, 0), (96, 32)])
def test_append_in_pieces_matches(dtype, code, dim, rot, pairs, block, slack):
    """Single tokens, pieces inside a block, over its end and over several blocks, with ranges that grow and ranges
    that do not; q within its roundings, keys and values code for code."""
    block = min(block, 32 if dim == 256 else 96)        # a page of a pool holds at most 32 KiB
    with KvCase(torch, dtype, code, 6, 3, dim, block, rot, pairs, max_tokens=320, slack=slack) as c:
        for counts, gain in (([1, 3, 0], 1.0), ([1, 28, 33], 2.0), ([1, 1, 1], 0.5), ([33, 1, 64], 4.0),
                             ([70, 5, 130], 0.1), ([0, 31, 1], 8.0)):
            c.append([0, 1, 3], counts, gain)
        c.check_read([0, 1, 3])
        c.check_read([3, 0])


@pytest.mark.parametrize("code", CODES)
def test_layers_and_order_of_sequences(code):
    with KvCase(torch, "f16", code, 4, 2, 64, 32, n_layers=3) as c:
        st, _, _ = c.step([2, 0], [40, 7])
        for layer in range(3):
            k, v = c.draw(47, 2), c.draw(47, 2)
            S.slora_kv_append(c.kv, st, layer, c.device(k), c.device(v), cos_sin=c.cos_sin,
                              stream=torch.cuda.current_stream())
            c.model.append(2, layer, k[:40], v[:40])
            c.model.append(0, layer, k[40:], v[40:])
        for layer in range(3):
            c.check_read([0, 2], layer)


@pytest.mark.parametrize("dtype,code,dim,heads,kv", [
    ("f16", 0, 64, 4, 4), ("f16", 1, 128, 8, 1), ("f16", 0, 128, 6, 2), ("f16", 1, 256, 4, 2), ("f16", 0, 256, 3, 3),
    ("f16", 1, 64, 20, 1), ("f16", 0, 128, 64, 2), ("f32", 0, 64, 4, 2), ("f32", 1, 128, 5, 1), ("f32", 0, 256, 2, 2)])
@pytest.mark.parametrize("window", [0, 1, 7, 50])
def test_attention_matches(dtype, code, dim, heads, kv, window):
    with KvCase(torch, dtype, code, heads, kv, dim, 64 if dim < 256 else 32, max_tokens=320) as c:
        seqs = [3, 0, 1, 2]
        for counts, gain in (([1, 0, 5, 33], 1.0), ([1, 1, 1, 1], 3.0), ([17, 130, 2, 40], 1.0), ([1, 64, 0, 3], 0.3)):
            st, info, ws, q, starts = c.append(seqs, counts, gain)
            out = c.attend(st, q, ws, 1 / np.sqrt(dim), window)
            c.check_attend(out, q, seqs, counts, starts, 1 / np.sqrt(dim), window)


@pytest.mark.parametrize("dtype,code", itertools.product(["f16", "f32"], CODES))
@pytest.mark.parametrize("length,rows", [(2500, 1), (2049, 3), (1100, 40)])
def test_long_sequences_split_their_keys(dtype, code, length, rows):
    with KvCase(torch, dtype, code, 8, 2, 64, 64, max_seqs=2, max_tokens=3000) as c:
        c.append([0, 1], [length - rows, 9], 1.0)
        st, info, ws, q, starts = c.append([0, 1], [rows, 2])
        assert info["workspace_bytes"] > 0
        for window in (0, 700):
            out = c.attend(st, q, ws, 0.125, window)
            c.check_attend(out, q, [0, 1], [rows, 2], starts, 0.125, window)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("rows", [3, 70])
def test_peaked_and_far_apart_scores(code, rows):
    """Scores of some hundreds: nearly all weight on one key, references raised again and again; scales of both signs
    and none (70 rows take the prompt tiles)."""
    with KvCase(torch, "f16", code, 4, 4, 64, 32) as c:
        c.append([0], [200], 6.0)
        st, info, ws, q, starts = c.append([0], [rows], 6.0, q=c.draw(rows, 4) * np.float16(6))
        for scale in (1.0, -0.5, 0.0):
            out = c.attend(st, q, ws, scale)
            c.check_attend(out, q, [0], [rows], starts, scale)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("heads,dim", [(2, 64), (8, 64), (8, 128), (4, 256)])
def test_block_ranges_of_very_different_size(code, heads, dim):
    """Value ranges that fall and rise by thousands from block to block, and blocks of zeros, in row tiles (2 heads)
    and prompt tiles."""
    with KvCase(torch, "f16", code, heads, 2, dim, 32) as c:
        for gain in (1.0, 2e-4, 3e3, 0.0, 1e-3, 50.0, 0.0):
            v = (c.draw(32, 2).astype(np.float32) * gain).astype(np.float16)
            st, info, ws, q, starts = c.append([0], [32], v=v)
            out = c.attend(st, q, ws, 0.125)
            c.check_attend(out, q, [0], [32], starts, 0.125)
        c.check_read([0])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("rows", [2, 40])
def test_a_row_of_nan_is_alone(dtype, rows):
    """A query row of NaN or infinity gives NaN there and changes no other row (split keys included)."""
    with KvCase(torch, dtype, 0, 4, 2, 64, 32, max_tokens=1200) as c:
        c.append([0, 1], [1000, 3])
        st, info, ws, q, starts = c.append([0, 1], [rows, 1])
        clean = c.attend(st, q, ws, 0.125)
        for bad in (float("nan"), float("inf")):
            x = q.clone()
            x[1, 2, 7] = bad
            out = c.attend(st, x, ws, 0.125)
            assert torch.isnan(out[1, 2]).all()
            out[1, 2] = clean[1, 2]
            assert torch.equal(out, clean)


@pytest.mark.parametrize("dim,tokens", [(128, 224), (64, 448), (256, 96)])
def test_blocks_of_the_second_page_class(dim, tokens):
    """A pool of two classes with the blocks in the larger pages: 224 tokens and more a block."""
    n = 40
    mem = [torch.full((n, 1024), 255, dtype=torch.uint8, device="cuda:0"),
           torch.full((n, 57344), 255, dtype=torch.uint8, device="cuda:0")]
    pool = S.slora_pool_create(S.SLORA_F16, 512, 28672, 1, 1, 1, mem, [n, n])
    desc = dict(cls=1, code=S.SLORA_KV_FP8, n_layers=1, n_heads=4, n_kv_heads=2, head_dim=dim,
                block_tokens=0 if dim != 256 else 96, max_seqs=2, max_tokens=900, rot_dim=dim)
    dev = torch.empty(S.slora_kv_device_bytes(pool, **desc), dtype=torch.uint8, device="cuda:0")
    kv = S.slora_kv_create(pool, dev, dev.numel(), **desc)
    cs = O.angles(900, dim)
    model, rng = O.KvModel(S.SLORA_KV_FP8, 4, 2, dim, tokens, dim, O.HALVES, cs), np.random.default_rng(1)
    cos_sin, steps, keep = torch.from_numpy(cs).to("cuda:0"), [], []
    try:
        for count in (1, 500, 1, 130, 30):
            st = S.slora_kv_build_step(kv, [1], [count])
            steps.append(st)
            info = S.slora_kv_step_get_info(st)
            meta, ws = (torch.empty(max(16, info[k]), dtype=torch.uint8, device="cuda:0")
                        for k in ("meta_bytes", "workspace_bytes"))
            keep += [meta, ws]
            S.slora_kv_step_upload(st, meta, meta.numel(), torch.cuda.current_stream())
            start = model.length(1)
            q, k, v = (rng.standard_normal((count, h, dim)).astype(np.float16) for h in (4, 2, 2))
            model.append(1, 0, k, v)
            dq, dk, dv = (torch.from_numpy(x).to("cuda:0") for x in (q, k, v))
            out = torch.empty_like(dq)
            S.slora_kv_append(kv, st, 0, dk, dv, dq, dq, cos_sin=cos_sin, stream=torch.cuda.current_stream())
            S.slora_kv_attend(kv, st, 0, dq, out, 0.1, 0, ws, ws.numel(), torch.cuda.current_stream())
            S.slora_kv_read(kv, st, 0, dk, dv, torch.cuda.current_stream())
            want, weight, *_ = model.attend(1, 0, dq.cpu().numpy(), start, 0.1)
            # a weight and the output are rounded to fp16 once each, everything else to fp32 or better
            assert (np.abs(out.cpu().numpy() - want) <= weight * 2.0 ** -10 + 2.0 ** -11 * np.abs(want) + 2.0 ** -24).all()
            for what, x in ((0, dk), (1, dv)):
                value = model.values(1, 0, what, start)
                assert (np.abs(x.cpu().numpy() - value) <= 2.0 ** -10 * np.abs(value) + 2.0 ** -24).all()
        assert len(S.slora_kv_pages(kv, 1)) == -(-662 // tokens)
    finally:
        torch.cuda.synchronize()
        for st in steps:
            S.slora_kv_step_destroy(st)
        S.slora_kv_destroy(kv)
        S.slora_pool_destroy(pool)


@pytest.mark.parametrize("dtype,code", itertools.product(["f16", "f32"], CODES))
@pytest.mark.parametrize("what", ["k", "v"])
def test_values_that_are_not_finite_mark_their_block_and_head(dtype, code, what):
    """A block and head with an infinity or NaN reads as NaN; rows that do not see the block stay as they are."""
    with KvCase(torch, dtype, code, 4, 2, 64, 32) as c:
        k, v = c.draw(70, 2), c.draw(70, 2)
        (k if what == "k" else v)[40, 1, 5] = np.inf
        (k if what == "k" else v)[33, 0, 6] = np.nan if dtype == "f16" else -np.inf
        st, info, ws, q, starts = c.append([0, 1], [70, 3], k=np.concatenate([k, c.draw(3, 2)]),
                                           v=np.concatenate([v, c.draw(3, 2)]))
        c.check_read([0, 1])
        out = c.attend(st, q, ws, 0.125, 20)
        got = out.cpu().numpy()
        # heads of 32-token blocks 0 and 2 are fine, block 1 is not: rows 0..31 see block 0, rows 32..63 see block 1
        assert np.isfinite(got[:32]).all() and np.isnan(got[32:64]).all() and np.isfinite(got[70:]).all()
        c.check_attend(out, q, [1], [0], [0], 0.125)
        want, *_ = c.model.attend(0, 0, q[:32].cpu().numpy(), 0, 0.125, 20, 70)
        assert np.abs(got[:32] - want).max() < 2e-2
        c.append([0], [30])                              # what follows in the block stays NaN
        c.check_read([0])


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("window", [0, 9])
def test_rows_beside_a_marked_block(code, what, window):
    """Rows of one tile on both sides of a block that reads as NaN: those that do not see it are numbers."""
    with KvCase(torch, "f16", code, 8, 2, 64, 32) as c:
        c.append([0], [25])
        k, v = c.draw(60, 2), c.draw(60, 2)
        (k if what == "k" else v)[40 - 25, :, 3] = np.inf              # in block 1: positions 32 .. 63
        st, info, ws, q, starts = c.append([0], [60], k=k, v=v)
        got = c.attend(st, q, ws, 0.125, window).cpu().numpy()
        pos = 25 + np.arange(60)
        sees = (pos >= 32) & ((pos - window + 1 <= 63) if window else True)
        assert np.isnan(got[sees]).all() and np.isfinite(got[~sees]).all()
        want, *_ = c.model.attend(0, 0, q.cpu().numpy(), 25, 0.125, window)
        assert np.abs(got[~sees] - want[~sees]).max() < 2e-2


def test_rows_behind_the_last_sequence_stay_as_they_were():
    with KvCase(torch, "f16", 0, 4, 2, 64, 32) as c:
        st, info, ws, q, starts = c.append([0, 2], [5, 40])
        out = torch.full((64, 4, 64), 7.0, dtype=torch.float16, device="cuda:0")
        qq = torch.full((64, 4, 64), float("nan"), dtype=torch.float16, device="cuda:0")
        qq[:45] = q
        c.attend(st, qq, ws, 0.125, out=out)
        assert (out[45:] == 7.0).all() and torch.isfinite(out[:45]).all()
        k = torch.full((50, 2, 64), 7.0, dtype=torch.float16, device="cuda:0")
        S.slora_kv_read(c.kv, st, 0, k, None, torch.cuda.current_stream())
        assert (k[45:] == 7.0).all() and not (k[:45] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_parts_of_one_projection_and_q_in_place(dtype):
    """q, k and v as strided parts of one tensor, q rotated in place, out and read rows strided."""
    with KvCase(torch, dtype, 1, 6, 3, 64, 32) as c:
        n = 41
        qkv = c.draw(n, 6 + 3 + 3)
        dev = c.device(qkv)
        q, k, v = dev[:, :6], dev[:, 6:9], dev[:, 9:]
        st, info, ws = c.step([1], [n])
        S.slora_kv_append(c.kv, st, 0, k, v, q, q, cos_sin=c.cos_sin, stream=torch.cuda.current_stream())
        c.model.append(1, 0, qkv[:, 6:9], qkv[:, 9:])
        c.check_rotated(q, qkv[:, :6], 0)
        np.testing.assert_array_equal(dev[:, 6:].cpu().numpy(), qkv[:, 6:])
        wide = torch.zeros((n, 10, 64), dtype=c.tdtype, device="cuda:0")
        c.attend(st, q, ws, 0.125, out=wide[:, 2:8])
        assert (wide[:, :2] == 0).all() and (wide[:, 8:] == 0).all()
        c.check_attend(wide[:, 2:8], q, [1], [n], [0], 0.125)
        back = torch.zeros((n, 8, 64), dtype=c.tdtype, device="cuda:0")
        S.slora_kv_read(c.kv, st, 0, back[:, 1:4], back[:, 5:], torch.cuda.current_stream())
        c.check_values(back[:, 5:], c.model.values(1, 0, 1))
        assert (back[:, 0] == 0).all() and (back[:, 4] == 0).all()


def test_reread_steps_attend_like_the_step_that_appended():
    with KvCase(torch, "f16", 0, 4, 2, 128, 64) as c:
        c.append([0, 1], [100, 20])
        st, info, ws, q, starts = c.append([0, 1], [30, 1])
        a = c.attend(st, q, ws, 0.1)
        re, _, ws2 = c.step([0, 1], [30, 1], True)
        b = c.attend(re, q, ws2, 0.1)
        assert torch.equal(a, b)
        # an older step still sees what it saw, whatever came behind it
        c.append([0, 1], [3, 3], 0.5)
        k2 = c.attend(st, q, ws, 0.1)
        c.check_attend(k2, q, [0, 1], [30, 1], starts, 0.1)


def test_repeated_launches_agree_and_appending_again_changes_nothing():
    with KvCase(torch, "f16", 0, 8, 2, 64, 64, max_tokens=2500) as c:
        c.append([0], [2400])
        q, k, v = c.draw(2, 8), c.draw(2, 2, 5.0), c.draw(2, 2, 5.0)
        st, info, ws, qr, starts = c.append([0], [2], q=q, k=k, v=v)
        first = c.attend(st, qr, ws, 0.125)
        for _ in range(3):
            S.slora_kv_append(c.kv, st, 0, c.device(k), c.device(v), cos_sin=c.cos_sin,
                              stream=torch.cuda.current_stream())
            ws.fill_(255)
            assert torch.equal(c.attend(st, qr, ws, 0.125), first)
        c.check_read([0])


def test_dropped_sequences_give_their_pages_to_others():
    with KvCase(torch, "f16", 1, 2, 2, 64, 32, max_seqs=2, max_tokens=96, extra_pages=0) as c:
        c.append([0, 1], [96, 96])
        with pytest.raises(S.SloraError):
            c.step([1], [1])
        S.slora_kv_drop(c.kv, 0)
        for w in (0, 1):
            del c.model.codes[0, 0, w], c.model.range[0, 0, w]
        st, info, ws, q, starts = c.append([0], [50], 0.01)
        out = c.attend(st, q, ws, 0.125)
        c.check_attend(out, q, [0], [50], starts, 0.125)
        c.check_read([0, 1])


def test_another_stream():
    with KvCase(torch, "f16", 0, 4, 2, 64, 32) as c:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            st, info, ws, q, starts = c.append([0, 1], [70, 9])
            out = c.attend(st, q, ws, 0.125)
            side.synchronize()
            c.check_attend(out, q, [0, 1], [70, 9], starts, 0.125)


def test_captured_and_replayed_with_work_between():
    """One graph with append, attention (split keys) and read; replayed on new inputs with eager launches between."""
    with KvCase(torch, "f16", 0, 8, 2, 64, 64, max_seqs=2, max_tokens=2500) as c:
        c.append([0, 1], [2304, 64])
        q, k, v = c.draw(2, 8), c.draw(2, 2), c.draw(2, 2)
        st, info, ws, qr, starts = c.append([0, 1], [1, 1], q=q, k=k, v=v)
        qd, kd, vd = c.device(q), c.device(k), c.device(v)
        qo, out, ko, vo = torch.empty_like(qd), torch.empty_like(qd), torch.empty_like(kd), torch.empty_like(vd)
        side = torch.cuda.Stream()

        def work(stream):
            S.slora_kv_append(c.kv, st, 0, kd, vd, qd, qo, cos_sin=c.cos_sin, stream=stream)
            S.slora_kv_attend(c.kv, st, 0, qo, out, 0.125, 0, ws, ws.numel(), stream)
            S.slora_kv_read(c.kv, st, 0, ko, vo, stream)

        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            work(torch.cuda.current_stream())
        for i in range(4):
            # the new tokens open blocks of their own (2304 and 64 are ends of blocks): the result does not depend on
            # what was there before
            x = [c.draw(2, 8), c.draw(2, 2), c.draw(2, 2)]
            for t, n in zip((qd, kd, vd), x):
                t.copy_(torch.from_numpy(n))
            work(torch.cuda.current_stream())
            torch.cuda.synchronize()
            want = [t.clone() for t in (qo, out, ko, vo)]
            for t in (qo, out, ko, vo):
                t.zero_()
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip((qo, out, ko, vo), want):
                assert torch.equal(a, b), i


def test_pages_beyond_four_gibibytes():
    """The first pages handed out lie at the end of a pool of 5 GiB."""
    n = 5 * (1 << 30) // 4096
    mem = torch.empty((n, 4096), dtype=torch.uint8, device="cuda:0")
    mem[-64:] = 255
    with KvCase(torch, "f16", 0, 4, 2, 64, 32, mem=mem, free_order=np.arange(n - 1, -1, -1, dtype=np.int32)) as c:
        st, info, ws, q, starts = c.append([0, 1], [40, 70])
        assert int(S.slora_kv_pages(c.kv, 0).min()) * 4096 > 1 << 32
        out = c.attend(st, q, ws, 0.125)
        c.check_attend(out, q, [0, 1], [40, 70], starts, 0.125)
        c.check_read([0, 1])


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes(seed):
    rng = np.random.default_rng(100 + seed)
    dtype, code = ("f16", "f32")[int(rng.integers(0, 4)) == 0], int(rng.integers(0, 2))
    dim, kv = int(rng.choice([64, 128, 256])), int(rng.choice([1, 2, 3, 5]))
    heads = kv * int(rng.choice([1, 2, 3, 4, 7, 16]))
    block = int(rng.choice([32, 64, 96, 128])) if dim < 256 else 32
    rot = int(rng.choice([0, 16, 32, dim]))
    with KvCase(torch, dtype, code, heads, kv, dim, block, rot, int(rng.integers(0, 2)), max_seqs=5, max_tokens=900,
                seed=seed) as c:
        for _ in range(4):
            seqs = rng.permutation(5)[:rng.integers(1, 6)].tolist()
            counts = [int(rng.choice([0, 1, 1, 2, rng.integers(1, 200)])) for _ in seqs]
            st, info, ws, q, starts = c.append(seqs, counts, float(rng.choice([0.3, 1.0, 3.0])))
            window = int(rng.choice([0, 0, 1, 33, 200]))
            out = c.attend(st, q, ws, 1 / np.sqrt(dim), window)
            c.check_attend(out, q, seqs, counts, starts, 1 / np.sqrt(dim), window)
        c.check_read([s for s in range(5) if c.model.length(s)])
