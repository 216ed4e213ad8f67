"""Attention over a window and the first tokens on the GPU against the 64-bit model."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

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


@pytest.mark.parametrize("dtype,code,dim,heads,kv", [
    ("f16", 0, 64, 4, 4), ("f16", 1, 128, 8, 1), ("f16", 0, 128, 6, 2), ("f16", 1, 256, 4, 2), ("f16", 1, 64, 20, 1),
    ("f16", 0, 128, 64, 2), ("f32", 0, 64, 4, 2), ("f32", 1, 128, 5, 1), ("f32", 0, 256, 2, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (7, 4), (50, 33), (50, 0), (33, 64), (100, 96), (40, 1000), (0, 5)])
def test_matches(dtype, code, dim, heads, kv, window, sinks):
    """Rows of all kinds of tiles; sinks that end inside a group of keys and at its end, meet the window or pass the
    sequence; steps cut for it and not."""
    with MoreCase(torch, dtype, code, heads, kv, dim, 64 if dim < 256 else 32, max_tokens=320) as c:
        seqs = [3, 0, 1, 2]
        for counts, gain in (([1, 0, 5, 33], 1.0), ([1, 1, 1, 1], 3.0), ([17, 130, 2, 40], 1.0), ([1, 64, 0, 3], 0.3)):
            st, info, ws, q, starts = c.append(seqs, counts, gain)
            out = c.attend_sinks(st, q, ws, 1 / np.sqrt(dim), window, sinks)
            c.check_sinks(out, q, seqs, counts, starts, 1 / np.sqrt(dim), window, sinks)
            st, info, ws = c.step(seqs, counts, True, window=window, sinks=sinks)
            out = c.attend_sinks(st, q, ws, 1 / np.sqrt(dim), window, sinks)
            c.check_sinks(out, q, seqs, counts, starts, 1 / np.sqrt(dim), window, sinks)


@pytest.mark.parametrize("dtype,code", itertools.product(["f16", "f32"], CODES))
@pytest.mark.parametrize("length,rows", [(2500, 1), (2049, 3), (1100, 40), (2600, 150)])
def test_long_sequences(dtype, code, length, rows):
    """Key splits that begin and end on both sides of the jump from the first tokens to the window, cut for another window
    than the launch's too."""
    with MoreCase(torch, dtype, code, 8, 2, 64, 64, max_seqs=2, max_tokens=3000) as c:
        c.append([0, 1], [length - rows, 9], 1.0)
        st, info, ws, q, starts = c.append([0, 1], [rows, 2])
        for window, sinks in ((700, 4), (1025, 600), (1, 700)):
            out = c.attend_sinks(st, q, ws, 0.125, window, sinks)
            c.check_sinks(out, q, [0, 1], [rows, 2], starts, 0.125, window, sinks)
        for cut in (dict(window=700, sinks=4), dict(window=1, sinks=0), dict(window=5000)):
            st, info, ws = c.step([0, 1], [rows, 2], True, **cut)
            for window, sinks in ((700, 4), (1025, 600), (0, 0)):
                out = c.attend_sinks(st, q, ws, 0.125, window, sinks)
                c.check_sinks(out, q, [0, 1], [rows, 2], starts, 0.125, window, sinks)


@pytest.mark.parametrize("rows", [1, 60])
@pytest.mark.parametrize("window", [40, 100])
def test_without_sinks_it_is_the_windows_attention(rows, window):
    """The same bits as slora_kv_attend's from the same step: its kernels are not the ones with sinks."""
    with MoreCase(torch, "f16", 0, 8, 2, 128, 32, max_tokens=900) as c:
        c.append([0], [800])
        st, info, ws, q, starts = c.append([0], [rows])
        assert torch.equal(c.attend(st, q, ws, 0.09, window), c.attend_sinks(st, q, ws, 0.09, window, 0))
        assert torch.equal(c.attend(st, q, ws, 0.09), c.attend_sinks(st, q, ws, 0.09, 0, 7))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("rows", [1, 50])
def test_blocks_between_sinks_and_window_stay_hidden(dtype, code, rows):
    """A block that reads as NaN between the two changes nothing; among the first tokens it shows in every row."""
    with MoreCase(torch, dtype, code, 4, 2, 64, 32, max_tokens=400) as c:
        for what in ("k", "v"):
            seq = 0 if what == "k" else 1
            x = c.draw(300 - rows, 2)
            x[130, 1, 5] = np.nan                              # block 4, kv head 1
            c.append([seq], [300 - rows], **{what: x})
            st, info, ws, q, starts = c.append([seq], [rows])
            for sinks, hidden in ((4, True), (128, True), (129, False), (140, False)):
                out = c.attend_sinks(st, q, ws, 0.125, 60, sinks)
                c.check_sinks(out, q, [seq], [rows], starts, 0.125, 60, sinks)
                assert torch.isnan(out[:, 2:]).all() == (not hidden)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("rows", [1, 40, 200])
def test_peaked_scores(code, rows):
    """Most weight on one of the first tokens or of the window, references raised late, scales of both signs."""
    with MoreCase(torch, "f16", code, 4, 4, 64, 32, max_tokens=600) as c:
        c.append([0], [300], 6.0)
        st, info, ws, q, starts = c.append([0], [rows], 6.0, q=c.draw(rows, 4) * np.float16(6))
        for scale in (1.0, -0.5, 0.0):
            out = c.attend_sinks(st, q, ws, scale, 45, 10)
            c.check_sinks(out, q, [0], [rows], starts, scale, 45, 10)


def test_captured_and_replayed_beside_eager_work():
    with MoreCase(torch, "f16", 0, 8, 2, 128, 32, max_tokens=2300) as c:
        c.append([0, 1], [2000, 1700])
        st, info, ws, q, starts = c.append([0, 1], [1, 1])
        st, info, ws = c.step([0, 1], [1, 1], True, window=900, sinks=4)
        assert info["n_row_tiles"] > 2                         # the keys are split: counters and workspace are used
        out = torch.empty_like(q)
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            S.slora_kv_attend_sinks(c.kv, st, 0, q, out, 0.09, 900, 4, ws, ws.numel(), torch.cuda.current_stream())
        for n in range(3):
            q.copy_(torch.from_numpy(c.draw(2, 8)))
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            c.check_sinks(out, q, [0, 1], [1, 1], starts, 0.09, 900, 4)
            assert torch.equal(out, c.attend_sinks(st, q, ws, 0.09, 900, 4))
            torch.cuda.synchronize()


def test_rows_behind_the_last_stay_as_they_were():
    with MoreCase(torch, "f16", 0, 8, 2, 64, 32, max_tokens=300) as c:
        for rows in (3, 70):
            st, info, ws, q, starts = c.append([0], [rows])
            out = torch.full((rows + 2, 8, 64), 7.0, dtype=torch.float16, device="cuda:0")
            S.slora_kv_attend_sinks(c.kv, st, 0, q, out, 0.1, 9, 2, ws, ws.numel(), torch.cuda.current_stream())
            assert (out[rows:] == 7).all()
            c.check_sinks(out[:rows], q, [0], [rows], starts, 0.1, 9, 2)
