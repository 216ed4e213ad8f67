"""The 8-bit paged KV cache on the GPU at the limits of its types, of its order of calls and of its launches."""
from types import SimpleNamespace

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kv_oracle as O  # noqa: E402
from rank_gemm_page_amd import slora as S  # noqa: E402
from tests.kv_case import KvCase, half_step  # noqa: E402

pytestmark = pytest.mark.gpu

CODES = [S.SLORA_KV_INT8, S.SLORA_KV_FP8]


@pytest.fixture(autouse=True)
def _gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.lib()
    print(f"[gpu] {request.node.name}", flush=True)


def weight_bits(c, out, q, seqs, counts, starts, scale, window=0):
    """Each output against the model's, with weights held in 22 bits or more:
    * scores, the exponential and the sums of the keys as in KvCase.check_attend: (dim + 8) 2^-24 of the score's
      magnitudes twice, 2^-20, and one fp32 rounding a key at most;
    * a weight is the sum of two fp16 numbers: the second is at most 2^-11 of the first and rounded by 2^-11 of itself,
      2^-22 together; where it falls below 2^-14 by up to 2^-25, in units of the largest block range that the kernel
      keeps sums in, at most 2^10 times the block's own;
    * the output is rounded once, half a step."""
    out, q = out.cpu().numpy().astype(np.float64), q.cpu().numpy()
    at = 0
    for s, n, start in zip(seqs, counts, starts):
        if n:
            want, weight, reach, spread = c.model.attend(s, 0, q[at:at + n], start, scale, window, start + n)
            r = c.model.range[s, 0, 1]
            ratio = min(1024.0, r.max() / r[r > 0].min())
            bound = weight * (2 * (c.dim + 8) * 2.0 ** -24 * reach + 2.0 ** -20 + (start + n + 8) * 2.0 ** -24)
            bound += weight * 2.0 ** -22 + spread * 2.0 ** -25 * ratio
            bound += half_step(np.abs(want) + bound, c.np_dtype)
            far = np.abs(out[at:at + n] - want) > bound
            assert not far.any(), (s, int(far.sum()), far.size, np.argwhere(far)[:4].tolist())
        at += n


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dim,heads,kv", [(64, 4, 4), (128, 8, 2), (256, 2, 1)])
@pytest.mark.parametrize("rows,window", [(10, 0), (150, 0), (150, 5)])
def test_weights_of_prompt_tiles_keep_their_bits(code, dim, heads, kv, rows, window):
    """10 rows of up to 4 query heads a kv head take the row tiles, 150 the prompt tiles: one bound for both.  Small
    scores keep the bound of their fp32 sums below a weight's 11th bit, and few keys its rounding from averaging out."""
    scale = 0.25 / np.sqrt(dim)
    with KvCase(torch, "f16", code, heads, kv, dim, 32, max_tokens=600) as c:
        c.append([0, 1], [300, 20])
        st, info, ws, q, starts = c.append([0, 1], [rows, rows])
        assert (info["n_prompt_tiles"] > 0) == (rows == 150)
        out = c.attend(st, q, ws, scale, window)
        weight_bits(c, out, q, [0, 1], [rows, rows], starts, scale, window)


@pytest.mark.parametrize("code", CODES)
def test_weights_of_split_prompt_tiles_keep_their_bits(code):
    """Keys split over workgroups."""
    with KvCase(torch, "f16", code, 8, 2, 64, 64, max_seqs=1, max_tokens=3000) as c:
        c.append([0], [2400])
        st, info, ws, q, starts = c.append([0], [24])
        assert info["n_prompt_tiles"] > 1 and info["workspace_bytes"] > 0
        out = c.attend(st, q, ws, 0.125)
        weight_bits(c, out, q, [0], [24], starts, 0.125)


def natural(c, out, q, seqs, counts, starts, scale, window=0):
    """fp32: as KvCase.check_attend, with what numbers below 2^-126 may lose: weights are at most 1 and their sum is at
    least 2^-8 (that of the largest score), so a value or a product that counts as 0 takes 2^-118 of the output, 2^-117
    a key together."""
    out, q = out.cpu().numpy().astype(np.float64), q.cpu().numpy()
    at = 0
    for s, n, start in zip(seqs, counts, starts):
        want, weight, reach, _ = c.model.attend(s, 0, q[at:at + n], start, scale, window, start + n)
        keys = start + n
        bound = weight * (2 * (c.dim + 8) * 2.0 ** -24 * reach + 2.0 ** -20 + (keys + 8) * 2.0 ** -24)
        bound += keys * 2.0 ** -117
        bound += half_step(np.abs(want) + bound, np.float32)
        far = ~(np.abs(out[at:at + n] - want) <= bound)
        assert not far.any(), (s, int(far.sum()), far.size, np.argwhere(far)[:4].tolist(), out[at:at + n][far][:4],
                               want[far][:4])
        at += n


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("gains", [(1.0, 1e-36, 1e-39, 1e30), (1e30, 1e-39, 1e-36, 1.0), (1e20, 1e-20, 0.0, 1e20),
                                   (1e-39, 1.0, 1e-37, 0.0)])
def test_fp32_value_ranges_far_apart(code, dim, gains):
    """Values whose blocks differ by up to 1e69, four blocks a wave, in every order; with a window some rows see small
    ones only."""
    with KvCase(torch, "f32", code, 4, 2, dim, 32, max_tokens=544) as c:
        for rows in (512, 5):
            gain = np.tile(np.repeat(gains, 32), 4)[:rows, None, None]
            v = (c.draw(rows, 2).astype(np.float64) * gain).astype(np.float32)
            st, info, ws, q, starts = c.append([0], [rows], v=v)
            for window in (0, 20, 150):
                out = c.attend(st, q, ws, 0.125, window)
                natural(c, out, q, [0], [rows], starts, 0.125, window)


@pytest.mark.parametrize("code", CODES)
def test_fp32_value_ranges_far_apart_over_split_keys(code):
    with KvCase(torch, "f32", code, 4, 2, 64, 32, max_seqs=1, max_tokens=2000) as c:
        gains = np.tile(np.repeat([1.0, 1e-39, 1e25, 1e-36, 1e10], 32), 11)[:1700, None, None]
        v = (c.draw(1700, 2).astype(np.float64) * gains).astype(np.float32)
        c.append([0], [1700], v=v)
        st, info, ws, q, starts = c.append([0], [2])
        assert info["workspace_bytes"] > 0
        for window in (0, 60, 500):
            out = c.attend(st, q, ws, 0.125, window)
            natural(c, out, q, [0], [2], starts, 0.125, window)


@pytest.mark.parametrize("code", CODES)
def test_fp32_magnitudes_that_products_of_codes_would_pass(code):
    """Large q on small keys, and values near the largest: scores of about 1 and outputs that fp32 holds, though
    q times a code, or a sum of codes in units of the range, would pass it."""
    with KvCase(torch, "f32", code, 2, 2, 64, 32, rot=0) as c:
        for rows in (100, 3):
            k = (c.draw(rows, 2).astype(np.float64) * 1e-37).astype(np.float32)
            v = (c.rng.uniform(-1, 1, (rows, 2, 64)) * 1e36).astype(np.float32)
            x = (c.draw(rows, 2).astype(np.float64) * 1e36).astype(np.float32)
            st, info, ws, q, starts = c.append([0], [rows], k=k, v=v, q=x)
            for scale in (1.0, -2.0):
                out = c.attend(st, q, ws, scale)
                natural(c, out, q, [0], [rows], starts, scale)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("first,then", [(10, 5), (1, 1), (40, 1), (3, 40), (33, 2)])
def test_a_step_is_appended_again_only_while_its_blocks_end_with_it(code, first, then):
    """An older step's append would leave the tokens behind it in its last block at another range: refused, and the
    cache stays as it was."""
    with KvCase(torch, "f16", code, 4, 2, 64, 32) as c:
        stream = torch.cuda.current_stream()
        x = [[c.draw(n, 2, g) for _ in range(2)] for n, g in ((first, 0.1), (then, 8.0))]
        old, *_ = c.append([0], [first], k=x[0][0], v=x[0][1])
        S.slora_kv_append(c.kv, old, 0, c.device(x[0][0]), c.device(x[0][1]), cos_sin=c.cos_sin, stream=stream)
        new, *_ = c.append([0], [then], k=x[1][0], v=x[1][1])
        for step, (k, v) in ((new, x[1]), (old, x[0])):
            if step is old:
                with pytest.raises(S.SloraError) as e:
                    S.slora_kv_append(c.kv, step, 0, c.device(k), c.device(v), cos_sin=c.cos_sin, stream=stream)
                assert e.value.status == S.SLORA_E_INVAL
            else:
                S.slora_kv_append(c.kv, step, 0, c.device(k), c.device(v), cos_sin=c.cos_sin, stream=stream)
            c.check_read([0])


@pytest.mark.parametrize("code", CODES)
def test_a_step_that_ends_its_block_is_appended_again_at_any_time(code):
    with KvCase(torch, "f16", code, 4, 2, 64, 32) as c:
        k, v = c.draw(64, 2), c.draw(64, 2)
        old, *_ = c.append([0], [64], k=k, v=v)
        c.append([0], [7], 3.0)
        S.slora_kv_append(c.kv, old, 0, c.device(k), c.device(v), cos_sin=c.cos_sin, stream=torch.cuda.current_stream())
        c.check_read([0])
        c.append([0], [7], 5.0)
        c.check_read([0])


def test_steps_built_ahead_are_appended_in_order():
    """Two steps of one block built and uploaded before either runs: the second is refused until the first is stored,
    layer by layer; a dropped sequence begins anew."""
    with KvCase(torch, "f16", 0, 4, 2, 64, 32, n_layers=2) as c:
        stream = torch.cuda.current_stream()
        steps = [c.step([1], [n])[0] for n in (6, 4, 30)]
        x = [[c.device(c.draw(n, 2)) for _ in range(2)] for n in (6, 4, 30)]

        def put(i, layer):
            S.slora_kv_append(c.kv, steps[i], layer, *x[i], cos_sin=c.cos_sin, stream=stream)

        for layer in range(2):
            for i in range(3):
                for late in range(i + 1, 3):
                    with pytest.raises(S.SloraError) as e:
                        put(late, layer)
                    assert e.value.status == S.SLORA_E_INVAL
                put(i, layer)
                c.model.append(1, layer, *(t.cpu().numpy() for t in x[i]))
            c.check_read([1], layer)
        S.slora_kv_drop(c.kv, 1)
        for layer in range(2):
            for w in range(2):
                del c.model.codes[1, layer, w], c.model.range[1, layer, w]
        c.append([1], [9])
        c.check_read([1])


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("size", [2e-45, 1e-44, 1e-42, 1e-39])
def test_fp32_subnormal_ranges(code, size):
    """Ranges of a few units of the smallest number: codes stay in -127 .. 127 and values within their steps.  Rotated
    keys lie between the units, so that the range is rounded from them; single tokens, pieces and older codes coded
    again."""
    with KvCase(torch, "f32", code, 4, 2, 64, 32, max_tokens=128) as c:
        unit = 2.0 ** -149
        for n, gain in ((1, 1.0), (1, 2.0), (29, 1.5), (1, 3.0), (40, 1.0)):
            k, v = ((np.rint(c.rng.uniform(-1, 1, (n, 2, 64)) * gain * size / unit) * unit).astype(np.float32)
                    for _ in range(2))
            c.append([0], [n], k=k, v=v)
        st, _, _ = c.step([0], [c.model.length(0)], True)
        got = [torch.zeros((c.model.length(0), 2, 64), dtype=torch.float32, device="cuda:0") for _ in range(2)]
        S.slora_kv_read(c.kv, st, 0, got[0], got[1], torch.cuda.current_stream())
        for what in range(2):
            want, have = c.model.values(0, 0, what), got[what].cpu().numpy().astype(np.float64)
            # the value is rounded once; half a unit
            assert (np.abs(have - want) <= 2.0 ** -24 * np.abs(want) + unit / 2).all()


def some_heads(c, kv_heads):
    """The model's part for a few kv heads, and their query heads."""
    g = c.n_heads // c.n_kv
    m = O.KvModel(c.desc["code"], g * len(kv_heads), len(kv_heads), c.dim, c.desc["block_tokens"])
    m.codes = {key: x[:, kv_heads] for key, x in c.model.codes.items()}
    m.range = {key: x[:, kv_heads] for key, x in c.model.range.items()}
    return SimpleNamespace(model=m, dim=c.dim, np_dtype=c.np_dtype), [h * g + i for h in kv_heads for i in range(g)]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("seqs,rows,window", [(1, 300, 0), (3, 300, 0), (3, 300, 90), (5, 280, 0), (6, 300, 0)])
def test_prompts_that_fill_the_chip_once_and_more(code, seqs, rows, window):
    """192 to 1152 workgroups of 64 heads of 128: both forms of the prompt kernel, one round of its places and more."""
    with KvCase(torch, "f16", code, 64, 64, 128, 32, max_seqs=6, max_tokens=400) as c:
        ids = list(range(seqs))
        c.append(ids, [17 * i for i in ids])
        st, info, ws, q, starts = c.append(ids, [rows] * seqs)
        assert info["n_prompt_tiles"] == 3 * seqs
        out = c.attend(st, q, ws, 0.09, window)
        part, heads = some_heads(c, [0, 37, 63])
        weight_bits(part, out[:, heads], q[:, heads], ids, [rows] * seqs, starts, 0.09, window)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dim,heads,kv,block", [(128, 8, 2, 64), (256, 8, 2, 32), (128, 100, 1, 32)])
@pytest.mark.parametrize("window", [0, 700, 10])
def test_split_prompt_tiles_of_wide_heads(code, dim, heads, kv, block, window):
    """Keys split over workgroups and joined, also where a window leaves some of them nothing; and a single token whose
    100 query heads share a kv head."""
    with KvCase(torch, "f16", code, heads, kv, dim, block, max_seqs=2, max_tokens=2500) as c:
        rows = [1, 1] if heads == 100 else [30, 25]
        c.append([0, 1], [2400, 1500])
        st, info, ws, q, starts = c.append([0, 1], rows)
        assert info["n_prompt_tiles"] > 2 and info["n_row_tiles"] == 0 and info["workspace_bytes"] > 0
        out = c.attend(st, q, ws, 1 / np.sqrt(dim), window)
        weight_bits(c, out, q, [0, 1], rows, starts, 1 / np.sqrt(dim), window)


@pytest.mark.parametrize("code", CODES)
def test_few_rows_after_a_long_context_fill_the_chip_with_splits(code):
    """64 rows of 4 query heads a kv head after 30000 tokens: near a thousand workgroups, 62 splits a tile."""
    with KvCase(torch, "f16", code, 32, 8, 128, 32, max_seqs=1, max_tokens=30100) as c:
        c.append([0], [30000])
        st, info, ws, q, starts = c.append([0], [64])
        assert 768 < info["n_prompt_tiles"] * 8 <= 1024
        out = c.attend(st, q, ws, 0.09)
        part, heads = some_heads(c, [5])
        weight_bits(part, out[:, heads], q[:, heads], [0], [64], starts, 0.09)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("rows", [48, 130])
def test_prompt_tiles_with_peaked_scores_and_a_row_of_nan(code, rows):
    """Scores of some hundreds of both signs and none; a query row of NaN or infinity is alone.  48 rows of a fresh
    prompt, 130 after 200 tokens with large values."""
    with KvCase(torch, "f16", code, 4, 4, 64, 32) as c:
        if rows == 130:
            c.append([0], [200], 6.0)
        st, info, ws, q, starts = c.append([0], [rows], 6.0, q=c.draw(rows, 4) * np.float16(6))
        assert info["n_prompt_tiles"] and not info["n_row_tiles"]
        for scale in (1.0, -0.5, 0.0):
            clean = c.attend(st, q, ws, scale)
            c.check_attend(clean, q, [0], [rows], starts, scale)
            for bad in (float("nan"), float("inf")):
                x = q.clone()
                x[40, 2, 7] = bad
                out = c.attend(st, x, ws, scale)
                assert torch.isnan(out[40, 2]).all()
                out[40, 2] = clean[40, 2]
                assert torch.equal(out, clean)
