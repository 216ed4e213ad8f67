"""The 8-bit paged KV cache on the GPU at the limits of its types and of its order of calls."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

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
            bound = weight * (2 * (c.dim + 8) * 2.0 ** -24 * reach + 2.0 ** -20 + (start + n + 8) * 2.0 ** -24 + 2.0 ** -22)
            bound += spread * 2.0 ** -25 * ratio
            bound += half_step(np.abs(want) + bound, c.np_dtype)
            far = np.abs(out[at:at + n] - want) > bound
            assert not far.any(), (s, int(far.sum()), far.size, np.argwhere(far)[:4].tolist())
        at += n


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dim,heads,kv", [(64, 4, 4), (128, 8, 2), (256, 2, 1)])
@pytest.mark.parametrize("rows,window", [(10, 0), (150, 0), (150, 5)])
def test_weights_of_prompt_tiles_keep_their_bits(code, dim, heads, kv, rows, window):
    """10 rows of up to 4 query heads a kv head take the row tiles, 150 the prompt tiles: the same bound for both.  Small
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
        st, info, ws, q, starts = c.append([0], [20])
        assert info["n_prompt_tiles"] > 1 and info["workspace_bytes"] > 0
        out = c.attend(st, q, ws, 0.125)
        weight_bits(c, out, q, [0], [20], starts, 0.125)
