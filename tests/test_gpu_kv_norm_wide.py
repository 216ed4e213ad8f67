"""Appends of fp32 pools norm and rotate q in 64 bits and round it once, on the GPU against the 64-bit model."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kv_oracle as O  # noqa: E402
from rank_gemm_page_amd import slora as S  # noqa: E402
from tests.kv_case import KvCase, half_step  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.lib()
    print(f"[gpu] {request.node.name}", flush=True)


@pytest.mark.parametrize("dim,rot,pairs,per_head", [
    (64, 64, 0, False), (64, 16, 1, True), (128, 128, 0, True), (128, 64, 1, False), (256, 256, 1, False),
    (256, 128, 0, True), (128, 0, 0, False)])
@pytest.mark.parametrize("gain,eps", [(1.0, 1e-6), (1e-4, 1e-5), (1e30, 2.0 ** -126)])
def test_q_is_rounded_once(dim, rot, pairs, per_head, gain, eps):
    """Of size |a c| + |b s|, v = 2^-53: a lane's 16 squares and sums and 4 sums over lanes (up to 36 v of the mean square,
    whose root halves them), eps, root and its reciprocal (5 v), two products, and a product and a sum of the rotation:
    27 v.  The model has as many: 54 v < 2^-47.  Then half a step of fp32, once."""
    with KvCase(torch, "f32", 0, 6, 3, dim, 32, rot, pairs, max_tokens=320) as c:
        size = lambda x, cs: O.rotation_error(x, cs, rot, pairs) * 2.0 ** 23  # noqa: E731
        for counts in ([1, 0, 1], [37, 1, 130], [1, 1, 1]):
            n, seqs = sum(counts), [0, 1, 3]
            starts = [S.slora_kv_length(c.kv, s) for s in seqs]
            st, _, _ = c.step(seqs, counts)
            q, k, v = c.draw(n, 6, gain), c.draw(n, 3), c.draw(n, 3)
            w = (1 + 0.4 * c.rng.standard_normal((6, dim) if per_head else dim)).astype(np.float32)
            out = torch.full((n, 6, dim), float("nan"), device="cuda:0")
            S.slora_kv_append_norm(c.kv, st, 0, c.device(k), c.device(v), c.device(q), out, c.device(w), None, eps,
                                   per_head, cos_sin=c.cos_sin, stream=torch.cuda.current_stream())
            y = O.normed(q, w, float(np.float32(eps)))
            got, at = out.cpu().numpy().astype(np.float64), 0
            for m, start in zip(counts, starts):
                cs = c.model.cs[start:start + m] if rot else None
                want = O.rotate(y[at:at + m], cs, rot, pairs)
                slack = 2.0 ** -47 * size(y[at:at + m], cs)
                off = np.abs(got[at:at + m] - want) / (half_step(np.abs(want) + slack, np.float32) + slack)
                assert (off <= 1).all(), (counts, float(off.max()), int((off > 1).sum()))
                at += m
