"""Long tables of angles, whose workgroups multiply a few positions' turns together, on the GPU against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kv_oracle as O  # noqa: E402
from rank_gemm_page_amd import slora as S  # noqa: E402
from tests.kv_case import KvCase, half_step  # noqa: E402

pytestmark = pytest.mark.gpu

FAR = 1 << 30
PLAIN, LINEAR = dict(), dict(scaling="linear", factor=4.0, amplitude=-0.5)
RAISED = dict(scaling="base", factor=8.0, base=500000.0, amplitude=3.0)
BANDS = dict(scaling="bands", factor=8.0, base=500000.0, trained=8192.0, low=1.0, high=4.0, amplitude=1.2)
RAMP = dict(scaling="ramp", factor=2.5, base=1e6, trained=4096.0, low=1.0, high=32.0, amplitude=1.0916)


@pytest.fixture(autouse=True)
def _gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.lib()
    print(f"[gpu] {request.node.name}", flush=True)


# (rot, positions, bases of a workgroup): positions / (256 / (rot / 2) * 4 * 1024), rounded down, in 1 .. 16
@pytest.mark.parametrize("rot,n,bases", [
    (256, 16384 + 7, 2), (256, 65536 + 129, 8), (256, 131072 + 1, 16), (256, 300001, 16), (16, 262144 + 77, 2),
    (16, 2097152 + 3, 16), (48, 327680 + 41, 8), (48, 655360 + 639, 16), (128, 131072 + 15, 8), (128, 262144, 16)])
@pytest.mark.parametrize("scaling,first", [(PLAIN, 0), (LINEAR, 12345), (RAISED, None), (BANDS, 1), (RAMP, None)])
def test_every_entry(rot, n, bases, scaling, first):
    """first None: as far as positions go.  u = 2^-53: a turn is off by its rounding (2 u) and its sine's and cosine's
    (2 u); an entry is a product of two of them (1 u for the amplitude, 2 u for the product): 11 u < 2^-49 of the
    amplitude.  Frequencies and their model leave (first + n) 2^-58 (test_rotary_table).  All of it once more in 64 bits
    without more care, which leaves half a step of frequencies and angles: 2^-52 of the position."""
    assert min(16, n // (256 // (rot // 2) * 4 * 1024)) == bases
    first = FAR - n if first is None else first
    amplitude = abs(scaling.get("amplitude", 1.0))
    with KvCase(torch, "f16", 0, 1, 1, 256, 32, rot=rot) as c:
        table = torch.full((n + 1, rot), float("nan"), dtype=torch.float32, device="cuda:0")
        S.slora_kv_rotary_table(c.kv, table[:n], first, stream=torch.cuda.current_stream(), **scaling)
        assert torch.isnan(table[n]).all()
        kw = {k: v for k, v in scaling.items() if k != "amplitude"}
        f = O.frequencies(rot, **kw)
        # some whole workgroups at either end, and rows between them
        rows = np.unique(np.r_[0:min(n, 2200), n - 700:n, c.rng.integers(0, n, 700)])
        angle = (rows.astype(np.longdouble) + first)[:, None] * f
        want = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float64) * scaling.get("amplitude", 1.0)
        got = table[torch.from_numpy(rows).cuda()].cpu().numpy().astype(np.float64)
        slack = (2.0 ** -49 + (first + n) * 2.0 ** -58) * amplitude
        bound = half_step(np.abs(want) + slack, np.float32) + slack
        off = np.abs(got - want) / bound
        assert (off <= 1).all(), (float(off.max()), rows[np.argwhere(off > 1)[:4, 0]].tolist())
        slack = (2.0 ** -49 + (first + n) * 2.0 ** -52) * amplitude
        wide = torch.from_numpy(f.astype(np.float64)).cuda()
        for r in range(0, n, 1 << 17):
            part = table[r:min(n, r + (1 << 17))].double()
            a = (torch.arange(r, r + len(part), device="cuda:0", dtype=torch.float64) + first)[:, None] * wide
            want = torch.cat([torch.cos(a), torch.sin(a)], 1) * scaling.get("amplitude", 1.0)
            assert ((part - want).abs() <= 2.0 ** -24 * amplitude + slack).all(), r
