"""Attention over a window and the first tokens on the CPU: refusals, and how its steps are cut.  No GPU is touched."""
import numpy as np
import pytest

from rank_gemm_page_amd import slora as S
from tests.test_kv_host import Cache, refused

X = 1 << 42
INVAL = S.SLORA_E_INVAL


def test_refusals():
    with Cache() as c:
        s, none = c.step([0], [40]), c.step([0], [0])
        call = lambda *a: S.slora_kv_attend_sinks(c.kv, *a)  # noqa: E731
        ok = (s, 0, X, X, 1.0, 10, 4, X, 1 << 30)
        assert "not uploaded" in refused(INVAL, call, *ok)
        for at, bad in ((1, -1), (1, 2), (2, 0), (3, 0), (2, X + 4), (4, float("inf")), (5, -1), (6, -1)):
            refused(INVAL, call, *ok[:at], bad, *ok[at + 1:])
        assert "not uploaded" in refused(INVAL, call, s, 0, X, X, 1.0, 2**31 - 1, 2**31 - 1, X, 1 << 30)
        call(none, 0, 0, 0, 1.0, 10, 4)
        for cut in (dict(window=-1), dict(sinks=-1), dict(window=3, sinks=-2)):
            refused(INVAL, S.slora_kv_build_step, c.kv, [0], [1], **cut)
        assert S.slora_kv_length(c.kv, 0) == 40
        for cut in (dict(window=2**31 - 1), dict(window=1, sinks=2**31 - 1), dict(sinks=7)):
            S.slora_kv_step_get_info(c.step([0], [1], **cut))
        S.slora_kv_drop(c.kv, 0)
        refused(S.SLORA_E_STALE, call, *ok)


def test_steps_are_cut_for_what_is_seen():
    with Cache(n_pages=4096, max_tokens=20000, n_layers=1) as c:
        c.step([0], [20000])
        tiles = lambda **cut: S.slora_kv_step_get_info(c.step([0], [1], True, **cut))["n_row_tiles"]  # noqa: E731
        whole = tiles()
        assert whole > 20 and tiles(sinks=4) == whole and tiles(window=20000, sinks=4) == whole
        assert tiles(window=2048) < whole and tiles(window=2048) <= 9
        assert tiles(window=1, sinks=4) == 1
        # the sinks count where the window does not reach them
        assert tiles(window=256, sinks=9000) == tiles(window=9256)


def test_model_of_the_first_tokens():
    """The model's mask against all pairs, one by one."""
    from oracle import kv_oracle as O
    rng = np.random.default_rng(0)
    m = O.KvModel(O.INT8, 2, 1, 64, 32)
    m.append(0, 0, rng.standard_normal((50, 1, 64)), rng.standard_normal((50, 1, 64)))
    q = rng.standard_normal((20, 2, 64))
    k, v = (m.values(0, 0, w)[:, 0] for w in (0, 1))
    for window, sinks in ((5, 3), (10, 40), (1, 0), (0, 3)):
        got = m.attend(0, 0, q, 30, 0.2, window, sinks=sinks)[0]
        for t in range(20):
            p = 30 + t
            js = [j for j in range(p + 1) if not window or j > p - window or j < sinks]
            for h in range(2):
                e = np.exp(0.2 * k[js] @ q[t, h])
                np.testing.assert_allclose(got[t, h], (e @ v[js]) / e.sum(), rtol=1e-12)
