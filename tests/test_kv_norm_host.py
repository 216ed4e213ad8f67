"""Normed appends and tables of angles on the CPU: refusals and the binding's checks.  No GPU is touched."""
import numpy as np
import pytest

from rank_gemm_page_amd import slora as S
from tests.test_kv_host import Cache, refused
from tests.test_kv_limits_host import OnGpu

X = 1 << 42
CS = dict(cos_sin=X, n_positions=100)
INVAL = S.SLORA_E_INVAL


def test_normed_appends_are_checked_like_others():
    with Cache() as c:
        s, r, none = c.step([0, 1], [40, 1]), c.step([0], [40], reread=True), c.step([0], [0])
        ok = dict(q_weight=X, k_weight=X, **CS)
        assert "not uploaded" in refused(INVAL, S.slora_kv_append_norm, c.kv, s, 0, X, X, X, X, **ok)
        assert "not uploaded" in refused(INVAL, S.slora_kv_append_norm, c.kv, s, 0, X, X, **CS)
        assert "reread" in refused(INVAL, S.slora_kv_append_norm, c.kv, r, 0, X, X, **ok)
        refused(INVAL, S.slora_kv_append_norm, c.kv, s, 2, X, X, **ok)
        refused(INVAL, S.slora_kv_append_norm, c.kv, s, 0, 0, X, **ok)
        refused(INVAL, S.slora_kv_append_norm, c.kv, s, 0, X, X, X, None, **ok)
        refused(INVAL, S.slora_kv_append_norm, c.kv, s, 0, X, X, cos_sin=X, n_positions=39)
        S.slora_kv_append_norm(c.kv, none, 0, 0, 0)
        S.slora_kv_drop(c.kv, 0)
        refused(S.SLORA_E_STALE, S.slora_kv_append_norm, c.kv, s, 0, X, X, **ok)


@pytest.mark.parametrize("eps", [0.0, -1e-6, 1e-39, float("inf"), float("nan"), 1e39])
def test_bad_eps(eps):
    with Cache() as c:
        assert "eps" in refused(INVAL, S.slora_kv_append_norm, c.kv, c.step([0], [5]), 0, X, X, eps=eps, **CS)


@pytest.mark.parametrize("bad", [dict(q_weight=X + 2), dict(k_weight=X + 8), dict(per_head=2), dict(per_head=-1)])
def test_bad_weights(bad):
    with Cache() as c:
        refused(INVAL, S.slora_kv_append_norm, c.kv, c.step([0], [5]), 0, X, X, **bad, **CS)


def test_binding_checks_weights():
    torch = pytest.importorskip("torch")
    with Cache() as c:
        s = c.step([0], [5])
        half = lambda *shape: torch.zeros(shape, dtype=torch.float16)  # noqa: E731
        for per_head, q, k in ((False, (64,), (64,)), (True, (4, 64), (2, 64))):
            good = dict(q_weight=OnGpu(half(*q)), k_weight=OnGpu(half(*k)), per_head=per_head)
            assert "not uploaded" in refused(INVAL, S.slora_kv_append_norm, c.kv, s, 0, X, X, **good, **CS)
            for bad in (dict(q_weight=half(*q)), dict(k_weight=OnGpu(half(*k).float())), dict(per_head=not per_head),
                        dict(q_weight=OnGpu(half(32))), dict(k_weight=OnGpu(half(5, 64))),
                        dict(k_weight=OnGpu(half(*k, 2)[..., 0]))):
                with pytest.raises(ValueError):
                    S.slora_kv_append_norm(c.kv, s, 0, X, X, **{**good, **bad}, **CS)


def rotary(c, first=0, n=10, **kw):
    return S.slora_kv_rotary_table(c.kv, kw.pop("cos_sin", X), first, n_positions=n, **kw)


GOOD = dict(scaling="bands", factor=2.0, trained=4096.0, low=1.0, high=4.0)


@pytest.mark.parametrize("bad", [
    dict(cos_sin=0), dict(cos_sin=X + 8), dict(first=-1), dict(n=-1), dict(first=1 << 30, n=1), dict(first=2 << 30, n=0),
    dict(n=(1 << 30) + 1), dict(first=1 << 62, n=1 << 62), dict(scaling=5), dict(scaling=-1), dict(base=1.0),
    dict(base=0.0), dict(base=-2.0), dict(base=float("inf")), dict(base=float("nan")), dict(amplitude=float("inf")),
    dict(amplitude=float("nan")), dict(factor=0.5), dict(factor=float("inf")), dict(factor=float("nan")),
    dict(trained=0.0), dict(trained=float("nan")), dict(trained=float("inf")), dict(low=0.0), dict(low=4.0),
    dict(low=float("nan")), dict(high=float("inf")), dict(high=0.5)])
def test_bad_tables_are_refused(bad):
    with Cache() as c:
        rotary(c, n=0, **GOOD)                           # nothing to write: nothing is launched
        rotary(c, n=0, first=1 << 30, scaling=S.SLORA_KV_ROT_RAMP, factor=1.0, trained=1.0, low=1e-9, high=2.0)
        rotary(c, n=0, factor=float("nan"), trained=-1.0, low=5.0)      # what a scaling does not use is not looked at
        rotary(c, n=0, scaling="linear", factor=3.0, trained=-1.0, low=5.0)
        refused(INVAL, rotary, c, **{**GOOD, **bad})
    with Cache(rot_dim=0) as c:
        assert "rot_dim" in refused(INVAL, rotary, c, n=0)


def test_binding_checks_the_table():
    torch = pytest.importorskip("torch")
    with Cache() as c:
        for bad in (torch.zeros((10, 64)), OnGpu(torch.zeros((10, 32))), OnGpu(torch.zeros((10, 64)).double()),
                    OnGpu(torch.zeros((64, 10)).T)):
            with pytest.raises(ValueError):
                S.slora_kv_rotary_table(c.kv, bad)
        with pytest.raises(ValueError):
            S.slora_kv_rotary_table(c.kv, OnGpu(torch.zeros((10, 64))), n_positions=11)
        S.slora_kv_rotary_table(c.kv, OnGpu(torch.zeros((0, 64))))


def test_model_of_frequencies():
    """The model's scalings against hand-made numbers."""
    from oracle import kv_oracle as O
    f = lambda **kw: O.frequencies(16, **kw).astype(float)  # noqa: E731
    plain = 10000.0 ** (-np.arange(8) / 8)
    np.testing.assert_allclose(f(), plain, rtol=1e-15)
    np.testing.assert_allclose(f(scaling="linear", factor=4.0), plain / 4, rtol=1e-15)
    raised = f(scaling="base", factor=4.0)
    np.testing.assert_allclose(raised, (10000.0 * 4 ** (16 / 14)) ** (-np.arange(8) / 8), rtol=1e-14)
    np.testing.assert_allclose(raised[7], plain[7] / 4, rtol=1e-14)           # the slowest pair: exactly the factor
    bands = f(scaling="bands", factor=4.0, trained=1000.0, low=1.0, high=4.0)
    turns = 1000 * plain / (2 * np.pi)
    assert (turns[:5] > [4, 4, 4, 4, 1]).all() and turns[4] < 4 and (turns[5:] < 1).all()
    np.testing.assert_allclose(bands[:4], plain[:4], rtol=1e-15)
    np.testing.assert_allclose(bands[5:], plain[5:] / 4, rtol=1e-14)
    s = (turns[4] - 1) / 3
    np.testing.assert_allclose(bands[4], plain[4] * (s + (1 - s) / 4), rtol=1e-14)
    ramp = f(scaling="ramp", factor=4.0, trained=1000.0, low=1.0, high=32.0)
    # pairs that would make 32 turns and 1: 16 ln(1000 / 64 pi) / (2 ln 10^4) = 1.39.., 16 ln(1000 / 2 pi) / .. = 4.40..
    r = np.clip((np.arange(8) - 1) / 4, 0, 1)
    np.testing.assert_allclose(ramp, plain * (1 - r + r / 4), rtol=1e-14)
