"""Sequences made of others' tokens on the CPU: refusals before anything is launched.  No GPU is touched."""
import pytest

from rank_gemm_page_amd import slora as S
from tests.test_kv_host import Cache, refused

INVAL = S.SLORA_E_INVAL
X = 1 << 42


def test_tokens_have_to_be_appended():
    with Cache() as c:
        c.step([0], [40])
        for call in (lambda *a: S.slora_kv_take_bytes(c.kv, *a), lambda *a: S.slora_kv_take(c.kv, *a, X, 1 << 20)):
            assert "uploaded" in refused(INVAL, call, [1], [0], [None])
            assert "uploaded" in refused(INVAL, call, [0], [0], [[(0, 1)]])
        assert S.slora_kv_length(c.kv, 0) == 40 and S.slora_free_count(c.pool, 0) == 40 - 8


def test_nothing_taken_is_an_empty_sequence():
    with Cache() as c:
        s = c.step([0], [40])
        S.slora_kv_take(c.kv, [], [], [])
        S.slora_kv_take(c.kv, [1, 2], [0, 2], [[], [(0, 0)]])                  # empty stays empty
        assert S.slora_kv_take_bytes(c.kv, [0], [0], [[(3, 3)]]) == 16
        S.slora_kv_take(c.kv, [0], [0], [[(3, 3), (9, 9)]])
        assert S.slora_kv_length(c.kv, 0) == 0 and S.slora_free_count(c.pool, 0) == 40
        assert [S.slora_kv_position(c.kv, i) for i in (0, 1, -1, 3)] == [0, 0, -1, -1]
        refused(S.SLORA_E_STALE, S.slora_kv_read, c.kv, s, 0, X, X)
        c.step([0], [40])
        assert S.slora_kv_position(c.kv, 0) == 40


@pytest.mark.parametrize("dst,src,ranges", [
    ([3], [0], [None]), ([-1], [0], [None]), ([1], [3], [None]), ([1], [-1], [None]), ([1, 1], [0, 0], [None, None]),
    ([1, 0], [0, 0], [None, []]), ([1, 2], [0, 1], [[], []]), ([2], [0], [[(0, 41)]]), ([2], [0], [[(-1, -1)]]),
    ([2], [0], [[(5, 4)]]), ([2], [0], [[(5, 5), (4, 4)]]), ([0], [2], [[]])])
def test_bad_calls(dst, src, ranges):
    with Cache() as c:
        c.step([0], [40])
        for call in (lambda *a: S.slora_kv_take_bytes(c.kv, *a), lambda *a: S.slora_kv_take(c.kv, *a, X, 1 << 20)):
            refused(INVAL, call, dst, src, ranges)
        assert [S.slora_kv_length(c.kv, i) for i in range(3)] == [40, 0, 0]


def test_binding_checks_its_lists():
    with Cache() as c:
        for args in (([1], [0, 0], [None]), ([1], [0], []), ([[1]], [[0]], [None])):
            with pytest.raises(ValueError):
                S.slora_kv_take(c.kv, *args)
        for bad in ([1, 2, 3], [1, 2], [(1, 2, 3)], [(0.0, 1.5)], [[[0, 1]]]):
            with pytest.raises(ValueError):
                S.slora_kv_take_bytes(c.kv, [1], [0], [bad])


def test_null_arguments():
    import ctypes
    lib = S.lib()
    one = (ctypes.c_int32 * 1)(0)
    with Cache() as c:
        for args in ((None, 1, one, one, one, None), (c.kv, -1, one, one, one, None), (c.kv, 1, None, one, one, None),
                     (c.kv, 1, one, None, one, None), (c.kv, 1, one, one, None, None),
                     (c.kv, 1, one, one, (ctypes.c_int32 * 1)(1), None), (c.kv, 1, one, one, (ctypes.c_int32 * 1)(-1), None)):
            assert lib.slora_kv_take_bytes(*args) == 0
            assert lib.slora_kv_take(*args, None, 0, None) == INVAL
        assert lib.slora_kv_take(c.kv, 0, None, None, None, None, None, 0, None) == 0
        assert lib.slora_kv_position(None, 0) == -1
