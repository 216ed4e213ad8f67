"""Handles and addresses at their limits, on the CPU.  No GPU is touched."""
import ctypes

from rank_gemm_page_amd import slora as S
from tests.test_kv_host import Cache, refused

INVAL = S.SLORA_E_INVAL


def test_sequences_are_dropped_by_any_handle():
    """A cache that is not there is refused with a status, and the C interface's plain handle will do."""
    refused(INVAL, S.slora_kv_drop, None, 0)
    with Cache() as c:
        c.step([0], [40])
        S.slora_kv_drop(ctypes.c_void_p(c.kv.value), 0)
        assert S.slora_kv_length(c.kv, 0) == 0


def test_a_table_of_no_positions_has_no_address():
    """An empty tensor's address is NULL; where there are positions, NULL is refused."""
    table = dict(first=5, scaling="linear", factor=2.0)
    with Cache() as c:
        S.slora_kv_rotary_table(c.kv, 0, n_positions=0, **table)
        refused(INVAL, S.slora_kv_rotary_table, c.kv, 0, n_positions=1, **table)
        refused(INVAL, S.slora_kv_rotary_table, c.kv, 8, n_positions=0, **table)
        refused(INVAL, S.slora_kv_rotary_table, c.kv, 0, n_positions=0, first=-1)
        refused(INVAL, S.slora_kv_rotary_table, c.kv, 0, n_positions=0, base=1.0)
