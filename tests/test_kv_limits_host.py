"""Host side of the KV cache on the CPU: order of appends, operands' types and positions.  No GPU is touched."""
from rank_gemm_page_amd import slora as S
from tests.test_kv_host import Cache, refused

X = 1 << 42
CS = dict(cos_sin=X, n_positions=100)


def test_appends_keep_the_order_of_their_tokens():
    """Steps built ahead: one whose block has earlier tokens that no append was launched for is refused."""
    with Cache() as c:
        first, second, third = (c.step([0, 1], n) for n in ([10, 0], [30, 3], [24, 1]))
        for layer in range(2):
            assert "not uploaded" in refused(S.SLORA_E_INVAL, S.slora_kv_append, c.kv, first, layer, X, X, **CS)
            for late in (second, third):
                msg = refused(S.SLORA_E_INVAL, S.slora_kv_append, c.kv, late, layer, X, X, **CS)
                assert "earlier tokens" in msg
        S.slora_kv_drop(c.kv, 0)
        # the sequence begins anew; what only begins blocks depends on nothing before it
        again, whole = c.step([0], [32]), c.step([0], [32])
        for step in (again, whole):
            assert "not uploaded" in refused(S.SLORA_E_INVAL, S.slora_kv_append, c.kv, step, 0, X, X, **CS)
