"""Host side of the KV cache on the CPU: order of appends, operands' types and positions.  No GPU is touched."""
import pytest

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


class OnGpu:
    """A tensor that says it lies on a GPU, at an address that nothing here touches."""

    def __init__(self, x, device=0):
        self.x, self.at = x, device

    def get_device(self):
        return self.at

    def data_ptr(self):
        return X

    def __getattr__(self, name):
        return getattr(self.x, name)


@pytest.mark.parametrize("dtype,right,wrong", [(S.SLORA_F16, "float16", ("float32", "bfloat16")),
                                               (S.SLORA_F32, "float32", ("float16", "float64"))])
def test_binding_takes_the_pools_type_on_its_gpu(dtype, right, wrong):
    """A smaller type than the pool's would be read past its end, a larger one as other numbers."""
    torch = pytest.importorskip("torch")
    with Cache(dtype=dtype, elems=2048) as c:
        s = c.step([0], [5])

        def rows(name, heads=2, device=0):
            x = torch.zeros((5, heads, 64), dtype=getattr(torch, name))
            return OnGpu(x, device) if device is not None else x

        cs = OnGpu(torch.zeros((100, 64)))
        ok = rows(right)
        # what is right gets as far as the library, which says that the step was not uploaded
        assert "not uploaded" in refused(S.SLORA_E_INVAL, S.slora_kv_append, c.kv, s, 0, ok, ok, cos_sin=cs)
        q = rows(right, 4)
        assert "not uploaded" in refused(S.SLORA_E_INVAL, S.slora_kv_attend, c.kv, s, 0, q, q, 1.0)
        assert "not uploaded" in refused(S.SLORA_E_INVAL, S.slora_kv_read, c.kv, s, 0, ok, ok)
        for bad in [rows(t) for t in wrong] + [rows(right, device=None)]:
            for k, v in ((ok, bad), (bad, ok)):
                with pytest.raises(ValueError):
                    S.slora_kv_append(c.kv, s, 0, k, v, cos_sin=cs)
                with pytest.raises(ValueError):
                    S.slora_kv_read(c.kv, s, 0, k, v)
        for bad in [rows(t, 4) for t in wrong] + [rows(right, 4, None)]:
            for q, out in ((rows(right, 4), bad), (bad, rows(right, 4))):
                with pytest.raises(ValueError):
                    S.slora_kv_append(c.kv, s, 0, ok, ok, q, out, cos_sin=cs)
                with pytest.raises(ValueError):
                    S.slora_kv_attend(c.kv, s, 0, q, out, 1.0)
        for bad in (torch.zeros((100, 64)), OnGpu(torch.zeros((100, 64), dtype=torch.float16)),
                    OnGpu(torch.zeros((100, 64), dtype=torch.float64)), OnGpu(torch.zeros((100, 32))),
                    OnGpu(torch.zeros((64, 100)).T)):
            with pytest.raises(ValueError):
                S.slora_kv_append(c.kv, s, 0, ok, ok, cos_sin=bad)
        with pytest.raises(ValueError):
            S.slora_kv_append(c.kv, s, 0, ok, ok, cos_sin=OnGpu(torch.zeros((4, 64))), n_positions=100)
        # rows further apart than the tensor's memory holds
        with pytest.raises(ValueError):
            S.slora_kv_append(c.kv, s, 0, ok, ok, cos_sin=cs, k_stride=192)
        wide = OnGpu(torch.zeros((5, 3, 64), dtype=getattr(torch, right))[:, :2])
        assert "not uploaded" in refused(S.SLORA_E_INVAL, S.slora_kv_append, c.kv, s, 0, wide, ok, cos_sin=cs,
                                         k_stride=192)


def test_binding_checks_the_memory_it_is_given():
    torch = pytest.importorskip("torch")
    with Cache() as c:
        s = c.step([0], [5])
        n = S.slora_kv_step_get_info(s)["meta_bytes"]
        room = torch.zeros(2 * n, dtype=torch.uint8)
        for bad in (room, OnGpu(room[:n - 1]), OnGpu(room[::2])):
            with pytest.raises(ValueError):
                S.slora_kv_step_upload(s, bad, n)
            with pytest.raises(ValueError):
                S.slora_kv_attend(c.kv, s, 0, X, X, 1.0, 0, bad, n)
            with pytest.raises(ValueError):
                S.slora_kv_create(c.pool, bad, n, **c.desc)


def test_binding_knows_another_gpu():
    torch = pytest.importorskip("torch")
    mem = OnGpu(torch.zeros((8, 2048), dtype=torch.float16), 1)
    pool = S.slora_pool_create(S.SLORA_F16, 2048, 2048, 1, 4, 4, [mem], [8])
    try:
        desc = dict(cls=0, n_layers=1, n_heads=2, n_kv_heads=2, head_dim=64, max_seqs=1, max_tokens=32)
        n = S.slora_kv_device_bytes(pool, **desc)
        with pytest.raises(ValueError):
            S.slora_kv_create(pool, OnGpu(torch.zeros(n, dtype=torch.uint8), 0), n, **desc)
        kv = S.slora_kv_create(pool, X, n, **desc)
        s = S.slora_kv_build_step(kv, [0], [5])
        x = torch.zeros((5, 2, 64), dtype=torch.float16)
        with pytest.raises(ValueError):
            S.slora_kv_read(kv, s, 0, OnGpu(x, 1), OnGpu(x, 0))
        assert "not uploaded" in refused(S.SLORA_E_INVAL, S.slora_kv_read, kv, s, 0, OnGpu(x, 1), OnGpu(x, 1))
        S.slora_kv_step_destroy(s)
        S.slora_kv_destroy(kv)
    finally:
        S.slora_pool_destroy(pool)


@pytest.mark.parametrize("dtype", [S.SLORA_F16, S.SLORA_F32])
@pytest.mark.parametrize("heads,before,rows,prompt", [(2, 0, 47, False), (2, 0, 48, True), (2, 10, 95, False),
                                                      (2, 10, 96, True), (8, 100, 23, False), (8, 100, 24, True),
                                                      (64, 100, 1, False), (192, 100, 1, True), (192, 0, 1, True)])
def test_which_rows_take_prompt_tiles(dtype, heads, before, rows, prompt):
    """96 packed rows of a kv head, or 48 of a fresh prompt, in fp16 pools; all others 16 at a time."""
    with Cache(dtype=dtype, elems=4096, n_heads=heads, max_tokens=200, n_pages=200) as c:
        if before:
            c.step([0], [before])
        info = S.slora_kv_step_get_info(c.step([0], [rows]))
        packed = rows * heads // 2
        if prompt and dtype == S.SLORA_F16:
            assert info["n_prompt_tiles"] == -(-packed // 128) and info["n_row_tiles"] == 0
        else:
            assert info["n_prompt_tiles"] == 0 and info["n_row_tiles"] == -(-packed // 16)


def test_the_table_of_angles_holds_the_rows_positions_only():
    """A sequence that gains nothing in a step needs no angles."""
    with Cache() as c:
        c.step([0], [90])
        s = c.step([0, 1], [0, 5])
        assert S.slora_kv_step_get_info(s)["max_len"] == 90
        msg = refused(S.SLORA_E_INVAL, S.slora_kv_append, c.kv, s, 0, X, X, cos_sin=X, n_positions=4)
        assert "position" in msg
        msg = refused(S.SLORA_E_INVAL, S.slora_kv_append, c.kv, s, 0, X, X, cos_sin=X, n_positions=5)
        assert "not uploaded" in msg


@pytest.mark.parametrize("scale", [3e38, -2.5e38, float("inf"), float("nan")])
def test_scales_beyond_fp32_are_refused(scale):
    """The kernels hold scale * log2(e): infinite, every score would be NaN."""
    with Cache() as c:
        s = c.step([0], [5])
        assert "scale" in refused(S.SLORA_E_INVAL, S.slora_kv_attend, c.kv, s, 0, X, X, scale)
        assert "not uploaded" in refused(S.SLORA_E_INVAL, S.slora_kv_attend, c.kv, s, 0, X, X, 2.3e38)
