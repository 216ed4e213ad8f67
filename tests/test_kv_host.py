"""Host side of the KV cache on the CPU: its pages, steps and refusals.  No GPU is touched."""
import os
import subprocess
import sys

import numpy as np
import pytest

from rank_gemm_page_amd import slora as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = [1 << 40]
DESC = dict(cls=0, code=S.SLORA_KV_INT8, n_layers=2, n_heads=4, n_kv_heads=2, head_dim=64, block_tokens=32, max_seqs=3,
            max_tokens=100, rot_dim=64, rot_pairs=S.SLORA_KV_HALVES)


class Cache:
    def __init__(self, n_pages=40, elems=2048, dtype=S.SLORA_F16, free_order=None, **kw):
        self.pool = S.slora_pool_create(dtype, elems, elems, 1, 4, 4, BASE, [n_pages],
                                        None if free_order is None else [free_order])
        self.desc = {**DESC, **kw}
        self.n = S.slora_kv_device_bytes(self.pool, **self.desc)
        self.kv = S.slora_kv_create(self.pool, 1 << 41, self.n, **self.desc)
        self.steps = []

    def step(self, *a, **kw):
        s = S.slora_kv_build_step(self.kv, *a, **kw)
        self.steps.append(s)
        return s

    def __enter__(self):
        return self

    def __exit__(self, *a):
        for s in self.steps:
            S.slora_kv_step_destroy(s)
        if self.kv is not None:
            S.slora_kv_destroy(self.kv)
        S.slora_pool_destroy(self.pool)


def refused(status, fn, *a, **kw):
    with pytest.raises(S.SloraError) as e:
        fn(*a, **kw)
    assert e.value.status == status, e.value
    return str(e.value)


def test_device_bytes_and_default_block():
    with Cache() as c:
        # 3 sequences x 2 layers x 2 heads x 4 blocks of 32 tokens, and two ranges a page
        assert c.n == 3 * 2 * 2 * 4 * 4 + 40 * 8
        # a page of 4096 bytes holds 32 tokens of 64; of 8192, 64 and of 10240 also 64 (whole groups of 32)
        for elems, tokens in ((2048, 32), (4096, 64), (5120, 64)):
            with Cache(elems=elems, block_tokens=0, max_tokens=tokens + 1) as d:
                d.step([0], [tokens + 1])
                assert len(S.slora_kv_pages(d.kv, 0)) == 2


@pytest.mark.parametrize("bad", [
    dict(cls=1), dict(cls=-1), dict(code=2), dict(n_layers=0), dict(n_layers=1025), dict(n_heads=0), dict(n_heads=3),
    dict(n_heads=1026), dict(n_kv_heads=0), dict(head_dim=96), dict(head_dim=128), dict(block_tokens=16),
    dict(block_tokens=64), dict(block_tokens=-32), dict(max_seqs=0), dict(max_tokens=0), dict(max_tokens=(1 << 30) + 1),
    dict(rot_dim=8), dict(rot_dim=80), dict(rot_dim=-16), dict(rot_pairs=2), dict(reserved0=1)])
def test_bad_descriptions_are_refused(bad):
    pool = S.slora_pool_create(S.SLORA_F16, 2048, 2048, 1, 4, 4, BASE, [8])
    try:
        desc = {**DESC, **bad}
        refused(S.SLORA_E_INVAL, S.slora_kv_device_bytes, pool, **desc)
        refused(S.SLORA_E_INVAL, S.slora_kv_create, pool, 1 << 41, 1 << 30, **desc)
    finally:
        S.slora_pool_destroy(pool)


def test_create_checks_its_memory():
    pool = S.slora_pool_create(S.SLORA_F16, 2048, 2048, 1, 4, 4, BASE, [8])
    try:
        n = S.slora_kv_device_bytes(pool, **DESC)
        refused(S.SLORA_E_INVAL, S.slora_kv_create, pool, 0, n, **DESC)
        refused(S.SLORA_E_INVAL, S.slora_kv_create, pool, (1 << 41) + 8, n, **DESC)
        refused(S.SLORA_E_NOMEM, S.slora_kv_create, pool, 1 << 41, n - 1, **DESC)
    finally:
        S.slora_pool_destroy(pool)


def test_pages_grow_with_the_tokens_and_come_from_the_pool_in_order():
    order = np.random.default_rng(3).permutation(40).astype(np.int32)
    with Cache(free_order=order) as c:
        c.step([1, 0], [33, 1])
        # sequence 1: two blocks, sequence 0: one; a block takes layers x heads pages, head by head within a layer
        want = order[:12].reshape(3, 2, 2)
        for layer in range(2):
            for head in range(2):
                assert S.slora_kv_pages(c.kv, 1, layer, head).tolist() == want[:2, layer, head].tolist()
                assert S.slora_kv_pages(c.kv, 0, layer, head).tolist() == want[2:, layer, head].tolist()
        assert S.slora_free_count(c.pool, 0) == 40 - 12
        s = c.step([0, 2, 1], [31, 0, 31])              # both fill up what they have, sequence 2 stays empty
        info = S.slora_kv_step_get_info(s)
        assert S.slora_free_count(c.pool, 0) == 40 - 12 and info["n_new_pages"] == 0
        assert info["n_rows"] == 62 and info["n_seqs"] == 3 and info["max_len"] == 64
        assert info["n_blocks"] == 2                    # the rows end inside one block each
        assert [S.slora_kv_length(c.kv, i) for i in range(3)] == [32, 64, 0]
        assert S.slora_kv_length(c.kv, 3) == -1 and S.slora_kv_length(c.kv, -1) == -1
        c.step([1], [1])
        assert len(S.slora_kv_pages(c.kv, 1)) == 3 and S.slora_free_count(c.pool, 0) == 40 - 16


def test_a_step_takes_all_its_pages_or_none():
    with Cache(n_pages=11) as c:
        c.step([0], [33])                               # 8 of 11 pages
        msg = refused(S.SLORA_E_NOMEM, S.slora_kv_build_step, c.kv, [0, 1], [1, 1])
        assert "free pages" in msg
        assert S.slora_free_count(c.pool, 0) == 3 and S.slora_kv_length(c.kv, 0) == 33 and S.slora_kv_length(c.kv, 1) == 0
        c.step([0], [1])                                # no new page is needed


def test_bad_steps_are_refused():
    with Cache() as c:
        c.step([0], [10])
        for seqs, counts, reread in (([3], [1], False), ([-1], [1], False), ([0, 0], [1, 1], False), ([0], [-1], False),
                                     ([0], [91], False), ([0], [11], True), ([1], [1], True)):
            refused(S.SLORA_E_INVAL, S.slora_kv_build_step, c.kv, seqs, counts, reread)
        assert S.slora_kv_length(c.kv, 0) == 10
        with pytest.raises(ValueError):
            S.slora_kv_build_step(c.kv, [0, 1], [1])
        refused(S.SLORA_E_INVAL, S.slora_kv_pages, c.kv, 0, 2, 0)
        refused(S.SLORA_E_INVAL, S.slora_kv_pages, c.kv, 0, 0, 2)
        refused(S.SLORA_E_INVAL, S.slora_kv_drop, c.kv, 3)


def test_a_step_too_large_for_a_launch_is_refused():
    with Cache(n_pages=1 << 20, n_layers=1, n_heads=64, n_kv_heads=64, max_seqs=1, max_tokens=1 << 26) as c:
        msg = refused(S.SLORA_E_INVAL, S.slora_kv_build_step, c.kv, [0], [1 << 24])
        assert "too large" in msg and S.slora_kv_length(c.kv, 0) == 0
        assert S.slora_free_count(c.pool, 0) == 1 << 20


def test_drop_returns_pages_and_makes_steps_stale():
    with Cache() as c:
        s = c.step([0, 1], [40, 40])
        S.slora_kv_drop(c.kv, 0)
        assert S.slora_free_count(c.pool, 0) == 40 - 8 and S.slora_kv_length(c.kv, 0) == 0
        S.slora_kv_drop(c.kv, 2)                        # an empty sequence may be dropped
        info = S.slora_kv_step_get_info(s)
        refused(S.SLORA_E_STALE, S.slora_kv_step_upload, s, 1 << 42, info["meta_bytes"])
        refused(S.SLORA_E_STALE, S.slora_kv_read, c.kv, s, 0, 1 << 42, 1 << 42)
        refused(S.SLORA_E_STALE, S.slora_kv_attend, c.kv, s, 0, 1 << 42, 1 << 42, 1.0)
        refused(S.SLORA_E_STALE, S.slora_kv_append, c.kv, s, 0, 1 << 42, 1 << 42, n_positions=100)


def test_destroy_returns_every_page():
    with Cache() as c:
        c.step([0, 1, 2], [1, 33, 64])
        S.slora_kv_destroy(c.kv)
        c.kv = None
        assert S.slora_free_count(c.pool, 0) == 40


def test_bad_launches_are_refused():
    x = 1 << 42
    with Cache() as c, Cache() as other:
        s = c.step([0, 1], [40, 1])
        r = c.step([0], [40], reread=True)
        none = c.step([0, 1], [0, 0])
        info = S.slora_kv_step_get_info(s)
        cs = dict(cos_sin=x, n_positions=100)
        inval = S.SLORA_E_INVAL
        # not uploaded
        assert "not uploaded" in refused(inval, S.slora_kv_append, c.kv, s, 0, x, x, **cs)
        assert "not uploaded" in refused(inval, S.slora_kv_attend, c.kv, s, 0, x, x, 1.0, 0, x, 1 << 30)
        assert "not uploaded" in refused(inval, S.slora_kv_read, c.kv, s, 0, x, x)
        refused(inval, S.slora_kv_step_upload, s, 0, info["meta_bytes"])
        refused(inval, S.slora_kv_step_upload, s, x + 8, info["meta_bytes"])
        refused(S.SLORA_E_NOMEM, S.slora_kv_step_upload, s, x, info["meta_bytes"] - 1)
        for layer in (-1, 2):
            refused(inval, S.slora_kv_append, c.kv, s, layer, x, x, **cs)
            refused(inval, S.slora_kv_attend, c.kv, s, layer, x, x, 1.0, 0, x, 1 << 30)
            refused(inval, S.slora_kv_read, c.kv, s, layer, x, x)
        assert "another cache" in refused(inval, S.slora_kv_append, other.kv, s, 0, x, x, **cs)
        assert "reread" in refused(inval, S.slora_kv_append, c.kv, r, 0, x, x, **cs)
        # operands
        refused(inval, S.slora_kv_append, c.kv, s, 0, 0, x, **cs)
        refused(inval, S.slora_kv_append, c.kv, s, 0, x, 0, **cs)
        refused(inval, S.slora_kv_append, c.kv, s, 0, x, x, x, None, **cs)
        refused(inval, S.slora_kv_append, c.kv, s, 0, x, x, None, x, **cs)
        refused(inval, S.slora_kv_append, c.kv, s, 0, x + 2, x, **cs)
        refused(inval, S.slora_kv_append, c.kv, s, 0, x, x, k_stride=120, **cs)
        refused(inval, S.slora_kv_append, c.kv, s, 0, x, x, v_stride=132, **cs)
        refused(inval, S.slora_kv_append, c.kv, s, 0, x, x, x, x, q_stride=256, q_out_stride=512, **cs)
        refused(inval, S.slora_kv_append, c.kv, s, 0, x, x, n_positions=100)
        refused(inval, S.slora_kv_append, c.kv, s, 0, x, x, cos_sin=x + 4, n_positions=100)
        assert "position" in refused(inval, S.slora_kv_append, c.kv, s, 0, x, x, cos_sin=x, n_positions=39)
        for bad in (float("inf"), float("nan")):
            refused(inval, S.slora_kv_attend, c.kv, s, 0, x, x, bad, 0, x, 1 << 30)
        refused(inval, S.slora_kv_attend, c.kv, s, 0, x, x, 1.0, -1, x, 1 << 30)
        refused(inval, S.slora_kv_attend, c.kv, s, 0, 0, x, 1.0, 0, x, 1 << 30)
        refused(inval, S.slora_kv_attend, c.kv, s, 0, x, x, 1.0, 0, x, 1 << 30, out_stride=255)
        refused(inval, S.slora_kv_read, c.kv, s, 0, 0, 0)
        refused(inval, S.slora_kv_read, c.kv, s, 0, x, x, v_stride=64)
        # a step without rows launches nothing
        S.slora_kv_append(c.kv, none, 0, 0, 0)
        S.slora_kv_attend(c.kv, none, 0, 0, 0, 1.0)
        S.slora_kv_read(c.kv, none, 0, x, x)


def test_a_split_step_asks_for_its_workspace():
    x = 1 << 42
    with Cache(n_pages=4096, max_tokens=20000, n_layers=1) as c:
        s = c.step([0], [20000])
        del s
        one = c.step([0], [1], reread=True)
        info = S.slora_kv_step_get_info(one)
        assert info["workspace_bytes"] > 0 and info["n_row_tiles"] > 1
        refused(S.SLORA_E_INVAL, S.slora_kv_attend, c.kv, one, 0, x, x, 1.0)
        refused(S.SLORA_E_INVAL, S.slora_kv_attend, c.kv, one, 0, x, x, 1.0, 0, x + 4, 1 << 30)
        refused(S.SLORA_E_NOMEM, S.slora_kv_attend, c.kv, one, 0, x, x, 1.0, 0, x, info["workspace_bytes"] - 1)


def test_binding_checks_shapes():
    import torch
    with Cache() as c:
        s = c.step([0], [5])
        ok = torch.zeros((5, 2, 64), dtype=torch.float16)
        for bad in (ok[:4], torch.zeros((5, 4, 64), dtype=torch.float16), torch.zeros((5, 2, 32), dtype=torch.float16),
                    ok.transpose(0, 1).contiguous().transpose(0, 1), torch.zeros((5, 2, 128), dtype=torch.float16)[..., ::2]):
            with pytest.raises(ValueError):
                S.slora_kv_append(c.kv, s, 0, ok, bad, cos_sin=1 << 42, n_positions=100)
        with pytest.raises(ValueError):
            S.slora_kv_append(c.kv, s, 0, ok, ok, cos_sin=torch.zeros((100, 32)))


@pytest.mark.parametrize("seed", range(4))
def test_random_sequences_never_share_a_page(seed):
    rng = np.random.default_rng(seed)
    with Cache(n_pages=400, max_seqs=6, max_tokens=400) as c:
        lens = [0] * 6
        for _ in range(40):
            seqs = rng.permutation(6)[:rng.integers(1, 7)]
            counts = rng.integers(0, 60, seqs.size)
            try:
                c.step(seqs, counts)
                for i, n in zip(seqs, counts):
                    lens[i] += int(n)
            except S.SloraError as e:
                assert e.status in (S.SLORA_E_NOMEM, S.SLORA_E_INVAL)
                i = int(rng.integers(0, 6))
                S.slora_kv_drop(c.kv, i)
                lens[i] = 0
            assert [S.slora_kv_length(c.kv, i) for i in range(6)] == lens
            pages = [p for i in range(6) for layer in range(2) for h in range(2)
                     for p in S.slora_kv_pages(c.kv, i, layer, h).tolist()]
            assert len(set(pages)) == len(pages) == sum(-(-n // 32) for n in lens) * 4
            assert S.slora_free_count(c.pool, 0) == 400 - len(pages)


def test_kernels_keep_matrix_instructions_in_uniform_flow(tmp_path):
    from rank_gemm_page_amd import build
    asm = build.device_assembly(str(tmp_path), "slora_kv.hip")
    with open(asm) as f:
        text = f.read()
    assert text.count("v_mfma") > 0 and "scratch_store" not in text
    assert build.masked_mfma_lines(asm) == []


def test_host_side_clean_under_asan_and_ubsan():
    from rank_gemm_page_amd.build import SANITIZED_LIB_PATH, asan_runtime, build_sanitized
    from tests.test_host_sanitized import _stale
    if os.environ.get("SLORA_LIB"):
        pytest.skip("the sanitized run itself")
    if _stale(SANITIZED_LIB_PATH):
        build_sanitized()
    env = dict(os.environ, LD_PRELOAD=asan_runtime(), SLORA_LIB=SANITIZED_LIB_PATH,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    cmd = [sys.executable, "-m", "pytest", os.path.abspath(__file__), "-x", "-q", "-p", "no:cacheprovider",
           "-k", "not binding and not matrix and not asan"]
    res = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-6000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-6000:]
