"""Metadata uploads of moderate size are one launch, with all that they do beside the copy: on the CPU with HIP calls
stubbed (kv_stub.c), in a child process under the sanitizers."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

from rank_gemm_page_amd import slora as S
from tests.test_kv_host import Cache, refused
from tests.test_kv_take_life import META, ROOT, STUB, Life, stubbed


def test_in_a_child_process_with_stubs(tmp_path):
    from rank_gemm_page_amd.build import SANITIZED_LIB_PATH, asan_runtime, build_sanitized
    from tests.test_host_sanitized import _stale
    if STUB:
        pytest.skip("the child process itself")
    if _stale(SANITIZED_LIB_PATH):
        build_sanitized()
    stub = str(tmp_path / "kv_stub.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", stub, os.path.join(ROOT, "tests", "kv_stub.c")], check=True)
    env = dict(os.environ, LD_PRELOAD=asan_runtime() + ":" + stub, SLORA_LIB=SANITIZED_LIB_PATH, SLORA_HIP_STUB=stub,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    cmd = [sys.executable, "-m", "pytest", os.path.abspath(__file__), "-x", "-q", "-p", "no:cacheprovider"]
    res = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and " passed" in out, out[-6000:]


class Launches:
    """Only the first n launches succeed."""

    def __init__(self, n):
        self.stub, self.n = ctypes.CDLL(STUB), n

    def __enter__(self):
        self.stub.kv_stub_fail_launch(self.n)

    def __exit__(self, *a):
        self.stub.kv_stub_fail_launch(-1)


@stubbed
def test_a_step_is_uploaded_by_one_launch():
    """Beside a large product of another stream, every further launch waits for the chip once more."""
    with Cache(n_pages=100, max_seqs=4, max_tokens=300) as c:
        st = c.step([0, 1], [100, 40])
        n = S.slora_kv_step_get_info(st)["meta_bytes"]
        with Launches(0):
            refused(S.SLORA_E_HIP, S.slora_kv_step_upload, st, META, n)
        with Launches(1):
            S.slora_kv_step_upload(st, META, n)
        life = Life(c, 4, 32)
        life.seqs[0], life.seqs[1] = [(i, i) for i in range(100)], [(100 + i, i) for i in range(40)]
        life.births = 140
        life.check(100)


@stubbed
@pytest.mark.parametrize("fused", [0, 1])
def test_segments_are_uploaded_by_one_launch(fused):
    pool = S.slora_pool_create(S.SLORA_F16, 64, 64, 2, 8, 8, [1 << 40], [400])
    try:
        S.slora_pool_set_tuning(pool, S.SLORA_TUNE_FUSED, fused)
        for i in range(3):
            S.slora_load_adapter(pool, i, 8, 0.5)
        seg = S.slora_build_segments(pool, np.array([0, 1, -1, 2, 2, 0, 1], np.int32))
        n = S.slora_segments_get_info(seg)["meta_bytes"]
        with Launches(0):
            refused(S.SLORA_E_HIP, S.slora_segments_upload, seg, META, n)
        with Launches(1):
            S.slora_segments_upload(seg, META, n)
        S.slora_segments_destroy(seg)
    finally:
        S.slora_pool_destroy(pool)
