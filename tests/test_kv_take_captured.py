"""Sequences that a call changes without a launch of its own, while its stream is captured: on the CPU with HIP calls
stubbed (kv_stub.c), in a child process under the sanitizers."""
import os
import subprocess
import sys

import pytest

from rank_gemm_page_amd import slora as S
from tests.test_kv_host import Cache, refused
from tests.test_kv_take_life import ROOT, STUB, X, Life, stubbed

CAPTURED = 0xC0                                                # the stub's stream that is captured


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


@stubbed
@pytest.mark.parametrize("made", [
    [(0, 0, [(0, 32)])], [(0, 0, [(0, 63)])], [(1, 1, [(0, 33)])], [(0, 0, [])], [(0, 0, None)], [(2, 2, [])],
    [(2, 0, [])], [(1, 1, [(0, 32)]), (2, 0, [])]])
def test_a_captured_stream_leaves_everything_as_it_was(made):
    """Blocks that are let go of, a last block that loses its end, an empty sequence: the call would launch nothing, but a
    launch that the stream's graph holds already may read the pages at every replay."""
    with Cache(n_pages=100, max_seqs=4, max_tokens=300) as c:
        life = Life(c, 4, 32)
        st = life.grow([0, 1], [64, 40])
        pages = [S.slora_kv_pages(c.kv, i).tolist() for i in range(4)]
        assert "captured" in refused(S.SLORA_E_INVAL, life.take, made, CAPTURED)
        life.check(100)
        assert [S.slora_kv_pages(c.kv, i).tolist() for i in range(4)] == pages
        S.slora_kv_append(c.kv, st, 0, X, X, cos_sin=X, n_positions=300)       # the step is not stale
        life.take(made)
        life.check(100)


@stubbed
def test_nothing_to_change_is_not_refused():
    with Cache(n_pages=100, max_seqs=4, max_tokens=300) as c:
        life = Life(c, 4, 32)
        life.grow([0], [64])
        life.take([], CAPTURED)
        life.check(100)
