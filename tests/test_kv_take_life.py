"""The host side of sequences made of others' tokens, under AddressSanitizer and UndefinedBehaviorSanitizer on the CPU:
HIP calls are stubs (kv_stub.c), so that appends count as launched and calls run to their end.  A child process runs this
file's other tests with the stubs and the sanitizers preloaded."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

from rank_gemm_page_amd import slora as S
from tests.test_kv_host import Cache, refused

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STUB = os.environ.get("SLORA_HIP_STUB")
stubbed = pytest.mark.skipif(not STUB, reason="runs in the child process with stubs")
X = 1 << 42
META = 1 << 44


def test_host_side_clean_under_asan_and_ubsan(tmp_path):
    from rank_gemm_page_amd.build import SANITIZED_LIB_PATH, asan_runtime, build_sanitized
    from tests.test_host_sanitized import _stale
    if STUB:
        pytest.skip("the child process itself")
    if _stale(SANITIZED_LIB_PATH):
        build_sanitized()
    stub = str(tmp_path / "kv_stub.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-Wall", "-Werror", "-o", stub,
                    os.path.join(ROOT, "tests", "kv_stub.c")], check=True)
    env = dict(os.environ, LD_PRELOAD=asan_runtime() + ":" + stub, SLORA_LIB=SANITIZED_LIB_PATH, SLORA_HIP_STUB=stub,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    cmd = [sys.executable, "-m", "pytest", os.path.abspath(__file__), "-x", "-q", "-p", "no:cacheprovider"]
    res = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-6000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-6000:]
    assert " passed" in out and " failed" not in out, out[-2000:]


class Life:
    """What the sequences of a cache hold, token by token: (birth, position) of each."""

    def __init__(self, c, seqs, block):
        self.c, self.block, self.seqs, self.births = c, block, [[] for _ in range(seqs)], 0

    def grow(self, seqs, counts, layers=2):
        c = self.c
        st = c.step(seqs, counts)
        S.slora_kv_step_upload(st, META, S.slora_kv_step_get_info(st)["meta_bytes"])
        for layer in range(layers):
            S.slora_kv_append(c.kv, st, layer, X, X, cos_sin=X, n_positions=1 << 30)
        for s, n in zip(seqs, counts):
            first = self.position(s)
            self.seqs[s] += [(self.births + i, first + i) for i in range(n)]
            self.births += n
        return st

    def position(self, s):
        return self.seqs[s][-1][1] + 1 if self.seqs[s] else 0

    def take(self, made, stream=None):
        args = [[m[i] for m in made] for i in range(3)]
        n = S.slora_kv_take_bytes(self.c.kv, *args)
        S.slora_kv_take(self.c.kv, *args, META, n, stream)
        old = [list(s) for s in self.seqs]
        for d, s, ranges in made:
            self.seqs[d] = [t for a, b in ([(0, len(old[s]))] if ranges is None else ranges) for t in old[s][a:b]]

    def check(self, total):
        """Lengths, positions, and whose the pages are: sequences share a block's pages only where their tokens there are
        the same ones and fill it."""
        kv = self.c.kv
        holders = {}
        for i, tokens in enumerate(self.seqs):
            assert S.slora_kv_length(kv, i) == len(tokens) and S.slora_kv_position(kv, i) == self.position(i)
            pages = np.stack([[S.slora_kv_pages(kv, i, layer, h) for h in range(2)] for layer in range(2)])
            assert pages.shape[2] == -(-len(tokens) // self.block)
            for b in range(pages.shape[2]):
                mine = [t[0] for t in tokens[b * self.block:(b + 1) * self.block]]
                assert len(set(pages[:, :, b].reshape(-1).tolist())) == 4
                for p in pages[:, :, b].reshape(-1).tolist():
                    if p in holders:
                        assert holders[p] == mine and len(mine) == self.block
                    holders[p] = mine
        assert S.slora_free_count(self.c.pool, 0) == total - len(holders)


@stubbed
@pytest.mark.parametrize("seed", range(20))
def test_random_life(seed):
    rng = np.random.default_rng(seed)
    total = int(rng.choice([60, 150, 400]))
    with Cache(n_pages=total, max_seqs=6, max_tokens=300) as c:
        life = Life(c, 6, 32)
        done = {"grow": 0, "fork": 0, "keep": 0, "drop": 0}
        for _ in range(120):
            lens = [len(s) for s in life.seqs]
            live, empty = [i for i in range(6) if lens[i]], [i for i in range(6) if not lens[i]]
            kind = rng.choice(["grow", "grow", "fork", "keep", "drop"])
            try:
                if kind == "grow" or not live:
                    seqs = [int(i) for i in rng.permutation(6)[:rng.integers(1, 5)]]
                    life.grow(seqs, [int(min(300 - lens[i], rng.integers(0, 100))) for i in seqs])
                elif kind in ("fork", "keep"):
                    made, used = [], set()
                    targets = empty[:rng.integers(1, 4)] if kind == "fork" else [int(rng.choice(live))]
                    for d in targets:
                        s = int(rng.choice(live)) if kind == "fork" else d
                        cut = np.sort(rng.integers(0, lens[s] + 1, 2 * rng.integers(1, 5)))
                        if rng.random() < 0.4:
                            cut = cut // 32 * 32
                        made.append((d, s, None if rng.random() < 0.2 else
                                     [(int(a), int(b)) for a, b in zip(cut[::2], cut[1::2])]))
                        used.add(d)
                    if not made:
                        continue
                    life.take(made)
                else:
                    i = int(rng.choice(live))
                    S.slora_kv_drop(c.kv, i)
                    life.seqs[i] = []
                done[kind] += 1
            except S.SloraError as e:
                assert e.status == S.SLORA_E_NOMEM, e
            life.check(total)
        assert min(done.values()) > 3, done
        for i in range(6):
            S.slora_kv_drop(c.kv, i)
        assert S.slora_free_count(c.pool, 0) == total


@stubbed
def test_a_failed_launch_changes_nothing():
    stub = ctypes.CDLL(STUB)
    with Cache(n_pages=100, max_seqs=4, max_tokens=300) as c:
        life = Life(c, 4, 32)
        life.grow([0, 1], [100, 40])
        order = S.slora_kv_pages(c.kv, 0).tolist()
        for n in range(3):                                     # the upload's launch, the copies', the rows'
            stub.kv_stub_fail_launch(n)
            for made in ([(0, 0, [(3, 90)]), (2, 1, None)],):
                refused(S.SLORA_E_HIP, life.take, made)
            stub.kv_stub_fail_launch(-1)
            life.check(100)
            assert S.slora_kv_pages(c.kv, 0).tolist() == order
        s = life.grow([3], [1])                                # the next pages are those that it would have had
        assert S.slora_kv_step_get_info(s)["n_new_pages"] == 4
        assert S.slora_kv_pages(c.kv, 3).tolist() == [24]
        life.take([(0, 0, [(3, 90)]), (2, 1, None)])
        life.check(100)


@stubbed
def test_errors_of_others_are_not_taken_for_its_own():
    """What an earlier HIP call of the program's failed with is still to be asked for when a launch succeeds."""
    stub = ctypes.CDLL(STUB)
    with Cache(n_pages=100, max_seqs=4, max_tokens=300) as c:
        life = Life(c, 4, 32)
        stub.kv_stub_leave_error()
        life.grow([0], [100])
        life.take([(1, 0, [(3, 90)])])
        life.check(100)
        stub.kv_stub_fail_launch(-1)


@stubbed
def test_captured_streams_shared_blocks_and_stale_steps():
    with Cache(n_pages=100, max_seqs=4, max_tokens=300) as c:
        life = Life(c, 4, 32)
        st = life.grow([0, 1], [64, 40])
        assert "captured" in refused(S.SLORA_E_INVAL, life.take, [(2, 0, None)], 0xC0)
        life.take([(2, 0, None)])
        again = lambda: S.slora_kv_append(c.kv, st, 0, X, X, cos_sin=X, n_positions=300)  # noqa: E731
        assert "shares" in refused(S.SLORA_E_INVAL, again)
        S.slora_kv_drop(c.kv, 2)
        life.seqs[2] = []
        again()
        life.take([(1, 1, [(0, 39)])])
        refused(S.SLORA_E_STALE, again)
        # half a step: what one layer has not stored cannot be taken
        life.grow([3], [50], layers=1)
        assert "every layer" in refused(S.SLORA_E_INVAL, life.take, [(2, 3, [(0, 1)])])
        life.take([(3, 3, [])])
        life.check(100)


@stubbed
def test_positions_end_at_their_largest():
    """A conversation that is shortened again and again counts its positions on, up to 2^30."""
    with Cache(n_pages=40, max_seqs=1, max_tokens=100) as c:
        life = Life(c, 1, 32)
        life.grow([0], [100])
        for _ in range(50):
            life.take([(0, 0, [(0, 4), (60, 100)])])
            life.grow([0], [56])
        assert S.slora_kv_position(c.kv, 0) == 100 + 50 * 56
        life.check(40)


@stubbed
def test_pages_freed_by_hand_are_not_freed_twice():
    with Cache(n_pages=40, max_seqs=3, max_tokens=100) as c:
        life = Life(c, 3, 32)
        life.grow([0], [70])
        ids = S.slora_kv_pages(c.kv, 0, 1, 1)[1:2]
        S.slora_free_pages(c.pool, 0, ids)
        assert "not an allocated" in refused(S.SLORA_E_INVAL, S.slora_kv_drop, c.kv, 0)
        S.slora_kv_take(c.kv, [0], [0], [[]])
        assert S.slora_free_count(c.pool, 0) == 40
