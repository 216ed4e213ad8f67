"""Appends that norm q and k head by head, and tables of angles, on the GPU against their 64-bit models."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kv_oracle as O  # noqa: E402
from rank_gemm_page_amd import slora as S  # noqa: E402
from tests.kv_case import KvCase, half_step  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.lib()
    print(f"[gpu] {request.node.name}", flush=True)


def append_normed(c, seqs, counts, weights, eps=1e-6, per_head=False, gain=1.0, q=None, k=None, in_place=False):
    """A step of drawn rows, normed, on the GPU and in the model; q is checked."""
    n = int(sum(counts))
    starts = [c.model.length(s) for s in seqs]
    st, _, _ = c.step(seqs, counts)
    q = c.draw(n, c.n_heads, gain) if q is None else q
    k = c.draw(n, c.n_kv, gain) if k is None else k
    v = c.draw(n, c.n_kv, gain)
    wq, wk = weights
    qd = c.device(q)
    out = qd if in_place else torch.full((n, c.n_heads, c.dim), float("nan"), dtype=c.tdtype, device="cuda:0")
    S.slora_kv_append_norm(c.kv, st, 0, c.device(k), c.device(v), qd, out, None if wq is None else c.device(wq),
                           None if wk is None else c.device(wk), eps, per_head, cos_sin=c.cos_sin,
                           stream=torch.cuda.current_stream())
    yq, yk = O.normed(q, wq, eps), O.normed(k, wk, eps)
    at = 0
    for s, m, start in zip(seqs, counts, starts):
        c.model.append(s, 0, yk[at:at + m], v[at:at + m])
        check_q(c, out[at:at + m], yq[at:at + m], start)
        at += m
    return st, out


def check_q(c, out, y, start):
    """Of the normed row y (64 bits), u = 2^-24.  fp16 pools: the squares' sum takes 16 products and sums in a lane and
    four sums over lanes (22 u), the mean, eps, root and reciprocal one rounding each: the root's factor is off by
    at most 22 / 2 + 4 u, and two products follow: 17 u of |y|, in each element of a pair.  fp32 pools: one rounding of
    y.  The rotation adds its two roundings (2 u of |a c| + |b s|), and the output is rounded to the pool's type."""
    m = c.model
    cs = m.cs[start:start + len(y)] if m.rot else None
    want = O.rotate(y, cs, m.rot, m.pairs)
    bound = O.rotation_error(y, cs, m.rot, m.pairs) * (1 + (17 if c.np_dtype == np.float16 else 1) / 2)
    bound += half_step(np.abs(want) + bound, c.np_dtype)
    got = out.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = np.abs(got - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(got - want) / bound)))


def weights_of(c, per_head, rng=None):
    rng = rng or c.rng
    shape = lambda h: (h, c.dim) if per_head else (c.dim,)  # noqa: E731
    return [(1 + 0.4 * rng.standard_normal(shape(h))).astype(c.np_dtype) for h in (c.n_heads, c.n_kv)]


@pytest.mark.parametrize("dtype,code,dim,rot,pairs,per_head", [
    ("f16", 0, 64, 64, 0, False), ("f16", 1, 64, 32, 1, True), ("f16", 0, 128, 128, 1, True),
    ("f16", 1, 128, 64, 0, False), ("f16", 0, 256, 64, 1, False), ("f16", 1, 256, 256, 0, True),
    ("f16", 0, 128, 0, 0, False), ("f32", 0, 64, 64, 1, True), ("f32", 1, 128, 128, 0, False),
    ("f32", 0, 256, 32, 0, False)])
@pytest.mark.parametrize("block", [32, 96])
def test_normed_append_in_pieces_matches(dtype, code, dim, rot, pairs, per_head, block):
    """Single tokens, pieces of a block and whole ones, ranges that grow and that do not; keys and values code for code.
    The norm takes the rows' sizes away, so the weights are other ones from step to step."""
    block = min(block, 32 if dim == 256 else 96)
    with KvCase(torch, dtype, code, 6, 3, dim, block, rot, pairs, max_tokens=320) as c:
        for n, counts in enumerate(([1, 3, 0], [1, 28, 33], [1, 1, 1], [33, 1, 64], [70, 5, 130], [0, 31, 1])):
            w = weights_of(c, per_head)
            append_normed(c, [0, 1, 3], counts, [x * c.np_dtype(1 + n % 3) for x in w], per_head=per_head)
        c.check_read([0, 1, 3])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("given", [(False, False), (True, False), (False, True)])
def test_missing_weights_are_ones(dtype, given):
    with KvCase(torch, dtype, 0, 8, 2, 64, 32) as c:
        for counts in ([40, 1], [1, 7]):
            w = [x if g else None for x, g in zip(weights_of(c, False), given)]
            append_normed(c, [0, 1], counts, w, in_place=True)
        c.check_read([0, 1])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("gain", [1e-4, 300.0])
@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-5, 10.0])
def test_small_and_large_rows_and_eps(dtype, gain, eps):
    """Rows far from the size of eps on either side, and rows of zeros, which stay zeros."""
    with KvCase(torch, dtype, 1, 4, 4, 128, 32) as c:
        for n in (1, 37, 1):
            q, k = c.draw(n, 4, gain), c.draw(n, 4, gain)
            q[0, 1], k[0, 2] = 0, 0
            append_normed(c, [2], [n], weights_of(c, True), eps, True, q=q, k=k)
        c.check_read([2])


def test_fp32_rows_beyond_the_squares_of_fp32():
    """1e30 and 1e-30: the squares pass fp32's range on both sides."""
    with KvCase(torch, "f32", 0, 2, 2, 64, 32) as c:
        for gain in (1e30, 1e-30):
            append_normed(c, [0], [5], weights_of(c, False), 2.0 ** -126, gain=gain)
            append_normed(c, [0], [1], weights_of(c, False), 2.0 ** -126, gain=gain)
        c.check_read([0])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("n", [1, 40])
def test_rows_that_are_not_finite(dtype, n):
    """A NaN or an infinity reaches its own head of q only (by the formula: the infinite elements NaN, the others 0, which
    the rotation joins in pairs), and makes the key block of its head read as NaN."""
    with KvCase(torch, dtype, 0, 4, 2, 64, 32, rot=32) as c:
        q, k = c.draw(n, 4), c.draw(n, 2)
        q[0, 1, 40], q[n - 1, 2, 3] = np.inf, np.nan
        k[n - 1, 0, 50] = -np.inf
        append_normed(c, [1], [n], weights_of(c, False), q=q, k=k)
        c.check_read([1])


@pytest.mark.parametrize("rows,heads,kv", [(1, 64, 8), (300, 64, 8), (2000, 12, 1)])
def test_strided_rows_of_one_projection(rows, heads, kv):
    """q, k and v as parts of one buffer, q in place, many heads a thread; rows behind the step stay as they were."""
    with KvCase(torch, "f16", 0, heads, kv, 128, 32, max_seqs=1, max_tokens=2100) as c:
        x = torch.randn((rows + 3, heads + 2 * kv, 128), generator=torch.Generator("cuda").manual_seed(3),
                        device="cuda:0").half()
        was = x.clone()
        wq, wk = weights_of(c, True)
        st, _, _ = c.step([0], [rows])
        S.slora_kv_append_norm(c.kv, st, 0, x[:, heads:heads + kv], x[:, heads + kv:], x[:, :heads], x[:, :heads],
                               c.device(wq), c.device(wk), 1e-5, True, cos_sin=c.cos_sin,
                               stream=torch.cuda.current_stream())
        host = was.cpu().numpy()[:rows]
        check_q(c, x[:rows, :heads], O.normed(host[:, :heads], wq, 1e-5), 0)
        c.model.append(0, 0, O.normed(host[:, heads:heads + kv], wk, 1e-5), host[:, heads + kv:])
        c.check_read([0])
        assert torch.equal(x[rows:], was[rows:]) and torch.equal(x[:, heads:], was[:, heads:])


def test_captured_and_replayed():
    """A captured append stores what its buffers hold at each replay."""
    with KvCase(torch, "f16", 0, 4, 2, 64, 32) as c:
        wq, wk = (c.device(w) for w in weights_of(c, False))
        st, _, _ = c.step([0, 1], [33, 1])
        q, k, v = (torch.empty((34, h, 64), dtype=torch.float16, device="cuda:0") for h in (4, 2, 2))
        out = torch.empty_like(q)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            S.slora_kv_append_norm(c.kv, st, 0, k, v, q, out, wq, wk, cos_sin=c.cos_sin,
                                   stream=torch.cuda.current_stream())
        for n in range(3):
            # (each time larger by more than the block ranges can have grown, for ranges of other appends only grow)
            hq, hk, hv = c.draw(34, 4), c.draw(34, 2), c.draw(34, 2, 4.0 ** n)
            for x, h in ((q, hq), (k, hk), (v, hv)):
                x.copy_(torch.from_numpy(h))
            graph.replay()
            torch.cuda.synchronize()
            c.model.codes.clear(), c.model.range.clear()
            at = 0
            for s, m in ((0, 33), (1, 1)):
                check_q(c, out[at:at + m], O.normed(hq, wq.cpu().numpy())[at:at + m], 0)
                c.model.append(s, 0, O.normed(hk, wk.cpu().numpy())[at:at + m], hv[at:at + m])
                at += m
            c.check_read([0, 1])


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0, base=500000.0),
            dict(scaling="bands", factor=8.0, base=500000.0, trained=8192.0, low=1.0, high=4.0),
            dict(scaling="ramp", factor=2.5, base=1e6, trained=4096.0, low=1.0, high=32.0, amplitude=1.0916),
            dict(scaling="ramp", factor=4.0, trained=3.0, low=1.0, high=32.0),
            dict(scaling="ramp", factor=4.0, trained=1e9, low=1.0, high=2.0, amplitude=-0.5)]


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("rot", [16, 48, 128, 256])
def test_rotary_table(scaling, rot):
    """Each entry is the 64-bit value rounded to fp32: half a step, and what a 64-bit angle near a zero of the function
    leaves, 2^-50 of the amplitude.  Frequencies (at most 1) are powers, that is exponentials of numbers up to 32, in
    floating point of 64 bits on either side: their arguments are off by up to 32 * 2^-64, the frequencies by that part
    of themselves, the angles of position p by 2 p 2^-59."""
    with KvCase(torch, "f16", 0, 1, 1, 256, 32, rot=rot) as c:
        amplitude = scaling.get("amplitude", 1.0)
        for first, n in ((0, 1), (0, 5), (3, 517), (100000, 64), ((1 << 30) - 200, 200)):
            table = torch.full((n + 1, rot), float("nan"), dtype=torch.float32, device="cuda:0")
            S.slora_kv_rotary_table(c.kv, table[:n], first, stream=torch.cuda.current_stream(), **scaling)
            want = O.rotary_table(first, n, rot, **scaling)
            got = table.cpu().numpy().astype(np.float64)
            bound = half_step(want, np.float32) + (2.0 ** -50 + (first + n) * 2.0 ** -58) * abs(amplitude)
            assert (np.abs(got[:n] - want) <= bound).all(), (first, float(np.max(np.abs(got[:n] - want) - bound)))
            assert np.isnan(got[n]).all()


@pytest.mark.parametrize("positions", [20000, 100001])
def test_long_rotary_table(positions):
    """Tables over the whole range of run lengths a thread takes."""
    with KvCase(torch, "f16", 0, 1, 1, 256, 32, rot=96) as c:
        table = torch.full((positions, 96), float("nan"), dtype=torch.float32, device="cuda:0")
        S.slora_kv_rotary_table(c.kv, table, 7, base=500000.0, stream=torch.cuda.current_stream())
        want = O.rotary_table(7, positions, 96, base=500000.0)
        bound = half_step(want, np.float32) + 2.0 ** -50
        assert (np.abs(table.cpu().numpy() - want) <= bound).all()


def test_a_table_made_here_is_what_appends_take():
    """The table of the tests' own model, to the last bit but where a 64-bit value lies at a rounding border."""
    with KvCase(torch, "f16", 0, 4, 2, 64, 32) as c:
        table = torch.empty_like(c.cos_sin)
        S.slora_kv_rotary_table(c.kv, table, stream=torch.cuda.current_stream())
        assert (table != c.cos_sin).float().mean() < 1e-3
        c.cos_sin = table
        c.model.cs = table.cpu().numpy()
        c.append([0, 1], [50, 3])
        c.check_read([0, 1])
