"""A small KV cache on the GPU beside its 64-bit model, driven step by step by the tests."""
import numpy as np

from oracle import kv_oracle as O
from rank_gemm_page_amd import slora as S


def half_step(x, dtype):
    """Half a unit in the last place of x in dtype."""
    with np.errstate(invalid="ignore"):
        return 0.5 * np.spacing(np.abs(x).astype(dtype)).astype(np.float64)


class KvCase:
    def __init__(self, torch, dtype="f16", code=S.SLORA_KV_INT8, n_heads=4, n_kv=2, dim=64, block=32, rot=None,
                 pairs=S.SLORA_KV_HALVES, n_layers=1, max_seqs=4, max_tokens=512, slack=0, extra_pages=3, seed=0,
                 free_order=None, mem=None):
        self.torch, self.rng = torch, np.random.default_rng(seed)
        self.np_dtype = np.float16 if dtype == "f16" else np.float32
        self.tdtype = torch.float16 if dtype == "f16" else torch.float32
        self.n_heads, self.n_kv, self.dim, self.n_layers = n_heads, n_kv, dim, n_layers
        rot = dim if rot is None else rot
        item = np.dtype(self.np_dtype).itemsize
        elems = (2 * block * dim + slack) // item
        blocks = -(-max_tokens // block)
        n_pages = max_seqs * blocks * n_layers * n_kv + extra_pages if mem is None else mem.shape[0]
        # every byte 0xFF: NaN as fp16, fp32 and e4m3, so that whatever is read beside the blocks shows
        self.mem = torch.full((n_pages, elems * item), 255, dtype=torch.uint8, device="cuda:0") if mem is None else mem
        order = self.rng.permutation(n_pages).astype(np.int32) if free_order is None else free_order
        self.pool = S.slora_pool_create(S.SLORA_F16 if dtype == "f16" else S.SLORA_F32, elems, elems, 1, 1, 1,
                                        [self.mem], [n_pages], [order])
        self.desc = dict(cls=0, code=code, n_layers=n_layers, n_heads=n_heads, n_kv_heads=n_kv, head_dim=dim,
                         block_tokens=block, max_seqs=max_seqs, max_tokens=max_tokens, rot_dim=rot, rot_pairs=pairs)
        nbytes = S.slora_kv_device_bytes(self.pool, **self.desc)
        self.dev = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda:0")
        self.kv = S.slora_kv_create(self.pool, self.dev, nbytes, **self.desc)
        cs = O.angles(max_tokens, rot) if rot else None
        self.cos_sin = torch.from_numpy(cs).to("cuda:0") if rot else None
        self.model = O.KvModel(code, n_heads, n_kv, dim, block, rot, pairs, cs)
        self.steps, self.metas = [], []

    def close(self):
        self.torch.cuda.synchronize()
        for s in self.steps:
            S.slora_kv_step_destroy(s)
        S.slora_kv_destroy(self.kv)
        S.slora_pool_destroy(self.pool)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def draw(self, n, heads, gain=1.0):
        x = self.rng.standard_normal((n, heads, self.dim)) * gain
        return x.astype(self.np_dtype)

    def device(self, x):
        return self.torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")

    def step(self, seqs, counts, reread=False, stream=None):
        s = S.slora_kv_build_step(self.kv, seqs, counts, reread)
        self.steps.append(s)
        info = S.slora_kv_step_get_info(s)
        meta = self.torch.empty(max(16, info["meta_bytes"]), dtype=self.torch.uint8, device="cuda:0")
        self.metas.append(meta)
        S.slora_kv_step_upload(s, meta, meta.numel(), stream or self.torch.cuda.current_stream())
        ws = self.torch.full((max(16, info["workspace_bytes"]),), 255, dtype=self.torch.uint8, device="cuda:0")
        self.metas.append(ws)
        return s, info, ws

    def append(self, seqs, counts, gain=1.0, layer=0, k=None, v=None, q=None):
        """A step of drawn rows on the GPU and in the model: (step, info, workspace, rotated q on the GPU, starts)."""
        n = int(sum(counts))
        starts = [self.model.length(s, layer) for s in seqs]
        st, info, ws = self.step(seqs, counts)
        q = self.draw(n, self.n_heads) if q is None else q
        k = self.draw(n, self.n_kv, gain) if k is None else k
        v = self.draw(n, self.n_kv, gain) if v is None else v
        qd, out = self.device(q), self.torch.zeros((n, self.n_heads, self.dim), dtype=self.tdtype, device="cuda:0")
        S.slora_kv_append(self.kv, st, layer, self.device(k), self.device(v), qd, out, cos_sin=self.cos_sin,
                          stream=self.torch.cuda.current_stream())
        at = 0
        for s, c, start in zip(seqs, counts, starts):
            self.model.append(s, layer, k[at:at + c], v[at:at + c])
            self.check_rotated(out[at:at + c], q[at:at + c], start)
            at += c
        return st, info, ws, out, starts

    def check_rotated(self, out, q, start):
        """fp32 rotation: a product and the sum rounded once each, then half a step of the pool dtype (elements behind
        the rotated part are copied)."""
        m, want = self.model, self.model.rotated(q, start)
        bound = O.rotation_error(q, m.cs[start:start + len(q)] if m.rot else None, m.rot, m.pairs)
        bound += half_step(np.abs(want) + bound, self.np_dtype)
        bound[..., m.rot:] = 0
        got = out.cpu().numpy().astype(np.float64)
        assert (np.abs(got - want) <= bound).all(), float(np.max(np.abs(got - want) - bound))

    def check_read(self, seqs, layer=0):
        """Everything the sequences hold."""
        counts = [self.model.length(s, layer) for s in seqs]
        st, _, _ = self.step(seqs, counts, True)
        n = sum(counts)
        k, v = (self.torch.zeros((n, self.n_kv, self.dim), dtype=self.tdtype, device="cuda:0") for _ in range(2))
        S.slora_kv_read(self.kv, st, layer, k, v, self.torch.cuda.current_stream())
        for what, x in ((0, k), (1, v)):
            self.check_values(x, np.concatenate([self.model.values(s, layer, what) for s in seqs]))
        return st, k, v

    def check_values(self, x, want):
        """code * (range / top) takes two fp32 roundings, 2^-24 of the value each, and one to the pool dtype, half a
        step; a code's neighbours are at least 8 fp16 steps away (e4m3: 64), so this pins every code."""
        got = x.cpu().numpy().astype(np.float64)
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        far = np.abs(got - want) > 2.0 ** -23 * np.abs(want) + half_step(want, self.np_dtype)
        assert not far.any(), (int(far.sum()), np.argwhere(far)[:4].tolist())

    def attend(self, st, q, ws, scale, window=0, layer=0, out=None, stream=None):
        out = self.torch.full_like(q, float("nan")) if out is None else out
        S.slora_kv_attend(self.kv, st, layer, q, out, scale, window, ws, ws.numel(),
                          stream or self.torch.cuda.current_stream())
        return out

    def check_attend(self, out, q, seqs, counts, starts, scale, window=0, layer=0):
        """Each output against the model's, with a bound from the arithmetic:
        * a score's error: dim products and sums of fp32 and a handful of roundings behind them, (dim + 8) 2^-24 of
          the sum of their magnitudes, which the exponential turns into that relative error of a weight, twice over
          numerator and denominator; 2^-21 more for the exponential itself;
        * fp16: each weight is rounded once, half a step 2^-11, and those below 2^-14 by up to 2^-25 in units of the
          largest block range that the kernel keeps sums in, at most 2^10 times the block's own;
        * the sums of the keys in fp32: one rounding a key at most;
        * the output is rounded once."""
        out, q = out.cpu().numpy().astype(np.float64), q.cpu().numpy()
        at = 0
        for s, c, start in zip(seqs, counts, starts):
            if c:
                want, weight, reach, spread = self.model.attend(s, layer, q[at:at + c], start, scale, window, start + c)
                got, keys = out[at:at + c], start + c
                bound = weight * (2 * (self.dim + 8) * 2.0 ** -24 * reach + 2.0 ** -20 + (keys + 8) * 2.0 ** -24)
                if self.np_dtype == np.float16:
                    r = self.model.range[s, layer, 1]
                    ratio = min(1024.0, np.nanmax(r) / max(np.nanmin(np.where(r > 0, r, np.inf)), 1e-30))
                    bound += weight * 2.0 ** -11 + spread * 2.0 ** -25 * ratio
                bound += half_step(np.abs(want) + bound, self.np_dtype)
                np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=f"sequence {s}")
                bad = np.abs(got - want) > bound
                bad &= ~np.isnan(want)
                assert not bad.any(), (s, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                                       float(np.nanmax(np.abs(got - want) / bound)))
            at += c
