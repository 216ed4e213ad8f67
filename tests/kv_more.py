"""KvCase with attention over a window and the first tokens, and with sequences made of others' tokens in all
layers."""
import numpy as np

from oracle import kv_oracle as O
from rank_gemm_page_amd import slora as S
from tests.kv_case import KvCase, half_step


class MoreCase(KvCase):
    def __init__(self, *a, positions=None, **kw):
        super().__init__(*a, **kw)
        if positions:
            self.model.cs = O.angles(positions, self.model.rot)
            self.cos_sin = self.torch.from_numpy(self.model.cs).to("cuda:0")

    def grow(self, seqs, counts, gain=1.0, attend=None):
        """A step of drawn rows in every layer; attend: (window, sinks) of the attention that follows, checked."""
        n = int(sum(counts))
        st, info, ws = self.step(seqs, counts)
        starts = [self.model.length(s) for s in seqs]
        for layer in range(self.n_layers):
            q, k, v = self.draw(n, self.n_heads), self.draw(n, self.n_kv, gain), self.draw(n, self.n_kv, gain)
            out = self.torch.zeros((n, self.n_heads, self.dim), dtype=self.tdtype, device="cuda:0")
            S.slora_kv_append(self.kv, st, layer, self.device(k), self.device(v), self.device(q), out,
                              cos_sin=self.cos_sin, stream=self.torch.cuda.current_stream())
            at = 0
            for s, m in zip(seqs, counts):
                first = self.model.position(s, layer)
                self.model.append(s, layer, k[at:at + m], v[at:at + m])
                self.check_rotated(out[at:at + m], q[at:at + m], first)
                at += m
            if attend:
                got = self.attend_sinks(st, out, ws, self.dim ** -0.5, *attend, layer=layer)
                self.check_sinks(got, out, seqs, counts, starts, self.dim ** -0.5, *attend, layer=layer)
        return st

    def take(self, made, stream=None):
        """made: (dst, src, ranges) of each."""
        args = [[m[i] for m in made] for i in range(3)]
        n = S.slora_kv_take_bytes(self.kv, *args)
        meta = self.torch.full((n,), 255, dtype=self.torch.uint8, device="cuda:0")
        self.metas.append(meta)
        S.slora_kv_take(self.kv, *args, meta, n, stream or self.torch.cuda.current_stream())
        self.model.take([(d, s, [(0, self.model.length(s))] if r is None else r) for d, s, r in made])
        for d, _, _ in made:
            assert S.slora_kv_length(self.kv, d) == self.model.length(d)
            assert S.slora_kv_position(self.kv, d) == self.model.position(d)

    def drop(self, seq):
        S.slora_kv_drop(self.kv, seq)
        self.model.drop(seq)

    def pages(self, seq):
        """[block, layer, head] page ids."""
        return np.stack([[S.slora_kv_pages(self.kv, seq, layer, h) for h in range(self.n_kv)]
                         for layer in range(self.n_layers)]).transpose(2, 0, 1)

    def free(self):
        return S.slora_free_count(self.pool, 0)

    def check_all(self, seqs):
        """What every sequence holds, in every layer."""
        seqs = [s for s in seqs if self.model.length(s)]
        for layer in range(self.n_layers if seqs else 0):
            self.check_read(seqs, layer)

    def step(self, seqs, counts, reread=False, stream=None, **cut):
        if not cut:
            return super().step(seqs, counts, reread, stream)
        s = S.slora_kv_build_step(self.kv, seqs, counts, reread, **cut)
        return self.uploaded(s, stream)

    def uploaded(self, s, stream=None):
        self.steps.append(s)
        info = S.slora_kv_step_get_info(s)
        meta = self.torch.empty(max(16, info["meta_bytes"]), dtype=self.torch.uint8, device="cuda:0")
        ws = self.torch.full((max(16, info["workspace_bytes"]),), 255, dtype=self.torch.uint8, device="cuda:0")
        self.metas += [meta, ws]
        S.slora_kv_step_upload(s, meta, meta.numel(), stream or self.torch.cuda.current_stream())
        return s, info, ws

    def attend_sinks(self, st, q, ws, scale, window, sinks, layer=0, stream=None):
        out = self.torch.full_like(q, float("nan"))
        S.slora_kv_attend_sinks(self.kv, st, layer, q, out, scale, window, sinks, ws, ws.numel(),
                                stream or self.torch.cuda.current_stream())
        return out

    def check_sinks(self, out, q, seqs, counts, starts, scale, window, sinks, layer=0):
        """Each output against the model's, within the bound that KvCase.check_attend derives: it counts the sequence's
        keys, of which fewer are seen here."""
        out, q = out.cpu().numpy().astype(np.float64), q.cpu().numpy()
        at = 0
        for s, c, start in zip(seqs, counts, starts):
            if c:
                want, weight, reach, spread = self.model.attend(s, layer, q[at:at + c], start, scale, window, start + c,
                                                                sinks)
                got, keys = out[at:at + c], start + c
                bound = weight * (2 * (self.dim + 8) * 2.0 ** -24 * reach + 2.0 ** -20 + (keys + 8) * 2.0 ** -24)
                if self.np_dtype == np.float16:
                    r = self.model.range[s, layer, 1]
                    ratio = min(1024.0, np.nanmax(r) / max(np.nanmin(np.where(r > 0, r, np.inf)), 1e-30))
                    bound += weight * 2.0 ** -11 + spread * 2.0 ** -25 * ratio
                bound += half_step(np.abs(want) + bound, self.np_dtype)
                np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=f"sequence {s}")
                with np.errstate(invalid="ignore"):
                    bad = np.abs(got - want) > bound
                assert not bad.any(), (s, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                                       float(np.nanmax(np.abs(got - want) / bound)))
            at += c
