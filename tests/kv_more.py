"""KvCase with attention over a window and the first tokens, for the tests of those."""
import numpy as np

from rank_gemm_page_amd import slora as S
from tests.kv_case import KvCase, half_step


class MoreCase(KvCase):
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
