"""The KV cache's operators as a server of long conversations uses them, one after another: a table of scaled angles,
prompts and tokens appended with normed heads, attention over a window and the first tokens, answers that fork from one
prompt, drafts taken back, and conversations shortened to what the window still sees; against the 64-bit model."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kv_oracle as O  # noqa: E402
from rank_gemm_page_amd import slora as S  # noqa: E402
from tests.kv_more import MoreCase  # noqa: E402

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, WINDOW, SINKS, POSITIONS = 8, 2, 128, 96, 4, 900


@pytest.fixture(autouse=True)
def _gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.lib()
    print(f"[gpu] {request.node.name}", flush=True)


class Server(MoreCase):
    """Two layers whose weights differ; the window's layers and those that see everything take turns."""

    def __init__(self, dtype, code, scaling):
        super().__init__(torch, dtype, code, HEADS, KV, DIM, 32, DIM, S.SLORA_KV_HALVES, n_layers=2, max_seqs=6,
                         max_tokens=400, extra_pages=-100, positions=POSITIONS)
        table = torch.empty((POSITIONS, DIM), dtype=torch.float32, device="cuda:0")
        S.slora_kv_rotary_table(self.kv, table, stream=torch.cuda.current_stream(), **scaling)
        want = O.rotary_table(0, POSITIONS, DIM, **scaling)
        assert np.abs(table.cpu().numpy() - want).max() < 2.0 ** -24 * 1.2     # half a step of numbers below 2^1
        self.cos_sin, self.model.cs = table, table.cpu().numpy()
        self.weights = [[(1 + 0.3 * self.rng.standard_normal(DIM)).astype(self.np_dtype) for _ in range(2)]
                        for _ in range(2)]

    def tokens(self, seqs, counts):
        """One step of the model: per layer the normed append and the attention, checked against what was given."""
        n = int(sum(counts))
        whole, _, ws_whole = self.step(seqs, counts)
        cut, _, ws_cut = self.step(seqs, counts, True, window=WINDOW, sinks=SINKS)
        starts = [self.model.length(s) for s in seqs]
        for layer in range(2):
            wq, wk = self.weights[layer]
            # one projection's output, of which q, k and v are parts
            x = self.draw(n, HEADS + 2 * KV, 1.5)
            xd = self.device(x)
            q = torch.empty((n, HEADS, DIM), dtype=self.tdtype, device="cuda:0")
            S.slora_kv_append_norm(self.kv, whole, layer, xd[:, HEADS:HEADS + KV], xd[:, HEADS + KV:], xd[:, :HEADS], q,
                                   self.device(wq), self.device(wk), 1e-6, cos_sin=self.cos_sin,
                                   stream=torch.cuda.current_stream())
            at = 0
            for s, m in zip(seqs, counts):
                self.model.append(s, layer, O.normed(x[at:at + m, HEADS:HEADS + KV], wk), x[at:at + m, HEADS + KV:])
                at += m
            sees = (WINDOW, SINKS) if layer else (0, 0)
            out = self.attend_sinks(cut if layer else whole, q, ws_cut if layer else ws_whole, DIM ** -0.5, *sees,
                                    layer=layer)
            self.check_sinks(out, q, seqs, counts, starts, DIM ** -0.5, *sees, layer=layer)


SCALINGS = [dict(scaling="ramp", base=10000.0, factor=4.0, trained=256.0, low=1.0, high=32.0, amplitude=1.1386),
            dict(scaling="bands", base=500000.0, factor=8.0, trained=200.0, low=1.0, high=4.0)]


@pytest.mark.parametrize("dtype,code,scaling", [("f16", 0, 0), ("f16", 1, 1), ("f32", 0, 1)])
def test_long_conversations(dtype, code, scaling):
    with Server(dtype, code, SCALINGS[scaling]) as c:
        pages = c.mem.shape[0]
        c.tokens([0, 1], [75, 130])                            # two prompts
        c.take([(2, 0, None), (3, 0, None), (4, 1, [(0, 64)])])        # three answers to them, one from halfway
        for _ in range(3):
            c.tokens([0, 1, 2, 3, 4], [1, 1, 1, 1, 1])
        c.tokens([2, 0], [6, 1])                               # a draft of six tokens, of which two hold
        n = c.model.length(2)
        c.take([(2, 2, [(0, n - 4)])])
        c.tokens([2, 3], [1, 20])
        c.drop(0)                                              # the first answer ends; its prompt stays with the others
        for _ in range(4):                                     # the second conversation goes on past what the cache holds
            c.tokens([1, 4], [100, 1])
            n = c.model.length(1)
            if n > 200:
                c.take([(1, 1, [(0, SINKS), (n - WINDOW, n)])])
        assert S.slora_kv_position(c.kv, 1) == 533 and c.model.length(1) < 400
        c.take([(5, 1, [(0, SINKS), (40, 60)]), (0, 3, None)])
        c.tokens([0, 1, 2, 3, 4, 5], [1, 2, 3, 1, 40, 33])
        c.check_all(range(6))
        for i in range(6):
            c.drop(i)
        assert c.free() == pages


def test_a_captured_decode_step_after_the_cache_was_rearranged():
    """A step's launches captured once and replayed over its layers' buffers: sequences that share a prompt's blocks and
    ones that were shortened.  The tokens begin blocks, whose ranges each replay takes anew."""
    with Server("f16", 0, SCALINGS[0]) as c:
        c.tokens([0, 1], [96, 160])
        c.take([(2, 0, None), (1, 1, [(0, SINKS), (36, 160)])])
        st, info, ws = c.step([0, 1, 2], [1, 1, 1], window=WINDOW, sinks=SINKS)
        starts = [c.model.length(s) for s in (0, 1, 2)]
        wq, wk = (c.device(w) for w in c.weights[0])
        x = torch.zeros((3, HEADS + 2 * KV, DIM), dtype=torch.float16, device="cuda:0")
        q, out = (torch.zeros((3, HEADS, DIM), dtype=torch.float16, device="cuda:0") for _ in range(2))
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            stream = torch.cuda.current_stream()
            S.slora_kv_append_norm(c.kv, st, 0, x[:, HEADS:HEADS + KV], x[:, HEADS + KV:], x[:, :HEADS], q, wq, wk,
                                   cos_sin=c.cos_sin, stream=stream)
            S.slora_kv_attend_sinks(c.kv, st, 0, q, out, DIM ** -0.5, WINDOW, SINKS, ws, ws.numel(), stream)
        keep = [{k: v.copy() for k, v in store.items()} for store in (c.model.codes, c.model.range)]
        for n in range(3):
            c.model.codes, c.model.range = ({k: v.copy() for k, v in store.items()} for store in keep)
            host = c.draw(3, HEADS + 2 * KV, 0.5)
            x.copy_(torch.from_numpy(host))
            graph.replay()
            torch.cuda.synchronize()
            for i, s in enumerate((0, 1, 2)):
                c.model.append(s, 0, O.normed(host[i:i + 1, HEADS:HEADS + KV], c.weights[0][1]),
                               host[i:i + 1, HEADS + KV:])
            c.check_read([0, 1, 2])
            c.check_sinks(out, q, [0, 1, 2], [1, 1, 1], starts, DIM ** -0.5, WINDOW, SINKS)
