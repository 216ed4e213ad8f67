"""One attention layer of a multi-adapter server, as its operators follow each other: the LoRA delta of the q, k and v
projections, append, attention, the delta of the o projection; adapters and KV blocks in one pool, a prompt and decode
steps, against the 64-bit models run on what each operator was given."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import build_from_workload, kv_oracle as O, lora_delta  # noqa: E402
from rank_gemm_page_amd import slora as S  # noqa: E402
from rank_gemm_page_amd.device_workload import DeviceWorkload  # noqa: E402
from synth import generate, small_spec  # noqa: E402
from tests.gates import check_gates  # noqa: E402

pytestmark = pytest.mark.gpu

HEADS, DIM, BLOCK, SEQS = 8, 64, 32, 3


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.lib()


@pytest.mark.parametrize("code", [S.SLORA_KV_INT8, S.SLORA_KV_FP8])
def test_layer_of_a_server(code):
    # pages of 2048 fp16 hold a block of 32 tokens of a head; the attention takes the first 512 columns of q, k and v
    wide = 4 * HEADS * DIM
    w = generate(small_spec("layer", h_in=wide, h_out=wide, n_adapters=4, n_proj=4, proj_x=(0, 0, 0, 1),
                            batch=("explicit", (0, 1, 1)), rank_set=(4, 8, 16), pool=("occ", 9, 10)), 11)
    dw = DeviceWorkload(w, "cuda:0")
    st = build_from_workload(w)
    kv = None
    steps = []
    try:
        S.slora_free_pages(dw.pool, 0, dw.kv[0])        # the pages a full server would hold blocks in
        desc = dict(cls=0, code=code, n_layers=1, n_heads=HEADS, n_kv_heads=HEADS, head_dim=DIM, block_tokens=BLOCK,
                    max_seqs=SEQS, max_tokens=128, rot_dim=DIM, rot_pairs=S.SLORA_KV_HALVES)
        dev = torch.empty(S.slora_kv_device_bytes(dw.pool, **desc), dtype=torch.uint8, device="cuda:0")
        kv = S.slora_kv_create(dw.pool, dev, dev.numel(), **desc)
        cs = O.angles(128, DIM)
        cos_sin = torch.from_numpy(cs).to("cuda:0")
        model = O.KvModel(code, HEADS, HEADS, DIM, BLOCK, DIM, O.HALVES, cs)
        rng = np.random.default_rng(5)
        stream = torch.cuda.current_stream()
        adapters = [0, 3, 1]
        for counts in ([40, 5, 17], [1, 1, 1], [1, 0, 1], [30, 1, 1]):
            rows = int(sum(counts))
            ids = np.repeat(np.array(adapters), counts).astype(np.int32)
            dw.build(ids)
            step = S.slora_kv_build_step(kv, [0, 1, 2], counts)
            steps.append(step)
            info = S.slora_kv_step_get_info(step)
            meta = torch.empty(max(16, info["meta_bytes"]), dtype=torch.uint8, device="cuda:0")
            ws = torch.empty(max(16, info["workspace_bytes"]), dtype=torch.uint8, device="cuda:0")
            S.slora_kv_step_upload(step, meta, meta.numel(), stream)
            x = rng.standard_normal((rows, wide)).astype(np.float16)
            base = [rng.standard_normal((rows, wide)).astype(np.float16) for _ in range(4)]
            xd, ys = torch.from_numpy(x).to("cuda:0"), [torch.from_numpy(b).to("cuda:0") for b in base]
            area = 3 * dw.info["workspace_bytes"]
            dws = torch.empty(area, dtype=torch.uint8, device="cuda:0")
            S.slora_lora_delta_multi(dw.pool, dw.seg, [0, 1, 2], [xd] * 3, ys[:3], dws, area, stream)
            q, k, v = (y.view(rows, 4 * HEADS, DIM)[:, :HEADS] for y in ys[:3])
            rotated = torch.empty((rows, HEADS, DIM), dtype=torch.float16, device="cuda:0")
            S.slora_kv_append(kv, step, 0, k, v, q, rotated, cos_sin=cos_sin, stream=stream)
            o_in = torch.zeros((rows, wide), dtype=torch.float16, device="cuda:0")
            S.slora_kv_attend(kv, step, 0, rotated, o_in.view(rows, 4 * HEADS, DIM)[:, :HEADS], 0.125, 0, ws, ws.numel(), stream)
            S.slora_lora_delta(dw.pool, dw.seg, 3, o_in, ys[3], dws, dw.info["workspace_bytes"], stream)
            torch.cuda.synchronize()
            # each operator against its model on what it was given
            got = [y.cpu().numpy() for y in ys]
            for p, given in ((0, x), (1, x), (2, x), (3, o_in.cpu().numpy())):
                want, sd = lora_delta(st.alloc, st.image, ids, given, base[p], p)
                check_gates(got[p], want, sd, np.float16, f"projection {p}")
            at = 0
            for s, c in enumerate(counts):
                start = model.length(s)
                heads = [g.reshape(rows, 4 * HEADS, DIM)[at:at + c, :HEADS] for g in got[:3]]
                if c:
                    model.append(s, 0, heads[1], heads[2])
                    rq = rotated[at:at + c].cpu().numpy()
                    want = model.rotated(heads[0], start)
                    # a product, the sum (fp32) and the result (fp16) are rounded once each
                    far = np.abs(rq - want) - 2.0 ** -11 * np.abs(want)
                    assert (far <= O.rotation_error(heads[0], cs[start:start + c], DIM, O.HALVES) + 2.0 ** -25).all()
                    want, weight, *_ = model.attend(s, 0, rq, start, 0.125)
                    have = o_in.view(rows, 4 * HEADS, DIM)[at:at + c, :HEADS].cpu().numpy()
                    # each weight and the output are rounded to fp16 once (2^-11 each), fp32 sums in between
                    assert (np.abs(have - want) <= weight * 2.0 ** -10 + 2.0 ** -11 * np.abs(want) + 2.0 ** -24).all()
                at += c
        assert S.slora_kv_length(kv, 0) == 72
    finally:
        torch.cuda.synchronize()
        for s in steps:
            S.slora_kv_step_destroy(s)
        if kv is not None:
            S.slora_kv_destroy(kv)
        dw.close()
