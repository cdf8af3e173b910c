"""The attention step as a decoder layer runs it: pages assigned, the SVQ linears q|k|v, head norms and rotary
positions into the cache, decode attention written in o's stored column order, the SVQ linear o.  A prompt step
(ragged prompts, padding rows), then decode steps with finished, idle and new requests, each checked against the
oracle on the step's own inputs; then decode steps replayed from one captured graph against the same steps run
eagerly, bit for bit."""
import numpy as np
import pytest

import synth
from oracle import attention as oa
from tests import test_gpu_paged_attention as tpa
from tests import test_gpu_rope_cache as trc
from tests.gpu_util import need_gpu, torch

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu
HID, HQ, HK, D, PAGE = 256, 8, 2, 64, 16


class Layer:
    def __init__(self, n_seqs, width, n_pages, kv):
        shapes = [(HQ * D, HID), (HK * D, HID), (HK * D, HID), (HID, HQ * D)]
        self.W = [svq.SvqWeight.from_synth(synth.make_matrix(61, i, n, k, 6 + i)) for i, (n, k) in enumerate(shapes)]
        g = torch.Generator(device="cuda").manual_seed(1)
        self.gamma, self.qg, self.kg = ((torch.rand(n, generator=g, device="cuda") + 0.5).half() for n in (HID, D, D))
        self.embed = torch.randn((4096, HID), generator=g, device="cuda").half()
        dt = trc.DT[kv]
        k, v = (torch.full((n_pages, PAGE, HK, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
        self.cache, self.rope = svq.KvCache(k, v), svq.Rope.make(D, 10000.0, svq.SVQ_ROPE_YARN, 2.0, 64)
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        self.table = torch.full((n_seqs, width), -1, dtype=torch.int32, device="cuda")
        self.free, self.n_free = i32(np.arange(n_pages)[::-1].copy()), i32([n_pages])
        self.lens, self.new, self.cu = i32([0] * n_seqs), i32([0] * n_seqs), i32([0] * (n_seqs + 1))
        self.order = torch.empty(HQ * D, dtype=torch.int32, device="cuda")
        self.order[self.W[3].perm.long()] = torch.arange(HQ * D, dtype=torch.int32, device="cuda")
        self.o_stored = self.W[3].without_perm()
        need = max(svq.svq_paged_attention_workspace_size(self.cache, HQ),
                   max(svq.svq_linear_gemv_workspace_size(w, m) for w in self.W for m in range(1, 17)),
                   svq.svq_linear_gemv_batched_workspace_size(self.W[:3], 16))
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        svq.svq_workspace_init(self.ws)

    def buffers(self, rows):
        f = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
        return dict(pos=f(rows, dt=torch.int32), slots=f(rows, dt=torch.int32), x=f(rows, HID, dt=torch.float16),
                    q=f(rows, HQ * D), k=f(rows, HK * D), v=f(rows, HK * D),
                    q_rot=f(rows, HQ, D, dt=self.cache.dtype), att=f(rows, HQ * D, dt=torch.float16),
                    att_nat=f(rows, HQ * D, dt=torch.float16), y=f(rows, HID), y_nat=f(rows, HID),
                    h=f(rows, HID, dt=torch.float16))

    def assign(self, b):
        svq.svq_kv_assign(self.lens, self.new, PAGE, self.table, self.free, self.n_free, self.lens, self.n_free, self.cu,
                          b["pos"], b["slots"])

    def to_cache(self, b):
        """From the rows' hidden states to rotated queries and a filled cache."""
        rows = b["h"].shape[0]
        svq.svq_rmsnorm_permute(b["h"], self.gamma, 1e-6, [None], [b["x"]])
        if rows <= 16:
            svq.svq_linear_gemv_batched(self.W[:3], [b["x"]] * 3, [b["q"], b["k"], b["v"]], self.ws)
        else:
            for w, y in zip(self.W, (b["q"], b["k"], b["v"])):
                ws = torch.empty(svq.svq_linear_gemm_workspace_size(w, rows), dtype=torch.uint8, device="cuda")
                svq.svq_linear_gemm(w, b["x"], y, ws)
        self.rot = dict(q=b["q"], k=b["k"], v=b["v"], q_gamma=self.qg, k_gamma=self.kg, eps=1e-6, rope=self.rope,
                        positions=b["pos"], slots=b["slots"], cache=self.cache, q_out=b["q_rot"])

    def attend(self, b):
        self.att = dict(q=b["q_rot"], cache=self.cache, lens=self.lens, block_table=self.table, scale=D ** -0.5,
                        out=b["att"], ws=self.ws, cu_rows=self.cu, order=self.order, lse=None)
        svq.svq_paged_attention(**self.att)
        svq.svq_linear_gemv(self.o_stored, b["att"], b["y"], self.ws)


@pytest.mark.parametrize("kv", ["f16", "bf16"])
def test_prompt_then_decode_steps(kv):
    need_gpu()
    layer = Layer(6, 12, 40, kv)
    rng = np.random.default_rng(3)
    steps = [([37, 5, 0, 64, 1, 16], 128), ([1, 1, 50, -1, 1, 0], 64), ([1, 1, 1, 7, 0, 1], 16), ([1] * 6, 6),
             ([0, 1, 1, 1, -1, 1], 6)]
    for new, rows in steps:
        before = (layer.lens.cpu().numpy(), layer.table.cpu().numpy(), layer.free.cpu().numpy(), int(layer.n_free))
        layer.new.copy_(torch.tensor(new, dtype=torch.int32))
        b = layer.buffers(rows)
        layer.assign(b)
        want = oa.kv_assign(before[0], new, PAGE, before[1], before[2], before[3], rows)
        assert np.array_equal(layer.lens.cpu().numpy(), want["lens_out"]) and int(layer.n_free) == want["n_free_out"]
        assert np.array_equal(b["slots"].cpu().numpy(), want["slots"])
        b["h"].copy_(layer.embed[torch.from_numpy(rng.integers(0, 4096, rows)).cuda()])
        layer.to_cache(b)
        c = layer.cache
        unused = torch.isnan(c.v[:, :, 0, 0])                 # places that no token has had yet
        c.k.nan_to_num_(7.0)                                  # the comparison wants numbers there
        c.v.nan_to_num_(7.0)
        trc.check(layer.rot)
        taken = b["slots"][b["slots"] >= 0].long()
        unused[taken // PAGE, taken % PAGE] = False
        c.k[unused] = float("nan")
        c.v[unused] = float("nan")
        if rows > 16:
            continue                                          # a prompt's own attention is the caller's
        b["att"].fill_(3.0)                                   # rows of a chunk but for its last stay as they are
        b["att_nat"].fill_(3.0)
        layer.attend(b)
        tpa.check(layer.att, run=False)
        svq.svq_paged_attention(**{**layer.att, "out": b["att_nat"], "order": None})
        svq.svq_linear_gemv(layer.W[3], b["att_nat"], b["y_nat"], layer.ws)
        live = int(layer.cu[-1])
        assert torch.equal(b["y"][:live], b["y_nat"][:live])
    assert svq.svq_get_device_status() == svq.SVQ_OK


def test_captured_decode_steps_equal_eager_ones():
    need_gpu()
    out = []
    for captured in (False, True):
        layer = Layer(4, 12, 40, "f16")
        layer.new.copy_(torch.tensor([30, 3, 16, 1], dtype=torch.int32))
        b = layer.buffers(64)
        layer.assign(b)
        b["h"].copy_(layer.embed[:64])
        layer.to_cache(b)
        svq.svq_qk_norm_rope_cache(**layer.rot)
        layer.new.fill_(1)
        d = layer.buffers(4)

        def step():
            layer.assign(d)
            layer.to_cache(d)
            svq.svq_qk_norm_rope_cache(**layer.rot)
            layer.attend(d)

        if captured:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        got = []
        for i in range(20):
            d["h"].copy_(layer.embed[100 + 4 * i:104 + 4 * i])
            g.replay() if captured else step()
            got.append(d["y"].clone())
        out.append(torch.stack(got))
        assert layer.lens.tolist() == [50, 23, 36, 21]
    assert torch.equal(out[0], out[1]) and bool(torch.isfinite(out[0]).all())
    assert svq.svq_get_device_status() == svq.SVQ_OK
