"""GPU parity of svq_qk_norm_rope_cache with the fp64 oracle.

Bar for each entry: half a step of the output type at the exact value (plus half a subnormal step) and 2e-6 of
factor times the length of the entry's pair.  Where the 2e-6 comes from, in units of u = 2^-24: the mean of
squares is a chain of at most 5 fused additions per lane and 5 in the butterfly (10 u; the product with 1/D
is exact) and eps one more, halved by the root: 5.5 u.  The reciprocal root adds 1 u; gamma, factor, the two
products and the sum 5 u.  The angle is exact to 3 u pi (its rounding to fp32 in turns: at most 2^-26 turns), sincospi adds 2 ulp (4 u):
cosine and sine are off by at most 13.5 u each, which turns the pair by sqrt(2) * 13.5 u = 19 u of its length.
Together 30.5 u; the bar of 34 u leaves the rest to the second-order terms."""
import numpy as np
import pytest

from oracle import attention as oa
from tests.gpu_util import need_gpu, torch

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu
REL = 34 * 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def f64(t):
    return t.detach().float().cpu().double().numpy()


def pools(pages, page, heads, dim, kv, layout="nhd", fill=7.0):
    if layout == "hnd":
        k, v = (torch.full((pages, heads, page, dim), fill, dtype=DT[kv], device="cuda").transpose(1, 2) for _ in range(2))
    elif layout == "both":                                   # k and v interleaved in one pool
        both = torch.full((pages, page, heads, 2, dim), fill, dtype=DT[kv], device="cuda")
        k, v = both[:, :, :, 0], both[:, :, :, 1]
    else:
        k, v = (torch.full((pages, page, heads, dim), fill, dtype=DT[kv], device="cuda") for _ in range(2))
    return svq.KvCache(k, v)


def case(seed, M, hq, hk, dim, rot, x="f32", kv="f16", norm=True, interleaved=False, layout="nhd", page=16, far=5000,
         factor=1.0, fused=True, base=1e6, pads=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wq, wk = hq * dim, hk * dim
    if fused:
        x_all = torch.randn((M, wq + 2 * wk + 8), generator=g, device="cuda").mul_(2).to(DT[x])
        q, k, v = x_all[:, :wq], x_all[:, wq:wq + wk], x_all[:, wq + wk:wq + 2 * wk]
    else:
        q, k, v = (torch.randn((M, w), generator=g, device="cuda").to(DT[x]) for w in (wq, wk, wk))
    gam = [(torch.rand(dim, generator=g, device="cuda") * 2 - 0.5).half() if norm else None for _ in range(2)]
    c = pools((M + page - 1) // page + 1, page, hk, dim, kv, layout)
    slots = torch.randperm(c.n_pages * page, generator=g, device="cuda")[:M].to(torch.int32)
    if pads:
        slots[torch.randperm(M, generator=g, device="cuda")[:pads]] = -1
    pos = torch.randint(0, far, (M,), generator=g, device="cuda", dtype=torch.int32)
    freq = svq.svq_rope_frequencies(rot, base)[0]
    r = svq.Rope(torch.from_numpy(freq).cuda(), interleaved, factor)
    return dict(q=q, k=k, v=v, q_gamma=gam[0], k_gamma=gam[1], eps=1e-6, rope=r, positions=pos, slots=slots, cache=c,
                q_out=torch.full((M, hq, dim), 9.0, dtype=DT[kv], device="cuda"))


def check(a, rows=None):
    """Runs the call and compares all of q_out and both pools (written and untouched entries)."""
    c, r = a["cache"], a["rope"]
    D, page, kv = c.head_dim, c.page_size, "f16" if c.dtype is torch.float16 else "bf16"
    eps = torch.finfo(c.dtype).eps
    before = [f64(t) for t in (a["q_out"], c.k, c.v)]
    svq.svq_qk_norm_rope_cache(**a)
    torch.cuda.synchronize()
    got = [f64(t) for t in (a["q_out"], c.k, c.v)]
    want = [b.copy() for b in before]
    tol = [np.zeros_like(b) for b in before]
    freq = r.inv_freq.cpu().numpy()
    pos, slots = a["positions"].cpu().numpy(), a["slots"].cpu().numpy()
    for m in range(len(slots)):
        if slots[m] < 0 or slots[m] >= c.n_pages * page:
            continue
        p, t = divmod(int(slots[m]), page)
        for i, (x, gamma) in enumerate(((a["q"], a["q_gamma"]), (a["k"], a["k_gamma"]), (a["v"], None))):
            heads = f64(x[m]).reshape(-1, D)
            if i == 2:
                want[2][p, t], tol[2][p, t] = heads, eps / 2 * np.abs(heads) + TINY[kv] / 2
                continue
            n = oa.head_norm(heads, None if gamma is None else f64(gamma), np.float32(a["eps"]))
            for h in range(len(heads)):
                y = oa.rotate(n[h], pos[m], freq, r.factor, r.interleaved)
                size = oa.pair_size(n[h], r.rot_dim, r.interleaved)
                size[:r.rot_dim] *= abs(r.factor)
                at = (m, h) if i == 0 else (p, t, h)
                want[i][at] = y
                tol[i][at] = eps / 2 * (np.abs(y) + REL * size) + REL * size + TINY[kv] / 2
    for i, name in enumerate(("q", "k", "v")):
        off = np.abs(got[i] - want[i]) - tol[i]
        assert off.max() <= 0, (name, np.unravel_index(off.argmax(), off.shape), off.max())


@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256), (256, 112)])
@pytest.mark.parametrize("x,kv", [("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("f16", "bf16"), ("bf16", "f16"),
                                  ("bf16", "bf16")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_and_head_layouts(dim, rot, x, kv, interleaved):
    need_gpu()
    check(case(dim + rot, 3, 6, 2, dim, rot, x, kv, interleaved=interleaved, layout="hnd" if interleaved else "nhd"))


@pytest.mark.parametrize("M,hq,hk,dim,kw", [
    (1, 32, 8, 128, {}), (16, 32, 4, 128, dict(x="f16", kv="bf16", factor=1.1386)), (1, 1, 1, 64, dict(norm=False)),
    (5, 7, 1, 128, dict(page=1, layout="both")), (2, 9, 3, 256, dict(page=24, pads=1)),
    (61, 14, 2, 64, dict(page=24, pads=9, norm=False, interleaved=True)),
    (300, 32, 8, 128, dict(x="bf16", kv="bf16", pads=4)),           # eight heads to a warp
    (257, 13, 3, 64, dict(pads=3, layout="hnd")), (150, 20, 5, 256, dict(factor=-0.5))])
def test_shapes(M, hq, hk, dim, kw):
    need_gpu()
    check(case(M, M, hq, hk, dim, kw.pop("rot", dim), **kw))


@pytest.mark.parametrize("far", [1, 131072, 10 ** 7, 10 ** 8])
def test_far_positions(far):
    need_gpu()
    a = case(3, 4, 4, 2, 128, 128, far=far, base=10000.0)
    a["positions"][:] = torch.tensor([far, far - 1, far // 2, max(far - 12345, 0)], dtype=torch.int32)
    check(a)


def test_separate_inputs_and_aligned_views():
    need_gpu()
    check(case(4, 5, 4, 2, 128, 128, fused=False))
    a = case(5, 4, 4, 2, 64, 64, fused=False)
    wide = torch.randn((4, 640), device="cuda")
    a["q"] = wide[:, 16:272]                                  # 64-byte offset, 640 apart
    check(a)


def test_zero_and_special_values():
    """A zero head stays zero (eps keeps the scale finite).  Infinities and NaN behind the rotated part stay what
    they are and where they are when there is no norm."""
    need_gpu()
    a = case(6, 2, 2, 1, 128, 64, norm=True)
    a["q"][0, :128] = 0.0
    svq.svq_qk_norm_rope_cache(**a)
    assert torch.all(a["q_out"][0, 0] == 0)
    for interleaved in (False, True):
        b = case(7, 2, 2, 1, 128, 64, norm=False, interleaved=interleaved)
        b["q"][0, 64], b["q"][0, 127], b["q"][1, 100] = float("inf"), float("-inf"), float("nan")
        svq.svq_qk_norm_rope_cache(**b)
        o = b["q_out"].float()
        assert o[0, 0, 64] == float("inf") and o[0, 0, 127] == float("-inf") and torch.isnan(o[1, 0, 100])
        assert int((~torch.isfinite(o)).sum()) == 3


def test_slots_beyond_the_cache_are_skipped():
    need_gpu()
    a = case(8, 6, 4, 2, 64, 64)
    a["slots"][2] = a["cache"].n_pages * 16
    a["slots"][4] = 2 ** 31 - 1
    check(a)
    assert svq.svq_get_device_status() == svq.SVQ_ERR_INVALID_ARG


def test_all_rows_padding():
    need_gpu()
    a = case(9, 12, 4, 2, 64, 64, pads=12)
    a["q"].fill_(float("nan"))
    check(a)


def test_pool_beyond_32_bit_offsets():
    need_gpu()
    page, hk, dim = 64, 8, 128
    a = case(10, 3, 16, hk, dim, dim)
    n_pages = (1 << 31) // (page * hk * dim) + 3
    k = torch.empty((n_pages, page, hk, dim), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    top = n_pages * page
    a["cache"], a["slots"] = svq.KvCache(k, v), torch.tensor([top - 1, 5, top - 100], dtype=torch.int32, device="cuda")
    svq.svq_qk_norm_rope_cache(**a)
    small = pools(2, page, hk, dim, "f16")
    b = dict(a, cache=small, slots=torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), q_out=a["q_out"].clone())
    svq.svq_qk_norm_rope_cache(**b)
    for i, s in enumerate((top - 1, 5, top - 100)):
        for big, ref in ((k, small.k), (v, small.v)):
            assert torch.equal(big.view(-1, hk, dim)[s], ref.view(-1, hk, dim)[i])


def test_other_stream_and_captured_call():
    need_gpu()
    a = case(11, 4, 8, 2, 128, 128)
    svq.svq_qk_norm_rope_cache(**a)
    want = [t.clone() for t in (a["q_out"], a["cache"].k, a["cache"].v)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svq.svq_qk_norm_rope_cache(**a)
    for t in (a["q_out"], a["cache"].k, a["cache"].v):
        t.fill_(7.0)
    a["cache"].k.copy_(torch.where(want[1] != 7, torch.zeros_like(want[1]), want[1]))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a["q_out"], want[0]) and torch.equal(a["cache"].k, want[1]) and torch.equal(a["cache"].v, want[2])
    a["q_out"].fill_(3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    svq.svq_qk_norm_rope_cache(**a, stream=s)
    s.synchronize()
    assert torch.equal(a["q_out"], want[0])


def test_binding_refuses_what_the_library_cannot_see():
    need_gpu()
    a = case(12, 4, 4, 2, 64, 64)
    z = torch.zeros
    for bad in (dict(q=a["q"][:, :192]), dict(k=a["k"][:3]), dict(v=a["v"].half()), dict(q_out=a["q_out"].bfloat16()),
                dict(q_out=a["q_out"].transpose(0, 1).contiguous().transpose(0, 1)), dict(q_gamma=z(64, device="cuda")),
                dict(k_gamma=z(32, dtype=torch.float16, device="cuda")), dict(positions=a["positions"].long()),
                dict(slots=a["slots"][:3]), dict(positions=a["positions"].cpu()), dict(q=a["q"].cpu()),
                dict(q=z((4, 512), device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            svq.svq_qk_norm_rope_cache(**{**a, **bad})
    with pytest.raises(svq.SvqError):                            # rows 8 bytes apart from a 16-byte boundary
        svq.svq_qk_norm_rope_cache(**{**a, "q": z((4, 268), device="cuda")[:, 2:258]})
    k = z((2, 4, 2, 64), dtype=torch.float16, device="cuda")
    for bad in ((k, k.bfloat16()), (k, k[:1]), (k.transpose(2, 3), k.transpose(2, 3)), (k, k.transpose(1, 2)),
                (k[0], k[0])):
        with pytest.raises(ValueError):
            svq.KvCache(*bad)
    for f in (z(32, device="cuda"), z(32, dtype=torch.float64), z((2, 16), dtype=torch.float64, device="cuda")):
        with pytest.raises(ValueError):
            svq.Rope(f)
