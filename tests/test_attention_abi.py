"""Host-side checks of the attention step's entry points (no GPU: every call returns before any launch)."""
import ctypes

import pytest

import bit_spherical_vector_b200 as svq

A = 0x1000                    # a pointer that is never dereferenced, 256-byte aligned
INV, SHAPE, WS, OK = svq.SVQ_ERR_INVALID_ARG, svq.SVQ_ERR_UNSUPPORTED_SHAPE, svq.SVQ_ERR_WORKSPACE, svq.SVQ_OK


def cache(**kw):
    f = dict(dtype=svq.SVQ_F16, n_pages=8, page_size=16, n_heads=2, head_dim=128, reserved=0,
             page_stride=16 * 2 * 128, token_stride=2 * 128, head_stride=128, k=A, v=A)
    f.update(kw)
    return svq.svq_kv_cache(**f)


def rope(**kw):
    f = dict(inv_freq=A, rot_dim=128, interleaved=0, factor=1.0, reserved=0)
    f.update(kw)
    return svq.svq_rope(**f)


def call_qk(c=None, r=None, **kw):
    c, r = c or cache(), r or rope()
    f = dict(q=A, k=A, v=A, x=svq.SVQ_F32, ldq=1024, ldk=256, ldv=256, M=1, n_q=8, qg=A, kg=A, eps=1e-6,
             rope=ctypes.addressof(r), pos=A, slots=A, cache=ctypes.addressof(c), out=A)
    f.update(kw)
    return svq.lib().svq_qk_norm_rope_cache(*f.values(), None)


def call_attn(c=None, **kw):
    c = c or cache()
    f = dict(q=A, rows=1, n_q=8, cache=ctypes.addressof(c), lens=A, cu=None, n=1, table=A, width=4, scale=0.1,
             order=None, out=A, dt=svq.SVQ_F16, lse=None, ws=A, nb=0)
    f.update(kw)
    return svq.lib().svq_paged_attention(*f.values(), None)


def call_assign(**kw):
    f = dict(lens=A, new=A, n=1, page=16, table=A, width=4, free=A, pages=8, n_free=A, lens_out=A, n_free_out=A, cu=A,
             pos=A, slots=A, rows=4)
    f.update(kw)
    return svq.lib().svq_kv_assign(*f.values(), None)


BAD_CACHE = [(dict(dtype=svq.SVQ_F32), INV), (dict(k=None), INV), (dict(v=0x1008), INV), (dict(n_pages=0), INV),
             (dict(page_size=0), INV), (dict(n_heads=0), INV), (dict(reserved=1), INV), (dict(token_stride=4), INV),
             (dict(head_stride=-8), INV), (dict(page_stride=12), INV), (dict(head_dim=96), SHAPE),
             (dict(n_pages=1 << 27), SHAPE), (dict(n_heads=2048), SHAPE)]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_cache_is_refused_everywhere(kw, status):
    c = cache(**kw)
    n = ctypes.c_size_t(0)
    assert call_qk(c) == status
    assert call_attn(c) == status
    assert svq.lib().svq_paged_attention_workspace_size(ctypes.addressof(c), 8, ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), INV), (dict(x=4), INV), (dict(ldq=1016), INV), (dict(ldq=1028), INV), (dict(ldk=248), INV),
    (dict(ldv=260), INV), (dict(M=-1), INV), (dict(M=(1 << 20) + 1), INV), (dict(n_q=0), INV), (dict(n_q=1025), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(q=None), INV),
    (dict(k=0x1008), INV), (dict(v=None), INV), (dict(qg=0x1002), INV), (dict(kg=0x1008), INV), (dict(pos=None), INV),
    (dict(slots=0x1002), INV), (dict(out=None), INV), (dict(out=0x1008), INV), (dict(rope=None), INV),
    (dict(cache=None), INV)])
def test_qk_norm_rope_cache_refusals(kw, status):
    assert call_qk(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(inv_freq=None), INV), (dict(inv_freq=0x1004), INV), (dict(interleaved=2), INV), (dict(reserved=1), INV),
    (dict(factor=float("nan")), INV), (dict(factor=float("inf")), INV), (dict(rot_dim=0), SHAPE),
    (dict(rot_dim=24), SHAPE), (dict(rot_dim=144), SHAPE)])
def test_bad_rope_is_refused(kw, status):
    assert call_qk(r=rope(**kw)) == status


def test_no_rows_is_a_no_op():
    assert call_qk(M=0, q=None, k=None, v=None, pos=None, slots=None, out=None) == OK
    assert call_attn(n=0, q=None, out=None, lens=None, table=None, ws=None) == OK
    assert call_attn(rows=0, q=None, out=None, lens=None, table=None, ws=None) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(dt=svq.SVQ_F32), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(n=-1), INV),
    (dict(rows=-1), INV), (dict(width=0), INV), (dict(n=4097), SHAPE), (dict(width=1 << 27), SHAPE),
    (dict(n=4096, width=1 << 20), SHAPE), (dict(n_q=0), SHAPE), (dict(n_q=7), SHAPE), (dict(n_q=1026), SHAPE),
    (dict(q=None), INV), (dict(q=0x1008), INV), (dict(out=0x1002), INV), (dict(lens=None), INV), (dict(lens=0x1002), INV),
    (dict(table=None), INV), (dict(cu=0x1001), INV), (dict(order=0x1008), INV), (dict(order=A, n_q=514), SHAPE), (dict(lse=0x1002), INV)])
def test_paged_attention_refusals(kw, status):
    assert call_attn(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), INV), (dict(page=0), INV), (dict(width=0), INV), (dict(pages=0), INV), (dict(rows=-1), INV),
    (dict(n=4097), SHAPE), (dict(width=1 << 28), SHAPE), (dict(pages=1 << 28), SHAPE), (dict(rows=(1 << 30) + 1), SHAPE),
    (dict(n=4096, width=1 << 19), SHAPE), (dict(lens=None), INV), (dict(new=0x1002), INV), (dict(table=None), INV),
    (dict(free=0x1001), INV), (dict(n_free=None), INV), (dict(lens_out=None), INV), (dict(n_free_out=0x1002), INV),
    (dict(cu=None), INV), (dict(pos=None), INV), (dict(slots=0x1002), INV)])
def test_kv_assign_refusals(kw, status):
    assert call_assign(**kw) == status
