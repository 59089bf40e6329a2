"""The latent-cache entry points refuse bad arguments before anything is enqueued
(no GPU needed: pointers are never followed)."""
import ctypes
import os

import pytest

from test_abi_exports import _ensure_built

_ensure_built()
import paged_kv_gqa_row_gb300 as lnk  # noqa: E402

OK, EINVAL, ERANGE, ECUDA, EUNSUPPORTED, EWORKSPACE = range(6)
A = 1 << 20  # an aligned address that nobody reads


def raw(fn, *args):
    import paged_kv_gqa_row_gb300.binding as b
    return b.raw_status(fn, *args)


def desc(**kw):
    base = dict(num_heads=16, latent_dim=512, rope_dim=64, num_pages=8, num_rows=4, pages_per_row=4, scale=0.1)
    base.update(kw)
    return lnk.latent_desc(**base)


BAD_DESC = [(dict(page_size=32), EUNSUPPORTED), (dict(latent_dim=576), EUNSUPPORTED), (dict(latent_dim=64), EUNSUPPORTED),
            (dict(latent_dim=0), EUNSUPPORTED), (dict(rope_dim=16), EUNSUPPORTED), (dict(rope_dim=128), EUNSUPPORTED),
            (dict(num_heads=0), EINVAL), (dict(num_heads=1025), ERANGE), (dict(num_pages=0), EINVAL),
            (dict(num_rows=-1), EINVAL), (dict(pages_per_row=0), EINVAL), (dict(window=-1), EINVAL), (dict(scale=0.0), EINVAL),
            (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), ERANGE),
            (dict(scale=3e38), ERANGE), (dict(num_pages=1 << 25), ERANGE), (dict(pages_per_row=1 << 25), ERANGE),
            (dict(num_rows=1 << 20, pages_per_row=1 << 12), ERANGE)]


def append(d, q=A, q_stride=64, kv=A, positions=A, rows=A, slots=None, table=A, norm_w=A, eps=1e-6, pool=A, q_out=A,
           q_out_stride=64, kv_out=None, T=2, rope=None):
    return raw("lnk_latent_append", ctypes.byref(d), ctypes.byref(rope or lnk.rope_desc(1e4)), q, q_stride, kv, positions,
               rows, slots, table, norm_w, eps, pool, q_out, q_out_stride, kv_out, T, None, None)


def decode(d, q=A, positions=A, table=A, pool=A, out=A, B=2, ws=A, ws_bytes=1 << 40):
    return raw("lnk_latent_decode_attn", ctypes.byref(d), q, positions, table, pool, out, B, ws, ws_bytes, None, None)


def step(d, q=A, rows=A, positions=A, step_positions=A, table=A, pool=A, out=A, P=2, B=2, ws=A, ws_bytes=1 << 40):
    return raw("lnk_latent_step_attn", ctypes.byref(d), q, rows, positions, step_positions, table, pool, out, P, B, ws,
               ws_bytes, None, None)


def copy(d, pools=(A,), src=A, dst=A, n=1, layers=None):
    a = (ctypes.c_void_p * max(1, len(pools)))(*pools)
    return raw("lnk_latent_copy_pages", ctypes.byref(d), a, len(pools) if layers is None else layers, src, dst, n, None, None)


@pytest.mark.parametrize("kw,status", BAD_DESC)
def test_descriptors(kw, status):
    d = desc(**kw)
    assert [append(d), decode(d), step(d), copy(d)] == [status] * 4
    assert lnk.lnk_latent_workspace_size(d) == 0


@pytest.mark.parametrize("kw", [dict(q=None), dict(kv=None), dict(positions=None), dict(pool=None), dict(q_out=None),
                                dict(table=None), dict(q=A + 2), dict(q_out=A + 2), dict(kv=A + 8), dict(pool=A + 8),
                                dict(kv_out=A + 8), dict(norm_w=A + 8), dict(q_stride=63), dict(q_stride=62),
                                dict(q_out_stride=65), dict(q_stride=-64), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(rows=None, T=5), dict(T=-1), dict(rope=lnk.rope_desc(1.0)),
                                dict(rope=lnk.rope_desc(1e4, (0.0, 1.0, 4.0, 8192.0)))])
def test_append_refusals(kw):
    assert append(desc(), **kw) == EINVAL


def test_append_ranges_and_nothing_to_do():
    assert append(desc(), q_stride=(1 << 30) + 2) == ERANGE
    assert append(desc(), T=0, q=None, kv=None, pool=None) == OK


@pytest.mark.parametrize("kw", [dict(q=None), dict(positions=None), dict(table=None), dict(pool=None), dict(out=None),
                                dict(q=A + 8), dict(out=A + 8), dict(pool=A + 8), dict(B=-1), dict(B=5)])
def test_decode_refusals(kw):
    assert decode(desc(), **kw) == EINVAL


@pytest.mark.parametrize("kw", [dict(rows=None), dict(positions=None), dict(step_positions=None), dict(P=-1), dict(B=5)])
def test_step_refusals(kw):
    assert step(desc(), **kw) == EINVAL


def test_step_ranges_and_nothing_to_do():
    assert decode(desc(num_rows=5000), B=4097) == ERANGE
    assert step(desc(num_heads=1024), P=1 << 21) == ERANGE
    assert decode(desc(), B=0, q=None, ws=None) == OK
    assert step(desc(), P=0, B=0, q=None, ws=None) == OK


def test_copy_refusals():
    assert copy(desc(), pools=(A, None)) == EINVAL
    assert copy(desc(), pools=(A + 8,)) == EINVAL
    assert copy(desc(), src=None) == EINVAL and copy(desc(), dst=None) == EINVAL
    assert copy(desc(), n=-1) == EINVAL and copy(desc(), layers=-1) == EINVAL
    assert copy(desc(), pools=(), n=3) == OK and copy(desc(), n=0) == OK


def test_workspace_on_a_gpu_less_machine():
    """Without a device the size is 0 and a call says so before it reads anything."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    assert lnk.lnk_latent_workspace_size(desc()) == 0
    assert decode(desc()) == ECUDA


def prompt(heads=4, d=128, r=64, scale=0.1, q=A, kv=A, kr=A, stride=64, qs=A, ks=A, out=A, Tq=10, Tk=10, N=2):
    return raw("lnk_latent_prompt_attn", heads, d, r, ctypes.c_float(scale), q, kv, kr, ctypes.c_int64(stride), qs, ks, out,
               Tq, Tk, N, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), EINVAL), (dict(heads=1025), ERANGE), (dict(d=96), EUNSUPPORTED), (dict(r=48), EUNSUPPORTED),
    (dict(scale=0.0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=3e38), ERANGE), (dict(q=None), EINVAL),
    (dict(kv=None), EINVAL), (dict(kr=None), EINVAL), (dict(qs=None), EINVAL), (dict(ks=None), EINVAL),
    (dict(out=None), EINVAL), (dict(q=A + 8), EINVAL), (dict(kv=A + 8), EINVAL), (dict(kr=A + 8), EINVAL),
    (dict(out=A + 8), EINVAL), (dict(stride=56), EINVAL), (dict(stride=68), EINVAL), (dict(stride=1 << 31), ERANGE),
    (dict(Tq=-1), EINVAL), (dict(Tk=-1), EINVAL), (dict(N=-1), EINVAL), (dict(heads=1024, Tq=2 ** 31 - 1), ERANGE),
    (dict(Tq=0, q=None, out=None), OK), (dict(N=0, q=None), OK)])
def test_prompt_refusals(kw, status):
    assert prompt(**kw) == status
