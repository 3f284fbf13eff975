"""CPU checks of the row operators' and the 8-bit projection's argument validation: the documented
status comes back before any CUDA call, so none of these needs a device."""
import ctypes

import pytest

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_27_b200 import build as b
    b.build()
    import mla_latent_kv_27_b200 as mla
    return mla


P = 4096  # a non-null address; every call below is refused before it would be read


def norm(mla, **kw):
    a = dict(act=mla.MLA_BF16, x=P, x_ld=64, res=P, res_ld=64, gamma=P, n=2, width=64, eps=1e-6, so=P, so_ld=64,
             y=P, y_ld=64, codes=P, codes_ld=64, scales=P)
    a.update(kw)
    return mla.lib_handle().mla_norm_rows(a["act"], a["x"], a["x_ld"], a["res"], a["res_ld"], a["gamma"], a["n"],
                                          a["width"], a["eps"], a["so"], a["so_ld"], a["y"], a["y_ld"], a["codes"],
                                          a["codes_ld"], a["scales"], None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x_ld=63), dict(res_ld=63), dict(so_ld=63), dict(y_ld=63), dict(codes_ld=63), dict(codes=None),
    dict(scales=None), dict(so=None, y=None, codes=None, scales=None), dict(n=-1), dict(width=0), dict(width=-8),
    dict(eps=-1.0), dict(eps=float("nan")), dict(act=7),
])
def test_norm_rows_refusals(mla, bad):
    assert norm(mla, **bad) == INVALID


def test_norm_rows_act_type(mla):
    assert norm(mla, act=mla.MLA_FP8_E4M3) == UNSUPPORTED


def test_no_rows_is_a_no_op(mla):
    lib = mla.lib_handle()
    assert norm(mla, n=0, x=None, so=None, y=None, codes=None, scales=None) == 0
    assert lib.mla_quantize_rows(mla.MLA_F32, None, 0, 0, 64, None, 0, None, None) == 0
    assert lib.mla_project_fp8(mla.MLA_F32, None, 0, None, 0, None, None, 8, 64, None, 0, None) == 0
    d = mla.mla_dims(64, 64, 16, 32, 32, 4, 64, mla.MLA_F32, mla.MLA_F32, 0.1)
    assert lib.mla_append_rows(ctypes.byref(d), None, 0, 0, None, None, None, 0.0, None, None, 0, None, None) == 0


@pytest.mark.parametrize("bad", [dict(x=None), dict(codes=None), dict(scales=None), dict(x_ld=63), dict(codes_ld=63),
                                 dict(n=-1), dict(width=0), dict(act=-1)])
def test_quantize_rows_refusals(mla, bad):
    a = dict(act=mla.MLA_F32, x=P, x_ld=64, n=2, width=64, codes=P, codes_ld=64, scales=P)
    a.update(bad)
    assert mla.lib_handle().mla_quantize_rows(*a.values(), None) == INVALID


@pytest.mark.parametrize("bad", [dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(out=None),
                                 dict(x_ld=63), dict(out_ld=7), dict(n=-1), dict(n_out=0), dict(width=0), dict(act=9)])
def test_project_fp8_refusals(mla, bad):
    a = dict(act=mla.MLA_F32, x=P, x_ld=64, xs=P, n=2, w=P, ws=P, n_out=8, width=64, out=P, out_ld=8)
    a.update(bad)
    assert mla.lib_handle().mla_project_fp8(*a.values(), None) == INVALID


@pytest.mark.parametrize("bad", [dict(kv=None), dict(kv_ld=79), dict(n=-1), dict(seq=None), dict(pos=None),
                                 dict(cos=None), dict(sin=None), dict(rows=0), dict(cache=None), dict(eps=-1.0)])
def test_append_rows_refusals(mla, bad):
    d = mla.mla_dims(64, 64, 16, 32, 32, 4, 64, mla.MLA_F32, mla.MLA_F32, 0.1)
    c = mla.mla_cache(P, None, None, P, 4, 8, 2)
    a = dict(dims=ctypes.byref(d), kv=P, kv_ld=80, n=2, seq=P, pos=P, gamma=None, eps=0.0, cos=P, sin=P, rows=16,
             cache=ctypes.byref(c))
    a.update(bad)
    assert mla.lib_handle().mla_append_rows(*a.values(), None) == INVALID


def test_append_rows_cache_descriptor(mla):
    lib = mla.lib_handle()
    d = mla.mla_dims(64, 128, 16, 32, 32, 4, 64, mla.MLA_BF16, mla.MLA_FP8_E4M3, 0.1)
    for c in (mla.mla_cache(P, None, P, P, 4, 8, 2), mla.mla_cache(P, P, None, P, 4, 8, 2),
              mla.mla_cache(P, P, P, None, 4, 8, 2), mla.mla_cache(P, P, P, P, 0, 8, 2)):
        assert lib.mla_append_rows(ctypes.byref(d), P, 144, 1, P, P, None, 0.0, P, P, 16, ctypes.byref(c), None) == INVALID
    odd = mla.mla_dims(64, 96, 16, 32, 32, 4, 64, mla.MLA_BF16, mla.MLA_FP8_E4M3, 0.1)
    c = mla.mla_cache(P, P, P, P, 4, 8, 2)
    assert lib.mla_append_rows(ctypes.byref(odd), P, 112, 1, P, P, None, 0.0, P, P, 16, ctypes.byref(c), None) == UNSUPPORTED


def test_host_tensors_are_refused(mla):
    import torch
    x = torch.zeros((2, 64))
    with pytest.raises(ValueError):
        mla.mla_quantize_rows(mla.MLA_F32, x, 64, 2, 64, 4096, 64, 4096, stream=0)


def test_addresses_between_elements_are_refused(mla):
    """A pointer that is no multiple of its element's size would fault on the device."""
    for name in ("x", "res", "gamma", "so", "y"):
        assert norm(mla, **{name: P + 1}) == INVALID
        assert norm(mla, act=mla.MLA_F32, **{name: P + 2}) == INVALID
    assert norm(mla, scales=P + 2) == INVALID
    lib = mla.lib_handle()
    assert lib.mla_quantize_rows(mla.MLA_BF16, P + 1, 64, 2, 64, P, 64, P, None) == INVALID
    assert lib.mla_quantize_rows(mla.MLA_BF16, P, 64, 2, 64, P, 64, P + 1, None) == INVALID
    for k in (3, 6, 9):
        a = [mla.MLA_F32, P, 64, P, 2, P, P, 8, 64, P, 8, None]
        a[k] = P + 2
        assert lib.mla_project_fp8(*a) == INVALID
    d = mla.mla_dims(64, 64, 16, 32, 32, 4, 64, mla.MLA_F32, mla.MLA_F32, 0.1)
    for k in (1, 4, 5, 6, 8, 9):
        c = mla.mla_cache(P, None, None, P, 4, 8, 2)
        a = [ctypes.byref(d), P, 80, 2, P, P, P, 0.0, P, P, 16, ctypes.byref(c), None]
        a[k] = P + 2
        assert lib.mla_append_rows(*a) == INVALID
    c = mla.mla_cache(P + 2, None, None, P, 4, 8, 2)
    assert lib.mla_append_rows(ctypes.byref(d), P, 80, 2, P, P, P, 0.0, P, P, 16, ctypes.byref(c), None) == INVALID


def test_extents_past_the_index_range_are_refused(mla):
    big = 2 ** 31 - 1
    assert norm(mla, n=big) == UNSUPPORTED
    assert norm(mla, width=big, x_ld=big, res_ld=big, so_ld=big, y_ld=big, codes_ld=big) == UNSUPPORTED
    lib = mla.lib_handle()
    assert lib.mla_quantize_rows(mla.MLA_BF16, P, 64, big, 64, P, 64, P, None) == UNSUPPORTED
    assert lib.mla_project_fp8(mla.MLA_F32, P, 64, P, big, P, P, 8, 64, P, 8, None) == UNSUPPORTED
    assert lib.mla_project_fp8(mla.MLA_F32, P, big, P, 2, P, P, 8, big, P, 8, None) == UNSUPPORTED
    assert lib.mla_project_fp8(mla.MLA_F32, P, 64, P, 2, P, P, big, 64, P, big, None) == UNSUPPORTED
