"""mla_absorb_query reads its q_nope only once the kernel in front has completed, whoever wrote it: another host
thread's call, a call with a refused one behind it, another library's kernel.  Each result is compared, bit for bit, with
the same calls with a synchronisation after each.  mla_absorb_query_early gives the same bits behind a call that does not
write q_nope, and checks its arguments as mla_absorb_query does."""
import ctypes
import dataclasses
import threading

import pytest
import torch

from mla_latent_kv_27_b200 import workloads as wl


# ------------------------------------------------------------------ on the CPU
@pytest.mark.parametrize("name", ["mla_absorb_query", "mla_absorb_query_early"])
def test_argument_checks(name):
    from mla_latent_kv_27_b200 import build as b
    b.build()
    import mla_latent_kv_27_b200 as mla
    f = getattr(mla.lib_handle(), name)
    d = lambda **kw: ctypes.byref(mla.mla_dims(**{**dict(  # noqa: E731
        d_model=64, d_c=64, d_rope=16, d_nope=32, d_v=32, n_heads=4, page_size=64, act_dtype=mla.MLA_F32,
        cache_dtype=mla.MLA_F32, scale=0.1), **kw}))
    good = [d(), 4096, 4096, 4096, 2, 4096, 4096, 4096, 16, 4096, None]
    for at, bad in [(0, None), (0, d(d_c=0)), (1, None), (2, None), (3, None), (4, -1), (5, None), (6, None), (7, None),
                    (8, 0), (9, None)]:
        args = list(good)
        args[at] = bad
        assert f(*args) == 1, (at, bad)
    assert f(d(act_dtype=mla.MLA_FP8_E4M3), *good[1:]) == 2
    assert f(d(), None, None, None, 0, None, None, None, 0, None, None) == 0


# ------------------------------------------------------------------ on the GPU
def layer():
    from mla_latent_kv_27_b200.runner import MLALayer
    w = dataclasses.replace(wl.WORKLOADS["v3_bf16"], d_model=512)
    L = MLALayer(w, 1536, lengths=(130,) * 40)
    L.draw_step_inputs()
    x = torch.randn((L.n_tok, 1536), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    L.B = __import__("mla_latent_kv_27_b200")
    L.B.mla_quantize_rows(L.act, x, 1536, L.n_tok, 1536, L.q8, 1536, L.q8_s)
    torch.cuda.synchronize()
    return L


def project(L, st):
    n = L.w.n_heads * L.w.d_nope
    L.B.mla_project_fp8(L.act, L.q8, 1536, L.q8_s, L.n_tok, L.w_qn, L.s_qn, n, 1536, L.q_nope, n, st)


def compare(L, prepare, write, times=6):
    """prepare(); write(q_nope); absorb(): with nothing between, against a synchronisation after each."""
    def once(wait):
        L.q_nope.zero_()
        L.q_packed.zero_()
        torch.cuda.synchronize()
        prepare()
        wait()
        write()
        wait()
        L.absorb()
        torch.cuda.synchronize()
        return L.q_packed.clone()

    want = once(torch.cuda.synchronize)
    assert want[..., :512].any()
    for _ in range(times):
        assert torch.equal(once(lambda: None), want)
    assert L.B.mla_check_device_error()[0] == 0


@pytest.mark.gpu
def test_behind_another_threads_projection(lib):
    """This thread's last call is an append; the projection comes from another one."""
    L = layer()
    st = torch.cuda.current_stream()

    def write():
        t = threading.Thread(target=lambda: project(L, st))
        t.start()
        t.join()

    compare(L, L.append, write)


@pytest.mark.gpu
def test_behind_a_projection_and_a_refused_call(lib):
    """The refused call enqueues nothing, so the projection is still directly in front."""
    L = layer()

    def write():
        project(L, None)
        h = torch.empty(L.h_new.numel() + 8, dtype=torch.bfloat16, device="cuda")[1:]
        with pytest.raises(lib.MlaError) as e:  # off the 16-byte boundary
            lib.mla_append_cache(L.dims, h, L.n_tok, L.seq_idx, L.pos, L.w_dkv, L.w_kr, L.rope_cos, L.rope_sin,
                                 L.rope_rows, L.cache.desc, L.append_ws, L.append_ws_bytes)
        assert e.value.status == 2

    compare(L, lambda: None, write)


@pytest.mark.gpu
def test_behind_another_stream_and_a_library_product(lib):
    """q_nope from a torch matrix product, behind calls of this library on this stream and on another one."""
    L = layer()
    side = torch.cuda.Stream()
    n = L.w.n_heads * L.w.d_nope
    a = torch.randn((L.n_tok, 2048), device="cuda").bfloat16()
    b = torch.randn((2048, n), device="cuda").bfloat16()
    o8, o8_s = torch.empty_like(L.q8), torch.empty_like(L.q8_s)

    def prepare():
        L.append()
        L.B.mla_quantize_rows(L.act, a, 2048, L.n_tok, 1536, o8, 1536, o8_s, side)

    compare(L, prepare, lambda: torch.mm(a, b, out=L.q_nope.view(L.n_tok, n)))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["tiny_fp32", "v2lite_bf16", "v3_bf16"])
def test_early_gives_the_same_bits(lib, name):
    """Behind an append, also with q_nope written by the call in front of that."""
    from mla_latent_kv_27_b200.runner import MLARunner
    w = dataclasses.replace(wl.WORKLOADS[name], d_model=min(wl.WORKLOADS[name].d_model, 512))
    r = MLARunner(w, lengths=(37, 100, 64))
    g = torch.linspace(0.5, 2, w.d_nope, device="cuda").to(r.q_nope.dtype)
    act = lib.MLA_F32 if w.act_dtype == "f32" else lib.MLA_BF16
    for seed in range(4):
        got = []
        for early in (False, True):
            r.draw_step_inputs(seed)
            rows, d = r.n_tok * w.n_heads, w.d_nope
            lib.mla_norm_rows(act, r.q_nope, d, None, 0, g, rows, d, 1e-6, None, 0, r.q_nope, d, None, 0, None)
            r.append()
            r.absorb(q_early=early)
            torch.cuda.synchronize()
            got.append(r.q_packed.clone())
        assert torch.equal(got[0], got[1])
