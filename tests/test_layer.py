"""The row operators and the 8-bit projection run together with the attention core (runner.MLALayer):
every stage's output against the fp64 formula of its actual input, so that each is held to its own
rounding and not to the 8-bit steps before it.

Tolerances.  Norms, 8-bit rows, appends: those of test_rows.py.  Projections: test_project_fp8.py's
(256 + blocks + 4) 2^-24 A plus half a step of the output.  Absorb, decode and output: the bounds
that the workloads state, 2e-2 absolute for bf16 and 1e-5 of the largest value for fp32."""
import dataclasses

import numpy as np
import pytest
import torch

from mla_latent_kv_27_b200 import workloads as wl
from oracle import mla_oracle as orc

W = wl.WORKLOADS


def test_quantize_weight_round_trip():
    """On the CPU: codes times scales within half an E4M3 step, whole blocks of zeros, ragged edges."""
    from mla_latent_kv_27_b200.runner import quantize_weight
    g = torch.Generator().manual_seed(3)
    w = torch.randn((300, 200), generator=g)
    w[128:256, :128] = 0
    codes, scales = quantize_weight(w)
    assert codes.shape == (300, 200) and codes.dtype == torch.uint8 and scales.shape == (3, 2)
    assert scales[1, 0] == 1 and (codes[128:256, :128] & 0x7F == 0).all()
    s = scales.double().repeat_interleave(128, 0)[:300].repeat_interleave(128, 1)[:, :200]
    v = codes.view(torch.float8_e4m3fn).double() * s
    # half a step of the code, 2^-4 of it (2^-10 scales where it is subnormal), and the division's rounding
    assert ((v - w.double()).abs() <= (2.0 ** -4 + 2.0 ** -20) * w.double().abs() + 2.0 ** -10 * s).all()
    assert (v.abs() <= 448 * s).all()


def _layer_case(lib, w, lengths, q_rank):
    from mla_latent_kv_27_b200.runner import MLALayer
    from tests.test_project_fp8 import check, reference
    from tests.test_rows import REL, check_codes, near, norm_ref
    L = MLALayer(w, q_rank, lengths=lengths)
    if w.cache_dtype == "fp8":
        L.fill_cache_projected()
    else:
        L.fill_cache_direct()
    L.draw_step_inputs()
    L.residual.copy_(2 * torch.randn(L.residual.shape, generator=torch.Generator(device="cuda").manual_seed(8),
                                     device="cuda"))
    res0 = L.residual.clone()
    T, R = L.n_tok, q_rank
    L.layer_step()
    torch.cuda.synchronize()
    assert lib.mla_check_device_error()[0] == 0

    def projected(out, x, xs, ws, ss):
        n, k = ws.shape
        check(out.reshape(T, n), *reference(x, xs, ws, ss, T, n, k), k)

    r, y = norm_ref(L.h_new, res0, L.g_in, L.eps)
    near(L.residual, r, 2.0 ** -24)
    check_codes(L.x8, L.x8_s, y, w.d_model)
    projected(L.down, L.x8, L.x8_s, L.w_down, L.s_down)
    check_codes(L.q8, L.q8_s, norm_ref(L.down[:, :R], None, L.g_q, L.eps)[1], R)
    projected(L.q_nope, L.q8, L.q8_s, L.w_qn, L.s_qn)
    projected(L.q_rope, L.q8, L.q8_s, L.w_qr, L.s_qr)
    # the step's cache rows
    at = (L.cache.block_table.long()[L.seq_idx.long(), L.pos.long() // 64] * 64 + L.pos.long() % 64)
    lat = norm_ref(L.down[:, R:R + w.d_c], None, L.g_kv, L.eps)[1]
    if w.cache_dtype == "fp8":
        check_codes(L.cache.rows.flatten(0, 1)[at], L.cache.scales.flatten(0, 1)[at], lat, w.d_c)
    else:
        near(L.cache.rows.flatten(0, 1)[at][:, :w.d_c], lat, REL)
    # attention core against the oracle on the actual queries and cache
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    pos = L.pos.cpu().numpy()
    q_lat, q_rot = orc.absorb_query(host(L.q_nope), host(L.q_rope), pos, host(L.w_uk), w.theta)
    rows = host(L.cache.rows)
    if w.cache_dtype == "fp8":
        codes = L.cache.rows.cpu().numpy()
        rows = np.concatenate([orc.fp8_dequantize_blocks(codes, L.cache.scales.cpu().numpy()), host(L.cache.rope)], -1)
    o, _ = orc.decode_paged(q_lat, q_rot, rows, L.block_table_np, L.lengths, w.s_q, w.scale, w.d_c, wl.PAGE_SIZE,
                            w.causal or w.s_q > 1)
    ref = orc.output_up(o, host(L.w_uv))
    err = np.abs(host(L.out) - ref).max()
    assert err <= (1e-5 * np.abs(ref).max() if w.act_dtype == "f32" else 2e-2), err
    out = L.out.reshape(T, -1)
    check_codes(L.o8, L.o8_s, out.double(), out.shape[1], 2.0 ** -24)
    projected(L.y, L.o8, L.o8_s, L.w_o, L.s_o)
    return L


@pytest.mark.gpu
@pytest.mark.parametrize("name,lengths,q_rank", [
    ("tiny_fp32", (37, 100), 48), ("v2lite_bf16", (130, 64, 1, 700), 768), ("v3_bf16", (300, 65, 1), 1536),
    ("fp8_mtp2", (513, 600, 64), 1536)])
def test_layer_step(lib, name, lengths, q_rank):
    w = dataclasses.replace(W[name], d_model=min(W[name].d_model, 1024))
    _layer_case(lib, w, lengths, q_rank)


@pytest.mark.gpu
def test_layer_step_captured(lib):
    """The layer's eleven calls in one graph: replays with new inputs equal eager steps, bit for bit."""
    from mla_latent_kv_27_b200.runner import MLALayer
    w = dataclasses.replace(W["v2lite_bf16"], d_model=512)
    st = torch.cuda.Stream()
    L = MLALayer(w, 256, lengths=(130, 64, 200))
    L.fill_cache_direct()
    L.draw_step_inputs(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        L.layer_step(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        L.layer_step(st)
    for seed in (1, 2):
        L.draw_step_inputs(seed)
        L.residual.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = L.y.clone()
        L.residual.zero_()
        torch.cuda.synchronize()
        L.layer_step(st)
        torch.cuda.synchronize()
        assert torch.equal(got, L.y)
    assert lib.mla_check_device_error()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("between", [False, True])
def test_absorb_directly_behind_the_projection(lib, between):
    """q_nope written by mla_project_fp8 directly in front of the absorb (or one append before it), which
    reads q_nope early: equal, bit for bit, to the same calls with a synchronisation between."""
    from mla_latent_kv_27_b200.runner import MLALayer
    w = dataclasses.replace(W["v3_bf16"], d_model=512)
    L = MLALayer(w, 1536, lengths=(130,) * 40)
    L.draw_step_inputs()
    T, n = L.n_tok, w.n_heads * w.d_nope

    def project_and_absorb(wait):
        lib.mla_quantize_rows(L.act, x, 1536, T, 1536, L.q8, 1536, L.q8_s)
        wait()
        lib.mla_project_fp8(L.act, L.q8, 1536, L.q8_s, T, L.w_qn, L.s_qn, n, 1536, L.q_nope, n)
        wait()
        if between:
            L.append()
            wait()
        L.absorb()

    for seed in range(6):
        x = torch.randn((T, 1536), generator=torch.Generator(device="cuda").manual_seed(seed),
                        device="cuda").bfloat16()
        torch.cuda.synchronize()
        project_and_absorb(lambda: None)
        torch.cuda.synchronize()
        got = L.q_packed.clone()
        L.q_packed.zero_()
        project_and_absorb(torch.cuda.synchronize)
        torch.cuda.synchronize()
        assert torch.equal(got, L.q_packed)


@pytest.mark.gpu
def test_absorb_directly_behind_the_norm(lib):
    """The same with q_nope normed in place by mla_norm_rows directly in front."""
    from mla_latent_kv_27_b200.runner import MLALayer
    w = dataclasses.replace(W["v3_bf16"], d_model=512)
    L = MLALayer(w, 1536, lengths=(130,) * 40)
    L.draw_step_inputs()
    rows, d = L.n_tok * w.n_heads, w.d_nope
    q = L.q_nope.clone()
    g = torch.linspace(0.5, 2, d, device="cuda").bfloat16()

    def norm_and_absorb(wait):
        L.q_nope.copy_(q)
        torch.cuda.synchronize()
        lib.mla_norm_rows(L.act, L.q_nope, d, None, 0, g, rows, d, 1e-6, None, 0, L.q_nope, d, None, 0, None)
        wait()
        L.absorb()
        torch.cuda.synchronize()
        return L.q_packed.clone()

    want = norm_and_absorb(torch.cuda.synchronize)
    L.q_packed.zero_()
    for _ in range(6):
        assert torch.equal(norm_and_absorb(lambda: None), want)


def test_quantize_weight_of_tiny_and_not_finite_blocks():
    """On the CPU: blocks of subnormals stay finite, and a NaN or an infinity makes its block NaN without touching the
    blocks beside it (a scale of 1 would round its neighbours to multiples of 2^-9 and say nothing)."""
    from mla_latent_kv_27_b200.runner import quantize_weight
    g = torch.Generator().manual_seed(4)
    w = torch.randn((256, 640), generator=g) / 40
    w[:128, 128:256] *= 2.0 ** -140
    w[3, 130] = 0
    w[5, 260] = float("nan")
    w[6, 390] = float("inf")
    w[7, 520] = -float("inf")
    codes, scales = quantize_weight(w)
    s = scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    v = codes.view(torch.float8_e4m3fn).double() * s
    for b in (2, 3, 4):
        assert torch.isnan(v[:128, 128 * b:128 * b + 128]).all()
    good = torch.ones((256, 640), dtype=torch.bool)
    good[:128, 256:] = False
    err = (v - w.double()).abs()
    # half a step of the code (2^-10 scales where it is subnormal), and the division's rounding
    assert (err <= (2.0 ** -4 + 2.0 ** -20) * w.double().abs() + 2.0 ** -10 * s)[good].all()
