"""GPU parity of the 8-bit block-scaled projection with the plain fp64 formula on the same codes and
scales.

Tolerance.  The products of two E4M3 values are exact in fp32.  With A = sum_b xs ws sum |x w|, every
partial sum is at most A: the 128 additions of a block err by at most 2^-23 of it each (a full step, in
case an adder truncates), the additions over blocks by 2^-24 each, and the scales' products by 2^-24
each, 3 of them.  So |out - ref| <= (256 + blocks + 4) 2^-24 A, and storing adds half a step of the
output type.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
GUARD = 77.0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def codes(shape, seed):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)


def scales(shape, seed):
    return torch.exp(torch.randn(shape, generator=gen(seed), device="cuda"))


def reference(x, xs, w, ws, t, n, k):
    xv = x.contiguous().view(torch.float8_e4m3fn).double() * xs.double().repeat_interleave(128, 1)[:, :k]
    wv = w.view(torch.float8_e4m3fn).double() * ws.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return xv @ wv.t(), xv.abs() @ wv.abs().t()


def check(out, ref, absref, k):
    kb = -(-k // 128)
    tol = (256 + kb + 4) * 2.0 ** -24 * absref
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol * (1 + HALF[out.dtype]) + HALF[out.dtype] * ref.abs()).all(), float((err / absref).max())


def run(lib, t, n, k, act=torch.bfloat16, x_pad=0, out_pad=0, offset=0, seed=0, stream=None):
    kb, nb = -(-k // 128), -(-n // 128)
    ld = k + x_pad
    xb = torch.full((t * ld + offset,), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes around the rows
    x = xb[offset:].view(t, ld)
    x[:, :k] = codes((t, k), seed)
    w = codes((n, k), seed + 1)
    xs, ws = scales((t, kb), seed + 2), scales((nb, kb), seed + 3)
    out = torch.full((t + 1, n + out_pad), GUARD, dtype=act, device="cuda")
    dt = lib.MLA_BF16 if act == torch.bfloat16 else lib.MLA_F32
    lib.mla_project_fp8(dt, x, ld, xs, t, w, ws, n, k, out, n + out_pad, stream)
    torch.cuda.synchronize()
    assert lib.mla_check_device_error()[0] == 0
    ref, absref = reference(x[:, :k], xs, w, ws, t, n, k)
    check(out[:t, :n], ref, absref, k)
    assert (out[t:] == GUARD).all() and (out[:, n:] == GUARD).all()


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (3, 5, 17), (70, 130, 300), (2, 64, 1000), (129, 65, 127)])
def test_any_layout(lib, act, t, n, k):
    run(lib, t, n, k, act)


@pytest.mark.parametrize("x_pad,offset", [(3, 0), (16, 0), (0, 1), (16, 16)])
def test_strides_and_alignment(lib, x_pad, offset):
    run(lib, 9, 200, 512, x_pad=x_pad, offset=offset, out_pad=5)
    run(lib, 300, 200, 512, x_pad=x_pad, offset=offset, out_pad=8)


# rows and outputs around every tile edge, widths that end inside a scale block
@pytest.mark.parametrize("t", [1, 2, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 256, 257])
def test_rows_around_the_tiles(lib, t):
    run(lib, t, 576, 512, seed=t)


@pytest.mark.parametrize("n", [1, 8, 63, 127, 128, 129, 255, 256, 257, 1000, 2112])
@pytest.mark.parametrize("t", [5, 64, 300])
def test_outputs_around_the_tiles(lib, t, n):
    run(lib, t, n, 384, seed=n)


@pytest.mark.parametrize("k", [16, 32, 48, 112, 128, 144, 256, 400, 1536, 2000, 7168])
@pytest.mark.parametrize("t", [4, 64, 200, 520])
def test_widths(lib, t, k):
    run(lib, t, 320, k, seed=k)


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,n,k", [(1, 576, 2048), (64, 2112, 7168), (64, 7168, 2048), (333, 1999, 2000), (1000, 2304, 1536),
                                   (2048, 1024, 2048), (4100, 700, 256)])
def test_larger(lib, act, t, n, k):
    run(lib, t, n, k, act, seed=7)


# few tokens: two token tiles, long ranges of the width per block of threads (split and not), more output tiles
# than streaming multiprocessors, and two of them on one
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,n,k", [(50, 576, 2048), (128, 570, 1040), (5, 18810, 2064), (32, 18810, 2064), (3, 9400, 4112),
                                   (30, 7000, 4112), (16, 24576, 400), (31, 19330, 272), (64, 24570, 400), (33, 19100, 1040),
                                   (100, 9500, 512), (64, 1100, 4112), (128, 1100, 4112)])
def test_few_rows_many_outputs(lib, act, t, n, k):
    run(lib, t, n, k, act, seed=9)


@pytest.mark.parametrize("out_pad", [1, 3, 7, 8])
def test_output_rows_apart(lib, out_pad):
    for t in (7, 300):
        run(lib, t, 250, 256, out_pad=out_pad)
        run(lib, t, 256, 256, torch.float32, out_pad=out_pad)


# many tokens and output rows that TMA stores do not take: 4-byte aligned or not, every end of a segment
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1025, 1026, 1028, 1032, 1087, 1090, 1103, 1106, 1118, 1119])
def test_many_rows_odd_outputs(lib, act, n):
    run(lib, 2300, n, 144, act, seed=n)
    run(lib, 2049, n, 144, act, out_pad=1, seed=n)
    run(lib, 2049, n, 144, act, out_pad=-n % 8 or 8, seed=n)  # aligned rows whose outputs end anywhere


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t", [3, 50, 2100])
@pytest.mark.parametrize("off", [1, 2, 8])
def test_output_begins_anywhere(lib, act, t, off):
    n, k = 1030, 256
    x, w, xs, ws = codes((t, k), 1), codes((n, k), 2), scales((t, 2), 3), scales((9, 2), 4)
    buf = torch.full((t * n + 16,), GUARD, dtype=act, device="cuda")
    out = buf[off:off + t * n].view(t, n)
    lib.mla_project_fp8(lib.MLA_BF16 if act == torch.bfloat16 else lib.MLA_F32, x, k, xs, t, w, ws, n, k, out, n)
    torch.cuda.synchronize()
    ref, absref = reference(x, xs, w, ws, t, n, k)
    check(out, ref, absref, k)
    assert (buf[:off] == GUARD).all() and (buf[off + t * n:] == GUARD).all()


def test_zero_scale_and_zero_codes(lib):
    """A block of zero codes or a zero scale contributes exactly nothing, whatever is beside it."""
    t, n, k = 20, 130, 384
    x, w = codes((t, k), 1), codes((n, k), 2)
    xs, ws = scales((t, 3), 3), scales((2, 3), 4)
    x[3], xs[5], ws[1] = 0, 0, 0
    out = torch.empty((t, n), device="cuda")
    lib.mla_project_fp8(lib.MLA_F32, x, k, xs, t, w, ws, n, k, out, n)
    torch.cuda.synchronize()
    assert (out[3] == 0).all() and (out[5] == 0).all() and (out[:, 128:] == 0).all()
    check(out, *reference(x, xs, w, ws, t, n, k), k)


def test_nan_row_stays_in_its_row(lib):
    for t in (20, 300):
        n, k = 200, 256
        x, w, xs, ws = codes((t, k), 1), codes((n, k), 2), scales((t, 2), 3), scales((2, 2), 4)
        x[4, 100] = 0x7F
        out = torch.empty((t, n), device="cuda")
        lib.mla_project_fp8(lib.MLA_F32, x, k, xs, t, w, ws, n, k, out, n)
        torch.cuda.synchronize()
        assert torch.isnan(out[4]).all()
        assert torch.isfinite(torch.cat((out[:4], out[5:]))).all()


def test_same_result_every_time(lib):
    for t, n, k in ((64, 640, 4096), (300, 640, 2048)):
        x, w, xs, ws = codes((t, k), 1), codes((n, k), 2), scales((t, k // 128), 3), scales((n // 128, k // 128), 4)
        outs = []
        for _ in range(4):
            o = torch.empty((t, n), device="cuda")
            lib.mla_project_fp8(lib.MLA_F32, x, k, xs, t, w, ws, n, k, o, n)
            outs.append(o)
        torch.cuda.synchronize()
        assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_two_streams_at_once(lib):
    """Calls on two streams share nothing."""
    t, n, k = 64, 1024, 2048
    a = [(codes((t, k), s), scales((t, 16), s + 1), codes((n, k), s + 2), scales((8, 16), s + 3),
          torch.empty((t, n), device="cuda"), torch.cuda.Stream()) for s in (10, 20)]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, xs, w, ws, o, st in a:
            lib.mla_project_fp8(lib.MLA_F32, x, k, xs, t, w, ws, n, k, o, n, st)
    torch.cuda.synchronize()
    for x, xs, w, ws, o, _ in a:
        check(o, *reference(x, xs, w, ws, t, n, k), k)


def test_captured_and_replayed_with_new_inputs(lib):
    """Quantise and project in one captured graph; weights and inputs change between replays."""
    t, n, k = 33, 300, 1024
    xr = torch.empty((t, k), device="cuda", dtype=torch.bfloat16)
    x, xs = torch.zeros((t, k), dtype=torch.uint8, device="cuda"), torch.zeros((t, 8), device="cuda")
    w, ws = codes((n, k), 2), scales((3, 8), 3)
    o = torch.empty((t, n), device="cuda")
    st = torch.cuda.Stream()

    def both():
        lib.mla_quantize_rows(lib.MLA_BF16, xr, k, t, k, x, k, xs, st)
        lib.mla_project_fp8(lib.MLA_F32, x, k, xs, t, w, ws, n, k, o, n, st)

    xr.normal_(generator=gen(1))
    torch.cuda.synchronize()
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        both()
        both()
    for seed in (5, 6):
        xr.normal_(generator=gen(seed))
        w.copy_(codes((n, k), seed + 50))
        graph.replay()
        torch.cuda.synchronize()
        check(o, *reference(x, xs, w, ws, t, n, k), k)


def test_offsets_past_32_bits(lib):
    """300 001 rows of 7168 values and 8000 outputs: the last ones lie past 2^31 bytes of x and 2^32
    bytes of out.  The first and last rows are compared."""
    t, n, k = 300_001, 8000, 7168
    x = torch.zeros((t, k), dtype=torch.uint8, device="cuda")
    x[:300], x[-300:] = codes((300, k), 1), codes((300, k), 2)
    xs = torch.ones((t, 56), device="cuda")
    xs[:300], xs[-300:] = scales((300, 56), 3), scales((300, 56), 4)
    w, ws = codes((n, k), 5), scales((63, 56), 6)
    out = torch.full((t, n), GUARD, dtype=torch.bfloat16, device="cuda")
    lib.mla_project_fp8(lib.MLA_BF16, x, k, xs, t, w, ws, n, k, out, n)
    torch.cuda.synchronize()
    assert lib.mla_check_device_error()[0] == 0
    for part in (slice(0, 300), slice(t - 300, t)):
        check(out[part], *reference(x[part], xs[part], w, ws, 300, n, k), k)
    assert not out[300:-300].any()


def test_chain_of_calls_without_a_wait_between(lib):
    """Each call's output is the next one's input, many times over, on one stream with nothing between:
    equal, bit for bit, to the same calls with a synchronisation after each."""
    t, k = 40, 1024
    w, ws = codes((k, k), 2), scales((8, 8), 3) / 2 ** 7
    g = torch.ones(k, device="cuda")

    def run_chain(wait):
        x = torch.randn((t, k), generator=gen(1), device="cuda")
        q, s = torch.empty((t, k), dtype=torch.uint8, device="cuda"), torch.empty((t, 8), device="cuda")
        r = x.clone()
        for _ in range(30):
            lib.mla_norm_rows(lib.MLA_F32, x, k, r, k, g, t, k, 1e-6, r, k, None, 0, q, k, s)
            wait()
            lib.mla_project_fp8(lib.MLA_F32, q, k, s, t, w, ws, k, k, x, k)
            wait()
        torch.cuda.synchronize()
        return r, x

    a, b = run_chain(lambda: None), run_chain(torch.cuda.synchronize)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[1]).all()


# many tokens in tiles of 256 x 160 (by the choice's times: from some 11 scale blocks on, where 128 outputs take a
# round of tiles more), 120 to 216 of them on 74 pairs, so that staging buffers, accumulators and scale slots go
# on from one tile to the next; 9 token tiles are a group of 8 and a last one of one
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,n,k", [(2304, 2560, 2048), (2304, 3840, 4096), (1300, 3200, 2560), (2300, 2552, 2000)])
def test_many_tiles_of_160_outputs(lib, act, t, n, k):
    run(lib, t, n, k, act, seed=21)
    run(lib, t, n, k, act, out_pad=3, seed=22)


@pytest.mark.parametrize("follower", ["few", "split", "many", "core"])
def test_behind_a_call_of_seconds(lib, follower):
    """One output of 60 million values on the general kernel takes longer than a kernel's own bounded waits (2 s); the call
    behind it does not count them from before that one's end, and nothing is reported."""
    from mla_latent_kv_27_b200 import workloads as wl
    k0 = 60_000_001
    x0, w0 = codes((1, k0), 1), codes((1, k0), 2)
    xs0, ws0 = scales((1, -(-k0 // 128)), 3) / 2 ** 10, scales((1, -(-k0 // 128)), 4) / 2 ** 10
    long_out = torch.empty((1, 1), device="cuda")
    if follower == "core":
        from mla_latent_kv_27_b200.runner import MLARunner
        r = MLARunner(wl.WORKLOADS["v2lite_bf16"], lengths=(130, 64))
        r.draw_step_inputs()
        call, outs = r.step, lambda: [r.cache.rows, r.q_packed, r.out]
    else:
        t, n, k = {"few": (5, 18810, 272), "split": (1, 576, 2048), "many": (300, 1000, 512)}[follower]
        x, w, xs, ws = codes((t, k), 5), codes((n, k), 6), scales((t, -(-k // 128)), 7), scales((-(-n // 128), -(-k // 128)), 8)
        out = torch.empty((t, n), device="cuda")
        call = lambda: lib.mla_project_fp8(lib.MLA_F32, x, k, xs, t, w, ws, n, k, out, n)  # noqa: E731
        outs = lambda: [out]  # noqa: E731
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs()]
    for o in outs():
        o.zero_()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    lib.mla_project_fp8(lib.MLA_F32, x0, k0, xs0, 1, w0, ws0, 1, k0, long_out, 1)
    call()
    b.record()
    torch.cuda.synchronize()
    assert a.elapsed_time(b) > 2500
    assert lib.mla_check_device_error()[0] == 0
    assert all(torch.equal(o, v) for o, v in zip(outs(), want))
    s = (xs0 * ws0).double().repeat_interleave(128, 1)[:, :k0]
    p = x0.view(torch.float8_e4m3fn).double() * w0.view(torch.float8_e4m3fn).double() * s
    assert abs(float(long_out) - float(p.sum())) <= (256 + -(-k0 // 128) + 4) * 2.0 ** -24 * float(p.abs().sum())


@pytest.mark.parametrize("t,n,k", [(2, 65535 * 128 + 130, 16), (40, 65535 * 128 + 130, 16), (65535 * 64 + 70, 3, 5),
                                   (3, 65535 * 64 + 70, 5)])
def test_more_tiles_than_a_grids_second_dimension(lib, t, n, k):
    run(lib, t, n, k, torch.bfloat16, seed=31)


def test_row_distance_past_a_tensor_maps(lib):
    """One row may be any distance from the next, which there is none of; other calls take such rows elsewhere."""
    n, k = 200, 512
    x, w, xs, ws = codes((1, k), 1), codes((n, k), 2), scales((1, 4), 3), scales((2, 4), 4)
    out = torch.full((1, n), GUARD, device="cuda")
    for ld in (2 ** 40, 2 ** 41 + 16, 2 ** 62):
        lib.mla_project_fp8(lib.MLA_F32, x, ld, xs, 1, w, ws, n, k, out, ld)
        torch.cuda.synchronize()
        check(out, *reference(x, xs, w, ws, 1, n, k), k)
        out.fill_(GUARD)
    assert lib.mla_check_device_error()[0] == 0
