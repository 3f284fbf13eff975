"""GPU parity of the row operators (norm, quantisation, append of projected rows) with plain fp64
formulas on the same inputs.

Tolerances.  U = 2^-24 is half a step of fp32.  The mean of squares is a sum of positive terms: a
value passes through at most ceil(width / 256) + 20 additions (one thread's values, then the
tree), so its relative error is below (ceil(width / 256) + 21) U, half of that after the root; the
root, two products and the residual's sum add a few U more.  At the widths used here (up to 33000)
that is under 80 U: REL = 128 U = 2^-17.  Storing rounds once: half a step of the output type,
2^-8 (bf16) or U (fp32) relative.  An E4M3 code is off by half a step of the code: 2^-4 of the
value, or 2^-10 scales where the code is subnormal (step 2^-9); a decision that falls the other
way because of REL costs REL more.
"""
import dataclasses

import numpy as np
import pytest
import torch

from mla_latent_kv_27_b200 import workloads as wl
from oracle import mla_oracle as orc

pytestmark = pytest.mark.gpu

REL = 2.0 ** -17
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ACT = [torch.bfloat16, torch.float32]
GUARD = 77.0


def dt(lib, t):
    return lib.MLA_BF16 if t == torch.bfloat16 else lib.MLA_F32


def randn(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def decoded(codes, scales, width):
    v = codes[:, :width].contiguous().view(torch.float8_e4m3fn).double()
    return v * scales.double().repeat_interleave(128, 1)[:, :width]


def check_codes(codes, scales, y, width, rel=REL):
    """8-bit rows against the exact values y [T, width] (fp64)."""
    assert torch.isfinite(scales).all()
    kb = -(-width // 128)
    pad = torch.nn.functional.pad(y, (0, kb * 128 - width)).view(y.shape[0], kb, 128)
    amax = pad.abs().amax(-1)
    want = torch.where(amax == 0, torch.ones_like(amax), amax.clamp(min=2.0 ** -100) / 448)
    assert ((scales.double() - want).abs() <= (rel + 2.0 ** -24) * want).all()
    s = scales.double().repeat_interleave(128, 1)[:, :width]
    err = (decoded(codes, scales, width) - y).abs()
    assert (err <= 2.0 ** -4 * y.abs() * (1 + 2 * rel) + 2.0 ** -10 * s + 2 * rel * y.abs()).all()


def near(got, want, extra=REL):
    tol = (HALF[got.dtype] + extra) * want.abs()
    assert ((got.double() - want).abs() <= tol).all(), float(((got.double() - want).abs() - tol).max())


def norm_ref(x, res, gamma, eps):
    r = x.double() if res is None else x.double() + res.double()
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    return r, y if gamma is None else y * gamma.double()


def strided(t, width, ld, act):
    return torch.full((t, ld), GUARD, dtype=act, device="cuda")


def run_norm(lib, act, t, width, *, res=True, gamma=True, outs=("sum", "y", "q"), pad=0, offset=0, seed=0, eps=1e-6,
             x=None):
    ld = width + pad
    cut = lambda m: m.reshape(-1)[offset:offset + t * ld].view(t, ld) if offset else m  # noqa: E731
    buf = torch.full((t * ld + offset,), GUARD, dtype=act, device="cuda")
    X = cut(buf) if offset else buf.view(t, ld)
    X[:, :width] = (randn((t, width), seed) if x is None else x).to(act)
    R = G = None
    if res:
        R = strided(t, width, ld, act)
        R[:, :width] = randn((t, width), seed + 1, 2.0).to(act)
    if gamma:
        G = (1 + 0.2 * randn((width,), seed + 2)).to(act)
    S = strided(t, width, ld, act) if "sum" in outs else None
    Y = strided(t, width, ld, act) if "y" in outs else None
    Q = torch.full((t, ld), 99, dtype=torch.uint8, device="cuda") if "q" in outs else None
    SC = torch.full((t, -(-width // 128)), float("nan"), device="cuda") if "q" in outs else None
    lib.mla_norm_rows(dt(lib, act), X, ld, R, ld, G, t, width, eps, S, ld, Y, ld, Q, ld, SC)
    torch.cuda.synchronize()
    assert lib.mla_check_device_error()[0] == 0
    r, y = norm_ref(X[:, :width], None if R is None else R[:, :width], G, eps)
    if S is not None:
        near(S[:, :width], r, 2.0 ** -24)
        assert (S[:, width:] == GUARD).all()
    if Y is not None:
        near(Y[:, :width], y)
        assert (Y[:, width:] == GUARD).all()
    if Q is not None:
        check_codes(Q, SC, y, width)
        assert (Q[:, width:] == 99).all()


# widths around the 8-value chunk, the 128-value block and the launch shapes (256, 1024, 4096 chunks)
WIDTHS = [1, 7, 8, 100, 127, 128, 136, 512, 1000, 1536, 2048, 2056, 7168, 8192, 8200, 16384, 32768, 33000]


@pytest.mark.parametrize("act", ACT)
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_widths(lib, act, width):
    run_norm(lib, act, 3, width, seed=width)


@pytest.mark.parametrize("act", ACT)
@pytest.mark.parametrize("t", [1, 2, 65, 1500])
def test_norm_rows_count(lib, act, t):
    run_norm(lib, act, t, 1536, seed=t)


@pytest.mark.parametrize("act", ACT)
@pytest.mark.parametrize("width", [72, 1000, 2056, 7168, 8200, 16384])
@pytest.mark.parametrize("res,gamma,outs", [(True, True, ("sum", "q")), (True, True, ("sum", "y")), (False, True, ("y", "q")),
                                            (True, False, ("q",)), (False, False, ("sum", "y"))])
def test_norm_many_rows(lib, act, width, res, gamma, outs):
    """More rows than CTAs that run at once: each CTA walks several, the last ones a row fewer."""
    run_norm(lib, act, 1201 if width <= 2056 else 641, width, res=res, gamma=gamma, outs=outs, pad=16, seed=width)


# widths off the 8-value chunk: one and several warps a row, two and four blocks a warp, rows read twice
@pytest.mark.parametrize("act", ACT)
@pytest.mark.parametrize("t,width", [(3, 129), (700, 301), (701, 511), (4, 513), (601, 1501), (5, 8191), (2, 8193), (600, 7169),
                                     (2, 16383), (3, 16385)])
def test_norm_odd_widths(lib, act, t, width):
    run_norm(lib, act, t, width, seed=width)
    run_norm(lib, act, t, width, res=False, outs=("y",), seed=width)


@pytest.mark.parametrize("act", ACT)
@pytest.mark.parametrize("t,width", [(1, 1), (3, 255), (700, 257), (601, 1501), (2, 40001)])
def test_quantize_odd_widths(lib, act, t, width):
    x = randn((t, width), width).to(act)
    q = torch.full((t, width + 3), 99, dtype=torch.uint8, device="cuda")
    s = torch.full((t, -(-width // 128)), float("nan"), device="cuda")
    lib.mla_quantize_rows(dt(lib, act), x, width, t, width, q, width + 3, s)
    torch.cuda.synchronize()
    check_codes(q, s, x.double(), width, 2.0 ** -24)
    assert (q[:, width:] == 99).all()


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (24, 8)])
def test_norm_strides_and_alignment(lib, pad, offset):
    for act in ACT:
        run_norm(lib, act, 5, 640, pad=pad, offset=offset)


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("gamma", [True, False])
@pytest.mark.parametrize("outs", [("sum",), ("y",), ("q",), ("sum", "q")])
def test_norm_optional_arguments(lib, res, gamma, outs):
    for width in (520, 515):
        run_norm(lib, torch.bfloat16, 4, width, res=res, gamma=gamma, outs=outs)


@pytest.mark.parametrize("width", [1024, 1001])
def test_norm_in_place(lib, width):
    """sum_out over the residual and y over x."""
    t = 6
    x, res = randn((t, width), 1).bfloat16(), randn((t, width), 2).bfloat16()
    g = (1 + 0.1 * randn((width,), 3)).bfloat16()
    r, y = norm_ref(x, res, g, 1e-5)
    lib.mla_norm_rows(lib.MLA_BF16, x, width, res, width, g, t, width, 1e-5, res, width, x, width, None, 0, None)
    torch.cuda.synchronize()
    near(res, r, 2.0 ** -24)
    near(x, y)


@pytest.mark.parametrize("width", [384, 385])
def test_norm_zero_rows(lib, width):
    """An all-zero row: y = 0, codes 0, scales 1; rows beside it are untouched by it."""
    x = randn((4, width), 5)
    x[2] = 0
    run_norm(lib, torch.float32, 4, width, res=False, x=x)
    q = torch.empty((4, width), dtype=torch.uint8, device="cuda")
    s = torch.empty((4, -(-width // 128)), device="cuda")
    lib.mla_quantize_rows(lib.MLA_F32, x, width, 4, width, q, width, s)
    torch.cuda.synchronize()
    assert (q[2] == 0).all() and (s[2] == 1).all()


@pytest.mark.parametrize("act", ACT)
@pytest.mark.parametrize("width", [8, 100, 128, 1000, 2048, 2304, 16384, 40000])
def test_quantize_equals_the_fp32_decision(lib, act, width):
    """Same inputs, same fp32 steps: codes and scales are the oracle's, bit for bit."""
    t = 7
    x = (randn((t, width), width) * torch.exp(randn((t, 1), 9))).to(act)
    q = torch.full((t, width), 99, dtype=torch.uint8, device="cuda")
    s = torch.empty((t, -(-width // 128)), device="cuda")
    lib.mla_quantize_rows(dt(lib, act), x, width, t, width, q, width, s)
    torch.cuda.synchronize()
    kb = -(-width // 128)
    padded = np.zeros((t, kb * 128), np.float32)
    padded[:, :width] = x.float().cpu().numpy()
    codes, scales = orc.fp8_quantize_blocks(padded)
    assert np.array_equal(s.cpu().numpy(), scales)
    got, want = q.cpu().numpy(), codes[:, :width]
    assert np.array_equal(got & 0x7F, want & 0x7F)
    assert np.array_equal(orc.e4m3_decode(got), orc.e4m3_decode(want))


@pytest.mark.parametrize("width", [256, 250])
def test_quantize_nan_inf_and_tiny_blocks(lib, width):
    x = randn((5, width), 3)
    x[0, 3] = float("nan")
    x[1, 3] = float("inf")
    x[2, :128] = 1e-38 * randn((128,), 4)
    x[3, :128] = 3.3e38
    x[4, :128] = 2.0 ** -99
    q = torch.empty((5, width), dtype=torch.uint8, device="cuda")
    s = torch.empty((5, 2), device="cuda")
    lib.mla_quantize_rows(lib.MLA_F32, x, width, 5, width, q, width, s)
    torch.cuda.synchronize()
    v = decoded(q, s, width)
    assert torch.isnan(v[0, :128]).all() and torch.isnan(v[1, :128]).all()
    check_codes(q[2:], s[2:], x[2:].double(), width)
    check_codes(q[:2, 128:].contiguous(), s[:2, 1:], x[:2, 128:].double(), width - 128)


def test_norm_nan_row_stays_in_its_row(lib):
    x = randn((3, 256), 3)
    x[1, 7] = float("nan")
    y = torch.empty_like(x)
    lib.mla_norm_rows(lib.MLA_F32, x, 256, None, 0, None, 3, 256, 1e-6, None, 0, y, 256, None, 0, None)
    torch.cuda.synchronize()
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()


# ------------------------------------------------------------------ append of projected rows
def rope_tables(lib, d_rope, rows):
    c = torch.empty((rows, d_rope // 2), device="cuda")
    s = torch.empty_like(c)
    lib.mla_rope_table(d_rope, rows, 10000.0, c, s)
    return c, s


class Cache:
    def __init__(self, lib, act, kind, d_c, d_rope, page, lengths, seed=0):
        self.kind, self.page, self.d_c, self.d_rope = kind, page, d_c, d_rope
        table, self.pages = wl.make_block_table(np.asarray(lengths), 0, True, np.random.default_rng(seed), page)
        self.table = torch.as_tensor(table, device="cuda")
        n = self.pages * page
        code = {"f32": lib.MLA_F32, "bf16": lib.MLA_BF16, "fp8": lib.MLA_FP8_E4M3}[kind]
        if kind == "fp8":
            self.rows = torch.full((n, d_c), 99, dtype=torch.uint8, device="cuda")
            self.scales = torch.full((n, d_c // 128), GUARD, device="cuda")
            self.rope = torch.full((n, d_rope), GUARD, dtype=torch.bfloat16, device="cuda")
        else:
            self.rows = torch.full((n, d_c + d_rope), GUARD, dtype=act, device="cuda")
            self.scales = self.rope = None
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.dims = lib.mla_dims(64, d_c, d_rope, 32, 32, 4, page, dt(lib, act), code, 0.1)
        self.desc = lib.mla_cache(p(self.rows), p(self.scales), p(self.rope), self.table.data_ptr(),
                                  table.shape[1], self.pages, table.shape[0])

    def slots(self, seq, pos):
        return self.table.long()[seq.long(), pos.long() // self.page] * self.page + pos.long() % self.page


def run_append(lib, act, kind, d_c=512, d_rope=64, page=64, lengths=(1, 64, 130), gamma=True, pad=0, offset=0, seed=0):
    c = Cache(lib, act, kind, d_c, d_rope, page, lengths, seed)
    T, W = int(sum(lengths)), d_c + d_rope
    seq = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths)).int().cuda()
    pos = torch.cat([torch.arange(n) for n in lengths]).int().cuda()
    order = torch.randperm(T, generator=torch.Generator().manual_seed(seed)).cuda()
    seq, pos = seq[order].contiguous(), pos[order].contiguous()
    ld = W + pad
    buf = torch.full((T * ld + offset,), GUARD, dtype=act, device="cuda")
    kv = buf[offset:].view(T, ld)
    kv[:, :W] = randn((T, W), seed + 1).to(act)
    G = (1 + 0.2 * randn((d_c,), seed + 2)).to(act) if gamma else None
    cos, sin = rope_tables(lib, d_rope, max(lengths))
    lib.mla_append_rows(c.dims, kv, ld, T, seq, pos, G, 1e-6, cos, sin, max(lengths), c.desc)
    torch.cuda.synchronize()
    assert lib.mla_check_device_error()[0] == 0
    x = kv[:, :W].double()
    lat = x[:, :d_c]
    if gamma:
        lat = norm_ref(kv[:, :d_c], None, G, 1e-6)[1]
    a, b = x[:, d_c::2], x[:, d_c + 1::2]
    cs, sn = cos.double()[pos.long()], sin.double()[pos.long()]
    rot = torch.stack((a * cs - b * sn, a * sn + b * cs), -1).flatten(1)
    # two products and a sum: 3 roundings of at most U (|a| + |b|) each, then the store's
    pair = (a.abs() + b.abs()).repeat_interleave(2, 1) * 3 * 2.0 ** -24
    at = c.slots(seq, pos)
    rest = torch.ones(c.pages * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    half = HALF[torch.bfloat16 if kind == "fp8" else act]
    got = c.rope[at] if kind == "fp8" else c.rows[at][:, d_c:]
    assert ((got.double() - rot).abs() <= half * rot.abs() + pair * (1 + half)).all()
    if kind == "fp8":
        check_codes(c.rows[at], c.scales[at], lat, d_c, REL if gamma else 2.0 ** -24)
        assert (c.rows[rest] == 99).all() and (c.scales[rest] == GUARD).all() and (c.rope[rest] == GUARD).all()
    else:
        near(c.rows[at][:, :d_c], lat, REL if gamma else 0.0)
        assert (c.rows[rest] == GUARD).all()


KINDS = [(torch.float32, "f32"), (torch.bfloat16, "bf16"), (torch.bfloat16, "fp8")]


@pytest.mark.parametrize("act,kind", KINDS)
@pytest.mark.parametrize("gamma", [True, False])
def test_append_rows(lib, act, kind, gamma):
    run_append(lib, act, kind, gamma=gamma)


@pytest.mark.parametrize("act,kind", KINDS)
@pytest.mark.parametrize("lengths", [(1,), (5,), (700, 1, 3)])
def test_append_rows_counts(lib, act, kind, lengths):
    run_append(lib, act, kind, lengths=lengths, seed=3)


@pytest.mark.parametrize("act,kind", KINDS)
@pytest.mark.parametrize("d_c,d_rope,page,lengths", [(512, 64, 64, (600,)), (512, 128, 16, (1, 5003, 2)), (128, 8, 7, (9000, 4)),
                                                     (384, 64, 64, (9001,)), (1024, 64, 64, (2000, 1))])
def test_append_rows_many_tokens(lib, act, kind, d_c, d_rope, page, lengths):
    """More tokens than run at once, odd counts among them: the last group of a warp has none."""
    run_append(lib, act, kind, d_c=d_c, d_rope=d_rope, page=page, lengths=lengths, pad=8, seed=4)


@pytest.mark.parametrize("act,kind", KINDS)
def test_append_rows_bad_tokens_among_many(lib, act, kind):
    n = 9001
    c = Cache(lib, act, kind, 512, 64, 64, (n, n))
    seq = (torch.arange(n) % 2).int().cuda()
    pos = torch.arange(n).int().cuda()
    bad = torch.tensor([0, 1, 592, 601, 4737, n - 1], device="cuda")
    good = torch.ones(n, dtype=torch.bool, device="cuda")
    good[bad] = False
    at = c.slots(seq, pos)[good]
    seq[bad[:3]] = 2
    pos[bad[3:]] = torch.tensor([n, -1, 1 << 30], dtype=torch.int32, device="cuda")
    kv = randn((n, 576), 6).to(act)
    cos, sin = rope_tables(lib, 64, n)
    lib.mla_append_rows(c.dims, kv, 576, n, seq, pos, None, 0.0, cos, sin, n, c.desc)
    status, detail = lib.mla_check_device_error()
    assert status == 4 and detail >> 24 in (2, 4)
    rest = torch.ones(c.pages * 64, dtype=torch.bool, device="cuda")
    rest[at] = False
    empty = 99 if kind == "fp8" else GUARD
    assert (c.rows[rest] == empty).all()
    if kind == "fp8":
        check_codes(c.rows[at], c.scales[at], kv[good][:, :512].double(), 512, 2.0 ** -24)
    else:
        near(c.rows[at][:, :512], kv[good][:, :512].double(), 0.0)


@pytest.mark.parametrize("act,kind", KINDS)
@pytest.mark.parametrize("d_c,d_rope,page", [(128, 16, 1), (256, 64, 16), (384, 8, 7), (1024, 256, 64), (1152, 64, 64),
                                             (512, 2, 64), (128, 258, 3)])
def test_append_rows_shapes(lib, act, kind, d_c, d_rope, page):
    run_append(lib, act, kind, d_c=d_c, d_rope=d_rope, page=page, lengths=(3, 20))


@pytest.mark.parametrize("d_c", [1, 9, 100, 520])
def test_append_rows_odd_latent(lib, d_c):
    run_append(lib, torch.float32, "f32", d_c=d_c, d_rope=6, lengths=(4, 9))
    run_append(lib, torch.bfloat16, "bf16", d_c=d_c, d_rope=6, lengths=(4, 9))


@pytest.mark.parametrize("pad,offset", [(1536, 0), (3, 0), (8, 8), (0, 1)])
def test_append_rows_strides(lib, pad, offset):
    for act, kind in KINDS:
        run_append(lib, act, kind, pad=pad, offset=offset)


def test_append_rows_bad_tokens_are_skipped(lib):
    """A bad sequence, position or page id skips that token alone and is reported; nothing else
    of the cache changes."""
    for d_c, d_rope in ((512, 64), (130, 6)):
        for what, kind in (("seq", 4), ("neg", 4), ("pos", 2), ("past", 2), ("page", 1)):
            c = Cache(lib, torch.bfloat16, "bf16", d_c, d_rope, 64, (64, 64))
            kv = randn((3, d_c + d_rope), 1).bfloat16()
            seq = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
            pos = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
            good = c.slots(seq, pos)[[0, 2]]
            if what == "seq":
                seq[1] = 2
            elif what == "neg":
                seq[1] = -1
            elif what == "pos":
                pos[1] = -3
            elif what == "past":
                pos[1] = 64
            else:
                seq[1], pos[2] = 0, 7
                good = c.slots(seq, pos)[[0, 1]]
                c.table[1, 0] = c.pages
            cos, sin = rope_tables(lib, d_rope, 128)
            lib.mla_append_rows(c.dims, kv, d_c + d_rope, 3, seq, pos, None, 0.0, cos, sin, 128, c.desc)
            status, detail = lib.mla_check_device_error()
            assert status == 4 and detail >> 24 == kind, (what, status, detail)
            rest = torch.ones(c.pages * 64, dtype=torch.bool, device="cuda")
            rest[good] = False
            assert (c.rows[rest] == GUARD).all() and not (c.rows[good] == GUARD).any()


def test_append_rows_writes_what_append_cache_writes(lib):
    """Same latents, same codes: the fused append's rows of an fp32 model, and append_rows on the
    rows that its projection gives (identity weights, so the products are exact)."""
    w = dataclasses.replace(wl.WORKLOADS["tiny_fp32"], d_model=80)
    lengths = (5, 70)
    T = sum(lengths)
    h = randn((T, 80), 11)
    eye = torch.eye(80, device="cuda")
    seq = torch.repeat_interleave(torch.arange(2), torch.tensor(lengths)).int().cuda()
    pos = torch.cat([torch.arange(n) for n in lengths]).int().cuda()
    cos, sin = rope_tables(lib, 16, 128)
    a, b = (Cache(lib, torch.float32, "f32", w.d_c, w.d_rope, 64, lengths) for _ in range(2))
    dims = lib.mla_dims(80, 64, 16, 32, 32, 4, 64, lib.MLA_F32, lib.MLA_F32, 0.1)
    n = lib.mla_append_workspace_size(dims, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    lib.mla_append_cache(dims, h, T, seq, pos, eye[:64].contiguous(), eye[64:].contiguous(), cos, sin, 128, a.desc, ws, n)
    lib.mla_append_rows(b.dims, h, 80, T, seq, pos, None, 0.0, cos, sin, 128, b.desc)
    torch.cuda.synchronize()
    # the rotation may contract a product and a sum: 3 roundings
    assert torch.equal(a.rows[:, :64], b.rows[:, :64])
    assert ((a.rows - b.rows).abs() <= 2.0 ** -21).all()


def test_rows_captured_and_replayed_with_new_inputs(lib):
    t, width = 9, 1536
    x, res = randn((t, width), 1).bfloat16(), randn((t, width), 2).bfloat16()
    g = (1 + 0.1 * randn((width,), 3)).bfloat16()
    q = torch.zeros((t, width), dtype=torch.uint8, device="cuda")
    s = torch.zeros((t, 12), device="cuda")
    y = torch.empty_like(x)
    st = torch.cuda.Stream()

    def both():
        lib.mla_norm_rows(lib.MLA_BF16, x, width, res, width, g, t, width, 1e-6, None, 0, y, width, None, 0, None, st)
        lib.mla_quantize_rows(lib.MLA_BF16, y, width, t, width, q, width, s, st)

    with torch.cuda.stream(st):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        both()
    for seed in (10, 11):
        x.copy_(randn((t, width), seed))
        graph.replay()
        torch.cuda.synchronize()
        near(y, norm_ref(x, res, g, 1e-6)[1])
        check_codes(q, s, y.double(), width, 2.0 ** -24)


# ------------------------------------------------------------------ offsets past 32 bits
def test_norm_and_quantize_offsets_past_32_bits(lib):
    """300 001 rows of 7168: the last ones lie past 2^31 elements (bf16) and bytes (codes)."""
    t, width = 300_001, 7168
    x = torch.empty((t, width), dtype=torch.bfloat16, device="cuda")
    x[:8], x[-8:] = randn((8, width), 1).bfloat16(), randn((8, width), 2).bfloat16()
    x[8:-8] = 1
    q = torch.empty((t, width), dtype=torch.uint8, device="cuda")
    s = torch.empty((t, 56), device="cuda")
    for norm in (True, False):
        q.fill_(99)
        if norm:
            lib.mla_norm_rows(lib.MLA_BF16, x, width, None, 0, None, t, width, 1e-6, None, 0, None, 0, q, width, s)
        else:
            lib.mla_quantize_rows(lib.MLA_BF16, x, width, t, width, q, width, s)
        torch.cuda.synchronize()
        for part in (slice(0, 8), slice(t - 8, t)):
            y = norm_ref(x[part], None, None, 1e-6)[1] if norm else x[part].double()
            check_codes(q[part], s[part], y, width, REL if norm else 2.0 ** -24)
    assert lib.mla_check_device_error()[0] == 0


@pytest.mark.parametrize("act,kind", KINDS)
def test_append_rows_offsets_past_32_bits(lib, act, kind):
    """Pages whose rows lie past 2^31 elements of the pool (2^32 bytes for the 8-bit one)."""
    d_c, d_rope, pages = 512, 64, 60_000 if kind != "fp8" else 140_000
    c = Cache(lib, act, kind, d_c, d_rope, 64, (128,))
    for name in ("rows", "scales", "rope"):
        old = getattr(c, name)
        if old is not None:
            setattr(c, name, torch.zeros((pages * 64, old.shape[1]), dtype=old.dtype, device="cuda"))
    c.table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    c.desc = lib.mla_cache(p(c.rows), p(c.scales), p(c.rope), c.table.data_ptr(), 2, pages, 1)
    kv = randn((128, 576), 5).to(act)
    seq = torch.zeros(128, dtype=torch.int32, device="cuda")
    pos = torch.arange(128, dtype=torch.int32, device="cuda")
    cos, sin = rope_tables(lib, d_rope, 128)
    lib.mla_append_rows(c.dims, kv, 576, 128, seq, pos, None, 0.0, cos, sin, 128, c.desc)
    torch.cuda.synchronize()
    assert lib.mla_check_device_error()[0] == 0
    at = c.slots(seq, pos)
    if kind == "fp8":
        check_codes(c.rows[at], c.scales[at], kv[:, :512].double(), 512, 2.0 ** -24)
    else:
        near(c.rows[at][:, :512], kv[:, :512].double(), 0.0)
    assert not c.rows[64:(pages - 1) * 64].any()


def test_calls_follow_the_current_stream(lib):
    """Without a stream argument a call goes to torch's current stream."""
    t, width = 2000, 4096
    st = torch.cuda.Stream()
    x = torch.zeros((t, width), dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty((t, width), dtype=torch.uint8, device="cuda"), torch.empty((t, 32), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(20):
            x.add_(0.25)  # (in order only on the same stream)
        lib.mla_quantize_rows(lib.MLA_BF16, x, width, t, width, q, width, s)
    st.synchronize()
    check_codes(q, s, torch.full((t, width), 5.0, dtype=torch.float64, device="cuda"), width, 2.0 ** -24)


def test_tensors_on_no_or_another_device_are_refused(lib):
    x = torch.zeros((2, 64), device="cuda")
    host = torch.zeros((2, 64))
    with pytest.raises(ValueError):
        lib.mla_quantize_rows(lib.MLA_F32, host, 64, 2, 64, x, 64, x)
    with pytest.raises(lib.MlaError):
        lib.mla_quantize_rows(lib.MLA_F32, x, 63, 2, 64, x, 64, x)


def test_append_rows_codes_are_append_caches_codes(lib):
    """8-bit cache, the same latents bit for bit (identity weights): the same codes and scales from both calls, for blocks
    of zeros and of any size from 2^-100 up."""
    lengths, d_c, d_rope = (5, 70), 512, 64
    T, W = sum(lengths), d_c + d_rope
    a, b = (Cache(lib, torch.bfloat16, "fp8", d_c, d_rope, 64, lengths) for _ in range(2))
    size = torch.exp2(torch.linspace(-99, 99, T, device="cuda"))[:, None]
    h = (randn((T, W), 12).clamp(-4, 4).sign() * (1 + randn((T, W), 13).abs().clamp(max=3)) * size).bfloat16()
    h[3, :128] = 0
    seq = torch.repeat_interleave(torch.arange(2), torch.tensor(lengths)).int().cuda()
    pos = torch.cat([torch.arange(n) for n in lengths]).int().cuda()
    cos, sin = rope_tables(lib, d_rope, 128)
    eye = torch.eye(W, device="cuda").bfloat16()
    dims = lib.mla_dims(W, d_c, d_rope, 64, 128, 4, 64, lib.MLA_BF16, lib.MLA_FP8_E4M3, 0.1)
    n = lib.mla_append_workspace_size(dims, T)
    ws = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    lib.mla_append_cache(dims, h, T, seq, pos, eye[:d_c].contiguous(), eye[d_c:].contiguous(), cos, sin, 128, a.desc, ws, n)
    lib.mla_append_rows(b.dims, h, W, T, seq, pos, None, 0.0, cos, sin, 128, b.desc)
    torch.cuda.synchronize()
    assert lib.mla_check_device_error()[0] == 0
    at = b.slots(seq, pos)
    assert torch.equal(a.rows[at], b.rows[at]) and torch.equal(a.scales[at], b.scales[at])


@pytest.mark.parametrize("d_rope", [64, 258])  # (the second goes by elements)
def test_append_rows_tiny_and_nan_blocks(lib, d_rope):
    """A latent block below 2^-100 is coded against 2^-100; one with a NaN or an infinity stands for NaN; the blocks
    beside it are as ever."""
    d_c, T = 256, 4
    c = Cache(lib, torch.bfloat16, "fp8", d_c, d_rope, 64, (T,))
    kv = randn((T, d_c + d_rope), 14).bfloat16()
    kv[0, :128] = (1e-38 * randn((128,), 15)).bfloat16()
    kv[0, 5] = 0
    kv[1, 3], kv[2, 4] = float("nan"), float("inf")
    seq, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    cos, sin = rope_tables(lib, d_rope, 64)
    lib.mla_append_rows(c.dims, kv, d_c + d_rope, T, seq, pos, None, 0.0, cos, sin, 64, c.desc)
    torch.cuda.synchronize()
    assert lib.mla_check_device_error()[0] == 0
    q, s, y = c.rows[c.slots(seq, pos)], c.scales[c.slots(seq, pos)], kv[:, :d_c].double()
    assert torch.isnan(decoded(q, s, d_c)[1:3, :128]).all()
    check_codes(q[[0, 3]], s[[0, 3]], y[[0, 3]], d_c, 2.0 ** -24)
    check_codes(q[1:3, 128:].contiguous(), s[1:3, 1:], y[1:3, 128:], 128, 2.0 ** -24)


# a warp a row; a CTA a row; walking CTAs; a CTA a row of more values; streaming CTAs (bf16, f32); four chunks a thread; by
# elements with a warp and with a CTA a row; rows read twice
@pytest.mark.parametrize("act", ACT)
@pytest.mark.parametrize("t,width", [(300, 512), (5, 1536), (2500, 1536), (40, 7168), (1300, 7168), (700, 16384), (3, 32768),
                                     (700, 301), (601, 1501), (5, 8191), (2, 16385)])
@pytest.mark.parametrize("sum_over", ["residual", "x"])
def test_norm_in_place_everywhere(lib, act, t, width, sum_over):
    """sum_out over the residual with y over x, and sum_out over x (with and without a residual), in every kernel."""
    g = (1 + 0.1 * randn((width,), 3)).to(act)
    for with_res in ((True,) if sum_over == "residual" else (True, False)):
        x = randn((t, width), 1).to(act)
        res = randn((t, width), 2).to(act) if with_res else None
        r, want = norm_ref(x, res, g, 1e-5)
        q = torch.empty((t, width), dtype=torch.uint8, device="cuda")
        s = torch.empty((t, -(-width // 128)), device="cuda")
        y = x if sum_over == "residual" else torch.empty_like(x)
        total = res if sum_over == "residual" else x
        lib.mla_norm_rows(dt(lib, act), x, width, res, width, g, t, width, 1e-5, total, width, y, width, q, width, s)
        torch.cuda.synchronize()
        near(total, r, 2.0 ** -24)
        near(y, want)
        check_codes(q, s, want, width)
    assert lib.mla_check_device_error()[0] == 0
