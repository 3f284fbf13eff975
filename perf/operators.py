"""Workloads of the operators around the attention core of an MLA layer: the norm in front of a projection (with the
residual's addition and an 8-bit output), the 8-bit quantisation of rows, the 8-bit projection with block scales, and
the append of already projected rows to the paged latent cache.

A case is a dict with ``op`` one of "norm", "quantize", "project", "append".  ``run`` computes it in elementary torch
operations, or with the library's calls where the module's ``own`` is true.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128      # values that share a scale
E4M3_MAX = 448.0
PAGE = 64
EPS = 1e-6
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of a small model: hidden 2048 to latent + rotary key; latency counts
        dict(name="project 1x576x2048", op="project", rows=1, n=576, k=2048, act="bf16"),
        # decode step of 64 sequences: hidden 7168 to a query rank of 1536 + latent 512 + rotary key 64
        dict(name="project 64x2112x7168", op="project", rows=64, n=2112, k=7168, act="bf16"),
        # the same step's output projection, 128 heads x 128 values to hidden
        dict(name="project 64x7168x16384", op="project", rows=64, n=7168, k=16384, act="bf16"),
        # ragged everywhere: an odd number of outputs, a reduction that ends inside a scale block, fp32 results
        dict(name="project 333x1999x2000 f32", op="project", rows=333, n=1999, k=2000, act="f32"),
        # prefill chunk through the output projection
        dict(name="project 2048x7168x16384", op="project", rows=2048, n=7168, k=16384, act="bf16"),
        # one token, hidden 7168, residual added, 8-bit output for the next projection
        dict(name="norm 1x7168", op="norm", rows=1, width=7168, act="bf16", residual=True, keep=False),
        # the query rank's norm of a mixed batch: no residual, the first columns of a fused down projection's rows
        dict(name="norm 391x1536", op="norm", rows=391, width=1536, act="bf16", residual=False, keep=True),
        # prefill: residual added, the sum, the normed rows and their 8-bit form all written
        dict(name="norm 8191x7168", op="norm", rows=8191, width=7168, act="bf16", residual=True, keep=True),
        # attention output of a decode step, 128 heads x 128 values
        dict(name="quantize 64x16384", op="quantize", rows=64, width=16384, act="bf16"),
        # prefill, 16 heads x 128 values, in fp32
        dict(name="quantize 4099x2048 f32", op="quantize", rows=4099, width=2048, act="f32"),
        # one new token for each of 64 sequences, latent norm applied, 8-bit cache
        dict(name="append 64 fp8", op="append", rows=64, seqs=64, act="bf16", cache="fp8", norm=True),
        # prefill of 5 sequences into a 16-bit cache with shuffled pages
        dict(name="append 40007 bf16", op="append", rows=40007, seqs=5, act="bf16", cache="bf16", norm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["project", "project", "norm", "quantize", "append"])
    act = rng.choice(["bf16", "bf16", "f32"])
    if op == "project":
        rows, n = _log(rng, 1, 4096), _log(rng, 64, 24576)
        k = 16 * _log(rng, 8, 1024) if rng.random() < 0.3 else 128 * _log(rng, 1, 128)
        most = 2048 * 7168 * 16384 // 2
        rows = max(1, min(rows, most // (n * k)))
        return dict(op=op, rows=rows, n=n, k=k, act=act)
    if op == "append":
        rows = _log(rng, 1, 40000)
        cache = "f32" if act == "f32" else rng.choice(["bf16", "fp8"])
        return dict(op=op, rows=rows, seqs=min(rows, _log(rng, 1, 128)), act=act, cache=cache, norm=rng.random() < 0.7)
    width = rng.choice([512, 1536, 2048, 7168, 16384, 8 * _log(rng, 16, 2048), _log(rng, 100, 16384)])
    rows = min(_log(rng, 1, 16384), max(1, (8191 * 7168 // 2) // width))
    if op == "quantize":
        return dict(op=op, rows=rows, width=width, act=act)
    return dict(op=op, rows=rows, width=width, act=act, residual=rng.random() < 0.6, keep=rng.random() < 0.5)


def work(case):
    e = 2 if case.get("act") == "bf16" else 4
    t, op = case["rows"], case["op"]
    if op == "project":
        n, k = case["n"], case["k"]
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        return dict(bytes=t * k + 4 * t * kb + n * k + 4 * nb * kb + t * n * e, flops=2 * t * n * k)
    if op == "append":
        out = 512 + 16 + 128 if case["cache"] == "fp8" else 576 * (2 if case["cache"] == "bf16" else 4)
        return dict(bytes=t * (576 * e + 64 * 4 + 12 + out) + (512 * e if case["norm"] else 0),
                    flops=t * (512 * 5 + 64 * 3))
    w = case["width"]
    out = t * w + 4 * t * -(-w // BLOCK)
    if op == "quantize":
        return dict(bytes=t * w * e + out, flops=t * w * 3)
    reads = t * w * e * (2 if case["residual"] else 1) + w * e
    writes = out + t * w * e * ((1 if case["residual"] else 0) + (1 if case["keep"] else 0))
    return dict(bytes=reads + writes, flops=t * w * 8)


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _codes(rows, width):
    return torch.zeros((rows, width), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)


def _quantize(x):
    """E4M3 codes and scales, one for each 128 values of a row, of fp32 rows [T, D]."""
    t, d = x.shape
    kb = -(-d // BLOCK)
    p = torch.nn.functional.pad(x, (0, kb * BLOCK - d)).view(t, kb, BLOCK)
    amax = p.abs().amax(-1)
    zero = amax == 0
    scales = torch.where(zero, torch.ones_like(amax), amax / E4M3_MAX)
    inv = torch.where(zero, torch.ones_like(amax), E4M3_MAX / amax)
    codes = (p * inv[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(t, kb * BLOCK)[:, :d].contiguous(), scales


def _weights(gen, n, k):
    """8-bit weights [n, k], N(0, 1/k) before rounding, with one scale for each 128 x 128 block."""
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    w = _randn(gen, n, k) / math.sqrt(k)
    p = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(nb, BLOCK, kb, BLOCK)
    scales = p.abs().amax((1, 3)) / E4M3_MAX
    codes = (p / scales[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(nb * BLOCK, kb * BLOCK)[:n, :k].contiguous(), scales.contiguous()


def _pages(case, gen):
    """Lengths already cached, and the new tokens' sequences and positions, with a shuffled block table."""
    t, b = case["rows"], case["seqs"]
    per = [t // b + (1 if i < t % b else 0) for i in range(b)]
    before = torch.randint(0, 2048, (b,), generator=gen, device="cuda")
    per_t = torch.tensor(per, device="cuda")
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), per_t)
    first = torch.cumsum(per_t, 0) - per_t
    pos = torch.arange(t, device="cuda") - first[seq] + before[seq]
    max_pages = (2048 + max(per) + PAGE - 1) // PAGE
    table = torch.randperm(b * max_pages, generator=gen, device="cuda").view(b, max_pages)
    return seq.to(torch.int32), pos.to(torch.int32), table.to(torch.int32).contiguous(), b * max_pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, t = case["op"], case["rows"]
    act = ACT[case["act"]]
    s = dict(case=case, op=op, act=act)
    if op == "project":
        n, k = case["n"], case["k"]
        s["x"], s["xs"] = _quantize(_randn(gen, t, k))
        s["w"], s["ws"] = _weights(gen, n, k)
        s["out"] = torch.empty((t, n), dtype=act, device="cuda")
    elif op == "append":
        s["kv"] = _randn(gen, t, 576).to(act)
        s["gamma"] = (1 + 0.1 * _randn(gen, 512)).to(act) if case["norm"] else None
        s["seq"], s["pos"], s["table"], pages = _pages(case, gen)
        top = s["table"].shape[1] * PAGE
        freq = 10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64)
        angle = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float().contiguous(), angle.sin().float().contiguous()
        if case["cache"] == "fp8":
            s["rows"] = _codes(pages * PAGE, 512).view(pages, PAGE, 512)
            s["scales"] = torch.ones((pages, PAGE, 4), dtype=torch.float32, device="cuda")
            s["rope"] = torch.zeros((pages, PAGE, 64), dtype=torch.bfloat16, device="cuda")
        else:
            s["rows"] = torch.zeros((pages, PAGE, 576), dtype=ACT[case["cache"]], device="cuda")
    else:
        w = case["width"]
        fused = 576 if op == "norm" and not case["residual"] else 0
        s["x"] = _randn(gen, t, w + fused).to(act)[:, :w]
        s["codes"] = _codes(t, w)
        s["scales"] = torch.empty((t, -(-w // BLOCK)), dtype=torch.float32, device="cuda")
        if op == "norm":
            s["gamma"] = (1 + 0.1 * _randn(gen, w)).to(act)
            s["residual"] = (2 * _randn(gen, t, w)).to(act) if case["residual"] else None
            s["sum"] = torch.empty((t, w), dtype=act, device="cuda") if case["residual"] else None
            s["y"] = torch.empty((t, w), dtype=act, device="cuda") if case["keep"] else None
    if own:
        _plan(s, case)
    return s


def _plan(s, case):
    """What a program that uses the library keeps between calls: the module, its enums and descriptors."""
    import mla_latent_kv_27_b200 as mla
    s["mla"] = mla
    s["dt"] = mla.MLA_BF16 if case["act"] == "bf16" else mla.MLA_F32
    if case["op"] == "append":
        kind = {"bf16": mla.MLA_BF16, "fp8": mla.MLA_FP8_E4M3, "f32": mla.MLA_F32}[case["cache"]]
        s["dims"] = mla.mla_dims(2048, 512, 64, 128, 128, 16, PAGE, s["dt"], kind, 1.0)
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        s["desc"] = mla.mla_cache(ptr(s["rows"]), ptr(s.get("scales")), ptr(s.get("rope")), ptr(s["table"]),
                                  s["table"].shape[1], s["rows"].shape[0], s["table"].shape[0])


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["op"]
    if own:
        return {"project": _own_project, "append": _own_append, "norm": _own_norm, "quantize": _own_quantize}[op](state)
    return {"project": _plain_project, "append": _plain_append, "norm": _plain_norm, "quantize": _plain_quantize}[op](state)


def _own_project(s):
    t, k = s["x"].shape
    n = s["w"].shape[0]
    s["mla"].mla_project_fp8(s["dt"], s["x"], k, s["xs"], t, s["w"], s["ws"], n, k, s["out"], n)
    return s["out"]


def _own_norm(s):
    t, w = s["x"].shape
    s["mla"].mla_norm_rows(s["dt"], s["x"], s["x"].stride(0), s["residual"], w, s["gamma"], t, w, EPS, s["sum"], w, s["y"], w,
                           s["codes"], w, s["scales"])
    return {"codes": s["codes"], "scales": s["scales"], "sum": s["sum"], "y": s["y"]}


def _own_quantize(s):
    t, w = s["x"].shape
    s["mla"].mla_quantize_rows(s["dt"], s["x"], w, t, w, s["codes"], w, s["scales"])
    return {"codes": s["codes"], "scales": s["scales"]}


def _own_append(s):
    s["mla"].mla_append_rows(s["dims"], s["kv"], 576, s["kv"].shape[0], s["seq"], s["pos"], s["gamma"], EPS, s["cos"],
                             s["sin"], s["cos"].shape[0], s["desc"])
    return {"rows": s["rows"], "scales": s.get("scales"), "rope": s.get("rope")}


def _spread(x, scales):
    """Codes times their scales, in fp32: scales [R, C] stand for blocks of [R', 128] values, R' = 1 or 128 rows."""
    r, c = x.shape
    s = scales.repeat_interleave(BLOCK, 1)[:, :c]
    if s.shape[0] != r:
        s = s.repeat_interleave(BLOCK, 0)[:r]
    return x.float() * s


def _plain_project(s):
    return (_spread(s["x"], s["xs"]) @ _spread(s["w"], s["ws"]).t()).to(s["act"])


def _rms(x, gamma):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.to(x.dtype)


def _plain_norm(s):
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = _rms(r, s["gamma"])
    codes, scales = _quantize(y)
    return {"codes": codes, "scales": scales, "sum": None if s["sum"] is None else r.to(s["act"]),
            "y": None if s["y"] is None else y.to(s["act"])}


def _plain_quantize(s):
    codes, scales = _quantize(s["x"].float())
    return {"codes": codes, "scales": scales}


def _rotate(k, cos, sin):
    a, b = k[:, 0::2], k[:, 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(1)


def _plain_append(s):
    kv = s["kv"].float()
    pos = s["pos"].long()
    c = kv[:, :512]
    if s["gamma"] is not None:
        c = _rms(c, s["gamma"])
    k = _rotate(kv[:, 512:], s["cos"][pos], s["sin"][pos])
    page, slot = s["table"][s["seq"].long(), pos // PAGE].long(), pos % PAGE
    rows = s["rows"]
    if "rope" in s:
        codes, scales = _quantize(c)
        rows.view(torch.uint8)[page, slot] = codes.view(torch.uint8)
        s["scales"][page, slot] = scales
        s["rope"][page, slot] = k.to(torch.bfloat16)
        return {"rows": rows, "scales": s["scales"], "rope": s["rope"]}
    rows[page, slot] = torch.cat((c, k), 1).to(rows.dtype)
    return {"rows": rows, "scales": None, "rope": None}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_blocks(y):
    """(code values before rounding, scales) of fp64 rows."""
    vals, scales = [], []
    for part in y.split(BLOCK, dim=1):
        top = part.abs().max(1, keepdim=True).values
        step = torch.where(top > 0, top / 448, torch.ones_like(top))
        vals.append(part / step)
        scales.append(step)
    return torch.cat(vals, 1), torch.cat(scales, 1)


def _exact_norm(r, gamma):
    size = torch.linalg.vector_norm(r, dim=1, keepdim=True) / math.sqrt(r.shape[1])
    return gamma.double() * r / torch.sqrt(size ** 2 + EPS)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "project":
        total = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        row = torch.arange(case["n"], device="cuda") // BLOCK
        for b, k0 in enumerate(range(0, case["k"], BLOCK)):
            part = s["x"][:, k0:k0 + BLOCK].double() @ s["w"][:, k0:k0 + BLOCK].double().t()
            total += part * s["xs"][:, b, None].double() * s["ws"][row, b].double()
        return total
    if op == "append":
        kv = s["kv"].double()
        c = kv[:, :512] if s["gamma"] is None else _exact_norm(kv[:, :512], s["gamma"])
        turn = torch.polar(torch.ones(1, 1, dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * 10000.0 ** (-torch.arange(32, device="cuda").double() / 32))
        k = torch.view_as_real(torch.view_as_complex(kv[:, 512:].reshape(-1, 32, 2).contiguous()) * turn).reshape(-1, 64)
        at = s["table"].long()[s["seq"].long(), s["pos"].long() // PAGE] * PAGE + s["pos"].long() % PAGE

        def put(buf, new):
            buf = buf.double().flatten(0, 1)
            buf[at] = new
            return buf.view(-1, PAGE, new.shape[1])

        if case["cache"] == "fp8":
            vals, scales = _exact_blocks(c)
            return {"rows": put(s["rows"], vals), "scales": put(s["scales"], scales), "rope": put(s["rope"], k)}
        return {"rows": put(s["rows"], torch.cat((c, k), 1)), "scales": None, "rope": None}
    r = s["x"].double()
    if op == "quantize":
        vals, scales = _exact_blocks(r)
        return {"codes": vals, "scales": scales}
    if s["residual"] is not None:
        r = r + s["residual"].double()
    y = _exact_norm(r, s["gamma"])
    vals, scales = _exact_blocks(y)
    return {"codes": vals, "scales": scales, "sum": None if s["sum"] is None else r, "y": None if s["y"] is None else y}
