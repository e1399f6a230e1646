"""The operators around the (grouped) MX GEMM of a feed-forward block, as cases to measure.

Six kinds of pass, each one call (or the two calls that always go together) of
the package's binding:

  norm          residual addition, RMS norm, MXFP8 output with E8M0 scales
  norm_back     its gradients (dx, dweight)
  dispatch      token slots sorted by expert, then each token's row quantised
                and written to its experts' rows
  combine       the experts' rows summed back to tokens with routing weights
                (or without them: dispatch's gradient)
  combine_back  combine's gradients (expert rows and routing weights)
  glu           gated activation, MXFP8 output, MXFP8 checkpoint of its inputs
  glu_back      its gradient and its recomputed output, from that checkpoint

``run`` computes a pass in elementary torch operations in FP32, or, with
``own`` set, through the package.  8-bit codes come back as float8 E4M3 values
and scales as E8M0 values; packed 4-bit codes come back as their bytes.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 32  # values that share a scale


# ---------------------------------------------------------------- the cases --

def listed():
    return [
        # one decode step of eight sequences, hidden size 8192: latency
        dict(name="norm_decode_8x8192", kind="norm", rows=8, K=8192, dtype="bf16", residual=True, plain=False,
             tiled=False),
        # a long prefill at the same hidden size, scales straight into the GEMM's tile layout
        dict(name="norm_prefill_16384x8192", kind="norm", rows=16384, K=8192, dtype="bf16", residual=True,
             plain=False, tiled=True),
        # first norm of a layer stack in FP32 (no residual yet), a ragged token count; the router also wants plain y
        dict(name="norm_f32_1023x5120", kind="norm", rows=1023, K=5120, dtype="f32", residual=False, plain=True,
             tiled=False),
        # a training step's norm gradient, hidden size 4096
        dict(name="norm_back_8192x4096", kind="norm_back", rows=8192, K=4096, dtype="bf16", residual=True),
        # a short ragged sequence trained in FP32, no gradient from the residual stream
        dict(name="norm_back_f32_301x5120", kind="norm_back", rows=301, K=5120, dtype="f32", residual=False),
        # decode batch of 32 tokens on 64 fine-grained experts
        dict(name="dispatch_decode_32x2048", kind="dispatch", tokens=32, topk=8, groups=64, K=2048, dtype="bf16",
             fmt="mxfp8", dropped=False),
        # long prefill on the same experts
        dict(name="dispatch_prefill_16384x2048", kind="dispatch", tokens=16384, topk=8, groups=64, K=2048,
             dtype="bf16", fmt="mxfp8", dropped=False),
        # eight wide experts, 4-bit codes, some slots dropped by an expert's capacity
        dict(name="dispatch_fp4_4099x4096", kind="dispatch", tokens=4099, topk=2, groups=8, K=4096, dtype="bf16",
             fmt="mxfp4", dropped=True),
        # the experts' rows back to tokens, added to the residual stream
        dict(name="combine_8192x4096", kind="combine", tokens=8192, topk=2, groups=8, N=4096, dtype="bf16",
             weighted=True, add=True, dropped=False),
        # its gradient on fine-grained experts with dropped slots
        dict(name="combine_back_8192x2048", kind="combine_back", tokens=8192, topk=8, groups=64, N=2048,
             dtype="bf16", dropped=True),
        # the gated activation of a training step, with its 8-bit checkpoint
        dict(name="glu_8192x14336", kind="glu", rows=8192, F=14336, dtype="bf16", act="silu", checkpoint=True,
             tiled=False),
        # and its gradient from that checkpoint
        dict(name="glu_back_8192x14336", kind="glu_back", rows=8192, F=14336, dtype="bf16", act="silu"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    """A row length up to 128 * hi: an odd count of 128-value tiles, or a power of two."""
    n = _spread(rng, 4, hi)
    return 128 * (2 ** int(math.log2(n)) if rng.random() < 0.4 else min(n | 1, hi - 1))


def draw(rng):
    kind = rng.choice(["norm", "norm_back", "dispatch", "combine", "combine_back", "glu", "glu_back"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    e = 2 if dtype == "bf16" else 4
    if kind in ("norm", "norm_back"):
        K = _width(rng, 64)
        if rng.random() < 0.5:
            K -= 32 * rng.randrange(1, 4)  # whole scale blocks, but no whole 128-value tiles
        rows = _spread(rng, 1, min(16384, 240_000_000 // (e * K)))
        c = dict(kind=kind, rows=rows, K=K, dtype=dtype, residual=rng.random() < 0.7)
        if kind == "norm":
            c.update(plain=rng.random() < 0.4, tiled=K % 128 == 0 and rng.random() < 0.5)
        return c
    if kind in ("glu", "glu_back"):
        F = _width(rng, 224)
        if kind == "glu_back" or rng.random() < 0.5:
            F -= 32 * rng.randrange(0, 4)
        rows = _spread(rng, 1, min(16384, 200_000_000 // (e * F)))
        c = dict(kind=kind, rows=rows, F=F, dtype=dtype, act=rng.choice(["silu", "silu", "gelu"]))
        if kind == "glu":
            c.update(checkpoint=rng.random() < 0.6, tiled=F % 128 == 0 and rng.random() < 0.5)
        return c
    groups = rng.choice([4, 8, 16, 60, 64, 128, 256])
    topk = rng.randrange(1, min(8, groups) + 1)
    K = _width(rng, 64)
    tokens = _spread(rng, 1, min(16384, 250_000_000 // (e * K * topk)))
    c = dict(kind=kind, tokens=tokens, topk=topk, groups=groups, dtype=dtype, dropped=rng.random() < 0.4)
    if kind == "dispatch":
        c.update(K=K, fmt=rng.choice(["mxfp8", "mxfp8", "mxfp4"]))
    elif kind == "combine":
        c.update(N=K, weighted=rng.random() < 0.7, add=rng.random() < 0.5)
    else:
        c.update(N=K)
    return c


# ---------------------------------------------------------------- their work --

def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    mx = 1 + 1 / BLOCK
    if c["kind"] == "norm":
        n = c["rows"] * c["K"]
        per = e + (2 * e if c["residual"] else 0) + (e if c["plain"] else 0) + mx
        return {"bytes": n * per + e * c["K"] + 4 * c["rows"], "flops": 8 * n}
    if c["kind"] == "norm_back":
        n = c["rows"] * c["K"]
        return {"bytes": n * e * (4 if c["residual"] else 3) + (e + 4) * c["K"] + 4 * c["rows"], "flops": 12 * n}
    if c["kind"] == "glu":
        n = c["rows"] * c["F"]
        return {"bytes": n * (2 * e + mx + (2 * mx if c["checkpoint"] else 0)), "flops": 10 * n}
    if c["kind"] == "glu_back":
        n = c["rows"] * c["F"]
        return {"bytes": n * (e + 2 * mx + 3 * e), "flops": 20 * n}
    T, k = c["tokens"], c["topk"]
    if c["kind"] == "dispatch":
        per = mx if c["fmt"] == "mxfp8" else 0.5 + 1 / BLOCK
        return {"bytes": T * c["K"] * (e + k * per) + T * k * (8 + 4 + 4) + 8 * (c["groups"] + 1),
                "flops": 3 * T * c["K"]}
    n = T * c["N"]
    if c["kind"] == "combine":
        return {"bytes": n * e * (k + 1 + (1 if c["add"] else 0)) + T * k * (8 if c["weighted"] else 4),
                "flops": 2 * n * k}
    return {"bytes": n * e * (1 + 2 * k) + T * k * 12, "flops": 3 * n * k}


# -------------------------------------------------------------------- inputs --

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)


def _hidden(gen, rows, K, dtype):
    """A hidden state: unit normal values and a few channels that are much larger, as residual streams have them."""
    x = torch.randn((rows, K), generator=gen, device=DEV, dtype=torch.float32)
    big = torch.randint(0, K, (max(1, K // 512),), generator=gen, device=DEV)
    x[:, big] *= 20.0
    return x.to(dtype)


def _route(gen, c):
    """Top-k expert ids (int64) with an uneven load, and their softmax weights; some slots dropped (-1), one token whole."""
    T, G, k = c["tokens"], c["groups"], c["topk"]
    scores = torch.randn((T, G), generator=gen, device=DEV) + torch.randn((G,), generator=gen, device=DEV)
    top, ids = torch.topk(scores, k, dim=1)
    weights = torch.softmax(top, dim=1)
    if c["dropped"]:
        ids = torch.where(torch.rand((T, k), generator=gen, device=DEV) < 0.05, -1, ids)
        ids[T // 3] = -1
    return ids.contiguous(), weights.contiguous()


def _sorted(ids, groups):
    """offsets, row_of_slot, slot_of_row of a stable sort of the slots by expert; dropped slots last, as -1 - row."""
    flat = ids.reshape(-1)
    good = (flat >= 0) & (flat < groups)
    key = torch.where(good, flat, groups)
    order = torch.sort(key, stable=True).indices
    rows = torch.empty_like(order)
    rows[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.bincount(key, minlength=groups + 1)[:groups]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return offsets, torch.where(good, rows, -1 - rows).to(torch.int32), order.to(torch.int32)


def _mx_buffers(s, rows, K, fmt="mxfp8", tiled=False, key=""):
    """Buffers for codes and scales that the program keeps from pass to pass, and the values they stand for."""
    s[key + "codes"] = torch.empty((rows, K if fmt == "mxfp8" else K // 2), dtype=torch.uint8, device=DEV)
    shape = (((rows + 127) // 128) * (K // 128) * 512,) if tiled else (rows, K // BLOCK)
    s[key + "scales"] = torch.empty(shape, dtype=torch.uint8, device=DEV)
    s[key + "code_values"] = s[key + "codes"].view(torch.float8_e4m3fn) if fmt == "mxfp8" else s[key + "codes"]
    s[key + "scale_values"] = s[key + "scales"].view(torch.float8_e8m0fnu)


def prepare(case, seed):
    c, dt = case, _dtype(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case=c)
    if c["kind"] in ("norm", "norm_back"):
        rows, K = c["rows"], c["K"]
        s["w"] = (1.0 + 0.2 * torch.randn((K,), generator=gen, device=DEV)).to(dt)
        if c["kind"] == "norm":
            s["x"] = _hidden(gen, rows, K, dt)
            s["r"] = _hidden(gen, rows, K, dt) if c["residual"] else None
            s["h"] = torch.empty((rows, K), dtype=dt, device=DEV) if c["residual"] else None
            s["y"] = torch.empty((rows, K), dtype=dt, device=DEV) if c["plain"] else None
            s["rstd"] = torch.empty((rows,), dtype=torch.float32, device=DEV)
            _mx_buffers(s, rows, K, tiled=c["tiled"])
        else:
            s["h"] = _hidden(gen, rows, K, dt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + 1e-5)
            s["dy"] = _normal(gen, (rows, K), dt, 0.02)
            s["dh"] = _normal(gen, (rows, K), dt, 0.02) if c["residual"] else None
            s["dx"] = torch.empty((rows, K), dtype=dt, device=DEV)
            s["dw"] = torch.empty((K,), dtype=torch.float32, device=DEV)
    elif c["kind"] in ("glu", "glu_back"):
        rows, F = c["rows"], c["F"]
        gu = _normal(gen, (rows, 2 * F), dt, 1.5)
        if c["kind"] == "glu":
            s["gu"] = gu
            _mx_buffers(s, rows, F, tiled=c["tiled"])
            if c["checkpoint"]:
                _mx_buffers(s, rows, 2 * F, key="kept_")
        else:
            v, sc = _quantize(gu.float(), "mxfp8")
            s["kept_codes"], s["kept_scales"] = v.view(torch.uint8), sc.view(torch.uint8)
            s["dy"] = _normal(gen, (rows, F), dt, 0.02)
            s["dgu"] = torch.empty((rows, 2 * F), dtype=dt, device=DEV)
            s["a"] = torch.empty((rows, F), dtype=dt, device=DEV)
    else:
        T, k = c["tokens"], c["topk"]
        s["ids"], s["weights"] = _route(gen, c)
        if c["kind"] == "dispatch":
            s["x"] = _hidden(gen, T, c["K"], dt)
            s["offsets"] = torch.empty((c["groups"] + 1,), dtype=torch.int64, device=DEV)
            s["row_of_slot"] = torch.empty((T * k,), dtype=torch.int32, device=DEV)
            s["slot_of_row"] = torch.empty((T * k,), dtype=torch.int32, device=DEV)
            _mx_buffers(s, T * k, c["K"], c["fmt"])
        else:
            N = c["N"]
            offsets, s["row_of_slot"], _ = _sorted(s["ids"], c["groups"])
            s["y"] = _normal(gen, (T * k, N), dt)
            if c["dropped"]:  # rows that no expert computes hold whatever the memory held
                s["y"][torch.arange(T * k, device=DEV) >= offsets[-1]] = float("nan")
            if c["kind"] == "combine":
                if not c["weighted"]:
                    s["weights"] = None
                s["add"] = _normal(gen, (T, N), dt) if c["add"] else None
                s["out"] = torch.empty((T, N), dtype=dt, device=DEV)
            else:
                s["dout"] = _normal(gen, (T, N), dt, 0.02)
                s["dy"] = torch.empty((T * k, N), dtype=dt, device=DEV)
                s["dweights"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------ the plain form --

def _pow2(code):
    """2^(code - 127) for whole codes 1..254, from the exponent bits."""
    return (code.to(torch.int32) << 23).view(torch.float32)


def _quantize(x, fmt):
    """MX codes and E8M0 scales of FP32 x [rows, K], one scale for 32 values."""
    b = x.reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1
    code = torch.where(amax > 0, (e - (8 if fmt == "mxfp8" else 2) + 127).clamp(min=0), 127)
    v = b * _pow2(254 - code).unsqueeze(-1)
    bad = ~torch.isfinite(amax)
    v = torch.where(bad.unsqueeze(-1), 0.0, v)
    code = torch.where(bad, 255, code)
    scales = code.to(torch.uint8).view(torch.float8_e8m0fnu)
    if fmt == "mxfp8":
        return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).reshape(x.shape), scales
    m = v.abs()
    n = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
         + 8 * torch.signbit(v)).to(torch.uint8).reshape(x.shape)
    return n[:, 0::2] | (n[:, 1::2] << 4), scales


def _dequantize(codes, scales, dtype=torch.float32):
    b = codes.view(torch.float8_e4m3fn).to(dtype)
    return (b.reshape(b.shape[0], -1, BLOCK) * scales.view(torch.float8_e8m0fnu).to(dtype).unsqueeze(-1)).reshape(b.shape)


def _tile(scales):
    """Row-major scales [rows, K/32] -> 512-byte tiles [ceil(rows/128)][K/128]: the scale of row 32q + p of a row
    block and block c of a K-tile at byte 16p + 4q + c; rows past the end hold 1.0."""
    rows, nb = scales.shape
    b = scales.view(torch.uint8)
    pad = -rows % 128
    b = torch.cat([b, b.new_full((pad, nb), 127)]) if pad else b
    b = b.reshape(-1, 4, 32, nb // 4, 4).permute(0, 3, 2, 1, 4)
    return b.contiguous().reshape(-1).view(torch.float8_e8m0fnu)


def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(g, act):
    if act == "silu":
        q = torch.sigmoid(g)
        return q * (1.0 + g * (1.0 - q))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _run_plain(s):
    c, dt = s["case"], _dtype(s["case"])
    if c["kind"] == "norm":
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
        rstd = torch.rsqrt(h.square().mean(1) + 1e-5)
        y = h * rstd.unsqueeze(1) * s["w"].float()
        codes, scales = _quantize(y, "mxfp8")
        return {"h": h.to(dt) if s["r"] is not None else None, "y": y.to(dt) if c["plain"] else None, "codes": codes,
                "scales": _tile(scales) if c["tiled"] else scales, "rstd": rstd}
    if c["kind"] == "norm_back":
        h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
        p = dy * s["w"].float()
        dx = rstd * p - h * (rstd * rstd * rstd * (p * h).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dw": (dy * h * rstd).sum(0)}
    if c["kind"] == "glu":
        gu = s["gu"].float()
        g, u = gu[:, :c["F"]], gu[:, c["F"]:]
        codes, scales = _quantize(_act(g, c["act"]) * u, "mxfp8")
        out = {"codes": codes, "scales": _tile(scales) if c["tiled"] else scales}
        if c["checkpoint"]:
            out["kept_codes"], out["kept_scales"] = _quantize(gu, "mxfp8")
        return out
    if c["kind"] == "glu_back":
        gu, dy = _dequantize(s["kept_codes"], s["kept_scales"]), s["dy"].float()
        g, u = gu[:, :c["F"]], gu[:, c["F"]:]
        f = _act(g, c["act"])
        dgu = torch.cat([dy * u * _act_slope(g, c["act"]), dy * f], 1)
        return {"dgu": dgu.to(dt), "a": (f * u).to(dt)}
    k = c["topk"]
    if c["kind"] == "dispatch":
        offsets, row_of_slot, slot_of_row = _sorted(s["ids"], c["groups"])
        codes, scales = _quantize(s["x"].float(), c["fmt"])
        token = (slot_of_row // k).long()
        kept = (torch.arange(token.numel(), device=DEV) < offsets[-1]).unsqueeze(1)
        rows = torch.where(kept, codes.view(torch.uint8)[token], 0)
        scales = torch.where(kept, scales.view(torch.uint8)[token], 127)
        return {"offsets": offsets, "row_of_slot": row_of_slot, "slot_of_row": slot_of_row,
                "codes": rows.view(torch.float8_e4m3fn) if c["fmt"] == "mxfp8" else rows,
                "scales": scales.view(torch.float8_e8m0fnu)}
    slot = s["row_of_slot"].reshape(-1, k).long()
    dead = (slot < 0).unsqueeze(-1)
    y = torch.where(dead, 0.0, s["y"][torch.where(slot < 0, -1 - slot, slot)].float())
    if c["kind"] == "combine":
        if s["weights"] is not None:
            y = y * torch.where(dead, 0.0, s["weights"].unsqueeze(-1))
        out = y.sum(1)
        if s["add"] is not None:
            out = out + s["add"].float()
        return {"out": out.to(dt)}
    dout = s["dout"].float().unsqueeze(1)
    dy = torch.empty_like(s["dy"])
    dy[torch.where(slot < 0, -1 - slot, slot).reshape(-1)] = torch.where(
        dead, 0.0, dout * s["weights"].unsqueeze(-1)).to(dt).reshape(-1, c["N"])
    return {"dy": dy, "dweights": (dout * y).sum(-1)}


# ----------------------------------------------------------- the package's --

def _run_own(s):
    from mx_block_scaled_gb300 import binding as mx
    c = s["case"]
    if c["kind"] == "norm":
        mx.rmsnorm(s["x"], s["w"], 1e-5, residual=s["r"], fmt=mx.MXGEMM_FMT_MXFP8_E4M3, tiled=c["tiled"], h=s["h"],
                   y=s["y"], codes=s["codes"], scales=s["scales"], rstd=s["rstd"])
        return {"h": s["h"], "y": s["y"], "codes": s["code_values"], "scales": s["scale_values"], "rstd": s["rstd"]}
    if c["kind"] == "norm_back":
        mx.rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["w"], dh=s["dh"], dx=s["dx"], dweight=s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if c["kind"] in ("glu", "glu_back"):
        act = mx.MXGEMM_ACT_SILU if c["act"] == "silu" else mx.MXGEMM_ACT_GELU_TANH
        if c["kind"] == "glu":
            F = c["F"]
            mx.glu(s["gu"][:, :F], s["gu"][:, F:], act, fmt=mx.MXGEMM_FMT_MXFP8_E4M3, tiled=c["tiled"],
                   codes=s["codes"], scales=s["scales"], kept_codes=s.get("kept_codes"),
                   kept_scales=s.get("kept_scales"))
            out = {"codes": s["code_values"], "scales": s["scale_values"]}
            if c["checkpoint"]:
                out["kept_codes"], out["kept_scales"] = s["kept_code_values"], s["kept_scale_values"]
            return out
        mx.glu_backward(s["dy"], act, kept_codes=s["kept_codes"], kept_scales=s["kept_scales"], dgu=s["dgu"], a=s["a"])
        return {"dgu": s["dgu"], "a": s["a"]}
    if c["kind"] == "dispatch":
        fmt = mx.MXGEMM_FMT_MXFP8_E4M3 if c["fmt"] == "mxfp8" else mx.MXGEMM_FMT_MXFP4_E2M1
        mx.moe_sort(s["ids"], c["groups"], offsets=s["offsets"], row_of_slot=s["row_of_slot"],
                    slot_of_row=s["slot_of_row"])
        mx.moe_dispatch(s["x"], s["row_of_slot"], fmt, rows=s["codes"], scales=s["scales"])
        return {"offsets": s["offsets"], "row_of_slot": s["row_of_slot"], "slot_of_row": s["slot_of_row"],
                "codes": s["code_values"], "scales": s["scale_values"]}
    if c["kind"] == "combine":
        mx.moe_combine(s["y"], s["row_of_slot"], c["topk"], weights=s["weights"], add=s["add"], out=s["out"])
        return {"out": s["out"]}
    mx.moe_combine_backward(s["dout"], s["y"], s["row_of_slot"], s["weights"], dy=s["dy"], dweights=s["dweights"])
    return {"dy": s["dy"], "dweights": s["dweights"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------- the definition in 64 bits --

def _x_quantize(x, fmt):
    """Code values and scale values of 64-bit x by rounding on the element grid (e4m3: 3 fraction bits from 2^-6 up to
    448; e2m1: 1 from 1 up to 6)."""
    top, low, bits, most = (8, -6, 3, 448.0) if fmt == "mxfp8" else (2, 0, 1, 6.0)
    b = x.reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, (torch.frexp(amax).exponent - 1 - top).clamp(min=-127), 0).double()
    v = b * torch.exp2(-s)
    q = torch.exp2(((torch.frexp(v).exponent - 1).clamp(min=low) - bits).double())
    v = (torch.round(v / q) * q).clamp(-most, most)
    return v.reshape(x.shape), torch.exp2(s).reshape(x.shape[0], -1)


def _x_tile(scales):
    rows, nb = scales.shape
    r = torch.arange((rows + 127) // 128 * 128, device=scales.device).unsqueeze(1)
    j = torch.arange(nb, device=scales.device).unsqueeze(0)
    at = (r // 128 * (nb // 4) + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4
    out = torch.ones(at.numel(), dtype=torch.float64, device=scales.device)
    out[at[:rows].reshape(-1)] = scales.reshape(-1)
    return out


def _x_slots(ids, groups):
    """(offsets, row_of_slot, slot_of_row), counted on the host."""
    flat = ids.reshape(-1).cpu().numpy()
    key = np.where((flat >= 0) & (flat < groups), flat, groups)
    order = np.argsort(key, kind="stable")
    rows = np.empty(flat.size, np.int64)
    rows[order] = np.arange(flat.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=groups + 1)[:groups])])
    return offsets.astype(np.int64), np.where(key < groups, rows, -1 - rows).astype(np.int32), order.astype(np.int32)


def _x_act(g, act):
    """Value and slope of the activation."""
    if act == "silu":
        q = 1.0 / (1.0 + torch.exp(-g))
        return g * q, q + g * q * (1.0 - q)
    z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    q = 1.0 / (1.0 + torch.exp(-z))  # (1 + tanh(z / 2)) / 2
    return g * q, q + g * q * (1.0 - q) * math.sqrt(8 / math.pi) * (1.0 + 0.134145 * g * g)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h += s["r"].double()
        rstd = (h.pow(2).sum(1) / c["K"] + 1e-5).pow(-0.5)
        y = h * s["w"].double() * rstd[:, None]
        codes, scales = _x_quantize(y, "mxfp8")
        return {"h": h if s["r"] is not None else None, "y": y if c["plain"] else None, "codes": codes,
                "scales": _x_tile(scales) if c["tiled"] else scales, "rstd": rstd}
    if c["kind"] == "norm_back":
        h, dy, w, rstd = s["h"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()[:, None]
        n = h * rstd
        dn = dy * w
        dx = rstd * (dn - n * ((dn * n).sum(1, keepdim=True) / c["K"]))
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dw": (dy * n).sum(0)}
    if c["kind"] == "glu":
        gu = s["gu"].double()
        f, _ = _x_act(gu[:, :c["F"]], c["act"])
        codes, scales = _x_quantize(f * gu[:, c["F"]:], "mxfp8")
        out = {"codes": codes, "scales": _x_tile(scales) if c["tiled"] else scales}
        if c["checkpoint"]:
            out["kept_codes"], out["kept_scales"] = _x_quantize(gu, "mxfp8")
        return out
    if c["kind"] == "glu_back":
        codes = s["kept_codes"].view(torch.float8_e4m3fn).double()
        gu = codes * torch.repeat_interleave(torch.exp2(s["kept_scales"].double() - 127), BLOCK, dim=1)
        f, slope = _x_act(gu[:, :c["F"]], c["act"])
        u, dy = gu[:, c["F"]:], s["dy"].double()
        return {"dgu": torch.cat([dy * u * slope, dy * f], 1), "a": f * u}
    offsets, row_of_slot, slot_of_row = _x_slots(s["ids"], c["groups"])
    k, dev = c["topk"], s["ids"].device
    dead = torch.from_numpy(row_of_slot < 0).to(dev)
    row = torch.from_numpy(np.where(row_of_slot < 0, -1 - row_of_slot, row_of_slot)).to(dev).long()
    if c["kind"] == "dispatch":
        v, sc = _x_quantize(s["x"].double(), c["fmt"])
        codes = v.new_zeros((c["tokens"] * k, c["K"]))
        scales = v.new_ones((c["tokens"] * k, c["K"] // BLOCK))
        live = torch.nonzero(~dead).reshape(-1)
        codes[row[live]] = v[live // k]
        scales[row[live]] = sc[live // k]
        if c["fmt"] == "mxfp4":  # whole numbers: each byte two positions among 0, .5, 1, 1.5, 2, 3, 4, 6, and their signs
            grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=dev)
            n = torch.searchsorted(grid, codes.abs().contiguous()) + 8 * torch.signbit(codes)
            codes = (n[:, 0::2] + 16 * n[:, 1::2]).to(torch.uint8)
        return {"offsets": offsets, "row_of_slot": row_of_slot, "slot_of_row": slot_of_row, "codes": codes,
                "scales": scales}
    y = s["y"].double()
    w = s["weights"].double().reshape(-1) if s["weights"] is not None else y.new_ones(row.numel())
    if c["kind"] == "combine":
        out = s["add"].double() if s["add"] is not None else y.new_zeros((c["tokens"], c["N"]))
        live = torch.nonzero(~dead).reshape(-1)
        out.index_add_(0, live // k, y[row[live]] * w[live, None])
        return {"out": out}
    dout = s["dout"].double()
    dy, dw = torch.zeros_like(y), y.new_zeros(row.numel())
    live = torch.nonzero(~dead).reshape(-1)
    dy[row[live]] = dout[live // k] * w[live, None]
    dw[live] = (dout[live // k] * y[row[live]]).sum(1)
    return {"dy": dy, "dweights": dw.reshape(-1, k)}
