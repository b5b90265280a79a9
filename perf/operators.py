"""Timed cases of the operators around the quantized GEMMs of a training step.

Four operators, each with the direction(s) a training step runs:

  gemm / gemm_bwd   block-scaled matrix product with bias, activation and residual in its epilogue, and the
                    backward pass of that epilogue (gradient of the pre-activation, bias gradient)
  norm / norm_bwd   root-mean-square norm of a residual stream, bf16 or 8-bit (E4M3 x UE8M0) output, and its backward
  balance           mixture-of-experts balance loss, per-expert counts and the gradient of the router's logits
  clip              global norm of many gradients, and the clipped gradients

``run`` computes them in elementary torch operations, or with the library's calls where ``own`` is set; ``exact``
computes the same definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
ACTS = ("none", "relu", "gelu", "silu")
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E1M2, E2M1, E4M3 = 0, 1, 3                     # grids of the quantized operands
E1M2_LEVELS = [k / 4 for k in range(8)]
E2M1_LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3_OF_E1M2 = [0x00, 0x28, 0x30, 0x34, 0x38, 0x3A, 0x3C, 0x3E]     # E4M3 bytes of k / 4
CORR_OF_E1M2 = [0, 1, 2, 3, 4, 4, 4, 2]        # E2M1 codes of k - e(k)


def listed():
    return [
        # the smallest layer of the tests: an FFN's first product on 8-bit activations, all of the epilogue
        {"name": "gemm_tiny", "op": "gemm", "kind": "mx", "m": 256, "n": 512, "k": 512, "act": "gelu", "bias": True,
         "residual": True, "pre": False, "out": "bf16"},
        # one linear layer, 8192 tokens: 8-bit activations from the norm, 4-bit weights, the pre-activation kept for
        # the backward pass
        {"name": "gemm_layer_mx", "op": "gemm", "kind": "mx", "m": 8192, "n": 8192, "k": 2048, "act": "gelu",
         "bias": True, "residual": False, "pre": True, "out": "bf16"},
        # the large layer's down projection, both operands in the uniform 4-bit grid, added to the residual stream
        {"name": "gemm_large_ufp4", "op": "gemm", "kind": "ufp4", "m": 16384, "n": 8192, "k": 28672, "act": "none",
         "bias": True, "residual": True, "pre": False, "out": "bf16"},
        # backward of a ragged batch's activation, fp32 gradient as DGRAD writes it
        {"name": "gemm_bwd_ragged", "op": "gemm_bwd", "m": 1111, "n": 1408, "act": "silu", "dout": "fp32"},
        # backward of the large layer's activation
        {"name": "gemm_bwd_large", "op": "gemm_bwd", "m": 16384, "n": 28672, "act": "gelu", "dout": "bf16"},
        # one token of the large layer's width: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 8192, "stream": "bf16", "residual": True, "y": "mx8"},
        # the large layer's input: residual stream in, 8-bit operand of the next product out
        {"name": "norm_large_mx8", "op": "norm", "rows": 16384, "cols": 8192, "stream": "bf16", "residual": True,
         "y": "mx8"},
        # the same norm's backward, with the gradient of the residual stream added in
        {"name": "norm_bwd_large", "op": "norm_bwd", "rows": 16384, "cols": 8192, "dy": "bf16", "stream": "bf16"},
        # a small router: 512 tokens, 8 experts, top-2, bf16 logits, padding tokens masked
        {"name": "balance_small", "op": "balance", "tokens": 512, "experts": 8, "topk": 2, "type": "bf16",
         "masked": True},
        # a long batch over many experts
        {"name": "balance_large", "op": "balance", "tokens": 131072, "experts": 256, "topk": 8, "type": "fp32",
         "masked": False},
        # the gradients of one small layer: few and short tensors, latency
        {"name": "clip_small", "op": "clip", "tensors": 6, "elements": 300_000, "type": "fp32", "out": "bf16"},
        # the fp32 weight gradients of a mixture-of-experts layer and its dense layers
        {"name": "clip_large", "op": "clip", "tensors": 48, "elements": 600_000_000, "type": "fp32", "out": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm_bwd", "norm", "norm", "norm_bwd", "balance", "clip"])
    if op == "gemm":
        # any number of tokens from one up; any width; K is padded to 64 by the operand's layout
        return {"op": op, "kind": rng.choice(["mx", "ufp4", "e2m1"]), "m": _spread(rng, 1, 8192),
                "n": _spread(rng, 33, 8192), "k": _spread(rng, 64, 8192), "act": rng.choice(ACTS),
                "bias": rng.random() < 0.7, "residual": rng.random() < 0.5, "pre": rng.random() < 0.3,
                "out": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "gemm_bwd":
        return {"op": op, "m": _spread(rng, 1, 16384), "n": _spread(rng, 33, 16384), "act": rng.choice(ACTS[1:]),
                "dout": rng.choice(["bf16", "fp32"])}
    if op == "norm":
        return {"op": op, "rows": _spread(rng, 1, 16384), "cols": _spread(rng, 64, 8192),
                "stream": rng.choice(["bf16", "fp32"]), "residual": rng.random() < 0.7, "y": rng.choice(["bf16", "mx8"])}
    if op == "norm_bwd":
        return {"op": op, "rows": _spread(rng, 1, 16384), "cols": _spread(rng, 64, 8192),
                "dy": rng.choice(["bf16", "fp32"]), "stream": rng.choice(["bf16", "fp32"])}
    if op == "balance":
        experts = _spread(rng, 4, 256)
        return {"op": op, "tokens": _spread(rng, 1, 131072), "experts": experts, "topk": min(experts, rng.randint(1, 8)),
                "type": rng.choice(["bf16", "fp32"]), "masked": rng.random() < 0.5}
    return {"op": op, "tensors": rng.randint(1, 48), "elements": _spread(rng, 1000, 200_000_000),
            "type": rng.choice(["bf16", "fp32"]), "out": rng.choice(["bf16", "fp32"])}


# ---------------------------------------------------------------- inputs
def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _kpad(k):
    return (k + 63) // 64 * 64


def _up(v, a):
    return (v + a - 1) // a * a


def _padded_blocks(x, block):
    """fp32 [rows, blocks, block] of a [rows, k] tensor, zero-padded to a multiple of 64 columns."""
    rows, k = x.shape
    full = torch.zeros(rows, _kpad(k), device=DEV)
    full[:, :k] = x
    return full.view(rows, -1, block)


def _exponents(amax, gmax):
    """The smallest X with amax <= gmax 2^X, within [-127, 127]; -127 for a zero block (whole numbers, exact)."""
    mant, ex = torch.frexp(amax.double())                  # amax = mant 2^ex, mant in [0.5, 1)
    gm, ge = math.frexp(gmax)
    x = ex - ge + (mant > gm).to(ex.dtype)
    return torch.where(amax > 0, x, torch.full_like(x, -127)).clamp(-127, 127)


def _atoms(fac, rows):
    """The factor-atom plane of block factors [blocks, >= rows]: 512-byte atoms of 128 rows x 4 factors."""
    nb = fac.shape[0]
    full = torch.zeros(_up(rows, 128), _up(nb, 4), dtype=torch.uint8, device=DEV)
    full[:rows, :nb] = fac[:, :rows].t()
    v = full.view(full.shape[0] // 128, 4, 32, full.shape[1] // 4, 4)
    return v.permute(0, 3, 2, 1, 4).reshape(full.shape[0] // 128, full.shape[1] // 4, 512).contiguous()


def _block_major(fac, rows):
    """[rows, blocks] bytes -> [blocks, rows rounded up to 64], the padding zero."""
    out = torch.zeros(fac.shape[1], _up(rows, 64), dtype=torch.uint8, device=DEV)
    out[:, :rows] = fac.t()
    return out


def _pack(nib):
    return (nib[:, 0::2] | (nib[:, 1::2] << 4)).contiguous()


def _quantized(x, kind, grid):
    """A quantized operand in the library's layout, as its quantizer leaves one (unrotated data stands for the
    rotated values; the codes are to the nearest level)."""
    rows, k = x.shape
    q = {"rows": rows, "k": k, "kpad": _kpad(k), "grid": grid, "kind": kind}
    if kind == "mx":
        b = _padded_blocks(x.float(), 32)
        e = _exponents(b.abs().amax(2), 448.0 if grid == E4M3 else 1.75)
        v = b * torch.exp2(-e.float())[:, :, None]
        q["scales"] = _block_major((e + 127).to(torch.uint8), rows)
        if grid == E4M3:
            q["elems8"] = v.to(torch.float8_e4m3fn).view(torch.uint8).view(rows, -1)
        else:
            mag = (v.abs() * 4).round().clamp(max=7).to(torch.int32).view(rows, -1)
            sign = (v.view(rows, -1) < 0) & (mag > 0)
            q["codes"] = _pack((mag + 8 * sign).to(torch.uint8))
            q["elems8"] = torch.tensor(E4M3_OF_E1M2, dtype=torch.uint8, device=DEV)[mag] | (128 * sign).to(torch.uint8)
    else:
        b = _padded_blocks(x.float(), 16)
        gmax = 1.75 if grid == E1M2 else 6.0
        amax = b.abs().amax(2)
        s = (amax.max() / (gmax * 448.0)).float()
        f8 = (amax / (gmax * s)).to(torch.float8_e4m3fn)
        step = (f8.float() * s)[:, :, None]
        v = torch.where(step > 0, b / step, torch.zeros_like(b)).view(rows, -1).clamp(-gmax, gmax)
        levels = torch.tensor(E1M2_LEVELS if grid == E1M2 else E2M1_LEVELS, device=DEV)
        mids = (levels[1:] + levels[:-1]) / 2
        mag = torch.bucketize(v.abs(), mids, out_int32=True)
        sign = (v < 0) & (mag > 0)
        nib = (mag + 8 * sign).to(torch.uint8)
        q["scales"] = _block_major(f8.view(torch.uint8), rows)
        q["tensor_scale"] = s.view(1).clone()
        if grid == E1M2:     # codes and their correction plane in one allocation, as the quantizer lays them out
            d = torch.tensor(CORR_OF_E1M2, dtype=torch.uint8, device=DEV)[mag] | (8 * sign).to(torch.uint8)
            q["planes"] = torch.stack([_pack(nib), _pack(d)])
        else:
            q["planes"] = _pack(nib)[None]
    q["atoms"] = _atoms(q["scales"], rows)
    return q


def _outliers(g, x, frac=0.01, factor=50.0):
    """A few input channels larger than the others, as in the large layer's activations."""
    cols = x.shape[1]
    at = torch.randperm(cols, generator=g, device=DEV)[: max(1, int(frac * cols))]
    x[:, at] *= factor
    return x


def _sizes(case):
    """Tensor sizes of a model's gradients: a few large matrices, some of them odd, and short vectors."""
    n, total = case["tensors"], case["elements"]
    w = [0.001 if i % 3 == 2 else 1.0 + (i * 7 % 5) for i in range(n)]
    return [max(1, int(total * v / sum(w))) + (i % 2) for i, v in enumerate(w)]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    op, s = case["op"], {"case": case, "op": case["op"]}
    if op == "gemm":
        m, n, k, kind = case["m"], case["n"], case["k"], case["kind"]
        x = _outliers(g, torch.randn(m, k, generator=g, device=DEV))
        w = torch.randn(n, k, generator=g, device=DEV) * 0.02
        s["a"] = _quantized(x, kind, {"mx": E4M3, "ufp4": E1M2, "e2m1": E2M1}[kind])
        s["b"] = _quantized(w, kind, {"mx": E1M2, "ufp4": E1M2, "e2m1": E2M1}[kind])
        s["hadamard"] = 0 if kind == "mx" else 16
        s["bias"] = _normal(g, n, std=0.5) if case["bias"] else None
        s["residual"] = _normal(g, m, n) if case["residual"] else None
        s["pre"] = torch.empty(m, n, dtype=torch.bfloat16, device=DEV) if case["pre"] else None
    elif op == "gemm_bwd":
        s["dout"] = _normal(g, case["m"], case["n"], std=1e-3, dtype=TYPES[case["dout"]])
        s["pre"] = _normal(g, case["m"], case["n"], std=1.5)
    elif op == "norm":
        rows, cols, st = case["rows"], case["cols"], TYPES[case["stream"]]
        s["x"] = _normal(g, rows, cols)
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=g, device=DEV)).to(torch.bfloat16)
        s["residual"] = _outliers(g, _normal(g, rows, cols, std=2.0, dtype=st)) if case["residual"] else None
        if not case["residual"]:
            s["x"] = s["x"].to(st)
        s["eps"] = 1e-5
        s["h"] = torch.empty(rows, cols, dtype=st, device=DEV) if case["residual"] else None
        if case["y"] == "mx8":   # the operand's planes, kept from step to step
            kp = _kpad(cols)
            s["elems8"] = torch.zeros(rows, kp, dtype=torch.uint8, device=DEV)
            s["scales"] = torch.zeros(kp // 32, _up(rows, 64), dtype=torch.uint8, device=DEV)
            s["atoms"] = torch.zeros(_up(rows, 128) // 128, _up(kp, 128) // 128, 512, dtype=torch.uint8, device=DEV)
    elif op == "norm_bwd":
        rows, cols, st = case["rows"], case["cols"], TYPES[case["stream"]]
        s["dy"] = _normal(g, rows, cols, std=1e-3, dtype=TYPES[case["dy"]])
        s["h"] = _outliers(g, _normal(g, rows, cols, std=2.0, dtype=st))
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=g, device=DEV)).to(torch.bfloat16)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + 1e-5).float()
        s["dh"] = _normal(g, rows, cols, std=1e-3, dtype=st)
    elif op == "balance":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        lean = torch.randn(e, generator=g, device=DEV)           # some experts are liked better
        logits = (torch.randn(t, e, generator=g, device=DEV) + lean).to(TYPES[case["type"]])
        s["logits"] = logits
        s["experts"] = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
        s["mask"] = (torch.rand(t, generator=g, device=DEV) < 0.9) if case["masked"] else None
        s["coef"] = 0.01
        s["dloss"] = torch.full((1,), 1.0, device=DEV)
    else:
        s["grads"] = [_normal(g, n, std=10.0 ** (-4 + i % 3), dtype=TYPES[case["type"]])
                      for i, n in enumerate(_sizes(case))]
        s["out"] = [torch.empty(t.numel(), dtype=TYPES[case["out"]], device=DEV) for t in s["grads"]]
        s["max_norm"] = 1.0
    return s


# ---------------------------------------------------------------- the framework's calls
def _operand(u, q, hadamard):
    mx = q["kind"] == "mx"
    cfg = u.QuantConfig(grid=q["grid"], hadamard_n=hadamard, block=32 if mx else 16,
                        scale_fmt=u.SCALE_UE8M0 if mx else u.SCALE_E4M3_X_FP32)
    planes = q.get("planes")
    return u.QTensor(codes=planes[0] if planes is not None else q.get("codes"), scales=q["scales"],
                     tensor_scale=q.get("tensor_scale"), rows=q["rows"], k=q["k"], kpad=q["kpad"],
                     scale_ld=q["scales"].shape[1], cfg=cfg,
                     corr=planes[1] if planes is not None and q["grid"] == E1M2 else None,
                     elems8=q.get("elems8"), sf_atoms=q["atoms"])


def _run_own(s):
    from fp4_quantized_gemms_b200 import ufp4 as u
    c = s["case"]
    act = {"none": u.ACT_NONE, "relu": u.ACT_RELU, "gelu": u.ACT_GELU, "silu": u.ACT_SILU}
    if s["op"] == "gemm":
        out = u.gemm_epilogue(_operand(u, s["a"], s["hadamard"]), _operand(u, s["b"], s["hadamard"]), bias=s["bias"],
                              act=act[c["act"]], residual=s["residual"], pre=s["pre"], out_dtype=TYPES[c["out"]])
        return {"out": out, "pre": s["pre"]}
    if s["op"] == "gemm_bwd":
        dpre, dbias = u.epilogue_backward(s["dout"], s["pre"], act[c["act"]])
        return {"dpre": dpre, "dbias": dbias}
    if s["op"] == "norm":
        q = None
        if c["y"] == "mx8":
            q = u.QTensor(codes=None, scales=s["scales"], tensor_scale=None, rows=c["rows"], k=c["cols"],
                          kpad=_kpad(c["cols"]), scale_ld=s["scales"].shape[1],
                          cfg=u.QuantConfig(grid=u.GRID_E4M3, hadamard_n=0, block=32, scale_fmt=u.SCALE_UE8M0),
                          elems8=s["elems8"], sf_atoms=s["atoms"])
        y, _, h, rstd = u.rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=s["eps"], q=q, h=s["h"])
        got = {"rstd": rstd}
        if s["residual"] is not None:
            got["h"] = h
        if q is None:
            got["y"] = y
        else:
            got.update(elems=s["elems8"].view(torch.float8_e4m3fn), scales=s["scales"].view(torch.float8_e8m0fnu),
                       atoms=s["atoms"].view(torch.float8_e8m0fnu))
        return got
    if s["op"] == "norm_bwd":
        dx, dw = u.rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dweight": dw}
    if s["op"] == "balance":
        loss, counts, tokens = u.moe_balance(s["logits"], s["experts"], coef=s["coef"], mask=s["mask"])
        dlogits = u.moe_balance_backward(s["logits"], counts, tokens, s["dloss"], topk=c["topk"], coef=s["coef"],
                                         mask=s["mask"])
        return {"loss": loss, "counts": counts, "dlogits": dlogits}
    norm = u.grad_clip(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "clipped": s["out"]}


# ---------------------------------------------------------------- the plain forms
def _decoded(q):
    """fp32 [rows, kpad] values of a quantized operand."""
    rows = q["rows"]
    if q["kind"] == "mx":
        v = q["elems8"].view(torch.float8_e4m3fn).float().view(rows, -1, 32)
        f = torch.exp2(q["scales"][:, :rows].t().float() - 127.0)
        return (v * f[:, :, None]).view(rows, -1)
    lv = E1M2_LEVELS if q["grid"] == E1M2 else E2M1_LEVELS
    lut = torch.tensor(lv + [-v for v in lv], device=DEV)
    codes = q["planes"][0]
    nib = torch.stack([codes & 15, codes >> 4], dim=2).view(rows, -1)
    f = q["scales"][:, :rows].t().contiguous().view(torch.float8_e4m3fn).float() * q["tensor_scale"]
    return (lut[nib.to(torch.int32)].view(rows, -1, 16) * f[:, :, None]).view(rows, -1)


def _act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _dact(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    if name == "gelu":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _run_plain(s):
    c = s["case"]
    if s["op"] == "gemm":
        z = torch.matmul(_decoded(s["a"]), _decoded(s["b"]).t())
        if s["hadamard"]:
            z = z / s["hadamard"]
        if s["bias"] is not None:
            z = z + s["bias"].float()
        v = _act(z, c["act"])
        if s["residual"] is not None:
            v = v + s["residual"].float()
        return {"out": v.to(TYPES[c["out"]]), "pre": z.to(torch.bfloat16) if c["pre"] else None}
    if s["op"] == "gemm_bwd":
        d = s["dout"].float() * _dact(s["pre"].float(), c["act"])
        return {"dpre": d.to(torch.bfloat16), "dbias": d.sum(0)}
    if s["op"] == "norm":
        h, got = s["x"], {}
        if s["residual"] is not None:
            h = (s["x"].float() + s["residual"].float()).to(TYPES[c["stream"]])
            got["h"] = h
        h = h.float()
        rstd = torch.rsqrt(h.square().mean(1) + s["eps"])
        got["rstd"] = rstd
        y = h * rstd[:, None] * s["weight"].float()
        if c["y"] == "bf16":
            got["y"] = y.to(torch.bfloat16)
        else:
            rows = c["rows"]
            b = _padded_blocks(y, 32)
            e = _exponents(b.abs().amax(2), 448.0)
            v = b * torch.exp2(-e.float())[:, :, None]
            fac = _block_major((e + 127).to(torch.uint8), rows)
            got.update(elems=v.to(torch.float8_e4m3fn).view(rows, -1), scales=fac.view(torch.float8_e8m0fnu),
                       atoms=_atoms(fac, rows).view(torch.float8_e8m0fnu))
        return got
    if s["op"] == "norm_bwd":
        xhat = s["h"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        gy = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (gy - xhat * (gy * xhat).mean(1, keepdim=True)) + s["dh"].float()
        return {"dx": dx.to(TYPES[c["stream"]]), "dweight": (dy * xhat).sum(0)}
    if s["op"] == "balance":
        x = s["logits"].float()
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        t, e, k = c["tokens"], c["experts"], c["topk"]
        chosen = s["experts"].long()
        if s["mask"] is not None:
            p = p * s["mask"][:, None]
            ones = s["mask"][:, None].expand(t, k).reshape(-1).long()
            n = s["mask"].sum()
        else:
            ones = torch.ones(t * k, dtype=torch.int64, device=DEV)
            n = torch.tensor(t, device=DEV)
        counts = torch.zeros(e, dtype=torch.int64, device=DEV).index_add_(0, chosen.reshape(-1), ones)
        n = n.clamp(min=1).float()
        f = counts.float() / (n * k)
        loss = s["coef"] * e * (f * (p.sum(0) / n)).sum()
        ge = s["dloss"] * s["coef"] * e * f / n
        d = p * (ge - (p * ge).sum(1, keepdim=True))       # masked rows have p = 0
        return {"loss": loss.view(1), "counts": counts, "dlogits": d.to(TYPES[c["type"]])}
    norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    return {"norm": norm.view(1), "clipped": [(t.float() * coef).to(TYPES[c["out"]]) for t in s["grads"]]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _values64(q):
    r = torch.arange(q["rows"], device=DEV)
    if q["kind"] == "mx":
        by = q["elems8"].to(torch.int32)
        ex, man = (by >> 3) & 15, (by & 7).double()
        mag = torch.where(ex == 0, man * 2.0 ** -9, torch.ldexp(1 + man / 8, ex - 7))
        v = torch.where(by >= 128, -mag, mag)
        e = q["scales"].to(torch.int32)[:, r] - 127
        step = torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)
        width = 32
    else:
        by = q["planes"][0]
        nib = torch.empty(q["rows"], 2 * by.shape[1], dtype=torch.uint8, device=DEV)
        nib[:, 0::2], nib[:, 1::2] = by % 16, by // 16
        k = (nib % 8).double()
        if q["grid"] == E2M1:
            mag = torch.where(k < 4, k / 2, torch.where(k < 6, k - 2, 2 * k - 8))
        else:
            mag = k / 4
        v = torch.where(nib >= 8, -mag, mag)
        sc = q["scales"].to(torch.int32)[:, r]
        ex, man = (sc >> 3) & 15, (sc & 7).double()
        step = torch.where(ex == 0, man * 2.0 ** -9, torch.ldexp(1 + man / 8, ex - 7)) * q["tensor_scale"].double()
        width = 16
    return v * step.t().repeat_interleave(width, dim=1)


def _sigmoid64(z):
    return torch.where(z >= 0, 1 / (1 + torch.exp(-z.abs())), torch.exp(-z.abs()) / (1 + torch.exp(-z.abs())))


def _e4m3_64(v):
    """The nearest E4M3 values, ties to even (at most 448)."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        z = _values64(s["a"]) @ _values64(s["b"]).T
        z *= 1.0 / max(1, s["hadamard"])
        if s["bias"] is not None:
            z += s["bias"].double()
        a = case["act"]
        if a == "relu":
            v = torch.where(z > 0, z, torch.zeros_like(z))
        elif a == "silu":
            v = z * _sigmoid64(z)
        elif a == "gelu":      # 0.5 (1 + tanh u) = sigmoid(2 u)
            v = z * _sigmoid64(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        else:
            v = z
        if s["residual"] is not None:
            v = v + s["residual"].double()
        return {"out": v, "pre": z if case["pre"] else None}
    if op == "gemm_bwd":
        z, a = s["pre"].double(), case["act"]
        if a == "relu":
            d = torch.where(z > 0, 1.0, 0.0).double()
        elif a == "silu":
            sg = _sigmoid64(z)
            d = sg + z * sg * _sigmoid64(-z)
        else:
            w = 2 * math.sqrt(2 / math.pi)
            sg = _sigmoid64(w * (z + 0.044715 * z ** 3))
            d = sg + z * sg * (1 - sg) * w * (1 + 0.134145 * z ** 2)
        d = d * s["dout"].double()
        return {"dpre": d, "dbias": d.sum(0)}
    if op == "norm":
        got, h = {}, s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(TYPES[case["stream"]]).double()     # the stream as it is stored
            got["h"] = h
        rstd = 1 / torch.sqrt((h * h).sum(1) / case["cols"] + s["eps"])
        got["rstd"] = rstd
        y = h * rstd[:, None] * s["weight"].double()
        if case["y"] == "bf16":
            got["y"] = y
            return got
        rows, kp = case["rows"], _kpad(case["cols"])
        full = torch.zeros(rows, kp, dtype=torch.float64, device=DEV)
        full[:, : case["cols"]] = y
        amax = full.view(rows, kp // 32, 32).abs().amax(2)
        m, ex = torch.frexp(amax)                               # 448 = 0.875 * 2^9
        x = (ex - 9 + (m > 0.875).to(ex.dtype)).clamp(-127, 127)
        x = torch.where(amax == 0, torch.full_like(x, -127), x)
        step = torch.ldexp(torch.ones_like(amax), x)
        got["elems"] = _e4m3_64(full / step.repeat_interleave(32, dim=1))
        low = 2.0 ** -127
        sc = torch.full((kp // 32, _up(rows, 64)), low, dtype=torch.float64, device=DEV)
        sc[:, :rows] = step.t()
        got["scales"] = sc
        at = torch.full((_up(rows, 128) // 128, _up(kp, 128) // 128, 512), low, dtype=torch.float64, device=DEV)
        r = torch.arange(rows, device=DEV)[:, None]
        b = torch.arange(kp // 32, device=DEV)[None, :]
        at[r // 128, b // 4, 16 * (r % 32) + 4 * ((r // 32) % 4) + b % 4] = step
        got["atoms"] = at
        return got
    if op == "norm_bwd":
        h, r, dy = s["h"].double(), s["rstd"].double()[:, None], s["dy"].double()
        gy = dy * s["weight"].double()
        dot = (gy * h).sum(1, keepdim=True) / case["cols"]
        return {"dx": gy * r - h * dot * r ** 3 + s["dh"].double(), "dweight": (dy * h * r).sum(0)}
    if op == "balance":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        keep = s["mask"] if s["mask"] is not None else torch.ones(t, dtype=torch.bool, device=DEV)
        x = s["logits"].double()
        p = torch.exp(x - torch.logsumexp(x, dim=1, keepdim=True))
        counts = torch.bincount(s["experts"][keep].long().reshape(-1), minlength=e)
        n = max(1, int(keep.sum()))
        f = counts.double() / (n * k)
        loss = s["coef"] * e * (f @ p[keep].sum(0)) / n
        w = s["dloss"].double() * s["coef"] * e * f / n
        d = p * w - p * (p @ w)[:, None]
        d[~keep] = 0
        return {"loss": loss.view(1), "counts": counts, "dlogits": d}
    total = math.sqrt(sum(float(t.double().square().sum()) for t in s["grads"]))
    coef = s["max_norm"] / total if total > s["max_norm"] else 1.0
    return {"norm": torch.tensor([total], dtype=torch.float64), "clipped": [t.double() * coef for t in s["grads"]]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "gemm":
        m, n, k = case["m"], case["n"], _kpad(case["k"])
        per = {"mx": (1 + 1 / 32, 0.5 + 1 / 32), "ufp4": (0.5 + 1 / 16,) * 2, "e2m1": (0.5 + 1 / 16,) * 2}[case["kind"]]
        out = m * n * (size[case["out"]] + 2 * case["residual"] + 2 * case["pre"]) + 2 * n * case["bias"]
        return {"bytes": m * k * per[0] + n * k * per[1] + out, "flops": 2.0 * m * n * case["k"]}
    if op == "gemm_bwd":
        mn = case["m"] * case["n"]
        return {"bytes": mn * (size[case["dout"]] + 2 + 2) + 4 * case["n"], "flops": 15.0 * mn}
    if op == "norm":
        rc, st = case["rows"] * case["cols"], size[case["stream"]]
        moved = 2 + 2 * st if case["residual"] else st
        y = 2 if case["y"] == "bf16" else 1 + 2 / 32
        return {"bytes": rc * (moved + y) + 4 * case["rows"] + 2 * case["cols"], "flops": 6.0 * rc}
    if op == "norm_bwd":
        rc = case["rows"] * case["cols"]
        return {"bytes": rc * (size[case["dy"]] + 3 * size[case["stream"]]) + 4 * case["rows"] + 6 * case["cols"],
                "flops": 12.0 * rc}
    if op == "balance":
        te = case["tokens"] * case["experts"]
        return {"bytes": te * 2 * size[case["type"]] + case["tokens"] * (4 * case["topk"] + case["masked"])
                + 8 * case["experts"], "flops": 12.0 * te}
    n = sum(_sizes(case))
    return {"bytes": n * (size[case["type"]] + size[case["out"]]), "flops": 3.0 * n}
