"""Helpers for the tests of the operators around the GEMMs: 64-bit values of
quantized operands, 8-bit operands from plain tensors, activations in 64 bits."""
import math

import torch

from fp4_quantized_gemms_b200 import ufp4

ACTS = {"none": ufp4.ACT_NONE, "relu": ufp4.ACT_RELU, "gelu": ufp4.ACT_GELU, "gelu_erf": ufp4.ACT_GELU_ERF,
        "silu": ufp4.ACT_SILU}
BF16, FP32 = torch.bfloat16, torch.float32


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def values64(q: ufp4.QTensor) -> torch.Tensor:
    """float64 [rows, kpad] values (rotated domain) of a quantized operand."""
    fmt, block = q.cfg.scale_fmt, q.cfg.block
    if fmt == ufp4.SCALE_FP32:
        step = q.scales.double()
    elif fmt == ufp4.SCALE_UE8M0:
        step = torch.exp2(q.scales.double() - 127)
    else:
        step = q.scales.view(torch.float8_e4m3fn).double() * q.tensor_scale.double()
    step = step[:, :q.rows].t().repeat_interleave(block, dim=1)
    if q.cfg.grid == ufp4.GRID_E4M3:
        return q.elems8.view(torch.float8_e4m3fn).double() * step
    lv = [k / 4 for k in range(8)] if q.cfg.grid == ufp4.GRID_E1M2 else [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    lut = torch.tensor(lv + [-v for v in lv], dtype=torch.float64, device=q.codes.device)
    nib = torch.stack([q.codes & 15, q.codes >> 4], dim=2).view(q.rows, q.kpad)
    return lut[nib.long()] * step


def product64(a: ufp4.QTensor, b: ufp4.QTensor) -> torch.Tensor:
    n = a.cfg.hadamard_n
    return values64(a) @ values64(b).t() / (n if n else 1)


def act64(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    return z


def slope64(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    if name == "gelu_erf":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


CFG8 = ufp4.QuantConfig(grid=ufp4.GRID_E4M3, hadamard_n=0, block=32, scale_fmt=ufp4.SCALE_UE8M0)


def eight_bit(x: torch.Tensor, atoms: bool = True) -> ufp4.QTensor:
    """An 8-bit operand of the float tensor x [rows, k], from the layout's definition."""
    rows, k = x.shape
    q = ufp4.empty_qtensor(rows, k, CFG8, device=x.device, with_atoms=atoms)
    full = torch.zeros(rows, q.kpad, dtype=torch.float64, device=x.device)
    full[:, :k] = x.double()
    b = full.view(rows, -1, 32)
    m, e = torch.frexp(b.abs().amax(2))
    X = torch.where(m > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -127)).clamp(-127, 127)
    v = (b * torch.exp2(-X.double())[:, :, None]).float().to(torch.float8_e4m3fn)
    q.elems8.copy_(v.view(torch.uint8).view(rows, -1))
    q.scales.zero_()
    q.scales[:, :rows] = (X + 127).to(torch.uint8).t()
    if atoms:
        q.sf_atoms.zero_()
        r = torch.arange(rows, device=x.device)[:, None]
        s = torch.arange(q.kpad // 32, device=x.device)[None, :]
        q.sf_atoms[r // 128, s // 4, 16 * (r % 32) + 4 * ((r // 32) % 4) + s % 4] = (X + 127).to(torch.uint8)
    return q


def rand(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def strided(t: torch.Tensor, pad: int, offset: int = 0) -> torch.Tensor:
    """The same matrix with a longer row pitch, `offset` elements into its allocation."""
    m, n = t.shape
    buf = torch.zeros(m * (n + pad) + offset, dtype=t.dtype, device=t.device)
    v = buf[offset:].view(m, n + pad)[:, :n]
    v.copy_(t)
    return v
