"""Refusals of the operators around the GEMMs: every bad argument is rejected
on the host, before any CUDA call (no GPU needed)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from fp4_quantized_gemms_b200 import build as ufp4_build
from fp4_quantized_gemms_b200 import ufp4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, BAD, UNSUP, ALIGN, MISMATCH = (ufp4.OK, ufp4.ERR_INVALID_ARG, ufp4.ERR_UNSUPPORTED, ufp4.ERR_ALIGNMENT,
                                   ufp4.ERR_OPERAND_MISMATCH)
P = 64 * 1024           # a made-up, well aligned device address


@pytest.fixture(scope="module")
def L():
    ufp4_build.build()
    return ufp4.lib()


def _layout_of(tmp_path, struct, fields):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ufp4.h"\nint main(void) {\n'
                   f'printf("%zu", sizeof({struct}));\n'
                   + "".join(f'printf(" %zu", offsetof({struct}, {f}));\n' for f in fields) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    return list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))


@pytest.mark.parametrize("struct,mirror", [("ufp4_epilogue_t", "EpilogueC"), ("ufp4_tensor_t", "TensorC")])
def test_struct_layouts(tmp_path, struct, mirror):
    c = getattr(ufp4, mirror)
    names = [f[0] for f in c._fields_]
    assert _layout_of(tmp_path, struct, names) == [ctypes.sizeof(c)] + [getattr(c, n).offset for n in names]


def _q(rows=128, k=256, elems8=None, **kw):
    cfg = ufp4.QuantConfig(**kw).c()
    kp = (k + 63) // 64 * 64
    codes = None if kw.get("grid") == ufp4.GRID_E4M3 else P
    return ufp4.QTensorC(codes, 2 * P, 3 * P if kw.get("scale_fmt") == 1 else None, rows, k, kp,
                         (rows + 63) // 64 * 64, cfg, None, elems8)


MX = dict(scale_fmt=ufp4.SCALE_UE8M0, block=32, hadamard_n=0)
E8 = dict(grid=ufp4.GRID_E4M3, **MX)


def test_eight_bit_operands(L):
    def layout(**kw):
        c = ufp4.QuantConfig(**kw).c()
        cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
        s = L.ufp4_qtensor_layout(100, 130, ctypes.byref(c), None, None, ctypes.byref(cb), ctypes.byref(sb))
        return s, cb.value, sb.value

    assert layout(**E8) == (OK, 0, 6 * 128)
    for bad in (dict(scale_fmt=ufp4.SCALE_FP32), dict(block=16), dict(hadamard_n=16), dict(rounding=1)):
        assert layout(**{**E8, **bad})[0] == BAD
    q8, q4 = _q(elems8=4 * P, **E8), _q(elems8=5 * P, grid=0, **MX)

    def gemm(a, b, ldc=64):           # ldc < N: a pair that is accepted gets as far as that check
        return L.ufp4_gemm_fprop(a, b, P, ldc, None)

    assert gemm(q8, q8) == BAD and gemm(q8, q4) == BAD and gemm(q4, q8) == BAD
    assert gemm(q8, _q(grid=0, **MX)) == MISMATCH                      # no element plane
    assert gemm(q8, _q(elems8=5 * P, grid=0, scale_fmt=2, block=32, hadamard_n=16)) == MISMATCH
    assert gemm(q8, _q(grid=1, **MX)) == MISMATCH
    assert gemm(_q(**E8), q8) == BAD                                   # no elements
    assert gemm(_q(elems8=4 * P + 8, **E8), q8) == ALIGN
    x = ctypes.c_void_p(P)
    assert L.ufp4_rht_quantize(x, 128, 256, 256, 0, None, q8, None) == UNSUP
    assert L.ufp4_quant_stats(x, 128, 256, 256, 0, q8, P, None) == UNSUP


def test_gemm_epilogue(L):
    a, b = _q(rows=128), _q(rows=64)

    def call(out=P, ldo=64, dt=0, a=a, b=b, **kw):
        return L.ufp4_gemm_epilogue(a, b, ufp4.EpilogueC(**kw), out, ldo, dt, None)

    assert call(out=None) == BAD and call(ldo=63) == BAD and call(dt=2) == BAD and call(dt=-1) == BAD
    assert call(out=P + 1) == ALIGN and call(out=P + 2, dt=1) == ALIGN
    assert call(act=5) == BAD and call(act=-1) == BAD
    assert call(bias=P, bias_dtype=3) == BAD and call(bias=P + 1) == ALIGN and call(bias=P + 2, bias_dtype=1) == ALIGN
    assert call(residual=P, ld_residual=63) == BAD and call(residual=P, ld_residual=0) == BAD
    assert call(residual=P, ld_residual=64, residual_dtype=2) == BAD
    assert call(residual=P + 1, ld_residual=64) == ALIGN
    assert call(pre=P, ld_pre=63) == BAD and call(pre=P, ld_pre=64, pre_dtype=9) == BAD
    assert call(pre=P + 2, ld_pre=64, pre_dtype=1) == ALIGN
    assert call(residual=P, ld_residual=65) == BAD and call(residual=P, ld_residual=64, residual_dtype=1) == BAD
    assert call(pre=P, ld_pre=64) == BAD and call(pre=2 * P, ld_pre=64, residual=2 * P, ld_residual=64) == BAD
    assert call(b=_q(rows=64, k=192)) == MISMATCH
    assert L.ufp4_gemm_epilogue(None, b, None, P, 64, 0, None) == BAD
    assert L.ufp4_gemm_epilogue(a, None, None, P, 64, 0, None) == BAD
    assert L.ufp4_gemm_epilogue(_q(rows=0), b, None, None, 64, 0, None) == OK      # nothing to write


def test_epilogue_backward(L):
    def call(dout=P, ldg=64, gd=0, pre=P, ldz=64, zd=0, act=2, m=128, n=64, dpre=2 * P, ldd=64, dd=0, dbias=3 * P,
             work=4 * P):
        return L.ufp4_epilogue_backward(dout, ldg, gd, pre, ldz, zd, act, m, n, dpre, ldd, dd, dbias, work, None)

    assert call(dout=None) == BAD and call(ldg=63) == BAD and call(gd=2) == BAD and call(dout=P + 1) == ALIGN
    assert call(pre=None) == BAD and call(ldz=1) == BAD and call(zd=-1) == BAD and call(pre=P + 2, zd=1) == ALIGN
    assert call(act=7) == BAD and call(m=-1) == BAD and call(n=-1) == BAD and call(m=1 << 32) == UNSUP
    assert call(ldd=63) == BAD and call(dd=2) == BAD and call(dpre=2 * P + 1) == ALIGN
    assert call(dpre=None, dbias=None) == BAD and call(dbias=3 * P + 2) == ALIGN
    assert call(work=None) == BAD and call(work=4 * P + 8) == ALIGN
    assert call(dpre=P, ldd=65) == BAD and call(dpre=P, gd=1) == BAD and call(dout=5 * P, dpre=P, zd=1) == BAD
    assert call(n=0) == OK
    W = L.ufp4_epilogue_backward_workspace
    assert W(0, 64) == 0 and W(64, 0) == 0 and W(1, 64) == 64 * 4
    assert W(16384, 28672) % (28672 * 4) == 0


def test_binding_refusals():
    """Wrong shapes, types and host tensors raise before the library is called."""
    cfg = ufp4.QuantConfig(**E8)
    t = torch.zeros(4, 8)
    with pytest.raises(RuntimeError, match="CUDA"):
        ufp4.epilogue_backward(t, t, ufp4.ACT_RELU)
    with pytest.raises(RuntimeError, match="CUDA"):
        ufp4.gemm_epilogue(ufp4.empty_qtensor(4, 64, cfg, device="cpu"), ufp4.empty_qtensor(8, 64, cfg, device="cpu"))
    q = ufp4.empty_qtensor(4, 64, cfg, device="cpu")
    assert q.codes is None and q.elems8.shape == (4, 64) and q.sf_atoms.shape == (1, 1, 512) and q.c().codes is None
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        ufp4._dtype(t.half(), "x")
    for bad in (t[:3], t.t(), torch.zeros(4, 16)[:, ::2], torch.zeros(8)):
        with pytest.raises(ValueError):
            ufp4._pitch(bad, 4, 8, "x")
    assert ufp4._pitch(torch.zeros(4, 10)[:, :8], 4, 8, "x") == 10
    with pytest.raises(ValueError):
        ufp4._vector(torch.zeros(16)[::2], 8, "x")


def test_rmsnorm(L):
    q = _q(rows=128, k=64, elems8=4 * P, **E8)

    def call(x=P, ldx=64, xd=0, res=2 * P, ldr=64, sd=0, w=3 * P, wd=0, eps=1e-6, rows=128, cols=64, h=5 * P, ldh=64,
             y=6 * P, ldy=64, q=None, rstd=7 * P):
        return L.ufp4_rmsnorm(x, ldx, xd, res, ldr, sd, w, wd, eps, rows, cols, h, ldh, y, ldy, q, rstd, None)

    assert call(x=None) == BAD and call(ldx=63) == BAD and call(xd=2) == BAD and call(x=P + 1) == ALIGN
    assert call(ldr=63) == BAD and call(sd=5) == BAD and call(res=2 * P + 2, sd=1) == ALIGN
    assert call(w=None) == BAD and call(wd=-1) == BAD and call(w=3 * P + 2, wd=1) == ALIGN
    assert call(eps=-1.0) == BAD and call(eps=float("nan")) == BAD
    assert call(rows=-1) == BAD and call(cols=-1) == BAD
    assert call(cols=32769, ldx=32769, ldr=32769, ldh=32769, ldy=32769) == UNSUP
    assert call(h=None) == BAD and call(ldh=1) == BAD
    assert call(res=None) == BAD                          # h without a residual
    assert call(res=None, h=None, sd=1) == BAD            # a stream type of its own
    assert call(y=None) == BAD and call(q=q) == BAD       # none, both
    assert call(ldy=63) == BAD and call(y=6 * P + 1) == ALIGN and call(rstd=7 * P + 2) == ALIGN
    assert call(y=None, q=_q(rows=127, k=64, elems8=4 * P, **E8)) == BAD
    assert call(y=None, q=_q(rows=128, k=128, elems8=4 * P, **E8)) == BAD
    assert call(y=None, q=_q(rows=128, k=64, **E8)) == BAD                     # no elements
    assert call(y=None, q=_q(rows=128, k=64, elems8=4 * P + 4, **E8)) == ALIGN
    assert call(y=None, q=_q(rows=128, k=64, elems8=4 * P, grid=0, **MX)) == UNSUP
    assert call(h=P, ldh=65) == BAD and call(h=P, xd=1) == BAD and call(h=2 * P, ldh=65) == BAD
    assert call(y=P) == BAD and call(y=5 * P) == BAD and call(y=2 * P) == BAD
    assert call(rows=0) == OK


def test_rmsnorm_backward(L):
    def call(dy=P, ldg=64, gd=0, h=2 * P, ldh=64, sd=0, w=3 * P, wd=0, rstd=4 * P, dh=5 * P, lddh=64, rows=128,
             cols=64, dx=6 * P, lddx=64, dd=0, dw=7 * P, work=8 * P):
        return L.ufp4_rmsnorm_backward(dy, ldg, gd, h, ldh, sd, w, wd, rstd, dh, lddh, rows, cols, dx, lddx, dd, dw,
                                       work, None)

    assert call(dy=None) == BAD and call(ldg=63) == BAD and call(gd=2) == BAD and call(dy=P + 1) == ALIGN
    assert call(h=None) == BAD and call(ldh=63) == BAD and call(sd=2) == BAD and call(h=2 * P + 2, sd=1) == ALIGN
    assert call(w=None) == BAD and call(wd=2) == BAD and call(rstd=None) == BAD and call(rstd=4 * P + 1) == ALIGN
    assert call(lddh=63) == BAD and call(dh=5 * P + 1) == ALIGN
    assert call(dx=None) == BAD and call(lddx=63) == BAD and call(dd=2) == BAD
    assert call(dw=7 * P + 2) == ALIGN and call(work=None) == BAD and call(work=8 * P + 4) == ALIGN
    assert call(rows=-1) == BAD and call(cols=40000, ldg=40000, ldh=40000, lddh=40000, lddx=40000) == UNSUP
    assert call(dx=P, lddx=65) == BAD and call(dx=P, gd=1) == BAD and call(dx=5 * P, dd=1) == BAD and call(dx=2 * P) == BAD
    assert call(cols=0) == OK and call(rows=0, dw=None) == OK
    W = L.ufp4_rmsnorm_backward_workspace
    assert W(0, 64) == 0 and W(5, 0) == 0 and W(1, 2048) == 2048 * 4 and W(1, 64) == 64 * 4


def test_moe_balance(L):
    def fwd(x=P, ld=64, dt=0, t=100, e=64, c=2 * P, k=2, mask=None, coef=1.0, loss=3 * P, counts=4 * P, valid=5 * P,
            work=6 * P):
        return L.ufp4_moe_balance(x, ld, dt, t, e, c, k, mask, coef, loss, counts, valid, work, None)

    assert fwd(x=None) == BAD and fwd(ld=63) == BAD and fwd(dt=2) == BAD and fwd(x=P + 1) == ALIGN
    assert fwd(t=-1) == BAD and fwd(e=0) == BAD and fwd(k=0) == BAD and fwd(coef=float("nan")) == BAD
    assert fwd(e=1025, ld=1025) == UNSUP and fwd(k=1025) == UNSUP and fwd(t=1 << 31) == UNSUP and fwd(t=1 << 30, k=128) == UNSUP
    assert fwd(c=None) == BAD and fwd(loss=None) == BAD and fwd(counts=None) == BAD and fwd(valid=None) == BAD
    assert fwd(work=None) == BAD and fwd(work=6 * P + 8) == ALIGN
    assert fwd(c=2 * P + 2) == ALIGN and fwd(loss=3 * P + 2) == ALIGN and fwd(counts=4 * P + 4) == ALIGN
    assert fwd(valid=5 * P + 4) == ALIGN

    def bwd(x=P, ld=64, dt=0, t=100, e=64, k=2, mask=None, coef=1.0, counts=4 * P, valid=5 * P, dl=6 * P, d=7 * P,
            ldd=64):
        return L.ufp4_moe_balance_backward(x, ld, dt, t, e, k, mask, coef, counts, valid, dl, d, ldd, None)

    assert bwd(x=None) == BAD and bwd(ld=63) == BAD and bwd(dt=3) == BAD and bwd(e=0) == BAD and bwd(k=0) == BAD
    assert bwd(e=2000, ld=2000, ldd=2000) == UNSUP
    assert bwd(counts=None) == BAD and bwd(valid=None) == BAD and bwd(dl=None) == BAD and bwd(d=None) == BAD
    assert bwd(ldd=63) == BAD and bwd(d=7 * P + 1) == ALIGN and bwd(counts=4 * P + 4) == ALIGN
    assert bwd(dl=6 * P + 2) == ALIGN and bwd(d=P, ldd=65) == BAD and bwd(t=0) == OK
    W = L.ufp4_moe_balance_workspace
    assert W(0) == 0 and W(1025) == 0 and W(64) > 0


def test_grad_clip(L):
    def table(*rows):
        return (ufp4.TensorC * len(rows))(*[ufp4.TensorC(*r) for r in rows])

    def clip(t, n=None, max_norm=1.0, norm=P, work=2 * P):
        return L.ufp4_grad_clip(t, len(t) if n is None else n, max_norm, norm, work, None)

    good = (4 * P, 4 * P, 100, 1, 1)
    assert clip(table(good), n=-1) == BAD and L.ufp4_grad_clip(None, 1, 1.0, P, 2 * P, None) == BAD
    assert clip(table(good), max_norm=-1.0) == BAD and clip(table(good), max_norm=float("nan")) == BAD
    assert clip(table(good), norm=None) == BAD and clip(table(good), work=None) == BAD
    assert clip(table(good), norm=P + 2) == ALIGN and clip(table(good), work=2 * P + 8) == ALIGN
    assert clip(table(good, (None, 8 * P, 10, 1, 1))) == BAD and clip(table((4 * P, None, 10, 1, 1))) == BAD
    assert clip(table((4 * P, 4 * P, -1, 1, 1))) == BAD and clip(table((4 * P, 8 * P, 10, 2, 1))) == BAD
    assert clip(table((4 * P, 8 * P, 10, 1, 7))) == BAD and clip(table((4 * P, 4 * P, 10, 1, 0))) == BAD
    assert clip(table((4 * P + 2, 8 * P, 10, 1, 1))) == ALIGN and clip(table((4 * P, 8 * P + 1, 10, 1, 0))) == ALIGN
    assert clip(table(good, good)) == BAD                                           # listed twice
    assert clip(table(good, (9 * P, 4 * P + 396, 5, 0, 1))) == BAD                  # overlap by one element
    assert L.ufp4_grad_norm(table((4 * P, None, 10, 5, 0)), 1, P, 2 * P, None) == BAD
    assert L.ufp4_grad_norm(table((4 * P + 1, None, 10, 0, 0)), 1, P, 2 * P, None) == ALIGN
    W = L.ufp4_grad_norm_workspace
    assert W(0) == W(1) == W(512) and W(513) == 2 * W(1) and W(1) % 8 == 0


def test_grad_clip_overlapping_sources(L):
    """A destination may be its own source, and overlaps no other tensor."""
    def clip(*rows):
        return L.ufp4_grad_clip((ufp4.TensorC * len(rows))(*[ufp4.TensorC(*r) for r in rows]), len(rows), 1.0, P, 2 * P, None)

    a, b, c = 4 * P, 5 * P, 6 * P
    for bad in ([(a, b, 100, 1, 1), (b, a, 100, 1, 1)],                      # exchanged
                [(a, c, 100, 1, 1), (b, a, 100, 1, 1)],                      # another's source
                [(b, a, 100, 1, 1), (a, a + 400, 100, 1, 1)],                # the same, in the other order
                [(a, a, 100, 1, 1), (a, c, 100, 1, 1)],                      # read by one, in place in the other
                [(a, a + 4, 100, 1, 1)], [(a + 4, a, 100, 1, 1)],            # its own source, shifted
                [(a, a + 196, 100, 0, 1)], [(a + 396, a, 100, 1, 1)],
                [(a, c, 100, 1, 1), (b, a + 396, 100, 1, 1)],                # by one element
                [(a, c, 100, 1, 1), (b, a - 200, 101, 1, 0)],                # by half of one
                [(a, c, 10, 1, 1)] * 1 + [(b, c + 4096 + 64 * i, 4, 1, 1) for i in range(600)] + [(b + 4096, a, 1, 1, 0)]):
        for rows in (bad, bad[::-1]):
            assert clip(*rows) == BAD, bad[:3]


def test_grad_clip_without_host_memory(L):
    """A list too long for the memory that its check needs is refused; no
    exception leaves the C entry."""
    script = f"""
import ctypes, resource, sys
import torch                     # (what the library's own loading needs, before the limit)
from fp4_quantized_gemms_b200 import ufp4
L = ufp4.lib()
n = 4_000_000
table = (ufp4.TensorC * n)()
ctypes.memset(table, 0, ctypes.sizeof(table))
for i in range(2):
    table[i] = ufp4.TensorC({P}, {P}, 1, 1, 1)       # twice the same: refused in any case
args = (table, n, 1.0, {P}, {2 * P}, None)
size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (size + (8 << 20),) * 2)
sys.exit(100 + L.ufp4_grad_clip(*args))
"""
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 100 + UNSUP, (r.returncode, r.stderr[-500:])
