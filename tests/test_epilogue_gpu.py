"""The GEMM epilogue (bias, activation, residual) and its backward pass against
64-bit formulas, over every operand format and its kernel family."""
import pytest
import torch

from fp4_quantized_gemms_b200 import ufp4
from tests.gpu_util import GEMM_RTOL, needs_gpu
from tests.op_util import ACTS, BF16, FP32, act64, eight_bit, half_step, product64, rand, slope64, strided

pytestmark = needs_gpu

TWO, MX = ufp4.SCALE_E4M3_X_FP32, ufp4.SCALE_UE8M0
# format name -> (config, options of the quantizer call)
FORMATS = {
    "e1m2_fp32": (dict(grid=0, block=16, scale_fmt=ufp4.SCALE_FP32), {}),
    "e2m1_fp32_b32": (dict(grid=1, block=32, scale_fmt=ufp4.SCALE_FP32), {}),
    "e1m2_lanes": (dict(grid=0, block=16, scale_fmt=TWO), {}),
    "e1m2_atoms": (dict(grid=0, block=16, scale_fmt=TWO), dict(with_lanes=False)),
    "e1m2_noatoms": (dict(grid=0, block=16, scale_fmt=TWO), dict(with_atoms=False)),
    "e1m2_nocorr": (dict(grid=0, block=16, scale_fmt=TWO), dict(with_corr=False)),
    "e2m1_two": (dict(grid=1, block=16, scale_fmt=TWO), {}),
    "e2m1_noatoms_b32": (dict(grid=1, block=32, scale_fmt=TWO), dict(with_atoms=False)),
    "mx": (dict(grid=0, block=32, scale_fmt=MX), {}),
    "mx_noatoms": (dict(grid=0, block=32, scale_fmt=MX), dict(with_atoms=False)),
    "mx_codes": (dict(grid=0, block=32, scale_fmt=MX), dict(with_elems8=False)),
    "mx_e2m1": (dict(grid=1, block=32, scale_fmt=MX), {}),
}


def _operands(fmt, m, n, k, seed=1):
    x, w = rand(seed, m, k), rand(seed + 1, n, k, std=0.05)
    if fmt in ("w4a8", "w4a8_noatoms", "w8a8"):
        atoms = fmt != "w4a8_noatoms"
        a = eight_bit(x.float() * 3, atoms)
        if fmt == "w8a8":
            return a, eight_bit(w.float())
        cfg = ufp4.QuantConfig(grid=0, block=32, scale_fmt=MX, hadamard_n=0)
        return a, ufp4.rht_quantize(w, ufp4.ALONG_COLS, cfg, with_atoms=atoms)
    kw, opt = FORMATS[fmt]
    cfg = ufp4.QuantConfig(**kw)
    return ufp4.rht_quantize(x, ufp4.ALONG_COLS, cfg, **opt), ufp4.rht_quantize(w, ufp4.ALONG_COLS, cfg, **opt)


def _check(got, want, z, dtype):
    """One rounding of the result (half a step of its value) on top of the
    product's bound (GEMM_RTOL of the product's norm, here also per element
    against its largest value) and of the activation's fp32 arithmetic
    (act_value: a few 1e-7 of max(|z|, 1)); slopes are at most 1.13."""
    slack = 1.2 * GEMM_RTOL * float(z.abs().max()) + 2e-6 * max(1.0, float(z.abs().max()))
    err = (got.double() - want).abs()
    lim = half_step(dtype) * want.abs() * 1.001 + slack
    assert torch.isfinite(got).all()
    assert bool((err <= lim).all()), float((err - lim).max())


def _ok():
    torch.cuda.synchronize()
    assert ufp4.check_device_status() == ufp4.OK


@pytest.mark.parametrize("fmt", [*FORMATS, "w4a8", "w4a8_noatoms", "w8a8"])
@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (257, 130, 200), (300, 520, 448)])
def test_formats(fmt, m, n, k):
    """Every operand format (so every kernel family), ragged shapes, the whole epilogue."""
    k8 = (k + 7) // 8 * 8
    a, b = _operands(fmt, m, n, k8)
    bias, res = rand(5, n, std=0.3), rand(6, m, n)
    pre = torch.full((m, n), float("nan"), dtype=BF16, device="cuda")
    y = ufp4.gemm_epilogue(a, b, bias=bias, act=ufp4.ACT_GELU, residual=res, pre=pre)
    _ok()
    z = product64(a, b) + bias.double()
    _check(pre, z, z, BF16)
    _check(y, act64(z, "gelu") + res.double(), z, BF16)


@pytest.mark.parametrize("path", [ufp4.GEMM_PATH_NATIVE_FP4])
@pytest.mark.parametrize("fmt", ["e1m2_lanes", "e2m1_two"])
def test_one_cta_path(fmt, path):
    a, b = _operands(fmt, 200, 450, 320)
    bias = rand(5, 450, dtype=FP32)
    ufp4.set_two_level_gemm_path(path)
    try:
        y = ufp4.gemm_epilogue(a, b, bias=bias, act=ufp4.ACT_SILU, out_dtype=FP32)
    finally:
        ufp4.set_two_level_gemm_path(ufp4.GEMM_PATH_AUTO)
    _ok()
    z = product64(a, b) + bias.double()
    _check(y, act64(z, "silu"), z, FP32)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out,bias_t,res_t,pre_t", [(BF16, BF16, BF16, BF16), (FP32, FP32, FP32, FP32),
                                                    (BF16, None, FP32, None), (FP32, BF16, None, None),
                                                    (BF16, None, None, None)])
def test_parts_and_types(act, out, bias_t, res_t, pre_t):
    m, n, k = 130, 264, 192
    a, b = _operands("e2m1_two", m, n, k)
    bias = rand(5, n, dtype=bias_t) if bias_t else None
    res = rand(6, m, n, dtype=res_t) if res_t else None
    pre = torch.empty(m, n, dtype=pre_t, device="cuda") if pre_t else None
    y = ufp4.gemm_epilogue(a, b, bias=bias, act=ACTS[act], residual=res, pre=pre, out_dtype=out)
    _ok()
    z = product64(a, b) + (bias.double() if bias_t else 0)
    if pre_t:
        _check(pre, z, z, pre_t)
    _check(y, act64(z, act) + (res.double() if res_t else 0), z, out)


@pytest.mark.parametrize("fmt", ["e2m1_two", "mx", "e1m2_fp32", "e1m2_nocorr"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (4, 0), (8, 4), (5, 0), (13, 8)])
def test_pitch_and_alignment(fmt, pad, offset):
    """Row pitches and start addresses that forbid vector accesses, odd N; the
    padding between rows stays as it was."""
    m, n, k = 140, 131, 128
    a, b = _operands(fmt, m, n, k)
    res = strided(rand(6, m, n), pad, offset)
    bias = rand(5, n + 1)[1:]
    buf = torch.full((m * (n + pad) + offset,), 7.0, dtype=BF16, device="cuda")
    out = buf[offset:].view(m, n + pad)[:, :n]
    ufp4.gemm_epilogue(a, b, bias=bias, residual=res, out=out)
    _ok()
    z = product64(a, b) + bias.double()
    _check(out, z + res.double(), z, BF16)
    assert bool((buf[offset:].view(m, n + pad)[:, n:] == 7.0).all()) and bool((buf[:offset] == 7.0).all())


def test_residual_in_place_and_large_values():
    m, n, k = 300, 200, 256
    a, b = _operands("mx", m, n, k)
    res = rand(6, m, n)
    res[3, 5], res[4, 6], res[7, 8] = float("inf"), float("-inf"), float("nan")
    want = product64(a, b) + res.double()
    ufp4.gemm_epilogue(a, b, residual=res, out=res)
    _ok()
    assert res[3, 5] == float("inf") and res[4, 6] == float("-inf") and bool(res[7, 8].isnan())
    ok = want.isfinite()
    assert bool((res.isfinite() == ok).all())
    _check(torch.where(ok, res, 0.0), torch.where(ok, want, 0.0), product64(a, b), BF16)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("act", ACTS)
def test_not_finite_bias(bad, act):
    """A bias that is not finite reaches its column as the formula says, and no other."""
    a, b = _operands("e2m1_two", 40, 72, 64)
    bias = torch.zeros(72, dtype=FP32, device="cuda")
    bias[9] = bad
    y = ufp4.gemm_epilogue(a, b, bias=bias, act=ACTS[act], out_dtype=FP32)
    _ok()
    want = act64(torch.full((1,), bad, dtype=torch.float64), act)
    col = y[:, 9].double().cpu()
    assert bool((col.isnan() if want.isnan() else col == want).all())
    y[:, 9] = 0
    assert bool(y.isfinite().all())


def test_no_reduction_and_empty():
    cfg = ufp4.QuantConfig(grid=1, scale_fmt=TWO)
    a, b = ufp4.empty_qtensor(70, 0, cfg), ufp4.empty_qtensor(33, 0, cfg)
    bias, res = rand(5, 33), rand(6, 70, 33, dtype=FP32)
    y = ufp4.gemm_epilogue(a, b, bias=bias, act=ufp4.ACT_SILU, residual=res, out_dtype=FP32)
    _ok()
    z = bias.double().expand(70, 33)
    _check(y, act64(z, "silu") + res.double(), z, FP32)
    a, b = _operands("mx", 64, 64, 64)
    none = ufp4.empty_qtensor(0, 64, a.cfg)
    assert ufp4.gemm_epilogue(none, b, bias=rand(1, 64)).shape == (0, 64)
    assert ufp4.gemm_epilogue(a, none).shape == (64, 0)


def test_agrees_with_the_plain_product():
    """Without an epilogue the fp32 output is the plain GEMM's, bit for bit."""
    for fmt in ("e1m2_lanes", "e2m1_two", "mx", "e1m2_fp32"):
        a, b = _operands(fmt, 512, 264, 320)
        assert torch.equal(ufp4.gemm_epilogue(a, b, out_dtype=FP32), ufp4.gemm_fprop(a, b))
    _ok()


def test_eight_bit_operands_in_the_plain_gemms():
    a, b = _operands("w4a8", 300, 200, 512)
    y = ufp4.gemm_fprop(a, b)
    _ok()
    want = product64(a, b)
    assert float((y.double() - want).norm() / want.norm()) <= GEMM_RTOL


def test_streams_and_graph():
    """On another stream, and captured once and replayed on new inputs."""
    m, n, k = 256, 512, 512
    a, b = _operands("mx", m, n, k)
    bias, res = rand(5, n), rand(6, m, n)
    first = ufp4.gemm_epilogue(a, b, bias=bias, act=ufp4.ACT_GELU, residual=res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = ufp4.gemm_epilogue(a, b, bias=bias, act=ufp4.ACT_GELU, residual=res)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first, other)
    out, pre = torch.empty_like(first), torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ufp4.gemm_epilogue(a, b, bias=bias, act=ufp4.ACT_GELU, residual=res, out=out, pre=pre)
        dpre, dbias = ufp4.epilogue_backward(out, pre, ufp4.ACT_GELU)
    res.copy_(rand(7, m, n))
    g.replay()
    eager = ufp4.gemm_epilogue(a, b, bias=bias, act=ufp4.ACT_GELU, residual=res)
    d2, b2 = ufp4.epilogue_backward(eager, pre, ufp4.ACT_GELU)
    assert torch.equal(out, eager) and torch.equal(dpre, d2) and torch.equal(dbias, b2)
    _ok()


# ---------------------------------------------------------------- backward
def _check_bwd(dpre, dbias, dout, pre, act, terms=1.0):
    """dpre: one rounding, plus the slope's fp32 arithmetic (2e-6: products of
    ex2 and reciprocal results within a few 2^-22 of values up to 1.13).
    dbias: m terms, each with that slope error and 2^-24 per addition along a
    path of at most 600 additions, against the sum of the terms' sizes."""
    d = dout.double() * (slope64(pre.double(), act) if pre is not None else 1.0)
    size = dout.double().abs()
    lim = half_step(dpre.dtype) * d.abs() * 1.001 + 2e-6 * size
    assert bool(((dpre.double() - d).abs() <= lim).all())
    if dbias is not None:
        lim = (2e-6 + 600 * 2.0 ** -24) * size.sum(0) * 1.2
        assert bool(((dbias.double() - d.sum(0)).abs() <= lim).all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gt,zt,dt", [(BF16, BF16, BF16), (FP32, BF16, BF16), (FP32, FP32, FP32), (BF16, FP32, FP32)])
@pytest.mark.parametrize("m,n", [(1, 8), (77, 264), (1030, 1408), (40, 131), (1100, 1021)])
def test_backward(act, gt, zt, dt, m, n):
    dout, pre = rand(1, m, n, std=0.01, dtype=gt), rand(2, m, n, std=3.0, dtype=zt)
    dpre, dbias = ufp4.epilogue_backward(dout, pre, ACTS[act], dpre=torch.empty(m, n, dtype=dt, device="cuda"))
    _ok()
    _check_bwd(dpre, dbias, dout, pre, act)


@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 0), (8, 3), (5, 2)])
def test_backward_pitch(pad, offset):
    m, n = 100, 264
    dout, pre = strided(rand(1, m, n), pad, offset), strided(rand(2, m, n), pad + 8, offset)
    buf = torch.full((m * (n + pad) + offset,), 7.0, dtype=BF16, device="cuda")
    dpre, dbias = ufp4.epilogue_backward(dout, pre, ufp4.ACT_SILU, dpre=buf[offset:].view(m, n + pad)[:, :n])
    _ok()
    _check_bwd(dpre, dbias, dout, pre, "silu")
    assert bool((buf[offset:].view(m, n + pad)[:, n:] == 7.0).all()) and bool((buf[:offset] == 7.0).all())


def test_backward_in_place_without_activation_and_empty():
    m, n = 200, 136
    dout, pre = rand(1, m, n), rand(2, m, n)
    want, wb = ufp4.epilogue_backward(dout, pre, ufp4.ACT_GELU)
    g = dout.clone()
    got, gb = ufp4.epilogue_backward(g, pre, ufp4.ACT_GELU, dpre=g)
    assert got is g and torch.equal(got, want) and torch.equal(gb, wb)
    d, b = ufp4.epilogue_backward(dout, None, ufp4.ACT_NONE)
    assert torch.equal(d, dout)
    _check_bwd(d, b, dout, None, "none")
    d, b = ufp4.epilogue_backward(dout, pre, ufp4.ACT_RELU, want_dbias=False)
    assert b is None
    _check_bwd(d, None, dout, pre, "relu")
    d, b = ufp4.epilogue_backward(dout[:0], pre[:0], ufp4.ACT_RELU)
    assert d.shape == (0, n) and bool((b == 0).all())
    _ok()


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
def test_backward_extreme_values(act):
    """Far pre-activations give slopes of 0 and 1, NaN stays NaN (but relu's, which compares)."""
    z = torch.tensor([[-1e30, -1e4, -60.0, -12.5, -0.0, 0.0, 12.5, 60.0, 1e4, 1e30, float("nan"), 1.0]], device="cuda")
    d, _ = ufp4.epilogue_backward(torch.ones_like(z), z, ACTS[act], dpre=torch.empty_like(z))
    _ok()
    at0 = 0.0 if act == "relu" else 0.5
    want = torch.tensor([0, 0, 0, 0, at0, at0, 1, 1, 1, 1], dtype=torch.float64)
    got = d[0, :10].double().cpu()
    # silu at +-12.5 is 4.4e-5 from its limit; the rest are within fp32 arithmetic
    assert bool(((got - want).abs() <= (5e-5 if act == "silu" else 2e-6)).all()), got
    assert act == "relu" or bool(d[0, 10].isnan())


def test_backward_against_differences():
    """The gradient of sum(w * out) with respect to the bias and to single
    pre-activations, by central differences of the forward's 64-bit formula."""
    m, n, h = 50, 72, 1e-4
    a, b = _operands("mx", m, n, 64)
    bias, w = rand(5, n, dtype=FP32), rand(6, m, n, dtype=FP32)
    for act in ACTS:
        pre = torch.empty(m, n, dtype=FP32, device="cuda")
        ufp4.gemm_epilogue(a, b, bias=bias, act=ACTS[act], pre=pre)
        dpre, dbias = ufp4.epilogue_backward(w, pre, ACTS[act], dpre=torch.empty(m, n, dtype=FP32, device="cuda"))
        _ok()
        z = pre.double()
        num = w.double() * (act64(z + h, act) - act64(z - h, act)) / (2 * h)
        away = z.abs() > h if act == "relu" else torch.ones_like(z, dtype=torch.bool)
        # third derivatives are below 3: h^2 / 6 * 3 per unit of w, plus the slope's own 2e-6
        lim = w.double().abs() * (0.5 * h * h + 2e-6) + half_step(FP32) * num.abs()
        assert bool(((dpre.double() - num).abs() <= lim)[away].all())
        if bool(away.all()):
            assert bool(((dbias.double() - num.sum(0)).abs() <= (lim.sum(0) + 1e-5 * w.double().abs().sum(0))).all())


def test_backward_same_bits_every_time():
    dout, pre = rand(1, 5000, 520), rand(2, 5000, 520)
    first = ufp4.epilogue_backward(dout, pre, ufp4.ACT_GELU)
    for _ in range(3):
        again = ufp4.epilogue_backward(dout, pre, ufp4.ACT_GELU)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
