"""The RMS norm of the residual stream, bf16 and 8-bit outputs, forward and
backward, against 64-bit formulas."""
import pytest
import torch

from fp4_quantized_gemms_b200 import ufp4
from tests.gpu_util import GEMM_RTOL, needs_gpu
from tests.op_util import BF16, FP32, half_step, product64, rand, strided, values64

pytestmark = needs_gpu

EPS = 1e-5
# y in fp32: a row's sum of squares takes at most 32 terms per thread and 10
# steps of a tree, 2^-24 each, halved by the square root; then mean, eps, root,
# reciprocal and two products: below 32 roundings in all.
ARITH = 32 * 2.0 ** -24


def _ok():
    torch.cuda.synchronize()
    assert ufp4.check_device_status() == ufp4.OK


def _around(v):
    """What the allocation of a strided matrix holds beside its rows."""
    whole = torch.empty(0, dtype=v.dtype, device=v.device).set_(v.untyped_storage())
    mine = torch.zeros(whole.numel(), dtype=torch.bool, device=v.device)
    r, c = v.shape
    mine[(v.storage_offset() + torch.arange(r, device=v.device)[:, None] * v.stride(0) +
          torch.arange(c, device=v.device)).reshape(-1)] = True
    return whole[~mine]


def _expect(x, res, w, eps=EPS):
    h = x.double() if res is None else (x.double() + res.double()).to(res.dtype).double()
    r = 1 / torch.sqrt((h * h).mean(1) + eps)
    return h, r, h * r[:, None] * w.double()


def _check_q(q, y):
    """The 8-bit operand: block exponents by their rule (where fp32 arithmetic
    cannot move amax across a power of two), elements within half an E4M3 step
    (2^-4 of the value, or half the step of the smallest exponents), zero
    padding, and the same factors in the atoms."""
    rows, cols = y.shape
    full = torch.zeros(rows, q.kpad, dtype=torch.float64, device=y.device)
    full[:, :cols] = y
    amax = full.view(rows, -1, 32).abs().amax(2)
    byte = q.scales[:, :rows].t()
    lo, hi = amax * (1 - ARITH), amax * (1 + ARITH)

    def rule(a):
        m, e = torch.frexp(a)
        x = torch.where(a > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -127)).clamp(-127, 127)
        return (x + 127).to(torch.uint8)

    assert bool(((byte == rule(lo)) | (byte == rule(hi))).all())
    step = torch.exp2(byte.double() - 127).repeat_interleave(32, dim=1)
    err = (values64(q) - full).abs()
    lim = torch.maximum(half_step(torch.float8_e4m3fn) * full.abs(), 2.0 ** -10 * step) * (1 + 1e-9) + ARITH * full.abs()
    assert bool((err <= lim).all()), float((err - lim).max())
    assert bool((q.elems8[:, cols:] == 0).all())
    if q.sf_atoms is not None:
        r = torch.arange(rows, device=y.device)[:, None]
        s = torch.arange(q.kpad // 32, device=y.device)[None, :]
        assert torch.equal(q.sf_atoms[r // 128, s // 4, 16 * (r % 32) + 4 * ((r // 32) % 4) + s % 4], byte)


COLS = [1, 7, 31, 64, 100, 256, 257, 520, 1000, 1024, 1032, 1408, 2048, 4096, 4100, 8192, 8200, 12000, 16384, 20001,
        32768]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 5, 133, 700])
@pytest.mark.parametrize("eight", [False, True])
def test_widths(rows, cols, eight):
    x, res, w = rand(1, rows, cols), rand(2, rows, cols, std=2.0), rand(3, cols)
    q = ufp4.empty_qtensor(rows, cols, ufp4.CFG_8BIT) if eight else None
    y, _, h, rstd = ufp4.rmsnorm(x, w, residual=res, eps=EPS, q=q)
    _ok()
    h64, r64, y64 = _expect(x, res, w)
    assert torch.equal(h.double(), h64)
    assert bool(((rstd.double() - r64).abs() <= ARITH * r64).all())
    if eight:
        assert y is None
        _check_q(q, y64)
    else:
        assert bool(((y.double() - y64).abs() <= (half_step(BF16) * 1.001 + ARITH) * y64.abs()).all())


@pytest.mark.parametrize("xt,st,wt", [(BF16, None, FP32), (FP32, None, BF16), (FP32, FP32, FP32), (BF16, FP32, BF16),
                                      (FP32, BF16, BF16)])
@pytest.mark.parametrize("rows,cols", [(9, 96), (200, 1000), (300, 1027), (40, 2056), (1300, 2055), (12, 8192),
                                       (200, 12345), (6, 30000)])
@pytest.mark.parametrize("eight", [False, True])
def test_types(xt, st, wt, rows, cols, eight):
    x, w = rand(1, rows, cols, dtype=xt), rand(3, cols, dtype=wt)
    res = rand(2, rows, cols, std=2.0, dtype=st) if st else None
    q = ufp4.empty_qtensor(rows, cols, ufp4.CFG_8BIT, with_atoms=False) if eight else None
    y, _, h, rstd = ufp4.rmsnorm(x, w, residual=res, eps=EPS, q=q)
    _ok()
    if st is None:
        assert h is x
        h64, r64, y64 = _expect(x, None, w)
    else:
        # an fp32 stream takes x + residual with one fp32 rounding
        h64, r64, y64 = _expect(x, res, w)
        assert torch.equal(h.double(), h64)
    assert bool(((rstd.double() - r64).abs() <= ARITH * r64).all())
    if eight:
        _check_q(q, y64)
    else:
        assert bool(((y.double() - y64).abs() <= (half_step(BF16) * 1.001 + ARITH) * y64.abs()).all())


@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 0), (8, 1), (3, 5)])
@pytest.mark.parametrize("rows,cols", [(70, 264), (70, 1410), (400, 1410), (300, 3001)])
def test_pitch_and_alignment(rows, cols, pad, offset):
    x, res, w = rand(1, rows, cols), rand(2, rows, cols), rand(3, cols + 1)[1:]
    y = strided(torch.full((rows, cols), 7.0, dtype=BF16, device="cuda"), pad, offset)
    y0, _, h0, r0 = ufp4.rmsnorm(x, w, residual=res, eps=EPS)
    hv = strided(res, pad, offset)
    around = [(v, _around(v).clone()) for v in (y, hv)]
    _, _, h, r = ufp4.rmsnorm(strided(x, pad, offset), w, residual=hv, h=hv, eps=EPS, y=y)
    _ok()
    assert all(torch.equal(_around(v), keep) for v, keep in around)      # nothing beside the rows was written
    h64, _, y64 = _expect(x, res, w)
    assert h is hv and torch.equal(h, h0) and torch.equal(h.double(), h64)
    assert bool(((y.double() - y64).abs() <= (half_step(BF16) * 1.001 + ARITH) * y64.abs()).all())


def test_in_place_stream():
    """h = residual, or h = x, in place: the same values."""
    x, res, w = rand(1, 300, 2048), rand(2, 300, 2048), rand(3, 2048)
    y, _, h, _ = ufp4.rmsnorm(x, w, residual=res, eps=EPS)
    r2, x2 = res.clone(), x.clone()
    y2, _, h2, _ = ufp4.rmsnorm(x, w, residual=r2, eps=EPS, h=r2)
    y3, _, h3, _ = ufp4.rmsnorm(x2, w, residual=res, eps=EPS, h=x2)
    assert h2 is r2 and h3 is x2
    for a, b in ((y, y2), (y, y3), (h, h2), (h, h3)):
        assert torch.equal(a, b)


def test_rows_beyond_the_last_stay():
    """Scale entries, atom bytes and elements that belong to no row keep their bytes."""
    rows, cols = 70, 200
    q = ufp4.empty_qtensor(rows, cols, ufp4.CFG_8BIT)
    for t in (q.scales, q.sf_atoms):
        t.fill_(0xA5)
    ufp4.rmsnorm(rand(1, rows, cols), rand(3, cols), q=q)
    _ok()
    assert bool((q.scales[:, rows:] == 0xA5).all())
    live = torch.zeros_like(q.sf_atoms, dtype=torch.bool)
    r = torch.arange(rows, device="cuda")[:, None]
    s = torch.arange(q.kpad // 32, device="cuda")[None, :]
    live[r // 128, s // 4, 16 * (r % 32) + 4 * ((r // 32) % 4) + s % 4] = True
    assert bool((q.sf_atoms[~live] == 0xA5).all())


@pytest.mark.parametrize("eight", [False, True])
def test_zero_small_and_large_rows(eight):
    """A zero row gives zeros (scale byte 0); tiny and huge rows keep their shape."""
    cols = 320
    x = rand(1, 4, cols, dtype=FP32)
    x[0] = 0
    x[1] *= 1e-25
    x[2] *= 1e15
    x[3, 32:64] = 0
    w = rand(3, cols, dtype=FP32)
    q = ufp4.empty_qtensor(4, cols, ufp4.CFG_8BIT) if eight else None
    y, _, _, rstd = ufp4.rmsnorm(x, w, eps=0.0 if not eight else EPS, q=q)
    _ok()
    if not eight:           # eps = 0: the zero row has no norm (0 / 0), the tiny row's squares leave fp32
        _, _, y64 = _expect(x[2:], None, w, 0.0)
        assert bool(((y[2:].double() - y64).abs() <= (half_step(BF16) * 1.001 + ARITH) * y64.abs()).all())
        return
    _, _, y64 = _expect(x, None, w)
    _check_q(q, y64)
    assert bool((q.elems8[0] == 0).all()) and bool((q.scales[:, 0] == 0).all())
    assert bool((q.elems8[3, 32:64] == 0).all()) and int(q.scales[1, 3]) == 0


def test_not_finite_rows_stay_apart():
    x, w = rand(1, 8, 512), rand(3, 512)
    clean, _, _, _ = ufp4.rmsnorm(x, w)
    x[2, 7], x[5, 9] = float("nan"), float("inf")
    y, _, _, _ = ufp4.rmsnorm(x, w)
    _ok()
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(y[keep], clean[keep]) and bool(y[2].isnan().all()) and bool(y[5, 9].isnan())


def test_feeds_the_gemm():
    """Norm -> 8-bit operand -> product with 4-bit weights, as a layer runs them."""
    rows, cols, n = 300, 512, 264
    x, res, w = rand(1, rows, cols), rand(2, rows, cols), rand(3, cols)
    q = ufp4.empty_qtensor(rows, cols, ufp4.CFG_8BIT)
    ufp4.rmsnorm(x, w, residual=res, q=q)
    wq = ufp4.rht_quantize(rand(4, n, cols, std=0.05), ufp4.ALONG_COLS,
                           ufp4.QuantConfig(block=32, scale_fmt=ufp4.SCALE_UE8M0, hadamard_n=0))
    out = ufp4.gemm_epilogue(q, wq, out_dtype=FP32)
    _ok()
    want = product64(q, wq)
    assert float((out.double() - want).norm() / want.norm()) <= GEMM_RTOL


# ---------------------------------------------------------------- backward
def _expect_bwd(dy, h, w, rstd, dh):
    h, dy, r = h.double(), dy.double(), rstd.double()[:, None]
    xh, g = h * r, dy * w.double()
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    return dx + (dh.double() if dh is not None else 0), (dy * xh).sum(0)


def _check_bwd(dx, dw, dy, h, w, rstd, dh):
    """dx: one rounding of the result, plus fp32 arithmetic on its terms: the
    dot's sum (at most 45 roundings against the sum of its terms' sizes) and
    eight more roundings of each term.  dw: at most `rows` additions of terms
    with two roundings each, against the sum of their sizes (a pessimistic
    chain: at most 600 in any partial sum here)."""
    dx64, dw64 = _expect_bwd(dy, h, w, rstd, dh)
    r = rstd.double()[:, None]
    xh, g = h.double() * r, dy.double() * w.double()
    size = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    lim = half_step(dx.dtype) * dx64.abs() * 1.001 + 64 * 2.0 ** -24 * size
    if dh is not None:
        lim = lim + 2 * 2.0 ** -24 * dh.double().abs()
    assert bool(((dx.double() - dx64).abs() <= lim).all()), float(((dx.double() - dx64).abs() - lim).max())
    if dw is not None:
        lim = 620 * 2.0 ** -24 * (dy.double() * xh).abs().sum(0)
        assert bool(((dw.double() - dw64).abs() <= lim).all())


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 37, 700])
def test_backward_widths(rows, cols):
    dy, h, w, dh = rand(1, rows, cols), rand(2, rows, cols, std=2.0), rand(3, cols), rand(4, rows, cols)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dx, dw = ufp4.rmsnorm_backward(dy, h, w, rstd, dh=dh)
    _ok()
    _check_bwd(dx, dw, dy, h, w, rstd, dh)


@pytest.mark.parametrize("gt,st,dt,wt", [(FP32, BF16, BF16, FP32), (BF16, FP32, FP32, BF16), (FP32, FP32, BF16, FP32),
                                         (BF16, BF16, FP32, BF16), (BF16, FP32, BF16, BF16), (FP32, FP32, FP32, FP32)])
@pytest.mark.parametrize("rows,cols", [(9, 96), (200, 1000), (300, 509), (40, 2056), (700, 2055), (350, 8192),
                                       (150, 12345), (6, 30000)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward_types(gt, st, dt, wt, rows, cols, with_dh):
    dy, h, w = rand(1, rows, cols, dtype=gt), rand(2, rows, cols, dtype=st), rand(3, cols, dtype=wt)
    dh = rand(4, rows, cols, dtype=st) if with_dh else None
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dx, dw = ufp4.rmsnorm_backward(dy, h, w, rstd, dh=dh, dx=torch.empty(rows, cols, dtype=dt, device="cuda"))
    _ok()
    _check_bwd(dx, dw, dy, h, w, rstd, dh)


@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 0), (8, 1)])
@pytest.mark.parametrize("rows,cols", [(90, 520), (700, 1411)])
def test_backward_pitch_in_place_and_empty(rows, cols, pad, offset):
    dy, h, w, dh = rand(1, rows, cols), rand(2, rows, cols), rand(3, cols), rand(4, rows, cols)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    want, wdw = ufp4.rmsnorm_backward(dy, h, w, rstd, dh=dh)
    dhv = strided(dh, pad, offset)
    keep = _around(dhv).clone()
    dx, dw = ufp4.rmsnorm_backward(strided(dy, pad, offset), strided(h, pad, offset), w, rstd, dh=dhv, dx=dhv)
    _ok()
    assert torch.equal(_around(dhv), keep)
    assert dx is dhv
    _check_bwd(dx, dw, dy, h, w, rstd, dh)
    dx, dw = ufp4.rmsnorm_backward(dy, h, w, rstd, dh=dh, want_dweight=False)
    assert dw is None and torch.equal(dx, want)
    dx, dw = ufp4.rmsnorm_backward(dy[:0], h[:0], w, rstd[:0])
    assert dx.shape == (0, cols) and bool((dw == 0).all())
    assert ufp4.rmsnorm(dy[:0], w)[0].shape == (0, cols)


def test_backward_against_differences():
    """d(sum(c * y)) by central differences of the 64-bit forward, along random directions."""
    rows, cols, t = 6, 200, 1e-5
    x, w, c = rand(1, rows, cols, dtype=FP32), rand(3, cols, dtype=FP32), rand(4, rows, cols, dtype=FP32)
    _, _, _, rstd = ufp4.rmsnorm(x, w, eps=EPS)
    dx, dw = ufp4.rmsnorm_backward(c, x, w, rstd)
    _ok()
    for seed in range(4):
        v, u = rand(10 + seed, rows, cols, dtype=FP32).double(), rand(20 + seed, cols, dtype=FP32).double()

        def f(s):
            h = x.double() + s * v
            r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
            return float((c.double() * h * r * (w.double() + s * u)).sum())

        num = (f(t) - f(-t)) / (2 * t)
        got = float((dx.double() * v).sum() + (dw.double() * u).sum())
        size = float((dx.double() * v).abs().sum() + (dw.double() * u).abs().sum())
        assert abs(got - num) <= 64 * 2.0 ** -24 * size + 1e-8 * size     # arithmetic; t^2 terms


def test_same_bits_streams_and_graph():
    rows, cols = 3000, 2048
    dy, h, w = rand(1, rows, cols), rand(2, rows, cols), rand(3, cols)
    y, _, _, rstd = ufp4.rmsnorm(h, w)
    dx, dw = ufp4.rmsnorm_backward(dy, h, w, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, _, _, r2 = ufp4.rmsnorm(h, w)
        dx2, dw2 = ufp4.rmsnorm_backward(dy, h, w, r2)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in ((y, y2), (rstd, r2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)
    q = ufp4.empty_qtensor(rows, cols, ufp4.CFG_8BIT)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, _, _, rg = ufp4.rmsnorm(h, w, q=q)
        dxg, dwg = ufp4.rmsnorm_backward(dy, h, w, rg)
    h.copy_(rand(5, rows, cols))
    g.replay()
    _, _, _, r3 = ufp4.rmsnorm(h, w)
    dx3, dw3 = ufp4.rmsnorm_backward(dy, h, w, r3)
    _ok()
    assert torch.equal(rg, r3) and torch.equal(dxg, dx3) and torch.equal(dwg, dw3)
    _check_q(q, _expect(h, None, w, 1e-6)[2])
