"""Global gradient norm and clipping against 64-bit sums."""
import math

import pytest
import torch

from fp4_quantized_gemms_b200 import ufp4
from tests.gpu_util import needs_gpu
from tests.op_util import BF16, FP32, half_step, rand

pytestmark = needs_gpu

# eight squares in fp32 (nine roundings at most, halved by the root), fp64
# after that, one rounding to fp32
N_REL = 6 * 2.0 ** -24


def _ok():
    torch.cuda.synchronize()
    assert ufp4.check_device_status() == ufp4.OK


def _norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def _check(ts, out, max_norm, before):
    n64 = _norm64(before)
    c = max_norm / n64 if n64 > max_norm else 1.0
    for o, b in zip(out, before):
        want = b.double() * c
        lim = half_step(o.dtype) * want.abs() * 1.001 + 2 * 2.0 ** -24 * want.abs() + 1e-45
        assert bool(((o.double() - want).abs() <= lim).all())


SIZES = [[1], [7], [8, 9], [16384], [16385, 3], [100_003, 1, 64, 5_000_000, 0, 17], [3] * 70, [1000] * 600]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("src,dst", [(FP32, None), (BF16, None), (FP32, BF16), (BF16, FP32), (FP32, FP32)])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_sizes(sizes, src, dst, max_norm):
    ts = [rand(i + 1, n, dtype=src) for i, n in enumerate(sizes)]
    before = [t.clone() for t in ts]
    n0 = ufp4.grad_norm(ts)
    out = [torch.empty(t.numel(), dtype=dst, device="cuda") for t in ts] if dst else None
    norm = ufp4.grad_clip(ts, max_norm, out=out)
    _ok()
    n64 = _norm64(before)
    assert abs(float(norm) - n64) <= N_REL * n64 and torch.equal(norm, n0)
    _check(ts, out if dst else ts, max_norm, before)
    if dst:
        assert all(torch.equal(a, b) for a, b in zip(ts, before))
    if max_norm > n64 and not dst:
        assert all(torch.equal(a, b) for a, b in zip(ts, before))


def test_shapes_views_and_alignment():
    """Matrices, views that start anywhere, mixed types in one list; what lies
    around a view stays."""
    buf = rand(1, 50_000, dtype=FP32)
    hb = rand(2, 50_000)
    ts = [buf[3:1004], buf[2000:12_000].view(100, 100), hb[1:778], hb[800:1600].view(2, 20, 20), buf[20_001:20_002]]
    keep, hkeep = buf.clone(), hb.clone()
    before = [t.clone() for t in ts]
    norm = ufp4.grad_clip(ts, 0.25)
    _ok()
    assert abs(float(norm) - _norm64(before)) <= N_REL * _norm64(before)
    _check(ts, ts, 0.25, before)
    for b, k, spans in ((buf, keep, [(3, 1004), (2000, 12_000), (20_001, 20_002)]), (hb, hkeep, [(1, 778), (800, 1600)])):
        rest = torch.ones(50_000, dtype=torch.bool, device="cuda")
        for s, e in spans:
            rest[s:e] = False
        assert torch.equal(b[rest], k[rest])


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-12, 1e15, 1e30])
def test_range(scale):
    """Squares that leave fp32 at either end still give the norm."""
    ts = [rand(1, 3001, dtype=FP32) * scale, rand(2, 40, dtype=FP32) * scale, torch.zeros(77, device="cuda")]
    before = [t.clone() for t in ts]
    norm = ufp4.grad_clip(ts, 0.5 * scale)
    _ok()
    assert abs(float(norm) - _norm64(before)) <= N_REL * _norm64(before)
    n64 = _norm64(before)
    for o, b in zip(ts, before):
        want = b.double() * (0.5 * scale / n64)
        assert bool(((o.double() - want).abs() <= 4 * 2.0 ** -24 * want.abs() + 2.0 ** -149).all())


def test_zero_gradients_and_zero_norm():
    ts = [torch.zeros(1000, device="cuda"), torch.zeros(10, dtype=BF16, device="cuda")]
    assert float(ufp4.grad_clip(ts, 1.0)) == 0.0 and bool((ts[0] == 0).all())
    ts = [rand(1, 500, dtype=FP32)]
    ufp4.grad_clip(ts, 0.0)
    assert bool((ts[0] == 0).all())
    e = [torch.empty(0, device="cuda")]
    assert float(ufp4.grad_norm(e)) == 0.0 and float(ufp4.grad_clip(e, 1.0)) == 0.0
    _ok()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("separate", [False, True])
def test_not_finite(bad, separate):
    """A gradient that is not finite shows in the norm, and nothing is scaled."""
    ts = [rand(1, 1000, dtype=FP32), rand(2, 333)]
    ts[1][100] = bad
    before = [t.clone() for t in ts]
    out = [torch.zeros_like(t) for t in ts] if separate else None
    norm = ufp4.grad_clip(ts, 0.1, out=out)
    _ok()
    assert bool(norm.isnan() if bad != bad else norm.isinf())
    for o, b in zip(out if separate else ts, before):
        assert torch.equal(torch.nan_to_num(o), torch.nan_to_num(b)) and torch.equal(o.isnan(), b.isnan())


def test_refusals():
    t = rand(1, 100, dtype=FP32)
    with pytest.raises(ufp4.UFP4Error):
        ufp4.grad_clip([t, t], 1.0)
    with pytest.raises(ufp4.UFP4Error):
        ufp4.grad_clip([t[:60], t[50:]], 1.0)
    with pytest.raises(ufp4.UFP4Error):
        ufp4.grad_clip([t], -1.0)
    with pytest.raises(ValueError):
        ufp4.grad_clip([t.view(10, 10).t()], 1.0)
    with pytest.raises(ValueError):
        ufp4.grad_clip([t], 1.0, out=[t[:50]])
    with pytest.raises(ValueError):
        ufp4.grad_clip([t], 1.0, out=[])
    with pytest.raises(ValueError):
        ufp4.grad_norm([])
    with pytest.raises(ValueError):
        ufp4.grad_norm([t.half()])
    ufp4.grad_norm([t, t])            # a norm may see a tensor twice
    _ok()


def test_same_bits_and_graph():
    ts = [rand(i + 1, n, dtype=FP32) for i, n in enumerate([3_000_001, 70_000, 9])]
    first = ufp4.grad_norm(ts)
    assert all(torch.equal(first, ufp4.grad_norm(ts)) for _ in range(3))
    g = torch.cuda.CUDAGraph()
    out = [torch.empty_like(t) for t in ts]
    with torch.cuda.graph(g):
        norm = ufp4.grad_clip(ts, 1.0, out=out)
    for i, t in enumerate(ts):
        t.copy_(rand(30 + i, t.numel(), dtype=FP32))
    g.replay()
    o2 = [torch.empty_like(t) for t in ts]
    n2 = ufp4.grad_clip(ts, 1.0, out=o2)
    _ok()
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(out, o2))
