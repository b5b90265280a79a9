"""Values at the ends of the operators' ranges: activations and slopes far from
zero, clipping factors below fp32's normal range, norms that have an exact
value, what stays 0 beside values that are not finite."""
import math

import pytest
import torch

from fp4_quantized_gemms_b200 import ufp4
from tests.gpu_util import needs_gpu
from tests.op_util import ACTS, BF16, FP32, eight_bit, half_step, rand, values64

pytestmark = needs_gpu

LOG2E = math.log2(math.e)
U = 2.0 ** -24


def _ok():
    torch.cuda.synchronize()
    assert ufp4.check_device_status() == ufp4.OK


def _terms(z, act):
    """(Phi, z Phi', A) of act = z Phi(z) in 64 bits, without cancellation on
    the left, and A = |log2| of the exponential that the kernels take."""
    if act == "silu":
        s = torch.sigmoid(z)
        return s, z * s * torch.sigmoid(-z), z.abs() * LOG2E
    if act == "gelu":
        a = 2 * math.sqrt(2 / math.pi)
        u = a * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(u)
        return s, z * s * torch.sigmoid(-u) * a * (1 + 3 * 0.044715 * z * z), u.abs() * LOG2E
    return (0.5 * torch.erfc(-z / math.sqrt(2)), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), z * z / 2 * LOG2E)


# The exponential's argument takes at most five roundings (its constants'
# among them), each 2^-24 of it, so ln 2 times that of the result; the
# exponential and reciprocal themselves (2^-22 and 2^-23) and the rest of the
# arithmetic are at most 24 roundings more.
def _relative(a):
    return (5 * math.log(2) * a + 24) * U


# left of these bounds 1 + exp leaves fp32, or the value its normal numbers
LEFT = {"silu": -86.0, "gelu": -9.8, "gelu_erf": -12.5}


@pytest.mark.parametrize("n", [4096, 4099])
@pytest.mark.parametrize("act,near", [("silu", -20.0), ("gelu", -5.0), ("gelu_erf", -3.0)])
def test_slopes_far_left(act, near, n):
    """The slope keeps its sign and its relative accuracy where it is tiny."""
    z = torch.linspace(LEFT[act], near, n, device="cuda").view(1, n)
    d, _ = ufp4.epilogue_backward(torch.ones_like(z), z, ACTS[act], dpre=torch.empty_like(z), want_dbias=False)
    _ok()
    p, q, a = _terms(z.double(), act)
    assert bool(((d.double() - (p + q)).abs() <= _relative(a) * (p.abs() + q.abs())).all())
    assert bool((d < 0).all())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_erf"])
def test_values_far_left(act):
    """act(z) itself, from a bias on a product of zeros and without a product."""
    n = 4096
    bias = torch.linspace(LEFT[act], 6.0, n, device="cuda")
    w = eight_bit(rand(1, n, 64, std=0.05).float())
    zeros = eight_bit(torch.zeros(3, 64, device="cuda"))
    p, _, a = _terms(bias.double(), act)
    want = bias.double() * p
    empty = [ufp4.empty_qtensor(r, 0, w.cfg) for r in (3, n)]
    for q in ((zeros, w), empty):
        y = ufp4.gemm_epilogue(*q, bias=bias, act=ACTS[act], out_dtype=FP32)
        yb = ufp4.gemm_epilogue(*q, bias=bias, act=ACTS[act])
        _ok()
        assert bool(((y.double() - want).abs() <= _relative(a) * want.abs()).all())
        assert bool(((yb.double() - want).abs() <= (_relative(a) + half_step(BF16)) * 1.001 * want.abs()).all())


@pytest.mark.parametrize("dst", [None, FP32, BF16])
@pytest.mark.parametrize("max_norm", [1e-4, 1e-8, 1e-20, 1e-38])
def test_clip_by_a_tiny_factor(max_norm, dst):
    """max_norm / N below fp32's normal numbers: the product need not be."""
    ts = [rand(1, 1003, dtype=FP32) * 3e36, rand(2, 64, dtype=FP32) * 1e20, rand(3, 520) * 1e36]
    before = [t.double() for t in ts]
    out = [torch.empty(t.numel(), dtype=dst, device="cuda") for t in ts] if dst else None
    ufp4.grad_clip(ts, max_norm, out=out)
    _ok()
    m = float(torch.tensor(max_norm, dtype=FP32))            # as the call takes it
    c = m / math.sqrt(sum(float(t.square().sum()) for t in before))
    for o, b in zip(out or ts, before):
        want = b * c
        # the norm's and the factor's roundings, one to the type, and its smallest step
        lim = (half_step(o.dtype) * 1.001 + 8 * U) * want.abs() + 2.0 ** -150 + (2.0 ** -134 if o.dtype == BF16 else 0)
        assert bool(((o.double() - want).abs() <= lim).all())


@pytest.mark.parametrize("rows", [3, 200])
def test_norm_of_ones(rows):
    """The mean of ones is 1 at every width: rstd is 1, and with a weight of
    1.0625, half way between two 8-bit values, the even one is taken."""
    for cols in [*range(1, 300), 999, 1000, 1025, 1409, 2047, 4099, 8191, 12345, 16383, 32761]:
        x = torch.ones(rows, cols, dtype=BF16, device="cuda")
        w = torch.full((cols,), 1.0625, device="cuda")
        q = ufp4.empty_qtensor(rows, cols, ufp4.CFG_8BIT)
        _, _, _, rstd = ufp4.rmsnorm(x, w, eps=0.0, q=q)
        assert bool((rstd == 1).all()), cols
        assert bool((values64(q)[:, :cols] == 1).all()), cols
    _ok()


@pytest.mark.parametrize("rows,cols", [(5, 200), (5, 1990), (300, 1500), (300, 5001)])
def test_padding_of_rows_that_are_not_finite(rows, cols):
    """Elements behind the row are 0 whatever the row holds."""
    x, w = rand(1, rows, cols), rand(2, cols)
    x[1, 3], x[2, 5], x[4] = float("nan"), float("inf"), 0
    q = ufp4.empty_qtensor(rows, cols, ufp4.CFG_8BIT)
    q.elems8.fill_(0x55)
    ufp4.rmsnorm(x, w, eps=0.0, q=q)
    _ok()
    assert q.kpad > cols and bool((q.elems8[:, cols:] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("e", [8, 24, 255, 256, 1000])
@pytest.mark.parametrize("dloss", [float("inf"), float("nan")])
def test_masked_tokens_stay_zero(e, dloss, dtype):
    """A loss gradient that is not finite reaches the tokens that count alone."""
    logits = rand(1, 300, e, dtype=dtype)
    choice = torch.topk(logits.float(), 2, dim=1).indices.to(torch.int32)
    mask = torch.arange(300, device="cuda") % 3 != 0
    _, counts, valid = ufp4.moe_balance(logits, choice, mask=mask)
    d = ufp4.moe_balance_backward(logits, counts, valid, torch.full((1,), dloss, device="cuda"), topk=2, mask=mask)
    _ok()
    assert bool((d[~mask] == 0).all()) and not bool(d[mask].isfinite().all())
