"""The router's balance loss, counts and logit gradient against 64-bit formulas."""
import pytest
import torch

from fp4_quantized_gemms_b200 import ufp4
from tests.gpu_util import needs_gpu
from tests.op_util import BF16, FP32, half_step, rand, strided

pytestmark = needs_gpu

# p in fp32: exp through ex2 (2^-22, plus 2^-24 per unit of its argument; the
# arguments here reach -40), the sum of up to 1024 terms in a tree of at most
# 32 + 5 additions per lane, a reciprocal and two products.
P_REL = (4 + 40 + 37 + 6) * 2.0 ** -24


def _ok():
    torch.cuda.synchronize()
    assert ufp4.check_device_status() == ufp4.OK


def _case(tokens, e, k, dtype, seed=1, ld_pad=0):
    logits = rand(seed, tokens, e, std=2.0, dtype=dtype)
    logits = strided(logits, ld_pad) if ld_pad else logits
    choice = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    return logits, choice


def _expect(logits, choice, coef, mask=None, dloss=1.0):
    t, e = logits.shape
    keep = torch.ones(t, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    x = logits.double()
    p = torch.softmax(x, 1)
    p = torch.where((x == float("-inf")).all(1, keepdim=True), torch.zeros_like(p), p) * keep[:, None]
    c = choice[keep].long().reshape(-1)
    c = c[(c >= 0) & (c < e)]
    counts = torch.bincount(c, minlength=e)
    n = int(keep.sum())
    if n == 0:
        return torch.zeros((), dtype=torch.float64, device="cuda"), counts, 0, torch.zeros_like(p)
    f = counts.double() / (n * choice.shape[1])
    loss = coef * e * (f * p.sum(0) / n).sum()
    g = dloss * coef * e * f / n
    return loss, counts, n, p * (g - (p * g).sum(1, keepdim=True))


def _check(logits, choice, coef, mask=None, dloss=0.7):
    loss, counts, valid = ufp4.moe_balance(logits, choice, coef=coef, mask=mask)
    d = ufp4.moe_balance_backward(logits, counts, valid, torch.full((1,), dloss, device="cuda"),
                                  topk=choice.shape[1], coef=coef, mask=mask)
    _ok()
    l64, c64, n64, d64 = _expect(logits, choice, coef, mask, dloss)
    assert torch.equal(counts, c64) and int(valid) == n64
    # all terms are positive; a lane adds at most 600 tokens here, then at most 5 + 16 + 296 partial sums
    assert abs(float(loss) - float(l64)) <= (P_REL + 917 * 2.0 ** -24) * abs(float(l64))
    # p (g - dot): p and dot each within P_REL of their size
    size = d64.abs() + 0.0
    p = torch.softmax(logits.double(), 1)
    p = torch.nan_to_num(p)
    g = dloss * coef * logits.shape[1] * c64.double() / max(1, n64 * n64 * choice.shape[1])
    size = p * (g + (p * g).sum(1, keepdim=True))
    lim = half_step(d.dtype) * d64.abs() * 1.001 + 2 * P_REL * size + 1e-37
    assert bool(((d.double() - d64).abs() <= lim).all()), float(((d.double() - d64).abs() - lim).max())
    return loss, counts, valid, d


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("e,k", [(1, 1), (2, 1), (4, 2), (7, 3), (8, 2), (9, 9), (16, 4), (33, 2), (60, 4), (64, 6), (65, 1),
                                 (128, 8), (160, 6), (200, 3), (256, 8), (257, 5), (384, 8), (510, 2), (1000, 8),
                                 (1024, 16)])
@pytest.mark.parametrize("tokens", [1, 37, 4000])
def test_shapes(tokens, e, k, dtype):
    _check(*_case(tokens, e, k, dtype), coef=0.01)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("e", [8, 64, 255, 256])
@pytest.mark.parametrize("pad", [1, 4])
def test_masked_and_strided(e, dtype, pad):
    logits, choice = _case(1500, e, 4, dtype, ld_pad=pad)
    for p in (0.5, 0.001):
        mask = torch.rand(1500, device="cuda") < p
        _, _, _, d = _check(logits, choice, 1.0, mask)
        assert bool((d[~mask] == 0).all())
        a = ufp4.moe_balance(logits, choice, mask=mask)
        b = ufp4.moe_balance(logits, choice, mask=mask.to(torch.uint8) * 3)      # any nonzero byte counts
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("tokens", [0, 5])
def test_nothing_counts(tokens):
    logits, choice = _case(5, 16, 2, FP32)
    mask = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    loss, counts, valid = ufp4.moe_balance(logits[:tokens], choice[:tokens], mask=mask)
    d = ufp4.moe_balance_backward(logits[:tokens], counts, valid, torch.ones(1, device="cuda"), topk=2, mask=mask)
    _ok()
    assert float(loss) == 0 and bool((counts == 0).all()) and int(valid) == 0
    assert d.shape == (tokens, 16) and bool((d == 0).all())


def test_dropped_and_repeated_choices():
    """Indices outside the experts count nowhere; a repeated index counts twice."""
    logits, choice = _case(600, 24, 3, FP32)
    choice[::2, 0] = -1
    choice[1::3, 1] = 24
    choice[5::7, 2] = 2 ** 31 - 1
    choice[3::5] = 7
    _check(logits, choice, 0.3)


def test_left_out_experts_and_empty_rows():
    """-inf logits: probability 0 and gradient 0; a row of nothing but -inf adds nothing."""
    logits, choice = _case(300, 32, 2, FP32)
    logits[:, 5] = float("-inf")
    logits[10] = float("-inf")
    _, _, _, d = _check(logits, choice, 1.0)
    assert bool((d[:, 5] == 0).all()) and bool((d[10] == 0).all())
    masked, _ = _case(300, 32, 2, FP32, seed=3)
    masked[7] = float("nan")
    mask = torch.ones(300, dtype=torch.bool, device="cuda")
    mask[7] = False
    loss, counts, valid = ufp4.moe_balance(masked, choice, mask=mask)      # NaN in a row that does not count
    d = ufp4.moe_balance_backward(masked, counts, valid, torch.ones(1, device="cuda"), topk=2, mask=mask)
    _ok()
    assert bool(loss.isfinite()) and bool(d.isfinite().all()) and bool((d[7] == 0).all())
    loss, counts, valid = ufp4.moe_balance(masked, choice)
    d = ufp4.moe_balance_backward(masked, counts, valid, torch.ones(1, device="cuda"), topk=2)
    _ok()
    assert bool(loss.isnan()) and bool(d[7].isnan().all()) and bool(d[8:].isfinite().all())


def test_large_logits():
    logits, choice = _case(200, 64, 2, FP32)
    _check(logits * 1e4, choice, 1.0)
    shifted = logits + 3e4
    _check(shifted, choice, 1.0)


def test_gradient_against_differences():
    tokens, e, k, t = 20, 12, 2, 1e-6
    logits, choice = _case(tokens, e, k, FP32)
    _, counts, valid, d = _check(logits, choice, 0.5, dloss=1.0)
    for seed in range(4):
        v = rand(50 + seed, tokens, e, dtype=FP32).double()

        def f(s):
            p = torch.softmax(logits.double() + s * v, 1)
            return float(0.5 * e * (counts.double() / (tokens * k) * p.mean(0)).sum())

        num = (f(t) - f(-t)) / (2 * t)
        size = float((d.double() * v).abs().sum())
        assert abs(float((d.double() * v).sum()) - num) <= 4 * P_REL * size + 1e-9


def test_balanced_router():
    """Counts that are equal have no gradient at all; counts that differ by one
    have the small gradient of the difference (to fp32 of itself, not of the
    large terms that cancel in it)."""
    tokens, e = 4096, 16
    logits, _ = _case(tokens, e, 1, FP32)
    choice = (torch.arange(tokens, device="cuda") % e).to(torch.int32)[:, None].contiguous()
    one = torch.ones(1, device="cuda")
    loss, counts, valid = ufp4.moe_balance(logits, choice)
    assert bool((counts == tokens // e).all())
    assert bool((ufp4.moe_balance_backward(logits, counts, valid, one, topk=1) == 0).all())
    choice[0] = 1
    loss, counts, valid = ufp4.moe_balance(logits, choice)
    d = ufp4.moe_balance_backward(logits, counts, valid, one, topk=1)
    _ok()
    want = _expect(logits, choice, 1.0)[3]
    p = torch.softmax(logits.double(), 1)
    # terms: p (g_e - sum p g) with g = +-1 count, each within P_REL of its size
    unit = e / float(tokens) ** 2
    size = p * unit * ((torch.arange(e, device="cuda") < 2).double() + p[:, :2].sum(1, keepdim=True))
    assert bool(((d.double() - want).abs() <= 2 * P_REL * size + half_step(FP32) * want.abs()).all())


def test_in_place_same_bits_streams_and_graph():
    logits, choice = _case(5000, 64, 6, FP32)
    one = torch.ones(1, device="cuda")
    first = ufp4.moe_balance(logits, choice, coef=0.1)
    d = ufp4.moe_balance_backward(logits, first[1], first[2], one, topk=6, coef=0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = ufp4.moe_balance(logits, choice, coef=0.1)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    buf = logits.clone()
    ufp4.moe_balance_backward(buf, first[1], first[2], one, topk=6, coef=0.1, dlogits=buf)
    assert torch.equal(buf, d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lg, cg, vg = ufp4.moe_balance(logits, choice, coef=0.1)
        dg = ufp4.moe_balance_backward(logits, cg, vg, one, topk=6, coef=0.1)
    new, nc = _case(5000, 64, 6, FP32, seed=9)
    logits.copy_(new)
    choice.copy_(nc)
    g.replay()
    l2, c2, v2 = ufp4.moe_balance(logits, choice, coef=0.1)
    d2 = ufp4.moe_balance_backward(logits, c2, v2, one, topk=6, coef=0.1)
    _ok()
    assert torch.equal(lg, l2) and torch.equal(cg, c2) and torch.equal(vg, v2) and torch.equal(dg, d2)
