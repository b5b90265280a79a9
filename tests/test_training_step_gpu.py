"""The operators together, as a training step runs them: a layer's forward and
backward pass around the quantized GEMMs, dense and mixture-of-experts, against
the same step in 64 bits on the same quantized operands, and against itself
captured into a graph."""
import math

import pytest
import torch

from fp4_quantized_gemms_b200 import ufp4
from tests.gpu_util import needs_gpu
from tests.op_util import BF16, FP32, act64, product64, rand, slope64, values64

pytestmark = needs_gpu

C, R = ufp4.ALONG_COLS, ufp4.ALONG_ROWS
MX0 = ufp4.QuantConfig(block=32, scale_fmt=ufp4.SCALE_UE8M0, hadamard_n=0)
TWO = ufp4.QuantConfig(block=16, scale_fmt=ufp4.SCALE_E4M3_X_FP32)
SR = TWO.with_(rounding=ufp4.ROUND_SR, sr_seed=7)


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


class Layer:
    """y = x + W2 gelu(W1 norm(x + prev) + b1): 8-bit activations into the
    first product, UFP4 operands everywhere else."""

    def __init__(self, m=384, d=256, f=704):
        self.m, self.d, self.f = m, d, f
        self.x, self.prev = rand(1, m, d), rand(2, m, d)
        self.w, self.b1 = rand(3, d, std=0.1) + 1, rand(4, f, std=0.1, dtype=FP32)
        self.W1, self.W2 = rand(5, f, d, std=0.06), rand(6, d, f, std=0.04)
        self.dout = rand(7, m, d, std=0.1)

    def step(self):
        t = self
        n8 = ufp4.empty_qtensor(t.m, t.d, ufp4.CFG_8BIT)
        _, _, h, rstd = ufp4.rmsnorm(t.x, t.w, residual=t.prev, q=n8)
        w1 = ufp4.rht_quantize(t.W1, C, MX0)
        pre = torch.empty(t.m, t.f, dtype=BF16, device="cuda")
        a = ufp4.gemm_epilogue(n8, w1, bias=t.b1, act=ufp4.ACT_GELU, pre=pre)
        aq, w2 = ufp4.rht_quantize(a, C, TWO), ufp4.rht_quantize(t.W2, C, TWO)
        y = ufp4.gemm_epilogue(aq, w2, residual=h)
        # backward
        dyq, w2t = ufp4.rht_quantize(t.dout, C, SR), ufp4.rht_quantize(t.W2, R, TWO)
        da = ufp4.gemm_dgrad(dyq, w2t)
        dyt, at = ufp4.rht_quantize(t.dout, R, SR.with_(sr_stream=1)), ufp4.rht_quantize(a, R, TWO)
        dW2 = ufp4.gemm_wgrad(dyt, at)
        dpre, db1 = ufp4.epilogue_backward(da, pre, ufp4.ACT_GELU)
        dpq, w1t = ufp4.rht_quantize(dpre, C, SR.with_(sr_stream=2)), ufp4.rht_quantize(t.W1, R, TWO)
        dn = ufp4.gemm_dgrad(dpq, w1t)
        dx, dw = ufp4.rmsnorm_backward(dn, h, t.w, rstd, dh=t.dout)
        grads = [dW2, db1, dw]
        clipped = [torch.empty(g.shape, dtype=BF16, device="cuda") for g in grads]
        norm = ufp4.grad_clip(grads, 0.5, out=clipped)
        self.kept = dict(n8=n8, w1=w1, aq=aq, w2=w2, dyq=dyq, w2t=w2t, dyt=dyt, at=at, dpq=dpq, w1t=w1t, pre=pre)
        return dict(h=h, a=a, y=y, da=da, dW2=dW2, dpre=dpre, db1=db1, dn=dn, dx=dx, dw=dw, norm=norm,
                    clipped=clipped, rstd=rstd)


def test_dense_layer_step():
    """Each result against its formula in 64 bits on the step's own quantized
    operands: fp32 results within 2e-5 (the GEMMs' bound and sums of a few
    hundred terms), bf16 ones within half a step of it."""
    t = Layer()
    o = t.step()
    torch.cuda.synchronize()
    assert ufp4.check_device_status() == ufp4.OK
    k = t.kept
    half = 2.0 ** -8
    h = (t.x.double() + t.prev.double()).to(BF16).double()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)
    n64 = h * r * t.w.double()
    assert torch.equal(o["h"].double(), h)
    # the 8-bit norm: half an E4M3 step of each element, or half the step of the block's smallest exponents
    err = (values64(k["n8"])[:, :t.d] - n64).abs()
    step = torch.exp2(k["n8"].scales[:, :t.m].t().double() - 127).repeat_interleave(32, 1)[:, :t.d]
    assert bool((err <= torch.maximum(n64.abs() / 16, step * 2.0 ** -10) * 1.001 + 1e-6).all())
    z = product64(k["n8"], k["w1"]) + t.b1.double()
    assert _rel(k["pre"], z) <= half and _rel(o["a"], act64(z, "gelu")) <= half
    assert _rel(o["y"], product64(k["aq"], k["w2"]) + h) <= half
    assert _rel(o["da"], product64(k["dyq"], k["w2t"])) <= 2e-5 and _rel(o["dW2"], product64(k["dyt"], k["at"])) <= 2e-5
    dp = o["da"].double() * slope64(k["pre"].double(), "gelu")
    assert _rel(o["dpre"], dp) <= half and _rel(o["db1"], dp.sum(0)) <= 2e-5
    dn = product64(k["dpq"], k["w1t"])
    assert _rel(o["dn"], dn) <= 2e-5
    xh, g = h * r, o["dn"].double() * t.w.double()
    assert _rel(o["dx"], r * (g - xh * (g * xh).mean(1, keepdim=True)) + t.dout.double()) <= half
    assert _rel(o["dw"], (o["dn"].double() * xh).sum(0)) <= 2e-5
    n = math.sqrt(sum(float(o[x].double().square().sum()) for x in ("dW2", "db1", "dw")))
    assert abs(float(o["norm"]) - n) <= 1e-6 * n and n > 0.5
    for c, x in zip(o["clipped"], ("dW2", "db1", "dw")):
        assert _rel(c, o[x].double() * (0.5 / n)) <= half


def test_dense_layer_step_in_a_graph():
    """Captured once, replayed on other inputs: the same bits as eagerly."""
    t = Layer()
    t.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = t.step()
    for name, seed in (("x", 11), ("prev", 12), ("dout", 13)):
        v = getattr(t, name)
        v.copy_(rand(seed, *v.shape, std=0.3))
    g.replay()
    torch.cuda.synchronize()
    got = {k: ([x.clone() for x in v] if isinstance(v, list) else v.clone()) for k, v in o.items()}
    want = t.step()
    torch.cuda.synchronize()
    assert ufp4.check_device_status() == ufp4.OK
    for k, v in want.items():
        for a, b in zip(v if isinstance(v, list) else [v], got[k] if isinstance(v, list) else [got[k]]):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("experts,topk", [(8, 2), (12, 3)])
def test_router_with_grouped_gemm(experts, topk):
    """Router -> counts -> the grouped GEMM's table -> expert products; the
    balance gradient joins the router's."""
    tokens, d, f = 512, 256, 192
    x = rand(1, tokens, d)
    logits = x.float() @ rand(2, d, experts, std=0.1, dtype=FP32)
    choice = torch.topk(logits, topk, dim=1).indices.to(torch.int32)
    loss, counts, valid = ufp4.moe_balance(logits, choice, coef=0.01)
    # routed rows, each expert's segment padded to 64
    order = torch.argsort(choice.reshape(-1).long(), stable=True)
    pad = (counts + 63) // 64 * 64
    start = torch.cumsum(pad, 0) - pad
    total = int(pad.sum())
    seg = torch.cumsum(counts, 0) - counts
    e = choice.reshape(-1).long()[order]
    rows = start[e] + torch.arange(tokens * topk, device="cuda") - seg[e]
    routed = torch.zeros(total, d, dtype=BF16, device="cuda")
    routed[rows] = x[order // topk]
    W = rand(3, experts * f, d, std=0.05)
    groups = torch.zeros(experts, 9, dtype=torch.int64, device="cuda")
    idx = torch.arange(experts, device="cuda")
    groups[:, 0], groups[:, 1], groups[:, 2] = counts, f, d
    groups[:, 3], groups[:, 5], groups[:, 7] = start, idx * f, start
    xq, wq = ufp4.rht_quantize(routed, C, TWO), ufp4.rht_quantize(W, C, TWO)
    out = torch.zeros(total, f, dtype=FP32, device="cuda")
    ufp4.grouped_gemm(xq, wq, groups, out)
    dl = ufp4.moe_balance_backward(logits, counts, valid, torch.ones(1, device="cuda"), topk=topk, coef=0.01)
    torch.cuda.synchronize()
    assert ufp4.check_device_status() == ufp4.OK
    assert int(valid) == tokens and int(counts.sum()) == tokens * topk
    a, b = values64(xq), values64(wq)
    for i in range(experts):
        s, c = int(start[i]), int(counts[i])
        if c:
            want = a[s:s + c] @ b[i * f:(i + 1) * f].t() / TWO.hadamard_n
            assert _rel(out[s:s + c], want) <= 1e-5
    p = torch.softmax(logits.double(), 1)
    fr = counts.double() / (tokens * topk)
    assert abs(float(loss) - float(0.01 * experts * (fr * p.mean(0)).sum())) <= 1e-5 * float(loss)
    g = 0.01 * experts * fr / tokens
    assert _rel(dl, p * (g - (p * g).sum(1, keepdim=True))) <= 1e-5
