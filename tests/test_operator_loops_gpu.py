"""The operators' persistent loops beyond their first turn: several tiles per
CTA pair with an epilogue, several tokens and rows per block; and 8-bit
operands on either side and in groups."""
import pytest
import torch

from fp4_quantized_gemms_b200 import ufp4
from tests import test_epilogue_gpu as epi
from tests import test_norm_gpu as norm
from tests import test_router_gpu as router
from tests.gpu_util import GEMM_RTOL, needs_gpu
from tests.op_util import ACTS, BF16, FP32, act64, eight_bit, product64, rand, values64

pytestmark = needs_gpu

# 17 x 18 tiles of 256 x 256 for the GPU's 74 CTA pairs; M and N end inside a
# tile, N is a whole number of 16-byte units (bulk copies) or odd.
M, N, N_ODD = 4300, 4360, 4359

PAIR = ["e2m1_two", "e2m1_noatoms_b32", "e1m2_lanes", "e1m2_atoms", "e1m2_noatoms", "mx", "mx_noatoms", "w4a8", "w8a8"]


def _ok():
    torch.cuda.synchronize()
    assert ufp4.check_device_status() == ufp4.OK


def _epilogue(fmt, n, k, act, out_t, res_t, pre_t, in_place):
    a, b = epi._operands(fmt, M, n, k)
    bias = rand(5, n, dtype=FP32)                             # another one in every column and tile
    res = rand(6, M, n, dtype=res_t) if res_t else None
    z = product64(a, b) + bias.double()
    want = act64(z, act) + (res.double() if res_t else 0)
    pre = torch.full((M, n), float("nan"), dtype=pre_t, device="cuda") if pre_t else None
    out = res if in_place else torch.full((M, n), float("nan"), dtype=out_t, device="cuda")
    ufp4.gemm_epilogue(a, b, bias=bias, act=ACTS[act], residual=res, pre=pre, out=out)
    _ok()
    if pre_t:
        epi._check(pre, z, z, pre_t)
    epi._check(out, want, z, out_t)


@pytest.mark.parametrize("fmt", PAIR)
@pytest.mark.parametrize("n,out_t,res_t,pre_t,in_place", [
    (N, BF16, BF16, None, True),          # two slots, residual in place
    (N, BF16, BF16, BF16, False),         # one slot and the stored pre-activation
    (N, BF16, None, BF16, False),
    (N, BF16, None, None, False),
    (N, FP32, FP32, None, True),          # one slot of fp32 pieces
    (N, FP32, FP32, FP32, False),         # element-wise: a stored fp32 pre-activation
    (N_ODD, BF16, BF16, BF16, True)])     # element-wise: odd rows
def test_epilogue_tiles_of_a_pair(fmt, n, out_t, res_t, pre_t, in_place):
    _epilogue(fmt, n, 192, "gelu", out_t, res_t, pre_t, in_place)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("fmt", ["mx", "e2m1_two"])
def test_epilogue_activations_over_tiles(fmt, act):
    _epilogue(fmt, N, 448, act, BF16, BF16, None, False)


@pytest.mark.parametrize("fmt", ["e1m2_fp32", "e1m2_nocorr", "mx_codes"])
@pytest.mark.parametrize("n", [N, N_ODD])
def test_epilogue_tiles_of_a_block(fmt, n):
    """The kernels with one CTA per tile."""
    _epilogue(fmt, n, 128, "silu", BF16, BF16, BF16, True)


@pytest.mark.parametrize("m,n", [(1500, 28672), (1500, 28671), (9001, 264)])
def test_epilogue_backward_rows(m, n):
    """Several steps of a chunk: at most 57 + 8 + 32 + 5 additions, fewer than
    the bound of _check_bwd counts."""
    dout, pre = rand(1, m, n, std=0.01), rand(2, m, n, std=3.0)
    dpre, dbias = ufp4.epilogue_backward(dout, pre, ufp4.ACT_GELU)
    _ok()
    epi._check_bwd(dpre, dbias, dout, pre, "gelu")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tokens,e,k", [(131_071, 8, 2), (131_071, 64, 6), (40_000, 255, 4), (131_071, 256, 8),
                                        (40_000, 33, 3), (40_000, 1000, 8), (20_003, 1021, 2)])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_tokens(tokens, e, k, dtype, masked):
    """296 blocks of 16 to 256 tokens at a time: at most 28 additions per lane,
    fewer than the 600 that _check counts."""
    logits, choice = router._case(tokens, e, k, dtype)
    mask = torch.rand(tokens, device="cuda") < 0.8 if masked else None
    _, _, _, d = router._check(logits, choice, 0.5, mask)
    if masked:
        assert bool((d[~mask] == 0).all())


# rows per block: above the ring's eight stages (1500), its three (4000, 8190,
# odd 8191) and two (16384); short rows: several rounds of every warp.
ROWS = [(20_001, 96), (20_001, 500), (12_001, 999), (12_001, 1000), (20_001, 1500), (3001, 4000), (1501, 8190),
        (1501, 8191), (700, 16384)]


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("eight", [False, True])
def test_norm_rows(rows, cols, eight):
    x, res, w = rand(1, rows, cols), rand(2, rows, cols, std=2.0), rand(3, cols)
    h64, r64, y64 = norm._expect(x, res, w)
    q = ufp4.empty_qtensor(rows, cols, ufp4.CFG_8BIT) if eight else None
    y, _, h, rstd = ufp4.rmsnorm(x, w, residual=res, eps=norm.EPS, q=q, h=res)
    _ok()
    assert torch.equal(h.double(), h64)
    assert bool(((rstd.double() - r64).abs() <= norm.ARITH * r64).all())
    if eight:
        norm._check_q(q, y64)
    else:
        assert bool(((y.double() - y64).abs() <= (2.0 ** -8 * 1.001 + norm.ARITH) * y64.abs()).all())


@pytest.mark.parametrize("rows,cols", ROWS)
def test_norm_backward_rows(rows, cols):
    """At most 148 * 4 blocks: a partial sum of at most 34 rows (short rows:
    8 and four warps), then 19 + 5 additions; fewer than _check_bwd counts."""
    dy, h, w, dh = rand(1, rows, cols), rand(2, rows, cols, std=2.0), rand(3, cols), rand(4, rows, cols)
    rstd = torch.rsqrt(h.double().square().mean(1) + norm.EPS).float()
    keep = dh.clone()
    dx, dw = ufp4.rmsnorm_backward(dy, h, w, rstd, dh=dh, dx=dh)
    _ok()
    norm._check_bwd(dx, dw, dy, h, w, rstd, keep)


# ------------------------------------------------- 8-bit operands on either side
def _mx4(x, **kw):
    cfg = ufp4.QuantConfig(grid=0, block=32, scale_fmt=ufp4.SCALE_UE8M0, hadamard_n=0)
    return ufp4.rht_quantize(x, ufp4.ALONG_COLS, cfg, **kw)


@pytest.mark.parametrize("atoms", [True, False])
@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (300, 520, 448), (257, 130, 1000)])
def test_four_bit_times_eight_bit(m, n, k, atoms):
    a, b = _mx4(rand(1, m, k), with_atoms=atoms), eight_bit(rand(2, n, k).float(), atoms)
    want = product64(a, b)
    for y in (ufp4.gemm_fprop(a, b), ufp4.gemm_epilogue(a, b, out_dtype=FP32)):
        _ok()
        assert float((y.double() - want).norm() / want.norm()) <= GEMM_RTOL


@pytest.mark.parametrize("first,second", [(8, 8), (8, 4), (4, 8)])
def test_eight_bit_groups(first, second):
    """Ragged experts (one empty) over windows of rows and of K; what lies
    between the groups stays."""
    hidden, ffn, counts = 320, 264, [70, 0, 300, 1, 513, 64]
    starts = [sum((c + 63) // 64 * 64 for c in counts[:e]) for e in range(len(counts))]
    total = starts[-1] + 64
    x, w = rand(1, total, 2 * hidden), rand(2, len(counts) * 272, hidden, std=0.05)
    a = eight_bit(x.float()) if first == 8 else _mx4(x)
    b = eight_bit(w.float()) if second == 8 else _mx4(w)
    table = [(c, ffn, hidden, s, hidden * (e % 2), 272 * e, 0, s, 8) for e, (c, s) in enumerate(zip(counts, starts))]
    out = torch.full((total, ffn + 16), 7.0, device="cuda")
    ufp4.grouped_gemm(a, b, torch.tensor(table, dtype=torch.int64, device="cuda"), out)
    _ok()
    av, bv = values64(a), values64(b)
    rest = torch.ones_like(out, dtype=torch.bool)
    for m, n, k, ar, ac, br, bc, cr, cc in table:
        if m:
            want = av[ar:ar + m, ac:ac + k] @ bv[br:br + n, bc:bc + k].t()
            got = out[cr:cr + m, cc:cc + n].double()
            assert float((got - want).norm() / want.norm()) <= GEMM_RTOL
            rest[cr:cr + m, cc:cc + n] = False
    assert bool((out[rest] == 7.0).all())
