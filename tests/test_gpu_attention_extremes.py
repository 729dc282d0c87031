"""Paged attention at the ends of the number range.  Expected values come from the formula in 64 bits."""
import math

import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests import serving as sv
from tests.serving import HND, NHD, Cache
from tests.test_gpu_serving import attend

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ infinities a row sees
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 40, 150])
@pytest.mark.parametrize("at", [10, 290])  # 300 keys: in a tile that every row sees whole, and in the last one
def test_attention_infinite_values_that_are_seen(gpu, dtype, nq, at):
    """An infinity in a value a row sees is that row's result in its dim (the weight is above 0), whatever tile it is
    in; every other dim is as without it."""
    c = Cache(dtype, HND, 2, 64, 16, [nq], [300], seed=21).fill()
    q = c.normal(nq, 4, 64)
    clean, _ = attend(c, q, False)
    c.values[0][at, 0, 5], c.values[0][at, 1, 63] = math.inf, -math.inf
    c.fill()
    out, lse = attend(c, q, False)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    assert (out[:, :2, 5] == math.inf).all() and (out[:, 2:, 63] == -math.inf).all()
    want = clean.clone()
    want[:, :2, 5], want[:, 2:, 63] = math.inf, -math.inf
    # the rest through another order of sums at most: both are within their bound of the same 64-bit value
    c.values[0][at] = torch.where(torch.isinf(c.values[0][at]), 0.0, c.values[0][at])
    for h in range(4):
        o, l, mass, terms = sv.attention_64(q[:, h], c.keys[0][:, h // 2], c.values[0][:, h // 2], 300 - nq, 0.125,
                                            False, -1)
        tol, tol_l = sv.attention_bounds(c.dt, 64, 300, o, mass, l, terms)
        fine = torch.isfinite(want[0, h])
        assert ((out[:, h].double() - o).abs() <= tol)[:, fine].all()
        assert ((lse[:, h].double() - l).abs() <= tol_l).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 40, 150])
@pytest.mark.parametrize("at", [10, 290])
def test_attention_keys_of_minus_infinity_that_are_seen(gpu, dtype, nq, at):
    """A score of -inf is a weight of 0: the row is what it is without that key.  (Factors with few significant bits
    are among the queries: 1, 0.5, 3.)"""
    c = Cache(dtype, NHD, 1, 64, 16, [nq], [300], seed=22).fill()
    q = c.normal(nq, 3, 64)
    q[:, 0, 7], q[:, 1, 7], q[:, 2, 7] = 1.0, 0.5, 3.0
    keys = c.keys[0].clone()
    c.keys[0][at, 0, 7] = -math.inf
    c.fill()
    out, lse = attend(c, q, False)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    left = [j for j in range(300) if j != at]
    for h in range(3):
        o, l, mass, terms = sv.attention_64(q[:, h], keys[left, 0], c.values[0][left, 0], 0, 0.125, False, -1)
        tol, tol_l = sv.attention_bounds(c.dt, 64, 300, o, mass, l, terms)
        assert ((out[:, h].double() - o).abs() <= tol).all()
        assert ((lse[:, h].double() - l).abs() <= tol_l).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 150])
def test_attention_nan_that_is_seen(gpu, dtype, nq):
    """NaN stays NaN, in its own dim, also where only its lowest bits are set."""
    c = Cache(dtype, HND, 1, 64, 16, [nq], [300], seed=23).fill()
    low = torch.tensor([0x7F800001], dtype=torch.int32).view(torch.float32) if dtype == "f32" else \
        torch.tensor([0x7F81], dtype=torch.int16).view(torch.bfloat16)
    c.values[0][10, 0, 3:4] = low.cuda()
    c.fill()
    q = c.normal(nq, 2, 64)
    out, _ = attend(c, q, False)
    nan = torch.isnan(out)
    assert nan[:, :, 3].all() and not nan[:, :, :3].any() and not nan[:, :, 4:].any()


# ------------------------------------------------------------------------------------------ scores of any size
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,kv,hq,h", [(1, 600, 2, 2), (1, 9000, 4, 1), (40, 600, 2, 2), (200, 600, 4, 2),
                                        (200, 5000, 2, 1)])
@pytest.mark.parametrize("scale", [3e4, 1e6, -1e9, 1e20, 3e35])
def test_attention_of_a_finite_scale(gpu, dtype, nq, kv, hq, h, scale):
    """Queries and keys are small whole numbers, so products are exact in 32 bits and the largest scores lie at least
    `scale` apart: a row is the mean of the values at its largest score, its lse that score (and the log of their
    number)."""
    c = Cache(dtype, HND, h, 64, 16, [nq], [kv], seed=24)
    c.keys[0] = torch.randint(-8, 9, (kv, h, 64), generator=c.g).to(c.dt).cuda()
    c.fill()
    q = torch.randint(-8, 9, (nq, hq, 64), generator=c.g).to(c.dt).cuda()
    out, lse = attend(c, q, True, -1, scale=scale)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    scale = float(torch.tensor(scale))  # as the call holds it
    step = sv.HALF_STEP[c.dt]
    hidden = torch.arange(kv, device="cuda")[None] > torch.arange(kv - nq, kv, device="cuda")[:, None]
    for i in range(hq):
        k, v = (x[:, i // (hq // h)].double() for x in (c.keys[0], c.values[0]))
        raw = math.copysign(1.0, scale) * (q[:, i].double() @ k.T)
        raw[hidden] = -math.inf
        top = raw.amax(-1, keepdim=True)
        won = (raw == top).double()
        n = won.sum(-1, keepdim=True)
        o, mass, l = won @ v / n, won @ v.abs() / n, (top * abs(scale) + n.log())[:, 0]
        # equal weights of 1 (exact in bf16 too), summed in 32 bits, one reciprocal, the result's rounding
        tol = mass * 8 * 2.0 ** -24 + step * o.abs()
        assert ((out[:, i].double() - o).abs() <= tol).all(), (i, (out[:, i].double() - o).abs().max().item())
        # the score in 32 bits: the scale in units of log2, the product, back, and the logarithm: a few roundings each
        assert ((lse[:, i].double() - l).abs() <= 2.0 ** -21 * l.abs() + 2.0 ** -20).all()


# ------------------------------------------------------------------------------------------ large values
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 200])
@pytest.mark.parametrize("rise", [7.0, 14.0, 30.0, 43.0])
@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** 90, 2.0 ** 100])
def test_attention_large_values_where_scores_rise(gpu, dtype, nq, rise, size):
    """One key late in a tile outweighs all before it by e^rise and its value is large: the quotient is finite, so the
    result is, however far the row's running level lags behind."""
    c = Cache(dtype, HND, 1, 64, 16, [nq], [520], seed=25)
    c.keys[0] = torch.zeros_like(c.keys[0])
    c.values[0] = torch.ones_like(c.values[0])
    for j in (178, 430):
        c.keys[0][j] = rise
        c.values[0][j] = (size * (1 + torch.arange(64) / 64)).to(c.dt).cuda()
    c.fill()
    q = torch.ones(nq, 2, 64, dtype=c.dt, device="cuda")
    out, lse = attend(c, q, False, -1, scale=1.0 / 64)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    o, l, mass, terms = sv.attention_64(q[:, 0], c.keys[0][:, 0], c.values[0][:, 0], 0, 1.0 / 64, False, -1)
    tol, tol_l = sv.attention_bounds(c.dt, 64, 520, o, mass, l, terms)
    for i in range(2):
        assert ((out[:, i].double() - o).abs() <= tol).all()
        assert ((lse[:, i].double() - l).abs() <= tol_l).all()
