"""The phase of the rotary append: the plan's fractions of a turn and the turned values against 60-digit arithmetic."""
import decimal
import math
import random
from decimal import Decimal

import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests.serving import NHD, Cache, ints

CTX = decimal.Context(prec=60)
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")

CONFIGS = [
    dict(rot_dim=128, base=10000.0),
    dict(rot_dim=44, base=500000.0, scaling=dcp.DCP_ROPE_LINEAR, factor=3.0),
    dict(rot_dim=64, base=10000.0, scaling=dcp.DCP_ROPE_BASE, factor=8.0),
    dict(rot_dim=96, base=500000.0, scaling=dcp.DCP_ROPE_PARTS, factor=8.0),
    dict(rot_dim=2, base=7.0, scaling=dcp.DCP_ROPE_BASE, factor=2.0),
]


def turns(cfg: dcp.RopeConfig):
    """theta_p / (2 pi) of every pair."""
    with decimal.localcontext(CTX):
        base, f, out = Decimal(cfg.base), Decimal(cfg.factor), []
        if cfg.scaling == dcp.DCP_ROPE_BASE and cfg.rot_dim > 2:
            base = ((f.ln() * cfg.rot_dim) / (cfg.rot_dim - 2)).exp() * base
        for p in range(cfg.rot_dim // 2):
            t = (base.ln() * (-2 * p) / cfg.rot_dim).exp()
            if cfg.scaling == dcp.DCP_ROPE_LINEAR:
                t /= f
            if cfg.scaling == dcp.DCP_ROPE_PARTS:
                fast, slow = Decimal(cfg.beta_fast), Decimal(cfg.beta_slow)
                g = (Decimal(cfg.orig_len) * t / TWO_PI - slow) / (fast - slow)
                g = min(max(g, Decimal(0)), Decimal(1))
                t = t * (g + (1 - g) / f)
            out.append(t / TWO_PI)
        return out


@pytest.mark.parametrize("kw", CONFIGS)
def test_plan_fractions(kw):
    """2^-62 turns a position: 2^-31 turns at the ends of the int32 range."""
    cfg = dcp.RopeConfig(**kw)
    plan = dcp.dcp_rope_plan(cfg)
    with decimal.localcontext(CTX):
        for p, t in enumerate(turns(cfg)):
            off = Decimal(plan.turns[p]) / 2 ** 64 - (t - t.to_integral_value(decimal.ROUND_FLOOR))
            assert abs(off - off.to_integral_value()) <= Decimal(2) ** -62, p


@pytest.mark.gpu
@pytest.mark.parametrize("kw", CONFIGS)
@pytest.mark.parametrize("far", [100, 10 ** 6, 2 ** 31 - 1])
def test_append_phase(gpu, kw, far):
    """Tokens whose pairs are (1, 0) turn to (cos, sin): off by 2^-30 turns, and by roundings relative to the value (2
    ulp of sine or cosine, a correction and a product)."""
    cfg = dcp.RopeConfig(pair_layout=dcp.DCP_ROPE_HALF, **kw)
    n, d, half = 60, 128, cfg.rot_dim // 2
    r = random.Random(far)
    pos = [r.randint(-far - 1 if far > 2 ** 30 else -far, far) for _ in range(n - 2)] + [far, -far]
    c = Cache("f32", NHD, 1, d, 16, [n], [n])
    x = torch.zeros(n, 1, d, device="cuda")
    x[:, :, :half] = 1.0
    out = torch.empty_like(x)
    dcp.dcp_rope_append(c.pool(), c.batch(), dcp.dcp_rope_plan(cfg), x, x, x, ints(pos), out)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    got = out[:, 0].double().cpu()
    want = torch.zeros(n, 2 * half, dtype=torch.float64)
    with decimal.localcontext(CTX):
        for p, t in enumerate(turns(cfg)):
            for i, y in enumerate(pos):
                z = y * t
                eighth = (z * 8).to_integral_value()            # nearest eighth of a turn, the rest below a sixteenth
                rest = float((z - eighth / 8) * TWO_PI)
                k = int(eighth) % 8
                a, b = math.cos(k * math.pi / 4), math.sin(k * math.pi / 4)
                a, b = (x if abs(x) > 0.5 else 0.0 for x in (a, b))
                want[i, p] = a * math.cos(rest) - b * math.sin(rest)
                want[i, p + half] = b * math.cos(rest) + a * math.sin(rest)
    tol = 2 * math.pi * 2.0 ** -30 + 2.0 ** -22 * want.abs()
    off = (got[:, :2 * half] - want).abs()
    assert (off <= tol).all(), (off - tol).max().item()
