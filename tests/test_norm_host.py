"""dcp_norm_rope_append on the host: the axes' plan and what the call refuses, before any CUDA call."""
import ctypes
import math

import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests.test_serving_binding import batch, device, ints, pool, refused
from tests.test_serving_host import BAD_BATCHES, BAD_POOLS, FAKE, B, _batch, _pool, no_gpu


def test_axes_hold_the_plans_of_their_configs():
    cfgs = [dcp.RopeConfig(44, base=10000.0), dcp.RopeConfig(42, base=5000.0, amplitude=1.5), dcp.RopeConfig(42)]
    axes, at = dcp.dcp_rope_axes(cfgs), 0
    for i, cfg in enumerate(cfgs):
        plan, n = dcp.dcp_rope_plan(cfg), cfg.rot_dim // 2
        assert axes.first[i] == at and axes.amplitude[i] == plan.amplitude
        assert list(axes.turns)[at:at + n] == list(plan.turns)[:n]
        at += n
    assert axes.rot_dim == 128 and axes.n_axes == 3
    one = dcp.dcp_rope_axes([dcp.RopeConfig(64, dcp.DCP_ROPE_HALF)])
    assert list(one.first) == [0, 32, 32] and one.pair_layout == dcp.DCP_ROPE_HALF and one.rot_dim == 64


@pytest.mark.parametrize("cfgs", [
    [], [dcp.RopeConfig(2)] * 4, [dcp.RopeConfig(3)], [dcp.RopeConfig(64), dcp.RopeConfig(66)],
    [dcp.RopeConfig(64, dcp.DCP_ROPE_HALF), dcp.RopeConfig(32)], [dcp.RopeConfig(8), dcp.RopeConfig(8, base=-1.0)]])
def test_axes_refused(cfgs):
    refused(dcp.dcp_rope_axes, cfgs)


def test_struct_sizes():
    for i, t in enumerate((dcp.DcpRopeAxesC, dcp.DcpNormConfigC)):
        assert dcp.lib.dcp_abi_norm_struct_size(i) == ctypes.sizeof(t)


def _norm(**over):
    kw = dict(q_weight=FAKE, k_weight=0, weight_dtype=dcp.DCP_BF16, weight_per_head=0, span=0, eps=1e-6)
    kw.update(over)
    return dcp.DcpNormConfigC(**kw)


def _append(pool=None, batch=None, axes=None, norm=None, q=FAKE, q_stride=40 * 128, Hq=40, k=FAKE, v=FAKE,
            kv_stride=8 * 128, positions=None, q_out=FAKE + 4096):
    pool, batch, norm = pool or _pool(), batch or _batch(), norm or _norm()
    axes = axes or dcp.dcp_rope_axes([dcp.RopeConfig(128)])
    return dcp.lib.dcp_norm_rope_append(B(pool), B(batch), B(axes), B(norm), q, q_stride, Hq, k, v, kv_stride, positions,
                                        q_out, None)


@no_gpu
@pytest.mark.parametrize("bad", BAD_POOLS)
def test_bad_pools_refused(bad):
    assert _append(pool=_pool(**bad)) == dcp.DCP_EINVAL


@no_gpu
@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_bad_batches_refused(bad):
    assert _append(batch=_batch(**bad)) == dcp.DCP_EINVAL


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(axes=dcp.DcpRopeAxesC()), dict(axes=dcp.dcp_rope_axes([dcp.RopeConfig(64)] * 2)), dict(q=0), dict(q_out=0),
    dict(k=0), dict(v=0), dict(k=FAKE + 4), dict(q=FAKE + 8), dict(q_stride=40 * 128 - 8), dict(q_stride=40 * 128 + 4),
    dict(kv_stride=8 * 128 - 8), dict(Hq=0), dict(positions=FAKE + 1), dict(q=FAKE, q_out=FAKE, q_stride=56 * 128),
    dict(batch=_batch(kv_len_per_head=1)), dict(norm=_norm(span=2)), dict(norm=_norm(span=-1)), dict(norm=_norm(eps=-1.0)),
    dict(norm=_norm(eps=math.nan)), dict(norm=_norm(eps=math.inf)), dict(norm=_norm(weight_dtype=2)),
    dict(norm=_norm(weight_per_head=2)), dict(norm=_norm(q_weight=FAKE + 8)), dict(norm=_norm(k_weight=FAKE + 2)),
    dict(pool=_pool(D=64, s_row=64, s_head=1024, s_block=8192), q_stride=40 * 64, kv_stride=8 * 64)])
def test_refusals(bad):
    assert _append(**bad) == dcp.DCP_EINVAL


def test_binding_refuses_tensors_of_another_kind():
    w = torch.ones(64)
    refused(dcp.NormConfig, w)
    for bad in (device(w.half()), device(torch.ones(128))[::2], device(torch.ones(2, 2, 64))):
        refused(dcp.NormConfig, bad)
    refused(dcp.NormConfig, device(w), device(w.bfloat16()))
    refused(dcp.NormConfig, device(w), device(torch.ones(2, 64)))
    p, b, axes = pool(), batch(), dcp.dcp_rope_axes([dcp.RopeConfig(64)])
    q, k = (device(torch.zeros(3, h, 64, dtype=torch.bfloat16)) for h in (4, 2))
    call = dcp.dcp_norm_rope_append
    for norm in (dcp.NormConfig(device(torch.ones(32))), dcp.NormConfig(device(torch.ones(2, 64))),
                 dcp.NormConfig(None, device(torch.ones(4, 64)))):
        refused(call, p, b, axes, norm, q, k, k, None, q)
    norm = dcp.NormConfig()
    refused(call, p, b, axes, norm, torch.zeros(3, 4, 64, dtype=torch.bfloat16), k, k, None, q)
    refused(call, p, b, axes, norm, q, k, k, ints(3), q)
    refused(call, p, b, axes, norm, q, k, k, device(ints(6)), q)
    refused(call, p, b, dcp.dcp_rope_axes([dcp.RopeConfig(32)] * 2), norm, q, k, k, device(ints(3)), q)
    refused(call, p, b, axes, norm, q, k, k, None, torch.zeros(3, 4, 64, dtype=torch.bfloat16))
