"""dcp_shared_attention on the host: what is refused, before any CUDA call."""
import math

import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests.test_serving_binding import batch, device, ints, pool, refused
from tests.test_serving_host import BAD_BATCHES, BAD_POOLS, FAKE, B, _batch, _pool, no_gpu


def _groups(**over):
    kw = dict(n_groups=1, max_q=10, max_prefix=60, start=FAKE, prefix_len=FAKE + 64)
    kw.update(over)
    return dcp.DcpPrefixGroupsC(**kw)


def _attend(pool=None, batch=None, groups=None, cfg=None, q=FAKE, q_stride=40 * 128, Hq=40, out=FAKE, lse=None, ws=FAKE,
            ws_bytes=1 << 40):
    pool, batch, groups, cfg = pool or _pool(), batch or _batch(), groups or _groups(), cfg or dcp.AttnConfig().c(128)
    return dcp.lib.dcp_shared_attention(B(pool), B(batch), B(groups), B(cfg), q, q_stride, Hq, out, lse, ws, ws_bytes,
                                        None)


@no_gpu
@pytest.mark.parametrize("bad", BAD_POOLS)
def test_bad_pools_refused(bad):
    assert _attend(pool=_pool(**bad)) == dcp.DCP_EINVAL


@no_gpu
@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_bad_batches_refused(bad):
    assert _attend(batch=_batch(**bad)) == dcp.DCP_EINVAL


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(n_groups=0), dict(n_groups=3), dict(max_q=0), dict(max_q=11), dict(max_prefix=-1), dict(start=0),
    dict(prefix_len=0), dict(start=FAKE + 2), dict(prefix_len=FAKE + 1)])
def test_bad_groups_refused(bad):
    assert _attend(groups=_groups(**bad)) == dcp.DCP_EINVAL
    assert dcp.lib.dcp_shared_attention_workspace_size(B(_pool()), B(_batch()), B(_groups(**bad)),
                                                       B(dcp.AttnConfig().c(128)), 40) == 0


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(q=0), dict(out=0), dict(q=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(q_stride=128), dict(Hq=0),
    dict(Hq=12), dict(ws=0), dict(ws=FAKE + 16), dict(ws_bytes=16), dict(cfg=dcp.DcpAttnConfigC(math.nan, 1, -1, 0)),
    dict(cfg=dcp.DcpAttnConfigC(0.1, 0, 5, 0)), dict(cfg=dcp.DcpAttnConfigC(0.1, 1, -1, 1))])
def test_refusals(bad):
    assert _attend(**bad) == dcp.DCP_EINVAL


def test_binding_refuses_tensors_of_another_kind():
    start, prefix = device(ints(2)), device(ints(1))
    for bad in ((ints(2), prefix), (start, ints(1)), (device(ints(3)), prefix), (start, device(torch.zeros(1)))):
        refused(dcp.PrefixGroups, *bad, 5, 3)
    g = dcp.PrefixGroups(start, prefix, 5, 3)
    p, b, cfg = pool(), batch(), dcp.AttnConfig()
    q, ws = (device(torch.zeros(3, h, 64, dtype=torch.bfloat16)) for h in (4, 8))
    host = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    call = dcp.dcp_shared_attention
    refused(call, p, b, g, cfg, host, q, None, ws)
    refused(call, p, b, g, cfg, q, host, None, ws)
    refused(call, p, b, g, cfg, q, q, torch.zeros(3, 4), ws)
    refused(call, p, b, g, cfg, q, q, None, torch.zeros(1 << 16, dtype=torch.uint8))
