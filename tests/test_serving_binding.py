"""The binding refuses tensors that the GPU cannot reach or that have another shape than the call's, before it passes their
addresses on.  No GPU is needed: a subclass that claims to be on the device stands for a device's tensor, and every call is
refused for another argument."""
import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp


class OnDevice(torch.Tensor):
    """Claims to be a device's; used where another argument is what is refused."""
    is_cuda = True


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def device(t):
    return t.as_subclass(OnDevice)


def pool():
    k = device(torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16))
    return dcp.KVPool(k, k.clone(), dcp.DCP_PAGED_HND)


def batch(n=3, **over):
    t = dict(q_start=device(ints(3)), tables=device(ints(2, 4)), kv_len=device(ints(2)), status=device(ints(1)))
    t.update(over)
    return dcp.SeqBatch(*t.values(), total_q=n, max_q=n, max_kv=9)


def page_pool():
    k = device(torch.zeros(1, 8, 2, 8, 64, dtype=torch.bfloat16))
    return dcp.PagePool(k, k.clone(), 8, device(ints(1)))


def refused(call, *args, **kw):
    with pytest.raises(dcp.DcpError) as e:
        call(*args, **kw)
    assert e.value.status == dcp.DCP_EINVAL


def test_descriptors():
    k = torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16)
    refused(dcp.KVPool, k, k, dcp.DCP_PAGED_HND)
    refused(dcp.KVPool, device(k), k, dcp.DCP_PAGED_HND)
    for name, t in (("q_start", ints(3)), ("tables", ints(2, 4)), ("kv_len", ints(2)), ("status", ints(1))):
        refused(batch, **{name: t})
    refused(batch, tables=device(ints(8)))
    refused(batch, q_start=device(ints(4)))
    p = torch.zeros(1, 8, 2, 8, 64)
    refused(dcp.PagePool, p, p, 8, device(ints(1)))
    refused(dcp.PagePool, device(p), device(p), 8, ints(1))
    refused(dcp.PagePool, device(p), device(p), 8, device(torch.zeros(1)))


def test_append_and_attention():
    p, b, plan, cfg = pool(), batch(), dcp.dcp_rope_plan(dcp.RopeConfig(64)), dcp.AttnConfig()
    q, k, ws = (device(torch.zeros(3, h, 64, dtype=torch.bfloat16)) for h in (4, 2, 8))
    host = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    refused(dcp.dcp_rope_append, p, b, plan, host, k, k, None, q)
    refused(dcp.dcp_rope_append, p, b, plan, q, host[:, :2], k, None, q)
    refused(dcp.dcp_rope_append, p, b, plan, q, k, k, ints(3), q)
    refused(dcp.dcp_rope_append, p, b, plan, q, k, k, None, host)
    refused(dcp.dcp_paged_attention, p, b, cfg, host, q, None, ws)
    refused(dcp.dcp_paged_attention, p, b, cfg, q, host, None, ws)
    refused(dcp.dcp_paged_attention, p, b, cfg, q, q, torch.zeros(3, 4), ws)
    refused(dcp.dcp_paged_attention, p, b, cfg, q, q, None, torch.zeros(1 << 16, dtype=torch.uint8))


def test_pages():
    p, t, ref, ws = page_pool(), device(ints(2, 4)), device(ints(8)), device(torch.zeros(1 << 16, dtype=torch.uint8))
    one, two = device(ints(1)), device(ints(2))
    refused(dcp.dcp_pages_copy, p, ints(1), one)
    refused(dcp.dcp_pages_copy, p, one, two)
    for i, bad in ((0, ints(2, 4)), (0, device(ints(8))), (1, ints(2)), (2, ints(1)), (5, ints(8)), (6, ints(1, 4)),
                   (7, ints(8)), (8, torch.zeros(1 << 16, dtype=torch.uint8))):
        args = [t, two, one, None, None, ref, device(ints(1, 4)), ref, ws]
        args[i] = bad
        refused(dcp.dcp_pages_fork, p, *args)
    for i, bad in ((0, ints(2, 4)), (0, device(ints(8))), (1, ints(8)), (2, ints(2, 4)), (3, ints(8)), (3, device(ints(7)))):
        args = [t, ref, t, ref]
        args[i] = bad
        refused(dcp.dcp_pages_free, p, *args)
        refused(dcp.dcp_pages_compact, p, *args, None, ws)
    refused(dcp.dcp_pages_compact, p, t, ref, t, ref, ints(1), ws)
    refused(dcp.dcp_pages_compact, p, t, ref, t, ref, device(ints(0)), ws)
    refused(dcp.dcp_pages_compact, p, t, ref, t, ref, None, torch.zeros(1 << 16, dtype=torch.uint8))
