"""Serving operators on the host: the rotary plan against its definition in 64 bits, and what each call refuses.  The
refusals return before any CUDA call, so they need no device."""
import ctypes
import math

import pytest

import autoregressive_video_diffusion_gb300 as dcp
from tests.conftest import has_gpu
from tests.serving import thetas_64

FAKE = 1 << 40  # aligned, never dereferenced: every call below is refused before any launch
no_gpu = pytest.mark.skipif(has_gpu(), reason="refused calls use fake device addresses")
B = ctypes.byref


@pytest.mark.parametrize("rot", [2, 6, 44, 64, 128])
@pytest.mark.parametrize("scaling,factor", [(dcp.DCP_ROPE_PLAIN, 1.0), (dcp.DCP_ROPE_LINEAR, 8.0),
                                            (dcp.DCP_ROPE_BASE, 4.0), (dcp.DCP_ROPE_PARTS, 8.0)])
def test_rope_plan_holds_the_frequencies(rot, scaling, factor):
    cfg = dcp.RopeConfig(rot, base=500000.0, scaling=scaling, factor=factor, orig_len=4096.0)
    plan = dcp.dcp_rope_plan(cfg)
    for p, theta in enumerate(thetas_64(cfg)):
        # a double's 53 bits through pow, a division and a product: a few ulps; then the fraction's own step
        assert abs(plan.turns[p] * 2.0 ** -64 * 2 * math.pi - theta) <= 16 * 2.0 ** -53 * theta + 2 * math.pi * 2.0 ** -64
    assert all(t == 0 for t in list(plan.turns)[rot // 2:])


@pytest.mark.parametrize("bad", [
    dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=130), dict(pair_layout=2), dict(scaling=4), dict(scaling=-1),
    dict(base=0.0), dict(base=float("nan")), dict(scaling=1, factor=0.0), dict(scaling=2, factor=float("inf")),
    dict(scaling=3, factor=2.0, orig_len=0.0), dict(scaling=3, factor=2.0, beta_fast=1.0, beta_slow=1.0),
    dict(amplitude=float("nan"))])
def test_rope_plan_refusals(bad):
    kw = dict(rot_dim=64)
    kw.update(bad)
    with pytest.raises(dcp.DcpError) as e:
        dcp.dcp_rope_plan(dcp.RopeConfig(**kw))
    assert e.value.status == dcp.DCP_EINVAL


def _pool(**over):
    kw = dict(k=FAKE, v=FAKE + (1 << 36), H=8, D=128, dtype=dcp.DCP_BF16, block_size=16, n_blocks=64,
              s_block=8 * 16 * 128, s_head=16 * 128, s_row=128)
    kw.update(over)
    return dcp.DcpKvPoolC(**kw)


def _batch(**over):
    kw = dict(n_seqs=2, total_q=10, max_q=7, kv_len_per_head=0, max_kv=100, table_stride=8, kv_len_add=0,
              q_start=FAKE, tables=FAKE + 256, kv_len=FAKE + 512, status=FAKE + 768)
    kw.update(over)
    return dcp.DcpSeqBatchC(**kw)


BAD_POOLS = [dict(k=0), dict(v=0), dict(k=FAKE + 8), dict(H=0), dict(D=0), dict(D=4), dict(D=136), dict(D=127),
             dict(dtype=3), dict(block_size=0), dict(n_blocks=0), dict(n_blocks=1 << 31), dict(s_row=0),
             dict(s_head=4), dict(s_block=-8), dict(s_row=1 << 40)]
BAD_BATCHES = [dict(n_seqs=0), dict(n_seqs=65536), dict(total_q=0), dict(max_q=0), dict(max_q=11),
               dict(kv_len_per_head=2), dict(max_kv=-1), dict(table_stride=0), dict(kv_len_add=-1), dict(q_start=0),
               dict(tables=0), dict(kv_len=0), dict(status=0), dict(q_start=FAKE + 2)]


def _append(pool=None, batch=None, plan=None, q=FAKE, q_stride=40 * 128, Hq=40, k=FAKE, v=FAKE, kv_stride=8 * 128,
            positions=None, q_out=FAKE + 4096):
    pool, batch = pool or _pool(), batch or _batch()
    plan = plan or dcp.dcp_rope_plan(dcp.RopeConfig(128))
    return dcp.lib.dcp_rope_append(B(pool), B(batch), B(plan), q, q_stride, Hq, k, v, kv_stride, positions, q_out,
                                   None)


def _attend(pool=None, batch=None, cfg=None, q=FAKE, q_stride=40 * 128, Hq=40, out=FAKE, lse=None, ws=FAKE,
            ws_bytes=1 << 40):
    pool, batch, cfg = pool or _pool(), batch or _batch(), cfg or dcp.AttnConfig().c(128)
    return dcp.lib.dcp_paged_attention(B(pool), B(batch), B(cfg), q, q_stride, Hq, out, lse, ws, ws_bytes, None)


@no_gpu
@pytest.mark.parametrize("bad", BAD_POOLS)
def test_bad_pools_refused(bad):
    assert _append(pool=_pool(**bad)) == dcp.DCP_EINVAL
    assert _attend(pool=_pool(**bad)) == dcp.DCP_EINVAL
    assert dcp.lib.dcp_attention_workspace_size(B(_pool(**bad)), B(_batch()), B(dcp.AttnConfig().c(128)), 40) == 0


@no_gpu
@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_bad_batches_refused(bad):
    assert _append(batch=_batch(**bad)) == dcp.DCP_EINVAL
    assert _attend(batch=_batch(**bad)) == dcp.DCP_EINVAL


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(plan=dcp.DcpRopePlanC()), dict(q=0), dict(q_out=0), dict(k=0), dict(v=0), dict(k=FAKE + 4), dict(q=FAKE + 8),
    dict(q_stride=40 * 128 - 8), dict(q_stride=40 * 128 + 4), dict(kv_stride=8 * 128 - 8), dict(Hq=0),
    dict(positions=FAKE + 1), dict(q=FAKE, q_out=FAKE, q_stride=56 * 128), dict(batch=_batch(kv_len_per_head=1))])
def test_append_refusals(bad):
    assert _append(**bad) == dcp.DCP_EINVAL


@no_gpu
def test_append_refuses_more_pairs_than_the_head_has():
    assert _append(pool=_pool(D=64, s_row=64, s_head=1024, s_block=8192), q_stride=40 * 64,
                   kv_stride=8 * 64) == dcp.DCP_EINVAL


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(q=0), dict(out=0), dict(q=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(q_stride=128),
    dict(q_stride=40 * 128 + 4), dict(Hq=0), dict(Hq=12), dict(ws=0), dict(ws=FAKE + 16), dict(ws_bytes=16),
    dict(cfg=dcp.DcpAttnConfigC(math.nan, 1, -1, 0)), dict(cfg=dcp.DcpAttnConfigC(0.1, 2, -1, 0)),
    dict(cfg=dcp.DcpAttnConfigC(0.1, 0, 5, 0)), dict(cfg=dcp.DcpAttnConfigC(0.1, 1, -2, 0)),
    dict(cfg=dcp.DcpAttnConfigC(0.1, 1, -1, 1))])
def test_attention_refusals(bad):
    assert _attend(**bad) == dcp.DCP_EINVAL


def _pages(**over):
    kw = dict(k=FAKE, v=FAKE, L=2, block_size=16, n_blocks=64, page_bytes=4096, status=FAKE)
    kw.update(over)
    return dcp.DcpPagePoolC(**kw)


@no_gpu
@pytest.mark.parametrize("bad", [dict(k=0), dict(v=0), dict(L=0), dict(block_size=0), dict(n_blocks=0),
                                 dict(n_blocks=1 << 31), dict(page_bytes=0), dict(page_bytes=24), dict(status=0),
                                 dict(k=FAKE + 8), dict(status=FAKE + 2)])
def test_bad_page_pools_refused(bad):
    p, F, L = _pages(**bad), FAKE, dcp.lib
    assert L.dcp_pages_workspace_size(B(p), 4, 8) == 0
    assert L.dcp_pages_copy(B(p), F, F, 1, None) == 1
    assert L.dcp_pages_fork(B(p), F, F, 4, 8, F, None, None, 4, F, F, F, F, 1 << 40, None) == 1
    assert L.dcp_pages_free(B(p), F, 4, 8, F, F, F, None) == 1
    assert L.dcp_pages_compact(B(p), F, 4, 8, F, F, F, F, F, 1 << 40, None) == 1


@no_gpu
def test_page_call_refusals():
    p, F, L = _pages(), FAKE, dcp.lib
    n = L.dcp_pages_workspace_size(B(p), 4, 8)
    assert n > 0 and n % 256 == 0
    assert L.dcp_pages_copy(B(p), None, F, 1, None) == 1
    assert L.dcp_pages_copy(B(p), F, F + 1, 1, None) == 1
    assert L.dcp_pages_copy(B(p), F, F, -1, None) == 1
    assert L.dcp_pages_copy(B(p), None, None, 0, None) == 0
    for k in (0, 1, 2, 5, 6, 7):  # tables, lens, parents, counts in, child tables, counts out
        a = [F, F, F, None, None, F, F, F]
        a[k] = None
        assert L.dcp_pages_fork(B(p), a[0], a[1], 4, 8, a[2], a[3], a[4], 4, a[5], a[6], a[7], F, n, None) == 1
    assert L.dcp_pages_fork(B(p), F, F, 4, 8, F, None, None, 0, F, F, F, F, n, None) == 1
    assert L.dcp_pages_fork(B(p), F, F, 4, 0, F, None, None, 4, F, F, F, F, n, None) == 1
    assert L.dcp_pages_fork(B(p), F, F, 4, 8, F, None, None, 4, F, F, F, F + 16, n, None) == 1
    assert L.dcp_pages_fork(B(p), F, F, 4, 8, F, None, None, 4, F, F, F, F, n - 1, None) == 1
    assert L.dcp_pages_free(B(p), F, 4, 8, F, None, F, None) == 1
    assert L.dcp_pages_free(B(p), F, 0, 8, F, F, F, None) == 1
    assert L.dcp_pages_compact(B(p), F, 4, 8, F, F, None, F, F, n, None) == 1
    assert L.dcp_pages_compact(B(p), F, 4, 8, F, F, F, F + 2, F, n, None) == 1
    assert L.dcp_pages_compact(B(p), F, 4, 8, F, F, F, F, F, 16, None) == 1


def test_serving_struct_sizes():
    for i, t in enumerate((dcp.DcpKvPoolC, dcp.DcpSeqBatchC, dcp.DcpRopeConfigC, dcp.DcpRopePlanC,
                           dcp.DcpAttnConfigC, dcp.DcpPagePoolC)):
        assert dcp.lib.dcp_abi_serving_struct_size(i) == ctypes.sizeof(t)
    assert dcp.lib.dcp_abi_serving_struct_size(6) == 0
