"""Attention under a window whose first positions stay visible, on the GPU against its 64-bit statement."""
import math

import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests.serving import HND, NHD, Cache, ints
from tests.serving_more import attention_sink_64, check_attention_sink

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, layout, hq, h, d, bs, q_lens, kv_lens, window, sink
    ("bf16", HND, 1, 1, 128, 16, [1], [1], 0, 1),
    ("bf16", NHD, 8, 1, 128, 16, [1, 1, 1], [1000, 17, 16], 100, 4),
    ("bf16", HND, 40, 8, 128, 32, [1, 1], [4097, 5], 1000, 64),
    ("bf16", HND, 40, 8, 128, 32, [1], [4097], 0, 1),
    ("bf16", HND, 8, 8, 64, 16, [1] * 20, [1, 7000, 0, 64, 65, 3, 129, 2048, 1, 1, 900, 16, 0, 5000, 33, 64, 63, 1, 2, 7],
     200, 70),
    ("bf16", NHD, 5, 5, 64, 24, [2, 3, 1, 0, 2, 1], [2, 500, 64, 9, 128, 4000], 63, 129),
    ("bf16", NHD, 16, 2, 80, 16, [8, 3, 1, 7], [900, 70, 2000, 7], 300, 37),
    ("bf16", HND, 5, 1, 128, 16, [129], [129], 20, 5),
    ("bf16", NHD, 10, 2, 128, 16, [257, 3], [2700, 258], 513, 130),
    ("bf16", HND, 4, 4, 64, 64, [300], [1111], 64, 64),
    ("bf16", HND, 4, 4, 64, 64, [300], [1111], 64, 900),       # the sink reaches into the rows' windows
    ("bf16", HND, 4, 4, 64, 64, [300], [1111], 100, 1 << 30),  # and past everything
    ("bf16", NHD, 7, 1, 64, 240, [50, 200], [500, 1999], 300, 250),
    ("bf16", NHD, 7, 1, 64, 240, [50, 200], [500, 1999], 300, 100),
    ("bf16", HND, 2, 1, 80, 24, [33, 70], [701, 90], 40, 11),
    ("bf16", NHD, 4, 2, 96, 100, [130], [1650], 129, 333),
    ("bf16", HND, 8, 8, 32, 5, [20, 1], [183, 7], 0, 3),
    ("bf16", HND, 3, 1, 8, 3, [165, 64, 1], [265, 200, 300], 17, 10),
    ("bf16", HND, 130, 1, 64, 16, [2, 5], [90, 900], 33, 20),
    ("bf16", HND, 1, 1, 64, 16, [600], [600], 100, 200),       # rows whose windows begin at 0 and rows behind the sink
    ("bf16", HND, 1, 1, 128, 128, [700], [900], 1, 1),
    ("bf16", HND, 2, 1, 64, 32, [100], [20000], 9000, 5000),   # items split over the keys
    ("f32", HND, 4, 4, 64, 16, [100], [700], 150, 40),
    ("f32", NHD, 8, 2, 128, 24, [1, 1], [1513, 2], 300, 33),
    ("f32", HND, 5, 1, 36, 7, [9, 40], [160, 41], 11, 6),
    ("f32", NHD, 14, 2, 80, 16, [130, 4], [400, 700], 100, 65),
]


def attend(c, q, window, sink, batch=None, scale=None):
    out = torch.full_like(q, math.nan, memory_format=torch.contiguous_format)
    lse = torch.full(q.shape[:2], math.nan, device="cuda")
    cfg, pool, batch = dcp.AttnConfig(scale, True, window, sink), c.pool(), batch or c.batch()
    ws = dcp.new_workspace(dcp.dcp_attention_workspace_size(pool, batch, cfg, q.shape[1]))
    for _ in range(2):  # the workspace is left ready for the next call
        dcp.dcp_paged_attention(pool, batch, cfg, q, out, lse, ws)
    return out, lse


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_sinks(gpu, case):
    dtype, layout, hq, h, d, bs, q_lens, kv_lens, window, sink = case
    c = Cache(dtype, layout, h, d, bs, q_lens, kv_lens, seed=hq + d).fill()
    q = c.normal(c.start[-1], hq, d)
    out, lse = attend(c, q, window, sink)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention_sink(c, q, out, lse, d ** -0.5, True, window, sink)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 6, 150])
def test_rows_that_see_nothing(gpu, dtype, nq):
    c = Cache(dtype, HND, 2, 64, 16, [nq, nq, nq], [0, max(nq // 2, 1), 200], seed=1).fill()
    q = c.normal(c.start[-1], 4, 64)
    out, lse = attend(c, q, 10, 3)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention_sink(c, q, out, lse, 0.125, True, 10, 3)
    assert (out[:nq] == 0).all() and (lse[:nq] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 7, 140, 300])
@pytest.mark.parametrize("sink", [1, 20, 64, 130])
def test_what_lies_between_is_not_read(gpu, dtype, nq, sink):
    """NaN and infinities behind the first positions and before the windows, and pages there that name no block."""
    c = Cache(dtype, NHD, 2, 64, 8, [nq], [1000], seed=sink)
    w, lo = 50, 1000 - nq - 50  # the first row's window begins at lo
    c.keys[0][sink:lo], c.values[0][sink:lo:2], c.values[0][sink + 1:lo:2] = math.nan, math.inf, math.nan
    c.fill()
    gone = range(-(-sink // 8), lo // 8)
    for i, page in enumerate(gone):
        if i % 3:
            c.tables[0, page] = -1 if i % 2 else 1 << 30
    q = c.normal(nq, 4, 64)
    out, lse = attend(c, q, w, sink)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention_sink(c, q, out, lse, 0.125, True, w, sink)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 140])
@pytest.mark.parametrize("page", [0, 1, 7])
def test_pages_of_the_sink_must_name_a_block(gpu, dtype, nq, page):
    c = Cache(dtype, NHD, 1, 64, 8, [nq], [1000]).fill()
    c.tables[0, page] = -1
    q = c.normal(nq, 2, 64)
    attend(c, q, 50, 60)  # pages 0 .. 7 hold the first 60 positions
    assert dcp.dcp_get_status(c.status) == dcp.DCP_EDEVICE
    dcp.dcp_reset_status(c.status)
    attend(c, q, 50, 8 * page)  # the page is the first one behind the sink
    assert dcp.dcp_get_status(c.status) == (dcp.DCP_OK)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 150])
def test_infinities_a_row_sees_in_the_sink(gpu, dtype, nq):
    """In the masked tile that holds the sink's last position: rows get their due."""
    c = Cache(dtype, HND, 1, 64, 16, [nq], [900], seed=3)
    c.values[0][3, 0, 5], c.values[0][40, 0, 6] = math.inf, math.nan  # seen, and behind the sink
    c.fill()
    q = c.normal(nq, 2, 64)
    out, lse = attend(c, q, 60, 30)
    assert (out[:, :, 5] == math.inf).all()
    out[:, :, 5] = 0
    c.values[0][:, 0, 5] = 0
    check_attention_sink(c, q, out, lse, 0.125, True, 60, 30)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 200])
def test_lengths_by_head_and_scores_that_rise(gpu, dtype, nq):
    c = Cache(dtype, HND, 4, 64, 16, [nq, nq], [500, 400], seed=6)
    for keys in c.keys:
        keys[-40:] = (keys[-40:].float() * 40).to(c.dt)
    c.fill()
    lens = [[500, 330, 401, nq], [400, 399, nq + 1, 310]]
    c.kv_len = ints(lens)
    q = c.normal(2 * nq, 8, 64)
    out, lse = attend(c, q, 64, 20)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention_sink(c, q, out, lse, 0.125, True, 64, 20, kv_of=lens)


def test_a_sink_that_covers_everything_is_no_window(gpu):
    for dtype, nq in (("bf16", 1), ("bf16", 200), ("f32", 30)):
        c = Cache(dtype, HND, 2, 64, 16, [nq], [700], seed=8).fill()
        q = c.normal(nq, 4, 64)
        out, lse = attend(c, q, 3, 1 << 30)
        check_attention_sink(c, q, out, lse, 0.125, True, -1, 0)


def test_long_cache_and_a_graph(gpu):
    """Element offsets past 2^31, replayed with other lengths."""
    bs, nb = 64, (1 << 31) // (64 * 128) + 700
    c = Cache("bf16", HND, 1, 128, bs, [1, 200], [30000, 12000], seed=9)
    k = torch.zeros((nb, 1, bs, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c.tables = torch.where(c.tables >= 0, c.tables + (nb - c.k.shape[0]), -1)
    c.table, c.k, c.v = c.tables.cpu().numpy(), k, v
    c.fill()
    q = c.normal(201, 4, 128)
    out, lse = attend(c, q, 4000, 1000)
    check_attention_sink(c, q, out, lse, 128 ** -0.5, True, 4000, 1000)
    cfg, pool, batch = dcp.AttnConfig(window=4000, sink=1000), c.pool(), c.batch()
    ws = dcp.new_workspace(dcp.dcp_attention_workspace_size(pool, batch, cfg, 4))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dcp.dcp_paged_attention(pool, batch, cfg, q, out, lse, ws)
    c.kv_len.copy_(ints([900, 7003]))
    c.kv_lens, c.keys, c.values = [900, 7003], [x[:n] for x, n in zip(c.keys, (900, 7003))], \
        [x[:n] for x, n in zip(c.values, (900, 7003))]
    g.replay()
    check_attention_sink(c, q, out, lse, 128 ** -0.5, True, 4000, 1000)
