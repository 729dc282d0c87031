"""The serving operators on the GPU against their plain 64-bit statements (tests/serving.py)."""
import math

import numpy as np
import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests import serving as sv
from tests.serving import HND, NHD, Cache, check_attention, check_turned, ints

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ append
APPEND = [
    # dtype, layout, hq, h, d, bs, q_lens, kv_lens, rot, pairs, positions
    ("bf16", HND, 5, 1, 128, 16, [1], [1], 128, 1, None),
    ("bf16", NHD, 8, 8, 64, 5, [3, 1, 7], [3, 12, 40], 64, 0, None),
    ("bf16", HND, 4, 2, 80, 24, [33, 2], [33, 50], 22, 1, 1000000),
    ("bf16", NHD, 2, 1, 40, 8, [9], [30], 14, 0, -70000),
    ("bf16", HND, 3, 3, 128, 32, [130], [1000], 44, 0, 240),
    ("f32", NHD, 4, 4, 32, 7, [5, 0, 6], [5, 3, 13], 30, 1, 2 ** 31 - 70),
    ("f32", HND, 6, 2, 96, 16, [17], [64], 64, 1, -2 ** 31 + 5),
    ("f32", HND, 1, 1, 4, 1, [3], [3], 2, 0, 5),
    ("bf16", NHD, 2, 2, 24, 3, [4], [9], 0, 1, None),
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
@pytest.mark.parametrize("fused", [False, True], ids=["dense", "fused"])
def test_append(gpu, case, fused):
    dtype, layout, hq, h, d, bs, q_lens, kv_lens, rot, pairs, far = case
    c = Cache(dtype, layout, h, d, bs, q_lens, kv_lens, seed=rot + hq).fill()
    n = c.start[-1]
    if fused:
        q, k, v = c.normal(n, hq + 2 * h, d).split([hq, h, h], dim=1)
    else:
        q, k, v = c.normal(n, hq, d), c.normal(n, h, d), c.normal(n, h, d)
    scaling = [dcp.DCP_ROPE_PLAIN, dcp.DCP_ROPE_LINEAR, dcp.DCP_ROPE_BASE, dcp.DCP_ROPE_PARTS][(rot + hq) % 4]
    cfg = dcp.RopeConfig(rot, pairs, scaling=scaling, factor=4.0, amplitude=1.25)
    place = np.concatenate([np.arange(nk - nq, nk) for nq, nk in zip(q_lens, kv_lens)])
    pos = place if far is None else far + np.arange(n) % 60
    out = torch.full((n, hq, d), math.nan, dtype=c.dt, device="cuda")
    k0, v0 = c.k.clone(), c.v.clone()
    dcp.dcp_rope_append(c.pool(), c.batch(), dcp.dcp_rope_plan(cfg), q, k, v, None if far is None else ints(pos), out)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_turned(out, q, pos, cfg)
    # only the new tokens' rows changed: keys turned, values as they are
    for i, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        r = slice(c.start[i], c.start[i + 1])
        block, row = c.rows(i, nk - nq, nk)
        at = (block, slice(None), row) if layout == HND else (block, row)
        check_turned(c.k[at], k[r], pos[r], cfg)
        assert torch.equal(c.v[at], v[r])
        k0[at], v0[at] = c.k[at], c.v[at]
    for a, b in ((c.k, k0), (c.v, v0)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_in_place_keys_only_and_rows_without_a_place(gpu):
    c = Cache("bf16", HND, 2, 64, 8, [6, 3], [4, 9], seed=3)  # the first two tokens of sequence 0 have no position
    n = c.start[-1]
    q, k, v = c.normal(n, 4, 64), c.normal(n, 2, 64), c.normal(n, 2, 64)
    q0, cfg = q.clone(), dcp.RopeConfig(64, dcp.DCP_ROPE_HALF)
    plan = dcp.dcp_rope_plan(cfg)
    dcp.dcp_rope_append(c.pool(), c.batch(), plan, q, k, v, None, q)
    pos = np.concatenate([np.arange(-2, 4), np.arange(6, 9)])
    check_turned(q, q0, pos, cfg)
    k1 = c.k.clone()
    c.k.fill_(math.nan)
    dcp.dcp_rope_append(c.pool(), c.batch(), plan, None, k, v, None, None)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    assert torch.equal(c.k.view(torch.int16), k1.view(torch.int16))
    for i, (lo, skip) in enumerate(((0, 2), (6, 0))):
        block, row = c.rows(i, lo, c.kv_lens[i])
        check_turned(c.k[block, :, row], k[c.start[i] + skip:c.start[i + 1]], np.arange(lo, c.kv_lens[i]), cfg)


@pytest.mark.parametrize("what", ["entry", "negative entry", "length", "q_start", "long"])
def test_append_bad_state_is_reported_and_written_nowhere(gpu, what):
    c = Cache("bf16", NHD, 2, 64, 8, [3, 4], [20, 30], seed=4)
    q, k, v = c.normal(7, 2, 64), c.normal(7, 2, 64), c.normal(7, 2, 64)
    out = torch.zeros_like(q)
    over = {}
    if what == "entry":
        c.tables[0, 2] = c.k.shape[0]
    elif what == "negative entry":
        c.tables[0, 2] = -1
    elif what == "length":
        c.kv_len[0] = c.tables.shape[1] * 8 + 1
    elif what == "q_start":
        c.q_start[0] = -5
    else:
        c.q_start[1], over = 6, dict(max_q=4)
    k0 = c.k.clone()
    dcp.dcp_rope_append(c.pool(), c.batch(**over), dcp.dcp_rope_plan(dcp.RopeConfig(64)), q, k, v, None, out)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_EDEVICE
    block, row = c.rows(1, 0, 30)
    k0[block, row] = c.k[block, row]  # the sound sequence's own rows
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16))


# ------------------------------------------------------------------------------------------ attention
ATTEND = [
    # dtype, layout, hq, h, d, bs, q_lens, kv_lens, causal, window
    ("bf16", HND, 1, 1, 128, 16, [1], [1], True, -1),
    ("bf16", NHD, 8, 1, 128, 16, [1, 1, 1], [1000, 17, 16], True, -1),
    ("bf16", HND, 40, 8, 128, 32, [1, 1], [4097, 5], True, -1),
    ("bf16", HND, 5, 1, 128, 16, [129], [129], True, -1),
    ("bf16", NHD, 10, 2, 128, 16, [257, 3], [700, 258], True, -1),
    ("bf16", HND, 4, 4, 64, 64, [300], [1111], False, -1),
    ("bf16", NHD, 7, 1, 64, 240, [50, 200], [500, 999], True, -1),
    ("bf16", HND, 2, 1, 80, 24, [33, 70], [701, 90], True, 40),
    ("bf16", NHD, 4, 2, 96, 100, [130], [650], True, 129),
    ("bf16", HND, 8, 8, 32, 5, [20, 1], [83, 7], True, 0),
    ("bf16", NHD, 16, 2, 40, 1, [40], [130], False, -1),
    ("bf16", HND, 3, 1, 8, 3, [65, 64, 1], [65, 200, 300], True, -1),
    ("bf16", HND, 130, 1, 64, 16, [2, 5], [90, 300], True, -1),
    ("bf16", HND, 16, 1, 128, 128, [2, 3, 4], [513, 640, 1], True, 1000),
    ("bf16", NHD, 2, 2, 128, 16, [0, 0, 4, 0], [30, 0, 4, 9], True, -1),
    ("f32", HND, 4, 4, 64, 16, [100], [300], True, -1),
    ("f32", NHD, 8, 2, 128, 24, [1, 1], [513, 2], True, -1),
    ("f32", HND, 5, 1, 36, 7, [9, 40], [60, 41], True, 11),
    ("f32", NHD, 2, 2, 32, 128, [64, 65], [64, 400], False, -1),
    ("f32", HND, 3, 1, 4, 1, [2], [5], True, -1),
    ("f32", NHD, 14, 2, 80, 16, [130, 4], [200, 700], True, -1),
]


def attend(c, q, causal=True, window=-1, batch=None, scale=None, lse=True):
    out = torch.full_like(q, math.nan, memory_format=torch.contiguous_format)
    lse = torch.full(q.shape[:2], math.nan, device="cuda") if lse else None
    cfg, pool, batch = dcp.AttnConfig(scale, causal, window), c.pool(), batch or c.batch()
    ws = dcp.new_workspace(dcp.dcp_attention_workspace_size(pool, batch, cfg, q.shape[1]))
    for _ in range(2):  # the workspace is left ready for the next call
        dcp.dcp_paged_attention(pool, batch, cfg, q, out, lse, ws)
    return out, lse


@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
def test_attention(gpu, case):
    dtype, layout, hq, h, d, bs, q_lens, kv_lens, causal, window = case
    c = Cache(dtype, layout, h, d, bs, q_lens, kv_lens, seed=hq + d).fill()
    q = c.normal(c.start[-1], hq, d)
    out, lse = attend(c, q, causal, window)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention(c, q, out, lse, d ** -0.5, causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 6, 150])
def test_attention_rows_that_see_nothing(gpu, dtype, nq):
    """No key at all, and more new tokens than cached positions: out 0, lse -inf for the rows without a key."""
    c = Cache(dtype, HND, 2, 64, 16, [nq, nq, nq], [0, max(nq // 2, 1), 200], seed=1).fill()
    q = c.normal(c.start[-1], 4, 64)
    out, lse = attend(c, q)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention(c, q, out, lse, 0.125, True, -1)
    assert (out[:nq] == 0).all() and (lse[:nq] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,kv", [(4, 40), (200, 333)])
def test_attention_poison_behind_the_masks(gpu, dtype, nq, kv):
    """NaN and infinities in the keys and values of later tokens reach no earlier row."""
    c = Cache(dtype, NHD, 1, 128, 16, [nq], [kv], seed=2)
    bad = kv - nq // 2
    c.keys[0][bad], c.keys[0][bad + 1] = math.nan, math.inf
    c.values[0][bad], c.values[0][bad + 1] = math.inf, math.nan
    c.fill()
    q = c.normal(nq, 4, 128)
    out, lse = attend(c, q)
    sound = bad - (kv - nq)
    c.keys[0], c.values[0] = c.keys[0][:bad], c.values[0][:bad]
    c.q_lens, c.start, c.kv_lens = [sound], [0, sound], [bad]
    check_attention(c, q[:sound], out[:sound], lse[:sound], 128 ** -0.5, True, -1)
    assert torch.isnan(out[sound]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [2, 140])
def test_attention_pages_behind_the_window_may_be_gone(gpu, dtype, nq):
    c = Cache(dtype, HND, 1, 64, 8, [nq], [600], seed=5).fill()
    w = 50
    gone = (600 - nq - w) // 8
    q = c.normal(nq, 2, 64)
    c.tables[0, :gone] = torch.where(torch.arange(gone, device="cuda") % 2 == 0, -1, 1 << 30).to(torch.int32)
    out, lse = attend(c, q, True, w)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention(c, q, out, lse, 0.125, True, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 300])
def test_attention_lengths_by_head(gpu, dtype, nq):
    """A head-specialised cache: each KV head sees its own length, an offset added to all."""
    c = Cache(dtype, HND, 4, 64, 16, [nq, nq], [500, 400], seed=6).fill()
    lens = [[500, 330, 401, nq], [400, 399, nq + 1, 310]]
    c.kv_len = ints([[x - 20 if x >= 20 else x for x in row] for row in lens])
    add = 20
    lens = [[x + add for x in row] for row in c.kv_len.tolist()]
    q = c.normal(2 * nq, 8, 64)
    out, lse = attend(c, q, False, -1, batch=c.batch(kv_len_add=add))
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention(c, q, out, lse, 0.125, False, -1, kv_of=lens)


RAGGED = [
    # dtype, hq, h, d, bs, q_lens, kv_lens: single tokens and drafts of ragged batches, with and without keys
    ("bf16", 8, 2, 128, 16, [1] * 20, [1, 7000, 0, 64, 65, 3, 129, 2048, 1, 1, 900, 16, 0, 5000, 33, 64, 63, 1, 2, 700]),
    ("bf16", 5, 5, 64, 24, [2, 3, 1, 0, 2, 1], [2, 500, 64, 9, 128, 4000]),
    ("f32", 4, 4, 32, 8, [1] * 9, [1, 300, 0, 32, 31, 33, 2, 65, 700]),
    ("f32", 6, 2, 128, 32, [4, 1, 0, 5], [4, 600, 5, 97]),
    ("bf16", 64, 64, 64, 16, [1] * 9, [30, 1, 200, 64, 0, 128, 77, 5, 300]),  # more items than are shared evenly
    ("bf16", 16, 2, 80, 16, [8, 3, 1, 7], [900, 70, 2000, 7]),                # 64 rows a head, keys cut by a span
]


@pytest.mark.parametrize("case", RAGGED, ids=[str(i) for i in range(len(RAGGED))])
@pytest.mark.parametrize("window", [-1, 100])
def test_attention_of_ragged_batches(gpu, case, window):
    dtype, hq, h, d, bs, q_lens, kv_lens = case
    c = Cache(dtype, NHD, h, d, bs, q_lens, kv_lens, seed=d + window).fill()
    q = c.normal(c.start[-1], hq, d)
    out, lse = attend(c, q, True, window)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention(c, q, out, lse, d ** -0.5, True, window)


@pytest.mark.parametrize("nq,kv,hq,h", [(1100, 1600, 40, 40), (100, 20000, 2, 1), (300, 3000, 4, 2)])
def test_attention_items_split_over_the_keys(gpu, nq, kv, hq, h):
    """An incomplete last round of items, and fewer items than SMs."""
    c = Cache("bf16", HND, h, 64, 32, [nq], [kv], seed=11).fill()
    q = c.normal(nq, hq, 64)
    out, lse = attend(c, q, False, -1)
    check_attention(c, q, out, lse, 0.125, False, -1)


def test_calls_of_different_sizes_share_a_workspace(gpu):
    cases = [("bf16", [1] * 12, [3000] * 12, 8, 4), ("bf16", [300], [5000], 4, 2), ("f32", [200, 90], [900, 90], 4, 4),
             ("bf16", [1], [9000], 8, 8)]
    caches = [Cache(t, HND, h, 64, 16, ql, kl, seed=i).fill() for i, (t, ql, kl, hq, h) in enumerate(cases)]
    cfg, size = dcp.AttnConfig(), 0
    for c, (_, _, _, hq, _) in zip(caches, cases):
        size = max(size, dcp.dcp_attention_workspace_size(c.pool(), c.batch(), cfg, hq))
    ws = dcp.new_workspace(size)
    for _ in range(2):
        for c, (_, _, _, hq, _) in zip(caches, cases):
            q = c.normal(c.start[-1], hq, 64)
            out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
            dcp.dcp_paged_attention(c.pool(), c.batch(), cfg, q, out, lse, ws)
            check_attention(c, q, out, lse, 0.125, True, -1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 130])
@pytest.mark.parametrize("rise", [3.0, 40.0, 1000.0])
def test_attention_scores_that_rise_along_the_keys(gpu, dtype, nq, rise):
    """Later keys outweigh the earlier ones by far: running maxima move, by more than 2^64 within a tile for the last."""
    c = Cache(dtype, HND, 1, 64, 16, [nq], [700], seed=12)
    j = torch.arange(700, device="cuda")[:, None, None]
    grow = torch.where(j >= 300, 1.0 + rise * (j // 150 - 1), 1.0)
    c.keys[0] = (c.keys[0].float() * grow).to(c.dt)
    c.fill()
    q = c.normal(nq, 2, 64)
    out, lse = attend(c, q, True, -1)
    check_attention(c, q, out, lse, 0.125, True, -1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 200])
@pytest.mark.parametrize("scale", [60.0, 500.0, -900.0])
def test_attention_scores_in_the_thousands(gpu, dtype, nq, scale):
    """A row is its largest score's value; levels and maxima of 10^4 and more must still be told apart."""
    c = Cache(dtype, HND, 2, 64, 16, [nq], [600], seed=13).fill()
    q = c.normal(nq, 4, 64)
    out, lse = attend(c, q, True, -1, scale=scale)
    check_attention(c, q, out, lse, scale, True, -1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 200])
def test_attention_large_scores_strided_q_no_lse(gpu, dtype, nq):
    """Scores in the hundreds (a softmax with almost one key), a fused projection's q, no lse; another stream."""
    c = Cache(dtype, NHD, 2, 128, 16, [nq], [300], seed=7).fill()
    q = c.normal(nq, 8, 128)[:, 2:6]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, _ = attend(c, q, True, -1, scale=3.0, lse=False)
    s.synchronize()
    check_attention(c, q, out, None, 3.0, True, -1)
    out, lse = attend(c, q, True, -1, scale=-0.05)
    check_attention(c, q, out, lse, -0.05, True, -1)
    out, lse = attend(c, q, True, -1, scale=0.0)
    check_attention(c, q, out, lse, 0.0, True, -1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 140])
@pytest.mark.parametrize("what", ["entry", "negative entry", "length", "negative length", "q_start", "long"])
def test_attention_bad_state_is_reported(gpu, dtype, nq, what):
    c = Cache(dtype, NHD, 1, 64, 8, [nq, nq], [200, 150], seed=8).fill()
    q = c.normal(2 * nq, 2, 64)
    over = {}
    if what == "entry":
        c.tables[0, 2] = c.k.shape[0]
    elif what == "negative entry":
        c.tables[0, 24] = -2
    elif what == "length":
        c.kv_len[0] = c.tables.shape[1] * 8 + 1
    elif what == "negative length":
        c.kv_len[0] = -1
    elif what == "q_start":
        c.q_start[0] = -5
    else:
        over = dict(max_q=max(nq - 1, 1))
        if nq == 1:
            c.q_start[1] = 2
    out, lse = attend(c, q, batch=c.batch(**over))
    assert dcp.dcp_get_status(c.status) == dcp.DCP_EDEVICE
    if what != "long":  # the sound sequence has its result
        c.keys, c.values, c.kv_lens, c.q_lens, c.start = c.keys[1:], c.values[1:], [150], [nq], [0, nq]
        check_attention(c, q[nq:], out[nq:], lse[nq:], 0.125, True, -1)


def test_attention_long_cache(gpu):
    """Element offsets past 2^31 in the pool."""
    bs, nb = 64, (1 << 31) // (64 * 128) + 600
    c = Cache("bf16", HND, 1, 128, bs, [1, 200], [3000, 9000], seed=9)
    k = torch.zeros((nb, 1, bs, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    shift = nb - c.k.shape[0]
    c.table = np.where(c.table >= 0, c.table + shift, -1).astype(np.int32)
    c.tables, c.k, c.v = torch.from_numpy(c.table).cuda(), k, v
    c.fill()
    q = c.normal(201, 4, 128)
    for rows in (slice(0, 201),):
        out, lse = attend(c, q[rows])
        check_attention(c, q[rows], out, lse, 128 ** -0.5, True, -1)


def test_attention_of_a_contiguous_cache_and_in_a_graph(gpu):
    """A KVCache's layer cut into pages (sink, history, one ring slot), replayed from a CUDA graph with new contents."""
    cache = dcp.KVCache(2, 2, 64, dcp.DCP_BF16, cap=16 * 12, hist_cap=32)
    for x in (cache.k, cache.v):
        x.normal_()
    pool = dcp.layer_pool(cache, 1, 16)
    table = ints([[9, 0, 1, 2, 3]])  # ring slot, sink, history (11 of its 32 rows)
    n, status = 4 * 16 + 11, cache.status
    batch = dcp.SeqBatch(ints([0, 7]), table, ints([n]), status, 7, 7, n)
    cfg = dcp.AttnConfig(causal=False)
    q = torch.randn(7, 4, 64, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty(7, 4, device="cuda")
    ws = dcp.new_workspace(dcp.dcp_attention_workspace_size(pool, batch, cfg, 4))
    dcp.dcp_paged_attention(pool, batch, cfg, q, out, lse, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dcp.dcp_paged_attention(pool, batch, cfg, q, out, lse, ws)
    cache.v[1].normal_()
    g.replay()
    torch.cuda.synchronize()
    rows = torch.cat([torch.arange(16 * b, 16 * b + 16) for b in (9, 0, 1, 2, 3)])[:n].cuda()
    for h in range(4):
        o, l, mass, terms = sv.attention_64(q[:, h], cache.k[1, h // 2, rows], cache.v[1, h // 2, rows], 0, 0.125, False,
                                            -1)
        tol, _ = sv.attention_bounds(torch.bfloat16, 64, n, o, mass, l, terms)
        assert ((out[:, h].double() - o).abs() <= tol).all()


def test_binding_refuses_mismatched_tensors(gpu):
    c = Cache("bf16", HND, 2, 64, 8, [3], [9]).fill()
    q = c.normal(3, 4, 64)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    out, cfg = torch.empty_like(q), dcp.AttnConfig()
    for bad in (q.float(), q[:2], q.transpose(1, 2), c.normal(3, 4, 32)):
        with pytest.raises(dcp.DcpError):
            dcp.dcp_paged_attention(c.pool(), c.batch(), cfg, bad, out, None, ws)
    with pytest.raises(dcp.DcpError):
        dcp.dcp_paged_attention(c.pool(), c.batch(), cfg, q, out, torch.empty(3, 4, device="cuda").double(), ws)
    with pytest.raises(dcp.DcpError):
        dcp.dcp_rope_append(c.pool(), c.batch(), dcp.dcp_rope_plan(dcp.RopeConfig(64)), q, q, q, None, out)


# ------------------------------------------------------------------------------------------ pages
class Pages:
    def __init__(self, layers, blocks, shape, bs, lens, stride, seed=0, dtype=torch.bfloat16):
        r = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = (torch.empty((layers, blocks, *shape), dtype=dtype, device="cuda").normal_(generator=g)
                          for _ in range(2))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.pool, self.bs, self.lens = dcp.PagePool(self.k, self.v, bs, self.status), bs, lens
        perm, at = r.permutation(blocks).astype(np.int32), 0
        self.tables = np.full((len(lens), stride), -1, np.int32)
        for i, n in enumerate(lens):
            p = -(-n // bs)
            self.tables[i, :p] = perm[at:at + p]
            at += p
            if i % 3 == 2:
                self.tables[i, :p // 2] = self.tables[i - 1, :p // 2] if -(-lens[i - 1] // bs) >= p // 2 else \
                    self.tables[i, :p // 2]
        self.ref = np.bincount(self.tables[self.tables >= 0], minlength=blocks).astype(np.int32)

    def ws(self, rows):
        return dcp.new_workspace(dcp.dcp_pages_workspace_size(self.pool, rows, self.tables.shape[1]))


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def moved(x, moves):
    y = x.clone()
    for a, b in moves:
        y[:, b] = x[:, a]
    return y


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


SHAPES = [((2, 16, 64), 16, torch.bfloat16), ((5, 3, 8), 5, torch.bfloat16), ((1, 1, 4), 1, torch.float32)]


@pytest.mark.parametrize("shape,bs,dtype", SHAPES)
@pytest.mark.parametrize("layers,n", [(1, 1), (3, 17), (2, 60)])
def test_pages_copy(gpu, shape, bs, dtype, layers, n):
    p = Pages(layers, 130, shape, bs, [1], 4, dtype=dtype)
    perm = np.random.default_rng(n).permutation(130)
    src, dst = np.r_[perm[:n - 1], perm[0]], perm[-n:]  # one source twice
    want = [moved(x, zip(src, dst)) for x in (p.k, p.v)]
    dcp.dcp_pages_copy(p.pool, dev(src), dev(dst))
    assert dcp.dcp_get_status(p.status) == dcp.DCP_OK
    assert same(p.k, want[0]) and same(p.v, want[1])
    dcp.dcp_pages_copy(p.pool, dev([-1, 3, perm[0], 130]), dev([2, 130, perm[-1], 4]))
    assert dcp.dcp_get_status(p.status) == dcp.DCP_EDEVICE
    assert same(p.k, want[0] if n == 1 else moved(want[0], [(perm[0], perm[-1])]))


@pytest.mark.parametrize("shape,bs,dtype", SHAPES)
@pytest.mark.parametrize("blocks,seqs,children,extra", [(40, 3, 1, False), (700, 9, 40, False), (3000, 6, 1100, True)])
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_fork(gpu, shape, bs, dtype, blocks, seqs, children, extra, in_place):
    r = np.random.default_rng(blocks)
    stride = 6
    lens = [int(r.integers(0 if i else 1, 5 * bs)) for i in range(seqs)]
    p = Pages(2, blocks, shape, bs, lens, stride, seed=blocks, dtype=dtype)
    parent = r.integers(0, seqs, children)
    shared = reserve = None
    if extra:
        shared = np.array([r.integers(0, -(-lens[a] // bs) + 1) for a in parent])
        reserve = np.array([int(r.integers(0, 2)) * bs for a in parent])
        need = sum(max(-(-lens[a] // bs), -(-int(e) // bs)) - int(s) for a, s, e in zip(parent, shared, reserve))
        if need > (p.ref == 0).sum():
            shared = np.array([lens[a] // bs for a in parent])
    child, ref, moves = sv.fork_plain(p.tables, lens, parent, shared, reserve, p.ref, bs)
    want = [moved(x, moves) for x in (p.k, p.v)]
    rin = dev(p.ref)
    rout = rin if in_place else torch.full_like(rin, 7)
    out = torch.full((children, stride), 99, dtype=torch.int32, device="cuda")
    dcp.dcp_pages_fork(p.pool, dev(p.tables), dev(lens), dev(parent), dev(shared), dev(reserve), rin, out, rout,
                       p.ws(children))
    assert dcp.dcp_get_status(p.status) == dcp.DCP_OK
    assert np.array_equal(out.cpu().numpy(), child) and np.array_equal(rout.cpu().numpy(), ref)
    assert same(p.k, want[0]) and same(p.v, want[1])
    if not in_place:
        assert np.array_equal(rin.cpu().numpy(), p.ref)


@pytest.mark.parametrize("what", ["full", "parent", "length", "shared", "entry", "free entry"])
def test_pages_fork_that_cannot_be_done_changes_nothing(gpu, what):
    lens, bs = [40, 33], 8
    p = Pages(1, 14, (1, 8, 8), bs, lens, 8, seed=1)
    parent, shared = [0, 1, 0], None
    if what == "full":
        parent, shared = [1, 1, 1], [1, 0, 0]
    elif what == "parent":
        parent = [0, 2, 0]
    elif what == "length":
        lens = [40, 65]
    elif what == "shared":
        shared = [5, 6, 0]
    elif what == "entry":
        p.tables[1, 1] = 14
    else:
        p.tables[1, 1] = int(np.flatnonzero(p.ref == 0)[0])
    k0, rin = p.k.clone(), dev(p.ref)
    rout, out = torch.full_like(rin, 7), torch.full((3, 8), 99, dtype=torch.int32, device="cuda")
    dcp.dcp_pages_fork(p.pool, dev(p.tables), dev(lens), dev(parent), dev(shared), None, rin, out, rout, p.ws(3))
    assert dcp.dcp_get_status(p.status) == (dcp.DCP_ECAPACITY if what == "full" else dcp.DCP_EDEVICE)
    assert (out == -1).all() and torch.equal(rout, rin) and same(p.k, k0)


@pytest.mark.parametrize("blocks,seqs,stride", [(7, 1, 4), (500, 20, 9), (20000, 40, 130)])
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_free(gpu, blocks, seqs, stride, in_place):
    p = Pages(1, blocks, (1, 1, 8), 1, [min(stride, blocks // seqs) - (i % 2) for i in range(seqs)], stride)
    drop = (seqs + 1) // 2
    t, rin = dev(p.tables[:drop]), dev(p.ref)
    tout, rout = (t, rin) if in_place else (torch.zeros_like(t), torch.full_like(rin, 9))
    want = p.ref - np.bincount(p.tables[:drop][p.tables[:drop] >= 0], minlength=blocks)
    dcp.dcp_pages_free(p.pool, t, rin, tout, rout)
    assert dcp.dcp_get_status(p.status) == dcp.DCP_OK
    assert (tout == -1).all() and np.array_equal(rout.cpu().numpy(), want)


@pytest.mark.parametrize("in_place", [False, True])
def test_pages_free_bad_entries(gpu, in_place):
    p = Pages(1, 20, (1, 1, 8), 1, [4, 4], 6)
    t = p.tables.copy()
    t[0, 0], t[1, :3] = 20, t[0, 1]  # past the pool; one block dropped more often than it is held
    rin, td = dev(p.ref), dev(t)
    tout, rout = (td, rin) if in_place else (torch.zeros_like(td), torch.zeros_like(rin))
    dcp.dcp_pages_free(p.pool, td, rin, tout, rout)
    assert dcp.dcp_get_status(p.status) == dcp.DCP_EDEVICE
    t[0, 0] = -1
    want = np.maximum(p.ref - np.bincount(t[t >= 0], minlength=20), 0)
    assert np.array_equal(rout.cpu().numpy(), want) and (tout == -1).all()


@pytest.mark.parametrize("shape,bs,dtype", SHAPES)
@pytest.mark.parametrize("blocks,seqs,stride", [(5, 1, 3), (300, 10, 12), (2500, 30, 40)])
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_compact(gpu, shape, bs, dtype, blocks, seqs, stride, in_place):
    lens = [max(1, bs * min(stride, blocks // (2 * seqs)) - i % bs) for i in range(seqs)]
    p = Pages(3, blocks, shape, bs, lens, stride, seed=seqs, dtype=dtype)
    tables, ref, live, moves = sv.compact_plain(p.tables, p.ref)
    want = [moved(x, moves) for x in (p.k, p.v)]
    t, rin, n = dev(p.tables), dev(p.ref), torch.zeros(1, dtype=torch.int32, device="cuda")
    tout, rout = (t, rin) if in_place else (torch.zeros_like(t), torch.full_like(rin, 9))
    dcp.dcp_pages_compact(p.pool, t, rin, tout, rout, n, p.ws(seqs))
    assert dcp.dcp_get_status(p.status) == dcp.DCP_OK
    assert np.array_equal(tout.cpu().numpy(), tables) and np.array_equal(rout.cpu().numpy(), ref)
    assert n.item() == live and same(p.k, want[0]) and same(p.v, want[1])


def test_pages_compact_all_free_all_live_and_bad_entry(gpu):
    for ref in (np.zeros(70, np.int32), np.ones(70, np.int32)):
        p = Pages(1, 70, (1, 1, 8), 1, [3], 5)
        k0, n = p.k.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        t = dev(p.tables)
        t[0, 4] = 70
        rin = dev(ref)
        out = torch.zeros_like(t)
        dcp.dcp_pages_compact(p.pool, t, rin, out, rin, n, p.ws(1))
        assert dcp.dcp_get_status(p.status) == dcp.DCP_EDEVICE
        assert n.item() == ref.sum() and same(p.k, k0) and np.array_equal(rin.cpu().numpy(), ref)
        assert torch.equal(out, t)
