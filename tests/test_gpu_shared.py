"""dcp_shared_attention on the GPU: every row against the 64-bit attention over its sequence's own positions."""
import math

import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests.serving import HND, NHD, ints
from tests.serving_more import FAR, Branches, check_attention_sink

pytestmark = pytest.mark.gpu


def token(n):
    return [(1, k) for k in n]


CASES = {
    "few": ("bf16", HND, 40, 8, 128, 16, [(1520, token([3, 1, 40, 17]))], (), ()),
    "one sequence": ("bf16", HND, 8, 8, 128, 16, [(100, token([1]))], (), ()),
    "tiles": ("bf16", NHD, 40, 8, 128, 32, [(3000, token(range(1, 33)))], (), ()),
    "two row tiles": ("bf16", HND, 16, 1, 64, 16, [(2500, token([9] * 40))], (), ()),
    "no group around": ("bf16", HND, 8, 2, 64, 16, [(300, token([5, 6])), (0, token([7, 1])), (64, [(1, 64)])],
                        [(1, 500), (3, 9)], [(2, 77)]),
    "empty": ("bf16", NHD, 4, 4, 64, 24, [(130, [(0, 4), (0, 0)]), (50, [(0, 3), (2, 2), (0, 9)]), (700, [(1, 1)])],
              (), [(0, 5)]),
    "partial pages": ("bf16", HND, 10, 2, 80, 24, [(131, token([1, 30, 2])), (25, token([24, 23]))], (), ()),
    "drafts": ("bf16", NHD, 32, 8, 128, 32, [(1000, [(5, 6), (1, 100), (3, 3), (4, 70)]), (77, [(2, 9)]),
                                             (513, [(3, 40), (5, 300)])], (), ()),
    "many groups": ("bf16", HND, 4, 2, 64, 16, [(16 * (i % 7), token([1 + i % 5] * (1 + i % 3))) for i in range(70)], (),
                    ()),
    "one long, many short": ("bf16", HND, 8, 8, 64, 16, [(9000, token([2, 3]))] + [(20, token([3]))] * 20, (), ()),
    "long rests": ("bf16", HND, 5, 1, 128, 16, [(200, token([3000, 2, 900, 64]))], (), ()),
    "many items": ("bf16", HND, 40, 40, 64, 16, [(400, token([5] * 20))], (), ()),
    "one head": ("bf16", HND, 4, 1, 128, 16, [(12000, token([30, 20, 10]))], (), ()),
    "rows of 64": ("bf16", NHD, 64, 1, 96, 100, [(650, token([129, 1]))], (), ()),
    "sequences of many rows": ("bf16", HND, 8, 2, 64, 16, [(300, [(40, 50), (17, 17)])], (), [(2, 30)]),
    "odd pages": ("bf16", HND, 8, 8, 32, 5, [(83, token([7, 1, 12])), (11, [(8, 8)])], (), ()),
    "large pages": ("bf16", HND, 20, 1, 64, 240, [(1000, token([7, 1, 12, 500]))], (), ()),
    "f32": ("f32", HND, 8, 8, 64, 16, [(1000, token([1, 50, 3])), (333, token([9] * 5))], (), ()),
    "f32 rows": ("f32", NHD, 20, 2, 128, 24, [(500, token([1, 50, 3, 20, 9, 8, 7, 6, 5, 4, 3, 2, 1, 90]))], (), ()),
    "f32 odd": ("f32", HND, 5, 1, 36, 7, [(60, [(9, 12), (4, 4)]), (3, [(1, 1)])], [(2, 2)], ()),
    "f32 drafts": ("f32", NHD, 14, 2, 80, 16, [(400, [(6, 60), (7, 7)])], (), [(1, 40)]),
    "f32 many rows": ("f32", NHD, 8, 2, 32, 16, [(300, [(40, 60), (3, 7)])], (), ()),
}


# Small prefixes are shared only where the bounds say that they may be long: the tests run with such bounds, and with bounds
# of what lies behind the prefixes that make an item one CTA's (0), a few CTAs' or an even share's (50000).
RESTS = [None, 0, 600, 50000]


def bounds(c, rest):
    return {} if rest is None else c.far(rest)


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "open"])
@pytest.mark.parametrize("rest", RESTS)
def test_shared(gpu, name, causal, rest):
    dtype, layout, hq, h, d, bs, groups, before, after = CASES[name]
    c = Branches(dtype, layout, h, d, bs, groups, before, after, seed=len(name)).fill()
    q = c.normal(c.start[-1], hq, d)
    out, lse = c.attend(q, causal, **bounds(c, rest))
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention_sink(c, q, out, lse, d ** -0.5, causal, -1, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,window,sink", [(1, 100, 0), (1, 100, 30), (30, 5, 2), (100, 300, 70)])
def test_windows(gpu, dtype, nq, window, sink):
    c = Branches(dtype, HND, 2, 64, 16, [(300, [(nq, nq + 40), (nq, nq)])], (), [(nq, 150)]).fill()
    q = c.normal(c.start[-1], 4, 64)
    out, lse = c.attend(q, True, window, sink)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention_sink(c, q, out, lse, 0.125, True, window, sink)


@pytest.mark.parametrize("rest", RESTS)
@pytest.mark.parametrize("dtype,hq", [("bf16", 4), ("bf16", 40), ("f32", 4), ("f32", 40)])
def test_extremes(gpu, rest, dtype, hq):
    """Scores that rise from the prefix to the rest or fall off, by far; an infinity that every row sees; nothing but
    unwritten rows behind the sequences."""
    c = Branches(dtype, NHD, 1, 64, 16, [(500, token([60, 1, 33])), (40, token([300, 2]))], seed=hq)
    for s in range(5):
        grow = 60.0 if s % 2 else 1 / 60.0
        c.keys[s][c.prefix[s // 3]:] = (c.keys[s][c.prefix[s // 3]:].float() * grow).to(c.dt)
    c.fill()
    q = c.normal(5, hq, 64)
    for scale in (0.125, 30.0, -3.0):
        out, lse = c.attend(q, scale=scale, **bounds(c, rest))
        check_attention_sink(c, q, out, lse, scale, True, -1, 0)
    c.values[0][7, 0, 3] = c.values[1][7, 0, 3] = c.values[2][7, 0, 3] = math.inf
    c.fill()
    out, lse = c.attend(q, **bounds(c, rest))
    assert (out[:3, :, 3] == math.inf).all() and torch.isfinite(out[3:]).all()
    out[:3, :, 3] = 0
    for s in range(3):
        c.values[s][:, 0, 3] = 0
    check_attention_sink(c, q, out, lse, 0.125, True, -1, 0)


@pytest.mark.parametrize("rest", RESTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_by_head(gpu, rest, dtype):
    c = Branches(dtype, HND, 4, 64, 16, [(130, token([300, 200, 40]))], (), [(1, 20)], seed=6).fill()
    lens = [[430, 131, 400, 200], [131, 132, 300, 330], [170, 160, 150, 140], [20, 1, 5, 0]]
    c.kv_len = ints(lens)
    q = c.normal(4, 8, 64)
    out, lse = c.attend(q, False, **bounds(c, rest))
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention_sink(c, q, out, lse, 0.125, False, -1, 0, kv_of=lens)


@pytest.mark.parametrize("dtype,hq,nq", [("bf16", 2, 1), ("bf16", 60, 1), ("bf16", 2, 60), ("f32", 2, 1), ("f32", 2, 100)])
@pytest.mark.parametrize("what", ["start", "start order", "prefix", "negative prefix", "prefix past the table",
                                  "prefix among the new tokens", "rows", "entry", "length", "q_start"])
@pytest.mark.parametrize("rest", [None, 0, 50000])
def test_bad_state_is_reported(gpu, rest, dtype, hq, nq, what):
    c = Branches(dtype, NHD, 1, 64, 8, [(100, [(nq, nq + 9), (nq, nq)]), (60, [(nq, nq + 3), (nq, nq + 8)])]).fill()
    q = c.normal(4 * nq, hq, 64)
    over = {}
    if what == "start":
        c.start_dev[2] = 5
    elif what == "start order":
        c.start_dev[0], c.start_dev[1] = 0, -3
    elif what == "prefix":
        c.prefix_dev[0] = 101 + 9
    elif what == "negative prefix":
        c.prefix_dev[0] = -1
    elif what == "prefix past the table":
        c.prefix_dev[0] = 1 << 20
    elif what == "prefix among the new tokens":
        c.prefix_dev[0] = 101
    elif what == "rows":
        over = dict(max_q=2 * nq - 1)
    elif what == "entry":
        c.tables[:2, 3] = -1
    elif what == "length":
        c.kv_len[1] = 1 << 28
    else:
        c.q_start[1] = -4
    if rest is not None:
        over["max_prefix"] = FAR
    out, lse = c.attend(q, groups=c.groups(**over), batch=c.batch() if rest is None else c.batch(max_kv=FAR + rest))
    assert dcp.dcp_get_status(c.status) == dcp.DCP_EDEVICE
    if what not in ("start", "start order", "rows"):  # the sound group has its result
        r = slice(2 * nq, None)
        c.keys, c.values, c.kv_lens, c.q_lens, c.start = c.keys[2:], c.values[2:], c.kv_lens[2:], [nq, nq], [0, nq, 2 * nq]
        check_attention_sink(c, q[r], out[r], lse[r], 0.125, True, -1, 0)


@pytest.mark.parametrize("rest", RESTS)
def test_rows_behind_the_last_sequence_are_left(gpu, rest):
    for dtype, hq in (("bf16", 4), ("bf16", 60), ("f32", 4)):
        c = Branches(dtype, HND, 1, 64, 16, [(100, token([5, 9, 1])), (40, token([300, 2]))], seed=hq).fill()
        q = c.normal(9, hq, 64)
        far = dict(total_q=9, **({} if rest is None else dict(max_kv=FAR + rest)))
        groups = c.groups() if rest is None else c.groups(max_prefix=FAR)
        out, lse = c.attend(q, batch=c.batch(**far), groups=groups)
        assert torch.isnan(out[5:]).all() and torch.isnan(lse[5:]).all()
        check_attention_sink(c, q[:5], out[:5], lse[:5], 0.125, True, -1, 0)


@pytest.mark.parametrize("rest", RESTS)
def test_same_as_alone(gpu, rest):
    """Branches read through their group's prefix give what they give one by one, up to the order of sums."""
    c = Branches("bf16", HND, 8, 128, 16, [(2000, token(range(1, 20)))]).fill()
    q = c.normal(19, 40, 128)
    out, lse = c.attend(q, **bounds(c, rest))
    ws = dcp.new_workspace(dcp.dcp_attention_workspace_size(c.pool(), c.batch(), dcp.AttnConfig(), 40))
    alone, lse_alone = torch.empty_like(out), torch.empty_like(lse)
    dcp.dcp_paged_attention(c.pool(), c.batch(), dcp.AttnConfig(), q, alone, lse_alone, ws)
    assert (lse - lse_alone).abs().max() <= 2.0 ** -16 and (out.float() - alone.float()).abs().max() <= 2.0 ** -8


@pytest.mark.parametrize("rest", RESTS)
def test_in_a_graph_with_other_lengths(gpu, rest):
    """Recorded once, replayed with other prefixes and lengths; the result does not depend on the run."""
    c = Branches("bf16", HND, 2, 64, 16, [(640, token([40, 50, 33])), (320, token([300, 20]))]).fill()
    q = c.normal(5, 20, 64)
    far = bounds(c, rest)
    cfg, pool, batch, groups = dcp.AttnConfig(), c.pool(), far.get("batch", c.batch()), far.get("groups", c.groups())
    ws = dcp.new_workspace(dcp.dcp_shared_attention_workspace_size(pool, batch, groups, cfg, 20))
    out, lse = torch.empty_like(q), torch.empty(5, 20, device="cuda")
    dcp.dcp_shared_attention(pool, batch, groups, cfg, q, out, lse, ws)
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dcp.dcp_shared_attention(pool, batch, groups, cfg, q, out, lse, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, first)
    c.prefix_dev.copy_(ints([0, 48]))
    g.replay()
    check_attention_sink(c, q, out, lse, 0.125, True, -1, 0)
    lens = [400, 301, 288, 60, 50]
    c.prefix_dev.copy_(ints([256, 48]))
    c.kv_len.copy_(ints(lens))
    c.kv_lens, c.keys, c.values = lens, [x[:n] for x, n in zip(c.keys, lens)], [x[:n] for x, n in zip(c.values, lens)]
    g.replay()
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention_sink(c, q, out, lse, 0.125, True, -1, 0)


def test_two_streams_and_a_workspace_that_others_use(gpu):
    a = Branches("bf16", HND, 8, 128, 16, [(3000, token(range(1, 30)))]).fill()
    b = Branches("f32", NHD, 4, 64, 16, [(900, token(range(1, 30)))]).fill()
    qa, qb = a.normal(29, 40, 128), b.normal(29, 4, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for rest in (None, 0, 50000):
        with torch.cuda.stream(s):
            outs.append((a, qa, *a.attend(qa, **bounds(a, rest))))
        outs.append((b, qb, *b.attend(qb, **bounds(b, rest))))
    s.synchronize()
    for c, q, out, lse in outs:
        check_attention_sink(c, q, out, lse, c.d ** -0.5, True, -1, 0)
    # one workspace, in turns with plain attention, a fork and a call of another size
    cfg, size = dcp.AttnConfig(), 0
    pages = dcp.PagePool(a.k[None], a.v[None], 16, a.status)
    for c, hq in ((a, 40), (b, 4)):
        size = max(size, dcp.dcp_shared_attention_workspace_size(c.pool(), *c.far().values(), cfg, hq),
                   dcp.dcp_attention_workspace_size(c.pool(), c.batch(), cfg, hq))
    size = max(size, dcp.dcp_pages_workspace_size(pages, 2, a.tables.shape[1]))
    ws = dcp.new_workspace(size)
    ref = torch.ones(a.k.shape[0], dtype=torch.int32, device="cuda")
    for _ in range(2):
        for c, q in ((a, qa), (b, qb)):
            out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
            dcp.dcp_shared_attention(c.pool(), *c.far().values(), cfg, q, out, lse, ws)
            check_attention_sink(c, q, out, lse, c.d ** -0.5, True, -1, 0)
            dcp.dcp_paged_attention(c.pool(), c.batch(), cfg, q, out, lse, ws)
            check_attention_sink(c, q, out, lse, c.d ** -0.5, True, -1, 0)
            child, tables = torch.empty_like(a.tables[:1]), a.tables[:1].contiguous()
            dcp.dcp_pages_fork(pages, tables, ints([16]), ints([0]), None, None, ref, child, ref, ws)
    assert dcp.dcp_get_status(a.status) == dcp.DCP_OK == dcp.dcp_get_status(b.status)


@pytest.mark.parametrize("rest", [None, 0, 50000])
def test_long_pool(gpu, rest):
    """Element offsets past 2^31 in the pool, strided q, no lse."""
    bs, nb = 64, (1 << 31) // (64 * 128) + 700
    c = Branches("bf16", HND, 1, 128, bs, [(12800, token([100, 70, 20, 9]))], seed=9)
    k = torch.zeros((nb, 1, bs, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c.tables = torch.where(c.tables >= 0, c.tables + (nb - c.k.shape[0]), -1)
    c.table, c.k, c.v = c.tables.cpu().numpy(), k, v
    c.fill()
    q = c.normal(4, 24, 128)[:, 4:22]
    far = bounds(c, rest)
    cfg, pool, batch, groups = dcp.AttnConfig(), c.pool(), far.get("batch", c.batch()), far.get("groups", c.groups())
    ws = dcp.new_workspace(dcp.dcp_shared_attention_workspace_size(pool, batch, groups, cfg, 18))
    out = torch.empty(4, 18, 128, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_shared_attention(pool, batch, groups, cfg, q, out, None, ws)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention_sink(c, q, out, None, 128 ** -0.5, True, -1, 0)
