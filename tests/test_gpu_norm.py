"""dcp_norm_rope_append on the GPU against its 64-bit statement (tests/serving_more.py)."""
import math

import numpy as np
import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests.serving import HND, NHD, Cache, ints
from tests.serving_more import check_norm_turned, normed_64

pytestmark = pytest.mark.gpu
HEAD, TOKEN = dcp.DCP_NORM_HEAD, dcp.DCP_NORM_TOKEN

CASES = [
    # dtype, layout, hq, h, d, bs, q_lens, kv_lens, rots, pairs, positions
    ("bf16", HND, 5, 1, 128, 16, [1], [1], [128], 1, None),
    ("bf16", NHD, 8, 8, 64, 5, [3, 1, 7], [3, 12, 40], [64], 0, None),
    ("bf16", HND, 4, 2, 80, 24, [33, 2], [33, 50], [22], 1, 1000000),
    ("bf16", NHD, 2, 1, 40, 8, [9], [30], [14], 0, -70000),
    ("bf16", HND, 40, 40, 128, 32, [13], [100], [44, 42, 42], 0, 240),
    ("bf16", HND, 12, 4, 96, 32, [21, 5], [100, 5], [16, 24, 40], 1, 1000),
    ("bf16", NHD, 3, 3, 72, 32, [4], [10], [2, 30], 1, -500),
    ("f32", NHD, 4, 4, 32, 7, [5, 0, 6], [5, 3, 13], [30], 1, 2 ** 31 - 70),
    ("f32", HND, 6, 2, 96, 16, [17], [64], [64], 1, -2 ** 31 + 5),
    ("f32", HND, 5, 5, 128, 16, [17], [64], [44, 42, 42], 0, 77),
    ("f32", HND, 1, 1, 4, 1, [3], [3], [2], 0, 5),
    ("bf16", NHD, 2, 2, 24, 3, [4], [9], [0], 1, None),
    ("bf16", NHD, 200, 3, 128, 16, [2], [9], [128], 1, None),     # many heads
    ("bf16", HND, 150, 150, 64, 16, [2], [9], [64], 0, None),
    ("f32", HND, 90, 1, 128, 16, [2], [9], [120], 1, None),
    ("bf16", NHD, 300, 3, 128, 16, [2, 3], [9, 3], [128], 1, None),  # and tokens that go through shared memory in pieces
    ("bf16", HND, 70, 280, 72, 16, [3], [9], [44], 0, 12),
    ("f32", HND, 100, 40, 128, 16, [2], [9], [128], 1, None),
    ("f32", NHD, 3, 130, 100, 16, [2], [9], [70], 1, None),
]


def weights_of(kind, c, hq, g):
    if kind == "none":
        return None, None
    dt = torch.float32 if kind.endswith("f32") else torch.bfloat16
    shapes = [(c.d,)] * 2 if kind.startswith("one") else [(hq, c.d), (c.h, c.d)]
    return [(1 + 0.3 * torch.randn(*s, generator=g)).to(dt).cuda() for s in shapes]


def new_rows(c, i):
    nq, nk = c.q_lens[i], c.kv_lens[i]
    block, row = c.rows(i, nk - nq, nk)
    return (block, slice(None), row) if c.layout == HND else (block, row)


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("span", [HEAD, TOKEN], ids=["head", "token"])
@pytest.mark.parametrize("weights", ["none", "one bf16", "heads f32", "one f32", "heads bf16"])
def test_norm_append(gpu, case, span, weights):
    dtype, layout, hq, h, d, bs, q_lens, kv_lens, rots, pairs, far = case
    c = Cache(dtype, layout, h, d, bs, q_lens, kv_lens, seed=rots[0] + hq).fill()
    n = c.start[-1]
    q, k, v = (3 * c.normal(n, hq + 2 * h, d)).split([hq, h, h], dim=1)
    qw, kw = weights_of(weights, c, hq, c.g)
    cfgs = [dcp.RopeConfig(r, pairs, base=10000.0 if i else 500000.0, amplitude=1.0 + 0.25 * i)
            for i, r in enumerate(rots)]
    place = np.concatenate([np.arange(nk - nq, nk) for nq, nk in zip(q_lens, kv_lens)])
    pos = np.stack([place if far is None else far + (np.arange(n) * (i + 1)) % 60 for i in range(len(rots))])
    out = torch.full((n, hq, d), math.nan, dtype=c.dt, device="cuda")
    k0, v0 = c.k.clone(), c.v.clone()
    norm = dcp.NormConfig(qw, kw, eps=1e-5, span=span)
    dcp.dcp_norm_rope_append(c.pool(), c.batch(), dcp.dcp_rope_axes(cfgs), norm, q, k, v,
                             None if far is None else ints(pos), out)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_norm_turned(out, q, qw, 1e-5, span, pos, cfgs)
    # only the new tokens' rows changed: keys turned, values as they are
    for i in range(len(q_lens)):
        r, at = slice(c.start[i], c.start[i + 1]), new_rows(c, i)
        check_norm_turned(c.k[at], k[r], kw, 1e-5, span, pos[:, r], cfgs)
        assert torch.equal(c.v[at], v[r])
        k0[at], v0[at] = c.k[at], c.v[at]
    for a, b in ((c.k, k0), (c.v, v0)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("span", [HEAD, TOKEN], ids=["head", "token"])
@pytest.mark.parametrize("rot", [0, 64, 20])
def test_sizes_of_values(gpu, dtype, span, rot):
    """Values whose squares leave fp32, beside ordinary ones."""
    c = Cache(dtype, HND, 2, 64, 8, [8], [8], seed=rot)
    scale = 2.0 ** torch.tensor([0, 70, 124, -60, -120, 63, -45, 10], dtype=torch.float64)[:, None, None].cuda()
    q, k, v = ((c.normal(8, n, 64).double() * scale).to(c.dt) for n in (6, 2, 2))
    for eps in (0.0, 1e-12, 1.0):
        cfg = dcp.RopeConfig(rot, dcp.DCP_ROPE_HALF)
        out = torch.empty_like(q)
        dcp.dcp_norm_rope_append(c.pool(), c.batch(), dcp.dcp_rope_axes([cfg]), dcp.NormConfig(eps=eps, span=span), q, k,
                                 v, None, out)
        pos = np.arange(8)[None]
        check_norm_turned(out, q, None, np.float32(eps).item(), span, pos, [cfg])
        check_norm_turned(c.k[c.rows(0, 0, 8)[0], :, c.rows(0, 0, 8)[1]], k, None, np.float32(eps).item(), span, pos,
                          [cfg])


@pytest.mark.parametrize("span", [HEAD, TOKEN], ids=["head", "token"])
def test_zeros_infinities_and_nan_stay_where_they_are(gpu, span):
    c = Cache("bf16", NHD, 2, 64, 8, [6], [6])
    q, k, v = c.normal(6, 4, 64), c.normal(6, 2, 64), c.normal(6, 2, 64)
    q[1] = 0
    q[2, 1, 5], q[3, 2, 7] = math.inf, math.nan
    k[4, 1, 0] = -math.inf
    out = torch.empty_like(q)
    axes = dcp.dcp_rope_axes([dcp.RopeConfig(0)])
    dcp.dcp_norm_rope_append(c.pool(), c.batch(), axes, dcp.NormConfig(eps=1e-6, span=span), q, k, v, None, out)
    for got, x in ((out, q), (c.k[c.rows(0, 0, 6)], k)):
        want = normed_64(x, None, np.float32(1e-6).item(), span)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert ((got.double() - want).abs()[fine] <= 2.0 ** -8 * 1.001 * want.abs()[fine]).all()


def test_in_place_keys_only_and_rows_without_a_place(gpu):
    c = Cache("bf16", HND, 2, 64, 8, [6, 3], [4, 9], seed=3)  # the first two tokens of sequence 0 have no position
    n = c.start[-1] + 2                                        # and the last two rows belong to no sequence
    q, k, v = c.normal(n, 4, 64), c.normal(n, 2, 64), c.normal(n, 2, 64)
    q0, cfg = q.clone(), dcp.RopeConfig(64, dcp.DCP_ROPE_HALF)
    axes, norm, b = dcp.dcp_rope_axes([cfg]), dcp.NormConfig(eps=1e-6, span=TOKEN), c.batch(total_q=n)
    dcp.dcp_norm_rope_append(c.pool(), b, axes, norm, q, k, v, None, q)
    pos = np.concatenate([np.arange(-2, 4), np.arange(6, 9)])[None]
    check_norm_turned(q[:9], q0[:9], None, 1e-6, TOKEN, pos, [cfg])
    assert torch.equal(q[9:], q0[9:])
    k1 = c.k.clone()
    c.k.fill_(math.nan)
    dcp.dcp_norm_rope_append(c.pool(), b, axes, norm, None, k, v, None, None)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    assert torch.equal(c.k.view(torch.int16), k1.view(torch.int16))


@pytest.mark.parametrize("what", ["entry", "negative entry", "length", "q_start", "long"])
def test_bad_state_is_reported_and_written_nowhere(gpu, what):
    c = Cache("bf16", NHD, 2, 64, 8, [3, 4], [20, 30], seed=4)
    q, k, v = c.normal(7, 2, 64), c.normal(7, 2, 64), c.normal(7, 2, 64)
    out, over = torch.zeros_like(q), {}
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
    dcp.dcp_norm_rope_append(c.pool(), c.batch(**over), dcp.dcp_rope_axes([dcp.RopeConfig(64)]), dcp.NormConfig(), q, k,
                             v, None, out)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_EDEVICE
    block, row = c.rows(1, 0, 30)
    k0[block, row] = c.k[block, row]  # the sound sequence's own rows
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16))


def test_without_norms_turn_as_the_plain_append(gpu):
    """Rows of size 1 a head, eps 0: what is appended is what dcp_rope_append appends, up to the norm's roundings."""
    a, b = (Cache("f32", HND, 2, 64, 8, [5], [11], seed=9) for _ in range(2))
    q, k, v = a.normal(5, 4, 64), a.normal(5, 2, 64), a.normal(5, 2, 64)
    q, k = (x / x.square().mean(-1, keepdim=True).sqrt() for x in (q, k))
    cfg = dcp.RopeConfig(64, dcp.DCP_ROPE_HALF, scaling=dcp.DCP_ROPE_PARTS, factor=8.0, amplitude=1.2)
    one, two = torch.empty_like(q), torch.empty_like(q)
    dcp.dcp_rope_append(a.pool(), a.batch(), dcp.dcp_rope_plan(cfg), q, k, v, None, one)
    dcp.dcp_norm_rope_append(b.pool(), b.batch(), dcp.dcp_rope_axes([cfg]), dcp.NormConfig(eps=0.0), q, k, v, None, two)
    assert (one - two).abs().max() <= 2.0 ** -20 * one.abs().max()
    at = new_rows(a, 0)
    assert (a.k[at] - b.k[at]).abs().max() <= 2.0 ** -20 * one.abs().max() and torch.equal(a.v[at], b.v[at])


@pytest.mark.parametrize("dtype,hq", [("bf16", 300), ("f32", 6)])
def test_values_past_the_squares_in_pieces_and_blocks(gpu, dtype, hq):
    """Tokens whose sums are taken again beside tokens whose sums are not, several in a CTA and one in pieces."""
    n = 700
    c = Cache(dtype, NHD, 2, 64 if hq < 10 else 128, 16, [n], [n], seed=hq)
    scale = 2.0 ** torch.randint(-1, 2, (n, 1, 1), generator=c.g).double().mul(70).cuda()
    q, k, v = ((c.normal(n, h, c.d).double() * scale).to(c.dt) for h in (hq, 2, 2))
    cfg, out = dcp.RopeConfig(64, dcp.DCP_ROPE_HALF), torch.empty_like(q)
    dcp.dcp_norm_rope_append(c.pool(), c.batch(), dcp.dcp_rope_axes([cfg]), dcp.NormConfig(eps=0.0, span=TOKEN), q, k, v,
                             None, out)
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_norm_turned(out, q, None, 0.0, TOKEN, np.arange(n)[None], [cfg])
    check_norm_turned(c.k[c.rows(0, 0, n)], k, None, 0.0, TOKEN, np.arange(n)[None], [cfg])


@pytest.mark.parametrize("span", [HEAD, TOKEN], ids=["head", "token"])
@pytest.mark.parametrize("shape", [(64,), (2, 64)], ids=["one", "heads"])
def test_weights_of_one_kind_only(gpu, span, shape):
    for which in range(2):
        c = Cache("bf16", HND, 2, 64, 8, [9], [20], seed=which)
        q, k, v = c.normal(9, 2, 64), c.normal(9, 2, 64), c.normal(9, 2, 64)
        w, cfg, out = (1 + 0.3 * torch.randn(*shape, generator=c.g)).cuda(), dcp.RopeConfig(44), torch.empty_like(q)
        weights = (w, None) if which == 0 else (None, w)
        dcp.dcp_norm_rope_append(c.pool(), c.batch(), dcp.dcp_rope_axes([cfg]), dcp.NormConfig(*weights, span=span), q, k, v,
                                 None, out)
        pos = np.arange(11, 20)[None]
        check_norm_turned(out, q, weights[0], 1e-6, span, pos, [cfg])
        check_norm_turned(c.k[new_rows(c, 0)], k, weights[1], 1e-6, span, pos, [cfg])


def test_in_a_graph_and_on_another_stream(gpu):
    c = Cache("bf16", NHD, 2, 64, 8, [3, 4], [20, 30], seed=4)
    q, k, v = c.normal(7, 4, 64), c.normal(7, 2, 64), c.normal(7, 2, 64)
    out = torch.empty_like(q)
    cfg = dcp.RopeConfig(64)
    args = (c.pool(), c.batch(), dcp.dcp_rope_axes([cfg]), dcp.NormConfig(), q, k, v, None, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dcp.dcp_norm_rope_append(*args, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dcp.dcp_norm_rope_append(*args)
    q.normal_()
    c.kv_len.copy_(ints([10, 9]))
    g.replay()
    check_norm_turned(out, q, None, 1e-6, HEAD, [np.concatenate([np.arange(7, 10), np.arange(5, 9)])], [cfg])
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
