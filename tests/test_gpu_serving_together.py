"""The serving operators of a decoding step together: branches of sessions (dcp_pages_fork) append their normalised and
turned tokens, attend through a window with first positions in one layer and over everything, their prefix shared, in
another; the step is recorded once and replayed as the sequences grow."""
import math

import numpy as np
import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests.serving import HND, NHD, attention_bounds, ints
from tests.serving_more import FAR, attention_sink_64, check_norm_turned

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [HND, NHD])
def test_decoding_steps_of_branches(gpu, dtype, layout):
    H, HQ, D, BS, N, STEPS = 2, 8, 64, 16, 6, 5
    parents, stride, blocks = [75, 130], 16, 120
    g = torch.Generator(device="cuda").manual_seed(3)
    shape = (2, blocks, H, BS, D) if layout == HND else (2, blocks, BS, H, D)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2))
    status = ints([0])
    pages = dcp.PagePool(k, v, BS, status)
    # two sessions, branched in four and two: full pages shared, the last one copied, room for the new tokens
    table = torch.full((2, stride), -1, dtype=torch.int32, device="cuda")
    table[0, :5], table[1, :9] = ints([7, 3, 90, 41, 8]), ints([1, 2, 60, 61, 5, 100, 33, 34, 9])
    ref = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    ref[table[table >= 0].long()] = 1
    of = [0, 0, 0, 0, 1, 1]
    tables = torch.empty(N, stride, dtype=torch.int32, device="cuda")
    ws = dcp.new_workspace(1 << 24)
    reserve = ints([parents[p] + STEPS + 1 for p in of])
    dcp.dcp_pages_fork(pages, table, ints(parents), ints(of), None, reserve, ref, tables, ref, ws)

    kv_len = ints([parents[p] for p in of])
    pools = [dcp.KVPool(k[i], v[i], layout) for i in range(2)]
    batch = dcp.SeqBatch(ints(list(range(N + 1))), tables, kv_len, status, N, 1, FAR + 200)
    groups = dcp.PrefixGroups(ints([0, 4, 6]), ints([n // BS * BS for n in parents]), FAR, 4)
    cfgs = [dcp.RopeConfig(24, dcp.DCP_ROPE_HALF), dcp.RopeConfig(20, dcp.DCP_ROPE_HALF), dcp.RopeConfig(20, dcp.DCP_ROPE_HALF)]
    axes = dcp.dcp_rope_axes(cfgs)
    qw, kw = (1 + 0.2 * torch.randn(n, D, generator=g, device="cuda") for n in (HQ, H))
    norm = dcp.NormConfig(qw, kw, span=dcp.DCP_NORM_TOKEN)
    windowed, full = dcp.AttnConfig(window=20, sink=5), dcp.AttnConfig()
    qkv = torch.empty(2, N, HQ + 2 * H, D, dtype=dtype, device="cuda")
    positions = torch.empty(3, N, dtype=torch.int32, device="cuda")
    turned, out = torch.empty(2, N, HQ, D, dtype=dtype, device="cuda"), torch.empty(2, N, HQ, D, dtype=dtype, device="cuda")
    lse = torch.empty(2, N, HQ, device="cuda")

    def step():
        kv_len.add_(1)
        for layer in range(2):
            q, new_k, new_v = qkv[layer].split([HQ, H, H], dim=1)
            dcp.dcp_norm_rope_append(pools[layer], batch, axes, norm, q, new_k, new_v, positions, turned[layer])
        dcp.dcp_paged_attention(pools[0], batch, windowed, turned[0], out[0], lse[0], ws)
        dcp.dcp_shared_attention(pools[1], batch, groups, full, turned[1], out[1], lse[1], ws)

    def fill():
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        positions.copy_(torch.randint(0, 500, positions.shape, generator=g, device="cuda"))

    def check():
        assert dcp.dcp_get_status(status) == dcp.DCP_OK
        half = positions.cpu().numpy()
        for layer in range(2):
            q, new_k, new_v = qkv[layer].split([HQ, H, H], dim=1)
            check_norm_turned(turned[layer], q, qw, 1e-6, dcp.DCP_NORM_TOKEN, half, cfgs)
            for s in range(N):
                n = int(kv_len[s])
                j = torch.arange(n, device="cuda")
                block, row = tables[s].long()[j // BS], j % BS
                keys, values = ((p[layer][block, :, row] if layout == HND else p[layer][block, row]) for p in (k, v))
                check_norm_turned(keys[-1:], new_k[s:s + 1], kw, 1e-6, dcp.DCP_NORM_TOKEN, half[:, s:s + 1], cfgs)
                assert torch.equal(values[-1], new_v[s])
                for h in range(HQ):
                    o, l, mass, terms = attention_sink_64(turned[layer, s:s + 1, h], keys[:, h // 4], values[:, h // 4], n - 1,
                                                          D ** -0.5, True, 20 if layer == 0 else -1, 5 if layer == 0 else 0)
                    tol, tol_l = attention_bounds(dtype, D, n, o, mass, l, terms)
                    assert ((out[layer, s, h].double() - o).abs() <= tol).all()
                    assert abs(lse[layer, s, h].double() - l) <= tol_l

    fill()
    step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(STEPS - 1):
        fill()
        graph.replay()
        check()
