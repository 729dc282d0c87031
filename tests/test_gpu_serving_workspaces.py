"""One workspace for every entry point: each call leaves it ready for the next, whichever that is."""
import numpy as np
import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
import oracle
from oracle import replay
from synth.workloads import TINY, scaled
from tests import devcache
from tests.serving import HND, Cache, check_attention, compact_plain, fork_plain
from tests.test_gpu_parity import _cuda, assert_cache_parity
from tests.test_gpu_serving import Pages, dev, moved, same

pytestmark = pytest.mark.gpu

W = scaled(TINY, R=2, S=4)  # keys turn: every part of a prune step's workspace is in use


class Calls:
    """Calls of every kind on one workspace, each checked against the oracle or the plain statements."""

    ATTEND = [("bf16", [1] * 12, [3000] * 12, 8, 4), ("bf16", [300], [5000], 4, 2), ("f32", [100], [900], 4, 2),
              ("bf16", [1], [9000], 8, 8)]

    def __init__(self):
        self.hc, self.ev = replay.state_before_last(W)
        self.x = W.score_inputs(self.ev[0])
        self.cfg = devcache.dcp_config(W)
        self.caches = [Cache(t, HND, h, 64, 16, ql, kl, seed=i).fill() for i, (t, ql, kl, _, h) in
                       enumerate(self.ATTEND)]
        p = self.pages()
        sizes = [dcp.dcp_workspace_size(devcache.to_device(self.hc, W), self.cfg),
                 dcp.dcp_pages_workspace_size(p.pool, 300, 12)]
        sizes += [dcp.dcp_attention_workspace_size(c.pool(), c.batch(), dcp.AttnConfig(), k[3])
                  for c, k in zip(self.caches, self.ATTEND)]
        self.ws = dcp.new_workspace(max(sizes))

    def pages(self):
        return Pages(2, 3000, (1, 2, 8), 2, [20, 11, 24, 7, 3], 12, seed=5)

    def score(self):
        (x0, xr), idx = self.x, torch.zeros(W.C, dtype=torch.int32, device="cuda")
        kept, status = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        dcp.dcp_score_mask(_cuda(x0), _cuda(xr), W.gamma, 0, None, None, idx, kept, status, self.ws)
        want = oracle.indices(oracle.keep(oracle.score(x0, xr)))
        assert int(kept) == len(want) and np.array_equal(idx[:len(want)].cpu().numpy(), want)

    def prune(self):
        c, q0_prev, q0 = self.ev
        d = devcache.to_device(self.hc, W)
        kept = torch.zeros(1, dtype=torch.int32, device="cuda")
        dcp.dcp_prune_step(d, self.cfg, _cuda(self.x[0]), _cuda(self.x[1]), W.slot_of(c), W.first_frame(c), q0_prev, q0,
                           None, kept, None, self.ws)
        o = self.hc.copy()
        rc, _, _, idx = oracle.prune_step(o, replay.cfg_of(W), *self.x, W.slot_of(c), W.first_frame(c), q0_prev, q0,
                                          None)
        assert rc == oracle.OK and dcp.dcp_get_status(d.status) == dcp.DCP_OK and int(kept) == len(idx)
        assert_cache_parity(devcache.from_device(d, W), o, W)

    def attend(self, i):
        c, hq = self.caches[i], self.ATTEND[i][3]
        q = c.normal(c.start[-1], hq, 64)
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")
        dcp.dcp_paged_attention(c.pool(), c.batch(), dcp.AttnConfig(), q, out, lse, self.ws)
        assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
        check_attention(c, q, out, lse, 0.125, True, -1)

    def fork(self):
        p, parent = self.pages(), np.arange(300) % 5
        child, ref, moves = fork_plain(p.tables, p.lens, parent, None, None, p.ref, p.bs)
        want = moved(p.k, moves)
        out, rin = torch.empty(300, 12, dtype=torch.int32, device="cuda"), dev(p.ref)
        dcp.dcp_pages_fork(p.pool, dev(p.tables), dev(p.lens), dev(parent), None, None, rin, out, rin, self.ws)
        assert dcp.dcp_get_status(p.status) == dcp.DCP_OK
        assert np.array_equal(out.cpu().numpy(), child) and np.array_equal(rin.cpu().numpy(), ref)
        assert same(p.k, want)

    def compact(self):
        p = self.pages()
        tables, ref, _, moves = compact_plain(p.tables, p.ref)
        want, t, rin = moved(p.k, moves), dev(p.tables), dev(p.ref)
        dcp.dcp_pages_compact(p.pool, t, rin, t, rin, None, self.ws)
        assert dcp.dcp_get_status(p.status) == dcp.DCP_OK
        assert np.array_equal(t.cpu().numpy(), tables) and np.array_equal(rin.cpu().numpy(), ref) and same(p.k, want)

    def run(self, name):
        self.attend(int(name[-1])) if name.startswith("attend") else getattr(self, name)()


NAMES = ["score", "prune", "fork", "compact"] + [f"attend {i}" for i in range(len(Calls.ATTEND))]


@pytest.mark.parametrize("before", NAMES)
def test_every_call_after_every_other(gpu, before):
    calls = Calls()
    for after in NAMES:
        calls.run(before)
        calls.run(after)
        calls.run(after)
