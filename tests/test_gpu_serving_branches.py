"""Pages that are held in common, or that nobody holds: what pruning and packing do about them."""
import copy

import numpy as np
import pytest
import torch

import autoregressive_video_diffusion_gb300 as dcp
import oracle
from oracle import replay
from synth.workloads import TINY, scaled
from tests import devcache
from tests.paged import PagedCopy
from tests.serving import HND, NHD, ints
from tests.test_gpu_parity import _cuda, assert_cache_parity
from tests.test_gpu_serving import Pages, dev, same

pytestmark = pytest.mark.gpu

BS = 16
TURNING = scaled(TINY, R=2, S=4)  # offsets past the span: every step turns the history's keys in place


class Family:
    """A paged cache before its last eviction and two branches of it, made by dcp_pages_fork."""

    def __init__(self, w, layout, shared):
        self.w, self.cfg = w, devcache.dcp_config(w)
        self.hc, self.ev = replay.state_before_last(w)
        self.dev = devcache.to_device(self.hc, w)
        self.n_sink, self.n_hist = w.sink_rows // BS, w.hist_cap // BS
        n_win = (w.window_chunks + 1) * w.C // BS
        pc = PagedCopy(self.dev, self.cfg, BS, layout, 3, spare=2 * (self.n_sink + self.n_hist + n_win) + 3)
        self.layout, cache = layout, pc.cache
        row = torch.cat([pc.sink_blocks, cache.hist_blocks, cache.window_blocks])
        self.ref = torch.zeros(cache.n_blocks, dtype=torch.int32, device="cuda")
        self.ref[row.long()] = 1
        pool, n = dcp.PagePool.of(cache), row.numel()
        children = torch.empty(2, n, dtype=torch.int32, device="cuda")
        ws = dcp.new_workspace(dcp.dcp_pages_workspace_size(pool, 2, n))
        dcp.dcp_pages_fork(pool, row[None].contiguous(), ints([n * BS]), ints([0, 0]),
                           None if shared is None else ints([shared] * 2), None, self.ref, children, self.ref, ws)
        assert dcp.dcp_get_status(cache.status) == dcp.DCP_OK
        cache.block_ref = self.ref
        self.members = [self.member(cache, r) for r in (row, children[0], children[1])]

    def member(self, cache, row):
        m = copy.copy(cache)
        m.hist_len, m.hist_t = cache.hist_len.clone(), cache.hist_t.clone()
        m.status = torch.zeros_like(cache.status)
        m.sink_blocks = row[:self.n_sink]
        m.hist_blocks = row[self.n_sink:self.n_sink + self.n_hist].contiguous()
        m.window_blocks = row[self.n_sink + self.n_hist:].contiguous()
        return m

    def step(self, m):
        c, q0_prev, q0 = self.ev
        x0, xr = self.w.score_inputs(c)
        ws = dcp.new_workspace(dcp.dcp_paged_workspace_size(m, self.cfg))
        dcp.dcp_paged_prune_step(m, self.cfg, _cuda(x0), _cuda(xr), self.w.slot_of(c), self.w.first_frame(c), q0_prev,
                                 q0, None, None, None, ws)
        return dcp.dcp_get_status(m.status)

    def check(self, m):
        """The member's state is what the oracle's step makes of the common state."""
        o, (c, q0_prev, q0) = self.hc.copy(), self.ev
        x0, xr = self.w.score_inputs(c)
        rc, _, _, _ = oracle.prune_step(o, replay.cfg_of(self.w), x0, xr, self.w.slot_of(c), self.w.first_frame(c),
                                        q0_prev, q0, None)
        assert rc == oracle.OK
        block, off = dcp.paged_row_map(self.cfg, m.hist_cap, BS, m.sink_blocks, m.hist_blocks, m.window_blocks)
        self.dev.k.copy_(dcp.paged_unpack(m.k_pool, block, off, self.layout))
        self.dev.v.copy_(dcp.paged_unpack(m.v_pool, block, off, self.layout))
        self.dev.hist_len.copy_(m.hist_len)
        self.dev.hist_t.copy_(m.hist_t)
        assert_cache_parity(devcache.from_device(self.dev, self.w), o, self.w)

    def all_go_on(self):
        assert [self.step(m) for m in self.members] == [dcp.DCP_OK] * 3
        for m in self.members:
            self.check(m)

    def all_refused(self):
        m = self.members[0]
        k0, v0 = m.k_pool.clone(), m.v_pool.clone()
        for m in self.members:
            len0, t0 = m.hist_len.clone(), m.hist_t.clone()
            assert self.step(m) == dcp.DCP_EDEVICE
            assert torch.equal(m.hist_len, len0) and torch.equal(m.hist_t, t0)
            assert same(m.k_pool, k0) and same(m.v_pool, v0)


@pytest.mark.parametrize("layout", [HND, NHD], ids=["hnd", "nhd"])
def test_branches_share_the_sink_where_the_history_turns(gpu, layout):
    Family(TURNING, layout, TURNING.sink_rows // BS).all_go_on()


@pytest.mark.parametrize("more", [None, 1, 3])
def test_a_step_that_would_turn_shared_history_is_refused(gpu, more):
    """The default (every full page) and any page of the history in use."""
    Family(TURNING, HND, None if more is None else TURNING.sink_rows // BS + more).all_refused()


def test_branches_share_full_history_where_no_key_turns(gpu):
    hc, _ = replay.state_before_last(TINY)
    full = (TINY.sink_rows + int(hc.hist_len[0])) // BS
    assert full > TINY.sink_rows // BS
    Family(TINY, HND, full).all_go_on()
    Family(TINY, HND, full + 1).all_refused()  # the page that the kept rows enter
    Family(TINY, HND, None).all_refused()
    f = Family(TINY, HND, full + 1)
    f.cfg.gamma = 1e9  # no row is kept: nothing is written
    assert [f.step(m) for m in f.members] == [dcp.DCP_OK] * 3


def test_prune_step_without_counts_and_with_bad_ones(gpu):
    f = Family(TURNING, HND, TURNING.sink_rows // BS)
    m = f.members[1]
    m.block_ref = None
    assert f.step(m) == dcp.DCP_OK
    f.check(m)
    m.block_ref = f.ref[:-1]
    with pytest.raises(dcp.DcpError):
        f.step(m)
    m.block_ref = f.ref.long()
    with pytest.raises(dcp.DcpError):
        f.step(m)


@pytest.mark.parametrize("in_place", [False, True])
def test_pages_compact_entries_that_name_free_blocks(gpu, in_place):
    """Reported; such an entry is emptied where a page moves into its block, so that it cannot come to name another
    row's page, and kept where the block stays free."""
    p = Pages(2, 40, (1, 1, 8), 1, [1], 6)
    p.ref[:] = 0
    p.ref[[1, 3, 30, 31]] = 1  # the 4 live blocks: 30 and 31 move into the free 0 and 2
    t = np.array([[1, 3, 30, 31, -1, -1], [2, 35, 3, 0, 7, -1]], np.int32)
    k0, v0 = p.k.clone(), p.v.clone()
    td, rin, n = dev(t), dev(p.ref), torch.zeros(1, dtype=torch.int32, device="cuda")
    tout, rout = (td, rin) if in_place else (torch.zeros_like(td), torch.full_like(rin, 9))
    ws = dcp.new_workspace(dcp.dcp_pages_workspace_size(p.pool, 2, 6))
    dcp.dcp_pages_compact(p.pool, td, rin, tout, rout, n, ws)
    assert dcp.dcp_get_status(p.status) == dcp.DCP_EDEVICE
    assert tout.tolist() == [[1, 3, 0, 2, -1, -1], [-1, 35, 3, -1, 7, -1]]
    assert n.item() == 4 and rout.tolist() == [1] * 4 + [0] * 36
    for x, x0 in ((p.k, k0), (p.v, v0)):
        assert same(x[:, :4], x0[:, [30, 1, 31, 3]])
