"""A session on the paged cache from chunk to chunk, branched in two: the serving operators as they are used together.

For every chunk: dcp_rope_append puts the new tokens' keys (turned to their frame) and values into the ring slot's
pages, dcp_paged_attention reads sink, history and window through one table, and dcp_paged_prune_step compacts the chunk
that leaves the window into the history.  dcp_pages_fork then branches the session (sink and full history pages are
shared, the rest is copied), each branch goes on by itself, one is dropped with dcp_pages_free, and dcp_pages_compact
packs the pool; the other branch reads the same through its moved pages.

Run it on a GPU:  python examples/branching_session.py
The q, k, v and score inputs are random: a model would stand where `Session.step` draws them.
"""
from __future__ import annotations

import copy
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import autoregressive_video_diffusion_gb300 as dcp  # noqa: E402

LAYERS, HEADS, KV_HEADS, D, BS = 2, 8, 4, 64, 16
# Every phase offset stays in g's identity range, so history pages never change and branches can share the full ones.
# (Past the span the prune steps turn the whole history: branches would then share the sink's pages only.)
CFG = dcp.Config(gamma=0.10, sink_chunks=1, window_chunks=2, tokens_per_frame=16, frames_per_chunk=4,
                 n_temporal_pairs=8, g_recent_R=1000.0, g_span_S=1000.0, max_frames=128)
C, SLOTS, HIST_CAP = CFG.C, CFG.window_chunks + 1, 512


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


class Session:
    """One sequence: a view of the pools through its own block table (sink | history | ring slots)."""

    def __init__(self, cache: dcp.PagedKVCache, table: torch.Tensor):
        self.cache, self.table = cache, table
        n_sink, n_hist = CFG.sink_chunks * C // BS, HIST_CAP // BS
        self.sink, self.hist, self.ring = table[:n_sink], table[n_sink:n_sink + n_hist], table[n_sink + n_hist:]
        cache.hist_blocks, cache.window_blocks = self.hist, self.ring
        self.chunk, self.live = 0, set()
        self.rope = dcp.dcp_rope_plan(dcp.RopeConfig(rot_dim=2 * CFG.n_temporal_pairs, base=CFG.rope_base))
        self.prune_ws = dcp.new_workspace(dcp.dcp_paged_workspace_size(cache, CFG))

    def branch(self, table: torch.Tensor) -> "Session":
        cache = copy.copy(self.cache)
        cache.hist_len, cache.hist_t = self.cache.hist_len.clone(), self.cache.hist_t.clone()
        cache.status = torch.zeros_like(self.cache.status)
        other = Session(cache, table)
        other.chunk, other.live = self.chunk, set(self.live)
        return other

    def slot(self, s: int) -> torch.Tensor:
        return self.ring[s * C // BS:(s + 1) * C // BS]

    def visible(self):
        """Block table of what a new chunk sees, its history last, and the positions before the history."""
        parts = [self.slot(s) for s in sorted(self.live)] + [self.sink, self.hist]
        return torch.cat(parts)[None].contiguous(), len(self.live) * C + CFG.sink_chunks * C

    def read(self, layer: int, q: torch.Tensor):
        """Attention of q over the visible cache; each KV head has its own history length."""
        table, before = self.visible()
        lens = self.cache.hist_len.view(LAYERS, KV_HEADS)[layer:layer + 1].contiguous()
        batch = dcp.SeqBatch(ints([0, C]), table, lens, self.cache.status, total_q=C, max_q=C,
                             max_kv=before + HIST_CAP, kv_len_add=before)
        pool, cfg = dcp.layer_pool(self.cache, layer), dcp.AttnConfig(causal=False)
        ws = dcp.new_workspace(dcp.dcp_attention_workspace_size(pool, batch, cfg, HEADS))
        out, lse = torch.empty_like(q), torch.empty(C, HEADS, device="cuda")
        dcp.dcp_paged_attention(pool, batch, cfg, q, out, lse, ws)
        return out

    def write(self, layer: int, blocks: torch.Tensor, q, k, v):
        batch = dcp.SeqBatch(ints([0, C]), blocks[None].contiguous(), ints([C]), self.cache.status, total_q=C, max_q=C,
                             max_kv=C)
        frame = ints(self.chunk * CFG.frames_per_chunk + torch.arange(C) // CFG.tokens_per_frame)
        turned = torch.empty_like(q)
        dcp.dcp_rope_append(dcp.layer_pool(self.cache, layer), batch, self.rope, q, k, v, frame, turned)
        return turned

    def step(self, g: torch.Generator):
        """One chunk: into the cache, attention over it, and the chunk that leaves the window into the history."""
        sink = self.chunk < CFG.sink_chunks
        s = (self.chunk - CFG.sink_chunks) % SLOTS
        outs = []
        for layer in range(LAYERS):
            qkv = torch.randn(C, HEADS + 2 * KV_HEADS, D, generator=g, device="cuda").bfloat16()
            q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], dim=1)
            q = self.write(layer, self.sink if sink else self.slot(s), q, k, v)
            if not sink:
                self.live.add(s)
                outs.append((q, self.read(layer, q)))
        self.chunk += 1
        leaving = self.chunk - 1 - CFG.window_chunks
        if leaving >= CFG.sink_chunks:
            e, q0 = (leaving - CFG.sink_chunks) % SLOTS, self.chunk * CFG.frames_per_chunk
            x = torch.randn(C, 16, generator=g, device="cuda")
            noise = 0.6 * torch.randn(C, 16, generator=g, device="cuda") * torch.rand(C, 1, generator=g, device="cuda")
            dcp.dcp_paged_prune_step(self.cache, CFG, x + noise, x, e, leaving * CFG.frames_per_chunk, q0, q0, None,
                                     None, None, self.prune_ws)
            self.live.discard(e)
        return outs

    def plain(self, layer: int, q: torch.Tensor):
        """The same attention in plain torch arithmetic."""
        table, before = self.visible()
        out = torch.empty(C, HEADS, D, device="cuda")
        for h in range(HEADS):
            kh = h // (HEADS // KV_HEADS)
            n = before + int(self.cache.hist_len[layer * KV_HEADS + kh])
            k, v = (p[layer][table[0].long(), kh].reshape(-1, D)[:n].float()
                    for p in (self.cache.k_pool, self.cache.v_pool))
            out[:, h] = torch.softmax(q[:, h].float() @ k.T * D ** -0.5, -1) @ v
        return out

    def error(self, outs) -> float:
        return max(float((o.float() - self.plain(layer, q)).abs().max()) for layer, (q, o) in enumerate(outs))


def main() -> float:
    g = torch.Generator(device="cuda").manual_seed(1)
    n_table = (CFG.sink_chunks * C + HIST_CAP + SLOTS * C) // BS
    n_blocks = 4 * n_table
    cache = dcp.PagedKVCache(LAYERS, KV_HEADS, D, dcp.DCP_BF16, BS, dcp.DCP_PAGED_HND, n_blocks, HIST_CAP,
                             SLOTS * C // BS)
    pages = dcp.PagePool.of(cache)
    perm = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)
    tables = perm[:n_table][None].contiguous()
    ref = torch.zeros(n_blocks, dtype=torch.int32, device="cuda")
    ref[tables[0].long()] = 1
    cache.block_ref = ref  # a prune step that would write a shared page is refused
    root = Session(cache, tables[0])
    worst = 0.0
    for _ in range(6):
        before = root.chunk
        outs = root.step(g)
        if outs and root.chunk - 1 - CFG.window_chunks < CFG.sink_chunks:  # nothing has left: the cache is as it was read
            worst = max(worst, root.error(outs))
        assert root.chunk == before + 1

    # two branches: sink and full history pages are shared, the history's last page and the ring are copied
    hist = int(root.cache.hist_len.max())
    ws = dcp.new_workspace(dcp.dcp_pages_workspace_size(pages, 3, n_table))
    shared = (CFG.sink_chunks * C + hist) // BS
    children = torch.empty(2, n_table, dtype=torch.int32, device="cuda")
    dcp.dcp_pages_fork(pages, tables, ints([n_table * BS]), ints([0, 0]), ints([shared, shared]), None, ref, children,
                       ref, ws)
    tables = torch.cat([tables, children])
    branches = [root.branch(tables[1]), root.branch(tables[2])]
    probe = torch.randn(C, HEADS, D, generator=g, device="cuda").bfloat16()
    want = root.read(0, probe)
    assert all(torch.equal(b.read(0, probe), want) for b in branches)
    for i, b in enumerate(branches):
        gb = torch.Generator(device="cuda").manual_seed(10 + i)
        for _ in range(3):
            b.step(gb)
        worst = max(worst, b.error([(probe, b.read(0, probe))]))
    assert torch.equal(root.read(0, probe), want), "a branch's writes must not reach its parent"

    # one branch is dropped, the pool packed: the others read the same through moved pages
    keep = branches[1].read(0, probe)
    dcp.dcp_pages_free(pages, tables[1:2], ref, tables[1:2], ref)
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    dcp.dcp_pages_compact(pages, tables, ref, tables, ref, n_live, ws)
    assert int(tables.max()) < int(n_live) == int((ref > 0).sum())
    for s, row in ((root, 0), (branches[1], 2)):
        moved = s.branch(tables[row])
        assert torch.equal(moved.read(0, probe), want if s is root else keep)
        assert dcp.dcp_get_status(s.cache.status) == dcp.DCP_OK
    print(f"history of {hist} positions a plane, {shared} of {n_table} pages shared by each branch, {int(n_live)} of "
          f"{n_blocks} blocks live after packing; largest difference from plain attention {worst:.4f}")
    return worst


if __name__ == "__main__":
    main()
