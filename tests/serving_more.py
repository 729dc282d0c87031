"""Plain 64-bit statements of the norms in front of the rotary turn, of windows with first positions, and of branches
that share a prefix, and the inputs their tests share.  Test infrastructure, as tests/serving.py."""
from __future__ import annotations

import math

import numpy as np
import torch

import autoregressive_video_diffusion_gb300 as dcp
from tests.serving import HALF_STEP, HND, Cache, attention_bounds, ints, thetas_64


# ------------------------------------------------------------------------------------------ norms
def normed_64(x, w, eps, span):
    """x [n][heads][d] normalised in 64 bits."""
    y = x.double()
    over = (2,) if span == dcp.DCP_NORM_HEAD else (1, 2)
    y = y / torch.sqrt(y.square().mean(over, keepdim=True) + eps)
    return y if w is None else y * w.double()


def norm_turned_64(x, w, eps, span, positions, cfgs):
    """x normalised and turned by positions [n_axes][n] in 64 bits, and |a| + |b| of each dim's (normalised) pair."""
    y = normed_64(x, w, eps, span)
    z, size, done = y.clone(), torch.zeros_like(y), 0
    pairs = sum(cfg.rot_dim for cfg in cfgs) // 2
    for cfg, at in zip(cfgs, positions):
        pos = torch.as_tensor(np.asarray(at), dtype=torch.float64)
        for t in thetas_64(cfg):
            i, j = (2 * done, 2 * done + 1) if cfg.pair_layout == dcp.DCP_ROPE_INTERLEAVED else (done, done + pairs)
            a, b = y[..., i], y[..., j]
            c = (torch.cos(pos * t) * cfg.amplitude).to(x.device)[:, None]
            s = (torch.sin(pos * t) * cfg.amplitude).to(x.device)[:, None]
            z[..., i], z[..., j] = a * c - b * s, a * s + b * c
            size[..., i] = size[..., j] = (a.abs() + b.abs()) * abs(cfg.amplitude)
            done += 1
    return z, size


def check_norm_turned(got, x, w, eps, span, positions, cfgs):
    want, size = norm_turned_64(x, w, eps, span, positions, cfgs)
    # a sum of squares (all positive): at most 16 terms of a head behind one another in a lane and 5 sums of lanes; of a
    # token at most 2 terms a head and 16 more, 5 sums of lanes and 8 of warps.  Half of it in the root; the mean, the root
    # and its correction and three products are a rounding each.
    chain = 24 if span == dcp.DCP_NORM_HEAD else 2 * x.shape[1] + 32
    norm = (0.5 * chain + 7) * 2.0 ** -24
    # the turn as in tests/serving.py: phase off by 2^-30 turns and its rounding, sine and cosine by 2 ulp, three roundings
    plain = torch.where(size > 0, size, want.abs())
    tol = plain * norm + size * 2.0 ** -21 + HALF_STEP[x.dtype] * want.abs() + 1e-37
    assert ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() / tol.clamp(min=1e-300)).max().item()


# ------------------------------------------------------------------------------------------ windows with first positions
def attention_sink_64(q, k, v, c0, scale, causal, window, sink):
    """out, lse, sum w|v| and the largest sum |scale q k| of one sequence and head in 64 bits (tests/serving.py's
    attention_64 with first positions that stay visible).  Only the visible positions of a row are touched."""
    q, k, v = q.double(), k.double(), v.double()
    nq, nk = q.shape[0], k.shape[0]
    c = c0 + torch.arange(nq, device=q.device)[:, None]
    j = torch.arange(nk, device=q.device)[None]
    seen = torch.ones(nq, nk, dtype=torch.bool, device=q.device)
    if causal:
        seen &= j <= c
    if window >= 0:
        seen &= (j >= c - window) | (j < sink)
    used = seen.any(0)
    k, v = torch.where(used[:, None], k, 0.0), torch.where(used[:, None], v, 0.0)
    s = (q @ k.T * scale).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if nk else torch.full((nq,), -math.inf, dtype=torch.float64, device=q.device)
    w = torch.where(seen, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
    terms = (q.abs() @ k.abs().T * abs(scale)).max().item() if nk and nq else 0.0
    return w @ v, lse, w @ v.abs(), terms


def check_attention_sink(cache, q, out, lse, scale, causal, window, sink, kv_of=None):
    """Every row of out and lse against 64 bits."""
    hq = q.shape[1]
    for i, nq in enumerate(cache.q_lens):
        r = slice(cache.start[i], cache.start[i + 1])
        for h in range(hq):
            kh = h // (hq // cache.h)
            nk = cache.kv_lens[i] if kv_of is None else kv_of[i][kh]
            o, l, mass, terms = attention_sink_64(q[r, h], cache.keys[i][:nk, kh], cache.values[i][:nk, kh], nk - nq,
                                                  scale, causal, window, sink)
            tol, tol_l = attention_bounds(cache.dt, cache.d, max(nk, 1), o, mass, l, terms)
            got = out[r, h].double()
            assert torch.isfinite(got).all(), (i, h)
            assert ((got - o).abs() <= tol).all(), (i, h, (got - o).abs().max().item())
            if lse is not None:
                empty = l == -math.inf
                assert torch.equal(lse[r, h] == -math.inf, empty), (i, h)
                assert ((lse[r, h].double() - l).abs()[~empty] <= tol_l[~empty]).all(), (i, h)


# ------------------------------------------------------------------------------------------ shared prefixes
FAR = 1 << 28


class Branches(Cache):
    """Pages of sequences in groups: [(prefix, [(new tokens, positions behind the prefix, new tokens among them), ...]),
    ...]; `before` and `after` further sequences that belong to no group.  A branch names its group's full pages and holds
    a copy of the prefix's last, partial one."""

    def __init__(self, dtype, layout, h, d, bs, groups, before=(), after=(), seed=0):
        self.prefix = [p for p, _ in groups]
        seqs = [(q, n) for q, n in before]
        self.group_at = [len(seqs)]
        for p, members in groups:
            seqs += [(q, p + n) for q, n in members]
            self.group_at.append(len(seqs))
        seqs += list(after)
        super().__init__(dtype, layout, h, d, bs, [q for q, _ in seqs], [n for _, n in seqs], seed)
        for g, p in enumerate(self.prefix):
            for s in range(self.group_at[g] + 1, self.group_at[g + 1]):
                first = self.group_at[g]
                self.keys[s][:p], self.values[s][:p] = self.keys[first][:p], self.values[first][:p]
                self.table[s, :p // bs] = self.table[first, :p // bs]
        self.tables = torch.from_numpy(self.table).cuda()
        self.start_dev, self.prefix_dev = ints(self.group_at), ints(self.prefix)

    def groups(self, **over):
        kw = dict(max_prefix=max(self.prefix), max_q=max(
            1, *(self.start[b] - self.start[a] for a, b in zip(self.group_at, self.group_at[1:]))))
        kw.update(over)
        return dcp.PrefixGroups(self.start_dev, self.prefix_dev, **kw)

    def far(self, rest=0):
        """The batch and the groups with bounds so large that prefixes are shared however short they are; `rest` is the bound
        of what lies behind them."""
        return dict(batch=self.batch(max_kv=FAR + rest), groups=self.groups(max_prefix=FAR))

    def attend(self, q, causal=True, window=-1, sink=0, scale=None, batch=None, groups=None):
        out = torch.full_like(q, math.nan, memory_format=torch.contiguous_format)
        lse = torch.full(q.shape[:2], math.nan, device="cuda")
        cfg, pool = dcp.AttnConfig(scale, causal, window, sink), self.pool()
        batch, groups = batch or self.batch(), groups or self.groups()
        ws = dcp.new_workspace(dcp.dcp_shared_attention_workspace_size(pool, batch, groups, cfg, q.shape[1]))
        for _ in range(2):  # the workspace is left ready for the next call
            dcp.dcp_shared_attention(pool, batch, groups, cfg, q, out, lse, ws)
        return out, lse
