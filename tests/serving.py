"""Plain 64-bit statements of the serving operators and the inputs their tests share.  Test infrastructure: no call of
the library is used to compute an expected value."""
from __future__ import annotations

import math

import numpy as np
import torch

import autoregressive_video_diffusion_gb300 as dcp

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HND, NHD = dcp.DCP_PAGED_HND, dcp.DCP_PAGED_NHD
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # a rounding's largest relative error


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


class Cache:
    """One layer's pages for a ragged batch: shuffled blocks, every page row filled with NaN until it is written."""

    def __init__(self, dtype, layout, h, d, bs, q_lens, kv_lens, seed=0, spare=2, table_pad=1):
        self.g = torch.Generator().manual_seed(seed)
        self.h, self.d, self.bs, self.layout, self.dt = h, d, bs, layout, DT[dtype]
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        pages = [-(-n // bs) for n in kv_lens]
        stride = max(max(pages), 1) + table_pad
        n_blocks = sum(pages) + spare
        perm = torch.randperm(n_blocks, generator=self.g).tolist()
        self.table = np.full((len(kv_lens), stride), -1, dtype=np.int32)
        at = 0
        for i, n in enumerate(pages):
            self.table[i, :n] = perm[at:at + n]
            at += n
        shape = (n_blocks, h, bs, d) if layout == HND else (n_blocks, bs, h, d)
        self.k = torch.full(shape, math.nan, dtype=self.dt, device="cuda")
        self.v = torch.full(shape, math.nan, dtype=self.dt, device="cuda")
        self.keys = [self.normal(n, h, d) for n in kv_lens]
        self.values = [self.normal(n, h, d) for n in kv_lens]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.tables = torch.from_numpy(self.table).cuda()
        start = np.concatenate([[0], np.cumsum(q_lens)])
        self.start = start.tolist()
        self.q_start, self.kv_len = ints(self.start), ints(self.kv_lens)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g).to(self.dt).cuda()

    def rows(self, i, lo, hi):
        j = torch.arange(lo, hi)
        return torch.from_numpy(self.table[i])[j // self.bs].long().cuda(), (j % self.bs).cuda()

    def write(self, pool, i, lo, x):
        block, row = self.rows(i, lo, lo + x.shape[0])
        if self.layout == HND:
            pool[block, :, row] = x
        else:
            pool[block, row] = x

    def fill(self):
        for i in range(len(self.kv_lens)):
            self.write(self.k, i, 0, self.keys[i])
            self.write(self.v, i, 0, self.values[i])
        return self

    def pool(self):
        return dcp.KVPool(self.k, self.v, self.layout)

    def batch(self, **over):
        kw = dict(total_q=self.start[-1], max_q=max(self.q_lens), max_kv=max(self.kv_lens))
        kw.update(over)
        return dcp.SeqBatch(self.q_start, self.tables, self.kv_len, self.status, **kw)


def attention_64(q, k, v, c0, scale, causal, window):
    """out, lse, sum w|v| and the largest sum |scale q k| of one sequence and head in 64 bits: q [nq][d] whose first
    row sits at cache position c0, k and v [nk][d].  Only the visible positions of a row are touched."""
    q, k, v = q.double(), k.double(), v.double()
    nq, nk = q.shape[0], k.shape[0]
    c = c0 + torch.arange(nq, device=q.device)[:, None]
    j = torch.arange(nk, device=q.device)[None]
    seen = torch.ones(nq, nk, dtype=torch.bool, device=q.device)
    if causal:
        seen &= j <= c
    if window >= 0:
        seen &= j >= c - window
    used = seen.any(0)
    k, v = torch.where(used[:, None], k, 0.0), torch.where(used[:, None], v, 0.0)
    s = (q @ k.T * scale).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if nk else torch.full((nq,), -math.inf, dtype=torch.float64, device=q.device)
    w = torch.where(seen, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
    terms = (q.abs() @ k.abs().T * abs(scale)).max().item() if nk and nq else 0.0
    return w @ v, lse, w @ v.abs(), terms


def attention_bounds(dt, d, n, out, mass, lse, terms):
    """Largest errors of out and lse: scores are sums of d products in 32 bits (each off by 2^-24 of the running sum's
    size, at most `terms`), exp and the sums over n keys in 32 bits, weights rounded to the cache's type before they
    meet the values (bf16), and the result's own rounding."""
    score = (d + 8) * 2.0 ** -24 * terms + 2.0 ** -21
    sums = (n + 64) * 2.0 ** -24
    half = HALF_STEP[dt]
    weight = half if dt == torch.bfloat16 else 0.0
    return mass * (2 * score + 2 * sums + 1.01 * weight) + half * out.abs() + 1e-30, \
        score + sums + 2.0 ** -22 * (1.0 + lse.abs())


def check_attention(cache, q, out, lse, scale, causal, window, kv_of=None):
    """Every row of out and lse against 64 bits."""
    hq = q.shape[1]
    for i, nq in enumerate(cache.q_lens):
        r = slice(cache.start[i], cache.start[i + 1])
        for h in range(hq):
            kh = h // (hq // cache.h)
            nk = cache.kv_lens[i] if kv_of is None else kv_of[i][kh]
            o, l, mass, terms = attention_64(q[r, h], cache.keys[i][:nk, kh], cache.values[i][:nk, kh], nk - nq,
                                             scale, causal, window)
            tol, tol_l = attention_bounds(cache.dt, cache.d, max(nk, 1), o, mass, l, terms)
            got = out[r, h].double()
            assert torch.isfinite(got).all(), (i, h)
            assert ((got - o).abs() <= tol).all(), (i, h, (got - o).abs().max().item())
            if lse is not None:
                empty = l == -math.inf
                assert torch.equal(lse[r, h] == -math.inf, empty), (i, h)
                assert ((lse[r, h].double() - l).abs()[~empty] <= tol_l[~empty]).all(), (i, h)


def thetas_64(cfg):
    """theta_p of a RopeConfig in 64 bits, from its definition."""
    out = []
    for p in range(cfg.rot_dim // 2):
        base = cfg.base
        if cfg.scaling == dcp.DCP_ROPE_BASE and cfg.rot_dim > 2:
            base = base * cfg.factor ** (cfg.rot_dim / (cfg.rot_dim - 2))
        t = math.exp(-2.0 * p / cfg.rot_dim * math.log(base))
        if cfg.scaling == dcp.DCP_ROPE_LINEAR:
            t /= cfg.factor
        if cfg.scaling == dcp.DCP_ROPE_PARTS:
            r = cfg.orig_len * t / (2 * math.pi)
            g = min(1.0, max(0.0, (r - cfg.beta_slow) / (cfg.beta_fast - cfg.beta_slow)))
            t = t * g + t / cfg.factor * (1 - g)
        out.append(t)
    return out


def turned_64(x, positions, cfg):
    """x [n][heads][d] turned to its positions in 64 bits, and |a| + |b| of each dim's pair."""
    y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    half = cfg.rot_dim // 2
    pos = torch.as_tensor(positions, dtype=torch.float64)
    for p, t in enumerate(thetas_64(cfg)):
        i, j = (2 * p, 2 * p + 1) if cfg.pair_layout == dcp.DCP_ROPE_INTERLEAVED else (p, p + half)
        a, b = x[..., i].double(), x[..., j].double()
        c = (torch.cos(pos * t) * cfg.amplitude).to(x.device)[:, None]
        s = (torch.sin(pos * t) * cfg.amplitude).to(x.device)[:, None]
        y[..., i], y[..., j] = a * c - b * s, a * s + b * c
        size[..., i] = size[..., j] = a.abs() + b.abs()
    return y, size


def check_turned(got, x, positions, cfg):
    want, size = turned_64(x, positions, cfg)
    half = HALF_STEP[x.dtype]
    # phase off by 2^-30 turns and its rounding to 24 bits, sine and cosine by 2 ulp, three roundings of the pair
    tol = abs(cfg.amplitude) * size * 2.0 ** -21 + half * want.abs() * (size > 0)
    assert ((got.double() - want).abs() <= tol).all(), (got.double() - want).abs().max().item()


# ------------------------------------------------------------------------------------------ pages
def fork_plain(tables, lens, parent, shared, reserve, ref, bs):
    """child tables, counts and moves of a fork, page by page."""
    ref, child, moves = ref.copy(), np.full((len(parent), tables.shape[1]), -1, np.int32), []
    free = [b for b in range(len(ref)) if ref[b] == 0]
    for c, p in enumerate(parent):
        n = -(-lens[p] // bs)
        ns = lens[p] // bs if shared is None else shared[c]
        total = max(n, 0 if reserve is None else -(-reserve[c] // bs))
        for j in range(total):
            if j < ns:
                child[c, j] = tables[p, j]
                ref[tables[p, j]] += 1
            else:
                b = free.pop(0)
                child[c, j], ref[b] = b, 1
                if j < n:
                    moves.append((tables[p, j], b))
    return child, ref, moves


def compact_plain(tables, ref):
    ref, tables = ref.copy(), tables.copy()
    live = int((ref > 0).sum())
    holes = [b for b in range(live) if ref[b] <= 0]
    movers = [b for b in range(live, len(ref)) if ref[b] > 0]
    for a, b in zip(movers, holes):
        ref[b], ref[a] = ref[a], 0
        tables[tables == a] = b
    return tables, ref, live, list(zip(movers, holes))
