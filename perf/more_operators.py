"""Further serving operators around the paged cache, as they are called: the cases that are measured, their inputs, one
pass in plain torch operations or through the library, and the work that a pass cannot do without.

Three operators, chosen by a case's "op":
  norm     the new tokens' q and k normalised (each head, or all heads of a token together), turned by one to three
           position axes, q returned and k, v written to the cache's pages
  sink     attention of the new tokens over the paged cache through a sliding window and a few first positions
  shared   attention of branches that hold a long prefix in common, which is read once for all of them
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases
def _norm(name, **kw):
    c = dict(name=name, op="norm", dtype="bf16", wdtype="bf16", layout="hnd", hq=40, h=8, d=128, bs=16, seqs=1, q_lo=1,
             q_hi=1, kv_lo=1024, kv_hi=1024, span="head", weights="shared", rot=128, rot2=0, rot3=0, pairs="half",
             base=10000.0, far=0, lens=1)
    c.update(kw)
    return c


def _sink(name, **kw):
    c = dict(name=name, op="sink", dtype="bf16", layout="hnd", hq=40, h=8, d=128, bs=16, seqs=1, q_lo=1, q_hi=1,
             kv_lo=1024, kv_hi=1024, window=1023, sink=4, lens=1)
    c.update(kw)
    return c


def _shared(name, **kw):
    c = dict(name=name, op="shared", dtype="bf16", layout="hnd", hq=40, h=8, d=128, bs=16, groups=1, per_lo=8, per_hi=8,
             q_lo=1, q_hi=1, pre_lo=1024, pre_hi=1024, own_lo=1, own_hi=64, causal=True, lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # a batch's next tokens: each head's q and k normalised and turned on their way into the pages
        _norm("norm tokens", layout="nhd", seqs=32, kv_lo=64, kv_hi=2048),
        # a video chunk (4 frames of 30 x 52 tokens): all heads normalised together, frame, row and column turned
        _norm("norm video chunk", q_lo=6240, q_hi=6240, kv_lo=6240, kv_hi=6240, h=40, bs=32, span="token",
              weights="heads", wdtype="f32", rot=44, rot2=42, rot3=42, pairs="interleaved", far=240),
        # prompts far into a long context, part of the head turned, fp32 cache
        _norm("norm prompts fp32", dtype="f32", wdtype="f32", hq=20, h=4, d=96, rot=64, seqs=5, q_lo=17, q_hi=1900,
              kv_lo=1900, kv_hi=4001, bs=24, base=500000.0, far=1000000, weights="heads"),
        # heads of 80 whose pairs fall into no vector
        _norm("norm odd heads", hq=12, h=4, d=80, rot=40, seqs=7, q_lo=1, q_hi=301, kv_lo=301, kv_hi=999, bs=24),
        # one session's next token in a windowed layer: nothing but latency
        _sink("sink token", kv_lo=5001, kv_hi=5001, window=1000, sink=4),
        # a serving batch's next tokens: ragged lengths, some shorter than the window
        _sink("sink tokens batch", layout="nhd", seqs=96, kv_lo=200, kv_hi=16000, bs=32, window=4095, sink=128, lens=2),
        # the Streaming policy over a video history: a chunk sees the sink chunk and the three chunks behind each token
        _sink("sink video chunk", q_lo=6240, q_hi=6240, kv_lo=43680, kv_hi=43680, bs=32, window=18720, sink=6240),
        # prompts' chunks with heads of 80 over pages of 24 positions: sizes that fill no tile
        _sink("sink prompts odd", hq=12, h=4, d=80, bs=24, seqs=5, q_lo=33, q_hi=1400, kv_lo=1401, kv_hi=6000, window=513,
              sink=37, lens=4),
        # a few branches of a short session: latency
        _shared("shared few", per_lo=4, per_hi=4, pre_lo=1520, pre_hi=1520, own_lo=3, own_hi=40),
        # many branches of one long session
        _shared("shared branches", per_lo=32, per_hi=32, pre_lo=24960, pre_hi=24960, own_lo=20, own_hi=700, lens=2),
        # several sessions' branches with drafts of a few tokens, position-major pages
        _shared("shared drafts", layout="nhd", bs=32, hq=32, groups=6, per_lo=1, per_hi=12, q_lo=1, q_hi=5, pre_lo=500,
                pre_hi=16000, own_lo=6, own_hi=400, lens=3),
        # the fp32 cache
        _shared("shared fp32", dtype="f32", hq=8, h=8, d=64, groups=2, per_lo=9, per_hi=13, pre_lo=1000, pre_hi=6001,
                own_lo=1, own_hi=200, lens=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "sink", "shared"])
    lens = rng.randrange(1 << 30)
    h = rng.choice([1, 2, 4, 8])
    hq = h * rng.choice([1, 2, 4, 5, 7, 8])
    d = rng.choice([32, 40, 64, 80, 96, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    bs = rng.choice([5, 8, 16, 16, 24, 32, 64, 100, 128, 240])
    layout = rng.choice(["hnd", "nhd"])
    seqs = _log(rng, 1, 64)
    if op == "norm":
        q_hi = _log(rng, 1, max(1, 8000 // seqs))
        half, axes = d // 2, rng.choice([1, 1, 2, 3])
        first = rng.randint(0 if axes == 1 else 1, half)
        second = rng.randint(0, half - first) if axes > 1 else 0
        third = rng.randint(0, half - first - second) if axes > 2 else 0
        if not second:
            third = 0
        return dict(op=op, dtype=dtype, wdtype=rng.choice([dtype, "f32"]), layout=layout, hq=hq, h=h, d=d, bs=bs,
                    seqs=seqs, q_lo=rng.randint(1, q_hi), q_hi=q_hi, kv_lo=q_hi, kv_hi=q_hi + _log(rng, 1, 4000),
                    span=rng.choice(["head", "head", "token"]), weights=rng.choice(["shared", "heads", "none"]),
                    rot=2 * first, rot2=2 * second, rot3=2 * third, pairs=rng.choice(["half", "interleaved"]),
                    base=rng.choice([10000.0, 500000.0]), far=rng.choice([0, 240, 100000, 1000000]), lens=lens)
    room = 2.0e9 if dtype == "bf16" else 2.5e8  # scores of a pass
    if op == "sink":
        q_hi = rng.choice([1, rng.randint(2, 9), _log(rng, 10, 4000)])
        kv_hi = q_hi + _log(rng, 1, 30000)
        kv_hi = max(q_hi, min(kv_hi, int(room / (q_hi * hq))))
        seqs = max(1, min(seqs, int(room / (q_hi * hq * kv_hi)), int(1.2e9 / (kv_hi * h * d))))
        return dict(op=op, dtype=dtype, layout=layout, hq=hq, h=h, d=d, bs=bs, seqs=seqs, q_lo=rng.randint(1, q_hi),
                    q_hi=q_hi, kv_lo=q_hi, kv_hi=kv_hi, window=_log(rng, 1, kv_hi), sink=_log(rng, 1, kv_hi), lens=lens)
    q_hi = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 200)])
    pre_hi, own_hi = _log(rng, 1, 30000), q_hi + _log(rng, 1, 1500)
    groups, per_hi = _log(rng, 1, 8), _log(rng, 1, 40)
    kv_hi = pre_hi + own_hi
    per_hi = max(1, min(per_hi, int(room / (q_hi * hq * kv_hi)), int(1.2e9 / (kv_hi * h * d))))
    groups = max(1, min(groups, int(room / (q_hi * hq * kv_hi * per_hi)), int(1.2e9 / (kv_hi * h * d * per_hi))))
    return dict(op=op, dtype=dtype, layout=layout, hq=hq, h=h, d=d, bs=bs, groups=groups, per_lo=rng.randint(1, per_hi),
                per_hi=per_hi, q_lo=rng.randint(1, q_hi), q_hi=q_hi, pre_lo=rng.randint(0, pre_hi), pre_hi=pre_hi,
                own_lo=q_hi, own_hi=own_hi, causal=rng.random() < 0.8, lens=lens)


def _lens(case):
    """New tokens and cache lengths of each sequence, from the case alone."""
    if case["op"] == "shared":
        _, q, pre, mine = _branches(case)
        return q, [p + m for p, m in zip(pre, mine)]
    r = random.Random(case["lens"])
    q = [case["q_hi"] if i == 0 else r.randint(case["q_lo"], case["q_hi"]) for i in range(case["seqs"])]
    kv = [case["kv_hi"] if i == 0 else r.randint(case["kv_lo"], case["kv_hi"]) for i in range(case["seqs"])]
    return q, kv


def _branches(case):
    """Branches of each group; new tokens, prefix and further positions (new tokens among them) of each branch."""
    r = random.Random(case["lens"])
    per, q, pre, mine = [], [], [], []
    for g in range(case["groups"]):
        per.append(case["per_hi"] if g == 0 else r.randint(case["per_lo"], case["per_hi"]))
        common = case["pre_hi"] if g == 0 else r.randint(case["pre_lo"], case["pre_hi"])
        for b in range(per[-1]):
            q.append(case["q_hi"] if not q else r.randint(case["q_lo"], case["q_hi"]))
            pre.append(common)
            mine.append(case["own_hi"] if b == 0 else r.randint(max(case["own_lo"], q[-1]), case["own_hi"]))
    return per, q, pre, mine


def _rots(case):
    return [r for r in (case["rot"], case["rot2"], case["rot3"]) if r] or [0]


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    st = {"case": case}
    q_len, kv_len = _lens(case)
    h, bs, d, n = case["h"], case["bs"], case["d"], sum(q_len)
    stride = -(-max(kv_len) // bs)
    n_blocks = sum(-(-x // bs) for x in kv_len) + 3
    if case["op"] == "shared":
        per, _, pre, _ = _branches(case)
        first = [sum(per[:i]) for i in range(len(per) + 1)]
        n_blocks -= sum(pre[first[i]] // bs * (m - 1) for i, m in enumerate(per))
    shape = (n_blocks, h, bs, d) if case["layout"] == "hnd" else (n_blocks, bs, h, d)
    st["k_pool"], st["v_pool"] = normal(*shape), normal(*shape)
    perm = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(q_len), stride), -1, dtype=torch.int32, device="cuda")
    at = 0
    if case["op"] == "shared":
        for i, m in enumerate(per):
            common, rest = divmod(pre[first[i]], bs)
            for s in range(first[i], first[i] + m):
                pages = -(-kv_len[s] // bs)
                if s > first[i]:  # a branch: the full pages are its parent's too, the last one of the prefix is a copy
                    tables[s, :common] = tables[first[i], :common]
                lo = common if s > first[i] else 0
                tables[s, lo:pages] = perm[at:at + pages - lo]
                at += pages - lo
            if rest:
                mine, its = tables[first[i] + 1:first[i] + m, common].long(), tables[first[i], common].long()
                for pool in (st["k_pool"], st["v_pool"]):
                    if case["layout"] == "hnd":
                        pool[mine, :, :rest] = pool[its, :, :rest]
                    else:
                        pool[mine, :rest] = pool[its, :rest]
        st["group_start"], st["prefix_len"] = ints(first), ints([pre[i] for i in first[:-1]])
    else:
        for i, x in enumerate(kv_len):
            tables[i, :-(-x // bs)] = perm[at:at + -(-x // bs)]
            at += -(-x // bs)
    start = [0]
    for x in q_len:
        start.append(start[-1] + x)
    st["tables"], st["kv_len"], st["q_start"] = tables, ints(kv_len), ints(start)
    st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "norm":
        qkv = normal(n, case["hq"] + 2 * h, d)
        st["q"], st["k"], st["v"] = qkv.split([case["hq"], h, h], dim=1)
        st["q_out"] = torch.empty(n, case["hq"], d, dtype=dt, device="cuda")
        st["q_weight"] = st["k_weight"] = st["positions"] = None
        if case["weights"] != "none":
            for name, heads in (("q_weight", case["hq"]), ("k_weight", h)):
                w = torch.empty((d,) if case["weights"] == "shared" else (heads, d), device="cuda")
                st[name] = w.normal_(1.0, 0.3, generator=g).to(DT[case["wdtype"]])
        axes = len(_rots(case))
        if case["far"] or axes > 1:
            far = max(case["far"], 2)
            st["positions"] = torch.randint(far // 2, far, (axes, n), generator=g, device="cuda").to(torch.int32)
    else:
        st["q"] = normal(n, case["hq"], d)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(n, case["hq"], dtype=torch.float32, device="cuda")
    if own:
        import autoregressive_video_diffusion_gb300 as dcp
        layout = dcp.DCP_PAGED_HND if case["layout"] == "hnd" else dcp.DCP_PAGED_NHD
        st["pool"] = dcp.KVPool(st["k_pool"], st["v_pool"], layout)
        st["batch"] = dcp.SeqBatch(st["q_start"], st["tables"], st["kv_len"], st["status"], total_q=n,
                                   max_q=max(q_len), max_kv=max(kv_len))
        if case["op"] == "norm":
            pairs = dcp.DCP_ROPE_HALF if case["pairs"] == "half" else dcp.DCP_ROPE_INTERLEAVED
            st["axes"] = dcp.dcp_rope_axes([dcp.RopeConfig(rot_dim=r, pair_layout=pairs, base=case["base"])
                                            for r in _rots(case)])
            st["norm"] = dcp.NormConfig(st["q_weight"], st["k_weight"], eps=EPS, span=dcp.DCP_NORM_TOKEN
                                        if case["span"] == "token" else dcp.DCP_NORM_HEAD)
        elif case["op"] == "sink":
            st["cfg"] = dcp.AttnConfig(causal=True, window=case["window"], sink=case["sink"])
            st["ws"] = dcp.new_workspace(dcp.dcp_attention_workspace_size(st["pool"], st["batch"], st["cfg"],
                                                                          case["hq"]))
        else:
            st["cfg"] = dcp.AttnConfig(causal=case["causal"])
            st["groups"] = dcp.PrefixGroups(st["group_start"], st["prefix_len"], max_prefix=max(pre),
                                            max_q=max(sum(q_len[a:b]) for a, b in zip(first, first[1:])))
            st["ws"] = dcp.new_workspace(dcp.dcp_shared_attention_workspace_size(
                st["pool"], st["batch"], st["groups"], st["cfg"], case["hq"]))
    return st


# ------------------------------------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"norm": _own_norm, "sink": _own_sink, "shared": _own_shared}[op](st)
    return _plain_norm(st) if op == "norm" else _plain_attend(st)


def _own_norm(st):
    import autoregressive_video_diffusion_gb300 as dcp
    dcp.dcp_norm_rope_append(st["pool"], st["batch"], st["axes"], st["norm"], st["q"], st["k"], st["v"],
                             st["positions"], st["q_out"])
    return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _own_sink(st):
    import autoregressive_video_diffusion_gb300 as dcp
    dcp.dcp_paged_attention(st["pool"], st["batch"], st["cfg"], st["q"], st["out"], st["lse"], st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_shared(st):
    import autoregressive_video_diffusion_gb300 as dcp
    dcp.dcp_shared_attention(st["pool"], st["batch"], st["groups"], st["cfg"], st["q"], st["out"], st["lse"], st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _plain_norm(st):
    case = st["case"]
    n = st["q"].shape[0]
    i = torch.arange(n, device="cuda")
    seq = torch.searchsorted(st["q_start"][1:].long(), i, right=True)
    pos = st["kv_len"].long()[seq] - st["q_start"].long()[seq + 1] + i
    block, row = st["tables"][seq, pos // case["bs"]].long(), pos % case["bs"]
    # cos and sin of every pair of every axis, the angles in 64 bits
    rots, angles = _rots(case), []
    for a, rot in enumerate(rots):
        theta = case["base"] ** (-2 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / max(rot, 1))
        at = pos if st["positions"] is None else st["positions"][a]
        angles.append(at.double()[:, None] * theta)
    angle = torch.cat(angles, 1)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = angle.shape[1]

    def turned(x, w):
        y = x.float()
        over = (-1,) if case["span"] == "head" else (-2, -1)
        y = y * torch.rsqrt((y * y).mean(over, keepdim=True) + EPS)
        if w is not None:
            y = y * w.float()
        rest = y[..., 2 * half:]
        if case["pairs"] == "half":
            a, b = y[..., :half], y[..., half:2 * half]
            z = torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
        else:
            a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            z = torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)
        return z.to(x.dtype)

    q, k = turned(st["q"], st["q_weight"]), turned(st["k"], st["k_weight"])
    if case["layout"] == "hnd":
        st["k_pool"][block, :, row] = k
        st["v_pool"][block, :, row] = st["v"]
    else:
        st["k_pool"][block, row] = k
        st["v_pool"][block, row] = st["v"]
    return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _plain_attend(st):
    """Every sequence against its own pages, the batch padded to its longest."""
    case = st["case"]
    hq, h, d, bs = case["hq"], case["h"], case["d"], case["bs"]
    q_len, kv_len = torch.diff(st["q_start"]).long(), st["kv_len"].long()
    lens = _lens(case)
    max_q, max_kv = max(lens[0]), max(lens[1])
    i, j = torch.arange(max_q, device="cuda"), torch.arange(max_kv, device="cuda")
    n = st["q"].shape[0]
    at = (st["q_start"][:-1].long()[:, None] + i).clamp(max=n - 1)                       # [b, max_q]
    block = st["tables"][:, j // bs].clamp(min=0).long()                                 # [b, max_kv]
    if case["layout"] == "hnd":
        k, v = st["k_pool"][block, :, j % bs].float(), st["v_pool"][block, :, j % bs].float()
    else:
        k, v = st["k_pool"][block, j % bs].float(), st["v_pool"][block, j % bs].float()  # [b, max_kv, h, d]
    b = block.shape[0]
    q = st["q"][at].float().view(b, max_q, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    s = (q * d ** -0.5) @ k.permute(0, 2, 3, 1)                                          # [b, h, g max_q, max_kv]
    s = s.view(b, h, hq // h, max_q, max_kv)
    c = (kv_len[:, None] - q_len[:, None] + i)[..., None]                                # [b, max_q, 1]
    seen = (j < kv_len[:, None])[:, None].expand(b, max_q, max_kv)
    if case.get("causal", True):
        seen = seen & (j <= c)
    if case["op"] == "sink":
        seen = seen & ((j >= c - case["window"]) | (j < case["sink"]))
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(b, h, -1, max_kv) @ v.permute(0, 2, 1, 3)).view(b, h, hq // h, max_q, d)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(b, max_q, hq, d)
    lse = lse.permute(0, 3, 1, 2).reshape(b, max_q, hq)
    rows = torch.arange(n, device="cuda")
    seq = torch.searchsorted(st["q_start"][1:].long(), rows, right=True)
    place = rows - st["q_start"].long()[seq]
    return {"out": out[seq, place].to(st["q"].dtype), "lse": lse[seq, place].contiguous()}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    es, d, bs = ES[case["dtype"]], case["d"], case["bs"]
    q_len, kv_len = _lens(case)
    n = sum(q_len)
    if case["op"] == "norm":
        heads, turned = case["hq"] + 2 * case["h"], case["hq"] + case["h"]
        w = {"none": 0, "shared": 2, "heads": turned}[case["weights"]] * d * ES[case["wdtype"]]
        axes = len(_rots(case)) if case["far"] or len(_rots(case)) > 1 else 0
        return {"bytes": 2 * n * heads * d * es + w + 4 * n * axes + 4 * len(q_len) * 3,
                "flops": n * turned * (4 * d + 6 * (sum(_rots(case)) // 2))}
    pairs = keys = 0
    if case["op"] == "sink":
        for nq, nk in zip(q_len, kv_len):
            w, sink, lo = case["window"], case["sink"], nk - nq
            full = max(0, nk - max(lo, w))                 # rows whose window begins at 0 or later: w + 1 keys
            short = nq - full                              # the others see c + 1 keys
            pairs += full * (w + 1) + short * (lo + 1) + short * (short - 1) // 2
            # keys before a row's window that are among the first ones: min(sink, c - w) where c > w
            a, b = max(0, lo - w), max(0, nk - 1 - w)      # where the first and the last row's window begins
            pairs += sink * max(0, b - max(a, sink) + 1) + sum(range(a, min(b, sink - 1) + 1))
            begin = max(0, lo - w)
            keys += nk - begin + min(sink, begin)
    else:
        per, _, pre, mine = _branches(case)
        at = 0
        for m in per:
            keys += pre[at] + sum(mine[at:at + m])
            at += m
        for nq, nk in zip(q_len, kv_len):
            pairs += nq * nk - (nq * (nq - 1) // 2 if case["causal"] else 0)
    return {"bytes": 2 * n * case["hq"] * d * es + 4 * n * case["hq"] + 2 * keys * case["h"] * d * es
            + 4 * (keys // bs + 1), "flops": 4 * pairs * case["hq"] * d}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, an axis, a sequence and a head at a time."""
    if case["op"] != "norm" and work(case)["flops"] > 5e12:
        return None
    st = prepare(case, seed)
    q_len, kv_len = _lens(case)
    hq, h, d, bs = case["hq"], case["h"], case["d"], case["bs"]
    if case["op"] == "norm":
        place = torch.cat([torch.arange(nk - nq, nk) for nq, nk in zip(q_len, kv_len)]).cuda()
        seq = torch.cat([torch.full((nq,), i) for i, nq in enumerate(q_len)]).cuda()
        pairs = sum(_rots(case)) // 2

        def definition(x, w):
            y = x.double()
            size = y.square().sum(-1) / d if case["span"] == "head" else y.square().sum((-2, -1))[:, None] / x[0].numel()
            y = y / (size + EPS).sqrt()[..., None]
            if w is not None:
                y = y * w.double()
            done = 0
            for a, rot in enumerate(_rots(case)):
                at = (place if st["positions"] is None else st["positions"][a]).double()
                for p in range(rot // 2):
                    i, j = (done, done + pairs) if case["pairs"] == "half" else (2 * done, 2 * done + 1)
                    angle = at * math.exp(-2.0 * p / rot * math.log(case["base"]))
                    z = torch.complex(y[..., i], y[..., j]) * torch.polar(torch.ones_like(angle), angle)[:, None]
                    y[..., i], y[..., j] = z.real, z.imag
                    done += 1
            return y

        k_pool = st["k_pool"].double()
        page, row = st["tables"].long()[seq, place // bs], place % bs
        if case["layout"] == "hnd":
            k_pool[page, :, row] = definition(st["k"], st["k_weight"])
        else:
            k_pool[page, row] = definition(st["k"], st["k_weight"])
        return {"q": definition(st["q"], st["q_weight"]), "k_pool": k_pool, "v_pool": None}
    n = sum(q_len)
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(n, hq, dtype=torch.float64, device="cuda")
    at = 0
    for i, (nq, nk) in enumerate(zip(q_len, kv_len)):
        pages = st["tables"][i, :-(-nk // bs)].long()
        c = torch.arange(nk - nq, nk, device="cuda")[:, None]
        j = torch.arange(nk, device="cuda")[None]
        hidden = (j > c) if case.get("causal", True) else torch.zeros(nq, nk, dtype=torch.bool, device="cuda")
        if case["op"] == "sink":
            hidden = hidden | ((j < c - case["window"]) & (j >= case["sink"]))
        for kh in range(h):
            def head(pool):
                x = pool[pages, kh] if case["layout"] == "hnd" else pool[pages, :, kh]
                return x.reshape(-1, d)[:nk].double()
            k, v = head(st["k_pool"]), head(st["v_pool"])
            for qh in range(kh * hq // h, (kh + 1) * hq // h):
                s = st["q"][at:at + nq, qh].double() @ k.T / math.sqrt(d)
                s[hidden] = -math.inf
                lse[at:at + nq, qh] = torch.logsumexp(s, -1)
                out[at:at + nq, qh] = torch.softmax(s, -1) @ v
        at += nq
    return {"out": out, "lse": lse}
