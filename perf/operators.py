"""The serving operators around the paged cache, as they are called: the cases that are measured, their inputs, one
pass in plain torch operations or through the library, and the work that a pass cannot do without.

Three operators, chosen by a case's "op":
  append   rotary turn of the new tokens' q and k, and k, v written to the cache's pages
  attend   attention of the new tokens of a ragged batch over the paged cache
  pages    copying, forking, compacting and freeing pages in every layer's pool
"""
import json
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases
def _attend(name, **kw):
    c = dict(name=name, op="attend", dtype="bf16", layout="hnd", hq=40, h=8, d=128, bs=16, seqs=1, q_lo=1, q_hi=1,
             kv_lo=1024, kv_hi=1024, causal=True, window=-1, lens=1)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(name=name, op="append", dtype="bf16", layout="hnd", hq=40, h=8, d=128, bs=16, seqs=1, q_lo=1, q_hi=1,
             kv_lo=1024, kv_hi=1024, rot=128, pairs="half", base=10000.0, scaling="none", factor=1.0, far=0, lens=1)
    c.update(kw)
    return c


def _pages(name, kind, **kw):
    c = dict(name=name, op="pages", kind=kind, dtype="bf16", layers=40, h=8, d=128, bs=16, blocks=1024, seqs=8,
             stride=64, children=0, moves=0, fill=0.5, lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # one session's next token over a short cache: nothing but latency
        _attend("attend token short", kv_lo=1531, kv_hi=1531),
        # a serving batch's next tokens: ragged lengths, position-major pages
        _attend("attend tokens batch", layout="nhd", seqs=48, kv_lo=200, kv_hi=16000, bs=32, lens=2),
        # one video chunk (4 frames of 30 x 52 tokens) denoised against sink, kept history, window and itself
        _attend("attend video chunk", q_lo=6240, q_hi=6240, kv_lo=25907, kv_hi=25907, bs=32, causal=False),
        # prompts' chunks behind what their caches hold: causal, ragged
        _attend("attend prompt chunks", hq=32, layout="nhd", seqs=6, q_lo=130, q_hi=2048, kv_lo=2100, kv_hi=12000,
                lens=3),
        # heads of 80 over pages of 24 positions, sliding window: sizes that fill no tile
        _attend("attend window odd", hq=12, h=4, d=80, bs=24, seqs=5, q_lo=33, q_hi=700, kv_lo=701, kv_hi=5000,
                window=513, lens=4),
        # the fp32 cache
        _attend("attend fp32", dtype="f32", hq=8, h=8, d=64, seqs=3, q_lo=100, q_hi=513, kv_lo=513, kv_hi=3001, lens=5),
        # a batch's next tokens enter the cache
        _append("append tokens", seqs=32, kv_lo=64, kv_hi=2048, layout="nhd"),
        # a video chunk enters its ring slot: the leading 22 interleaved pairs carry the frame
        _append("append video chunk", q_lo=6240, q_hi=6240, kv_lo=6240, kv_hi=6240, h=40, rot=44, pairs="interleaved",
                bs=32, far=240),
        # prompts far into a long context, frequencies scaled by parts, fp32 cache
        _append("append far fp32", dtype="f32", hq=32, d=96, rot=64, seqs=5, q_lo=17, q_hi=900, kv_lo=900, kv_hi=4001,
                scaling="parts", factor=8.0, far=1000000, bs=24, base=500000.0),
        # sessions branch: every child shares its parent's full pages and gets its own copy of the last one
        _pages("pages fork", "fork", seqs=8, children=32, blocks=1024, stride=48, fill=0.35),
        # a pool half full of scattered pages is packed to its front
        _pages("pages compact", "compact", blocks=2048, seqs=32, stride=60, fill=0.5),
        # branches are dropped
        _pages("pages free", "free", layers=1, blocks=16384, seqs=64, stride=128, fill=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "pages"])
    lens = rng.randrange(1 << 30)
    if op == "pages":
        kind = rng.choice(["copy", "fork", "compact", "free"])
        h, d, dtype = rng.choice([1, 2, 8, 40]), rng.choice([32, 64, 96, 128]), rng.choice(["bf16", "f32"])
        bs, layers = rng.choice([4, 16, 24, 32]), _log(rng, 1, 40)
        blocks = _log(rng, 64, 4096)
        most = 6 << 30  # bytes of one pool
        blocks = max(48, min(blocks, most // (layers * h * bs * d * ES[dtype])))
        seqs = _log(rng, 2, min(64, blocks // 16))
        return dict(op=op, kind=kind, dtype=dtype, layers=layers, h=h, d=d, bs=bs, blocks=blocks, seqs=seqs,
                    stride=rng.randint(2, 160), children=rng.randint(1, max(1, min(40, blocks // 8))),
                    moves=rng.randint(1, blocks // 3), fill=rng.uniform(0.1, 0.5), lens=lens)
    h = rng.choice([1, 2, 4, 8])
    hq = h * rng.choice([1, 2, 4, 5, 7, 8])
    d = rng.choice([32, 40, 64, 80, 96, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    bs = rng.choice([5, 8, 16, 16, 24, 32, 64, 100, 128, 240])
    layout = rng.choice(["hnd", "nhd"])
    seqs = _log(rng, 1, 64)
    if op == "append":
        q_hi = _log(rng, 1, max(1, 8000 // seqs))
        scaling = rng.choice(["none", "linear", "base", "parts"])
        return dict(op=op, dtype=dtype, layout=layout, hq=hq, h=h, d=d, bs=bs, seqs=seqs, q_lo=rng.randint(1, q_hi),
                    q_hi=q_hi, kv_lo=q_hi, kv_hi=q_hi + _log(rng, 1, 4000), rot=2 * rng.randint(1, d // 2),
                    pairs=rng.choice(["half", "interleaved"]), base=rng.choice([10000.0, 500000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                    far=rng.choice([0, 0, 240, 100000, 1000000]), lens=lens)
    q_hi = rng.choice([1, rng.randint(2, 9), _log(rng, 10, 4000)])
    room = 2.0e9 if dtype == "bf16" else 2.5e8  # scores of a pass
    kv_hi = q_hi + _log(rng, 1, 30000)
    kv_hi = max(q_hi, min(kv_hi, int(room / (q_hi * hq))))
    seqs = max(1, min(seqs, int(room / (q_hi * hq * kv_hi)), int(1.2e9 / (kv_hi * h * d))))
    causal = rng.random() < 0.7
    return dict(op=op, dtype=dtype, layout=layout, hq=hq, h=h, d=d, bs=bs, seqs=seqs, q_lo=rng.randint(1, q_hi),
                q_hi=q_hi, kv_lo=q_hi, kv_hi=kv_hi, causal=causal,
                window=_log(rng, 1, kv_hi) if causal and rng.random() < 0.4 else -1, lens=lens)


def _lens(case):
    """New tokens and cache lengths of each sequence, from the case alone."""
    r = random.Random(case["lens"])
    q = [case["q_hi"] if i == 0 else r.randint(case["q_lo"], case["q_hi"]) for i in range(case["seqs"])]
    kv = [case["kv_hi"] if i == 0 else r.randint(case["kv_lo"], case["kv_hi"]) for i in range(case["seqs"])]
    return q, kv


def _table_lens(case):
    """Positions of each sequence of a page case: together about `fill` of the pool, at most the table's row."""
    r = random.Random(case["lens"])
    most = min(case["stride"], max(1, int(case["fill"] * case["blocks"]) // case["seqs"]))
    pages = [most if i == 0 else r.randint(max(1, most // 3), most) for i in range(case["seqs"])]
    return [(n - 1) * case["bs"] + r.randint(1, case["bs"]) for n in pages]


def _freed(case):
    return (case["seqs"] + 1) // 2


def _fork_plan(case):
    """Positions of the parents, and the parent of each child."""
    r = random.Random(case["lens"] + 1)
    lens = _table_lens(case)
    return lens, [r.randrange(case["seqs"]) for _ in range(case["children"])]


# ------------------------------------------------------------------------------------------------ inputs
def _pool_shape(case, n_blocks):
    h, bs, d = case["h"], case["bs"], case["d"]
    return (n_blocks, h, bs, d) if case["layout"] == "hnd" else (n_blocks, bs, h, d)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape):
        x = torch.empty(shape, dtype=dt, device="cuda")
        return x.normal_(generator=g)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    st = {"case": case}
    if case["op"] == "pages":
        lens = _table_lens(case)
        bs, nb, stride = case["bs"], case["blocks"], case["stride"]
        st["k"] = normal(case["layers"], nb, case["h"], bs, case["d"])
        st["v"] = normal(case["layers"], nb, case["h"], bs, case["d"])
        perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        tables = torch.full((case["seqs"], stride), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(lens):
            pages = -(-n // bs)
            tables[i, :pages] = perm[at:at + pages]
            at += pages
            if i:  # a branch: it shares its first pages with the sequence before it
                common = min(pages, -(-lens[i - 1] // bs)) // 3
                tables[i, :common] = tables[i - 1, :common]
        st["tables"], st["lens"] = tables, ints(lens)
        used = torch.where(tables >= 0, tables, nb).flatten().long()
        st["ref"] = torch.zeros(nb + 1, dtype=torch.int32, device="cuda").index_add_(
            0, used, torch.ones_like(used, dtype=torch.int32))[:nb].contiguous()
        st["ref_out"] = torch.zeros_like(st["ref"])
        if case["kind"] == "free":  # half of the branches are dropped, the others live on
            st["tables"] = tables[:_freed(case)].clone()
        rows = case["children"] if case["kind"] == "fork" else st["tables"].shape[0]
        st["tables_out"] = torch.zeros((rows, stride), dtype=torch.int32, device="cuda")
        st["n_live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["kind"] == "fork":
            st["parent"] = ints(_fork_plan(case)[1])
        if case["kind"] == "copy":
            pages = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
            st["src"], st["dst"] = pages[:case["moves"]].clone(), pages[-case["moves"]:].clone()
        if own:
            import autoregressive_video_diffusion_gb300 as dcp
            st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
            st["pool"] = dcp.PagePool(st["k"], st["v"], bs, st["status"])
            st["ws"] = dcp.new_workspace(dcp.dcp_pages_workspace_size(st["pool"], rows, stride))
        return st

    q_len, kv_len = _lens(case)
    bs, n = case["bs"], sum(q_len)
    stride = -(-max(kv_len) // bs)
    n_blocks = sum(-(-x // bs) for x in kv_len) + 3
    st["k_pool"], st["v_pool"] = normal(*_pool_shape(case, n_blocks)), normal(*_pool_shape(case, n_blocks))
    perm = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(q_len), stride), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, x in enumerate(kv_len):
        tables[i, :-(-x // bs)] = perm[at:at + -(-x // bs)]
        at += -(-x // bs)
    start = [0]
    for x in q_len:
        start.append(start[-1] + x)
    st["tables"], st["kv_len"], st["q_start"] = tables, ints(kv_len), ints(start)
    st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        qkv = normal(n, case["hq"] + 2 * case["h"], case["d"])
        st["q"], st["k"], st["v"] = qkv.split([case["hq"], case["h"], case["h"]], dim=1)
        st["q_out"] = torch.empty(n, case["hq"], case["d"], dtype=dt, device="cuda")
        if case["far"]:
            st["positions"] = torch.randint(case["far"] // 2, case["far"], (n,), generator=g, device="cuda").to(
                torch.int32)
        else:
            st["positions"] = None
    else:
        st["q"] = normal(n, case["hq"], case["d"])
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(n, case["hq"], dtype=torch.float32, device="cuda")
    if own:
        import autoregressive_video_diffusion_gb300 as dcp
        layout = dcp.DCP_PAGED_HND if case["layout"] == "hnd" else dcp.DCP_PAGED_NHD
        st["pool"] = dcp.KVPool(st["k_pool"], st["v_pool"], layout)
        st["batch"] = dcp.SeqBatch(st["q_start"], st["tables"], st["kv_len"], st["status"], total_q=n,
                                   max_q=max(q_len), max_kv=max(kv_len))
        if case["op"] == "append":
            st["plan"] = dcp.dcp_rope_plan(dcp.RopeConfig(
                rot_dim=case["rot"], pair_layout=dcp.DCP_ROPE_HALF if case["pairs"] == "half"
                else dcp.DCP_ROPE_INTERLEAVED, base=case["base"], scaling={
                    "none": dcp.DCP_ROPE_PLAIN, "linear": dcp.DCP_ROPE_LINEAR, "base": dcp.DCP_ROPE_BASE,
                    "parts": dcp.DCP_ROPE_PARTS}[case["scaling"]], factor=case["factor"], orig_len=4096.0,
                amplitude=_amplitude(case)))
        else:
            st["cfg"] = dcp.AttnConfig(causal=case["causal"], window=case["window"])
            st["ws"] = dcp.new_workspace(dcp.dcp_attention_workspace_size(st["pool"], st["batch"], st["cfg"],
                                                                          case["hq"]))
    return st


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


# ------------------------------------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "pages": _own_pages}[op](st)
    return {"append": _plain_append, "attend": _plain_attend, "pages": _plain_pages}[op](st)


def _own_append(st):
    import autoregressive_video_diffusion_gb300 as dcp
    dcp.dcp_rope_append(st["pool"], st["batch"], st["plan"], st["q"], st["k"], st["v"], st["positions"], st["q_out"])
    return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _own_attend(st):
    import autoregressive_video_diffusion_gb300 as dcp
    dcp.dcp_paged_attention(st["pool"], st["batch"], st["cfg"], st["q"], st["out"], st["lse"], st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_pages(st):
    import autoregressive_video_diffusion_gb300 as dcp
    kind = st["case"]["kind"]
    if kind == "copy":
        dcp.dcp_pages_copy(st["pool"], st["src"], st["dst"])
        return {"k": st["k"], "v": st["v"]}
    if kind == "fork":
        dcp.dcp_pages_fork(st["pool"], st["tables"], st["lens"], st["parent"], None, None, st["ref"],
                           st["tables_out"], st["ref_out"], st["ws"])
        return {"k": st["k"], "v": st["v"], "tables": st["tables_out"], "ref": st["ref_out"]}
    if kind == "compact":
        dcp.dcp_pages_compact(st["pool"], st["tables"], st["ref"], st["tables_out"], st["ref_out"], st["n_live"],
                              st["ws"])
        return {"k": st["k"], "v": st["v"], "tables": st["tables_out"], "ref": st["ref_out"], "n": st["n_live"]}
    dcp.dcp_pages_free(st["pool"], st["tables"], st["ref"], st["tables_out"], st["ref_out"])
    return {"tables": st["tables_out"], "ref": st["ref_out"]}


def _theta(case):
    """Angle a position of each rotary pair, 64 bits."""
    rot, f = case["rot"], case["factor"]
    p = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    base = case["base"]
    if case["scaling"] == "base" and rot > 2:
        base = base * f ** (rot / (rot - 2))
    theta = base ** (-2 * p / rot)
    if case["scaling"] == "linear":
        theta = theta / f
    if case["scaling"] == "parts":
        g = ((4096.0 * theta / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        theta = theta * (g + (1 - g) / f)
    return theta


def _rows(st):
    """Sequence, cache position and page row of every new token."""
    n = st["q"].shape[0]
    i = torch.arange(n, device="cuda")
    seq = torch.searchsorted(st["q_start"][1:].long(), i, right=True)
    start, end = st["q_start"].long()[seq], st["q_start"].long()[seq + 1]
    pos = st["kv_len"].long()[seq] - (end - start) + (i - start)
    bs = st["case"]["bs"]
    return seq, pos, st["tables"][seq, pos // bs].long(), pos % bs


def _plain_append(st):
    case = st["case"]
    _, pos, block, row = _rows(st)
    at = pos if st["positions"] is None else st["positions"]
    angle = at.double()[:, None] * _theta(case)
    amp = _amplitude(case)
    cos, sin = (angle.cos() * amp).float()[:, None], (angle.sin() * amp).float()[:, None]
    rot = case["rot"]

    def turn(x):
        y = x.float()
        if case["pairs"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat([a * cos - b * sin, a * sin + b * cos, y[..., rot:]], -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), y[..., rot:]], -1)
        return z.to(x.dtype)

    q, k = turn(st["q"]), turn(st["k"])
    if case["layout"] == "hnd":
        st["k_pool"][block, :, row] = k
        st["v_pool"][block, :, row] = st["v"]
    else:
        st["k_pool"][block, row] = k
        st["v_pool"][block, row] = st["v"]
    return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _plain_attend(st):
    case = st["case"]
    hq, h, d, bs = case["hq"], case["h"], case["d"], case["bs"]
    q_len, kv_len = (torch.diff(st["q_start"]).long(), st["kv_len"].long())
    max_q, max_kv = case["q_hi"], case["kv_hi"]
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
    c = kv_len[:, None] - q_len[:, None] + i                                             # [b, max_q]
    seen = (j < kv_len[:, None])[:, None].expand(b, max_q, max_kv)
    if case["causal"]:
        seen = seen & (j <= c[..., None])
    if case["window"] >= 0:
        seen = seen & (j >= c[..., None] - case["window"])
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
    seq, place = torch.searchsorted(st["q_start"][1:].long(), torch.arange(n, device="cuda"), right=True), None
    place = torch.arange(n, device="cuda") - st["q_start"].long()[seq]
    return {"out": out[seq, place].to(st["q"].dtype), "lse": lse[seq, place].contiguous()}


def _plain_pages(st):
    case, k, v = st["case"], st["k"], st["v"]
    if case["kind"] == "copy":
        src, dst = st["src"].long(), st["dst"].long()
        k[:, dst] = k[:, src]
        v[:, dst] = v[:, src]
        return {"k": k, "v": v}
    ref, nb, bs = st["ref"], case["blocks"], case["bs"]
    block = torch.arange(nb, device="cuda")
    if case["kind"] == "free":
        gone = torch.zeros(nb + 1, dtype=torch.int32, device="cuda")
        used = torch.where(st["tables"] >= 0, st["tables"], nb).flatten().long()
        gone.index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
        return {"tables": torch.full_like(st["tables"], -1), "ref": ref - gone[:nb]}
    if case["kind"] == "compact":
        live = ref > 0
        n_live = live.sum()
        src = torch.nonzero(live & (block >= n_live)).flatten()
        dst = torch.nonzero(~live & (block < n_live)).flatten()
        k[:, dst] = k[:, src]
        v[:, dst] = v[:, src]
        to, ref = block.clone(), ref.clone()
        to[src] = dst
        ref[dst] = ref[src]
        ref[src] = 0
        tables = torch.where(st["tables"] >= 0, to[st["tables"].clamp(min=0).long()], -1).to(torch.int32)
        return {"k": k, "v": v, "tables": tables, "ref": ref, "n": n_live.to(torch.int32).view(1)}
    rows = st["tables"][st["parent"].long()]
    length = st["lens"][st["parent"].long()].long()[:, None]
    j = torch.arange(case["stride"], device="cuda")
    share, fresh = j < length // bs, (j >= length // bs) & (j < (length + bs - 1) // bs)
    free = torch.sort((ref > 0).to(torch.int32), stable=True).indices
    dst = free[(fresh.flatten().cumsum(0) - 1).clamp(min=0)].view(fresh.shape)
    tables = torch.where(share, rows, torch.where(fresh, dst.to(torch.int32), -1))
    counts = torch.zeros(nb + 1, dtype=torch.int32, device="cuda")
    used = torch.where(tables >= 0, tables, nb).flatten().long()
    counts.index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
    at, to = rows[fresh].long(), dst[fresh]
    k[:, to] = k[:, at]
    v[:, to] = v[:, at]
    return {"k": k, "v": v, "tables": tables, "ref": ref + counts[:nb]}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    es = ES[case["dtype"]]
    if case["op"] == "append":
        n = sum(_lens(case)[0])
        heads = case["hq"] + 2 * case["h"]
        return {"bytes": 2 * n * heads * case["d"] * es + 4 * n,
                "flops": 6 * n * (case["hq"] + case["h"]) * (case["rot"] // 2)}
    if case["op"] == "attend":
        q_len, kv_len = _lens(case)
        pairs = keys = 0
        for nq, nk in zip(q_len, kv_len):
            if not case["causal"]:
                pairs, keys = pairs + nq * nk, keys + nk
                continue
            w = case["window"] if case["window"] >= 0 else nk
            first, last = nk - nq, nk - 1                  # cache positions of the first and last new token
            full = max(0, last - max(first, w) + 1)        # rows that see w + 1 keys
            short = nq - full                              # the others see c + 1 keys
            pairs += full * (w + 1) + short * (first + 1) + short * (short - 1) // 2
            keys += nk - max(0, first - w)
        n, d = sum(q_len), case["d"]
        return {"bytes": 2 * n * case["hq"] * d * es + 4 * n * case["hq"] + 2 * keys * case["h"] * d * es
                + 4 * sum(-(-x // case["bs"]) for x in kv_len), "flops": 4 * pairs * case["hq"] * d}
    page = case["h"] * case["bs"] * case["d"] * es
    nb, lens, bs = case["blocks"], _table_lens(case), case["bs"]
    meta = 4 * 2 * (nb + case["seqs"] * case["stride"])
    if case["kind"] == "copy":
        moved, meta = case["moves"], 8 * case["moves"]
    elif case["kind"] == "free":
        moved, meta = 0, 4 * 2 * (nb + _freed(case) * case["stride"])
    elif case["kind"] == "compact":
        pages = [-(-x // bs) for x in lens]
        live = sum(p - (min(p, pages[i - 1]) // 3 if i else 0) for i, p in enumerate(pages))
        moved = live * (nb - live) // nb                   # pages are scattered evenly
    else:
        lens, parents = _fork_plan(case)
        moved = sum(1 for p in parents if lens[p] % bs)
        meta = 4 * (2 * nb + (case["seqs"] + case["children"]) * case["stride"])
    return {"bytes": 2 * 2 * case["layers"] * moved * page + meta, "flops": 0}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, a sequence and a head at a time."""
    if case["op"] == "pages":
        return None  # whole pages and whole numbers: there is nothing to round
    st = prepare(case, seed)
    q_len, kv_len = _lens(case)
    hq, h, d, bs = case["hq"], case["h"], case["d"], case["bs"]
    if case["op"] == "append":
        rot, half = case["rot"], case["rot"] // 2
        freq = []
        for p in range(half):
            base = case["base"]
            if case["scaling"] == "base" and rot > 2:
                base *= case["factor"] ** (rot / (rot - 2.0))
            t = math.exp(-2.0 * p / rot * math.log(base))
            if case["scaling"] == "linear":
                t /= case["factor"]
            elif case["scaling"] == "parts":
                turns = 4096.0 * t / (2 * math.pi)
                ramp = min(1.0, max(0.0, (turns - 1.0) / 31.0))
                t = (1 - ramp) * t / case["factor"] + ramp * t
            freq.append(t)
        place = torch.cat([torch.arange(nk - nq, nk) for nq, nk in zip(q_len, kv_len)]).cuda()
        seq = torch.cat([torch.full((nq,), i) for i, nq in enumerate(q_len)]).cuda()
        x = (place if st["positions"] is None else st["positions"]).double()
        z = torch.polar(torch.full((x.numel(), half), _amplitude(case), dtype=torch.float64, device="cuda"),
                        x[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))[:, None]
        first = torch.arange(half, device="cuda") if case["pairs"] == "half" else torch.arange(0, rot, 2, device="cuda")
        second = first + (half if case["pairs"] == "half" else 1)

        def turned(y):
            y = y.double()
            c = torch.complex(y[..., first], y[..., second]) * z
            y[..., first], y[..., second] = c.real, c.imag
            return y

        k_pool = st["k_pool"].double()
        page = st["tables"].long()[seq, place // bs]
        if case["layout"] == "hnd":
            k_pool[page, :, place % bs] = turned(st["k"])
        else:
            k_pool[page, place % bs] = turned(st["k"])
        return {"q": turned(st["q"]), "k_pool": k_pool, "v_pool": None}
    w = work(case)
    if w["flops"] > 5e12:
        return None
    n = sum(q_len)
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(n, hq, dtype=torch.float64, device="cuda")
    at = 0
    for i, (nq, nk) in enumerate(zip(q_len, kv_len)):
        pages = st["tables"][i, :-(-nk // bs)].long()
        c = torch.arange(nk - nq, nk, device="cuda")[:, None]
        j = torch.arange(nk, device="cuda")[None]
        hidden = (j > c) if case["causal"] else torch.zeros(nq, nk, dtype=torch.bool, device="cuda")
        if case["window"] >= 0:
            hidden = hidden | (j < c - case["window"])
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
