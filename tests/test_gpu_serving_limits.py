"""What the attention's contract says of its bounds and of host threads."""
import os
import subprocess
import sys
import textwrap

import pytest

import autoregressive_video_diffusion_gb300 as dcp
from tests.serving import NHD, Cache, check_attention
from tests.test_gpu_serving import attend

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

LONGER = [
    # dtype, hq, h, q_lens, kv_lens: all lengths may exceed the bound that the work is divided by
    ("bf16", 8, 2, [1] * 6, [3000, 1, 700, 64, 5000, 0]),
    ("bf16", 4, 2, [1], [9000]),
    ("bf16", 16, 2, [7, 1], [2000, 900]),
    ("bf16", 4, 2, [200, 30], [3000, 500]),
    ("f32", 4, 2, [1, 1, 1], [900, 33, 400]),
    ("f32", 4, 2, [100, 9], [1500, 60]),
]


@pytest.mark.parametrize("case", LONGER, ids=[str(i) for i in range(len(LONGER))])
@pytest.mark.parametrize("bound", [0, 1, 130, 1000])
@pytest.mark.parametrize("window", [-1, 333])
def test_lengths_above_max_kv(gpu, case, bound, window):
    dtype, hq, h, q_lens, kv_lens = case
    c = Cache(dtype, NHD, h, 64, 16, q_lens, kv_lens, seed=41).fill()
    q = c.normal(c.start[-1], hq, 64)
    out, lse = attend(c, q, True, window, batch=c.batch(max_kv=bound))
    assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
    check_attention(c, q, out, lse, 0.125, True, window)


CHILD = textwrap.dedent('''
    import threading
    import torch
    import autoregressive_video_diffusion_gb300 as dcp
    from tests.serving import HND, Cache, check_attention

    cases = [("bf16", [300], [2000], 4, 2, 128), ("bf16", [300], [2000], 4, 2, 64), ("bf16", [1, 1], [700, 90], 8, 2, 128),
             ("f32", [100], [600], 4, 2, 64), ("f32", [1], [5000], 4, 2, 64), ("bf16", [9], [3000], 8, 2, 64)]
    jobs = []
    for i, (t, ql, kl, hq, h, d) in enumerate(cases):
        c = Cache(t, HND, h, d, 16, ql, kl, seed=i).fill()
        q = c.normal(c.start[-1], hq, d)
        cfg = dcp.AttnConfig()
        ws = dcp.new_workspace(dcp.dcp_attention_workspace_size(c.pool(), c.batch(), cfg, hq))
        jobs.append((c, q, torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), cfg, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(jobs)), []

    def run(c, q, out, lse, cfg, ws, stream):
        try:
            pool, batch = c.pool(), c.batch()
            start.wait()
            for _ in range(20):
                dcp.dcp_paged_attention(pool, batch, cfg, q, out, lse, ws, stream=stream)
            stream.synchronize()
        except Exception as e:  # reported by the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=run, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for c, q, out, lse, _, _, _ in jobs:
        assert dcp.dcp_get_status(c.status) == dcp.DCP_OK
        check_attention(c, q, out, lse, c.d ** -0.5, True, -1)
    print("threads ok", len(jobs))
''')


def test_host_threads_with_the_attention(gpu):
    """Each on its own cache, workspace and stream, the first launches of every kernel at the same time."""
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "threads ok 6" in r.stdout
