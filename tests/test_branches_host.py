"""What the prune step on a cache with shared pages refuses on the host, before any CUDA call."""
import ctypes

import pytest

import autoregressive_video_diffusion_gb300 as dcp
from tests.conftest import has_gpu

FAKE = 1 << 40  # aligned, never dereferenced


@pytest.mark.skipif(has_gpu(), reason="refused calls use fake device addresses")
def test_shared_prune_step_refusals():
    cfg = dcp.Config(max_frames=256).c()
    c = dcp.DcpPagedCacheC(FAKE, FAKE + (1 << 36), 2, 2, 128, dcp.DCP_BF16, 16, dcp.DCP_PAGED_HND, 4096, 6240,
                           FAKE + (2 << 36), FAKE + (3 << 36), FAKE + (4 << 36), FAKE + (5 << 36), FAKE + (6 << 36))
    n = dcp.lib.dcp_paged_workspace_size(ctypes.byref(c), ctypes.byref(cfg))
    assert n > 0

    def step(ref, slot=0):
        return dcp.lib.dcp_paged_prune_step_shared(ctypes.byref(c), ctypes.byref(cfg), ref, FAKE, FAKE, 64, slot, 4, 20,
                                                   20, None, None, None, FAKE + (7 << 36), n, None)

    assert step(None) == dcp.DCP_EINVAL and step(FAKE + 2) == dcp.DCP_EINVAL
    assert step(FAKE, slot=9) == dcp.DCP_EINVAL
