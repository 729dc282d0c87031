"""Windows with first positions on the host: what is refused, before any CUDA call."""
import pytest

import autoregressive_video_diffusion_gb300 as dcp
from tests.test_serving_host import B, _attend, _batch, _pool, no_gpu


@no_gpu
@pytest.mark.parametrize("causal,window,sink", [(1, -1, 4), (0, -1, 1), (1, 100, -1), (0, 100, 4)])
def test_refusals(causal, window, sink):
    cfg = dcp.DcpAttnConfigC(0.1, causal, window, sink)
    assert _attend(cfg=cfg) == dcp.DCP_EINVAL
    assert dcp.lib.dcp_attention_workspace_size(B(_pool()), B(_batch()), B(cfg), 40) == 0


def test_the_sink_reaches_the_struct():
    c = dcp.AttnConfig(0.5, True, 7, 3).c(64)
    assert (c.scale, c.causal, c.window, c.sink) == (0.5, 1, 7, 3)
    assert dcp.AttnConfig().c(64).sink == 0
