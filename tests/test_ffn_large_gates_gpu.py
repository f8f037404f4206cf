"""Gradients where the gate is far from 0: slopes of 0 and 1, whatever the
gate's square is."""
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests.gpu_util import stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [64, 300])
@pytest.mark.parametrize("recompute", [False, True])
@pytest.mark.parametrize("activation", ["silu", "gelu", "gelu_tanh", "relu"])
def test_slopes_far_from_0(activation, recompute, rows):
    """x = (g, 1), weights that pick them, dh = 1: dx = (a'(g), a(g)) = (1, g) on the right and 0 on the left, exactly."""
    torch.cuda.set_device(0)
    sat.build()
    size = 2.0**torch.linspace(8, 126, rows // 2).floor().double()
    g = torch.cat([size, -size]).cuda().bfloat16()
    x, w = torch.zeros(rows, 8, device="cuda", dtype=torch.bfloat16), torch.zeros(2, 8, device="cuda", dtype=torch.bfloat16)
    x[:, 0], x[:, 1], w[0, 0], w[1, 1] = g, 1, 1, 1
    pre, dh, dx = x[:, :2].contiguous(), torch.ones_like(x), torch.full_like(x, float("nan"))
    args = sat.FfnArgs(rows=rows, width=8, hidden=1, type="bf16", activation=activation, w_by_output=1, x=x, ldx=8, w=w, ldw=8,
                       **({} if recompute else dict(preact=pre, ldp=2)))
    grads = sat.FfnGrads(dh=dh, lddh=8, dx=dx, lddx=8)
    size = sat.ffn_gated_backward_workspace(args, grads)
    grads.workspace, grads.workspace_bytes = torch.empty(size, device="cuda", dtype=torch.uint8), size
    assert sat.ffn_gated_backward(args, grads, stream()) == 0, sat.gemm_last_error()
    torch.cuda.synchronize()
    assert torch.equal(dx[:, 0].float(), (g > 0).float())
    assert torch.equal(dx[:, 1], torch.where(g > 0, g, torch.zeros_like(g)))
