"""Gradients of rows as wide as sizes may be."""
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests.gpu_util import stream

pytestmark = pytest.mark.gpu

WIDTH, LD = (1 << 31) - 9, (1 << 31) - 8


def test_the_last_columns_before_2_to_the_31():
    """One row, one hidden output: dx = dg wg + du wu, dw = (x dg, x du), products of small whole numbers and their sums,
    exactly. The element between the row's end and its stride is left as it is."""
    torch.cuda.set_device(0)
    sat.build()
    w = torch.randint(-4, 5, (2, LD), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    x = torch.randint(-4, 5, (1, LD), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    pre = torch.tensor([[3.0, 5.0]], device="cuda", dtype=torch.bfloat16)
    dh = torch.full((1, 8), 2.0, device="cuda", dtype=torch.bfloat16)
    args = sat.FfnArgs(rows=1, width=WIDTH, hidden=1, type="bf16", activation="none", w_by_output=1, x=x, ldx=LD, w=w, ldw=LD,
                       preact=pre, ldp=2)
    dx, dw = (torch.full((n, LD), float("nan"), device="cuda", dtype=t) for n, t in ((1, torch.bfloat16), (2, torch.float32)))
    grads = sat.FfnGrads(dh=dh, lddh=8, dx=dx, lddx=LD, dw=dw, lddw=LD, dw_type="fp32")
    size = sat.ffn_gated_backward_workspace(args, grads)
    grads.workspace, grads.workspace_bytes = torch.empty(size, device="cuda", dtype=torch.uint8), size
    assert sat.ffn_gated_backward(args, grads, stream()) == 0, sat.gemm_last_error()
    torch.cuda.synchronize()
    assert bool(dx[:, WIDTH:].isnan().all()) and bool(dw[:, WIDTH:].isnan().all())
    dg, du = 10, 6  # dh u, dh g
    step = 1 << 28
    for at in range(0, WIDTH, step):
        c = slice(at, min(at + step, WIDTH))
        assert torch.equal(dx[0, c], dg * w[0, c] + du * w[1, c])
        assert torch.equal(dw[0, c], dg * x[0, c].float()) and torch.equal(dw[1, c], du * x[0, c].float())
