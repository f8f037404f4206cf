"""A teacher's NaN among the entries that are present makes its row NaN, by
itself or beside others, as the formula has it; absent entries do not matter."""
import numpy as np
import pytest
import torch

import shape_adaptive_tile_gb300 as sat
from tests.test_distill_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)
    sat.build()
    sat.lib()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("k", [1, 20, 300])
@pytest.mark.parametrize("rows,vocab", [(6, 1000), (90, 700), (6, 60000), (6, 280000)])
def test_rows_of_nan(rows, vocab, k, dtype):
    c = Case(5, rows, vocab, k, dtype, "bf16")
    good = c.run()
    c.teacher[0] = float("nan")           # all of them
    c.teacher[1, k - 1] = float("nan")    # the last one
    c.teacher[2] = float("nan")           # all that are present
    c.ids[2, :k // 2] = -1
    c.teacher[3] = float("-inf")          # none is present
    c.teacher[3, 0] = float("nan")
    c.ids[3, 0] = -1
    loss, lse, d, d2, alone = c.run()
    for r in (0, 1, 2):
        assert bool(loss[r].isnan()) and bool(alone[r].isnan())
        assert bool(d[r].isnan().all()) and bool(d2[r].isnan().all())
        assert lse[r] == good[1][r]  # of the student's alone
    assert loss[3] == 0 and lse[3] == 0 and bool((d[3] == 0).all()) and bool((d2[3] == 0).all())
    for a, b in zip((loss, lse, d, d2, alone), good):
        assert torch.equal(a[4:], b[4:])
    assert np.isfinite(good[0].cpu().numpy()).all()
