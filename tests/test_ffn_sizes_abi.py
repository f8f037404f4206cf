"""Sizes of which 64 bits cannot count twice, or a product: refused on the host
before anything is computed from them."""
import pytest

import shape_adaptive_tile_gb300 as sat

AT = 1 << 20  # an aligned address; nothing may touch it
HUGE = [1 << 30, 1 << 31, 1 << 61, 1 << 62, (1 << 62) + 1, 3 << 61, (1 << 63) - 1]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sat.build()
    sat.lib()


@pytest.mark.parametrize("rows", [0, 4])
@pytest.mark.parametrize("preact", [None, AT])
@pytest.mark.parametrize("by_output", [1, 0])
@pytest.mark.parametrize("hidden", HUGE)
def test_hidden(hidden, by_output, preact, rows):
    f = dict(rows=rows, width=16, hidden=hidden, type="bf16", activation="silu", w_by_output=by_output, x=AT, ldx=16, w=AT, ldw=1 << 30,
             h=AT, ldh=1 << 30, preact=preact, ldp=1 << 30)
    a = sat.FfnArgs(**f)
    g = sat.FfnGrads(dh=AT, lddh=1 << 30, dx=AT, lddx=16, dw=AT, lddw=1 << 30, dw_type="fp32", workspace=AT, workspace_bytes=1 << 62)
    for call in (lambda: sat.ffn_gated_workspace(a), lambda: sat.ffn_gated_backward_workspace(a, g)):
        with pytest.raises(sat.GemmError):
            call()
    assert sat.ffn_gated(a) == -1 and sat.ffn_gated_backward(a, g) == -1


@pytest.mark.parametrize("n", [1 << 31, 1 << 62, (1 << 63) - 1])
def test_others(n):
    for size in ("rows", "width"):
        a = sat.FfnArgs(**{**dict(rows=4, width=16, hidden=8, type="bf16", x=AT, ldx=16, w=AT, ldw=16, w_by_output=1, h=AT, ldh=8), size: n})
        with pytest.raises(sat.GemmError):
            sat.ffn_gated_workspace(a)
        assert sat.ffn_gated(a) == -1
    for sizes in ((n, 4), (4, n)):
        with pytest.raises(sat.GemmError):
            sat.mxfp4_scale_bytes(*sizes)
