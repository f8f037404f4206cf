"""Refusals of the feed-forward operators, which are decided on the host before
any launch, their structs' layout and their sizes of scratch. Pointers are
made-up addresses: nothing may touch them."""
import ctypes
import os
import re
import subprocess

import pytest

import shape_adaptive_tile_gb300 as sat

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
AT = 1 << 20  # an aligned address


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sat.build()
    sat.lib()


def _header():
    return open(os.path.join(ROOT, "include", "ffn.h")).read()


def test_exports():
    names = set(re.findall(r"\b((?:ffn|mxfp4)_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", _header(), flags=re.S)))
    assert names == set(sat.FFN_EXPORTS)
    for fn in names:
        assert hasattr(sat.lib(), fn) and callable(getattr(sat, fn))


def test_struct_layouts_match_the_header(tmp_path):
    structs = {"ffn_gated_args": sat.FfnArgs, "ffn_gated_grads": sat.FfnGrads, "mxfp4_args": sat.Mxfp4Args,
               "mxfp4_gemm_args": sat.Mxfp4GemmArgs}
    text = '#include <stddef.h>\n#include <stdio.h>\n#include "ffn.h"\nint main(void) {\n'
    for name, cls in structs.items():
        text += f'printf("{name} %zu\\n", sizeof({name}));\n'
        text += "".join(f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));\n' for f, _ in cls._fields_)
    (tmp_path / "a.c").write_text(text + "return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")], check=True)
    said = dict(line.split() for line in subprocess.run([str(tmp_path / "a")], check=True, capture_output=True,
                                                         text=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(said[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(said[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)
        body = re.search(r"typedef struct \{([^}]*)\} " + name, _header()).group(1)
        assert re.findall(r"(\w+)\s*[,;]", re.sub(r"/\*.*?\*/", "", body, flags=re.S)) == [f for f, _ in cls._fields_]
    for name, value in sat.ACTIVATIONS.items():
        assert re.search(rf"FFN_{name.upper()} = {value}\b", _header())


def test_args_take_names_and_reject_unknown_fields():
    a = sat.FfnArgs(type="fp16", activation="gelu_tanh", x=AT)
    assert a.type == sat.C_TYPES["fp16"] and a.activation == 3 and a.x == AT
    with pytest.raises(AttributeError):
        sat.FfnGrads(dz=AT)
    with pytest.raises(KeyError):
        sat.Mxfp4GemmArgs(activation="tanh")


def _ffn(**kw):
    f = dict(rows=4, width=16, hidden=24, type="bf16", activation="silu", w_by_output=1, x=AT, ldx=16, w=AT, ldw=16, h=AT, ldh=24)
    return sat.FfnArgs(**{**f, **kw})


def _grads(**kw):
    f = dict(dh=AT, lddh=24, dx=AT, lddx=16, dw=AT, lddw=16, dw_type="fp32", workspace=AT, workspace_bytes=1 << 40)
    return sat.FfnGrads(**{**f, **kw})


SHARED = [(-1, dict(rows=-1)), (-1, dict(width=-1)), (-1, dict(hidden=-1)), (-1, dict(rows=1 << 31)), (-1, dict(hidden=1 << 30)),
          (-1, dict(type="fp32")), (-1, dict(type=3)), (-1, dict(activation=5)), (-1, dict(activation=-1)), (-1, dict(x=None)),
          (-1, dict(w=None)), (-1, dict(ldx=15)), (-1, dict(ldw=15)), (-1, dict(w_by_output=0, ldw=47)), (-1, dict(ldx=1 << 31)),
          (-1, dict(preact=AT, ldp=47)), (-3, dict(x=AT + 1)), (-3, dict(w=AT + 1)), (-3, dict(preact=AT + 1, ldp=48))]


@pytest.mark.parametrize("status,bad", SHARED + [
    (-1, dict(h=None)), (-1, dict(ldh=23)), (-3, dict(h=AT + 1)), (-1, dict(ldx=17)), (-1, dict(w=AT + 2)),
    (-1, dict(hidden=20, ldw=40, w_by_output=0)), (-1, dict(ldx=17, workspace=AT, workspace_bytes=8)),
    (-3, dict(ldx=17, workspace=AT + 8, workspace_bytes=1 << 30))])
def test_gated_refuses(status, bad):
    assert sat.ffn_gated(_ffn(**bad)) == status
    assert sat.gemm_last_error()


@pytest.mark.parametrize("status,bad,grads", [(s, b, {}) for s, b in SHARED] + [
    (-1, {}, dict(dh=None)), (-1, {}, dict(lddh=23)), (-1, {}, dict(lddx=15)), (-1, {}, dict(lddw=15)),
    (-1, dict(w_by_output=0, ldw=48), dict(lddw=47)), (-1, {}, dict(dw_type="fp16")), (-1, {}, dict(dw_type=7)),
    (-1, {}, dict(dw_type="bf16", accumulate=1)), (-1, {}, dict(workspace=None)), (-1, {}, dict(workspace_bytes=8)),
    (-3, {}, dict(workspace=AT + 8)), (-3, {}, dict(dh=AT + 1)), (-3, {}, dict(dx=AT + 1)), (-3, {}, dict(dw=AT + 2)),
    (-1, {}, dict(lddw=1 << 31))])
def test_gated_backward_refuses(status, bad, grads):
    assert sat.ffn_gated_backward(_ffn(**bad), _grads(**grads)) == status
    assert sat.gemm_last_error()


def test_workspaces():
    assert sat.ffn_gated_workspace(_ffn()) == 0                         # read as they lie
    assert sat.ffn_gated_workspace(_ffn(rows=0, x=None, ldx=0)) == 0
    assert sat.ffn_gated_workspace(_ffn(ldx=17)) >= 4 * 16 * 2          # a copy of x
    assert sat.ffn_gated_workspace(_ffn(w=AT + 2)) >= 48 * 16 * 2       # of w
    assert sat.ffn_gated_workspace(_ffn(w_by_output=0, ldw=48)) == 0
    assert sat.ffn_gated_workspace(_ffn(w_by_output=0, hidden=20, ldw=40)) >= 16 * 40 * 2
    need = sat.ffn_gated_backward_workspace(_ffn(), _grads())
    assert need >= 4 * 48 * 2
    assert sat.ffn_gated_backward_workspace(_ffn(), _grads(lddh=25)) > need
    assert sat.ffn_gated_backward_workspace(_ffn(preact=AT, ldp=48), _grads(lddh=25)) == need  # only read element by element
    assert sat.ffn_gated_backward_workspace(_ffn(), _grads(dx=None, dw=None)) == 0
    for bad in (dict(rows=-1), dict(type=0)):
        with pytest.raises(sat.GemmError):
            sat.ffn_gated_workspace(_ffn(**bad))
        with pytest.raises(sat.GemmError):
            sat.ffn_gated_backward_workspace(_ffn(**bad), _grads())
    assert sat.mxfp4_scale_bytes(0, 100) == 0 and sat.mxfp4_scale_bytes(1, 1) == 512
    assert sat.mxfp4_scale_bytes(129, 129) == 4 * 512 and sat.mxfp4_scale_bytes(128, 128) == 512
    with pytest.raises(sat.GemmError):
        sat.mxfp4_scale_bytes(-1, 4)


def _quant(**kw):
    f = dict(rows=4, width=40, type="bf16", values=AT, ldv=40, codes=AT, ldc=32, scales=AT)
    return sat.Mxfp4Args(**{**f, **kw})


@pytest.mark.parametrize("status,bad", [
    (-1, dict(rows=-1)), (-1, dict(width=-1)), (-1, dict(width=1 << 31)), (-1, dict(type=3)), (-1, dict(values=None)),
    (-1, dict(codes=None)), (-1, dict(scales=None)), (-1, dict(ldv=39)), (-1, dict(ldc=16)), (-3, dict(ldc=40)),
    (-3, dict(values=AT + 1)), (-3, dict(codes=AT + 8)), (-3, dict(scales=AT + 4))])
def test_quantize_refuses(status, bad):
    for call in (sat.mxfp4_quantize, sat.mxfp4_dequantize):
        assert call(_quant(**bad)) == status
        assert sat.gemm_last_error()


def _gemm(**kw):
    f = dict(rows=4, cols=8, width=40, out_type="bf16", alpha=1.0, a_codes=AT, lda=32, a_scales=AT, b_codes=AT, ldb=32,
             b_scales=AT, out=AT, ldo=8)
    return sat.Mxfp4GemmArgs(**{**f, **kw})


@pytest.mark.parametrize("status,bad", [
    (-1, dict(rows=-1)), (-1, dict(cols=-1)), (-1, dict(width=-1)), (-1, dict(cols=1 << 31)), (-1, dict(out_type=3)),
    (-1, dict(activation=9)), (-1, dict(activation="silu")), (-1, dict(out=None)), (-1, dict(a_codes=None)),
    (-1, dict(a_scales=None)), (-1, dict(b_codes=None)), (-1, dict(b_scales=None)), (-1, dict(up_codes=AT, ldu=32)),
    (-1, dict(lda=16)), (-1, dict(ldb=16)), (-1, dict(up_codes=AT, up_scales=AT, ldu=16)), (-1, dict(ldo=7)),
    (-3, dict(out=AT + 1)), (-3, dict(lda=40)), (-3, dict(ldb=40)), (-3, dict(a_codes=AT + 8)), (-3, dict(b_scales=AT + 8)),
    (-3, dict(up_codes=AT + 4, up_scales=AT, ldu=32)), (-3, dict(up_codes=AT, up_scales=AT, ldu=40))])
def test_gemm_refuses(status, bad):
    assert sat.mxfp4_gemm(_gemm(**bad)) == status
    assert sat.gemm_last_error()


def test_null_structs_and_empty_calls():
    for call in (sat.ffn_gated, sat.mxfp4_quantize, sat.mxfp4_dequantize, sat.mxfp4_gemm):
        assert call(None) == -1
    assert sat.ffn_gated_backward(None, _grads()) == -1 and sat.ffn_gated_backward(_ffn(), None) == -1
    # Nothing to do, whatever the pointers.
    assert sat.ffn_gated(sat.FfnArgs(rows=0, width=4, hidden=4, type="bf16")) == 0
    assert sat.ffn_gated(sat.FfnArgs(rows=3, width=4, hidden=0, type="fp16")) == 0
    assert sat.ffn_gated_backward(_ffn(), _grads(dx=None, dw=None, dh=None)) == 0
    assert sat.mxfp4_quantize(sat.Mxfp4Args(rows=0, width=4)) == 0 and sat.mxfp4_dequantize(sat.Mxfp4Args(rows=4)) == 0
    assert sat.mxfp4_gemm(sat.Mxfp4GemmArgs(rows=0, cols=4, width=4)) == 0
    assert sat.mxfp4_gemm(sat.Mxfp4GemmArgs(rows=3, cols=0, width=4)) == 0


def test_no_device_is_an_error_and_not_a_crash():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert sat.ffn_gated(_ffn()) in (-2, -4) and sat.ffn_gated_backward(_ffn(), _grads()) in (-2, -4)
    assert sat.mxfp4_gemm(_gemm()) in (-2, -4) and sat.mxfp4_quantize(_quant()) == -4


@pytest.mark.parametrize("big", [("rows", "width"), ("rows", "hidden"), ("width", "hidden")])
def test_bytes_that_64_bits_cannot_count_are_refused(big):
    most = (1 << 30) - 9  # (2 hidden columns in one row)
    sizes = {**dict(rows=3, width=5, hidden=7), **{n: most for n in big}}
    f = dict(ldx=2 * most + 1, ldw=2 * most + 1, ldh=2 * most + 1, x=AT + 2, w=AT + 2, w_by_output=0)
    for preact in (None, AT):
        a = _ffn(**{**f, **sizes, "preact": preact, "ldp": 2 * most + 1})
        g = _grads(lddh=2 * most + 1, lddx=2 * most + 1, lddw=2 * most + 1)
        for call in (lambda: sat.ffn_gated_workspace(a), lambda: sat.ffn_gated_backward_workspace(a, g)):
            with pytest.raises(sat.GemmError, match="2\\^56"):
                call()
        assert sat.ffn_gated(a) == sat.ffn_gated_backward(a, g) == -1
