"""Refusals of the language-model row operators, which are decided on the host
before any launch, and their structs' layout. Pointers are made-up addresses:
nothing may touch them."""
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


def test_struct_layouts_match_the_header(tmp_path):
    structs = {"rowop_block_norm_args": sat.BlockNormArgs, "rowop_block_norm_grads": sat.BlockNormGrads,
               "rowop_distill_args": sat.DistillArgs, "rowop_verify_args": sat.VerifyArgs}
    text = '#include <stddef.h>\n#include <stdio.h>\n#include "rowops.h"\nint main(void) {\n'
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
    header = open(os.path.join(ROOT, "include", "rowops.h")).read()
    for name, cls in structs.items():
        body = re.search(r"typedef struct \{([^}]*)\} " + name, header).group(1)
        fields = re.findall(r"(\w+)\s*[,;]", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
        assert fields == [f for f, _ in cls._fields_]


def test_args_take_names_and_reject_unknown_fields():
    a = sat.BlockNormArgs(block_type="bf16", post_norm="layer", x=AT)
    assert a.block_type == sat.C_TYPES["bf16"] and a.post_norm == 2 and a.x == AT
    with pytest.raises(AttributeError):
        sat.DistillArgs(rowz=1)
    with pytest.raises(KeyError):
        sat.DistillArgs(logits_type="int8")


def _norm(**kw):
    f = dict(rows=4, width=16, block_type="bf16", stream_type="fp32", gate_type="bf16", post_norm="rms", pre_norm="layer",
             residual_scale=1.0, branch_scale=1.0, x=AT, ldx=16, y=AT, ldy=16, h=AT, ldh=16, z=AT, ldz=16, gate=AT, ldg=16,
             rows_per_gate=2, post_stats=AT, pre_stats=AT)
    return sat.BlockNormArgs(**{**f, **kw})


def _grads(**kw):
    f = dict(dh=AT, lddh=16, dz=AT, lddz=16, dx=AT, lddx=16, dy=AT, lddy=16, workspace=AT, workspace_bytes=1 << 40)
    return sat.BlockNormGrads(**{**f, **kw})


@pytest.mark.parametrize("status,bad", [
    (-1, dict(rows=-1)), (-1, dict(width=-1)), (-1, dict(rows=1 << 31)), (-1, dict(width=16385)), (-1, dict(block_type=3)),
    (-1, dict(stream_type="fp16")), (-1, dict(gate_type="fp16")), (-1, dict(post_norm=3)), (-1, dict(pre_norm=-1)),
    (-1, dict(x=None)), (-1, dict(y=None)), (-1, dict(h=None)), (-1, dict(z=None)), (-1, dict(ldx=15)), (-1, dict(ldy=15)),
    (-1, dict(ldh=15)), (-1, dict(ldz=15)), (-1, dict(rows_per_gate=0)), (-1, dict(ldg=15)), (-3, dict(x=AT + 2)),
    (-3, dict(y=AT + 1)), (-3, dict(h=AT + 2)), (-3, dict(z=AT + 1)), (-3, dict(gate=AT + 1)), (-3, dict(pre_gamma=AT + 2)),
    (-3, dict(post_stats=AT + 1))])
def test_block_norm_refuses(status, bad):
    assert sat.rowop_block_norm(_norm(**bad)) == status
    assert sat.gemm_last_error()


@pytest.mark.parametrize("status,bad,grads", [
    (-1, {}, dict(dz=None)), (-1, dict(h=None), {}), (-1, dict(pre_norm="none"), dict(dh=None)), (-1, {}, dict(lddh=15)),
    (-1, {}, dict(lddz=15)), (-1, {}, dict(lddx=15)), (-1, {}, dict(lddy=15)), (-1, dict(post_stats=None), {}),
    (-1, dict(pre_stats=None), {}), (-1, {}, dict(workspace=None)), (-1, {}, dict(workspace_bytes=8)),
    (-1, {}, dict(dpost_beta=AT)), (-1, dict(pre_norm="none"), dict(dpre_gamma=AT)), (-1, dict(gate=None), dict(dgate=AT, lddg=16)),
    (-1, {}, dict(dgate=AT, lddg=15)), (-3, {}, dict(workspace=AT + 16)), (-3, {}, dict(dh=AT + 2)), (-3, {}, dict(dy=AT + 1)),
    (-3, {}, dict(dpre_gamma=AT + 2)), (-3, {}, dict(dgate=AT + 1, lddg=16))])
def test_block_norm_backward_refuses(status, bad, grads):
    assert sat.rowop_block_norm_backward(_norm(**bad), _grads(**grads)) == status
    assert sat.gemm_last_error()


def test_null_structs_and_empty_calls():
    for call in (sat.rowop_block_norm, sat.rowop_distill, sat.rowop_distill_backward, sat.rowop_verify):
        assert call(None) == -1
    assert sat.rowop_block_norm_backward(None, _grads()) == -1
    assert sat.rowop_block_norm_backward(_norm(), None) == -1
    # No rows, no columns or no sequences: nothing to do, whatever the pointers.
    assert sat.rowop_block_norm(sat.BlockNormArgs(rows=0, width=16)) == 0
    assert sat.rowop_block_norm(sat.BlockNormArgs(rows=3, width=0)) == 0
    assert sat.rowop_block_norm_backward(sat.BlockNormArgs(rows=3, width=0), sat.BlockNormGrads()) == 0
    assert sat.rowop_distill(sat.DistillArgs(rows=0)) == 0
    assert sat.rowop_distill_backward(sat.DistillArgs(rows=0)) == 0
    assert sat.rowop_verify(sat.VerifyArgs(batch=0)) == 0


def test_workspaces():
    assert sat.rowop_block_norm_workspace(_norm(rows=0)) == 0
    for rows, width in ((1, 1), (5, 300), (100, 4096), (70000, 16384), (1 << 30, 64)):
        size = sat.rowop_block_norm_workspace(_norm(rows=rows, width=width, ldg=width))
        # At least a set of sums for a part; at most 5 sums for about four rounds of CTAs that fill the GPU.
        assert 3 * width * 4 <= size <= 5 * 4 * (width + 8) * 4 * 1300
    with pytest.raises(sat.GemmError):
        sat.rowop_block_norm_workspace(_norm(width=1 << 20))
    assert sat.rowop_verify_workspace(0, 4, 100) >= 0 and sat.rowop_verify_workspace(3, 4, 100) > 0
    for bad in ((-1, 4, 100), (1, -1, 100), (1, 65, 100), (1, 4, 0), (1, 4, 1 << 31), ((1 << 20) + 1, 1, 8)):
        with pytest.raises(sat.GemmError):
            sat.rowop_verify_workspace(*bad)


def _distill(**kw):
    f = dict(rows=2, vocab=100, k=4, logits_type="bf16", teacher_type="fp32", temperature=1.0, logits=AT, ldl=100, ids=AT,
             ldi=4, teacher=AT, ldt=4, loss=AT, lse=AT, dlogits=AT, ldd=100)
    return sat.DistillArgs(**{**f, **kw})


@pytest.mark.parametrize("status,bad", [
    (-1, dict(rows=-1)), (-1, dict(vocab=-1)), (-1, dict(vocab=0)), (-1, dict(vocab=(1 << 30) + 1)), (-1, dict(k=-1)),
    (-1, dict(k=1025)), (-1, dict(logits_type=7)), (-1, dict(teacher_type=-1)), (-1, dict(temperature=0.0)),
    (-1, dict(temperature=-1.0)), (-1, dict(temperature=float("nan"))), (-1, dict(temperature=float("inf"))),
    (-1, dict(logits=None)), (-1, dict(ids=None)), (-1, dict(teacher=None)), (-1, dict(ldl=99)), (-1, dict(ldi=3)),
    (-1, dict(ldt=3)), (-1, dict(ldd=99)), (-3, dict(logits=AT + 1)), (-3, dict(dlogits=AT + 1)), (-3, dict(ids=AT + 2)),
    (-3, dict(teacher=AT + 2)), (-3, dict(weight=AT + 2)), (-3, dict(dloss=AT + 2)), (-3, dict(teacher_lse=AT + 1))])
def test_distill_refuses(status, bad):
    assert sat.rowop_distill(_distill(**bad)) == status
    assert sat.gemm_last_error()
    assert sat.rowop_distill_backward(_distill(**bad)) == status


def test_distill_refuses_missing_outputs():
    assert sat.rowop_distill(_distill(loss=None)) == -1
    assert sat.rowop_distill_backward(_distill(lse=None)) == -1
    assert sat.rowop_distill_backward(_distill(dlogits=None)) == -1


@pytest.mark.parametrize("status,bad", [
    (-1, dict(batch=-1)), (-1, dict(drafts=-1)), (-1, dict(drafts=65)), (-1, dict(vocab=0)), (-1, dict(batch=(1 << 20) + 1)),
    (-1, dict(logits_type=3)), (-1, dict(temperature=-0.5)), (-1, dict(temperature=float("nan"))),
    (-1, dict(draft_temperature=0.0)), (-1, dict(target=None)), (-1, dict(tokens=None)), (-1, dict(uniforms=None)),
    (-1, dict(noise=None)), (-1, dict(accepted=None)), (-1, dict(out=None)), (-1, dict(ldt=99)), (-1, dict(ldq=99)),
    (-1, dict(ldn=99)), (-1, dict(workspace=None)), (-1, dict(workspace_bytes=1)), (-3, dict(target=AT + 1)),
    (-3, dict(draft=AT + 1)), (-3, dict(tokens=AT + 2)), (-3, dict(noise=AT + 2)), (-3, dict(workspace=AT + 8)),
    (-3, dict(logprobs=AT + 2)), (-3, dict(lengths=AT + 1))])
def test_verify_refuses(status, bad):
    f = dict(batch=2, drafts=3, vocab=100, logits_type="fp16", temperature=1.0, draft_temperature=1.0, target=AT, ldt=100,
             draft=AT, ldq=100, tokens=AT, uniforms=AT, noise=AT, ldn=100, accepted=AT, out=AT, workspace=AT,
             workspace_bytes=1 << 30)
    assert sat.rowop_verify(sat.VerifyArgs(**{**f, **bad})) == status
    assert sat.gemm_last_error()
