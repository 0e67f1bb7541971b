"""Host-side tests of the FP8 layer operators' ABI (no GPU needed): exports,
structure layout, and every refusal before any launch, in C and in Python."""
import ctypes as C
import os
import re
import subprocess

import pytest
import torch

from routed_moe_decode_router_gb300 import build as B
from routed_moe_decode_router_gb300 import native as N
from routed_moe_decode_router_gb300 import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_ops.h")
P = 1 << 20      # a well-aligned address that no refused call may touch


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return N.lib()


def test_exports_match_header():
    declared = set(re.findall(r"MOE_API\s+[\w\s\*]+?\b(moeop_\w+)\s*\(", open(HEADER).read()))
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB], capture_output=True, text=True,
                         check=True).stdout
    assert declared == set(re.findall(r"\sT\s(moeop_\w+)", out)) == set(N.OPS_EXPORTS)


def test_struct_layout(tmp_path):
    structs = {"moeop_route_config": N.RouteConfig, "moeop_experts_config": N.ExpertsConfig,
               "moeop_experts_weights": N.ExpertsWeights}
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_ops.h"', 'int main(void){']
    for c, py in structs.items():
        src.append('printf("%s %%zu\\n", sizeof(%s));' % (c, c))
        src += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (c, f, c, f) for f, _ in py._fields_]
    (tmp_path / "l.c").write_text("\n".join(src + ["return 0;}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    got = dict(line.split() for line in subprocess.run(
        [str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.splitlines())
    for c, py in structs.items():
        assert int(got[c]) == C.sizeof(py)
        for f, _ in py._fields_:
            assert int(got["%s.%s" % (c, f)]) == getattr(py, f).offset


def refused(fn, *a, status=1, text=""):
    with pytest.raises(N.MoeError) as e:
        fn(*a)
    assert e.value.status == status and text in str(e.value), str(e.value)


def norm_args(**kw):
    d = dict(x=P, xs=256, r=0, rs=0, w=2 * P, rows=4, hidden=256, dtype=0, eps=1e-6, y=3 * P,
             ro=0, q=0, sc=0)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,text", [
    (dict(dtype=3), "dtype"), (dict(rows=-1), "rows"), (dict(rows=(1 << 30) + 1), "rows"),
    (dict(hidden=0), "hidden"),
    (dict(hidden=32769, xs=40000), "hidden"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(y=0), "required"), (dict(q=4 * P), "together"),
    (dict(sc=4 * P), "together"), (dict(x=0), "NULL"), (dict(x=P + 1), "aligned"),
    (dict(w=0), "NULL"), (dict(xs=255), "stride"), (dict(r=5 * P, rs=10), "stride"),
    (dict(y=P), "overlaps an input"), (dict(y=2 * P), "overlaps an input"),
    (dict(r=5 * P, rs=256, ro=3 * P), "two outputs"),
    (dict(xs=512, r=5 * P, rs=256, ro=P), "overlaps an input"),
    (dict(q=3 * P, sc=4 * P), "two outputs")])
def test_norm_refusals(kw, text):
    refused(N.moeop_rms_norm, *norm_args(**kw), text=text)


def test_empty_calls_touch_nothing():
    N.moeop_rms_norm(*norm_args(rows=0))
    N.moeop_route_topk(route_cfg(), 0, 16, 0, 0, 0, 0)
    N.moeop_matmul_fp8(*mm_args(m=0, a=0, out=0))


def route_cfg(**kw):
    d = dict(num_experts=16, top_k=4, scoring=0, groups=1, group_limit=1, group_score=0,
             norm_topk_prob=1, routed_scaling_factor=1.0, dtype=2)
    d.update(kw)
    return N.RouteConfig(**d)


@pytest.mark.parametrize("kw,text", [
    (dict(num_experts=0), "num_experts"), (dict(num_experts=1025), "num_experts"),
    (dict(top_k=0), "top_k"), (dict(top_k=17), "top_k"),
    (dict(num_experts=1024, top_k=65), "top_k"), (dict(groups=3), "groups"),
    (dict(groups=0), "groups"), (dict(num_experts=64, groups=64), "groups"),
    (dict(groups=4, group_limit=5), "group_limit"), (dict(groups=4, group_limit=0), "group_limit"),
    (dict(groups=8, group_limit=1), "top_k"), (dict(scoring=2), "scoring"),
    (dict(group_score=2), "group_score"), (dict(norm_topk_prob=2), "norm_topk_prob"),
    (dict(routed_scaling_factor=float("inf")), "finite"), (dict(dtype=-1), "dtype")])
def test_route_config_refusals(kw, text):
    refused(N.moeop_route_topk, route_cfg(**kw), P, 1024, 0, 4, 2 * P, 3 * P, text=text)


@pytest.mark.parametrize("a,text", [
    ((0, 16, 0, 4, 2 * P, 3 * P), "NULL"), ((P + 2, 16, 0, 4, 2 * P, 3 * P), "aligned"),
    ((P, 15, 0, 4, 2 * P, 3 * P), "stride"), ((P, 16, 0, -1, 2 * P, 3 * P), "rows"),
    ((P, 16, 0, 4, P, 3 * P), "overlap"), ((P, 16, 0, 4, 2 * P, 2 * P), "overlap"),
    ((P, 16, 3 * P, 4, 2 * P, 3 * P), "overlap"), ((P, 16, 0, 4, 0, 3 * P), "NULL")])
def test_route_argument_refusals(a, text):
    refused(N.moeop_route_topk, route_cfg(), *a, text=text)


def mm_args(**kw):
    d = dict(a=P, ast=256, sa=2 * P, b=3 * P, bst=256, sb=4 * P, m=4, n=100, k=256, out=5 * P,
             dt=0)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,text", [
    (dict(dt=3), "out_dtype"), (dict(m=-1), "m="), (dict(n=0), "n="), (dict(k=0), "k="),
    (dict(k=24), "k="), (dict(a=P + 8), "aligned"), (dict(b=0), "aligned"), (dict(sa=0), "NULL"),
    (dict(sb=4 * P + 2), "aligned"), (dict(out=0), "NULL"), (dict(ast=248), "strides"),
    (dict(bst=264), "strides"), (dict(out=P), "overlaps"), (dict(out=3 * P), "overlaps"),
    (dict(out=2 * P), "overlaps"), (dict(m=1 << 30, n=1 << 24), "tiles")])
def test_matmul_refusals(kw, text):
    refused(N.moeop_matmul_fp8, *mm_args(**kw), text=text)


def ex_cfg(**kw):
    d = dict(hidden=256, inter=128, num_experts=8, top_k=2)
    d.update(kw)
    return N.ExpertsConfig(**d)


@pytest.mark.parametrize("kw,rows", [
    (dict(hidden=200), 4), (dict(hidden=0), 4), (dict(hidden=32896), 4), (dict(inter=64), 4),
    (dict(num_experts=0), 4), (dict(num_experts=1025), 4), (dict(top_k=0), 4), (dict(top_k=65), 4),
    (dict(), -1), (dict(top_k=64), 1 << 21)])
def test_experts_config_refusals(kw, rows):
    refused(N.moeop_experts_workspace_size, ex_cfg(**kw), rows)


def ex_args(cfg=None, w=None, **kw):
    d = dict(q=P, sc=2 * P, ids=3 * P, wts=4 * P, add=0, out=5 * P, rows=4, ws=64 * P,
             n=1 << 30)
    d.update(kw)
    return [cfg or ex_cfg(), w or N.ExpertsWeights(10 * P, 12 * P, 14 * P, 16 * P, 17 * P, 18 * P)
            ] + list(d.values())


@pytest.mark.parametrize("kw,status,text", [
    (dict(q=0), 1, "q"), (dict(q=P + 8), 1, "aligned"), (dict(out=0), 1, "out"),
    (dict(add=P + 2), 1, "addend"), (dict(ids=0), 1, "ids"), (dict(wts=4 * P + 1), 1, "wts"),
    (dict(ws=0), 3, "NULL"), (dict(ws=64 * P + 128), 3, "256"), (dict(n=100), 3, "needs"),
    (dict(out=P), 1, "overlaps"), (dict(out=10 * P), 1, "overlaps"),
    (dict(out=64 * P), 1, "workspace"), (dict(q=64 * P), 1, "workspace"),
    (dict(rows=-1), 1, "rows"), (dict(add=5 * P + 16), 1, "overlaps"),
    (dict(w=N.ExpertsWeights(10 * P, 0, 14 * P, 16 * P, 17 * P, 18 * P)), 1, "up"),
    (dict(w=N.ExpertsWeights(10 * P, 12 * P, 14 * P, 16 * P, 17 * P, 0)), 1, "scale")])
def test_experts_refusals(kw, status, text):
    refused(N.moeop_experts_fp8, *ex_args(**kw), status=status, text=text)


def test_python_refuses_host_tensors_before_the_library():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    f = torch.zeros(4, 256, dtype=ops.F8)
    s = torch.zeros(4, 2)
    for call in (lambda: ops.rms_norm(x, x[0]), lambda: ops.route_topk(x.float(), 2),
                 lambda: ops.matmul_fp8(f, s, f, s[:1]),
                 lambda: ops.experts_fp8(f, s, None, None, None, None, None, None, None, None)):
        with pytest.raises((ValueError, TypeError), match="CUDA|Tensor"):
            call()
    with pytest.raises(TypeError):
        ops.rms_norm(None, None)
    with pytest.raises(ValueError, match="dimensions"):
        ops.rms_norm(x[0], x[0])


def test_workspace_size_covers_rows():
    a, b = (N.moeop_experts_workspace_size(ex_cfg(), r) for r in (1, 1000))
    assert a % 256 == 0 and b > 1000 * 2 * (128 + 256 * 2)
    assert N.moeop_experts_workspace_size(ex_cfg(), 0) > 0
