"""CPU-only checks of the experts' C-ABI boundary and binding: the library
builds, loads and exports what include/lapsum_experts.h declares, and bad calls
are refused before any CUDA work.  No kernel is launched here."""
import os
import re
import subprocess

import pytest

import differentiable_soft_top_b200 as lt
from differentiable_soft_top_b200 import experts as ex

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EBADK, EWORKSPACE, ETOOLARGE = lt.LAPSUM_OK, lt.LAPSUM_EINVAL, lt.LAPSUM_EBADK, lt.LAPSUM_EWORKSPACE, lt.LAPSUM_ETOOLARGE
A = 1 << 30  # aligned, non-null, far apart: checks fail before any use


def at(i):
    return A * (i + 1)


@pytest.fixture(scope="module")
def lib():
    return ex._load()


def test_library_exports_what_the_header_declares(lib):
    src = open(os.path.join(ROOT, "include", "lapsum_experts.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"LAPSUM_API\s+[\w\s\*]+?\b(lapsum_\w+)\s*\(", src)))
    out = subprocess.run(["nm", "-D", "--defined-only", ex.library_path()], capture_output=True, text=True).stdout
    assert sorted(ln.split()[-1] for ln in out.splitlines() if " T " in ln) == names
    for limit, value in (("MAX", ex.MAX_EXPERTS), ("MAX_K", ex.MAX_K), ("MAX_GROUPS", ex.MAX_GROUPS)):
        assert re.search(rf"#define LAPSUM_EXPERTS_{limit} {value}\b", src)


def refused(fn, names, good, cases):
    for change, code in cases:
        args = dict(good, **change)
        assert fn(*[args[n] for n in names]) == code, change


ROUTE = "scores dtype tokens experts stride k score bias groups kept top renorm scale weights chosen stream".split()


def test_route_fwd_rejects_bad_arguments(lib):
    good = dict(scores=at(0), dtype=0, tokens=4, experts=16, stride=16, k=2, score=0, bias=None, groups=1, kept=1, top=1,
                renorm=1, scale=1.0, weights=at(1), chosen=at(2), stream=None)
    inf = float("inf")
    refused(lib.lapsum_experts_route_fwd, ROUTE, good, [
        (dict(scores=None), EINVAL), (dict(weights=None), EINVAL), (dict(chosen=None), EINVAL), (dict(dtype=3), EINVAL),
        (dict(tokens=0), EINVAL), (dict(experts=0), EINVAL), (dict(stride=15), EINVAL), (dict(score=3), EINVAL),
        (dict(scores=at(0) + 2), EINVAL), (dict(dtype=1, scores=at(0) + 1), EINVAL), (dict(weights=at(1) + 2), EINVAL),
        (dict(bias=at(3) + 2), EINVAL), (dict(k=0), EBADK), (dict(k=17), EBADK),
        (dict(experts=2048, stride=2048), ETOOLARGE), (dict(experts=64, stride=64, k=33), ETOOLARGE),
        (dict(tokens=1 << 40), ETOOLARGE), (dict(groups=3), EINVAL), (dict(groups=0), EINVAL),
        (dict(experts=128, stride=128, groups=64), EINVAL), (dict(groups=4, kept=5), EINVAL), (dict(groups=4, kept=0), EINVAL),
        (dict(groups=8, kept=1, k=3), EBADK), (dict(top=3), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
        (dict(scale=inf), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(weights=at(0) + 64), EINVAL),
        (dict(chosen=at(1)), EINVAL), (dict(bias=at(1)), EINVAL),
    ])


def test_route_bwd_rejects_bad_arguments(lib):
    names = "scores dtype tokens experts stride k score bias renorm scale chosen weights gw grad gstride stream".split()
    good = dict(scores=at(0), dtype=1, tokens=4, experts=16, stride=16, k=2, score=0, bias=None, renorm=1, scale=1.0,
                chosen=at(1), weights=at(2), gw=at(3), grad=at(4), gstride=16, stream=None)
    refused(lib.lapsum_experts_route_bwd, names, good, [
        (dict(grad=None), EINVAL), (dict(gw=None), EINVAL), (dict(chosen=None), EINVAL), (dict(weights=None), EINVAL),
        (dict(gstride=15), EINVAL), (dict(grad=at(0)), EINVAL), (dict(grad=at(3)), EINVAL), (dict(grad=at(4) + 1), EINVAL),
        (dict(k=0), EBADK), (dict(score=-1), EINVAL),
    ])


def test_plan_rejects_bad_arguments(lib):
    names = "chosen slots experts offsets rows slot_of ws wsb stream".split()
    good = dict(chosen=at(0), slots=100000, experts=64, offsets=at(1), rows=at(2), slot_of=at(3), ws=at(4), wsb=1 << 20,
                stream=None)
    need = lib.lapsum_experts_plan_workspace_size(100000, 64)
    assert 0 < need < 1 << 20
    assert lib.lapsum_experts_plan_workspace_size(4096, 1024) == 0  # one block
    assert lib.lapsum_experts_plan_workspace_size(0, 4) == 0 and lib.lapsum_experts_plan_workspace_size(8, 0) == 0
    assert lib.lapsum_experts_plan_workspace_size(2**31 - 1, 1024) <= 256 * 1024 * 4
    refused(lib.lapsum_experts_plan, names, good, [
        (dict(chosen=None), EINVAL), (dict(offsets=None), EINVAL), (dict(rows=None), EINVAL), (dict(slot_of=None), EINVAL),
        (dict(slots=0), EINVAL), (dict(experts=0), EINVAL), (dict(experts=1025), ETOOLARGE), (dict(slots=1 << 31), ETOOLARGE),
        (dict(rows=at(2) + 1), EINVAL), (dict(rows=at(0)), EINVAL), (dict(slot_of=at(2)), EINVAL), (dict(offsets=at(3)), EINVAL),
        (dict(ws=None), EWORKSPACE), (dict(wsb=need - 1), EWORKSPACE), (dict(ws=at(4) + 128), EWORKSPACE),
    ])


def test_exchange_rejects_bad_arguments(lib):
    names = "x dtype tokens k dim xs slot_of out os stream".split()
    good = dict(x=at(0), dtype=1, tokens=8, k=2, dim=64, xs=64, slot_of=at(1), out=at(2), os=64, stream=None)
    refused(lib.lapsum_experts_dispatch, names, good, [
        (dict(x=None), EINVAL), (dict(slot_of=None), EINVAL), (dict(out=None), EINVAL), (dict(dtype=-1), EINVAL),
        (dict(tokens=0), EINVAL), (dict(k=0), EINVAL), (dict(dim=0), EINVAL), (dict(xs=63), EINVAL), (dict(os=63), EINVAL),
        (dict(k=33), ETOOLARGE), (dict(tokens=1 << 31), ETOOLARGE), (dict(x=at(0) + 1), EINVAL), (dict(out=at(0) + 64), EINVAL),
        (dict(out=at(1)), EINVAL), (dict(slot_of=at(1) + 2), EINVAL),
    ])
    names = "y dtype tokens k dim ys w rows res rs out os stream".split()
    good = dict(y=at(0), dtype=0, tokens=8, k=2, dim=64, ys=64, w=at(1), rows=at(2), res=at(3), rs=64, out=at(4), os=64,
                stream=None)
    refused(lib.lapsum_experts_combine, names, good, [
        (dict(y=None), EINVAL), (dict(rows=None), EINVAL), (dict(out=None), EINVAL), (dict(ys=1), EINVAL), (dict(rs=1), EINVAL),
        (dict(out=at(3)), EINVAL), (dict(out=at(1)), EINVAL), (dict(res=at(3) + 2), EINVAL), (dict(k=40), ETOOLARGE),
    ])
    names = "g dtype tokens k dim gs y ys w rows slot_of gy gys gw stream".split()
    good = dict(g=at(0), dtype=2, tokens=8, k=2, dim=64, gs=64, y=at(1), ys=64, w=at(2), rows=at(3), slot_of=at(4), gy=at(5),
                gys=64, gw=at(6), stream=None)
    refused(lib.lapsum_experts_combine_bwd, names, good, [
        (dict(g=None), EINVAL), (dict(y=None), EINVAL), (dict(rows=None), EINVAL), (dict(slot_of=None), EINVAL),
        (dict(gy=None, gw=None), EINVAL), (dict(gs=8), EINVAL), (dict(gys=8), EINVAL), (dict(gy=at(1)), EINVAL),
        (dict(gw=at(2)), EINVAL), (dict(gw=at(5)), EINVAL), (dict(gw=at(6) + 2), EINVAL),
    ])


def test_products_reject_bad_arguments(lib):
    names = "x dtype rows in_ xs w experts out off b act res rs y ys pre ps status stream".split()
    good = dict(x=at(0), dtype=1, rows=32, in_=64, xs=64, w=at(1), experts=4, out=128, off=at(2), b=at(3), act=1, res=at(4),
                rs=128, y=at(5), ys=128, pre=at(6), ps=128, status=at(7), stream=None)
    refused(lib.lapsum_experts_linear_fwd, names, good, [
        (dict(dtype=0), EINVAL), (dict(rows=0), EINVAL), (dict(rows=2**31 - 1), EINVAL), (dict(in_=60), EINVAL),
        (dict(out=100), EINVAL), (dict(in_=0), EINVAL), (dict(act=5), EINVAL), (dict(act=-1), EINVAL),
        (dict(act=4, out=136), EINVAL), (dict(experts=0), EINVAL), (dict(experts=1025), EINVAL), (dict(off=None), EINVAL),
        (dict(off=at(2) + 2), EINVAL), (dict(x=None), EINVAL), (dict(x=at(0) + 8), EINVAL), (dict(xs=68), EINVAL),
        (dict(xs=56), EINVAL), (dict(w=None), EINVAL), (dict(w=at(1) + 2), EINVAL), (dict(y=None), EINVAL),
        (dict(ys=120), EINVAL), (dict(rs=120), EINVAL), (dict(ps=120), EINVAL), (dict(y=at(0)), EINVAL), (dict(y=at(1)), EINVAL),
        (dict(y=at(4)), EINVAL), (dict(pre=at(5)), EINVAL), (dict(y=at(2)), EINVAL), (dict(status=at(7) + 2), EINVAL),
        (dict(rows=2**30, out=1 << 20, ys=1 << 20, rs=1 << 20, ps=1 << 20), ETOOLARGE),
    ])
    names = "gy dtype rows out gys pre ps experts off act gh ghs gb ws wsb stream".split()
    good = dict(gy=at(0), dtype=1, rows=32, out=128, gys=128, pre=at(1), ps=128, experts=4, off=at(2), act=2, gh=at(3), ghs=128,
                gb=at(4), ws=at(5), wsb=1 << 20, stream=None)
    need = lib.lapsum_experts_linear_act_workspace_size(32, 4, 128)
    refused(lib.lapsum_experts_linear_act_bwd, names, good, [
        (dict(gy=None), EINVAL), (dict(pre=None), EINVAL), (dict(gh=None), EINVAL), (dict(act=0, gh=None, gb=None), EINVAL),
        (dict(gy=at(0) + 2), EINVAL), (dict(gys=132), EINVAL), (dict(ghs=120), EINVAL), (dict(gh=at(0)), EINVAL),
        (dict(gb=at(1)), EINVAL), (dict(gh=at(4)), EINVAL), (dict(ws=None), EWORKSPACE), (dict(wsb=need - 1), EWORKSPACE),
        (dict(ws=at(5) + 16), EWORKSPACE), (dict(act=4, out=136, ghs=136, ps=136, gys=136), EINVAL),
    ])
    names = "gh dtype rows out ghs w experts in_ off gx gxs status stream".split()
    good = dict(gh=at(0), dtype=1, rows=32, out=128, ghs=128, w=at(1), experts=4, in_=64, off=at(2), gx=at(3), gxs=64, status=None,
                stream=None)
    refused(lib.lapsum_experts_linear_dx, names, good, [
        (dict(gh=None), EINVAL), (dict(ghs=132), EINVAL), (dict(w=at(1) + 8), EINVAL), (dict(gx=None), EINVAL),
        (dict(gxs=56), EINVAL), (dict(gx=at(0)), EINVAL), (dict(gx=at(1)), EINVAL), (dict(off=None), EINVAL),
    ])
    names = "gh dtype rows out ghs x in_ xs experts off gw status stream".split()
    good = dict(gh=at(0), dtype=1, rows=32, out=128, ghs=128, x=at(1), in_=64, xs=64, experts=4, off=at(2), gw=at(3), status=None,
                stream=None)
    refused(lib.lapsum_experts_linear_dweight, names, good, [
        (dict(gh=None), EINVAL), (dict(x=None), EINVAL), (dict(xs=60), EINVAL), (dict(gw=at(3) + 8), EINVAL),
        (dict(gw=at(0)), EINVAL), (dict(gw=at(1)), EINVAL), (dict(experts=0), EINVAL),
    ])


def test_linear_backward_rejects_bad_arguments(lib):
    names = "gy dtype rows out gys pre x in_ xs w experts off act gx gw gb status ws wsb stream".split()
    good = dict(gy=at(0), dtype=2, rows=32, out=128, gys=128, pre=at(1), x=at(2), in_=64, xs=64, w=at(3), experts=4, off=at(4),
                act=2, gx=at(5), gw=at(6), gb=at(7), status=None, ws=at(8), wsb=1 << 20, stream=None)
    size = lib.lapsum_experts_linear_bwd_workspace_size
    need = size(32, 4, 128, 2, 1)
    assert need == 32 * 128 * 2 + lib.lapsum_experts_linear_act_workspace_size(32, 4, 128)
    assert size(32, 4, 128, 0, 0) == 0 and size(0, 4, 128, 2, 1) == 0
    refused(lib.lapsum_experts_linear_bwd, names, good, [
        (dict(gy=None), EINVAL), (dict(pre=None), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(off=None), EINVAL),
        (dict(gx=None, gw=None, gb=None), EINVAL), (dict(dtype=0), EINVAL), (dict(rows=0), EINVAL), (dict(in_=60), EINVAL),
        (dict(act=5), EINVAL), (dict(act=4, out=136, gys=136), EINVAL), (dict(gys=132), EINVAL), (dict(xs=56), EINVAL),
        (dict(gx=at(5) + 8), EINVAL), (dict(gw=at(6) + 8), EINVAL), (dict(gx=at(0)), EINVAL), (dict(gw=at(2)), EINVAL),
        (dict(gx=at(3)), EINVAL), (dict(gb=at(6)), EINVAL), (dict(gw=at(1)), EINVAL), (dict(ws=at(5)), EINVAL),
        (dict(ws=None), EWORKSPACE), (dict(wsb=need - 1), EWORKSPACE), (dict(ws=at(8) + 16), EWORKSPACE),
    ])


def test_layer_rejects_bad_arguments(lib):
    names = "x dtype tokens dim xs w chosen k wi bi experts up act wo bo dim_out res rs out os keep status ws wsb stream".split()
    good = dict(x=at(0), dtype=1, tokens=8, dim=64, xs=64, w=at(1), chosen=at(2), k=2, wi=at(3), bi=at(4), experts=4, up=128,
                act=4, wo=at(5), bo=at(6), dim_out=72, res=at(7), rs=72, out=at(8), os=72, keep=0, status=at(9), ws=at(10),
                wsb=1 << 20, stream=None)
    size = lib.lapsum_experts_mlp_workspace_size
    need = size(8, 2, 4, 64, 128, 4, 72, 0)
    assert need >= 16 * 2 * (64 + 64 + 72)
    assert size(8, 2, 4, 64, 128, 4, 72, 1) == need + 16 * 2 * 128
    assert size(0, 2, 4, 64, 128, 4, 72, 0) == 0 and size(8, 33, 4, 64, 128, 4, 72, 0) == 0
    refused(lib.lapsum_experts_mlp_fwd, names, good, [
        (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(chosen=None), EINVAL), (dict(wi=None), EINVAL),
        (dict(wo=None), EINVAL), (dict(out=None), EINVAL), (dict(dtype=0), EINVAL), (dict(tokens=0), EINVAL), (dict(k=0), EINVAL),
        (dict(k=33), EINVAL), (dict(dim=60), EINVAL), (dict(xs=56), EINVAL), (dict(up=120), EINVAL), (dict(act=0, up=100), EINVAL),
        (dict(act=7), EINVAL), (dict(dim_out=70), EINVAL), (dict(os=64), EINVAL), (dict(rs=64), EINVAL), (dict(experts=0), EINVAL),
        (dict(experts=1025), EINVAL), (dict(wi=at(3) + 8), EINVAL), (dict(out=at(0)), EINVAL), (dict(out=at(10) + 256), EINVAL),
        (dict(ws=at(5)), EINVAL), (dict(ws=None), EWORKSPACE), (dict(wsb=need - 1), EWORKSPACE), (dict(ws=at(10) + 16), EWORKSPACE),
        (dict(wsb=need, keep=1), EWORKSPACE),
    ])


def test_layer_backward_rejects_bad_arguments(lib):
    names = "g dtype tokens dim gs w k wi experts up act wo dim_out kept own gx gw gwi gbi gwo gbo status ws wsb stream".split()
    good = dict(g=at(0), dtype=1, tokens=8, dim=64, gs=64, w=at(1), k=2, wi=at(2), experts=4, up=128, act=4, wo=at(3), dim_out=64,
                kept=at(4), own=1, gx=at(5), gw=at(6), gwi=at(7), gbi=at(8), gwo=at(9), gbo=at(10), status=None, ws=at(11),
                wsb=1 << 22, stream=None)
    size = lib.lapsum_experts_mlp_bwd_workspace_size
    need = size(8, 2, 4, 64, 128, 4, 64)
    assert need >= 16 * 2 * (64 + 64 + 64 + 128) and size(0, 2, 4, 64, 128, 4, 64) == 0
    none = dict(gx=None, gw=None, gwi=None, gbi=None, gwo=None, gbo=None)
    refused(lib.lapsum_experts_mlp_bwd, names, good, [
        (dict(g=None), EINVAL), (dict(w=None), EINVAL), (dict(wi=None), EINVAL), (dict(wo=None), EINVAL), (dict(kept=None), EINVAL),
        (none, EINVAL), (dict(dim_out=72, gs=72), EINVAL), (dict(gs=56), EINVAL), (dict(dtype=0), EINVAL), (dict(act=9), EINVAL),
        (dict(up=120), EINVAL), (dict(k=0), EINVAL), (dict(experts=0), EINVAL), (dict(gx=at(5) + 8), EINVAL),
        (dict(gwi=at(7) + 8), EINVAL), (dict(kept=at(4) + 16), EINVAL), (dict(gx=at(0)), EINVAL), (dict(gwi=at(2)), EINVAL),
        (dict(gwo=at(7)), EINVAL), (dict(gw=at(4) + 1024), EINVAL), (dict(ws=at(4)), EINVAL), (dict(ws=None), EWORKSPACE),
        (dict(wsb=need - 1), EWORKSPACE), (dict(ws=at(11) + 16), EWORKSPACE),
    ])


def test_binding_refuses_cpu_tensors_and_bad_types():
    torch = pytest.importorskip("torch")
    x, c = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    p = ex.Plan(torch.zeros(17, dtype=torch.int32), c, torch.zeros(8, dtype=torch.int32))
    for call in (lambda: ex.route(x, 2), lambda: ex.plan(c, 16), lambda: ex.dispatch(x, p),
                 lambda: ex.combine(x, x, p), lambda: ex.linear(x.bfloat16(), x.bfloat16()),
                 lambda: ex.mlp(x, x, c, x[None], x[None])):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_row_layouts_the_binding_passes_on():
    """What needs no copy is passed as it is; overlapping, column-major or
    unaligned rows are copied."""
    torch = pytest.importorskip("torch")
    base = torch.zeros(10, 64, dtype=torch.bfloat16)
    v = base[:, 8:40]
    assert ex._rows16(v) is v and ex._stride(v) == 64
    assert ex._rows_of(base[:, 3:20]).data_ptr() == base[:, 3:20].data_ptr()
    assert ex._rows16(base[:, 3:35]).is_contiguous()  # starts off the 16-byte grid
    odd = torch.zeros(10, 65, dtype=torch.bfloat16)[:, :64]
    assert ex._rows16(odd).stride(0) == 64
    assert ex._rows_of(base.t()).is_contiguous()
    wide = torch.zeros(1, 8).expand(5, 8)
    assert ex._rows_of(wide).stride(0) == 8
    assert ex._stride(torch.zeros(1, 8)[:, :5]) == 5  # of one row the stride is never used
    assert ex._dense16(base[:, :32]).is_contiguous()
    flat = torch.zeros(65, dtype=torch.bfloat16)[1:].view(8, 8)
    assert ex._dense16(flat).data_ptr() % 16 == 0
