"""Refusals of the mixture-of-experts calls that need no GPU: the C ABI's argument checks
(fake pointers, never dereferenced: every call must fail before a launch) and the binding's."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import precision_quantized_linear_amd as pql

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = pql.PQL_ERR_INVALID_ARGUMENT, pql.PQL_ERR_UNSUPPORTED, pql.PQL_ERR_WORKSPACE
P = 1 << 20                      # a fake 16-byte aligned device pointer
ROW, BLOCK, MXFP8 = (pql.SCHEMES[s] for s in ("fp8_row", "fp8_block128", "mxfp8"))


def _route(score=0, dtype=0, logits=P, T=4, E=16, ldl=16, bias=None, k=2, groups=1, top=1, gs=0, renorm=1, scale=1.0,
           ids=P, weights=P):
    return pql.lib().pql_moe_route(score, dtype, logits, T, E, ldl, bias, k, groups, top, gs, renorm,
                                   ctypes.c_float(scale), ids, weights, None)


@pytest.mark.parametrize("bad", [
    dict(score=2), dict(score=-1), dict(dtype=3), dict(gs=2), dict(T=-1), dict(E=0), dict(E=1025, ldl=1025),
    dict(k=0), dict(k=33, E=64, ldl=64), dict(k=17), dict(groups=3), dict(groups=0), dict(groups=16, top=17),
    dict(groups=4, top=0), dict(groups=8, top=1, k=3), dict(E=130, ldl=130, groups=65), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(ldl=15), dict(logits=None), dict(ids=None), dict(weights=None),
    dict(logits=P + 2), dict(dtype=1, logits=P + 1), dict(bias=P + 2), dict(T=1 << 24, k=1), dict(T=1 << 40),
    dict(T=3, ldl=1 << 40),
])
def test_route_refusals(bad):
    assert _route(**bad) == INVALID and pql.lib().pql_last_error()


def test_route_empty_is_a_no_op():
    assert _route(T=0, logits=None, ids=None, weights=None) == pql.PQL_OK


def _plan(ids=P, T=4, k=2, E=16, offsets=P, order=P, slots=P, ws=P, wsb=1 << 30):
    return pql.lib().pql_moe_plan(ids, T, k, E, offsets, order, slots, ws, wsb, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(ids=None), dict(offsets=None), dict(order=None),
    dict(slots=None), dict(ids=P + 2), dict(offsets=P + 1), dict(T=1 << 23, k=2),
])
def test_plan_refusals(bad):
    assert _plan(**bad) == INVALID and pql.lib().pql_last_error()


def test_plan_workspace_refusal():
    need = ctypes.c_size_t()
    assert pql.lib().pql_moe_plan_workspace(1 << 20, 8, 256, ctypes.byref(need)) == pql.PQL_OK
    if need.value:
        assert _plan(T=1 << 20, k=8, E=256, ws=None, wsb=0) == WORKSPACE
        assert _plan(T=1 << 20, k=8, E=256, wsb=need.value - 1) == WORKSPACE
        assert _plan(T=1 << 20, k=8, E=256, ws=P + 4) == INVALID
    assert pql.lib().pql_moe_plan_workspace(4, 2, 2000, ctypes.byref(need)) == INVALID
    assert pql.lib().pql_moe_plan_workspace(4, 2, 8, None) == INVALID


def _gemm(scheme=ROW, a=P, sa=P, rows=8, gather=0, w=P, sw=P, offsets=P, order=P, T=4, k=2, E=8, N=256, K=256, c=P,
          ldc=256):
    return pql.lib().pql_moe_qgemm(scheme, a, sa, rows, gather, w, sw, offsets, order, T, k, E, N, K, c, ldc, None)


@pytest.mark.parametrize("bad,want", [
    (dict(scheme=MXFP8), UNSUPPORTED), (dict(scheme=99), UNSUPPORTED), (dict(K=200), INVALID), (dict(K=0), INVALID),
    (dict(N=0), INVALID), (dict(N=(1 << 20) + 128, ldc=(1 << 20) + 128), INVALID), (dict(ldc=255), INVALID),
    (dict(scheme=BLOCK, N=200, ldc=200), INVALID), (dict(rows=7), INVALID), (dict(gather=1), INVALID),
    (dict(gather=1, rows=4, order=None), INVALID), (dict(a=None), INVALID), (dict(sa=None), INVALID),
    (dict(w=None), INVALID), (dict(sw=None), INVALID), (dict(offsets=None), INVALID), (dict(c=None), INVALID),
    (dict(a=P + 8), INVALID), (dict(w=P + 4), INVALID), (dict(c=P + 1), INVALID), (dict(E=0), INVALID),
    (dict(E=1025), INVALID), (dict(k=33), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 23, rows=1 << 24), INVALID),
    (dict(E=1024, N=1 << 20, K=1 << 20, ldc=1 << 20), INVALID),
])
def test_gemm_refusals(bad, want):
    assert _gemm(**bad) == want and pql.lib().pql_last_error()


def test_gemm_empty_is_a_no_op():
    assert _gemm(T=0, rows=0, a=None, c=None) == pql.PQL_OK
    assert pql.moe_kernel_name("fp8_row", 0, 8, 64, 256, 256) == ""
    assert pql.moe_kernel_name("mxfp8", 4, 8, 64, 256, 256) == ""
    assert pql.moe_kernel_name("fp8_block128", 4, 8, 64, 256, 256).startswith("k_moe_")


def _swiglu(scheme=ROW, x=P, rows=4, cols=256, ldx=512, count=None, codes=P, scales=P):
    return pql.lib().pql_swiglu_quantize(scheme, x, rows, cols, ldx, count, codes, scales, None)


@pytest.mark.parametrize("bad,want", [
    (dict(scheme=MXFP8), UNSUPPORTED), (dict(cols=100), INVALID), (dict(scheme=BLOCK, cols=64, ldx=128), INVALID),
    (dict(ldx=256), INVALID), (dict(ldx=516), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 24), INVALID),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(x=P + 8), INVALID),
    (dict(count=P + 2), INVALID),
])
def test_swiglu_refusals(bad, want):
    assert _swiglu(**bad) == want and pql.lib().pql_last_error()


def _combine(y=P, rows=8, ldy=64, slots=P, weights=P, T=4, k=2, N=64, add=None, ldadd=64, out=P, ldo=64):
    return pql.lib().pql_moe_combine(y, rows, ldy, slots, weights, T, k, N, add, ldadd, out, ldo, None)


@pytest.mark.parametrize("bad", [
    dict(N=0), dict(N=(1 << 20) + 1), dict(ldy=63), dict(ldo=63), dict(add=P, ldadd=60), dict(T=-1), dict(k=0),
    dict(k=33), dict(rows=-1), dict(rows=1 << 24), dict(y=None), dict(slots=None), dict(weights=None), dict(out=None),
    dict(y=P + 1), dict(out=P + 1), dict(add=P + 1), dict(slots=P + 2), dict(T=1 << 24, k=1),
])
def test_combine_refusals(bad):
    assert _combine(**bad) == INVALID and pql.lib().pql_last_error()


def test_empty_calls_are_no_ops():
    assert _swiglu(rows=0, x=None, codes=None, scales=None) == pql.PQL_OK
    assert _combine(T=0, slots=None, out=None) == pql.PQL_OK


# ---------------------------------------------------------------- binding
def _cpu_plan(T=4, k=2, E=8):
    z = lambda n: torch.zeros(n, dtype=torch.int32)   # noqa: E731
    return pql.MoePlan(T, k, E, z(E + 1), z(T * k), z(T * k))


@pytest.mark.parametrize("call,message", [
    (lambda: pql.moe_route(torch.zeros(4, 8, dtype=torch.float64), 2), "float32"),
    (lambda: pql.moe_route(torch.zeros(8), 2), "2-D"),
    (lambda: pql.moe_route(torch.zeros(8, 4).t(), 2), "unit stride"),
    (lambda: pql.moe_route(torch.zeros(4, 8), 2, score="tanh"), "unknown score"),
    (lambda: pql.moe_route(torch.zeros(4, 8), 2, group_score="sum"), "unknown group score"),
    (lambda: pql.moe_route(torch.zeros(4, 8), 2, bias=torch.zeros(7)), "bias"),
    (lambda: pql.moe_route(torch.zeros(4, 8), 2, bias=torch.zeros(8).double()), "bias"),
    (lambda: pql.moe_route(torch.zeros(4, 8), 2), "HIP device"),
    (lambda: pql.moe_plan(torch.zeros(4, 2), 8), "int32"),
    (lambda: pql.moe_plan(torch.zeros(8, dtype=torch.int32), 8), "int32"),
    (lambda: pql.moe_plan(torch.zeros(2, 4, dtype=torch.int32).t(), 8), "contiguous"),
    (lambda: pql.moe_plan(torch.zeros(4, 2, dtype=torch.int32), 8), "HIP device"),
])
def test_binding_refusals(call, message):
    with pytest.raises(ValueError, match=message):
        call()


def test_moe_qgemm_binding_refusals():
    plan = _cpu_plan()
    a, w = pql._alloc_q("fp8_row", "activation", 8, 256, "cpu"), pql._alloc_q("fp8_row", "weight", 8 * 32, 256, "cpu")
    with pytest.raises(ValueError, match="HIP device"):
        pql.moe_qgemm(a, w, plan)
    with pytest.raises(ValueError, match="4 rows"):
        pql.moe_qgemm(a, w, plan, gather=True)
    with pytest.raises(ValueError, match="K mismatch"):
        pql.moe_qgemm(pql._alloc_q("fp8_row", "activation", 8, 128, "cpu"), w, plan)
    with pytest.raises(ValueError, match="schemes differ"):
        pql.moe_qgemm(pql._alloc_q("fp8_block128", "activation", 8, 256, "cpu"), w, plan)
    with pytest.raises(ValueError, match="activation"):
        pql.moe_qgemm(w, w, plan)
    with pytest.raises(ValueError, match="divide"):
        pql.moe_qgemm(a, pql._alloc_q("fp8_row", "weight", 8 * 32 + 1, 256, "cpu"), plan)
    with pytest.raises(ValueError, match="MoePlan"):
        pql.moe_qgemm(a, w, (plan.offsets, plan.order, plan.slots))
    with pytest.raises(ValueError, match="bfloat16"):
        pql.moe_qgemm(a, w, plan, out=torch.empty(8, 32))
    m = pql._alloc_q("mxfp8", "weight", 8 * 32, 256, "cpu")
    with pytest.raises(NotImplementedError):
        pql.moe_qgemm(pql._alloc_q("mxfp8", "activation", 8, 256, "cpu"), m, plan)
    short = pql.MoePlan(4, 2, 8, plan.offsets[:-1], plan.order, plan.slots)
    with pytest.raises(ValueError, match="plan.offsets"):
        pql.moe_qgemm(a, w, short)


def test_swiglu_and_combine_binding_refusals():
    plan = _cpu_plan()
    with pytest.raises(ValueError, match="HIP device"):
        pql.swiglu_quantize(torch.zeros(8, 256, dtype=torch.bfloat16), "fp8_row")
    y, w = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="HIP device"):
        pql.moe_combine(y, plan, w)
    with pytest.raises(ValueError, match="weights"):
        pql.moe_combine(y, plan, w.double())
    with pytest.raises(ValueError, match="weights"):
        pql.moe_combine(y, plan, w.t().contiguous())
    with pytest.raises(ValueError, match="y must"):
        pql.moe_combine(y[:4], plan, w)
    with pytest.raises(ValueError, match="add must"):
        pql.moe_combine(y, plan, w, add=torch.zeros(4, 63, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="out must"):
        pql.moe_combine(y, plan, w, out=torch.zeros(4, 64))


def test_rejected_calls_are_logged():
    code = ("import ctypes, precision_quantized_linear_amd as p; L = p.lib();"
            "L.pql_moe_plan(None, 4, 2, 0, None, None, None, None, 0, None);"
            "L.pql_moe_qgemm(3, None, None, 0, 0, None, None, None, None, 4, 2, 8, 256, 256, None, 256, None)")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, PQL_LOG="1"), capture_output=True,
                       text=True, timeout=300)
    lines = [x for x in r.stderr.splitlines() if x.startswith("[pql] ")]
    assert lines == ["[pql] moe_plan T=4 k=2 E=0: rejected (status 1): E must be 1 .. 1024 (got 0)",
                     "[pql] moe_qgemm MXFP8 T=4 k=2 E=8 N=256 K=256: rejected (status 2): "
                     "defined for FP8_ROW and FP8_BLOCK128 only (got MXFP8)"]


@pytest.mark.parametrize("scheme,T,k,E,N,K", [
    ("fp8_block128", 4, 2, 8, 200, 256), ("fp8_row", 4, 2, 8, 256, 100), ("fp8_block128", 4, 2, 8, 256, 200),
    ("fp8_row", 1 << 23, 2, 8, 256, 256), ("fp8_block128", (1 << 24) - 1, 32, 8, 256, 256), ("fp8_row", 1 << 24, 1, 8, 256, 256),
    ("fp8_row", 4, 2, 1024, 1 << 20, 1 << 20), ("fp8_row", 4, 2, 8, 1 << 20, 1 << 18), ("fp8_row", 4, 2, 8, (1 << 20) + 1, 256),
    ("fp8_row", (1 << 24) - 1, 1, 8, 1 << 17, 256), ("fp8_row", 4, 33, 64, 256, 256), ("fp8_row", 4, 2, 1025, 256, 256), ("fp8_row", -1, 2, 8, 256, 256),
    ("fp8_row", 4, 2, 8, 256, 1 << 21), ("fp8_row", 4, 0, 8, 256, 256), ("fp8_row", 4, 2, 0, 256, 256), ("int8_row", 4, 2, 8, 256, 256)])
@pytest.mark.parametrize("gather", [0, 1])
def test_no_kernel_is_named_for_a_refused_product(scheme, T, k, E, N, K, gather):
    """Every shape that pql_moe_qgemm refuses has the name "", and asking leaves the error text alone."""
    rows = T if gather else T * k
    assert _gemm(pql.SCHEMES[scheme], rows=rows, gather=gather, T=T, k=k, E=E, N=N, K=K, ldc=N) in (INVALID, UNSUPPORTED)
    before = pql.lib().pql_last_error()
    assert pql.moe_kernel_name(scheme, T, k, E, N, K, gather) == ""
    assert pql.lib().pql_last_error() == before


@pytest.mark.parametrize("scheme,N", [("fp8_block128", 256), ("fp8_row", 200), ("fp8_row", 1)])
def test_kernels_are_named_for_accepted_products(scheme, N):
    for T, k in ((1, 1), (37, 6), ((1 << 24) - 1, 1), ((1 << 19) - 1, 32)):
        assert pql.moe_kernel_name(scheme, T, k, 64, N, 512).startswith("k_moe_")
