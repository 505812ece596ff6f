"""Refusals of the calls around the cache of keys and values that need no GPU: the C ABI's argument checks
(fake pointers, never dereferenced: every call must fail before a launch) and the binding's; the
rotary tables; sizes, workspaces and kernel names."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as pql

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = pql.PQL_ERR_INVALID_ARGUMENT, pql.PQL_ERR_UNSUPPORTED, pql.PQL_ERR_WORKSPACE
P = 1 << 20                      # a fake 16-byte aligned device pointer
BF16, TENSOR, ROW = 0, 1, 2


def _rope(layout=0, x=P, T=4, H=2, D=128, lxt=256, lxh=128, pos=P, freqs=P, rotary=128, scale=1.0, out=P, lot=256,
          loh=128):
    return pql.lib().pql_rope(layout, x, T, H, D, lxt, lxh, pos, freqs, rotary, ctypes.c_float(scale), out, lot, loh, None)


@pytest.mark.parametrize("bad", [
    dict(layout=2), dict(layout=-1), dict(x=None), dict(out=None), dict(pos=None), dict(freqs=None), dict(T=-1),
    dict(H=0), dict(D=0), dict(D=100), dict(D=8, rotary=16), dict(D=1032, lxt=4128), dict(rotary=0), dict(rotary=8),
    dict(rotary=24), dict(rotary=144), dict(scale=math.nan), dict(scale=math.inf), dict(x=P + 8), dict(out=P + 2),
    dict(pos=P + 2), dict(freqs=P + 4), dict(lxt=-8), dict(lxt=260), dict(lxh=132), dict(lot=128), dict(loh=64),
    dict(lot=264), dict(T=1 << 40), dict(T=1 << 31, H=1), dict(T=1 << 28, H=4), dict(lxt=1 << 40),
    dict(lxh=1 << 41), dict(lot=0, T=2),
])
def test_rope_refusals(bad):
    assert _rope(**bad) == INVALID and pql.lib().pql_last_error()


def test_rope_empty_is_a_no_op():
    assert _rope(T=0, x=None, out=None, pos=None, freqs=None) == pql.PQL_OK
    assert _rope(T=0, x=None, out=None, pos=None, freqs=None, rotary=8) == INVALID


CACHES = [
    (dict(scheme=3), UNSUPPORTED), (dict(scheme=-1), UNSUPPORTED), (dict(D=96), INVALID), (dict(D=0), INVALID),
    (dict(D=512), INVALID), (dict(ps=0), INVALID), (dict(ps=8), INVALID), (dict(ps=48), INVALID), (dict(ps=131072), INVALID),
    (dict(n_pages=0), INVALID), (dict(n_pages=-1), INVALID), (dict(n_pages=1 << 27), INVALID), (dict(Hk=0), INVALID),
    (dict(Hk=-1), INVALID), (dict(Hk=1 << 40), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(kc=P + 8), INVALID),
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(vs=P + 4), INVALID),
]


def _append(scheme=ROW, k=P, kt=256, kh=128, v=P, vt=256, vh=128, T=4, slots=P, layout=0, pos=None, freqs=None, rotary=0,
            scale=1.0, kc=P, vc=P, ks=P, vs=P, n_pages=4, ps=16, Hk=2, D=128):
    return pql.lib().pql_kv_append(scheme, k, kt, kh, v, vt, vh, T, slots, layout, pos, freqs, rotary,
                                   ctypes.c_float(scale), kc, vc, ks, vs, n_pages, ps, Hk, D, None)


def _read(scheme=ROW, kc=P, vc=P, ks=P, vs=P, n_pages=4, ps=16, Hk=2, D=128, slots=P, n=4, k=P, kt=256, kh=128, v=P,
          vt=256, vh=128):
    return pql.lib().pql_kv_read(scheme, kc, vc, ks, vs, n_pages, ps, Hk, D, slots, n, k, kt, kh, v, vt, vh, None)


def _attend(scheme=ROW, q=P, qt=512, qh=128, T=4, H=4, kc=P, vc=P, ks=P, vs=P, n_pages=4, ps=16, Hk=2, D=128, starts=P,
            lens=P, pages=P, B=2, width=2, ldp=2, causal=1, window=0, scale=0.1, out=P, ot=512, oh=128, lse=None, ws=P,
            wsb=1 << 40):
    return pql.lib().pql_kv_attention(scheme, q, qt, qh, T, H, kc, vc, ks, vs, n_pages, ps, Hk, D, starts, lens, pages, B,
                                      width, ldp, causal, window, ctypes.c_float(scale), out, ot, oh, lse, ws, wsb, None)


@pytest.mark.parametrize("call", [_append, _read, _attend])
@pytest.mark.parametrize("bad,status", CACHES)
def test_cache_refusals(call, bad, status):
    assert call(**bad) == status and pql.lib().pql_last_error()


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 40), dict(k=None), dict(v=None), dict(slots=None), dict(k=P + 8), dict(v=P + 2),
    dict(slots=P + 2), dict(kt=100), dict(kh=-8), dict(vt=1 << 40), dict(pos=P, freqs=None, rotary=128),
    dict(pos=P, freqs=P, rotary=0), dict(pos=P, freqs=P, rotary=136), dict(pos=P, freqs=P, rotary=128, layout=5),
    dict(pos=P, freqs=P, rotary=128, scale=math.nan), dict(pos=P + 1, freqs=P, rotary=128),
])
def test_append_refusals(bad):
    assert _append(**bad) == INVALID and pql.lib().pql_last_error()


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=1 << 40), dict(slots=None), dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 8),
    dict(slots=P + 1), dict(kt=128), dict(kh=0), dict(vt=0), dict(vh=64), dict(vt=-256),
])
def test_read_refusals(bad):
    assert _read(**bad) == INVALID and pql.lib().pql_last_error()


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(H=3), dict(H=1, Hk=2), dict(H=65536, Hk=1, D=64), dict(B=-1), dict(B=(1 << 20) + 1),
    dict(width=-1), dict(width=1 << 28, ldp=1 << 28), dict(ldp=1), dict(window=-1), dict(scale=math.nan),
    dict(scale=-math.inf), dict(q=None), dict(out=None), dict(starts=None), dict(lens=None), dict(pages=None),
    dict(q=P + 8), dict(out=P + 8), dict(starts=P + 2), dict(lens=P + 1), dict(pages=P + 3), dict(lse=P + 2),
    dict(qt=516), dict(qh=-8), dict(ot=256), dict(oh=0), dict(T=1 << 27, H=64, Hk=64),
    dict(T=1 << 20, B=1 << 20, H=64, Hk=64, D=64, qt=4096, qh=64, ot=4096, oh=64),
])
def test_attention_refusals(bad):
    assert _attend(**bad) == INVALID and pql.lib().pql_last_error()


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(width=-1), dict(ldp=1), dict(ps=0), dict(ps=24), dict(T=-1), dict(T=1 << 31), dict(starts=None),
    dict(lens=None), dict(pages=None), dict(slots=None), dict(pos=None), dict(starts=P + 2), dict(slots=P + 2),
])
def test_slots_refusals(bad):
    a = dict(starts=P, lens=P, pages=P, B=2, width=2, ldp=2, ps=16, T=4, slots=P, pos=P)
    a.update(bad)
    assert pql.lib().pql_kv_slots(*a.values(), None) == INVALID and pql.lib().pql_last_error()


def test_empty_calls_are_no_ops():
    assert _append(T=0, k=None, v=None, slots=None) == pql.PQL_OK
    assert _read(n=0, k=None, v=None, slots=None) == pql.PQL_OK
    assert _attend(T=0, q=None, out=None) == pql.PQL_OK and _attend(B=0, starts=None, lens=None, pages=None) == pql.PQL_OK
    assert pql.lib().pql_kv_slots(None, None, None, 2, 2, 2, 16, 0, None, None, None) == pql.PQL_OK


def test_sizes():
    assert pql.kv_sizes("bf16", 10, 16, 8, 128) == (10 * 16 * 8 * 128 * 2, 0)
    assert pql.kv_sizes("fp8_tensor", 10, 16, 8, 128) == (10 * 16 * 8 * 128, 4)
    assert pql.kv_sizes("fp8_row", 10, 16, 8, 128) == (10 * 16 * 8 * 128, 10 * 16 * 8 * 4)
    with pytest.raises(ValueError):
        pql.kv_sizes("fp8_row", 10, 16, 8, 100)
    with pytest.raises(ValueError):
        pql.kv_sizes("mxfp8", 10, 16, 8, 128)


@pytest.mark.parametrize("T,H,Hk,D,B,width,ps", [(1, 32, 8, 128, 1, 400, 16), (64, 32, 4, 128, 64, 300, 64), (8192, 32, 8, 128, 1, 512, 64),
                                                  (300, 16, 2, 64, 5, 200, 32), (40, 256, 1, 256, 40, 4000, 16)])
def test_workspace(T, H, Hk, D, B, width, ps):
    need = pql.kv_attention_workspace("fp8_row", T, H, Hk, D, B, width, ps)
    name = pql.kv_kernel_name("fp8_row", T, H, Hk, D, B, width, ps)
    assert name and need % 4 == 0
    if need:
        a = dict(T=T, H=H, Hk=Hk, D=D, B=B, width=width, ldp=width, ps=ps, qt=H * D, qh=D, ot=H * D, oh=D)
        assert _attend(**a, ws=None, wsb=0) == WORKSPACE and _attend(**a, wsb=need - 1) == WORKSPACE
        assert _attend(**a, ws=P + 4, wsb=need) == INVALID
    assert pql.kv_attention_workspace("fp8_row", 0, H, Hk, D, B, width, ps) == 0
    assert pql.kv_kernel_name("fp8_row", 0, H, Hk, D, B, width, ps) == ""
    assert pql.kv_kernel_name("fp8_row", T, H, Hk, 100, B, width, ps) == ""


# ---------------------------------------------------------------- the binding
def _cache(scheme="fp8_row", **kw):
    return pql.kv_cache(4, 16, 2, 64, scheme, device="cpu", **kw)


def test_cache_arguments():
    c = _cache("fp8_tensor", k_scale=0.5, v_scale=2.0)
    assert c.k_scales.tolist() == [0.5] and c.v_scales.tolist() == [2.0] and c.k.shape == (4, 2, 16, 64)
    assert _cache().k_scales.shape == (4, 2, 16) and _cache("bf16").k.dtype is torch.bfloat16
    for kw in (dict(scheme="fp8_tensor"), dict(scheme="fp8_tensor", k_scale=1.0), dict(scheme="fp8_row", k_scale=1.0, v_scale=1.0),
               dict(scheme="fp8_tensor", k_scale=0.0, v_scale=1.0), dict(scheme="fp8_tensor", k_scale=math.inf, v_scale=1.0),
               dict(scheme="int8")):
        with pytest.raises(ValueError):
            _cache(**kw)
    with pytest.raises(ValueError):
        pql.kv_cache(4, 17, 2, 64, device="cpu")


def test_binding_refusals():
    """No GPU here: whatever gets past the binding's checks is refused for its device."""
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((3,), dtype=torch.int32)
    t = pql.rope_freqs(64)
    c = _cache()
    starts, lens, pages = torch.zeros(2, dtype=torch.int32), i[:1], torch.zeros((1, 2), dtype=torch.int32)
    bad = [
        lambda: pql.rope(x.float(), i, t), lambda: pql.rope(x[0], i, t), lambda: pql.rope(x, i.long(), t),
        lambda: pql.rope(x, i[:2], t), lambda: pql.rope(x, i, pql.Rope(t.freqs.float())), lambda: pql.rope(x, i, t.freqs),
        lambda: pql.rope(x, i, pql.rope_freqs(128)), lambda: pql.rope(x, i, pql.Rope(t.freqs, 1.0, "odd")),
        lambda: pql.rope(x, i, t, out=x[:2]), lambda: pql.rope(x.transpose(1, 2), i, t), lambda: pql.rope(x, i, t),
        lambda: pql.kv_append(x, x[:2], c, i), lambda: pql.kv_append(x, x, c, i[:1]), lambda: pql.kv_append(x, x, "c", i),
        lambda: pql.kv_append(x, x, c, i, t), lambda: pql.kv_append(x, x, c, i, None, i),
        lambda: pql.kv_append(x[:, :1], x[:, :1], c, i), lambda: pql.kv_append(x, x, c, i),
        lambda: pql.kv_append(x, x, pql.KVCache("fp8_row", 4, 16, 2, 64, c.k, c.v), i),
        lambda: pql.kv_append(x, x, pql.KVCache("odd", 4, 16, 2, 64, c.k, c.v), i),
        lambda: pql.kv_append(x, x, pql.KVCache("bf16", 4, 16, 2, 64, c.k, c.v), i),
        lambda: pql.kv_append(x, x, pql.KVCache("fp8_row", 5, 16, 2, 64, c.k, c.v, c.k_scales, c.v_scales), i),
        lambda: pql.kv_read(c, i.float()), lambda: pql.kv_read(c, i, out=(x, x[:1])), lambda: pql.kv_read(c, i),
        lambda: pql.kv_slots(starts, lens, pages, 16, -1), lambda: pql.kv_slots(starts[:1], lens, pages, 16, 1),
        lambda: pql.kv_slots(starts, lens, pages[0], 16, 1), lambda: pql.kv_slots(starts, lens, pages.long(), 16, 1),
        lambda: pql.kv_attention(x, c, starts[:1], lens, pages), lambda: pql.kv_attention(x[:, :, :32], c, starts, lens, pages),
        lambda: pql.kv_attention(x, c, starts, lens.long(), pages), lambda: pql.kv_attention(x, c, starts, lens, pages[:, ::2].t()),
        lambda: pql.kv_attention(x, c, starts, lens, pages, out=x[:1]), lambda: pql.kv_attention(x, c, starts, lens, pages),
    ]
    for n, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted", n)


# ---------------------------------------------------------------- rotary tables
def test_rope_freqs():
    plain = pql.rope_freqs(64, 10000.0)
    assert plain.freqs.dtype is torch.float64 and plain.scale == 1.0 and plain.layout == "half"
    f = plain.freqs.numpy()
    assert np.allclose(f, [10000.0 ** (-2 * i / 64) for i in range(32)], rtol=1e-15)
    assert np.allclose(pql.rope_freqs(64, scaling=dict(type="linear", factor=4.0)).freqs.numpy(), f / 4, rtol=1e-15)
    ntk = pql.rope_freqs(64, scaling=dict(type="ntk", factor=4.0)).freqs.numpy()
    assert np.isclose(ntk[0], 1.0) and np.isclose(ntk[-1], f[-1] / 4, rtol=1e-12)       # the slowest pair is stretched by the factor
    for kind, lo, hi in (("yarn", 1.0, 32.0), ("bands", 1.0, 4.0)):
        t = pql.rope_freqs(64, scaling=dict(type=kind, factor=8.0, original=4096))
        ratio, turns = t.freqs.numpy() / f, 4096 * f / (2 * math.pi)
        assert np.isclose(ratio[0], 1.0) and np.isclose(ratio[-1], 1 / 8)
        assert (ratio <= 1 + 1e-12).all() and (ratio >= 1 / 8 - 1e-12).all() and (np.diff(ratio) <= 1e-12).all()
        assert np.allclose(ratio[turns > hi * 1.4], 1.0) and np.allclose(ratio[turns < lo / 1.4], 1 / 8)
        assert np.isclose(t.scale, 0.1 * math.log(8) + 1 if kind == "yarn" else 1.0)
    bands = pql.rope_freqs(64, scaling=dict(type="bands", factor=8.0, original=4096, fast=4.0, slow=1.0)).freqs.numpy()
    turns = 4096 * f / (2 * math.pi)
    keep = np.clip((turns - 1) / 3, 0, 1)
    assert np.allclose(bands, f * (keep + (1 - keep) / 8), rtol=1e-14)
    for kw in (dict(dim=60), dict(dim=0), dict(dim=64, base=0.5), dict(dim=64, layout="x"), dict(dim=64, scaling={"type": "?"}),
               dict(dim=64, scaling={"type": "linear"}), dict(dim=64, scaling={"type": "linear", "factor": 0.5}),
               dict(dim=64, scaling={"type": "linear", "factor": 2.0, "original": 1}),
               dict(dim=64, scaling={"type": "yarn", "factor": 2.0}),
               dict(dim=64, scaling={"type": "yarn", "factor": 2.0, "original": 4096, "fast": 1.0, "slow": 2.0})):
        with pytest.raises(ValueError):
            pql.rope_freqs(**kw)


def test_launch_log_names_the_calls():
    """PQL_LOG writes one line a call, a refusal with its reason."""
    code = ("import sys; sys.path.insert(0, %r)\n"
            "import precision_quantized_linear_amd as pql\n"
            "L = pql.lib()\n"
            "L.pql_rope(0, None, 0, 2, 128, 256, 128, None, None, 128, 1.0, None, 256, 128, None)\n"
            "L.pql_kv_append(2, None, 0, 0, None, 0, 0, 4, None, 0, None, None, 0, 1.0, None, None, None, None, 4, 16, 2, 100, None)\n"
            % ROOT)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=dict(os.environ, PQL_LOG="1"))
    assert "[pql] rope T=0 H=2 D=128: nothing to do" in r.stderr, r.stderr
    assert "[pql] kv_append" in r.stderr and "rejected (status 1): a cache's head size" in r.stderr, r.stderr
