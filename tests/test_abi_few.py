"""The few-token entry points on the host: their argument checks, before any
HIP call. No kernel is launched here."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import w4a16_grouped_moe_amd as dg
from tests import few_ref
from w4a16_grouped_moe_amd import binding as B

P = 1 << 12


def _few(routed=False, **kw):
    a = dict(x=P, ids=P, w=P, lg=P, T=4, topk=2, E=8, d=512, m=192, gq=P, gs=P, gz=P, gg=128,
             dq=P, ds=P, dz=P, dg=64, ws=P, out=P, n=1 << 30)
    a.update(kw)
    n = None if a["n"] is None else ctypes.byref(ctypes.c_size_t(a["n"]))
    head = (a["x"], a["lg"]) if routed else (a["x"], a["ids"], a["w"])
    f = dg.lib().dgw4_moe_few_routed if routed else dg.lib().dgw4_moe_few
    return f(*head, a["T"], a["topk"], a["E"], a["d"], a["m"], a["gq"], a["gs"], a["gz"], a["gg"],
             a["dq"], a["ds"], a["dz"], a["dg"], a["ws"], n, a["out"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), B.ERR_INVALID_ARG),
    (dict(gq=None), B.ERR_INVALID_ARG),
    (dict(gs=None), B.ERR_INVALID_ARG),
    (dict(gz=None), B.ERR_INVALID_ARG),
    (dict(dq=None), B.ERR_INVALID_ARG),
    (dict(ds=None), B.ERR_INVALID_ARG),
    (dict(dz=None), B.ERR_INVALID_ARG),
    (dict(out=None), B.ERR_INVALID_ARG),
    (dict(n=None), B.ERR_INVALID_ARG),
    (dict(T=-1), B.ERR_INVALID_ARG),
    (dict(topk=0), B.ERR_INVALID_ARG),
    (dict(topk=9), B.ERR_INVALID_ARG),                 # > E
    (dict(E=1025), B.ERR_INVALID_ARG),
    (dict(E=0), B.ERR_INVALID_ARG),
    (dict(d=500), B.ERR_INVALID_ARG),
    (dict(m=100), B.ERR_INVALID_ARG),
    (dict(gg=96), B.ERR_UNSUPPORTED),
    (dict(dg=32), B.ERR_UNSUPPORTED),
    (dict(gg=0), B.ERR_INVALID_ARG),
    (dict(gg=128 | B.ROWS_TILES), B.ERR_INVALID_ARG),
    (dict(gg=128 | B.ROWS_CHUNKS), B.ERR_INVALID_ARG),
    (dict(dg=64 | 0x80000), B.ERR_INVALID_ARG),
    (dict(T=257), B.ERR_UNSUPPORTED),                  # 514 assignments
    (dict(T=2**30), B.ERR_UNSUPPORTED),
    (dict(d=1 << 20, m=2048), B.ERR_UNSUPPORTED),      # one expert's weights from 2 GiB
    (dict(ws=P + 64), B.ERR_INVALID_ARG),
    (dict(x=P + 8), B.ERR_INVALID_ARG),
    (dict(gz=P + 2), B.ERR_INVALID_ARG),
    (dict(dq=P + 4), B.ERR_INVALID_ARG),
    (dict(out=P + 4), B.ERR_INVALID_ARG),
    (dict(n=16), B.ERR_WORKSPACE),
])
@pytest.mark.parametrize("routed", [False, True])
def test_few_rejects(routed, kw, code):
    assert _few(routed, **kw) == code


def test_few_route_arguments():
    assert _few(ids=None) == B.ERR_INVALID_ARG
    assert _few(w=None) == B.ERR_INVALID_ARG
    assert _few(ids=P + 2) == B.ERR_INVALID_ARG
    assert _few(w=P + 1) == B.ERR_INVALID_ARG
    assert _few(True, lg=None) == B.ERR_INVALID_ARG
    assert _few(True, lg=P + 2) == B.ERR_INVALID_ARG
    assert _few(True, E=80, topk=65) == B.ERR_INVALID_ARG
    for routed in (False, True):
        assert _few(routed, T=0, x=None, ids=None, w=None, lg=None, out=None) == B.OK


def test_few_workspace():
    # the intermediate, the router's ids and weights, the tile list, and past 64
    # assignments their outputs, each in whole 256 bytes
    assert dg.moe_few_workspace_bytes(1, 8, 128, 2816, 704) == 8 * 704 * 2 + 2 * 256 + 6400
    assert dg.moe_few_workspace_bytes(8, 8, 128, 2816, 704) == 64 * 704 * 2 + 2 * 256 + 6400
    assert dg.moe_few_workspace_bytes(64, 8, 128, 2816, 704) == 512 * 704 * 2 + 2 * 2048 + 6400 + 512 * 2816 * 4
    assert dg.moe_few_workspace_bytes(0, 8, 128, 2816, 704) == 0
    with pytest.raises(dg.Dgw4Error, match="UNSUPPORTED"):
        dg.moe_few_workspace_bytes(65, 8, 128, 2816, 704)


def test_quantize_rows_rejects():
    f = dg.lib().dgw4_quantize_rows_i8
    ok = dict(x=P, t=1, rows=4, K=100, ldx=100, q=P, ldq=112, s=P)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["x"], a["t"], a["rows"], a["K"], a["ldx"], a["q"], a["ldq"], a["s"], None)

    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(t=3), dict(t=-1), dict(rows=-1),
               dict(K=0), dict(K=2**31 - 1, ldx=2**31), dict(ldx=99), dict(ldq=100), dict(ldq=96),
               dict(ldq=120), dict(q=P + 8), dict(x=P + 1), dict(t=0, x=P + 2), dict(s=P + 2)):
        assert call(**kw) == B.ERR_INVALID_ARG, kw
    assert call(rows=0, x=None, q=None, s=None) == B.OK


def test_quantize_rows_longest():
    # the longest row there is room for in 32 bits with its padding, and one more
    f = dg.lib().dgw4_quantize_rows_i8
    for K, code in ((2**31 - 17, B.OK), (2**31 - 16, B.ERR_INVALID_ARG)):
        assert f(None, 1, 0, K, 2**31, None, 2**31, None, None) == code


def test_w8a8_rejects():
    f = dg.lib().dgw4_w8a8_linear
    ok = dict(xq=P, xs=P, T=4, K=64, ldx=64, wq=P, ws=P, N=5, ldw=64, y=P, t=1, ldy=5)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["xq"], a["xs"], a["T"], a["K"], a["ldx"], a["wq"], a["ws"], a["N"], a["ldw"],
                 a["y"], a["t"], a["ldy"], None)

    for kw in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(y=None), dict(T=-1),
               dict(K=0), dict(N=0), dict(ldx=48), dict(ldx=72), dict(ldw=48), dict(ldw=72),
               dict(ldy=4), dict(t=7), dict(xq=P + 8), dict(wq=P + 4), dict(xs=P + 2), dict(ws=P + 1),
               dict(y=P + 1), dict(t=0, y=P + 2)):
        assert call(**kw) == B.ERR_INVALID_ARG, kw
    for kw in (dict(K=40, ldx=48, ldw=48), dict(K=131072, ldx=131072, ldw=131072),
               dict(ldx=(1 << 22) + 16), dict(ldw=(1 << 22) + 16), dict(T=2**31 - 1),
               dict(N=2**31 - 1, ldy=2**31)):
        assert call(**kw) == B.ERR_UNSUPPORTED, kw
    assert call(T=0, xq=None, xs=None, y=None) == B.OK


def test_w8a8_tokens_rejects():
    f = dg.lib().dgw4_w8a8_linear_tokens
    ok = dict(x=P, xt=1, T=4, K=50, ldx=50, wq=P, ws=P, N=5, ldw=64, y=P, t=1, ldy=5, b=P, n=1 << 20)

    def call(**kw):
        a = {**ok, **kw}
        n = None if a["n"] is None else ctypes.byref(ctypes.c_size_t(a["n"]))
        return f(a["x"], a["xt"], a["T"], a["K"], a["ldx"], a["wq"], a["ws"], a["N"], a["ldw"],
                 a["y"], a["t"], a["ldy"], a["b"], n, None)

    for kw in (dict(x=None), dict(wq=None), dict(ws=None), dict(y=None), dict(n=None), dict(T=-1),
               dict(K=0), dict(N=0), dict(xt=5), dict(t=5), dict(ldx=49), dict(ldw=48), dict(ldw=72),
               dict(ldy=4), dict(x=P + 1), dict(xt=0, x=P + 2), dict(wq=P + 8), dict(b=P + 16),
               dict(y=P + 1)):
        assert call(**kw) == B.ERR_INVALID_ARG, kw
    assert call(n=16) == B.ERR_WORKSPACE
    assert call(K=131057, ldx=131057, ldw=131072) == B.ERR_UNSUPPORTED
    assert call(ldw=(1 << 22) + 16) == B.ERR_UNSUPPORTED
    assert call(T=0, x=None, y=None) == B.OK
    assert call(T=0, b=None) == B.OK                       # a query
    assert dg.w8a8_workspace_bytes(1, 1) == 512
    assert dg.w8a8_workspace_bytes(16, 2803) == 16 * 2816 + 256


def test_binding_rejects_host_tensors():
    x = torch.zeros((2, 32), dtype=torch.float16)
    with pytest.raises(ValueError, match="ROCm"):
        dg.quantize_rows_i8(x)
    q = torch.zeros((2, 32), dtype=torch.int8)
    with pytest.raises(ValueError, match="ROCm"):
        dg.w8a8_linear(q, torch.ones(2), (q, torch.ones(2)))
    with pytest.raises(TypeError):
        dg.quantize_rows_i8([[1.0]])


def test_binding_refuses_sizes_past_32_bits():
    # the C ABI takes 32-bit sizes: a larger one is refused, not taken modulo 2^32
    big = 2**32 + 1
    for shape in ((big, 16), (1, big), (2**31, 1)):
        t = torch.empty(shape, dtype=torch.int8, device="meta")
        with pytest.raises(ValueError, match="32 bits"):
            B._rows(t, "x", B._I8, t.get_device())
    edge = torch.empty((1, 2**31 - 1), dtype=torch.int8, device="meta")
    assert B._rows(edge, "x", B._I8, edge.get_device())[1:3] == (1, 2**31 - 1)
    for args in ((big, 8, 128, 2816, 704), (1, big, 128, 2816, 704), (1, 8, big, 2816, 704),
                 (1, 8, 128, 2816 + 2**32, 704), (1, 8, 128, 2816, 704 - 2**32),
                 (1, 8, 128, 2816, 704, 2**32 + 128), (1, 8, 128, 2816, 704, 128, 2**32 + 64)):
        with pytest.raises(ValueError, match="32 bits"):
            dg.moe_few_workspace_bytes(*args)
    for T, K in ((big, 16), (1, big)):
        with pytest.raises(ValueError, match="32 bits"):
            dg.w8a8_workspace_bytes(T, K)
    x, lg = torch.zeros((1, 64), dtype=torch.float16), torch.zeros((1, 4))
    w = (torch.zeros((4, 2, 2), dtype=torch.uint8),)
    with pytest.raises(ValueError, match="32 bits"):
        dg.moe_few_routed(x, lg, 2**32 + 2, w, w)


def test_binding_refuses_an_empty_workspace():
    none, one = torch.empty(0, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        B._workspace(none, 1, none.get_device())
    B._workspace(none, 0, none.get_device())
    assert B._workspace(one, 1, one.get_device())[0] == one.data_ptr()


def test_plain_form_agrees_with_the_oracle():
    # the 64-bit form the GPU tests use, against the oracle's layer
    rng = np.random.default_rng(1)
    T, E, topk, d, m = 6, 5, 3, 256, 128
    gw = rng.standard_normal((E, 2 * m, d), dtype=np.float32) * np.float32(0.02)
    dw = rng.standard_normal((E, d, m), dtype=np.float32) * np.float32(0.02)
    gu = (*oracle.quantize_rtn(gw, 128), 128)
    dn = (*oracle.quantize_rtn(dw, 64), 64)
    x = rng.standard_normal((T, d), dtype=np.float32).astype(np.float16)
    ids, w = oracle.router(rng.standard_normal((T, E), dtype=np.float32), topk)
    ids[2, 1] = ids[2, 0]                      # the same expert twice
    ref = oracle.moe_forward(x, ids, w.astype(np.float32), gu, dn, E)
    as_f16 = lambda p: (p[0], *(v.view(np.float16) for v in p[1:3]), p[3])
    out, bound = few_ref.moe(x, ids, w.astype(np.float32), as_f16(gu), as_f16(dn), E)
    assert np.abs(out - ref).max() <= 1e-12 * np.abs(ref).max()
    assert (bound < 0.02 * np.abs(ref).max()).all()
