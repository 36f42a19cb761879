"""The entry points at the end of a step on the host: their argument checks,
before any HIP call. No kernel is launched here."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import w4a16_grouped_moe_amd as dg
from tests import rules_ref
from w4a16_grouped_moe_amd import binding as B

P = 1 << 12
BAD, NO = B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED


def _linear(**kw):
    a = dict(x=P, xt=1, T=4, K=256, ldx=256, q=P, s=P, z=P, N=32, g=64, y=P, yt=0, ldy=32)
    a.update(kw)
    return dg.lib().dgw4_w4a16_linear_few(*[a[k] for k in ("x", "xt", "T", "K", "ldx", "q", "s", "z", "N",
                                                           "g", "y", "yt", "ldy")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BAD), (dict(q=None), BAD), (dict(s=None), BAD), (dict(z=None), BAD), (dict(y=None), BAD),
    (dict(T=-1), BAD), (dict(T=65), NO), (dict(K=0), BAD), (dict(K=255, ldx=256), BAD), (dict(K=320, g=128, ldx=320), BAD),
    (dict(N=0), BAD), (dict(ldx=255), BAD), (dict(ldy=31), BAD), (dict(xt=0), NO), (dict(xt=3), BAD),
    (dict(yt=3), BAD), (dict(yt=-1), BAD), (dict(g=0), BAD), (dict(g=32), NO), (dict(g=-64), BAD),
    (dict(g=64 | B.ROWS_TILES), BAD), (dict(g=64 | B.ROWS_CHUNKS), BAD), (dict(g=64 | 0x80000), BAD),
    (dict(g=64 | B.WEIGHTS_TILED, N=33, ldy=33), BAD), (dict(x=P + 1), BAD), (dict(q=P + 8), BAD), (dict(s=P + 2), BAD),
    (dict(z=P + 8), BAD), (dict(y=P + 2), BAD), (dict(yt=2, y=P + 1), BAD),
    (dict(K=(1 << 24) + 128, ldx=1 << 25), NO), (dict(N=2**31 - 256, ldy=2**31), NO),
])
def test_linear_few_rejects(kw, code):
    assert _linear(**kw) == code


def test_linear_few_of_no_tokens():
    assert _linear(T=0, x=None, q=None, s=None, z=None, y=None) == B.OK


RULES = dict(row_seq=None, tokens=P, lengths=P, prompt_lengths=P, repetition=P, frequency=P, presence=P, scale=P,
             bias_ids=P, bias=P, mask=P, mask_row=P, ld_tokens=100, ld_bias=8, ld_mask=32, sequences=4,
             max_tokens=100, n_bias=8, mask_rows=2)


def _rules(**kw):
    u = B._Rules()
    for k, v in {**RULES, **kw}.items():
        setattr(u, k, v)
    return u


def _adjust(rules=None, **kw):
    a = dict(x=P, t=0, R=4, V=1000, ld=1000, out=1 << 20, ot=0, ldo=1000)
    a.update(kw)
    u = None if rules is False else ctypes.byref(_rules(**(rules or {})))
    return dg.lib().dgw4_adjust_logits(a["x"], a["t"], a["R"], a["V"], a["ld"], u, a["out"], a["ot"],
                                       a["ldo"], None)


def _sample(rules=None, **kw):
    a = dict(x=P, t=0, R=4, V=1000, ld=1000, h=P, s=P, a=P, ws=P, n=1 << 30)
    a.update(kw)
    u = None if rules is False else ctypes.byref(_rules(**(rules or {})))
    n = None if a["n"] is None else ctypes.byref(ctypes.c_size_t(a["n"]))
    return dg.lib().dgw4_sample_adjusted(a["x"], a["t"], a["R"], a["V"], a["ld"], u, 7, a["h"], a["s"],
                                         a["a"], a["ws"], n, None)


BAD_RULES = [
    (dict(sequences=-1), BAD), (dict(n_bias=-1), BAD), (dict(mask_rows=-1), BAD),
    (dict(sequences=3), BAD),                                     # row r is sequence r: four rows
    (dict(tokens=None), BAD),                                     # penalties without tokens
    (dict(lengths=None), BAD), (dict(max_tokens=0), BAD), (dict(ld_tokens=99), BAD),
    (dict(max_tokens=1 << 21, ld_tokens=1 << 21), NO),
    (dict(n_bias=1024, ld_bias=1024), NO), (dict(bias=None), BAD), (dict(bias_ids=None), BAD), (dict(ld_bias=7), BAD),
    (dict(ld_mask=31), BAD), (dict(mask_row=None), BAD),          # four rows, two masks
] + [({k: P + 2}, BAD) for k in ("row_seq", "tokens", "lengths", "prompt_lengths", "repetition", "frequency",
                                 "presence", "scale", "bias_ids", "bias", "mask", "mask_row")]


@pytest.mark.parametrize("rules,code", BAD_RULES)
def test_rules_rejects(rules, code):
    assert _adjust(rules) == code
    assert _sample(rules) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BAD), (dict(R=-1), BAD), (dict(V=0), BAD), (dict(ld=999), BAD), (dict(t=3), BAD),
    (dict(t=-1), BAD), (dict(x=P + 2), BAD), (dict(t=1, x=P + 1), BAD),
    (dict(V=1 << 30, ld=1 << 30, ldo=1 << 30), NO), (dict(R=2**31 - 1, V=1 << 20, ld=1 << 20, ldo=1 << 20), NO),
])
def test_logits_rejects(kw, code):
    assert _adjust(**kw) == code
    kw.pop("ldo", None)
    assert _sample(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(out=None), BAD), (dict(ot=3), BAD), (dict(ldo=999), BAD), (dict(out=(1 << 20) + 2), BAD),
    (dict(t=0, ot=1), NO), (dict(t=1, ot=2), NO),
    # overlaps: shifted, another type, another row distance, rows that run into each other
    (dict(out=P + 4), BAD), (dict(x=P, out=P, t=1, ot=0), BAD), (dict(out=P, ldo=1001), BAD),
    (dict(out=P + 4000, ld=1999, ldo=1999), BAD), (dict(out=P + 7996, ld=1999, ldo=1999), BAD),
    (dict(out=P + 3996, R=1), BAD), (dict(x=P + 3996, out=P, R=1), BAD),
])
def test_adjust_rejects(kw, code):
    assert _adjust(**kw) == code


def test_adjust_of_no_rows():
    assert _adjust(R=0, x=None, out=None) == B.OK
    assert _adjust(False) == BAD and _sample(False) == BAD


def test_sample_rejects():
    assert _sample(n=None) == BAD
    assert _sample(ws=P + 8) == BAD
    for k in ("h", "s", "a"):
        assert _sample(**{k: P + 2}) == BAD
    need = dg.sample_adjusted_workspace_bytes(4, 1000)
    assert need > 0 and _sample(n=need - 1) == B.ERR_WORKSPACE
    assert _sample(R=0, x=None, n=0) == B.OK
    assert _sample(False, ws=None) == B.OK                 # a query needs no rules
    assert dg.sample_adjusted_workspace_bytes(0, 1000) == 0
    with pytest.raises(ValueError, match="32 bits"):
        dg.sample_adjusted_workspace_bytes(2**32 + 1, 4)


def test_layout_of_the_struct():
    # dgw4_logit_rules as the header lays it out: twelve pointers, three
    # long longs, four ints
    assert ctypes.sizeof(B._Rules) == 12 * 8 + 3 * 8 + 4 * 4
    assert B._Rules.sequences.offset == 120 and B._Rules.mask_rows.offset == 132


def test_binding_rejects():
    x = torch.zeros((2, 64), dtype=torch.float16)
    w = (torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.float16),
         torch.zeros((4, 1), dtype=torch.float16), 64)
    with pytest.raises(ValueError, match="ROCm"):
        dg.w4a16_linear_few(x, w)
    with pytest.raises(TypeError):
        dg.w4a16_linear_few([1.0], w)
    with pytest.raises(ValueError, match="ROCm"):
        dg.LogitRules(scale=torch.ones(2))
    with pytest.raises(ValueError, match="ROCm"):
        dg.adjust_logits(x, dg.LogitRules())
    one = torch.ones(2)
    for kw in (dict(tokens=one), dict(lengths=one), dict(bias=one), dict(bias_ids=one)):
        with pytest.raises(ValueError):
            dg.LogitRules(**kw)


def test_plain_forms_agree_with_the_oracle():
    rng = np.random.default_rng(3)
    w = rng.standard_normal((40, 256), dtype=np.float32) * np.float32(0.02)
    q, s, z = oracle.quantize_rtn(w[None], 64)
    x = rng.standard_normal((5, 256), dtype=np.float32).astype(np.float16)
    f16 = lambda v: v[0].view(np.float16)
    y, bound = rules_ref.linear(torch.from_numpy(x), q[0], f16(s), f16(z), 64, torch.float32)
    ref = oracle.w4a16_linear(x, q[0], s[0], z[0], 64)
    assert np.abs(y - ref).max() <= 1e-12 * np.abs(ref).max()
    assert (bound < 1e-3 * np.abs(ref).max()).all()
    l = rng.standard_normal((4, 64)).astype(np.float32)
    h, _ = rules_ref.entropies(l)
    assert np.allclose(h, oracle.sample(l, 1)[0], rtol=1e-12)


def test_plain_rules():
    # one row by hand: token 1 in the prompt, 2 generated twice, 3 in both
    u = dict(tokens=[[1, 3, 2, 2, 3, 9]], lengths=[6], prompt_lengths=[2], repetition=[2.0], frequency=[0.25],
             presence=[1.0], scale=[0.5], bias_ids=[[4, 2, 4, -1]], bias=[[7.0, 1.0, 3.0, 5.0]], mask=[[0b111110]])
    t = {k: torch.tensor(v, dtype=torch.int32 if k in ("tokens", "lengths", "prompt_lengths", "bias_ids", "mask")
                         else torch.float32) for k, v in u.items()}
    l = torch.tensor([[8.0, 4.0, -4.0, 4.0, 1.0, 0.0]])
    got = rules_ref.adjusted(l, t)
    # 1: 4/2; 2: -8 - 0.5 - 1 + 1; 3: 2 - 0.25 - 1; 4: 1 + 3; halves; 0 masked
    assert got.tolist() == [[-np.inf, 1.0, -4.25, 0.375, 2.0, 0.0]]
