"""What the binding makes of a batch's rules, on the host: tensors in host memory
pass its checks where the device's index is that of host memory (-1). No kernel
is launched here."""
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from w4a16_grouped_moe_amd import binding as B

HOST = -1


@pytest.fixture(autouse=True)
def _host_tensors(monkeypatch):
    monkeypatch.setattr(B, "_gpu", lambda t, name: HOST)


def _ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("with_row", [False, True])
def test_a_mask_of_no_words_is_too_short(with_row):
    # rows of no words lie nowhere in memory: they are refused as any other rows
    # that are too short, and not taken for no mask
    x = torch.zeros(3, 40)
    for words in (0, 1):
        rules = dg.LogitRules(mask=_ints(3, words), mask_row=_ints(3) if with_row else None)
        with pytest.raises(ValueError, match=f"mask has {words} words"):
            B._logits(x, rules, HOST)
    B._logits(x, dg.LogitRules(mask=_ints(3, 2), mask_row=_ints(3) if with_row else None), HOST)


def test_a_mask_of_no_rows_that_no_row_has():
    # every place of mask_row is outside a mask of no rows: no row has one
    for words in (0, 1, 2):
        B._logits(torch.zeros(3, 40), dg.LogitRules(mask=_ints(0, words), mask_row=_ints(3)), HOST)
    with pytest.raises(ValueError, match="reach 0 rows"):
        B._logits(torch.zeros(3, 40), dg.LogitRules(mask=_ints(0, 2)), HOST)


def test_rules_of_no_sequences():
    # a batch none of whose rows has a sequence: biases as well as tokens and scales
    # are absent then (biases without an address were handed on, which the call refuses)
    none = dict(tokens=_ints(0, 5), lengths=_ints(0), repetition=torch.zeros(0), scale=torch.zeros(0),
                bias_ids=_ints(0, 4), bias=torch.zeros(0, 4))
    for kw in (none, {k: none[k] for k in ("bias_ids", "bias")}):
        rules = dg.LogitRules(row_seq=torch.full((3,), -1, dtype=torch.int32), **kw)
        assert (rules._c.sequences, rules._c.n_bias, rules._c.tokens) == (0, 0, None)
        B._logits(torch.zeros(3, 40), rules, HOST)
        # the library's own checks (of no rows: nothing is launched)
        assert dg.lib().dgw4_adjust_logits(None, 0, 0, 40, 40, rules._ref, None, 0, 40, None) == B.OK
    one = dg.LogitRules(bias_ids=_ints(1, 4), bias=torch.zeros(1, 4))
    assert (one._c.sequences, one._c.n_bias) == (1, 4)


def test_masks_of_either_sign():
    for dtype in (torch.int32, torch.uint32):
        B._logits(torch.zeros(3, 40), dg.LogitRules(mask=torch.zeros((3, 2), dtype=dtype)), HOST)
    with pytest.raises(TypeError):
        dg.LogitRules(mask=torch.zeros((3, 2), dtype=torch.int64))
