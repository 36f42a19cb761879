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
