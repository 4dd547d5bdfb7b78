"""Attention over packed prompts at its edges: rows whose every score is -infinity, and offsets that are out of order."""
import numpy as np
import pytest
import torch

from gqa_decode_attention_fa_gb300 import binding
from test_gpu_packed import D, attend, make, near, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv", [(40, 8), (8, 8), (16, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_whose_every_score_is_minus_infinity(Hq, Hkv, causal):
    """They are zeros, be the values that they see finite or not, in tiles that all rows see or on the diagonal; rows with other scores
    see those values."""
    n = [300, 70, 1]
    w = make(Hq, Hkv, n, [x + 20 for x in n], seed=31)
    at = w["qa"]
    w["k"][..., 5] = float("-inf")
    w["q"][..., 5] = 1.0
    lone = torch.tensor([0, 60, 200, 299, int(at[1]) + 40], device="cuda")  # rows that see finite scores too: 0 x -inf there is NaN
    for j in (3, 90, 150, 318, int(w["ka"][1]) + 50):
        w["v"][j, :, j % D] = float("inf") if j % 2 else float("nan")
    out, err = run(w, causal)
    assert err == 0 and bool((out[:at[-1]] == 0).all()) and torch.equal(out[at[-1]:], w["out"][at[-1]:])
    w["q"][lone, :, 5] = 0.0
    out, err = run(w, causal)
    rest = torch.ones(int(at[-1]), dtype=torch.bool, device="cuda")
    rest[lone] = False
    assert err == 0 and bool((out[:at[-1]][rest] == 0).all()) and bool(torch.isnan(out[lone]).all())
