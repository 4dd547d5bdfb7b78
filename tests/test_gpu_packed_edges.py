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


@pytest.mark.parametrize("qa,ka", [
    ([0, 40, 20, 130, 180], None),
    ([-5, 40, 100, 130, 180], None),
    ([0, 40, 100, 130, 200], None),
    ([10, 5, 60, 60, 170], None),
    ([0, 40, 100, 130, 170], [0, 50, 30, 150, 181]),     # the keys' alone: a sequence without keys
    ([0, 40, 30, 130, 170], [-1, 50, 60, 150, 999]),
])
def test_offsets_out_of_order(qa, ka):
    """Each sequence by its own offsets: one with bad ones is left out, its rows and those of none as they were, the others as ever
    (but in rows that two of them hold)."""
    w = make(8, 2, [180], [180], seed=33)
    N = len(w["out"])
    w["qa"], w["ka"], w["given"] = np.array(qa), np.array(qa if ka is None else ka), ka is not None
    out, err = run(w)
    assert err == binding.DEVERR_SEQLEN
    ref, mag, owners = w["out"].double().clone(), torch.zeros(w["out"].shape, dtype=torch.float64, device="cuda"), np.zeros(N, int)
    for b in range(4):
        (x, y), (j, k) = w["qa"][b:b + 2], w["ka"][b:b + 2]
        if not 0 <= x <= y <= N:
            continue
        if not 0 <= j <= k <= N:
            j = k = 0
        owners[x:y] += 1
        o, m = attend({**w, "qa": np.array([x, y]), "ka": np.array([j, k])})
        ref[x:y], mag[x:y] = o[x:y], m[x:y]
    one = torch.as_tensor(owners == 1, device="cuda")
    near(out[one], ref[one], mag[one], norm=False)
    none = torch.as_tensor(owners == 0, device="cuda")
    assert bool(none.any()) and torch.equal(out[none], w["out"][none])
