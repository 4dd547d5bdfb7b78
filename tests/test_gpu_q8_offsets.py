"""Rows of an 8-bit cache under offsets that are out of order: what is stored and read is right, and nothing else changes."""
import numpy as np
import pytest
import torch

from gqa_decode_attention_fa_gb300 import binding
from test_gpu_q8 import Cache, errors, i32, quantised, rows_of, values

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("at,every", [
    ([0, 50, 3, 9, 9, 9, 12], False),
    ([0, 5, 3, 9, 9, 9, 12], False),
    ([7, 6, 5, 4, 3, 2, 1], False),
    ([0, 3, 6, 2, 8, 12, 11], False),
    ([-2, 3, 6, 9, 10, 11, 12], True),       # ascending ones that begin below 0 or end behind the last row
    ([0, 3, 6, 9, 10, 11, 13], True),
    ([-9, -9, -1, 0, 5, 12, 99], True),
])
def test_offsets_out_of_order(fmt, paged, at, every):
    B, Hkv, cap, N = 6, 3, 70, 12
    c = Cache(B, Hkv, cap, fmt, paged)
    start = [60, 0, 3, 7, 1, 55]
    k, v = rows_of(1, N, Hkv), rows_of(2, N, Hkv)
    before = [bits(t) for t in c.tensors]
    good = [b for b in range(B) if 0 <= at[b] <= at[b + 1] <= N]
    err = errors()
    binding.q8_append(B, Hkv, N, cap, k, v, *c.tensors, c.table, i32(at), i32(start), device_errors=err, **c.layout)
    assert err.item() == binding.DEVERR_SEQLEN
    after = [bits(t) for t in c.tensors]
    same = np.logical_and.reduce([(x == y).reshape(c.rows, -1).all(1) for x, y in zip(after, before)])
    stored, other = {}, np.ones(c.rows, bool)
    want = [quantised(x.double().cpu().numpy(), fmt) for x in (k, v)]
    for b in good:
        for i, row in enumerate(c.slots(b, start[b], at[b + 1] - at[b])):
            other[row] = False
            if not same[row]:
                stored[b, i] = row
                for (codes, scale), got, f in zip(want, (c.k, c.v), (c.ks, c.vs)):
                    assert (values(got)[row] == codes[at[b] + i]).all() and (f[row].cpu().numpy() == scale[at[b] + i]).all()
    assert same[other].all()
    if every:
        assert len(stored) == sum(at[b + 1] - at[b] for b in good)
    # read back: a row that changes is the slot of a sequence that holds it
    ko, vo = rows_of(3, N, Hkv), rows_of(4, N, Hkv)
    old = ko.clone(), vo.clone()
    err.zero_()
    binding.q8_read(B, Hkv, N, cap, *c.tensors, c.table, i32(at), i32(start), ko, vo, device_errors=err, **c.layout)
    assert err.item() == binding.DEVERR_SEQLEN
    dense = [x.reshape(c.rows, Hkv, 128) for x in c.dense()]
    for n in range(N):
        mine = [c.slots(b, start[b] + n - at[b], 1)[0] for b in good if at[b] <= n < at[b + 1]]
        left = torch.equal(ko[n], old[0][n]) and torch.equal(vo[n], old[1][n])
        assert left or any(all((np.abs(x[n].double().cpu().numpy() - y[r]) <= 2.0 ** -8 * (1 + 2.0 ** -12) * np.abs(y[r])).all()
                               for x, y in zip((ko, vo), dense)) for r in mine)
        assert not (every and mine and left)
