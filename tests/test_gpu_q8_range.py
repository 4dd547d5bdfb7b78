"""One token's attention over an 8-bit cache at the ends of binary32's range: weights, V scales and their products that
leave it where the result does not, and scores so large that a logarithm beside them has no bits left.

A query has one dim that is not zero, so a score is one product of binary32 numbers: the code times powers of two, a scale and
log2(e) / sqrt(128) rounded once, each product by 2^-24.  With scores of at most S in size a weight is off by at most 2^-21 S
relatively (both its own score and the largest), which the tests add to the tolerance of test_gpu_q8.py; half of the least
bf16 step, 2^-134, where the result is smaller than bf16's normal numbers; and n Q 2^-32 of the largest product of a weight and
a scale for products of many sizes (derived there); and the keys whose weights may count as 0: a weight is 2^x beside the largest score
its warp holds, at most 8 below the largest so far, times 2^y that joins the warps, and either is 0 below 2^-126, the smallest
normal number; so those below 2^-118 of the largest key's."""
import numpy as np
import pytest
import torch

from test_gpu_q8 import Cache, MOST, D, near, token, values

pytestmark = pytest.mark.gpu
CODE = 64.0  # of a key's one dim: a level of both formats


def scored(c, scores, Hq):
    """Keys of `scores` [B, cap, Hkv] (natural logarithms); the queries for them."""
    k = c.k.view(c.B, c.cap, c.Hkv, D)
    k[..., 0] = torch.where(scores < 0, -CODE, CODE).to(k.dtype)
    c.ks = (scores.abs() * (D ** 0.5 / CODE)).float().view(c.B * c.cap, c.Hkv).contiguous()
    q = torch.zeros(c.B, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    return q


def attend(c, q, lens):
    """(out, sum_j p_j |v_j|, that sum over keys that may count as 0, the largest p_j vs_j [B, Hq, 1]) in 64 bits."""
    B, Hq, G = *q.shape[:2], q.shape[1] // c.Hkv
    (out, mag, lost), most = np.zeros((3, B, Hq, D)), np.zeros((B, Hq, 1))
    k, v = values(c.k).reshape(B, c.cap, c.Hkv, D), values(c.v).reshape(B, c.cap, c.Hkv, D)
    ks, vs = (x.double().cpu().numpy().reshape(B, c.cap, c.Hkv) for x in (c.ks, c.vs))
    qd = q.double().cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(Hq):
            kv = h // G
            s = (k[b, :n, kv] @ qd[b, h]) * ks[b, :n, kv] / np.sqrt(D)
            p = np.exp(s - s.max())
            small = p < 2.0 ** -118
            p /= p.sum()
            x, y = p * vs[b, :n, kv], np.abs(v[b, :n, kv])
            out[b, h], mag[b, h], lost[b, h], most[b, h] = x @ v[b, :n, kv], np.abs(x) @ y, np.abs(x) * small @ y, np.abs(x).max()
    return out, mag, lost, most


def check(c, q, lens, size):
    out, err = token(c, q, lens, q.shape[1])
    ref, mag, lost, most = attend(c, q, lens)
    assert err == 0 and bool(torch.isfinite(out).all())
    near(out, ref, mag, 2.0 ** -21 * size * mag + lost + 2.0 ** -134 + max(lens) * MOST[c.fmt] * 2.0 ** -32 * most)
    again, _ = token(c, q, lens, q.shape[1])
    assert torch.equal(out, again)
    return out


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("cap", [300, 2500])
@pytest.mark.parametrize("first", [0, 9, 200])
def test_zeros_far_above_small_values(fmt, cap, first):
    """A key with the largest score and a V row of zeros, every other 60 to 87 below it with V scales of 2^-20 to 2^-70: the
    products of a weight and a scale lie around the least binary32 number."""
    B, Hq, Hkv = 5, 8, 4
    c = Cache(B, Hkv, cap, fmt, False)
    scores = torch.zeros(B, cap, Hkv, device="cuda", dtype=torch.float64)
    scores[:, first] = torch.tensor([60.0, 68, 75, 81, 87], device="cuda", dtype=torch.float64)[:, None]
    vs = c.vs.view(B, cap, Hkv)
    vs *= torch.exp2(torch.tensor([-20.0, -31, -50, -70], device="cuda"))
    vs[:, first] = 0
    c.v.view(torch.uint8).view(B, cap, Hkv, D)[:, first] = 0
    check(c, scored(c, scores, Hq), [cap, cap - 1, cap - 64, cap, cap - 9], 87)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("cap", [300, 2500])
def test_zeros_rise_above_the_least_values(fmt, cap):
    """V scales of 2^-140, then in every other eight units of 16 keys one of zeros 30 (log2) above all before it and one with such a
    scale 12 below that."""
    B, Hq, Hkv = 3, 4, 2
    c = Cache(B, Hkv, cap, fmt, False)
    scores = torch.zeros(B, cap, Hkv, device="cuda", dtype=torch.float64)
    slot = torch.arange(cap, device="cuda")
    late = slot // 128 % 2 == 1
    zero = late & (slot % 16 == 3)
    scores[:, zero] = 30 * np.log(2.0)
    scores[:, late & (slot % 16 == 11)] = 18 * np.log(2.0)
    c.vs = torch.full_like(c.vs, 2.0 ** -140)
    c.vs.view(B, cap, Hkv)[:, zero] = 0
    check(c, scored(c, scores, Hq), [cap, cap - 5, 256], 21)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("cap", [300, 2500])
def test_weights_and_scales_of_many_sizes(fmt, cap):
    """Scores over 150 binades, V scales over 250, a third of the V rows zeros."""
    B, Hq, Hkv = 6, 8, 4
    c = Cache(B, Hkv, cap, fmt, False, seed=3)
    g = torch.Generator(device="cuda").manual_seed(8)
    draw = lambda lo, hi: torch.randint(lo, hi, (B, cap, Hkv), generator=g, device="cuda").double()  # noqa: E731
    scores = draw(-150, 1) * np.log(2.0) * (torch.arange(B, device="cuda") % 3 + 1)[:, None, None] / 3
    rise = torch.arange(cap, device="cuda").double()[None, :, None] / cap * 100
    scores[B // 2:] += rise - 100
    vs = c.vs.view(B, cap, Hkv)
    vs *= torch.exp2(draw(-140, 100)).float()
    zero = draw(0, 3) == 0
    vs[zero] = 0
    check(c, scored(c, scores, Hq), [cap, 77, cap - 1] * 2, 210)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("cap", [300, 2500])
def test_a_weight_times_a_large_scale(fmt, cap):
    """V rows of 3e38: a weight of up to 2^8, which a key has whose score passes the maximum held by less than 8 (log2), times
    their scales is beyond binary32, their mean is not."""
    B, Hq, Hkv = 2, 4, 2
    c = Cache(B, Hkv, cap, fmt, False)
    slot = torch.arange(cap, device="cuda")
    scores = torch.zeros(B, cap, Hkv, device="cuda", dtype=torch.float64)
    top = slot == 16 * 8 + 5                    # in the second unit of a warp
    scores[:, top] = 7.9 * np.log(2.0)
    c.vs = torch.full_like(c.vs, 1e20)
    c.vs.view(B, cap, Hkv)[:, top] = 3e38 / MOST[fmt]
    c.v.view(B, cap, Hkv, D)[:, top, :, ::2] = torch.tensor(MOST[fmt], device="cuda").to(c.v.dtype)
    out = check(c, scored(c, scores, Hq), [cap, 200], 6)
    assert bool((out[1, :, ::2] > 1e38).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Hkv,cap", [(2, 300), (2, 2500), (1, 40000)])
def test_means_near_the_largest_number(fmt, Hkv, cap):
    """All V rows alike, of 3e38: so is their mean, whatever the warps and ranges (a hundred in the longest) it is joined from."""
    B, Hq = 3, 4
    c = Cache(B, Hkv, cap, fmt, False)
    c.vs = torch.full_like(c.vs, 3e38 / MOST[fmt])
    sign = 1 - 2 * (torch.arange(D, device="cuda") % 2).float()
    c.v.view(B, cap, Hkv, D)[:] = (MOST[fmt] * sign).to(c.v.dtype)
    scores = torch.randn(B, cap, Hkv, device="cuda", dtype=torch.float64, generator=torch.Generator(device="cuda").manual_seed(2))
    out = check(c, scored(c, scores, Hq), [cap, 33, cap - 17], 6)
    assert bool((out.abs() > 2.9e38).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Hkv,cap", [(3, 300), (3, 2500), (1, 40000)])
@pytest.mark.parametrize("power", [0, 12, 20, 26, 30, 100])
def test_tied_keys_with_large_scores(fmt, Hkv, cap, power):
    """Keys with one score of 2^power (log2), spread unevenly over warps and ranges, all others 0: the mean of their values.  (At
    2^0 the others have weights too.)"""
    B, Hq = 3, 6
    c = Cache(B, Hkv, cap, fmt, False)
    scores = torch.zeros(B, cap, Hkv, device="cuda", dtype=torch.float64)
    at = [4, 5, 7, 30, cap // 2, cap // 2 + 1, cap - 90, cap - 89, cap - 88, cap - 87, cap - 86, cap - 40, cap - 11]
    scores[:, at] = 2.0 ** power * np.log(2.0)
    # (bit-equal scores: the others lie 2^power below, beyond every weight but at 2^0, so their size is no source of error)
    check(c, scored(c, scores, Hq), [cap, cap - 20, cap - 87], 2)
