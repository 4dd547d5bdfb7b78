"""Rotary append on the GPU against the definition in extended precision (numpy longdouble).

A stored key element must be the bf16 rounding of its exact value unless that lies within the
kernel's error bound of a rounding midpoint (check_rounded_rows); a query element likewise with
a binary32 bound.  The bounds, times the pair's size m r (|y_i| + |y_j|): the angle p f is at
most 2^-53 p from exact (the frequency's own product), 2^-40 covers the double-word
arithmetic of keys and 2^-18 the binary32 arithmetic of queries, as in the decode step."""
import itertools

import numpy as np
import pytest
import torch

import oracle
from _util import K_WINDOW, Q_WINDOW, check_rounded_rows
from gqa_decode_attention_fa_gb300 import binding

pytestmark = pytest.mark.gpu
LD = np.longdouble


def as_bits(t):
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def value(t):
    return t.detach().double().cpu().numpy().astype(LD)


def rotated(x, w, eps, positions, rope):
    """x [N, H, 128] rows at positions [N]: exact z and the pair sizes the bounds scale with."""
    f, m = rope.frequencies()
    r, f = rope.rotary_dim, f.astype(LD)
    y = x
    if w is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + LD(np.float32(eps))) * w
    i = np.arange(r // 2)
    first, second = (i, i + r // 2) if rope.layout == 0 else (2 * i, 2 * i + 1)
    a = positions.astype(LD)[:, None, None] * f
    c, s = np.cos(a) * LD(m), np.sin(a) * LD(m)
    z, size = y.copy(), np.abs(y)
    z[..., first] = y[..., first] * c - y[..., second] * s
    z[..., second] = y[..., second] * c + y[..., first] * s
    size[..., first] = size[..., second] = LD(m) * (np.abs(y[..., first]) + np.abs(y[..., second]))
    return z, size


def check(got, x, w, eps, positions, rope, window, what):
    z, size = rotated(value(x), None if w is None else value(w), eps, positions, rope)
    bound = size * (window + np.abs(positions.astype(np.float64))[:, None, None] * 2.0 ** -53)
    z64 = z.astype(np.float64)
    check_rounded_rows(as_bits(got), oracle.round_bf16(z64), z64, bound.astype(np.float64) + 1e-300, what)


def setup(B, Hq, Hkv, T, cap, paged, seed, positions_max=None, ragged=False, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    ri = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda").to(torch.int32)  # noqa: E731
    d = dict(B=B, Hq=Hq, Hkv=Hkv, T=T, cap=cap)
    if fused:
        qkv = rn(B, T, Hq + 2 * Hkv, 128)
        d["q"], d["k"], d["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    else:
        d["q"], d["k"], d["v"] = rn(B, T, Hq, 128), rn(B, T, Hkv, 128), rn(B, T, Hkv, 128)
    d["counts"] = ri(0, T, B) if ragged else None
    d["start"] = ri(0, cap - T, B)
    d["positions"] = None if positions_max is None else ri(0, positions_max, B, T)
    per = (cap + 63) // 64
    d["blocks"] = B * per + 2 if paged else 0
    d["table"] = torch.randperm(d["blocks"], generator=g, device="cuda")[:B * per].view(B, per).to(torch.int32) if paged else None
    rows = d["blocks"] * 64 if paged else B * cap
    d["kc"], d["vc"] = rn(rows, Hkv, 128), rn(rows, Hkv, 128)
    d["out"] = rn(B, T, Hq, 128)
    d["wq"], d["wk"] = (1 + 0.2 * rn(128).float()).to(torch.bfloat16), (1 + 0.2 * rn(128).float()).to(torch.bfloat16)
    d["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return d


def call(d, rope, norm=True, eps=1e-6, **over):
    a = dict(d)
    a.update(over)
    binding.rope_append(a["B"], a["Hq"], a["Hkv"], a["T"], a["cap"], a["q"], a["k"], a["v"], a["kc"], a["vc"], a["table"], a["start"],
                        a["positions"], a["counts"], a["wq"] if norm else None, a["wk"] if norm else None, rope, eps, a["out"],
                        block_size=64 if a["table"] is not None else 0, num_cache_blocks=a["blocks"], device_errors=a["err"])


def rows_of(d, b, slots):
    if d["table"] is None:
        return b * d["cap"] + slots
    return d["table"].cpu().numpy()[b][slots // 64].astype(np.int64) * 64 + slots % 64


def verify(d, rope, before, norm=True, eps=1e-6, skip=()):
    """Every output row and every cache row, new and old, of a call on `d`."""
    kc0, vc0, out0, q0 = before
    kw, vw, ow = as_bits(kc0).copy(), as_bits(vc0).copy(), as_bits(d["out"]).copy()
    kg = as_bits(d["kc"])
    start = d["start"].cpu().numpy()
    for b in range(d["B"]):
        n = d["T"] if d["counts"] is None else int(d["counts"][b])
        if b in skip or n == 0:
            np.testing.assert_array_equal(ow[b], as_bits(out0)[b])
            continue
        slots = start[b] + np.arange(n)
        pos = slots if d["positions"] is None else d["positions"][b, :n].cpu().numpy()
        rows = rows_of(d, b, slots)
        check(d["out"][b, :n], q0[b, :n], d["wq"] if norm else None, eps, pos, rope, Q_WINDOW, f"q of sequence {b}")
        check(d["kc"][torch.from_numpy(rows).cuda()], d["k"][b, :n], d["wk"] if norm else None, eps, pos, rope, K_WINDOW, f"k of sequence {b}")
        kw[rows] = kg[rows]
        vw[rows] = as_bits(d["v"][b, :n])
        np.testing.assert_array_equal(ow[b, n:], as_bits(out0)[b, n:])   # padded tokens: left as they were
    np.testing.assert_array_equal(kg, kw)       # no other row changed
    np.testing.assert_array_equal(as_bits(d["vc"]), vw)
    assert int(d["err"]) == 0


def snapshot(d):
    return d["kc"].clone(), d["vc"].clone(), d["out"].clone(), d["q"].clone()


LAYOUTS = [("half", 128), ("half", 64), ("half", 24), ("half", 8), ("half", 120), ("interleaved", 128), ("interleaved", 64),
           ("interleaved", 8), ("interleaved", 40)]


@pytest.mark.parametrize("layout,r", LAYOUTS)
@pytest.mark.parametrize("norm", [True, False])
def test_layouts(layout, r, norm):
    d = setup(3, 10, 2, 5, 150, paged=True, seed=r, positions_max=131071, ragged=True)
    before, rope = snapshot(d), binding.Rope(rotary_dim=r, layout=layout)
    call(d, rope, norm)
    verify(d, rope, before, norm)


@pytest.mark.parametrize("scaling", [dict(scaling="linear", factor=4.0),
                                     dict(theta=5e5, scaling="banded", factor=8.0, original_max_len=8192),
                                     dict(theta=5e5, scaling="yarn", factor=4.0, original_max_len=32768),
                                     dict(scaling="custom", freqs=np.geomspace(3.0, 1e-7, 64), magnitude=0.75)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scalings_at_far_positions(scaling, layout):
    d = setup(2, 8, 8, 7, 64, paged=False, seed=11, positions_max=(1 << 21))
    before, rope = snapshot(d), binding.Rope(layout=layout, **scaling)
    call(d, rope)
    verify(d, rope, before)


@pytest.mark.parametrize("B,Hq,Hkv,T,cap,paged", [(1, 1, 1, 1, 1, False), (1, 40, 8, 1, 256, True), (2, 16, 1, 3, 65, True),
                                                  (1, 64, 8, 200, 333, True), (33, 5, 5, 2, 64, False), (1, 32, 2, 64, 64, True),
                                                  (2, 320, 40, 3, 64, True), (1, 640, 80, 1, 2, False), (1, 1, 1, 500, 500, True)])
@pytest.mark.parametrize("fused", [False, True])
def test_sizes_and_strides(B, Hq, Hkv, T, cap, paged, fused):
    d = setup(B, Hq, Hkv, T, cap, paged, seed=B + T, ragged=T > 2, fused=fused)
    before, rope = snapshot(d), binding.Rope(theta=1e4)
    call(d, rope)
    verify(d, rope, before)


def test_positions_up_to_the_largest_int():
    d = setup(1, 4, 2, 4, 64, paged=False, seed=3)
    d["positions"] = torch.tensor([[0, 1, (1 << 24) + 1, (1 << 31) - 1]], dtype=torch.int32, device="cuda")
    before, rope = snapshot(d), binding.Rope()
    call(d, rope)
    verify(d, rope, before)


def test_in_place_queries():
    d = setup(2, 8, 2, 9, 64, paged=False, seed=5)
    d["out"] = d["q"]
    before, rope = snapshot(d), binding.Rope(layout="interleaved", rotary_dim=64)
    call(d, rope)
    verify(d, rope, before)


def test_large_and_zero_rows():
    """Values at the ends of bf16's range: zero rows, tiny rows (the norm's eps rules) and rows whose
    squares stay finite in binary32."""
    d = setup(1, 4, 4, 4, 64, paged=False, seed=6)
    for t, s in enumerate((0.0, 1e-20, 1e18, 3e-3)):
        for x in (d["q"], d["k"]):
            x[:, t] = (x[:, t].float() * s).to(torch.bfloat16)
    for norm in (True, False):
        before, rope = snapshot(d), binding.Rope()
        call(d, rope, norm)
        verify(d, rope, before, norm)


def test_nonfinite_values_stay_in_their_pairs():
    d = setup(1, 2, 2, 1, 64, paged=False, seed=7)
    d["k"][0, 0, 0, 3] = float("inf")
    d["k"][0, 0, 1, 100] = float("nan")
    call(d, binding.Rope(rotary_dim=64), norm=False)
    row = d["kc"][int(d["start"][0])]
    assert set(torch.nonzero(~torch.isfinite(row[0])).flatten().tolist()) <= {3, 35}
    assert not bool(torch.isfinite(row[0, [3, 35]]).any())
    assert torch.nonzero(~torch.isfinite(row[1])).flatten().tolist() == [100]


def test_keys_are_the_bits_the_prefill_chunk_appends():
    """Half-split, full width, unscaled: the cache rows are those of gqa_prefill_attn."""
    B, Hq, Hkv, T, cap = 2, 40, 8, 150, 400
    d = setup(B, Hq, Hkv, T, cap, paged=True, seed=8)
    rope = binding.Rope(theta=1e6)
    kc, vc, out = d["kc"].clone(), d["vc"].clone(), torch.empty_like(d["out"])
    call(d, rope)
    binding.prefill_attn(B, Hq, Hkv, T, cap, d["q"], d["k"], d["v"], kc, vc, d["table"], d["start"], d["wq"], d["wk"], 1e6, 1e-6, out,
                         block_size=64, num_cache_blocks=d["blocks"])
    torch.cuda.synchronize()
    differ = int((as_bits(kc) != as_bits(d["kc"])).sum())
    assert differ <= 1e-6 * kc.numel(), differ     # both round the exact value: 2^-40 of all values lie too near a midpoint
    np.testing.assert_array_equal(as_bits(vc), as_bits(d["vc"]))


def test_bad_pages_store_nothing():
    d = setup(2, 4, 2, 4, 130, paged=True, seed=13)
    d["start"] = torch.tensor([62, 62], dtype=torch.int32, device="cuda")
    d["table"][0, 1], d["table"][1, 0] = d["blocks"], -1
    before, rope = snapshot(d), binding.Rope()
    call(d, rope)
    assert int(d["err"]) == binding.DEVERR_PAGE
    changed = set(np.nonzero((as_bits(d["kc"]) != as_bits(before[0])).any((1, 2)))[0].tolist())
    assert changed == set(rows_of(d, 0, np.array([62, 63])).tolist()) | set(rows_of(d, 1, np.array([64, 65])).tolist())
    d["err"].zero_()
    for b in range(2):                           # the queries are rotated all the same
        check(d["out"][b], before[3][b], d["wq"], 1e-6, 62 + np.arange(4), rope, Q_WINDOW, "q")


def test_bad_lengths_and_positions_are_contained():
    B, T, cap = 6, 4, 130
    d = setup(B, 4, 2, T, cap, paged=True, seed=9)
    d["start"] = torch.tensor([0, -1, 127, 5, 60, 3], dtype=torch.int32, device="cuda")
    d["counts"] = torch.tensor([4, 2, 4, 5, 4, 4], dtype=torch.int32, device="cuda")
    d["positions"] = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
    d["positions"][5, 2] = -7
    d["table"][4, 1] = d["blocks"]               # slots 64.. of sequence 4, which the call does not touch
    before, rope = snapshot(d), binding.Rope()
    call(d, rope)
    err = int(d["err"])
    assert err == binding.DEVERR_POSITION | binding.DEVERR_SEQLEN
    out = as_bits(d["out"])
    for b in (1, 2, 3):
        assert not out[b].any()
    assert not out[5, 2].any() and out[5, [0, 1, 3]].any(-1).all()
    changed = set(np.nonzero((as_bits(d["kc"]) != as_bits(before[0])).any((1, 2)))[0].tolist())
    want = set(rows_of(d, 0, np.arange(4)).tolist()) | set(rows_of(d, 4, np.arange(60, 64)).tolist()) | set(
        rows_of(d, 5, np.array([3, 4, 6])).tolist())
    assert changed == want


def test_captured_and_replayed():
    d = setup(2, 8, 2, 3, 64, paged=False, seed=10)
    rope = binding.Rope()
    call(d, rope)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(d, rope)
    d["q"].copy_(torch.randn_like(d["q"]))
    d["k"].copy_(torch.randn_like(d["k"]))
    before = snapshot(d)
    g.replay()
    torch.cuda.synchronize()
    verify(d, rope, before)


def test_wrapper_refuses_wrong_tensors():
    d = setup(2, 8, 2, 3, 64, paged=False, seed=12)
    rope = binding.Rope()
    for name, bad in [("q", d["q"].float()), ("q", d["q"].cpu()), ("k", d["k"][:, :2]), ("v", d["v"].transpose(1, 2)),
                      ("start", d["start"].long()), ("kc", d["kc"][:-1]), ("out", d["out"][:1]), ("err", torch.zeros(2, dtype=torch.int32, device="cuda"))]:
        with pytest.raises((ValueError, binding.GqaError)):
            call(d, rope, **{name: bad})


def test_random_geometries():
    rng = np.random.default_rng(0)
    for seed, paged in itertools.product(range(6), (False, True)):
        Hkv = int(rng.choice([1, 2, 5, 8]))
        Hq, T = Hkv * int(rng.integers(1, 17)), int(rng.integers(1, 40))
        d = setup(int(rng.integers(1, 6)), Hq, Hkv, T, T + int(rng.integers(0, 300)), paged, seed, positions_max=int(rng.integers(0, 200000)),
                  ragged=bool(rng.integers(0, 2)), fused=bool(rng.integers(0, 2)))
        rope = binding.Rope(theta=float(rng.choice([1e4, 5e5])), rotary_dim=8 * int(rng.integers(1, 17)),
                            layout=["half", "interleaved"][int(rng.integers(0, 2))])
        before, norm = snapshot(d), bool(rng.integers(0, 2))
        call(d, rope, norm)
        verify(d, rope, before, norm)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("r", [8, 40, 96])
def test_dims_that_do_not_turn_keep_their_bits(layout, r):
    """Without a norm, z = y = x there: every finite bf16, zeros of either sign and infinities."""
    B, T = 2, 150
    d = setup(B, 6, 3, T, 256, True, seed=r)
    every = np.array([x for x in range(1 << 16) if x & 0x7fff <= 0x7f80], np.uint16)   # all but NaN
    rng = np.random.default_rng(r)
    for name in ("q", "k"):
        bits = as_bits(d[name]).copy()
        bits[..., r:] = rng.choice(every, bits[..., r:].shape)
        bits[..., -1] = 0x8000
        d[name] = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    call(d, binding.Rope(layout=layout, rotary_dim=r), norm=False)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(as_bits(d["out"])[..., r:], as_bits(d["q"])[..., r:])
    for b in range(B):
        s = int(d["start"][b])
        kept = as_bits(d["kc"])[rows_of(d, b, np.arange(s, s + T))]
        np.testing.assert_array_equal(kept[..., r:], as_bits(d["k"][b])[..., r:])


def round_to_bf16(z):
    """float64 values rounded once to bf16, ties to even, as float64."""
    b = z.view(torch.int64)
    return ((b + ((1 << 44) - 1) + ((b >> 45) & 1)) >> 45 << 45).view(torch.float64)


@pytest.mark.parametrize("size", [8e17, 1e16, 1.0])
def test_keys_of_many_rows_round_as_the_exact_value(size):
    """10^8 key elements of normalised rows up to the largest that the norm takes, at position 0, where
    z = r x w: a relative error of r of 2^-31 would change several of the roundings.  The 64-bit
    value's own error is 2^-50."""
    B, H, T = 8, 8, 4096
    for seed in range(4):
        d = setup(B, H, H, T, T, paged=False, seed=20 + seed)
        d["k"] = (d["k"].float() * size).to(torch.bfloat16)
        d["start"].zero_()
        d["positions"] = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        call(d, binding.Rope())
        x = d["k"].double()
        z = x / torch.sqrt(x.square().mean(-1, keepdim=True) + float(np.float32(1e-6))) * d["wk"].double()
        assert bool(torch.isfinite(x.float().square().sum(-1)).all())
        want, got = round_to_bf16(z), d["kc"].view(B, T, H, 128).double()
        off = (got != want) & ((z - 0.5 * (got + want)).abs() > K_WINDOW * z.abs())   # (want is a midpoint's neighbour)
        assert int(off.sum()) == 0, (int(off.sum()), float(z[off][0]), float(got[off][0]))
    assert int(d["err"]) == 0


@pytest.mark.parametrize("eps,size", [(0.0, 3e-15), (0.0, 1.0), (0.0, 5e17), (1e-30, 3e-20), (1e-30, 1e-30)])
def test_small_rows_with_little_or_no_eps(eps, size):
    """Rows down to the least mean(x^2) + eps that the header names."""
    d = setup(2, 8, 4, 9, 64, paged=True, seed=30)
    for x in (d["q"], d["k"]):
        x.copy_((x.float() * size).to(torch.bfloat16))
    before, rope = snapshot(d), binding.Rope()
    call(d, rope, eps=eps)
    verify(d, rope, before, eps=eps)


def test_rows_below_the_norms_range_reach_no_other_row():
    """eps = 0 with zero rows and rows whose squares vanish in binary32: no other row, query, key
    or value, and no other token is changed by them."""
    d = setup(2, 8, 4, 9, 64, paged=True, seed=31)
    rope = binding.Rope()
    kc0, vc0 = d["kc"].clone(), d["vc"].clone()
    call(d, rope, eps=0.0)
    kc, vc, out = d["kc"].clone(), d["vc"].clone(), d["out"].clone()
    small = [(0, 0, 0, 0.0), (0, 4, 3, 1e-23), (1, 8, 1, 1e-38), (1, 2, 2, 0.0)]
    for b, t, h, f in small:
        d["k"][b, t, h] = (d["k"][b, t, h].float() * f).to(torch.bfloat16)
        d["q"][b, t, 2 * h + 1] = (d["q"][b, t, 2 * h + 1].float() * f).to(torch.bfloat16)
    d["kc"].copy_(kc0)
    d["vc"].copy_(vc0)
    call(d, rope, eps=0.0)
    start = d["start"].cpu().numpy()
    for b, t, h, _ in small:
        row = int(rows_of(d, b, np.array([start[b] + t]))[0])
        kc[row, h] = d["kc"][row, h]
        out[b, t, 2 * h + 1] = d["out"][b, t, 2 * h + 1]
    np.testing.assert_array_equal(as_bits(d["kc"]), as_bits(kc))
    np.testing.assert_array_equal(as_bits(d["vc"]), as_bits(vc))
    np.testing.assert_array_equal(as_bits(d["out"]), as_bits(out))
    assert int(d["err"]) == 0
