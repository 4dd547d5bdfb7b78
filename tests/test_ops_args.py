"""CPU checks of the draft-step operators (rotary append, draft trees, cache pages): the rotary
frequencies against their definitions, and the refusals of the C entry points, made before
any device work (the dummy pointers are never followed)."""
import ctypes
import math

import numpy as np
import pytest

from gqa_decode_attention_fa_gb300 import binding

INV, UNS = binding.GQA_ERR_INVALID_ARG, binding.GQA_ERR_UNSUPPORTED
DUMMY = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 2)


# ------------------------------------------------------------------------------- frequencies

def base(theta, r):
    return [np.float32(theta).astype(np.float64) ** (-2.0 * i / r) for i in range(r // 2)]


def test_unscaled_and_linear_frequencies():
    for r in (8, 24, 64, 128):
        f, m = binding.Rope(theta=1e6, rotary_dim=r).frequencies()
        np.testing.assert_allclose(f, base(1e6, r), rtol=1e-14)
        assert m == 1.0 and f[0] == 1.0
        g, m = binding.Rope(theta=1e6, rotary_dim=r, scaling="linear", factor=4.0).frequencies()
        np.testing.assert_allclose(g, f / 4.0, rtol=1e-15)
        assert m == 1.0


def test_banded_frequencies_keep_short_divide_long_and_mix_between():
    n, lo, hi, factor = 8192, 1.0, 4.0, 8.0
    f, m = binding.Rope(theta=5e5, scaling="banded", factor=factor, low_freq_factor=lo, high_freq_factor=hi,
                        original_max_len=n).frequencies()
    assert m == 1.0
    kinds = set()
    for got, w in zip(f, base(5e5, 128)):
        wavelength = 2 * math.pi / w
        if wavelength < n / hi:
            kinds.add("short")
            assert got == pytest.approx(w, rel=1e-14)
        elif wavelength > n / lo:
            kinds.add("long")
            assert got == pytest.approx(w / factor, rel=1e-14)
        else:
            kinds.add("between")
            mix = (n / wavelength - lo) / (hi - lo)
            assert got == pytest.approx((1 - mix) * w / factor + mix * w, rel=1e-12)
    assert kinds == {"short", "between", "long"}


def test_yarn_frequencies_ramp_and_magnitude():
    r, n, factor, theta = 64, 32768, 4.0, 1e4
    f, m = binding.Rope(theta=theta, rotary_dim=r, scaling="yarn", factor=factor, original_max_len=n).frequencies()
    assert m == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-15)
    d = lambda b: r * math.log(n / (2 * math.pi * b)) / (2 * math.log(theta))  # noqa: E731
    low, high = max(math.floor(d(32.0)), 0), min(math.ceil(d(1.0)), r - 1)
    for i, (got, w) in enumerate(zip(f, base(theta, r))):
        ramp = min(1.0, max(0.0, (i - low) / (high - low)))
        assert got == pytest.approx(w / factor * ramp + w * (1 - ramp), rel=1e-12)
    assert f[0] == 1.0 and f[-1] == pytest.approx(base(theta, r)[-1] / factor, rel=1e-12)
    assert binding.Rope(theta=theta, scaling="yarn", factor=factor, original_max_len=n, magnitude=1.5).frequencies()[1] == 1.5


def test_custom_frequencies_are_the_callers():
    table = np.linspace(2.0, -0.5, 16)
    f, m = binding.Rope(rotary_dim=32, scaling="custom", freqs=table).frequencies()
    np.testing.assert_array_equal(f, table)
    assert m == 1.0


@pytest.mark.parametrize("over", [
    dict(rotary_dim=0), dict(rotary_dim=12), dict(rotary_dim=136), dict(theta=0.0), dict(theta=float("nan")),
    dict(magnitude=-1.0), dict(magnitude=float("inf")), dict(scaling="linear", factor=0.0),
    dict(scaling="banded", factor=2.0, original_max_len=0), dict(scaling="banded", factor=2.0, original_max_len=64, low_freq_factor=4.0),
    dict(scaling="yarn", factor=0.5, original_max_len=64), dict(scaling="yarn", factor=2.0, original_max_len=64, beta_fast=1.0),
    dict(scaling="yarn", factor=2.0, original_max_len=64, theta=1.0), dict(scaling="custom"),
    dict(scaling="custom", freqs=[float("inf")] * 64), dict(scaling="custom", freqs=[65537.0] * 64),
    dict(scaling="linear", factor=1e-6),
])
def test_bad_rotary_embeddings_are_refused(over):
    with pytest.raises(binding.GqaError) as e:
        binding.Rope(**over).frequencies()
    assert e.value.status == INV


def test_unknown_rotary_names_are_refused():
    for over in (dict(layout="split"), dict(scaling="ntk"), dict(scaling="custom", freqs=[1.0])):
        with pytest.raises(ValueError):
            binding.Rope(**over)
    assert binding.load().gqa_rope_freqs(None, None, None) == INV
    for field in ("layout", "scaling"):
        r = binding.Rope()
        setattr(r, field, 9)
        assert binding.load().gqa_rope_freqs(ctypes.byref(r), None, None) == INV


# ------------------------------------------------------------------------------ rotary append

def _rope(rope=None, eps=1e-6, args=None, **over):
    d = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, num_tokens=4, block_size=0, max_seq_len=64,
             num_cache_blocks=0, device=0, q_stride=0, k_stride=0, v_stride=0)
    d.update(over)
    desc = binding.RopeDesc(*[d[n] for n, _ in binding.RopeDesc._fields_])
    a = dict(q=DUMMY, k=DUMMY, v=DUMMY, kc=DUMMY, vc=DUMMY, pt=DUMMY if d["block_size"] else None, start=DUMMY, pos=None,
             counts=None, qw=None, kw=None, out=DUMMY, err=None)
    a.update(args or {})
    return binding.load().gqa_rope_append(
        ctypes.byref(desc), a["q"], a["k"], a["v"], a["kc"], a["vc"], a["pt"], a["start"], a["pos"], a["counts"], a["qw"],
        a["kw"], ctypes.byref(rope or binding.Rope()), ctypes.c_float(eps), a["out"], a["err"], None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), INV), (dict(batch=1025), INV), (dict(num_tokens=0), INV), (dict(num_tokens=65), INV),
    (dict(max_seq_len=0), INV), (dict(num_q_heads=0), INV), (dict(head_dim=64), UNS),
    (dict(num_q_heads=9), UNS), (dict(num_q_heads=34), UNS), (dict(block_size=32, num_cache_blocks=4), UNS),
    (dict(block_size=64, num_cache_blocks=0), INV), (dict(q_stride=1020), INV), (dict(q_stride=1028), INV),
    (dict(num_q_heads=801, num_kv_heads=801), UNS), (dict(num_q_heads=1280, num_kv_heads=80), UNS), (dict(k_stride=128), INV), (dict(v_stride=-256), INV), (dict(batch=1024, max_seq_len=1 << 22), UNS),
])
def test_rope_append_refuses_bad_geometry(over, status):
    assert _rope(**over) == status


def test_rope_append_refuses_bad_arguments():
    for name in ("q", "k", "v", "kc", "vc", "start", "out"):
        assert _rope(args={name: None}) == INV
    for name in ("q", "k", "v", "kc", "vc", "out", "qw", "kw", "start", "pos", "counts", "err"):
        assert _rope(args={name: ODD}) == INV
    assert _rope(args=dict(pt=DUMMY)) == INV                           # a table for a contiguous cache
    assert _rope(block_size=64, num_cache_blocks=4, args=dict(pt=None)) == INV
    assert _rope(eps=-1.0) == INV and _rope(eps=float("nan")) == INV
    assert _rope(q_stride=2048) == INV                                 # in place needs dense queries
    assert _rope(rope=binding.Rope(rotary_dim=20)) == INV
    assert binding.load().gqa_rope_append(*([None] * 13), ctypes.c_float(1e-6), None, None, None) == INV


# -------------------------------------------------------------------------------- draft trees

def _tree(args=None, **over):
    d = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, tree_len=4, block_size=0, max_seq_len=512,
             num_cache_blocks=0, device=0)
    d.update(over)
    desc = binding.TreeDesc(*[d[n] for n, _ in binding.TreeDesc._fields_])
    n = ctypes.c_size_t()
    sized = binding.load().gqa_tree_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    a = dict(q=DUMMY, kc=DUMMY, vc=DUMMY, pt=DUMMY if d["block_size"] else None, ctx=DUMMY, counts=None, mask=DUMMY,
             out=DUMMY, ws=DUMMY, err=None)
    a.update(args or {})
    ran = binding.load().gqa_tree_attn(ctypes.byref(desc), a["q"], a["kc"], a["vc"], a["pt"], a["ctx"], a["counts"], a["mask"],
                                       a["out"], a["ws"], a["err"], None)
    return sized, ran


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), INV), (dict(batch=1025), INV), (dict(tree_len=0), INV), (dict(tree_len=257), INV),
    (dict(tree_len=9, max_seq_len=8), INV), (dict(head_dim=64), UNS), (dict(num_q_heads=9), UNS),
    (dict(num_q_heads=34), UNS), (dict(block_size=16, num_cache_blocks=4), UNS),
    (dict(block_size=64, num_cache_blocks=0), INV), (dict(block_size=64, num_cache_blocks=1 << 26), UNS),
])
def test_tree_attn_refuses_bad_geometry(over, status):
    assert _tree(**over) == (status, status)


def test_tree_attn_refuses_bad_arguments():
    for name in ("q", "kc", "vc", "ctx", "mask", "out", "ws"):
        assert _tree(args={name: None})[1] == INV
    for name in ("q", "kc", "vc", "ctx", "counts", "mask", "out", "ws", "err"):
        assert _tree(args={name: ODD})[1] == INV
    assert _tree(args=dict(mask=ctypes.c_void_p(4100)))[1] == INV
    assert _tree(args=dict(ws=ctypes.c_void_p(4096 + 128)))[1] == INV
    assert _tree(args=dict(pt=DUMMY))[1] == INV
    assert _tree(block_size=64, num_cache_blocks=4, args=dict(pt=None))[1] == INV
    lib = binding.load()
    assert lib.gqa_tree_attn(*([None] * 12)) == INV and lib.gqa_tree_workspace_bytes(None, None) == INV


def test_tree_prepare_refuses_bad_arguments():
    f = binding.load().gqa_tree_prepare
    ok = [2, 4, DUMMY, DUMMY, None, DUMMY, DUMMY, 0, None, None]
    for at, bad in [(0, 0), (0, 1025), (1, 0), (1, 257), (2, None), (3, None), (5, None), (6, None), (2, ODD), (3, ODD), (4, ODD),
                    (5, ctypes.c_void_p(4100)), (6, ODD), (8, ODD)]:
        assert f(*[bad if i == at else x for i, x in enumerate(ok)]) == INV, (at, bad)


# -------------------------------------------------------------------------------- cache pages

def test_page_state_refusals():
    lib = binding.load()
    good = (2, 4, 16, 0)
    for bad in [(0, 4, 16, 0), (1025, 4, 16, 0), (2, 0, 16, 0), (2, 4, 0, 0), (2, 4, 1 << 25, 0), (1024, 1 << 21, 16, 0)]:
        d = binding.PagesDesc(*bad)
        assert lib.gqa_pages_fork(ctypes.byref(d), DUMMY, DUMMY, DUMMY, DUMMY, DUMMY, 1, None, None) == INV
        assert lib.gqa_pages_resize(ctypes.byref(d), DUMMY, DUMMY, DUMMY, DUMMY, DUMMY, DUMMY, None, None) == INV
    d = binding.PagesDesc(*good)
    for bad in (None, ODD):
        for at in range(6):
            a = [bad if i == at else DUMMY for i in range(6)]
            assert lib.gqa_pages_resize(ctypes.byref(d), *a, None, None) == INV
            if at < 5:
                assert lib.gqa_pages_fork(ctypes.byref(d), *a[:5], 1, None, None) == INV
    assert lib.gqa_pages_resize(ctypes.byref(d), *[DUMMY] * 6, ODD, None) == INV
    for n in (0, -1, 1025):
        assert lib.gqa_pages_fork(ctypes.byref(d), *[DUMMY] * 5, n, None, None) == INV
    assert lib.gqa_pages_fork(None, *[DUMMY] * 5, 1, None, None) == INV


def _pools(*rows, base=4096):
    return (binding.Pool * len(rows))(*[binding.Pool(base, r) for r in rows])


def test_copy_and_keep_refusals():
    lib = binding.load()
    good = _pools(2048, 32)

    def copy(pools=good, n=2, blocks=8, src=DUMMY, dst=DUMMY, pairs=1, err=None):
        return lib.gqa_pages_copy(pools, n, blocks, src, dst, pairs, 0, err, None)

    def keep(pools=good, n=2, pt=DUMMY, start=DUMMY, lst=DUMMY, counts=DUMMY, err=None, **over):
        d = dict(batch=2, max_keep=4, max_seq_len=128, block_size=64, num_blocks=8, device=0)
        d.update(over)
        desc = binding.KeepDesc(*[d[k] for k, _ in binding.KeepDesc._fields_])
        return lib.gqa_cache_keep_rows(ctypes.byref(desc), pools, n, pt, start, lst, counts, err, None)

    for f in (copy, keep):
        assert f(pools=None) == INV and f(n=0) == INV and f(n=257) == INV and f(err=ODD) == INV
        for rows in ((8,), (24,), (0,), (-16,), ((1 << 20) + 16,)):
            assert f(pools=_pools(*rows), n=1) == INV
        assert f(pools=_pools(2048, base=4100), n=1) == INV and f(pools=_pools(2048, base=0), n=1) == INV
    for over in (dict(blocks=0), dict(blocks=1 << 25), dict(pairs=0), dict(pairs=4097), dict(src=None), dict(dst=ODD)):
        assert copy(**over) == INV
    for over in (dict(batch=0), dict(batch=1025), dict(max_keep=0), dict(max_keep=129), dict(max_seq_len=0), dict(num_blocks=0),
                 dict(pt=None), dict(block_size=0), dict(start=None), dict(lst=ODD), dict(counts=None)):
        assert keep(**over) == INV, over
    assert keep(block_size=32) == UNS and keep(num_blocks=1 << 26) == UNS
    assert lib.gqa_cache_keep_rows(None, good, 2, *[DUMMY] * 4, None, None) == INV


def test_fields_beyond_32_bits_are_refused():
    for field in (1 << 31, (1 << 32) + 64, -(1 << 31) - 1):
        with pytest.raises(ValueError):
            binding._desc(binding.PagesDesc, 2, field, 16, 0)
        with pytest.raises(ValueError):
            binding.tree_workspace_bytes(2, 8, 2, 4, field)
    binding._desc(binding.PagesDesc, 2, (1 << 31) - 1, 16, 0)


def test_tree_geometry_at_the_largest_capacity():
    """2^31 - 1 tokens a sequence over a small pool: the limit on B (ceil(max_seq_len/64) + 7) is reached at 64."""
    big = dict(block_size=64, num_cache_blocks=1, max_seq_len=2 ** 31 - 1)
    for batch, refused in [(64, True), (63, False)]:
        for status in _tree(batch=batch, args=dict(ws=ODD), **big)[:1 if not refused else 2]:
            assert (status == UNS) == refused, (batch, status)


def test_keep_lists_longer_than_any_index_are_refused():
    """Lists past 2^30 entries: the kernel counts in steps of thousands below 2^31."""
    desc = lambda n: ctypes.byref(binding.KeepDesc(1, n, 2 ** 31 - 1, 0, 0, 0))  # noqa: E731
    call = lambda n: binding.load().gqa_cache_keep_rows(desc(n), _pools(16), 1, None, DUMMY, DUMMY, ODD, None, None)  # noqa: E731
    assert call((1 << 30) + 1) == UNS and call(2 ** 31 - 1) == UNS
    assert call(1 << 30) == INV                                        # goes on to the misaligned counts
