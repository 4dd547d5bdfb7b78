"""CPU checks of the 8-bit cache and packed-prompt calls: the refusals of the C entry points, made
before any device work (the dummy pointers are never followed), and of the Python ones."""
import ctypes

import pytest
import torch

from gqa_decode_attention_fa_gb300 import binding

INV, UNS = binding.GQA_ERR_INVALID_ARG, binding.GQA_ERR_UNSUPPORTED
DUMMY = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 2)


def _desc(over):
    d = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, format=0, num_tokens=4, block_size=0, max_seq_len=64,
             num_cache_blocks=0, device=0, k_stride=0, v_stride=0)
    d.update(over)
    return d, ctypes.byref(binding.Q8Desc(*[d[n] for n, _ in binding.Q8Desc._fields_]))


def _rows(call, args=None, **over):
    d, desc = _desc(over)
    a = dict(k=DUMMY, v=DUMMY, kc=DUMMY, vc=DUMMY, ks=DUMMY, vs=DUMMY, pt=DUMMY if d["block_size"] else None, off=DUMMY, start=DUMMY,
             err=None)
    a.update(args or {})
    packed, cache = [a["k"], a["v"]], [a["kc"], a["vc"], a["ks"], a["vs"]]
    where = [a["pt"], a["off"], a["start"]]
    every = packed + cache + where if call == "append" else cache + where + packed
    return getattr(binding.load(), "gqa_q8_" + call)(desc, *every, a["err"], None)


def _attn(args=None, **over):
    d, desc = _desc(over)
    n = ctypes.c_size_t()
    sized = binding.load().gqa_q8_workspace_bytes(desc, ctypes.byref(n))
    a = dict(q=DUMMY, kc=DUMMY, vc=DUMMY, ks=DUMMY, vs=DUMMY, pt=DUMMY if d["block_size"] else None, lens=DUMMY, out=DUMMY, ws=DUMMY,
             err=None)
    a.update(args or {})
    return sized, binding.load().gqa_q8_attn(desc, *a.values(), None)


GEOMETRY = [
    (dict(batch=0), INV), (dict(batch=1025), INV), (dict(num_kv_heads=0), INV), (dict(max_seq_len=0), INV), (dict(head_dim=64), UNS),
    (dict(format=2), INV), (dict(format=-1), INV), (dict(block_size=32, num_cache_blocks=4), UNS),
    (dict(block_size=64, num_cache_blocks=0), INV), (dict(block_size=64, num_cache_blocks=1 << 26), UNS),
    (dict(batch=1024, max_seq_len=1 << 22), UNS),
]


@pytest.mark.parametrize("call", ["append", "read"])
@pytest.mark.parametrize("over,status", GEOMETRY + [
    (dict(num_tokens=0), INV), (dict(num_tokens=-1), INV), (dict(k_stride=128), INV), (dict(v_stride=260), INV), (dict(v_stride=-256), INV),
    (dict(num_tokens=1 << 30), UNS),
])
def test_rows_refuse_bad_geometry(call, over, status):
    assert _rows(call, **over) == status


@pytest.mark.parametrize("call", ["append", "read"])
def test_rows_refuse_bad_arguments(call):
    for name in ("k", "v", "kc", "vc", "ks", "vs") + (("start",) if call == "append" else ()):
        assert _rows(call, args={name: None}) == INV
    for name in ("k", "v", "kc", "vc", "ks", "vs", "off", "start", "err"):
        assert _rows(call, args={name: ODD}) == INV
    assert _rows(call, args=dict(kc=ctypes.c_void_p(4096 + 8))) == INV
    assert _rows(call, args=dict(off=None)) == INV                          # 4 tokens of 2 sequences
    assert _rows(call, args=dict(pt=DUMMY)) == INV                          # a table for a contiguous cache
    assert _rows(call, block_size=64, num_cache_blocks=4, args=dict(pt=None)) == INV
    assert getattr(binding.load(), "gqa_q8_" + call)(*([None] * 12)) == INV


@pytest.mark.parametrize("over,status", GEOMETRY + [
    (dict(num_q_heads=0), INV), (dict(num_q_heads=9), UNS), (dict(num_q_heads=34), UNS),
    (dict(batch=64, block_size=64, num_cache_blocks=1, max_seq_len=2 ** 31 - 1), UNS),
    (dict(num_q_heads=1 << 22, num_kv_heads=1 << 22, max_seq_len=1), UNS),
])
def test_attn_refuses_bad_geometry(over, status):
    assert _attn(**over) == (status, status)


@pytest.mark.parametrize("num_kv_heads", [1, 2, 64])
@pytest.mark.parametrize("batch", [300, 1023, 1024])
def test_attn_counts_the_numbers_of_a_batch(batch, num_kv_heads):
    """The batch's units of 16 tokens, with 24 numbers behind each sequence (the end of a piece that eight warps share, 3 units of each
    warp), are fewer than 2^31: the last capacity that keeps to it, and the next."""
    units = (2 ** 31 - 1) // batch - 24
    geometry = dict(batch=batch, num_q_heads=num_kv_heads, num_kv_heads=num_kv_heads, block_size=64, num_cache_blocks=1)
    n = ctypes.c_size_t()
    sized = lambda cap: binding.load().gqa_q8_workspace_bytes(_desc(dict(geometry, max_seq_len=cap))[1], ctypes.byref(n))  # noqa: E731
    assert sized(16 * units) != UNS  # (not called: on a device it would run)
    assert sized(16 * units + 1) == UNS
    assert _attn(max_seq_len=16 * units + 1, **geometry) == (UNS, UNS)


def test_attn_refuses_bad_arguments():
    for name in ("q", "kc", "vc", "ks", "vs", "lens", "out", "ws"):
        assert _attn(args={name: None})[1] == INV
    for name in ("q", "kc", "vc", "ks", "vs", "lens", "out", "ws", "err"):
        assert _attn(args={name: ODD})[1] == INV
    assert _attn(args=dict(ws=ctypes.c_void_p(4096 + 128)))[1] == INV
    assert _attn(args=dict(pt=DUMMY))[1] == INV
    assert _attn(block_size=64, num_cache_blocks=4, args=dict(pt=None))[1] == INV
    lib = binding.load()
    assert lib.gqa_q8_attn(*([None] * 12)) == INV and lib.gqa_q8_workspace_bytes(None, None) == INV


# ------------------------------------------------------------------------------- packed prompts

def _packed(args=None, **over):
    d = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, num_queries=10, num_keys=12, causal=1, device=0, q_stride=0,
             k_stride=0, v_stride=0)
    d.update(over)
    desc = ctypes.byref(binding.PackedDesc(*[d[n] for n, _ in binding.PackedDesc._fields_]))
    a = dict(q=DUMMY, k=DUMMY, v=DUMMY, qo=DUMMY, ko=None, out=DUMMY, err=None)
    a.update(args or {})
    return binding.load().gqa_packed_attn(desc, *a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), INV), (dict(batch=1025), INV), (dict(num_q_heads=0), INV), (dict(num_kv_heads=0), INV), (dict(head_dim=64), UNS),
    (dict(num_q_heads=9), UNS), (dict(num_q_heads=34), UNS), (dict(num_queries=0), INV), (dict(num_keys=0), INV), (dict(num_keys=-1), INV),
    (dict(q_stride=1020), INV), (dict(q_stride=1016), INV), (dict(k_stride=128), INV), (dict(v_stride=-256), INV), (dict(v_stride=260), INV),
    (dict(num_queries=1 << 29), UNS), (dict(num_keys=1 << 30), UNS), (dict(num_q_heads=1, num_kv_heads=1, num_keys=(1 << 26) + 1), UNS),
])
def test_packed_attn_refuses_bad_geometry(over, status):
    assert _packed(**over) == status


def test_packed_attn_refuses_bad_arguments():
    for name in ("q", "k", "v", "qo", "out"):
        assert _packed(args={name: None}) == INV
    for name in ("q", "k", "v", "qo", "ko", "out", "err"):
        assert _packed(args={name: ODD}) == INV
    assert binding.load().gqa_packed_attn(*([None] * 9)) == INV


# ------------------------------------------------------------------------------- the Python entry points

def test_python_entry_points_refuse_host_tensors_and_other_types():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i32 = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    cache = (z(64, 2, 128, dtype=torch.int8), z(64, 2, 128, dtype=torch.int8), z(64, 2, dtype=torch.float32), z(64, 2, dtype=torch.float32))
    with pytest.raises(ValueError, match="cuda:0"):
        binding.q8_append(1, 2, 3, 64, z(3, 2, 128), z(3, 2, 128), *cache, None, i32(2), i32(1), fmt="int8")
    with pytest.raises(ValueError, match="cuda:0"):
        binding.q8_read(1, 2, 3, 64, *cache, None, i32(2), i32(1), z(3, 2, 128), z(3, 2, 128), fmt="int8")
    with pytest.raises(ValueError, match="cuda:0"):
        binding.packed_attn(z(5, 4, 128), z(5, 2, 128), z(5, 2, 128), i32(3), None, z(5, 4, 128))
    with pytest.raises(ValueError, match="fmt"):
        binding._q8_cache(*cache, "e5m2", 64, 2, -1)
    with pytest.raises(ValueError, match="k_codes"):
        binding._q8_cache(*cache, "e4m3", 64, 2, -1)                        # int8 codes as e4m3
    with pytest.raises(ValueError, match="rows"):
        binding._q8_cache(*cache, "int8", 65, 2, -1)
    with pytest.raises(ValueError, match="strides"):
        binding._packed(z(4, 2, 256)[:, :, ::2], "k", 4, 2, -1)
    with pytest.raises(ValueError, match="strides"):
        binding._packed(z(2, 4, 128).transpose(0, 1), "k", 4, 2, -1)        # heads outside tokens
    p, stride = binding._packed(z(4, 6, 128)[:, 2:4], "k", 4, 2, -1)
    assert stride == 6 * 128
    assert binding._packed(z(1, 6, 128)[:, 2:4], "k", 1, 2, -1)[1] == 2 * 128
    with pytest.raises(ValueError):
        binding.q8_workspace_bytes(2, 8, 2, 1 << 31)
