"""Serving over an 8-bit cache end to end: prompts packed one behind the other are rotated, attended to
and quantised into pages; a second chunk goes on over the prefixes read back; then tokens, one a
sequence, over the cache, captured in a graph -- each step against the formula in 64 bits on the rows that the
step before has left."""
import threading

import numpy as np
import pytest
import torch

from gqa_decode_attention_fa_gb300 import binding
from test_gpu_packed import attend as attend_packed, near as near_packed, offsets
from test_gpu_q8 import Cache, attend as attend_token, i32, near as near_token, quantised, rows_of

pytestmark = pytest.mark.gpu
Hq, Hkv, D, EPS = 40, 8, 128, 1e-6
ROPE = binding.Rope(theta=1e6)


class Server:
    """Two layers' 8-bit pools over one page table, empty pages; what never was written reads as NaN."""

    def __init__(self, B, cap, blocks, fmt):
        self.B, self.cap, self.blocks, self.fmt = B, cap, blocks, fmt
        i32z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.refs, self.lens, self.err, self.zero = i32z(blocks), i32z(B), i32z(1), i32z(1)
        self.table, self.cow = i32z(B, (cap + 63) // 64) - 1, i32z(2, B) - 1
        self.layers = []
        for _ in range(2):
            c = Cache(B, Hkv, cap, fmt, True)
            c.blocks, c.rows, c.table = blocks, blocks * 64, self.table
            kind = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
            c.k, c.v = (torch.full((c.rows, Hkv, D), 0x7f, dtype=torch.uint8, device="cuda").view(kind) for _ in range(2))
            c.ks, c.vs = (torch.full((c.rows, Hkv), float("nan"), device="cuda") for _ in range(2))
            self.layers.append(c)
        self.pools = binding.CachePools([t for c in self.layers for t in c.tensors], num_blocks=blocks)
        self.wq, self.wk = ((1 + 0.1 * rows_of(s, 1, 1).view(D).float()).to(torch.bfloat16) for s in (1, 2))

    def grow(self, new):
        binding.pages_resize(self.refs, self.table, self.lens, new, self.cow[0], self.cow[1], device_errors=self.err)
        binding.pages_copy(self.pools, self.cow[0], self.cow[1], device_errors=self.err)

    def rotated(self, x, positions):
        """Rotated queries, and keys and values as packed rows: the rows as one sequence of a contiguous cache."""
        n = x.shape[0]
        q, k, v = x[None].split([Hq, Hkv, Hkv], 2)
        q_rot = torch.empty(1, n, Hq, D, dtype=torch.bfloat16, device="cuda")
        kr, vr = (torch.empty(n, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        binding.rope_append(1, Hq, Hkv, n, n, q, k, v, kr, vr, None, self.zero, positions[None], None, self.wq, self.wk, ROPE, EPS,
                            q_rot, device_errors=self.err)
        return q_rot[0], kr, vr

    def append(self, layer, n, k, v, at, start):
        c = self.layers[layer]
        binding.q8_append(self.B, Hkv, n, self.cap, k, v, *c.tensors, self.table, at, start, device_errors=self.err, **c.layout)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_prompts_chunks_and_tokens(fmt):
    B, cap = 4, 640
    s = Server(B, cap, 44, fmt)
    first, second = [130, 1, 300, 64], [50, 129, 0, 7]
    held = np.zeros(B, np.int64)
    for lengths in (first, second):
        n, before = int(sum(lengths)), held.copy()
        held += lengths
        qa, ka = offsets(lengths), offsets(held)
        positions = i32(np.concatenate([np.arange(a, b) for a, b in zip(before, held)]))
        s.grow(i32(held))
        for layer in range(2):
            q, k, v = s.rotated(rows_of(10 * layer + n, n, Hq + 2 * Hkv), positions)
            s.append(layer, n, k, v, i32(qa), i32(before))
            c = s.layers[layer]
            for b in range(B):  # the rows as the format keeps them
                ref, scale = quantised(k[qa[b]:qa[b + 1]].double().cpu().numpy(), fmt)
                rows = c.slots(b, int(before[b]), lengths[b])
                got = c.k[torch.as_tensor(rows, device="cuda")] if fmt == "int8" else c.k.view(torch.uint8)[torch.as_tensor(rows, device="cuda")].view(c.k.dtype)
                assert (got.double().cpu().numpy() == ref).all() and (c.ks[torch.as_tensor(rows, device="cuda")].cpu().numpy() == scale).all()
            if before.any():  # a chunk attends to its sequence's rows as the cache holds them
                m = int(held.sum())
                k, v = (torch.empty(m, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                binding.q8_read(B, Hkv, m, cap, *c.tensors, s.table, i32(ka), None, k, v, device_errors=s.err, **c.layout)
            out = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
            binding.packed_attn(q, k, v, i32(qa), i32(ka), out, device_errors=s.err)
            near_packed(out, *attend_packed(dict(q=q, k=k, v=v, qa=qa, ka=ka, out=out, given=True)))
    # sequence 2 goes to sequence 1's place too: the pages are shared, then split as both grow
    binding.pages_resize(s.refs, s.table, s.lens, i32([held[0], 0, held[2], held[3]]), s.cow[0], s.cow[1], device_errors=s.err)
    binding.pages_fork(s.refs, s.table, s.lens, i32([2]), i32([1]), device_errors=s.err)
    assert s.lens.tolist() == [held[0], held[2], held[2], held[3]]
    # tokens: the whole step of both layers is captured once and replayed
    x = [torch.empty(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = [torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q_rot = [None, None]
    ws = binding.q8_workspace(B, Hq, Hkv, cap, block_size=64, num_cache_blocks=s.blocks)
    new = s.lens.clone()

    def step():
        positions = s.lens.clone()
        new.copy_(s.lens + 1)
        s.grow(new)
        for layer in range(2):
            c = s.layers[layer]
            q_rot[layer], k, v = s.rotated(x[layer], positions)
            s.append(layer, B, k, v, None, positions)
            binding.q8_attn(B, Hq, Hkv, cap, q_rot[layer], *c.tensors, s.table, s.lens, out[layer], workspace=ws, device_errors=s.err,
                            **c.layout)

    graph = None
    for i in range(4):
        for layer in range(2):
            x[layer].copy_(rows_of(100 + 2 * i + layer, B, Hq + 2 * Hkv))
        if i == 1:
            state = [t.clone() for t in (s.refs, s.table, s.lens)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for t, old in zip((s.refs, s.table, s.lens), state):
                assert torch.equal(t, old)  # nothing ran yet
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        lens = s.lens.tolist()
        for layer in range(2):
            c = s.layers[layer]
            c.table = s.table
            K, V = c.dense()
            K[np.isnan(K)], V[np.isnan(V)] = 0, 0  # rows that nobody holds
            c.dense = lambda k=K, v=V: (k, v)
            near_token(out[layer], *attend_token(c, q_rot[layer], lens, Hq))
            del c.dense
    assert s.err.item() == 0
    # the last three tokens of every sequence are given up again: rows moved, pages kept consistent
    keep = i32([[2]] * B)
    before = [t.clone() for t in s.layers[0].tensors]
    binding.cache_keep_rows(s.pools, s.table, s.lens - 3, keep, i32([1] * B), max_seq_len=cap, device_errors=s.err)
    for b, n in enumerate(s.lens.tolist()):
        to, frm = s.layers[0].slots(b, n - 3, 1), s.layers[0].slots(b, n - 1, 1)
        for now, old in zip(s.layers[0].tensors, before):
            assert torch.equal(now.view(torch.uint8)[torch.as_tensor(to, device="cuda")], old.view(torch.uint8)[torch.as_tensor(frm, device="cuda")])
    assert s.err.item() == 0


def test_calls_on_streams_of_their_own_and_several_threads():
    """The calls of several threads, each with its own stream, cache and workspace, give what they give alone."""
    def work(seed, stream):
        c = Cache(3, 4, 700, "e4m3", True, seed=seed)
        k, v, q = rows_of(seed, 30, 4), rows_of(seed + 1, 30, 4), rows_of(seed + 2, 30, 8)
        at, start, lens = i32([0, 10, 11, 30]), i32([500, 0, 640]), i32([510, 1, 659])
        ws = binding.q8_workspace(3, 8, 4, 700, block_size=64, num_cache_blocks=c.blocks)
        outs = [torch.zeros(3, 8, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(30, 8, D, dtype=torch.bfloat16, device="cuda")]
        ko, vo = torch.zeros_like(k), torch.zeros_like(v)
        torch.cuda.synchronize()
        for _ in range(20):
            binding.q8_append(3, 4, 30, 700, k, v, *c.tensors, c.table, at, start, stream=stream, **c.layout)
            binding.q8_read(3, 4, 30, 700, *c.tensors, c.table, at, start, ko, vo, stream=stream, **c.layout)
            binding.packed_attn(q, ko, vo, at, None, outs[1], stream=stream)
            binding.q8_attn(3, 8, 4, 700, q[:3].contiguous() if stream is None else work.q[seed], *c.tensors, c.table, lens, outs[0], workspace=ws,
                            stream=stream, **c.layout)
        torch.cuda.synchronize()
        return outs + [ko, vo]

    work.q = {seed: rows_of(seed + 2, 30, 8)[:3].contiguous() for seed in (10, 20, 30)}
    alone = {seed: work(seed, None) for seed in (10, 20, 30)}
    got = {}

    def thread(seed):
        got[seed] = work(seed, torch.cuda.Stream())

    threads = [threading.Thread(target=thread, args=(seed,)) for seed in alone]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for seed, want in alone.items():
        for a, b in zip(got[seed], want):
            assert torch.equal(a, b)


def test_a_call_on_a_stream_needs_a_workspace_and_out_is_not_q():
    c = Cache(1, 2, 100, "int8", False)
    q = rows_of(1, 1, 4)
    with pytest.raises(ValueError, match="workspace"):
        binding.q8_attn(1, 4, 2, 100, q, *c.tensors, None, i32([50]), torch.empty_like(q), stream=torch.cuda.Stream(), **c.layout)
    with pytest.raises(ValueError, match="out"):
        binding.q8_attn(1, 4, 2, 100, q, *c.tensors, None, i32([50]), q, **c.layout)
    with pytest.raises(ValueError, match="workspace"):
        binding.q8_attn(1, 4, 2, 100, q, *c.tensors, None, i32([50]), torch.empty_like(q), workspace=torch.empty(8, dtype=torch.uint8, device="cuda"),
                        **c.layout)
    k = rows_of(2, 1, 2)
    with pytest.raises(ValueError, match="out"):
        binding.packed_attn(q, k, k, i32([0, 1]), None, q)
    with pytest.raises(ValueError, match="k_offsets"):
        binding.packed_attn(q, k, k, i32([0, 1]), i32([0, 1, 1]), torch.empty_like(q))
