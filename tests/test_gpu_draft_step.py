"""A speculative decoding step end to end, as a serving loop runs it: fork, grow with
copy-on-write, rotary append of the drafted tree, tree attention, the accepted path moved into
place, the rest of the pages given back -- against plain decode steps of the accepted tokens."""
import threading

import numpy as np
import pytest
import torch

from _util import MAX_ABS, REL_L2
from gqa_decode_attention_fa_gb300 import binding

pytestmark = pytest.mark.gpu

Hq, Hkv, D, THETA, EPS = 40, 8, 128, 1e6, 1e-6
LAYERS = 2


def bits(t):
    return t.detach().contiguous().view(torch.int16)


class Loop:
    """The state of the draft loop: pages, two layers' pools, a page per 64 tokens."""

    def __init__(self, B, capacity, blocks, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.B, self.cap, self.blocks = B, capacity, blocks
        self.refs, self.lens = torch.zeros(blocks, **i32), torch.zeros(B, **i32)
        self.table = torch.full((B, capacity // 64), -1, **i32)
        self.cow = torch.full((2, B), -1, **i32)
        self.err = torch.zeros(1, **i32)
        rows = blocks * 64
        self.k = [torch.full((rows, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
        self.v = [torch.full((rows, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
        self.pools = binding.CachePools(self.k + self.v, num_blocks=blocks)
        self.wq, self.wk = (1 + 0.1 * self.rn(D).float()).to(torch.bfloat16), (1 + 0.1 * self.rn(D).float()).to(torch.bfloat16)

    def rn(self, *s):
        return torch.randn(*s, generator=self.g, device="cuda").to(torch.bfloat16)

    def resize(self, new):
        binding.pages_resize(self.refs, self.table, self.lens, new, self.cow[0], self.cow[1], device_errors=self.err)
        binding.pages_copy(self.pools, self.cow[0], self.cow[1], device_errors=self.err)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def test_draft_steps_equal_decode_steps():
    B, cap, T = 4, 512, 11
    s = Loop(B, cap, 24, seed=0)
    prompt = [130, 63, 0, 0]
    rope = binding.Rope(theta=THETA)
    # prompts of sequences 0 and 1, one prefill chunk each; 2 and 3 become forks of them
    s.resize(i32(prompt))
    history = [[None] * B for _ in range(LAYERS)]        # per layer and sequence: the (q, k, v) rows so far
    for layer in range(LAYERS):
        for b in (0, 1):
            n = prompt[b]
            q, k, v = s.rn(1, n, Hq, D), s.rn(1, n, Hkv, D), s.rn(1, n, Hkv, D)
            binding.prefill_attn(1, Hq, Hkv, n, cap, q, k, v, s.k[layer], s.v[layer], s.table[b:b + 1].contiguous(), i32([0]), s.wq,
                                 s.wk, THETA, EPS, torch.empty_like(q), block_size=64, num_cache_blocks=s.blocks, device_errors=s.err)
            history[layer][b] = (k[0], v[0])
    binding.pages_fork(s.refs, s.table, s.lens, i32([0, 1]), i32([2, 3]), device_errors=s.err)
    for layer in range(LAYERS):
        history[layer][2], history[layer][3] = history[layer][0], history[layer][1]

    rng = np.random.default_rng(1)
    for step in range(3):
        ctx = s.lens.clone()
        host_ctx = ctx.tolist()
        counts = [T, T - 3, 1, T - 1] if step else [T, T, T, T]
        parents = np.stack([[rng.integers(max(-1, t - 4), t) if t else -1 for t in range(T)] for _ in range(B)]).astype(np.int32)
        s.resize(ctx + i32(counts))
        if step == 0:
            assert (s.cow[0] >= 0).tolist() == [True, True, False, False]     # the first of each pair of holders splits
        mask = torch.zeros(B, T, 1, dtype=torch.int64, device="cuda")
        positions = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        binding.tree_prepare(i32(parents), ctx, i32(counts), mask, positions, device_errors=s.err)
        # an accepted path of each sequence: from a random node up to the context
        paths = []
        for b in range(B):
            t, path = int(rng.integers(0, counts[b])), []
            while t >= 0:
                path.append(t)
                t = int(parents[b][t])
            paths.append(path[::-1])
        outs, news = [], []
        for layer in range(LAYERS):
            qkv = s.rn(B, T, Hq + 2 * Hkv, D)
            q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
            q_rot, out = torch.empty(B, T, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
            binding.rope_append(B, Hq, Hkv, T, cap, q, k, v, s.k[layer], s.v[layer], s.table, ctx, positions, i32(counts), s.wq, s.wk, rope,
                                EPS, q_rot, block_size=64, num_cache_blocks=s.blocks, device_errors=s.err)
            binding.tree_attn(B, Hq, Hkv, T, cap, q_rot, s.k[layer], s.v[layer], s.table, ctx, i32(counts), mask, out, block_size=64,
                              num_cache_blocks=s.blocks, device_errors=s.err)
            outs.append(out)
            news.append((q, k, v))
        keep = np.full((B, T), -1, np.int32)
        for b, path in enumerate(paths):
            keep[b, :len(path)] = path
        took = i32([len(p) for p in paths])
        binding.cache_keep_rows(s.pools, s.table, ctx, i32(keep), took, max_seq_len=cap, device_errors=s.err)
        s.resize(ctx + took)
        assert int(s.err) == 0

        # the same tokens by plain decode steps over contiguous caches of the whole history
        for layer in range(LAYERS):
            q, k, v = news[layer]
            for b, path in enumerate(paths):
                kc = torch.zeros(cap, Hkv, D, dtype=torch.bfloat16, device="cuda")
                vc = torch.zeros_like(kc)
                hk, hv = history[layer][b]
                n0 = host_ctx[b]
                assert hk.shape[0] == n0
                if n0:
                    binding.prefill_attn(1, Hq, Hkv, n0, cap, s.rn(1, n0, Hq, D), hk[None].contiguous(), hv[None].contiguous(), kc, vc, None,
                                         i32([0]), s.wq, s.wk, THETA, EPS, torch.empty(1, n0, Hq, D, dtype=torch.bfloat16, device="cuda"))
                plan = binding.Plan(1, Hq, Hkv, cap)
                for depth, t in enumerate(path):
                    want = torch.empty(1, Hq, D, dtype=torch.bfloat16, device="cuda")
                    plan.decode_attn(q[b, t][None].contiguous(), k[b, t][None].contiguous(), v[b, t][None].contiguous(), kc, vc, None,
                                     i32([n0 + depth + 1]), i32([n0 + depth]), s.wq, s.wk, THETA, EPS, want)
                    got, ref = outs[layer][b, t].double(), want[0].double()
                    # both are within the step's tolerance of the exact output
                    assert float((got - ref).abs().max()) <= 2 * MAX_ABS
                    assert float((got - ref).norm() / ref.norm()) <= 2 * REL_L2
                assert plan.device_errors() == 0
                history[layer][b] = (torch.cat([hk, k[b, path]]), torch.cat([hv, v[b, path]]))
                # the sequence's cache rows are those of the decode steps, in order
                n1 = n0 + len(path)
                slots = torch.arange(n1, device="cuda")
                rows = s.table[b].long()[slots // 64] * 64 + slots % 64
                assert int((bits(s.k[layer][rows]) != bits(kc[:n1])).sum()) <= 1   # two roundings of one exact value (see _util)
                assert torch.equal(bits(s.v[layer][rows]), bits(vc[:n1]))
    s.resize(i32([0] * B))
    assert not bool(s.refs.any()) and bool((s.table == -1).all()) and int(s.err) == 0


def test_a_captured_draft_step_replays():
    """rope_append -> tree_attn -> keep_rows of one layer in a graph, replayed on new inputs."""
    B, cap, T = 3, 256, 6
    s = Loop(B, cap, 15, seed=2)
    s.resize(i32([cap] * B))
    s.k[0].copy_(s.rn(*s.k[0].shape))
    s.v[0].copy_(s.rn(*s.v[0].shape))
    ctx, counts, parents = i32([100, 0, 63]), i32([6, 4, 5]), i32([[-1, 0, 0, 1, 2, -1]] * B)
    keep, took = i32([[0, 2, 4, -1, -1, -1], [1, 3, -1, -1, -1, -1], [3, -1, -1, -1, -1, -1]]), i32([3, 2, 1])
    mask = torch.zeros(B, T, 1, dtype=torch.int64, device="cuda")
    positions = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    q, k, v = s.rn(B, T, Hq, D), s.rn(B, T, Hkv, D), s.rn(B, T, Hkv, D)
    q_rot, out = torch.zeros_like(q), torch.zeros_like(q)
    pools = binding.CachePools([s.k[0], s.v[0]], num_blocks=s.blocks)
    rope = binding.Rope(theta=5e5, layout="interleaved", rotary_dim=64, scaling="yarn", factor=4.0, original_max_len=128)

    def step():
        binding.tree_prepare(parents, ctx, counts, mask, positions, device_errors=s.err)
        binding.rope_append(B, Hq, Hkv, T, cap, q, k, v, s.k[0], s.v[0], s.table, ctx, positions, counts, None, s.wk, rope, EPS, q_rot,
                            block_size=64, num_cache_blocks=s.blocks, device_errors=s.err)
        binding.tree_attn(B, Hq, Hkv, T, cap, q_rot, s.k[0], s.v[0], s.table, ctx, counts, mask, out, block_size=64,
                          num_cache_blocks=s.blocks, device_errors=s.err)
        binding.cache_keep_rows(pools, s.table, ctx, keep, took, max_seq_len=cap, device_errors=s.err)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for x in (q, k, v):
            x.copy_(s.rn(*x.shape))
        k0, v0 = s.k[0].clone(), s.v[0].clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (q_rot, out, s.k[0], s.v[0])]
        s.k[0].copy_(k0)
        s.v[0].copy_(v0)
        step()
        for a, b in zip(got, (q_rot, out, s.k[0], s.v[0])):
            assert torch.equal(bits(a), bits(b))
    assert int(s.err) == 0


def test_threads_with_streams_of_their_own():
    """Steps of several host threads at once, each with its rotary embedding, sizes and stream, give
    the bits of the same steps one after another."""
    ropes = [binding.Rope(theta=1e6), binding.Rope(theta=1e4, layout="interleaved", rotary_dim=64),
             binding.Rope(theta=5e5, scaling="linear", factor=4.0), binding.Rope(rotary_dim=32, scaling="custom", freqs=np.linspace(1, 0.1, 16))]

    def inputs(i):
        s = Loop(2 + i, 256, 16 + 4 * i, seed=10 + i)
        B, T = s.B, 3 + 2 * i
        for x in s.k + s.v:
            x.copy_(s.rn(*x.shape))
        d = dict(s=s, T=T, ctx=i32([10 + 17 * b for b in range(B)]), parents=i32([[t // 2 - 1 if t else -1 for t in range(T)]] * B))
        d["mask"] = torch.zeros(B, T, 1, dtype=torch.int64, device="cuda")
        d["positions"] = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        d["qkv"] = [(s.rn(B, T, Hq, D), s.rn(B, T, Hkv, D), s.rn(B, T, Hkv, D)) for _ in range(6)]
        d["rot"], d["out"] = [s.rn(B, T, Hq, D) for _ in range(6)], [s.rn(B, T, Hq, D) for _ in range(6)]
        d["ws"] = binding.tree_workspace(B, Hq, Hkv, T, s.cap)
        d["keep"], d["took"] = i32([[0, 2, -1]] * B), i32([2] * B)
        return d

    def steps(i, d, stream):
        s, T, B = d["s"], d["T"], d["s"].B
        to = dict(device_errors=s.err, stream=stream)
        paged = dict(block_size=64, num_cache_blocks=s.blocks)
        binding.pages_resize(s.refs, s.table, s.lens, d["full"], s.cow[0], s.cow[1], **to)
        for (q, k, v), rot, out in zip(d["qkv"], d["rot"], d["out"]):
            binding.tree_prepare(d["parents"], d["ctx"], None, d["mask"], d["positions"], **to)
            binding.rope_append(B, Hq, Hkv, T, s.cap, q, k, v, s.k[0], s.v[0], s.table, d["ctx"], d["positions"], None, s.wq, s.wk,
                                ropes[i], EPS, rot, **paged, **to)
            binding.tree_attn(B, Hq, Hkv, T, s.cap, rot, s.k[0], s.v[0], s.table, d["ctx"], None, d["mask"], out, workspace=d["ws"],
                              **paged, **to)
            binding.cache_keep_rows(s.pools, s.table, d["ctx"], d["keep"], d["took"], max_seq_len=s.cap, **to)

    def results(d):
        return [bits(x) for x in d["rot"] + d["out"] + d["s"].k + d["s"].v]

    want = []
    for i in range(4):
        d = inputs(i)
        d["full"] = i32([d["s"].cap] * d["s"].B)
        steps(i, d, None)
        torch.cuda.synchronize()
        assert int(d["s"].err) == 0
        want.append(results(d))
    again = [inputs(i) for i in range(4)]
    for d in again:
        d["full"] = i32([d["s"].cap] * d["s"].B)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            steps(i, again[i], streams[i])
        except Exception as e:  # a thread's own would not reach the test
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in range(4):
        assert int(again[i]["s"].err) == 0
        for a, b in zip(results(again[i]), want[i]):
            assert torch.equal(a, b)


def test_a_captured_step_whose_growth_fails_changes_no_page():
    """resize -> copy -> prepare -> rope_append -> tree_attn -> keep_rows -> resize in one graph, with too few free pages
    for one replay.  The step's counts are what the resize granted, seq_lens less the lengths before it, so
    the page that two sequences still share is not written; with pages enough the same graph splits it."""
    B, cap, T = 3, 256, 5
    s = Loop(B, cap, 6, seed=30)
    s.resize(i32([100, 0, 128]))                                            # two pages, none, two
    binding.pages_fork(s.refs, s.table, s.lens, i32([0]), i32([1]), device_errors=s.err)
    for x in s.k + s.v:
        x.copy_(s.rn(*x.shape))
    ctx, granted, took, wanted = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(4))
    drafted, accepted = i32([T, T, T]), i32([2, 3, 1])
    parents, keep = i32([list(range(-1, T - 1))] * B), i32([[0, 2, 4, -1, -1], [1, 2, 3, -1, -1], [4, -1, -1, -1, -1]])
    mask, positions = torch.zeros(B, T, 1, dtype=torch.int64, device="cuda"), torch.zeros(B, T, dtype=torch.int32, device="cuda")
    q, k, v = s.rn(B, T, Hq, D), s.rn(B, T, Hkv, D), s.rn(B, T, Hkv, D)
    q_rot, out = s.rn(B, T, Hq, D), s.rn(B, T, Hq, D)
    rope, paged, err = binding.Rope(theta=THETA), dict(block_size=64, num_cache_blocks=s.blocks), dict(device_errors=s.err)

    def step():
        ctx.copy_(s.lens)
        torch.add(ctx, drafted, out=wanted)
        s.resize(wanted)
        torch.sub(s.lens, ctx, out=granted)
        torch.minimum(accepted, granted, out=took)
        binding.tree_prepare(parents, ctx, granted, mask, positions, **err)
        for layer in range(LAYERS):
            binding.rope_append(B, Hq, Hkv, T, cap, q, k, v, s.k[layer], s.v[layer], s.table, ctx, positions, granted, s.wq, s.wk, rope,
                                EPS, q_rot, **paged, **err)
            binding.tree_attn(B, Hq, Hkv, T, cap, q_rot, s.k[layer], s.v[layer], s.table, ctx, granted, mask, out, **paged, **err)
        binding.cache_keep_rows(s.pools, s.table, ctx, keep, took, max_seq_len=cap, **err)
        torch.add(ctx, took, out=wanted)
        s.resize(wanted)

    state = [s.refs, s.table, s.lens, out, q_rot] + s.k + s.v
    start = [x.clone() for x in state]
    step()                                                                  # loads every kernel
    for x, y in zip(state, start):
        x.copy_(y)
    s.err.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # 6 pages, 4 in use; needed: one for the split of the shared page, one for the full sequence: enough
    graph.replay()
    torch.cuda.synchronize()
    assert int(s.err) == 0 and s.lens.tolist() == [102, 103, 129] and granted.tolist() == [T] * 3
    a, b = s.table[0, 1].item(), s.table[1, 1].item()
    assert a != b and s.refs[a].item() == s.refs[b].item() == 1
    # one free page: the growth fails as a whole
    for x, y in zip(state, start):
        x.copy_(y)
    free = (s.refs == 0).nonzero().flatten()[0]
    s.refs[free] = 1
    before = [x.clone() for x in state]
    graph.replay()
    torch.cuda.synchronize()
    assert int(s.err) == binding.DEVERR_NOPAGE
    assert granted.tolist() == [0] * 3 and took.tolist() == [0] * 3 and bool((s.cow == -1).all())
    for x, y in zip(state, before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # and with the page back the same graph goes on
    s.err.zero_()
    s.refs[free] = 0
    graph.replay()
    torch.cuda.synchronize()
    assert int(s.err) == 0 and s.lens.tolist() == [102, 103, 129]


def test_page_tables_of_the_largest_capacity():
    """max_seq_len = 2^31 - 1 (2^25 columns a sequence) over a small pool: every call finds the second
    sequence's pages and gives what it gives with a table of three columns."""
    B, T, blocks, small, large = 2, 5, 9, 192, 2 ** 31 - 1
    narrow = i32([[4, 1, 7], [8, 0, 3]])
    wide = torch.full((B, 2 ** 25), -1, dtype=torch.int32, device="cuda")
    wide[:, :3] = narrow
    ctx, counts = i32([70, 127]), i32([5, 4])
    parents, keep, took = i32([[-1, 0, 0, 1, 2]] * B), i32([[1, 3, -1, -1, -1], [0, 2, 3, -1, -1]]), i32([2, 3])
    mask, positions = torch.zeros(B, T, 1, dtype=torch.int64, device="cuda"), torch.zeros(B, T, dtype=torch.int32, device="cuda")
    binding.tree_prepare(parents, ctx, counts, mask, positions)
    got = []
    for cap, table in ((small, narrow), (large, wide)):
        s = Loop(1, 64, blocks, seed=50)
        for x in s.k + s.v:
            x.copy_(s.rn(*x.shape))
        q, k, v = s.rn(B, T, Hq, D), s.rn(B, T, Hkv, D), s.rn(B, T, Hkv, D)
        rot, out, pre = s.rn(B, T, Hq, D), s.rn(B, T, Hq, D), s.rn(B, T, Hq, D)
        paged = dict(block_size=64, num_cache_blocks=blocks, device_errors=s.err)
        binding.prefill_attn(B, Hq, Hkv, T, cap, q, k, v, s.k[1], s.v[1], table, i32([62, 127]), s.wq, s.wk, THETA, EPS, pre, **paged)
        binding.rope_append(B, Hq, Hkv, T, cap, q, k, v, s.k[0], s.v[0], table, ctx, positions, counts, s.wq, s.wk, binding.Rope(theta=THETA),
                            EPS, rot, **paged)
        binding.tree_attn(B, Hq, Hkv, T, cap, rot, s.k[0], s.v[0], table, ctx, counts, mask, out, **paged)
        binding.cache_keep_rows(s.pools, table, ctx, keep, took, max_seq_len=cap, device_errors=s.err)
        torch.cuda.synchronize()
        assert int(s.err) == 0
        got.append((out, [rot, pre] + s.k + s.v))
    for a, b in zip(got[0][1], got[1][1]):
        assert torch.equal(bits(a), bits(b))
    a, b = (x[0].double() for x in got)      # the sequences may be cut otherwise: two roundings of values near each other
    for x, y, n in zip(a, b, counts.tolist()):
        assert float((x[:n] - y[:n]).norm() / y[:n].norm()) <= 2 * REL_L2
        assert torch.equal(bits(x[n:].bfloat16()), bits(y[n:].bfloat16()))
