"""Draft-tree attention on the GPU against the definition in 64 bits.

Tolerance of an output element, derived before the first run: half a bf16 step of the value,
2^-8 |o|, and 2^-12 sum_j p_j |v_j| for the arithmetic before it -- a score is a binary32 sum of
128 exact products, off by at most 128 2^-24 sum |q k| / sqrt(128) (5.5e-5 for N(0,1) data, and a
weight by as much relatively); 2^x and the scaling add about 2^-21; P is kept to 2^-16 in two
bf16 terms; sums of at most 2^13 weights in 64-key steps add 2^-14.  Together under 2^-12."""
import numpy as np
import pytest
import torch

from gqa_decode_attention_fa_gb300 import binding

pytestmark = pytest.mark.gpu
D = 128


def ancestors(parents, n):
    """[n, n] bool: node t sees u (its ancestors and itself)."""
    seen = np.zeros((n, n), bool)
    for t in range(n):
        if parents[t] >= 0:
            seen[t] = seen[parents[t]]
        seen[t, t] = True
    return seen


def pack(seen, T):
    words = (T + 63) // 64
    out = np.zeros((T, words), np.uint64)
    for t, u in zip(*np.nonzero(seen)):
        out[t, u // 64] |= np.uint64(1) << np.uint64(u % 64)
    return out.view(np.int64)


def make(B, Hq, Hkv, T, ctx, counts=None, paged=True, seed=0, slack=7, parents=None, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    rn = lambda *s: (scale * torch.randn(*s, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    ctx = np.asarray(ctx, np.int32)
    n = np.full(B, T, np.int32) if counts is None else np.asarray(counts, np.int32)
    cap = int(max(ctx.max(), 0)) + T + slack
    w = dict(B=B, Hq=Hq, Hkv=Hkv, T=T, cap=cap, ctx=ctx, n=n)
    per = (cap + 63) // 64
    w["blocks"] = B * per + 1 if paged else 0
    w["table"] = torch.randperm(w["blocks"], generator=g, device="cuda")[:B * per].view(B, per).to(torch.int32) if paged else None
    rows = w["blocks"] * 64 if paged else B * cap
    w["q"], w["out"] = rn(B, T, Hq, D), rn(B, T, Hq, D)
    w["k"], w["v"] = rn(rows, Hkv, D), rn(rows, Hkv, D)
    if parents is None:
        parents = np.stack([[rng.integers(-1, t) if t else -1 for t in range(T)] for _ in range(B)])
    w["parents"] = np.asarray(parents, np.int32)
    mask = np.stack([pack(ancestors(w["parents"][b], T), T) for b in range(B)])
    w["mask"] = torch.from_numpy(mask).cuda()
    w["ctx_d"] = torch.from_numpy(ctx).cuda()
    w["n_d"] = None if counts is None else torch.from_numpy(n).cuda()
    w["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return w


def call(w, **over):
    a = dict(w)
    a.update(over)
    binding.tree_attn(a["B"], a["Hq"], a["Hkv"], a["T"], a["cap"], a["q"], a["k"], a["v"], a["table"], a["ctx_d"], a["n_d"], a["mask"], a["out"],
                      block_size=64 if a["table"] is not None else 0, num_cache_blocks=a["blocks"], device_errors=a["err"],
                      workspace=a.get("ws"), stream=a.get("stream"))


def rows_of(w, b, slots):
    if w["table"] is None:
        return b * w["cap"] + slots
    return w["table"][b].long()[slots // 64] * 64 + slots % 64


def reference(w, b):
    """[n, Hq, D] outputs and the sizes sum p |v| of sequence b, in 64 bits (on the GPU)."""
    c, n, G = int(w["ctx"][b]), int(w["n"][b]), w["Hq"] // w["Hkv"]
    slots = torch.arange(c + n, device="cuda")
    rows = rows_of(w, b, slots)
    seen = torch.ones(n, c + n, dtype=torch.bool, device="cuda")
    bits = w["mask"][b, :n]
    for u in range(n):
        seen[:, c + u] = ((bits[:, u // 64] >> (u % 64)) & 1) == 1
    o = torch.zeros(n, w["Hq"], D, dtype=torch.float64, device="cuda")
    s = torch.zeros_like(o)
    for kv in range(w["Hkv"]):
        k, v = w["k"][rows, kv].double(), w["v"][rows, kv].double()
        for t in range(n):   # only the keys the node sees take part
            m = seen[t]
            if not bool(m.any()):
                continue
            p = torch.softmax(w["q"][b, t, kv * G:(kv + 1) * G].double() @ k[m].T / D ** 0.5, -1)
            o[t, kv * G:(kv + 1) * G] = p @ v[m]
            s[t, kv * G:(kv + 1) * G] = p @ v[m].abs()
    return o, s


def verify(w, before, sequences=None, l2=2e-3):
    torch.cuda.synchronize()
    for b in range(w["B"]) if sequences is None else sequences:
        n = int(w["n"][b])
        assert torch.equal(w["out"][b, n:].view(torch.int16), before[b, n:].view(torch.int16)), f"padded rows of {b}"
        if n == 0:
            continue
        o, s = reference(w, b)
        got = w["out"][b, :n].double()
        assert bool(torch.isfinite(got).all()), b
        over = (got - o).abs() - (2.0 ** -8 * o.abs() + 2.0 ** -12 * s)
        assert float(over.max()) <= 0, (b, float(over.max()), np.argwhere((over > 0).cpu().numpy())[:4].tolist())
        if float(o.norm()) > 0:
            assert float((got - o).norm() / o.norm()) <= l2, b
    assert int(w["err"]) == 0


def run(w, **over):
    before = w["out"].clone()
    call(w, **over)
    verify(w, before)


@pytest.mark.parametrize("Hq,Hkv", [(40, 8), (64, 8), (8, 8), (16, 1), (6, 2), (3, 1), (12, 1)])
@pytest.mark.parametrize("T", [1, 5, 17, 64])
@pytest.mark.parametrize("paged", [True, False])
def test_heads_and_tree_sizes(Hq, Hkv, T, paged):
    run(make(2, Hq, Hkv, T, [70, 333], paged=paged, seed=T))


@pytest.mark.parametrize("ctx", [0, 1, 2, 31, 32, 33, 62, 63, 64, 65, 126, 127, 128, 129, 200])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130])
def test_where_the_tree_meets_the_tiles(ctx, T):
    run(make(1, 4, 2, T, [ctx], seed=ctx * 7 + T))


@pytest.mark.parametrize("T", [200, 255, 256])
def test_the_largest_trees(T):
    run(make(2, 32, 2, T, [100, 1], seed=T))
    chain = [list(range(-1, T - 1))] * 2
    run(make(2, 8, 8, T, [0, 65], seed=T, parents=chain))


def test_ragged_batches_and_counts():
    rng = np.random.default_rng(4)
    for B in (3, 33, 70):
        ctx, n = rng.integers(0, 900, B), rng.integers(0, 17, B)
        run(make(B, 20, 4, 16, ctx, n, seed=B))


def test_many_short_sequences_fill_whole_pieces():
    run(make(600, 4, 2, 2, np.arange(600) % 130, seed=1))
    run(make(1024, 1, 1, 1, np.zeros(1024, int), seed=2))


def test_one_long_sequence_is_cut_over_the_gpu():
    run(make(1, 10, 2, 12, [8000], seed=3))
    run(make(1, 16, 1, 40, [8150], seed=4))


def test_long_contexts():
    """131072 tokens of one sequence; every row of two KV heads against the 64-bit definition."""
    run(make(1, 10, 2, 7, [131072 - 7], paged=False, seed=5))
    run(make(2, 4, 1, 3, [100001, 31], seed=6))


def test_any_mask_and_empty_rows():
    """Masks that are not trees: later nodes seen, self not seen, nothing seen at all."""
    rng = np.random.default_rng(6)
    w = make(4, 8, 2, 70, [0, 0, 64, 37], [70, 3, 65, 70], seed=7)
    m = rng.integers(-2 ** 63, 2 ** 63 - 1, w["mask"].shape, dtype=np.int64)
    m[:, ::5] = 0
    w["mask"] = torch.from_numpy(m).cuda()
    run(w)
    out = w["out"].float()
    assert not bool(out[0, ::5].any()) and not bool(out[1, 0].any())     # no context and nothing seen: zeros
    assert bool(out[2, 0].any())


def test_unwritten_slots_and_unseen_nodes_may_hold_anything():
    """NaN and infinities in slots past the tree, in unseen nodes' keys and values, in padded queries."""
    for ctx, T, n in ((60, 9, 6), (0, 70, 66), (130, 5, 5)):
        w = make(1, 8, 2, T, [ctx], [n], seed=ctx + T, slack=200)
        last = ctx + n
        slots = torch.arange(last, w["cap"], device="cuda")
        w["k"][rows_of(w, 0, slots)] = float("nan")
        w["v"][rows_of(w, 0, slots)] = float("inf")
        w["q"][0, n:] = float("nan")
        seen = ((w["mask"][0, :n, 0] >> 1) & 1) == 1               # node 1: some see it, some do not
        row = rows_of(w, 0, torch.tensor([ctx + 1], device="cuda"))
        before = w["out"].clone()
        clean = w["v"][row].clone()
        call(w)
        verify(w, before)
        base = w["out"].clone()
        w["v"][row, 0, 3] = float("inf")
        w["v"][row, 1, 77] = float("nan")
        w["k"][row, 1, 5] = float("nan")
        call(w)
        torch.cuda.synchronize()
        other = [t for t in range(n) if not bool(seen[t])]
        assert other and bool(seen.any())
        assert torch.equal(w["out"][0, other], base[0, other])
        for t in np.nonzero(seen.cpu().numpy())[0]:
            assert bool((w["out"][0, t, :4, 3] == float("inf")).all()) and bool(torch.isnan(w["out"][0, t, 4:]).all())
            keep = [e for e in range(D) if e != 3]
            assert torch.equal(w["out"][0, t, :4][:, keep], base[0, t, :4][:, keep])
        w["v"][row] = clean


def test_growing_scores_rescale():
    """Keys whose scores climb by far more than the lazy rescale's threshold from tile to tile."""
    w = make(1, 8, 1, 20, [900], seed=8)
    slots = torch.arange(920, device="cuda")
    rows = rows_of(w, 0, slots)
    w["q"][:] = w["q"].abs()
    w["k"][rows] = (w["k"][rows].float().abs() * (0.05 + slots.float() / 100)[:, None, None]).to(torch.bfloat16)
    before = w["out"].clone()
    call(w)
    torch.cuda.synchronize()
    o, s = reference(w, 0)
    got = w["out"][0].double()
    # scores reach 9 128 0.64 0.64 / 11.3 = 42 x ... about 500: their binary32 sums are off by up to
    # 128 2^-24 x 500 = 0.004 relative in a weight, which the output's size carries
    assert float(((got - o).abs() - 2.0 ** -8 * o.abs() - 2.0 ** -7 * s).max()) <= 0


def test_same_inputs_same_bits():
    w = make(5, 40, 8, 16, [3000, 17, 800, 0, 5001], [16, 1, 9, 4, 16], seed=9)
    call(w)
    first = w["out"].clone()
    for _ in range(3):
        call(w)
        assert torch.equal(first.view(torch.int16), w["out"].view(torch.int16))


def test_bad_lengths_and_pages_are_contained():
    w = make(5, 8, 2, 4, [100, 50, 60, 200, 90], [4, 4, 4, 4, 4], seed=10)
    w["ctx_d"] = torch.tensor([100, -1, 60, w["cap"] - 3, 90], dtype=torch.int32, device="cuda")
    w["n_d"] = torch.tensor([4, 4, 5, 4, -1], dtype=torch.int32, device="cuda")
    w["table"][0, 0] = w["blocks"]                       # reads as zeros
    before = w["out"].clone()
    call(w)
    torch.cuda.synchronize()
    assert int(w["err"]) == binding.DEVERR_POSITION | binding.DEVERR_SEQLEN | binding.DEVERR_PAGE
    for b in (1, 2, 3, 4):
        assert not bool(w["out"][b].any())
    # sequence 0 with its first page as zeros
    w["err"].zero_()
    w["table"][0, 0] = w["blocks"] - 1 if w["blocks"] - 1 not in w["table"].flatten().tolist() else 0
    free = sorted(set(range(w["blocks"])) - set(w["table"].flatten().tolist()[1:]))[0]
    w["table"][0, 0] = free
    w["k"][free * 64:(free + 1) * 64] = 0
    w["v"][free * 64:(free + 1) * 64] = 0
    verify(w, before, sequences=[0])


def test_two_graphs_with_workspaces_of_their_own():
    ws = [make(3, 40, 8, 16, [1500, 200, 700], seed=s) for s in (11, 12)]
    graphs, streams = [], [torch.cuda.Stream() for _ in ws]
    for w in ws:
        w["ws"] = binding.tree_workspace(w["B"], w["Hq"], w["Hkv"], w["T"], w["cap"])
        call(w)
    torch.cuda.synchronize()
    for w, s in zip(ws, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(w)
        graphs.append(g)
    want = [w["out"].clone() for w in ws]
    for w in ws:
        w["out"].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, x in zip(ws, want):
        assert torch.equal(w["out"].view(torch.int16), x.view(torch.int16))


def test_a_stream_of_the_callers():
    w = make(2, 8, 2, 9, [400, 3], seed=13)
    w["ws"] = binding.tree_workspace(w["B"], w["Hq"], w["Hkv"], w["T"], w["cap"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    before = w["out"].clone()
    torch.cuda.synchronize()
    call(w, stream=s)
    s.synchronize()
    verify(w, before)
    with pytest.raises(ValueError):
        call(w, stream=s, ws=None)
    with pytest.raises(ValueError):
        call(w, ws=w["ws"][:256])


def test_outputs_at_any_16_byte_boundary():
    w = make(3, 8, 2, 5, [100, 0, 70], seed=18)
    call(w)
    want = w["out"].clone()
    room = torch.zeros(w["out"].numel() + 8, dtype=torch.bfloat16, device="cuda")
    w["out"] = room[8:].view(want.shape)
    assert w["out"].data_ptr() % 32 == 16
    call(w)
    assert torch.equal(w["out"].view(torch.int16), want.view(torch.int16)) and not bool(room[:8].any())


def test_wrapper_refuses_wrong_tensors():
    w = make(2, 8, 2, 4, [40, 3], seed=14)
    for name, bad in [("q", w["q"].float()), ("q", w["q"][:, :3]), ("k", w["k"].cpu()), ("mask", w["mask"][:, :, :0]), ("mask", w["mask"].int()),
                      ("ctx_d", w["ctx_d"].long()), ("out", w["out"].transpose(0, 1)), ("v", w["v"][:-1])]:
        with pytest.raises(ValueError):
            call(w, **{name: bad})


def test_no_node_anywhere():
    w = make(3, 8, 2, 5, [100, 0, 7], [0, 0, 0], seed=16)
    before = w["out"].clone()
    call(w)
    torch.cuda.synchronize()
    assert torch.equal(w["out"].view(torch.int16), before.view(torch.int16)) and int(w["err"]) == 0


def test_caches_past_4_gib():
    """Pages at the far end of 4.4 GB pools, filled by rope_append, read by the tree."""
    Hq, Hkv, T, blocks = 16, 8, 9, 34000
    k = torch.empty(blocks * 64, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() * 2 > 1 << 32
    table = torch.tensor([[blocks - 1, 3, blocks - 2], [blocks - 7, blocks - 3, 0]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(17)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    for p in table.flatten().tolist():
        k[p * 64:(p + 1) * 64], v[p * 64:(p + 1) * 64] = rn(64, Hkv, D), rn(64, Hkv, D)
    w = make(2, Hq, Hkv, T, [60, 120], seed=17, slack=192 - 120 - T)
    assert w["cap"] == 192
    w.update(k=k, v=v, table=table, blocks=blocks)
    q, kn, vn = rn(2, T, Hq, D), rn(2, T, Hkv, D), rn(2, T, Hkv, D)
    binding.rope_append(2, Hq, Hkv, T, 192, q, kn, vn, k, v, table, w["ctx_d"], None, None, None, None, binding.Rope(), 1e-6, w["q"],
                        block_size=64, num_cache_blocks=blocks, device_errors=w["err"])
    for b in range(2):
        rows = rows_of(w, b, torch.arange(int(w["ctx"][b]), int(w["ctx"][b]) + T, device="cuda"))
        assert torch.equal(v[rows], vn[b])
    run(w)


def test_random_geometries():
    rng = np.random.default_rng(15)
    for seed in range(25):
        Hkv = int(rng.choice([1, 2, 3, 8]))
        B, T = int(rng.integers(1, 9)), int(rng.integers(1, 100))
        ctx = rng.integers(0, int(rng.choice([5, 200, 3000])), B)
        run(make(B, Hkv * int(rng.integers(1, 17)), Hkv, T, ctx, rng.integers(0, T + 1, B), bool(rng.integers(0, 2)), seed=seed,
                 slack=int(rng.integers(0, 90))))


# ------------------------------------------------------------------------- masks and positions

@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 129, 200, 256])
def test_prepare(T):
    rng = np.random.default_rng(T)
    B = 5
    kinds = [np.full(T, -1), np.arange(-1, T - 1), [rng.integers(max(-1, t - 3), t) for t in range(T)], [rng.integers(-1, t) if t else -1 for t in range(T)],
             np.minimum(np.arange(T) - 1, 0)]
    parents = np.stack(kinds).astype(np.int32)
    ctx = np.array([0, 5, 100000, 7, 2 ** 31 - 1 - T], np.int32)
    counts = np.array([T, T, T // 2, 1, T], np.int32)
    words = (T + 63) // 64
    mask = torch.full((B, T, words), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((B, T), -5, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    garbage = parents.copy()
    for b in range(B):
        garbage[b, counts[b]:] = 10 ** 6           # not read
    binding.tree_prepare(cu(garbage), cu(ctx), cu(counts), mask, pos, device_errors=err)
    assert int(err) == 0
    for b in range(B):
        n = counts[b]
        seen = ancestors(parents[b], n)
        np.testing.assert_array_equal(mask[b, :n].cpu().numpy(), pack(seen, T)[:n])
        np.testing.assert_array_equal(pos[b, :n].cpu().numpy(), ctx[b] + seen.sum(1) - 1)
        assert bool((mask[b, n:] == 77).all()) and bool((pos[b, n:] == -5).all())
    binding.tree_prepare(cu(parents), cu(ctx), None, mask, pos)
    np.testing.assert_array_equal(mask[3].cpu().numpy(), pack(ancestors(parents[3], T), T))


def test_prepare_contains_bad_parents_and_lengths():
    T, cu = 6, lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    parents = [[-1, 0, 2, 1, -2, 4], [-1, 0, 1, 2, 3, 4], [-1, 0, 1, 2, 3, 4], [-1, 0, 1, 2, 3, 4]]
    mask = torch.full((4, T, 1), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((4, T), -5, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.tree_prepare(cu(parents), cu([10, -1, 4, 2 ** 31 - 3]), cu([6, 6, 7, 6]), mask, pos, device_errors=err)
    assert int(err) == binding.DEVERR_POSITION | binding.DEVERR_SEQLEN
    fixed = [-1, 0, -1, 1, -1, 4]                  # node 2's parent was itself, node 4's below -1
    np.testing.assert_array_equal(mask[0].cpu().numpy(), pack(ancestors(fixed, T), T))
    assert pos[0].tolist() == [10, 11, 10, 12, 10, 11]
    assert bool((mask[1:] == 77).all()) and bool((pos[1:] == -5).all())


def test_output_over_the_queries_is_refused():
    z = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ctx, mask, q = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones((1, 1, 1), dtype=torch.int64, device="cuda"), z(1, 1, 4, 128)
    with pytest.raises(ValueError):
        binding.tree_attn(1, 4, 1, 1, 64, q, z(64, 1, 128), z(64, 1, 128), None, ctx, None, mask, q.view(1, 1, 4, 128))


@pytest.mark.parametrize("T", [9, 70])
@pytest.mark.parametrize("ctx", [40, 3001])
def test_values_that_are_not_finite_reach_the_nodes_that_see_them(ctx, T):
    """In sequences whole to a range and in cut ones, with one row tile and with two: +inf, both
    infinities, NaN, each in a dim of its own."""
    w = make(1, 8, 2, T, [ctx], seed=ctx + T, slack=70)
    before = w["out"].clone()
    call(w)
    verify(w, before)
    base = w["out"].clone()
    bits = w["mask"][0].cpu().numpy()
    sees = lambda t, u: bool((int(bits[t, u // 64]) >> (u % 64)) & 1)  # noqa: E731
    pairs = [(t, u, x) for t in range(T) for u in range(t) for x in range(u) if sees(t, u) and sees(t, x)]
    node, u, x = pairs[-1]                                  # a node and two that it sees
    row = lambda y: rows_of(w, 0, torch.tensor([ctx + y], device="cuda"))  # noqa: E731
    w["v"][row(u), 0, 5] = float("inf")
    w["v"][row(u), 0, 100] = float("inf")
    w["v"][row(x), 0, 100] = float("-inf")
    w["v"][row(u), 1, 40] = float("nan")
    w["v"][row(x), 1, 127] = float("-inf")
    call(w)
    torch.cuda.synchronize()
    for t in range(T):
        want = base[0, t].clone()
        first, second = want[:4], want[4:]
        if sees(t, u):
            first[:, 5] = float("inf")
            first[:, 100] = float("nan") if sees(t, x) else float("inf")
            second[:, 40] = float("nan")
        elif sees(t, x):
            first[:, 100] = float("-inf")
        if sees(t, x):
            second[:, 127] = float("-inf")
        got = w["out"][0, t]
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan), t
        assert torch.equal(got[~nan], want[~nan]), t
    assert int(w["err"]) == 0


@pytest.mark.parametrize("T", [9, 70])
@pytest.mark.parametrize("where", ["context", "node"])
def test_values_that_are_not_finite_count_however_small_their_weight(T, where):
    """A cut sequence with one row tile and with two; scores of some ranges lie 2^300 in weight below the
    row's largest, and those hold the values: 0 x inf is NaN, so no rounding of a weight to zero
    makes such a dim finite.  Nodes that do not see the value keep their bits."""
    ctx = 8000
    w = make(1, 8, 2, T, [ctx], seed=T, slack=70)
    rows = rows_of(w, 0, torch.arange(ctx + T, device="cuda"))
    w["q"].fill_(2.0)
    high = slice(4000, None) if where == "context" else slice(0, 4000)
    w["k"][rows] = (0.25 * w["k"][rows].float()).to(torch.bfloat16)
    w["k"][rows[high]] += 10.0                              # scores of 128 x 20 / 11.3 = 226, 2^326 in weight
    call(w)
    o, s = reference(w, 0)
    # scores of 226 sum 128 products of 20: binary32 is off by at most 128 2^-24 2560 / 11.3 = 0.0017
    # in a weight, which with the rest (2^-12) stays below 2^-8
    assert float(((w["out"][0].double() - o).abs() - 2.0 ** -8 * o.abs() - 2.0 ** -8 * s).max()) <= 0
    base = w["out"].clone()
    at = 100 if where == "context" else ctx + T // 2
    seen = [where == "context" or bool((int(w["mask"][0, t, (T // 2) // 64]) >> ((T // 2) % 64)) & 1) for t in range(T)]
    assert any(seen)
    hit = {(0, 7): float("inf"), (0, 100): float("nan"), (1, 64): float("-inf")}
    for (kv, d), x in hit.items():
        w["v"][rows[at], kv, d] = x
    call(w)
    torch.cuda.synchronize()
    for t in range(T):
        touched = torch.zeros(8, D, dtype=torch.bool, device="cuda")
        if seen[t]:
            for kv, d in hit:
                touched[4 * kv:4 * kv + 4, d] = True
        got = w["out"][0, t]
        assert torch.equal(torch.isfinite(got), ~touched), t
        assert torch.equal(got[~touched], base[0, t][~touched]), t
    assert int(w["err"]) == 0


def test_workspace_of_a_page_table_larger_than_any_pool():
    """batch * max_seq_len past 2^31 - 1 rows over a small pool: no contiguous cache has that size, a paged
    one does, and a call on an explicit stream gets its workspace and runs."""
    B, Hq, Hkv, T, cap, blocks = 80, 8, 2, 3, 1 << 25, 9
    assert B * cap > 2 ** 31
    with pytest.raises(binding.GqaError):
        binding.tree_workspace(B, Hq, Hkv, T, cap)
    ws = binding.tree_workspace(B, Hq, Hkv, T, cap, block_size=64, num_cache_blocks=blocks)
    assert ws.numel() == binding.tree_workspace_bytes(B, Hq, Hkv, T, cap, block_size=64, num_cache_blocks=blocks)
    small = make(B, Hq, Hkv, T, np.arange(B) % 9, seed=19)
    assert ws.numel() >= binding.tree_workspace(B, Hq, Hkv, T, small["cap"]).numel()
    # the first column of a table that wide: nine pages, shared by the sequences (the call only reads)
    w = dict(small, cap=cap, blocks=blocks, ws=ws, stream=torch.cuda.Stream())
    w["table"] = torch.full((B, cap // 64), -1, dtype=torch.int32, device="cuda")
    w["table"][:, 0] = torch.arange(B, device="cuda") % blocks
    w["k"], w["v"] = small["k"][:blocks * 64].contiguous(), small["v"][:blocks * 64].contiguous()
    before = w["out"].clone()
    torch.cuda.synchronize()
    call(w)
    verify(w, before)


def test_a_context_that_ends_in_the_last_tile_of_int32():
    """2^31 - 9 cached slots over a table that repeats three pages: the last tile ends at slot 2^31.  With
    keys of zero every weight is alike; a node's infinity reaches those that see it and no other."""
    T, cap = 8, 2 ** 31 - 1
    ctx = cap - T
    blocks = 5
    w = make(1, 2, 1, T, [3], seed=40, parents=[[-1, 0, 0, 1, 2, 4, 4, -1]])
    w.update(cap=cap, ctx=np.array([ctx]), ctx_d=torch.tensor([ctx], dtype=torch.int32, device="cuda"), blocks=blocks)
    w["table"] = (torch.arange(2 ** 25, dtype=torch.int32, device="cuda") % 3)[None].contiguous()
    w["table"][0, -1] = 4                                    # slots 2^31 - 64 on: 55 of the context, then the nodes
    w["k"] = torch.zeros(blocks * 64, 1, D, dtype=torch.bfloat16, device="cuda")
    w["v"] = torch.ones_like(w["k"])
    call(w)
    torch.cuda.synchronize()
    base = w["out"].clone()
    # a part's sums are whole numbers below 2^24, exact; the parts' add up to 2^31 within 152 2^-24
    assert bool((base.float() == 1).all()) and int(w["err"]) == 0
    row = 4 * 64 + (ctx + 2) % 64
    w["v"][row, 0, 9] = float("inf")
    call(w)
    torch.cuda.synchronize()
    sees = [bool((int(w["mask"][0, t, 0]) >> 2) & 1) for t in range(T)]
    assert sees == [False, False, True, False, True, True, True, False]
    for t in range(T):
        touched = torch.zeros(2, D, dtype=torch.bool, device="cuda")
        touched[:, 9] = sees[t]
        assert torch.equal(torch.isfinite(w["out"][0, t]), ~touched), t
        assert torch.equal(w["out"][0, t][~touched], base[0, t][~touched]), t
