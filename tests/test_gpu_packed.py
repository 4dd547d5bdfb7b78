"""Attention over packed prompts on the GPU against the definition in 64 bits.

Tolerance of an output element, derived before the first run: half a bf16 step, 2^-8 |o|; each weight
is rounded to bf16, by at most 2^-8 of it, and divided by the sum of the rounded ones, which moves
the result by at most 2^-8 sum_j p_j |v_j - o| <= 2^-8 (sum_j p_j |v_j| + |o|); and 2^-11 sum_j p_j |v_j| for
the rest: a score is a binary32 sum of 128 exact products, off by at most 128 2^-24 sum |q k| / sqrt(128)
(below 2^-13 for N(0, 1) data, and a weight by as much relatively), 2^x and the scaling add 2^-20, sums of at most
2^13 weights 2^-13.  In the 2-norm over N(0, 1) data both roundings are 2^-8 / sqrt(12) 1.44 = 1.6e-3 of the
result, independent of each other: 2.3e-3 together, of which 3e-3 is allowed."""
import numpy as np
import pytest
import torch

from gqa_decode_attention_fa_gb300 import binding

pytestmark = pytest.mark.gpu
D = 128


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)])


def rows(seed, n, H):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, H, D, generator=g, device="cuda").to(torch.bfloat16)


def make(Hq, Hkv, nq, nk=None, seed=0, spare=3, fused=False):
    qa, ka = offsets(nq), offsets(nq if nk is None else nk)
    N, M = int(qa[-1]) + spare, int(ka[-1]) + spare
    if fused:
        x = rows(seed, N, Hq + 2 * Hkv)
        q, k, v = x.split([Hq, Hkv, Hkv], 1)
    else:
        q, k, v = rows(seed, N, Hq), rows(seed + 1, M, Hkv), rows(seed + 2, M, Hkv)
    return dict(q=q, k=k, v=v, qa=qa, ka=ka, out=torch.full((N, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda"),
                given=nk is not None)


def attend(w, causal=True):
    """(out, sum_j p_j |v_j|) in 64 bits; rows of no sequence as they were."""
    q, k, v = (w[x].double() for x in "qkv")
    out, mag = w["out"].double().clone(), torch.zeros(w["out"].shape, dtype=torch.float64, device="cuda")
    G = q.shape[1] // k.shape[1]
    for b in range(len(w["qa"]) - 1):
        i, j = slice(w["qa"][b], w["qa"][b + 1]), slice(w["ka"][b], w["ka"][b + 1])
        n, m = i.stop - i.start, j.stop - j.start
        if n == 0:
            continue
        kk, vv = (x[j].repeat_interleave(G, 1).transpose(0, 1) for x in (k, v))
        s = q[i].transpose(0, 1) @ kk.transpose(1, 2) / D ** 0.5
        hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1) if causal else torch.zeros(n, m, dtype=torch.bool, device="cuda")
        s = s.masked_fill(hidden, -float("inf"))
        p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0) if m else s
        out[i], mag[i] = (p @ vv).transpose(0, 1), (p @ vv.abs()).transpose(0, 1)
    return out, mag


def run(w, causal=True, **more):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = w["out"].clone()
    binding.packed_attn(w["q"], w["k"], w["v"], i32(w["qa"]), i32(w["ka"]) if w["given"] else None, out, causal=causal,
                        device_errors=err, **more)
    return out, err.item()


def near(out, ref, mag, norm=True):
    off = (out.double() - ref).abs()
    tol = 2.0 ** -7 * ref.abs() + (2.0 ** -8 + 2.0 ** -11) * mag
    assert bool((off <= tol).all()), (off.max().item(), (off / tol.clamp_min(1e-300)).max().item())
    if norm and ref.numel() > 20000:
        assert (out.double() - ref).norm() <= 3e-3 * ref.norm()


@pytest.mark.parametrize("Hq,Hkv,nq,nk,causal", [
    (40, 8, [1], None, True),
    (40, 8, [150], None, True),
    (40, 8, [1, 0, 24, 25, 26, 49, 50, 51, 127, 128, 129, 300], None, True),
    (64, 8, [700, 3, 255], None, True),
    (8, 8, [513, 128, 1, 257], None, True),                 # one head a KV head: 128 tokens a tile
    (16, 1, [333, 40], None, True),                         # 16 heads a KV head
    (18, 2, [100, 9, 0, 77], None, True),                   # 9 heads
    (6, 3, [1000], None, True),
    (40, 8, [64, 1, 130], [1000, 257, 131], True),          # over prefixes
    (32, 8, [200, 1, 5], [201, 129, 1030], True),
    (8, 2, [200, 5, 30], [50, 0, 29], True),                # more queries than keys: the first see none
    (40, 8, [150, 1, 64], [300, 128, 1], False),            # not causal
    (4, 4, [130, 0, 3], [0, 7, 600], False),
    (12, 4, [2500], None, True),
])
def test_packed(Hq, Hkv, nq, nk, causal):
    w = make(Hq, Hkv, nq, nk, seed=Hq + len(nq))
    out, err = run(w, causal)
    ref, mag = attend(w, causal)
    near(out, ref, mag)
    assert err == 0 and torch.equal(out[w["qa"][-1]:], w["out"][w["qa"][-1]:])
    again, _ = run(w, causal)
    assert torch.equal(out, again)


def test_slices_of_one_projection_and_offsets_that_start_later():
    w = make(20, 4, [70, 130, 1], fused=True, spare=9)
    w["qa"] = w["ka"] = w["qa"] + 5
    out, err = run(w)
    ref, mag = attend(w)
    near(out, ref, mag)
    assert err == 0


def test_many_sequences():
    """More sequences than a warp has lanes, up to the largest batch; each result as the sequence's alone."""
    for B, top in ((33, 200), (300, 90), (1024, 40)):
        rng = np.random.default_rng(B)
        nq = rng.integers(0, top + 1, B)
        nk = nq + rng.integers(-10, 60, B).clip(-nq)
        w = make(8, 2, nq, nk, seed=B)
        out, err = run(w)
        ref, mag = attend(w)
        near(out, ref, mag)
        assert err == 0
        b = int(nq.argmax())
        one = {**w, "qa": w["qa"][b:b + 2], "ka": w["ka"][b:b + 2]}
        alone, _ = run(one)
        assert torch.equal(alone[w["qa"][b]:w["qa"][b + 1]], out[w["qa"][b]:w["qa"][b + 1]])


def test_scores_that_grow_and_large_ones():
    """Maxima that rise along the keys (the running maximum is raised often), and scores of hundreds."""
    for scale, slope in ((1.0, 1.0), (6.0, 0.0), (0.01, 0.0)):
        w = make(8, 2, [400, 150], seed=3)
        pos = torch.cat([torch.arange(400), torch.arange(150), torch.zeros(3)]).cuda()
        w["q"][..., 0], w["k"][..., 0] = 10.0, (slope * pos / 8)[:, None].to(torch.bfloat16)
        w["q"][..., 1:] *= scale
        out, err = run(w)
        ref, mag = attend(w)
        # (the scores' error bound grows with them: 2^-24 128 sum |q k| / sqrt(128), under 2^-8 here)
        off = (out.double() - ref).abs()
        assert bool((off <= 2.0 ** -7 * ref.abs() + (2.0 ** -7 + 2.0 ** -11) * mag).all()) and err == 0


@pytest.mark.parametrize("Hq,Hkv", [(40, 8), (8, 8), (16, 1)])
def test_what_a_query_does_not_see_has_no_effect(Hq, Hkv):
    """NaN and infinities in later keys and values, in other sequences and in rows of none."""
    nq = [150, 40, 300, 7]
    w = make(Hq, Hkv, nq, [x + 30 for x in nq], seed=5)
    clean, _ = run(w)
    cut = 90  # query index of sequence 2 from which on it sees the bad rows
    first = int(w["ka"][2]) + cut + 30
    for x, a, b in ((w["k"], float("nan"), float("-inf")), (w["v"], float("inf"), float("nan"))):
        x[first], x[first + 57, :, 9] = a, b
        x[w["ka"][1]:w["ka"][2]] = a
        x[w["ka"][4]:] = b
    w["q"][w["qa"][1]:w["qa"][2]] = float("nan")
    out, err = run(w)
    keep = torch.ones(len(out), dtype=torch.bool, device="cuda")
    keep[w["qa"][1]:w["qa"][2]] = False
    keep[int(w["qa"][2]) + cut:int(w["qa"][3])] = False
    assert err == 0 and torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[int(w["qa"][2]) + cut:int(w["qa"][3])]).all())


@pytest.mark.parametrize("Hq,Hkv", [(40, 8), (8, 8), (16, 1)])
def test_values_that_are_not_finite_reach_what_sees_them(Hq, Hkv):
    w = make(Hq, Hkv, [200, 333], seed=6)
    clean, _ = run(w)
    at = {60: float("inf"), 130: float("-inf"), 131: float("nan"), 299: float("inf")}  # key of sequence 1 -> value in dim 3 + key % 5
    for j, x in at.items():
        w["v"][200 + j, :, 3 + j % 5] = x
    out, err = run(w)
    assert err == 0 and torch.equal(out[:200], clean[:200])
    for i in range(333):
        want = clean[200 + i].clone()
        for j, x in at.items():
            if j <= i:
                want[:, 3 + j % 5] = want[:, 3 + j % 5] + x
        assert torch.equal(torch.isnan(out[200 + i]), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(torch.isinf(out[200 + i][fine]), torch.isinf(want[fine]))
        mine = fine & ~torch.isinf(want)
        assert torch.equal(out[200 + i][mine], want[mine])


def test_offsets_out_of_order():
    w = make(8, 2, [40, 60, 30, 50], seed=7)
    clean, _ = run(w)
    N = len(w["out"])
    for qa, good in (([0, 40, 20, 130, 180], [(20, 130)]), ([-5, 40, 100, 130, 180], [(40, 100), (100, 130), (130, 180)]),
                     ([0, 40, 100, 130, N + 1], [(0, 40), (40, 100), (100, 130)])):
        bad = {**w, "qa": np.array(qa), "ka": np.array(qa)}
        out, err = run(bad)
        assert err == binding.DEVERR_SEQLEN
        touched = torch.zeros(N, dtype=torch.bool, device="cuda")
        for a, b in good:
            touched[a:b] = True
        if qa[1:4] == [40, 100, 130]:
            rows_ = touched & (torch.arange(N, device="cuda") < 130)
            assert torch.equal(out[rows_], clean[rows_])
    # keys out of order: as a sequence without keys
    out, err = run({**w, "ka": np.array([0, 40, 100, 130, N + 1]), "given": True})
    assert err == binding.DEVERR_SEQLEN
    assert bool((out[130:180] == 0).all()) and torch.equal(out[:130], clean[:130])


def test_long_sequences_and_rows_beyond_four_gib():
    """One query a sequence over long keys (the last tiles alone are masked), at byte offsets beyond 32 bits."""
    Hkv = 8
    M = (1 << 32) // (Hkv * D * 2) + 5000
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("not enough device memory")
    k = torch.zeros(M, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    n, m = [1, 70], [3000, 4001]
    ka = np.array([M - sum(m), M - m[1], M])
    k[ka[0]:], v[ka[0]:] = rows(1, sum(m), Hkv), rows(2, sum(m), Hkv)
    w = dict(q=rows(3, 71, Hkv), k=k, v=v, qa=offsets(n), ka=ka, out=torch.zeros(71, Hkv, D, dtype=torch.bfloat16, device="cuda"), given=True)
    out, err = run(w)
    w["k"], w["v"], w["ka"] = k[ka[0]:], v[ka[0]:], ka - ka[0]
    ref, mag = attend(w)
    near(out, ref, mag)
    assert err == 0


def test_padding_and_replay():
    """Many packed rows, all of them prompts (a prompt's bits do not depend on the others) or nearly all padding; and a captured
    call replayed with other lengths."""
    n = [900, 1300, 40, 2000, 1, 700] * 4
    w = make(4, 4, n, seed=11)                       # one head a KV head: units of 256 tokens
    alone = {b: run({**w, "qa": w["qa"][b:b + 2], "ka": w["ka"][b:b + 2]})[0][w["qa"][b]:w["qa"][b + 1]] for b in (3, 4, 21)}
    out, err = run(w)
    ref, mag = attend(w)
    near(out, ref, mag)
    assert err == 0
    for b, x in alone.items():
        assert torch.equal(out[w["qa"][b]:w["qa"][b + 1]], x)
    big = make(32, 32, [40, 333], seed=12, spare=40000)
    out, err = run(big)
    small = {x: big[x][:400] for x in "qkv"} | dict(qa=big["qa"], ka=big["ka"], out=big["out"][:400], given=False)
    ref, mag = attend(small)
    near(out[:400], ref, mag)
    assert err == 0 and torch.equal(out[373:], big["out"][373:])
    # captured with these lengths, replayed with others
    w = make(40, 8, [150, 0, 300, 77], seed=13, spare=700)
    at, out = i32(w["qa"]), w["out"].clone()
    graph = torch.cuda.CUDAGraph()
    binding.packed_attn(w["q"], w["k"], w["v"], at, None, out)
    with torch.cuda.graph(graph):
        binding.packed_attn(w["q"], w["k"], w["v"], at, None, out)
    for lengths in ([150, 0, 300, 77], [1, 1, 1, 1], [0, 0, 0, 0], [600, 500, 100, 20]):
        w["qa"] = w["ka"] = offsets(lengths)
        at.copy_(i32(w["qa"]))
        out.copy_(w["out"])
        graph.replay()
        ref, mag = attend(w)
        near(out, ref, mag, norm=False)


@pytest.mark.parametrize("power", [8, 12])
def test_scores_far_apart(power):
    """Scores of about 2^(2 power): most of the next lie so far below the largest that its value alone counts."""
    w = make(20, 4, [300, 1, 77], [500, 1, 130], seed=21)
    w["q"], w["k"] = w["q"] * 2.0 ** power, w["k"] * 2.0 ** power
    for causal in (True, False):
        out, err = run(w, causal)
        ref, mag = attend(w, causal)
        near(out, ref, mag)
        assert err == 0
