"""The page operators on the GPU against a plain restatement on host integers and bytes: whole
state after every call, valid or not."""
import numpy as np
import pytest
import torch

from gqa_decode_attention_fa_gb300 import binding
from gqa_decode_attention_fa_gb300.binding import DEVERR_CONFLICT, DEVERR_NOPAGE, DEVERR_PAGE, DEVERR_POSITION, DEVERR_SEQLEN

pytestmark = pytest.mark.gpu


def pages(n):
    return -(-n // 64)


class Model:
    """The state and the rules of the page operators, on the host."""

    def __init__(self, B, max_blocks, blocks):
        self.refs = np.zeros(blocks, np.int32)
        self.table = np.full((B, max_blocks), -1, np.int32)
        self.lens = np.zeros(B, np.int32)

    def held(self, b, lo, hi):
        return all(0 <= p < len(self.refs) and self.refs[p] > 0 for p in self.table[b, lo:hi])

    def fork(self, src, dst):
        err, B = 0, len(self.lens)
        plan = []
        for i, (a, b) in enumerate(zip(src, dst)):
            if a < 0:
                continue
            if a >= B or not 0 <= b < B:
                err |= DEVERR_POSITION
            elif any(s >= 0 and (s == b or (j < i and d == b)) for j, (s, d) in enumerate(zip(src, dst))):
                err |= DEVERR_CONFLICT
            elif self.lens[b] != 0 or self.lens[a] < 0 or pages(self.lens[a]) > self.table.shape[1]:
                err |= DEVERR_SEQLEN
            elif not self.held(a, 0, pages(self.lens[a])):
                err |= DEVERR_PAGE
            else:
                plan.append((a, b))
        for a, b in plan:
            n = pages(self.lens[a])
            self.table[b, :n] = self.table[a, :n]
            for p in self.table[a, :n]:
                self.refs[p] += 1
            self.lens[b] = self.lens[a]
        return err

    def resize(self, new):
        B, cap = self.table.shape
        err, act = 0, {}
        cow = np.full((2, B), -1, np.int32)
        for b in range(B):
            if new[b] < 0:
                continue
            if self.lens[b] < 0 or pages(self.lens[b]) > cap or pages(new[b]) > cap:
                err |= DEVERR_SEQLEN
                continue
            have, need = pages(self.lens[b]), pages(new[b])
            if need < have and not self.held(b, need, have):
                err |= DEVERR_PAGE
                continue
            act[b] = (have, need)
        refs = self.refs.copy()
        for b, (have, need) in act.items():
            for p in self.table[b, need:have]:
                refs[p] -= 1
        last = {}
        for b, (have, need) in list(act.items()):
            if new[b] > self.lens[b] and self.lens[b] % 64:
                p = self.table[b, have - 1]
                if not 0 <= p < len(refs) or refs[p] < 1:
                    err |= DEVERR_PAGE
                    del act[b]
                else:
                    last[b] = p
        split = {b for b, p in last.items() if refs[p] - sum(q == p for j, q in last.items() if j < b) > 1}
        take = sum(max(0, act[b][1] - act[b][0]) + (b in split) for b in act)
        free = [int(p) for p in np.nonzero(refs <= 0)[0]]
        if take > len(free):
            return err | DEVERR_NOPAGE, cow
        self.refs = refs
        for b in sorted(act):
            have, need = act[b]
            if b in split:
                p = free.pop(0)
                cow[0, b], cow[1, b] = last[b], p
                self.table[b, have - 1] = p
                refs[p] = 1
            for c in range(have, need):
                p = free.pop(0)
                self.table[b, c] = p
                refs[p] = 1
            self.table[b, need:have] = -1
            self.lens[b] = new[b]
        for b in split:
            refs[last[b]] -= 1
        return err, cow


class Device:
    def __init__(self, m):
        cu = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
        self.refs, self.table, self.lens = cu(m.refs), cu(m.table), cu(m.lens)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cow = torch.full((2, len(m.lens)), -7, dtype=torch.int32, device="cuda")

    def fork(self, src, dst):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.err.zero_()
        binding.pages_fork(self.refs, self.table, self.lens, i(src), i(dst), device_errors=self.err)
        return int(self.err)

    def resize(self, new):
        self.err.zero_()
        binding.pages_resize(self.refs, self.table, self.lens, torch.tensor(np.asarray(new), dtype=torch.int32, device="cuda"),
                             self.cow[0], self.cow[1], device_errors=self.err)
        return int(self.err), self.cow.cpu().numpy()

    def same(self, m):
        np.testing.assert_array_equal(self.lens.cpu().numpy(), m.lens)
        np.testing.assert_array_equal(self.table.cpu().numpy(), m.table)
        np.testing.assert_array_equal(self.refs.cpu().numpy(), m.refs)


def both_resize(m, d, new):
    want, cow = m.resize(np.asarray(new))
    got, gcow = d.resize(new)
    assert got == want
    np.testing.assert_array_equal(gcow, cow)
    d.same(m)
    return want


def both_fork(m, d, src, dst):
    want = m.fork(src, dst)
    assert d.fork(src, dst) == want
    d.same(m)
    return want


@pytest.mark.parametrize("B,max_blocks,blocks", [(1, 1, 1), (3, 4, 9), (8, 6, 40), (40, 33, 700), (1024, 3, 2500), (5, 2100, 9000)])
def test_random_walks(B, max_blocks, blocks):
    """Grow, shrink, free and fork at random, far past the pool's size at times."""
    rng = np.random.default_rng(B)
    m = Model(B, max_blocks, blocks)
    d = Device(m)
    seen = 0
    for step in range(40):
        if rng.random() < 0.4 and B > 1:
            n = int(rng.integers(1, min(B, 64) + 1))
            src = [int(x) for x in rng.integers(-1, B, n)]
            dst = [int(x) for x in rng.integers(0, B, n)]
            seen |= both_fork(m, d, src, dst)
        else:
            new = rng.integers(0, 64 * max_blocks + 1, B)
            near = np.clip(m.lens + rng.integers(-70, 90, B), 0, 64 * max_blocks)
            new = np.where(rng.random(B) < 0.6, near, new)
            new = np.where(rng.random(B) < 0.3, -1, new)
            new = np.where(rng.random(B) < 0.15, 0, new)
            seen |= both_resize(m, d, new)
        held = np.zeros_like(m.refs)                      # the counts are the table's
        for b in range(B):
            np.add.at(held, m.table[b, :pages(m.lens[b])], 1)
        np.testing.assert_array_equal(held, m.refs)
    assert not seen & (DEVERR_PAGE | DEVERR_POSITION)


def test_every_holder_grows_at_once_and_the_last_keeps_the_page():
    m = Model(5, 4, 12)
    d = Device(m)
    both_resize(m, d, [100, -1, -1, -1, 0])
    both_fork(m, d, [0, 0, 0], [1, 2, 3])
    assert both_resize(m, d, [101, 130, 164, 102, -1]) == 0
    assert m.refs[0] == 4 and m.refs[1] == 1 and m.table[3, 1] == 1      # the shared full page, the page sequence 3 keeps
    both_resize(m, d, [0, 0, 0, 0, 0])
    assert not m.refs.any()


def test_too_few_pages_changes_nothing():
    m = Model(3, 8, 4)
    d = Device(m)
    both_resize(m, d, [64, 128, 0])
    assert both_resize(m, d, [0, 512, 64]) == DEVERR_NOPAGE
    assert both_resize(m, d, [0, 256, 0]) == 0            # freed pages are taken by the same call


def test_lengths_and_pages_out_of_range_are_left_alone():
    m = Model(4, 3, 10)
    d = Device(m)
    both_resize(m, d, [100, 100, 100, 192])
    assert both_resize(m, d, [193, -1, 130, 10]) == DEVERR_SEQLEN
    m.table[0, 1], m.table[1, 1] = 10, -1
    m.refs[m.table[2, 1]] = 0                              # a table that names a free page
    d = Device(m)
    assert both_resize(m, d, [120, 10, 135, -1]) == DEVERR_PAGE
    m.lens[3] = -5
    d = Device(m)
    assert both_resize(m, d, [-1, -1, -1, 0]) == DEVERR_SEQLEN


def test_fork_refusals():
    m = Model(6, 3, 10)
    d = Device(m)
    both_resize(m, d, [100, 70, 0, 0, 0, 0])
    assert both_fork(m, d, [0, 1], [2, 2]) == DEVERR_CONFLICT           # the first takes it
    assert both_fork(m, d, [0, 3], [3, 4]) == DEVERR_CONFLICT           # 3 is a source
    assert both_fork(m, d, [5, 0], [5, 6]) == DEVERR_CONFLICT | DEVERR_POSITION
    assert both_fork(m, d, [6, 0, -1], [4, -1, 99]) == DEVERR_POSITION
    assert both_fork(m, d, [0], [1]) == DEVERR_SEQLEN
    m.table[0, 1] = 10
    d = Device(m)
    assert both_fork(m, d, [0], [5]) == DEVERR_PAGE


def bytes_pools(rng, rows, widths):
    return [torch.from_numpy(rng.integers(0, 256, (rows, w), dtype=np.uint8)).cuda() for w in widths]


WIDTHS = [(2048, 2048), (512, 512, 32, 32), (16,), (272, 4112, 65536), (256, 1 << 14)]


@pytest.mark.parametrize("widths", WIDTHS)
def test_copy_pages(widths):
    rng = np.random.default_rng(len(widths))
    blocks = 12
    pools = bytes_pools(rng, blocks * 64, widths)
    want = [p.cpu().numpy().reshape(blocks, -1).copy() for p in pools]
    src, dst = [3, -1, 3, 7, 0, 9], [1, 99, 2, 7, 11, 4]
    for w in want:
        old = w.copy()
        for a, b in zip(src, dst):
            if a >= 0:
                w[b] = old[a]
    cp = binding.CachePools(pools, num_blocks=blocks)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.pages_copy(cp, torch.tensor(src, dtype=torch.int32, device="cuda"), torch.tensor(dst, dtype=torch.int32, device="cuda"),
                       device_errors=err)
    for p, w in zip(pools, want):
        np.testing.assert_array_equal(p.cpu().numpy().reshape(blocks, -1), w)
    assert int(err) == 0


def test_copy_conflicts_and_bad_pages_copy_nothing():
    rng = np.random.default_rng(0)
    pools = bytes_pools(rng, 8 * 64, (64, 2048))
    want = [p.cpu().numpy().reshape(8, -1).copy() for p in pools]
    for w in want:
        w[1] = w[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # (0, 1) is good; (2, 1) names its page again; (4, 3) writes a page that (3, 5) reads, which is fine itself
    src, dst = [0, 2, 4, 3, 8, 6], [1, 1, 3, 5, 7, -1]
    for w in want:
        w[5] = w[3]
    binding.pages_copy(binding.CachePools(pools, num_blocks=8), torch.tensor(src, dtype=torch.int32, device="cuda"),
                       torch.tensor(dst, dtype=torch.int32, device="cuda"), device_errors=err)
    for p, w in zip(pools, want):
        np.testing.assert_array_equal(p.cpu().numpy().reshape(8, -1), w)
    assert int(err) == DEVERR_CONFLICT | DEVERR_PAGE


def test_copy_the_largest_list_and_pools():
    """4096 pairs, 256 pools (an L2-sized cache of thin rows)."""
    rng = np.random.default_rng(5)
    blocks = 8192 + 16
    pools = [torch.from_numpy(rng.integers(0, 256, (blocks * 64, 16), dtype=np.uint8)).cuda() for _ in range(2)]
    perm = rng.permutation(blocks)
    src, dst = perm[:4096].astype(np.int32), perm[4096:8192].astype(np.int32)
    want = [p.cpu().numpy().reshape(blocks, -1).copy() for p in pools]
    for w in want:
        w[dst] = w[src]
    binding.pages_copy(binding.CachePools(pools, num_blocks=blocks), torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
    for p, w in zip(pools, want):
        np.testing.assert_array_equal(p.cpu().numpy().reshape(blocks, -1), w)
    many = [torch.from_numpy(rng.integers(0, 256, (64 * 3, 16), dtype=np.uint8)).cuda() for _ in range(256)]
    want = [p.cpu().numpy().reshape(3, -1)[1].copy() for p in many]
    binding.pages_copy(binding.CachePools(many, num_blocks=3), torch.tensor([1], dtype=torch.int32, device="cuda"),
                       torch.tensor([2], dtype=torch.int32, device="cuda"))
    for p, w in zip(many, want):
        np.testing.assert_array_equal(p.cpu().numpy().reshape(3, -1)[2], w)


def keep_case(rng, B, cap, N, paged, widths, lists=None):
    per = pages(cap)
    blocks = B * per + 1
    rows = blocks * 64 if paged else B * cap
    pools = bytes_pools(rng, rows, widths)
    table = rng.permutation(blocks)[:B * per].reshape(B, per).astype(np.int32) if paged else None
    start = rng.integers(0, cap - N + 1, B).astype(np.int32)
    counts = rng.integers(0, N + 1, B).astype(np.int32)
    keep = np.full((B, N), -1, np.int32)
    for b in range(B):
        kept = np.sort(rng.permutation(N)[:counts[b]])
        keep[b, :counts[b]] = kept
    if lists is not None:
        for b, (s, ks) in enumerate(lists):
            start[b], counts[b] = s, len(ks)
            keep[b] = -1
            keep[b, :len(ks)] = ks
    return pools, table, start, keep, counts, blocks


def run_keep(pools, table, start, keep, counts, blocks, cap, stream=None):
    cu = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cp = binding.CachePools(pools, num_blocks=blocks) if table is not None else binding.CachePools(pools, rows=pools[0].shape[0])
    binding.cache_keep_rows(cp, cu(table), cu(start), cu(keep), cu(counts), max_seq_len=cap, device_errors=err)
    return int(err)


def expect_keep(pools, table, start, keep, counts, cap, skip=()):
    want = []
    for p in pools:
        w = p.cpu().numpy().copy()
        old = w.copy()
        for b in range(len(start)):
            if b in skip:
                continue
            row = lambda s: b * cap + s if table is None else int(table[b, s // 64]) * 64 + s % 64  # noqa: E731,B023
            for i in range(counts[b]):
                w[row(start[b] + i)] = old[row(start[b] + keep[b, i])]
        want.append(w)
    return want


@pytest.mark.parametrize("B,cap,N,paged", [(1, 1, 1, False), (1, 64, 64, True), (3, 200, 16, True), (4, 300, 300, True),
                                           (2, 700, 650, False), (1, 5000, 4700, True), (37, 130, 9, True)])
@pytest.mark.parametrize("widths", WIDTHS[:4])
def test_keep_rows(B, cap, N, paged, widths):
    rng = np.random.default_rng(B + N + len(widths))
    case = keep_case(rng, B, cap, N, paged, widths)
    pools, table, start, keep, counts, blocks = case
    want = expect_keep(pools, table, start, keep, counts, cap)
    assert run_keep(*case, cap) == 0
    for p, w in zip(pools, want):
        np.testing.assert_array_equal(p.cpu().numpy(), w)


def test_keep_edges_of_the_list():
    """All kept, none kept, only the last, every other one, a run after a gap."""
    cap, N = 640, 500
    lists = [(0, list(range(N))), (7, []), (140, [N - 1]), (63, list(range(0, N, 2))), (1, [0, 1, 2] + list(range(100, N)))]
    rng = np.random.default_rng(2)
    case = keep_case(rng, 5, cap, N, True, (2048, 512, 32), lists)
    want = expect_keep(*case[:5], cap)
    assert run_keep(*case, cap) == 0
    for p, w in zip(case[0], want):
        np.testing.assert_array_equal(p.cpu().numpy(), w)


def test_keep_refuses_broken_lists_whole():
    cap, N = 256, 10
    lists = [(0, [1, 1, 2]), (0, [3, 2]), (0, [-1, 2]), (250, [2, 6]), (-1, [1]), (0, [2, 4]), (0, [1, 2]), (5, [2, 3])]
    rng = np.random.default_rng(3)
    pools, table, start, keep, counts, blocks = keep_case(rng, 8, cap, N, True, (2048,), lists)
    want = expect_keep(pools, table, start, keep, counts, cap, skip=(0, 1, 2, 3, 4))
    assert run_keep(pools, table, start, keep, counts, blocks, cap) == DEVERR_POSITION
    np.testing.assert_array_equal(pools[0].cpu().numpy(), want[0])
    counts[5], counts[6], table[7, 0] = 11, -1, blocks
    assert run_keep(pools, table, start, keep, counts, blocks, cap) == DEVERR_POSITION | DEVERR_SEQLEN | DEVERR_PAGE
    np.testing.assert_array_equal(pools[0].cpu().numpy(), want[0])


def test_keep_rows_past_32_bit_offsets():
    """Rows behind the 4 GiB mark of a pool."""
    rows, width = 70000 * 64 // 64 * 64, 65536
    pool = torch.zeros(rows, width // 4, dtype=torch.int32, device="cuda")
    blocks, cap = rows // 64, 128
    table = np.array([[blocks - 1, blocks - 3]], np.int32)
    pool[(blocks - 1) * 64:] = torch.arange(64, dtype=torch.int32, device="cuda")[:, None]
    pool[(blocks - 3) * 64:(blocks - 2) * 64] = torch.arange(64, 128, dtype=torch.int32, device="cuda")[:, None]
    keep = np.array([[5, 60, 99, 127]], np.int32)
    err = run_keep([pool], table, np.array([0], np.int32), keep, np.array([4], np.int32), blocks, cap)
    got = pool[(blocks - 1) * 64:(blocks - 1) * 64 + 5].cpu().numpy()
    assert err == 0 and [int(x) for x in got[:, 0]] == [5, 60, 99, 127, 4] and (got == got[:, :1]).all()
    binding.pages_copy(binding.CachePools([pool], num_blocks=blocks), torch.tensor([blocks - 1], dtype=torch.int32, device="cuda"),
                       torch.tensor([1], dtype=torch.int32, device="cuda"))
    assert torch.equal(pool[64:128], pool[(blocks - 1) * 64:])


def test_captured_growth_and_copy():
    """A graph that grows by one token and splits shared pages, replayed step after step."""
    m = Model(3, 4, 9)
    d = Device(m)
    both_resize(m, d, [60, 0, 0])
    both_fork(m, d, [0], [1])
    rng = np.random.default_rng(1)
    pools = bytes_pools(rng, 9 * 64, (256, 32))
    cp = binding.CachePools(pools, num_blocks=9)
    want = [p.cpu().numpy().reshape(9, -1).copy() for p in pools]
    new = torch.empty(3, dtype=torch.int32, device="cuda")
    grow = torch.tensor([1, 2, 0], dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        torch.add(d.lens, grow, out=new)
        binding.pages_resize(d.refs, d.table, d.lens, new, d.cow[0], d.cow[1], device_errors=d.err)
        binding.pages_copy(cp, d.cow[0], d.cow[1], device_errors=d.err)
    for _ in range(6):
        _, cow = m.resize(m.lens + np.array([1, 2, 0], np.int32))
        for w in want:
            for a, b in cow.T:
                if a >= 0:
                    w[b] = w[a]
        g.replay()
        torch.cuda.synchronize()
        d.same(m)
        for p, w in zip(pools, want):
            np.testing.assert_array_equal(p.cpu().numpy().reshape(9, -1), w)


def test_wrapper_refuses_wrong_tensors():
    m = Model(2, 3, 8)
    d = Device(m)
    with pytest.raises(ValueError):
        binding.pages_resize(d.refs, d.table, d.lens[:1], d.lens, d.cow[0], d.cow[1])
    with pytest.raises(ValueError):
        binding.pages_fork(d.refs, d.table.cpu(), d.lens, d.lens, d.lens)
    with pytest.raises(ValueError):
        binding.CachePools([torch.zeros(100, dtype=torch.uint8, device="cuda")], num_blocks=1)
    with pytest.raises(ValueError):
        binding.CachePools([], num_blocks=1)


def test_pools_that_overlap_are_refused():
    """Two pools on the same memory would have their rows moved twice."""
    whole = torch.zeros(4 * 64 * 48, dtype=torch.uint8, device="cuda")
    row = 4 * 64 * 16
    binding.CachePools([whole[:row], whole[row:2 * row]], num_blocks=4)   # next to each other
    for pools in ([whole[:row], whole[:row]], [whole[16:row + 16], whole[:row]], [whole[row - 16:2 * row - 16], whole[:row]]):
        with pytest.raises(ValueError):
            binding.CachePools(pools, num_blocks=4)


@pytest.mark.parametrize("heads", [1, 2, 3, 5, 6, 7])
def test_pools_whose_rows_the_calls_cannot_move_are_refused_by_name(heads):
    """A 4-bit cache's scales (4 bytes a head) where that is no multiple of 16 bytes, and rows past 2^20."""
    blocks = 3
    idx = torch.zeros(blocks * 64, heads, 64, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(blocks * 64, heads, dtype=torch.float32, device="cuda")
    binding.CachePools([idx], num_blocks=blocks)
    with pytest.raises(ValueError, match="multiple of 4"):
        binding.CachePools([idx, scale], num_blocks=blocks)
    with pytest.raises(ValueError, match="multiple of 16"):
        binding.CachePools([torch.zeros(2, (1 << 20) + 16, dtype=torch.uint8, device="cuda")], rows=2)


@pytest.mark.parametrize("heads", [4, 8, 12])
def test_pages_of_a_4_bit_cache(heads):
    """Indices and scales as the 4-bit decode step lays them out: pages copied, rows kept."""
    blocks, rng = 6, np.random.default_rng(heads)
    idx = [torch.from_numpy(rng.integers(0, 256, (blocks * 64, heads, 64), dtype=np.uint8)).cuda() for _ in range(2)]
    scale = [torch.from_numpy(rng.random((blocks * 64, heads), dtype=np.float32)).cuda() for _ in range(2)]
    pools = binding.CachePools(idx + scale, num_blocks=blocks)
    want = [x.cpu().numpy().copy() for x in idx + scale]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    binding.pages_copy(pools, i32([2, -1, 0]), i32([5, -1, 1]))
    binding.cache_keep_rows(pools, i32([[4, 3]]), i32([60]), i32([[1, 5, 9, -1]]), i32([3]), max_seq_len=128)
    for w, x in zip(want, idx + scale):
        w[5 * 64:], w[64:128] = w[2 * 64:3 * 64], w[:64].copy()
        at = lambda slot: [4, 3][slot // 64] * 64 + slot % 64  # noqa: E731
        old = w.copy()
        for i, k in enumerate((1, 5, 9)):
            w[at(60 + i)] = old[at(60 + k)]
        np.testing.assert_array_equal(x.cpu().numpy(), w)
