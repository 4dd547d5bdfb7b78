"""The 8-bit cache on the GPU: rows quantised and read back, and the attention of one token over
it, against the definitions in 64 bits.

Codes and scales have one right value each (the scale a correctly rounded quotient, the code the level
next to the exact quotient, ties to even): they are compared for equality.  A row read back is
code * scale, a binary32 product (off by 2^-24 of it) rounded to bf16 (half a step, 2^-8 of the value):
the tests allow 2^-8 (1 + 2^-12) |value|, and half of the least bf16 step where that is more.

Tolerance of an output element of the attention, derived before the first run: half a bf16 step,
2^-8 |o|, and 2^-10 sum_j p_j |v_j| for what comes before it: a score is a binary32 sum of 128 exact
products, off by at most 128 2^-24 sum |q k| / sqrt(128) (below 2^-12 for the data here, and a weight by
as much relatively), 2^x and the scalings add 2^-20, the weights times the scale of V are rounded to
binary16 (half a step, 2^-11), sums of at most 2^13 weights add 2^-13."""
import numpy as np
import pytest
import torch

from gqa_decode_attention_fa_gb300 import binding

pytestmark = pytest.mark.gpu
D = 128
MOST = {"e4m3": 448.0, "int8": 127.0}


def levels(fmt):
    if fmt == "int8":
        return np.arange(128.0)
    return np.array([(c % 8) / 8 * 2.0 ** -6 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) for c in range(127)])


def quantised(x, fmt):
    """(codes as values [..., 128] float64, scales float32) of bf16 rows x given as float64."""
    with np.errstate(invalid="ignore", divide="ignore"):
        most = np.abs(x).max(-1)
        scale = (most.astype(np.float32) / np.float32(MOST[fmt])).astype(np.float32)
        bad = ~np.isfinite(x).all(-1)
        scale[bad] = np.nan
        q = np.abs(x) / scale.astype(np.float64)[..., None]
    q = np.where((scale > 0)[..., None], q, 0.0)
    lv = levels(fmt)
    hi = np.clip(np.searchsorted(lv, q), 1, len(lv) - 1)
    below, above = q - lv[hi - 1], lv[hi] - q
    at = np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)
    return np.copysign(lv[at], x) * (lv[at] != 0), scale


def values(codes):
    return codes.cpu().float().double().numpy() if codes.dtype != torch.int8 else codes.cpu().double().numpy()


class Cache:
    """An 8-bit cache of B sequences of `cap` tokens, filled with random codes."""

    def __init__(self, B, Hkv, cap, fmt="e4m3", paged=True, seed=0, spare=2):
        g = torch.Generator(device="cuda").manual_seed(seed + 100)
        self.B, self.Hkv, self.cap, self.fmt, per = B, Hkv, cap, fmt, (cap + 63) // 64
        self.blocks = B * per + spare if paged else 0
        self.table = torch.randperm(self.blocks, generator=g, device="cuda")[:B * per].view(B, per).to(torch.int32) if paged else None
        self.rows = self.blocks * 64 if paged else B * cap
        x = torch.randn(2, self.rows, Hkv, D, generator=g, device="cuda") * MOST[fmt] * 0.37
        x = x.clamp(-MOST[fmt], MOST[fmt])
        x = x.round().to(torch.int8) if fmt == "int8" else x.to(torch.float8_e4m3fn)
        self.k, self.v = x[0].clone(), x[1].clone()
        s = (0.5 + torch.rand(2, self.rows, Hkv, generator=g, device="cuda")) * 2.7 / MOST[fmt]
        self.ks, self.vs = s[0].clone(), s[1].clone()

    @property
    def tensors(self):
        return self.k, self.v, self.ks, self.vs

    @property
    def layout(self):
        return dict(fmt=self.fmt, block_size=64 if self.blocks else 0, num_cache_blocks=self.blocks)

    def slots(self, b, first, n):
        s = np.arange(first, first + n)
        return b * self.cap + s if self.table is None else self.table[b].cpu().numpy()[s // 64].astype(np.int64) * 64 + s % 64

    def dense(self):
        """(K, V) as float64 [rows, Hkv, 128]."""
        return [values(c) * s.cpu().double().numpy()[..., None] for c, s in ((self.k, self.ks), (self.v, self.vs))]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def offsets_of(lengths):
    return np.concatenate([[0], np.cumsum(lengths)])


def errors():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def bf16(x):
    return torch.as_tensor(x).to(torch.bfloat16).cuda()


def rows_of(seed, n, Hkv, kind="normal"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, Hkv, D, generator=g, device="cuda")
    if kind == "wide":  # magnitudes over the whole range of bf16, rows alike within a few binades
        x = x * torch.exp2(torch.randint(-120, 110, (n, Hkv, 1), generator=g, device="cuda").float())
    if kind == "ties":  # quotients on the borders of levels: small whole numbers under a largest one of each kind
        x = torch.randint(-255, 256, (n, Hkv, D), generator=g, device="cuda").float()
        x[..., 0] = torch.randint(128, 256, (n, Hkv), generator=g, device="cuda").float()
        x = torch.where(x.abs() > x[..., :1], x[..., :1], x)
    if kind == "least":  # multiples of the least bf16 number
        x = (x * 40).round() * 2.0 ** -133
    return x.to(torch.bfloat16)


# ------------------------------------------------------------------------------- append and read

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Hkv,lengths,start,paged,kind", [
    (8, [1, 1, 1], [0, 63, 64], True, "normal"),
    (8, [130, 0, 1, 77], [5, 9, 62, 0], True, "wide"),
    (1, [300, 5], [0, 200], True, "ties"),
    (2, [33, 64], [1, 0], False, "least"),
    (5, [40, 0, 0, 90], [0, 0, 3, 63], False, "ties"),
    (16, [20, 300], [7, 0], True, "normal"),
    (3, [1], [0], True, "wide"),
])
def test_append_and_read(fmt, Hkv, lengths, start, paged, kind):
    cap = max(a + b for a, b in zip(lengths, start)) + 3
    c = Cache(len(lengths), Hkv, cap, fmt, paged)
    at = np.concatenate([[0], np.cumsum(lengths)])
    N = int(at[-1]) + 4  # rows behind the last sequence
    k, v = rows_of(1, N, Hkv, kind), rows_of(2, N, Hkv, kind)
    k[N - 2:], v[N - 2:] = float("nan"), float("inf")
    want = [values(t) if t.dim() == 3 else t.cpu().numpy().copy() for t in c.tensors]
    kq, kf = quantised(k.double().cpu().numpy(), fmt)
    vq, vf = quantised(v.double().cpu().numpy(), fmt)
    for b, n in enumerate(lengths):
        rows, mine = c.slots(b, start[b], n), slice(at[b], at[b + 1])
        want[0][rows], want[1][rows], want[2][rows], want[3][rows] = kq[mine], vq[mine], kf[mine], vf[mine]
    err = errors()
    binding.q8_append(c.B, Hkv, N, cap, k, v, *c.tensors, c.table, i32(at), i32(start), device_errors=err, **c.layout)
    for got, ref in zip(c.tensors, want):
        np.testing.assert_array_equal(values(got) if got.dim() == 3 else got.cpu().numpy(), ref)
    ko, vo = rows_of(3, N, Hkv), rows_of(4, N, Hkv)
    ko0, vo0 = ko.clone(), vo.clone()
    binding.q8_read(c.B, Hkv, N, cap, *c.tensors, c.table, i32(at), i32(start), ko, vo, device_errors=err, **c.layout)
    assert err.item() == 0
    for got, before, q, f in ((ko, ko0, kq, kf), (vo, vo0, vq, vf)):
        assert torch.equal(got[at[-1]:], before[at[-1]:])
        ref = (q * f.astype(np.float64)[..., None])[:at[-1]]
        off = np.abs(got[:at[-1]].double().cpu().numpy() - ref)
        assert (off <= np.maximum(2.0 ** -8 * (1 + 2.0 ** -12) * np.abs(ref), 2.0 ** -134)).all(), off.max()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_one_row_each_from_a_projection(fmt):
    """offsets None, k and v slices of one projection, uint8 codes."""
    B, Hkv = 7, 4
    c = Cache(B, Hkv, 100, fmt, True)
    x = rows_of(5, B, 8 + 2 * Hkv)
    k, v = x[:, 8:8 + Hkv], x[:, 8 + Hkv:]
    start = np.arange(B) * 13
    binding.q8_append(B, Hkv, B, 100, k, v, c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks, c.vs, c.table, None, i32(start),
                      **c.layout)
    y = torch.zeros(B, 3 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    binding.q8_read(B, Hkv, B, 100, *c.tensors, c.table, None, i32(start), y[:, Hkv:2 * Hkv], y[:, 2 * Hkv:], **c.layout)
    assert (y[:, :Hkv] == 0).all()
    for got, src in ((y[:, Hkv:2 * Hkv], k), (y[:, 2 * Hkv:], v)):
        q, f = quantised(src.double().cpu().numpy(), fmt)
        ref = q * f.astype(np.float64)[..., None]
        assert (np.abs(got.double().cpu().numpy() - ref) <= 2.0 ** -8 * (1 + 2.0 ** -12) * np.abs(ref)).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rows_of_zeros_and_rows_that_are_not_finite(fmt):
    Hkv, N = 2, 6
    c = Cache(1, Hkv, 70, fmt, True)
    k, v = rows_of(1, N, Hkv), rows_of(2, N, Hkv)
    k[0], v[1, 0] = 0, -0.0
    k[2, 1, 77], v[3, 0, 0], k[4, 0, 127] = float("nan"), float("-inf"), float("inf")
    at, start = i32([0, N]), i32([60])
    binding.q8_append(1, Hkv, N, 70, k, v, *c.tensors, c.table, at, start, **c.layout)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    binding.q8_read(1, Hkv, N, 70, *c.tensors, c.table, at, start, ko, vo, **c.layout)
    for got, src in ((ko, k), (vo, v)):
        bad = ~torch.isfinite(src).all(-1)
        assert bool(torch.isnan(got[bad]).all()) and bool(torch.isfinite(got[~bad]).all())
        assert bool((got[(src == 0).all(-1)] == 0).all())
    rows = torch.as_tensor(c.slots(0, 60, N), device="cuda")
    assert bool((values(c.k)[rows.cpu().numpy()][0] == 0).all()) and bool((c.ks[rows][0] == 0).all())


def test_device_side_errors_are_contained():
    """Bad offsets, starts, capacities and pages: flagged, nothing of the sequence stored or read."""
    B, Hkv, cap = 6, 2, 128
    c = Cache(B, Hkv, cap, "e4m3", True)
    table = c.table.clone()
    table[4, 1] = 10 ** 6
    table[5, 0] = -1
    lengths = [3, 3, 3, 3, 66, 3]
    at = np.concatenate([[0], np.cumsum(lengths)])
    N = int(at[-1])
    start = [0, -1, 126, 0, 60, 0]
    k, v = rows_of(1, N, Hkv), rows_of(2, N, Hkv)
    before = [t.clone() for t in c.tensors]
    err = errors()
    binding.q8_append(B, Hkv, N, cap, k, v, *c.tensors, table, i32(at), i32(start), device_errors=err, **c.layout)
    assert err.item() == binding.DEVERR_POSITION | binding.DEVERR_SEQLEN | binding.DEVERR_PAGE
    written = np.concatenate([c.slots(0, 0, 3), c.slots(3, 0, 3), c.slots(4, 60, 4)])
    for got, old in zip(c.tensors, before):
        same = (got.view(torch.uint8) == old.view(torch.uint8)).view(c.rows, -1).all(1).cpu().numpy()
        assert not same[written].any() and same.sum() == c.rows - len(written)
    ko, vo = rows_of(3, N, Hkv), rows_of(4, N, Hkv)
    ko0 = ko.clone()
    err.zero_()
    binding.q8_read(B, Hkv, N, cap, *c.tensors, table, i32(at), i32(start), ko, vo, device_errors=err, **c.layout)
    assert err.item() == binding.DEVERR_POSITION | binding.DEVERR_SEQLEN | binding.DEVERR_PAGE
    assert torch.equal(ko[3:9], ko0[3:9])
    assert bool((ko[at[4] + 4:] == 0).all()) and bool((vo[at[4] + 4:] == 0).all())
    assert bool((ko[at[4]:at[4] + 4] != ko0[at[4]:at[4] + 4]).any())
    # offsets that descend, start below 0 or pass N
    for bad in ([0, 5, 3, 9, 9, 9, 12], [-2, 3, 6, 9, 10, 11, 12], [0, 3, 6, 9, 10, 11, N + 1]):
        err.zero_()
        binding.q8_append(B, Hkv, N, cap, k, v, *c.tensors, c.table, i32(bad), i32([0] * B), device_errors=err, **c.layout)
        assert err.item() == binding.DEVERR_SEQLEN


def test_many_sequences():
    """Batches of more than 32 and of 1024 sequences, most of them empty or short."""
    for B in (33, 64, 1000, 1024):
        rng = np.random.default_rng(B)
        lengths = rng.integers(0, 4, B)
        c = Cache(B, 1, 10, "int8", False)
        at = np.concatenate([[0], np.cumsum(lengths)])
        N = int(at[-1])
        k, v = rows_of(1, N, 1), rows_of(2, N, 1)
        start = rng.integers(0, 7, B)
        err = errors()
        binding.q8_append(B, 1, N, 10, k, v, *c.tensors, None, i32(at), i32(start), device_errors=err, **c.layout)
        ref, f = quantised(v.double().cpu().numpy(), "int8")
        got, gf = values(c.v), c.vs.cpu().numpy()
        for b in range(B):
            rows = c.slots(b, start[b], lengths[b])
            np.testing.assert_array_equal(got[rows], ref[at[b]:at[b + 1]])
            np.testing.assert_array_equal(gf[rows], f[at[b]:at[b + 1]])
        assert err.item() == 0


# ------------------------------------------------------------------------------- one token's attention

def attend(c, q, lens, Hq):
    """(out [B, Hq, 128], sum_j p_j |v_j|) in 64 bits over the cache's values."""
    G = Hq // c.Hkv
    K, V = c.dense()
    out = np.zeros((c.B, Hq, D))
    mag = np.zeros((c.B, Hq, D))
    qd = q.double().cpu().numpy()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        rows = c.slots(b, 0, n)
        for h in range(Hq):
            k, v = K[rows, h // G], V[rows, h // G]
            s = (k @ qd[b, h]) / np.sqrt(D)
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h], mag[b, h] = p @ v, p @ np.abs(v)
    return out, mag


def token(c, q, lens, Hq, **more):
    out = torch.full((c.B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    err = errors()
    ws = binding.q8_workspace(c.B, Hq, c.Hkv, c.cap, block_size=64 if c.blocks else 0, num_cache_blocks=c.blocks)
    ws.fill_(255)
    binding.q8_attn(c.B, Hq, c.Hkv, c.cap, q, *c.tensors, more.get("table", c.table), i32(lens), out, workspace=ws,
                    device_errors=err, **c.layout)
    return out, err.item()


def near(out, ref, mag, least=0.0):
    off = np.abs(out.double().cpu().numpy() - ref)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag + least
    assert (off <= tol).all(), (off.max(), (off / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Hq,Hkv,lens,paged,slack", [
    (40, 8, [256], False, 0),
    (40, 8, [1, 0, 15, 16, 17, 63, 64, 65, 300], True, 5),          # one CTA a sequence and head (small capacity)
    (40, 8, [1, 0, 15, 16, 17, 63, 64, 65, 1300], True, 5),         # cut into ranges
    (64, 8, [5000], True, 0),
    (8, 8, [700, 900, 0, 33], False, 1),
    (16, 1, [2000, 1, 0, 777], True, 0),                            # 16 heads a KV head, 8 warps a head
    (18, 2, [900, 1000], False, 3),                                 # 9 heads
    (6, 3, [600, 601, 602], True, 0),                               # KV heads that are no power of two
    (20, 4, [3000, 10, 4000, 0, 0, 1], True, 0),
    (32, 32, [520, 100], True, 0),
    (15, 5, [1111], False, 2),
    (4, 4, [0, 0], True, 600),
])
def test_one_token(fmt, Hq, Hkv, lens, paged, slack):
    c = Cache(len(lens), Hkv, max(max(lens), 1) + slack, fmt, paged, seed=len(lens))
    q = rows_of(9, len(lens), Hq)
    out, err = token(c, q, lens, Hq)
    ref, mag = attend(c, q, lens, Hq)
    near(out, ref, mag)
    assert err == 0
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((out[b] == 0).all())
    again, _ = token(c, q, lens, Hq)
    assert torch.equal(out, again)


def test_many_sequences_attend():
    """More sequences than ranges; ragged, some empty."""
    for B, cap in ((400, 700), (700, 520), (1024, 40)):
        rng = np.random.default_rng(B)
        lens = rng.integers(0, cap + 1, B)
        lens[rng.random(B) < 0.2] = 0
        c = Cache(B, 2, cap, "int8", False)
        q = rows_of(3, B, 4)
        out, err = token(c, q, lens, 4)
        ref, mag = attend(c, q, lens, 4)
        near(out, ref, mag)
        assert err == 0


@pytest.mark.parametrize("B,Hq,Hkv,cap,top,wide", [
    (700, 4, 2, 6000, 100, 3),       # more sequences than ranges, most of them short
    (90, 4, 1, 30000, 60, 900),
    (40, 64, 16, 9000, 50, 1000),    # KV heads in twos, in fours, in eights
    (10, 32, 32, 9000, 300, 500),
    (6, 64, 64, 5000, 300, 500),
    (5, 48, 3, 4000, 200, 1500),     # 16 heads a KV head
])
def test_lengths_far_below_the_capacity(B, Hq, Hkv, cap, top, wide):
    """A pool smaller than every sequence at full length: the sequences are cut by the lengths on the device."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, top + 1, B)
    lens[rng.random(B) < 0.2] = 0
    lens[rng.integers(0, B)] = wide
    need = (lens + 63) // 64
    c = Cache(1, Hkv, 64 * int(need.sum()), "e4m3", True, seed=B)
    pages, at = c.table[0].cpu().numpy(), offsets_of(need)
    table = np.full((B, (cap + 63) // 64), -7, np.int32)
    for b in range(B):
        table[b, :need[b]] = pages[at[b]:at[b + 1]]
    c.B, c.cap, c.table = B, cap, i32(table)
    q = rows_of(3, B, Hq)
    out, err = token(c, q, lens, Hq)
    ref, mag = attend(c, q, lens, Hq)
    near(out, ref, mag)
    assert err == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("cap", [400, 3000])
def test_slots_behind_the_length_have_no_effect(fmt, cap):
    B, Hq, Hkv = 3, 16, 4
    c = Cache(B, Hkv, cap, fmt, True)
    lens = [cap - 65, 1, cap - 7]
    q = rows_of(4, B, Hq)
    out, _ = token(c, q, lens, Hq)
    keep = np.concatenate([c.slots(b, 0, n) for b, n in enumerate(lens)])
    rest = torch.as_tensor(np.setdiff1d(np.arange(c.rows), keep), device="cuda")
    c.k.view(torch.uint8)[rest] = 0x7f
    c.v.view(torch.uint8)[rest] = 0xff
    c.ks[rest], c.vs[rest] = float("nan"), float("inf")
    again, err = token(c, q, lens, Hq)
    assert err == 0 and torch.equal(out, again)


@pytest.mark.parametrize("cap", [300, 2500])
def test_scales_over_the_whole_range(cap):
    """Rows of V whose scales lie many binades apart, growing, falling and mixed; a head whose weight sits
    on a row of small values (as where a first token takes the weight); tiny and large queries."""
    B, Hq, Hkv = 4, 8, 4
    c = Cache(B, Hkv, cap, "e4m3", False)
    slot = torch.arange(cap, device="cuda").float()
    vs = c.vs.view(B, cap, Hkv)
    vs[0] *= torch.exp2(-20 + 40 * slot / cap)[:, None]
    vs[1] *= torch.exp2(20 - 40 * slot / cap)[:, None]
    vs[2] *= torch.exp2(torch.randint(-10, 10, (cap, Hkv), device="cuda").float())
    vs[3, 1:] *= 2.0 ** 10
    c.ks.view(B, cap, Hkv)[:, :, 3] *= 2.0 ** -60
    q = rows_of(6, B, Hq)
    q[:, 6:] *= 2.0 ** 60
    q[:, :2] *= 2.0 ** -40
    c.k.view(B, cap, Hkv, D)[3, 0, 1] = q[3, 2].float().mul(100).clamp(-448, 448).to(torch.float8_e4m3fn)
    lens = [cap, cap - 1, cap - 17, cap]
    out, err = token(c, q, lens, Hq)
    ref, mag = attend(c, q, lens, Hq)
    near(out, ref, mag)
    assert err == 0


@pytest.mark.parametrize("power", [-135, -100, 100, 115])
def test_extreme_scales(power):
    """Values near the ends of binary32's range: alike within a few binades."""
    c = Cache(2, 2, 600, "int8", True)
    c.vs *= 2.0 ** power
    q = rows_of(6, 2, 4)
    out, err = token(c, q, [600, 77], 4)
    ref, mag = attend(c, q, [600, 77], 4)
    near(out, ref, mag, 2.0 ** -134)
    # (at 2^-135 a value is 2^-135 and the mean of 77 of them about 2^-138, below half of the least bf16 number, 2^-133)
    assert err == 0 and bool((out != 0).any()) == bool((np.abs(ref) >= 2.0 ** -133).any())


@pytest.mark.parametrize("power", [8, 26])
@pytest.mark.parametrize("cap", [300, 2500])
def test_a_key_far_above_the_others(cap, power):
    """One slot's score is 2^(power + 3) and more above all others, which weigh nothing beside it: the output is its value, be that
    zeros (nothing else may then be scaled up in its place) or far smaller or larger than the values before it."""
    B, Hq, Hkv = 4, 12, 4
    c = Cache(B, Hkv, cap, "int8", False)
    q = rows_of(9, B, Hq).abs()
    at = torch.arange(B, device="cuda") * cap + torch.tensor([200, 0, 76, 55], device="cuda")
    c.k[at] = 127
    c.ks[at] = 2.0 ** (power - 7)
    c.vs[at[:, None], torch.arange(4, device="cuda")] *= torch.tensor([0.0, 1.0, 2.0 ** -40, 2.0 ** 40], device="cuda")
    lens = [cap, cap - 1, 77, 60]
    out, err = token(c, q, lens, Hq)
    ref, mag = attend(c, q, lens, Hq)
    near(out, ref, mag)
    assert err == 0 and bool((out[:, :3] == 0).all())


@pytest.mark.parametrize("fmt,Hq,Hkv,cap,lens", [
    ("int8", 20, 4, 300, [300, 1, 150, 0, 47]),
    ("e4m3", 40, 8, 300, [299, 64]),
    ("int8", 8, 1, 2600, [2600, 900, 17]),
    ("e4m3", 32, 2, 5000, [4100, 33]),
])
def test_scales_of_many_sizes(fmt, Hq, Hkv, cap, lens):
    """V scales over 60 binades.  A product x of a weight and a scale is a binary16 number under a power of two by which the
    largest is at least 2^8: half a step below 2^-14 is 2^-25, 2^-33 of the largest.  n of them, times codes of at most Q, may be off by
    n Q 2^-33 of it, beside what `near` allows (twice that is: a warp's largest is its own)."""
    c = Cache(len(lens), Hkv, cap, fmt, True, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    c.vs *= torch.exp2(torch.randint(-30, 30, c.vs.shape, generator=g, device="cuda").float())
    q = rows_of(7, len(lens), Hq)
    out, err = token(c, q, lens, Hq)
    ref, mag = attend(c, q, lens, Hq)
    K, _ = c.dense()
    floor = np.zeros((len(lens), Hq, 1))
    for b, n in enumerate(lens):
        rows = c.slots(b, 0, n)
        for h in range(Hq if n else 0):
            s = (K[rows, h // (Hq // Hkv)] @ q[b, h].double().cpu().numpy()) / np.sqrt(D)
            p = np.exp(s - s.max())
            floor[b, h] = n * MOST[fmt] * 2.0 ** -32 * (p / p.sum() * c.vs[:, h // (Hq // Hkv)].double().cpu().numpy()[rows]).max()
    near(out, ref, mag, floor)
    assert err == 0


@pytest.mark.parametrize("cap", [300, 2500])
def test_values_that_are_not_finite_reach_what_sees_them(cap):
    B, Hq, Hkv = 3, 8, 4
    c = Cache(B, Hkv, cap, "e4m3", False)
    clean, _ = token(c, q := rows_of(4, B, Hq), [cap] * B, Hq)
    c.ks.view(B, cap, Hkv)[0, 5, 1] = float("nan")
    c.vs.view(B, cap, Hkv)[1, cap - 1, 2] = float("nan")
    c.v.view(torch.uint8).view(B, cap, Hkv, D)[2, 17, 3, 9] = 0x7f
    out, err = token(c, q, [cap] * B, Hq)
    bad = torch.zeros(B, Hq, D, dtype=torch.bool, device="cuda")
    bad[0, 2:4], bad[1, 4:6], bad[2, 6:8, 9] = True, True, True
    assert err == 0 and bool(torch.isnan(out[bad]).all()) and torch.equal(out[~bad], clean[~bad])
    q[0, 0, 3] = float("inf")
    q[1, 0, 3] = float("nan")
    out, _ = token(c, q, [cap] * B, Hq)
    assert bool(torch.isnan(out[:2, 0]).all()) and torch.equal(out[:, 1][~bad[:, 1]], clean[:, 1][~bad[:, 1]])


@pytest.mark.parametrize("cap", [300, 2500])
def test_bad_lengths_and_pages(cap):
    B, Hq, Hkv = 4, 8, 2
    c = Cache(B, Hkv, cap, "e4m3", True)
    q = rows_of(4, B, Hq)
    lens = [cap, -1, cap + 1, cap]
    table = c.table.clone()
    table[3, 1], table[3, 2] = c.blocks, -5
    out, err = token(c, q, lens, Hq, table=table)
    assert err == binding.DEVERR_SEQLEN | binding.DEVERR_PAGE
    assert bool((out[1:3] == 0).all())
    zero = torch.as_tensor(c.slots(3, 64, 128), device="cuda")
    for x in c.tensors:
        x.view(torch.uint8)[zero] = 0
    ref, mag = attend(c, q, [cap, 0, 0, cap], Hq)
    near(out, ref, mag)


def test_rows_beyond_four_gib():
    """A cache whose byte offsets pass 32 bits."""
    Hkv, cap = 8, (1 << 32) // (8 * 128) + 700
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("not enough device memory")
    k = torch.zeros(cap, Hkv, D, dtype=torch.int8, device="cuda")
    v, s = torch.zeros_like(k), torch.zeros(2, cap, Hkv, device="cuda")
    c = Cache(1, Hkv, 4, "int8", False)
    c.cap = c.rows = cap
    c.k, c.v, c.ks, c.vs = k, v, s[0], s[1]
    n = 600
    x, y = rows_of(1, n, Hkv), rows_of(2, n, Hkv)
    binding.q8_append(1, Hkv, n, cap, x, y, *c.tensors, None, i32([0, n]), i32([cap - n]), **c.layout)
    ko, vo = torch.empty_like(x), torch.empty_like(y)
    binding.q8_read(1, Hkv, n, cap, *c.tensors, None, i32([0, n]), i32([cap - n]), ko, vo, **c.layout)
    kq, kf = quantised(x.double().cpu().numpy(), "int8")
    vq, vf = quantised(y.double().cpu().numpy(), "int8")
    kd, vd = kq * kf.astype(float)[..., None], vq * vf.astype(float)[..., None]
    assert (np.abs(ko.double().cpu().numpy() - kd) <= 2.0 ** -8 * (1 + 2.0 ** -12) * np.abs(kd)).all()
    q = rows_of(3, 1, Hkv) * 4
    out, err = token(c, q, [cap], Hkv)
    assert err == 0
    for h in range(Hkv):
        z = kd[:, h] @ q[0, h].double().cpu().numpy() / np.sqrt(D)
        top = max(z.max(), 0.0)
        p = np.exp(z - top)
        total = p.sum() + (cap - n) * np.exp(-top)
        ref, mag = (p @ vd[:, h]) / total, (p @ np.abs(vd[:, h])) / total
        off = np.abs(out[0, h].double().cpu().numpy() - ref)
        assert (off <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag).all()
