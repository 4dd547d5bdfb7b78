"""Cases for the operators of one speculative decoding step over a KV cache: attention of a tree of
drafted tokens over the cache (and the tree's mask and positions), QK-norm + rotary embedding +
append in the layouts and scalings models use, and the page operations around them (fork, grow
with copy-on-write, copy, keep the accepted rows).

`run` with `own` false computes each operator from its definition in elementary torch operations;
with `own` true it calls the package.  Caches are bf16, head_dim 128, pages of 64 tokens."""
import math

import torch

own = False

D = 128
PAGE = 64
DEV = "cuda"
BF16 = torch.bfloat16


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # the latency end: a 4-node draft on a short contiguous cache (40/8 heads, 256 tokens)
        dict(name="tree_draft4_256", op="tree", B=1, Hq=40, Hkv=8, T=4, lo=251, hi=251, paged=False, ragged=False),
        # one new token a sequence (the plain decode shape), 8 sequences of 32k: one layer of the 40-layer workload
        dict(name="tree_one_token_8x32k", op="tree", B=8, Hq=40, Hkv=8, T=1, lo=32767, hi=32767, paged=True, ragged=False),
        # serving batch: 32 ragged contexts, up to 16 drafted nodes each (ragged counts), paged
        dict(name="tree_draft16_ragged", op="tree", B=32, Hq=40, Hkv=8, T=16, lo=512, hi=8176, paged=True, ragged=True),
        # a wide draft on one 128k context with 64/8 heads: bound by the tensor core, not by the cache
        dict(name="tree_draft64_128k", op="tree", B=1, Hq=64, Hkv=8, T=64, lo=131008, hi=131008, paged=False, ragged=False),
        # the step's tree tables: small and large batches of drafts
        dict(name="prepare_32x16", op="prepare", B=32, T=16, lo=512, hi=8176, ragged=True),
        # decode-sized rotary: one token a sequence, half-split, unscaled, QK-norm
        dict(name="rope_decode_32", op="rope", B=32, Hq=40, Hkv=8, T=1, lo=512, hi=8176, layout="half", r=128,
             scaling="none", norm=True, paged=True, ragged=False),
        # drafts at far positions: interleaved pairs over half of the head, YaRN, ragged counts
        dict(name="rope_yarn_32x16_far", op="rope", B=32, Hq=64, Hkv=8, T=16, lo=65536, hi=131000, layout="interleaved",
             r=64, scaling="yarn", norm=False, paged=False, ragged=True),
        # a prefill-sized chunk, banded scaling
        dict(name="rope_banded_8x1000", op="rope", B=8, Hq=40, Hkv=8, T=1000, lo=0, hi=7168, layout="half", r=128,
             scaling="banded", norm=True, paged=True, ragged=False),
        # two continuations of one prompt, a two-layer draft model: latency of the bookkeeping
        dict(name="fork_grow_2", op="fork", n=2, pools=4, lo=100, hi=300, T=9, blocks=64),
        # beam fork of 32 sequences, 40 layers (80 pools): each copies its last, shared page in every layer
        dict(name="fork_grow_32x40", op="fork", n=32, pools=80, lo=65, hi=190, T=17, blocks=256),
        # accepted drafts of 32 sequences moved into place in all 40 layers
        dict(name="keep_draft_32x40", op="keep", B=32, pools=80, start_lo=70, start_hi=110, n=16, keep=5),
        # eviction: half of 8000 cached tokens kept in each of 4 sequences, 8 layers
        dict(name="keep_evict_4x8000", op="keep", B=4, pools=16, start_lo=4, start_hi=64, n=8000, keep=4000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "prepare", "rope", "rope", "fork", "keep"])
    heads = rng.choice([(40, 8), (64, 8), (32, 8), (8, 8), (16, 1), (20, 4)])
    if op == "tree":
        T = _log(rng, 1, 130)
        B = _log(rng, 1, 48)
        # tokens of cache in the batch, bounded by the largest listed cases' bytes and products
        room = min(262144, int(131072 * 64 * 64 / max(1, T * heads[0])))
        hi = max(2, min(131072 - T, room // B))
        hi = _log(rng, 1, hi)
        return dict(op="tree", B=B, Hq=heads[0], Hkv=heads[1], T=T, lo=rng.randint(0, hi), hi=hi, paged=rng.random() < 0.6,
                    ragged=rng.random() < 0.5)
    if op == "prepare":
        return dict(op="prepare", B=_log(rng, 1, 256), T=_log(rng, 1, 256), lo=0, hi=rng.randint(1, 9000),
                    ragged=rng.random() < 0.5)
    if op == "rope":
        T = _log(rng, 1, 900)
        B = _log(rng, 1, max(1, min(64, 7000 // T)))
        lo = rng.choice([0, 5, 4096, 100001])
        return dict(op="rope", B=B, Hq=heads[0], Hkv=heads[1], T=T, lo=lo, hi=lo + rng.randint(0, 4000),
                    layout=rng.choice(["half", "interleaved"]), r=rng.choice([128, 128, 96, 64, 32, 24]),
                    scaling=rng.choice(["none", "linear", "banded", "yarn"]), norm=rng.random() < 0.5,
                    paged=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "fork":
        n = _log(rng, 1, 40)
        lo = rng.randint(1, 150)
        hi = lo + rng.randint(0, 150)
        return dict(op="fork", n=n, pools=2 * _log(rng, 1, 24), lo=lo, hi=hi, T=rng.randint(1, 40), blocks=n * 8 + rng.randint(0, 50))
    n = _log(rng, 1, 4000)
    B = _log(rng, 1, max(1, min(32, 16000 // n)))
    lo = rng.randint(0, 200)
    return dict(op="keep", B=B, pools=2 * _log(rng, 1, 8), start_lo=lo, start_hi=lo + rng.randint(0, 100), n=n,
                keep=rng.randint(0, n))


# --------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(BF16)


def _randint(g, lo, hi, *shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(int(lo), int(hi) + 1, shape, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)


def _twice(a):
    return ((a @ a) > 0).float()


def _closure(parents):
    """[B, T, T] float 0/1: node t's ancestors and itself, from parents[b][t] in [-1, t)."""
    T = parents.shape[1]
    u = torch.arange(T, device=parents.device)
    a = ((parents[:, :, None] == u) | (u[:, None] == u)).float()
    return _twice(_twice(_twice(_twice(_twice(_twice(_twice(_twice(a))))))))  # paths of up to 2^8 edges


def _pack(seen):
    """[B, T, T] 0/1 -> [B, T, ceil(T/64)] int64 words, bit u of word u/64 for node u."""
    B, T, _ = seen.shape
    W = (T + 63) // 64
    bits = torch.zeros(B, T, W * 64, dtype=torch.int64, device=seen.device)
    bits[:, :, :T] = seen.to(torch.int64)
    return (bits.view(B, T, W, 64) << torch.arange(64, device=seen.device)).sum(-1)


def _tree(g, B, T):
    """Drafted trees: each node hangs from one of the few before it, the first from the context."""
    back = _randint(g, 1, 4, B, T)
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    return torch.clamp(t - back, min=-1).to(torch.int32)


def _counts(g, B, T, ragged):
    return _randint(g, 1, T, B) if ragged else torch.full((B,), T, device=DEV, dtype=torch.int32)


def _table(g, B, capacity):
    """A page table of capacity tokens a sequence over a permuted pool with a few spare pages."""
    per = (capacity + PAGE - 1) // PAGE
    blocks = B * per + 3
    perm = torch.randperm(blocks, generator=g, device=DEV)[: B * per]
    return perm.view(B, per).to(torch.int32), blocks


def _cache(g, rows, Hkv):
    return _randn(g, rows, Hkv, D)


def _capacity(case):
    return case["hi"] + case["T"] + 5


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c}
    op = c["op"]
    if op in ("tree", "rope"):
        B, T = c["B"], c["T"]
        cap = _capacity(c)
        s["cap"] = cap
        s["ctx"] = _randint(g, c["lo"], c["hi"], B)
        s["counts"] = _counts(g, B, T, c["ragged"])
        if c["paged"]:
            s["table"], s["blocks"] = _table(g, B, cap)
            rows = s["blocks"] * PAGE
        else:
            s["table"], s["blocks"] = None, 0
            rows = B * cap
        # what a pass leaves as it was (rows of padded nodes; for rope the cache around the new rows) is kept
        # small, so that it does not hide the size of an error in what the pass writes
        small = 1e-3
        s["k_cache"], s["v_cache"] = _cache(g, rows, c["Hkv"]), _cache(g, rows, c["Hkv"])
        if op == "rope":
            s["k_cache"].mul_(small), s["v_cache"].mul_(small)
        s["out"] = small * _randn(g, B, T, c["Hq"], D)
        s["q"] = _randn(g, B, T, c["Hq"], D)
        parents = _tree(g, B, T)
        if op == "tree":
            s["mask"] = _pack(_closure(parents))
            if own:
                from gqa_decode_attention_fa_gb300 import binding
                s["workspace"] = binding.tree_workspace(B, c["Hq"], c["Hkv"], T, cap)
        else:
            s["k"], s["v"] = _randn(g, B, T, c["Hkv"], D), _randn(g, B, T, c["Hkv"], D)
            depth = _closure(parents).sum(-1).to(torch.int32) - 1 if T <= 256 else torch.arange(T, device=DEV, dtype=torch.int32)
            s["positions"] = (s["ctx"][:, None] + depth).to(torch.int32).contiguous()
            s["wq"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(BF16) if c["norm"] else None
            s["wk"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(BF16) if c["norm"] else None
            if own:
                from gqa_decode_attention_fa_gb300 import binding
                s["rope"] = binding.Rope(**_rope_args(c))
        return s
    if op == "prepare":
        B, T = c["B"], c["T"]
        s["ctx"] = _randint(g, c["lo"], c["hi"], B)
        s["counts"] = _counts(g, B, T, c["ragged"])
        s["parents"] = _tree(g, B, T)
        s["mask"] = torch.zeros(B, T, (T + 63) // 64, dtype=torch.int64, device=DEV)
        s["positions"] = torch.zeros(B, T, dtype=torch.int32, device=DEV)
        return s
    if op == "fork":
        n, P, blocks = c["n"], c["pools"], c["blocks"]
        per = (c["hi"] + c["T"] + PAGE - 1) // PAGE + 1
        lens = _randint(g, c["lo"], c["hi"], n)
        have = (lens + PAGE - 1) // PAGE
        perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
        cols = torch.arange(per, device=DEV)
        used = cols < have[:, None]
        s["table"] = torch.full((2 * n, per), -1, device=DEV, dtype=torch.int32)
        at = (torch.cumsum(used.reshape(-1).int(), 0) - 1).view(n, per).clamp(min=0)
        s["table"][:n] = torch.where(used, perm[at], torch.full_like(perm[at], -1))
        s["refs"] = torch.zeros(blocks, device=DEV, dtype=torch.int32)
        s["refs"].index_add_(0, s["table"][:n][used].long(), torch.ones(int(used.sum()), device=DEV, dtype=torch.int32))
        s["lens"] = torch.cat([lens, torch.zeros_like(lens)])
        s["src"] = torch.arange(n, device=DEV, dtype=torch.int32)
        s["dst"] = torch.arange(n, 2 * n, device=DEV, dtype=torch.int32)
        s["grown"] = torch.cat([lens, lens + c["T"]]).to(torch.int32)
        s["freed"] = torch.cat([lens, torch.zeros_like(lens)]).to(torch.int32)
        s["cow_src"] = torch.full((2 * n,), -1, device=DEV, dtype=torch.int32)
        s["cow_dst"] = torch.full((2 * n,), -1, device=DEV, dtype=torch.int32)
        s["none"] = torch.full((2 * n,), -1, device=DEV, dtype=torch.int32)
        s["none2"] = torch.full((2 * n,), -1, device=DEV, dtype=torch.int32)
        s["cache"] = _pool_bytes(g, P, blocks * PAGE)
        s["blocks"] = blocks
    else:
        B, P, n = c["B"], c["pools"], c["n"]
        cap = c["start_hi"] + n + 3
        s["start"] = _randint(g, c["start_lo"], c["start_hi"], B)
        s["counts"] = torch.full((B,), c["keep"], device=DEV, dtype=torch.int32)
        order = torch.argsort(torch.rand(B, n, generator=g, device=DEV), dim=1)[:, : c["keep"]]
        s["keep"] = torch.full((B, n), -1, device=DEV, dtype=torch.int32)
        s["keep"][:, : c["keep"]] = torch.sort(order, dim=1).values.to(torch.int32)
        s["table"], s["blocks"] = _table(g, B, cap)
        s["cap"] = cap
        s["cache"] = _pool_bytes(g, P, s["blocks"] * PAGE)
    if own:
        from gqa_decode_attention_fa_gb300 import binding
        s["pools"] = binding.CachePools(list(s["cache"].unbind(0)), num_blocks=s["blocks"])
    return s


def _pool_bytes(g, P, rows):
    """P pools (K and V of the layers) of bf16 rows of 8 heads: [P, rows, 8, 128]."""
    bits = torch.randint(0, 0x3f80, (P, rows, 8, D), generator=g, device=DEV, dtype=torch.int16)
    return bits.view(BF16)


def _rope_args(c):
    a = dict(theta=1e6 if c["scaling"] == "none" else 5e5, rotary_dim=c["r"], layout=c["layout"])
    if c["scaling"] == "linear":
        a.update(scaling="linear", factor=4.0)
    elif c["scaling"] == "banded":
        a.update(scaling="banded", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original_max_len=8192)
    elif c["scaling"] == "yarn":
        a.update(scaling="yarn", factor=4.0, beta_fast=32.0, beta_slow=1.0, original_max_len=32768)
    return a


EPS = 1e-6


# ------------------------------------------------------------------------------- plain forms

def _rows(s, slots):
    """Cache rows of slots [B, n]."""
    b = torch.arange(slots.shape[0], device=slots.device)[:, None]
    slots = slots.long()
    if s["table"] is None:
        return b * s["cap"] + slots
    return s["table"].long()[b, slots // PAGE] * PAGE + slots % PAGE


def _plain_tree(s):
    c = s["case"]
    B, T, Hq, Hkv = c["B"], c["T"], c["Hq"], c["Hkv"]
    G = Hq // Hkv
    n = c["hi"] + T
    slot = torch.arange(n, device=DEV)
    rows = _rows(s, slot.expand(B, n))
    ctx, cnt = s["ctx"].long(), s["counts"].long()
    in_ctx = slot < ctx[:, None]
    u = slot - ctx[:, None]
    in_tree = (u >= 0) & (u < cnt[:, None])
    uc = u.clamp(0, T - 1)
    word = torch.gather(s["mask"], 2, (uc // 64)[:, None, :].expand(B, T, n))
    seen = in_ctx[:, None, :] | (in_tree[:, None, :] & (((word >> (uc % 64)[:, None, :]) & 1) > 0))   # [B, T, n]
    live = (in_ctx | in_tree)
    k = s["k_cache"][rows].float().permute(0, 2, 3, 1)                                               # [B, Hkv, D, n]
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    p = torch.matmul(q, k).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, T, n)
    del k
    p.masked_fill_(~seen[:, None, None], float("-inf"))
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    l = p.sum(-1, keepdim=True)
    v = torch.where(live[:, :, None, None], s["v_cache"][rows].float(), torch.zeros((), device=DEV)).permute(0, 2, 1, 3)
    o = torch.matmul(p.view(B, Hkv, G * T, n), v).view(B, Hkv, G, T, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(BF16)
    valid = torch.arange(T, device=DEV) < cnt[:, None]
    s["out"].copy_(torch.where(valid[:, :, None, None], o, s["out"]))
    return s["out"]


def _plain_prepare(s):
    c = s["case"]
    valid = torch.arange(c["T"], device=DEV) < s["counts"][:, None]
    seen = _closure(s["parents"])
    mask = _pack(seen)
    pos = s["ctx"][:, None] + seen.sum(-1).to(torch.int32) - 1
    s["mask"].copy_(torch.where(valid[:, :, None], mask, s["mask"]))
    s["positions"].copy_(torch.where(valid, pos.to(torch.int32), s["positions"]))
    return s["mask"], s["positions"]


def _frequencies(c):
    """The pairs' angular frequencies and the magnitude, in 64 bits."""
    a = _rope_args(c)
    r = a["rotary_dim"]
    f = a["theta"] ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
    mag = 1.0
    if c["scaling"] == "linear":
        f = f / a["factor"]
    elif c["scaling"] == "banded":
        turns = a["original_max_len"] * f / (2 * math.pi)     # periods of each pair in the trained length
        keep = ((turns - a["low_freq_factor"]) / (a["high_freq_factor"] - a["low_freq_factor"])).clamp(0, 1)
        f = keep * f + (1 - keep) * f / a["factor"]
    elif c["scaling"] == "yarn":
        at = [r * math.log(a["original_max_len"] / (b * 2 * math.pi)) / (2 * math.log(a["theta"])) for b in (a["beta_fast"], a["beta_slow"])]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        ramp = ((torch.arange(r // 2, device=DEV, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        f = ramp * f / a["factor"] + (1 - ramp) * f
        mag = 0.1 * math.log(a["factor"]) + 1.0
    return f, mag


def _rotate(x, w, c, cs, sn):
    """RMSNorm (w given) and rotation of x [B, T, H, D] in x's own precision."""
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(x.dtype)
    r = c["r"]
    rest = x[..., r:]
    if c["layout"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2:r]
        return torch.cat([a * cs - b * sn, b * cs + a * sn, rest], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cs - b * sn, b * cs + a * sn], -1).flatten(-2), rest], -1)


def _plain_rope(s):
    c = s["case"]
    T = c["T"]
    f, mag = _frequencies(c)
    angle = s["positions"].double()[..., None] * f
    cs, sn = (mag * angle.cos()).float()[:, :, None], (mag * angle.sin()).float()[:, :, None]
    q = _rotate(s["q"].float(), s["wq"], c, cs, sn).to(BF16)
    k = _rotate(s["k"].float(), s["wk"], c, cs, sn).to(BF16)
    t = torch.arange(T, device=DEV)
    valid = t < s["counts"][:, None]
    rows = _rows(s, s["ctx"][:, None] + t)[valid]
    s["k_cache"].index_copy_(0, rows, k[valid])
    s["v_cache"].index_copy_(0, rows, s["v"][valid])
    s["out"].copy_(torch.where(valid[:, :, None, None], q, s["out"]))
    return s["out"], s["k_cache"], s["v_cache"]


def _plain_resize(s, new, cow_src, cow_dst):
    refs, table, lens = s["refs"], s["table"], s["lens"]
    n, per = table.shape
    have, need = (lens + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    cols = torch.arange(per, device=DEV)
    one = torch.ones_like(table)
    gone = (cols >= need[:, None]) & (cols < have[:, None])
    refs.index_add_(0, table.clamp(min=0).view(-1).long(), torch.where(gone, -one, 0 * one).view(-1))
    table.masked_fill_(gone, -1)
    grows = (new > lens) & (lens % PAGE != 0)
    last = torch.gather(table, 1, (have - 1).clamp(min=0)[:, None].long())[:, 0]
    b = torch.arange(n, device=DEV)
    same = grows[:, None] & grows & (last[:, None] == last) & (b < b[:, None])
    cow = grows & (refs[last.clamp(min=0).long()] - same.sum(1) > 1)
    fresh = ((cols >= have[:, None]) & (cols < need[:, None])) | (cow[:, None] & (cols == (have - 1)[:, None]))
    order = torch.argsort((refs != 0).to(torch.int8), stable=True).to(torch.int32)      # free pages, lowest first
    page = order[(torch.cumsum(fresh.view(-1).int(), 0) - 1).clamp(0, order.numel() - 1)].view(n, per)
    refs.index_add_(0, last.clamp(min=0).long(), torch.where(cow, -torch.ones_like(last), torch.zeros_like(last)))
    refs.index_add_(0, page.view(-1).long(), fresh.view(-1).to(torch.int32))
    table.copy_(torch.where(fresh, page, table))
    at = torch.gather(table, 1, (have - 1).clamp(min=0)[:, None].long())[:, 0]
    cow_src.copy_(torch.where(cow, last, torch.full_like(last, -1)))
    cow_dst.copy_(torch.where(cow, at, torch.full_like(last, -1)))
    lens.copy_(new)


def _plain_fork(s):
    refs, table, lens = s["refs"], s["table"], s["lens"]
    src, dst = s["src"].long(), s["dst"].long()
    have = (lens[src] + PAGE - 1) // PAGE
    mine = torch.arange(table.shape[1], device=DEV) < have[:, None]
    pages = table[src]
    refs.index_add_(0, pages.clamp(min=0).view(-1).long(), mine.view(-1).to(torch.int32))
    table[dst] = torch.where(mine, pages, torch.full_like(pages, -1))
    lens[dst] = lens[src]
    _plain_resize(s, s["grown"], s["cow_src"], s["cow_dst"])
    paged = s["cache"].view(s["cache"].shape[0], s["blocks"], -1)
    ok = s["cow_src"] >= 0
    paged[:, s["cow_dst"][ok].long()] = paged[:, s["cow_src"][ok].long()]
    got = [x.clone() for x in (table, refs, lens, s["cow_src"], s["cow_dst"])]
    _plain_resize(s, s["freed"], s["none"], s["none2"])
    return got + [table, refs, s["cache"]]


def _plain_keep(s):
    n = s["keep"].shape[1]
    i = torch.arange(n, device=DEV)
    valid = i < s["counts"][:, None]
    to = _rows(s, s["start"][:, None] + i)[valid]
    frm = _rows(s, s["start"][:, None] + s["keep"].clamp(min=0))[valid]
    s["cache"][:, to] = s["cache"][:, frm]
    return s["cache"]


# --------------------------------------------------------------------------------- one pass

def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        return {"tree": _plain_tree, "prepare": _plain_prepare, "rope": _plain_rope, "fork": _plain_fork, "keep": _plain_keep}[op](s)
    from gqa_decode_attention_fa_gb300 import binding
    if op == "tree":
        binding.tree_attn(c["B"], c["Hq"], c["Hkv"], c["T"], s["cap"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"],
                          s["counts"], s["mask"], s["out"], block_size=PAGE if c["paged"] else 0, num_cache_blocks=s["blocks"],
                          workspace=s["workspace"])
        return s["out"]
    if op == "prepare":
        binding.tree_prepare(s["parents"], s["ctx"], s["counts"], s["mask"], s["positions"])
        return s["mask"], s["positions"]
    if op == "rope":
        binding.rope_append(c["B"], c["Hq"], c["Hkv"], c["T"], s["cap"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                            s["table"], s["ctx"], s["positions"], s["counts"], s["wq"], s["wk"], s["rope"], EPS, s["out"],
                            block_size=PAGE if c["paged"] else 0, num_cache_blocks=s["blocks"])
        return s["out"], s["k_cache"], s["v_cache"]
    if op == "fork":
        refs, table, lens = s["refs"], s["table"], s["lens"]
        binding.pages_fork(refs, table, lens, s["src"], s["dst"])
        binding.pages_resize(refs, table, lens, s["grown"], s["cow_src"], s["cow_dst"])
        binding.pages_copy(s["pools"], s["cow_src"], s["cow_dst"])
        got = [x.clone() for x in (table, refs, lens, s["cow_src"], s["cow_dst"])]
        binding.pages_resize(refs, table, lens, s["freed"], s["none"], s["none2"])
        return got + [table, refs, s["cache"]]
    binding.cache_keep_rows(s["pools"], s["table"], s["start"], s["keep"], s["counts"], max_seq_len=s["cap"])
    return s["cache"]


# ------------------------------------------------------------------------------------- work

def work(case):
    c = case
    op = c["op"]
    if op in ("tree", "prepare", "rope"):
        B, T = c["B"], c["T"]
        nodes = B * (T + 1) / 2 if c["ragged"] else B * T
        ctx = (c["lo"] + c["hi"]) / 2
    if op == "tree":
        keys = B * (ctx + nodes / B)
        return {"bytes": keys * c["Hkv"] * D * 4 + nodes * c["Hq"] * D * 4, "flops": 4 * D * c["Hq"] * (nodes / B) * keys}
    if op == "prepare":
        return {"bytes": nodes * (4 + 4 + 8 * ((T + 63) // 64)), "flops": 0}
    if op == "rope":
        return {"bytes": nodes * (c["Hq"] + 2 * c["Hkv"]) * D * 4, "flops": nodes * (c["Hq"] + c["Hkv"]) * D * 4}
    if op == "fork":
        # nearly every fork's last page is partial and shared: one page copied in each pool
        return {"bytes": c["n"] * c["pools"] * PAGE * 8 * D * 4 + c["blocks"] * 8, "flops": 0}
    return {"bytes": max(1, c["B"] * c["keep"] * c["pools"] * 8 * D * 4), "flops": 0}


# ------------------------------------------------------------------------------------ exact

def exact(case, seed):
    """The operator's definition in 64 bits, sequence by sequence."""
    c = case
    if c["op"] not in ("tree", "rope"):
        return None  # whole numbers and moved bytes
    s = prepare(c, seed)
    B, T, Hq, Hkv = c["B"], c["T"], c["Hq"], c["Hkv"]
    out = s["out"].double()
    if c["op"] == "tree":
        for b in range(B):
            n0, n = int(s["ctx"][b]), int(s["counts"][b])
            slots = torch.arange(n0 + n, device=DEV)
            if s["table"] is None:
                rows = b * s["cap"] + slots
            else:
                rows = s["table"][b].long()[slots // PAGE] * PAGE + slots % PAGE
            seen = torch.ones(n, n0 + n, dtype=torch.bool, device=DEV)
            for u in range(n):
                seen[:, n0 + u] = ((s["mask"][b, :n, u // 64] >> (u % 64)) & 1) == 1
            for kv in range(Hkv):
                k, v = s["k_cache"][rows, kv].double(), s["v_cache"][rows, kv].double()
                for h in range(kv * Hq // Hkv, (kv + 1) * Hq // Hkv):
                    x = (s["q"][b, :n, h].double() @ k.T) / D ** 0.5
                    x[~seen] = -float("inf")
                    out[b, :n, h] = torch.nan_to_num(torch.softmax(x, -1), nan=0.0) @ v
        return out
    a = _rope_args(c)
    r = a["rotary_dim"]
    freq, mag = [], 1.0
    for i in range(r // 2):
        w = a["theta"] ** (-2.0 * i / r)
        if c["scaling"] == "linear":
            w /= a["factor"]
        elif c["scaling"] == "banded":
            wavelength = 2 * math.pi / w
            long, short = a["original_max_len"] / a["low_freq_factor"], a["original_max_len"] / a["high_freq_factor"]
            if wavelength > long:
                w /= a["factor"]
            elif wavelength > short:
                mix = (a["original_max_len"] / wavelength - a["low_freq_factor"]) / (a["high_freq_factor"] - a["low_freq_factor"])
                w = (1 - mix) * w / a["factor"] + mix * w
        elif c["scaling"] == "yarn":
            mag = 1.0 + 0.1 * math.log(a["factor"])
            dim = lambda beta: r * math.log(a["original_max_len"] / (beta * 2 * math.pi)) / (2 * math.log(a["theta"]))  # noqa: E731
            first, last = max(0, math.floor(dim(a["beta_fast"]))), min(r - 1, math.ceil(dim(a["beta_slow"])))
            far = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            w = w * (1 - far) + w / a["factor"] * far
        freq.append(w)
    angle = s["positions"].double()[:, :, None, None] * torch.tensor(freq, dtype=torch.float64, device=DEV)
    turn = mag * torch.polar(torch.ones_like(angle), angle)

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * w.double()
        y = x.clone()
        i = torch.arange(r // 2, device=DEV)
        first, second = (i, i + r // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    q, k = turned(s["q"], s["wq"]), turned(s["k"], s["wk"])
    for b in range(B):
        n = int(s["counts"][b])
        slots = int(s["ctx"][b]) + torch.arange(n, device=DEV)
        rows = b * s["cap"] + slots if s["table"] is None else s["table"][b].long()[slots // PAGE] * PAGE + slots % PAGE
        out[b, :n], kc[rows], vc[rows] = q[b, :n], k[b, :n], s["v"][b, :n].double()
    return out, kc, vc
