"""Cases for the operators of serving over an 8-bit KV cache: rows quantised as they are written and read
back, attention of one new token over the quantised cache, and causal attention over prompts of
different lengths packed one behind the other.

`run` with `own` false computes each operator from its definition in elementary torch operations;
with `own` true it calls the package.  Rows are bf16, head_dim 128, pages of 64 tokens; codes are e4m3 or
int8 with one fp32 scale a (token, KV head) row."""
import math
import random

import torch

own = False

D = 128
PAGE = 64
DEV = "cuda"
BF16 = torch.bfloat16
LARGEST = {"e4m3": 448.0, "int8": 127.0}


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's new rows of 32 sequences: latency
        dict(name="append_decode_32", op="append", B=32, Hkv=8, lo=1, hi=1, at=500, fmt="e4m3", paged=True),
        # 16 prompts of up to 2000 tokens stored, one layer
        dict(name="append_prompts_16", op="append", B=16, Hkv=8, lo=64, hi=2000, at=0, fmt="e4m3", paged=True),
        # chunks of three long prompts behind their prefixes, 4 KV heads, int8, contiguous
        dict(name="append_chunks_int8", op="append", B=3, Hkv=4, lo=700, hi=1100, at=3001, fmt="int8", paged=False),
        # the prefixes of 8 prompts read back for their next chunk
        dict(name="read_prefixes_8", op="read", B=8, Hkv=8, lo=1000, hi=6000, at=0, fmt="e4m3", paged=True),
        # a few rows in the middle of two caches
        dict(name="read_rows_int8", op="read", B=2, Hkv=5, lo=30, hi=90, at=77, fmt="int8", paged=True),
        # the latency end: one sequence of 256 tokens
        dict(name="token_256", op="token", B=1, Hq=40, Hkv=8, lo=256, hi=256, fmt="e4m3", paged=False),
        # a serving batch: 32 ragged contexts
        dict(name="token_ragged_32", op="token", B=32, Hq=40, Hkv=8, lo=512, hi=8192, fmt="e4m3", paged=True),
        # one layer of a step of 8 sequences of 32k
        dict(name="token_8x32k", op="token", B=8, Hq=40, Hkv=8, lo=32768, hi=32768, fmt="e4m3", paged=True),
        # one 128k context, 64/8 heads, int8
        dict(name="token_128k_int8", op="token", B=1, Hq=64, Hkv=8, lo=131072, hi=131072, fmt="int8", paged=False),
        # one short prompt: latency
        dict(name="prompt_150", op="prompt", B=1, Hq=40, Hkv=8, lo=150, hi=150, pre_lo=0, pre_hi=0),
        # a serving batch's prompts, packed
        dict(name="prompts_ragged_16", op="prompt", B=16, Hq=40, Hkv=8, lo=64, hi=2000, pre_lo=0, pre_hi=0),
        # two chunks of 6000 tokens with 64/8 heads, each over a prefix: bound by the tensor core
        dict(name="prompts_prefix_2x6000", op="prompt", B=2, Hq=64, Hkv=8, lo=6000, hi=6000, pre_lo=1500, pre_hi=2000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "token", "token", "prompt", "prompt"])
    fmt = rng.choice(["e4m3", "int8"])
    paged = rng.random() < 0.6
    if op in ("append", "read"):
        Hkv = rng.choice([1, 2, 4, 5, 8, 16])
        rows = (16000 if op == "append" else 28000) * 8 // Hkv       # at most as many as the largest listed case's
        B = _log(rng, 1, 200)
        hi = _log(rng, 4, max(4, min(30000, rows // B)))
        return dict(op=op, B=B, Hkv=Hkv, lo=rng.randint(0 if B > 3 else 1, hi), hi=hi, at=rng.choice([0, 1, 63, 500, 1999]), fmt=fmt, paged=paged)
    if op == "token":
        Hq, Hkv = rng.choice([(40, 8), (64, 8), (32, 8), (8, 8), (16, 1), (20, 4), (32, 32), (6, 3)])
        B = _log(rng, 1, 200)
        hi = _log(rng, 4, max(4, min(131072, 260000 * 8 // (max(8, Hkv) * B))))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, lo=rng.randint(0 if B > 3 else 1, hi), hi=hi, fmt=fmt, paged=paged)
    Hq, Hkv = rng.choice([(40, 8), (64, 8), (32, 8), (8, 8), (16, 1), (20, 4), (6, 3)])
    B = _log(rng, 1, 64)
    pairs = 2 * 6000 * 6000 // 2 * 64 // Hq                          # query-key pairs a head, as the largest listed case
    hi = _log(rng, 4, max(4, min(9000, int(math.sqrt(2 * pairs / B)))))
    pre = rng.choice([0, 0, _log(rng, 1, max(1, min(9000, pairs // (2 * B * hi))))])
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, lo=rng.randint(0 if B > 3 else 1, hi), hi=hi, pre_lo=rng.randint(0, pre), pre_hi=pre)


# --------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(BF16)


def _i32(values):
    return torch.tensor(list(values), dtype=torch.int32, device=DEV)


def _lengths(seed, n, lo, hi):
    """n lengths in [lo, hi]: a batch of these sizes has the same ones for every seed, in another order."""
    r = random.Random(1000003 * n + 1009 * lo + hi)
    lengths = [r.randint(lo, hi) for _ in range(n)]
    random.Random(seed).shuffle(lengths)
    return lengths


def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _keys(g, *shape):
    """Rows as a model's keys have them: a few channels of every head are large."""
    x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)
    return x.mul_(torch.where(torch.arange(D, device=DEV) % 41 == 7, 6.0, 1.0)).to(BF16)


def _code_type(fmt):
    return torch.float8_e4m3fn if fmt == "e4m3" else torch.int8


def _codes(g, fmt, rows, Hkv, spread):
    """Codes of normally distributed rows whose standard deviation is `spread` of the largest level."""
    x = torch.empty(rows, Hkv, D, dtype=_code_type(fmt), device=DEV)
    for part in x.split(max(1, (1 << 26) // (Hkv * D))):
        y = torch.randn(part.shape, generator=g, device=DEV).mul_(LARGEST[fmt] * spread).clamp_(-LARGEST[fmt], LARGEST[fmt])
        part.copy_(y.round_() if fmt == "int8" else y)
    return x


def _table(seed, g, B, capacity):
    per = (capacity + PAGE - 1) // PAGE
    blocks = B * per + 3
    return torch.randperm(blocks, generator=g, device=DEV)[: B * per].view(B, per).to(torch.int32), blocks


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    B, op = c["B"], c["op"]
    s = {"case": c}
    lengths = _lengths(seed, B, c["lo"], c["hi"])
    s["longest"] = max(1, max(lengths))
    if op == "prompt":
        prefix = _lengths(seed + 1, B, c["pre_lo"], c["pre_hi"])
        q_at, k_at = _offsets(lengths), _offsets(a + b for a, b in zip(lengths, prefix))
        s["longest_k"] = max(1, max(a + b for a, b in zip(lengths, prefix)))
        # q, k and v of prompts without a prefix are slices of one projection; with one, keys and values are tensors of their own
        n, m = max(1, q_at[-1]), max(1, k_at[-1])
        if c["pre_hi"] == 0:
            x = _randn(g, n, c["Hq"] + 2 * c["Hkv"], D)
            s["q"], s["k"], s["v"] = x.split([c["Hq"], c["Hkv"], c["Hkv"]], 1)
        else:
            s["q"], s["k"], s["v"] = _randn(g, n, c["Hq"], D), _randn(g, m, c["Hkv"], D), _randn(g, m, c["Hkv"], D)
        s["q_offsets"], s["k_offsets"] = _i32(q_at), _i32(k_at)
        s["out"] = torch.zeros(n, c["Hq"], D, dtype=BF16, device=DEV)
        return s
    s["cap"] = cap = c["hi"] + c.get("at", 0) + 5
    if c["paged"]:
        s["table"], s["blocks"] = _table(seed, g, B, cap)
        rows = s["blocks"] * PAGE
    else:
        s["table"], s["blocks"], rows = None, 0, B * cap
    # what an append leaves as it was is kept small, so that it does not hide the size of an error in what it writes
    small = 0.004 if op == "append" else 0.37
    s["k_codes"], s["v_codes"] = (_codes(g, c["fmt"], rows, c["Hkv"], small) for _ in range(2))
    s["k_scale"], s["v_scale"] = ((0.8 + 0.4 * torch.rand(rows, c["Hkv"], generator=g, device=DEV)) * (2.7 / LARGEST[c["fmt"]])
                                  for _ in range(2))
    if op == "token":
        s["lens"] = _i32(lengths)
        s["q"] = _randn(g, B, c["Hq"], D)
        s["out"] = torch.zeros(B, c["Hq"], D, dtype=BF16, device=DEV)
        if own:
            from gqa_decode_attention_fa_gb300 import binding
            s["workspace"] = binding.q8_workspace(B, c["Hq"], c["Hkv"], cap, block_size=PAGE if c["paged"] else 0,
                                                  num_cache_blocks=s["blocks"])
        return s
    at = _offsets(lengths)
    n = at[-1] + 7  # a few rows behind the last sequence, as where a batch is padded
    s["offsets"] = _i32(at)
    s["start"] = _i32(_lengths(seed + 1, B, 0, c["at"]))
    s["rows"] = n
    if op == "append":
        s["k"], s["v"] = _keys(g, n, c["Hkv"], D), _randn(g, n, c["Hkv"], D)
    else:
        s["k_out"], s["v_out"] = (1e-3 * _randn(g, n, c["Hkv"], D) for _ in range(2))
    return s


# ------------------------------------------------------------------------------- plain forms

def _slots(s, seq, slot):
    """Cache rows of slots of sequences."""
    if s["table"] is None:
        return seq * s["cap"] + slot
    return s["table"].long()[seq, slot // PAGE] * PAGE + slot % PAGE


def _packed_rows(s):
    """The packed rows that belong to a sequence and the cache rows they go to."""
    at = s["offsets"].long()
    row = torch.arange(s["rows"], device=DEV)
    row = row[row < at[-1]]
    seq = torch.searchsorted(at, row, right=True) - 1
    return row, _slots(s, seq, s["start"].long()[seq] + row - at[seq])


def _quantise(x, fmt):
    """Codes and scales of rows: in 64 bits, since values next to the border of two codes go by the exact quotient."""
    most = x.float().abs().amax(-1)
    scale = most / torch.full_like(most, LARGEST[fmt])  # (a division by a number may be done as a product)
    q = x.double() / scale.double()[..., None]
    q = torch.where(scale[..., None] > 0, q, torch.zeros_like(q))
    if fmt == "int8":
        return q.round().clamp(-127, 127).to(torch.int8), scale
    step = torch.ldexp(torch.ones_like(q), torch.clamp(torch.frexp(q).exponent - 1, min=-6) - 3)
    return ((q / step).round() * step).clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _plain_append(s):
    row, to = _packed_rows(s)
    for x, codes, scales in ((s["k"], s["k_codes"], s["k_scale"]), (s["v"], s["v_codes"], s["v_scale"])):
        c, f = _quantise(x[row], s["case"]["fmt"])
        codes.view(torch.uint8)[to] = c.view(torch.uint8)
        scales[to] = f
    return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]


def _plain_read(s):
    row, frm = _packed_rows(s)
    for codes, scales, out in ((s["k_codes"], s["k_scale"], s["k_out"]), (s["v_codes"], s["v_scale"], s["v_out"])):
        c = codes.view(torch.uint8)[frm].view(codes.dtype)
        out[row] = (c.float() * scales[frm][..., None]).to(BF16)
    return s["k_out"], s["v_out"]


def _softmax_(p):
    """Softmax over the last axis in place; rows without a finite score become zeros."""
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _plain_token(s):
    c = s["case"]
    B, Hq, Hkv, n = c["B"], c["Hq"], c["Hkv"], s["longest"]
    slot = torch.arange(n, device=DEV)
    live = slot < s["lens"][:, None]
    rows = _slots(s, torch.arange(B, device=DEV)[:, None], slot.expand(B, n))

    def values(codes, scales):
        x = codes.view(torch.uint8)[rows].view(codes.dtype).float() * scales[rows][..., None]
        return torch.where(live[..., None, None], x, torch.zeros((), device=DEV)).permute(0, 2, 1, 3)  # [B, Hkv, n, D]

    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    p = torch.matmul(q, values(s["k_codes"], s["k_scale"]).transpose(-1, -2)).mul_(1 / math.sqrt(D))
    p = _softmax_(p.masked_fill_(~live[:, None, None], float("-inf")))
    s["out"].copy_(torch.matmul(p, values(s["v_codes"], s["v_scale"])).reshape(B, Hq, D))
    return s["out"]


def _plain_prompt(s):
    c = s["case"]
    B, Hq, Hkv, n, m = c["B"], c["Hq"], c["Hkv"], s["longest"], s["longest_k"]
    q_at, k_at = s["q_offsets"].long(), s["k_offsets"].long()
    nq, nk = q_at[1:] - q_at[:-1], k_at[1:] - k_at[:-1]
    i, j = torch.arange(n, device=DEV), torch.arange(m, device=DEV)
    live_q, live_k = i < nq[:, None], j < nk[:, None]
    qi = torch.where(live_q, q_at[:-1, None] + i, torch.zeros_like(i))
    kj = torch.where(live_k, k_at[:-1, None] + j, torch.zeros_like(j))
    q = s["q"][qi].float().view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    k, v = (torch.where(live_k[..., None, None], x[kj].float(), torch.zeros((), device=DEV)).permute(0, 2, 1, 3)
            for x in (s["k"], s["v"]))
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(D)).view(B, Hkv, Hq // Hkv, n, m)
    seen = live_k[:, None, :] & (j <= i[:, None] + (nk - nq)[:, None, None])
    p = _softmax_(p.masked_fill_(~seen[:, None, None], float("-inf"))).view(B, Hkv, -1, m)
    o = torch.matmul(p, v).view(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    s["out"][qi[live_q]] = o[live_q].to(BF16)
    return s["out"]


# --------------------------------------------------------------------------------- one pass

def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "token": _plain_token, "prompt": _plain_prompt}[op](s)
    from gqa_decode_attention_fa_gb300 import binding
    if op == "prompt":
        binding.packed_attn(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], s["out"])
        return s["out"]
    cache = dict(fmt=c["fmt"], block_size=PAGE if c["paged"] else 0, num_cache_blocks=s["blocks"])
    if op == "append":
        binding.q8_append(c["B"], c["Hkv"], s["rows"], s["cap"], s["k"], s["v"], s["k_codes"], s["v_codes"], s["k_scale"],
                          s["v_scale"], s["table"], s["offsets"], s["start"], **cache)
        return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]
    if op == "read":
        binding.q8_read(c["B"], c["Hkv"], s["rows"], s["cap"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
                        s["table"], s["offsets"], s["start"], s["k_out"], s["v_out"], **cache)
        return s["k_out"], s["v_out"]
    binding.q8_attn(c["B"], c["Hq"], c["Hkv"], s["cap"], s["q"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
                    s["table"], s["lens"], s["out"], workspace=s["workspace"], **cache)
    return s["out"]


# ------------------------------------------------------------------------------------- work

def work(case):
    c = case
    lengths = _lengths(0, c["B"], c["lo"], c["hi"])
    mean, square = sum(lengths) / c["B"], sum(n * n for n in lengths) / c["B"]
    if c["op"] in ("append", "read"):
        values = c["B"] * mean * c["Hkv"] * D * 2
        return {"bytes": max(1, values * 3 + values / D * 4), "flops": values}
    if c["op"] == "token":
        tokens = c["B"] * mean
        return {"bytes": tokens * c["Hkv"] * (2 * D + 8) + c["B"] * c["Hq"] * D * 4, "flops": 4 * D * c["Hq"] * tokens}
    prefix = (c["pre_lo"] + c["pre_hi"]) / 2
    pairs = c["B"] * ((square + mean) / 2 + mean * prefix)
    return {"bytes": max(1, c["B"] * 4 * D * (mean * c["Hq"] + (mean + prefix) * c["Hkv"])), "flops": 4 * D * c["Hq"] * pairs}


# ------------------------------------------------------------------------------------ exact

def _levels(fmt):
    """The format's levels, ascending, and whether each one's code is even."""
    if fmt == "int8":
        v = torch.arange(-127, 128, dtype=torch.float64, device=DEV)
        return v, v.long() % 2 == 0
    mag = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    mag = mag[:127]  # the last code is no number
    v = torch.tensor([-x for x in mag[:0:-1]] + mag, dtype=torch.float64, device=DEV)
    return v, torch.arange(-126, 127, device=DEV) % 2 == 0


def _nearest(x, fmt):
    level, even = _levels(fmt)
    hi = torch.searchsorted(level, x.contiguous()).clamp(1, level.numel() - 1)
    below, above = x - level[hi - 1], level[hi] - x
    up = (above < below) | ((above == below) & even[hi])
    return level[torch.where(up, hi, hi - 1)]


def exact(case, seed):
    """The operator's definition in 64 bits, sequence by sequence."""
    c = case
    s = prepare(c, seed)
    B, Hkv, op = c["B"], c["Hkv"], c["op"]
    if op == "prompt":
        G = c["Hq"] // Hkv
        out = s["out"].double()
        q_at, k_at = s["q_offsets"].tolist(), s["k_offsets"].tolist()
        for b in range(B):
            n, m = q_at[b + 1] - q_at[b], k_at[b + 1] - k_at[b]
            if n == 0 or m == 0:
                continue
            ahead = torch.ones(n, m, dtype=torch.bool, device=DEV).triu(m - n + 1)
            for h in range(c["Hq"]):
                k, v = (s[x][k_at[b]:k_at[b + 1], h // G].double() for x in "kv")
                x = (s["q"][q_at[b]:q_at[b + 1], h].double() @ k.T) / D ** 0.5
                out[q_at[b]:q_at[b + 1], h] = torch.softmax(x.masked_fill_(ahead, -float("inf")), -1) @ v
        return out

    def rows_of(b, first, n):
        slot = torch.arange(first, first + n, device=DEV)
        return b * s["cap"] + slot if s["table"] is None else s["table"][b].long()[slot // PAGE] * PAGE + slot % PAGE

    def values(codes, rows):
        return codes.view(torch.uint8)[rows].view(codes.dtype).double()

    if op == "token":
        G = c["Hq"] // Hkv
        out = s["out"].double()
        for b, n in enumerate(s["lens"].tolist()):
            if n == 0:
                continue
            rows = rows_of(b, 0, n)
            for kv in range(Hkv):
                k = values(s["k_codes"][:, kv], rows) * s["k_scale"][rows, kv, None].double()
                v = values(s["v_codes"][:, kv], rows) * s["v_scale"][rows, kv, None].double()
                x = (s["q"][b, kv * G:(kv + 1) * G].double() @ k.T) / D ** 0.5
                out[b, kv * G:(kv + 1) * G] = torch.softmax(x, -1) @ v
        return out
    at, start = s["offsets"].tolist(), s["start"].tolist()
    if op == "read":
        outs = []
        for x in "kv":
            out = s[x + "_out"].double()
            for b in range(B):
                rows = rows_of(b, start[b], at[b + 1] - at[b])
                out[at[b]:at[b + 1]] = values(s[x + "_codes"], rows) * s[x + "_scale"][rows, :, None].double()
            outs.append(out)
        return tuple(outs)
    codes, scales = [], []
    for x in "kv":
        code, scale = s[x + "_codes"].double(), s[x + "_scale"].double()
        for b in range(B):
            rows = rows_of(b, start[b], at[b + 1] - at[b])
            y = s[x][at[b]:at[b + 1]].double()
            most = y.abs().max(-1).values if y.shape[0] else y.new_zeros(0, Hkv)
            scale[rows] = most / LARGEST[c["fmt"]]
            kept = scale[rows].float().double()[..., None]  # the codes go by the scale that is kept
            code[rows] = _nearest(torch.where(kept > 0, y / kept, 0 * y), c["fmt"])
        codes.append(code if c["fmt"] == "e4m3" else None)
        scales.append(scale)
    return (*codes, *scales)
