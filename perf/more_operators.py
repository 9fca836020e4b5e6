"""The latent cache in 4 bits, as cases for measuring: its writer (RMS norm and
quantising), its reader, and the absorbed latent attention over it, with several
new tokens a sequence and with a prefix that a batch shares.

``run`` computes each in its plain form with elementary torch operations in 32
bits (64 where a value lies next to a border of the 4-bit values), or, with
``own`` set, by the library's entry points.  ``exact`` is the definition in 64
bits.

A cached row is 400 bytes: 512 latent values as e2m1 codes (the value of an even
channel in the low half of its byte), one scale byte s of 2^(s - 127) for each 32
of them (255: they are NaN), and the 64 shared key channels in bf16.
"""
import random

import torch

own = False

D_LATENT, D_PE = 512, 64
D_ROW = D_LATENT + D_PE
GROUP = 32                                   # latent values with one scale
GROUPS = D_LATENT // GROUP
CODES, ROW_BYTES = D_LATENT // 2, D_LATENT // 2 + GROUPS + 2 * D_PE
SCALE = 192 ** -0.5
EPS = 1e-5
LEAST, MOST = -120, 125                      # a scale's exponent


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user's next token: latency
        {"name": "decode 1x777", "op": "decode", "batch": 1, "new": 1, "heads": 32, "shortest": 777,
         "longest": 777, "prefix": 0, "page": 64, "lse": False, "split": 0},
        # one user's next token behind a book
        {"name": "decode 1x131072", "op": "decode", "batch": 1, "new": 1, "heads": 32, "shortest": 131072,
         "longest": 131072, "prefix": 0, "page": 64, "lse": False, "split": 1},
        # a current token and two drafts for a batch of 32
        {"name": "decode 32x3", "op": "decode", "batch": 32, "new": 3, "heads": 32, "shortest": 512,
         "longest": 8192, "prefix": 0, "page": 64, "lse": True, "split": 2},
        # a full batch's next tokens
        {"name": "decode 256x1", "op": "decode", "batch": 256, "new": 1, "heads": 32, "shortest": 512,
         "longest": 8192, "prefix": 0, "page": 64, "lse": False, "split": 3},
        # a model of 40 heads, odd lengths, small pages
        {"name": "decode 61x1 40 heads", "op": "decode", "batch": 61, "new": 1, "heads": 40, "shortest": 1,
         "longest": 5001, "prefix": 0, "page": 16, "lse": True, "split": 4},
        # eight samples of one question: a common prompt, answers just begun
        {"name": "shared 8x1 4097", "op": "decode", "batch": 8, "new": 1, "heads": 32, "shortest": 1,
         "longest": 100, "prefix": 4097, "page": 64, "lse": False, "split": 5},
        # a long system prompt before every request of a batch, with two drafts each
        {"name": "shared 128x3 16384", "op": "decode", "batch": 128, "new": 3, "heads": 32,
         "shortest": 16, "longest": 512, "prefix": 16384, "page": 64, "lse": False, "split": 6},
        # the new rows of a decoding batch, written and looked at again
        {"name": "store 256x3", "op": "store", "seqs": 256, "tokens": 768, "ragged": False,
         "cached": 1024, "page": 64, "norm": True, "split": 7},
        # the rows of a batch of prompts
        {"name": "store 8 of 32768", "op": "store", "seqs": 8, "tokens": 32768, "ragged": True,
         "cached": 0, "page": 64, "norm": True, "split": 8},
        # what one prompt in pieces has cached so far
        {"name": "read 1x1025", "op": "read", "seqs": 1, "tokens": 1025, "ragged": False,
         "cached": 0, "page": 64, "split": 9},
        # a batch of prompts in pieces: the rows before their next piece
        {"name": "read 5 of 65537", "op": "read", "seqs": 5, "tokens": 65537, "ragged": True,
         "cached": 0, "page": 128, "split": 10},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["decode", "long", "shared", "store", "read"])
    split, page = rng.randrange(1 << 20), rng.choice([16, 32, 64, 128, 256])
    if op in ("decode", "long", "shared"):
        batch, new, heads = _log(rng, 1, 256), rng.choice([1, 1, 2, 3, 5, 8]), rng.choice([8, 16, 32, 40])
        longest = _log(rng, 1, {"decode": 8192, "long": 131072, "shared": 600}[op])
        prefix = _log(rng, 1, 16384) if op == "shared" else 0
        while batch > 1 and (batch * new * heads * (longest + prefix) > 1 << 27 or batch * longest > 1 << 20):
            batch = batch * 3 // 4
        return {"op": "decode", "batch": batch, "new": new, "heads": heads, "shortest": rng.randint(0, longest),
                "longest": longest, "prefix": prefix, "page": page, "lse": rng.random() < 0.5, "split": split}
    seqs = _log(rng, 1, 256)
    few = rng.random() < 0.4
    tokens = seqs * rng.randint(1, 4) if few else _log(rng, seqs, 30000)
    case = {"op": op, "seqs": seqs, "tokens": tokens, "ragged": not few,
            "cached": rng.choice([0, _log(rng, 1, 1024)]), "page": page, "split": split}
    if op == "store":
        case["norm"] = rng.random() < 0.8
    return case


def _parts(total, n, rng):
    """n whole numbers that sum to total, drawn at random."""
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _decode_lengths(c):
    rng = random.Random(c["split"])
    return [rng.randint(c["shortest"], c["longest"]) for _ in range(c["batch"])]


def _row_lengths(c):
    """(rows of the call, cached rows after them) of each sequence."""
    rng = random.Random(c["split"])
    n = c["seqs"]
    new = _parts(c["tokens"], n, rng) if c["ragged"] else [c["tokens"] // n] * n
    return new, [a + rng.randint(0, c["cached"]) for a in new]


def work(case):
    c = case
    if c["op"] == "decode":
        lens, t = _decode_lengths(c), c["new"]
        rows = c["batch"] * t * c["heads"]
        seen = sum(c["prefix"] + max(0, n - i) for n in lens for i in range(t))
        return {"bytes": (sum(lens) + c["prefix"]) * ROW_BYTES + 2 * rows * (D_ROW + D_LATENT),
                "flops": 2 * c["heads"] * seen * (D_ROW + D_LATENT)}
    moved = c["tokens"] * (ROW_BYTES + 2 * D_ROW)
    if c["op"] == "read":
        return {"bytes": moved, "flops": c["tokens"] * D_LATENT}
    return {"bytes": 2 * moved, "flops": 7 * c["tokens"] * D_LATENT}


# ---------------------------------------------------------------------------
# the format
# ---------------------------------------------------------------------------
def _encode(latent, pe):
    """Rows of the cache from latent values [n, 512] (64 bits) and pe [n, 64] bf16."""
    n = latent.shape[0]
    y = latent.reshape(n, GROUPS, GROUP)
    most = y.abs().amax(-1, keepdim=True)
    part, e = torch.frexp(most)                       # most = part 2^e, part in [1/2, 1)
    e = (e - 3 + (part > 0.875).to(e.dtype)).clamp(LEAST, MOST)
    e = torch.where(most > 0, e, torch.full_like(e, LEAST))
    t = torch.ldexp(y.abs(), -e)
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0)).to(t.dtype)
    t = (torch.round(t / step) * step).clamp(max=6)   # (round takes ties to even)
    code = torch.where(t < 2, 2 * t, torch.where(t < 4, t + 2, t / 2 + 4)).to(torch.uint8)
    code = (code | ((y < 0) & (t > 0)).to(torch.uint8) * 8).reshape(n, CODES, 2)
    good = torch.isfinite(most[..., 0])
    scale = torch.where(good, e[..., 0] + 127, 255).to(torch.uint8)
    return torch.cat([code[..., 0] | code[..., 1] << 4, scale, pe.contiguous().view(torch.uint8)], 1)


def _decode_rows(rows):
    """The 576 values of cached rows [..., 400], in 32 bits."""
    codes, scale = rows[..., :CODES], rows[..., CODES:CODES + GROUPS]
    pe = rows[..., CODES + GROUPS:].contiguous().view(torch.bfloat16).float()
    both = torch.stack([codes & 15, codes >> 4], -1).reshape(*rows.shape[:-1], GROUPS, GROUP)
    size = (both & 7).float()
    size = torch.where(size < 4, size / 2, torch.where(size < 6, size - 2, 2 * size - 8))
    size = torch.where(both > 7, -size, size)
    factor = torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.int() - 127)
    factor = torch.where(scale == 255, float("nan"), factor)
    return torch.cat([(size * factor[..., None]).flatten(-2), pe], -1)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=_device())


def _pages(lens, page, width, gen, spare):
    """A block table over shuffled pages (-1 behind a sequence's last) and the number of pages in the pool."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=gen, device=_device()).to(torch.int32)
    col = torch.arange(width, device=_device())[None, :]
    need_t = torch.tensor(need, device=_device())[:, None]
    first = torch.cumsum(need_t[:, 0], 0)[:, None] - need_t
    table = torch.where(col < need_t, order[(first + col).clamp(max=pool - 1)], -1)
    return table.to(torch.int32).contiguous(), order, pool


def _filled(pool, page, gen):
    """A cache of rows as a model leaves them: normalised latents, some channels larger than others."""
    dev = _device()
    out = torch.empty(pool * page, ROW_BYTES, dtype=torch.uint8, device=dev)
    size = torch.exp(0.3 * torch.randn(D_LATENT, generator=gen, device=dev))
    for at in range(0, pool * page, 1 << 16):
        x = torch.randn(min(1 << 16, pool * page - at), D_ROW, generator=gen, device=dev)
        out[at:at + x.shape[0]] = _encode(x[:, :D_LATENT] * size, x[:, D_LATENT:].bfloat16())
    return out.reshape(pool, page, ROW_BYTES)


def prepare(case, seed):
    c, dev = case, _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    page = c["page"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if c["op"] == "decode":
        lens = _decode_lengths(c)
        npre = -(-c["prefix"] // page)
        table, order, pool = _pages(lens, page, max(1, -(-c["longest"] // page)), gen, npre + 3)
        return {"c": c, "q": normal(c["batch"], c["new"], c["heads"], D_ROW).bfloat16(),
                "cache": _filled(pool, page, gen), "table": table, "lens": _ints(lens),
                "prefix": order[pool - npre:].contiguous() if npre else None}
    new, after = _row_lengths(c)
    table, _, pool = _pages(after, page, max(1, -(-max(after) // page)), gen, 3)
    s = {"c": c, "cache": _filled(pool, page, gen), "table": table, "lens": _ints(after),
         "cu": _ints(_offsets(new)) if c["ragged"] else None}
    if c["op"] == "store":
        s["kv"] = (3 * normal(c["tokens"], D_ROW)).bfloat16()
        s["weight"] = 1 + 0.1 * normal(D_LATENT) if c["norm"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _softmax_parts(scores):
    """exp(scores - max), its sum and the log of the sum of exp(scores), rows with nothing to see included."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total > 0, total, torch.ones_like(total)), (top + torch.log(total))[..., 0]


def _plain_decode(s):
    c, cache = s["c"], s["cache"]
    b, t, h = c["batch"], c["new"], c["heads"]
    q = s["q"].float().reshape(b, t * h, D_ROW) * SCALE
    kv = _decode_rows(cache[s["table"].clamp(min=0).long()].reshape(b, -1, ROW_BYTES))
    last = s["lens"].long()[:, None] - (t - 1 - torch.arange(t, device=q.device))[None, :]
    seen = torch.arange(kv.shape[1], device=q.device)[None, None, :] < last[:, :, None]
    scores = torch.matmul(q, kv.transpose(1, 2))
    scores = scores.reshape(b, t, h, -1).masked_fill_(~seen[:, :, None, :], float("-inf")).reshape(b, t * h, -1)
    n = c["prefix"]
    if n:
        pre = _decode_rows(cache[s["prefix"].long()].reshape(-1, ROW_BYTES)[:n])
        scores = torch.cat([torch.matmul(q, pre.t()), scores], -1)
    p, total, lse = _softmax_parts(scores)
    o = torch.matmul(p[..., n:], kv[..., :D_LATENT])
    if n:
        o = o + torch.matmul(p[..., :n], pre[:, :D_LATENT])
    o = (o / total).bfloat16().reshape(b, t, h, D_LATENT)
    return (o, lse.reshape(b, t, h)) if c["lse"] else o


def _slots(s):
    """The page and the row in it of each row of the call."""
    c, lens = s["c"], s["lens"].long()
    at = torch.arange(c["tokens"], device=lens.device)
    if s["cu"] is not None:
        cu = s["cu"].long()
        seq = (at[:, None] >= cu[None, 1:]).sum(1)
        place, new = at - cu[seq], cu[1:] - cu[:-1]
    else:
        each = c["tokens"] // c["seqs"]
        seq, place, new = at // each, at % each, torch.full_like(lens, each)
    place = place + (lens - new)[seq]
    return s["table"].long()[seq, place // c["page"]], place % c["page"]


def _plain_read(s):
    page, row = _slots(s)
    return _decode_rows(s["cache"][page, row]).bfloat16()


def _plain_store(s):
    y = s["kv"][:, :D_LATENT].double()
    if s["weight"] is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * s["weight"].double()
    page, row = _slots(s)
    s["cache"][page, row] = _encode(y, s["kv"][:, D_LATENT:])
    return _plain_read(s)


def _own(s):
    from gated_delta_amd import rda
    c = s["c"]
    if c["op"] == "decode":
        o, lse = rda.rda_mla_decode_q4(s["q"], s["cache"], s["table"], s["lens"], SCALE, prefix_table=s["prefix"],
                                       prefix_len=c["prefix"], want_lse=c["lse"])
        return (o, lse) if c["lse"] else o
    if c["op"] == "store":
        rda.rda_mla_append_q4(s["kv"], s["cache"], s["table"], s["lens"], s["cu"], weight=s["weight"], eps=EPS)
    return rda.rda_mla_read_q4(s["cache"], s["table"], s["lens"], c["tokens"], s["cu"])


def run(state):
    if own:
        return _own(state)
    return {"decode": _plain_decode, "store": _plain_store, "read": _plain_read}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _values(rows):
    """Cached rows [n, 400] as values [n, 576] in 64 bits."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=torch.float64, device=rows.device)
    out = torch.empty(rows.shape[0], D_ROW, dtype=torch.float64, device=rows.device)
    out[:, 0:D_LATENT:2] = table[(rows[:, :CODES] % 16).long()]
    out[:, 1:D_LATENT:2] = table[(rows[:, :CODES] // 16).long()]
    for g in range(GROUPS):
        s = rows[:, CODES + g].double()
        factor = torch.where(s == 255, float("nan"), torch.exp2(s - 127))
        out[:, g * GROUP:(g + 1) * GROUP] *= factor[:, None]
    out[:, D_LATENT:] = rows[:, CODES + GROUPS:].contiguous().view(torch.bfloat16).double()
    return out


def _nearest(y):
    """Latent values [n, 512] in 64 bits as the 4-bit values that hold them."""
    steps = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=y.device)
    borders = (steps[1:] + steps[:-1]) / 2
    out = torch.empty_like(y)
    for g in range(GROUPS):
        x = y[:, g * GROUP:(g + 1) * GROUP]
        most = x.abs().amax(1)
        e = torch.full_like(most, LEAST)
        for n in range(LEAST + 1, MOST + 1):
            e = torch.where(most > 7 * 2.0 ** (n - 1), float(n), e)
        unit = torch.exp2(e)[:, None]
        t = x.abs() / unit
        at = (t[..., None] > borders).sum(-1)
        # a value on a border goes to the neighbour with an even place
        on = (t[..., None] == borders).any(-1)
        at = torch.where(on & (at % 2 == 1), at + 1, at)
        out[:, g * GROUP:(g + 1) * GROUP] = torch.sign(x) * steps[at] * unit
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    cache, dev, page = s["cache"], s["cache"].device, c["page"]
    if c["op"] != "decode":
        new, after = _row_lengths(c)
        if c["op"] == "store":
            x = s["kv"].double()
            if s["weight"] is not None:
                rms = torch.sqrt(x[:, :D_LATENT].pow(2).mean(1, keepdim=True) + EPS)
                x[:, :D_LATENT] = x[:, :D_LATENT] / rms * s["weight"].double()
            for at in range(0, x.shape[0], 4096):
                x[at:at + 4096, :D_LATENT] = _nearest(x[at:at + 4096, :D_LATENT])
            return x
        table = s["table"].tolist()
        at = [table[i][p // page] * page + p % page for i, (m, n) in enumerate(zip(new, after)) for p in range(n - m, n)]
        return _values(cache.reshape(-1, ROW_BYTES)[torch.tensor(at, device=dev)])
    b, t, h = c["batch"], c["new"], c["heads"]
    o = torch.zeros(b, t, h, D_LATENT, dtype=torch.float64, device=dev)
    lse = torch.full((b, t, h), float("-inf"), dtype=torch.float64, device=dev)
    pre = torch.zeros(0, D_ROW, dtype=torch.float64, device=dev)
    if c["prefix"]:
        pre = _values(cache[s["prefix"].long()].reshape(-1, ROW_BYTES)[:c["prefix"]])
    for i, n in enumerate(_decode_lengths(c)):
        rows = _values(cache[s["table"][i, :-(-n // page)].long()].reshape(-1, ROW_BYTES)[:n])
        for j in range(t):
            k = torch.cat([pre, rows[:max(0, n - (t - 1 - j))]])
            if k.shape[0] == 0:
                continue
            x = (s["q"][i, j].double() @ k.T) * SCALE
            lse[i, j] = torch.logsumexp(x, -1)
            o[i, j] = torch.exp(x - lse[i, j][:, None]) @ k[:, :D_LATENT]
    return (o, lse) if c["lse"] else o
