"""The serving operators around the RDA mixer, as cases for measuring: the
latent attention of the hybrid's other layers (expanded for prompts, absorbed
over a paged latent cache for decoding, with a prefix that a batch shares), the
write into that cache, and the verification of drafted tokens that yields
``rda_decode_tokens``' accept counts.

``run`` computes each in its plain form with elementary torch operations in 32
bits (64 where a value lies next to a border), or, with ``own`` set, by the
library's entry points.  ``exact`` is the definition in 64 bits.
"""
import random

import torch

own = False

# Widths of the latent attention: 128 key and value channels a head, 64 key
# channels shared by the heads, a latent vector of 512; a cache row is the
# latent followed by the shared key channels.
D_NOPE, D_PE, D_V, D_LATENT = 128, 64, 128, 512
D_QK, D_ROW = D_NOPE + D_PE, D_LATENT + D_PE
SCALE = D_QK ** -0.5
EPS = 1e-5


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a short question to a model that is waiting: one prompt of 65 tokens
        {"name": "prefill 65", "op": "prefill", "heads": 32, "seqs": 1, "tokens": 65,
         "context": 0, "causal": True, "lse": True, "split": 0},
        # a serving batch: five ragged prompts, each behind what is already cached of it
        {"name": "prefill ragged 4096+3001", "op": "prefill", "heads": 16, "seqs": 5, "tokens": 4096,
         "context": 3001, "causal": True, "lse": False, "split": 1},
        # one long prompt
        {"name": "prefill 8192", "op": "prefill", "heads": 32, "seqs": 1, "tokens": 8192,
         "context": 0, "causal": True, "lse": False, "split": 2},
        # one user's next token: latency
        {"name": "decode 1x777", "op": "decode", "batch": 1, "new": 1, "heads": 32, "shortest": 777,
         "longest": 777, "prefix": 0, "page": 64, "lse": False, "split": 3},
        # a current token and two drafts for a batch of 32
        {"name": "decode 32x3", "op": "decode", "batch": 32, "new": 3, "heads": 32, "shortest": 512,
         "longest": 8192, "prefix": 0, "page": 64, "lse": True, "split": 4},
        # a full batch's next tokens
        {"name": "decode 256x1", "op": "decode", "batch": 256, "new": 1, "heads": 32, "shortest": 512,
         "longest": 8192, "prefix": 0, "page": 64, "lse": False, "split": 5},
        # eight samples of one question: a common prompt, answers just begun
        {"name": "shared 8x1 4097", "op": "decode", "batch": 8, "new": 1, "heads": 32, "shortest": 1,
         "longest": 100, "prefix": 4097, "page": 64, "lse": False, "split": 6},
        # a long system prompt before every request of a batch, with two drafts each
        {"name": "shared 128x3 16384", "op": "decode", "batch": 128, "new": 3, "heads": 32,
         "shortest": 16, "longest": 512, "prefix": 16384, "page": 64, "lse": False, "split": 7},
        # drafts taken greedily (no draft probabilities) over a small odd vocabulary
        {"name": "verify 8x3 32003", "op": "verify", "batch": 8, "drafts": 3, "vocab": 32003,
         "sampled": False, "ragged": True},
        # a full batch with two sampled drafts each over the whole vocabulary
        {"name": "verify 256x2 259840", "op": "verify", "batch": 256, "drafts": 2, "vocab": 259840,
         "sampled": True, "ragged": False},
        # the new rows of a decoding batch
        {"name": "append 256x3", "op": "append", "seqs": 256, "tokens": 768, "ragged": False,
         "cached": 1024, "page": 64, "norm": True, "split": 8},
        # the rows of a batch of prompts
        {"name": "append 8 of 32768", "op": "append", "seqs": 8, "tokens": 32768, "ragged": True,
         "cached": 0, "page": 64, "norm": True, "split": 9},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prefill", "decode", "shared", "verify", "append"])
    split = rng.randrange(1 << 20)
    if op == "prefill":
        heads, tokens = rng.choice([4, 8, 16, 32, 40]), _log(rng, 1, 8192)
        context = rng.choice([0, _log(rng, 1, 8192)])
        while heads * tokens * (tokens + context) > 1 << 30:
            tokens, context = tokens * 3 // 4, context * 3 // 4
        return {"op": op, "heads": heads, "seqs": rng.randint(1, min(8, tokens)), "tokens": tokens,
                "context": context, "causal": rng.random() < 0.8, "lse": rng.random() < 0.5, "split": split}
    if op in ("decode", "shared"):
        batch, new, heads = _log(rng, 1, 256), rng.choice([1, 1, 2, 3, 5, 8]), rng.choice([8, 16, 32, 40])
        longest = _log(rng, 1, 8192 if op == "decode" else 600)
        prefix = 0 if op == "decode" else _log(rng, 1, 16384)
        while batch > 1 and batch * new * heads * (longest + prefix) > 1 << 27:
            batch = batch * 3 // 4
        return {"op": "decode", "batch": batch, "new": new, "heads": heads, "shortest": rng.randint(0, longest),
                "longest": longest, "prefix": prefix, "page": rng.choice([16, 32, 64, 128, 256]),
                "lse": rng.random() < 0.5, "split": split}
    if op == "verify":
        return {"op": op, "batch": _log(rng, 1, 256), "drafts": rng.randint(1, 4), "vocab": _log(rng, 997, 200000),
                "sampled": rng.random() < 0.7, "ragged": rng.random() < 0.5}
    seqs = _log(rng, 1, 256)
    return {"op": op, "seqs": seqs, "tokens": seqs * rng.randint(1, 4) if rng.random() < 0.5 else _log(rng, seqs, 30000),
            "ragged": True, "cached": rng.choice([0, _log(rng, 1, 1024)]), "page": rng.choice([16, 32, 64, 128, 256]),
            "norm": rng.random() < 0.8, "split": split}


def _parts(total, n, rng):
    """n whole numbers that sum to total, drawn at random."""
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _prefill_lengths(c):
    """(query tokens, key tokens) of each sequence."""
    rng = random.Random(c["split"])
    lq = _parts(c["tokens"], c["seqs"], rng)
    return lq, [a + b for a, b in zip(lq, _parts(c["context"], c["seqs"], rng))]


def _decode_lengths(c):
    rng = random.Random(c["split"])
    return [rng.randint(c["shortest"], c["longest"]) for _ in range(c["batch"])]


def _append_lengths(c):
    """(new tokens, cached tokens after them) of each sequence."""
    rng = random.Random(c["split"])
    n = c["seqs"]
    new = _parts(c["tokens"], n, rng) if c["ragged"] else [c["tokens"] // n] * n
    return new, [a + rng.randint(0, c["cached"]) for a in new]


def _seen(lq, lk, causal):
    """Keys that the queries of one sequence see, in all."""
    return sum(max(0, min(lk, i + 1 + lk - lq)) for i in range(lq)) if causal else lq * lk


def work(case):
    c = case
    if c["op"] == "prefill":
        lq, lk = _prefill_lengths(c)
        h = c["heads"]
        pairs = sum(_seen(a, b, c["causal"]) for a, b in zip(lq, lk))
        return {"bytes": 2 * (sum(lq) * h * (D_QK + D_V) + sum(lk) * (h * (D_NOPE + D_V) + D_PE)),
                "flops": 2 * pairs * h * (D_QK + D_V)}
    if c["op"] == "decode":
        lens = _decode_lengths(c)
        rows = c["batch"] * c["new"] * c["heads"]
        pairs = c["heads"] * sum(c["new"] * c["prefix"] + _seen(c["new"], n, True) for n in lens)
        return {"bytes": 2 * ((sum(lens) + c["prefix"]) * D_ROW + rows * (D_ROW + D_LATENT)),
                "flops": 2 * pairs * (D_ROW + D_LATENT)}
    if c["op"] == "verify":
        # the rows of the position where the drafts end, and the drafts' own probabilities
        return {"bytes": c["batch"] * (4 * c["vocab"] * (2 if c["sampled"] else 1) + 8 * c["drafts"]),
                "flops": c["batch"] * c["vocab"] * 2}
    return {"bytes": 4 * c["tokens"] * D_ROW, "flops": 4 * c["tokens"] * D_LATENT}


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


def prepare(case, seed):
    c, dev = case, _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if c["op"] == "prefill":
        lq, lk = _prefill_lengths(c)
        h = c["heads"]
        # kv is the up-projection's output (keys and values of a head side by side);
        # the shared key channels are a slice of the latent projection's rows
        rows = normal(sum(lk), D_ROW).bfloat16()
        return {"c": c, "q": (2 * normal(sum(lq), h, D_QK)).bfloat16(),
                "kv": normal(sum(lk), h, D_NOPE + D_V).bfloat16(), "pe": rows[:, D_LATENT:],
                "cu_q": _ints(_offsets(lq)), "cu_k": _ints(_offsets(lk))}
    if c["op"] == "decode":
        lens, page = _decode_lengths(c), c["page"]
        npre = -(-c["prefix"] // page)
        table, order, pool = _pages(lens, page, max(1, -(-c["longest"] // page)), gen, npre + 3)
        return {"c": c, "q": normal(c["batch"], c["new"], c["heads"], D_ROW).bfloat16(),
                "cache": normal(pool, page, D_ROW).bfloat16(), "table": table, "lens": _ints(lens),
                "prefix": order[pool - npre:].contiguous() if npre else None}
    if c["op"] == "verify":
        b, d, v = c["batch"], c["drafts"], c["vocab"]
        logits = 3 * normal(b, d + 1, v)
        target = torch.softmax(logits, -1)
        draft = torch.softmax(logits[:, :d] + normal(b, d, v), -1)
        if c["sampled"]:
            tok = torch.multinomial(draft.reshape(b * d, v), 1, generator=gen).reshape(b, d)
        else:
            tok, draft = draft.argmax(-1), None
        num = torch.randint(0, d + 1, (b,), generator=gen, device=dev).to(torch.int32) if c["ragged"] else None
        return {"c": c, "target": target, "draft": draft, "tokens": tok.to(torch.int32),
                "u": torch.rand(b, d + 1, generator=gen, device=dev), "num": num}
    new, after = _append_lengths(c)
    page = c["page"]
    table, _, pool = _pages(after, page, max(1, -(-max(after) // page)), gen, 3)
    return {"c": c, "kv": (3 * normal(c["tokens"], D_ROW)).bfloat16(), "cache": normal(pool, page, D_ROW).bfloat16(),
            "table": table, "lens": _ints(after), "cu": _ints(_offsets(new)) if c["ragged"] else None,
            "weight": 1 + 0.1 * normal(D_LATENT) if c["norm"] else None}


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


def _of_sequence(cu, total):
    """The sequence of each packed token and its place in it."""
    at = torch.arange(total, device=cu.device)
    seq = (at[:, None] >= cu[None, 1:]).sum(1)
    return seq, at - cu.long()[seq]


def _plain_prefill(s):
    c, q, kv = s["c"], s["q"].float(), s["kv"].float()
    lens_q, lens_k = (cu.long()[1:] - cu.long()[:-1] for cu in (s["cu_q"], s["cu_k"]))
    qs, qp = _of_sequence(s["cu_q"], q.shape[0])
    ks, kp = _of_sequence(s["cu_k"], kv.shape[0])
    k = torch.cat([kv[..., :D_NOPE], s["pe"].float()[:, None].expand(-1, c["heads"], -1)], -1)
    scores = torch.matmul(q.transpose(0, 1) * SCALE, k.permute(1, 2, 0))
    seen = qs[:, None] == ks[None, :]
    if c["causal"]:
        seen &= kp[None, :] <= (qp + (lens_k - lens_q)[qs])[:, None]
    p, total, lse = _softmax_parts(scores.masked_fill_(~seen, float("-inf")))
    o = (torch.matmul(p, kv[..., D_NOPE:].transpose(0, 1)) / total).transpose(0, 1).contiguous().bfloat16()
    return (o, lse.transpose(0, 1).contiguous()) if c["lse"] else o


def _plain_decode(s):
    c, cache = s["c"], s["cache"]
    b, t, h = c["batch"], c["new"], c["heads"]
    q = s["q"].float().reshape(b, t * h, D_ROW) * SCALE
    kv = cache[s["table"].clamp(min=0).long()].reshape(b, -1, D_ROW).float()
    last = s["lens"].long()[:, None] - (t - 1 - torch.arange(t, device=q.device))[None, :]
    seen = torch.arange(kv.shape[1], device=q.device)[None, None, :] < last[:, :, None]
    scores = torch.matmul(q, kv.transpose(1, 2))
    scores = scores.reshape(b, t, h, -1).masked_fill_(~seen[:, :, None, :], float("-inf")).reshape(b, t * h, -1)
    n = c["prefix"]
    if n:
        pre = cache[s["prefix"].long()].reshape(-1, D_ROW)[:n].float()
        scores = torch.cat([torch.matmul(q, pre.t()), scores], -1)
    p, total, lse = _softmax_parts(scores)
    o = torch.matmul(p[..., n:], kv[..., :D_LATENT])
    if n:
        o = o + torch.matmul(p[..., :n], pre[:, :D_LATENT])
    o = (o / total).bfloat16().reshape(b, t, h, D_LATENT)
    return (o, lse.reshape(b, t, h)) if c["lse"] else o


def _plain_verify(s):
    c, target, tok = s["c"], s["target"], s["tokens"].long()
    b, d, v = c["batch"], c["drafts"], c["vocab"]
    at = torch.arange(b, device=tok.device)
    p_tok = target[:, :d].gather(2, tok[:, :, None])[..., 0].double()
    q_tok = s["draft"].gather(2, tok[:, :, None])[..., 0].double() if c["sampled"] else torch.ones_like(p_tok)
    ok = s["u"][:, :d].double() * q_tok < p_tok
    count = s["num"].long() if s["num"] is not None else torch.full_like(at, d)
    ok &= torch.arange(d, device=tok.device)[None, :] < count[:, None]
    good = torch.cumprod(ok.long(), 1).sum(1)
    p = target[at, good].double()
    row, rejected = good.clamp(max=d - 1), good < count
    if c["sampled"]:
        left = p - s["draft"][at, row].double()
    else:
        left = p.clone()
        left[at, tok[at, row]] = 0
    left = torch.where(rejected[:, None], left, p).clamp(min=0)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, p)
    run_sum = torch.cumsum(left, 1)
    beyond = run_sum > s["u"][:, d].double()[:, None] * run_sum[:, -1:]
    pick = (beyond & (left > 0)).long().argmax(1)
    col = torch.arange(d + 1, device=tok.device)[None, :]
    drafted = torch.cat([tok, tok[:, :1]], 1)
    out = torch.where(col < good[:, None], drafted, torch.where(col == good[:, None], pick[:, None], -1))
    return (good + 1).to(torch.int32), out.to(torch.int32)


def _slots(s):
    """The page and the row in it of each new token."""
    c, lens = s["c"], s["lens"].long()
    n = c["tokens"]
    if s["cu"] is not None:
        cu = s["cu"].long()
        seq, place = _of_sequence(cu, n)
        new = cu[1:] - cu[:-1]
    else:
        each = n // c["seqs"]
        at = torch.arange(n, device=lens.device)
        seq, place, new = at // each, at % each, torch.full_like(lens, each)
    place = place + (lens - new)[seq]
    return s["table"].long()[seq, place // c["page"]], place % c["page"]


def _plain_append(s):
    x = s["kv"].float()
    if s["weight"] is not None:
        head = x[:, :D_LATENT]
        head = head / torch.sqrt((head * head).mean(-1, keepdim=True) + EPS) * s["weight"]
        x = torch.cat([head, x[:, D_LATENT:]], 1)
    page, row = _slots(s)
    s["cache"][page, row] = x.bfloat16()
    return s["cache"]


def _own(s):
    from gated_delta_amd import rda
    c = s["c"]
    if c["op"] == "prefill":
        o, lse = rda.rda_mla_prefill(s["q"], s["kv"], s["pe"], SCALE, s["cu_q"], s["cu_k"],
                                     causal=c["causal"], want_lse=c["lse"])
        return (o, lse) if c["lse"] else o
    if c["op"] == "decode":
        o, lse = rda.rda_mla_decode(s["q"], s["cache"], s["table"], s["lens"], SCALE, prefix_table=s["prefix"],
                                    prefix_len=c["prefix"], want_lse=c["lse"])
        return (o, lse) if c["lse"] else o
    if c["op"] == "verify":
        return rda.rda_verify_drafts(s["target"], s["draft"], s["tokens"], s["u"], s["num"])
    return rda.rda_mla_append(s["kv"], s["cache"], s["table"], s["lens"], s["cu"], weight=s["weight"], eps=EPS)


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "verify": _plain_verify,
            "append": _plain_append}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _attend(q, k, v, causal):
    """softmax(q k^T SCALE) v of one head in 64 bits, the queries at the keys' end; (o, log-sum-exp)."""
    x = (q @ k.T) * SCALE
    if causal:
        last = torch.arange(q.shape[0], device=q.device) + (k.shape[0] - q.shape[0])
        x[torch.arange(k.shape[0], device=q.device)[None, :] > last[:, None]] = float("-inf")
    lse = torch.logsumexp(x, -1) if k.shape[0] else torch.full_like(q[:, 0], float("-inf"))
    return torch.nan_to_num(torch.exp(x - lse[:, None])) @ v, lse


def exact(case, seed):
    c = case
    if c["op"] == "verify":
        return None
    s = prepare(c, seed)
    dev = s["lens"].device if "lens" in s else s["q"].device
    if c["op"] == "prefill":
        lq, lk = _prefill_lengths(c)
        o = torch.zeros(sum(lq), c["heads"], D_V, dtype=torch.float64, device=dev)
        lse = torch.zeros(sum(lq), c["heads"], dtype=torch.float64, device=dev)
        for q0, nq, k0, nk in zip(_offsets(lq), lq, _offsets(lk), lk):
            for h in range(c["heads"]):
                kv = s["kv"][k0:k0 + nk, h].double()
                k = torch.cat([kv[:, :D_NOPE], s["pe"][k0:k0 + nk].double()], 1)
                o[q0:q0 + nq, h], lse[q0:q0 + nq, h] = _attend(s["q"][q0:q0 + nq, h].double(), k, kv[:, D_NOPE:], c["causal"])
        return (o, lse) if c["lse"] else o
    if c["op"] == "decode":
        b, t, h = c["batch"], c["new"], c["heads"]
        o = torch.zeros(b, t, h, D_LATENT, dtype=torch.float64, device=dev)
        lse = torch.zeros(b, t, h, dtype=torch.float64, device=dev)
        pre = s["cache"][:0].reshape(-1, D_ROW).double()
        if c["prefix"]:
            pre = s["cache"][s["prefix"].long()].reshape(-1, D_ROW)[:c["prefix"]].double()
        for i, n in enumerate(_decode_lengths(c)):
            rows = s["cache"][s["table"][i, :-(-n // c["page"])].long()].reshape(-1, D_ROW)[:n].double()
            for j in range(t):
                k = torch.cat([pre, rows[:max(0, n - (t - 1 - j))]])
                o[i, j], lse[i, j] = _attend(s["q"][i, j].double(), k, k[:, :D_LATENT], False)
        return (o, lse) if c["lse"] else o
    cache, x = s["cache"].double(), s["kv"].double()
    if s["weight"] is not None:
        rms = torch.sqrt(x[:, :D_LATENT].pow(2).mean(1, keepdim=True) + EPS)
        x[:, :D_LATENT] = x[:, :D_LATENT] / rms * s["weight"].double()
    new, after = _append_lengths(c)
    table = s["table"].tolist()
    page = [table[i][p // c["page"]] for i, (m, n) in enumerate(zip(new, after)) for p in range(n - m, n)]
    row = [p % c["page"] for m, n in zip(new, after) for p in range(n - m, n)]
    cache[page, row] = x
    return cache
