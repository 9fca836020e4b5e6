"""Plain 64-bit forms of the latent attention, its cache and the verification
of drafted tokens (test infrastructure), with bounds of what the kernels'
roundings may add.

Error bounds.  A score is a sum of K exact products in fp32 (at most K
roundings of 2^-24 relative to the sum of magnitudes), scaled and shifted in
one fused operation: off by at most ds = scale (K + 8) 2^-24 sum |q k|.  A
probability takes that as a relative error, an exponential's few 2^-23, and
one rounding to bf16 of at most 2^-8; the output one more of 2^-8:

    |o - o_ref| <= 2^-8 |o_ref| + (2^-8 (1 + 2^-8) + 2 (e^ds - 1) + n 2^-23) sum_j p_j |v_j|

(n fp32 additions, of the sum of probabilities and of the products, each).
The log-sum-exp carries the score's error and that of the sum:

    |lse - lse_ref| <= ds + (n + 16) 2^-23 + 2^-22 |lse_ref|
"""
import numpy as np
import torch

LATENT, ROW, NOPE, PE, V = 512, 576, 128, 64, 128
BF16_HALF_STEP = torch.finfo(torch.bfloat16).eps / 2     # 2^-8


def attend(q, k, v, scale, limit):
    """q [n, K], k [m, K], v [m, D], limit [n]: keys that each query sees (the
    first limit_i).  Returns o, lse and the bounds of both, in 64 bits."""
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    n, m = q.shape[0], k.shape[0]
    o = torch.zeros(n, v.shape[1], dtype=torch.float64)
    lse = torch.full((n,), float("-inf"), dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    for i in range(n):
        c = int(min(max(int(limit[i]), 0), m))
        if c == 0:
            continue
        s = scale * (k[:c] @ q[i])
        lse[i] = torch.logsumexp(s, 0)
        p = torch.exp(s - lse[i])
        o[i] = p @ v[:c]
        ds = float(scale * (q.shape[1] + 8) * 2.0 ** -24 * (k[:c].abs() @ q[i].abs()).max())
        most = p @ v[:c].abs()
        h = BF16_HALF_STEP
        bo[i] = h * o[i].abs() + (h * (1 + h) + 2 * np.expm1(ds) + c * 2.0 ** -23) * most + 1e-38
        bl[i] = ds + (c + 16) * 2.0 ** -23 + 2.0 ** -22 * lse[i].abs()
    return o, lse, bo, bl


def prefill(q, kv, pe, scale, cu_q, cu_k, causal):
    """q [Tq, H, 192], kv [Tk, H, 256], pe [Tk, 64] and offsets (lists)."""
    Tq, H = q.shape[:2]
    o = torch.zeros(Tq, H, V, dtype=torch.float64)
    lse = torch.full((Tq, H), float("-inf"), dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    for a, b, c, d in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        lq, lk = b - a, d - c
        limit = [i + 1 + lk - lq if causal else lk for i in range(lq)]
        for h in range(H):
            k = torch.cat([kv[c:d, h, :NOPE], pe[c:d]], 1)
            o[a:b, h], lse[a:b, h], bo[a:b, h], bl[a:b, h] = attend(
                q[a:b, h], k, kv[c:d, h, NOPE:], scale, limit)
    return o, lse, bo, bl


def cached_rows(cache, table, n):
    """The first n cached rows behind a page list."""
    page = cache.shape[1]
    pages = [int(x) for x in table[:-(-n // page)]]
    return (torch.cat([cache[p] for p in pages])[:n] if pages else cache[:0].reshape(0, ROW)).cpu()


def decode(q, cache, table, lens, scale, prefix_table=None, prefix_len=0):
    """q [B, T, H, 576]; rows of a sequence behind table[b], lens [B]."""
    B, T, H, _ = q.shape
    o = torch.zeros(B, T, H, LATENT, dtype=torch.float64)
    lse = torch.full((B, T, H), float("-inf"), dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    pre = cached_rows(cache, prefix_table, prefix_len) if prefix_len else None
    for b in range(B):
        n = int(lens[b])
        rows = cached_rows(cache, table[b], n)
        for t in range(T):
            own = rows[:max(0, n - (T - 1 - t))]
            k = torch.cat([pre, own]) if pre is not None else own
            o[b, t], lse[b, t], bo[b, t], bl[b, t] = attend(
                q[b, t], k, k[:, :LATENT], scale, [k.shape[0]] * H)
    return o, lse, bo, bl


def check(name, got, ref, bound):
    """got within bound of ref, element by element; infinities equal."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, f"{name}: shape {tuple(got.shape)}"
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), f"{name}: finite in other places"
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{name}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{name}: other infinities"
    over = ((got - ref).abs() - bound)[fin]
    if over.numel():
        worst = float((((got - ref).abs()) / (bound + 1e-300))[fin].max())
        print(f"{name}: largest error {worst:.3f} of its bound", flush=True)
        assert float(over.max()) <= 0, f"{name}: {worst:.3f} times the bound"


def append(kv, cache, table, lens, cu, weight, eps):
    """The cache after the call, in 64 bits (its bf16 values where untouched)."""
    out = cache.detach().cpu().double().clone()
    page = cache.shape[1]
    for n in range(len(cu) - 1):
        new = cu[n + 1] - cu[n]
        for i in range(new):
            x = kv[cu[n] + i].detach().cpu().double().clone()
            pos = int(lens[n]) - new + i
            if pos < 0 or pos >= table.shape[1] * page:
                continue
            p = int(table[n, pos // page])
            if p < 0 or p >= cache.shape[0]:
                continue
            if weight is not None:
                x[:LATENT] = x[:LATENT] / torch.sqrt((x[:LATENT] ** 2).mean() + eps) * weight.cpu().double()
            out[p, pos % page] = x
    return out


def verify(target, draft, tokens, u, num=None):
    """(accept, out_tokens) as int lists, with Python's exact sums of doubles."""
    import math
    B, T, V_ = target.shape
    acc, out = [], []
    for b in range(B):
        D = T - 1 if num is None else max(0, min(int(num[b]), T - 1))
        r = 0
        while r < D:
            d = int(tokens[b, r])
            if not 0 <= d < V_:
                break
            q = float(draft[b, r, d]) if draft is not None else 1.0
            if not float(u[b, r]) * q < float(target[b, r, d]):
                break
            r += 1
        p = target[b, r].double().numpy()
        if r < D:
            if draft is not None:
                w = p - draft[b, r].double().numpy()
            else:
                w = p.copy()
                if 0 <= int(tokens[b, r]) < V_:
                    w[int(tokens[b, r])] = 0
        else:
            w = p

        def clean(x):
            return np.where((x > 0) & (x < np.inf), x, 0.0)

        w = clean(w)
        if not w.sum() > 0:
            w = clean(p)
        pick = -1
        if w.sum() > 0:
            t = float(u[b, T - 1]) * math.fsum(w)
            over = np.nonzero((np.cumsum(w) > t) & (w > 0))[0]
            pick = int(over[0]) if len(over) else int(np.nonzero(w > 0)[0][-1])
        acc.append(r + 1)
        out.append([int(x) for x in tokens[b, :r]] + [pick] + [-1] * (T - 1 - r))
    return acc, out
