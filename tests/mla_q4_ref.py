"""The 4-bit latent cache in 64 bits (test infrastructure), written from the
format, and bounds of what the attention kernel's roundings may add.

A cached row: 512 e2m1 codes (two a byte, the even channel's in the low half),
16 scale bytes (2^(s - 127), 255: NaN), 64 bf16 values.

Error bounds of the attention: those of mla_ref, and the query's.  It enters the
products as hi + lo, 8-bit floats (4 significant bits, least step 2^-9) scaled
by powers of two so that the row's largest latent magnitude M becomes at least
128 for hi and lo has 1/32 of hi's scale.  hi is off by at most half its step, which lo
holds exactly unless its own step of 2^-9 / 32 is too large: off by at most
2^-10 / 32 = 2^-15 where M is 128 or more, that is 2^-22 M.  So a score is off by
2^-22 M sum |c_j| scale more.
"""
import numpy as np
import torch

import mla_ref
from mla_ref import BF16_HALF_STEP, LATENT, ROW, check  # noqa: F401

ROW_BYTES, GROUP, GROUPS = 400, 32, 16
SIZES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def values(rows):
    """Cached rows [..., 400] uint8 as values [..., 576] in 64 bits."""
    x = rows.detach().cpu().numpy()
    flat = x.reshape(-1, ROW_BYTES)
    out = np.empty((flat.shape[0], ROW), np.float64)
    signed = np.concatenate([SIZES, -SIZES])
    codes = flat[:, :256]
    out[:, 0:LATENT:2], out[:, 1:LATENT:2] = signed[codes & 15], signed[codes >> 4]
    scale = np.ldexp(1.0, flat[:, 256:272].astype(np.int32) - 127)
    scale[flat[:, 256:272] == 255] = np.nan
    out[:, :LATENT] *= np.repeat(scale, GROUP, 1)
    pe = np.ascontiguousarray(flat[:, 272:]).view(np.uint16).astype(np.uint32) << 16
    out[:, LATENT:] = pe.view(np.float32)
    return torch.from_numpy(out.reshape(*x.shape[:-1], ROW))


def encode_row(latent, pe):
    """One row from 512 Python floats / a float64 array and 64 bf16 values."""
    out = np.zeros(ROW_BYTES, np.uint8)
    y = np.asarray(latent, np.float64)
    for g in range(GROUPS):
        part = y[g * GROUP:(g + 1) * GROUP]
        if not np.isfinite(part).all():
            out[256 + g] = 255
            continue
        most = np.abs(part).max()
        e = -120
        while e < 125 and most > 7 * 2.0 ** e:
            e += 1
        out[256 + g] = e + 127
        t = np.abs(part) / 2.0 ** e
        dist = np.abs(t[:, None] - SIZES[None, :])
        near = dist.min(1, keepdims=True)
        for i in range(GROUP):
            tied = [c for c in range(8) if dist[i, c] == near[i, 0]]
            # a value half way goes to the even code
            c = tied[0] if len(tied) == 1 else [c for c in tied if c % 2 == 0][0]
            if part[i] < 0 and c:
                c |= 8
            ch = g * GROUP + i
            out[ch // 2] |= c << (4 * (ch % 2))
    out[272:] = pe.detach().cpu().contiguous().view(torch.uint8).numpy()
    return torch.from_numpy(out)


def normed(kv, weight, eps):
    """The latent parts [n, 512] in 64 bits."""
    x = kv[:, :LATENT].detach().cpu().double()
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(1, keepdim=True) + float(np.float32(eps))) * weight.cpu().double()


def append(kv, cache, table, lens, cu, weight, eps):
    """The cache's bytes after the call."""
    out = cache.detach().cpu().clone()
    y, kv = normed(kv, weight, eps), kv.detach().cpu()
    page = cache.shape[1]
    for n in range(len(cu) - 1):
        new = cu[n + 1] - cu[n]
        for i in range(new):
            pos = int(lens[n]) - new + i
            if pos < 0 or pos >= table.shape[1] * page:
                continue
            p = int(table[n, pos // page])
            if 0 <= p < cache.shape[0]:
                out[p, pos % page] = encode_row(y[cu[n] + i].numpy(), kv[cu[n] + i, LATENT:])
    return out


def read(cache, table, lens, cu, total, before=None):
    """[total, 576] in 64 bits; rows outside every part as they are in `before`."""
    out = torch.zeros(total, ROW, dtype=torch.float64) if before is None else before.detach().cpu().double()
    page = cache.shape[1]
    for n in range(len(cu) - 1):
        rows = cu[n + 1] - cu[n]
        for i in range(rows):
            pos = int(lens[n]) - rows + i
            p = int(table[n, pos // page]) if 0 <= pos < table.shape[1] * page else -1
            out[cu[n] + i] = values(cache[p, pos % page]) if 0 <= p < cache.shape[0] else 0.0
    return out


def attend(q, k, v, scale):
    """q [n, 576], k [m, 576], v [m, 512] in 64 bits: o, lse and their bounds."""
    n, c = q.shape[0], k.shape[0]
    o = torch.zeros(n, v.shape[1], dtype=torch.float64)
    lse = torch.full((n,), float("-inf"), dtype=torch.float64)
    if c == 0:
        return o, lse, torch.zeros_like(o), torch.zeros_like(lse)
    q = q.detach().cpu().double()
    s = scale * (q @ k.T)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    o, most = p @ v, p @ v.abs()
    ds = scale * ((ROW + 8) * 2.0 ** -24 * (q.abs() @ k.abs().T).amax(1) +
                  2.0 ** -22 * q[:, :LATENT].abs().amax(1) * k[:, :LATENT].abs().sum(1).max())
    h = BF16_HALF_STEP
    bo = h * o.abs() + (h * (1 + h) + 2 * torch.expm1(ds)[:, None] + c * 2.0 ** -23) * most + 1e-38
    bl = ds + (c + 16) * 2.0 ** -23 + 2.0 ** -22 * lse.abs()
    return o, lse, bo, bl


def cached(cache, table, n):
    page = cache.shape[1]
    pages = [int(x) for x in table[:-(-n // page)]]
    rows = torch.cat([cache[p] for p in pages])[:n] if pages else cache[:0].reshape(0, ROW_BYTES)
    return values(rows)


def decode(q, cache, table, lens, scale, prefix_table=None, prefix_len=0):
    """q [B, T, H, 576] over the 4-bit cache: (o, lse, bounds of both)."""
    B, T, H, _ = q.shape
    cache, q = cache.detach().cpu(), q.detach().cpu()
    res = [torch.zeros(B, T, H, LATENT, dtype=torch.float64), torch.zeros(B, T, H, dtype=torch.float64),
           torch.zeros(B, T, H, LATENT, dtype=torch.float64), torch.zeros(B, T, H, dtype=torch.float64)]
    pre = cached(cache, prefix_table, prefix_len) if prefix_len else torch.zeros(0, ROW, dtype=torch.float64)
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * cache.shape[1])
        rows = cached(cache, table[b], n)
        for t in range(T):
            k = torch.cat([pre, rows[:max(0, n - (T - 1 - t))]])
            for x, y in zip(res, attend(q[b, t], k, k[:, :LATENT], scale)):
                x[b, t] = y
    return res
