"""Decodes over long 8-bit caches in 64 bits on the GPU (test oracle), and which pieces the decode's walk cuts a batch into."""
import math

import torch

from paged8_ref import values

TILE, ROWS = 128, 16  # tokens of a tile, rows of an item


def attention(q, kc, vc, scales, table, lens, scale=None):
    """paged8_ref.attention for batches whose sequences are long and many: (o, lse, bound), in 64 bits on the device of q.
    Sequences with the same pages and length are computed together.  bound: per row X (see there) and M = max_n p_n vs_n (weight
    times value scale, of the tokens that the row sees), per element A = sum_n p_n |v_n| and C = sum_n |code of v_n|."""
    B, Hq, T, d = q.shape
    pages, Hkv, page, _ = kc.shape
    R = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    dev = q.device
    o, A, C = (torch.zeros(B, Hq, T, d, dtype=torch.float64, device=dev) for _ in range(3))
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=dev)
    X, M = (torch.zeros(B, Hq, T, dtype=torch.float64, device=dev) for _ in range(2))
    K, V, S = values(kc, scales[..., 0]), values(vc, scales[..., 1]), scales[..., 1].double()
    tab, ln = table.cpu(), lens.cpu()
    alike = {}
    for b in range(B):
        alike.setdefault((min(int(ln[b]), tab.shape[1] * page), tuple(tab[b].tolist())), []).append(b)
    for (n, row), bs in alike.items():
        if n == 0:
            continue
        i = torch.arange(n, device=dev)
        pg, sl = torch.tensor(row, device=dev)[i // page], i % page
        for g in range(Hkv):
            k, v, vs, code = K[pg, g, sl], V[pg, g, sl], S[pg, g, sl // 16], vc[pg, g, sl].double().abs()
            for b0 in range(0, len(bs), 64):
                at = torch.tensor(bs[b0:b0 + 64], device=dev)
                x = q[at, g * R:(g + 1) * R].double()                       # [b, R, T, d]
                s = x @ k.T * scale
                seen = i < n - T + 1 + torch.arange(T, device=dev)[:, None]  # [T, n]
                s.masked_fill_(~seen, -math.inf)
                lse[at, g * R:(g + 1) * R] = torch.logsumexp(s, -1)
                p = torch.softmax(s, -1)
                p = torch.where(seen.any(-1)[:, None], p, 0.0)
                put = lambda t, y: t.__setitem__((at, slice(g * R, (g + 1) * R)), y)  # noqa: E731
                put(o, p @ v)
                put(A, p @ v.abs())
                put(C, seen.double() @ code + torch.zeros_like(x))
                put(M, (p * vs).amax(-1))
                put(X, (x.abs() @ k.abs().T).amax(-1) * scale
                    + 2.0 ** -21 * x.abs().amax(-1) * k.abs().sum(-1).max() * scale / (d + 4) * 2 ** 23)
    return o, lse, (A, X, M, C)


def tolerance(dtype, d, n, bound):
    """Elementwise bounds on o and on lse for at most n tokens, made of what each row's own weights carry.

    Scores: sums of d exact products in fp32, (d + 4) roundings (truncations in the tensor cores: 2^-23 each) of at most X in
    all; a weight's relative error is twice that (its own and the sum's), plus 2^-20 for the exponential, and the sums take a rounding
    per 32 tokens (a product of the tensor cores) and 16 at a piece's end.
    bf16: a weight times its value scale is an f16: within 2^-11 of itself, or 2^-25 where it is below 2^-14, while the largest of the
    tokens that the row sees is at least 2^11 (to 2^-20): 2^-36 M, times a code; and the output is rounded (2^-8)."""
    A, X, M, C = bound
    ds = (d + 4) * 2.0 ** -23 * X
    sums = 2.0 ** -20 + (n / 32 + 16) * 2.0 ** -23
    w = (2 * ds + 2 * sums)[..., None]
    if dtype == torch.bfloat16:
        return lambda o: 2.0 ** -8 * o.abs() + (w + 2.0 ** -11) * A + 2.0 ** -36 * M[..., None] * C, ds + sums
    return lambda o: 2.0 ** -24 * o.abs() + w * A, ds + sums


def pieces(lens, Hq, Hkv, T, dtype, sms):
    """The tiles of every piece, CTA by CTA, as the decode cuts a batch: all items' tiles one after the other (and half a tile an item
    where ranges are long), in equal ranges."""
    rows = Hq // Hkv * T
    items = Hkv * -(-rows // ROWS)
    per_sm = 2 if dtype == torch.float32 else 4 if rows <= 4 else 3 if rows <= 8 else 2
    nt = [-(-max(n, 0) // TILE) for n in lens for _ in range(items)]
    G = min(sms * per_sm, sum(nt))
    extra = 2 * sum(nt) + sum(n > 0 for n in nt) >= 4 * G
    cost = [(n << extra) + extra if n else 0 for n in nt]
    total, got = sum(cost), [[] for _ in range(G)]
    lo = [g * (total // G) + min(g, total % G) for g in range(G + 1)]
    begin = g = 0
    for n, c in zip(nt, cost):
        end = begin + c
        while c:
            t0, t1 = (max(lo[g], begin) - begin) >> extra, n if lo[g + 1] >= end else (lo[g + 1] - begin) >> extra
            if t1 > t0:
                got[g].append(t1 - t0)
            if lo[g + 1] > end or g + 1 == G:
                break
            g += 1
            if lo[g] == end:
                break
        begin = end
    assert sum(map(sum, got)) == sum(nt)
    return got
