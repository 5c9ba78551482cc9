"""Paged decode row by row: every (sequence, query head) has to be as good as its own size allows.

Bound of a row's error, relative to the row's own norm.  A score is a sum of d products in fp32, so it is off by at
most e = (d + 4) 2^-24 max|score| (the four: the scale, log2(e), the subtraction of the maximum and exp2), which is
its weight's relative error; the sums over n tokens add n 2^-24, and the weights' two bf16 parts leave 2^-17.  These are
relative to sum_n w_n |v_n|, which cancellation may make much larger than |o|: their ratio multiplies them.  The
output's rounding is 2^-8 of the row in bf16, 2^-24 in fp32.  lse: e + n 2^-24, and its own rounding, two steps of
2^-24 of the larger of |lse| and 1."""
import pytest
import torch

import chunked_state_scan_causal_gb300 as la

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_state_scan_causal_gb300 import build
    build.build()


def case(seed, lens, Hq, Hkv, d, page, dtype):
    """q, caches, table and lengths; what no length covers holds NaN."""
    g = torch.Generator().manual_seed(seed)
    B, blocks = len(lens), max(1, -(-max(lens) // page))
    pages = B * blocks + 2
    table = torch.randperm(pages, generator=g)[: B * blocks].view(B, blocks).to(torch.int32)
    q = torch.randn(B, Hq, 1, d, generator=g).to(dtype)
    kc, vc = (torch.randn(pages, Hkv, page, d, generator=g).to(dtype) for _ in range(2))
    for b, n in enumerate(lens):
        for j in range(blocks):
            used = max(0, min(page, n - j * page))
            kc[table[b, j], :, used:] = NAN
            vc[table[b, j], :, used:] = NAN
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32)


def run(c):
    x = [t.cuda() for t in c]
    ws = la.workspace(x[0], la.OP_PAGED_DECODE)
    o, lse = la.paged_decode(*x, want_lse=True, ws=ws)
    assert la.device_status(ws) == la.OK
    return o.cpu(), lse.cpu()


def rows(c):
    """Per (b, h): o, lse, and the bounds of their errors, in 64 bits (finite inputs)."""
    q, kc, vc, table, lens = c
    (B, Hq, _, d), Hkv, page = q.shape, kc.shape[1], kc.shape[2]
    for b in range(B):
        n = int(lens[b])
        blocks = table[b, : -(-n // page)].long()
        K, V = (x[blocks].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :n] for x in (kc, vc))
        for h in range(Hq):
            if n == 0:
                yield b, h, torch.zeros(d, dtype=torch.float64), -INF, 0.0, 0.0
                continue
            k, v = K[h // (Hq // Hkv)], V[h // (Hq // Hkv)]
            x = (k @ q[b, h, 0].double()) * d ** -0.5
            w, lse = torch.softmax(x, 0), float(torch.logsumexp(x, 0))
            o = w @ v
            e = (d + 4) * 2 ** -24 * max(float(x.abs().max()), 1.0) + n * 2 ** -24
            ratio = float((w * v.norm(dim=-1)).sum() / o.norm())
            bf16 = q.dtype == BF16
            yield (b, h, o, lse, (2 ** -8 if bf16 else 2 ** -24) + (e + (2 ** -17 if bf16 else 0.0)) * ratio,
                   e + 2 ** -23 * max(abs(lse), 1.0))


def check_rows(c, o, lse, skip=()):
    for b, h, ro, rl, bound, lbound in rows(c):
        if (b, h) in skip:
            continue
        if rl == -INF:
            assert (o[b, h] == 0).all() and lse[b, h] == -INF
            continue
        err = float((o[b, h, 0].double() - ro).norm() / ro.norm())
        assert err <= bound, (b, h, err, bound)
        assert abs(float(lse[b, h]) - rl) <= lbound, (b, h, float(lse[b, h]), rl, lbound)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("Hq,Hkv,d,page,lens", [
    (4, 2, 128, 32, [5] * 40 + [2000]),              # whole items beside one that is cut over CTAs
    (8, 1, 128, 64, [20000, 3, 0, 700]),
    (16, 1, 64, 16, [129, 128, 127, 1, 4000]),
    (20, 1, 128, 24, [300, 65, 1500]),               # two slices of query heads
    (2, 2, 64, 3, [1000, 10]),                       # pages copied piece by piece
    (32, 8, 128, 16, [125 + 3 * i for i in range(64)]),
])
def test_every_row(dtype, Hq, Hkv, d, page, lens):
    c = case(1, lens, Hq, Hkv, d, page, dtype)
    check_rows(c, *run(c))
