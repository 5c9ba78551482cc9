"""Paged decode row by row: every (sequence, query head) has to be as good as its own size allows, and what is not a
number inside a length has to reach the rows that read it.

Bound of a row's error, relative to the row's own norm.  A score is a sum of d products in fp32, so it is off by at
most e = (d + 4) 2^-24 max|score| (the four: the scale, log2(e), the subtraction of the maximum and exp2), which is
its weight's relative error; the sums over n tokens add n 2^-24, and the weights' two bf16 parts leave 2^-17.  These are
relative to sum_n w_n |v_n|, which cancellation may make much larger than |o|: their ratio multiplies them.  The
output's rounding is 2^-8 of the row in bf16, 2^-24 in fp32.  lse: e + n 2^-24, and its own rounding, two steps of
2^-24 of the larger of |lse| and 1."""
import math

import pytest
import torch

import chunked_state_scan_causal_gb300 as la
from delta_ref import paged_attention

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


def same_or_nan(c, o, lse, want_nan):
    """Rows in want_nan (b, key head): all NaN; the others as good as ever."""
    group = c[0].shape[1] // c[1].shape[1]
    bad = {(b, hk * group + i) for b, hk in want_nan for i in range(group)}
    for b, h in bad:
        assert o[b, h].isnan().all() and lse[b, h].isnan().all(), (b, h, o[b, h], lse[b, h])
    return bad


HEADS = [(4, 2, 128, 16), (8, 1, 64, 128), (16, 1, 128, 24), (4, 4, 64, 3), (20, 1, 128, 16)]


def slot(c, b, n):
    page = c[1].shape[2]
    return int(c[3][b, n // page]), n % page


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("Hq,Hkv,d,page", HEADS)
def test_nan_key(dtype, Hq, Hkv, d, page):
    """One NaN key in the first, a middle or the last token: NaN for its key head's rows, nothing else moves."""
    c = case(2, [300, 1, 900, 640, 77], Hq, Hkv, d, page, dtype)
    clean = [t.clone() for t in c]
    for b, n in ((0, 0), (2, 500), (3, 639)):
        p, s = slot(c, b, n)
        c[1][p, 0, s, d // 2] = NAN
    o, lse = run(c)
    bad = same_or_nan(c, o, lse, [(0, 0), (2, 0), (3, 0)])
    check_rows(clean, o, lse, bad)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("Hq,Hkv,d,page", HEADS)
def test_nan_query(dtype, Hq, Hkv, d, page):
    """A NaN query is not an empty sequence: o and lse are NaN for its row alone."""
    c = case(3, [300, 1, 2000], Hq, Hkv, d, page, dtype)
    clean = [t.clone() for t in c]
    for b, h in ((0, 0), (1, Hq - 1), (2, Hq // 2)):
        c[0][b, h, 0, 3] = NAN
    o, lse = run(c)
    bad = {(0, 0), (1, Hq - 1), (2, Hq // 2)}
    for b, h in bad:
        assert o[b, h].isnan().all() and lse[b, h].isnan().all()
    check_rows(clean, o, lse, bad)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("first", [0, 128, 1024, 1920])
def test_pages_never_appended(dtype, first):
    """A tile's worth of NaN inside the length, wherever it is: NaN, not attention over the rest of the tokens."""
    c = case(4, [2048, 2048, 30], 4, 2, 128, 64, dtype)
    clean = [t.clone() for t in c]
    for n in range(first, first + 128, 64):
        p, _ = slot(c, 0, n)
        c[1][p] = NAN
        c[2][p] = NAN
    o, lse = run(c)
    bad = same_or_nan(c, o, lse, [(0, 0), (0, 1)])
    check_rows(clean, o, lse, bad)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("Hq,Hkv,d,page", HEADS)
def test_infinite_keys(dtype, Hq, Hkv, d, page):
    """A score of +inf has no softmax (NaN); one of -inf is a weight of zero."""
    lens = [300, 700, 129]
    c = case(5, lens, Hq, Hkv, d, page, dtype)
    c[0][:, :, 0, 0] = c[0][:, :, 0, 0].abs() + 0.5
    clean = [t.clone() for t in c]
    p, s = slot(c, 0, 200)
    c[1][p, :, s, 0] = INF
    gone = [(1, n) for n in (0, 5, 350, 699)] + [(2, n) for n in range(128)]   # (2: one token is left)
    for b, n in gone:
        p, s = slot(c, b, n)
        c[1][p, :, s, 0] = -INF
    o, lse = run(c)
    assert o[0].isnan().all() and not lse[0].isfinite().any()
    # the same without the tokens of weight zero, in an order of its own
    for b in (1, 2):
        keep = [n for n in range(lens[b]) if (b, n) not in gone]
        at = [slot(clean, b, n) for n in keep]
        K, V = (torch.stack([x[p, :, s] for p, s in at], 1)[None] for x in clean[1:3])
        alone = (clean[0][b:b + 1], K, V, torch.zeros(1, 1, dtype=torch.int32), torch.tensor([len(keep)]))
        check_rows(alone, o[b:b + 1], lse[b:b + 1])


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("Hq,Hkv,d,page", HEADS)
def test_no_weight_left(dtype, Hq, Hkv, d, page):
    """Tokens are there and every score is -inf: 0 / 0, where an empty sequence gives 0."""
    c = case(6, [300, 0, 1, 3000], Hq, Hkv, d, page, dtype)
    c[0][:, :, 0, 0] = c[0][:, :, 0, 0].abs() + 0.5
    c[1][..., 0] = -INF
    o, lse = run(c)
    assert o[0].isnan().all() and o[2].isnan().all() and o[3].isnan().all()
    assert (o[1] == 0).all() and (lse == -INF).all()


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("Hq,Hkv,d,page", HEADS)
def test_nan_value(dtype, Hq, Hkv, d, page):
    """A NaN in one dimension of one value: that dimension of its key head's rows, and no other."""
    c = case(7, [300, 900], Hq, Hkv, d, page, dtype)
    clean = [t.clone() for t in c]
    for b, n in ((0, 131), (1, 899)):
        p, s = slot(c, b, n)
        c[2][p, 0, s, 7] = NAN
    o, lse = run(c)
    ref, _ = paged_attention(*c)
    assert torch.equal(o.isnan(), ref.isnan())
    assert torch.equal(lse, run(clean)[1])
    full = run(clean)[0]
    assert torch.equal(torch.where(ref.isnan(), full, o), full)


def test_two_layers_agree():
    """The hybrid's softmax layer in its two forms, on the same tokens: NaN where a key is NaN, in both."""
    g = torch.Generator().manual_seed(8)
    T, H, d = 256, 2, 128
    q, k, v = (torch.randn(1, H, T, d, generator=g).to(BF16).cuda() for _ in range(3))
    k[0, 1, 100, 5] = NAN
    o1, _ = la.softmax_segment_fwd(q[:, :, -1:].contiguous(), k, v, want_lse=True)
    pages = lambda x: x.view(H, T // 64, 64, d).transpose(0, 1).contiguous()  # noqa: E731
    o2, _ = la.paged_decode(q[:, :, -1:].contiguous(), pages(k[0]), pages(v[0]),
                            torch.arange(T // 64, dtype=torch.int32, device="cuda")[None],
                            torch.tensor([T], dtype=torch.int32, device="cuda"))
    assert torch.equal(o1.isnan(), o2.isnan()) and o2[0, 1].isnan().all() and not o2[0, 0].isnan().any()
    assert math.isfinite(float(o2[0, 0].float().norm()))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_append_status_is_this_call_s(dtype):
    """The status word tells of this call alone, also when the call has no tokens."""
    kc, vc = (torch.zeros(3, 2, 16, 64, dtype=dtype, device="cuda") for _ in range(2))
    k = torch.ones(1, 2, 4, 64, dtype=dtype, device="cuda")
    bad, good = (torch.tensor([[i]], dtype=torch.int32, device="cuda") for i in (9, 1))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    status = torch.full((3,), 5, dtype=torch.int32, device="cuda")[1:2]   # a word of its own, 4-byte aligned
    for table, T, want in ((bad, 4, la.ERR_INVALID), (bad, 0, la.OK), (bad, 1, la.ERR_INVALID), (good, 1, la.OK)):
        la.paged_append(k[:, :, :T], k[:, :, :T], kc, vc, table, zero, device_status=status)
        assert int(status) == want, (T, int(status))
    assert (kc[1, :, 0] == 1).all() and int((kc != 0).sum()) == 2 * 64
