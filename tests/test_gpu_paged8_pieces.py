"""Decoding over the 8-bit cache where a CTA's range is long: pieces of up to 70 tiles (rings, scales, score and output buffers used
again and again, references that move inside a piece), and more pieces than a CTA keeps published at once."""
import pytest
import torch

import chunked_state_scan_causal_gb300 as la
import paged8_long as ref

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_state_scan_causal_gb300 import build
    build.build()


def ranges(rows, dtype):
    """CTAs of a decode with so many rows of a key head."""
    n = torch.cuda.get_device_properties(0).multi_processor_count
    return n * (2 if dtype == F32 else 4 if rows <= 4 else 3 if rows <= 8 else 2)


def batch(seed, lens, count, Hq, d, T, dtype, page, keys, vals, Hkv=1):
    """`count` sequences with queries of their own over len(lens) documents (of their lengths) in turn.  keys, vals: by how much the
    scales of keys (all scores positive, times up to 16) and values (2^20) rise (1) or fall (-1) along a document."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    D, blocks = len(lens), max(1, -(-max(lens) // page))
    pages = D * blocks + 1
    kc, vc = (rn(pages, Hkv, page, d) * 60).clamp(-448, 448), (rn(pages, Hkv, page, d) * 60).clamp(-448, 448)
    q = rn(count, Hq, T, d).to(dtype)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[: D * blocks].view(D, blocks).cuda()
    scales = torch.full((pages, Hkv, page // 16, 2), 2.0 ** -6, device="cuda")
    for j, n in enumerate(lens):
        at = (torch.arange(blocks * page // 16, device="cuda") / max(1, n / 16)).clamp(max=1)  # 0 .. 1 along the document
        up = lambda s, top: torch.exp2(top * (at if s > 0 else 1 - at)) if s else torch.ones_like(at)  # noqa: E731
        both = torch.stack((2.0 ** -7 * up(keys, 4.0), 1.3 * 2.0 ** -16 * up(vals, 20.0)), -1)
        scales[table[j]] = both.view(blocks, 1, page // 16, 2).expand(-1, Hkv, -1, -1)
        # what the length does not cover: NaN codes, and NaN scales of blocks that it does not reach
        for i in range(n // page, blocks):
            used = max(0, min(page, n - i * page))
            kc[table[j, i], :, used:], vc[table[j, i], :, used:] = float("nan"), float("nan")
            scales[table[j, i], :, -(-used // 16):] = float("nan")
    if keys:
        q, kc = q.abs(), kc.abs()
    pick = torch.arange(count) % D
    return [q, kc.to(E4M3), vc.to(E4M3), scales, table.int()[pick.cuda()].contiguous(),
            torch.tensor(lens, dtype=torch.int32)[pick].cuda()]


def check(c):
    q, kc, vc, sc, table, lens = c
    o, lse = la.paged_decode_q8(*c, want_lse=True)
    again, lse2 = la.paged_decode_q8(*c, want_lse=True)
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    # (the codes and scales behind a length are no part of the definition)
    ro, rl, bound = ref.attention(q, kc.float().nan_to_num(0.0), vc.float().nan_to_num(0.0), sc.nan_to_num(1.0), table, lens)
    to, tl = ref.tolerance(q.dtype, q.shape[-1], int(lens.max()), bound)
    off = (o.double() - ro).abs() - to(ro)
    assert bool((off <= 0).all()), float(off.max())
    live = rl.isfinite()
    assert torch.equal(lse.isfinite(), live) and not o[~live].any()
    assert bool(((lse.double() - rl).abs() <= tl + 2.0 ** -23 * rl.abs())[live].all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,page", [(64, 48), (128, 64)])
@pytest.mark.parametrize("Hq,T", [(4, 1), (2, 2), (8, 1), (2, 8), (5, 3), (40, 1)])
@pytest.mark.parametrize("tiles", [3, 9, 20, 70])
def test_long_pieces(dtype, d, page, Hq, T, tiles):
    rows = Hq * T
    count = -(-ranges(rows, dtype) // -(-rows // ref.ROWS))
    lens = [tiles * 128 - 37 * j for j in range(3)]
    got = ref.pieces([lens[i % 3] for i in range(count)], Hq, 1, T, dtype, torch.cuda.get_device_properties(0).multi_processor_count)
    assert max(map(max, got)) >= tiles * 3 // 4
    for keys, vals in ((0, 0), (1, -1), (-1, 1), (1, 1)):
        check(batch(tiles + rows, lens, count, Hq, d, T, dtype, page, keys, vals))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
@pytest.mark.parametrize("Hq,T", [(4, 1), (8, 1), (4, 4), (2, 1)])
def test_many_pieces(dtype, d, page, Hq, T):
    """More than 16 sequences of one tile for every CTA, some of them empty, with long ones among them."""
    count = ranges(Hq * T, dtype) * 24
    lens = [100, 1, 128, 0, 77, 16, 127, 3, 50, 0, 128, 99]
    got = ref.pieces([lens[i % 12] for i in range(count)], Hq, 1, T, dtype, torch.cuda.get_device_properties(0).multi_processor_count)
    assert min(map(len, got)) > 16
    check(batch(1, lens, count, Hq, d, T, dtype, page, 0, 0))
    lens = lens[:11] + [700]
    got = ref.pieces([lens[i % 12] for i in range(count // 2)], Hq, 1, T, dtype, torch.cuda.get_device_properties(0).multi_processor_count)
    assert max(map(len, got)) >= 9 and max(map(max, got)) >= 6
    check(batch(2, lens, count // 2, Hq, d, T, dtype, page, 1, -1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,T", [(8, 2, 1), (32, 4, 1), (6, 3, 4)])
def test_ragged(dtype, Hq, Hkv, T):
    """Documents from nothing to 70 tiles in one batch, several key heads."""
    lens = [8960, 0, 5, 3000, 129, 8000, 1, 640, 128, 4097]
    check(batch(3, lens, 200, Hq, 128, T, dtype, 80, 1, 1, Hkv))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,T", [(4, 1), (8, 1), (4, 4)])
def test_not_a_number_in_long_pieces(dtype, Hq, T):
    """NaN scores of a whole first tile, of a token further on, and a NaN value: the rows (or the dimension) that see them are NaN, and
    nothing else is."""
    count = ranges(Hq * T, dtype)
    c = batch(5, [2000, 2000, 2000, 2000], count, Hq, 64, T, dtype, 128, 0, 0)
    q, kc, vc, sc, table, lens = c
    raw = lambda x, doc, n: x.view(torch.uint8)[table[doc, n // 128].long(), 0, n % 128]  # noqa: E731
    for n in range(128):
        raw(kc, 0, n)[5] = 0x7f
    raw(kc, 1, 1500)[0] = 0xff
    raw(vc, 2, 900)[7] = 0x7f
    o, lse = la.paged_decode_q8(*c, want_lse=True)
    bad = torch.zeros_like(o, dtype=torch.bool)
    doc = torch.arange(count, device="cuda") % 4
    bad[(doc == 0) | (doc == 1)] = True
    bad[..., 7] |= (doc == 2)[:, None, None]
    assert torch.equal(o.isnan(), bad) and o[~bad].isfinite().all()
    assert torch.equal(lse.isnan(), ((doc == 0) | (doc == 1))[:, None, None].expand_as(lse))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,T", [(4, 1), (8, 1), (16, 1), (2, 2)])
@pytest.mark.parametrize("power", [-126, -90, 60, 105])
def test_value_scales_of_any_size(dtype, Hq, T, power):
    """Values of the smallest and of very large scales; and a first tile whose values are all zero (their scale is the smallest)
    before ordinary ones."""
    lens = [700, 90, 333]
    c = batch(6, lens, 60, Hq, 128, T, dtype, 64, 0, 0)
    c[3][..., 1] = 2.0 ** power
    # r is at most 2^120: a row's largest weight is 2^-6 at a scale of 2^-126, and its smallest step 2^-19 of that
    ro, rl, (A, X, M, C) = ref.attention(c[0], c[1].float().nan_to_num(0.0), c[2].float().nan_to_num(0.0), c[3].nan_to_num(1.0), *c[4:])
    to, _ = ref.tolerance(dtype, 128, 700, (A, X, M * 2.0 ** 17, C))
    o, _ = la.paged_decode_q8(*c)
    assert bool(((o.double() - ro).abs() <= to(ro)).all())
    c = batch(7, lens, 60, Hq, 128, T, dtype, 64, 0, 0)
    for j in range(3):
        at = c[4][j, :2].long()
        c[2].view(torch.uint8)[at] = 0
        c[3][at, ..., 1] = 2.0 ** -126
    check(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,T", [(4, 1), (8, 1), (16, 1)])
@pytest.mark.parametrize("size", [20, 30, 60])
@pytest.mark.parametrize("power", [-60, 0, 60])
def test_one_token_takes_all(dtype, Hq, T, size, power):
    """Scores so far apart that one token has all the weight: o is its value, whatever its scale is beside the others'."""
    g = torch.Generator().manual_seed(size)
    n, page, d = 1000, 128, 64
    kc = torch.ones(8, 1, page, d)
    kc[..., 0] = torch.tensor([1.0, 2.0, 4.0, 8.0])[torch.randint(0, 4, (8, 1, page), generator=g)]
    kc[5, 0, 77, 0] = 64.0
    vc = (torch.randn(8, 1, page, d, generator=g) * 60).clamp(-448, 448).to(E4M3)
    sc = torch.ones(8, 1, page // 16, 2)
    sc[5, 0, 77 // 16, 1] = 2.0 ** power
    q = torch.zeros(3, Hq, T, d, dtype=dtype)
    q[..., 0] = 2.0 ** size
    table = torch.arange(8, dtype=torch.int32).expand(3, 8).contiguous()
    o, lse = la.paged_decode_q8(q.cuda(), kc.to(E4M3).cuda(), vc.cuda(), sc.cuda(), table.cuda(),
                                torch.full((3,), n, dtype=torch.int32, device="cuda"), scale=1.0, want_lse=True)
    want = (vc[5, 0, 77].double() * 2.0 ** power).cuda()
    assert bool(((o.double() - want).abs() <= torch.finfo(dtype).eps * want.abs()).all())
    assert bool(((lse.double() / (64 * 2.0 ** size) - 1).abs() <= 2.0 ** -21).all())
