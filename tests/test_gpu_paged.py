"""The paged cache: append and decode against a 64-bit gather.

Tolerances on ||got - ref|| / ||ref||.  fp32: dots of d <= 128 terms and sums of up to n weights, each term rounded by
2^-24: the weights' relative error is the scores' absolute one, (d + 4) 2^-24 |x| with |x| < 8 here, so 8 * 132 * 2^-24
= 6.3e-5.  bf16: the output's rounding, 2^-8, and the weights' rounding to bf16, 2^-8 (both at most): 7.9e-3.
lse: fp32 from exact bf16 products, as fp32 above: 6.3e-5 absolute."""
import pytest
import torch

import chunked_state_scan_causal_gb300 as la
from delta_ref import paged_attention, rel

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
TOL = {torch.float32: 6.3e-5, BF16: 7.9e-3}


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_state_scan_causal_gb300 import build
    build.build()


def case(seed, lens, Hq, Hkv, d, page, dtype, blocks=None, poison=True):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    blocks = blocks or max(1, -(-max(max(lens), 1) // page))
    pages = B * blocks + 3
    table = torch.randperm(pages, generator=g)[: B * blocks].view(B, blocks).to(torch.int32)
    q = torch.randn(B, Hq, 1, d, generator=g).to(dtype)
    kc, vc = (torch.randn(pages, Hkv, page, d, generator=g).to(dtype) for _ in range(2))
    if poison:  # slots that no length covers hold NaN and infinities
        for b, n in enumerate(lens):
            for j in range(blocks):
                used = max(0, min(page, n - j * page))
                kc[table[b, j], :, used:] = float("nan")
                vc[table[b, j], :, used:] = float("inf")
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32)


def run(c, **kw):
    x = [t.cuda() for t in c]
    ws = la.workspace(x[0], la.OP_PAGED_DECODE)
    o, lse = la.paged_decode(*x, want_lse=True, ws=ws, **kw)
    return o, lse, la.device_status(ws)


def check(c, scale=None):
    o, lse, status = run(c, scale=scale or 0.0)
    ro, rl = paged_attention(*c, scale=scale)
    assert status == la.OK
    assert rel(o, ro) < TOL[c[0].dtype]
    live = rl.isfinite()
    assert torch.equal(lse.cpu().isfinite(), live) and (lse.cpu()[~live] == -float("inf")).all()
    assert (o.cpu()[~live[..., 0]] == 0).all()
    if live.any():
        assert float((lse.cpu().double() - rl)[live].abs().max()) < 6.3e-5


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 2), (16, 1), (20, 1), (34, 2)])
def test_heads(dtype, d, Hq, Hkv):
    check(case(1, [1, 130, 0, 77], Hq, Hkv, d, 16, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 128, 200, 256])
def test_page_sizes(dtype, page):
    check(case(2, [5, 128, 129, 300, 64], 4, 2, 128, page, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("lens", [[0], [1], [127], [128], [0, 0, 1, 0], [0, 0], [3000], [5] * 40 + [2000]])
def test_lengths(dtype, lens):
    check(case(3, lens, 4, 2, 128, 32, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_many_short_sequences(dtype):
    check(case(4, [(7 * i) % 40 for i in range(700)], 2, 1, 64, 8, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_long_split_over_all_ctas(dtype):
    check(case(5, [70000], 2, 1, 64, 128, dtype), scale=0.3)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_large_scores(dtype):
    """Scores in the hundreds that grow along the sequence: the running maximum moves at every tile."""
    c = case(6, [1000, 400], 4, 2, 128, 16, dtype, poison=False)
    q, kc, vc, table, lens = c
    q = q.abs()
    kc.copy_(kc.abs() * 0.1)
    for b in range(2):
        for j in range(table.shape[1]):
            kc[table[b, j]] *= 1 + 0.5 * j
    c = (q, kc, vc, table, lens)
    o, lse, _ = run(c)
    ro, rl = paged_attention(*c)
    # scores up to 300: their fp32 rounding, 132 * 2^-24 * 300, is the weights' relative error
    assert rel(o, ro) < TOL[dtype] + 2.4e-3 and rel(lse, rl) < 132 * 2 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_layouts(dtype):
    """[pages, page, H, d] caches, rows longer than d, a table that is a slice, q and o in [B, 1, H, d] order."""
    q, kc, vc, table, lens = case(7, [90, 33, 150], 8, 4, 64, 16, dtype)
    ro, rl = paged_attention(q, kc, vc, table, lens)

    def pack(x):
        buf = torch.zeros(x.shape[0], x.shape[2], x.shape[1], 64 + 8, dtype=dtype, device="cuda")
        view = buf[..., :64].permute(0, 2, 1, 3)
        view.copy_(x)
        return view
    wide = torch.full((3, table.shape[1] + 5), -5, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = table.cuda()
    qq = q.cuda().permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    o, lse = la.paged_decode(qq, pack(kc), pack(vc), wide[:, 2:2 + table.shape[1]], lens.cuda(), want_lse=True)
    assert o.stride() == qq.stride() and rel(o, ro) < TOL[dtype]


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_bad_pages_and_lengths(dtype):
    """Ids outside the cache are absent tokens and are reported; lengths are clamped to the table."""
    q, kc, vc, table, lens = case(8, [100, 60, 40, 300], 4, 2, 128, 16, dtype, poison=False)
    table[0, 2], table[1, 0], table[2, :] = -1, kc.shape[0], 1 << 30
    c = (q, kc, vc, table, torch.tensor([100, 60, 40, 100000], dtype=torch.int32))
    o, lse, status = run(c)
    ro, rl = paged_attention(*c)
    assert status == la.ERR_INVALID
    assert rel(o, ro) < TOL[dtype] and (lse[2].cpu() == -float("inf")).all() and (o[2] == 0).all()
    c = (q, kc, vc, table, torch.tensor([-3, 0, -(1 << 31), 20], dtype=torch.int32))
    o, lse, status = run(c)
    assert status == la.OK and rel(o, paged_attention(*c)[0]) < TOL[dtype]


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("page,T", [(16, 1), (1, 5), (24, 40), (128, 300)])
def test_append(dtype, page, T):
    B, H, d, blocks = 4, 2, 64, -(-(50 + T) // page)
    g = torch.Generator().manual_seed(9)
    pages = B * blocks + 2
    table = torch.randperm(pages, generator=g)[: B * blocks].view(B, blocks).to(torch.int32)
    kc, vc = (torch.randn(pages, H, page, d, generator=g).to(dtype) for _ in range(2))
    k, v = (torch.randn(B, T, H, d, generator=g).to(dtype).transpose(1, 2) for _ in range(2))
    start = torch.tensor([0, 50, 13, 7], dtype=torch.int32)
    new = torch.tensor([T, 0, -2, T // 2], dtype=torch.int32)
    for lens in (None, new):
        gk, gv = kc.cuda(), vc.cuda()
        status = torch.full((4,), 9, dtype=torch.int32, device="cuda")
        la.paged_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), start.cuda(),
                        new_lens=None if lens is None else lens.cuda(), device_status=status)
        wk, wv = kc.clone(), vc.clone()
        for b in range(B):
            for t in range(T if lens is None else max(0, int(lens[b]))):
                n = int(start[b]) + t
                wk[table[b, n // page], :, n % page] = k[b, :, t]
                wv[table[b, n // page], :, n % page] = v[b, :, t]
        assert torch.equal(gk.cpu(), wk) and torch.equal(gv.cpu(), wv) and int(status[0]) == la.OK


def test_append_outside():
    """Positions outside the table and bad page ids are reported and written nowhere."""
    k = torch.randn(3, 1, 4, 64, device="cuda")
    kc, vc = torch.zeros(5, 1, 2, 64, device="cuda"), torch.zeros(5, 1, 2, 64, device="cuda")
    table = torch.tensor([[0, 1], [2, 5], [-1, 4]], dtype=torch.int32, device="cuda")
    start = torch.tensor([2, 0, -1], dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    la.paged_append(k, k, kc, vc, table, start, device_status=status)
    want = torch.zeros_like(kc)
    want[1, 0], want[2, 0] = k[0, 0, :2], k[1, 0, :2]
    assert int(status[0]) == la.ERR_INVALID and torch.equal(kc, want) and torch.equal(vc, want)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_serving_steps_captured(dtype):
    """Prompts appended as a padded batch, then decode steps (append, attend) in one captured graph whose lengths
    move on the device."""
    B, Hq, Hkv, d, page, blocks = 3, 4, 2, 128, 16, 8
    g = torch.Generator().manual_seed(10)
    rn = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    plen, steps = torch.tensor([50, 1, 17], dtype=torch.int32), 6
    K, V, Q = rn(B, Hkv, 60, d), rn(B, Hkv, 60, d), rn(B, Hq, steps, d)
    table = torch.randperm(B * blocks, generator=g).view(B, blocks).to(torch.int32)
    kc, vc = (torch.full((B * blocks, Hkv, page, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    tab, n = table.cuda(), plen.cuda()
    la.paged_append(K[:, :, :50].cuda(), V[:, :, :50].cuda(), kc, vc, tab, zero, new_lens=n)
    k1, v1, q1 = (torch.zeros(B, h, 1, d, dtype=dtype, device="cuda") for h in (Hkv, Hkv, Hq))
    ws = la.workspace(q1, la.OP_PAGED_DECODE)
    out = torch.empty_like(q1)
    lens = n.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.paged_append(k1, v1, kc, vc, tab, lens)
        lens.add_(1)
        la.paged_decode(q1, kc, vc, tab, lens, out=out, ws=ws)
    for s in range(steps):
        at = (plen.long() + s)[:, None, None, None]
        k1.copy_(K.gather(2, at.expand(B, Hkv, 1, d)))
        v1.copy_(V.gather(2, at.expand(B, Hkv, 1, d)))
        q1.copy_(Q[:, :, s:s + 1])
        graph.replay()
        for b in range(B):
            m = int(plen[b]) + s + 1
            kk, vv = (x[b].repeat_interleave(Hq // Hkv, 0)[:, :m].double() for x in (K, V))
            p = torch.softmax((kk @ Q[b, :, s, :, None].double())[..., 0] * d ** -0.5, -1)
            assert rel(out[b, :, 0], (p[:, None] @ vv)[:, 0]) < TOL[dtype]
    assert torch.equal(lens.cpu(), plen + steps)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_repeatable_and_concurrent(dtype):
    """Two calls at once with their own workspaces, and the same call again: the same bits."""
    c = [t.cuda() for t in case(11, [900, 40, 3000], 8, 2, 128, 64, dtype)]
    want = la.paged_decode(*c, want_lse=True)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got += [la.paged_decode(*c, want_lse=True) for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_offsets_past_32_bits(dtype):
    """A cache of more than 2^31 elements, its last pages in use."""
    pages, Hq, Hkv, page, d = 66000, 8, 4, 64, 128
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * pages * Hkv * page * d * torch.finfo(dtype).bits // 8:
        pytest.skip("not enough free memory")
    kc, vc = (torch.empty(pages, Hkv, page, d, dtype=dtype, device="cuda") for _ in range(2))
    assert kc.numel() > 1 << 31
    q, sk, sv, small, lens = case(12, [250, 130], Hq, Hkv, d, page, dtype, poison=False)
    far = (pages - 1 - small.long() * 7).to(torch.int32)
    K, V = (torch.stack([c[small[b].long()].transpose(0, 1).reshape(Hkv, -1, d) for b in range(2)]) for c in (sk, sv))
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    la.paged_append(K.cuda(), V.cuda(), kc, vc, far.cuda(), zero, new_lens=lens.cuda())
    o, lse = la.paged_decode(q.cuda(), kc, vc, far.cuda(), lens.cuda(), want_lse=True)
    ro, rl = paged_attention(q, sk, sv, small, lens)
    assert rel(o, ro) < TOL[dtype] and float((lse.cpu().double() - rl).abs().max()) < 6.3e-5


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_shared_pages(dtype):
    """Sequences with a common prefix of pages, and a page twice in one sequence."""
    q, kc, vc, table, lens = case(13, [300, 290, 64, 7], 8, 2, 128, 32, dtype, poison=False)
    table[1, :6], table[2, 1], table[3] = table[0, :6], table[2, 0], table[0]
    check((q, kc, vc, table, lens))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_named_stream(dtype):
    """stream=: the workspace that a call allocates is not handed out again while it still runs."""
    c = [t.cuda() for t in case(14, [5000, 300], 8, 2, 128, 64, dtype, poison=False)]
    k = c[1][0, :, :1][None].expand(2, -1, -1, -1).contiguous()
    side = torch.cuda.Stream()

    def step(**kw):
        la.paged_append(k, k, c[1], c[2], c[3], c[4] - 1, **kw)
        return la.paged_decode(*c, want_lse=True, **kw)

    want, last = step(), c[4] - 1
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200000)
    la.paged_append(k, k, c[1], c[2], c[3], last, stream=side)
    got = la.paged_decode(*c, want_lse=True, stream=side)
    n = la.workspace(c[0], la.OP_PAGED_DECODE).numel()
    for _ in range(200):
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
