"""Decoding over the 8-bit cache where the softmax concentrates: what few tokens leave to the others must reach the output."""
import math

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


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def sink_case(seed, dtype, d, rows, tokens, items, sink, value, spread):
    """`items` items of `tokens` tokens (all sequences on the same pages, with queries of their own): the first token's score is
    `sink` nats above the mean of the others', whose deviation is `spread`; its value is `value` times the others' size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    Hkv, page = 2, 64
    B, blocks = -(-items // Hkv), -(-tokens // page)
    k, v = rn(blocks, Hkv, page, d).clamp(-4, 4), (rn(blocks, Hkv, page, d) * 60).clamp(-448, 448)
    k[..., 0] = 0
    k[0, :, 0] = 0
    k[0, :, 0, 0] = sink
    v[0, :, 0] *= value
    scales = torch.ones(blocks, Hkv, page // 16, 2, device="cuda")
    scales[..., 1] = 2.0 ** -6
    q = rn(B, Hkv * rows, 1, d) * (spread / math.sqrt(d - 1))
    q[..., 0] = 1
    table = torch.randperm(blocks, generator=torch.Generator().manual_seed(seed)).cuda()
    kc, vc = torch.empty_like(k), torch.empty_like(v)
    kc[table], vc[table] = k, v
    return [q.to(dtype), kc.to(E4M3), vc.to(E4M3), scales, table.int().expand(B, blocks).contiguous(),
            torch.full((B,), tokens, dtype=torch.int32, device="cuda")]


def check(c, scale=1.0, tol=ref.tolerance):
    q, kc, vc, sc, table, lens = c
    o, lse = la.paged_decode_q8(*c, scale=scale, want_lse=True)
    ro, rl, bound = ref.attention(*c, scale=scale)
    to, tl = tol(q.dtype, q.shape[-1], int(lens.max()), bound)
    off = (o.double() - ro).abs() - to(ro)
    assert bool((off <= 0).all()), (float(off.max()), float(((o.double() - ro).abs() / bound[0].clamp(min=1e-300)).max()))
    assert bool(((lse.double() - rl).abs() <= tl + 2.0 ** -23 * rl.abs()).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [4, 8, 16])
@pytest.mark.parametrize("sink,value,spread", [(8, 1.0, 1.0), (11, 0.02, 1.0), (14, 0.0, 0.5), (14, 0.02, 0.0), (15, 0.0, 1.0),
                                               (18, 0.0, 0.5)])
def test_sinks(dtype, d, rows, sink, value, spread):
    """A first token that takes most of the mass and has a small value, in pieces of 64 tiles and more."""
    tokens, items = 9000, 2 * 2 * sms()
    assert max(map(max, ref.pieces([tokens] * (items // 2), 2 * rows, 2, 1, dtype, sms()))) >= 64
    check(sink_case(rows + sink, dtype, d, rows, tokens, items, sink, value, spread))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rows", [(64, 4), (128, 4), (64, 8), (128, 8), (64, 16), (128, 16)])
@pytest.mark.parametrize("larger", [4, 8, 14, 20, 40])
@pytest.mark.parametrize("sink,block", [(0, 0), (11, 3), (11, 70), (0, 561)])
def test_large_values_without_weight(dtype, d, rows, larger, sink, block):
    """A block of values 2^larger times the others' at tokens of a weight of e^-30 (the first block of a piece, one of its first
    tile, one further on, the last one) costs the other tokens nothing."""
    c = sink_case(rows + larger, dtype, d, rows, 9000, 2 * 2 * sms(), sink, 0.02, 1.0)
    page, slot = c[4][0, block // 4].long(), block % 4
    c[1][page, :, slot * 16:slot * 16 + 16, 0] = torch.tensor(-30.0).to(E4M3)
    c[3][page, :, slot, 1] *= 2.0 ** larger
    check(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,T", [(2, 2), (2, 4), (2, 8), (4, 8)])
@pytest.mark.parametrize("larger", [10, 30])
def test_large_values_not_seen(dtype, d, Hq, T, larger):
    """The last token's value, alone in its block and 2^larger times the others', reaches the last row and no other."""
    q, kc, vc, sc, table, lens = sink_case(T, dtype, d, 1, 2001, 80, 8, 0.02, 1.0)
    q = torch.randn(len(lens), Hq, T, d, generator=torch.Generator().manual_seed(T)).cuda().to(dtype)
    sc[table[0, 2000 // 64].long(), :, 2000 % 64 // 16, 1] *= 2.0 ** larger
    check((q, kc, vc, sc, table, lens), scale=d ** -0.5)
