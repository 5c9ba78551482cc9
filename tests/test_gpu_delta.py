"""The gated delta rule (fwd_delta / bwd_delta / decode_delta) against its 64-bit recurrence.

Tolerances are on ||got - ref|| / ||ref||.
  fp32 inputs: every value is a chain of fp32 sums of at most d + T terms; each term is rounded by at most 2^-24
    relative, so (d + T) 2^-24 with d + T <= 512 gives 3.1e-5.
  bf16 inputs, bf16 outputs: the output's own rounding and at most three roundings of operands to bf16 lie on the way
    to a value.  Each is at most 2^-8 relative, 2^-8 / sqrt(3) = 2.3e-3 in the mean square; added as if they all
    agreed: 9.1e-3.  The log-gate's gradient is a difference of three such values: 2.8e-2 when those agree in size.
  bf16 inputs, fp32 states: operands in two bf16 parts leave 2^-16 relative each, four on the way: 6.2e-5.
"""
import pytest
import torch

import chunked_state_scan_causal_gb300 as la
from delta_ref import delta_backward, delta_forward, rel

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
TOL = {torch.float32: dict(out=3.1e-5, gate=3.1e-5, state=3.1e-5), BF16: dict(out=9.1e-3, gate=2.8e-2, state=6.2e-5)}


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_state_scan_causal_gb300 import build
    build.build()


def case(seed, B, H, T, d, dtype, gate=None, decay=0.3):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    k = rn(B, H, T, d)
    c = dict(q=rn(B, H, T, d) / d ** 0.5, k=k / k.norm(dim=-1, keepdim=True), v=rn(B, H, T, d), dO=rn(B, H, T, d))
    c = {n: x.to(dtype) for n, x in c.items()}
    gate = gate or dtype
    c["lg"] = (-decay * torch.rand(B, H, T, generator=g)).to(gate)
    c["beta"] = torch.sigmoid(rn(B, H, T)).to(gate)
    c["init"], c["D"] = rn(B, H, d, d) / d ** 0.5, rn(B, H, d, d) / d ** 0.5
    return c


def run(c, lg=True, init=True, D=True, place=lambda x: x.cuda()):
    """(o, final, dq, dk, dv, dlg, dbeta, dinit) on the GPU; `place` puts the sequence tensors there."""
    q, k, v, dO = (place(c[n]) for n in ("q", "k", "v", "dO"))
    gl, gb = c["lg"].cuda() if lg else None, c["beta"].cuda()
    i, d = c["init"].cuda() if init else None, c["D"].cuda() if D else None
    ck = la.checkpoint_delta(q)
    ws = la.workspace(q, la.OP_FWD_DELTA)
    o, fin = la.fwd_delta(q, k, v, gl, gb, init_state=i, want_final=True, ckpt=ck, ws=ws)
    ws2 = la.workspace(q, la.OP_BWD_DELTA)
    outs = la.bwd_delta(q, k, v, dO, gl, gb, ck, init_state=i, d_final=d, want_dinit=True, ws=ws2)
    assert la.device_status(ws) == la.OK and la.device_status(ws2) == la.OK
    return (o, fin, *outs)


def check(c, got, lg=True, init=True, D=True):
    i, d = c["init"] if init else None, c["D"] if D else None
    gl = c["lg"] if lg else None
    o, fin, _, _ = delta_forward(c["q"], c["k"], c["v"], gl, c["beta"], i)
    grads = delta_backward(c["q"], c["k"], c["v"], c["dO"], gl, c["beta"], i, d)
    tol = TOL[c["q"].dtype]
    # gates in fp32 beside bf16 sequences: their gradients come from the same bf16 products
    names = ("o", "final", "dq", "dk", "dv", "dlg", "dbeta", "dinit")
    kinds = ("out", "state", "out", "out", "out", "gate", "gate", "state")
    errs = {}
    for n, kind, x, r in zip(names, kinds, got, (o, fin, *grads)):
        if n == "dlg" and not lg:
            assert x is None
            continue
        errs[n] = rel(x, r)
        assert errs[n] < tol[kind], (n, errs[n], tol[kind], errs)


@pytest.mark.parametrize("T", [1, 2, 7, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("d,dtype", [(64, torch.float32), (128, torch.float32), (64, BF16), (128, BF16)])
def test_lengths(d, dtype, T):
    c = case(T + d, 1, 2, T, d, dtype)
    check(c, run(c))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("lg,init,D", [(False, False, False), (True, False, True), (False, True, False),
                                       (True, True, False)])
def test_optional_operands(dtype, lg, init, D):
    c = case(5, 2, 3, 150, 128, dtype)
    check(c, run(c, lg, init, D), lg, init, D)


@pytest.mark.parametrize("dtype,gate", [(BF16, torch.float32), (torch.float32, BF16)])
def test_gate_types(dtype, gate):
    """Gates of the other type; their gradients have it too."""
    c = case(6, 1, 2, 100, 128, dtype, gate)
    got = run(c)
    assert got[5].dtype == gate and got[6].dtype == gate
    if gate == BF16:  # the gradients' own rounding
        o, fin, _, _ = delta_forward(c["q"], c["k"], c["v"], c["lg"], c["beta"], c["init"])
        grads = delta_backward(c["q"], c["k"], c["v"], c["dO"], c["lg"], c["beta"], c["init"], c["D"])
        assert rel(got[0], o) < 3.1e-5 and rel(got[3], grads[1]) < 3.1e-5
        for x, r in zip(got[5:7], grads[3:5]):
            assert rel(x, r) < 2 ** -8 + 3.1e-5
    else:
        check(c, got)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_strong_decay_and_zero_strengths(dtype):
    """Log-gates down to -100 a token (the state is wiped: factors underflow, nothing overflows), exact zeros among
    the strengths (their gradient is not zero) and strengths of one."""
    c = case(7, 1, 2, 130, 128, dtype)
    c["lg"] = c["lg"].clone()
    c["lg"][:, 0, 10:20] = -100.0
    c["lg"][:, 1] = -3.0
    c["beta"] = c["beta"].clone()
    c["beta"][:, :, 5::9] = 0.0
    c["beta"][:, :, 6::9] = 1.0
    check(c, run(c))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_repeated_keys(dtype):
    """One key for a whole chunk, strengths of one, no decay: every write replaces the last one's value."""
    c = case(8, 1, 1, 96, 64, dtype)
    c["k"] = c["k"][:, :, :1].expand_as(c["k"]).contiguous()
    c["beta"] = torch.ones_like(c["beta"])
    o, fin, _, _ = delta_forward(c["q"], c["k"], c["v"], None, c["beta"], c["init"])
    got = run(c, lg=False)
    assert rel(got[0], o) < TOL[dtype]["out"] and rel(got[1], fin) < TOL[dtype]["state"]


@pytest.mark.parametrize("B,H,T,d", [(2, 20, 200, 128), (5, 16, 70, 64), (1, 160, 65, 128)])
def test_many_heads(B, H, T, d):
    """More (batch, head, slice)s than the GPU has SMs: the wider slices, and several waves of them."""
    c = case(15, B, H, T, d, BF16)
    check(c, run(c))


def test_longer_bf16():
    c = case(9, 1, 3, 1000, 128, BF16, decay=0.05)
    check(c, run(c))


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, BF16), (128, torch.float32)])
def test_strides(d, dtype):
    """[B, T, H, d] order and rows longer than d, outputs in the inputs' layout and nothing written between rows."""
    c = case(10, 2, 2, 70, d, dtype)

    def place(x):
        buf = torch.full((2, 70, 2, d + 16), 7.0, dtype=dtype, device="cuda")
        view = buf[..., :d].permute(0, 2, 1, 3)
        view.copy_(x)
        return view
    check(c, run(c, place=place))
    q = place(c["q"])
    outs = [place(torch.zeros_like(c["q"])) for _ in range(4)]
    ck = la.checkpoint_delta(q)
    gl, gb = c["lg"].cuda(), c["beta"].cuda()
    k, v, dO = (place(c[n]) for n in ("k", "v", "dO"))
    la.fwd_delta(q, k, v, gl, gb, ckpt=ck, out=outs[0])
    la.bwd_delta(q, k, v, dO, gl, gb, ck, outs=outs[1:])
    for x in outs:
        rows = x.permute(0, 2, 1, 3).as_strided((2, 70, 2, 16), x.permute(0, 2, 1, 3).stride(), x.storage_offset() + d)
        assert (rows == 7.0).all()


def test_empty_sequence():
    for dtype in (torch.float32, BF16):
        q = torch.zeros(1, 2, 0, 64, device="cuda", dtype=dtype)
        g = torch.zeros(1, 2, 0, device="cuda")
        S, D = torch.randn(1, 2, 64, 64, device="cuda"), torch.randn(1, 2, 64, 64, device="cuda")
        ck = la.checkpoint_delta(q)
        o, fin = la.fwd_delta(q, q, q, g, g, init_state=S, want_final=True, ckpt=ck)
        *_, dinit = la.bwd_delta(q, q, q, q, g, g, ck, init_state=S, d_final=D, want_dinit=True)
        assert o.numel() == 0 and torch.equal(fin, S) and torch.equal(dinit, D)


@pytest.mark.parametrize("d,dtype,B,T", [(128, BF16, 3, 1), (64, BF16, 1, 1), (128, torch.float32, 2, 4),
                                         (64, torch.float32, 5, 3)])
def test_decode(d, dtype, B, T):
    c = case(11, B, 2, T, d, dtype)
    S = c["init"].cuda()
    o = la.decode_delta(*(c[n].cuda() for n in ("q", "k", "v", "lg", "beta")), S)
    ro, rS, _, _ = delta_forward(c["q"], c["k"], c["v"], c["lg"], c["beta"], c["init"])
    # one rounding of o (2^-8 in bf16); the state is fp32: d + T terms at 2^-24
    assert rel(o, ro) < (2 ** -8 if dtype == BF16 else 3.1e-5)
    assert rel(S, rS) < 3.1e-5


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_prefill_in_pieces_then_decode(dtype):
    """A prompt in two pieces through the state, then tokens one by one: as used when serving."""
    c = case(12, 2, 2, 150, 128, dtype)
    x = {n: c[n].cuda() for n in ("q", "k", "v", "lg", "beta")}
    part = lambda a, b: [x[n][:, :, a:b].contiguous() for n in ("q", "k", "v", "lg", "beta")]  # noqa: E731
    o1, S = la.fwd_delta(*part(0, 90), want_final=True)
    o2, S = la.fwd_delta(*part(90, 147), init_state=S, want_final=True)
    outs = [o1, o2] + [la.decode_delta(*part(t, t + 1), S) for t in range(147, 150)]
    ro, rS, _, _ = delta_forward(c["q"], c["k"], c["v"], c["lg"], c["beta"])
    assert rel(torch.cat(outs, 2), ro) < TOL[dtype]["out"] and rel(S, rS) < TOL[dtype]["state"]


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_graph_and_streams(dtype):
    """Captured and replayed with new inputs, and two calls at once on two streams: bitwise the eager results."""
    c, c2 = case(13, 1, 2, 200, 128, dtype), case(14, 1, 2, 200, 128, dtype)
    names = ("q", "k", "v", "dO", "lg", "beta")
    x, y = ({n: e[n].cuda() for n in names} for e in (c, c2))

    def step(z, ck, ws, ws2):
        o, _ = la.fwd_delta(z["q"], z["k"], z["v"], z["lg"], z["beta"], ckpt=ck, ws=ws)
        return (o, *la.bwd_delta(z["q"], z["k"], z["v"], z["dO"], z["lg"], z["beta"], ck, ws=ws2)[:5])

    bufs = lambda: (la.checkpoint_delta(x["q"]), la.workspace(x["q"], la.OP_FWD_DELTA),  # noqa: E731
                    la.workspace(x["q"], la.OP_BWD_DELTA))
    want = [[t.clone() for t in step(z, *bufs())] for z in (x, y)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    held = [bufs(), bufs()]
    for s, z, b in zip(streams, (x, y), held):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                r = step(z, *b)
            got.append(r)
    torch.cuda.synchronize()
    for w, r in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, r))
    z = {n: t.clone() for n, t in x.items()}
    b = bufs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step(z, *b)
    for w, src in zip(want, (x, y)):
        for n in names:
            z[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(w, r))


def test_offsets_past_32_bits():
    """Records of more than 2^32 bytes: the same bits as the sequence in two pieces (cut between two chunks)."""
    B, H, T, d = 4, 32, 32832, 128
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough free memory")
    g = torch.Generator(device="cuda").manual_seed(31)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    k = rn(B, H, T, d)
    k = (k / k.norm(dim=-1, keepdim=True)).bfloat16()
    q, v, dO = ((rn(B, H, T, d) * s).bfloat16() for s in (d ** -0.5, 1.0, 1.0))
    beta, lg = torch.rand(B, H, T, generator=g, device="cuda"), -0.1 * torch.rand(B, H, T, generator=g, device="cuda")
    ck = la.checkpoint_delta(q)
    assert ck.numel() > 1 << 32
    o, fin = la.fwd_delta(q, k, v, lg, beta, want_final=True, ckpt=ck)
    grads = la.bwd_delta(q, k, v, dO, lg, beta, ck, want_dinit=True)
    cut, state, pieces = T // 128 * 64, None, []
    for part in (slice(0, cut), slice(cut, T)):
        x = [t[:, :, part] for t in (q, k, v)] + [t[:, :, part].contiguous() for t in (lg, beta)]
        ckp = la.checkpoint_delta(x[0])
        op, nxt = la.fwd_delta(*x, init_state=state, want_final=True, ckpt=ckp)
        assert torch.equal(op, o[:, :, part])
        pieces.append((x, ckp, state, dO[:, :, part], part))
        state = nxt
    assert torch.equal(state, fin)
    D = None
    for x, ckp, init, up, part in reversed(pieces):
        got = la.bwd_delta(*x[:3], up, *x[3:], ckp, init_state=init, d_final=D, want_dinit=True)
        for a, b in zip(got[:5], grads[:5]):
            assert torch.equal(a, b[:, :, part])
        D = got[5]
    assert torch.equal(D, grads[5])


def test_two_graphs_one_workspace():
    """Two captured steps of different shapes that share one workspace and checkpoint, replayed in turn."""
    steps = []
    for B, H, T in ((1, 3, 200), (2, 2, 129)):
        g = torch.Generator(device="cuda").manual_seed(T)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        k = torch.nn.functional.normalize(rn(B, H, T, 128), dim=-1).bfloat16()
        q, v, dO = ((rn(B, H, T, 128) * s).bfloat16() for s in (0.1, 1.0, 1.0))
        beta, lg = torch.rand(B, H, T, generator=g, device="cuda"), -torch.rand(B, H, T, generator=g, device="cuda")
        steps.append((q, k, v, dO, lg, beta))
    sizes = [max(f(s[0]).numel() for s in steps) for f in (
        la.checkpoint_delta, lambda q: la.workspace(q, la.OP_FWD_DELTA), lambda q: la.workspace(q, la.OP_BWD_DELTA))]
    ck, w1, w2 = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes)

    def step(s):
        o, fin = la.fwd_delta(*s[:3], *s[4:], want_final=True, ckpt=ck, ws=w1)
        return (o, fin, *la.bwd_delta(*s, ck, ws=w2, want_dinit=True))

    want = [[t.clone() for t in step(s)] for s in steps]
    graphs, got = [], []
    for s in steps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(step(s))
    for i in (0, 1, 1, 0, 1):
        for t in got[i]:
            t.fill_(7)
        graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_named_stream(dtype):
    """stream=: workspaces and outputs that a call allocates are not handed out again while it still runs."""
    c = {n: x.cuda() for n, x in case(41, 2, 4, 300, 128, dtype).items()}
    seq, gates = (c["q"], c["k"], c["v"]), (c["lg"], c["beta"])
    state = c["init"].clone()

    def steps(**kw):
        ck = la.checkpoint_delta(c["q"])
        o, fin = la.fwd_delta(*seq, *gates, init_state=c["init"], want_final=True, ckpt=ck, **kw)
        grads = la.bwd_delta(*seq, c["dO"], *gates, ck, init_state=c["init"], d_final=c["D"], want_dinit=True, **kw)
        one = [x[:, :, :1] for x in seq] + [x[:, :, :1].contiguous() for x in gates]
        return (o, fin, *grads, la.decode_delta(*one, state, **kw)), ck, one

    want, _, _ = steps()
    state.copy_(c["init"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200000)
    got, *keep = steps(stream=side)
    sizes = {la.workspace(c["q"], op).numel() for op in (la.OP_FWD_DELTA, la.OP_BWD_DELTA)}
    for _ in range(200):
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
