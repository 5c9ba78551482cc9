"""The gated delta rule's gradients and states beyond single short sequences."""
import pytest
import torch

import chunked_state_scan_causal_gb300 as la
from delta_ref import delta_backward, delta_forward, rel

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_state_scan_causal_gb300 import build
    build.build()


def inputs(seed, B, H, T, d, dtype, gate, decay, device="cpu"):
    """q, k, v, dO, log-gates and strengths."""
    g = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    k = rn(B, H, T, d)
    seq = (rn(B, H, T, d) / d ** 0.5, k / k.norm(dim=-1, keepdim=True), rn(B, H, T, d), rn(B, H, T, d))
    lg = -decay * torch.rand(B, H, T, generator=g, device=device)
    return [x.to(dtype) for x in seq] + [lg.to(gate), torch.sigmoid(rn(B, H, T)).to(gate)]


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_repeat_over_many_chunks(d):
    """Many chunks for every CTA of the gradient kernel: each call gives the same bits."""
    q, k, v, dO, lg, beta = inputs(1, 2, 20, 2560, d, BF16, torch.float32, 0.1, "cuda")
    ck = la.checkpoint_delta(q)
    la.fwd_delta(q, k, v, lg, beta, ckpt=ck)
    want = la.bwd_delta(q, k, v, dO, lg, beta, ck)[:5]
    for _ in range(10):
        for a, b in zip(la.bwd_delta(q, k, v, dO, lg, beta, ck)[:5], want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, BF16), (64, torch.float32)])
def test_checkpointed_forward_needs_no_workspace(d, dtype):
    """A training forward allocates its output and 256 bytes, and gives the bits of the one without a checkpoint."""
    q, k, v, dO, lg, beta = inputs(2, 1, 3, 300, d, dtype, torch.float32, 0.1, "cuda")
    want, fin = la.fwd_delta(q, k, v, lg, beta, want_final=True)
    ck = la.checkpoint_delta(q)
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    o, _ = la.fwd_delta(q, k, v, lg, beta, ckpt=ck)
    assert torch.cuda.max_memory_allocated() - held <= o.numel() * o.element_size() + 1024
    assert torch.equal(o, want)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    o, f = la.fwd_delta(q, k, v, lg, beta, want_final=True, ckpt=ck, ws=ws)
    assert torch.equal(o, want) and torch.equal(f, fin) and la.device_status(ws) == la.OK


# Independent roundings of b bits leave 2^-b / sqrt(3) in the mean square at most (2.3e-3 in bf16).  A gradient has its
# own rounding and at most three operands' on the way: sqrt(4) 2.3e-3 = 4.5e-3.  A log-gate's gradient is the sum of three
# values (<R, S>, q . dq, k . dk) made of products of two rounded operands, sqrt(3 x 2) 2.3e-3, and its own rounding:
# sqrt(7) 2.3e-3 = 6.0e-3.  The output has its own rounding, 2^-8 at most, and operands in two parts, 2^-16 each: eight of
# them, 1.2e-4.  States: four of those, 6.2e-5, whatever the length, since a step takes from an error as from the state
# (beta |k|^2 <= 1).  fp32: sums of d + T terms, 2^-24 each.
def bounds(dtype, d, T):
    if dtype == BF16:
        return dict(o=2 ** -8 + 1.2e-4, state=6.2e-5, grad=4.5e-3, gate=6.0e-3)
    e = (d + T) * 2 ** -24
    return dict(o=e, state=e, grad=e, gate=e)


NAMES = (("o", "o"), ("final", "state"), ("dq", "grad"), ("dk", "grad"), ("dv", "grad"), ("dlg", "gate"),
         ("dbeta", "grad"), ("dinit", "state"))


@pytest.mark.parametrize("d,dtype,gate,T,decay", [
    (128, BF16, BF16, 1000, 0.05), (64, BF16, torch.float32, 777, 0.3), (128, BF16, torch.float32, 8192, 0.002),
    (128, BF16, BF16, 4099, 0.02), (64, torch.float32, torch.float32, 2050, 0.002)])
def test_long_against_64_bits(d, dtype, gate, T, decay):
    """Up to 128 chunks, memories of hundreds of tokens, every result against the recurrence in 64 bits."""
    q, k, v, dO, lg, beta = inputs(T, 1, 2, T, d, dtype, gate, decay, "cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    init, D = (torch.randn(1, 2, d, d, generator=g, device="cuda") / d ** 0.5 for _ in range(2))
    ck = la.checkpoint_delta(q)
    o, fin = la.fwd_delta(q, k, v, lg, beta, init_state=init, want_final=True, ckpt=ck)
    got = (o, fin, *la.bwd_delta(q, k, v, dO, lg, beta, ck, init_state=init, d_final=D, want_dinit=True))
    ro, rfin, _, _ = delta_forward(q, k, v, lg, beta, init)
    want = (ro, rfin, *delta_backward(q, k, v, dO, lg, beta, init, D))
    tol = bounds(dtype, d, T)
    errs = {n: rel(a, b.cpu()) for (n, _), a, b in zip(NAMES, got, want)}
    for n, kind in NAMES:
        assert errs[n] <= tol[kind], (n, errs, tol)


@pytest.mark.parametrize("d,dtype,H,T", [(128, BF16, 3, 200), (64, BF16, 2, 64), (128, BF16, 50, 130),
                                         (64, torch.float32, 2, 70), (128, BF16, 2, 0)])
def test_states_in_place(d, dtype, H, T):
    """final_state may be init_state itself, and d_init_state d_final_state: the bits of separate buffers."""
    q, k, v, dO, lg, beta = inputs(5, 1, H, T, d, dtype, torch.float32, 0.3, "cuda")
    init, D = (torch.randn(1, H, d, d, device="cuda") for _ in range(2))
    ck = la.checkpoint_delta(q)
    o, fin = la.fwd_delta(q, k, v, lg, beta, init_state=init, want_final=True, ckpt=ck)
    grads = la.bwd_delta(q, k, v, dO, lg, beta, ck, init_state=init, d_final=D, want_dinit=True)
    sh, s = la.shape_of(q), torch.cuda.current_stream().cuda_stream
    w1, w2 = la.workspace(q, la.OP_FWD_DELTA), la.workspace(q, la.OP_BWD_DELTA)
    state, dstate, o2, out = init.clone(), D.clone(), torch.empty_like(q), [torch.empty_like(t) for t in grads[:5]]
    p = lambda t: t.data_ptr()  # noqa: E731
    assert la.linattn_fwd_delta(sh, p(q), p(k), p(v), p(lg), p(beta), la.F32, p(o2), p(state), p(state), None, 0, p(w1),
                                w1.numel(), s) == la.OK
    assert la.linattn_bwd_delta(sh, p(q), p(k), p(v), p(dO), p(lg), p(beta), la.F32, p(init), p(dstate), p(ck),
                                ck.numel(), *(p(t) for t in out), p(dstate), p(w2), w2.numel(), s) == la.OK
    assert la.device_status(w1) == la.OK and la.device_status(w2) == la.OK
    assert torch.equal(o2, o) and torch.equal(state, fin) and torch.equal(dstate, grads[5])
    for a, b in zip(out, grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_decode_captured(dtype):
    """A captured token, replayed with new inputs, goes on from the state that the last replay left."""
    B, H, d, n = 3, 4, 128, 5
    q, k, v, _, lg, beta = inputs(6, B, H, n, d, dtype, dtype, 0.3, "cuda")
    S = torch.randn(B, H, d, d, device="cuda")
    want_S = S.clone()
    tok = lambda t: [x[:, :, t:t + 1].contiguous() for x in (q, k, v, lg, beta)]  # noqa: E731
    want = [la.decode_delta(*tok(t), want_S) for t in range(n)]
    x, state = tok(0), S.clone()
    o = torch.empty_like(x[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.decode_delta(*x, state, out=o)
    for t in range(n):
        for a, b in zip(x, tok(t)):
            a.copy_(b)
        graph.replay()
        assert torch.equal(o, want[t])
    assert torch.equal(state, want_S)
