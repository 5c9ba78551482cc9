"""The gated delta rule's gradients and states beyond single short sequences."""
import pytest
import torch

import chunked_state_scan_causal_gb300 as la

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
