"""The 64-bit references of the delta rule and the paged cache against differences and a dense form (no GPU),
and the host-side refusals of their entry points (no kernel is launched)."""
import ctypes

import pytest
import torch

import chunked_state_scan_causal_gb300 as la
from delta_ref import delta_backward, delta_forward, paged_attention


def inputs(seed, B, H, T, d):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    k = rn(B, H, T, d)
    return (rn(B, H, T, d) / d ** 0.5, k / k.norm(dim=-1, keepdim=True), rn(B, H, T, d), rn(B, H, T, d),
            -0.3 * torch.rand(B, H, T, generator=g, dtype=torch.float64), torch.sigmoid(rn(B, H, T)),
            rn(B, H, d, d), rn(B, H, d, d))


def test_reference_gradients_against_differences():
    q, k, v, dO, lg, beta, init, D = inputs(1, 1, 2, 5, 4)

    def loss(q, k, v, lg, beta, init):
        o, fin, _, _ = delta_forward(q, k, v, lg, beta, init)
        return float((o * dO).sum() + (fin * D).sum())

    args = [q, k, v, lg, beta, init]
    grads = delta_backward(q, k, v, dO, lg, beta, init, D)
    h = 1e-6
    for i, g in enumerate(grads):
        for e in range(0, args[i].numel(), max(1, args[i].numel() // 7)):
            lo, hi = [x.clone() for x in args], [x.clone() for x in args]
            lo[i].view(-1)[e] -= h
            hi[i].view(-1)[e] += h
            num = (loss(*hi) - loss(*lo)) / (2 * h)
            # central differences: the loss' rounding 2^-53 * |loss| / h, about 1e-9, and h^2
            assert abs(num - float(g.reshape(-1)[e])) < 1e-7, (i, e)


def test_reference_is_the_dense_solution():
    """beta (I + tril(A, -1))^-1 form of one chunk without decay."""
    q, k, v, _, _, beta, init, _ = inputs(2, 1, 1, 9, 4)
    o, fin, y, _ = delta_forward(q, k, v, None, beta, init)
    A = torch.tril(k @ k.transpose(-1, -2), -1) * beta[..., None, :]
    Y = torch.linalg.solve(torch.eye(9, dtype=torch.float64) + A, v - k @ init)
    assert torch.allclose(Y, y, atol=1e-12)
    assert torch.allclose(fin, init + k.transpose(-1, -2) @ (beta[..., None] * Y), atol=1e-12)


FAKE = 1 << 20


def _shape(**kw):
    s = la.Shape()
    s.abi_version, s.B, s.H, s.T, s.dk, s.dv, s.chunk, s.dtype = la.ABI_VERSION, 1, 2, 256, 128, 128, 64, la.BF16
    s.stride_b, s.stride_h, s.stride_t = 2 * 256 * 128, 256 * 128, 128
    for n, x in kw.items():
        setattr(s, n, x)
    return s


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_state_scan_causal_gb300 import build
    build.build()


def fwd(s, q=FAKE, lg=FAKE, beta=FAKE, gdt=la.F32, o=FAKE, init=None, ck=None, nck=0, ws=FAKE, nws=1 << 40):
    return la.linattn_fwd_delta(s, q, FAKE, FAKE, lg, beta, gdt, o, init, None, ck, nck, ws, nws, None)


def bwd(s, dO=FAKE, lg=FAKE, dlg=FAKE, gdt=la.F32, ck=FAKE, nck=1 << 40, ws=FAKE, nws=1 << 40, db=FAKE):
    return la.linattn_bwd_delta(s, FAKE, FAKE, FAKE, dO, lg, FAKE, gdt, None, None, ck, nck, FAKE, FAKE, FAKE, dlg, db,
                                None, ws, nws, None)


def test_delta_refusals():
    lam = (ctypes.c_float * 2)(0.9, 0.9)
    decayed = _shape(decay=ctypes.cast(lam, ctypes.c_void_p))
    for call in (fwd, bwd):
        assert call(decayed) == la.ERR_INVALID
        assert call(_shape(), gdt=7) == la.ERR_INVALID
        assert call(_shape(dk=96)) == la.ERR_UNSUPPORTED
        assert call(_shape(stride_t=129)) == la.ERR_ALIGN
        assert call(_shape(T=-1)) == la.ERR_INVALID
        assert call(_shape(), ws=None) == la.ERR_WORKSPACE
        assert call(_shape(), ws=FAKE + 16) == la.ERR_WORKSPACE
        assert call(_shape(), lg=FAKE + 4) == la.ERR_ALIGN
    assert fwd(_shape(), q=None) == la.ERR_INVALID
    assert fwd(_shape(), beta=None) == la.ERR_INVALID
    assert fwd(_shape(), o=FAKE + 2) == la.ERR_ALIGN
    assert fwd(_shape(), init=FAKE + 4) == la.ERR_ALIGN
    for s in (_shape(), _shape(dtype=la.F32)):
        st, n = la.linattn_workspace_size(s, la.OP_CHECKPOINT_DELTA)
        assert st == la.OK and n > 0 and n % 256 == 0
        assert fwd(s, ck=FAKE, nck=n - 1) == la.ERR_INVALID
        assert fwd(s, ck=FAKE + 16, nck=n) == la.ERR_INVALID
        assert bwd(s, nck=n - 1) == la.ERR_INVALID
        for op, call in ((la.OP_FWD_DELTA, fwd), (la.OP_BWD_DELTA, bwd)):
            st, n = la.linattn_workspace_size(s, op)
            assert st == la.OK and n >= 256
            assert call(s, nws=n - 1) == la.ERR_WORKSPACE
    assert bwd(_shape(), ck=None) == la.ERR_INVALID
    assert bwd(_shape(), dO=None) == la.ERR_INVALID
    assert bwd(_shape(), db=None) == la.ERR_INVALID
    # the log-gates and their gradient come together
    assert bwd(_shape(), dlg=None) == la.ERR_INVALID
    assert bwd(_shape(), lg=None) == la.ERR_INVALID

    def dec(s, beta=FAKE, state=FAKE, gdt=la.BF16):
        return la.linattn_decode_delta(s, FAKE, FAKE, FAKE, None, beta, gdt, FAKE, state, None)
    assert dec(_shape(T=1), beta=None) == la.ERR_INVALID
    assert dec(_shape(T=1), state=FAKE + 8) == la.ERR_ALIGN
    assert dec(_shape(T=1), gdt=-1) == la.ERR_INVALID
    assert dec(decayed) == la.ERR_INVALID
    assert dec(_shape(T=0)) == la.OK


def _cache(**kw):
    return _shape(**{**dict(B=40, H=2, T=16, stride_b=2 * 16 * 128, stride_h=16 * 128, stride_t=128), **kw})


def test_paged_refusals():
    new = _shape(T=3, stride_b=2 * 3 * 128, stride_h=3 * 128)

    def app(s=new, c=None, k=FAKE, tab=FAKE, n=4, ts=4, start=FAKE):
        return la.linattn_paged_append(s, c or _cache(), k, FAKE, FAKE, FAKE, tab, n, ts, start, None, None, None)
    q = _shape(H=8, T=1, stride_b=8 * 128, stride_h=128)
    st, need = la.linattn_workspace_size(q, la.OP_PAGED_DECODE)
    assert st == la.OK and need > 256

    def dec(s=q, c=None, k=FAKE, tab=FAKE, n=4, ts=4, lens=FAKE, scale=0.0, ws=FAKE, nws=need):
        return la.linattn_paged_decode(s, c or _cache(), FAKE, k, FAKE, FAKE, None, tab, n, ts, lens, scale, ws, nws,
                                       None)
    for call in (app, dec):
        assert call(c=_cache(dtype=la.F32)) == la.ERR_INVALID            # another type
        assert call(c=_cache(dk=64, dv=64)) == la.ERR_INVALID            # another head dimension
        assert call(c=_cache(T=0)) == la.ERR_INVALID                     # no page
        assert call(tab=None) == la.ERR_INVALID
        assert call(n=0) == la.ERR_INVALID
        assert call(ts=3) == la.ERR_INVALID
        assert call(n=1 << 28, ts=1 << 28) == la.ERR_UNSUPPORTED         # positions past 31 bits
        assert call(k=None) == la.ERR_INVALID
        assert call(k=FAKE + 8) == la.ERR_ALIGN
        assert call(c=_cache(stride_t=132)) == la.ERR_ALIGN
    assert app(start=None) == la.ERR_INVALID
    assert app(s=_shape(H=4)) == la.ERR_INVALID
    assert app(s=_shape(T=0)) == la.OK
    assert dec(lens=None) == la.ERR_INVALID
    assert dec(s=_shape(H=7, T=1)) == la.ERR_UNSUPPORTED                 # not a multiple of the key heads
    assert dec(s=_shape(H=8, T=2)) == la.ERR_UNSUPPORTED
    for scale in (-1.0, float("nan"), float("inf")):
        assert dec(scale=scale) == la.ERR_INVALID
    assert dec(ws=None) == la.ERR_WORKSPACE
    assert dec(nws=need - 1) == la.ERR_WORKSPACE


def test_python_checks():
    q = torch.zeros(1, 2, 8, 64)
    g = torch.zeros(1, 2, 8)
    ck = torch.empty(0, dtype=torch.uint8)
    for lg, b in ((g, g.bfloat16()), (g[:, :, :4], g), (g, g.half()), (g.transpose(1, 2).contiguous().transpose(1, 2), g)):
        with pytest.raises(ValueError):
            la.fwd_delta(q, q, q, lg, b)
        with pytest.raises(ValueError):
            la.bwd_delta(q, q, q, q, lg, b, ck)
    with pytest.raises(ValueError):
        la.fwd_delta(q, q, q, g, g, init_state=torch.zeros(1, 2, 64, 64).bfloat16())
    with pytest.raises(ValueError):
        la.decode_delta(q, q, q, g, g, torch.zeros(1, 2, 64, 32))
    kc = torch.zeros(4, 2, 16, 64)
    tab, n = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for t, m in ((tab.long(), n), (tab, n.long()), (tab[0], n), (tab, torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            la.paged_decode(q[:, :, :1], kc, kc, t, m)
        with pytest.raises(ValueError):
            la.paged_append(q, q, kc, kc, t, m)


def test_paged_reference_skips_bad_pages():
    g = torch.Generator().manual_seed(3)
    q, kc = torch.randn(1, 2, 1, 8, generator=g), torch.randn(3, 1, 4, 8, generator=g)
    o, lse = paged_attention(q, kc, kc, torch.tensor([[2, 9, 0]]), torch.tensor([10]))
    K = torch.cat((kc[2, 0], kc[0, 0, :2])).double()
    x = (q[0, :, 0].double() @ K.T) * 8 ** -0.5
    assert torch.allclose(o[0, :, 0], torch.softmax(x, -1) @ K) and torch.allclose(lse[0, :, 0], torch.logsumexp(x, -1))


def test_overlapping_table_rows():
    """A row expanded over the batch (stride 0) or rows that overlap are refused, not read as if they were apart; one
    sequence may have any row stride, and rows may be further apart than they are long."""
    q, kc = torch.zeros(2, 2, 1, 64), torch.zeros(4, 2, 16, 64)
    n, flat = torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    for tab in (flat[:3].expand(2, 3), flat.as_strided((2, 3), (2, 1)), flat[:1].expand(2, 1)):
        with pytest.raises(ValueError, match="overlap"):
            la.paged_decode(q, kc, kc, tab, n)
        with pytest.raises(ValueError, match="overlap"):
            la.paged_append(q, q, kc, kc, tab, n)
    assert la._table(q, flat.as_strided((2, 3), (5, 1)))[1:] == (3, 5)
    assert la._table(q, flat.view(2, 4))[1:] == (4, 4)
    assert la._table(q[:1], flat.as_strided((1, 3), (0, 1)))[1:] == (3, 3)


def test_words_of_32_bits():
    """A status word, lengths, positions, page ids and lse off a 4-byte boundary are refused (a kernel would read or
    write them whole); so is a status tensor that is not int32 or is empty."""
    new = _shape(T=3, stride_b=2 * 3 * 128, stride_h=3 * 128)
    q = _shape(H=8, T=1, stride_b=8 * 128, stride_h=128)
    _, need = la.linattn_workspace_size(q, la.OP_PAGED_DECODE)
    for off in (1, 2, 3):
        for i in range(4):
            tab, start, lens, status = (FAKE + (off if i == j else 0) for j in range(4))
            assert la.linattn_paged_append(new, _cache(), FAKE, FAKE, FAKE, FAKE, tab, 4, 4, start, lens, status,
                                           None) == la.ERR_ALIGN
        for i in range(3):
            tab, lens, lse = (FAKE + (off if i == j else 0) for j in range(3))
            assert la.linattn_paged_decode(q, _cache(), FAKE, FAKE, FAKE, FAKE, lse, tab, 4, 4, lens, 0.0, FAKE, need,
                                           None) == la.ERR_ALIGN
    x, kc = torch.zeros(1, 2, 1, 64), torch.zeros(4, 2, 16, 64)
    tab, n = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for status in (torch.zeros(1, dtype=torch.int8), torch.zeros(1), torch.zeros(0, dtype=torch.int32),
                   torch.zeros(1, dtype=torch.int32, device="meta")):
        with pytest.raises(ValueError, match="device_status"):
            la.paged_append(x, x, kc, kc, tab, n, device_status=status)


def test_forward_workspace_with_a_checkpoint():
    """With a checkpoint the forward's workspace is its status word's 256 bytes; without one, what the size query says."""
    for s in (_shape(), _shape(dtype=la.F32), _shape(dk=64, dv=64)):
        _, nck = la.linattn_workspace_size(s, la.OP_CHECKPOINT_DELTA)
        _, nws = la.linattn_workspace_size(s, la.OP_FWD_DELTA)
        assert fwd(s, ck=FAKE, nck=nck, nws=255) == la.ERR_WORKSPACE
        # (the next refusal after the workspace's: it was long enough)
        assert fwd(s, q=None, ck=FAKE, nck=nck, nws=256) == la.ERR_INVALID
        assert fwd(s, nws=nws - 1) == la.ERR_WORKSPACE


def test_tensors_of_the_host_are_refused():
    """Every kind of call says so (ValueError) before the library gets a pointer."""
    q, kc = torch.zeros(1, 2, 8, 64), torch.zeros(4, 2, 16, 64)
    g, S = torch.zeros(1, 2, 8), torch.zeros(1, 2, 64, 64)
    tab, n = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ck, one = torch.zeros(1 << 20, dtype=torch.uint8), q[:, :, :1]
    for call in (lambda: la.fwd(q, q, q), lambda: la.decode(q, q, q, S), lambda: la.fwd_delta(q, q, q, g, g),
                 lambda: la.bwd_delta(q, q, q, q, g, g, ck), lambda: la.decode_delta(q, q, q, g, g, S),
                 lambda: la.paged_append(one, one, kc, kc, tab, n), lambda: la.paged_decode(one, kc, kc, tab, n),
                 lambda: la.device_status(ck)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_buffers_of_another_device_are_refused():
    """A workspace or checkpoint elsewhere, or one whose bytes are not its own (expanded), never reaches a kernel."""
    q, g = torch.zeros(1, 2, 8, 64), torch.zeros(1, 2, 8)
    kc, n = torch.zeros(4, 2, 16, 64), torch.zeros(1, dtype=torch.int32)
    tab, ck = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1 << 20, dtype=torch.uint8)
    for bad in (torch.zeros(1 << 20, dtype=torch.uint8, device="meta"), torch.zeros(1, dtype=torch.uint8).expand(1 << 20)):
        for call in (lambda: la.fwd_delta(q, q, q, g, g, ws=bad), lambda: la.fwd_delta(q, q, q, g, g, ckpt=bad),
                     lambda: la.bwd_delta(q, q, q, q, g, g, bad), lambda: la.bwd_delta(q, q, q, q, g, g, ck, ws=bad),
                     lambda: la.paged_decode(q[:, :, :1], kc, kc, tab, n, ws=bad)):
            with pytest.raises(ValueError, match="workspaces and checkpoints"):
                call()
