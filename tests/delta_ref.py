"""The gated delta rule and attention over a paged cache in 64 bits, one token at a time (test oracle)."""
import torch


def delta_forward(q, k, v, lg, beta, init=None):
    """(o, final state, y [B,H,T,d], S' and S per token)."""
    q, k, v, beta = (x.double() for x in (q, k, v, beta))
    B, H, T, d = q.shape
    a = torch.ones(B, H, T, dtype=torch.float64) if lg is None else torch.exp(lg.double())
    S = torch.zeros(B, H, d, d, dtype=torch.float64) if init is None else init.double()
    o, y, states = torch.zeros_like(q), torch.zeros_like(q), []
    for t in range(T):
        Sd = a[:, :, t, None, None] * S
        y[:, :, t] = v[:, :, t] - (Sd.transpose(-1, -2) @ k[:, :, t, :, None])[..., 0]
        S = Sd + k[:, :, t, :, None] * (beta[:, :, t, None] * y[:, :, t])[:, :, None]
        o[:, :, t] = (S.transpose(-1, -2) @ q[:, :, t, :, None])[..., 0]
        states.append((Sd, S))
    return o, S, y, states


def delta_backward(q, k, v, dO, lg, beta, init=None, d_final=None):
    """(dq, dk, dv, d_log_gate, d_beta, d_init)."""
    _, _, y, states = delta_forward(q, k, v, lg, beta, init)
    q, k, v, dO, beta = (x.double() for x in (q, k, v, dO, beta))
    B, H, T, d = q.shape
    a = torch.ones(B, H, T, dtype=torch.float64) if lg is None else torch.exp(lg.double())
    R = torch.zeros(B, H, d, d, dtype=torch.float64) if d_final is None else d_final.double()
    dq, dk, dv = (torch.zeros_like(q) for _ in range(3))
    dlg, db = torch.zeros_like(beta), torch.zeros_like(beta)
    mv = lambda M, x: (M @ x[..., None])[..., 0]  # noqa: E731
    for t in reversed(range(T)):
        Sd, S = states[t]
        R = R + q[:, :, t, :, None] * dO[:, :, t, None]
        dq[:, :, t] = mv(S, dO[:, :, t])
        du = mv(R.transpose(-1, -2), k[:, :, t])
        dy = beta[:, :, t, None] * du
        db[:, :, t] = (du * y[:, :, t]).sum(-1)
        dv[:, :, t] = dy
        dk[:, :, t] = mv(R, beta[:, :, t, None] * y[:, :, t]) - mv(Sd, dy)
        R = R - k[:, :, t, :, None] * dy[:, :, None]
        dlg[:, :, t] = (R * Sd).sum((-1, -2))
        R = a[:, :, t, None, None] * R
    return dq, dk, dv, dlg, db, R


def paged_attention(q, kc, vc, table, lens, scale=None):
    """(o [B,Hq,1,d], lse [B,Hq,1]); tokens on page ids outside the cache are absent."""
    B, Hq, _, d = q.shape
    pages, Hkv, page, _ = kc.shape
    scale = d ** -0.5 if scale is None else scale
    o = torch.zeros(B, Hq, 1, d, dtype=torch.float64)
    lse = torch.full((B, Hq, 1), -float("inf"), dtype=torch.float64)
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * page))
        keep = [(int(table[b, i // page]), i % page) for i in range(n) if 0 <= int(table[b, i // page]) < pages]
        if not keep:
            continue
        pg, sl = (torch.tensor(x) for x in zip(*keep))
        for h in range(Hq):
            K, V = (c[pg, h // (Hq // Hkv), sl].double() for c in (kc, vc))
            x = (K @ q[b, h, 0].double()) * scale
            lse[b, h, 0] = torch.logsumexp(x, 0)
            o[b, h, 0] = torch.softmax(x, 0) @ V
    return o, lse


def rel(got, ref):
    """2-norm of the difference over the 2-norm of the reference."""
    got, ref = got.detach().double().cpu(), ref.double().cpu()
    assert torch.isfinite(got).all()
    return float((got - ref).norm() / max(float(ref.norm()), 1e-30))
