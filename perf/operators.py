"""Cases that measure the gated delta rule and the paged key-value cache, with the operators in plain torch.

Two families, the two layer kinds of a hybrid model:

* the gated delta rule (a linear-attention layer that overwrites what its state holds at a key),
      S_t = a_t S_{t-1} + b_t k_t (v_t - (a_t S_{t-1})^T k_t)^T,   o_t = S_t^T q_t,   a_t = exp(log_gate_t),
  as a training step, as a prefill from and to a state, and as one decoded token;
* softmax attention served from a paged cache: appending new keys and values through a block
  table, and one new query per sequence over everything its pages hold.

`own` selects between the plain forms (False) and the library's calls (True).
"""
import math
import random

import torch

own = False

CHUNK = 64


# ------------------------------------------------------------------ cases
def listed():
    return [
        # training steps: a toy layer, a ragged small-head layer, the fp32 check of a small model,
        # a layer at the forward benchmark's length, and the headline forward + backward shape
        {"name": "delta train B1 H2 T640 d128", "op": "train", "B": 1, "H": 2, "T": 640, "d": 128, "dtype": "bf16"},
        {"name": "delta train B2 H3 T1001 d64", "op": "train", "B": 2, "H": 3, "T": 1001, "d": 64, "dtype": "bf16"},
        {"name": "delta train B1 H2 T257 d64 fp32", "op": "train", "B": 1, "H": 2, "T": 257, "d": 64, "dtype": "f32"},
        {"name": "delta train B2 H16 T16384 d128", "op": "train", "B": 2, "H": 16, "T": 16384, "d": 128,
         "dtype": "bf16"},
        {"name": "delta train B2 H16 T65536 d128", "op": "train", "B": 2, "H": 16, "T": 65536, "d": 128,
         "dtype": "bf16"},
        # a later piece of a prompt: state in, state out
        {"name": "delta prefill B4 H16 T2049 d128", "op": "prefill", "B": 4, "H": 16, "T": 2049, "d": 128,
         "dtype": "bf16"},
        # one token per sequence: a single user, and a full serving batch
        {"name": "delta decode B1 H16", "op": "decode", "B": 1, "H": 16, "d": 128, "dtype": "bf16"},
        {"name": "delta decode B512 H16", "op": "decode", "B": 512, "H": 16, "d": 128, "dtype": "bf16"},
        # new keys and values into their pages: a decode step of a batch, and a padded batch of prompts
        {"name": "append B64 H8 T1", "op": "append", "B": 64, "Hkv": 8, "T": 1, "ctx": 2000, "page": 16, "d": 128,
         "dtype": "bf16"},
        {"name": "append B8 H8 T4096", "op": "append", "B": 8, "Hkv": 8, "T": 4096, "ctx": 777, "page": 64, "d": 128,
         "dtype": "bf16"},
        # one query per sequence over its pages: a single short chat, and a long-context serving batch
        {"name": "paged decode B1 H16 700", "op": "paged", "B": 1, "Hq": 16, "Hkv": 4, "len": 700, "page": 16,
         "d": 128, "dtype": "bf16"},
        {"name": "paged decode B64 H32 16384", "op": "paged", "B": 64, "Hq": 32, "Hkv": 8, "len": 16384, "page": 64,
         "d": 128, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["train", "train", "train", "prefill", "decode", "append", "paged", "paged"])
    d = rng.choice([64, 128, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("train", "prefill"):
        B, H = rng.choice([1, 2, 4]), rng.choice([1, 2, 3, 4, 8, 16, 32])
        # fp32 runs on the CUDA cores and is meant for checks: short sequences
        T = _log(rng, 1, 1024) if dtype == "f32" else _log(rng, 16, min(65536, (1 << 21) // (B * H)))
        return {"op": op, "B": B, "H": H, "T": T, "d": d, "dtype": dtype}
    if op == "decode":
        return {"op": op, "B": _log(rng, 1, 512), "H": rng.choice([1, 4, 16]), "d": d, "dtype": dtype}
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        T = rng.choice([1, 1, _log(rng, 2, 4096)])
        return {"op": op, "B": _log(rng, 1, 8 if T > 1 else 256), "Hkv": Hkv, "T": T, "ctx": _log(rng, 1, 4000),
                "page": page, "d": d, "dtype": dtype}
    n = _log(rng, 1, 16384)
    return {"op": op, "B": max(1, min(_log(rng, 1, 256), (1 << 20) // n)), "Hq": Hkv * rng.choice([1, 2, 4, 8]),
            "Hkv": Hkv, "len": n, "page": page, "d": d, "dtype": dtype}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case, g):
    """Ragged lengths of a batch: the first sequence the longest, the others anything down to a quarter of it."""
    B, n = case["B"], case.get("len", case.get("T"))
    r = torch.rand(B, generator=g, device="cuda")
    r[0] = 1.0
    return (n * (0.25 + 0.75 * r)).ceil().clamp(1, n).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op, B, d = case["op"], case["B"], case["d"]
    s = dict(case)
    if op in ("train", "prefill", "decode"):
        H, T = case["H"], case.get("T", 1)
        s["q"] = (rn(B, H, T, d) / math.sqrt(d)).to(dt)
        k = rn(B, H, T, d)
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
        s["v"] = rn(B, H, T, d).to(dt)
        # strengths from a sigmoid; log-gates -A softplus(x - 2) with a rate A per head between 0.05 and 0.8:
        # memories from a few tokens to hundreds.  Both come out of a projection in the model's type.
        s["beta"] = torch.sigmoid(rn(B, H, T)).to(dt)
        A = torch.exp(torch.rand(1, H, 1, generator=g, device="cuda") * math.log(16.0)) * 0.05
        s["lg"] = (-A * torch.nn.functional.softplus(rn(B, H, T) - 2)).to(dt)
        if op == "train":
            s["dO"] = rn(B, H, T, d).to(dt)
        else:
            s["state"] = rn(B, H, d, d) / math.sqrt(d)
        return s
    Hkv, page = case["Hkv"], case["page"]
    if op == "append":
        T = case["T"]
        s["new"] = _lens(case, g)
        s["start"] = (torch.rand(B, generator=g, device="cuda") * case["ctx"]).to(torch.int32)
        blocks = -(-(case["ctx"] + T) // page)
        s["k"], s["v"] = rn(B, Hkv, T, d).to(dt), rn(B, Hkv, T, d).to(dt)
    else:
        s["lens"] = _lens(case, g)
        blocks = -(-case["len"] // page)
        s["q"] = rn(B, case["Hq"], 1, d).to(dt)
    pages = B * blocks + 7
    s["table"] = torch.randperm(pages, generator=g, device="cuda")[: B * blocks].view(B, blocks).to(torch.int32)
    s["kc"], s["vc"] = rn(pages, Hkv, page, d).to(dt), rn(pages, Hkv, page, d).to(dt)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "train":
        leaves = [s[n].float().requires_grad_() for n in ("q", "k", "v", "lg", "beta")]
        with torch.enable_grad():
            o, _ = _delta(*leaves, None)
            grads = torch.autograd.grad(o, leaves, s["dO"].float())
        dt = s["q"].dtype
        return {n: x.detach().to(dt) for n, x in zip(("o", "dq", "dk", "dv", "dlg", "dbeta"), (o, *grads))}
    with torch.no_grad():
        if s["op"] == "prefill":
            o, fin = _delta(*(s[n].float() for n in ("q", "k", "v", "lg", "beta")), s["state"])
            return {"o": o.to(s["q"].dtype), "final": fin}
        if s["op"] == "decode":
            return _decode(s)
        return _append(s) if s["op"] == "append" else _paged(s)


def _run_own(s):
    import chunked_state_scan_causal_gb300 as la
    if s["op"] == "train":
        ck = la.checkpoint_delta(s["q"])
        o, _ = la.fwd_delta(s["q"], s["k"], s["v"], s["lg"], s["beta"], ckpt=ck)
        dq, dk, dv, dlg, dbeta, _ = la.bwd_delta(s["q"], s["k"], s["v"], s["dO"], s["lg"], s["beta"], ck)
        return {"o": o, "dq": dq, "dk": dk, "dv": dv, "dlg": dlg, "dbeta": dbeta}
    if s["op"] == "prefill":
        o, fin = la.fwd_delta(s["q"], s["k"], s["v"], s["lg"], s["beta"], init_state=s["state"], want_final=True)
        return {"o": o, "final": fin}
    if s["op"] == "decode":
        return {"o": la.decode_delta(s["q"], s["k"], s["v"], s["lg"], s["beta"], s["state"]), "state": s["state"]}
    if s["op"] == "append":
        la.paged_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["start"], new_lens=s["new"])
        return {"k_cache": s["kc"], "v_cache": s["vc"]}
    o, lse = la.paged_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], want_lse=True)
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------ plain forms
def _inverse(A):
    """(I + A)^-1 of strictly lower triangular blocks, by halves: [[X, 0], [-Y C X, Y]]."""
    n = A.shape[-1]
    if n == 1:
        return torch.ones_like(A)
    h = n // 2
    XY = _inverse(torch.stack((A[..., :h, :h], A[..., h:, h:])))
    X, Y = XY[0], XY[1]
    return torch.cat((torch.cat((X, torch.zeros_like(X)), -1), torch.cat((-Y @ A[..., h:, :h] @ X, Y), -1)), -2)


def _delta(q, k, v, lg, beta, state):
    """The delta rule by chunks: what a chunk's tokens write is the solution of a triangular system given the
    state that enters it, so the one loop, over the chunks, is the recurrence itself."""
    B, H, T, d = q.shape
    N = -(-T // CHUNK)
    fill = N * CHUNK - T
    pad = torch.nn.functional.pad
    q, k, v = (pad(x, (0, 0, 0, fill)).view(B, H, N, CHUNK, d) for x in (q, k, v))
    g = pad(lg, (0, fill)).view(B, H, N, CHUNK).cumsum(-1)
    b = pad(beta, (0, fill)).view(B, H, N, CHUNK, 1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    gam = torch.exp((g[..., :, None] - g[..., None, :]).masked_fill(~low, -math.inf))
    kk = (k @ k.transpose(-1, -2)) * gam
    inv = _inverse((b * kk).tril(-1))
    att = (q @ k.transpose(-1, -2)) * gam
    eg = torch.exp(g)[..., None]
    tv, tk = inv @ (b * v), inv @ (b * eg * k)
    qe, ke, last = eg * q, torch.exp(g[..., -1:] - g)[..., None] * k, torch.exp(g[..., -1])[..., None, None]
    S = torch.zeros(B, H, d, d, device=q.device) if state is None else state.float()
    outs = []
    for tvn, tkn, qen, attn, ken, lastn in zip(*(x.unbind(2) for x in (tv, tk, qe, att, ke, last))):
        u = tvn - tkn @ S
        outs.append(qen @ S + attn @ u)
        S = lastn * S + ken.transpose(-1, -2) @ u
    return torch.stack(outs, 2).view(B, H, N * CHUNK, d)[:, :, :T], S


def _decode(s):
    q, k, v, b = (s[n][:, :, 0].float() for n in ("q", "k", "v", "beta"))
    S = s["state"].mul_(torch.exp(s["lg"][:, :, 0].float())[..., None, None])
    y = v - (S * k[..., None]).sum(-2)
    S.add_(k[..., None] * (b[..., None] * y)[..., None, :])
    return {"o": (S * q[..., None]).sum(-2).to(s["q"].dtype)[:, :, None], "state": S}


def _append(s):
    B, _, T, _ = s["k"].shape
    page = s["page"]
    t = torch.arange(T, device="cuda")
    pos = s["start"].long()[:, None] + t
    keep = t < s["new"].long()[:, None]
    block = s["table"].long().gather(1, pos // page)[keep]
    slot = (pos % page)[keep]
    s["kc"][block, :, slot] = s["k"].transpose(1, 2)[keep]
    s["vc"][block, :, slot] = s["v"].transpose(1, 2)[keep]
    return {"k_cache": s["kc"], "v_cache": s["vc"]}


def _paged(s):
    B, Hq, Hkv, d, page = s["B"], s["Hq"], s["Hkv"], s["d"], s["page"]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    k, v = (s[n][s["table"].long()].float().transpose(1, 2).reshape(B, Hkv, -1, d) for n in ("kc", "vc"))
    x = (q @ k.transpose(-1, -2)) / math.sqrt(d)
    hidden = torch.arange(x.shape[-1], device="cuda") >= s["lens"].long()[:, None]
    x = x.masked_fill(hidden[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / l
    return {"o": o.view(B, Hq, 1, d).to(s["q"].dtype), "lse": (m + torch.log(l)).view(B, Hq, 1)}


# ------------------------------------------------------------------ work of one pass
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, B, d = case["op"], case["B"], case["d"]
    if op in ("train", "prefill", "decode"):
        n = B * case["H"] * case.get("T", 1)
        state = B * case["H"] * d * d * 4
        # per token of the recurrence: the read-out of the old value, the rank-one write and the output
        fwd = n * 6 * d * d
        if op == "train":
            # forward reads q, k, v and writes o; backward reads them and dO again and writes dq, dk, dv
            return {"bytes": n * (11 * d * e + 6 * e), "flops": 3 * fwd}
        return {"bytes": n * (4 * d * e + 2 * e) + 2 * state, "flops": fwd}
    if op == "append":
        return {"bytes": 4 * _mean_len(case, "T") * case["Hkv"] * d * e, "flops": 0}
    kv = _mean_len(case, "len") * case["Hkv"] * d
    return {"bytes": 2 * kv * e + 2 * B * case["Hq"] * d * e, "flops": 4 * kv * (case["Hq"] // case["Hkv"])}


def _mean_len(case, key):
    """Tokens of the batch: one full-length sequence and the others at the mean of their range."""
    return case[key] * (1 + 0.625 * (case["B"] - 1)) if case[key] > 1 else case["B"]


# ------------------------------------------------------------------ 64-bit values, from the definitions
def exact(case, seed):
    if case["op"] in ("train", "prefill") and case["T"] > 20000:
        return None  # a step per token: too long
    s = prepare(case, seed)
    D = lambda n: s[n].double()  # noqa: E731
    if case["op"] == "append":
        kc, vc, start, new, tab = D("kc"), D("vc"), s["start"].tolist(), s["new"].tolist(), s["table"].tolist()
        for b in range(case["B"]):
            t = 0
            while t < new[b]:  # page by page
                at = start[b] + t
                m = min(case["page"] - at % case["page"], new[b] - t)
                blk, sl = tab[b][at // case["page"]], at % case["page"]
                kc[blk, :, sl:sl + m] = s["k"][b, :, t:t + m].double()
                vc[blk, :, sl:sl + m] = s["v"][b, :, t:t + m].double()
                t += m
        return {"k_cache": kc, "v_cache": vc}
    if case["op"] == "paged":
        o, lse = [], []
        for b, n in enumerate(s["lens"].tolist()):
            blocks = s["table"][b, : -(-n // case["page"])].long()
            K, V = (s[c][blocks].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :n] for c in ("kc", "vc"))
            grp = case["Hq"] // case["Hkv"]
            K, V = K.repeat_interleave(grp, 0), V.repeat_interleave(grp, 0)
            x = torch.einsum("hd,hnd->hn", D("q")[b, :, 0], K) * case["d"] ** -0.5
            w = torch.logsumexp(x, -1)
            o.append(torch.einsum("hn,hnd->hd", torch.exp(x - w[:, None]), V))
            lse.append(w)
        return {"o": torch.stack(o)[:, :, None], "lse": torch.stack(lse)[:, :, None]}
    return _exact_delta(s, case, D)


def _exact_delta(s, case, D):
    """Token by token in 64 bits; the backward walks the tokens in reverse over states kept for one block at a time."""
    q, k, v, lg, b = (D(n) for n in ("q", "k", "v", "lg", "beta"))
    B, H, T, d = q.shape
    a = torch.exp(lg)[..., None, None]
    S = D("state") if "state" in s else torch.zeros(B, H, d, d, dtype=torch.float64, device="cuda")
    o, Y = torch.empty_like(q), torch.empty_like(q)

    def forward(S, t):
        Sd = a[:, :, t] * S
        y = v[:, :, t] - torch.einsum("bhij,bhi->bhj", Sd, k[:, :, t])
        return Sd, y, Sd + k[:, :, t, :, None] * (b[:, :, t, None] * y)[:, :, None]

    step, kept = 64, {}
    for t in range(T):
        if t % step == 0:
            kept[t] = S
        _, Y[:, :, t], S = forward(S, t)
        o[:, :, t] = torch.einsum("bhij,bhi->bhj", S, q[:, :, t])
    if case["op"] == "prefill":
        return {"o": o, "final": S}
    if case["op"] == "decode":
        return {"o": o, "state": S}
    do = D("dO")
    dq, dk, dv, dlg, db = (torch.empty_like(x) for x in (q, k, v, lg, b))
    R = torch.zeros_like(S)
    for t0 in reversed(range(0, T, step)):
        S, saved = kept.pop(t0), []
        for t in range(t0, min(T, t0 + step)):
            Sd, _, S = forward(S, t)
            saved.append((Sd, S))
        for t in reversed(range(t0, min(T, t0 + step))):
            Sd, St = saved.pop()
            R = R + q[:, :, t, :, None] * do[:, :, t, None]
            dq[:, :, t] = torch.einsum("bhij,bhj->bhi", St, do[:, :, t])
            du = torch.einsum("bhij,bhi->bhj", R, k[:, :, t])
            dy = b[:, :, t, None] * du
            db[:, :, t] = (du * Y[:, :, t]).sum(-1)
            dv[:, :, t] = dy
            dk[:, :, t] = (torch.einsum("bhij,bhj->bhi", R, b[:, :, t, None] * Y[:, :, t])
                           - torch.einsum("bhij,bhj->bhi", Sd, dy))
            R = R - k[:, :, t, :, None] * dy[:, :, None]
            dlg[:, :, t] = (R * Sd).sum((-1, -2))
            R = a[:, :, t] * R
    return {"o": o, "dq": dq, "dk": dk, "dv": dv, "dlg": dlg, "dbeta": db}
