"""The compiled marshalling and the Python functions make the same checks: every argument that one refuses, the other refuses too,
and every call that the Python way takes in its ordinary form, the compiled one takes."""
import pytest
import torch

import chunked_state_scan_causal_gb300 as la

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
B, HQ, HKV, T, D, PAGE, PAGES, BLOCKS = 2, 4, 2, 2, 64, 32, 12, 4


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_state_scan_causal_gb300 import build
    build.build()


class Never:
    paged_append_q8 = paged_gather_q8 = paged_decode_q8 = rope = staticmethod(lambda *a: None)


def good():
    """Arguments by name, all of them views of larger zeroed buffers."""
    z = lambda shape, dtype: torch.zeros(8 * torch.Size(shape).numel(), dtype=dtype, device="cuda")[  # noqa: E731
        : torch.Size(shape).numel()].view(shape)
    codes = lambda: z((PAGES, HKV, PAGE, D), torch.uint8).view(E4M3)  # noqa: E731
    return dict(q=z((B, HQ, T, D), BF16), k=z((B, HKV, T, D), BF16), v=z((B, HKV, T, D), BF16), kc=codes(), vc=codes(),
                scales=z((PAGES, HKV, PAGE // 16, 2), F32) + 1, table=z((B, BLOCKS), torch.int32),
                start=z((B,), torch.int32), lens=z((B,), torch.int32) + 5, freqs=la.rope_frequencies(D, device="cuda"),
                pos=z((B,), torch.int32), out=z((B, HQ, T, D), BF16), ws=la.workspace(z((B, HQ, T, D), BF16), la.OP_PAGED_DECODE))


CALLS = {
    "append": (("k", "v", "kc", "vc", "scales", "table", "start", "lens"),
               lambda a: la.paged_append_q8(*a), lambda m, a: m.paged_append_q8(*a)),
    "gather": (("kc", "vc", "scales", "table", "lens", "start"),
               lambda a: la.paged_gather_q8(*a[:5], 7, F32, a[5]), lambda m, a: m.paged_gather_q8(*a[:5], 7, F32, a[5])),
    "decode": (("q", "kc", "vc", "scales", "table", "lens", "out", "ws"),
               lambda a: la.paged_decode_q8(*a[:6], 0.5, True, a[6], a[7]),
               lambda m, a: m.paged_decode_q8(*a[:6], 0.5, True, a[6], a[7])),
    "rope": (("q", "k", "freqs", "pos"),
             lambda a: la.rope_fwd(*a), lambda m, a: m.rope(False, *a, la.ROPE_LAYOUTS["half"], 1.0, None, None)),
}


def odd(x):
    """Strides of two in the last dimension."""
    return torch.zeros(*x.shape[:-1], 2 * x.shape[-1], dtype=x.dtype, device=x.device)[..., ::2]


def wide(x):
    """The same values with other strides."""
    y = torch.zeros(*x.shape[:-1], 2 * x.shape[-1], dtype=torch.uint8 if x.dtype == E4M3 else x.dtype, device=x.device)
    y = y.view(E4M3) if x.dtype == E4M3 else y
    return y[..., : x.shape[-1]]


SEQ = [("half", lambda x: x.half()), ("codes", lambda x: x.to(E4M3)), ("three dimensions", lambda x: x[0]), ("odd", odd),
       ("another d", lambda x: torch.zeros(*x.shape[:3], 96, dtype=x.dtype, device="cuda")), ("host", lambda x: x.cpu())]
ROWS = [("long", lambda x: x.long()), ("one more", lambda x: torch.cat((x, x[:1]))), ("every other", lambda x: x.repeat(2)[::2]),
        ("two dimensions", lambda x: x[None]), ("host", lambda x: x.cpu())]
REFUSED = {
    "q": SEQ, "k": [*SEQ, ("another batch", lambda x: x[:1])],
    "v": [("float", lambda x: x.float()), ("wide", wide), ("another batch", lambda x: x[:1]), ("host", lambda x: x.cpu())],
    "kc": [("bytes", lambda x: x.view(torch.uint8)), ("wide", wide), ("fewer pages", lambda x: x[:1]), ("no heads", lambda x: x[:, 0]),
           ("host", lambda x: x.cpu())],
    "vc": [("bytes", lambda x: x.view(torch.uint8)), ("wide", wide), ("fewer pages", lambda x: x[:1]), ("host", lambda x: x.cpu())],
    "scales": [("double", lambda x: x.double()), ("one head", lambda x: x[:, :1]), ("one block", lambda x: x[:, :, :1]),
               ("one number", lambda x: x[..., :1]), ("keys and values apart", lambda x: x.transpose(2, 3).contiguous().transpose(2, 3)),
               ("host", lambda x: x.cpu())],
    "table": [("long", lambda x: x.long()), ("one more", lambda x: torch.cat((x, x[:1]))), ("odd", odd), ("one row", lambda x: x[0]),
              ("a row twice", lambda x: x[:1].expand(B, BLOCKS)), ("host", lambda x: x.cpu())],
    "start": ROWS, "lens": ROWS,
    "freqs": [("float", lambda x: x.float()), ("every other", lambda x: x.repeat(2)[::2]), ("two dimensions", lambda x: x[None]),
              ("too many", lambda x: x.repeat(2)), ("none", lambda x: x[:0]), ("host", lambda x: x.cpu())],
    "pos": [("long", lambda x: x.long()), ("one more", lambda x: torch.cat((x, x[:1]))), ("every other", lambda x: x.repeat(2)[::2]),
            ("another T", lambda x: x[:, None].repeat(1, T + 1)), ("host", lambda x: x.cpu())],
    "out": [("float", lambda x: x.float()), ("wide", wide), ("another batch", lambda x: x[:1]), ("host", lambda x: x.cpu())],
    "ws": [("every other", lambda x: x.repeat(2)[::2]), ("short", lambda x: x[:256]), ("host", lambda x: x.cpu())],
}
TABLE = [(call, name, label) for call, (names, *_) in CALLS.items() for name in names for label, _ in REFUSED[name]]


@pytest.mark.parametrize("call,name,label", TABLE)
def test_refused_both_ways(call, name, label, monkeypatch):
    names, python, compiled = CALLS[call]
    a = good()
    a[name] = dict(REFUSED[name])[label](a[name])
    args = [a[n] for n in names]
    assert compiled(la._bind(), args) is None
    errors = []
    for way in (la._bind(), Never):
        monkeypatch.setattr(la, "_fast", way)
        with pytest.raises((ValueError, la.LinattnError)) as e:
            python(args)
        errors.append((e.type, str(e.value)))
    assert errors[0] == errors[1]


@pytest.mark.parametrize("call", CALLS)
def test_ordinary_both_ways(call, monkeypatch):
    """Without a change, and with what is left out or laid out otherwise, the compiled way takes the call."""
    names, python, compiled = CALLS[call]
    changes = [{}, {n: None for n in ("start", "lens") if (call, n) in (("append", "lens"), ("gather", "start"))},
               {n: None for n in ("out", "ws", "k") if (call, n) in (("decode", "out"), ("decode", "ws"), ("rope", "k"))},
               {n: wide for n in ("k", "v", "kc", "vc")}, {"scales": lambda x: x.repeat(1, 2, 1, 1)[:, :HKV]}]  # (longer pages)
    for change in changes:
        a = good()
        for n, f in change.items():
            a[n] = f(a[n]) if f else None
        args = [a[n] for n in names]
        assert compiled(la._bind(), args) is not None, change
        monkeypatch.setattr(la, "_fast", Never)
        python(args)
        monkeypatch.undo()
