"""The library is built and used without torch's headers; the compiled marshalling is a shortcut that may be missing."""
import os
import subprocess
import sys

import pytest
import torch

import chunked_state_scan_causal_gb300 as la
from chunked_state_scan_causal_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("without", ["sys.modules['torch'] = None", "b._bind_flags = lambda: ['--no-such-flag']"])
def test_library_without_the_module(tmp_path, without):
    code = f"""
import sys
sys.path.insert(0, {ROOT!r})
from chunked_state_scan_causal_gb300 import build as b
{without}
b.OUT_DIR, b.SOURCES = {str(tmp_path)!r}, ["pad.cu"]
b.LIB = {str(tmp_path / "liblinattn.so")!r}
assert b.build() == b.LIB
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert (tmp_path / "liblinattn.so").exists() and not list(tmp_path.glob("_bind*.so"))
    assert "marshalling" in r.stderr


def test_calls_without_the_module(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(build, "bind_path", lambda: str(tmp_path / "_bind.so"))
    monkeypatch.setattr(la, "_fast", None)
    q = torch.zeros(1, 2, 3, 64)
    c = torch.zeros(2, 1, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s, t, n = torch.zeros(2, 1, 1, 2), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for f in (lambda: la.rope_fwd(q, None, la.rope_frequencies(64), n), lambda: la.paged_append_q8(q, q, c, c, s, t, n),
              lambda: la.paged_gather_q8(c, c, s, t, n, 4), lambda: la.paged_decode_q8(q, c, c, s, t, n)):
        with pytest.raises(ValueError, match="CUDA"):  # what the Python way says, on a machine with or without a GPU
            f()
