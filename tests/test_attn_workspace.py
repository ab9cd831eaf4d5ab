"""A workspace made for the largest call serves the smaller ones (CPU: sizes and plans only)."""
import os
import random
import subprocess

from sparse_matrix_vector_amd import _lib as L
from test_sanitize_cpu import SAN, SAN_ENV, _cxx, pytestmark as needs_sanitizers


def test_sizes_grow_with_every_argument():
    f = L.attn_lib().nm_attn_workspace_bytes
    assert f(1, 32, 8, 128, 0, 0, 8193) >= f(1, 32, 8, 128, 0, 0, 8192) > 0
    assert f(32, 64, 8, 128, 1, 32768, 4096) >= f(32, 64, 8, 128, 1, 32768, 512) >= f(32, 64, 8, 128, 1, 32768, 0) > 0
    r = random.Random(3)
    for _ in range(20000):
        heads, G = r.choice((1, 2, 4, 8, 16)), r.choice((1, 3, 4, 8, 16, 17, 32))
        shape = (heads * G, heads, r.choice((64, 128, 256)), r.randrange(3))
        B, P, ml = r.randrange(1, 100), r.choice((0, r.randrange(40000))), r.choice((0, r.randrange(40000)))
        small = f(r.randrange(1, B + 1), *shape, r.choice((0, r.randrange(P + 1))), r.choice((0, r.randrange(ml + 1))))
        assert 0 <= small <= f(B, *shape, P, ml)


@needs_sanitizers
def test_sizes_hold_every_smaller_plan(tmp_path):
    exe = _cxx(str(tmp_path / "attn_workspace"), os.path.join(SAN, "attn_workspace.cpp"))
    proc = subprocess.run([exe, "1000000"], capture_output=True, text=True, env=dict(os.environ, **SAN_ENV), timeout=600)
    assert proc.returncode == 0, proc.stdout + proc.stderr
    assert "shapes checked" in proc.stdout
    print(proc.stdout)
