"""Host code behind include/nmattn.h under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/sanitize/attn_checks.cpp."""
import os
import subprocess

from test_sanitize_cpu import CSRC, SAN, SAN_ENV, _cxx, pytestmark  # noqa: F401


def test_attention_layout_plans_and_checks(tmp_path):
    exe = _cxx(str(tmp_path / "attn_checks"), os.path.join(SAN, "attn_checks.cpp"), os.path.join(CSRC, "nmattn_api.cpp"))
    proc = subprocess.run([exe, "400000"], capture_output=True, text=True, env=dict(os.environ, **SAN_ENV), timeout=600)
    out = proc.stdout + proc.stderr
    assert proc.returncode == 0, out[-4000:]
    assert "plans checked" in out and "runtime error" not in out
    print(out)
