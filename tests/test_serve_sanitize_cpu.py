"""Host code behind include/nmserve.h under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/sanitize/serve_checks.cpp."""
import os
import subprocess

from test_sanitize_cpu import CSRC, SAN, SAN_ENV, _cxx, pytestmark  # noqa: F401


def test_serving_plans_sizes_and_checks(tmp_path):
    exe = _cxx(str(tmp_path / "serve_checks"), os.path.join(SAN, "serve_checks.cpp"),
               os.path.join(CSRC, "nmserve_api.cpp"), os.path.join(CSRC, "nmattn_api.cpp"))
    proc = subprocess.run([exe, "200000"], capture_output=True, text=True, env=dict(os.environ, **SAN_ENV), timeout=600)
    out = proc.stdout + proc.stderr
    assert proc.returncode == 0, out[-4000:]
    assert "tree plans checked" in out and "launches" in out and "runtime error" not in out
    print(out)
