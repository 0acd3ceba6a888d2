"""The attention calls' entry points without a GPU, over pools that none could hold."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "c"))
import build as cbuild  # noqa: E402


def test_slots_beyond_32_bits_are_refused():
    exe = cbuild.build_sanitized("asan", "attend_host")
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="halt_on_error=1 print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "attend_host ok" in r.stdout and "runtime error" not in r.stderr
