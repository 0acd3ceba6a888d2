"""The forward-pass calls' host side without a GPU."""
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "c"))
import build as cbuild  # noqa: E402


def test_host_arithmetic_under_sanitizers():
    """Extents of tensors and tables from sizes and strides, those that pass 64 bits among them, overlaps
    of strided tensors, and reports made between the steps of a sync that takes others."""
    exe = cbuild.build_sanitized("asan", "forward_host")
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="halt_on_error=1 print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "forward_host ok" in r.stdout and "runtime error" not in r.stderr


def test_inline_assembly_names_the_registers_it_writes():
    """Statements that set m0 tell the compiler so."""
    csrc = os.path.join(os.path.dirname(HERE), "host_device_page_amd", "csrc")
    found = 0
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            for text in re.findall(r"\basm\b[^;]*;", f.read()):
                if re.search(r"s_mov_b32 m0", text):
                    found += 1
                    assert re.search(r':[^:]*"m0"\s*\)\s*;$', text), (name, text)
    assert found == 2
