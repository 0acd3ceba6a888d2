"""How attention calls are split, without a GPU."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "c"))
import build as cbuild  # noqa: E402


def test_places_for_partial_results():
    """Two million calls' sizes, bounds of no rows among them: whoever writes partial results has a workspace for them."""
    exe = cbuild.build_attend_plan()
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "attend_plan ok" in r.stdout
