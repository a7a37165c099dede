"""The entry script: it ends well when it is run, and its smoke run reaches every operator."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_script_builds_and_ends():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "__graft_entry__.py")], cwd=ROOT,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.gpu
def test_smoke_reaches_every_operator(capsys):
    import __graft_entry__

    __graft_entry__.smoke()
    out = capsys.readouterr().out
    for name in ("float32", "bfloat16", "short conv", "layer operators", "linear attention"):
        assert f"smoke {name}" in out or f"smoke torch.{name}" in out, (name, out)
