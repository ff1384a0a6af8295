"""What is built against what: the library needs no torch binding, and a binding fits one torch."""
import os
import subprocess
import sys

from certified_fixed_stabilizer_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_without_its_torch_binding(tmp_path):
    """No binding, and no compiler to build one: the calls that need libclis.so alone work, the others say why not."""
    build.build()
    code = f"""
import certified_fixed_stabilizer_gb300.build as b
b.TORCH_EXT = {str(tmp_path / "_clis_torch.so")!r}
import torch
from certified_fixed_stabilizer_gb300 import clis
assert clis.clis_status_string(0) and clis.load_library() is not None
assert clis.load_library().clis_attn_fwd(None, *[None] * 8, 0.1, 0, 0, None) == 1
t = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
try:
    clis.rope(t, None, torch.zeros(4, 1, dtype=torch.int32), torch.ones(8, dtype=torch.float64), torch.zeros(8, dtype=torch.int32))
except Exception as e:
    print("refused:", type(e).__name__)
"""
    env = {**os.environ, "PATH": str(tmp_path), "CUDA_HOME": str(tmp_path), "PYTHONPATH": ROOT}
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "refused:" in r.stdout and "ValueError" not in r.stdout, r.stdout


def test_a_binding_for_another_torch_is_stale(monkeypatch):
    build.build()
    assert not build._binding_stale()
    monkeypatch.setattr(build, "_torch_tag", lambda: "another torch")
    assert build._binding_stale() and not build._stale()
