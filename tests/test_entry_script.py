"""The entry file run as a script: what its functions use is there by then."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ENTRY = os.path.join(ROOT, "__graft_entry__.py")


def test_script_runs_its_functions_when_all_are_defined():
    """Nothing is defined below the block that runs them."""
    import ast
    with open(ENTRY) as f:
        body = ast.parse(f.read()).body
    blocks = [n for n in body if isinstance(n, ast.If) and "__main__" in ast.unparse(n.test)]
    assert blocks == [body[-1]]


@pytest.mark.gpu
def test_smoke_as_a_script():
    r = subprocess.run([sys.executable, ENTRY, "smoke"], capture_output=True, text=True, cwd=ROOT, timeout=600)
    assert r.returncode == 0 and "smoke ok" in r.stdout, r.stdout + r.stderr
