"""The paged cache's C ABI used from a plain C11 program
(tests/capi/cache_check.c): every entry point of tb_cache.h once, no Python
binding and no torch in the process."""
import os
import subprocess

import pytest

from gpu_util import note

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIN = os.path.join(ROOT, "tests", "capi", "cache_check")

pytestmark = pytest.mark.gpu


def test_c_program_uses_the_cache():
    if not os.path.exists(BIN):
        pytest.fail(f"{BIN} is missing: build first (python -c 'import __graft_entry__ as g; g.build()')")
    note("C-ABI consumer of the paged cache: append, fork, attention, page copy, resize, compact from plain C")
    r = subprocess.run([BIN], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, f"rc={r.returncode}\n{r.stdout}\n{r.stderr}"
    assert "cache ok" in r.stdout
