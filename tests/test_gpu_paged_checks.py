"""The MP_CHECKS build over the paged cache: tests/paged_checks_child.py in a child process that loads
libmagicpig_checks.so."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_paged_cache_passes_the_index_checks():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lsh_sampled_sparse_gb300.build import build
    build(checks=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "paged_checks_child.py")],
                       env=dict(os.environ, MAGICPIG_CHECKS="1"), cwd=ROOT, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "checks ok" in r.stdout
