"""What the preparation of the paged cache's kernels failing refuses: their calls, and no others. The error is a
fake one, made on the host: the library is linked once more with that function replaced."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_paged_cache_that_cannot_be_prepared_refuses_its_own_calls_only(tmp_path):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lsh_sampled_sparse_gb300 import build as b
    b.build()
    objs = [os.path.join(b.OBJDIR, os.path.basename(s)[:-3] + ".o") for s in b.sources()]
    if not all(os.path.exists(o) for o in objs):
        b.build(force=True)
    fake, lib = tmp_path / "fake.cu", tmp_path / "libmagicpig_unprepared.so"
    fake.write_text('#include <cuda_runtime.h>\n'
                    'extern "C" cudaError_t __wrap__ZN2mp13prepare_pagedEv() { return cudaErrorInvalidValue; }\n')
    subprocess.run([b.nvcc(), *b.NVCC_FLAGS, "-c", str(fake), "-o", str(tmp_path / "fake.o")], check=True)
    subprocess.run([b.nvcc(), *b.ARCH, "-shared", "-Xlinker", "--wrap=_ZN2mp13prepare_pagedEv", "-o", str(lib),
                    *objs, str(tmp_path / "fake.o")], check=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "paged_unprepared_child.py"), str(lib)],
                       cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "unprepared ok" in r.stdout
