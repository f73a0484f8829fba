"""Child process of tests/test_gpu_kv4_checks.py: run with MAGICPIG_CHECKS=1, so that the binding
loads the build whose kernels check the indices of their global accesses. The calls over the 4-bit
cache on clean inputs, at ragged sizes and with positions that leave the cache: no check fails.
Prints "checks ok" and exits 0 when every assertion holds."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import lsh_sampled_sparse_gb300 as mp  # noqa: E402
from tests import kv4_reference as R  # noqa: E402
from workloads import make_hyperplanes, make_layer, small_workload  # noqa: E402


def main() -> None:
    assert mp.library_path().endswith("libmagicpig_checks.so")
    assert mp.check_report() == (True, 0) and mp.device_status() == 0
    for dt in (torch.bfloat16, torch.float32):
        for B, Hkv, G, m, cap in ((2, 3, 4, 700, 777), (1, 8, 8, 9001, 9001), (3, 1, 1, 1, 5),
                                  (2, 5, 2, 2003, 2005)):
            x = torch.randn(2, B, Hkv, m, 128, device="cuda").to(dt)
            cache = mp.kv4_cache(B, Hkv, cap)
            cache.params.zero_()
            mp.kv4_write(cache, x[0], x[1])
            pos = torch.arange(B, dtype=torch.int32, device="cuda") * 3 - 2
            mp.kv4_write(cache, x[0], x[1], positions=pos)
            mp.kv4_read(cache, m, positions=pos, dtype=dt)
            q = torch.randn(B, Hkv * G, 128, device="cuda").to(dt)
            lengths = torch.randint(0, cap + 9, (B,), device="cuda").int()
            for L in (None, lengths):
                out = mp.kv4_attention(q, cache, lengths=L)
                used = [cap] * B if L is None else [min(cap, int(v)) for v in L]
                want, tol = R.attention64(q, cache, used, 128 ** -0.5)
                assert ((out.double() - want).abs() <= tol).all()
    wl = small_workload(name="kv4checks", index=770, B=2, Hq=8, Hkv=2, n=5000, K=10, L=150)
    x = {k: v.cuda() for k, v in make_layer(wl).items()}
    W = make_hyperplanes(wl).cuda()
    centre = mp.key_mean(x["keys"])
    codes = mp.build_tables(x["keys"], centre, W, wl.K, wl.L)
    cache = mp.kv4_write(mp.kv4_cache(2, 2, wl.n), x["keys"], x["values"], centre=centre)
    out = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, wl.K, wl.L, 4, 64)
    assert torch.isfinite(out).all()
    torch.cuda.synchronize()
    assert mp.check_report() == (True, 0) and mp.device_status() == 0
    print("checks ok", flush=True)


if __name__ == "__main__":
    main()
