"""Child process of tests/test_gpu_paged_checks.py: run with MAGICPIG_CHECKS=1, so that the binding loads
the build whose kernels check the indices of their global accesses. The calls over the paged cache on
clean inputs, at ragged sizes, with places and pages that do not exist: no check fails. Prints "checks
ok" and exits 0 when every assertion holds."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import lsh_sampled_sparse_gb300 as mp  # noqa: E402
from tests import paged_reference as R  # noqa: E402


def main() -> None:
    assert mp.library_path().endswith("libmagicpig_checks.so")
    assert mp.check_report() == (True, 0) and mp.device_status() == 0
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    freq = (1e4 ** (-torch.arange(0, 128, 2, device="cuda").double() / 128)).float()
    for dt in (torch.bfloat16, torch.float32):
        for B, Hkv, G, n, page in ((2, 3, 4, 700, 16), (1, 8, 8, 9001, 64), (3, 1, 1, 1, 8),
                                   (5, 2, 12, 2003, 48), (9, 2, 2, 300, 24), (70, 1, 4, 90, 8)):
            slots = -(-n // page)
            n_pages = B * slots + 1
            table = torch.randperm(n_pages, generator=gen, device="cuda")[:B * slots].view(B, -1).int()
            cache = mp.paged_cache(n_pages, Hkv, page, dt)
            for t in cache:
                t.zero_()
            x = torch.randn(2, B, Hkv, n, 128, generator=gen, device="cuda").to(dt)
            q = torch.randn(B, Hkv * G, 1, 128, generator=gen, device="cuda").to(dt)
            mp.paged_append(cache, table, x[0], x[1], inv_freq=freq)
            places = (torch.arange(B, device="cuda") * 3 - 2).int()      # the first before the cache
            counts = torch.randint(-1, n + 2, (B,), generator=gen, device="cuda").int()
            mp.paged_append(cache, table, x[0], x[1], positions=places, counts=counts)
            q = mp.paged_append(cache, table, x[0][:, :, :1], x[1][:, :, :1], n_begin=n - 1,
                                inv_freq=freq, interleaved=True, q=q,
                                keys_out=torch.empty(B, Hkv, 1, 128, dtype=dt, device="cuda"))[:, :, 0]
            q = q.contiguous()
            lengths = torch.randint(0, n + 9, (B,), generator=gen, device="cuda").int()
            for L in (None, lengths):
                out = mp.paged_attention(q, cache, table, n=n, lengths=L)
                used = [n] * B if L is None else [min(n, int(v)) for v in L]
                want, tol = R.attention(q, cache.keys, cache.values, table.cpu(), used, 128 ** -0.5)
                assert ((out.double() - want).abs() <= tol).all()
            table[0, 0] = -1                                             # and a page that is not there
            mp.paged_attention(q, cache, table, n=n)
            if G <= 8 and G != 3:
                K, L = 6, 40
                W = torch.randn(128, K * L, generator=gen, device="cuda").to(dt)
                centre = torch.randn(B, Hkv, 128, generator=gen, device="cuda")
                codes = mp.encode_rows(x[0], centre, W, K, L, 0, slots * page)
                mp.encode_rows_at(x[0][:, :, :33].contiguous(), centre, W, K, L, places, slots * page,
                                  codes)
                for ln in (None, lengths):
                    out = mp.paged_decode_attention(q, codes, centre, W, cache, table, K, L, 4, 64, n=n,
                                                    lengths=ln)
                    assert torch.isfinite(out).all()
                    # most keys sampled
                    out = mp.paged_decode_attention(q, codes, centre, W, cache, table, 1, 40, 40, 640, n=n,
                                                    lengths=ln)
                    assert torch.isfinite(out).all()
    torch.cuda.synchronize()
    assert mp.check_report() == (True, 0) and mp.device_status() == 0
    print("checks ok", flush=True)


if __name__ == "__main__":
    main()
