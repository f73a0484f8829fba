"""Child process of tests/test_gpu_paged_unprepared.py: a library whose preparation of the paged cache's kernels
reports an error (argv[1]: its path). The calls that need it say so and launch nothing; all others run. Prints
"unprepared ok" and exits 0 when every assertion holds."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import lsh_sampled_sparse_gb300 as mp  # noqa: E402
from lsh_sampled_sparse_gb300 import binding  # noqa: E402


def main() -> None:
    binding.library_path = lambda: sys.argv[1]
    B, Hq, Hkv, n, K, L, page = 1, 4, 2, 640, 4, 30, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    keys, values, q, W = rand(B, Hkv, n, 128), rand(B, Hkv, n, 128), rand(B, Hq, 128), rand(128, K * L)
    centre = mp.key_mean(keys)
    codes = mp.build_tables(keys, centre, W, K, L)
    want = mp.decode_attention(q, codes, centre, W, keys, values, K, L, 4, 64)
    assert torch.isfinite(want).all()
    kv4 = mp.kv4_cache(B, Hkv, n)
    mp.kv4_write(kv4, keys, values)
    assert torch.isfinite(mp.kv4_attention(q, kv4)).all()
    table = torch.arange(n // page, device="cuda").int()[None]
    cache = mp.PagedCache(*(t[0].view(Hkv, n // page, page, 128).transpose(0, 1).contiguous()
                            for t in (keys, values)))
    for _ in range(2):
        for call in (lambda: mp.paged_attention(q, cache, table),
                     lambda: mp.paged_append(cache, table, keys, values)):
            try:
                call()
            except mp.MagicPIGError as e:
                assert "MP_ERR_CUDA" in str(e)
            else:
                raise AssertionError("a call ran whose kernels are not prepared")
    # (the sampled decode over pages is the contiguous cache's kernels')
    out = mp.paged_decode_attention(q, codes, centre, W, cache, table, K, L, 4, 64)
    assert (out - want).abs().max() <= 2 * 4e-5 * 5          # log u: 2e-5 of the contiguous form's table, twice
    torch.cuda.synchronize()
    assert mp.device_status() == 0
    print("unprepared ok", flush=True)


if __name__ == "__main__":
    main()
