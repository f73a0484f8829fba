"""Child process of tests/test_gpu_kv4_forms_checks.py: run with MAGICPIG_CHECKS=1, so that the
binding loads the build whose kernels check the indices of their global accesses. The forms of the
4-bit cache's calls that tests/kv4_checks_child.py does not reach, on clean inputs: the sampled
decode whose rows are shared by clusters of two, four and eight CTAs, over bucketed tables with
appended keys, over MIPS and cross-polytope codes; rows encoded in every mode of mp_encode_rows
and mp_encode_keys. No check fails, and results equal those of the calls they have to equal.
Prints "checks ok" and exits 0 when every assertion holds."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import lsh_sampled_sparse_gb300 as mp  # noqa: E402
from workloads import make_hyperplanes, make_layer, small_workload  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def clean():
    torch.cuda.synchronize()
    assert mp.check_report() == (True, 0) and mp.device_status() == 0


def layer(B, Hq, Hkv, n, K, L, cap):
    """Inputs, hyperplanes, centre, codes and the 4-bit cache of a layer, laid out for cap."""
    wl = small_workload(name="kv4forms", index=771, B=B, Hq=Hq, Hkv=Hkv, n=n, K=K, L=L)
    x = {k: v.cuda() for k, v in make_layer(wl).items()}
    W = make_hyperplanes(wl).cuda()
    centre = mp.key_mean(x["keys"])
    cache = mp.kv4_cache(B, Hkv, cap)
    mp.kv4_write(cache, x["keys"], x["values"], centre=centre)
    codes = mp.encode_rows(x["keys"], centre, W, K, L, 0, cap)
    return x, W, centre, codes, cache


def main() -> None:
    assert mp.library_path().endswith("libmagicpig_checks.so")
    clean()
    # clusters of eight, four and two CTAs a partial; the bucketed call; the variants
    for B, Hq, Hkv, n, K, L, sink, local in ((1, 16, 8, 3194, 7, 195, 4, 64),
                                             (4, 32, 8, 901, 6, 99, 0, 64),
                                             (8, 64, 8, 1500, 5, 100, 4, 64),
                                             (1, 2, 1, 2000, 10, 150, 300, 1200)):
        cap = n + 5
        x, W, centre, codes, cache = layer(B, Hq, Hkv, n, K, L, cap)
        args = (K, L, sink, local)
        out = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, *args, n=n)
        assert torch.isfinite(out).all()
        ws = torch.empty(mp.decode_workspace_bytes(B, Hq, Hkv, n, 128, *args), dtype=torch.uint8,
                         device="cuda")
        indexed = n - 300
        buckets = mp.build_buckets(codes, B, Hkv, indexed, K, L, n_capacity=cap)
        mp.encode_query(x["q"], centre, W, (B, Hkv, cap, 128), *args, ws, n=n)
        again = mp.kv4_sampled_attention_buckets(x["q"], buckets, centre, cache, *args,
                                                 torch.empty_like(out), ws, codes=codes, n=n,
                                                 n_indexed=indexed)
        assert torch.equal(again, out)
        clean()
        W_aug = torch.cat([W, torch.randn(1, K * L, device="cuda").to(W.dtype)]).contiguous()
        radius = mp.key_radius(x["keys"], centre)
        kc = torch.zeros(B, Hkv, cap, 128, dtype=BF, device="cuda")
        kc[:, :, :n] = x["keys"]
        mcodes = mp.encode_keys_mips(kc, centre, W_aug, radius, K, L, 0, n)
        out = mp.kv4_decode_attention(x["q"], mcodes, centre, W_aug, cache, *args, n=n,
                                      radius=radius)
        assert torch.isfinite(out).all()
        G = torch.randn(16, 128, 128, device="cuda").to(BF)
        ccodes = mp.encode_keys_cp(kc, centre, G, 16, 0, n)
        out = mp.kv4_decode_attention(x["q"], ccodes, centre, G, cache, 1, 16, sink, local, n=n,
                                      logu_table=mp.cp_logu_table(1, 16))
        assert torch.isfinite(out).all()
        clean()
    # rows that begin and end inside blocks, short and long, on tensor cores and CUDA cores
    for kd, wd in ((BF, BF), (F32, F32), (BF, F32)):
        for B, Hkv, m, cap, n0 in ((2, 2, 1, 1500, 1499), (1, 3, 64, 2048, 1000),
                                   (2, 2, 500, 1700, 300), (1, 2, 2500, 5000, 100),
                                   (2, 1, 3100, 4200, 1024), (1, 1, 1024, 1024, 0)):
            K, L = 9, 20
            keys = torch.randn(B, Hkv, cap, 128, device="cuda").to(kd)
            W = torch.randn(128, K * L, device="cuda").to(wd)
            centre = mp.key_mean(keys)
            want = mp.build_tables(keys, centre, W, K, L)
            mp.encode_keys(keys, centre, W, K, L, n0, n0 + m, want)
            got = want.clone()
            rows = keys[:, :, n0:n0 + m].contiguous()
            mp.encode_rows(rows, centre, W, K, L, n0, cap, codes=got)
            # the same bits but for signs that float32 cannot tell; none outside the range
            differ = mp.codes_unpack(got, B, Hkv, cap, K, L) != mp.codes_unpack(want, B, Hkv, cap,
                                                                               K, L)
            assert differ[:, :, n0:n0 + m].double().mean() < 1e-3
            assert not differ[:, :, :n0].any() and not differ[:, :, n0 + m:].any()
            clean()
    print("checks ok", flush=True)


if __name__ == "__main__":
    main()
