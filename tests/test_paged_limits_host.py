"""The largest sizes that the calls over the paged cache take, on the host: what is past them is refused before
anything is launched."""
import ctypes

import pytest

from tests.test_paged_host import INVALID, OK, L, _cache  # noqa: F401  (L: a fixture)

HUGE = dict(page=8, slots=2 ** 28 - 1)           # a table of 2^31 - 8 tokens, of ten pages again and again


def _decode(L, B=1, Hq=4, Hkv=1, n=100, K=0, cache=None, cap=0, scale=0.0, size=2 ** 62):
    import lsh_sampled_sparse_gb300 as mp
    prm = mp.Params(K, 150, 4, 64, scale, 0, cap)
    return L.mp_paged_decode_attention(OK, 1, OK, OK, OK, 1, cache or _cache(**HUGE), B, Hq, Hkv, n, 128,
                                       None, ctypes.byref(prm), OK, OK, size, None)


@pytest.mark.parametrize("n", [2 ** 30 + 1, 2 ** 31 - 4095, 2 ** 31 - 1024, 2 ** 31 - 8])
def test_sampled_decode_refuses_more_tokens_than_it_numbers(L, n):  # noqa: F811
    assert _decode(L, n=n) == INVALID
    assert _decode(L, n=n, K=10, cap=n) == INVALID


@pytest.mark.parametrize("kw", [dict(n=2 ** 30 + 1), dict(n=2 ** 31 - 8), dict(B=2 ** 20 + 1, n=1),
                                dict(B=2 ** 11, n=2 ** 22 + 1), dict(B=2 ** 31 - 1, n=1)])
def test_attention_refuses_more_than_it_numbers(L, kw):  # noqa: F811
    a = dict(B=1, Hq=4, Hkv=1, n=100)
    a.update(kw)
    assert L.mp_paged_attention(OK, 1, _cache(**HUGE), a["B"], a["Hq"], a["Hkv"], a["n"], 128, None, 0.0, OK,
                                OK, 2 ** 62, None) == INVALID


@pytest.mark.parametrize("B,Hq,Hkv", [(2048, 32, 8), (65536, 1, 1), (8192, 8, 8), (2 ** 28, 32, 8)])
def test_sampled_decodes_refuse_more_query_rows_than_a_grid_has(L, B, Hq, Hkv):  # noqa: F811
    """Before anything is launched: not by the last kernel's launch, behind the first ones."""
    import lsh_sampled_sparse_gb300 as mp
    from lsh_sampled_sparse_gb300.binding import _KV4
    assert _decode(L, B=B, Hq=Hq, Hkv=Hkv) == INVALID
    prm = ctypes.byref(mp.Params(0, 150, 4, 64, 0.0, 0, 100))
    dims, end = (B, Hq, Hkv, 100, 128, prm, OK, OK, 2 ** 62, None), INVALID
    kv4 = ctypes.byref(_KV4(0x10000, 0x10000, 0x10000, 100))
    assert L.mp_decode_attention(OK, 1, OK, OK, OK, 1, OK, OK, 1, *dims) == end
    assert L.mp_sampled_attention(OK, 1, OK, OK, OK, OK, 1, *dims) == end
    assert L.mp_sampled_attention_buckets(OK, 1, OK, OK, OK, OK, OK, 1, *dims) == end
    assert L.mp_kv4_decode_attention(OK, 1, OK, OK, OK, 1, kv4, *dims) == end
    assert L.mp_kv4_sampled_attention(OK, 1, OK, OK, kv4, *dims) == end
    # as many as there are places is not what is wrong
    small = (1, 4, 1, 100, 128, prm, OK, OK, 16, None)
    assert L.mp_decode_attention(OK, 1, OK, OK, OK, 1, OK, OK, 1, *small) == 5          # the workspace


def test_scales_that_make_no_number_are_refused(L):  # noqa: F811
    """The exact attention's kernels take the scale times log2 e, which has to be finite too: every score would
    be an infinity or NaN."""
    def att(scale, size=2 ** 62):
        return L.mp_paged_attention(OK, 1, _cache(), 1, 4, 1, 100, 128, None, scale, OK, OK, size, None)

    for scale in (3.0e38, 2.36e38, float("inf"), float("nan"), -1e-30):
        assert att(scale) == INVALID
    assert att(2.35e38, 16) == 5                 # refused for its workspace
    for scale in (float("inf"), float("nan"), -1.0):
        assert _decode(L, scale=scale) == INVALID
