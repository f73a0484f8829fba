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
