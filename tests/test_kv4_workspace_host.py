"""The workspace of the 4-bit cache's attention on the host: one size serves a growing decode."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from lsh_sampled_sparse_gb300.build import build
    build()
    import lsh_sampled_sparse_gb300 as mp
    return mp.lib()


SHAPES = [(1, 32, 8, 98304), (4, 32, 8, 16384), (1, 32, 8, 8192), (2, 64, 8, 131072),
          (32, 32, 8, 32768), (7, 12, 12, 3001), (1, 8, 1, 5000), (1, 24, 1, 70000), (3, 5, 1, 257)]


@pytest.mark.parametrize("B,Hq,Hkv,cap", SHAPES)
def test_the_size_of_a_capacity_serves_every_smaller_n(L, B, Hq, Hkv, cap):
    sizes = [L.mp_kv4_attention_workspace_bytes(B, Hq, Hkv, n, 128)
             for n in [*range(1, min(cap, 600)), *range(600, cap, 97), cap]]
    assert sizes == sorted(sizes)
    assert sizes[-1] <= 8 << 20                                # partial states of a few waves of CTAs
    for n in (1, cap // 7 + 1, cap):
        uses = L.mp_kv4_attention_uses_workspace(B, Hq, Hkv, n, 128)
        assert uses in (0, 1) and (not uses or L.mp_kv4_attention_workspace_bytes(B, Hq, Hkv, n, 128))


def test_a_call_that_uses_no_workspace_says_so(L):
    uses = L.mp_kv4_attention_uses_workspace
    assert uses(1, 32, 8, 200, 128) == 0                       # one split
    assert uses(4, 32, 8, 16384, 128) == 0                     # a cluster
    assert uses(1, 32, 8, 98304, 128) == 1
    assert uses(1, 6, 4, 98304, 128) == 0 and uses(1, 32, 8, 98304, 64) == 0   # invalid


def test_no_workspace_is_asked_for_only_where_one_is_used(L):
    from lsh_sampled_sparse_gb300.binding import _KV4
    ok, WORKSPACE, INVALID = ctypes.c_void_p(0x10000), 5, 1

    def att(n, ws, size):
        cache = _KV4(0x10000, 0x10000, 0x10000, n)
        return L.mp_kv4_attention(ok, 1, ctypes.byref(cache), 1, 32, 8, n, 128, None, 0.0, ok, ws,
                                  size, None)

    need = L.mp_kv4_attention_workspace_bytes(1, 32, 8, 98304, 128)
    assert att(98304, None, need) == INVALID and att(98304, ok, need - 1) == WORKSPACE
