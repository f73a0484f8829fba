"""Calls over the paged cache that its documentation allows and the other tests do not make."""
import pytest
import torch

from tests.test_gpu_paged import BF, F32, _attend_and_check, _gen, _ints, _randn, _random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lsh_sampled_sparse_gb300 as mp
    mp.lib()
    return mp


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G", [1, 4, 8, 16, 20])
def test_many_units_of_one_tile(mp, dtype, G):
    """Runs of units of one tile, whose sums of weights differ by a hundred: a unit's sums are its own."""
    B, Hkv, n = 611, 2, 256
    g = _gen(G + 1)
    lens = [(1, 128, 2, 127, 129, 256, 1, 100)[b % 8] for b in range(B)]
    cache, table = _random_cache(mp, g, B, Hkv, n, 16, dtype, lens)
    q = (_randn(g, B, Hkv * G, 128) * 0.1).to(dtype)
    first = _attend_and_check(mp, q, cache, table, n, lens, _ints(lens))
    for _ in range(20):
        assert torch.equal(mp.paged_attention(q, cache, table, n=n, lengths=_ints(lens)), first)
    assert mp.device_status() == 0
