"""Attention over the 4-bit cache where tokens of very different sizes stand side by side, against 64
bits, with tolerances that follow the weights: a token that has none may not cost the others
anything."""
import pytest
import torch

from tests import kv4_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lsh_sampled_sparse_gb300 as mp
    mp.lib()
    return mp


def _weighted64(q, cache, scale, held=0.0):
    """softmax(scale q.k) . v in 64 bits and the error [B, Hq, 128] that a float32 evaluation may
    have of it, by the weights w_i: with V_i the largest value of token i in a dim's group and V the
    mean of V_i under the weights,

        sum_i w_i e_i (V_i + V) + 2^-24 (4 sqrt(n) + 16) V,   e_i = 2^-24 (32 A_i + 2 D_i + 4).

    A_i = scale sum_d |q_d k_id|: a logit is off by a random walk over 128 products and their sum,
    about sqrt(128) = 11.3 roundings of up to 2 2^-24 A_i (32 leaves a factor of 1.4), and by the
    rounding of its distance D_i from the largest logit; the exponential adds 4. A weight that is
    off by e_i moves the output by w_i e_i (v_i - out). The sums over n tokens add a random walk of
    sqrt(n) roundings of 2 2^-24, in numerator and denominator. `held`: what a query's elements may be
    off by, as a share of the row's largest, besides 2^-22 of themselves (counted if it is not 0)."""
    k, v = R.values64(cache[0], cache[2], 0), R.values64(cache[1], cache[2], 1)
    B, Hq, _ = q.shape
    G = Hq // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    n, e = k.shape[2], 2.0 ** -24
    qd = q.double().unsqueeze(-1)
    s = scale * (k @ qd).squeeze(-1)                                     # [B, Hq, n]
    w = torch.softmax(s, -1)
    A = scale * (k.abs() @ qd.abs()).squeeze(-1)
    D = s.amax(-1, keepdim=True) - s
    big = v.abs().unflatten(-1, (2, 64)).amax(-1)                        # [B, Hq, n, 2]
    mean = (w.unsqueeze(-1) * big).sum(2, keepdim=True)
    if held:
        A = A + scale / (32 * e) * (k.abs() @ (2.0 ** -22 * qd.abs()
                                               + held * qd.abs().amax(-2, keepdim=True))).squeeze(-1)
    tol = (w.unsqueeze(-1) * e * (32 * A + 2 * D + 4).unsqueeze(-1) * (big + mean)).sum(2) \
        + e * (4 * n ** 0.5 + 16) * mean.squeeze(2)
    return (w.unsqueeze(2) @ v).squeeze(2), tol.repeat_interleave(64, -1)


def _opposed(mp, B, Hkv, G, n, at, far, seed):
    """Queries q of every KV head near one direction, the last head's against it; random keys but for
    token `at`, whose key lies `far` times against that direction: next to no weight for all
    heads but the last, which has next to no other."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    base = torch.randn(B, Hkv, 1, 128, generator=g, device="cuda")
    q = base + 0.3 * torch.randn(B, Hkv, G, 128, generator=g, device="cuda")
    if G > 1:
        q[:, :, -1] = -q[:, :, -1]
    keys = torch.randn(B, Hkv, n, 128, generator=g, device="cuda")
    keys[:, :, at] = -far * base[:, :, 0]
    values = torch.randn(B, Hkv, n, 128, generator=g, device="cuda")
    return q.flatten(1, 2).contiguous(), keys, values, g


# far 20: the weight is 0 in float32 (e^-220 and less); far 2: about e^-22, so that the large value
# counts for something again
@pytest.mark.parametrize("far", [20.0, 2.0])
@pytest.mark.parametrize("ratio", [2.0 ** 20, 2.0 ** 27, 2.0 ** 34, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("G,n,at", [(1, 64, 37), (4, 500, 77), (8, 500, 78), (3, 4100, 4099), (11, 90, 3)])
def test_a_large_value_that_has_no_weight_costs_the_others_nothing(mp, G, n, at, ratio, far):
    q, keys, values, _ = _opposed(mp, 2, 2, G, n, at, far, seed=n + G)
    values[:, :, at] *= ratio
    cache = mp.kv4_write(mp.kv4_cache(2, 2, n), keys, values)
    out = mp.kv4_attention(q, cache)
    want, tol = _weighted64(q, cache, 128 ** -0.5)
    off = (out.double() - want).abs()
    assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("G", [1, 4, 8])
def test_heads_of_one_tile_do_not_share_a_scale(mp, G):
    """Tiles in which one head finds its weight and the others next to none (e^-22), over values
    2^30 times larger than the earlier tiles': each head's sums keep their own bits."""
    n = 600
    q, keys, values, _ = _opposed(mp, 1, 2, G, n, n - 1, 2.0, seed=40 + G)
    keys[:, :, 512:] = keys[:, :, -1:]
    values[:, :, :512] *= 2.0 ** -30
    cache = mp.kv4_write(mp.kv4_cache(1, 2, n), keys, values)
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    want, tol = _weighted64(q, cache, 128 ** -0.5)
    for out in (mp.kv4_attention(q, cache), mp.kv4_attention(q, cache, lengths=lengths)):
        off = (out.double() - want).abs()
        assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("at", [3, 12])
@pytest.mark.parametrize("ends", [(0.0, 2.0 ** 126), (-2.0 ** 126, 2.0 ** 126), (-2.0 ** 126, 0.0)])
def test_values_of_the_documented_size(mp, G, at, ends):
    """Values up to 2^126 in size, whose codes the sums take in 15 steps at once: without weight they
    cost the others nothing; with all the weight (the last head) they come out."""
    n = 40
    q, keys, values, _ = _opposed(mp, 1, 2, G, n, at, 20.0, seed=60 + G)
    values[:, :, at, :64] = torch.linspace(*ends, 64, device="cuda")
    cache = mp.kv4_write(mp.kv4_cache(1, 2, n), keys, values)
    assert torch.isfinite(cache.params.float()).all()
    out = mp.kv4_attention(q, cache)
    want, tol = _weighted64(q, cache, 128 ** -0.5)
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("ratio", [2.0 ** 6, 2.0 ** 12, 2.0 ** 18])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_queries_and_keys_of_opposite_sizes(mp, G, ratio):
    """The small elements of a query meet the large ones of the keys and the other way round: an
    element is held to 2^-25 of its row's largest, as the header says."""
    n = 300
    g = torch.Generator(device="cuda")
    g.manual_seed(80 + G)
    q = torch.randn(1, 2 * G, 128, generator=g, device="cuda")
    keys = torch.randn(1, 2, n, 128, generator=g, device="cuda")
    values = torch.randn(1, 2, n, 128, generator=g, device="cuda")
    q[..., 64:] /= ratio
    keys[..., 64:] *= ratio
    cache = mp.kv4_write(mp.kv4_cache(1, 2, n), keys, values)
    want, tol = _weighted64(q, cache, 128 ** -0.5, held=2.0 ** -25)
    assert ((mp.kv4_attention(q, cache).double() - want).abs() <= tol).all()


def test_keys_up_to_the_documented_size(mp):
    n = 70
    g = torch.Generator(device="cuda")
    g.manual_seed(90)
    keys = torch.randn(1, 2, n, 128, generator=g, device="cuda")
    keys = keys / keys.abs().max() * 2.0 ** 124
    values = torch.randn(1, 2, n, 128, generator=g, device="cuda")
    q = torch.randn(1, 8, 128, generator=g, device="cuda") * 2.0 ** -121
    cache = mp.kv4_write(mp.kv4_cache(1, 2, n), keys, values)
    want, tol = _weighted64(q, cache, 128 ** -0.5)
    assert ((mp.kv4_attention(q, cache).double() - want).abs() <= tol).all()


def test_one_workspace_serves_a_growing_decode(mp):
    B, Hq, Hkv, cap = 4, 32, 8, 16384              # a cluster at the capacity, a merge below it
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    cache = mp.kv4_write(mp.kv4_cache(B, Hkv, cap),
                         *(torch.randn(B, Hkv, cap, 128, generator=g, device="cuda")
                           for _ in range(2)))
    q = torch.randn(B, Hq, 128, generator=g, device="cuda")
    ws = torch.empty(mp.kv4_attention_workspace_bytes(B, Hq, Hkv, cap), dtype=torch.uint8,
                     device="cuda")
    for n in (1, 300, 5000, 10001, 16128, cap):
        assert torch.equal(mp.kv4_attention(q, cache, n=n, workspace=ws),
                           mp.kv4_attention(q, cache, n=n))


def test_a_small_scale_of_small_queries_over_large_keys(mp):
    """scale times a query below 2^-126: a product that float32 holds only as a subnormal number."""
    n = 200
    g = torch.Generator(device="cuda")
    g.manual_seed(91)
    keys = torch.randn(1, 2, n, 128, generator=g, device="cuda")
    keys = keys / keys.abs().max() * 2.0 ** 124
    values = torch.randn(1, 2, n, 128, generator=g, device="cuda")
    q = torch.randn(1, 8, 128, generator=g, device="cuda") * 2.0 ** -121
    cache = mp.kv4_write(mp.kv4_cache(1, 2, n), keys, values)
    want, tol = _weighted64(q, cache, 2.0 ** -20)
    assert ((mp.kv4_attention(q, cache, scale=2.0 ** -20).double() - want).abs() <= tol).all()
