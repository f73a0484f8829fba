"""The 4-bit K/V cache on the host: its reference pinned by the definition, and the calls'
refusals, which happen before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

from tests import kv4_reference as R

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def L():
    from lsh_sampled_sparse_gb300.build import build
    build()
    import lsh_sampled_sparse_gb300 as mp
    return mp.lib()


def test_reference_meets_its_definition():
    rng = np.random.default_rng(5)
    x = np.concatenate([rng.normal(size=(300, 128)), 1e-3 * rng.normal(size=(50, 128)) + 7,
                        1e20 * rng.normal(size=(50, 128)), np.full((3, 128), 0.3),
                        np.zeros((1, 128))]).astype(np.float32)
    c, sb, zb = R.quantise(x)
    s, z = R.bf16_values(sb), R.bf16_values(zb)
    g = x.astype(np.float64).reshape(-1, 2, 64)
    assert c.min() >= 0 and c.max() <= 15
    assert (z <= g.min(-1)).all() and (z + 15 * s >= g.max(-1)).all()
    held = z[..., None] + s[..., None] * c.reshape(-1, 2, 64)
    assert (np.abs(held - g) <= s[..., None] / 2 * (1 + 1e-12)).all()
    # one bf16 step more or less breaks a condition: the next z above passes the minimum, the
    # next s below misses the maximum
    up = np.where(zb == 0x8000, 0x0001, np.where(zb >> 15, zb - 1, zb + 1)).astype(np.uint16)
    assert (R.bf16_values(up) > g.min(-1)).all()
    pos = sb > 0
    assert ((z + 15 * R.bf16_values((sb - pos).astype(np.uint16)))[pos] < g.max(-1)[pos]).all()


def test_reference_holds_what_is_not_finite_as_nan():
    x = np.zeros((4, 128), dtype=np.float32)
    x[0, 3], x[1, 64], x[2, 127] = np.nan, np.inf, -np.inf
    x[3, 0], x[3, 1] = 3e38, -3e38                     # the spread passes float32
    _, sb, zb = R.quantise(x)
    bad = np.array([[1, 0], [0, 1], [0, 1], [1, 0]], bool)
    assert ((sb == 0x7FC0) == bad).all() and ((zb == 0x7FC0) == bad).all()


def _cache(ptr=0x10000, cap=100, params=0x10000):
    from lsh_sampled_sparse_gb300.binding import _KV4
    return ctypes.byref(_KV4(ptr, ptr, params, cap))


def test_rows_reject_bad_arguments_before_launch(L):
    P = ctypes.c_void_p
    ok = P(0x10000)

    def write(keys=ok, dt=1, centre=ok, B=1, Hkv=1, m=10, d=128, n0=0, pos=None, cache=None):
        return L.mp_kv4_write(keys, ok, dt, centre, B, Hkv, m, d, n0, pos, cache or _cache(), None)

    def read(keys=ok, dt=1, centre=ok, B=1, Hkv=1, m=10, d=128, n0=0, pos=None, cache=None):
        return L.mp_kv4_read(cache or _cache(), centre, B, Hkv, m, d, n0, pos, keys, ok, dt, None)

    for f in (write, read):
        assert f(keys=None) == INVALID
        assert f(keys=P(0x10008)) == INVALID                   # misaligned
        assert f(centre=P(0x10008)) == INVALID
        assert f(pos=P(0x10002)) == INVALID
        assert f(dt=2) == INVALID
        assert f(B=0) == INVALID and f(Hkv=0) == INVALID and f(m=-1) == INVALID
        assert f(d=64) == UNSUPPORTED
        assert f(n0=-1) == INVALID and f(n0=91) == INVALID     # past the capacity
        assert f(n0=2 ** 31 - 5) == INVALID
        assert f(cache=_cache(cap=0)) == INVALID
        assert f(cache=_cache(ptr=0x10008)) == INVALID
        assert f(cache=_cache(params=None)) == INVALID
        assert f(B=2 ** 20, Hkv=2 ** 11, m=100) == INVALID     # more rows than a grid takes
        assert f(m=0, keys=None) == 0                          # nothing to do


def test_attention_rejects_bad_arguments_before_launch(L):
    P = ctypes.c_void_p
    ok = P(0x10000)

    def att(q=ok, dt=1, cache=None, B=1, Hq=4, Hkv=1, n=100, d=128, lengths=None, scale=0.0,
            out=ok, ws=ok, size=1 << 24):
        return L.mp_kv4_attention(q, dt, cache or _cache(), B, Hq, Hkv, n, d, lengths, scale, out,
                                  ws, size, None)

    assert att(q=None) == INVALID and att(out=None) == INVALID
    assert att(dt=3) == INVALID
    assert att(B=0) == INVALID and att(n=0) == INVALID and att(n=101) == INVALID
    assert att(Hq=6, Hkv=4) == INVALID
    assert att(scale=-1.0) == INVALID and att(scale=float("nan")) == INVALID
    assert att(scale=float("inf")) == INVALID
    assert att(q=P(0x10001)) == INVALID and att(out=P(0x10008)) == INVALID
    assert att(lengths=P(0x10002)) == INVALID
    assert att(cache=_cache(ptr=None)) == INVALID
    assert att(d=64) == UNSUPPORTED
    big = dict(n=100000, cache=_cache(cap=100000), Hq=32, Hkv=8)
    need = L.mp_kv4_attention_workspace_bytes(1, 32, 8, 100000, 128)
    assert need > 0 and need % 256 == 0
    assert att(**big, ws=None) == INVALID
    assert att(**big, ws=P(0x10010)) == INVALID
    assert att(**big, size=need - 1) == WORKSPACE
    assert L.mp_kv4_attention_workspace_bytes(1, 6, 4, 100, 128) == 0
    assert L.mp_kv4_attention_workspace_bytes(1, 4, 1, 0, 128) == 0
    assert L.mp_kv4_attention_workspace_bytes(1, 4, 1, 100, 64) == 0


def test_sampled_decode_rejects_bad_arguments_before_launch(L):
    import lsh_sampled_sparse_gb300 as mp
    P = ctypes.c_void_p
    ok = P(0x10000)
    prm = mp.Params(10, 150, 4, 64, 0.0, 0)

    def dec(cache=None, n=100, Hq=4, d=128, ws=1 << 24, q=ok):
        return L.mp_kv4_decode_attention(q, 1, ok, ok, ok, 1, cache or _cache(), 1, Hq, 1, n, d,
                                         ctypes.byref(prm), ok, ok, ws, None)

    def half(cache=None, n=100, Hq=4, d=128, ws=1 << 24, q=ok):
        return L.mp_kv4_sampled_attention(q, 1, ok, ok, cache or _cache(), 1, Hq, 1, n, d,
                                          ctypes.byref(prm), ok, ok, ws, None)

    def buckets(cache=None, n=100, Hq=4, d=128, ws=1 << 24, q=ok):
        return L.mp_kv4_sampled_attention_buckets(q, 1, ok, ok, ok, cache or _cache(), 1, Hq, 1, n,
                                                  d, ctypes.byref(prm), ok, ok, ws, None)

    for f in (dec, half, buckets):
        assert f(q=None) == INVALID
        assert f(cache=_cache(params=None)) == INVALID
        assert f(cache=_cache(ptr=0x10004)) == INVALID
        assert f(n=101) == INVALID                             # longer than the cache
        assert f(Hq=3) == UNSUPPORTED and f(d=64) == UNSUPPORTED
        assert f(ws=16) == WORKSPACE
    assert L.mp_kv4_sampled_attention_buckets(ok, 1, None, ok, ok, _cache(), 1, 4, 1, 100, 128,
                                              ctypes.byref(prm), ok, ok, 1 << 24, None) == INVALID


def test_binding_refuses_cpu_tensors(L):
    import lsh_sampled_sparse_gb300 as mp
    cache = mp.kv4_cache(1, 1, 16, device="cpu")
    x = torch.zeros(1, 1, 4, 128)
    with pytest.raises(TypeError):
        mp.kv4_write(cache, x, x)
    with pytest.raises(TypeError):
        mp.kv4_read(cache, 4)
    with pytest.raises(TypeError):
        mp.kv4_attention(torch.zeros(1, 1, 128), cache)


def test_encode_rows_rejects_bad_arguments_before_launch(L):
    P = ctypes.c_void_p
    ok = P(0x10000)

    def enc(keys=ok, kd=1, centre=ok, W=ok, wd=1, B=1, Hkv=1, m=10, cap=100, n0=0, d=128, K=10,
            tables=5, codes=ok):
        return L.mp_encode_rows(keys, kd, centre, W, wd, B, Hkv, m, cap, n0, d, K, tables, codes,
                                None)

    assert enc(keys=None) == INVALID and enc(centre=None) == INVALID
    assert enc(W=None) == INVALID and enc(codes=None) == INVALID
    assert enc(kd=2) == INVALID and enc(wd=-1) == INVALID
    assert enc(B=0) == INVALID and enc(Hkv=0) == INVALID and enc(m=-1) == INVALID
    assert enc(cap=0) == INVALID and enc(n0=-1) == INVALID and enc(n0=91) == INVALID
    assert enc(m=101) == INVALID and enc(n0=2 ** 31 - 5) == INVALID
    assert enc(K=33) == INVALID and enc(tables=0) == INVALID
    assert enc(keys=P(0x10008)) == INVALID and enc(codes=P(0x10004)) == INVALID
    assert enc(centre=P(0x10002)) == INVALID and enc(W=P(0x10001)) == INVALID
    assert enc(d=64) == UNSUPPORTED
    assert enc(m=0, keys=None) == 0 and enc(K=0, codes=None) == 0      # nothing to do
