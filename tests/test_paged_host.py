"""The paged cache on the host: the calls' refusals, which happen before anything is launched, and what
reading the source of its kernels has to show."""
import ctypes
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "lsh_sampled_sparse_gb300", "csrc")
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
P = ctypes.c_void_p
OK = P(0x10000)


@pytest.fixture(scope="module")
def L():
    from lsh_sampled_sparse_gb300.build import build
    build()
    import lsh_sampled_sparse_gb300 as mp
    return mp.lib()


def _cache(keys=0x10000, table=0x10000, dtype=1, n_pages=10, page=16, slots=7, stride=None):
    from lsh_sampled_sparse_gb300.binding import _PAGED
    return _PAGED(keys or 0, 0x10000, table or 0, dtype, n_pages, page, slots,
                  slots if stride is None else stride)


def _rows(data=0x10000, sb=1 << 20, sh=1 << 10, sm=128):
    from lsh_sampled_sparse_gb300.binding import _ROWS
    return _ROWS(data or 0, sb, sh, sm)


BAD_CACHES = [(dict(keys=None), INVALID), (dict(keys=0x10008), INVALID), (dict(table=None), INVALID),
              (dict(table=0x10002), INVALID), (dict(dtype=2), INVALID), (dict(n_pages=0), INVALID),
              (dict(page=0), INVALID), (dict(slots=0), INVALID), (dict(stride=6), INVALID),
              (dict(page=12), UNSUPPORTED), (dict(page=2 ** 30, slots=2), INVALID),
              (dict(n_pages=2 ** 27 + 1), INVALID)]


def test_append_rejects_bad_arguments_before_launch(L):
    def app(k=None, v=None, q=None, dt=1, freq=OK, rotary=128, B=2, Hq=4, Hkv=2, m=10, d=128, n0=0,
            pos=None, counts=None, cache=None, q_out=OK, k_out=None):
        return L.mp_paged_append(k or _rows(), v or _rows(), q, dt, freq, rotary, 0, B, Hq, Hkv, m, d,
                                 n0, pos, counts, cache or _cache(), q_out, k_out, None)

    for kw, status in BAD_CACHES:
        assert app(cache=_cache(**kw)) == status, kw
    assert app(k=_rows(data=None)) == INVALID and app(v=_rows(data=0x10008)) == INVALID
    assert app(k=_rows(sb=4)) == INVALID and app(k=_rows(sh=4)) == INVALID
    assert app(v=_rows(sm=4)) == INVALID
    assert app(dt=0, v=_rows(sm=2)) == INVALID             # 8 bytes in float32
    assert app(dt=3) == INVALID
    assert app(q=_rows(data=0x10008)) == INVALID and app(q=_rows(), q_out=None) == INVALID
    assert app(q=_rows(), Hq=0) == INVALID
    assert app(q_out=P(0x10008)) == INVALID and app(k_out=P(0x10004)) == INVALID
    assert app(freq=P(0x10002)) == INVALID
    assert app(pos=P(0x10002)) == INVALID and app(counts=P(0x10001)) == INVALID
    assert app(B=0) == INVALID and app(Hkv=0) == INVALID and app(m=-1) == INVALID
    assert app(n0=-1) == INVALID and app(n0=103) == INVALID                # past 7 pages of 16
    assert app(n0=2 ** 31 - 5) == INVALID
    assert app(d=64) == UNSUPPORTED
    for r in (0, 8, 24, 144):
        assert app(rotary=r) == UNSUPPORTED
    assert app(B=2 ** 20, m=2 ** 10, pos=OK, Hkv=2) == INVALID             # rows past 2^31
    assert app(q=_rows(), Hq=2 ** 18, B=1, m=1) == INVALID                 # more heads than a grid has
    assert app(m=0, k=_rows(data=None)) == 0                               # nothing to do


def test_attention_rejects_bad_arguments_before_launch(L):
    def att(q=OK, dt=1, cache=None, B=1, Hq=4, Hkv=1, n=100, d=128, lengths=None, scale=0.0, out=OK,
            ws=OK, size=1 << 28):
        return L.mp_paged_attention(q, dt, cache or _cache(), B, Hq, Hkv, n, d, lengths, scale, out, ws,
                                    size, None)

    for kw, status in BAD_CACHES:
        assert att(cache=_cache(**kw)) == status, kw
    assert att(q=None) == INVALID and att(out=None) == INVALID and att(ws=None) == INVALID
    assert att(dt=3) == INVALID
    assert att(B=0) == INVALID and att(n=0) == INVALID and att(n=113) == INVALID
    assert att(Hq=6, Hkv=4) == INVALID
    assert att(scale=-1.0) == INVALID and att(scale=float("nan")) == INVALID
    assert att(scale=float("inf")) == INVALID
    assert att(q=P(0x10001)) == INVALID and att(out=P(0x10008)) == INVALID
    assert att(lengths=P(0x10002)) == INVALID and att(ws=P(0x10010)) == INVALID
    assert att(d=64) == UNSUPPORTED
    need = L.mp_paged_attention_workspace_bytes(1, 4, 1, 100, 128)
    assert need > 0 and need % 256 == 0
    assert need == L.mp_paged_attention_workspace_bytes(1, 4, 1, 100000, 128)
    assert att(size=need - 1) == WORKSPACE
    assert L.mp_paged_attention_workspace_bytes(1, 6, 4, 100, 128) == 0
    assert L.mp_paged_attention_workspace_bytes(1, 4, 1, 0, 128) == 0
    assert L.mp_paged_attention_workspace_bytes(1, 4, 1, 100, 64) == 0


def test_sampled_decode_rejects_bad_arguments_before_launch(L):
    import lsh_sampled_sparse_gb300 as mp

    def dec(cache=None, n=100, Hq=4, d=128, ws=1 << 24, q=OK, lengths=None, cap=0, codes=OK):
        prm = mp.Params(10, 150, 4, 64, 0.0, 0, cap)
        return L.mp_paged_decode_attention(q, 1, codes, OK, OK, 1, cache or _cache(), 1, Hq, 1, n, d,
                                           lengths, ctypes.byref(prm), OK, OK, ws, None)

    for kw, status in BAD_CACHES:
        assert dec(cache=_cache(**kw)) == status, kw
    assert dec(q=None) == INVALID and dec(codes=None) == INVALID
    assert dec(lengths=P(0x10002)) == INVALID
    assert dec(n=113) == INVALID and dec(n=0) == INVALID and dec(cap=99) == INVALID
    assert dec(Hq=3) == UNSUPPORTED and dec(d=64) == UNSUPPORTED
    assert dec(ws=16) == WORKSPACE


def test_encode_rows_at_rejects_bad_arguments_before_launch(L):
    def enc(keys=OK, B=2, Hkv=2, m=3, cap=100, pos=OK, d=128, K=10, codes=OK, W=OK):
        return L.mp_encode_rows_at(keys, 1, OK, W, 1, B, Hkv, m, cap, pos, d, K, 150, codes, None)

    assert enc(keys=None) == INVALID and enc(codes=None) == INVALID and enc(W=None) == INVALID
    assert enc(pos=None) == INVALID and enc(pos=P(0x10002)) == INVALID
    assert enc(keys=P(0x10008)) == INVALID and enc(codes=P(0x10008)) == INVALID
    assert enc(B=0) == INVALID and enc(m=-1) == INVALID and enc(cap=0) == INVALID
    assert enc(K=33) == INVALID
    assert enc(B=2 ** 18, Hkv=2) == INVALID
    assert enc(m=65) == UNSUPPORTED and enc(d=64) == UNSUPPORTED
    assert enc(m=0, keys=None) == 0 and enc(K=0, keys=None) == 0


@pytest.mark.parametrize("name,count", [("mp_paged.cu", 3), ("mp_paged_tc.cu", 1), ("mp_paged_mma.cu", 1)])
def test_dependent_kernels_of_the_paged_cache_make_no_non_coherent_load(name, count):
    """A kernel launched as a dependent begins before its predecessor has written positions, lengths,
    tables, queries or rows; a non-coherent load promises that nobody writes them during its life."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "__ldg(" not in code and ".global.nc" not in code and "__restrict__" not in code
    assert "<<<" not in code
    kernels = re.findall(r"__global__.*?\n}\n", code, re.S)
    assert len(kernels) >= count and all("wait_for_predecessor();" in k for k in kernels)


@pytest.mark.parametrize("total", [1, 2, 7, 151, 152, 153, 1000, 10007, 2 ** 45 + 3])
@pytest.mark.parametrize("ctas", [1, 152, 304])
def test_the_shares_of_a_call_cover_its_tiles_once(total, ctas):
    """The arithmetic that shares tiles out to CTAs and finds a tile's CTA again."""
    n = min(ctas, total)
    each, more = total // n, total % n
    first = [each * c + min(c, more) for c in range(n + 1)]
    assert first[0] == 0 and first[-1] == total and all(a < b for a, b in zip(first, first[1:]))
    for c in range(n):
        for t in {first[c], (first[c] + first[c + 1] - 1) // 2, first[c + 1] - 1}:
            of = t // (each + 1) if t < more * (each + 1) else more + (t - more * (each + 1)) // each
            assert of == c
    for size in range(1, 9):                     # a cluster's ranks
        part = [r * total // size for r in range(size + 1)]
        assert part[0] == 0 and part[-1] == total and all(a <= b for a, b in zip(part, part[1:]))
