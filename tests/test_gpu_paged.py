"""The paged cache on the GPU against its definition in 64 bits (tests/paged_reference.py): tokens
appended with their rotary positions, exact attention and the sampled decode over the pages, codes of
tokens that join sequences of different lengths, and a run of them together."""
import pytest
import torch

from tests import paged_reference as R
from workloads import make_hyperplanes, make_layer, small_workload

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lsh_sampled_sparse_gb300 as mp
    mp.lib()
    return mp


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, B, slots, extra=2):
    """Pages dealt out at random, and how many there are."""
    n = B * slots + extra
    return torch.randperm(n, generator=g, device="cuda")[:B * slots].view(B, slots).int(), n


def _inv_freq(r, theta=500000.0):
    return (theta ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)).float()


def _bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def _filled(mp, n_pages, Hkv, page, dtype):
    """A pool whose every element is a NaN of its own."""
    c = mp.paged_cache(n_pages, Hkv, page, dtype)
    for t in c:
        _bits(t).fill_(0x7FA5 if dtype == BF else 0x7FA5A5A5)
    return c


# ---------------------------------------------------------------- append
def _check_append(cache, before, table, starts, counts, k_want, k_tol, v_want):
    """Every row of the pool: the written ones within the tolerance, the others as before."""
    n_pages, Hkv, page, _ = cache.keys.shape
    B, _, m, _ = k_want.shape
    dtype = cache.keys.dtype
    left = [t.clone() for t in before]
    for b in range(B):
        for i in range(counts[b]):
            p = starts[b] + i
            if not 0 <= p < table.shape[1] * page:
                continue
            pg = int(table[b, p // page])
            if not 0 <= pg < n_pages:
                continue
            got = cache.keys[pg, :, p % page].double()
            tol = R.rounded(k_tol[b, :, i], k_want[b, :, i], dtype)
            assert ((got - k_want[b, :, i]).abs() <= tol).all(), (b, i)
            left[0][pg, :, p % page] = cache.keys[pg, :, p % page]
            left[1][pg, :, p % page] = v_want[b, :, i].to(dtype)
    assert torch.equal(_bits(cache.keys), _bits(left[0]))
    assert torch.equal(_bits(cache.values), _bits(left[1]))


@pytest.mark.parametrize("rows", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hq,Hkv,m,page,r,interleaved", [
    (1, 1, 1, 1, 8, 128, False), (3, 6, 2, 17, 24, 64, True), (2, 10, 5, 133, 16, 96, False),
    (32, 4, 1, 1, 64, 16, True), (1, 32, 8, 700, 48, 128, True), (5, 3, 3, 9, 8, 112, False)])
def test_append_turns_and_writes(mp, rows, dtype, B, Hq, Hkv, m, page, r, interleaved):
    g = _gen(m + r)
    slots = -(-(m + 40) // page)
    table, n_pages = _table(g, B, slots)
    cache = _filled(mp, n_pages, Hkv, page, dtype)
    before = [t.clone() for t in cache]
    x = _randn(g, B, m, Hq + 2 * Hkv, 128).to(rows).transpose(1, 2)      # one projection's output
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    starts = [int(s) for s in torch.randint(0, slots * page - m + 1, (B,))]
    pos, freq = _ints(starts), _inv_freq(r)
    keys_out = torch.full((B, Hkv, m, 128), 7.0, dtype=dtype, device="cuda")
    q_out = mp.paged_append(cache, table, k, v, positions=pos, inv_freq=freq,
                            interleaved=interleaved, q=q, keys_out=keys_out)
    q_want, q_tol = R.turned(q, pos, freq, interleaved)
    assert q_out.dtype == rows and q_out.shape == q.shape
    assert ((q_out.double() - q_want).abs() <= R.rounded(q_tol, q_want, rows)).all()
    k_want, k_tol = R.turned(k, pos, freq, interleaved)
    _check_append(cache, before, table.cpu(), starts, [m] * B, k_want, k_tol, v)
    for b in range(B):                           # the keys returned are the ones held
        for i in range(m):
            p = starts[b] + i
            assert torch.equal(keys_out[b, :, i], cache.keys[table[b, p // page], :, p % page])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_without_rotation_counts_and_places_that_do_not_exist(mp, dtype):
    B, Hkv, m, page, slots = 9, 3, 13, 8, 5
    g = _gen(3)
    table, n_pages = _table(g, B, slots)
    table[3, 1], table[4, 0], table[4, 2] = -1, n_pages, 2 ** 31 - 1     # no pages
    wide = torch.full((B, 11), -7, dtype=torch.int32, device="cuda")     # a view of a wider table
    wide[:, 2:2 + slots] = table
    view = wide[:, 2:2 + slots]
    cache = _filled(mp, n_pages, Hkv, page, dtype)
    before = [t.clone() for t in cache]
    k, v = _randn(g, B, Hkv, m, 128).to(dtype), _randn(g, B, Hkv, m, 128).to(dtype)
    starts = [0, 30, 27, 5, 3, -4, 2 ** 31 - 1, -2 ** 31, 40]
    counts = [13, 99, 13, 13, 13, 7, 13, 13, -1]
    used = [max(0, min(m, c)) for c in counts]
    keys_out = torch.full((B, Hkv, m, 128), 7.0, dtype=dtype, device="cuda")
    assert mp.paged_append(cache, view, k, v, positions=_ints(starts), counts=_ints(counts),
                           keys_out=keys_out) is None
    _check_append(cache, before, table.cpu(), starts, used, k.double(), torch.zeros_like(k).double(), v)
    for b in range(B):
        assert torch.equal(keys_out[b, :, :used[b]], k[b, :, :used[b]])
        assert (keys_out[b, :, used[b]:] == 7).all()
    # no positions: every sequence from n_begin on
    cache = _filled(mp, n_pages, Hkv, page, dtype)
    before = [t.clone() for t in cache]
    mp.paged_append(cache, view, k, v, n_begin=27)
    _check_append(cache, before, table.cpu(), [27] * B, [m] * B, k.double(),
                  torch.zeros_like(k).double(), v)


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_of_far_positions(mp, interleaved):
    """float32 angles would be off by 4e-3 at 2^17 already; the reduction's 2^-51 of the angle is 5e-7 at
    2^30."""
    starts = [0, 1, 131071, 2 ** 20 + 3, 2 ** 25 + 1, 2 ** 30 - 77, -5, -2 ** 30]
    B = len(starts)
    g = _gen(4)
    cache = mp.paged_cache(B, 1, 8, F32)
    table = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    k = _randn(g, B, 1, 3, 128)
    freq = torch.cat([_inv_freq(124), torch.tensor([37.5, 0.0], device="cuda")])
    keys_out = torch.empty_like(k)
    mp.paged_append(cache, table, k, k, positions=_ints(starts), inv_freq=freq,
                    interleaved=interleaved, keys_out=keys_out)
    want, tol = R.turned(k, _ints(starts), freq, interleaved)
    far = torch.tensor([abs(s) for s in starts], dtype=torch.float64, device="cuda").view(B, 1, 1, 1)
    # 2^-51 of an angle of the fastest pair, in the kernel and (its product and its own reduction) in
    # the reference
    tol = tol + 2 * 2.0 ** -51 * 37.5 * far * tol / (10 * R.E)
    assert ((keys_out.double() - want).abs() <= R.rounded(tol, want, F32)).all()


def test_append_in_place_and_rows_of_repeated_heads(mp):
    B, H, m, page = 2, 4, 6, 8
    g = _gen(5)
    table, n_pages = _table(g, B, 2)
    cache = mp.paged_cache(n_pages, H, page, F32)
    one = _randn(g, B, 1, m, 128)
    k = one.expand(B, H, m, 128)                                         # stride 0
    q = _randn(g, B, H, m, 128)
    want = mp.paged_append(cache, table, k, k, n_begin=3, inv_freq=_inv_freq(128), q=q.clone())
    first = cache.keys.clone()
    assert mp.paged_append(cache, table, k.contiguous(), k, n_begin=3, inv_freq=_inv_freq(128), q=q,
                           q_out=q) is q
    assert torch.equal(q, want) and torch.equal(_bits(cache.keys), _bits(first))
    assert torch.equal(cache.keys[table[0, 0], 0, 3:], cache.keys[table[0, 0], 3, 3:])


# ---------------------------------------------------------------- exact attention
def _random_cache(mp, g, B, Hkv, n, page, dtype, used, fill=float("nan")):
    """A cache of random rows; what lies behind a sequence's length, and in no page, is `fill`."""
    slots = -(-n // page)
    table, n_pages = _table(g, B, slots)
    cache = mp.paged_cache(n_pages, Hkv, page, dtype)
    for t in cache:
        t.fill_(fill)
    for b in range(B):
        for t in cache:
            x = torch.full((Hkv, slots * page, 128), fill, device="cuda")
            x[:, :used[b]] = _randn(g, Hkv, used[b], 128)
            t[table[b].long()] = x.view(Hkv, slots, page, 128).transpose(0, 1).to(dtype)
        table[b, -(-used[b] // page):] = -1
    return cache, table


def _attend_and_check(mp, q, cache, table, n, used, lengths=None, scale=0.0, **kw):
    out = mp.paged_attention(q, cache, table, n=n, lengths=lengths, scale=scale, **kw)
    want, tol = R.attention(q, cache.keys, cache.values, table.cpu(), used, scale or 128 ** -0.5)
    bad = (out.double() - want).abs() > tol
    assert not bad.any(), (bad.nonzero()[:5].tolist(),
                           ((out.double() - want).abs() / tol.clamp_min(1e-300)).max().item())
    return out


@pytest.mark.parametrize("qt", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hkv,G,n,page", [
    (1, 1, 1, 1, 8), (1, 2, 4, 127, 16), (2, 3, 5, 128, 24), (1, 8, 4, 129, 64), (3, 1, 8, 1000, 48),
    (1, 2, 12, 777, 128), (1, 1, 16, 4100, 8), (2, 2, 20, 300, 256), (1, 8, 4, 20000, 16),
    (1, 1, 3, 30001, 40), (5, 7, 2, 1333, 1024)])
def test_attention_against_64_bits(mp, qt, dtype, B, Hkv, G, n, page):
    g = _gen(n + G)
    cache, table = _random_cache(mp, g, B, Hkv, n, page, dtype, [n] * B)
    q = (_randn(g, B, Hkv * G, 128) * 2).to(qt)
    _attend_and_check(mp, q, cache, table, n, [n] * B)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G", [1, 4, 7, 12])
def test_attention_of_sequences_of_different_lengths(mp, dtype, G):
    lens = [0, 1, 5, 128, 0, 129, 127, 2000, 2003, 64, 1999, 0]
    g = _gen(G)
    n, page = 2003, 16
    cache, table = _random_cache(mp, g, 12, 2, n, page, dtype, lens)
    q = _randn(g, 12, 2 * G, 128).to(dtype)
    out = _attend_and_check(mp, q, cache, table, n, lens, _ints(lens))
    assert all((out[b] == 0).all() for b in (0, 4, 11))
    # lengths outside [0, n] are taken into it
    wild = [v - 3 if v == 0 else v + (2 ** 31 - 1 - v if v == n else 0) for v in lens]
    assert torch.equal(mp.paged_attention(q, cache, table, n=n, lengths=_ints(wild)), out)
    # the table's whole capacity in place of n
    assert torch.equal(mp.paged_attention(q, cache, table, lengths=_ints(lens)), out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B", [151, 700])
def test_attention_of_many_sequences(mp, dtype, B):
    """More sequences than a CTA has threads, many of them empty."""
    g = _gen(B)
    n = 400
    lens = torch.randint(-100, n + 1, (B,), generator=torch.Generator().manual_seed(B)).clamp_min(0)
    lens = [int(v) for v in lens]
    cache, table = _random_cache(mp, g, B, 2, n, 16, dtype, lens)
    q = _randn(g, B, 6, 128).to(dtype)
    _attend_and_check(mp, q, cache, table, n, lens, _ints(lens))
    none = torch.zeros(B, dtype=torch.int32, device="cuda")
    assert (mp.paged_attention(q, cache, table, n=n, lengths=none) == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_tokens_without_a_page_are_not_there(mp, dtype, page):
    B, n = 3, 1500
    g = _gen(page)
    cache, table = _random_cache(mp, g, B, 2, n, page, dtype, [n] * B)
    table[0, 0], table[0, 3] = -1, cache.keys.shape[0]
    table[1, :] = -2 ** 31
    table[2, 2:] = 2 ** 31 - 1
    q = _randn(g, B, 8, 128).to(dtype)
    out = _attend_and_check(mp, q, cache, table, n, [n] * B)
    assert (out[1] == 0).all()
    # pages that sequences share
    table[1] = table[2] = table[0]
    q[1:] = q[0]
    out = _attend_and_check(mp, q, cache, table, n, [n] * B)
    # (sums of the same keys, shared out to CTAs at other places)
    assert (out[1] - out[0]).abs().max() < 1e-4


@pytest.mark.parametrize("qt", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_with_sharp_scores_and_a_scale_of_its_own(mp, qt, dtype):
    g = _gen(6)
    n = 3000
    cache, table = _random_cache(mp, g, 2, 2, n, 16, dtype, [n, n])
    q = (_randn(g, 2, 8, 128) * 30).to(qt)
    _attend_and_check(mp, q, cache, table, n, [n, n], scale=0.25)
    _attend_and_check(mp, q, cache, table, n, [n, n], scale=1e-20)
    for t in cache:
        t.mul_(1e18)
    _attend_and_check(mp, q.mul(1e-18), cache, table, n, [n, n])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_where_a_new_maximum_comes_late(mp, dtype):
    """Scores that grow along the sequence: every tile moves the running maximum."""
    g = _gen(7)
    n = 2500
    cache, table = _random_cache(mp, g, 1, 1, n, 16, dtype, [n])
    q = _randn(g, 1, 4, 128).to(dtype)
    u = q[0].float().mean(0) / q[0].float().mean(0).norm() ** 2
    rows = cache.keys[table[0].long()].transpose(0, 1).reshape(1, -1, 128)
    rows = rows.float() + torch.arange(rows.shape[1], device="cuda").view(1, -1, 1) * 0.3 * u
    cache.keys[table[0].long()] = rows.to(dtype).view(1, -1, 16, 128).transpose(0, 1)
    _attend_and_check(mp, q, cache, table, n, [n])
    flipped = table.flip(1)                      # ... and scores that fall
    _attend_and_check(mp, q, cache, flipped, n - 2500 % 16, [n - 2500 % 16])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G", [2, 7, 11])
def test_attention_passes_nan_and_infinity_on(mp, dtype, G):
    n = 400
    g = _gen(12)
    cache, table = _random_cache(mp, g, 3, 1, n, 16, dtype, [n] * 3)

    def at(b, i):
        return int(table[b, i // 16]), 0, i % 16

    cache.values[at(0, 111)][100] = float("nan")
    cache.keys[at(1, 222)][5] = float("nan")
    q = _randn(g, 3, G, 128)
    q[2, 1, 7] = float("inf")
    out = mp.paged_attention(q, cache, table, n=n)
    nan = torch.isnan(out)
    assert nan[0, :, 100].all() and not nan[0, :, :100].any() and not nan[0, :, 101:].any()
    assert nan[1].all()
    assert not nan[2, 0].any() and nan[2, 1].all() and not nan[2, 2:].any()
    short = _ints([111, 222, 400])               # ends before the bad token
    q[2, 1, 7] = 0.0
    _attend_and_check(mp, q, cache, table, n, [111, 222, 400], short)
    for b in range(2):                           # the page that holds it is shut out
        table[b, (111, 222)[b] // 16] = -1
    _attend_and_check(mp, q, cache, table, n, [n] * 3)
    cache.keys[at(2, 17)][:] = float("-inf")     # scores of -inf and NaN
    assert torch.isnan(mp.paged_attention(q, cache, table, n=n)[2]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_queries_aligned_to_their_element_only(mp, dtype):
    g = _gen(8)
    n = 500
    cache, table = _random_cache(mp, g, 1, 2, n, 16, dtype, [n])
    for qt in (BF, F32):
        q = _randn(g, 1, 8, 128).to(qt)
        room = torch.empty(q.numel() + 1, dtype=qt, device="cuda")
        odd = room[1:].view(q.shape)
        odd.copy_(q)
        assert torch.equal(mp.paged_attention(odd, cache, table, n=n),
                           mp.paged_attention(q, cache, table, n=n))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_beyond_2_to_the_32_bytes(mp, dtype):
    size = 2 if dtype == BF else 4
    page, Hkv = 256, 3
    n_pages = (1 << 32) // (page * Hkv * 128 * size) + 9
    cache = mp.paged_cache(n_pages, Hkv, page, dtype)
    g = _gen(4)
    table = torch.stack([torch.arange(n_pages - 3, n_pages), torch.arange(3)]).int().cuda()
    n = 700
    k, v = _randn(g, 2, Hkv, n, 128).to(dtype), _randn(g, 2, Hkv, n, 128).to(dtype)
    mp.paged_append(cache, table, k, v)
    q = _randn(g, 2, 6, 128)
    _attend_and_check(mp, q, cache, table, n, [n, n])
    want, _ = R.held(cache.keys, table.cpu(), 0, n)
    assert torch.equal(want, k[0].double())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_runs_agree_bit_for_bit_and_streams_and_graphs_do_not_mix(mp, dtype):
    B, Hkv, n, page = 2, 4, 6000, 16
    g = _gen(21)
    cache, table = _random_cache(mp, g, B, Hkv, n, page, dtype, [n] * B, fill=0.0)
    q = _randn(g, B, 16, 128).to(dtype)
    first = mp.paged_attention(q, cache, table, n=n)
    assert all(torch.equal(mp.paged_attention(q, cache, table, n=n), first) for _ in range(5))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out = mp.paged_attention(q, cache, table, n=n, stream=other)
    other.synchronize()
    assert torch.equal(out, first)
    # one token appended and attended to, captured, replayed on new data
    k, v = _randn(g, B, Hkv, 1, 128).to(dtype), _randn(g, B, Hkv, 1, 128).to(dtype)
    qr = _randn(g, B, 16, 1, 128).to(dtype)
    pos = torch.full((B,), 100, dtype=torch.int32, device="cuda")
    lengths, freq = pos + 1, _inv_freq(128)
    size = mp.paged_attention_workspace_bytes(B, 16, Hkv, n)
    graphs = []
    for _ in range(2):
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        res, turned = torch.empty(B, 16, 128, device="cuda"), torch.empty_like(qr)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mp.paged_append(cache, table, k, v, positions=pos, inv_freq=freq, q=qr, q_out=turned)
            mp.paged_attention(turned[:, :, 0], cache, table, lengths=lengths, out=res, workspace=ws)
        graphs.append((graph, res, ws, turned))
    for step in range(3):
        k.normal_()
        v.normal_()
        pos.copy_(_ints([200 * step + 7, 5990 - step]))
        lengths.copy_(pos + 1)
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        expect = _attend_and_check(mp, graphs[0][3][:, :, 0].contiguous(), cache, table, n,
                                   lengths.tolist(), lengths)
        assert torch.equal(graphs[0][1], expect) and torch.equal(graphs[1][1], expect)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_back_to_back_equal_calls_waited_for(mp, dtype):
    """Queued calls overlap at their ends: lengths, tables and queries written just before a call, and
    one workspace and output for all of them."""
    B, Hkv, n, page = 6, 4, 1500, 16
    g = _gen(33)
    cache, table = _random_cache(mp, g, B, Hkv, n, page, dtype, [n] * B)
    qs = [_randn(g, B, 16, 128).to(dtype) for _ in range(12)]
    lens = [torch.randint(0, n + 1, (B,), device="cuda").int() for _ in range(12)]
    tables = [table[torch.randperm(B, device="cuda")].contiguous() for _ in range(12)]
    ws = torch.empty(mp.paged_attention_workspace_bytes(B, 16, Hkv, n), dtype=torch.uint8,
                     device="cuda")
    want = []
    for q, ln, tb in zip(qs, lens, tables):
        want.append(mp.paged_attention(q, cache, tb, lengths=ln, n=n))
        torch.cuda.synchronize()
    q, ln, tb = torch.empty_like(qs[0]), torch.empty_like(lens[0]), torch.empty_like(tables[0])
    out, got = torch.empty_like(want[0]), []
    for i in range(12):
        q.copy_(qs[i])
        ln.copy_(lens[i])
        tb.copy_(tables[i])
        mp.paged_attention(q, cache, tb, lengths=ln, n=n, out=out, workspace=ws)
        got.append(out.clone())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_table_that_repeats_pages_over_a_long_context(mp, dtype):
    """Four million tokens in 37 pages, and a table that is a view of a wider one."""
    g = _gen(41)
    page, pages, slots = 8, 37, 1 << 19
    n = slots * page - 3
    cache = mp.paged_cache(pages, 1, page, dtype)
    for t in cache:
        t.copy_(_randn(g, *t.shape))
    wide = torch.full((2, slots + 5), -1, dtype=torch.int32, device="cuda")
    table = wide[:, :slots]
    table.copy_(torch.randint(0, pages, (2, slots), generator=g, device="cuda"))
    q = _randn(g, 2, 2, 128).to(dtype)
    lens = [n, n // 3]
    out = mp.paged_attention(q, cache, table, n=n, lengths=_ints(lens))
    k, v = (t.double().view(-1, 128) for t in cache)
    for b in range(2):
        tok = torch.arange(lens[b], device="cuda")
        times = torch.bincount(table[b, tok // page].long() * page + tok % page, minlength=pages * page)
        logits = q[b].double() @ k.T * 128 ** -0.5
        want = torch.softmax(logits + times.double().log(), -1) @ v
        A = (q[b].double().abs() @ k.abs().T * 128 ** -0.5).max()
        # paged_reference.attention's
        tol = R.E * (2 * (32 * A + 4) + 4 * lens[b] ** 0.5 + 16) * v.abs().max()
        assert ((out[b].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_on_two_streams_at_once(mp, dtype):
    """Each with its workspace, on one pool: one stream's sequences grow while the other's are read."""
    B, Hkv, n, page = 4, 4, 3000, 16
    g = _gen(51)
    cache, table = _random_cache(mp, g, 2 * B, Hkv, n, page, dtype, [n] * 2 * B)
    q = _randn(g, 2 * B, 16, 128).to(dtype)
    rows = [_randn(g, 2, B, Hkv, 1, 128).to(dtype) for _ in range(8)]
    halves = (slice(0, B), slice(B, 2 * B))
    want = [[], []]
    start = [t.clone() for t in cache]
    for i in range(8):
        for j, part in enumerate(halves):
            mp.paged_append(cache, table[part], rows[i][j], rows[i][j], n_begin=7 * i)
            want[j].append(mp.paged_attention(q[part], cache, table[part], n=n - 100 * i))
            torch.cuda.synchronize()
    for t, was in zip(cache, start):
        t.copy_(was)
    streams = [torch.cuda.Stream() for _ in halves]
    ws = [torch.empty(mp.paged_attention_workspace_bytes(B, 16, Hkv, n), dtype=torch.uint8, device="cuda")
          for _ in halves]
    outs = [[torch.empty(B, 16, 128, device="cuda") for _ in range(8)] for _ in halves]
    torch.cuda.synchronize()
    for i in range(8):
        for j, part in enumerate(halves):
            mp.paged_append(cache, table[part], rows[i][j], rows[i][j], n_begin=7 * i, stream=streams[j])
            mp.paged_attention(q[part], cache, table[part], n=n - 100 * i, out=outs[j][i], workspace=ws[j],
                               stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[j], want[j]))


def test_what_was_handed_in_is_filled_and_no_more(mp):
    g = _gen(31)
    for dtype, Hq in ((BF, 8), (F32, 8), (BF, 24), (F32, 16), (F32, 24)):
        cache, table = _random_cache(mp, g, 1, 2, 30000, 16, dtype, [30000])
        q = _randn(g, 1, Hq, 128).to(BF)
        room = torch.full((3, Hq, 128), 7.0, device="cuda")
        size = mp.paged_attention_workspace_bytes(1, Hq, 2, 30000)
        ws = torch.full((size + 4096,), 0xEE, dtype=torch.uint8, device="cuda")
        out = mp.paged_attention(q, cache, table, out=room[1:2], workspace=ws, n=30000)
        assert out.data_ptr() == room[1].data_ptr()
        assert torch.equal(out, mp.paged_attention(q, cache, table, n=30000))
        assert (room[0] == 7).all() and (room[2] == 7).all()
        assert (ws[size:] == 0xEE).all()


# ---------------------------------------------------------------- codes
@pytest.mark.parametrize("kd,wd", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("B,Hkv,m,cap,K,L", [(1, 1, 1, 1, 10, 150), (5, 3, 17, 3001, 8, 75),
                                             (9, 2, 64, 2000, 3, 5), (40, 1, 2, 1100, 12, 33)])
def test_codes_at_places_of_their_own_equal_encode_rows(mp, kd, wd, B, Hkv, m, cap, K, L):
    g = _gen(cap)
    keys, W = _randn(g, B, Hkv, m, 128).to(kd), _randn(g, 128, K * L).to(wd)
    centre = _randn(g, B, Hkv, 128)
    starts = [int(s) for s in torch.randint(0, cap - m + 1, (B,))]
    words = mp.codes_bytes(1, Hkv, cap, K, L) // 4
    codes = torch.randint(-2 ** 31, 2 ** 31, (B, words), device="cuda", dtype=torch.int32)
    want = codes.clone()
    for b, s in enumerate(starts):
        # short ranges go the same way in the sums
        mp.encode_rows(keys[b:b + 1], centre[b:b + 1], W, K, L, s, cap, codes=want[b])
    got = mp.encode_rows_at(keys, centre, W, K, L, _ints(starts), cap, codes)
    assert got is codes and torch.equal(codes, want)


def test_codes_outside_the_capacity_are_left_out(mp):
    B, m, cap, K, L = 7, 5, 70, 4, 9
    g = _gen(2)
    keys, W = _randn(g, B, 1, m, 128), _randn(g, 128, K * L)
    centre = torch.zeros(B, 1, 128, device="cuda")
    starts = [-3, 0, 66, 70, -5, 2 ** 31 - 1, -2 ** 31]
    codes = torch.full((B, mp.codes_bytes(1, 1, cap, K, L) // 4), 0x5A5A5A5A, dtype=torch.int32,
                       device="cuda")
    want = codes.clone()
    for b, s in enumerate(starts):
        lo, hi = max(0, -s), min(m, cap - s)
        if lo < hi:
            mp.encode_rows(keys[b:b + 1, :, lo:hi].contiguous(), centre[b:b + 1], W, K, L, s + lo, cap,
                           codes=want[b])
    mp.encode_rows_at(keys, centre, W, K, L, _ints(starts), cap, codes)
    assert torch.equal(codes, want)


# ---------------------------------------------------------------- the sampled decode
def _pages_of(mp, g, x, cap, page):
    """The rows of a contiguous cache [B, Hkv, n, 128] in pages of a table for cap tokens."""
    B, Hkv, n, _ = x["keys"].shape
    slots = -(-cap // page)
    table, n_pages = _table(g, B, slots)
    cache = mp.paged_cache(n_pages, Hkv, page, x["keys"].dtype)
    for t in cache:
        t.fill_(float("nan"))
    mp.paged_append(cache, table, x["keys"], x["values"])
    return cache, table


def _chosen(mp, x, codes, centre, W, lens, cap, args, Hkv, **extra):
    """What each query samples, from the contiguous cache's inspection call (tested against the oracle
    elsewhere), a sequence at a time."""
    B, Hq, _ = x["q"].shape
    n = x["keys"].shape[2]
    wide = torch.zeros(B, Hkv, cap, 128, dtype=x["keys"].dtype, device="cuda")
    wide[:, :, :n] = x["keys"]
    per = codes.numel() // B
    chosen = []
    for b in range(B):
        rows = []
        if lens[b] > 0:
            one = {k: (v[b * Hkv:(b + 1) * Hkv] if k == "radius" and v.dim() == 1 else
                       v[b:b + 1].contiguous() if k == "radius" else v) for k, v in extra.items()}
            dbg = mp.debug_select(x["q"][b:b + 1], codes.view(-1)[b * per:(b + 1) * per],
                                  centre[b:b + 1], W, wide[b:b + 1], wide[b:b + 1], *args, n=lens[b],
                                  counts=False, **one)
            for h in range(Hq):
                mask = torch.zeros(cap, dtype=torch.bool, device="cuda")
                mask[dbg["sel_idx"][0, h, :int(dbg["sel_count"][0, h])].long()] = True
                rows.append(mask)
        chosen.append(rows)
    return chosen


@pytest.mark.parametrize("dt,Hq,Hkv,n,page,K,L,n_sink,n_local", [
    (BF, 8, 2, 5000, 16, 10, 150, 4, 64), (F32, 4, 4, 1500, 24, 6, 40, 0, 3),
    (BF, 8, 1, 4097, 128, 9, 120, 4, 64), (F32, 2, 1, 900, 8, 0, 2, 4, 64),
    (BF, 4, 2, 2000, 48, 3, 49, 0, 0), (BF, 2, 2, 3000, 64, 20, 1000, 4, 64),
    # many keys sampled, many in T: CTAs that share a partial's rows, and list them a window at a time
    (BF, 1, 1, 9000, 16, 6, 180, 4, 64), (F32, 4, 2, 5000, 24, 6, 100, 100, 1500),
    (BF, 8, 4, 2500, 8, 4, 60, 700, 300)])
def test_sampled_decode_over_pages(mp, dt, Hq, Hkv, n, page, K, L, n_sink, n_local):
    lens = [n, n // 2 + 1, 0, 1, 70]
    wl = small_workload(name="paged", index=780, B=len(lens), Hq=Hq, Hkv=Hkv, n=n, K=K, L=L,
                        kv_dtype=dt, q_dtype=dt, w_dtype=dt)
    g = _gen(n)
    x = {k: v.cuda() for k, v in make_layer(wl).items()}
    W = make_hyperplanes(wl).cuda()
    centre = mp.key_mean(x["keys"])
    cap = n + 1200                               # the codes' capacity, and the table's another
    cache, table = _pages_of(mp, g, x, n + 2 * page, page)
    codes = mp.encode_rows(x["keys"], centre, W, K, L, 0, cap) if K else \
        torch.zeros(4, dtype=torch.int32, device="cuda")
    args = (K, L, n_sink, n_local)
    chosen = _chosen(mp, x, codes if K else codes.new_zeros(len(lens) * 4), centre, W, lens, cap, args,
                     Hkv)

    def check(lengths, used, n_call):
        out = mp.paged_decode_attention(x["q"], codes, centre, W, cache, table, *args, n=n_call,
                                        lengths=lengths, n_capacity=cap)
        want, tol = R.sampled(x["q"], centre, cache.keys, cache.values, table.cpu(), used, chosen, *args,
                              128 ** -0.5)
        bad = (out.double() - want).abs() > tol
        assert not bad.any(), (bad.nonzero()[:5].tolist(),
                               ((out.double() - want).abs() / tol.clamp_min(1e-300)).max().item())
        return out

    out = check(_ints(lens), lens, n)
    assert (out[2] == 0).all()
    assert torch.equal(check(_ints(lens), lens, n + page), out)          # a larger n, the same lengths
    # pages that are not there: their tokens are neither sampled nor attended to
    table[0, 0], table[0, 5], table[1, :] = -1, 2 ** 31 - 1, -5
    assert (check(_ints(lens), lens, n)[1] == 0).all()
    # every sequence n tokens long
    chosen = _chosen(mp, x, codes if K else codes.new_zeros(len(lens) * 4), centre, W, [n] * len(lens),
                     cap, args, Hkv)
    check(None, [n] * len(lens), n)


@pytest.mark.parametrize("dt,B,Hq,Hkv,K,L", [(BF, 12, 8, 2, 10, 150), (F32, 9, 8, 4, 6, 40), (BF, 41, 8, 1, 8, 75),
                                             (F32, 70, 4, 4, 5, 23), (BF, 33, 16, 4, 3, 49)])
def test_sampled_decode_of_many_sequences(mp, dt, B, Hq, Hkv, K, L):
    """Batches whose queries are encoded several rows at a time (and hyperplanes that are no multiple of
    four): the keys that the contiguous cache's encoding samples."""
    n, page, n_sink, n_local = 300, 16, 2, 9
    lens = [(37 * b) % (n + 1) for b in range(B)]
    wl = small_workload(name="pagedb", index=782, B=B, Hq=Hq, Hkv=Hkv, n=n, K=K, L=L, kv_dtype=dt,
                        q_dtype=dt, w_dtype=dt)
    g = _gen(B)
    x = {k: v.cuda() for k, v in make_layer(wl).items()}
    W = make_hyperplanes(wl).cuda()
    centre = mp.key_mean(x["keys"])
    cache, table = _pages_of(mp, g, x, n, page)
    codes = mp.encode_rows(x["keys"], centre, W, K, L, 0, n)
    args = (K, L, n_sink, n_local)
    chosen = _chosen(mp, x, codes, centre, W, lens, n, args, Hkv)
    out = mp.paged_decode_attention(x["q"], codes, centre, W, cache, table, *args, n=n,
                                    lengths=_ints(lens), n_capacity=n)
    want, tol = R.sampled(x["q"], centre, cache.keys, cache.values, table.cpu(), lens, chosen, *args,
                          128 ** -0.5)
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("variant,K,L", [("mips", 8, 75), ("cp", 1, 32)])
def test_variants_run_over_pages(mp, variant, K, L):
    """The same weights as over the contiguous cache: outputs agree to a few roundings of log u."""
    lens = [3000, 1777]
    wl = small_workload(name="pagedv", index=781, B=2, Hq=4, Hkv=2, n=3000, K=K, L=L, kv_dtype=BF,
                        q_dtype=BF, w_dtype=BF)
    g = _gen(1)
    x = {k: v.cuda() for k, v in make_layer(wl).items()}
    centre = mp.key_mean(x["keys"])
    extra = {}
    if variant == "mips":
        W = torch.cat([make_hyperplanes(wl).cuda(), _randn(g, 1, K * L).to(BF)]).contiguous()
        extra["radius"] = mp.key_radius(x["keys"], centre)
        codes = mp.encode_keys_mips(x["keys"], centre, W, extra["radius"], K, L, 0, 3000)
    else:
        W = _randn(g, L, 128, 128).to(BF)
        extra["logu_table"] = mp.cp_logu_table(1, L)
        codes = mp.encode_keys_cp(x["keys"], centre, W, L, 0, 3000)
    cache, table = _pages_of(mp, g, x, 3000, 16)
    out = mp.paged_decode_attention(x["q"], codes, centre, W, cache, table, K, L, 4, 64, n=3000,
                                    lengths=_ints(lens), n_capacity=3000, **extra)
    per = codes.numel() // 2
    for b in range(2):
        one = dict(extra)
        if "radius" in one:
            one["radius"] = extra["radius"][b:b + 1].contiguous()
        want = mp.decode_attention(x["q"][b:b + 1], codes.view(-1)[b * per:(b + 1) * per],
                                   centre[b:b + 1], W, x["keys"][b:b + 1], x["values"][b:b + 1], K, L,
                                   4, 64, n=lens[b], **one)
        # log u: 2e-5 of the contiguous form's table, twice (weights), of values of up to 5
        assert (out[b] - want[0]).abs().max() <= 2 * 4e-5 * 5


def test_a_prompt_and_decode_steps_as_they_are_used(mp):
    """Two sequences of different lengths: prompts appended with their rotation and encoded, then decode
    steps, each appended, encoded and attended to, exactly and sampled."""
    B, Hq, Hkv, K, L, page, steps = 2, 8, 2, 8, 60, 16, 4
    prompts = [1500, 333]
    g = _gen(77)
    slots = 110
    table, n_pages = _table(g, B, slots)
    cap = slots * page
    cache = _filled(mp, n_pages, Hkv, page, BF)
    W, freq = _randn(g, 128, K * L).to(BF), _inv_freq(128)
    codes = torch.zeros(B, mp.codes_bytes(1, Hkv, cap, K, L) // 4, dtype=torch.int32, device="cuda")
    centre = torch.empty(B, Hkv, 128, device="cuda")
    raw_k = [_randn(g, Hkv, n + steps, 128).to(BF) + 2 for n in prompts]
    raw_v = [_randn(g, Hkv, n + steps, 128).to(BF) for n in prompts]
    for b, n in enumerate(prompts):
        rows = torch.empty(1, Hkv, n, 128, dtype=BF, device="cuda")
        mp.paged_append(cache, table[b:b + 1], raw_k[b][None, :, :n], raw_v[b][None, :, :n],
                        inv_freq=freq, keys_out=rows)
        mp.key_mean(rows, centre=centre[b:b + 1])
        mp.encode_rows(rows, centre[b:b + 1], W, K, L, 0, cap, codes=codes[b])
    pos = _ints(prompts)
    for step in range(steps):
        at = [n + step for n in prompts]
        k = torch.stack([raw_k[b][:, at[b]:at[b] + 1] for b in range(B)])
        v = torch.stack([raw_v[b][:, at[b]:at[b] + 1] for b in range(B)])
        q = _randn(g, B, Hq, 1, 128).to(BF)
        rows = torch.empty(B, Hkv, 1, 128, dtype=BF, device="cuda")
        q_out = mp.paged_append(cache, table, k, v, positions=pos, inv_freq=freq, q=q, keys_out=rows)
        mp.encode_rows_at(rows, centre, W, K, L, pos, cap, codes)
        pos += 1
        lens = [n + 1 for n in at]
        assert pos.tolist() == lens
        qq = q_out[:, :, 0].contiguous()
        _attend_and_check(mp, qq, cache, table, None, lens, pos)
        out = mp.paged_decode_attention(qq, codes, centre, W, cache, table, K, L, 4, 64, lengths=pos)
        # what the pages hold, in a contiguous cache with codes of its own
        for b in range(B):
            keys, _ = R.held(cache.keys, table.cpu(), b, lens[b])
            values, _ = R.held(cache.values, table.cpu(), b, lens[b])
            keys, values = keys[None].to(BF), values[None].to(BF)
            own = mp.encode_rows(keys, centre[b:b + 1], W, K, L, 0, lens[b])
            again = mp.decode_attention(qq[b:b + 1], own, centre[b:b + 1], W, keys, values, K, L, 4, 64)
            # the prompt's codes come from the tensor cores here and there, the step's from CUDA cores
            # there; log u is the contiguous form's table: as in the test of the variants
            assert (out[b] - again[0]).abs().max() <= 2 * 4e-5 * 5
    held, _ = R.held(cache.keys, table.cpu(), 0, prompts[0] + steps)
    want, tol = R.turned(raw_k[0][None], _ints([0]), freq, False)
    assert ((held - want[0]).abs() <= R.rounded(tol, want, BF)[0]).all()


@pytest.mark.parametrize("captured", [False, True])
def test_a_step_with_its_codes_back_to_back(mp, captured):
    """Append, codes and both attentions of several steps, queued or captured as one graph, against the
    same calls each waited for: bit for bit."""
    B, Hq, Hkv, K, L, page, slots, steps = 3, 8, 2, 8, 60, 16, 40, 5
    g = _gen(78)
    lens0 = [500, 1, 257]
    table, n_pages = _table(g, B, slots)
    cap = slots * page
    W, freq = _randn(g, 128, K * L).to(BF), _inv_freq(128)
    start = mp.paged_cache(n_pages, Hkv, page)
    first = _randn(g, 2, B, Hkv, max(lens0), 128).to(BF)
    for t in start:
        t.zero_()
    mp.paged_append(start, table, first[0], first[1], counts=_ints(lens0))
    centre = _randn(g, B, Hkv, 128) * 0.1
    codes0 = mp.encode_rows(first[0], centre, W, K, L, 0, cap)
    x = [_randn(g, 2, B, Hkv, 1, 128).to(BF) for _ in range(steps)]
    q = [_randn(g, B, Hq, 1, 128).to(BF) for _ in range(steps)]
    ws = torch.empty(max(mp.paged_attention_workspace_bytes(B, Hq, Hkv, cap),
                         mp.decode_workspace_bytes(B, Hq, Hkv, cap, 128, K, L, 4, 64)), dtype=torch.uint8,
                     device="cuda")
    rows, turned = torch.empty(B, Hkv, 1, 128, dtype=BF, device="cuda"), torch.empty_like(q[0])

    def run(wait):
        cache, codes, pos = mp.PagedCache(*(t.clone() for t in start)), codes0.clone(), _ints(lens0)
        outs = [torch.empty(B, Hq, 128, device="cuda") for _ in range(2 * steps)]

        def go():
            for i in range(steps):
                for call in (
                        lambda: mp.paged_append(cache, table, x[i][0], x[i][1], positions=pos, inv_freq=freq,
                                                q=q[i], q_out=turned, keys_out=rows),
                        lambda: mp.encode_rows_at(rows, centre, W, K, L, pos, cap, codes),
                        lambda: pos.add_(1),
                        lambda: mp.paged_attention(turned[:, :, 0], cache, table, lengths=pos,
                                                   out=outs[2 * i], workspace=ws),
                        lambda: mp.paged_decode_attention(turned[:, :, 0], codes, centre, W, cache, table, K,
                                                          L, 4, 64, lengths=pos, out=outs[2 * i + 1],
                                                          workspace=ws)):
                    call()
                    if wait:
                        torch.cuda.synchronize()

        if captured and not wait:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                go()
            for _ in range(3):                   # on what it started from
                for t, was in zip((*cache, codes), (*start, codes0)):
                    t.copy_(was)
                pos.copy_(_ints(lens0))
                graph.replay()
        else:
            go()
        torch.cuda.synchronize()
        return (*cache, codes, *outs)

    want = run(True)
    for _ in range(1 if captured else 4):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
    assert mp.device_status() == 0


# ---------------------------------------------------------------- refusals
def test_refusals_of_the_binding(mp):
    cache = mp.paged_cache(6, 2, 16)
    table = torch.arange(6, device="cuda").view(2, 3).int()
    k = torch.zeros(2, 2, 4, 128, dtype=BF, device="cuda")
    q = torch.zeros(2, 4, 128, device="cuda")
    lens = _ints([3, 3])

    def refused(kind, f):
        with pytest.raises(kind):
            f()

    for call in (lambda c, t: mp.paged_append(c, t, k, k), lambda c, t: mp.paged_attention(q, c, t)):
        refused(TypeError, lambda: call(mp.PagedCache(cache.keys.cpu(), cache.values), table))
        refused(TypeError, lambda: call(mp.PagedCache(cache.keys, cache.values.float()), table))
        refused(ValueError, lambda: call(mp.PagedCache(cache.keys, cache.values[:5]), table))
        refused(ValueError, lambda: call(mp.PagedCache(cache.keys[..., :64], cache.values[..., :64]),
                                         table))
        refused(ValueError, lambda: call(mp.PagedCache(*(t.transpose(1, 2) for t in cache)), table))
        refused(TypeError, lambda: call(mp.PagedCache(*(t.half() for t in cache)), table))
        refused(TypeError, lambda: call(cache, table.long()))
        refused(TypeError, lambda: call(cache, table.cpu()))
        refused(ValueError, lambda: call(cache, table.t()))
        refused(ValueError, lambda: call(cache, table[0]))
        refused(ValueError, lambda: call(cache, table[:1].expand(2, 3)))
    bad_pages = mp.paged_cache(6, 2, 12)
    refused(mp.MagicPIGError, lambda: mp.paged_attention(q, bad_pages, table))
    refused(ValueError, lambda: mp.paged_append(cache, table, k[:1], k[:1]))
    refused(ValueError, lambda: mp.paged_append(cache, table, k, k[:, :1]))
    refused(TypeError, lambda: mp.paged_append(cache, table, k, k.float()))
    refused(ValueError, lambda: mp.paged_append(cache, table, k.transpose(2, 3), k.transpose(2, 3)))
    refused(mp.MagicPIGError, lambda: mp.paged_append(cache, table, k, k, n_begin=45))
    refused(mp.MagicPIGError, lambda: mp.paged_append(cache, table, k, k, n_begin=-1))
    refused(ValueError, lambda: mp.paged_append(cache, table, k, k, n_begin=2 ** 40))
    refused(TypeError, lambda: mp.paged_append(cache, table, k, k, positions=lens.long()))
    refused(ValueError, lambda: mp.paged_append(cache, table, k, k, counts=lens[:1]))
    refused(mp.MagicPIGError, lambda: mp.paged_append(cache, table, k, k, inv_freq=_inv_freq(24)))
    refused(TypeError, lambda: mp.paged_append(cache, table, k, k, inv_freq=_inv_freq(64).double()))
    refused(ValueError, lambda: mp.paged_append(cache, table, k, k, q=k[:, :, :3]))
    refused(ValueError, lambda: mp.paged_append(cache, table, k, k, q_out=k))
    refused(ValueError, lambda: mp.paged_append(cache, table, k, k, q=k, q_out=k[:1]))
    refused(TypeError, lambda: mp.paged_append(cache, table, k, k, keys_out=k.float()))
    refused(ValueError, lambda: mp.paged_attention(q[:1], cache, table))
    refused(ValueError, lambda: mp.paged_attention(q.transpose(1, 2), cache, table))
    refused(ValueError, lambda: mp.paged_attention(q, cache, table, n=49))
    refused(ValueError, lambda: mp.paged_attention(q, cache, table, n=0))
    refused(TypeError, lambda: mp.paged_attention(q, cache, table, lengths=lens.long()))
    refused(ValueError, lambda: mp.paged_attention(q, cache, table, lengths=lens[:1]))
    refused(TypeError, lambda: mp.paged_attention(q, cache, table, out=q.to(BF)))
    refused(mp.MagicPIGError, lambda: mp.paged_attention(q[:, :3].contiguous(), cache, table))
    refused(mp.MagicPIGError, lambda: mp.paged_attention(q, cache, table, scale=-1.0))
    refused(mp.MagicPIGError, lambda: mp.paged_attention(
        q, cache, table, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")))
    W, centre = torch.zeros(128, 80, device="cuda"), torch.zeros(2, 2, 128, device="cuda")
    codes = torch.zeros(mp.codes_bytes(2, 2, 48, 8, 10) // 4, dtype=torch.int32, device="cuda")

    def dec(q=q, codes=codes, centre=centre, W=W, **kw):
        return mp.paged_decode_attention(q, codes, centre, W, cache, table, 8, 10, 4, 64, **kw)

    dec()
    refused(ValueError, lambda: dec(codes=codes[:-4]))
    refused(ValueError, lambda: dec(codes=None))
    refused(ValueError, lambda: dec(n_capacity=1100))
    refused(ValueError, lambda: dec(W=W[:127].contiguous()))
    refused(ValueError, lambda: dec(centre=centre[:1]))
    refused(TypeError, lambda: dec(centre=None))
    refused(ValueError, lambda: dec(n=49))
    refused(mp.MagicPIGError, lambda: dec(n_capacity=47))
    enc = lambda **kw: mp.encode_rows_at(**{**dict(keys=k, centre=centre, W=W, K=8, L=10,
                                                   positions=lens, n_capacity=48, codes=codes), **kw})
    enc()
    refused(TypeError, lambda: enc(positions=None))
    refused(ValueError, lambda: enc(positions=lens[:1]))
    refused(ValueError, lambda: enc(codes=codes[:-4]))
    refused(ValueError, lambda: enc(W=W[:, :-1].contiguous()))
    refused(ValueError, lambda: enc(n_capacity=0))
    refused(mp.MagicPIGError, lambda: enc(keys=torch.zeros(2, 2, 65, 128, device="cuda")))
    torch.cuda.synchronize()
    assert mp.device_status() == 0
