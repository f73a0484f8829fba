"""The 4-bit K/V cache on the GPU against its definition in 64 bits (tests/kv4_reference.py):
rows written (codes and parameters equal bit for bit), rows read back, exact attention over the
cache, and the LSH-sampled decode over it against the oracle."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import kv4_reference as R
from tests.parity import OUT_REL_TOL, row_rel_err
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


def _filled(mp, B, Hkv, cap):
    """A cache whose every byte is a sentinel; the parameters are NaN."""
    c = mp.kv4_cache(B, Hkv, cap)
    c.k_codes.fill_(0xA5)
    c.v_codes.fill_(0x5A)
    c.params.fill_(float("nan"))
    return c


def _clone(c):
    return type(c)(*(t.clone() for t in c))


def _same(a, b):
    return a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _check_rows(cache, before, keys, values, centre, starts):
    """Every row of the cache: the written ones by the definition, the others as before."""
    B, Hkv, m, _ = keys.shape
    cap = cache.k_codes.shape[2]
    kx = keys.float() if centre is None else keys.float() - centre.unsqueeze(2)
    kc, ks, kz = R.quantise(kx.cpu().numpy())
    vc, vs, vz = R.quantise(values.float().cpu().numpy())
    want = [t.cpu().clone() for t in before]
    prm = R.params(ks, kz, vs, vz)
    for b in range(B):
        for i in range(m):
            p = starts[b] + i
            if 0 <= p < cap:
                want[0][b, :, p] = torch.from_numpy(R.pack(kc[b, :, i]))
                want[1][b, :, p] = torch.from_numpy(R.pack(vc[b, :, i]))
                want[2][b, :, p] = torch.from_numpy(prm[b, :, i].view(np.int16)).view(BF)
    assert torch.equal(cache.k_codes.cpu(), want[0])
    assert torch.equal(cache.v_codes.cpu(), want[1])
    got, exp = cache.params.cpu().float(), want[2].float()
    assert torch.equal(torch.isnan(got), torch.isnan(exp))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(exp))     # -0 equals 0


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("B,Hkv,m,cap,n0,centred", [
    (1, 1, 1, 1, 0, True), (1, 2, 17, 40, 23, True), (3, 5, 33, 77, 9, False),
    (2, 1, 300, 301, 1, True), (32, 8, 1, 65, 64, True)])
def test_write_is_the_definition_bit_for_bit(mp, dt, B, Hkv, m, cap, n0, centred):
    g = _gen(m + cap)
    keys = (torch.randn(B, Hkv, m, 128, generator=g, device="cuda") * 3 + 1).to(dt)
    values = torch.randn(B, Hkv, m, 128, generator=g, device="cuda").to(dt)
    centre = torch.randn(B, Hkv, 128, generator=g, device="cuda") if centred else None
    cache = _filled(mp, B, Hkv, cap)
    before = _clone(cache)
    assert mp.kv4_write(cache, keys, values, n_begin=n0, centre=centre) is cache
    _check_rows(cache, before, keys, values, centre, [n0] * B)


def _at_16_bytes(t):
    """The same tensor 16 bytes past a 32-byte boundary."""
    n = 16 // t.element_size()
    room = torch.empty(t.numel() + 2 * n, dtype=t.dtype, device=t.device)
    assert room.data_ptr() % 32 == 0
    u = room[n:n + t.numel()].view(t.shape)
    u.copy_(t)
    return u


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("m,shifted", [(31, True), (2003, False), (2003, True)])
def test_many_rows_and_rows_aligned_to_16_bytes_only(mp, dt, m, shifted):
    """20030 bf16 rows go through the kernel of four lanes a row; hard rows among them."""
    B, Hkv, cap = 2, 5, m + 3
    g = _gen(m)
    keys = torch.randn(B, Hkv, m, 128, generator=g, device="cuda") * 2
    values = torch.randn(B, Hkv, m, 128, generator=g, device="cuda")
    hard = torch.from_numpy(_hard_rows()).cuda()[:m]
    keys[1, 2, -hard.shape[0]:] = hard
    values[1, 3, :hard.shape[0]] = hard
    keys, values = keys.to(dt), values.to(dt)
    centre = torch.randn(B, Hkv, 128, generator=g, device="cuda")
    if shifted:
        keys, values = _at_16_bytes(keys), _at_16_bytes(values)
    cache = _filled(mp, B, Hkv, cap)
    before = _clone(cache)
    mp.kv4_write(cache, keys, values, n_begin=2, centre=centre)
    _check_rows(cache, before, keys, values, centre, [2] * B)
    k, v = mp.kv4_read(cache, m, n_begin=2, centre=centre, dtype=dt)
    if shifted:
        out = _at_16_bytes(torch.zeros_like(k)), _at_16_bytes(torch.zeros_like(v))
        mp.kv4_read(cache, m, n_begin=2, centre=centre, keys=out[0], values=out[1])
        assert _same(out[0], k) and _same(out[1], v)


def _hard_rows():
    """Rows whose groups sit where the format can go wrong."""
    rng = np.random.default_rng(11)
    rows = [np.zeros(128), -np.zeros(128), np.full(128, 0.3), np.full(128, -1e-40),
            np.full(128, 3e38), rng.normal(size=128) * 1e-42, rng.normal(size=128) * 1e37,
            rng.normal(size=128) * 1e-38, np.where(np.arange(128) == 70, 1e4, 1e-4),
            1000 + rng.normal(size=128) * 1e-3, -1000 + rng.normal(size=128) * 1e-3,
            np.linspace(0, 15, 128), np.linspace(-7.5, 7.5, 128)]
    # exactly half-way values: z = 0, s = 1, x = c + 1/2 (ties to even), and z = -4, s = 1/2
    half = np.concatenate([np.arange(16), np.arange(15) + 0.5, np.zeros(33)])
    rows += [np.tile(half, 2), np.tile(half / 2 - 4, 2)]
    for bad in (np.nan, np.inf, -np.inf):
        r = rng.normal(size=128)
        r[rng.integers(0, 64)] = bad
        rows.append(r)
    r = rng.normal(size=128)
    r[64], r[65] = 3.3e38, -3.3e38
    rows.append(r)
    r = rng.normal(size=128)
    r[:] = np.nan
    rows.append(r)
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("dt", [BF, F32])
def test_write_of_constant_tiny_huge_tied_and_non_finite_groups(mp, dt):
    x = torch.from_numpy(_hard_rows()).cuda()
    # many rows whose values lie next to a border between two codes: multiples of s / 2 moved by
    # one step of their type
    g = _gen(3)
    base = torch.randint(0, 31, (400, 128), generator=g, device="cuda").float() / 2
    base[:, 0::64], base[:, 1::64] = 0.0, 15.0
    scale = 2.0 ** torch.randint(-8, 8, (400, 1), generator=g, device="cuda").float() * \
        (1 + torch.randint(0, 128, (400, 1), generator=g, device="cuda").float() / 128)
    near = base * scale
    bits = near.view(torch.int32) + torch.randint(-1, 2, near.shape, generator=g,
                                                  device="cuda").int()
    near = torch.where(near > 0, bits.view(torch.float32), near)
    keys = torch.cat([x, near]).to(dt)[None, None].contiguous()
    values = keys.flip(2).contiguous()
    m = keys.shape[2]
    cache = _filled(mp, 1, 1, m + 2)
    before = _clone(cache)
    mp.kv4_write(cache, keys, values, n_begin=1)
    _check_rows(cache, before, keys, values, None, [1])


def test_positions_may_leave_the_cache_and_are_then_not_written_or_read(mp):
    B, Hkv, m, cap = 7, 3, 5, 20
    g = _gen(8)
    keys = torch.randn(B, Hkv, m, 128, generator=g, device="cuda")
    values = torch.randn(B, Hkv, m, 128, generator=g, device="cuda")
    starts = [0, 15, 18, 20, -2, 2 ** 31 - 1, -2 ** 31]
    pos = torch.tensor(starts, dtype=torch.int32, device="cuda")
    cache = _filled(mp, B, Hkv, cap)
    before = _clone(cache)
    mp.kv4_write(cache, keys, values, positions=pos)
    _check_rows(cache, before, keys, values, None, starts)
    k, v = mp.kv4_read(cache, m, positions=pos, centre=torch.ones(B, Hkv, 128, device="cuda"),
                       dtype=F32)
    for b, s in enumerate(starts):
        for i in range(m):
            inside = 0 <= s + i < cap
            assert bool((k[b, :, i] == 0).all()) != inside, (b, i)
            assert bool((v[b, :, i] == 0).all()) != inside, (b, i)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("B,Hkv,m,cap,n0,ragged,centred", [
    (1, 1, 1, 3, 2, False, True), (2, 3, 19, 50, 31, False, False), (4, 2, 133, 190, 0, True, True),
    (1, 8, 1025, 1030, 5, False, True)])
def test_read_returns_the_values_held(mp, dt, B, Hkv, m, cap, n0, ragged, centred):
    g = _gen(m)
    x = torch.randn(2, B, Hkv, cap, 128, generator=g, device="cuda")
    centre = torch.randn(B, Hkv, 128, generator=g, device="cuda") * 4 if centred else None
    cache = mp.kv4_write(mp.kv4_cache(B, Hkv, cap), x[0], x[1])
    pos = torch.randint(0, cap - m + 1, (B,), generator=g, device="cuda").int() if ragged else None
    k, v = mp.kv4_read(cache, m, n_begin=n0, centre=centre, positions=pos, dtype=dt)
    assert k.shape == v.shape == (B, Hkv, m, 128) and k.dtype == v.dtype == dt
    for b in range(B):
        s = n0 if pos is None else int(pos[b])
        held = [R.values64(c[b, :, s:s + m], cache.params[b, :, s:s + m], i).float()
                for i, c in ((0, cache.k_codes), (1, cache.v_codes))]
        if centred:
            held[0] = held[0] + centre[b].unsqueeze(1)
        assert torch.equal(k[b], held[0].to(dt)) and torch.equal(v[b], held[1].to(dt))
    # within half a step of what was written
    k32, v32 = mp.kv4_read(cache, cap, dtype=F32)
    step = cache.params.float()
    for got, wrote, at in ((k32, x[0], 0), (v32, x[1], 4)):
        s = step[..., at:at + 4:2].repeat_interleave(64, -1)
        # half a step, and the rounding of the float32 value (2^-24 of it)
        assert ((got - wrote).abs() <= s / 2 + 2.0 ** -23 * wrote.abs().max()).all()


def _random_cache(mp, B, Hkv, cap, n, seed, scale=1.0):
    """A cache of n random tokens per head; the rest of the capacity is NaN and sentinels."""
    g = _gen(seed)
    cache = _filled(mp, B, Hkv, cap)
    keys = torch.randn(B, Hkv, n, 128, generator=g, device="cuda") * scale
    values = torch.randn(B, Hkv, n, 128, generator=g, device="cuda")
    mp.kv4_write(cache, keys, values)
    return cache


def _attend_and_check(mp, q, cache, n, lengths=None, scale=0.0):
    out = mp.kv4_attention(q, cache, n=n, lengths=lengths, scale=scale)
    used = [n] * q.shape[0] if lengths is None else \
        [max(0, min(n, int(x))) for x in lengths]
    want, tol = R.attention64(q, cache, used, scale or 128 ** -0.5)
    off = (out.double() - want).abs()
    assert (off <= tol).all(), float((off / tol.clamp_min(1e-30)).nan_to_num().max())
    return out


@pytest.mark.parametrize("qt", [BF, F32])
@pytest.mark.parametrize("B,Hkv,G,n", [
    (1, 1, 1, 1), (1, 1, 4, 2), (2, 3, 3, 15), (1, 2, 5, 16), (1, 2, 8, 17), (3, 1, 7, 63),
    (1, 1, 16, 64), (2, 2, 2, 65), (1, 1, 11, 127), (1, 3, 6, 256), (2, 1, 4, 257), (1, 2, 1, 511),
    (1, 2, 4, 1000), (2, 2, 8, 4097), (1, 1, 32, 777), (5, 4, 4, 2049), (1, 8, 4, 20011)])
def test_attention_against_64_bits(mp, qt, B, Hkv, G, n):
    cache = _random_cache(mp, B, Hkv, n + 37, n, seed=n)
    q = (torch.randn(B, Hkv * G, 128, generator=_gen(n + 1), device="cuda") * 2).to(qt)
    _attend_and_check(mp, q, cache, n)


@pytest.mark.parametrize("G", [1, 4, 8])
def test_attention_of_sequences_of_different_lengths(mp, G):
    n = 3000
    raw = [0, 1, 2, 63, 64, 65, 1500, 2999, 3000, 3001, 2 ** 31 - 1, -1, -2 ** 31]
    B = len(raw)
    cache = _random_cache(mp, B, 2, 3100, n, seed=G)
    lengths = torch.tensor(raw, dtype=torch.int32, device="cuda")
    q = torch.randn(B, 2 * G, 128, generator=_gen(5), device="cuda")
    out = _attend_and_check(mp, q, cache, n, lengths)
    for b, x in enumerate(raw):
        if x <= 0:
            assert (out[b] == 0).all()


@pytest.mark.parametrize("qt", [BF, F32])
def test_attention_with_sharp_scores_and_a_scale_of_its_own(mp, qt):
    cache = _random_cache(mp, 2, 2, 1500, 1500, seed=2, scale=4.0)
    q = torch.randn(2, 8, 128, generator=_gen(6), device="cuda").to(qt)
    for scale in (1e-6, 0.3, 1.7):
        _attend_and_check(mp, q, cache, 1500, scale=scale)
    # queries far from 1, up and down
    for f in (2.0 ** 60, 2.0 ** -60):
        _attend_and_check(mp, (q.float() * f).to(qt), cache, 1500, scale=0.1 / f)
    _attend_and_check(mp, torch.zeros_like(q), cache, 1500)


@pytest.mark.parametrize("qt", [BF, F32])
def test_attention_of_queries_aligned_to_their_element_only(mp, qt):
    cache = _random_cache(mp, 2, 3, 700, 700, seed=77)
    for G in (2, 7):
        q = torch.randn(2, 3 * G, 128, generator=_gen(G), device="cuda").to(qt)
        room = torch.empty(q.numel() + 1, dtype=qt, device="cuda")
        shifted = room[1:].view(q.shape)
        shifted.copy_(q)
        assert torch.equal(mp.kv4_attention(shifted, cache), _attend_and_check(mp, q, cache, 700))


def test_attention_layouts_of_one_two_and_three_ctas_an_sm(mp):
    """Shapes that the plan lays out with one split, as many as fill one or two CTAs an SM, and in
    several waves, long sequences among them."""
    for B, Hkv, G, n in ((1, 8, 4, 16384), (2, 8, 4, 30000), (40, 8, 1, 1100), (9, 8, 8, 2500),
                         (1, 1, 2, 70001), (150, 4, 3, 300), (1, 2, 24, 5000)):
        cache = _random_cache(mp, B, Hkv, n, n, seed=n)
        q = torch.randn(B, Hkv * G, 128, generator=_gen(n), device="cuda")
        _attend_and_check(mp, q, cache, n)
        lengths = torch.randint(0, n + 1, (B,), generator=_gen(B), device="cuda").int()
        _attend_and_check(mp, q, cache, n, lengths)


def test_attention_over_values_of_very_different_sizes(mp):
    n = 900
    g = _gen(9)
    keys = torch.randn(1, 2, n, 128, generator=g, device="cuda")
    values = torch.randn(1, 2, n, 128, generator=g, device="cuda")
    values[..., :64] *= 1e-20                                     # one group tiny, one huge
    values[..., 64:] *= 1e20
    cache = mp.kv4_write(mp.kv4_cache(1, 2, n), keys, values)
    q = torch.randn(1, 8, 128, generator=g, device="cuda")
    out = mp.kv4_attention(q, cache)
    want, _ = R.attention64(q, cache, [n], 128 ** -0.5)
    for part in (slice(0, 64), slice(64, 128)):
        # each group by its own largest value: the bound of attention64 at A < 8, n = 900
        tol = 2.0 ** -24 * (2 * (32 * 8 + 4) + 4 * 30 + 16) * values[..., part].abs().max()
        assert ((out.double() - want)[..., part].abs() <= tol).all()
    # sizes that differ from token to token
    values = torch.randn(1, 2, n, 128, generator=g, device="cuda") * \
        10.0 ** torch.randint(-6, 7, (1, 2, n, 1), generator=g, device="cuda")
    cache = mp.kv4_write(mp.kv4_cache(1, 2, n), keys, values)
    _attend_and_check(mp, q, cache, n)


def test_attention_passes_nan_and_infinity_on(mp):
    n = 400
    g = _gen(12)
    keys = torch.randn(3, 1, n, 128, generator=g, device="cuda")
    values = torch.randn(3, 1, n, 128, generator=g, device="cuda")
    values[0, 0, 111, 100] = float("nan")          # a value: its 64 dims
    keys[1, 0, 222, 5] = float("inf")              # a key: the whole row
    cache = mp.kv4_write(mp.kv4_cache(3, 1, n), keys, values)
    q = torch.randn(3, 2, 128, generator=g, device="cuda")
    q[2, 1, 7] = float("inf")                      # a query element: its own row
    out = mp.kv4_attention(q, cache)
    nan = torch.isnan(out)
    assert nan[0, :, 64:].all() and not nan[0, :, :64].any()
    assert nan[1].all()
    assert not nan[2, 0].any() and nan[2, 1].all()
    # the group that is not hurt keeps its values; so does the row without the bad element
    want, tol = R.attention64(q, cache, [n] * 3, 128 ** -0.5)
    assert ((out.double() - want)[0, :, :64].abs() <= tol[2, 0]).all()
    assert ((out.double() - want)[2, 0].abs() <= tol[2, 0]).all()
    q[2, 1, 7] = float("nan")
    assert torch.isnan(mp.kv4_attention(q, cache)[2, 1]).all()
    # a length that ends before the bad token never sees it
    short = torch.tensor([111, 222, 400], dtype=torch.int32, device="cuda")
    out = mp.kv4_attention(q, cache, lengths=short)
    assert torch.isfinite(out[:2]).all()


def test_offsets_beyond_2_to_the_31_bytes(mp):
    cap, n = (1 << 25) + 1234, 700                 # a head of codes is 2 GiB and more
    cache = mp.kv4_cache(1, 3, cap)
    g = _gen(4)
    keys = torch.randn(1, 3, n, 128, generator=g, device="cuda")
    values = torch.randn(1, 3, n, 128, generator=g, device="cuda")
    mp.kv4_write(cache, keys, values)
    q = torch.randn(1, 6, 128, generator=g, device="cuda")
    small = mp.kv4_write(mp.kv4_cache(1, 3, n), keys, values)
    assert torch.equal(mp.kv4_attention(q, cache, n=n), mp.kv4_attention(q, small))
    end = torch.tensor([cap - n], dtype=torch.int32, device="cuda")
    mp.kv4_write(cache, keys, values, positions=end)
    got = mp.kv4_read(cache, n, n_begin=cap - n, dtype=F32)
    want = mp.kv4_read(small, n, dtype=F32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # one head of 2^25 tokens attended to in whole: equal keys, so the mean of the values
    cache.k_codes[:, 2].zero_()
    cache.v_codes[:, 2, :, :] = 0x77
    cache.params[:, 2].copy_(torch.tensor([0.5, 1.0] * 4, dtype=BF, device="cuda"))
    cache.params[:, :2].zero_()
    cache.v_codes[:, :2].zero_()
    cache.k_codes[:, :2].zero_()
    out = mp.kv4_attention(q, cache)
    # 1 + 7/2 everywhere; two sums of 2^25 equal terms, in whatever order, are each off by less
    # than 2^-24 a term added: pieces of at most 2^14 terms
    assert (out[0, 4:] - 4.5).abs().max() <= 4.5 * 2.0 ** -24 * 2 ** 14
    assert (out[0, :4] == 0).all()


def test_runs_agree_bit_for_bit_and_streams_and_graphs_do_not_mix(mp):
    n = 6000
    cache = _random_cache(mp, 2, 4, n, n, seed=21)
    q = torch.randn(2, 16, 128, generator=_gen(1), device="cuda")
    first = mp.kv4_attention(q, cache)
    assert all(torch.equal(mp.kv4_attention(q, cache), first) for _ in range(5))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out = mp.kv4_attention(q, cache, stream=other)
    other.synchronize()
    assert torch.equal(out, first)
    # one token appended and attended to, captured, replayed on new data
    B, Hkv = 2, 4
    new_k = torch.randn(B, Hkv, 1, 128, device="cuda")
    new_v = torch.randn(B, Hkv, 1, 128, device="cuda")
    pos = torch.full((B,), 100, dtype=torch.int32, device="cuda")
    lengths = pos + 1
    size = mp.kv4_attention_workspace_bytes(B, 16, Hkv, n)
    graphs = []
    for _ in range(2):
        ws = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
        res = torch.empty(B, 16, 128, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mp.kv4_write(cache, new_k, new_v, positions=pos)
            mp.kv4_attention(q, cache, lengths=lengths, out=res, workspace=ws)
        graphs.append((graph, res, ws))
    for step in range(3):
        new_k.normal_()
        new_v.normal_()
        pos.fill_(200 * step + 7)
        lengths.copy_(pos + 1)
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        expect = mp.kv4_attention(q, cache, lengths=lengths)
        assert torch.equal(graphs[0][1], expect) and torch.equal(graphs[1][1], expect)
        k, _ = mp.kv4_read(cache, 1, positions=pos, dtype=F32)
        step_size = cache.params[:, :, int(pos[0]), 0:4:2].float().repeat_interleave(64, -1)
        assert ((k[:, :, 0] - new_k[:, :, 0]).abs() <= step_size / 2 + 1e-6).all()


def test_an_output_that_was_handed_in_is_filled_and_no_more(mp):
    cache = _random_cache(mp, 1, 2, 300, 300, seed=31)
    q = torch.randn(1, 8, 128, generator=_gen(2), device="cuda").to(BF)
    room = torch.full((3, 8, 128), 7.0, device="cuda")
    size = mp.kv4_attention_workspace_bytes(1, 8, 2, 300)
    ws = torch.full((size + 4096,), 0xEE, dtype=torch.uint8, device="cuda")
    out = mp.kv4_attention(q, cache, out=room[1:2], workspace=ws)
    assert out.data_ptr() == room[1].data_ptr()
    assert torch.equal(out, mp.kv4_attention(q, cache))
    assert (room[0] == 7).all() and (room[2] == 7).all()
    assert (ws[max(size, 0):] == 0xEE).all()


# ---------------------------------------------------------------- the sampled decode
def _sampled_case(mp, wl, cap, variant="simhash"):
    x = {k: v.cuda() for k, v in make_layer(wl).items()}
    W = make_hyperplanes(wl).cuda()
    kc = torch.full((wl.B, wl.Hkv, cap, 128), 50.0, dtype=wl.kv_dtype, device="cuda")
    kc[:, :, :wl.n] = x["keys"]
    centre = mp.key_mean(kc, n=wl.n)
    cache = mp.kv4_write(_filled(mp, wl.B, wl.Hkv, cap), x["keys"], x["values"], centre=centre)
    extra = {}
    if variant == "mips":
        W = torch.cat([W, torch.randn(1, W.shape[1], generator=_gen(9), device="cuda").to(W.dtype)])
        extra["radius"] = mp.key_radius(kc, centre, n=wl.n)
        codes = mp.encode_keys_mips(kc, centre, W.contiguous(), extra["radius"], wl.K, wl.L, 0,
                                    wl.n)
    elif variant == "cp":
        W = torch.randn(wl.L, 128, 128, generator=_gen(9), device="cuda").to(wl.w_dtype)
        extra["logu_table"] = mp.cp_logu_table(1, wl.L)
        codes = mp.encode_keys_cp(kc, centre, W, wl.L, 0, wl.n)
    else:
        codes = torch.empty(max(mp.codes_bytes(wl.B, wl.Hkv, cap, wl.K, wl.L) // 4, 4),
                            dtype=torch.int32, device="cuda")
        mp.encode_keys(kc, centre, W, wl.K, wl.L, 0, wl.n, codes)
    return x, W.contiguous(), kc, centre, cache, codes, extra


def _oracle_out(wl, x, W, centre, cache, codes, mp, q, n, counts):
    """The estimator over the cache's own keys and values, the sample sets those of the codes."""
    k = R.values64(cache.k_codes, cache.params, 0).cpu().numpy()
    v = R.values64(cache.v_codes, cache.params, 1).cpu().numpy()
    out = np.zeros((wl.B, wl.Hq, 128))
    T = O.exact_set_mask(n, wl.n_sink, wl.n_local)
    G = wl.Hq // wl.Hkv
    for b in range(wl.B):
        for h in range(wl.Hq):
            kk, vv = k[b, h // G, :n], v[b, h // G, :n]
            qq = O.as64(q[b, h])
            S = O.sampled_set(counts[b, h], T)
            p = O.collision_probability(qq, kk)
            logw = kk @ qq / 128 ** 0.5
            logw[S] -= O.log_inclusion_probability(p[S], wl.K, wl.L)
            keep = T.copy()
            keep[S] = True
            w = np.exp(logw[keep] - logw[keep].max())
            out[b, h] = (w @ vv[keep]) / w.sum()
    return out


@pytest.mark.parametrize("dt,B,Hq,Hkv,n,cap,K,L", [
    (BF, 2, 8, 2, 5000, 5000, 10, 150), (F32, 1, 2, 2, 1500, 2100, 6, 40),
    (BF, 1, 8, 1, 4097, 9000, 9, 120), (BF, 3, 4, 4, 70, 100, 8, 75),
    (F32, 1, 2, 1, 900, 900, 0, 2)])
def test_sampled_decode_against_the_oracle_on_the_stored_cache(mp, dt, B, Hq, Hkv, n, cap, K, L):
    wl = small_workload(name="kv4", index=760, B=B, Hq=Hq, Hkv=Hkv, n=n, K=K, L=L, kv_dtype=dt,
                        q_dtype=dt, w_dtype=dt)
    x, W, kc, centre, cache, codes, _ = _sampled_case(mp, wl, cap)
    args = (wl.K, wl.L, wl.n_sink, wl.n_local)
    out = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, *args, n=n)
    # the sample sets do not depend on the cache: those of the same codes over the bf16/fp32 rows
    # (tested against the oracle elsewhere)
    vc = torch.zeros_like(kc)
    dbg = mp.debug_select(x["q"], codes, centre, W, kc, vc, *args, n=n)
    counts = dbg["cnt"].cpu().numpy()
    want = _oracle_out(wl, x, W, centre, cache, codes, mp, x["q"], n, counts)
    for b in range(B):
        for h in range(Hq):
            assert row_rel_err(out[b, h].cpu().numpy(), want[b, h]) <= OUT_REL_TOL
    # the two halves, and the bucketed tables, give the same bits
    ws = torch.empty(mp.decode_workspace_bytes(B, Hq, Hkv, n, 128, *args), dtype=torch.uint8,
                     device="cuda")
    half = torch.empty_like(out)
    mp.encode_query(x["q"], centre, W, kc.shape, *args, ws, n=n)
    mp.kv4_sampled_attention(x["q"], codes, centre, cache, *args, half, ws, n=n)
    assert torch.equal(half, out)
    if 0 < K <= 12:
        indexed = max(1, n - 600)
        buckets = mp.build_buckets(codes, B, Hkv, indexed, K, L, n_capacity=cap)
        bucketed = torch.empty_like(out)
        mp.encode_query(x["q"], centre, W, kc.shape, *args, ws, n=n)
        mp.kv4_sampled_attention_buckets(x["q"], buckets, centre, cache, *args, bucketed, ws,
                                         codes=codes, n=n, n_indexed=indexed)
        assert torch.equal(bucketed, out)


@pytest.mark.parametrize("K,L", [(1, 2), (2, 3), (3, 49), (4, 200), (7, 50), (12, 300), (20, 1000)])
def test_sampled_decode_weighs_keys_to_a_few_millionths(mp, K, L):
    """Over few and many tables, where the weights' log u takes each of its forms. The tolerance is
    attention64's, and 2 x 3e-6 of the largest value for log u off by 3e-6 at most (twelve fp32
    roundings of numbers up to 2 K log 2 = 28, the largest of the pairs)."""
    wl = small_workload(name="kv4u", index=763, B=1, Hq=4, Hkv=2, n=4000, K=K, L=L, kv_dtype=F32,
                        q_dtype=F32, w_dtype=F32, key_spread=4.0)
    x, W, kc, centre, cache, codes, _ = _sampled_case(mp, wl, wl.n)
    args = (wl.K, wl.L, wl.n_sink, wl.n_local)
    out = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, *args)
    counts = mp.debug_select(x["q"], codes, centre, W, kc, torch.zeros_like(kc),
                             *args)["cnt"].cpu().numpy()
    want = _oracle_out(wl, x, W, centre, cache, codes, mp, x["q"], wl.n, counts)
    _, tol = R.attention64(x["q"], cache, [wl.n], 128 ** -0.5)
    vmax = R.values64(cache.v_codes, cache.params, 1).abs().max()
    off = (out.double().cpu() - torch.from_numpy(want)).abs()
    assert (off <= (tol + 6e-6 * vmax).cpu()).all(), float(off.max())


@pytest.mark.parametrize("B,Hq,Hkv,n,K,L,n_sink,n_local", [
    (1, 16, 8, 3194, 7, 195, 4, 64), (4, 16, 8, 700, 6, 180, 4, 64), (4, 32, 8, 901, 6, 99, 0, 64),
    (8, 64, 8, 1500, 5, 100, 4, 64), (1, 2, 1, 2000, 10, 150, 300, 1200),
    (1, 1, 1, 200, 10, 150, 150, 150), (1, 2, 2, 8200, 4, 90, 1, 1)])
def test_sampled_decode_where_much_is_sampled(mp, B, Hq, Hkv, n, K, L, n_sink, n_local):
    """A CTA's many rows, alone or shared with one, three or seven others; a long exact set. The
    tolerance is that of the test above."""
    wl = small_workload(name="kv4d", index=764, B=B, Hq=Hq, Hkv=Hkv, n=n, K=K, L=L, kv_dtype=BF,
                        q_dtype=F32, w_dtype=BF, n_sink=n_sink, n_local=n_local)
    x, W, kc, centre, cache, codes, _ = _sampled_case(mp, wl, n + 3)
    args = (wl.K, wl.L, wl.n_sink, wl.n_local)
    out = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, *args, n=n)
    counts = mp.debug_select(x["q"], codes, centre, W, kc, torch.zeros_like(kc), *args,
                             n=n)["cnt"].cpu().numpy()
    want = _oracle_out(wl, x, W, centre, cache, codes, mp, x["q"], n, counts)
    _, tol = R.attention64(x["q"], cache, [n] * B, 128 ** -0.5)
    vmax = R.values64(cache.v_codes, cache.params, 1)[:, :, :n].abs().max()
    off = (out.double().cpu() - torch.from_numpy(want)).abs()
    assert (off <= (tol + 6e-6 * vmax).cpu()).all(), float(off.max())
    again = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, *args, n=n)
    assert torch.equal(out, again)


@pytest.mark.parametrize("variant,K,L", [("mips", 9, 100), ("cp", 1, 16)])
def test_variants_run_over_the_stored_cache(mp, variant, K, L):
    """Against the same variant's decode over the rows read back: the same values, at most
    rounded to fp32, so the outputs agree to the decode's own rounding."""
    wl = small_workload(name="kv4v", index=761, B=1, Hq=4, Hkv=2, n=3000, K=K, L=L, kv_dtype=F32,
                        q_dtype=F32, w_dtype=F32)
    x, W, kc, centre, cache, codes, extra = _sampled_case(mp, wl, 3100, variant)
    args = (wl.K, wl.L, wl.n_sink, wl.n_local)
    out = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, *args, n=wl.n, **extra)
    zero = torch.zeros_like(centre)
    k, v = mp.kv4_read(cache, wl.n, dtype=F32)
    kk = torch.zeros_like(kc)
    kk[:, :, :wl.n] = k
    vv = torch.zeros_like(kc)
    vv[:, :, :wl.n] = v
    want = mp.decode_attention(x["q"], codes, zero, W, kk, vv, *args, n=wl.n, **extra)
    for h in range(wl.Hq):
        assert row_rel_err(out[0, h].cpu().numpy(), want[0, h].double().cpu().numpy()) <= 1e-5


def test_a_prompt_and_decode_steps_as_they_are_used(mp):
    """A prompt stored, then tokens appended one by one: written to the cache, encoded, attended
    to exactly and by sampling; every K = 0 table collides, so that decode is the exact one."""
    B, Hq, Hkv, n0, steps, cap = 2, 8, 2, 2500, 5, 2600
    wl = small_workload(name="kv4run", index=762, B=B, Hq=Hq, Hkv=Hkv, n=n0 + steps, K=10, L=150)
    x = {k: v.cuda() for k, v in make_layer(wl).items()}
    W = make_hyperplanes(wl).cuda()
    args = (wl.K, wl.L, wl.n_sink, wl.n_local)
    kc = torch.zeros(B, Hkv, cap, 128, dtype=BF, device="cuda")
    kc[:, :, :n0] = x["keys"][:, :, :n0]
    centre = mp.key_mean(kc, n=n0)
    codes = torch.zeros(mp.codes_bytes(B, Hkv, cap, wl.K, wl.L) // 4, dtype=torch.int32,
                        device="cuda")
    mp.encode_keys(kc, centre, W, wl.K, wl.L, 0, n0, codes)
    cache = _filled(mp, B, Hkv, cap)
    mp.kv4_write(cache, x["keys"][:, :, :n0].contiguous(), x["values"][:, :, :n0].contiguous(),
                 centre=centre)
    pos = torch.full((B,), n0, dtype=torch.int32, device="cuda")
    for i in range(steps):
        n = n0 + i + 1
        k1 = x["keys"][:, :, n - 1:n].contiguous()
        kc[:, :, n - 1:n] = k1
        mp.encode_keys(kc, centre, W, wl.K, wl.L, n - 1, n, codes)
        mp.kv4_write(cache, k1, x["values"][:, :, n - 1:n].contiguous(), centre=centre,
                     positions=pos)
        pos += 1
        exact = mp.kv4_attention(x["q"], cache, n=cap, lengths=pos)
        want, tol = R.attention64(x["q"], cache, [n] * B, 128 ** -0.5)
        assert ((exact.double() - want).abs() <= tol).all()
        all_keys = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, 0, 2, wl.n_sink,
                                           wl.n_local, n=n)
        assert ((all_keys.double() - want).abs() <= 4 * tol + 1e-5).all()
        sampled = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, *args, n=n)
    dbg = mp.debug_select(x["q"], codes, centre, W, kc, torch.zeros_like(kc), *args, n=n)
    want = _oracle_out(wl, x, W, centre, cache, codes, mp, x["q"], n, dbg["cnt"].cpu().numpy())
    assert row_rel_err(sampled.cpu().numpy(), want) <= OUT_REL_TOL
    # and the whole is near the decode over the cache in bf16: the 4-bit rounding, not a fault
    vc = torch.zeros_like(kc)
    vc[:, :, :n] = x["values"][:, :, :n]
    full = mp.decode_attention(x["q"], codes, centre, W, kc, vc, *args, n=n)
    assert (full - sampled).norm() / full.norm() < 0.35


def test_refusals_of_the_binding(mp):
    cache = _random_cache(mp, 2, 2, 64, 64, seed=1)
    x = torch.zeros(2, 2, 4, 128, device="cuda")
    q = torch.zeros(2, 4, 128, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        mp.kv4_write(cache, x.half(), x.half())
    with pytest.raises(ValueError):
        mp.kv4_write(cache, x, x[:, :, :3].contiguous())
    with pytest.raises(ValueError):
        mp.kv4_write(cache, x[:, :1].contiguous(), x[:, :1].contiguous())    # heads
    with pytest.raises(ValueError):
        mp.kv4_write(cache, x.transpose(1, 2), x.transpose(1, 2))            # strides
    with pytest.raises(mp.MagicPIGError):
        mp.kv4_write(cache, x, x, n_begin=61)
    with pytest.raises(TypeError):
        mp.kv4_write(cache, x, x, positions=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        mp.kv4_write(cache, x, x, positions=torch.zeros(3, **i32))
    with pytest.raises(ValueError):
        mp.kv4_write(cache, x, x, centre=torch.zeros(2, 128, device="cuda"))
    with pytest.raises(TypeError):
        mp.kv4_write(cache, x, x, centre=torch.zeros(2, 2, 128, device="cuda").bfloat16())
    with pytest.raises(TypeError):
        mp.kv4_write(cache._replace(params=cache.params.float()), x, x)
    with pytest.raises(ValueError):
        mp.kv4_write(cache._replace(v_codes=cache.v_codes[:, :, :60]), x, x)
    for big in (2 ** 31, -2 ** 31 - 1, 2 ** 32):
        with pytest.raises(ValueError):
            mp.kv4_write(cache, x, x, n_begin=big)
        with pytest.raises(ValueError):
            mp.kv4_read(cache, 4, n_begin=big)
    with pytest.raises(mp.MagicPIGError):
        mp.kv4_read(cache, 65)
    with pytest.raises(TypeError):
        mp.kv4_read(cache, 4, dtype=torch.float16)
    with pytest.raises(ValueError):
        mp.kv4_read(cache, 4, keys=x[:, :, :2].contiguous())
    with pytest.raises(ValueError):
        mp.kv4_attention(q[:1].contiguous(), cache)
    with pytest.raises(ValueError):
        mp.kv4_attention(q, cache, n=65)
    with pytest.raises(ValueError):
        mp.kv4_attention(q, cache, n=0)
    with pytest.raises(TypeError):
        mp.kv4_attention(q.half(), cache)
    with pytest.raises(mp.MagicPIGError):
        mp.kv4_attention(torch.zeros(2, 3, 128, device="cuda"), cache)
    with pytest.raises(mp.MagicPIGError):
        mp.kv4_attention(torch.zeros(2, 4, 64, device="cuda"), cache)
    with pytest.raises(TypeError):
        mp.kv4_attention(q, cache, out=torch.zeros(2, 4, 128, device="cuda").bfloat16())
    with pytest.raises(ValueError):
        mp.kv4_attention(q, cache, lengths=torch.zeros(1, **i32))
    centre = torch.zeros(2, 2, 128, device="cuda")
    W = torch.zeros(128, 80, device="cuda")
    codes = torch.zeros(mp.codes_bytes(2, 2, 64, 8, 10) // 4, **i32)
    with pytest.raises(ValueError):
        mp.kv4_decode_attention(q, codes[:-1], centre, W, cache, 8, 10, 4, 8)
    with pytest.raises(ValueError):
        mp.kv4_decode_attention(q, codes, centre, W[:, :70].contiguous(), cache, 8, 10, 4, 8)
    with pytest.raises(ValueError):
        mp.kv4_decode_attention(q, codes, centre[:1], W, cache, 8, 10, 4, 8)
    with pytest.raises(ValueError):
        mp.kv4_decode_attention(q, codes, centre, W, cache, 8, 10, 4, 8,
                                radius=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        mp.kv4_attention(q, cache, workspace=torch.zeros(2, 512, device="cuda")[:, ::2])
    # a workspace too small for what the call needs, here or in the sampled decode
    long = mp.kv4_cache(1, 8, 98304)
    assert mp.kv4_attention_workspace_bytes(1, 32, 8, 98304) > 256
    with pytest.raises(mp.MagicPIGError):
        mp.kv4_attention(torch.zeros(1, 32, 128, device="cuda"), long,
                         workspace=torch.zeros(64, device="cuda"))
    with pytest.raises(mp.MagicPIGError):
        mp.kv4_decode_attention(q, codes, centre, W, cache, 8, 10, 4, 8,
                                workspace=torch.zeros(64, device="cuda"))
    assert mp.device_status() == 0


def _code_bits(mp, codes, B, Hkv, cap, C):
    """The sign bits [B, Hkv, blocks * 1024, C] of bit-sliced codes."""
    w = codes.view(B, Hkv, -(-cap // 1024), C, 32, 1)
    bits = (w >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1
    return bits.flatten(4).transpose(3, 4).flatten(2, 3)


# whole blocks, parts of blocks (short and long; begun or ended by the range, or both), fp32
@pytest.mark.parametrize("kd, wd, B, Hkv, m, cap, n0, K, L", [
    (BF, BF, 2, 2, 1, 1500, 0, 10, 150), (BF, BF, 1, 3, 64, 2048, 1000, 10, 13),
    (BF, BF, 2, 2, 65, 5000, 1023, 9, 20), (BF, BF, 1, 2, 2500, 5000, 0, 10, 150),
    (BF, BF, 2, 1, 3100, 4200, 1024, 5, 7), (BF, BF, 1, 1, 1024, 1024, 0, 10, 30),
    (BF, BF, 2, 3, 500, 1700, 300, 10, 150), (BF, BF, 1, 2, 900, 1000, 100, 10, 33),
    (BF, BF, 2, 2, 66, 2000, 958, 10, 20), (BF, BF, 1, 2, 1300, 2600, 1100, 8, 25),
    (F32, F32, 1, 2, 2300, 4000, 700, 10, 30), (F32, BF, 1, 2, 1, 1024, 1023, 10, 30),
    (BF, F32, 3, 1, 130, 300, 170, 1, 5)])
def test_codes_of_rows_that_no_cache_holds(mp, kd, wd, B, Hkv, m, cap, n0, K, L):
    """Signs of w . (k - mu) in 64 bits wherever float32 can tell (128 products and sums: an error
    below 2^-16 of the sum of the magnitudes); every other key's bits stay."""
    g = _gen(900 + m)
    C = K * L
    keys = (torch.randn(B, Hkv, m, 128, generator=g, device="cuda") + 0.5).to(kd)
    W = torch.randn(128, C, generator=g, device="cuda").to(wd)
    centre = 0.5 + 0.1 * torch.randn(B, Hkv, 128, generator=g, device="cuda")
    before = torch.randint(-2 ** 31, 2 ** 31, (mp.codes_bytes(B, Hkv, cap, K, L) // 4,),
                           generator=g, device="cuda", dtype=torch.int32)
    codes = mp.encode_rows(keys, centre, W, K, L, n0, cap, codes=before.clone())
    was = _code_bits(mp, before, B, Hkv, cap, C)
    got = _code_bits(mp, codes, B, Hkv, cap, C)
    kd64, mu, Wd = keys.double(), centre.double().unsqueeze(2), W.double()
    P = (kd64 - mu) @ Wd
    sure = P.abs() > 2.0 ** -16 * (kd64.abs() + mu.abs()) @ Wd.abs()
    assert sure.double().mean() > 0.99
    new = got[:, :, n0:n0 + m]
    assert torch.equal(new[sure], (P > 0).int()[sure])
    assert torch.equal(got[:, :, :n0], was[:, :, :n0])
    assert torch.equal(got[:, :, n0 + m:], was[:, :, n0 + m:])


def test_a_run_without_a_full_precision_cache(mp):
    """Prompt and appended tokens encoded and stored from their own rows alone, in pieces that
    begin and end inside blocks: the codes and the sampled decode are those of a bf16 cache."""
    B, Hq, Hkv, n0, steps, cap = 2, 8, 2, 3200, 3, 3300
    wl = small_workload(name="kv4rows", index=763, B=B, Hq=Hq, Hkv=Hkv, n=n0 + steps, K=10, L=150)
    x = {k: v.cuda() for k, v in make_layer(wl).items()}
    W = make_hyperplanes(wl).cuda()
    n = n0 + steps
    prompt = x["keys"][:, :, :n0].contiguous()
    centre = mp.key_mean(prompt)
    cache = _filled(mp, B, Hkv, cap)
    codes = None
    for a, b in [(0, 700), (700, 2900), (2900, n0)] + [(i, i + 1) for i in range(n0, n)]:
        k, v = (x[t][:, :, a:b].contiguous() for t in ("keys", "values"))
        codes = mp.encode_rows(k, centre, W, wl.K, wl.L, a, cap, codes=codes)
        mp.kv4_write(cache, k, v, n_begin=a, centre=centre)
    kc = torch.zeros(B, Hkv, cap, 128, dtype=BF, device="cuda")
    kc[:, :, :n] = x["keys"][:, :, :n]
    dbg = mp.debug_select(x["q"], codes, centre, W, kc, torch.zeros_like(kc), wl.K, wl.L,
                          wl.n_sink, wl.n_local, n=n)
    sampled = mp.kv4_decode_attention(x["q"], codes, centre, W, cache, wl.K, wl.L, wl.n_sink,
                                      wl.n_local, n=n)
    want = _oracle_out(wl, x, W, centre, cache, codes, mp, x["q"], n, dbg["cnt"].cpu().numpy())
    assert row_rel_err(sampled.cpu().numpy(), want) <= OUT_REL_TOL
    one = mp.build_tables(x["keys"][:, :, :n].contiguous(), centre, W, wl.K, wl.L)
    C, blocks = wl.K * wl.L, -(-n // 1024)
    differ = _code_bits(mp, codes, B, Hkv, cap, C)[:, :, :n] \
        != _code_bits(mp, one, B, Hkv, blocks * 1024, C)[:, :, :n]
    assert differ.double().mean() < 1e-5                     # signs that float32 cannot tell
    side = torch.cuda.Stream()                               # codes made and written there
    side.wait_stream(torch.cuda.current_stream())
    there = mp.encode_rows(prompt, centre, W, wl.K, wl.L, 0, cap, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(there, mp.encode_rows(prompt, centre, W, wl.K, wl.L, 0, cap))
    with pytest.raises(TypeError):
        mp.encode_rows(prompt, centre.to(BF), W, wl.K, wl.L, 0, cap)
    with pytest.raises(TypeError):
        mp.encode_rows(prompt, centre, W.cpu(), wl.K, wl.L, 0, cap)
    with pytest.raises(ValueError):
        mp.encode_rows(prompt, centre, W, wl.K, wl.L, cap - n0 + 1, cap)
    with pytest.raises(ValueError):
        mp.encode_rows(prompt, centre, W, wl.K, wl.L, 0, cap, codes=codes[:-1].contiguous())
    with pytest.raises(ValueError):
        mp.encode_rows(prompt, centre[:, :1].contiguous(), W, wl.K, wl.L, 0, cap)


def _chain(mp, x, n0, steps, sync):
    """Tokens appended and attended to, the calls back to back or each waited for."""
    B, Hkv = x["keys"].shape[:2]
    cap = n0 + steps
    cache = _filled(mp, B, Hkv, cap)
    pos = torch.full((B,), n0, dtype=torch.int32, device="cuda")
    mp.kv4_write(cache, x["keys"][:, :, :n0].contiguous(), x["values"][:, :, :n0].contiguous(),
                 centre=x["centre"])
    q = x["q"].clone()
    codes = mp.encode_rows(x["keys"][:, :, :n0].contiguous(), x["centre"], x["W"], 4, 20, 0, cap)
    rows = [[x[t][:, :, n0 + i:n0 + i + 1].contiguous() for t in ("keys", "values")]
            for i in range(steps)]
    outs = []
    wait = torch.cuda.synchronize if sync else (lambda: None)
    wait()
    for i, (k, v) in enumerate(rows):
        mp.kv4_write(cache, k, v, centre=x["centre"], positions=pos)
        wait()
        mp.encode_rows(k, x["centre"], x["W"], 4, 20, n0 + i, cap, codes=codes)
        wait()
        pos += 1
        outs.append(mp.kv4_attention(q, cache, n=cap, lengths=pos))
        wait()
        outs.append(mp.kv4_decode_attention(q, codes, x["centre"], x["W"], cache, 4, 20, 4, 64,
                                            n=n0 + i + 1))
        wait()
        q.mul_(0.5).add_(outs[-2].to(q.dtype))               # what the next step attends with
        outs.extend(mp.kv4_read(cache, 5, n_begin=n0 + i - 4, dtype=F32))
        wait()
    return outs + list(cache)


@pytest.mark.parametrize("B, Hq, Hkv, n0", [(1, 8, 2, 600), (2, 16, 4, 9000), (24, 32, 8, 700)])
def test_calls_back_to_back_equal_calls_waited_for(mp, B, Hq, Hkv, n0):
    """The kernels may start before their predecessors end: a step's output feeds the next one's
    queries, rows and codes, over layouts with one split, a cluster and a merge."""
    g = _gen(77)
    steps = 6
    x = {t: torch.randn(B, Hkv, n0 + steps, 128, generator=g, device="cuda").to(BF)
         for t in ("keys", "values")}
    x["q"] = torch.randn(B, Hq, 128, generator=g, device="cuda")
    x["W"] = torch.randn(128, 80, generator=g, device="cuda").to(BF)
    x["centre"] = mp.key_mean(x["keys"])
    want = _chain(mp, x, n0, steps, True)
    for _ in range(3):
        got = _chain(mp, x, n0, steps, False)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert _same(a, b)


def test_captured_behind_copies_and_other_streams(mp):
    """In a graph the calls follow a copy from the host, a fill, a join of two streams, or
    nothing."""
    B, Hq, Hkv, cap = 2, 8, 2, 5000
    g = _gen(78)
    kv = [torch.randn(B, Hkv, 3, 128, generator=g, device="cuda").to(BF) for _ in range(2)]
    cache = _random_cache(mp, B, Hkv, cap, cap, seed=79)
    before = _clone(cache)
    host = torch.randn(B, Hq, 128).pin_memory()
    q, q2 = torch.zeros(B, Hq, 128, device="cuda"), torch.zeros(B, Hq, 128, device="cuda")
    out = [torch.zeros(B, Hq, 128, device="cuda") for _ in range(3)]
    ws = torch.empty(mp.kv4_attention_workspace_bytes(B, Hq, Hkv, cap) + 256, dtype=torch.uint8,
                     device="cuda")
    kr = [torch.zeros_like(kv[0]) for _ in range(2)]
    side = torch.cuda.Stream()

    def work():
        mp.kv4_attention(q2, cache, out=out[0], workspace=ws)            # first in the graph
        q.copy_(host, non_blocking=True)
        mp.kv4_attention(q, cache, out=out[1], workspace=ws)             # behind a copy
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q2.copy_(q).mul_(2.0)
        mp.kv4_write(cache, *kv, n_begin=7)
        torch.cuda.current_stream().wait_stream(side)
        mp.kv4_attention(q2, cache, out=out[2], workspace=ws)            # behind two streams
        kr[0].zero_()
        mp.kv4_read(cache, 3, n_begin=7, keys=kr[0], values=kr[1])       # behind a fill

    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in out[1:] + kr]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for t, was in zip(cache, before):
        t.copy_(was)
    for t in out + kr:
        t.zero_()
    q2.copy_(host.cuda())
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    # the second replay's first two calls meet the rows that the first one wrote
    first = mp.kv4_attention(2.0 * host.cuda(), cache)
    assert _same(out[0], first)
    assert _same(out[1], mp.kv4_attention(host.cuda(), cache))
    for a, b in zip(out[2:] + kr, want[1:]):
        assert _same(a, b)
