"""Calls over the paged cache that its documentation allows and the other tests do not make."""
import pytest
import torch

from tests import paged_reference as R
from tests.test_gpu_paged import (BF, F32, _attend_and_check, _chosen, _gen, _ints, _pages_of, _randn,
                                  _random_cache)
from workloads import make_hyperplanes, make_layer, small_workload

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


def test_codes_laid_out_for_the_largest_capacity(mp):
    """2^31 - 1 tokens a head: the codes' stride is that of 2^21 blocks, and places near the end are there."""
    Hkv, m, cap, K, L = 3, 64, 2 ** 31 - 1, 1, 1
    g = _gen(31)
    keys = _randn(g, 1, Hkv, m, 128)
    W, centre = _randn(g, 128, K * L), _randn(g, 1, Hkv, 128) * 0.1
    codes = torch.zeros(Hkv, 2 ** 21, 32, dtype=torch.int32, device="cuda")
    assert codes.numel() * 4 == mp.codes_bytes(1, Hkv, cap, K, L)
    for pos, left in ((1024 * 3 + 5, m), (cap - 40, 40), (1024 * 2 ** 20 - 17, m)):
        codes.zero_()
        mp.encode_rows_at(keys, centre, W, K, L, _ints([pos]), cap, codes)
        at = pos % 1024
        want = mp.encode_rows_at(keys[:, :, :left].contiguous(), centre, W, K, L, _ints([at]), 2048,
                                 torch.zeros(Hkv, 2, 32, dtype=torch.int32, device="cuda"))
        first = pos // 1024
        for h in range(Hkv):
            nonzero = codes[h].any(-1).nonzero().flatten().tolist()
            assert nonzero and all(first <= b <= first + 1 for b in nonzero)
            assert torch.equal(codes[h, first:first + 2], want[h, :min(2, 2 ** 21 - first)])


def test_sampled_decode_with_codes_of_the_largest_capacity(mp):
    B, Hq, Hkv, n, page, K, L = 1, 4, 2, 3000, 16, 2, 3
    g = _gen(32)
    cache, table = _random_cache(mp, g, B, Hkv, n, page, BF, [n])
    keys = _randn(g, B, Hkv, n, 128).to(BF)
    W, centre = _randn(g, 128, K * L).to(BF), _randn(g, B, Hkv, 128) * 0.1
    q = _randn(g, B, Hq, 128).to(BF)
    near = mp.encode_rows(keys, centre, W, K, L, 0, n)
    want = mp.paged_decode_attention(q, near, centre, W, cache, table, K, L, 4, 64, n=n, n_capacity=n)
    far = torch.zeros(Hkv, 2 ** 21, K * L * 32, dtype=torch.int32, device="cuda")
    far[:, :3] = near.view(torch.int32).view(Hkv, 3, -1)
    assert torch.equal(mp.paged_decode_attention(q, far, centre, W, cache, table, K, L, 4, 64, n=n,
                                                 n_capacity=2 ** 31 - 1), want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sampled_decode_of_the_most_rows(mp, dtype):
    """65520 query rows of 65535: every row is that of a batch of its own."""
    B, Hq, Hkv, n, page, K, L = 4095, 16, 2, 72, 8, 2, 20
    g = _gen(33)
    lens = [b % (n + 1) for b in range(B)]
    slots = n // page
    cache = mp.paged_cache(64, Hkv, page, dtype)
    for t in cache:
        t.copy_(_randn(g, *t.shape))
    table = torch.randint(0, 64, (B, slots), generator=g, device="cuda").int()
    W, centre = _randn(g, 128, K * L).to(dtype), _randn(g, B, Hkv, 128) * 0.1
    q = _randn(g, B, Hq, 128).to(dtype)
    rows = cache.keys[table.long()].transpose(1, 2).reshape(B, Hkv, n, 128)
    codes = mp.encode_rows(rows.contiguous(), centre, W, K, L, 0, n)
    out = mp.paged_decode_attention(q, codes, centre, W, cache, table, K, L, 2, 9, n=n, lengths=_ints(lens),
                                    n_capacity=n)
    per = codes.view(torch.int32).view(B, -1)
    for b in (0, 1, 5, 72, 2047, 2048, 4000, 4094):
        own = mp.paged_decode_attention(q[b:b + 1], per[b], centre[b:b + 1], W, cache, table[b:b + 1], K, L, 2,
                                        9, n=n, lengths=_ints(lens[b:b + 1]), n_capacity=n)
        # (a single sequence's rows are shared by clusters: sums of the same keys in another order)
        assert (out[b] - own[0]).abs().max() <= 2e-5
        assert lens[b] > 0 or (out[b] == 0).all()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sink", [0, 96])
def test_sampled_decode_of_the_lowest_logits_behind_a_missing_page(mp, dtype, sink):
    """Logits of -3.2e38 behind a page that is not there: what stands for its tokens is no higher. The keys are
    one and the same row, so that all weights are 1, and the output is the mean of the values."""
    n, page = 96, 32
    g = _gen(34)
    q = torch.full((1, 1, 128), -1.0, device="cuda").to(dtype)
    cache = mp.paged_cache(3, 1, page, dtype)
    cache.keys.fill_(2.5)                        # q.k = -320, exactly
    cache.values.copy_(_randn(g, *cache.values.shape))
    table = _ints([[-1, 0, 2]])
    W, centre = _randn(g, 128, 2), torch.zeros(1, 1, 128, device="cuda")
    codes = torch.zeros(4, dtype=torch.int32, device="cuda")             # K = 0: every key is sampled, log u = 0
    out = mp.paged_decode_attention(q, codes, centre, W, cache, table, 0, 2, sink, 0, scale=1e36)
    v = torch.cat([cache.values[0, 0], cache.values[2, 0]]).double()
    # sums of 64 values, each step rounded: 64 half steps of the largest sum at most, and the division
    assert (out[0, 0].double() - v.mean(0)).abs().max() <= 2.0 ** -24 * 66 * v.abs().max()


@pytest.mark.parametrize("interleaved", [False, True])
def test_cosines_and_sines_of_all_quarters_of_a_turn(mp, interleaved):
    """A pair (1, 0) becomes (cos, sin) exactly, so that these show by themselves: off by what the header gives
    for the angle, and by a unit in the last place of each (at most 2^-23 of it)."""
    starts = [0, 1, 2, 3, 5, 97, 1000, 4095, 65537, 2 ** 20 - 3, -1, -4, -70001]
    B, m, r = len(starts), 64, 128
    x = torch.zeros(B, 1, m, 128, device="cuda")
    first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, 64), slice(64, 128))
    x[..., first] = 1.0
    # every eighth of a turn among the angles at position 1, the quarters and their neighbours too
    freq = (torch.arange(64, device="cuda").double() / 32 * torch.pi).float()
    table, cache = torch.full((B, 1), -1, dtype=torch.int32, device="cuda"), mp.paged_cache(1, 1, 8, F32)
    out = torch.empty_like(x)
    mp.paged_append(cache, table, x, x, positions=_ints(starts), inv_freq=freq, interleaved=interleaved,
                    keys_out=out)
    p = torch.tensor(starts, device="cuda").double()[:, None] + torch.arange(m, device="cuda")
    a = (p[..., None] * freq.double())[:, None]
    # 2^-52 of the angle twice: the reference's product and its own reduction
    angle = 2.0 ** -25 + (2.0 ** -61 * (1 + freq.double()) * p[..., None].abs())[:, None] + 2.0 ** -51 * a.abs()
    for got, want in ((out[..., first], a.cos()), (out[..., second], a.sin())):
        off = (got.double() - want).abs() - angle - 2.0 ** -23 * want.abs()
        assert (off <= 0).all(), off.max().item()
    assert (out[0, 0, 0, first] == 1).all() and (out[0, 0, 0, second] == 0).all()        # position 0


def _layer(B, Hq, Hkv, n, K, L, seed):
    wl = small_workload(name="pagede", index=seed, B=B, Hq=Hq, Hkv=Hkv, n=n, K=K, L=L, kv_dtype=F32, q_dtype=F32,
                        w_dtype=F32)
    return {k: v.cuda() for k, v in make_layer(wl).items()}, make_hyperplanes(wl).cuda()


@pytest.mark.parametrize("qt,kt,wt", [(F32, BF, BF), (BF, F32, F32), (BF, BF, F32), (F32, F32, BF),
                                      (F32, BF, F32), (BF, F32, BF)])
@pytest.mark.parametrize("B,Hq,Hkv", [(3, 8, 2), (23, 8, 4), (37, 16, 2)])
def test_sampled_decode_of_mixed_types(mp, qt, kt, wt, B, Hq, Hkv):
    """Queries, cache and hyperplanes of different types, at batches of each form of the query encoding (24, 184
    and 592 rows)."""
    n, page, K, L, args = 600, 24, 6, 50, (6, 50, 3, 20)
    lens = [(n, 0, 1, 333, 70, 24, 23)[b % 7] for b in range(B)]
    x, W = _layer(B, Hq, Hkv, n, K, L, 790)
    x = dict(q=x["q"].to(qt), keys=x["keys"].to(kt), values=x["values"].to(kt))
    W = W.to(wt)
    centre = mp.key_mean(x["keys"])
    g = _gen(B)
    cache, table = _pages_of(mp, g, x, n, page)
    codes = mp.encode_rows(x["keys"], centre, W, K, L, 0, n)
    chosen = _chosen(mp, x, codes, centre, W, lens, n, args, Hkv)
    out = mp.paged_decode_attention(x["q"], codes, centre, W, cache, table, *args, n=n, lengths=_ints(lens),
                                    n_capacity=n)
    want, tol = R.sampled(x["q"], centre, cache.keys, cache.values, table.cpu(), lens, chosen, *args, 128 ** -0.5)
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("wt", [BF, F32])
@pytest.mark.parametrize("B,Hq,Hkv", [(2, 4, 2), (33, 2, 2), (43, 3, 3), (33, 4, 2), (70, 8, 4), (129, 4, 4), (100, 3, 3)])
def test_hyperplanes_aligned_to_their_element_only(mp, wt, B, Hq, Hkv):
    """And heads without a group, in each form of the query encoding: the outputs and codes of aligned ones."""
    n, page, K, L = 200, 8, 4, 40
    x, W = _layer(B, Hq, Hkv, n, K, L, 791)
    W = W.to(wt)
    off = torch.empty(W.numel() + 1, dtype=wt, device="cuda")[1:].view(W.shape)
    off.copy_(W)
    assert off.data_ptr() % (2 * off.element_size()) == off.element_size() and W.data_ptr() % 16 == 0
    lens = [(37 * b) % (n + 1) for b in range(B)]
    centre = mp.key_mean(x["keys"])
    g = _gen(B)
    cache, table = _pages_of(mp, g, x, n, page)
    codes = mp.encode_rows(x["keys"], centre, W, K, L, 0, n)
    rows = x["keys"][:, :, :7].contiguous()
    for kt in (BF, F32):
        at = _ints([(11 * b) % n for b in range(B)])
        two = [mp.encode_rows_at(rows.to(kt), centre, w, K, L, at, n, codes.clone()) for w in (W, off)]
        assert torch.equal(*two)
    args, kw = (K, L, 2, 9), dict(n=n, lengths=_ints(lens), n_capacity=n)
    out = mp.paged_decode_attention(x["q"], codes, centre, off, cache, table, *args, **kw)
    assert torch.equal(mp.paged_decode_attention(x["q"], codes, centre, W, cache, table, *args, **kw), out)
    chosen = _chosen(mp, x, codes, centre, W, lens, n, args, Hkv)
    want, tol = R.sampled(x["q"], centre, cache.keys, cache.values, table.cpu(), lens, chosen, *args, 128 ** -0.5)
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("B,Hkv,m,cap,K,L", [(5, 3, 17, 3001, 8, 75), (64, 8, 1, 1500, 10, 150), (2, 1, 64, 1100, 3, 7)])
def test_codes_of_float32_keys_by_bf16_hyperplanes(mp, B, Hkv, m, cap, K, L):
    g = _gen(cap)
    keys, centre = _randn(g, B, Hkv, m, 128), _randn(g, B, Hkv, 128) * 0.1
    W = _randn(g, 128, K * L).to(BF)
    starts = [(997 * b) % (cap - m + 1) for b in range(B)]
    old = torch.randint(-2 ** 31, 2 ** 31 - 1, (mp.codes_bytes(B, Hkv, cap, K, L) // 4,), generator=g,
                        device="cuda").int()
    codes = mp.encode_rows_at(keys, centre, W, K, L, _ints(starts), cap, old.clone())
    per = old.numel() // B
    for b in range(B):
        want = old[b * per:(b + 1) * per].clone()
        mp.encode_rows(keys[b:b + 1], centre[b:b + 1], W, K, L, starts[b], cap, codes=want)
        assert torch.equal(codes[b * per:(b + 1) * per], want)


@pytest.mark.parametrize("variant,K,L", [("mips", 8, 75), ("cp", 1, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_variants_over_pages_of_empty_sequences_and_missing_pages(mp, variant, K, L, dtype):
    n, page, lens = 2100, 16, [0, 2100, 1, 1500, 0]
    B, Hq, Hkv = len(lens), 4, 2
    x, W = _layer(B, Hq, Hkv, n, 1 if variant == "cp" else K, L, 792)
    x = {k: v.to(dtype) for k, v in x.items()}
    g = _gen(2)
    centre, extra = mp.key_mean(x["keys"]), {}
    if variant == "mips":
        W = torch.cat([W, _randn(g, 1, K * L)]).to(dtype).contiguous()
        extra["radius"] = mp.key_radius(x["keys"], centre)
        codes = mp.encode_keys_mips(x["keys"], centre, W, extra["radius"], K, L, 0, n)
    else:
        W = _randn(g, L, 128, 128).to(dtype)
        extra["logu_table"] = mp.cp_logu_table(1, L)
        codes = mp.encode_keys_cp(x["keys"], centre, W, L, 0, n)
    cache, table = _pages_of(mp, g, x, n, page)

    def run(**kw):
        return mp.paged_decode_attention(x["q"], codes, centre, W, cache, table, K, L, 4, 64, n=n, n_capacity=n,
                                         lengths=_ints(lens), **extra, **kw)

    out = run()
    per = codes.numel() // B
    for b, used in enumerate(lens):
        if used == 0:
            assert (out[b] == 0).all()
            continue
        one = {k: v[b:b + 1].contiguous() if k == "radius" else v for k, v in extra.items()}
        want = mp.decode_attention(x["q"][b:b + 1], codes.view(-1)[b * per:(b + 1) * per], centre[b:b + 1], W,
                                   x["keys"][b:b + 1], x["values"][b:b + 1], K, L, 4, 64, n=used, **one)
        # log u: 2e-5 of the contiguous form's table, twice (weights), of values of up to 5
        assert (out[b] - want[0]).abs().max() <= 2 * 4e-5 * 5
    table[1] = -1                                # nothing left of the longest
    again = run()
    assert (again[1] == 0).all()
    assert torch.equal(again[[0, 2, 3, 4]], out[[0, 2, 3, 4]])
    mp.paged_decode_attention(x["q"], codes, centre, W, cache, table, K, L, 4, 64, n=n, n_capacity=n,
                              lengths=_ints([0] * B), out=out, **extra)
    assert (out == 0).all()


def test_radii_and_tables_of_other_types_are_refused(mp):
    """They are read as float32: half as many bytes would be read past their end."""
    cache = mp.paged_cache(6, 2, 16)
    table = torch.arange(6, device="cuda").view(2, 3).int()
    q, W, centre = _randn(_gen(1), 2, 4, 128), torch.zeros(128, 80, device="cuda"), torch.zeros(2, 2, 128, device="cuda")
    codes = torch.zeros(mp.codes_bytes(2, 2, 48, 8, 10) // 4, dtype=torch.int32, device="cuda")
    kv4 = mp.kv4_cache(2, 2, 48)
    entries = torch.zeros(mp.MP_LOGU_TABLE_ENTRIES, device="cuda")
    for t in (BF, torch.float16, torch.float64, torch.int32):
        for kw in (dict(radius=torch.ones(2, 2, device="cuda").to(t)), dict(logu_table=entries.to(t))):
            K, L = (1, 10) if "logu_table" in kw else (8, 10)
            with pytest.raises(TypeError):
                mp.paged_decode_attention(q, codes, centre, W, cache, table, K, L, 4, 64, **kw)
            with pytest.raises(TypeError):
                mp.kv4_decode_attention(q, codes, centre, W, kv4, K, L, 4, 64, **kw)
    with pytest.raises(ValueError):
        mp.paged_decode_attention(q, codes, centre, W, cache, table, 8, 10, 4, 64, radius=torch.ones(3, device="cuda"))
    torch.cuda.synchronize()
    assert mp.device_status() == 0
