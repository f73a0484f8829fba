"""Measured cases of the paged K/V cache: tokens appended with their rotary positions, exact
attention of single tokens over the pages, the LSH-sampled decode over them, and the codes of
tokens that join sequences of different lengths.

The cache is a pool of pages, keys and values [n_pages, Hkv, page_size, 128] (bf16 or float32);
page_table int32 [B, pages] says which page holds the tokens [j page_size, (j + 1) page_size) of a
sequence. The rotation takes a pair (x, y) of a row's first rotary_dims dims, number j, at position p to
(x cos a - y sin a, y cos a + x sin a), a = p inv_freq[j]; pairs are (j, j + rotary_dims / 2), or
(2 j, 2 j + 1) where they are interleaved. Codes are bit-sliced in blocks of 1024 keys: int32
[B, Hkv, blocks, K L, 32], bit i % 32 of word (i % 1024) / 32 the sign of key i.
"""
import functools
import math

import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
N_SINK, N_LOCAL = 4, 64
# Share of the keys that a query head samples on these inputs at (K, L) = (10, 150), as the pages
# quote it.
SAMPLED_SHARE = 0.0157


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 sequences: a token each
        dict(name="append_b64", op="append", dtype="bf16", B=64, Hq=32, Hkv=8, m=1, cap=512,
             page=16, rotary=128, interleaved=False, ragged=True),
        # a padded chunk of an fp32 model that rotates half of its dims, pairs interleaved
        dict(name="append_f32_odd", op="append", dtype="f32", B=5, Hq=12, Hkv=3, m=333, cap=1801,
             page=24, rotary=64, interleaved=True, ragged=True),
        # the last chunk of the 96K-token prompt
        dict(name="append_8k", op="append", dtype="bf16", B=1, Hq=32, Hkv=8, m=8192, cap=98304,
             page=64, rotary=128, interleaved=False, ragged=False),
        # a short context, one sequence: latency
        dict(name="attend_b1_512", op="attend", dtype="bf16", B=1, Hq=32, Hkv=8, n=512, page=16,
             ragged=False),
        # one query head per KV head in fp32, sequences of different odd lengths
        dict(name="attend_mha_f32", op="attend", dtype="f32", B=7, Hq=12, Hkv=12, n=3001, page=48,
             ragged=True),
        # the 96K-token workload, one layer
        dict(name="attend_b1_96k", op="attend", dtype="bf16", B=1, Hq=32, Hkv=8, n=98304, page=64,
             ragged=False),
        # the 70B-shaped workload: eight query heads per KV head, 128K tokens, two sequences
        dict(name="attend_b2_128k_g8", op="attend", dtype="bf16", B=2, Hq=64, Hkv=8, n=131072,
             page=128, ragged=False),
        # large-batch decode, 32 sequences of up to 32K tokens
        dict(name="attend_b32_32k", op="attend", dtype="bf16", B=32, Hq=32, Hkv=8, n=32768,
             page=16, ragged=True),
        # sampled decode of four sequences of up to 16K tokens
        dict(name="sampled_b4_16k", op="sampled", dtype="bf16", B=4, Hq=32, Hkv=8, n=16384,
             page=16, K=10, L=150, ragged=True),
        # sampled decode of the 96K-token workload, one layer
        dict(name="sampled_b1_96k", op="sampled", dtype="bf16", B=1, Hq=32, Hkv=8, n=98304,
             page=64, K=10, L=150, ragged=False),
        # the codes of a decode step's tokens, one for each of 32 sequences
        dict(name="encode_b32", op="encode", dtype="bf16", B=32, Hkv=8, m=1, cap=2048, K=10, L=150),
        # the codes of a few tokens at once, fp32
        dict(name="encode_f32_m17", op="encode", dtype="f32", B=5, Hkv=3, m=17, cap=5001, K=8, L=75),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "sampled", "encode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([8, 16, 16, 24, 32, 48, 64, 64, 128, 256])
    size = 2 if dtype == "bf16" else 1
    if op == "append":
        B, Hkv, G = _log_int(rng, 1, 64), rng.randint(1, 12), rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
        m = _log_int(rng, 1, max(1, min(8192, 40_000 * size // (B * Hkv))))
        cap = m + _log_int(rng, 1, max(2, 400_000 * size // (B * Hkv) - m))
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, m=m, cap=cap, page=page,
                    rotary=rng.choice([128, 128, 64, 96, 32]), interleaved=rng.random() < 0.4,
                    ragged=rng.random() < 0.5)
    if op == "attend":
        B, Hkv = _log_int(rng, 1, 32), rng.randint(1, 12)
        G = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 12, 16])
        n = _log_int(rng, 1, min(131072, 2_000_000 * size // (B * Hkv)))
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, n=n, page=page,
                    ragged=rng.random() < 0.5)
    Hkv, K, L = rng.choice([1, 2, 4, 8]), rng.randint(6, 12), rng.randint(40, 200)
    if op == "encode":
        B, m = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        cap = m + _log_int(rng, 1, max(2, 400_000_000 // (B * Hkv * K * L)))
        return dict(op=op, dtype=dtype, B=B, Hkv=Hkv, m=m, cap=cap, K=K, L=L)
    G, B = rng.choice([1, 2, 4, 8]), rng.randint(1, 4)
    most = 4_000_000_000 // (B * Hkv * G * K * L)
    n = _log_int(rng, 500, max(600, min(98304, most)))
    return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, n=n, page=page, K=K, L=L,
                ragged=rng.random() < 0.5)


def work(case):
    B, Hkv = case["B"], case["Hkv"]
    size = 2 if case["dtype"] == "bf16" else 4
    row = D * size
    if case["op"] == "append":
        # sequences of different counts append between half of m and m tokens
        tokens = B * (case["m"] * 0.75 if case["ragged"] and case["m"] > 1 else case["m"])
        Hq = case["Hq"]
        return {"bytes": tokens * row * (2 * Hq + 5 * Hkv),          # rotated keys are returned too
                "flops": tokens * (Hq + Hkv) * case["rotary"] * 3}
    if case["op"] == "encode":
        C = case["K"] * case["L"]
        tokens = B * Hkv * case["m"]
        return {"bytes": tokens * (row + C / 8) + D * C * size + B * Hkv * D * 4,
                "flops": tokens * 2 * D * C}
    Hq, n = case["Hq"], case["n"]
    ends = B * Hq * (row + 4 * D)
    # sequences of different lengths are between half of n and n
    tokens = B * n * (0.75 if case["ragged"] else 1.0)
    if case["op"] == "attend":
        return {"bytes": tokens * Hkv * 2 * row + ends, "flops": tokens * Hq * 4 * D}
    C = case["K"] * case["L"]
    per_head = tokens / B * SAMPLED_SHARE
    exact = min(tokens / B, N_SINK + N_LOCAL)
    rows = B * Hkv * min(tokens / B, Hq // Hkv * per_head + exact)
    return {"bytes": tokens * Hkv * C / 8 + rows * 2 * row + ends + D * C * 2 + B * Hkv * D * 4,
            "flops": B * Hq * ((per_head + exact) * 6 * D + 2 * D * C)}


# ------------------------------------------------------------------------------------- inputs
def _ceil_div(a, b):
    return -(-a // b)


def _pages(B, cap, page, gen, device):
    """A table of pages dealt out at random, and how many pages there are."""
    per = _ceil_div(cap, page)
    n_pages = B * per + 3
    table = torch.randperm(n_pages, generator=gen, device=device)[:B * per]
    return table.view(B, per).to(torch.int32), n_pages


def _between(lo, hi, B, gen, device):
    return torch.randint(lo, hi + 1, (B,), generator=gen, device=device).to(torch.int32)


def _fill(pool, pages, rows):
    """rows [Hkv, n, 128] into the pages of one sequence."""
    Hkv, n, _ = rows.shape
    page = pool.shape[2]
    used = _ceil_div(n, page)
    padded = torch.zeros(Hkv, used * page, D, dtype=pool.dtype, device=pool.device)
    padded[:, :n] = rows.to(pool.dtype)
    pool[pages[:used].long()] = padded.view(Hkv, used, page, D).transpose(0, 1)


def _geometry(B, Hkv, Hq, gen, device):
    """The cone of the keys and the opposite cone of the queries: centre 8 u, queries around
    -4 u. Queries lie on a grid of 1/32 (all of it bf16): with hyperplanes on a grid of 1/16 every
    projection is exact in float32, so that no sign depends on the order of a sum."""
    u = torch.randn(B, Hkv, D, generator=gen, device=device)
    u = u / u.norm(dim=-1, keepdim=True)
    q = 0.5 * torch.randn(B, Hq, D, generator=gen, device=device)
    q = q - 4 * u.repeat_interleave(Hq // Hkv, dim=1)
    return 8 * u, (q * 32).round().clamp(-255, 255) / 32


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    op, dtype, B, Hkv = case["op"], DTYPES[case["dtype"]], case["B"], case["Hkv"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    s = dict(op=op)
    if op == "append":
        Hq, m, cap, page, r = case["Hq"], case["m"], case["cap"], case["page"], case["rotary"]
        s["table"], n_pages = _pages(B, cap, page, gen, device)
        s["keys"] = torch.zeros(n_pages, Hkv, page, D, dtype=dtype, device=device)
        s["values"] = torch.zeros_like(s["keys"])
        # one projection's output: queries, keys and values of a token next to each other
        x = randn(B, m, Hq + 2 * Hkv, D).to(dtype).transpose(1, 2)
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s["positions"] = _between(0, cap - m, B, gen, device) if case["ragged"] else torch.full(
            (B,), cap - m, dtype=torch.int32, device=device)
        s["counts"] = _between(_ceil_div(m, 2), m, B, gen, device) if case["ragged"] else None
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, r, 2, device=device,
                                                    dtype=torch.float64) / r)).float()
        s["interleaved"] = case["interleaved"]
        # rows past a sequence's count keep what these hold
        s["q_out"] = torch.zeros(B, Hq, m, D, dtype=dtype, device=device)
        s["keys_out"] = torch.zeros(B, Hkv, m, D, dtype=dtype, device=device)
        return s
    if op == "encode":
        m, cap, K, L = case["m"], case["cap"], case["K"], case["L"]
        # on grids, as the queries above: every projection is exact in float32
        s["centre"] = (8 * torch.nn.functional.normalize(randn(B, Hkv, D), dim=-1) * 32
                       ).round() / 32
        k = randn(B, Hkv, m, D) + s["centre"].unsqueeze(2)
        s["k"] = ((k * 32).round().clamp(-255, 255) / 32).to(dtype)
        s["W"] = ((randn(D, K * L) * 16).round() / 16).to(dtype)
        s["positions"] = _between(0, cap - m, B, gen, device)
        s["codes"] = torch.randint(-2**31, 2**31, (B, Hkv, _ceil_div(cap, 1024), K * L, 32),
                                   generator=gen, device=device, dtype=torch.int32)
        s["K"], s["L"], s["cap"] = K, L, cap
        return s
    Hq, n, page = case["Hq"], case["n"], case["page"]
    centre, q = _geometry(B, Hkv, Hq, gen, device)
    s["n"], s["q"] = n, q.to(dtype)
    s["table"], n_pages = _pages(B, n, page, gen, device)
    s["keys"] = torch.zeros(n_pages, Hkv, page, D, dtype=dtype, device=device)
    s["values"] = torch.zeros_like(s["keys"])
    lengths = torch.full((B,), n, dtype=torch.int32, device=device)
    if case["ragged"]:
        lengths = _between(_ceil_div(n, 2), n, B, gen, device)
    s["lengths"] = lengths if case["ragged"] else None
    C = case["K"] * case["L"] if op == "sampled" else 0
    if C:
        s["K"], s["L"], s["centre"] = case["K"], case["L"], centre
        s["W"] = ((randn(D, C) * 16).round() / 16).to(dtype)
        nblk = _ceil_div(s["table"].shape[1] * page, 1024)
        codes = torch.zeros(B, Hkv, nblk, C, 128, dtype=torch.uint8, device=device)
    # keys: noise around the centre, and the first token twelve deviations along the mean query
    # of its head (the attention sink)
    sink = 12 * torch.nn.functional.normalize(q.unflatten(1, (Hkv, Hq // Hkv)).mean(2), dim=-1)
    for b in range(B):
        k = randn(Hkv, n, D)
        k[:, 0] = sink[b]
        k = (k + centre[b].unsqueeze(1)).to(dtype)
        _fill(s["keys"], s["table"][b], k)
        _fill(s["values"], s["table"][b], randn(Hkv, n, D))
        for g in range(Hkv if C else 0):
            bits = torch.zeros(nblk * 1024, C, dtype=torch.bool, device=device)
            bits[:n] = (k[g].float() - centre[b, g]) @ s["W"].float() > 0
            bits = bits.view(nblk, 128, 8, C).to(torch.uint8)
            bits <<= torch.arange(8, dtype=torch.uint8, device=device)[:, None]
            codes[b, g] = bits.sum(2, dtype=torch.uint8).transpose(1, 2)
    if C:
        s["codes"] = codes.view(torch.int32)
    if case["ragged"]:
        # pages that a sequence has not come to are not in its table yet
        j = torch.arange(s["table"].shape[1], device=device)
        s["table"] = torch.where(j * page < lengths.unsqueeze(1), s["table"], -1)
    s["out"] = torch.empty(B, Hq, D, dtype=torch.float32, device=device)
    s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device=device)
    return s


# -------------------------------------------------------------------------------- plain forms
def _rotated(x, positions, inv_freq, interleaved):
    """x [B, H, m, 128], its first dims turned by their positions; float32, angles in 64 bits."""
    m, r = x.shape[2], 2 * inv_freq.numel()
    p = positions.double().unsqueeze(1) + torch.arange(m, device=x.device)
    angle = (p.unsqueeze(-1) * inv_freq.double()).unsqueeze(1)
    cos, sin = angle.cos().float(), angle.sin().float()
    x = x.float()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _append_plain(s):
    B, _, m, _ = s["k"].shape
    page, device = s["keys"].shape[2], s["k"].device
    i = torch.arange(m, device=device)
    live = (i < (m if s["counts"] is None else s["counts"].unsqueeze(1))).expand(B, m)
    q = _rotated(s["q"], s["positions"], s["inv_freq"], s["interleaved"]).to(s["q"].dtype)
    k = _rotated(s["k"], s["positions"], s["inv_freq"], s["interleaved"]).to(s["k"].dtype)
    keep = live[:, None, :, None]
    torch.where(keep, q, s["q_out"], out=s["q_out"])
    torch.where(keep, k, s["keys_out"], out=s["keys_out"])
    at = s["positions"].long().unsqueeze(1) + i
    pages = s["table"].long().gather(1, at // page)
    where = (pages, at % page)
    keep = live[:, :, None, None]
    for pool, rows in ((s["keys"], k), (s["values"], s["v"])):
        was = pool[where[0], :, where[1]]                              # [B, m, Hkv, 128]
        pool[where[0], :, where[1]] = torch.where(keep, rows.transpose(1, 2), was)
    return s["q_out"], s["keys_out"], s["keys"], s["values"]


def _encode_plain(s):
    B, Hkv, m, _ = s["k"].shape
    C = s["K"] * s["L"]
    bits = (s["k"].float() - s["centre"].unsqueeze(2)) @ s["W"].float() > 0
    codes = s["codes"].view(torch.uint8)                               # bytes of eight keys
    b = torch.arange(B, device=codes.device)
    for i in range(m):
        p = s["positions"].long() + i
        at = (b, slice(None), p // 1024, slice(None), p % 1024 // 8)
        mask = (1 << (p % 8)).to(torch.uint8)[:, None, None]
        codes[at] = (codes[at] & ~mask) | torch.where(bits[:, :, i], mask, 0)
    return s["codes"].view(B, Hkv, -1, C, 32)


def _sequence(s, pool, b):
    """The first n rows of one sequence, [Hkv, n, 128] float32."""
    pages = s["table"][b, :_ceil_div(s["n"], pool.shape[2])].long().clamp_min(0)
    return pool[pages].transpose(0, 1).flatten(1, 2)[:, :s["n"]].float()


def _softmax_values(logits, v):
    w = torch.exp(logits - logits.amax(-1, keepdim=True).clamp_min(-3e38))
    total = w.sum(-1, keepdim=True)
    return torch.where(total > 0, (w @ v) / total.clamp_min(1e-37), 0.0)


def _attend_plain(s):
    B, _, D_ = s["q"].shape
    Hkv = s["keys"].shape[1]
    i = torch.arange(s["n"], device=s["q"].device)
    out = s["out"]
    for b in range(B):
        q = s["q"][b].float().unflatten(0, (Hkv, -1))
        logits = q @ _sequence(s, s["keys"], b).transpose(-1, -2) / math.sqrt(D)
        if s["lengths"] is not None:
            logits = logits.masked_fill(i >= s["lengths"][b], -math.inf)
        out[b] = _softmax_values(logits, _sequence(s, s["values"], b)).flatten(0, 1)
    return out


def _log_inclusion(p, K, L):
    """log P[Binomial(L, p^K) >= 2], in 64 bits."""
    x = p ** K
    lx = torch.log1p(-x)
    return torch.log(-torch.expm1(L * lx) - L * x * torch.exp((L - 1) * lx))


def _sampled_plain(s):
    n, K, L = s["n"], s["K"], s["L"]
    B, Hkv, device = s["q"].shape[0], s["keys"].shape[1], s["q"].device
    i = torch.arange(n, device=device)
    out = s["out"]
    for b in range(B):
        q = s["q"][b].float().unflatten(0, (Hkv, -1))
        # the query's sign bits against the packed planes of the keys: a table matches a key where
        # none of its K bits differ; keys that match in two tables or more are sampled
        bits = (q @ s["W"].float() > 0).to(torch.uint8) * 255
        bits = bits.view(Hkv, -1, 1, L, K, 1)
        planes = s["codes"][b].view(torch.uint8).view(Hkv, 1, -1, L, K, 128)
        differ = functools.reduce(torch.bitwise_or, [(a ^ c) for a, c in zip(planes.unbind(4),
                                                                            bits.unbind(4))])
        same = ((~differ).unsqueeze(-1) >> torch.arange(8, dtype=torch.uint8, device=device)) & 1
        count = same.sum(3, dtype=torch.int32).flatten(2)[..., :n]
        length = n if s["lengths"] is None else s["lengths"][b]
        exact = ((i < N_SINK) | (i >= length - N_LOCAL)) & (i < length)
        sampled = (count >= 2) & ~exact & (i < length)
        k = _sequence(s, s["keys"], b)
        dot = q @ k.transpose(-1, -2)
        centred = k - s["centre"][b].unsqueeze(1)
        cos = (q @ centred.transpose(-1, -2)).double() / (
            q.double().norm(dim=-1, keepdim=True) * centred.double().norm(dim=-1).unsqueeze(1))
        p = 1 - torch.arccos(cos.clamp(-1, 1)) / math.pi
        weight = torch.where(sampled, _log_inclusion(p, K, L), 0.0)
        logits = (dot / math.sqrt(D) - weight.float()).masked_fill(~(sampled | exact), -math.inf)
        out[b] = _softmax_values(logits, _sequence(s, s["values"], b)).flatten(0, 1)
    return out


def run(s):
    if own:
        import lsh_sampled_sparse_gb300 as mp
        if s["op"] == "append":
            cache = mp.PagedCache(s["keys"], s["values"])
            mp.paged_append(cache, s["table"], s["k"], s["v"], positions=s["positions"],
                            counts=s["counts"], inv_freq=s["inv_freq"],
                            interleaved=s["interleaved"], q=s["q"], q_out=s["q_out"],
                            keys_out=s["keys_out"])
            return s["q_out"], s["keys_out"], s["keys"], s["values"]
        if s["op"] == "encode":
            return mp.encode_rows_at(s["k"], s["centre"], s["W"], s["K"], s["L"], s["positions"],
                                     s["cap"], s["codes"])
        cache = mp.PagedCache(s["keys"], s["values"])
        if s["op"] == "attend":
            return mp.paged_attention(s["q"], cache, s["table"], n=s["n"], lengths=s["lengths"],
                                      out=s["out"], workspace=s["workspace"])
        return mp.paged_decode_attention(s["q"], s["codes"], s["centre"], s["W"], cache,
                                         s["table"], s["K"], s["L"], N_SINK, N_LOCAL, n=s["n"],
                                         lengths=s["lengths"], out=s["out"],
                                         workspace=s["workspace"])
    return {"append": _append_plain, "encode": _encode_plain, "attend": _attend_plain,
            "sampled": _sampled_plain}[s["op"]](s)


# ----------------------------------------------------------------------- from the definitions
def _turn64(x, start, inv_freq, interleaved):
    """One sequence's rows x [H, m, 128] in 64 bits: pairs as complex numbers times e^{i angle}."""
    r = 2 * inv_freq.numel()
    z = x.double().clone()
    for i in range(x.shape[1]):
        angle = float(start + i) * inv_freq.double()
        pair = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2),
                                                                      slice(r // 2, r))
        turned = torch.complex(z[:, i, pair[0]], z[:, i, pair[1]]) * torch.polar(
            torch.ones_like(angle), angle)
        z[:, i, pair[0]], z[:, i, pair[1]] = turned.real, turned.imag
    return z


def _exact_append(s):
    B, Hkv, m, _ = s["k"].shape
    q_out, keys_out = s["q_out"].double(), s["keys_out"].double()
    keys, values = s["keys"].double(), s["values"].double()
    page = keys.shape[2]
    for b in range(B):
        start, count = int(s["positions"][b]), m if s["counts"] is None else int(s["counts"][b])
        q_out[b, :, :count] = _turn64(s["q"][b, :, :count], start, s["inv_freq"], s["interleaved"])
        keys_out[b, :, :count] = _turn64(s["k"][b, :, :count], start, s["inv_freq"],
                                         s["interleaved"])
        where = [(int(s["table"][b, j]), j) for j in range(start // page,
                                                          (start + count - 1) // page + 1)]
        for pg, j in where:
            lo, hi = max(start, j * page), min(start + count, (j + 1) * page)
            keys[pg, :, lo - j * page:hi - j * page] = keys_out[b, :, lo - start:hi - start]
            values[pg, :, lo - j * page:hi - j * page] = s["v"][b, :, lo - start:hi - start].double()
    return q_out, keys_out, keys, values


def _exact_encode(s):
    B, Hkv, m, _ = s["k"].shape
    C = s["K"] * s["L"]
    codes = s["codes"].to(torch.int64) % 2**32
    for b in range(B):
        for i in range(m):
            p = int(s["positions"][b]) + i
            side = (s["k"][b, :, i].double() - s["centre"][b].double()) @ s["W"].double()
            word = codes[b, :, p // 1024, :, p % 1024 // 32]
            bit = 2 ** (p % 32)
            word += ((side > 0).to(torch.int64) - word // bit % 2) * bit
    return (codes - (codes >= 2**31) * 2**32).to(torch.int32).view(B, Hkv, -1, C, 32)


def exact(case, seed):
    s = prepare(case, seed)
    op, B, Hkv = case["op"], case["B"], case["Hkv"]
    if op == "append":
        return _exact_append(s)
    if op == "encode":
        return _exact_encode(s)
    Hq, n, page = case["Hq"], case["n"], case["page"]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        length = n if s["lengths"] is None else int(s["lengths"][b])
        pages = s["table"][b, :_ceil_div(length, page)].long()
        for g in range(Hkv if length else 0):
            k = s["keys"][pages, g].reshape(-1, D)[:length].double()
            v = s["values"][pages, g].reshape(-1, D)[:length].double()
            q = s["q"][b, g * G:(g + 1) * G].double()
            logits = q @ k.T / D ** 0.5
            if op == "sampled":
                K, L, mu = case["K"], case["L"], s["centre"][b, g].double()
                planes = s["codes"].view(torch.uint8)[b, g]          # [nblk, C, 128]
                bit = torch.arange(8, device=planes.device)
                keybits = ((planes.unsqueeze(-1) >> bit.to(torch.uint8)) & 1).flatten(2)
                power = 2 ** torch.arange(K, device=planes.device)
                code = (keybits.unflatten(1, (L, K)).to(torch.int16)
                        * power.to(torch.int16)[:, None]).sum(2)      # [nblk, L, 1024]
                mine = ((q @ s["W"].double() > 0).unflatten(1, (L, K)) * power).sum(2)
                i = torch.arange(length, device=planes.device)
                static = (i < N_SINK) | (i >= length - N_LOCAL)
                for h in range(G):
                    hits = (code == mine[h][None, :, None]).sum(1).flatten()[:length]
                    chosen = (hits >= 2) & ~static
                    kc = k[chosen] - mu
                    cos = (kc @ q[h]) / (kc.norm(dim=1) * q[h].norm())
                    x = (1 - torch.arccos(cos.clamp(-1, 1)) / math.pi) ** K
                    miss = torch.log1p(-x)
                    u = 1 - torch.exp(L * miss) - L * x * torch.exp((L - 1) * miss)
                    row = torch.full((length,), -math.inf, dtype=torch.float64, device=planes.device)
                    row[static] = logits[h][static]
                    row[chosen] = logits[h][chosen] - torch.log(u)
                    logits[h] = row
            w = torch.exp(logits - logits.max(1, keepdim=True).values)
            out[b, g * G:(g + 1) * G] = (w @ v) / w.sum(1, keepdim=True)
    return out
