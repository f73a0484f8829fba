"""Measured cases of the 4-bit K/V cache: writing rows and reading them back, reading rows,
attention of single tokens over the cache, and the LSH-sampled decode over it.

A cache row (one token of one KV head, 128 dims) holds, for the key minus the head's centre and
for the value, 4-bit codes in two groups of 64 dims: with z the largest bf16 not above the group's
minimum and s the smallest bf16 with z + 15 s not below its maximum, c = rint((x - z) / s) and
x ~ z + s c. Tensors: k_codes and v_codes uint8 [B, Hkv, capacity, 64] (dim 2 i in the low half of
byte i), params bf16 [B, Hkv, capacity, 8] = s, z of key group 0, key group 1, value group 0,
value group 1.
"""
import functools
import math

import torch

own = False

D = 128
GROUP = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 32 sequences of different lengths: a token each is appended
        dict(name="append_b32", op="store", dtype="bf16", B=32, Hkv=8, m=1, cap=2048, ragged=True),
        # a chunk of odd length of an fp32 model with few heads
        dict(name="store_f32_odd", op="store", dtype="f32", B=3, Hkv=5, m=777, cap=1801,
             ragged=True),
        # the prompt of the 96K-token workload, one layer, stored and read back for its attention
        dict(name="store_96k", op="store", dtype="bf16", B=1, Hkv=8, m=98304, cap=98304,
             ragged=False),
        # a stretch of a 16K-token cache of four sequences read back as bf16
        dict(name="read_b4_16k", op="read", dtype="bf16", B=4, Hkv=8, m=16384, cap=16384,
             ragged=False),
        # an odd stretch read back in fp32 from places of each sequence's own
        dict(name="read_f32_odd", op="read", dtype="f32", B=3, Hkv=4, m=1333, cap=5001,
             ragged=True),
        # a short context, one sequence: latency
        dict(name="attend_b1_512", op="attend", dtype="bf16", B=1, Hq=32, Hkv=8, n=512, cap=512,
             ragged=False),
        # one query head per KV head, fp32 queries, sequences of different odd lengths
        dict(name="attend_mha_ragged", op="attend", dtype="f32", B=7, Hq=12, Hkv=12, n=3001,
             cap=3333, ragged=True),
        # the 96K-token workload, one layer
        dict(name="attend_b1_96k", op="attend", dtype="bf16", B=1, Hq=32, Hkv=8, n=98304,
             cap=98304, ragged=False),
        # the 70B-shaped workload: eight query heads per KV head, 128K tokens, two sequences
        dict(name="attend_b2_128k_g8", op="attend", dtype="bf16", B=2, Hq=64, Hkv=8, n=131072,
             cap=131072, ragged=False),
        # large-batch decode, 32 sequences of up to 32K tokens
        dict(name="attend_b32_32k", op="attend", dtype="bf16", B=32, Hq=32, Hkv=8, n=32768,
             cap=32768, ragged=True),
        # sampled decode of four 16K-token sequences
        dict(name="sampled_b4_16k", op="sampled", dtype="bf16", B=4, Hq=32, Hkv=8, n=16384,
             cap=16384, K=10, L=150),
        # sampled decode of the 96K-token workload, one layer
        dict(name="sampled_b1_96k", op="sampled", dtype="bf16", B=1, Hq=32, Hkv=8, n=98304,
             cap=98304, K=10, L=150),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "read", "attend", "attend", "sampled"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("store", "read"):
        B, Hkv = _log_int(rng, 1, 32), rng.randint(1, 12)
        most = max(1, 700_000 // (B * Hkv) // (2 if dtype == "f32" else 1))
        m = _log_int(rng, 1, min(most, 98304))
        return dict(op=op, dtype=dtype, B=B, Hkv=Hkv, m=m, cap=m + rng.randint(0, 999),
                    ragged=rng.random() < 0.5)
    if op == "attend":
        B, Hkv = _log_int(rng, 1, 32), rng.randint(1, 12)
        G = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8])
        n = _log_int(rng, 1, min(131072, 6_000_000 // (B * Hkv)))
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, n=n, cap=n + rng.randint(0, 999),
                    ragged=rng.random() < 0.5)
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    K, L = rng.randint(6, 12), rng.randint(40, 200)
    B = rng.randint(1, 4)
    most = 4_400_000_000 // (B * Hkv * G * K * L)
    n = _log_int(rng, 500, max(600, min(98304, most)))
    return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, n=n, cap=n + rng.randint(0, 999),
                K=K, L=L)


# Share of the keys that a KV head's query heads sample together on these inputs: what the pages
# quote for (K, L) = (10, 150), four query heads a KV head, is about 1.6% each.
SAMPLED_SHARE = 0.0157
N_SINK, N_LOCAL = 4, 64
ROW_BYTES = 2 * (D // 2) + 16


def work(case):
    B, Hkv = case["B"], case["Hkv"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("store", "read"):
        rows = B * Hkv * case["m"]
        wide = 2 * D * size
        centre = B * Hkv * D * 4
        if case["op"] == "store":
            return {"bytes": rows * (wide + ROW_BYTES + wide) + centre, "flops": rows * 2 * D * 8}
        return {"bytes": rows * (ROW_BYTES + wide) + centre, "flops": rows * 2 * D * 3}
    Hq, n = case["Hq"], case["n"]
    ends = B * Hq * D * (size + 4)
    if case["op"] == "attend":
        # sequences of different lengths are between half of n and n
        tokens = B * n * (0.75 if case["ragged"] else 1.0)
        return {"bytes": tokens * Hkv * ROW_BYTES + ends, "flops": tokens * Hq * 4 * D}
    C = case["K"] * case["L"]
    per_head = n * SAMPLED_SHARE
    exact = min(n, N_SINK + N_LOCAL)
    rows = B * Hkv * min(n, Hq // Hkv * per_head + exact)
    return {"bytes": B * Hkv * n * C / 8 + rows * ROW_BYTES + ends + D * C * 2 + B * Hkv * D * 4,
            "flops": B * Hq * ((per_head + exact) * 6 * D + 2 * D * C)}


# ------------------------------------------------------------------------- the format, plainly
def _bf16_below(x):
    """The largest bf16 that is not above x (float32)."""
    r = x.to(torch.bfloat16)
    bits = r.view(torch.int16)
    down = torch.where(r == 0, torch.full_like(bits, -32767), torch.where(r > 0, bits - 1, bits + 1))
    return torch.where(r.float() > x, down.view(torch.bfloat16), r)


def _bf16_above(x):
    """The smallest bf16 that is not below x (float64, not negative)."""
    r = x.float().to(torch.bfloat16)
    return torch.where(r.double() < x, (r.view(torch.int16) + 1).view(torch.bfloat16), r)


def _quantise(x):
    """x float32 [..., 128] -> codes uint8 [..., 64], params bf16 [..., 4] = s, z of both groups."""
    g = x.unflatten(-1, (D // GROUP, GROUP))
    z = _bf16_below(g.amin(-1))
    s = _bf16_above((g.amax(-1).double() - z.double()) / 15)
    s64, z64 = s.double().unsqueeze(-1), z.double().unsqueeze(-1)
    c = torch.where(s64 > 0, torch.round((g.double() - z64) / s64), 0.0)
    c = c.to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([s, z], -1).flatten(-2)


def _values(codes, params):
    """float32 [..., 128] of codes [..., 64] and params [..., 4] = s, z of both groups."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (D // GROUP, GROUP))
    p = params.double().unflatten(-1, (D // GROUP, 2)).unsqueeze(-2)
    return (p[..., 1] + p[..., 0] * c).float().flatten(-2)


# ------------------------------------------------------------------------------------- inputs
def _cache_of(case, keys_of, values_of, device):
    """A cache whose first n rows of each head hold the given rows (a function per sequence);
    the rest of the capacity is zero."""
    B, Hkv, cap = case["B"], case["Hkv"], case["cap"]
    k_codes = torch.zeros(B, Hkv, cap, D // 2, dtype=torch.uint8, device=device)
    v_codes = torch.zeros_like(k_codes)
    params = torch.zeros(B, Hkv, cap, 8, dtype=torch.bfloat16, device=device)
    for b in range(B):
        for codes, at, rows in ((k_codes, 0, keys_of(b)), (v_codes, 4, values_of(b))):
            n = rows.shape[-2]
            codes[b, :, :n], params[b, :, :n, at:at + 4] = _quantise(rows)
    return k_codes, v_codes, params


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
    op, dtype, B, Hkv, cap = case["op"], DTYPES[case["dtype"]], case["B"], case["Hkv"], case["cap"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    s = dict(op=op)
    if op in ("store", "read"):
        m = case["m"]
        s["m"], s["dtype"] = m, dtype
        s["centre"] = 8 * torch.nn.functional.normalize(randn(B, Hkv, D), dim=-1)
        s["positions"] = (torch.randint(0, cap - m + 1, (B,), generator=gen, device=device)
                          .to(torch.int32) if case["ragged"] else None)
        if op == "store":
            s["keys"] = (randn(B, Hkv, m, D) + s["centre"].unsqueeze(2)).to(dtype)
            s["values"] = randn(B, Hkv, m, D).to(dtype)
            s["cache"] = _cache_of(case, lambda b: torch.zeros(Hkv, 0, D, device=device),
                                   lambda b: torch.zeros(Hkv, 0, D, device=device), device)
        else:
            s["cache"] = _cache_of(case, lambda b: randn(Hkv, cap, D),
                                   lambda b: randn(Hkv, cap, D), device)
        return s
    Hq, n = case["Hq"], case["n"]
    centre, q = _geometry(B, Hkv, Hq, gen, device)
    s["n"], s["q"] = n, q.to(dtype)
    lengths = None
    if op == "attend" and case["ragged"]:
        lengths = torch.randint(n // 2, n + 1, (B,), generator=gen, device=device)
    # what a key is minus the centre: noise, and the first token twelve deviations along the
    # mean query of its head (the attention sink)
    sink = 12 * torch.nn.functional.normalize(q.unflatten(1, (Hkv, Hq // Hkv)).mean(2), dim=-1)
    keep = {}

    def keys_of(b):
        k = randn(Hkv, n, D)
        k[:, 0] = sink[b]
        keep[b] = k
        return k

    s["cache"] = _cache_of(case, keys_of, lambda b: randn(Hkv, n, D), device)
    s["out"] = torch.empty(B, Hq, D, dtype=torch.float32, device=device)
    if op == "attend":
        s["lengths"] = None if lengths is None else lengths.to(torch.int32)
        s["scale"] = 1 / math.sqrt(D)
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=device)
        return s
    K, L = case["K"], case["L"]
    C, nblk = K * L, -(-cap // 1024)
    s["K"], s["L"], s["centre"] = K, L, centre
    s["W"] = ((randn(D, C) * 16).round() / 16).to(dtype)
    codes = torch.zeros(B, Hkv, nblk, C, 128, dtype=torch.uint8, device=device)
    for b in range(B):
        for g in range(Hkv):
            bits = torch.zeros(nblk * 1024, C, dtype=torch.bool, device=device)
            bits[:n] = keep[b][g] @ s["W"].float() > 0
            bits = bits.view(nblk, 128, 8, C).to(torch.uint8)
            bits <<= torch.arange(8, dtype=torch.uint8, device=device)[:, None]
            codes[b, g] = bits.sum(2, dtype=torch.uint8).transpose(1, 2)
    s["codes"] = codes.view(torch.int32)
    s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device=device)
    return s


# -------------------------------------------------------------------------------- plain forms
def _rows(s, t):
    """The stored rows [B, Hkv, m, ...] of a cache tensor, and where they are."""
    B, m = t.shape[0], s["m"]
    b = torch.arange(B, device=t.device)[:, None]
    start = torch.zeros(B, 1, dtype=torch.int64, device=t.device)
    at = (start if s["positions"] is None else s["positions"][:, None]) + torch.arange(
        m, device=t.device)
    return b, at


def _read_plain(s):
    k_codes, v_codes, params = s["cache"]
    b, at = _rows(s, params)
    p = params[b, :, at].transpose(1, 2)
    k = _values(k_codes[b, :, at].transpose(1, 2), p[..., :4]) + s["centre"].unsqueeze(2)
    return k.to(s["dtype"]), _values(v_codes[b, :, at].transpose(1, 2), p[..., 4:]).to(s["dtype"])


def _store_plain(s):
    k_codes, v_codes, params = s["cache"]
    b, at = _rows(s, params)
    kc, kp = _quantise(s["keys"].float() - s["centre"].unsqueeze(2))
    vc, vp = _quantise(s["values"].float())
    k_codes[b, :, at] = kc.transpose(1, 2)
    v_codes[b, :, at] = vc.transpose(1, 2)
    params[b, :, at] = torch.cat([kp, vp], -1).transpose(1, 2)
    return _read_plain(s)


def _softmax_values(logits, v):
    w = torch.exp(logits - logits.amax(-1, keepdim=True).clamp_min(-3e38))
    total = w.sum(-1, keepdim=True)
    return torch.where(total > 0, (w @ v) / total.clamp_min(1e-300 if v.dtype == torch.float64
                                                            else 1e-37), 0.0)


def _attend_plain(s):
    k_codes, v_codes, params = (t[:, :, :s["n"]] for t in s["cache"])
    B, Hkv = params.shape[:2]
    q = s["q"].float().unflatten(1, (Hkv, -1))
    logits = q @ _values(k_codes, params[..., :4]).transpose(-1, -2) * s["scale"]
    if s["lengths"] is not None:
        i = torch.arange(s["n"], device=q.device)
        logits = logits.masked_fill(i >= s["lengths"].view(B, 1, 1, 1), -math.inf)
    return _softmax_values(logits, _values(v_codes, params[..., 4:])).flatten(1, 2)


def _log_inclusion(p, K, L):
    """log P[Binomial(L, p^K) >= 2], in 64 bits."""
    x = p ** K
    lx = torch.log1p(-x)
    return torch.log(-torch.expm1(L * lx) - L * x * torch.exp((L - 1) * lx))


def _sampled_plain(s):
    n, K, L = s["n"], s["K"], s["L"]
    k_codes, v_codes, params = (t[:, :, :n] for t in s["cache"])
    B, Hkv = params.shape[:2]
    device = params.device
    q = s["q"].float().unflatten(1, (Hkv, -1))
    # the query's sign bits against the packed planes of the keys: a table matches a key where
    # none of its K bits differ; keys that match in two tables or more are sampled
    bits = (q @ s["W"].float() > 0).to(torch.uint8) * 255
    bits = bits.view(B, Hkv, -1, 1, L, K, 1)
    planes = s["codes"].view(torch.uint8).view(B, Hkv, 1, -1, L, K, 128)
    differ = functools.reduce(torch.bitwise_or, [(a ^ c) for a, c in zip(planes.unbind(5),
                                                                        bits.unbind(5))])
    same = ((~differ).unsqueeze(-1) >> torch.arange(8, dtype=torch.uint8, device=device)) & 1
    count = same.sum(4, dtype=torch.int32).flatten(3)[..., :n]
    i = torch.arange(n, device=device)
    exact = (i < N_SINK) | (i >= n - N_LOCAL)
    sampled = (count >= 2) & ~exact
    k = _values(k_codes, params[..., :4])
    dot = q @ k.transpose(-1, -2)
    cos = dot.double() / (q.double().norm(dim=-1, keepdim=True)
                          * k.double().norm(dim=-1).unsqueeze(2))
    p = 1 - torch.arccos(cos.clamp(-1, 1)) / math.pi
    weight = torch.where(sampled, _log_inclusion(p, K, L), 0.0)
    logits = dot / math.sqrt(D) - weight.float()
    logits = logits.masked_fill(~(sampled | exact), -math.inf)
    return _softmax_values(logits, _values(v_codes, params[..., 4:])).flatten(1, 2)


def run(s):
    if own:
        import lsh_sampled_sparse_gb300 as mp
        cache = mp.KV4Cache(*s["cache"])
        if s["op"] == "store":
            mp.kv4_write(cache, s["keys"], s["values"], centre=s["centre"],
                         positions=s["positions"])
        if s["op"] in ("store", "read"):
            return mp.kv4_read(cache, s["m"], centre=s["centre"], positions=s["positions"],
                               dtype=s["dtype"])
        if s["op"] == "attend":
            return mp.kv4_attention(s["q"], cache, n=s["n"], lengths=s["lengths"],
                                    scale=s["scale"], out=s["out"], workspace=s["workspace"])
        return mp.kv4_decode_attention(s["q"], s["codes"], s["centre"], s["W"], cache, s["K"],
                                       s["L"], N_SINK, N_LOCAL, n=s["n"], out=s["out"],
                                       workspace=s["workspace"])
    return {"store": _store_plain, "read": _read_plain, "attend": _attend_plain,
            "sampled": _sampled_plain}[s["op"]](s)


# ----------------------------------------------------------------------- from the definitions
def _dequantised64(codes, params):
    """[n, 128] float64 of one head's rows: code by code, from the definition."""
    out = torch.empty(codes.shape[0], D, dtype=torch.float64, device=codes.device)
    for e0 in (0, 1):
        nibble = (codes.to(torch.int32) >> (4 * e0)) % 16
        for g in range(D // GROUP):
            part = slice(g * GROUP // 2, (g + 1) * GROUP // 2)
            out[:, g * GROUP + e0:(g + 1) * GROUP:2] = (
                params[:, 2 * g + 1, None].double()
                + params[:, 2 * g, None].double() * nibble[:, part].double())
    return out


def _stored64(x):
    """What rows x [n, 128] (float32) are stored as, in 64 bits: bf16 steps are tried one by one
    against the two conditions that define them."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    inf = torch.full((), math.inf, dtype=torch.bfloat16, device=x.device)
    for g in range(D // GROUP):
        v = x[:, g * GROUP:(g + 1) * GROUP].double()
        lo, hi = v.min(1).values, v.max(1).values
        z = lo.to(torch.bfloat16)
        for _ in range(2):
            z = torch.where(z.double() > lo, torch.nextafter(z, -inf), z)
        step = ((hi - z.double()) / 15).to(torch.bfloat16)
        for _ in range(2):
            lower = torch.nextafter(step, -inf)
            step = torch.where((lower >= 0) & (z.double() + 15 * lower.double() >= hi), lower, step)
        for _ in range(3):
            step = torch.where(z.double() + 15 * step.double() < hi, torch.nextafter(step, inf),
                               step)
        z64, s64 = z.double()[:, None], step.double()[:, None]
        code = torch.where(s64 > 0, ((v - z64) / s64).round(), 0.0)
        out[:, g * GROUP:(g + 1) * GROUP] = z64 + s64 * code
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, B, Hkv = case["op"], case["B"], case["Hkv"]
    k_codes, v_codes, params = s["cache"]
    if op in ("store", "read"):
        m = case["m"]
        k = torch.empty(B, Hkv, m, D, dtype=torch.float64, device=params.device)
        v = torch.empty_like(k)
        for b in range(B):
            p = 0 if s["positions"] is None else int(s["positions"][b])
            for g in range(Hkv):
                mu = s["centre"][b, g]
                if op == "store":
                    k[b, g] = _stored64(s["keys"][b, g].float() - mu) + mu.double()
                    v[b, g] = _stored64(s["values"][b, g].float())
                else:
                    at = (b, g, slice(p, p + m))
                    k[b, g] = _dequantised64(k_codes[at], params[at][:, :4]) + mu.double()
                    v[b, g] = _dequantised64(v_codes[at], params[at][:, 4:])
        return k, v
    Hq, n = case["Hq"], case["n"]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=params.device)
    for b in range(B):
        length = n
        if op == "attend" and s["lengths"] is not None:
            length = int(s["lengths"][b])
        for g in range(Hkv):
            if length == 0:
                continue
            at = (b, g, slice(0, length))
            k = _dequantised64(k_codes[at], params[at][:, :4])
            v = _dequantised64(v_codes[at], params[at][:, 4:])
            q = s["q"][b, g * G:(g + 1) * G].double()
            logits = q @ k.T / D ** 0.5
            if op == "sampled":
                K, L = case["K"], case["L"]
                planes = s["codes"].view(torch.uint8)[b, g]          # [nblk, C, 128]
                bit = torch.arange(8, device=planes.device)
                keybits = ((planes.unsqueeze(-1) >> bit.to(torch.uint8)) & 1).flatten(2)
                power = 2 ** torch.arange(K, device=planes.device)
                code = (keybits.unflatten(1, (L, K)).to(torch.int16)
                        * power.to(torch.int16)[:, None]).sum(2)      # [nblk, L, 1024]
                mine = ((q @ s["W"].double() > 0).unflatten(1, (L, K)) * power).sum(2)
                i = torch.arange(n, device=planes.device)
                static = (i < N_SINK) | (i >= n - N_LOCAL)
                for h in range(G):
                    hits = (code == mine[h][None, :, None]).sum(1).flatten()[:n]
                    chosen = (hits >= 2) & ~static
                    cos = (k[chosen] @ q[h]) / (k[chosen].norm(dim=1) * q[h].norm())
                    x = (1 - torch.arccos(cos.clamp(-1, 1)) / math.pi) ** K
                    miss = torch.log1p(-x)
                    u = 1 - torch.exp(L * miss) - L * x * torch.exp((L - 1) * miss)
                    row = torch.full((n,), -math.inf, dtype=torch.float64, device=planes.device)
                    row[static] = logits[h][static]
                    row[chosen] = logits[h][chosen] - torch.log(u)
                    logits[h] = row
            w = torch.exp(logits - logits.max(1, keepdim=True).values)
            out[b, g * G:(g + 1) * G] = (w @ v) / w.sum(1, keepdim=True)
    return out
