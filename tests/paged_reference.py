"""The paged cache from its definition, in 64 bits (test infrastructure; shares no code with the
product): rows found through the page table, the rotation, attention, and the sampled estimator,
with the tolerances of a float32 evaluation."""
from __future__ import annotations

import math

import torch

E = 2.0 ** -24                                   # half a step of float32, relative


def held(pool, table, b, n):
    """(rows float64 [Hkv, n, 128], there bool [n]) of sequence b; rows without a page are zero."""
    n_pages, Hkv, page, d = pool.shape
    rows = torch.zeros(Hkv, n, d, dtype=torch.float64, device=pool.device)
    there = torch.zeros(n, dtype=torch.bool, device=pool.device)
    for j in range(-(-n // page)):
        pg = int(table[b, j])
        if 0 <= pg < n_pages:
            end = min(n, (j + 1) * page)
            rows[:, j * page:end] = pool[pg, :, :end - j * page].double()
            there[j * page:end] = True
    return rows, there


def turned(x, positions, inv_freq, interleaved):
    """x [B, H, m, 128] turned by the positions [B] + i, float64, and the tolerance of float32.

    The tolerance, of a pair (x, y): the angle is rounded to 24 bits of at most pi, sin and cos are off
    by two units of 2^-24 each way (four half steps), the product and the fused sum round once each: (pi + 4 + 2)
    half steps of |x| + |y|, 10 with the angle's reduction (2^-51 of it) at positions below 2^26."""
    B, H, m, d = x.shape
    r = 2 * inv_freq.numel()
    p = positions.double()[:, None] + torch.arange(m, device=x.device)
    a = (p[..., None] * inv_freq.double())[:, None]
    c, s = a.cos(), a.sin()
    x = x.double()
    first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2),
                                                                         slice(r // 2, r))
    out, tol = x.clone(), torch.zeros_like(x)
    out[..., first] = x[..., first] * c - x[..., second] * s
    out[..., second] = x[..., second] * c + x[..., first] * s
    size = x[..., first].abs() + x[..., second].abs()
    tol[..., first] = tol[..., second] = 10 * E * size
    return out, tol


def rounded(tol, want, dtype):
    """A tolerance with the rounding to the type that a value is stored in."""
    return tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) if dtype != torch.float32 \
        else tol + E * (want.abs() + tol)


def attention(q, keys, values, table, lengths, scale, drop=None):
    """softmax(scale q.k) . v in 64 bits, zero rows where nothing is attended to; and the tolerance
    of a float32 evaluation, per query row.

    The tolerance, with a row's A = max_i scale sum_d |q_d k_id|: a logit's 128 products, each off by a
    few E, and their sum are off by a random walk of about sqrt(128) = 11.3 roundings of up to 2 E A
    (sums that round toward zero: all of 2 E a step): 32 E A leaves a factor of 1.4; the exponential
    adds 4 E. A softmax whose logits are off by D each moves by at most 2 D max|v|. The two sums
    over n keys add a random walk of sqrt(n) roundings of 2 E, twice."""
    B, Hq, d = q.shape
    Hkv = keys.shape[1]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros(B, Hq, 1, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        k, there = held(keys, table, b, n)
        v, _ = held(values, table, b, n)
        if not there.any():
            continue
        k, v = k[:, there], v[:, there]
        qq = q[b].double().view(Hkv, G, d)
        logits = scale * (qq @ k.transpose(1, 2))
        out[b] = (torch.softmax(logits, -1) @ v).flatten(0, 1)
        A = scale * (qq.abs() @ k.abs().transpose(1, 2)).amax(-1)
        big = v.abs().flatten(1).amax(1)[:, None]
        tol[b] = (E * (2 * (32 * A + 4) + 4 * n ** 0.5 + 16) * big).view(Hq, 1)
    return out, tol


def log_u(c, K, L):
    """log P[Binomial(L, p^K) >= 2], p = 1 - arccos(c) / pi, in 64 bits."""
    if K == 0:
        return torch.zeros_like(c)
    x = ((1 - torch.arccos(c.clamp(-1, 1)) / math.pi) ** K).clamp(max=1 - 1e-16)
    l1 = torch.log1p(-x)
    r = x / (1 - x)
    # from the binomial terms where few collide, else one minus the first two of them
    term, tail = torch.ones_like(x), torch.ones_like(x)
    for j in range(2, 40):
        term = term * max(L - j, 0) / (j + 1) * r
        tail = tail + term
    few = math.log(L * (L - 1) / 2) + 2 * torch.log(x) + (L - 2) * l1 + torch.log(tail)
    many = torch.log(-torch.expm1(L * l1) - L * x * torch.exp((L - 1) * l1))
    return torch.where(L * x < 0.5, few, many)


def sampled(q, centre, keys, values, table, lengths, chosen, K, L, n_sink, n_local, scale):
    """The estimator over the keys that `chosen` (bool [B][Hq] of [n]) samples, and the tolerance: that
    of the attention, and of log u: 3e-6 for its evaluation, and what it moves by where the cosine
    moves by 32 E (sum |q k| + sum |q mu|) / (|q| |k - mu|)."""
    B, Hq, d = q.shape
    Hkv = keys.shape[1]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros(B, Hq, 1, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        k, there = held(keys, table, b, n)
        v, _ = held(values, table, b, n)
        i = torch.arange(n, device=q.device)
        T = (i < n_sink) | (i >= n - n_local)
        for h in range(Hq):
            g = h // G
            S = chosen[b][h][:n] & ~T & there
            keep = (S | T) & there
            if not keep.any():
                continue
            qq, mu = q[b, h].double(), centre[b, g].double()
            kc = k[g] - mu
            den = (qq.norm() * kc.norm(dim=1)).clamp_min(1e-300)
            cos = kc @ qq / den
            off = 32 * E * (k[g].abs() @ qq.abs() + mu.abs() @ qq.abs()) / den
            lw = torch.where(S, log_u(cos, K, L), 0.0)
            move = torch.where(S, (log_u(cos + off, K, L) - log_u(cos - off, K, L)).abs(), 0.0)
            logits = (scale * (k[g] @ qq) - lw)[keep]
            vv = v[g][keep]
            out[b, h] = torch.softmax(logits, 0) @ vv
            A = scale * (k[g][keep].abs() @ qq.abs()).max()
            D = E * (32 * A + 4) + 3e-6 + move[keep].max()
            tol[b, h] = (2 * D + E * (4 * n ** 0.5 + 16)) * vv.abs().max()
    return out, tol
