"""The 4-bit K/V cache from its definition, in 64 bits (test infrastructure; shares no code with
the product). A group of 64 dims x is held by z, the largest bf16 <= min x, s, the smallest bf16
with z + 15 s >= max x, and codes rint((x - z) / s), ties to even; the value is z + s code. A group
without finite s and z is NaN throughout."""
from __future__ import annotations

import numpy as np
import torch

GROUP = 64


def bf16_values(bits: np.ndarray) -> np.ndarray:
    """float64 of bf16 bit patterns (uint16)."""
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


# every bf16 that is not NaN, ascending, with both infinities: a search table
_BITS = np.concatenate([np.arange(0xFF80, 0x7FFF, -1, dtype=np.int64),
                        np.arange(0x0000, 0x7F81, dtype=np.int64)]).astype(np.uint16)
_VALUES = bf16_values(_BITS)


def quantise(x) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """x float32 [..., 128] -> codes [..., 128] (0..15), s and z bf16 bits [..., 2] (uint16); the
    bits of a group that is held as NaN are 0x7fc0."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    finite = np.isfinite(g).all(-1)
    safe = np.where(finite[..., None], g, 0.0)
    lo, hi = safe.min(-1), safe.max(-1)
    zi = np.searchsorted(_VALUES, lo, side="right") - 1            # largest value <= lo
    z = _VALUES[zi]
    need = np.where(np.isfinite(z), hi - np.where(np.isfinite(z), z, 0.0), np.inf)
    # 15 s is exact in float64; the smallest s with 15 s >= need
    si = np.searchsorted(15.0 * _VALUES[_VALUES >= 0][1:], need, side="left")
    pos_bits = _BITS[_VALUES >= 0][1:]                             # +0 first (after -0)
    pos = _VALUES[_VALUES >= 0][1:]
    s = pos[np.minimum(si, len(pos) - 1)]
    # a difference past the largest float32 has no finite step in float32 arithmetic
    ok = finite & np.isfinite(z) & np.isfinite(s) & (need <= np.finfo(np.float32).max)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] > 0, np.rint((safe - z[..., None]) / s[..., None]), 0.0)
    c = np.where(ok[..., None], c, 0.0).astype(np.int64)
    zb = np.where(ok, _BITS[zi], 0x7FC0).astype(np.uint16)
    sb = np.where(ok, pos_bits[np.minimum(si, len(pos) - 1)], 0x7FC0).astype(np.uint16)
    return c.reshape(x.shape), sb, zb


def pack(c: np.ndarray) -> np.ndarray:
    """codes [..., 128] -> bytes [..., 64]."""
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def params(ks, kz, vs, vz) -> np.ndarray:
    """bf16 bits [..., 8] of a row."""
    return np.concatenate([np.stack([ks, kz], -1).reshape(*ks.shape[:-1], -1),
                           np.stack([vs, vz], -1).reshape(*vs.shape[:-1], -1)], -1)


def values64(codes: torch.Tensor, prm: torch.Tensor, value: int) -> torch.Tensor:
    """float64 [..., 128] that a cache's rows hold: value 0 the (centred) keys, 1 the values."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    p = prm.double()[..., 4 * value:4 * value + 4]
    s = p[..., 0::2].repeat_interleave(GROUP, -1)
    z = p[..., 1::2].repeat_interleave(GROUP, -1)
    return z + s * c


def attention64(q, cache, lengths, scale):
    """softmax(scale q.k) . v in 64 bits, zero rows for length 0; and the tolerance of a float32
    evaluation, per query row.

    The tolerance, with e = 2^-24 and a row's A = max_i scale sum_d |q_d k_id|: a logit's 128
    products, each off by a few e, and their sum are off by a random walk of about sqrt(128) = 11.3
    roundings of up to 2 e A: 32 e A leaves a factor of 1.4; the exponential adds 4 e. A softmax
    whose logits are off by D each moves by at most 2 D max|v|. The two sums over n keys add a
    random walk of sqrt(n) roundings of 2 e, twice."""
    k, v = values64(cache[0], cache[2], 0), values64(cache[1], cache[2], 1)
    B, Hq, d = q.shape
    Hkv, cap = k.shape[1:3]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros(B, Hq, 1, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        for h in range(Hq):
            kk, vv, qq = k[b, h // G, :n], v[b, h // G, :n], q[b, h].double()
            out[b, h] = torch.softmax(scale * (kk @ qq), 0) @ vv
            A = scale * (kk.abs() @ qq.abs()).max()
            tol[b, h] = (2.0 ** -24 * (2 * (32 * A + 4) + 4 * n ** 0.5 + 16)) * vv.abs().max()
    return out, tol
