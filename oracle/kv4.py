"""The 4-bit key/value cache in exact numpy arithmetic: its format, attention on it with the
weight each row gets, and the rows an eviction keeps.

Test infrastructure, written from the definitions in include/pasa.h and sharing no code with
the CUDA library. Every rounding is done in float64, where it is exact: fp16 inputs, scales
of 8 bits and quotients that are compared with half integers.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
FP16_MAX = 65504.0


def round_bits(x, bits):
    """x to `bits` significant bits, ties to even."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.rint(m * 2.0 ** bits), e - bits)


def to_fp16(x):
    """x rounded once to fp16 (11 bits, multiples of 2^-24), overflow to infinity; as float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        y = np.where(np.abs(x) < 2.0 ** -14, np.rint(x * 2.0 ** 24) * 2.0 ** -24, round_bits(x, 11))
        return np.where(np.abs(y) > FP16_MAX, np.copysign(np.inf, x), y)


def quantise(x, shift=None):
    """(codes uint8 [..., D/2], scales fp16 [..., D/32]) of fp16 rows x [B, H, S, D]; shift fp16 [B, H, D]."""
    x = np.asarray(x, np.float64)
    if shift is not None:
        with np.errstate(invalid="ignore"):
            x = to_fp16(x - np.asarray(shift, np.float64)[:, :, None])
    x = np.where(np.isnan(x), 0.0, np.clip(x, -FP16_MAX, FP16_MAX))
    x = x.reshape(*x.shape[:-1], -1, GROUP)
    s = to_fp16(round_bits(np.abs(x).max(-1) / 7.0, 8))
    c = np.clip(np.rint(x / np.where(s > 0, s, 1.0)[..., None]), -7, 7) * (s > 0)[..., None]
    n = (c + 8).astype(np.uint8).reshape(*x.shape[:-2], -1)
    return n[..., 0::2] | (n[..., 1::2] << 4), s.astype(np.float16)


def values(codes, scales):
    """What cache rows stand for (without the shift), float64 [..., D]."""
    c = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]))
    c[..., 0::2] = (codes & 15).astype(np.float64) - 8
    c[..., 1::2] = (codes >> 4).astype(np.float64) - 8
    return c * np.repeat(np.asarray(scales, np.float64), GROUP, -1)


def decode(q, kv, vv, lengths, causal, scale, shift=None):
    """O, LSE and row weights of q [B, Hq, Sq, D] on cache values kv, vv [B, Hkv, S, D]: a dict with
    o [B, Hq, Sq, D], lse, weights [B, Hkv, S], and for error bounds pv = sum_j p_j |v_j| (like o),
    n (keys seen), vabs = sum_j |v_j| and sabs = max_j scale * sum_groups max|k_j in group| sum |q in group|
    (at least the sum of the magnitudes of a score's products)."""
    q = np.asarray(q, np.float64)
    B, Hq, Sq, D = q.shape
    H, S = kv.shape[1:3]
    g = Hq // H
    out = {"o": np.zeros(q.shape), "lse": np.full((B, Hq, Sq), -np.inf), "weights": np.zeros((B, H, S)),
           "pv": np.zeros(q.shape), "n": np.zeros((B, Hq, Sq)), "sabs": np.zeros((B, Hq, Sq)), "vabs": np.zeros(q.shape)}
    for b in range(B):
        for h in range(Hq):
            for i in range(Sq):
                n = int(np.clip(lengths[b], 0, S))
                see = min(n, i + n - Sq + 1) if causal else n
                if see <= 0:
                    continue
                k, v = kv[b, h // g, :see], vv[b, h // g, :see]
                x = scale * (k @ q[b, h, i])
                m = x.max()
                p = np.exp(x - m)
                out["lse"][b, h, i] = m + np.log(p.sum())
                p /= p.sum()
                if shift is not None:
                    out["lse"][b, h, i] += scale * float(q[b, h, i] @ np.asarray(shift[b, h // g], np.float64))
                out["o"][b, h, i] = p @ v
                out["pv"][b, h, i] = p @ np.abs(v)
                out["vabs"][b, h, i] = np.abs(v).sum(0)
                out["weights"][b, h // g, :see] += p
                out["n"][b, h, i] = see
                kg = np.abs(k).reshape(see, -1, GROUP).max(-1)
                out["sabs"][b, h, i] = scale * (kg @ np.abs(q[b, h, i]).reshape(-1, GROUP).sum(-1)).max()
    return out


def select(weights, length, budget, recent):
    """The rows one head keeps, ascending: weights fp32 [>= length]."""
    length = int(length)
    if length <= budget:
        return list(range(max(length, 0)))
    old = length - recent
    w = np.where(np.isnan(weights[:old]), -np.inf, weights[:old].astype(np.float64))
    best = sorted(range(old), key=lambda j: (-w[j], j))[:budget - recent]
    return sorted(best) + list(range(old, length))
