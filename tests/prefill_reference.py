"""Norms, rotation, 4-bit rows and prompt attention in 64 bits: plain
restatements of the definitions in include/gbtopk.h for the tests, float64
arrays and nothing of the package."""
import math

import numpy as np


def turned(x, positions, freqs, interleaved, weight, eps):
    """[rows, heads, dim] normalised and rotated, and the sum of the magnitudes
    that each element is a sum of."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    y, mag = x.copy(), np.abs(x)
    n = 0 if freqs is None else len(freqs)
    if n:
        angle = positions.astype(np.float64)[:, None] * freqs.astype(np.float64)
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        at = np.arange(n)
        i, j = (2 * at, 2 * at + 1) if interleaved else (at, at + n)
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
        mag[..., i] = mag[..., j] = np.abs(a) + np.abs(b)
    return y, mag


def areas(dim):
    return 16 * -(-dim // 32), 8 if dim <= 128 else 16


SCALES = np.array([b / 512 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 10) for b in range(128)])


def codes(x, unit=1.0):
    """Scale bytes [..., dim/16] and codes [..., dim/16, 16] of [..., dim]."""
    x = x.astype(np.float64).reshape(x.shape[:-1] + (-1, 16)) / unit
    top = np.where(np.isnan(x), 0, np.abs(x)).max(-1) / 7
    top = np.minimum(top, 448)
    # the nearest of the scales, ties to the even byte
    at = np.searchsorted(SCALES[:127], top, side="right").clip(1, 126)
    low, high = SCALES[at - 1], SCALES[at]
    up = (top - low > high - top) | ((top - low == high - top) & (at % 2 == 0))
    byte = np.where(up, at, at - 1)
    s = SCALES[byte][..., None]
    with np.errstate(all="ignore"):
        c = np.where(s > 0, np.rint(x / s), 0)
    c = np.where(np.isnan(c), 0, c).clip(-7, 7)
    return byte, c.astype(np.int64)


def row_bytes(byte_k, code_k, byte_v, code_v):
    """The bytes of rows."""
    dim = byte_k.shape[-1] * 16
    c, s = areas(dim)
    out = np.zeros(byte_k.shape[:-1] + (2 * c + 2 * s,), dtype=np.uint8)
    for part, (byte, code) in enumerate(((byte_k, code_k), (byte_v, code_v))):
        code = code.reshape(code.shape[:-2] + (dim // 8, 8))
        word = np.zeros(code.shape[:-1], dtype=np.uint64)
        for e in range(8):
            j, odd = divmod(e, 2)
            mag, sign = np.abs(code[..., e]).astype(np.uint64), (code[..., e] < 0).astype(np.uint64)
            word |= mag << np.uint64(4 * j + 16 * odd) | sign << np.uint64((4 * j + 15 + 16 * odd) % 32)
        for b in range(4):
            out[..., part * c + b:part * c + dim // 2:4] = (word >> np.uint64(8 * b)) & np.uint64(255)
        out[..., 2 * c + part * s:2 * c + part * s + dim // 16] = byte
    return out


def values(rows, dim):
    """Keys and values [..., dim] that rows of any bytes stand for."""
    c, s = areas(dim)
    got = []
    for part in range(2):
        raw = rows[..., part * c:part * c + dim // 2].astype(np.uint64).reshape(rows.shape[:-1] + (dim // 8, 4))
        word = sum(raw[..., b] << np.uint64(8 * b) for b in range(4))
        x = np.zeros(word.shape + (8,))
        for e in range(8):
            j, odd = divmod(e, 2)
            mag = (word >> np.uint64(4 * j + 16 * odd)) & np.uint64(7)
            sign = (word >> np.uint64((4 * j + 15 + 16 * odd) % 32)) & np.uint64(1)
            x[..., e] = np.where(sign == 1, -1.0, 1.0) * mag
        scale = SCALES[rows[..., 2 * c + part * s:2 * c + part * s + dim // 16] & 127]
        got.append((x.reshape(scale.shape + (16,)) * scale[..., None]).reshape(rows.shape[:-1] + (dim,)))
    return got


def attend(q, k, v, group, scale):
    """As decode_reference.attend, over [n, kv_heads, dim] arrays, all seen."""
    heads, dim = q.shape
    out, mag = np.zeros((heads, dim)), np.zeros((heads, dim))
    lse, eta = np.full(heads, -math.inf), np.zeros(heads)
    if k.shape[0] == 0:
        return out, lse, eta, mag
    for h in range(heads):
        kk, vv = k[:, h // group], v[:, h // group]
        s = scale * (kk @ q[h])
        top = s.max()
        lse[h] = top + math.log(np.exp(s - top).sum())
        p = np.exp(s - lse[h])
        out[h], mag[h] = p @ vv, p @ np.abs(vv)
        eta[h] = (dim + 8) * 2.0 ** -23 * (scale * (np.abs(kk) @ np.abs(q[h]))).max() + 2.0 ** -20
    return out, lse, eta, mag
