"""Definitions of the 4-bit row operators in 64 bits (numpy), for the tests."""

from __future__ import annotations

import numpy as np

LATENT, ROPE, VALUES, BYTES, GROUP = 512, 64, 576, 416, 16
FLAG = 1 << 30
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the non-negative finite e4m3 values, by code
E4M3 = np.array([f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
                 for e in range(16) for f in range(8)][:127])


def nearest(v, table):
    """Code of the table entry nearest to v >= 0, ties to the even code."""
    v = np.minimum(v, table[-1])
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    below, above = v - table[lo], table[hi] - v
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def bits_to_float(bits, dtype):
    """float64 of uint16 bf16 / f16 bits."""
    if dtype == "f16":
        return bits.view(np.float16).astype(np.float64)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def pack(bits, dtype):
    """uint8 [n][416] of uint16 value bits [n][576]."""
    n = bits.shape[0]
    rows = np.zeros((n, BYTES), dtype=np.uint8)
    x = bits_to_float(bits[:, :LATENT], dtype).reshape(n, -1, GROUP)
    a = np.abs(x)
    nan = np.isnan(a).any(2)
    top = np.where(nan, 0, np.where(np.isnan(a), 0, a).max(2))
    e8 = nearest(top / 6, E4M3)
    scale = E4M3[e8][:, :, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(scale > 0, nearest(np.where(np.isnan(a), 0, a) / np.where(scale > 0, scale, 1), LEVELS), 0)
    code = code | (np.signbit(x).astype(np.int64) << 3)
    code = code.reshape(n, LATENT)
    rows[:, :256] = code[:, 0::2] | (code[:, 1::2] << 4)
    rows[:, 256:288] = np.where(nan, 0x7F, e8)
    rows[:, 288:] = np.ascontiguousarray(bits[:, LATENT:]).view(np.uint8)
    return rows


def unpack(rows, dtype):
    """float64 latent [n][512], rope [n][64]."""
    n = rows.shape[0]
    code = np.empty((n, LATENT), dtype=np.int64)
    code[:, 0::2], code[:, 1::2] = rows[:, :256] & 15, rows[:, :256] >> 4
    e8 = rows[:, 256:288].astype(np.int64)
    scale = np.where((e8 & 0x7F) == 0x7F, np.nan, E4M3[np.minimum(e8 & 0x7F, 126)])
    v = np.where(code >= 8, -1.0, 1.0) * LEVELS[code & 7]
    lat = v * np.repeat(scale, GROUP, axis=1)
    rope = bits_to_float(np.ascontiguousarray(rows[:, 288:]).view(np.uint16), dtype)
    return lat, rope


def attend(q, lat, rope, scale):
    """(out [H][512], lse [H], weight [n], spread) of q [H][576] over n rows;
    spread = {"abs": sum_i p |lat|, "dot": the largest scale * sum |q||row|}."""
    H = q.shape[0]
    if lat.shape[0] == 0:
        return (np.zeros((H, LATENT)), np.full(H, -np.inf), np.zeros(0),
                {"abs": np.zeros((H, LATENT)), "dot": np.zeros(H)})
    x = np.concatenate([lat, rope], axis=1)
    s = scale * (q @ x.T)
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    total = e.sum(1, keepdims=True)
    p = e / total
    return (p @ lat, (top + np.log(total))[:, 0], p.sum(0),
            {"abs": p @ np.abs(lat), "dot": abs(scale) * (np.abs(q) @ np.abs(x).T).max(1)})


def evict(weights, slot2tok, seq, recent, want):
    """Chosen slots of one request, ascending; weights [tokens], slot2tok [D]."""
    D = slot2tok.size
    if seq <= D or want <= 0:
        return np.zeros(0, dtype=np.int64)
    tok = slot2tok.astype(np.int64)
    at = np.nonzero((tok >= 0) & (tok < min(seq - recent, weights.size)))[0]
    w = weights[tok[at]].astype(np.float64) + 0.0
    w = np.where(np.isnan(w), np.inf, w)
    last = np.isnan(weights[tok[at]])
    order = np.lexsort((at, last, w))
    return np.sort(at[order[:want]])
