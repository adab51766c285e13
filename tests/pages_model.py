"""Definitions of the resident pages' operators, for the tests: block tables with
a list, rows and attention in 64 bits (numpy)."""

from __future__ import annotations

import numpy as np

import rows4_model as M4

LATENT, ROPE, VALUES = 512, 64, 576
ROW4, ROW8, ROW16 = 416, 656, 1152
BAD_INDEX, BAD_SEQ_LEN, BAD_POSITION, BAD_RESIDENT, CAPACITY = 1, 3, 4, 5, 7
FLAG = 1 << 30
E4M3 = M4.E4M3


class Tables:
    """hisparse_page_tables on Python lists."""

    def __init__(self, tables, held, free_list, free_count, shared, bs):
        self.tables, self.held = np.array(tables, dtype=np.int64), [int(h) for h in held]
        self.list = np.array(free_list, dtype=np.int64)
        self.count = int(free_count)
        self.shared, self.bs = [int(p) for p in shared], bs
        self.status = np.zeros(len(self.held), dtype=np.int64)

    def call(self, lens, new=None, tokens=0):
        """offsets, slots, positions (with new)."""
        R, W = self.tables.shape
        S = len(self.shared)
        need, left = [], []
        for r in range(R):
            n = -(-int(lens[r]) // self.bs)
            bad = not 0 <= self.held[r] <= W
            if bad:
                self.status[r] |= 1 << BAD_INDEX
            elif lens[r] >= 0 and n > W:
                self.status[r] |= 1 << BAD_SEQ_LEN
                bad = True
            left.append(bad or lens[r] < 0)
            need.append(self.held[r] if left[r] else n)
        back = []
        for r in range(R):
            if not left[r] and need[r] < self.held[r]:
                back += [int(p) for p in self.tables[r, max(need[r], S):self.held[r]]]
                self.tables[r, need[r]:self.held[r]] = -1
                self.held[r] = need[r]
        free = [int(p) for p in self.list[:self.count]] + back[::-1]
        self.list[self.count:len(free)] = free[self.count:]
        room, want = len(free), 0
        for r in range(R):
            if left[r]:
                continue
            more = max(need[r] - S, 0) - max(self.held[r] - S, 0)
            want += max(more, 0)
            if more > 0 and want > room:
                left[r] = True
                self.status[r] |= 1 << CAPACITY
                continue
            for b in range(self.held[r], need[r]):
                self.tables[r, b] = self.shared[b] if b < S else free.pop()
            self.held[r] = need[r]
        self.count = len(free)
        if new is None:
            return None
        offsets = np.zeros(R + 1, dtype=np.int64)
        slots = np.full(tokens, -1, dtype=np.int64)
        positions = slots.copy()
        at = 0
        for r in range(R):
            offsets[r] = at
            n = int(new[r])
            if n < 0 or n > max(int(lens[r]), 0):
                self.status[r] |= 1 << BAD_POSITION
            if n > 0 and at + n > tokens:
                self.status[r] |= 1 << CAPACITY
            for i in range(max(n, 0)):
                p = int(lens[r]) - n + i
                if at + i < tokens and not left[r] and n <= lens[r]:
                    page = int(self.tables[r, p // self.bs])
                    if page >= 0 and (page + 1) * self.bs <= FLAG:
                        slots[at + i], positions[at + i] = page * self.bs + p % self.bs, p
                    elif page >= 0:
                        self.status[r] |= 1 << BAD_RESIDENT
            at += max(n, 0)
        offsets[R] = at
        return offsets, slots, positions


def norm(x, weight, eps):
    """float64 [n][512] of float64 [n][512]."""
    return x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * weight


def scale8(top):
    """The least power of two s >= 2^-126 with top <= 448 s."""
    s = np.exp2(np.clip(np.ceil(np.log2(np.maximum(top, 1e-300) / 448)), -126, 200))
    s = np.where(top > 448 * s, 2 * s, s)
    return np.where((top <= 224 * s) & (s > 2.0 ** -126), s / 2, s)


def values_of_rows(rows, dtype):
    """float64 latent [n][512], rope [n][64] of uint8 rows of any format."""
    n, row = rows.shape
    if row == ROW4:
        return M4.unpack(rows, dtype)
    rope = M4.bits_to_float(np.ascontiguousarray(rows[:, row - 128:]).view(np.uint16), dtype)
    if row == ROW16:
        return M4.bits_to_float(np.ascontiguousarray(rows[:, :1024]).view(np.uint16), dtype), rope
    scale = np.ascontiguousarray(rows[:, 512:528]).view(np.float32).astype(np.float64)
    b = rows[:, :512].astype(np.int64)
    v = np.where((b & 0x7F) == 0x7F, np.nan, E4M3[np.minimum(b & 0x7F, 126)]) * np.where(b >= 128, -1.0, 1.0)
    return v * np.repeat(scale, 128, axis=1), rope


def attend_prefix(q, lat, rope, scale, part=None, part_lse=None):
    """(out [M][512], lse [M], spread) of q [M][576] over rows and a part."""
    M = q.shape[0]
    x = np.concatenate([lat, rope], axis=1)
    s = scale * (q @ x.T)
    both = s if part is None else np.concatenate([s, part_lse[:, None]], axis=1)
    if both.shape[1] == 0:
        return np.zeros((M, LATENT)), np.full(M, -np.inf), {"abs": np.zeros((M, LATENT)), "dot": np.zeros(M)}
    top = both.max(1, keepdims=True)
    base = np.where(np.isfinite(top), top, 0)
    e = np.exp(both - base)
    total = e.sum(1, keepdims=True)
    p = e / np.where(total == 0, 1, total)
    n = s.shape[1]
    out, spread = p[:, :n] @ lat, p[:, :n] @ np.abs(lat)
    if part is not None:
        w = np.where(part_lse[:, None] == -np.inf, 0, part)
        out, spread = out + p[:, n:] * w, spread + p[:, n:] * np.abs(w)
    dot = abs(scale) * (np.abs(q) @ np.abs(x).T).max(1) if n else np.zeros(M)
    with np.errstate(divide="ignore"):
        return out, (base + np.log(total))[:, 0], {"abs": spread, "dot": dot}
