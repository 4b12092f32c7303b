"""Plain 64-bit reference of the paged key/value cache and its attention (numpy), written from the
formulas: one token, one element, one key at a time where it matters, no tiling, no online softmax.
"""
from __future__ import annotations

import numpy as np

BLOCK = 64


def quantise(x):
    """fp rows [..., D] -> (codes int8, scales fp32). a = max|x|, scale = a / 127 in fp32,
    code = rint(127 x / a); a row with an infinity or NaN: scale NaN, codes 0."""
    x = np.asarray(x, np.float64)
    a = np.abs(x).max(axis=-1)
    finite = np.isfinite(x).all(axis=-1)
    live = finite & (a > 0)
    div = np.where(live, a, 1.0)[..., None]
    code = np.where(live[..., None], np.rint(127.0 * np.where(finite[..., None], x, 0.0) / div), 0.0)
    with np.errstate(invalid="ignore"):
        scale = np.where(finite, a.astype(np.float32) / np.float32(127.0), np.float32(np.nan)).astype(np.float32)
    return code.astype(np.int8), scale


def element_place(D, which, j, d):
    """(byte inside a plane, nibble) of element (slot j, dim d); which: "k" or "v"."""
    if which == "k":
        g, n = 2 * (j // 16) + j % 2, (d % 8) // 2 + 4 * (d % 2)
        byte = (16 * (32 * ((D // 64) * ((j // 4) % 4) + d // 64) + 4 * g + (d % 64) // 16)
                + 8 * ((j // 2) % 2) + 4 * ((d % 16) // 8) + n // 2)
        return byte, n % 2
    byte = 16 * (32 * (d // 16) + 4 * (d % 8) + j // 16) + 4 * ((j // 4) % 4) + (j % 4) // 2 + 2 * (j % 2)
    return byte, (d // 8) % 2


_places = {}


def places(D, which):
    """element_place as arrays [64, D]; every (byte, nibble) pair is used once."""
    if (D, which) not in _places:
        pl = np.array([[element_place(D, which, j, d) for d in range(D)] for j in range(BLOCK)])
        assert len({(int(b), int(n)) for b, n in pl.reshape(-1, 2)}) == BLOCK * D
        _places[D, which] = pl[..., 0], pl[..., 1]
    return _places[D, which]


def record_bytes(D):
    return 512 + 128 * D


def write_token(record, D, j, kc, ks, vc, vs):
    """Slot j of one head's record (uint8 [record_bytes]) in place."""
    record[4 * j:4 * j + 4] = np.frombuffer(np.float32(ks).tobytes(), np.uint8)
    record[256 + 4 * j:260 + 4 * j] = np.frombuffer(np.float32(vs).tobytes(), np.uint8)
    for which, code, hi0, lo0 in (("k", kc, 512, 512 + 64 * D), ("v", vc, 512 + 32 * D, 512 + 96 * D)):
        byte, nib = (p[j] for p in places(D, which))
        u = code.astype(np.int16) + 128
        for base, val in ((hi0, u >> 4), (lo0, u & 15)):
            for d in range(D):
                at, s = base + byte[d], 4 * nib[d]
                record[at] = (int(record[at]) & (0xF0 >> s)) | (int(val[d]) << s)


def read_record(record, D, level):
    """(k, v) float64 [64, D] of a head's record at a level (0, 1-2, 3+), and their scales."""
    sc = record[:512].view(np.float32).reshape(2, BLOCK)
    out = []
    for which, hi0, lo0, s in (("k", 512, 512 + 64 * D, sc[0]), ("v", 512 + 32 * D, 512 + 96 * D, sc[1])):
        byte, nib = places(D, which)
        h = (record[hi0 + byte].astype(np.int64) >> (4 * nib)) & 15
        l = (record[lo0 + byte].astype(np.int64) >> (4 * nib)) & 15
        w = (16 * h + l - 128).astype(np.float64) if level >= 3 else 16.0 * (h - 8) + 7.5
        out.append(np.zeros((BLOCK, D)) if level == 0 else s.astype(np.float64)[:, None] * w)
    return out[0], out[1], sc


def gather(pages, table_row, levels_row, length, D, head):
    """(k, v [length, D], level of each token, scales [2, length]) of one sequence and head.
    pages: uint8 [num_pages, kv_heads, record_bytes]; a page index out of range reads as ZERO."""
    ks, vs, lv, sc = [], [], [], []
    for b in range(max(1, -(-length // BLOCK))):
        page = int(table_row[b])
        level = int(levels_row[b]) if levels_row is not None else 4
        if not 0 <= page < pages.shape[0]:
            page, level = 0, 0
        k, v, s = read_record(pages[page, head], D, level)
        ks.append(k), vs.append(v), sc.append(s)
        lv.append(np.full(BLOCK, level))
    return (np.concatenate(ks)[:length], np.concatenate(vs)[:length], np.concatenate(lv)[:length],
            np.concatenate(sc, axis=1)[:, :length])


def attention(q, k, v, level, sc, pos, scale, window, sinks):
    """One head's queries q [n, D] at positions pos over its cached tokens. Returns the output and the
    bound of a computation that keeps scores and statistics in fp32 and rounds each probability
    times its value's scale, and the output, to bf16."""
    n, D = q.shape
    out, tol = np.zeros((n, D)), np.zeros((n, D))
    j = np.arange(len(k))
    for r in range(n):
        see = (j <= pos[r]) & (level > 0)
        if window:
            see &= (pos[r] - j < window) | (j < sinks)
        if not see.any():
            continue
        kk, vv, s = k[see], v[see], sc[:, see].astype(np.float64)
        z = scale * (kk @ q[r])
        e = np.exp(z - z.max())
        w = e / e.sum()
        out[r] = w @ vv
        # |d score|: D products and sums in fp32 on codes off by their centre (8 scales at most)
        mass = abs(scale) * np.max((np.abs(kk) + 8 * s[0][:, None]) @ np.abs(q[r]))
        dz = (D + 8) * 2.0 ** -23 * mass
        room = w @ (np.abs(vv) + 8 * s[1][:, None])
        tol[r] = 2.0 ** -8 * np.abs(out[r]) + room * (2.0 ** -8 + 2 * dz + len(vv) * 2.0 ** -23 + 2.0 ** -18)
    return out, tol * 1.0000001 + 1e-37
