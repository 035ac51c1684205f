"""Plain fp64 / integer definitions of the paged-cache operators (numpy, loops over requests and rows).

TEST INFRASTRUCTURE ONLY, like the rest of this package: shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ROW_BYTES = 416


def _bf16(t):
    """bf16 torch tensor -> float64 array."""
    import torch
    return t.detach().cpu().to(torch.float64).numpy()


def block_tables(seq, new, table, free, page, pages, max_tokens, start=0):
    """(slots, positions, requests, starts, free_next, table, bad) of one step, request by request."""
    table = np.array(table, np.int64)
    slots, pos_, req_ = [], [], []
    starts, at, bad = [0], start, False
    for r, (n, w) in enumerate(zip(seq, new)):
        n, w = int(n), int(w)
        if w < 0 or n < w or n > table.shape[1] * page:
            bad, n, w = True, 0, 0
            starts.append(starts[-1])
            continue
        for b in range(-(-(n - w) // page), -(-n // page)):
            p = int(free[at]) if at < len(free) else -1
            if not 0 <= p < pages:
                bad, p = True, -1
            table[r, b] = p
            at += 1
        for s in range(n - w, n):
            p = int(table[r, s // page])
            if not 0 <= p < pages:
                bad, p = True, -1
            slots.append(-1 if p < 0 else p * page + s % page)
            pos_.append(s)
            req_.append(r)
        starts.append(starts[-1] + w)
    if len(slots) > max_tokens:
        bad = True
    pad = [-1] * max(0, max_tokens - len(slots))
    return (np.array((slots + pad)[:max_tokens], np.int64), np.array((pos_ + pad)[:max_tokens], np.int32),
            np.array((req_ + pad)[:max_tokens], np.int32), np.array(starts, np.int32),
            min(at, len(free)), table.astype(np.int32), bad)


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    f = []
    if scaling == "yarn":
        pair = [rot * math.log(original_len / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (beta_fast, beta_slow)]
        lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), rot - 1)
    for i in range(rot // 2):
        v = base ** (-2.0 * i / rot)
        if scaling == "linear":
            v /= factor
        if scaling == "yarn":
            ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            v = v / factor * ramp + v * (1 - ramp)
        f.append(v)
    return np.array(f)


def rope(x, positions, freq, layout, offset, mscale):
    """x float64 [N,H,D] -> rotated; rows with a negative position as they are."""
    y = np.array(x, np.float64)
    n = len(freq)
    for t, p in enumerate(positions):
        if p < 0:
            continue
        for i in range(n):
            a, b = (offset + i, offset + n + i) if layout == "half" else (offset + 2 * i, offset + 2 * i + 1)
            c, s = math.cos(int(p) * freq[i]), math.sin(int(p) * freq[i])
            u, v = x[t, :, a], x[t, :, b]
            y[t, :, a], y[t, :, b] = mscale * (u * c - v * s), mscale * (u * s + v * c)
    return y


def _e4m3_table():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m / 512 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if c & 127 == 127 else -a if c & 128 else a
    return v


E4M3 = _e4m3_table()


def kv4_pack(rows):
    """bf16 rows [n, 576] -> uint8 [n, 416], by distance to every representable value."""
    import torch
    x = _bf16(rows)[:, :512].reshape(-1, 32, 16)
    amax = np.abs(x).max(2)                              # NaN stays
    want = np.minimum(amax / 6, 448.0)
    grid = E4M3[:127]
    # ties to the even code: bf16 / 6 is a tie or off one by 2^-12 of itself and more
    d = np.abs(want[:, :, None] - grid) + 1e-9 * want[:, :, None] * (np.arange(127) % 2)
    code = np.where(np.isnan(want), 127, np.argmin(np.where(np.isnan(d), 0, d), axis=2)).astype(np.uint8)
    s = E4M3[code][:, :, None]
    with np.errstate(all="ignore"):
        q = np.where(s == 0, 0.0, np.minimum(np.abs(x), 1e6) / np.where(s == 0, 1.0, s))
    mag = np.array(MAGNITUDES)
    e = np.abs(q[..., None] - mag) + 1e-12 * (np.arange(8) % 2)
    nib = np.argmin(np.where(np.isnan(e), 0, e), axis=3).astype(np.uint8) + 8 * np.signbit(x).astype(np.uint8)
    nib = nib.reshape(-1, 256, 2)
    raw = rows.detach().cpu()[:, 512:].contiguous().view(torch.uint8).numpy()
    return np.concatenate([nib[:, :, 0] | (nib[:, :, 1] << 4), code, raw], axis=1).astype(np.uint8)


def kv4_unpack(raw):
    """uint8 [n, 416] -> float64 [n, 576]."""
    import torch
    raw = np.asarray(raw, np.uint8)
    val = np.array(MAGNITUDES + tuple(-m for m in MAGNITUDES))
    c = raw[:, :256]
    v = val[np.stack([c & 15, c >> 4], 2).reshape(-1, 512)]
    s = np.repeat(E4M3[raw[:, 256:288]], 16, axis=1)
    r = torch.from_numpy(np.ascontiguousarray(raw[:, 288:])).view(torch.bfloat16).to(torch.float64).numpy()
    return np.concatenate([v * s, r], axis=1)


def visible(position, window, sinks):
    """Positions a token at `position` sees, ascending."""
    s = np.arange(position + 1)
    return s[(s < sinks) | (s > position - window)]


def attention(q, rows, scale):
    """q float64 [H,576], rows float64 [n,576] -> (o [H,512], sum_i p_i |v_i|, the largest
    scale * sum_d |q_d k_d| of a head) with o = 0 when there is no row."""
    if rows.shape[0] == 0:
        z = np.zeros((q.shape[0], 512))
        return z, z, np.zeros(q.shape[0])
    lg = scale * (q @ rows.T)
    p = np.exp(lg - lg.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return p @ rows[:, :512], p @ np.abs(rows[:, :512]), scale * (np.abs(q) @ np.abs(rows).T).max(1)
