"""CPU oracle of the attention half of a layer: head norms and position
rotation, the 8-bit cache, attention over it. numpy, float64; the cache's
quantizer with its binary32 roundings written out. Test infrastructure only;
shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np

TINY = 2.0 ** -126


def norm_rope(x, w, eps, positions, inv_freq, interleaved):
    """(y, amp): float64 rows [N, H, d] rotated after an optional RMS norm, and
    the length of each value's pair (or its own size where not rotated)."""
    y = np.asarray(x, np.float64).copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    out, amp = y.copy(), np.abs(y)
    rot = 2 * len(inv_freq)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        t = (np.asarray(positions, np.float64) * np.float64(inv_freq[i]))[:, None]
        c, s = np.cos(t), np.sin(t)
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        amp[..., a] = amp[..., b] = np.hypot(y[..., a], y[..., b])
    return out, amp


def _f32(x):
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def append(codes, scale, x, cu, kv_len, table, P):
    """Quantize the new rows x [N, H, d] of a ragged batch into codes
    [pages, H, P, d] int8 and scale [pages, H] float32, in place."""
    for b in range(len(kv_len)):
        q = int(cu[b + 1] - cu[b])
        n = int(kv_len[b])
        for p in range((n - q) // P, -(-n // P) if q else 0):
            lo, hi = max(n - q, p * P), min(n, (p + 1) * P)
            page = int(table[b, p])
            r = int(cu[b]) + lo - (n - q)
            for h in range(codes.shape[1]):
                new = np.asarray(x[r:r + hi - lo, h], np.float64)
                old = float(scale[page, h]) if lo > p * P else 0.0
                fin = np.abs(new[np.isfinite(new)])
                s = max(old, float(_f32((fin.max() if fin.size else 0.0) / 127.0)))
                if s < TINY:
                    s = 0.0
                k = lo - p * P
                if s == 0.0:
                    codes[page, h, :hi - p * P] = 0
                else:
                    c = codes[page, h, :k].astype(np.float64)
                    codes[page, h, :k] = np.rint(_f32(c * _f32(old / s))).astype(np.int8)
                    c = _f32(new * _f32(1.0 / s))
                    c = np.where(np.isnan(c), 0.0, np.clip(c, -127, 127))
                    codes[page, h, k:hi - p * P] = np.rint(c).astype(np.int8)
                scale[page, h] = np.float32(s)


def values(codes, scale, table_row, n, P):
    """float64 [n, H, d]: the first n tokens of a sequence."""
    ids = [int(i) for i in table_row[:-(-n // P)]]
    if not ids:
        return np.zeros((0,) + codes.shape[1:2] + codes.shape[3:])
    v = codes[ids].astype(np.float64) * scale[ids].astype(np.float64)[:, :, None, None]
    return v.transpose(0, 2, 1, 3).reshape(-1, codes.shape[1], codes.shape[3])[:n]


def attention(q, kc, vc, ks, vs, cu, kv_len, table, P, *, scale, causal=True, window=0):
    """(out, lse, spread, top): float64 outputs, lse, sum_j w_j |v_j|, and the
    largest single weight times v scale times 127 of each row."""
    N, Hq, d = q.shape
    H = kc.shape[1]
    G = Hq // H
    out, spread = np.zeros((N, Hq, d)), np.zeros((N, Hq, d))
    lse, top = np.full((N, Hq), -np.inf), np.zeros((N, Hq))
    for b in range(len(kv_len)):
        n, r0, r1 = int(kv_len[b]), int(cu[b]), int(cu[b + 1])
        if r1 <= r0 or n == 0:
            continue
        K, V = values(kc, ks, table[b], n, P), values(vc, vs, table[b], n, P)
        sc = np.repeat(vs[[int(i) for i in table[b, :-(-n // P)]]].astype(np.float64), P, 0)[:n]
        pos = n - (r1 - r0) + np.arange(r1 - r0)
        j = np.arange(n)
        ok = np.ones((r1 - r0, n), bool)
        if causal:
            ok = j[None] <= pos[:, None]
            if window:
                ok &= j[None] > pos[:, None] - window
        for h in range(Hq):
            t = np.where(ok, q[r0:r1, h].astype(np.float64) @ K[:, h // G].T * scale, -np.inf)
            m = t.max(1, keepdims=True)
            m[np.isinf(m)] = 0.0
            e = np.exp(t - m)
            l = e.sum(1, keepdims=True)
            some = l[:, 0] > 0
            w = e / np.where(l > 0, l, 1.0)
            out[r0:r1, h] = w @ V[:, h // G]
            spread[r0:r1, h] = w @ np.abs(V[:, h // G])
            lse[r0:r1, h][some] = (m + np.log(np.where(l > 0, l, 1.0)))[some, 0]
            top[r0:r1, h] = (w * sc[None, :, h // G]).max(1) * 127
    return out, lse, spread, top
