"""Plain CPU oracle for the 8-bit serving operators (test infrastructure).

TEST INFRASTRUCTURE ONLY, like the rest of `oracle/`: imported by `tests/` and by nothing on
the product path, with which it shares no code. Everything is written from the definitions in
float64 (or int64), one sequence, page and head at a time:

* per-token INT8: quantScale = max|x''| / (127 / clipRatio), codes rounded half to even and
  clamped to [-128, 127];
* the INT8 product: the exact integer sum times the two scales;
* E4M3 (1 sign, 4 exponent bits with bias 7, 3 fraction bits, largest 448, no infinity);
* a page's exponent: the smallest e with max|value| <= 448 * 2^e, clamped to [-40, 40];
* rotary positions, appending to pages, and attention over them.
"""

import numpy as np

E_MIN, E_MAX = -40, 40


def per_token_quantize8(x2, clip_ratio):
    """(codes int64 [K, L], quantScale float64 [K], v [K, L] before rounding)."""
    x2 = np.asarray(x2, dtype=np.float64).reshape(len(x2), -1)
    qs = np.abs(x2).max(axis=1) / (127.0 / clip_ratio)
    v = x2 / np.where(qs > 0, qs, 1.0)[:, None]
    return np.clip(np.rint(v), -128, 127).astype(np.int64), qs, v


def int8_matmul(a, a_scale, w, w_scale):
    """C [T, O] float64. The float64 product of 8-bit integers is exact (sums below 2^53)."""
    acc = np.asarray(a, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    return acc * np.asarray(a_scale, dtype=np.float64)[:, None] * np.asarray(w_scale, dtype=np.float64)[None, :]


def _e4m3_table():
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = -v if c & 128 else v
    t[0x7F] = t[0xFF] = np.nan
    return t


E4M3 = _e4m3_table()


def e4m3_encode(x):
    """Nearest code, ties to the even code, saturating; the sign of zero kept."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    mag = E4M3[:0x7F]  # rising magnitudes of the codes 0 .. 126
    hi = np.clip(np.searchsorted(mag, a), 1, 126)
    lo = hi - 1
    dl, dh = a - mag[lo], mag[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def page_exponent(amax):
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def rotary(x, pos, inv_freq, interleaved):
    """x [T, H, D] turned by pos[t] * inv_freq[j] in the pair j of every head."""
    y = np.array(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    n = len(f)
    for j in range(n):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
        ang = np.asarray(pos, dtype=np.float64) * f[j]
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = np.array(x[..., i0], dtype=np.float64), np.array(x[..., i1], dtype=np.float64)
        y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    return y


def kv_store(codes, scale, new, cu, lens, table):
    """Appends new [T, H, D] (float64) to codes [P, H, page, D] (uint8) and scale [P, H]
    (uint8), in place."""
    page = codes.shape[2]
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        first = lens[b] - n
        for p in range(first // page, -(-lens[b] // page)):
            r0, r1 = max(first - p * page, 0), min(lens[b] - p * page, page)
            if r1 <= r0:
                continue
            t0 = cu[b] + p * page + r0 - first
            pg = table[b][p]
            for h in range(codes.shape[1]):
                rows = new[t0:t0 + r1 - r0, h]
                e = page_exponent(np.abs(rows).max())
                old = int(scale[pg, h]) - 127
                if r0 > 0 and old >= e:
                    e = old
                elif r0 > 0:
                    codes[pg, h, :r0] = e4m3_encode(E4M3[codes[pg, h, :r0]] * 2.0 ** (old - e))
                codes[pg, h, r0:r1] = e4m3_encode(rows * 2.0 ** -e)
                scale[pg, h] = e + 127


def kv_values(codes, scale, table_row, n):
    """Cached values [n, H, D] of one sequence."""
    page = codes.shape[2]
    pages = [table_row[p] for p in range(-(-n // page))]
    x = E4M3[codes[pages]] * np.exp2(scale[pages].astype(np.float64) - 127)[..., None, None]
    return x.transpose(0, 2, 1, 3).reshape(-1, codes.shape[1], codes.shape[3])[:n]


def kv_attention(q, k_codes, k_scale, v_codes, v_scale, cu, lens, table, scale, causal):
    """(out [T, Hq, D], lse [T, Hq], info) in float64; rows of no sequence are NaN. info holds,
    per row and head, sum_j p_j |v_j| ("pv", [T, Hq, D]), the largest sum_d |q_d k_jd| * scale
    over the row's keys ("a") and max|v| ("vmax")."""
    T, Hq, D = q.shape
    H = k_codes.shape[1]
    G = Hq // H
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    info = {"pv": np.zeros((T, Hq, D)), "a": np.zeros((T, Hq)), "vmax": np.zeros((T, Hq))}
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        k = kv_values(k_codes, k_scale, table[b], lens[b])
        v = kv_values(v_codes, v_scale, table[b], lens[b])
        for i in range(n):
            t = cu[b] + i
            seen = max(lens[b] - n + i + 1, 0) if causal else lens[b]
            for h in range(Hq):
                if seen == 0:
                    out[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                kk, vv = k[:seen, h // G], v[:seen, h // G]
                z = scale * (kk @ q[t, h])
                m = z.max()
                p = np.exp(z - m)
                lse[t, h] = m + np.log(p.sum())
                p /= p.sum()
                out[t, h] = p @ vv
                info["pv"][t, h] = p @ np.abs(vv)
                info["a"][t, h] = abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
                info["vmax"][t, h] = np.abs(vv).max()
    return out, lse, info
