"""Plain 64-bit definitions of the operators between a decoder layer's matvecs,
in numpy, and the bounds their results are held to."""
import math

import numpy as np

QMAX = {"e4m3": 448.0, "i8": 127.0}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def e4m3_values():
    """The value of each of the 256 codes."""
    v = []
    for c in range(128):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    v[127] = math.nan
    return np.array(v + [-x for x in v])


E4M3 = e4m3_values()
E4M3_POS = E4M3[:127]


def decode(codes, fmt):
    return codes.astype(np.uint8).view(np.int8).astype(np.float64) if fmt == "i8" else E4M3[codes]


def encode(x, fmt):
    """Nearest code, ties to even; |x| <= QMAX."""
    x = np.asarray(x, np.float64)
    if fmt == "i8":
        return np.rint(x).astype(np.int8).view(np.uint8)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3_POS[hi] - a, a - E4M3_POS[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def same_codes(a, b, fmt):
    """Equal as the values they stand for (the sign of a zero is free)."""
    return np.array_equal(decode(a, fmt), decode(b, fmt), equal_nan=True)


def scale_of(amax, fmt):
    """Least 2^e, e >= -64, with amax <= QMAX 2^e."""
    e = -64
    if amax > 0:
        e = max(-64, math.frexp(amax / QMAX[fmt])[1] - 2)
        while amax > QMAX[fmt] * 2.0 ** e:
            e += 1
    return 2.0 ** e


def rope_rows(base, rows, rot):
    ang = np.arange(rows, dtype=np.float64)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def rotate(x, cs, inter):
    """x [..., dim] float64, cs [rot / 2][2]."""
    half = cs.shape[0]
    y = x.copy()
    i = np.arange(half) * 2 if inter else np.arange(half)
    j = i + 1 if inter else i + half
    c, s = cs[:, 0].astype(np.float64), cs[:, 1].astype(np.float64)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def positions(lens, starts, tokens):
    """[(row, sequence, position)] of every row that a sequence has."""
    out = []
    for s in range(len(lens)):
        a, b = min(max(starts[s], 0), tokens), min(max(starts[s + 1], 0), tokens)
        out += [(a + i, s, int(lens[s]) - (b - a) + i) for i in range(b - a)]
    return out


def append(cache, table, lens, starts, k, v, cs, inter, fmt):
    """cache: dict of numpy arrays k, v (codes), ks, vs, changed in place."""
    pages, heads, T, _ = cache["k"].shape
    cap = table.shape[1] * T
    groups = {}
    for row, s, p in positions(lens, starts, len(k)):
        if 0 <= p < cap and 0 <= table[s, p // T] < pages:
            groups.setdefault(int(table[s, p // T]), []).append((p % T, row, p))
    for page, rows in groups.items():
        rows.sort()
        slots, src = [r[0] for r in rows], [r[1] for r in rows]
        for name, x in (("k", k), ("v", v)):
            new = x[src].astype(np.float64)  # [m][heads][dim]
            if name == "k" and cs is not None:
                new = np.stack([rotate(new[i], cs[r[2]], inter) for i, r in enumerate(rows)])
            for h in range(heads):
                y, old = new[:, h], float(cache[name + "s"][page, h])
                fresh = slots[0] == 0
                if not np.isfinite(y).all() or (not fresh and (not math.isfinite(old) or np.signbit(old))):
                    cache[name + "s"][page, h] = np.nan
                    cache[name][page, h, slots] = 0
                    continue
                now = scale_of(float(np.abs(y).max()), fmt)
                if not fresh:
                    now = max(now, old)
                    if now > old:
                        c = cache[name][page, h, :slots[0]]
                        cache[name][page, h, :slots[0]] = encode(decode(c, fmt) * (old / now), fmt)
                cache[name + "s"][page, h] = now
                cache[name][page, h, slots] = encode(y / now, fmt)


def attend(cache, table, lens, starts, q, scale, window, fmt, dtype):
    """(out, bound) in float64; bound is how far a right kernel may be off.
    Rows that no sequence has are NaN in both."""
    pages, heads, T, D = cache["k"].shape
    tokens, qh, _ = q.shape
    group = qh // heads
    out, tol = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    with np.errstate(invalid="ignore"):
        kk = decode(cache["k"], fmt) * cache["ks"].astype(np.float64)[:, :, None, None]
        vv = decode(cache["v"], fmt) * cache["vs"].astype(np.float64)[:, :, None, None]
    u = HALF_STEP[dtype]
    w_err = 2.0 ** -20 if dtype == "f32" else 2.0 ** -11
    for row, s, p in positions(lens, starts, tokens):
        t = np.arange(max(0, p + 1 - window) if window else 0, max(0, min(p + 1, table.shape[1] * T)))
        pg = table[s, t // T] if len(t) else np.zeros(0, np.int64)
        ok = (pg >= 0) & (pg < pages)
        t, pg = t[ok], pg[ok]
        if not len(t):
            out[row], tol[row] = 0.0, 0.0
            continue
        for h in range(heads):
            keys, vals = kk[pg, h, t % T], vv[pg, h, t % T]
            if not (np.isfinite(cache["ks"][pg, h]).all() and np.isfinite(cache["vs"][pg, h]).all()):
                continue  # poisoned: NaN
            x = q[row, h * group:(h + 1) * group].astype(np.float64)
            sc = x @ keys.T * scale
            w = np.exp(sc - sc.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            o = w @ vals
            # a score is off by its products' rounding (D fp32 additions; q kept to 2^-22) and by
            # the rounding of its own size; a weight by twice that; sums of len(t) weights
            ds = (np.abs(x) @ np.abs(keys).T).max(-1) * abs(scale) * (D * 2.0 ** -24 + 2.0 ** -21) + \
                np.abs(sc).max(-1) * 2.0 ** -22
            rel = w_err + 2.0 * ds + (len(t) + 16) * 2.0 ** -24
            out[row, h * group:(h + 1) * group] = o
            tol[row, h * group:(h + 1) * group] = rel[:, None] * (w @ np.abs(vals)) + u * np.abs(o) + 2.0 ** -25 * (
                dtype == "f16")  # half a step of the smallest fp16 numbers
    return out, tol


def norm(x, resid, post_w, gate, scale, pre_w, eps):
    """(r, out, size of r's terms) in float64."""
    def unit(t):
        return t / np.sqrt((t * t).mean(-1, keepdims=True) + eps)

    t = x.astype(np.float64)
    if post_w is not None:
        t = unit(t) * post_w
    t = scale * (1.0 if gate is None else gate) * t
    r = t if resid is None else resid + t
    size = np.abs(t) + (0.0 if resid is None else np.abs(resid))
    out = unit(r) * (1.0 if pre_w is None else pre_w)
    return r, out, size
