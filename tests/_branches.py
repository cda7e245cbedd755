"""Plain 64-bit definitions, in numpy, of the operators for several continuations
of a sequence: trees of new tokens, norms of heads, pages that sequences share,
accepted paths, beam search's selection; and the bounds results are held to."""
import math

import _layer as L
import numpy as np

MAX_TREE = 512


def line(tree, i):
    """Token i's ancestors and itself, the first one first; what is no earlier token ends the line."""
    out = [i]
    while 0 <= tree[i] < i:
        i = tree[i]
        out.append(i)
    return out[::-1]


def random_tree(rng, n, wide=0.3):
    return [-1 if i == 0 or rng.random() < wide / (1 + i) else int(rng.integers(max(-1, i - 6), i)) for i in range(n)]


def rows_of(lens, starts, tokens, parents):
    """[(row, sequence, slot's position, position, line's positions of slots)] of the
    rows that have a place or at least a sequence; position None: no tree."""
    out = []
    for s in range(len(lens)):
        a, b = min(max(starts[s], 0), tokens), min(max(starts[s + 1], 0), tokens)
        n = max(b - a, 0)
        base = int(lens[s]) - n
        for i in range(n):
            if parents is None:
                out.append((a + i, s, base + i, base + i, [base + j for j in range(i + 1)]))
            elif n > MAX_TREE or base < 0:
                out.append((a + i, s, None, None, []))
            else:
                ln = line(parents[a:b], i)
                out.append((a + i, s, base + i, base + len(ln) - 1, [base + j for j in ln]))
    return out


def normed(x, w, eps):
    """Heads of x [..., heads, dim] normed; w [dim] or [heads][dim]."""
    if w is None:
        return x.astype(np.float64)
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def append(cache, table, lens, starts, q, k, v, cs, inter, fmt, parents=None, q_norm=None, k_norm=None, eps=1e-5):
    """Changes `cache` (numpy k, v, ks, vs) in place; returns (q, size of its terms), rows that are
    not written NaN."""
    pages, heads, T, _ = cache["k"].shape
    cap = table.shape[1] * T
    kn, qn = normed(k, k_norm, eps), normed(q, q_norm, eps)
    qo, size = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    groups = {}
    for row, s, at, pos, _ in rows_of(lens, starts, len(k), parents):
        if at is None or not 0 <= at < cap:
            continue
        if cs is None:
            qo[row], size[row] = qn[row], np.abs(qn[row])
        else:
            qo[row] = L.rotate(qn[row], cs[pos], inter)
            size[row] = L.rotate(np.abs(qn[row]), np.abs(cs[pos]) * [1, -1], inter)  # |a c| + |b s|
            half = cs.shape[1]
            j = (np.arange(half) * 2 + 1) if inter else np.arange(half) + half
            size[row][..., j] = L.rotate(np.abs(qn[row]), np.abs(cs[pos]), inter)[..., j]
        if 0 <= table[s, at // T] < pages:
            groups.setdefault(int(table[s, at // T]), []).append((at % T, row, pos))
    for page, rows in groups.items():
        rows.sort()
        slots, src = [r[0] for r in rows], [r[1] for r in rows]
        for name, x in (("k", kn), ("v", v.astype(np.float64))):
            new = x[src]
            if name == "k" and cs is not None:
                new = np.stack([L.rotate(new[i], cs[r[2]], inter) for i, r in enumerate(rows)])
            for h in range(heads):
                y, old = new[:, h], float(cache[name + "s"][page, h])
                fresh = slots[0] == 0
                if not np.isfinite(y).all() or (not fresh and (not math.isfinite(old) or np.signbit(old))):
                    cache[name + "s"][page, h] = np.nan
                    cache[name][page, h, slots] = 0
                    continue
                now = L.scale_of(float(np.abs(y).max()), fmt)
                if not fresh:
                    now = max(now, old)
                    if now > old:
                        c = cache[name][page, h, :slots[0]]
                        cache[name][page, h, :slots[0]] = L.encode(L.decode(c, fmt) * (old / now), fmt)
                cache[name + "s"][page, h] = now
                cache[name][page, h, slots] = L.encode(y / now, fmt)
    return qo, size


def attend(cache, table, lens, starts, q, scale, window, fmt, dtype, parents):
    """(out, bound): rows that no sequence has are NaN in both.  The bound counts as that of L.attend."""
    pages, heads, T, D = cache["k"].shape
    tokens, qh, _ = q.shape
    group = qh // heads
    out, tol = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    with np.errstate(invalid="ignore"):
        kk = L.decode(cache["k"], fmt) * cache["ks"].astype(np.float64)[:, :, None, None]
        vv = L.decode(cache["v"], fmt) * cache["vs"].astype(np.float64)[:, :, None, None]
    u = L.HALF_STEP[dtype]
    w_err = 2.0 ** -20 if dtype == "f32" else 2.0 ** -11
    cap = table.shape[1] * T
    for row, s, at, pos, own in rows_of(lens, starts, tokens, parents):
        t = []
        if at is not None:
            base = own[0] if parents is None else pos - len(own) + 1
            t = [(p, p) for p in range(max(0, base))] + [(p, base + i) for i, p in enumerate(own)]
            t = [p for p, where in t if 0 <= p < cap and (not window or where > pos - window)]
        t = np.array(t, np.int64)
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
            ds = (np.abs(x) @ np.abs(keys).T).max(-1) * abs(scale) * (D * 2.0 ** -24 + 2.0 ** -21) + \
                np.abs(sc).max(-1) * 2.0 ** -22
            rel = w_err + 2.0 * ds + (len(t) + 16) * 2.0 ** -24
            out[row, h * group:(h + 1) * group] = o
            # Weights are held as fp16 numbers (two of them, the second for what the first leaves off), the
            # row's largest as 2^6 or more, times their page's scale by the largest one: half a step of the
            # smallest fp16 numbers, 2^-25, is 2^-31 of the largest weight, in units of the largest scale.
            least = 2.0 ** -31 * cache["vs"][pg, h].max() * np.abs(L.decode(cache["v"][pg, h, t % T], fmt)).sum(0)
            tol[row, h * group:(h + 1) * group] = rel[:, None] * (w @ np.abs(vals)) + least + u * np.abs(o) + \
                2.0 ** -25 * (dtype == "f16")
    return out, tol


class Book:
    """Page tables, lengths, counts of holders and some caches (dicts of numpy arrays)."""

    def __init__(self, table, lens, pages, T, caches):
        self.table, self.lens, self.T, self.caches = np.array(table), [int(x) for x in lens], T, caches
        self.pages = pages

    def refs(self):
        t = self.table[(self.table >= 0) & (self.table < self.pages)]
        return np.bincount(t, minlength=self.pages)

    def fork(self, source, keep=None):
        old, had = self.table.copy(), list(self.lens)
        for s, src in enumerate(source):
            ok = 0 <= src < len(had)
            n = had[src] if ok else 0
            if keep is not None:
                n = min(n, keep[s])
            self.lens[s] = max(0, n)
            for c in range(old.shape[1]):
                p = old[src, c] if ok and c * self.T < self.lens[s] else -1
                self.table[s, c] = p if 0 <= p < self.pages else -1

    def grow(self, more):
        """Pages missing (then nothing changes)."""
        refs, T = self.refs(), self.T
        first = [n // T if n % T else None for n in self.lens]
        needs, beyond = [], 0
        there = lambda p: 0 <= p < self.pages  # noqa: E731
        for s, n in enumerate(self.lens):
            a = max(0, more[s])
            for c in range(n // T, -(-(n + a) // T) if a else 0):
                if c >= self.table.shape[1]:
                    beyond += 1
                    continue
                p = self.table[s, c]
                if c == first[s]:
                    if not there(p) or refs[p] <= 1:
                        continue
                    same = [i for i in range(len(self.lens)) if more[i] > 0 and first[i] is not None and
                            first[i] < self.table.shape[1] and self.table[i, first[i]] == p]
                    if len(same) == refs[p] and s == same[-1]:
                        continue
                    needs.append((s, c, p, n % T))
                elif not there(p) or refs[p] > 1:
                    needs.append((s, c, -1, 0))
        free = [p for p in range(self.pages) if refs[p] == 0]
        missing = beyond + max(0, len(needs) - len(free))
        if beyond or len(needs) > len(free):
            return missing
        for (s, c, p, slots), now in zip(needs, free):
            self.table[s, c] = now
            if p >= 0:
                for x in self.caches:
                    for n in "kv":
                        x[n][now, :, :slots] = x[n][p, :, :slots]
                        x[n + "s"][now] = x[n + "s"][p]
        for s in range(len(self.lens)):
            self.lens[s] += max(0, more[s])
        return 0


def accept(caches, fmt, table, lens, starts, tokens, parents, leaf):
    """New lengths; changes the caches (dicts of numpy arrays) in place."""
    out = []
    for s in range(len(lens)):
        a, b = min(max(starts[s], 0), tokens), min(max(starts[s + 1], 0), tokens)
        n, length = max(b - a, 0), int(lens[s])
        base = length - n
        if n == 0 or base < 0 or (parents is not None and n > MAX_TREE):
            out.append(length)
            continue
        ln = []
        if 0 <= leaf[s] < n:
            ln = list(range(leaf[s] + 1)) if parents is None else line(parents[a:b], leaf[s])
        pages, _, T, _ = caches[0]["k"].shape

        def page(pos):
            p = table[s, pos // T] if pos // T < table.shape[1] else -1  # noqa: B023
            return int(p) if 0 <= p < pages else None  # noqa: B023

        for i, t in enumerate(ln):
            if page(base + i) is None or page(base + t) is None:
                ln = ln[:i]
                break
        out.append(base + len(ln))
        if ln == list(range(len(ln))):
            continue
        good = lambda x: math.isfinite(x) and not np.signbit(x)  # noqa: E731
        for x in caches:
            for name in "kv":
                codes, scales = x[name], x[name + "s"]
                for h in range(codes.shape[1]):
                    # codes and scales as they were: a path's tokens come from their own slots or later ones
                    src = [(page(base + t), codes[page(base + t), h, (base + t) % T].copy(),
                            float(scales[page(base + t), h])) for t in ln]
                    by_page = {}
                    for i in range(len(ln)):
                        by_page.setdefault(page(base + i), []).append(i)
                    for p, items in by_page.items():
                        old, slot0 = float(scales[p, h]), (base + items[0]) % T
                        others = [i for i in items if src[i][0] != p]
                        poison = any(not good(src[i][2]) for i in others)
                        now = old
                        if good(old):
                            top = max([0.0] + [np.abs(L.decode(src[i][1], fmt)).max() * src[i][2] for i in others if
                                               good(src[i][2])])
                            if poison:
                                now = math.nan
                            elif top > 0:
                                now = max(old, L.scale_of(top, fmt))
                        raised = good(now) and now > old
                        if raised:
                            codes[p, h, :slot0] = L.encode(L.decode(codes[p, h, :slot0], fmt) * old / now, fmt)
                        if not good(now) and good(old):
                            scales[p, h] = np.nan
                        elif raised:
                            scales[p, h] = now
                        for i in items:
                            q, c, sc = src[i]
                            if q != p and not good(now):
                                c = np.zeros_like(c)
                            elif q != p or raised:
                                c = L.encode(L.decode(c, fmt) * sc / now, fmt) if now > 0 else np.zeros_like(c)
                            codes[p, h, (base + i) % T] = c
    return out


def beams(logits, scores, keep, ended=None, end_token=0):
    """(scores, parents, tokens) as nested lists; logits [items][beams][vocab] in float64."""
    out = ([], [], [])
    items, nb, _ = logits.shape
    for i in range(items):
        found = []
        for b in range(nb):
            x, s = logits[i, b], float(scores[i, b])
            if not math.isfinite(s):
                continue
            if ended is not None and ended[i, b]:
                found.append((-s, b, 0.0, end_token))
                continue
            if np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any():
                continue
            top = x.max()
            y = s + (x - (top + math.log(np.exp(x - top).sum())))
            t = np.flatnonzero(x > -np.inf)
            least = np.sort(x[t])[::-1][min(keep, len(t)) - 1]
            found += [(-y[j], b, -x[j], int(j)) for j in t[x[t] >= least]]
        found = sorted(found)[:keep]
        out[0].append([-f[0] for f in found] + [-math.inf] * (keep - len(found)))
        out[1].append([i * nb + f[1] for f in found] + [-1] * (keep - len(found)))
        out[2].append([f[3] for f in found] + [-1] * (keep - len(found)))
    return out
