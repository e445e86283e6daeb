"""Plain 64-bit forms of the paged 8-bit cache's operators (numpy), and the bounds their results are held to."""
import math

import numpy as np

U_OUT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step of the output type, relative to the value
TINY_OUT = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # half the smallest step


def e4m3_table():
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            v = math.nan
        t[c] = -v if c & 128 else v
    return t


E4M3 = e4m3_table()
_POS = E4M3[:127]


def round_e4m3(x):
    """Codes of x (64 bits): nearest, ties to even, saturating; infinities saturate, NaN is kept."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.searchsorted(_POS, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(_POS[hi] == a, hi, code)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def need_exp(amax):
    """Least exponent byte whose scale holds amax within 448."""
    if amax == 0:
        return 7
    e = -400
    m, x = math.frexp(amax / 448.0)
    e = x if m > 0.5 else x - 1
    while amax > 448.0 * 2.0 ** e:
        e += 1
    while amax <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return min(max(e + 127, 7), 247)


class Cache:
    """Host copy of a cache's tensors with the operators' plain forms."""

    def __init__(self, k, v, ke, ve, table, lens, refs):
        self.k, self.v, self.ke, self.ve = k, v, ke, ve
        self.table, self.lens, self.refs = table, lens, refs
        self.pages, self.heads, self.page, self.dim = k.shape
        self.status = 0

    def copy(self):
        return Cache(*(a.copy() for a in (self.k, self.v, self.ke, self.ve, self.table, self.lens, self.refs)))

    def values(self, s, head, which):
        codes, exps = (self.k, self.ke) if which == "k" else (self.v, self.ve)
        n = int(self.lens[s])
        used = self.table[s, :-(-n // self.page)]
        x = E4M3[codes[used, head]] * 2.0 ** (exps[used, head].astype(np.float64) - 127)[:, None, None]
        return x.reshape(-1, self.dim)[:n]

    # ---- attention: (out, lse, bound of out, bound of lse)
    def attention(self, q, starts, scale, dtype, selected=None, causal=True):
        rows, hq, d = q.shape
        g = hq // self.heads
        out, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -np.inf)
        tol, ltol = np.zeros((rows, hq, d)), np.zeros((rows, hq))
        for s in range(len(self.lens)):
            a, b = int(starts[s]), int(starts[s + 1])
            if a == b:
                continue
            for h in range(self.heads):
                K, V = self.values(s, h, "k"), self.values(s, h, "v")
                nan = np.isnan(K).any(1) | np.isnan(V).any(1)
                for r in range(a, b):
                    last = int(self.lens[s]) - (b - a) + (r - a) if causal else int(self.lens[s]) - 1
                    t = np.arange(max(last + 1, 0))
                    if selected is not None:
                        t = selected[r][(selected[r] >= 0) & (selected[r] <= last)]
                    for x in range(h * g, h * g + g):
                        if len(t) == 0:
                            continue
                        if nan[t].any() or not np.isfinite(q[r, x]).all():
                            out[r, x], lse[r, x] = np.nan, np.nan
                            continue
                        kt, vt = K[t], V[t]
                        sc = scale * (kt @ q[r, x])
                        top = sc.max()
                        p = np.exp(sc - top)
                        total = p.sum()
                        out[r, x] = p @ vt / total
                        lse[r, x] = top + math.log(total)
                        # scores: fp32 products summed in chunks of 16 by the tensor cores (each sum
                        # may lose 2^-22 of the magnitudes in it), then a product and a difference
                        mag = scale * (np.abs(kt) @ np.abs(q[r, x]))
                        ds = ((d / 16 + 2) * 2.0 ** -22 * mag + 2.0 ** -22 * (np.abs(sc) + abs(top))).max() + 2.0 ** -21
                        # query values as sums of e4m3 terms: 2^-10 of a largest value of 224 or more is lost
                        ds += (scale * np.abs(q[r, x]).max() * 2.0 ** -10 / 224 * np.abs(kt).sum(1)).max()
                        sums = (len(t) / 16 + 64) * 2.0 ** -22
                        mean = p @ np.abs(vt) / total
                        # a weight is rounded to fp16: 2^-11 of it, or 2^-25 of the largest weight times scale
                        big = (p * np.abs(vt).max(1)).max() / total
                        err = mean * (2.0 ** -11 + 2 * ds + sums) + len(t) * 2.0 ** -25 * 2 * big
                        tol[r, x] = (np.abs(out[r, x]) + err) * U_OUT[dtype] * 1.01 + err + TINY_OUT[dtype]
                        ltol[r, x] = 2 * ds + sums + 2.0 ** -22 * abs(lse[r, x])
        return out, lse, tol, ltol

    # ---- appending
    def append(self, k, v, starts):
        for s in range(len(self.lens)):
            a, b = int(starts[s]), int(starts[s + 1])
            first = int(self.lens[s]) - (b - a)
            for lo in range(max(first, 0), int(self.lens[s])):
                if lo % self.page and lo != max(first, 0):
                    continue
                hi = min((lo // self.page + 1) * self.page, int(self.lens[s]))
                p, held = self.table[s, lo // self.page], lo % self.page
                for codes, exps, x in ((self.k, self.ke, k), (self.v, self.ve, v)):
                    for h in range(self.heads):
                        part = x[a + lo - first:a + hi - first, h].astype(np.float64)
                        fin = np.abs(part[np.isfinite(part)])
                        e = need_exp(fin.max() if fin.size else 0.0)
                        if held:
                            was = int(exps[p, h])
                            e = max(e, was)
                            if e > was:
                                codes[p, h, :held] = round_e4m3(E4M3[codes[p, h, :held]] * 2.0 ** (was - e))
                        codes[p, h, held:held + hi - lo] = round_e4m3(part * 2.0 ** (127 - e))
                        exps[p, h] = e

    # ---- pages
    def _count(self, n):
        return -(-int(n) // self.page)

    def _free_pages(self, n):
        f = np.nonzero(self.refs == 0)[0]
        return f[:n] if len(f) >= n else None

    def reserve(self, counts):
        cap = self.table.shape[1] * self.page
        if (counts < 0).any():
            return 4
        if ((self.lens.astype(np.int64) + counts) > cap).any():
            return 8
        need = [self._count(n + c) - self._count(n) for n, c in zip(self.lens, counts)]
        got = self._free_pages(sum(need))
        if got is None:
            return 1
        at = 0
        for s, n in enumerate(need):
            have = self._count(self.lens[s])
            self.table[s, have:have + n] = got[at:at + n]
            self.refs[got[at:at + n]] = 1
            at += n
            self.lens[s] += counts[s]
        return 0

    def fork(self, parents, children):
        if len(set(children.tolist())) < len(children) or (self.lens[children] != 0).any():
            return 4
        part = [int(self.lens[p]) % self.page != 0 for p in parents]
        got = self._free_pages(sum(part))
        if got is None:
            return 1
        got = list(got)
        lens = self.lens.copy()
        for p, c, x in zip(parents, children, part):
            full = int(lens[p]) // self.page
            self.table[c, :full] = self.table[p, :full]
            np.add.at(self.refs, self.table[p, :full], 1)
            if x:
                new = got.pop(0)
                self.copy_pages([self.table[p, full]], [new])
                self.table[c, full] = new
                self.refs[new] = 1
            self.lens[c] = lens[p]
        return 0

    def free(self, seqs):
        for s in seqs:
            n = self._count(self.lens[s])
            np.subtract.at(self.refs, self.table[s, :n], 1)
            self.table[s, :n] = -1
            self.lens[s] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        dst = np.nonzero(self.refs[:live] == 0)[0]
        src = live + np.nonzero(self.refs[live:] > 0)[0]
        to = np.arange(self.pages)
        to[src] = dst
        self.copy_pages(src, dst)
        for s in range(len(self.lens)):
            n = self._count(self.lens[s])
            self.table[s, :n] = to[self.table[s, :n]]
        self.refs[dst] = self.refs[src]
        self.refs[src] = 0

    def copy_pages(self, src, dst):
        for a in (self.k, self.v, self.ke, self.ve):
            a[dst] = a[src]


def random_cache(rng, pages, heads, page, dim, lens, max_pages, spread=2, garbage=True, shuffle=True):
    """A cache whose sequences hold `lens` positions of normal values; unused codes are anything (NaN too)."""
    codes = rng.integers(0, 256, (2, pages, heads, page, dim)).astype(np.uint8) if garbage else \
        np.zeros((2, pages, heads, page, dim), np.uint8)
    exps = rng.integers(127 - spread, 128 + spread, (2, pages, heads)).astype(np.uint8)
    table = rng.integers(-3, pages + 3, (len(lens), max_pages)).astype(np.int32)  # entries behind the pages: anything
    refs = np.zeros(pages, np.int32)
    order = rng.permutation(pages) if shuffle else np.arange(pages)
    at = 0
    for s, n in enumerate(lens):
        c = -(-n // page)
        table[s, :c] = order[at:at + c]
        refs[order[at:at + c]] = 1
        at += c
        for j in range(c):
            m = min(page, n - j * page)
            x = rng.standard_normal((2, heads, m, dim)) * 60
            codes[:, order[at - c + j], :, :m] = round_e4m3(x)
    assert at <= pages
    return Cache(codes[0], codes[1], exps[0], exps[1], table, np.array(lens, np.int32), refs)


def to_device(c, mqa, extra=()):
    import torch
    t = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    return mqa.KVCache(t(c.k), t(c.v), t(c.ke), t(c.ve), t(c.table), t(c.lens), t(c.refs), extra=extra)


def same(c, dev):
    """Names of the tensors in which a device cache differs from the plain one."""
    pairs = {"k": c.k, "v": c.v, "k_exps": c.ke, "v_exps": c.ve, "page_table": c.table, "seq_lens": c.lens,
             "refcounts": c.refs}
    return [n for n, a in pairs.items() if not np.array_equal(getattr(dev, n).cpu().numpy(), a)]
