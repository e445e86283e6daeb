"""Plain forms of what rows of the paged cache see (windows, trees of drafted rows), of the trees' masks and of accepting
drafted rows, on the host copies of kv_reference.py."""
import numpy as np

import kv_reference as ref


def listed(seen):
    """Lists of positions as the rows of an array, -1 behind them (what kv_reference's attention takes as selected)."""
    out = np.full((len(seen), max([len(t) for t in seen] + [1])), -1, np.int32)
    for r, t in enumerate(seen):
        out[r, :len(t)] = t
    return out


def rows_of(c, starts):
    """(row, sequence, first position of the sequence's rows, number of the row among them, rows)."""
    for s in range(len(c.lens)):
        a, b = int(starts[s]), int(starts[s + 1])
        for r in range(a, b):
            yield r, s, int(c.lens[s]) - (b - a), r - a, b - a


def window_seen(c, starts, window, sinks):
    seen = []
    for r, s, first, i, n in rows_of(c, starts):
        p = first + i
        seen.append([t for t in range(p + 1) if t > p - window or t < sinks])
    return listed(seen)


def tree_seen(c, starts, mask):
    seen = []
    for r, s, first, i, n in rows_of(c, starts):
        bits = [j for j in range(min(n, 32 * mask.shape[1])) if int(mask[r, j // 32]) >> (j % 32) & 1]
        seen.append(list(range(max(first, 0))) + [first + j for j in bits if first + j >= 0])
    return listed(seen)


def tree_mask(c, starts, parents, words):
    """(mask, positions) from parents; one that is no earlier row counts as none."""
    n = int(starts[-1])
    mask, positions = np.zeros((n, words), np.int64), np.zeros(n, np.int32)
    for r, s, first, i, _ in rows_of(c, starts):
        at, depth = i, 0
        while True:
            if at < 32 * words:
                mask[r, at // 32] |= 1 << (at % 32)
            up = int(parents[r - i + at])
            if not 0 <= up < at:
                break
            at, depth = up, depth + 1
        positions[r] = first + depth
    return mask.astype(np.uint32).view(np.int32), positions


def random_parents(rng, rows):
    out = []
    for n in rows:
        out += [int(rng.integers(-1, i)) if rng.random() < 0.5 else i - 1 for i in range(n)]
    return np.array(out, np.int32)


def random_accepted(rng, rows):
    """(counts, accepted): ascending parts of each sequence's rows, entries behind them anything."""
    counts, out = [], []
    for n in rows:
        k = int(rng.integers(0, n + 1))
        out += sorted(rng.choice(n, k, replace=False).tolist()) + rng.integers(-5, 9, n - k).tolist()
        counts.append(k)
    return np.array(counts, np.int32), np.array(out, np.int32)


def accept(c, starts, counts, accepted=None):
    """Kept rows behind one another, written as their values would be appended; pages behind the last given back."""
    for s in range(len(c.lens)):
        a, n = int(starts[s]), int(starts[s + 1]) - int(starts[s])
        if n <= 0:
            continue
        old, keep = int(c.lens[s]), int(counts[s])
        first = old - n
        if accepted is not None:
            rows = accepted[a:a + keep].astype(int)
            stay = int((rows == np.arange(keep)).sum())
            kv = [np.stack([c.values(s, h, w)[first + rows[stay:]] for h in range(c.heads)], 1) for w in "kv"]
            c.lens[s] = first + keep
            only = np.zeros(len(c.lens) + 1, np.int64)
            only[s + 1:] = keep - stay
            c.append(kv[0], kv[1], only)
        c.lens[s] = first + keep
        for j in range(-(-(first + keep) // c.page), -(-old // c.page)):
            c.refs[c.table[s, j]] -= 1
            c.table[s, j] = -1


__all__ = ["ref", "listed", "window_seen", "tree_seen", "tree_mask", "random_parents", "random_accepted", "accept"]
