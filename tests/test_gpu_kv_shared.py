"""Accepted rows and roll-backs of forked sequences, whose pages are shared: what a call writes into, or leaves partly
filled, becomes the sequence's own, and nobody else's codes change."""
import numpy as np
import pytest

import kv_reference as ref
import view_reference as view
from test_gpu_kv import ints, mqa, rows_of, starts_of  # noqa: F401

pytestmark = pytest.mark.gpu


def only(starts, s):
    """Bounds that give rows to sequence s alone."""
    out = np.full(len(starts), starts[s], np.int32)
    out[s + 1:] = starts[s + 1]
    return out


def accept(c, starts, counts, accepted=None, extra=()):
    """The plain form: sequences that move rows into shared pages, or would end in one that is not full, get pages of
    their own for them (the lowest free ones, by sequence, then position; none of them where there are too few)."""
    before, wants = c.refs.copy(), {}
    for s in range(len(c.lens)):
        a, n = int(starts[s]), int(starts[s + 1] - starts[s])
        if n <= 0:
            continue
        keep, now = int(counts[s]), int(c.lens[s]) - n + int(counts[s])
        if keep == n:
            wants[s] = []
            continue
        rows = np.arange(keep) if accepted is None else accepted[a:a + keep]
        stay = int((rows == np.arange(keep)).sum())
        first = now - keep + stay if stay < keep else now - 1 if now % c.page else now
        wants[s] = [j for j in range(first // c.page, -(-now // c.page)) if before[c.table[s, j]] > 1]
    free = list(np.nonzero(before == 0)[0])
    short = sum(map(len, wants.values())) > len(free)
    for s, pages in wants.items():
        if short and pages:
            continue
        for j in pages:
            old, new = c.table[s, j], free.pop(0)
            c.copy_pages([old], [new])
            for x in extra:
                x[new] = x[old]
            c.table[s, j], c.refs[new] = new, 1
            c.refs[old] -= 1
        view.accept(c, only(starts, s), counts, accepted)
    return 1 if short else 0


def forked(rng, parents, page=16, heads=2, dim=64, pages=60, seqs=None, shape=()):
    """Sequences of the lengths `parents`, and room for children; their device cache with an extra pool."""
    lens = list(parents) + [0] * ((seqs or 2 * len(parents)) - len(parents))
    c = ref.random_cache(rng, pages, heads, page, dim, lens, 30)
    return c, rng.integers(0, 256, (pages,) + shape).astype(np.uint8)


def on_device(c, extra, mqa):  # noqa: F811
    import torch
    return ref.to_device(c, mqa, extra=(torch.from_numpy(extra.copy()).cuda(),))


def same(c, extra, dev):
    """Names of what differs.  The two NaN codes count as one: rows that were reserved and never written may hold either,
    and one that is rounded anew loses its sign."""
    pairs = {n: (getattr(c, n), getattr(dev, n).cpu().numpy()) for n in "kv"}
    codes = [n for n, (a, b) in pairs.items() if not np.array_equal(*(np.where(x == 255, 127, x) for x in (a, b)))]
    return codes + [n for n in ref.same(c, dev) if n not in pairs] + (
        [] if np.array_equal(dev.extra[0].cpu().numpy(), extra) else ["extra"])


@pytest.mark.parametrize("page,heads,dim", [(16, 2, 64), (64, 1, 128), (128, 3, 64)])
@pytest.mark.parametrize("who", [0, 1])
def test_a_roll_back_into_a_shared_page(mqa, page, heads, dim, who):  # noqa: F811
    """Fork at a page's end, roll one of the two back into the last page, go on with it: the other keeps its codes."""
    rng = np.random.default_rng(page + who)
    c, extra = forked(rng, [2 * page], page, heads, dim, shape=(7,))
    assert c.fork(np.array([0]), np.array([1])) == 0
    dev, other = on_device(c, extra, mqa), 1 - who
    held = [[c.values(other, h, w).copy() for h in range(heads)] for w in "kv"]
    st = np.array([0, 5, 5] if who == 0 else [0, 0, 5], np.int32)
    mqa.kv_accept(dev, ints(st), ints([0, 0]), rows=5)
    assert mqa.kv_status(dev) == 0 and accept(c, st, np.zeros(2, np.int32), extra=(extra,)) == 0
    assert same(c, extra, dev) == []
    assert c.table[0, 1] != c.table[1, 1] and c.table[0, 0] == c.table[1, 0]
    add = np.zeros(2, np.int32)
    add[who] = 5
    mqa.kv_reserve(dev, ints(add))
    assert c.reserve(add) == 0
    k, kd = rows_of(rng, 5, heads, dim, "bf16", 1e4)  # a larger scale for the page
    mqa.kv_append(dev, k, k, ints(st))
    c.append(kd, kd, st)
    assert same(c, extra, dev) == [] and mqa.kv_status(dev) == 0
    for w, rows in zip("kv", held):
        assert all(np.array_equal(c.values(other, h, w), x, equal_nan=True) for h, x in enumerate(rows))


def test_what_ends_with_a_page_or_keeps_everything_stays_shared(mqa):  # noqa: F811
    rng = np.random.default_rng(3)
    c, extra = forked(rng, [48, 64])
    assert c.fork(np.array([0, 1]), np.array([2, 3])) == 0
    dev = on_device(c, extra, mqa)
    for rows, counts in (([20, 0, 0, 9], [4, 0, 0, 9]), ([0, 0, 32, 0], [0, 0, 0, 0]), ([0, 64, 0, 0], [0, 0, 0, 0])):
        st = starts_of(rows)
        mqa.kv_accept(dev, ints(st), ints(counts), rows=int(st[-1]))
        assert accept(c, st, np.array(counts)) == 0
        assert same(c, extra, dev) == [] and mqa.kv_status(dev) == 0
    assert c.table[0, 0] == c.table[2, 0] and (c.refs <= 2).all() and c.lens.tolist() == [32, 0, 16, 64]


def test_rows_that_move_into_shared_pages(mqa):  # noqa: F811
    """A list that moves rows through several shared pages, from shared pages."""
    rng = np.random.default_rng(4)
    c, extra = forked(rng, [160], heads=3, shape=(3, 5))
    assert c.fork(np.array([0]), np.array([1])) == 0
    dev = on_device(c, extra, mqa)
    held = [c.values(1, h, "v").copy() for h in range(3)]
    st = np.array([0, 100, 100], np.int32)
    rows = np.sort(np.concatenate([np.arange(10), rng.choice(np.arange(11, 100), 60, replace=False)]))
    accepted, counts = np.concatenate([rows, np.zeros(30)]).astype(np.int32), np.array([70, 0], np.int32)
    mqa.kv_accept(dev, ints(st), ints(counts), ints(accepted))
    assert accept(c, st, counts, accepted, (extra,)) == 0
    assert same(c, extra, dev) == [] and mqa.kv_status(dev) == 0
    assert all(np.array_equal(c.values(1, h, "v"), x) for h, x in enumerate(held))
    assert (c.table[0, :4] == c.table[1, :4]).all() and (c.table[0, 4:9] != c.table[1, 4:9]).all()


def test_both_of_a_pair_in_one_call(mqa):  # noqa: F811
    """Counts are those before the call, whichever sequence is served first: one keeps part of a shared page that the
    other gives back, keeps part of as well, or moves rows into."""
    rng = np.random.default_rng(5)
    for rows, counts in (([20, 40], [3, 0]), ([40, 20], [0, 3]), ([20, 20], [3, 7]), ([30, 30], [5, 12])):
        for lists in (False, True):
            c, extra = forked(rng, [64], shape=(4,))
            assert c.fork(np.array([0]), np.array([1])) == 0
            dev, st = on_device(c, extra, mqa), starts_of(rows)
            accepted = None
            if lists:
                accepted = np.concatenate([np.sort(rng.choice(n, n, replace=False)) for n in rows]).astype(np.int32)
                for s, k in enumerate(counts):
                    accepted[st[s]:st[s] + k] = np.sort(rng.choice(rows[s], k, replace=False))
            for _ in range(3):
                mqa.kv_accept(dev, ints(st), ints(counts), None if accepted is None else ints(accepted), rows=int(st[-1]))
                assert accept(c, st, np.array(counts), accepted, (extra,)) == 0
                assert same(c, extra, dev) == [] and mqa.kv_status(dev) == 0
                mqa.kv_reserve(dev, ints(np.array(rows) - counts))
                assert c.reserve(np.array(rows) - counts) == 0


def test_too_few_free_pages(mqa):  # noqa: F811
    """None of the sequences that need a page is changed then; the others are served."""
    rng = np.random.default_rng(6)
    c, extra = forked(rng, [32, 32, 40], pages=9)
    assert c.fork(np.array([0, 1]), np.array([3, 4])) == 0  # 7 pages used, 2 free
    c.lens[5] = 0
    dev = on_device(c, extra, mqa)
    rows = [3, 3, 9, 3, 0, 0]  # sequences 0, 1 and 3 need a page each
    st, counts = starts_of(rows), np.array([1, 1, 2, 2, 0, 0], np.int32)
    mqa.kv_accept(dev, ints(st), ints(counts), rows=int(st[-1]))
    assert accept(c, st, counts, extra=(extra,)) == 1
    assert same(c, extra, dev) == [] and mqa.kv_status(dev) == 1
    assert c.lens.tolist() == [32, 32, 33, 32, 32, 0]
    counts[3] = 3  # now two of them do
    mqa.kv_accept(dev, ints(st[:3].tolist() + [6, 9, 9, 9]), ints(counts), rows=9)
    assert accept(c, np.array(st[:3].tolist() + [6, 9, 9, 9]), counts, extra=(extra,)) == 0
    assert same(c, extra, dev) == [] and mqa.kv_status(dev) == 0


def test_a_refused_list_takes_no_page(mqa):  # noqa: F811
    rng = np.random.default_rng(7)
    c, extra = forked(rng, [48, 48])
    assert c.fork(np.array([0, 1]), np.array([2, 3])) == 0
    dev = on_device(c, extra, mqa)
    st = starts_of([20, 20, 0, 0])
    accepted = np.zeros(40, np.int32)
    accepted[:3], accepted[20:23] = [5, 4, 9], [1, 7, 19]
    mqa.kv_accept(dev, ints(st), ints([3, 3, 0, 0]), ints(accepted))
    assert mqa.kv_status(dev) == 4
    assert accept(c, only(st, 1), np.array([0, 3, 0, 0]), accepted, (extra,)) == 0
    assert same(c, extra, dev) == []


@pytest.mark.parametrize("seed", range(6))
def test_any_forks_and_calls(mqa, seed):  # noqa: F811
    """Families of forks, then calls with and without lists, room for new rows in between."""
    rng = np.random.default_rng(100 + seed)
    page = (16, 32, 64)[seed % 3]
    n = 5
    c, extra = forked(rng, rng.integers(1, 5 * page, n), page, 1 + seed % 2, (64, 128)[seed // 3], pages=150, seqs=4 * n,
                      shape=(1 + 15 * (seed % 2),))
    dev = on_device(c, extra, mqa)
    for first in (n, 2 * n, 3 * n):
        parents = rng.integers(0, first, n)
        at = rng.integers(0, 2, n) * n  # half of them forks of forks
        parents = np.where(parents < at + n, parents, parents % n).astype(np.int32)
        children = np.arange(first, first + n, dtype=np.int32)
        mqa.kv_fork(dev, ints(parents), ints(children))
        free = np.nonzero(c.refs == 0)[0]
        part = [int(p) for p in parents if c.lens[p] % page]
        assert c.fork(parents, children) == 0
        for old, new in zip([c.table[p, c.lens[p] // page] for p in part], free):
            extra[new] = extra[old]
    for step in range(6):
        rows = np.array([int(rng.integers(0, k + 1)) if rng.random() < 0.7 else 0 for k in c.lens], np.int32)
        counts, accepted = view.random_accepted(rng, rows)
        st = starts_of(rows)
        if step % 2:
            accepted = None
        mqa.kv_accept(dev, ints(st), ints(counts), None if accepted is None else ints(accepted), rows=int(st[-1]))
        assert accept(c, st, counts, accepted, (extra,)) == mqa.kv_status(dev)
        assert same(c, extra, dev) == [], step
        add = rng.integers(0, 2 * page, len(c.lens)).astype(np.int32)
        mqa.kv_reserve(dev, ints(add))
        assert c.reserve(add) == 0 and same(c, extra, dev) == []
        k, kd = rows_of(rng, int(add.sum()), c.heads, c.dim, "bf16", 10.0 ** step)
        mqa.kv_append(dev, k, k, ints(starts_of(add)))
        c.append(kd, kd, starts_of(add))
        assert same(c, extra, dev) == [] and mqa.kv_status(dev) == 0


def test_in_a_graph(mqa):  # noqa: F811
    """One captured call, replayed as lengths, counts and sharing change; with and without pages to copy."""
    import torch
    rng = np.random.default_rng(8)
    c, extra = forked(rng, [64, 50], pages=80, shape=(9,))
    dev = on_device(c, extra, mqa)
    st, counts, accepted = starts_of([10, 10, 10, 10]), np.zeros(4, np.int32), np.zeros(40, np.int32)
    sd, cd, ad = ints(st), ints(counts), ints(accepted)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.kv_accept(dev, sd, cd, ad)
    fork = np.array([0, 1]), np.array([2, 3])
    for i in range(8):
        if i % 2 == 0:
            mqa.kv_free(dev, ints([2, 3]))
            c.free([2, 3])
            mqa.kv_fork(dev, ints(fork[0]), ints(fork[1]))
            free = np.nonzero(c.refs == 0)[0]
            part = [c.table[p, c.lens[p] // 16] for p in fork[0] if c.lens[p] % 16]
            assert c.fork(*fork) == 0
            for old, new in zip(part, free):
                extra[new] = extra[old]
        counts, accepted = view.random_accepted(rng, [10] * 4)
        cd.copy_(ints(counts))
        ad.copy_(ints(accepted))
        graph.replay()
        assert accept(c, st, counts, accepted, (extra,)) == 0
        assert same(c, extra, dev) == [] and mqa.kv_status(dev) == 0, i
        add = 10 - counts
        mqa.kv_reserve(dev, ints(add))
        assert c.reserve(add) == 0
        if i % 2:  # whole pages behind them, so that the next forks share what the next calls leave
            add = (16 - c.lens % 16) % 16
            mqa.kv_reserve(dev, ints(add))
            assert c.reserve(add) == 0


def test_among_as_many_sequences_as_there_may_be(mqa):  # noqa: F811
    rng = np.random.default_rng(9)
    n = 65536
    lens = np.zeros(n, np.int64)
    pick = np.sort(rng.choice(n, 60, replace=False))
    parents, children = pick[::2], pick[1::2]
    lens[parents] = 16 * rng.integers(1, 4, 30)
    c = ref.random_cache(rng, 250, 1, 16, 64, lens, 6)
    assert c.fork(parents, children) == 0
    extra = rng.integers(0, 256, (250, 3)).astype(np.uint8)
    dev = on_device(c, extra, mqa)
    rows = np.zeros(n, np.int64)
    rows[pick] = rng.integers(0, 17, 60)
    st = starts_of(rows)
    counts, accepted = view.random_accepted(rng, rows)
    mqa.kv_accept(dev, ints(st), ints(counts), ints(accepted))
    assert accept(c, st, counts, accepted, (extra,)) == 0
    assert same(c, extra, dev) == [] and mqa.kv_status(dev) == 0
