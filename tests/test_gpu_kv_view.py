"""Windows and trees over the paged 8-bit cache, the trees' masks and accepted rows, against plain 64-bit forms."""
import numpy as np
import pytest

import kv_reference as ref
import view_reference as view
from test_gpu_kv import check, ints, mqa, rows_of, starts_of  # noqa: F401

pytestmark = pytest.mark.gpu


def attend(mqa, c, rng, rows, group, dtype="bf16", max_rows=None, extra_rows=0, mask=None, only=None,  # noqa: F811
           **sees):
    """only: how many rows of each sequence are compared (its first and last among them)."""
    import torch
    st = starts_of(rows)
    m, n = int(st[-1]), int(st[-1]) + extra_rows
    q, qd = rows_of(rng, n, c.heads * group, c.dim, dtype)
    dev = ref.to_device(c, mqa)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    if mask is not None:
        wide = np.concatenate([mask, np.full((extra_rows, mask.shape[1]), -1, np.int32)])
        mqa.kv_attention(q, dev, ints(st), tree=ints(wide), max_rows=max_rows, out=out, lse=lse)
        seen = view.tree_seen(c, st, mask)
    else:
        mqa.kv_attention(q, dev, ints(st), max_rows=max_rows, out=out, lse=lse, **sees)
        seen = view.window_seen(c, st, sees["window"], sees.get("sinks", 0))
    assert mqa.kv_status(dev) == 0
    assert (out[m:] == 7).all() and (lse[m:] == 7).all()  # rows behind the last sequence
    pick, part = np.arange(m), st
    if only is not None:
        at = [np.unique(np.concatenate([rng.integers(0, n, only), np.arange(n)[:3], np.arange(n)[-3:]])) if n else
              np.arange(0) for n in rows]
        pick, part = np.concatenate([a + s for a, s in zip(at, st)]), starts_of([len(a) for a in at])
    check(out[pick], lse[pick], c.attention(qd[pick], part, c.dim ** -0.5, dtype, seen[pick], causal=False))
    return out, lse, dev, q, st


LITTLE = 10 ** 7  # rows x query heads x positions seen: views of more go to the tiled kernel


CASES = [  # page, heads, group, dim, lens, rows
    (16, 1, 1, 128, [1], [1]),
    (64, 2, 4, 128, [0, 1, 63, 64, 65, 700], [1, 1, 1, 1, 1, 1]),
    (32, 2, 8, 64, [0, 5, 333, 0], [0, 3, 2, 1]),
    (16, 3, 3, 64, [100, 257], [5, 7]),
    (128, 1, 16, 128, [129, 1000], [1, 2]),
    (64, 2, 5, 128, [700], [9]),
    (32, 2, 2, 128, [2, 40], [5, 40]),            # more rows than positions
    (64, 1, 4, 128, [130, 77, 64], [130, 77, 1]),
    (16, 2, 8, 128, [700], [70]),
    (128, 1, 3, 64, [400, 0, 90, 513], [200, 0, 90, 9]),
    (64, 2, 1, 128, [1500], [600]),
    (64, 1, 7, 64, [100, 260], [150, 200]),
    (16, 3, 5, 64, [257, 256, 255], [255, 256, 100]),
]
WINDOWS = [(1, 0), (1, 1), (16, 0), (64, 4), (100, 17), (128, 128), (300, 0), (257, 200), (5000, 3), (7, 5000),
           (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_window(mqa, case, window, sinks):  # noqa: F811
    page, heads, group, dim, lens, rows = case
    rng = np.random.default_rng(len(lens) * 100 + group + window % 1000)
    c = ref.random_cache(rng, sum(-(-n // page) for n in lens) + 2, heads, page, dim, lens, 100)
    dtype = "bf16" if (window + dim) % 3 else "fp16"
    attend(mqa, c, rng, rows, group, dtype, extra_rows=3, window=window, sinks=sinks)
    attend(mqa, c, rng, rows, group, dtype, max_rows=1, window=window, sinks=sinks)  # every sequence on the split kernel


TILED = [  # page, heads, group, dim, lens, rows
    (16, 2, 8, 128, [2500, 900], [1400, 900]),
    (64, 1, 4, 64, [3000], [2900]),
    (128, 3, 5, 128, [1700, 1000, 130], [1000, 700, 1]),
    (32, 1, 7, 64, [1200, 2000], [1500, 1000]),   # more rows than positions
]


@pytest.mark.parametrize("window,sinks", WINDOWS + [(700, 3), (900, 400)])
@pytest.mark.parametrize("case", TILED, ids=str)
def test_window_in_the_tiled_kernel(mqa, case, window, sinks):  # noqa: F811
    page, heads, group, dim, lens, rows = case
    assert sum(rows) * heads * group * max(rows) > LITTLE
    rng = np.random.default_rng(len(lens) * 100 + group + window % 1000)
    c = ref.random_cache(rng, sum(-(-n // page) for n in lens) + 2, heads, page, dim, lens, 200)
    attend(mqa, c, rng, rows, group, "bf16" if (window + dim) % 3 else "fp16", extra_rows=3, only=20, window=window,
           sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(1000, 4), (4096, 0), (129, 300)])
@pytest.mark.parametrize("rows", [1, 8, 300, 2400])
def test_window_far_behind_the_first_positions(mqa, rows, window, sinks):  # noqa: F811
    rng = np.random.default_rng(rows + window)
    c = ref.random_cache(rng, 200, 1, 64, 128, [9001, 2500], 160)
    attend(mqa, c, rng, [rows, 2 * rows // 3], 4, only=40, window=window, sinks=sinks)


@pytest.mark.parametrize("rows,max_rows", [([9, 1], 1), ([1100, 40], None)])
def test_a_window_as_long_as_the_sequences_is_no_window(mqa, rows, max_rows):  # noqa: F811
    """What the call without one gives: in the split kernel bit by bit.  (The tiled kernel cuts the keys of windows in
    other places, whose sums are added in another order: there every score is the same, and so are the largest ones, so
    the logarithms of the sums differ by what the order of at most 1,300 fp32 additions of up to 1 can do.)"""
    import torch
    rng = np.random.default_rng(5)
    c = ref.random_cache(rng, 100, 2, 16, 128, [1300, 200], 90)
    out, lse, dev, q, st = attend(mqa, c, rng, rows, 4, window=1300, max_rows=max_rows, only=20)
    l2 = torch.zeros_like(lse)
    o2 = mqa.kv_attention(q, dev, ints(st), max_rows=max_rows, lse=l2)
    if max_rows == 1:
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert ((lse - l2).abs() <= 1300 * 2.0 ** -23 + lse.abs() * 2.0 ** -21).all()


def test_nan_codes_outside_a_window(mqa):  # noqa: F811
    """A NaN key or value counts for the rows whose window holds it, in tiles that other rows see as well."""
    for rows in ([6, 5], [1100, 1000]):
        for window, sinks in ((20, 0), (20, 3)):
            rng = np.random.default_rng(14)
            c = ref.random_cache(rng, 150, 2, 16, 128, [1170, 1140], 80)
            c.v[c.table[0, 1150 // 16], 0, 1150 % 16, 3] = 127
            c.k[c.table[1, 1120 // 16], 1, 1120 % 16, 100] = 255
            if sinks:
                c.v[c.table[1, 0], 0, 1, 0] = 127
            out, _, _, _, st = attend(mqa, c, rng, rows, 4, window=window, sinks=sinks, only=60)
            o, a, b = out.isnan().any(2).cpu().numpy(), int(st[1]), int(st[2])
            sees = np.arange(1170 - rows[0], 1170)
            assert np.array_equal(o[:a, 0], (sees >= 1150) & (sees < 1170)) and not o[:a, 4:].any()
            sees = np.arange(1140 - rows[1], 1140)
            assert np.array_equal(o[a:b, 4], sees >= 1120) and o[a:b, 0].all() == (sinks > 0)


def test_a_window_over_bad_tables(mqa):  # noqa: F811
    """Pages that no row's window needs are not looked at; one that is needed and outside the pool is not followed."""
    rng = np.random.default_rng(17)
    for n, heads in ((2, 8), (60, 8), (1200, 8)):
        length = n + 240
        c = ref.random_cache(rng, 100, 2, 16, 64, [length], 100)
        dev = ref.to_device(c, mqa)
        dev.page_table[0, 3:9] = 1 << 30
        q, qd = rows_of(rng, n, heads, 64, "fp16")
        st, pick = np.array([0, n]), np.unique(rng.integers(0, n, 40))
        part = np.array([0, len(pick)])
        got = mqa.kv_attention(q, dev, ints(st), window=90, sinks=20)
        assert mqa.kv_status(dev) == 0
        seen = view.window_seen(c, st, 90, 20)
        check(got[pick], None, c.attention(qd[pick], part, 0.125, "fp16", seen[pick], causal=False))
        dev.page_table[0, (length - 20) // 16] = -5
        seen[seen // 16 == (length - 20) // 16] = -1
        got = mqa.kv_attention(q, dev, ints(st), window=90, sinks=20)
        assert mqa.kv_status(dev) == 2
        check(got[pick], None, c.attention(qd[pick], part, 0.125, "fp16", seen[pick], causal=False))


TREES = CASES + [(64, 2, 4, 128, [1000, 900], [64, 37]), (16, 1, 1, 64, [400], [333]), (32, 1, 32, 128, [500], [12])]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", TREES, ids=str)
def test_tree(mqa, case, dtype):  # noqa: F811
    page, heads, group, dim, lens, rows = case
    rng = np.random.default_rng(len(lens) * 100 + group)
    c = ref.random_cache(rng, sum(-(-n // page) for n in lens) + 2, heads, page, dim, lens, 100)
    parents = view.random_parents(rng, rows)
    mask, _ = view.tree_mask(c, starts_of(rows), parents, -(-max(rows) // 32))
    attend(mqa, c, rng, rows, group, dtype, mask=mask, extra_rows=3)
    attend(mqa, c, rng, rows, group, dtype, mask=mask, max_rows=1)
    # a table long enough for the tiled kernel
    c.table = np.concatenate([c.table, np.full((len(lens), LITTLE // (sum(rows) * heads * group * page) + 1), -1,
                                               np.int32)], 1)
    attend(mqa, c, rng, rows, group, dtype, mask=mask, extra_rows=3, only=30)


@pytest.mark.parametrize("max_rows", [1, None])
@pytest.mark.parametrize("words", [1, 2, 5])
def test_tree_masks_of_any_kind(mqa, words, max_rows):  # noqa: F811
    """Random bits (later rows and rows behind the sequence's last among them), no bit at all, too few words."""
    rng = np.random.default_rng(words)
    c = ref.random_cache(rng, 60, 2, 16, 64, [0, 100, 7, 300], 20 if words == 2 else 2000)
    rows = [3, 70, 7, 40]  # sequence 0 has no positions, sequence 2 none before its rows
    mask = rng.integers(-2 ** 31, 2 ** 31, (120, words)).astype(np.int32)
    mask[5] = 0
    mask[74:77] = 0
    out, lse, *_ = attend(mqa, c, rng, rows, 4, mask=mask, max_rows=max_rows)
    assert not out[:3].any() and not out[74:77].any() and lse[74:77].isneginf().all()


def test_a_chain_is_causal(mqa):  # noqa: F811
    """Rows that hang on the one before them see what they see without a mask."""
    rng = np.random.default_rng(9)
    c = ref.random_cache(rng, 40, 2, 16, 128, [300, 200], 30)
    rows = [40, 33]
    parents = np.concatenate([np.arange(n) - 1 for n in rows])
    mask, pos = view.tree_mask(c, starts_of(rows), parents, 2)
    assert np.array_equal(pos, np.concatenate([np.arange(260, 300), np.arange(167, 200)]))
    out, _, dev, q, st = attend(mqa, c, rng, rows, 4, mask=mask)
    check(mqa.kv_attention(q, dev, ints(st)), None, c.attention(q.double().cpu().numpy(), st, 128 ** -0.5, "bf16"))


def test_tree_nan_codes(mqa):  # noqa: F811
    """A drafted row with a NaN value counts for the rows that hang on it."""
    rng = np.random.default_rng(10)
    for rows in ([6, 4], [60, 50]):
        c = ref.random_cache(rng, 40, 2, 16, 128, [200, 150], 1000)
        p = 200 - rows[0] + 2
        c.v[c.table[0, p // 16], 1, p % 16, 9] = 127
        parents = view.random_parents(rng, rows)
        mask, _ = view.tree_mask(c, starts_of(rows), parents, 2)
        attend(mqa, c, rng, rows, 4, mask=mask)


def test_least_alignment_of_masks_and_strided_rows(mqa):  # noqa: F811
    import torch
    rng = np.random.default_rng(11)
    c = ref.random_cache(rng, 40, 2, 16, 64, [200], 13)
    for n in (5, 50):
        wide = torch.from_numpy(rng.standard_normal((n, 12, 64))).to(torch.bfloat16).cuda()
        q, st = wide[:, 2:10], np.array([0, n])
        mask, _ = view.tree_mask(c, st, view.random_parents(rng, [n]), 2)
        odd = torch.zeros(2 * n + 1, dtype=torch.int32, device="cuda")[1:].view(n, 2)
        odd.copy_(ints(mask))
        dev = ref.to_device(c, mqa)
        qd = q.double().cpu().numpy()
        check(mqa.kv_attention(q, dev, ints(st), tree=odd), None,
              c.attention(qd, st, 0.125, "bf16", view.tree_seen(c, st, mask), causal=False))
        check(mqa.kv_attention(q, dev, ints(st), window=60, sinks=2), None,
              c.attention(qd, st, 0.125, "bf16", view.window_seen(c, st, 60, 2)))


# ---------------------------------------------------------------- masks
@pytest.mark.parametrize("rows", [[1], [5, 0, 33], [64] * 7, [300, 2, 1], [1500, 40]], ids=str)
def test_masks_and_positions(mqa, rows):  # noqa: F811
    import torch
    rng = np.random.default_rng(sum(rows))
    lens = [n + int(rng.integers(0, 50)) for n in rows]
    c = ref.random_cache(rng, sum(-(-n // 16) for n in lens) + 2, 1, 16, 64, lens, 200)
    dev, st = ref.to_device(c, mqa), starts_of(rows)
    parents = view.random_parents(rng, rows)
    for max_rows in (max(rows), 32, 700):
        mask, pos = mqa.kv_tree_mask(dev, ints(parents), ints(st), max_rows)
        want = view.tree_mask(c, st, parents, -(-max_rows // 32))
        assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(pos.cpu().numpy(), want[1])
    # rows of no sequence are left alone; bounds that leave the rows are cut to them
    n = int(st[-1])
    held = torch.full((n + 3, 2), 5, dtype=torch.int32, device="cuda")
    pos = torch.full((n + 3,), 5, dtype=torch.int32, device="cuda")
    more = np.concatenate([[0, 0], parents, [9]]).astype(np.int32)
    mqa.kv_tree_mask(dev, ints(more), ints(st + 2), 64, mask=held, positions=pos)
    want = view.tree_mask(c, st, parents, 2)
    assert np.array_equal(held[2:-1].cpu().numpy(), want[0]) and np.array_equal(pos[2:-1].cpu().numpy(), want[1])
    assert (held[:2] == 5).all() and (held[-1] == 5).all() and (pos[:2] == 5).all() and pos[-1] == 5
    assert mqa.kv_status(dev) == 0


def test_parents_that_are_no_earlier_rows(mqa):  # noqa: F811
    rng = np.random.default_rng(3)
    c = ref.random_cache(rng, 10, 1, 16, 64, [50], 5)
    dev, st = ref.to_device(c, mqa), np.array([0, 6])
    for bad in (3, 5, 2 ** 31 - 1, -2, -2 ** 31):
        parents = np.array([-1, 0, 1, bad, 3, 1], np.int32)
        mask, pos = mqa.kv_tree_mask(dev, ints(parents), ints(st), 6)
        assert mqa.kv_status(dev) == 2
        want = view.tree_mask(c, st, parents, 1)
        assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(pos.cpu().numpy(), want[1])


# ---------------------------------------------------------------- accepting
ACCEPT = [  # page, heads, dim, lens, rows
    (16, 1, 64, [1], [1]),
    (16, 2, 128, [40, 33, 16, 100], [7, 16, 16, 50]),
    (64, 3, 64, [200, 90, 0, 64], [64, 1, 0, 64]),
    (128, 1, 128, [500, 129], [300, 129]),
    (32, 2, 64, [333] * 9, [20] * 9),
    (16, 20, 64, [50, 21], [30, 5]),              # more heads than a CTA has warps for
    (16, 1, 128, [3001, 5], [2500, 5]),           # more rows than are looked up at once
    (128, 1, 64, [4000], [3900]),
]


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("case", ACCEPT, ids=str)
def test_accept(mqa, case, seed):  # noqa: F811
    page, heads, dim, lens, rows = case
    rng = np.random.default_rng(seed * 100 + page)
    c = ref.random_cache(rng, sum(-(-n // page) for n in lens) + 2, heads, page, dim, lens, 200, spread=1 + 3 * seed)
    dev, st = ref.to_device(c, mqa), starts_of(rows)
    counts, accepted = view.random_accepted(rng, rows)
    if seed == 3:  # everything stays
        counts = np.array(rows, np.int32)
        accepted = np.concatenate([np.arange(n) for n in rows]).astype(np.int32)
    mqa.kv_accept(dev, ints(st), ints(counts), ints(accepted))
    view.accept(c, st, counts, accepted)
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0
    mqa.kv_accept(dev, ints(st * 0), ints(counts), ints(accepted))  # no rows: nothing changes
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0


def test_accept_the_first_rows(mqa):  # noqa: F811
    """Without a list: a plain roll-back; shared pages are given back once."""
    rng = np.random.default_rng(4)
    lens, rows = [40, 33, 16, 100], [7, 16, 16, 50]
    c = ref.random_cache(rng, 30, 2, 16, 64, lens, 9)
    c.refs[c.table[3, 4]] = 2
    dev, st = ref.to_device(c, mqa), starts_of(rows)
    counts = np.array([7, 0, 0, 3], np.int32)
    mqa.kv_accept(dev, ints(st), ints(counts), rows=int(st[-1]))
    view.accept(c, st, counts)
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0


def test_roll_backs_of_many_sequences(mqa):  # noqa: F811
    """Without a list, again and again: every thread reads a sequence's length before it changes."""
    rng = np.random.default_rng(41)
    n = 700
    rows = rng.integers(0, 30, n)
    c = ref.random_cache(rng, 3 * n, 1, 16, 64, rows + rng.integers(0, 12, n), 3)
    dev, st = ref.to_device(c, mqa), starts_of(rows)
    for _ in range(20):
        counts = np.array([rng.integers(0, k + 1) for k in rows], np.int32)
        mqa.kv_accept(dev, ints(st), ints(counts), rows=int(st[-1]))
        view.accept(c, st, counts)
        assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0
        mqa.kv_reserve(dev, ints(rows - counts))
        assert c.reserve(rows - counts) == 0


def test_accept_nan_and_extreme_scales(mqa):  # noqa: F811
    """NaN codes move and set no scale; scales up to both ends of their range."""
    rng = np.random.default_rng(6)
    lens, rows = [60, 61], [30, 40]
    c = ref.random_cache(rng, 12, 2, 16, 64, lens, 5, spread=100)
    for s in (0, 1):
        p = lens[s] - 3
        c.k[c.table[s, p // 16], 0, p % 16, :7] = 127
        c.v[c.table[s, p // 16], 1, p % 16, :] = 127
    dev, st = ref.to_device(c, mqa), starts_of(rows)
    counts = np.array([20, 11], np.int32)
    accepted = np.zeros(70, np.int32)
    accepted[:20] = np.sort(rng.choice(27, 20, replace=False))
    accepted[19] = 27
    accepted[30:41] = [0, 1, 5, 7, 8, 20, 30, 35, 36, 37, 39]
    mqa.kv_accept(dev, ints(st), ints(counts), ints(accepted))
    view.accept(c, st, counts, accepted)
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0


@pytest.mark.parametrize("change,status", [
    (dict(counts=[8, 2, 1]), 4), (dict(counts=[-1, 2, 1]), 4), (dict(accepted=[1, 1, 2]), 4),
    (dict(accepted=[2, 1, 3]), 4), (dict(accepted=[-1, 0, 1]), 4), (dict(accepted=[0, 1, 7]), 4),
    (dict(len=6), 8), (dict(len=10 ** 6), 8), (dict(len=-1), 8)])
def test_a_refused_list_changes_its_sequence_not_the_others(mqa, change, status):  # noqa: F811
    rng = np.random.default_rng(7)
    c = ref.random_cache(rng, 20, 2, 16, 64, [40, 33, 20], 9)
    rows = [7, 16, 3]
    counts, accepted = np.array([3, 2, 1], np.int32), np.arange(26, dtype=np.int32) % 7
    accepted[:3], accepted[7:9], accepted[23] = [1, 3, 6], [4, 15], 2
    if "counts" in change:
        counts[:] = change["counts"]
    if "accepted" in change:
        accepted[:3] = change["accepted"]
    st = starts_of(rows)
    if "len" in change:
        c.lens[0] = change["len"]
    dev = ref.to_device(c, mqa)
    mqa.kv_accept(dev, ints(st), ints(counts), ints(accepted))
    others = st.copy()
    others[0] = 7  # sequence 0 without rows
    view.accept(c, others, counts, accepted)
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == status


def test_accept_over_bad_tables(mqa):  # noqa: F811
    """Pages outside the pool are not followed: nothing moves from them, to them or into their place."""
    rng = np.random.default_rng(8)
    c = ref.random_cache(rng, 20, 1, 16, 64, [60, 60], 6)
    dev, st = ref.to_device(c, mqa), np.array([0, 40, 80])
    dev.page_table[0, 2] = 99
    dev.page_table[1, 3] = -1
    accepted = np.concatenate([np.arange(0, 40, 3), np.zeros(26), np.arange(1, 40, 2), np.zeros(20)]).astype(np.int32)
    before = dev.page_table.clone()
    mqa.kv_accept(dev, ints(st), ints([14, 20]), ints(accepted))
    assert mqa.kv_status(dev) == 2 and dev.seq_lens.tolist() == [34, 40]
    assert (dev.page_table[:, :2] == before[:, :2]).all() and (dev.page_table[:, 3] == -1).all()


# ---------------------------------------------------------------- together
def test_a_speculative_step(mqa):  # noqa: F811
    """Prompt; then rounds of: room for a draft, its masks and positions, rotated heads appended and attended, what was
    accepted taken over.  Against the plain forms, and the kept rows against a cache that never held the others."""
    import torch
    rng = np.random.default_rng(20)
    heads, group, dim, page = 2, 4, 64, 16
    c = ref.random_cache(rng, 40, heads, page, dim, [0, 0], 16, garbage=False)
    dev = ref.to_device(c, mqa)
    turns = mqa.rope_turns(10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim))
    ws = mqa.alloc_kv_workspace(dev, 100, heads * group)
    for step, rows in enumerate(([37, 50], [9, 13], [16, 1], [5, 20])):
        st, n = starts_of(rows), sum(rows)
        mqa.kv_reserve(dev, ints(rows))
        assert c.reserve(np.array(rows)) == 0
        parents = view.random_parents(rng, rows) if step else np.concatenate([np.arange(k) - 1 for k in rows])
        mask, pos = mqa.kv_tree_mask(dev, ints(parents), ints(st), max(rows))
        want = view.tree_mask(c, st, parents, mask.shape[1])
        assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(pos.cpu().numpy(), want[1])
        qkv, _ = rows_of(rng, n, heads * (group + 2), dim, "bf16")
        q, k = mqa.qk_norm_rope(qkv[:, :heads * group], qkv[:, heads * group:heads * (group + 1)], turns, pos)
        v = qkv[:, heads * (group + 1):]
        mqa.kv_append(dev, k, v, ints(st))
        c.append(k.double().cpu().numpy(), v.double().cpu().numpy(), st)
        assert ref.same(c, dev) == []
        qd = q.double().cpu().numpy()
        got = mqa.kv_attention(q, dev, ints(st), tree=mask, max_rows=max(rows), workspace=ws)
        check(got, None, c.attention(qd, st, dim ** -0.5, "bf16", view.tree_seen(c, st, want[0]), causal=False))
        got = mqa.kv_attention(q, dev, ints(st), window=20, sinks=2, max_rows=max(rows), workspace=ws)
        check(got, None, c.attention(qd, st, dim ** -0.5, "bf16", view.window_seen(c, st, 20, 2)))
        if step:  # a path from a random row up
            counts, accepted = np.zeros(2, np.int32), np.zeros(n, np.int32)
            for s, r in enumerate(rows):
                path, at = [], int(rng.integers(0, r))
                while at >= 0:
                    path.append(at)
                    at = int(parents[st[s] + at])
                counts[s] = len(path)
                accepted[st[s]:st[s] + len(path)] = path[::-1]
            mqa.kv_accept(dev, ints(st), ints(counts), ints(accepted))
            view.accept(c, st, counts, accepted)
            assert ref.same(c, dev) == []
    assert mqa.kv_status(dev) == 0


def test_a_speculative_step_in_a_graph(mqa):  # noqa: F811
    """Reserve, masks, attention in both forms and acceptance captured once, replayed with other contents."""
    import torch
    rng = np.random.default_rng(21)
    heads, group, dim, page = 2, 4, 64, 16
    c = ref.random_cache(rng, 60, heads, page, dim, [30, 100], 30)
    dev = ref.to_device(c, mqa)
    rows = np.array([12, 20], np.int32)
    st, n = starts_of(rows), 32
    drows, dst = ints(rows), ints(st)
    q, k, v = (torch.zeros((n, h, dim), dtype=torch.bfloat16, device="cuda") for h in (heads * group, heads, heads))
    parents, counts, accepted = ints(np.zeros(n) - 1), ints([0, 0]), ints(np.zeros(n))
    mask, pos = ints(np.zeros((n, 1))), ints(np.zeros(n))
    ws = [mqa.alloc_kv_workspace(dev, n, heads * group) for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(2)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        mqa.kv_reserve(dev, drows)
        mqa.kv_tree_mask(dev, parents, dst, 32, mask=mask, positions=pos)
        mqa.kv_append(dev, k, v, dst)
        mqa.kv_attention(q, dev, dst, tree=mask, workspace=ws[0], out=outs[0])
        mqa.kv_attention(q, dev, dst, window=40, sinks=4, workspace=ws[1], out=outs[1])
        mqa.kv_accept(dev, dst, counts, accepted)
    torch.cuda.synchronize()
    for i in range(8):
        qn, kn, vn = (rows_of(rng, n, h, dim, "bf16") for h in (heads * group, heads, heads))
        pn = view.random_parents(rng, rows)
        cn, an = view.random_accepted(rng, rows)
        cn = np.minimum(cn, 15)
        for t, x in ((q, qn[0]), (k, kn[0]), (v, vn[0]), (parents, ints(pn)), (counts, ints(cn)), (accepted, ints(an))):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert c.reserve(rows) == 0
        want = view.tree_mask(c, st, pn, 1)
        assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(pos.cpu().numpy(), want[1])
        c.append(kn[1], vn[1], st)
        check(outs[0], None, c.attention(qn[1], st, 0.125, "bf16", view.tree_seen(c, st, want[0]), causal=False), i)
        check(outs[1], None, c.attention(qn[1], st, 0.125, "bf16", view.window_seen(c, st, 40, 4)), i)
        view.accept(c, st, cn, an)
        assert ref.same(c, dev) == [], i
    assert mqa.kv_status(dev) == 0


def test_as_many_sequences_as_there_may_be(mqa):  # noqa: F811
    rng = np.random.default_rng(79)
    n = 65536
    lens, rows = np.zeros(n, np.int64), np.zeros(n, np.int64)
    pick = rng.choice(n, 40, replace=False)
    pick[:2] = 0, n - 1
    lens[pick] = rng.integers(1, 90, 40)
    rows[pick] = np.minimum(lens[pick], rng.integers(1, 60, 40))
    lens[pick[5]], rows[pick[5]] = 700, 300
    c = ref.random_cache(rng, 600, 1, 16, 64, lens, 45)
    st = starts_of(rows)
    attend(mqa, c, rng, rows, 4, window=33, sinks=4)
    attend(mqa, c, rng, rows, 4, "fp16", max_rows=2, window=33, sinks=4)
    parents = view.random_parents(rng, rows)
    mask, pos = view.tree_mask(c, st, parents, 10)
    _, _, dev, _, _ = attend(mqa, c, rng, rows, 4, mask=mask)
    got = mqa.kv_tree_mask(dev, ints(parents), ints(st), 300)
    assert np.array_equal(got[0].cpu().numpy(), mask) and np.array_equal(got[1].cpu().numpy(), pos)
    counts, accepted = view.random_accepted(rng, rows)
    mqa.kv_accept(dev, ints(st), ints(counts), ints(accepted))
    view.accept(c, st, counts, accepted)
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0


# ---------------------------------------------------------------- values that are hard, in every kernel
HARD = [  # heads, group, lens, rows: split kernel; tiled, halves in turns; tiled, two halves
    (2, 4, [300], [6]), (1, 4, [700, 400], [30, 25]), (1, 8, [700, 300], [60, 31])]


def both_views(mqa, c, rng, rows, group, q, qd, st, scale=None, dtype="bf16"):  # noqa: F811
    """A tree and a window call, each in the kernel that the sizes choose, and their plain answers."""
    parents = view.random_parents(rng, rows)
    mask, _ = view.tree_mask(c, st, parents, -(-max(rows) // 32))
    dev = ref.to_device(c, mqa)
    scale = c.dim ** -0.5 if scale is None else scale
    got = mqa.kv_attention(q, dev, ints(st), tree=ints(mask), scale=scale)
    yield got, c.attention(qd, st, scale, dtype, view.tree_seen(c, st, mask), causal=False)
    got = mqa.kv_attention(q, dev, ints(st), window=100, sinks=3, scale=scale)
    yield got, c.attention(qd, st, scale, dtype, view.window_seen(c, st, 100, 3))
    assert mqa.kv_status(dev) == 0


def long_tables(c, rows, group):
    """Tables so long that trees go to the tiled kernel."""
    c.table = np.concatenate([c.table, np.full((len(c.lens), LITTLE // (sum(rows) * c.heads * group * c.page) + 1), -1,
                                               np.int32)], 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", HARD, ids=str)
def test_infinite_and_nan_queries(mqa, case, dtype):  # noqa: F811
    heads, group, lens, rows = case
    rng = np.random.default_rng(30)
    c = ref.random_cache(rng, 100, heads, 16, 128, lens, 60)
    if sum(rows) > 10:
        long_tables(c, rows, group)
    st, n = starts_of(rows), sum(rows)
    q, _ = rows_of(rng, n, heads * group, 128, dtype)
    q[0, 1, 5], q[n - 1, 0, 0], q[n // 2, 2, 127] = float("nan"), float("inf"), -float("inf")
    for got, want in both_views(mqa, c, rng, rows, group, q, q.double().cpu().numpy(), st, dtype=dtype):
        check(got, None, want)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("case", HARD, ids=str)
def test_scales_far_apart_and_sharp_softmax(mqa, case, dim):  # noqa: F811
    heads, group, lens, rows = case
    rng = np.random.default_rng(31)
    st, n = starts_of(rows), sum(rows)
    c = ref.random_cache(rng, 100, heads, 16, dim, lens, 60, spread=20)
    if sum(rows) > 10:
        long_tables(c, rows, group)
    q, qd = rows_of(rng, n, heads * group, dim, "fp16")
    for got, (out, _, tol, _) in both_views(mqa, c, rng, rows, group, q, qd, st, scale=1e-6, dtype="fp16"):
        g = got.double().cpu().numpy()
        fine, past = np.abs(out) + tol < 65504, np.abs(out) - tol >= 65520  # what rounds to fp16's infinity
        assert fine.any() and (np.abs(g - out)[fine] <= tol[fine]).all()
        assert np.array_equal(g[past], np.copysign(np.inf, out[past]))
    c.ke[:] = 127
    q, qd = rows_of(rng, n, heads * group, dim, "bf16", 200.0)  # scores of thousands
    for got, want in both_views(mqa, c, rng, rows, group, q, qd, st):
        check(got, None, want)
    # values whose scales span 2^120: those within bf16's range are compared
    c.ve[:] = rng.integers(60, 180, c.ve.shape)
    q, qd = rows_of(rng, n, heads * group, dim, "bf16")
    for got, (out, _, tol, _) in both_views(mqa, c, rng, rows, group, q, qd, st, scale=0.01):
        fine = np.abs(out) < 3e38
        assert fine.any() and (np.abs(got.double().cpu().numpy() - out)[fine] <= tol[fine]).all()


@pytest.mark.parametrize("case", HARD, ids=str)
def test_a_tree_over_bad_tables(mqa, case):  # noqa: F811
    heads, group, lens, rows = case
    rng = np.random.default_rng(32)
    c = ref.random_cache(rng, 100, heads, 16, 64, lens, 60)
    if sum(rows) > 10:
        long_tables(c, rows, group)
    st, n = starts_of(rows), sum(rows)
    q, qd = rows_of(rng, n, heads * group, 64, "fp16")
    mask, _ = view.tree_mask(c, st, view.random_parents(rng, rows), 2)
    seen = view.tree_seen(c, st, mask)
    dev = ref.to_device(c, mqa)
    for col, bad in ((2, 1 << 30), (9, -5), (17, -2 ** 31)):
        dev.page_table[0, col] = bad
        seen[:rows[0]][seen[:rows[0]] // 16 == col] = -1
    got = mqa.kv_attention(q, dev, ints(st), tree=ints(mask))
    assert mqa.kv_status(dev) == 2
    check(got, None, c.attention(qd, st, 0.125, "fp16", seen, causal=False))


def test_on_streams_of_their_own(mqa):  # noqa: F811
    """Each operator on a stream that is not the current one, outputs made there; two layers' calls at once."""
    import torch
    rng = np.random.default_rng(33)
    c = ref.random_cache(rng, 60, 1, 16, 128, [400, 300], 2000)
    rows = [40, 33]
    st, n = starts_of(rows), sum(rows)
    parents = view.random_parents(rng, rows)
    want = view.tree_mask(c, st, parents, 2)
    dev, pd, sd = ref.to_device(c, mqa), ints(parents), ints(st)
    q, qd = rows_of(rng, n, 8, 128, "bf16")
    counts, accepted = view.random_accepted(rng, rows)
    cd, ad = ints(counts), ints(accepted)
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    mask, pos = mqa.kv_tree_mask(dev, pd, sd, 40, stream=sides[0])
    a = mqa.kv_attention(q, dev, sd, tree=mask, stream=sides[0])
    b = mqa.kv_attention(q, dev, sd, window=50, sinks=1, stream=sides[1])
    for s in sides:
        s.synchronize()
    assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(pos.cpu().numpy(), want[1])
    check(a, None, c.attention(qd, st, 128 ** -0.5, "bf16", view.tree_seen(c, st, want[0]), causal=False))
    check(b, None, c.attention(qd, st, 128 ** -0.5, "bf16", view.window_seen(c, st, 50, 1)))
    mqa.kv_accept(dev, sd, cd, ad, stream=sides[1])
    sides[1].synchronize()
    view.accept(c, st, counts, accepted)
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0


def test_results_do_not_depend_on_the_run(mqa):  # noqa: F811
    """The same call again and again gives the same bits, whatever ran before on its workspace."""
    import torch
    rng = np.random.default_rng(34)
    c = ref.random_cache(rng, 300, 2, 16, 128, [2000, 1500], 2000)
    rows = [30, 60]
    st, n = starts_of(rows), sum(rows)
    q, _ = rows_of(rng, n, 8, 128, "bf16")
    dev, sd = ref.to_device(c, mqa), ints(st)
    mask, _ = mqa.kv_tree_mask(dev, ints(view.random_parents(rng, rows)), sd, 60)
    ws = mqa.alloc_kv_workspace(dev, n, 8)
    first = None
    for i in range(20):
        ws.random_(0, 256)
        got = (mqa.kv_attention(q, dev, sd, tree=mask, workspace=ws), mqa.kv_attention(q, dev, sd, window=900, sinks=5,
                                                                                       workspace=ws))
        first = got if first is None else first
        assert all(torch.equal(x, y) for x, y in zip(got, first)), i


@pytest.mark.parametrize("case", HARD + [(1, 8, [1300], [1200])], ids=str)
def test_values_near_the_top_of_the_range(mqa, case):  # noqa: F811
    """Value scales of 2^118: results within bf16's range come out, also in tiles of which some keys are not needed."""
    heads, group, lens, rows = case
    rng = np.random.default_rng(35)
    c = ref.random_cache(rng, 130, heads, 16, 128, lens, 90)
    c.v[:] = ref.round_e4m3(rng.standard_normal(c.v.shape))
    c.ve[:] = 127 + 118
    if sum(rows) > 10:
        long_tables(c, rows, group)
    st, n = starts_of(rows), sum(rows)
    q, qd = rows_of(rng, n, heads * group, 128, "bf16", 0.01)
    pick = np.arange(n) if n < 1000 else np.unique(np.concatenate([np.arange(5), rng.integers(0, n, 20), [n - 1]]))
    part = st if n < 1000 else np.array([0, len(pick)])
    dev = ref.to_device(c, mqa)
    mask, _ = view.tree_mask(c, st, view.random_parents(rng, rows), -(-max(rows) // 32))
    for kw, seen in ((dict(tree=ints(mask)), view.tree_seen(c, st, mask)),
                     (dict(window=100, sinks=3), view.window_seen(c, st, 100, 3)),
                     (dict(), view.window_seen(c, st, 10 ** 6, 0))):
        got = mqa.kv_attention(q, dev, ints(st), **kw)
        check(got[pick], None, c.attention(qd[pick], part, 128 ** -0.5, "bf16", seen[pick], causal=False), sorted(kw))


# ---------------------------------------------------------------- pages outside the pool, whole tiles of them
OUTSIDE = [  # what rows see, heads, group, lens, rows: in the tiled kernel parts of several tiles, in both forms
    ("split", 1, 8, [1500, 700], [3, 1]), ("dense", 1, 8, [2600, 900], [700, 20]), ("all", 8, 8, [1700, 700], [130, 77]),
    ("window", 1, 8, [2600, 1500], [1200, 900]), ("tree", 32, 4, [3000, 700], [30, 25]),
    ("tree", 8, 8, [2900, 900], [60, 31])]


@pytest.mark.parametrize("size", ["large", "small", "low"])
@pytest.mark.parametrize("page,dim", [(16, 128), (128, 64)])
@pytest.mark.parametrize("kind,heads,group,lens,rows", OUTSIDE, ids=str)
def test_tiles_of_pages_outside_the_pool(mqa, kind, heads, group, lens, rows, page, dim, size):  # noqa: F811
    """Runs of 128 and 256 positions in pages outside the pool, the first ones among them, so that parts begin with tiles
    in which nothing is seen; in the tiled kernel as in the split one they count as not seen.  size: of the scores; low:
    about -270 in powers of two, whose weights vanish unless the references follow."""
    import torch
    rng = np.random.default_rng(page + dim + len(kind))
    n, st = sum(rows), starts_of(rows)
    c = ref.random_cache(rng, sum(-(-k // page) for k in lens) + 2, heads, page, dim, lens, 4096 // page)
    q, _ = rows_of(rng, n, heads * group, dim, "bf16", 1.5 if size == "large" else 0.003)
    scale = dim ** -0.5
    if size == "low":
        c.k[:], c.ke[:], scale = 56, 127, 1.0  # keys of 1
        q = (q - 187.0 / dim).to(torch.bfloat16)
    qd = q.double().cpu().numpy()
    pick = np.unique(np.concatenate([rng.integers(0, n, 16 if heads == 1 else 2), [0, n - 1, rows[0] - 1, rows[0]]]))
    part = np.array([0, (pick < rows[0]).sum(), len(pick)])
    if kind == "tree":
        long_tables(c, rows, group)
        mask, _ = view.tree_mask(c, st, view.random_parents(rng, rows), 2)
        kw, seen = dict(tree=ints(mask)), view.tree_seen(c, st, mask)
    elif kind == "window":
        assert n * group * max(rows) > LITTLE
        kw, seen = dict(window=400), view.window_seen(c, st, 400, 0)
    elif kind == "all":
        kw, seen = dict(causal=False), np.stack([np.where(np.arange(max(lens)) < lens[s], np.arange(max(lens)), -1)
                                                 for s, _ in enumerate(rows) for _ in range(rows[s])])
    else:
        kw, seen = dict(max_rows=1 if kind == "split" else None), view.window_seen(c, st, 10 ** 6, 0)
    for bad in (lambda t: (t >= 0) & (t < 256), lambda t: (t >= 0) & (t // 128 % 3 != 2)):
        dev = ref.to_device(c, mqa)
        at = np.arange(c.table.shape[1]) * page
        for s, k in enumerate(lens):
            dev.page_table[s, torch.from_numpy((at < k) & bad(at)).cuda()] = (1 << 30) - 3 * s
        sees = np.where(bad(seen), -1, seen)[pick]
        lse = torch.zeros((n, heads * group), device="cuda")
        got = mqa.kv_attention(q, dev, ints(st), lse=lse, scale=scale, **kw)
        assert mqa.kv_status(dev) == 2
        check(got[pick], lse[pick], c.attention(qd[pick], part, scale, "bf16", sees, causal=False), kind)


# ---------------------------------------------------------------- windows in the tiled kernel: hard values, repeated, replayed
BROAD = [  # heads, group, lens, rows: the last block has 128 columns, whose halves take turns; blocks of two full halves
    (1, 8, [1300], [1200]), (2, 4, [1500, 1400], [700, 640])]


def broad(case, window, sinks, rng, dim=128, spread=2):
    """A cache, and rows whose windows are so much work that the tiled kernel serves them; a sample of the rows."""
    heads, group, lens, rows = case
    assert sum(rows) * heads * group * min(1600, window + sinks + sum(rows)) > LITTLE
    c = ref.random_cache(rng, 200, heads, 16, dim, lens, 100, spread=spread)
    st, n = starts_of(rows), sum(rows)
    pick = np.unique(np.concatenate([np.arange(3), rng.integers(0, n, 16), [rows[0] - 1, n - 1]]))
    part = np.concatenate([[0], np.searchsorted(pick, st[1:])])
    return c, st, n, pick, part, view.window_seen(c, st, window, sinks)[pick]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", BROAD, ids=str)
def test_infinite_and_nan_queries_in_broad_windows(mqa, case, dtype):  # noqa: F811
    rng = np.random.default_rng(50)
    c, st, n, pick, part, seen = broad(case, 100, 3, rng)
    q, _ = rows_of(rng, n, c.heads * case[1], 128, dtype)
    q[0, 1, 5], q[n - 1, 0, 0], q[pick[8], 2, 127] = float("nan"), float("inf"), -float("inf")
    dev = ref.to_device(c, mqa)
    got = mqa.kv_attention(q, dev, ints(st), window=100, sinks=3)
    check(got[pick], None, c.attention(q.double().cpu().numpy()[pick], part, 128 ** -0.5, dtype, seen, causal=False))
    assert mqa.kv_status(dev) == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("case", BROAD, ids=str)
def test_scales_far_apart_and_sharp_softmax_in_broad_windows(mqa, case, dim):  # noqa: F811
    rng = np.random.default_rng(51)
    c, st, n, pick, part, seen = broad(case, 300, 20, rng, dim, spread=20)
    attention = lambda q, scale: mqa.kv_attention(q, ref.to_device(c, mqa), ints(st), window=300, sinks=20,  # noqa: E731
                                                  scale=scale)[pick]
    plain = lambda qd, scale, dtype: c.attention(qd[pick], part, scale, dtype, seen, causal=False)  # noqa: E731
    heads = c.heads * case[1]
    q, qd = rows_of(rng, n, heads, dim, "fp16")
    g, (out, _, tol, _) = attention(q, 1e-6).double().cpu().numpy(), plain(qd, 1e-6, "fp16")
    fine, past = np.abs(out) + tol < 65504, np.abs(out) - tol >= 65520  # what rounds to fp16's infinity
    assert fine.any() and (np.abs(g - out)[fine] <= tol[fine]).all()
    assert np.array_equal(g[past], np.copysign(np.inf, out[past]))
    c.ke[:] = 127
    q, qd = rows_of(rng, n, heads, dim, "bf16", 200.0)  # scores of thousands
    check(attention(q, dim ** -0.5), None, plain(qd, dim ** -0.5, "bf16"))
    # values whose scales span 2^120: those within bf16's range are compared
    c.ve[:] = rng.integers(60, 180, c.ve.shape)
    q, qd = rows_of(rng, n, heads, dim, "bf16")
    out, _, tol, _ = plain(qd, 0.01, "bf16")
    fine = np.abs(out) < 3e38
    assert fine.any() and (np.abs(attention(q, 0.01).double().cpu().numpy() - out)[fine] <= tol[fine]).all()


@pytest.mark.parametrize("case", BROAD, ids=str)
def test_broad_windows_give_the_same_bits_again(mqa, case):  # noqa: F811
    """Whatever ran on the workspace before, on two streams at once, and in a graph whose lengths and queries change."""
    import torch
    rng = np.random.default_rng(52)
    c, st, n, pick, part, seen = broad(case, 500, 5, rng)
    q, qd = rows_of(rng, n, c.heads * case[1], 128, "bf16")
    dev, sd = ref.to_device(c, mqa), ints(st)
    ws = [mqa.alloc_kv_workspace(dev, n, c.heads * case[1]) for _ in range(2)]
    call = lambda q=q, **kw: mqa.kv_attention(q, dev, sd, window=500, sinks=5, **kw)  # noqa: E731
    first = call(workspace=ws[0])
    check(first[pick], None, c.attention(qd[pick], part, 128 ** -0.5, "bf16", seen, causal=False))
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for w in ws:
            w.random_(0, 256)
        torch.cuda.synchronize()
        got = [call(workspace=w, stream=s) for w, s in zip(ws, sides)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], first) and torch.equal(got[1], first)
    held, out, graph = torch.zeros_like(q), torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(held, workspace=ws[0], out=out)
    for cut in (0, 77, 1):
        c.lens[:] -= cut
        dev.seq_lens.copy_(ints(c.lens))
        held.copy_(q)
        graph.replay()
        assert torch.equal(out, call(workspace=ws[1]))
        seen = view.window_seen(c, st, 500, 5)[pick]
        check(out[pick], None, c.attention(qd[pick], part, 128 ** -0.5, "bf16", seen, causal=False), cut)
    assert mqa.kv_status(dev) == 0


# ---------------------------------------------------------------- the waits' time limit
LIMITS = [  # what rows see, heads, group, dim, type, lens, rows: halves in turns, values staged or not, full halves
    ("tree", 1, 4, 128, "bf16", [900, 700], [30, 25]), ("tree", 1, 4, 64, "fp16", [900, 700], [30, 25]),
    ("tree", 1, 4, 128, "fp16", [900, 700], [30, 25]), ("tree", 2, 8, 64, "bf16", [900, 0, 700], [60, 0, 1]),
    ("window", 1, 8, 128, "bf16", [1300], [1200]), ("window", 2, 4, 64, "fp16", [1500, 1400], [700, 640])]


@pytest.mark.parametrize("stall", [1, 2])
@pytest.mark.parametrize("case", LIMITS, ids=str)
def test_waits_of_views_end_at_their_limit(mqa, case, stall):  # noqa: F811
    """A wait for what never comes runs out: the status says so, nothing but the outputs has changed, and the next call on
    the same workspace answers as if nothing had been."""
    import ctypes

    import torch
    from sparse_attention_indexer_relu_gb300 import kv_cache as kv
    kind, heads, group, dim, dtype, lens, rows = case
    rng = np.random.default_rng(60)
    c = ref.random_cache(rng, 220, heads, 16, dim, lens, 100)
    n, st = sum(rows), ints(starts_of(rows))
    if kind == "tree":
        long_tables(c, rows, group)
        mask = ints(view.tree_mask(c, starts_of(rows), view.random_parents(rng, rows), 2)[0])
        seen, kw = kv._View(0, 0, mask.data_ptr(), 2), dict(tree=mask)
    else:
        assert n * heads * group * min(1600, 103 + n) > LITTLE
        seen, kw = kv._View(100, 3, None, 0), dict(window=100, sinks=3)
    dev = ref.to_device(c, mqa)
    q, _ = rows_of(rng, n, heads * group, dim, dtype)
    ws = mqa.alloc_kv_workspace(dev, n, heads * group)
    ws.fill_(0xAB)
    want, got = mqa.kv_attention(q, dev, st, workspace=ws, **kw), torch.empty_like(q)
    assert mqa.kv_status(dev) == 0

    def call(**options):
        mqa._check(mqa.lib().mqa_kv_attention_view_debug(
            dev._ref, q.data_ptr(), heads * group * dim, kv._types()[q.dtype], heads * group, st.data_ptr(), n, 0,
            ctypes.byref(seen), dim ** -0.5, got.data_ptr(), None, ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream, ctypes.byref(kv.KVDebugOptions(**options))), "view")
        return mqa.kv_status(dev)

    for _ in range(2):
        assert call(stall=stall, wait_timeout_ms=30) == 16 and ref.same(c, dev) == []
        assert call(wait_timeout_ms=500) == 0 and torch.equal(got, want)
