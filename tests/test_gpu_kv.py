"""The paged 8-bit cache on the GPU, against the plain 64-bit forms of kv_reference.py."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


@pytest.fixture(scope="module")
def mqa():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_attention_indexer_relu_gb300 as m
    m.lib()
    return m


def ints(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.int32).copy()).cuda()


def rows_of(rng, n, heads, dim, dtype, scale=1.5):
    """Random rows of a type, and their values in 64 bits."""
    import torch
    t = (torch.from_numpy(rng.standard_normal((n, heads, dim))) * scale).to(getattr(torch, TYPES[dtype])).cuda()
    return t, t.double().cpu().numpy()


def starts_of(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def check(got, lse, want, what=""):
    """Against (out, lse, bound of out, bound of lse): NaN where NaN, else within the bound."""
    out, l, tol, ltol = want
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(out)), what
    bad = np.abs(np.nan_to_num(g - out)) > tol
    assert not bad.any(), (what, np.argwhere(bad)[:5], np.abs(g - out)[bad][:5], tol[bad][:5])
    if lse is not None:
        gl = lse.double().cpu().numpy()
        assert np.array_equal(np.isnan(gl), np.isnan(l)) and np.array_equal(np.isneginf(gl), np.isneginf(l)), what
        d = np.abs(np.where(np.isfinite(l), gl, 0) - np.where(np.isfinite(l), l, 0))
        assert (d <= ltol + 1e-30).all(), (what, d.max())


def attend(mqa, c, rng, rows, group, dtype="bf16", causal=True, selected=None, max_rows=None, q_scale=1.5, scale=None,
           extra_rows=0):
    import torch
    st = starts_of(rows)
    n = int(st[-1]) + extra_rows
    q, qd = rows_of(rng, n, c.heads * group, c.dim, dtype, q_scale)
    dev = ref.to_device(c, mqa)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    sel = None if selected is None else ints(selected)
    scale = c.dim ** -0.5 if scale is None else scale
    mqa.kv_attention(q, dev, ints(st), selected=sel, causal=causal, scale=scale, max_rows=max_rows, out=out, lse=lse)
    assert mqa.kv_status(dev) == 0
    m = int(st[-1])
    assert (out[m:] == 7).all() and (lse[m:] == 7).all()  # rows behind the last sequence
    want = c.attention(qd[:m], st, scale, dtype, None if selected is None else selected[:m], causal)
    check(out[:m], lse[:m], want)
    return out, dev, q, st


# ---------------------------------------------------------------- attention
CASES = [  # page, heads, group, dim, lens, rows
    (16, 1, 1, 128, [1], [1]),
    (64, 2, 4, 128, [0, 1, 63, 64, 65, 200], [1, 1, 1, 1, 1, 1]),
    (32, 2, 8, 64, [0, 5, 333, 0], [0, 3, 2, 1]),
    (16, 3, 3, 64, [100, 257], [5, 7]),
    (128, 1, 16, 128, [129, 1000], [1, 2]),
    (64, 2, 5, 128, [700], [9]),
    (64, 1, 32, 128, [300, 31], [1, 3]),
    (16, 1, 71, 64, [90], [2]),
    (32, 2, 2, 128, [2, 40], [5, 40]),          # more rows than positions: the first see nothing
    (64, 1, 4, 128, [130, 77, 64], [130, 77, 1]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention(mqa, case, dtype, causal):
    page, heads, group, dim, lens, rows = case
    rng = np.random.default_rng(len(lens) * 100 + group)
    c = ref.random_cache(rng, sum(-(-n // page) for n in lens) + 2, heads, page, dim, lens, 20)
    attend(mqa, c, rng, rows, group, dtype, causal, extra_rows=3)


@pytest.mark.parametrize("max_rows", [None, 1, 4, 100])
def test_attention_answers_for_any_max_rows(mqa, max_rows):
    rng = np.random.default_rng(7)
    c = ref.random_cache(rng, 40, 2, 16, 128, [150, 90, 33], 12)
    attend(mqa, c, rng, [40, 1, 7], 4, max_rows=max_rows)


def test_attention_long_context_is_split_and_joined(mqa):
    rng = np.random.default_rng(8)
    c = ref.random_cache(rng, 700, 1, 64, 128, [40001], 640)
    attend(mqa, c, rng, [2], 8)


def test_attention_sharp_and_flat_softmax(mqa):
    """Scores of thousands (one key takes all) and of almost zero (all alike)."""
    rng = np.random.default_rng(9)
    c = ref.random_cache(rng, 30, 2, 32, 64, [500, 300], 20)
    attend(mqa, c, rng, [2, 2], 4, "fp16", q_scale=200.0)
    attend(mqa, c, rng, [2, 2], 4, "bf16", q_scale=1e-30)


def test_attention_scales_far_apart(mqa):
    """Blocks whose scales span 2^120: keys stay within reach of the softmax, values do not."""
    rng = np.random.default_rng(10)
    c = ref.random_cache(rng, 20, 2, 16, 128, [200], 16)
    c.ve[:] = rng.integers(60, 180, c.ve.shape)
    c.ke[:] = rng.integers(90, 128, c.ke.shape)
    rng2 = np.random.default_rng(11)
    q, qd = rows_of(rng2, 3, 8, 128, "bf16")
    dev = ref.to_device(c, mqa)
    got = mqa.kv_attention(q, dev, ints([0, 3]), scale=0.01)
    want = c.attention(qd, np.array([0, 3]), 0.01, "bf16")
    out, _, tol, _ = want
    fine = np.abs(out) < 3e38  # the rest leave bf16's range
    assert fine.any() and (np.abs(got.double().cpu().numpy() - out)[fine] <= tol[fine]).all()


def test_small_scale_block_with_all_the_weight(mqa):
    """The key with all the softmax weight sits in a block whose value scale is 2^30 below the others'."""
    rng = np.random.default_rng(12)
    c = ref.random_cache(rng, 8, 1, 16, 64, [96], 8)
    c.ve[:] = 127
    c.ve[c.table[0, 2], 0] = 97
    c.k[c.table[0, 2], 0, 5] = ref.round_e4m3(np.full(64, 400.0))
    import torch
    q = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    dev = ref.to_device(c, mqa)
    got = mqa.kv_attention(q, dev, ints([0, 1]), scale=0.125)
    out, l, tol, ltol = c.attention(np.ones((1, 2, 64)), np.array([0, 1]), 0.125, "bf16")
    check(got, None, (out, l, tol, ltol))


def test_nan_codes_count_only_where_they_are_seen(mqa):
    rng = np.random.default_rng(13)
    c = ref.random_cache(rng, 20, 2, 16, 128, [100, 60], 10)
    c.v[c.table[0, 97 // 16], 0, 97 % 16, 3] = 127    # a value of position 97, head 0
    c.k[c.table[1, 58 // 16], 1, 58 % 16, 100] = 255  # a key of position 58, head 1
    for rows in ([5, 4], [100, 60]):
        out, _, _, st = attend(mqa, c, np.random.default_rng(14), rows, 4)
        o = out.float().cpu().numpy()
        first = int(st[1])
        assert np.isnan(o[first - 3:first, :4]).all() and not np.isnan(o[:first - 3]).any()
        assert not np.isnan(o[:first, 4:]).any()


def test_infinite_and_nan_queries(mqa):
    import torch
    rng = np.random.default_rng(15)
    c = ref.random_cache(rng, 20, 2, 16, 64, [100], 10)
    q, qd = rows_of(rng, 3, 8, 64, "bf16")
    q[1, 2, 5] = float("nan")
    q[2, 4, 0] = float("inf")
    out = mqa.kv_attention(q, ref.to_device(c, mqa), ints([0, 3])).float().cpu().numpy()
    qd[1, 2], qd[2, 4] = 0, 0
    want = c.attention(qd, np.array([0, 3]), 0.125, "bf16")
    assert np.isnan(out[1, 2]).all()
    keep = np.ones((3, 8), bool)
    keep[1, 2] = keep[2, 4] = False
    assert (np.abs(out - want[0])[keep] <= want[2][keep]).all() and not np.isnan(out[keep]).any()
    assert torch.cuda.current_stream() is not None


def test_strided_queries(mqa):
    import torch
    rng = np.random.default_rng(16)
    c = ref.random_cache(rng, 12, 2, 32, 64, [150], 6)
    wide = torch.from_numpy(rng.standard_normal((4, 12, 64))).to(torch.bfloat16).cuda()
    q = wide[:, 2:10]
    got = mqa.kv_attention(q, ref.to_device(c, mqa), ints([0, 4]))
    check(got, None, c.attention(q.double().cpu().numpy(), np.array([0, 4]), 0.125, "bf16"))


def test_bad_tables_are_not_followed(mqa):
    """A page index outside the pool: its keys are not seen; the status word tells."""
    rng = np.random.default_rng(17)
    c = ref.random_cache(rng, 12, 2, 16, 64, [100, 40], 8)
    dev = ref.to_device(c, mqa)
    dev.page_table[0, 2] = 1 << 30
    dev.page_table[1, 0] = -5
    q, qd = rows_of(rng, 2, 4, 64, "fp16")
    sel = np.full((2, 128), -1, np.int32)
    sel[0, :84] = [t for t in range(100) if not 32 <= t < 48]
    sel[1, :24] = range(16, 40)
    got = mqa.kv_attention(q, dev, ints([0, 1, 2]))
    assert mqa.kv_status(dev) == 2
    check(got, None, c.attention(qd, np.array([0, 1, 2]), 0.125, "fp16", sel))
    dev.seq_lens[0] = 10 ** 6
    mqa.kv_attention(q, dev, ints([0, 1, 2]))
    assert mqa.kv_status(dev) & 8
    assert mqa.kv_status(dev) == 0


def test_row_starts_outside_the_rows(mqa):
    """Bounds that leave the call's rows are cut to them; decreasing ones give a sequence no rows."""
    import torch
    rng = np.random.default_rng(18)
    c = ref.random_cache(rng, 30, 1, 16, 64, [50, 40, 30], 8)
    q, qd = rows_of(rng, 4, 4, 64, "bf16")
    out = torch.zeros_like(q)
    mqa.kv_attention(q, ref.to_device(c, mqa), ints([-3, 2, 2, 1000]), out=out)
    want = c.attention(qd, np.array([0, 2, 2, 4]), 0.125, "bf16")
    check(out, None, want)
    mqa.kv_attention(q, ref.to_device(c, mqa), ints([3, 1, 4, 4]), out=out)
    torch.cuda.synchronize()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention_with_few_rows_announced(mqa, case, causal):
    """max_rows = 1 keeps every sequence on the split kernel."""
    page, heads, group, dim, lens, rows = case
    rng = np.random.default_rng(len(lens) * 100 + group)
    c = ref.random_cache(rng, sum(-(-n // page) for n in lens) + 2, heads, page, dim, lens, 20)
    attend(mqa, c, rng, rows, group, "fp16", causal, max_rows=1)


TILED = [  # page, heads, group, dim, lens, rows: 17 to thousands of columns per sequence
    (64, 1, 4, 128, [128], [32]),                 # one 128-column half, one full tile of keys
    (64, 1, 4, 128, [129], [33]),
    (16, 2, 8, 128, [700], [70]),                 # two full halves and a rest
    (32, 2, 8, 64, [700], [70]),
    (128, 1, 3, 64, [400, 0, 90, 513], [200, 0, 90, 9]),
    (16, 1, 16, 128, [300, 5, 1100], [17, 2, 40]),
    (64, 2, 1, 128, [3000], [600]),
    (64, 1, 7, 64, [100, 260], [150, 200]),       # more rows than positions, then a chunk
    (32, 1, 32, 128, [2500], [9]),                # split along the keys
    (16, 3, 5, 64, [257, 256, 255], [255, 256, 100]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", TILED, ids=str)
def test_tiled_attention(mqa, case, dtype, causal):
    page, heads, group, dim, lens, rows = case
    rng = np.random.default_rng(sum(lens) + dim)
    c = ref.random_cache(rng, sum(-(-n // page) for n in lens) + 2, heads, page, dim, lens, 190)
    attend(mqa, c, rng, rows, group, dtype, causal, extra_rows=5)


def test_tiled_attention_scales_far_apart_and_sharp(mqa):
    rng = np.random.default_rng(25)
    c = ref.random_cache(rng, 30, 1, 16, 64, [400], 30, spread=20)
    attend(mqa, c, rng, [60], 4, "fp16", scale=1e-6)
    c.ke[:] = 127
    attend(mqa, c, rng, [60], 4, "bf16", q_scale=200.0)
    c.ve[:] = 127
    c.ve[c.table[0, 3], 0] = 27  # values 2^100 below the others', in the block that has all the weight
    c.k[c.table[0, 3], 0, 5] = ref.round_e4m3(np.full(64, 440.0))
    import torch
    q = torch.ones((60, 4, 64), dtype=torch.bfloat16, device="cuda")
    got = mqa.kv_attention(q, ref.to_device(c, mqa), ints([0, 60]), scale=0.5)
    check(got, None, c.attention(np.ones((60, 4, 64)), np.array([0, 60]), 0.5, "bf16"))


def test_tiled_attention_bad_page(mqa):
    rng = np.random.default_rng(26)
    c = ref.random_cache(rng, 40, 2, 16, 64, [300], 30)
    dev = ref.to_device(c, mqa)
    dev.page_table[0, 7] = 40
    q, qd = rows_of(rng, 50, 8, 64, "fp16")
    sel = np.array([[t for t in range(300) if t // 16 != 7]] * 50, np.int32)
    got = mqa.kv_attention(q, dev, ints([0, 50]))
    assert mqa.kv_status(dev) == 2
    check(got, None, c.attention(qd, np.array([0, 50]), 0.125, "fp16", sel))

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [3, 8])
def test_one_workspace_holds_for_every_form(mqa, dim, group):
    """alloc_kv_workspace(rows) serves calls of fewer rows, of any max_rows, and over selected keys."""
    rng = np.random.default_rng(60)
    c = ref.random_cache(rng, 20, 2, 16, dim, [90, 60], 8)
    dev = ref.to_device(c, mqa)
    q, qd = rows_of(rng, 8, 2 * group, dim, "bf16")
    ws = mqa.alloc_kv_workspace(dev, 8, 2 * group)
    for rows in ([8, 0], [4, 4], [1, 1], [0, 3]):
        st = starts_of(rows)
        n = int(st[-1])
        sel = random_selection(rng, c, rows, 20)
        for max_rows in (None, 1, 2, 3, 4, 7):
            got = mqa.kv_attention(q[:n], dev, ints(st), max_rows=max_rows, workspace=ws)
            check(got, None, c.attention(qd[:n], st, dim ** -0.5, "bf16"), (rows, max_rows))
        got = mqa.kv_attention(q[:n], dev, ints(st), selected=ints(sel), workspace=ws)
        check(got, None, c.attention(qd[:n], st, dim ** -0.5, "bf16", sel), rows)


def test_short_sequences_beside_a_prompt(mqa):
    """Sequences of one row, of none and of no position in one call with a prompt."""
    rng = np.random.default_rng(61)
    c = ref.random_cache(rng, 60, 2, 16, 128, [0, 400, 150, 7, 1], 26)
    attend(mqa, c, rng, [0, 400, 1, 3, 1], 8, extra_rows=2)
    attend(mqa, c, rng, [2, 300, 0, 1, 0], 8, "fp16", causal=False)


def test_many_sequences(mqa):
    """More sequences than the kernels hold bounds of at once, most of them without rows."""
    rng = np.random.default_rng(62)
    n = 1500
    lens = rng.integers(0, 40, n)
    rows = np.where(rng.random(n) < 0.1, np.minimum(rng.integers(1, 9, n), lens), 0)
    rows[[0, 1023, 1024, 1025, n - 1]] = 1
    lens[[0, 1023, 1024, 1025, n - 1]] = 17
    c = ref.random_cache(rng, int((-(-lens // 16)).sum()) + 1, 1, 16, 64, lens, 3)
    out, dev, q, st = attend(mqa, c, rng, rows, 4)
    attend(mqa, c, rng, rows, 4, max_rows=1)
    k, kd = rows_of(rng, int(st[-1]), 1, 64, "bf16")
    mqa.kv_append(dev, k, k, ints(st))
    c.append(kd, kd, st)
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0


def test_offsets_past_32_bits(mqa):
    """A pool of more than 2^32 bytes: its last pages are appended to, read in each form, copied and moved."""
    import torch
    rng = np.random.default_rng(63)
    heads, page, dim = 8, 128, 128
    pages = 2 ** 32 // (heads * page * dim) + 64
    tail = 40  # the host holds the last pages only; page p of the pool is page p - (pages - tail) there
    lens, width = [1000, 300], 12
    c = ref.random_cache(rng, tail, heads, page, dim, lens, width)
    base = pages - tail
    z = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    dev = mqa.KVCache(z(pages, heads, page, dim), z(pages, heads, page, dim), z(pages, heads), z(pages, heads),
                      ints(c.table + base), ints(c.lens), z(pages, t=torch.int32))
    for t, a in ((dev.k, c.k), (dev.v, c.v), (dev.k_exps, c.ke), (dev.v_exps, c.ve), (dev.refcounts, c.refs)):
        t[base:] = torch.from_numpy(a).cuda()

    def same():
        return [n for n, a in (("k", c.k), ("v", c.v), ("k_exps", c.ke), ("v_exps", c.ve))
                if not np.array_equal(getattr(dev, n)[base:].cpu().numpy(), a)]

    for rows in ([1, 2], [40, 3]):
        st = starts_of(rows)
        n = int(st[-1])
        k, kd = rows_of(rng, n, heads, dim, "bf16")
        mqa.kv_append(dev, k, k, ints(st))
        c.append(kd, kd, st)
        assert same() == []
        q, qd = rows_of(rng, n, heads * 4, dim, "bf16")
        check(mqa.kv_attention(q, dev, ints(st)), None, c.attention(qd, st, dim ** -0.5, "bf16"))
        sel = random_selection(rng, c, rows, 33)
        check(mqa.kv_attention(q, dev, ints(st), selected=ints(sel)), None,
              c.attention(qd, st, dim ** -0.5, "bf16", sel))
    free = np.nonzero(c.refs == 0)[0][:2]
    src = c.table[0, :2].copy()
    mqa.kv_copy_pages(dev, ints(src + base), ints(free + base))
    c.copy_pages(src, free)
    assert same() == [] and not dev.k[:base].any() and not dev.v[:base].any()  # nothing landed 2^32 bytes lower
    want = mqa.kv_attention(q, dev, ints(st))
    mqa.kv_compact(dev)
    assert mqa.kv_status(dev) == 0 and int(dev.page_table[0, :8].max()) < 64
    assert torch.equal(mqa.kv_attention(q, dev, ints(st)), want)


@pytest.mark.parametrize("rows", [3, 70])
def test_tiny_queries_and_scales(mqa, rows):
    """Scores whose factor leaves fp32's range: all alike, and masked keys stay masked."""
    rng = np.random.default_rng(66)
    c = ref.random_cache(rng, 12, 1, 16, 64, [100], 8)
    c.ke[:] = 7
    attend(mqa, c, rng, [rows], 4, q_scale=1e-30)
    attend(mqa, c, rng, [rows], 4, q_scale=1e-30, selected=random_selection(rng, c, [rows], 20))


# ---------------------------------------------------------------- selected keys
def random_selection(rng, c, rows, k, seen_only=False):
    sel = []
    for n, r in zip(c.lens, rows):
        for i in range(r):
            last = int(n) - r + i
            hi = max(1, last + 1 if seen_only else int(n) + 5)
            x = rng.permutation(hi)[:k]
            x = np.concatenate([x, np.full(k - len(x), -1)]) if len(x) < k else x
            if not seen_only:
                x[rng.random(k) < 0.1] = rng.integers(-5, 0)
            sel.append(x)
    return np.array(sel, np.int32).reshape(-1, k)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", [(16, 1, 1, 128, [1], [1], 4), (64, 2, 4, 128, [500, 0, 90], [3, 2, 2], 100),
                                  (32, 1, 32, 64, [700, 64], [2, 5], 65), (128, 2, 9, 128, [1200], [3], 512),
                                  (16, 4, 16, 64, [33, 400], [33, 1], 48)], ids=str)
def test_selected_attention(mqa, case, dtype):
    page, heads, group, dim, lens, rows, k = case
    rng = np.random.default_rng(k)
    c = ref.random_cache(rng, sum(-(-n // page) for n in lens) + 1, heads, page, dim, lens, 30)
    sel = random_selection(rng, c, rows, k)
    sel = np.concatenate([sel, np.full((2, k), 3, np.int32)])  # rows of no sequence
    attend(mqa, c, rng, rows, group, dtype, True, sel, extra_rows=2)


def test_selected_all_entries_and_none(mqa):
    """A list of every visible position gives the dense answer's value; an empty one and one of -1 give zeros; a
    position listed twice counts twice."""
    rng = np.random.default_rng(20)
    c = ref.random_cache(rng, 20, 2, 16, 128, [150], 12)
    allk = np.stack([np.where(np.arange(150) <= 145 + i, np.arange(150), -1) for i in range(5)]).astype(np.int32)
    attend(mqa, c, rng, [5], 4, selected=allk)
    attend(mqa, c, rng, [5], 4, selected=np.full((5, 7), -1, np.int32))
    attend(mqa, c, rng, [5], 4, selected=np.zeros((5, 0), np.int32))
    attend(mqa, c, rng, [5], 4, selected=np.tile(np.array([[9, 3, 9, 9]], np.int32), (5, 1)))


def test_selected_long(mqa):
    rng = np.random.default_rng(21)
    c = ref.random_cache(rng, 330, 1, 64, 128, [20000], 320)
    attend(mqa, c, rng, [3], 8, selected=random_selection(rng, c, [3], 2048, True))


# ---------------------------------------------------------------- streams, graphs
def test_attention_in_a_graph_on_a_side_stream(mqa):
    import torch
    rng = np.random.default_rng(22)
    c = ref.random_cache(rng, 60, 2, 16, 128, [300, 120], 24)
    dev = ref.to_device(c, mqa)
    q, qd = rows_of(rng, 4, 8, 128, "bf16")
    st = ints([0, 2, 4])
    ws = mqa.alloc_kv_workspace(dev, 4, 8)
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mqa.kv_attention(q, dev, st, workspace=ws, out=out, stream=side)
    side.synchronize()
    check(out, None, c.attention(qd, np.array([0, 2, 4]), 128 ** -0.5, "bf16"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mqa.kv_attention(q, dev, st, workspace=ws, out=out)
    for lens in ([300, 120], [17, 1], [0, 64]):
        c.lens[:] = lens
        dev.seq_lens.copy_(ints(lens))
        out.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        check(out, None, c.attention(qd, np.array([0, 2, 4]), 128 ** -0.5, "bf16"), lens)


def test_two_streams_with_a_workspace_each(mqa):
    import torch
    rng = np.random.default_rng(23)
    c = ref.random_cache(rng, 340, 2, 32, 128, [9000, 500], 300)
    dev = ref.to_device(c, mqa)
    q, _ = rows_of(rng, 2, 8, 128, "fp16")
    st = ints([0, 1, 2])
    want = mqa.kv_attention(q, dev, st)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [mqa.kv_attention(q, dev, st, stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)  # and the same bits every time


def test_tiled_attention_in_graphs(mqa):
    """Two graphs of a call for many columns on one workspace, replayed on a side stream with other lengths."""
    import torch
    rng = np.random.default_rng(64)
    c = ref.random_cache(rng, 60, 2, 16, 64, [300, 120], 24)
    dev = ref.to_device(c, mqa)
    q, qd = rows_of(rng, 90, 8, 64, "fp16")
    bounds = [np.array([0, 60, 90]), np.array([0, 1, 90])]
    st = [ints(b) for b in bounds]
    ws = mqa.alloc_kv_workspace(dev, 90, 8)
    outs = [torch.zeros_like(q) for _ in st]
    mqa.kv_attention(q, dev, st[0], workspace=ws, out=outs[0])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in st]
    for g, s, o in zip(graphs, st, outs):
        with torch.cuda.graph(g):
            mqa.kv_attention(q, dev, s, workspace=ws, out=o)
    side = torch.cuda.Stream()
    for lens in ([300, 120], [60, 89], [5, 0], [257, 128]):
        c.lens[:] = lens
        dev.seq_lens.copy_(ints(lens))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for g in graphs:
                g.replay()
        side.synchronize()
        for o, b in zip(outs, bounds):
            check(o, None, c.attention(qd, b, 0.125, "fp16"), lens)


def test_calls_follow_one_another_without_a_pause(mqa):
    """Appending and attention for few and for many columns in turn on one workspace: each call reads what the call
    before it wrote, and the answers are those of calls made one at a time."""
    import torch
    rng = np.random.default_rng(65)
    c = ref.random_cache(rng, 90, 2, 16, 128, [500, 260], 36)
    c.k &= 0x7E  # whatever the unused positions hold, no NaN
    c.v &= 0x7E
    ks = [rows_of(rng, n, 2, 128, "bf16")[0] for n in (3, 80, 3, 80)]
    qs = [rows_of(rng, k.shape[0], 16, 128, "bf16")[0] for k in ks]
    sts = [ints([0, k.shape[0] - 1, k.shape[0]]) for k in ks]

    def run(pause):
        dev, outs = ref.to_device(c, mqa), []
        ws = mqa.alloc_kv_workspace(dev, 80, 16)
        for k, q, st in list(zip(ks, qs, sts)) * 3:
            mqa.kv_append(dev, k, k, st)
            outs.append(mqa.kv_attention(q, dev, st, workspace=ws))
            mqa.kv_reserve(dev, ints([1, 2]))
            if pause:
                torch.cuda.synchronize()
        assert mqa.kv_status(dev) == 0
        return outs
    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_prompts_on_two_streams_from_two_threads(mqa):
    """Calls for many columns that overlap, a workspace each: the same bits as one at a time."""
    import threading

    import torch
    rng = np.random.default_rng(67)
    c = ref.random_cache(rng, 130, 2, 32, 128, [2000, 700, 900], 70)
    dev = ref.to_device(c, mqa)
    q, _ = rows_of(rng, 500, 8, 128, "bf16")
    st = ints([0, 300, 301, 500])
    want = mqa.kv_attention(q, dev, st)
    torch.cuda.synchronize()
    outs = [[], []]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ws = mqa.alloc_kv_workspace(dev, 500, 8)
            for _ in range(20):
                outs[i].append(mqa.kv_attention(q, dev, st, workspace=ws))
        s.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(outs[0]) == len(outs[1]) == 20
    assert all(torch.equal(o, want) for o in outs[0] + outs[1]) and mqa.kv_status(dev) == 0


# ---------------------------------------------------------------- appending
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("case", [(16, 1, 128, [1], [1]), (64, 2, 64, [64, 65, 200, 5], [1, 2, 130, 0]),
                                  (32, 3, 128, [31, 33, 400], [31, 33, 77]), (128, 2, 64, [300, 0, 4], [2, 0, 9]),
                                  (16, 8, 128, [17, 18, 19, 20, 40, 16, 1, 2], [1] * 8)], ids=str)
def test_append_bit_exact(mqa, case, dtype):
    import torch
    page, heads, dim, lens, rows = case
    rng = np.random.default_rng(dim + len(lens))
    c = ref.random_cache(rng, sum(-(-n // page) for n in lens) + 2, heads, page, dim, lens, 14)
    dev = ref.to_device(c, mqa)
    st = starts_of(rows)
    n = int(st[-1]) + 2
    size = torch.from_numpy(2.0 ** rng.integers(-6, 14, (n, heads, 1))).cuda()  # some blocks' scales grow
    k, v = (rows_of(rng, n, heads, dim, dtype)[0] * size for _ in range(2))
    k, v = (x.clamp(-6e4, 6e4).to(getattr(torch, TYPES[dtype])) for x in (k, v))
    mqa.kv_append(dev, k, v, ints(st))
    c.append(k.double().cpu().numpy(), v.double().cpu().numpy(), st)
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0


def test_append_extremes(mqa):
    """Zeros, the smallest and largest values, infinities and NaN, and a block of a given, larger scale."""
    import torch
    rng = np.random.default_rng(31)
    c = ref.random_cache(rng, 12, 2, 16, 64, [40, 20, 16, 9], 4)
    c.ke[c.table[1, 1]] = 200
    dev = ref.to_device(c, mqa)
    st = starts_of([20, 4, 16, 5])
    k = torch.from_numpy(rng.standard_normal((45, 2, 64))).float().cuda()
    k[3] = 0
    k[4:12] *= 1e38
    k[22:24] = 1e-44
    k[24:40] = 0
    v = k.clone()
    v[1, 0, 5], v[2, 1, 6], v[41, 0, 0] = float("inf"), float("-inf"), float("nan")
    v[40:45, 1] = float("nan")
    mqa.kv_append(dev, k, v, ints(st))
    c.append(k.double().cpu().numpy(), v.double().cpu().numpy(), st)
    bad = ref.same(c, dev)
    if bad:  # a NaN's sign is not kept by every path
        for n, a in (("k", c.k), ("v", c.v)):
            g = getattr(dev, n).cpu().numpy()
            nan = np.isnan(ref.E4M3[a])
            assert np.array_equal(np.isnan(ref.E4M3[g]), nan) and np.array_equal(g[~nan], a[~nan])
    assert [n for n in bad if n not in ("k", "v")] == []


def test_append_strided_and_refused_rows(mqa):
    import torch
    rng = np.random.default_rng(32)
    c = ref.random_cache(rng, 12, 2, 16, 64, [3, 40], 4)
    dev = ref.to_device(c, mqa)
    wide = torch.from_numpy(rng.standard_normal((9, 6, 64))).to(torch.bfloat16).cuda()
    k, v = wide[:, 1:3], wide[:, 4:6]
    st = starts_of([5, 4])  # five rows for a sequence of three: two lie before it
    mqa.kv_append(dev, k, v, ints(st))
    kd, vd = k.double().cpu().numpy(), v.double().cpu().numpy()
    c.append(np.concatenate([kd[2:], kd[:2]]), np.concatenate([vd[2:], vd[:2]]), starts_of([3, 4]))
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0
    dev.page_table[1, 2] = 99  # positions 36 .. 39 have no page now
    before = dev.k.clone()
    mqa.kv_append(dev, k[5:], v[5:], ints([0, 0, 4]))
    assert mqa.kv_status(dev) == 2 and torch.equal(before, dev.k)
    dev.seq_lens[1] = 1000
    mqa.kv_append(dev, k[5:], v[5:], ints([0, 0, 4]))
    assert mqa.kv_status(dev) == 8 and torch.equal(before, dev.k)


# ---------------------------------------------------------------- pages
def test_random_page_operations(mqa):
    import torch
    rng = np.random.default_rng(40)
    pages, heads, page, dim, seqs, width = 90, 2, 16, 64, 12, 9
    c = ref.random_cache(rng, pages, heads, page, dim, [0] * seqs, width, shuffle=False)
    c.table[:] = -1
    index = torch.from_numpy(rng.integers(0, 255, (pages, page, 5)).astype(np.uint8)).cuda()
    plain_index = index.cpu().numpy().copy()
    dev = ref.to_device(c, mqa, extra=(index,))
    plain_copy = c.copy_pages

    def copy_all(src, dst):
        plain_copy(src, dst)
        plain_index[dst] = plain_index[src]
    c.copy_pages = copy_all
    seen = set()
    for step in range(300):
        op = rng.choice(["reserve", "reserve", "fork", "fork", "free", "compact"])
        live = np.nonzero(c.lens)[0]
        empty = np.nonzero(c.lens == 0)[0]
        want = 0
        if op == "reserve":
            counts = np.where(rng.random(seqs) < 0.4, rng.integers(0, 40, seqs), 0).astype(np.int32)
            # a shared partial page cannot arise: fork copies it
            mqa.kv_reserve(dev, ints(counts))
            want = c.reserve(counts)
        elif op == "fork":
            n = int(rng.integers(1, 4))
            parents = rng.integers(0, seqs, n).astype(np.int32)
            children = rng.permutation(empty)[:n].astype(np.int32)
            if len(children) < n or rng.random() < 0.1:
                children = rng.integers(0, seqs, n).astype(np.int32)
            mqa.kv_fork(dev, ints(parents), ints(children))
            want = c.fork(parents, children)
        elif op == "free":
            gone = rng.permutation(live)[:2].astype(np.int32)
            mqa.kv_free(dev, ints(np.concatenate([gone, gone[:1]])))  # one of them listed twice
            c.free(gone)
        else:
            mqa.kv_compact(dev)
            c.compact()
        seen.add((op, want))
        assert mqa.kv_status(dev) == want, (step, op)
        assert ref.same(c, dev) == [], (step, op, ref.same(c, dev))
        assert np.array_equal(index.cpu().numpy(), plain_index)
    assert {("reserve", 0), ("reserve", 8), ("fork", 0), ("fork", 4), ("free", 0), ("compact", 0)} <= seen, seen


def test_too_few_pages_change_nothing(mqa):
    rng = np.random.default_rng(42)
    c = ref.random_cache(rng, 10, 1, 16, 64, [70, 40, 0, 0, 0], 9)  # two free pages
    dev = ref.to_device(c, mqa)
    for counts, want in (([0, 9, 33, 0, 0], 1), ([0, 0, 17, 16, 0], 1), ([10, 8, 16, 16, 0], 0), ([0, 0, 1, 0, 0], 1)):
        counts = np.array(counts, np.int32)
        mqa.kv_reserve(dev, ints(counts))
        assert c.reserve(counts) == want and mqa.kv_status(dev) == want and ref.same(c, dev) == []
    c = ref.random_cache(rng, 10, 1, 16, 64, [70, 40, 0, 0, 0], 9)
    dev = ref.to_device(c, mqa)
    for parents, children, want in (([0, 1, 0], [2, 3, 4], 1), ([0, 1], [2, 3], 0), ([1], [4], 1)):
        parents, children = np.array(parents), np.array(children)
        mqa.kv_fork(dev, ints(parents), ints(children))
        assert c.fork(parents, children) == want and mqa.kv_status(dev) == want and ref.same(c, dev) == []


@pytest.mark.parametrize("pages", [16384, 40001])
def test_reserve_in_large_pools(mqa, pages):
    """Free pages far apart and far behind are found lowest first, over all steps of the search."""
    rng = np.random.default_rng(pages)
    c = ref.random_cache(rng, pages, 1, 16, 64, [0] * 6, 1000, garbage=False)
    c.refs[:] = rng.random(pages) < 0.97
    c.refs[:pages // 2] = 1
    c.refs[[5, pages - 1]] = 0
    dev = ref.to_device(c, mqa)
    free = int((c.refs == 0).sum())
    for counts, want in (([16, 0, 0, 33, 0, 1], 0), ([0, 16 * (free // 2), 0, 0, 15, 0], 0), ([0, 0, 16 * free, 0, 0, 0], 1),
                         ([0, 0, 16 * (free - free // 2 - 6), 0, 0, 0], 0), ([0, 0, 0, 0, 16, 0], 1)):
        counts = np.array(counts, np.int32)
        assert c.reserve(counts) == want
        mqa.kv_reserve(dev, ints(counts))
        assert mqa.kv_status(dev) == want and ref.same(c, dev) == [], counts


@pytest.mark.parametrize("pages", [1, 7, 4096, 5000, 12289])
def test_compact_sizes(mqa, pages):
    rng = np.random.default_rng(pages)
    lens, left = [], pages
    while left > 0 and len(lens) < 40:
        n = int(rng.integers(1, max(2, min(left, 700) + 1)))
        n = min(n, left)
        lens.append(16 * n - int(rng.integers(0, 16)))
        left -= n
    c = ref.random_cache(rng, pages, 1, 16, 64, lens, 700)
    c.table[c.table < 0] = 0
    dev = ref.to_device(c, mqa)
    gone = np.nonzero(rng.random(len(lens)) < 0.5)[0].astype(np.int32)
    c.free(gone)
    mqa.kv_free(dev, ints(gone))
    mqa.kv_compact(dev)
    c.compact()
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0
    mqa.kv_compact(dev)  # nothing left to move
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0


def test_page_lists_that_are_refused(mqa):
    rng = np.random.default_rng(41)
    c = ref.random_cache(rng, 20, 2, 16, 64, [40, 33, 0, 0], 8)
    dev = ref.to_device(c, mqa)
    for src, dst in (([1, 2], [3, 3]), ([1, 2], [2, 3]), ([1], [20]), ([-1], [3]), ([4], [4])):
        mqa.kv_copy_pages(dev, ints(src), ints(dst))
        assert mqa.kv_status(dev) == 4 and ref.same(c, dev) == [], (src, dst)
    mqa.kv_copy_pages(dev, ints([1, 1, 5]), ints([3, 4, 6]))
    c.copy_pages([1, 1, 5], [3, 4, 6])
    assert mqa.kv_status(dev) == 0 and ref.same(c, dev) == []
    for parents, children in (([0], [1]), ([0, 1], [2, 2]), ([4], [2]), ([0], [-1])):
        mqa.kv_fork(dev, ints(parents), ints(children))
        assert mqa.kv_status(dev) == 4 and ref.same(c, dev) == []
    mqa.kv_free(dev, ints([7, -1]))
    assert mqa.kv_status(dev) == 2 and ref.same(c, dev) == []
    mqa.kv_reserve(dev, ints([0, 0, 16 * 9, 0]))
    assert mqa.kv_status(dev) == 8 and ref.same(c, dev) == []
    mqa.kv_reserve(dev, ints([0, -1, 0, 0]))
    assert mqa.kv_status(dev) == 4 and ref.same(c, dev) == []


# ---------------------------------------------------------------- together
def test_prompt_selection_attention_fork_and_decode(mqa):
    """A prompt is written, the indexer selects keys for its rows, attention reads them; two samples are forked, each
    gets a token of its own, the prompt's sequence is freed, the pool compacted, and the samples answer as before."""
    import torch
    rng = np.random.default_rng(50)
    heads, group, dim, page, n = 2, 8, 128, 64, 1000
    dev = mqa.alloc_kv_cache(60, page, heads, dim, 3, 20)
    c = ref.Cache(*(t.cpu().numpy().copy() for t in (dev.k, dev.v, dev.k_exps, dev.v_exps, dev.page_table,
                                                     dev.seq_lens, dev.refcounts)))

    def grow(counts):
        counts = np.array(counts, np.int32)
        st = starts_of(counts)
        k, kd = rows_of(rng, int(st[-1]), heads, dim, "bf16")
        v, vd = rows_of(rng, int(st[-1]), heads, dim, "bf16")
        mqa.kv_reserve(dev, ints(counts))
        mqa.kv_append(dev, k, v, ints(st))
        assert c.reserve(counts) == 0
        c.append(kd, vd, st)
        return st

    st = grow([n, 0, 0])
    # the indexer over the prompt's own index keys
    rows = 6
    iq = torch.from_numpy(ref.round_e4m3(rng.standard_normal((rows, 32, 128)))).cuda()
    ik = torch.from_numpy(ref.round_e4m3(rng.standard_normal((n, 128)))).cuda()
    ends = ints(n - rows + 1 + np.arange(rows))
    idx = mqa.mqa_topk_prefill(iq, ik, torch.ones(n, device="cuda"), torch.rand((rows, 32), device="cuda"),
                               torch.zeros_like(ends), ends, 512)
    q, qd = rows_of(rng, rows, heads * group, dim, "bf16")
    last = np.array([0, rows, rows, rows])
    got = mqa.kv_attention(q, dev, ints(last), selected=idx)
    check(got, None, c.attention(qd, last, dim ** -0.5, "bf16", idx.cpu().numpy()))
    mqa.kv_fork(dev, ints([0, 0]), ints([1, 2]))
    assert c.fork(np.array([0, 0]), np.array([1, 2])) == 0
    st = grow([0, 1, 1])
    assert ref.same(c, dev) == []
    q, qd = rows_of(rng, 2, heads * group, dim, "bf16")
    want = mqa.kv_attention(q, dev, ints(st))
    check(want, None, c.attention(qd, st, dim ** -0.5, "bf16"))
    mqa.kv_free(dev, ints([0]))
    mqa.kv_compact(dev)
    c.free([0])
    c.compact()
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0
    assert torch.equal(mqa.kv_attention(q, dev, ints(st)), want)


# ---------------------------------------------------------------- the least alignment
def shifted(t, by):
    """A copy of t that begins `by` elements behind an aligned address, and the elements before it."""
    import torch
    flat = torch.zeros(t.numel() + by, dtype=t.dtype, device="cuda")
    flat[by:].copy_(t.reshape(-1))
    return flat[by:].view(t.shape), flat[:by]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,max_rows", [([60, 1, 300], None), ([40, 0, 0], None), ([2, 1, 3], 3)])
def test_least_alignment(mqa, dim, rows, max_rows):
    """Rows, outputs and codes at 16 bytes behind a multiple of 32, counts and tables at 4, exponents at 1: every form
    of attention, appending and the page operations answer as ever and write nothing before their outputs."""
    import torch
    rng = np.random.default_rng(70)
    c = ref.random_cache(rng, 60, 2, 16, dim, [300, 41, 310], 24)
    dev = mqa.KVCache(*(shifted(torch.from_numpy(a).cuda(), by)[0]
                        for a, by in ((c.k, 16), (c.v, 16), (c.ke, 1), (c.ve, 1), (c.table, 1), (c.lens, 1), (c.refs, 1))))
    assert dev.k.data_ptr() % 32 == 16
    st = starts_of(rows)
    n = int(st[-1])
    k, kd = rows_of(rng, n, 2, dim, "bf16")
    k, _ = shifted(k, 8)
    starts, _ = shifted(ints(st), 1)
    mqa.kv_append(dev, k, k, starts)
    c.append(kd, kd, st)
    assert ref.same(c, dev) == []
    for dtype in ("bf16", "fp16"):
        q, qd = rows_of(rng, n, 8, dim, dtype)
        q, _ = shifted(q, 8)
        for sel in (None, random_selection(rng, c, rows, 20)):
            out, before = shifted(torch.zeros_like(q), 8)
            lse, lse_before = shifted(torch.zeros((n, 8), device="cuda"), 1)
            assert q.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16 and lse.data_ptr() % 8 == 4
            mqa.kv_attention(q, dev, starts, selected=None if sel is None else shifted(ints(sel), 1)[0],
                             max_rows=max_rows, out=out, lse=lse)
            check(out, lse, c.attention(qd, st, dim ** -0.5, dtype, sel))
            assert not before.any() and not lse_before.any()
    c.free([0])
    mqa.kv_free(dev, ints([0]))
    mqa.kv_fork(dev, ints([2]), ints([0]))
    assert c.fork(np.array([2]), np.array([0])) == 0
    mqa.kv_compact(dev)
    c.compact()
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0


# ---------------------------------------------------------------- requests far past the pool
def test_reserve_requests_whose_pages_pass_32_bits(mqa):
    """Requests of up to 2^26 pages each, whose sum passes 2^31 and 2^32 pages, in a pool of 40: too few pages, and
    nothing changes.  (Sums in 32 bits would read as negative, as zero and as three pages.)"""
    import torch
    pages, seqs, width = 40, 65, 1 << 26
    z = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    dev = mqa.KVCache(z(pages, 1, 16, 64), z(pages, 1, 16, 64), z(pages, 1), z(pages, 1),
                      torch.full((seqs, width), -1, dtype=torch.int32, device="cuda"), z(seqs, t=torch.int32),
                      z(pages, t=torch.int32))
    full = 1 << 30  # positions of 2^26 pages of 16
    for counts in ([full] * 32 + [0] * 33, [0] * 33 + [full] * 32, [full] * 64 + [0], [full] * 64 + [40], [full] * 65):
        need = sum(-(-n // 16) for n in counts)
        assert need >= 1 << 31
        mqa.kv_reserve(dev, ints(counts))
        assert mqa.kv_status(dev) == 1, need
        assert not dev.seq_lens.any() and not dev.refcounts.any()
        assert int(dev.page_table.max()) == -1 and int(dev.page_table.min()) == -1
    mqa.kv_reserve(dev, ints([0] * 64 + [40]))
    assert mqa.kv_status(dev) == 0 and dev.page_table[64, :4].tolist() == [0, 1, 2, -1] and int(dev.seq_lens[64]) == 40
    assert int(dev.refcounts.sum()) == 3


# ---------------------------------------------------------------- the waits' time limit
@pytest.mark.parametrize("stall", [1, 2])
@pytest.mark.parametrize("rows,max_rows", [([1, 1, 2], 2), ([150, 0, 90], None), ([400, 1, 300], None)])
def test_waits_end_at_their_limit(mqa, rows, max_rows, stall):
    """A wait for what never comes runs out (of few columns, of many, and of both in one call): the status says so,
    nothing but the outputs has changed, and the next call on the same workspace answers as if nothing had been."""
    import torch
    rng = np.random.default_rng(71)
    c = ref.random_cache(rng, 130, 2, 16, 128, [900, 40, 700], 60)
    dev = ref.to_device(c, mqa)
    st = starts_of(rows)
    q, _ = rows_of(rng, int(st[-1]), 8, 128, "bf16")
    ws = mqa.alloc_kv_workspace(dev, int(st[-1]), 8)
    ws.fill_(0xAB)
    want = mqa.kv_attention(q, dev, ints(st), max_rows=max_rows, workspace=ws)
    assert mqa.kv_status(dev) == 0
    for _ in range(2):
        got = mqa.kv_attention(q, dev, ints(st), max_rows=max_rows, workspace=ws,
                               debug={"stall": stall, "wait_timeout_ms": 30})
        assert got.shape == q.shape and mqa.kv_status(dev) == 16
        assert ref.same(c, dev) == []
        got = mqa.kv_attention(q, dev, ints(st), max_rows=max_rows, workspace=ws, debug={"wait_timeout_ms": 500})
        assert torch.equal(got, want) and mqa.kv_status(dev) == 0


# ---------------------------------------------------------------- rows of no sequence
@pytest.mark.parametrize("form", ["dense", "selected"])
@pytest.mark.parametrize("rows", [[1, 2], [40, 9], [0, 3], [0, 0]])
def test_rows_before_the_first_bound(mqa, rows, form):
    """A first bound above zero: the rows before it belong to no sequence, in no form of the call."""
    import torch
    rng = np.random.default_rng(72)
    c = ref.random_cache(rng, 20, 2, 16, 64, [90, 70], 8)
    dev = ref.to_device(c, mqa)
    before, behind, n = 3, 2, sum(rows)
    st = starts_of(rows) + before
    q, qd = rows_of(rng, before + n + behind, 8, 64, "bf16")
    q[:before] = float("nan")
    sel = random_selection(rng, c, rows, 20)
    pad = lambda k: np.zeros((k, 20), np.int32)  # noqa: E731
    sel = np.concatenate([pad(before), sel, pad(behind)]) if form == "selected" else None
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    mqa.kv_attention(q, dev, ints(st), selected=None if sel is None else ints(sel), out=out, lse=lse)
    assert mqa.kv_status(dev) == 0
    at = slice(before, before + n)
    for t in (out, lse):
        assert (t[:before] == 7).all() and (t[before + n:] == 7).all()
    check(out[at], lse[at], c.attention(qd[at], st - before, 0.125, "bf16", None if sel is None else sel[at]))
    k, kd = rows_of(rng, before + n + behind, 2, 64, "bf16")
    mqa.kv_append(dev, k, k, ints(st))
    c.append(kd[at], kd[at], st - before)
    assert ref.same(c, dev) == []


# ---------------------------------------------------------------- the status word and captures
def test_status_is_refused_in_a_capture(mqa):
    """Reading the status waits for the stream, which a capture does not allow: the call is refused, and the capture
    is not lost."""
    import torch
    rng = np.random.default_rng(73)
    c = ref.random_cache(rng, 12, 2, 16, 64, [100], 8)
    dev = ref.to_device(c, mqa)
    q, qd = rows_of(rng, 2, 8, 64, "bf16")
    st = ints([0, 2])
    ws = mqa.alloc_kv_workspace(dev, 2, 8)
    out = torch.zeros_like(q)
    mqa.kv_attention(q, dev, st, workspace=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mqa.kv_attention(q, dev, st, workspace=ws, out=out)
        with pytest.raises(mqa.MQAError) as e:
            mqa.kv_status(dev)
        assert e.value.code == 1
    dev.page_table[0, 1] = -7
    out.zero_()
    g.replay()
    assert mqa.kv_status(dev) == 2 and mqa.kv_status(dev) == 0
    sel = np.array([[t for t in range(100) if t // 16 != 1]] * 2, np.int32)
    check(out, None, c.attention(qd, np.array([0, 2]), 0.125, "bf16", sel))


# ---------------------------------------------------------------- forms that only few columns had been tested in
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens", [([3, 2], [100, 60]), ([90, 40], [400, 60]), ([30, 70], [2900, 70])], ids=str)
def test_infinite_and_nan_query_values(mqa, rows, lens, dtype):
    """A query value that is no finite number gives NaN in every component and the lse of its row and head, and
    nothing else: in both kernels, whole and joined from parts, over selected keys, and zeros where the row sees
    nothing."""
    import torch
    rng = np.random.default_rng(74)
    c = ref.random_cache(rng, sum(-(-n // 16) for n in lens) + 2, 2, 16, 64, lens, 190)
    dev = ref.to_device(c, mqa)
    st = starts_of(rows)
    n = int(st[-1])
    q, _ = rows_of(rng, n, 8, 64, dtype)
    marks = [(1, 2, 5, float("nan")), (2, 4, 0, float("inf")), (n - 1, 7, 63, float("-inf")), (n - 2, 0, 8, float("inf"))]
    for r, h, d, x in marks:
        q[r, h, d] = x
    q[0, 1] = float("nan")
    qd = q.double().cpu().numpy()
    for sel in (None, random_selection(rng, c, rows, 30)):
        if sel is not None:
            sel[n - 1] = -1  # sees nothing: zeros
        lse = torch.zeros((n, 8), device="cuda")
        out = mqa.kv_attention(q, dev, ints(st), selected=None if sel is None else ints(sel), lse=lse)
        want = c.attention(qd, st, 0.125, dtype, sel)
        for r, h in [m[:2] for m in marks] + [(0, 1)]:
            assert np.isnan(want[0][r, h]).all() or (sel is not None and not want[0][r, h].any())
        assert np.isnan(want[0]).any()
        check(out, lse, want)
    assert mqa.kv_status(dev) == 0


@pytest.mark.parametrize("rows,max_rows", [([90, 40, 1], None), ([3, 2, 1], 3)])
def test_strided_queries_in_every_kernel(mqa, rows, max_rows):
    """Queries that are a slice of a wider projection."""
    import torch
    rng = np.random.default_rng(75)
    c = ref.random_cache(rng, 40, 2, 32, 128, [400, 60, 70], 14)
    dev = ref.to_device(c, mqa)
    st = starts_of(rows)
    wide = torch.from_numpy(rng.standard_normal((int(st[-1]), 14, 128))).to(torch.float16).cuda()
    q = wide[:, 3:11]
    qd = q.double().cpu().numpy()
    sel = random_selection(rng, c, rows, 30)
    check(mqa.kv_attention(q, dev, ints(st), max_rows=max_rows), None, c.attention(qd, st, 128 ** -0.5, "fp16"))
    check(mqa.kv_attention(q, dev, ints(st), selected=ints(sel)), None, c.attention(qd, st, 128 ** -0.5, "fp16", sel))


@pytest.mark.parametrize("case", [(1, 72, 64, [90, 3], [2, 1]), (2, 128, 128, [300, 40], [1, 5]),
                                  (1, 300, 64, [200, 129], [1, 3]), (256, 1, 64, [20, 33], [1, 20])], ids=str)
def test_many_query_heads(mqa, case):
    """Groups beyond a block's columns (one row in several blocks), and many key/value heads."""
    heads, group, dim, lens, rows = case
    rng = np.random.default_rng(76)
    c = ref.random_cache(rng, 40, heads, 16, dim, lens, 20)
    for max_rows in (None, 1):
        attend(mqa, c, rng, rows, group, "bf16", max_rows=max_rows)
    attend(mqa, c, rng, rows, group, "fp16", selected=random_selection(rng, c, rows, 25))
    attend(mqa, c, rng, rows, group, "fp16", False, selected=random_selection(rng, c, rows, 25))


def test_decreasing_bounds_give_the_others_their_rows(mqa):
    """A bound below the one before it leaves its sequence without rows; the others' rows are answered."""
    import torch
    rng = np.random.default_rng(77)
    c = ref.random_cache(rng, 30, 1, 16, 64, [50, 40, 30], 8)
    dev = ref.to_device(c, mqa)
    for n, group in ((4, 4), (70, 4)):
        q, qd = rows_of(rng, n, group, 64, "bf16")
        out = torch.zeros_like(q)
        mqa.kv_attention(q, dev, ints([3, 1, n, n]), out=out)  # sequence 1: rows [1, n)
        want = c.attention(qd[1:], np.array([0, 0, n - 1, n - 1]), 0.125, "bf16")
        check(out[1:], None, want)
        assert not out[0].any() and mqa.kv_status(dev) == 0


def test_rows_past_32_bits(mqa):
    """More than 2^32 bytes of queries, outputs and new rows: the last of them are read and written where they lie."""
    import torch
    rng = np.random.default_rng(78)
    base, rows = (1 << 24) + 3, [40, 1]
    c = ref.random_cache(rng, 30, 1, 64, 128, [300, 129], 6)
    dev = ref.to_device(c, mqa)
    n = sum(rows)
    st = starts_of(rows)
    starts = ints(st + base)
    k = torch.zeros((base + n, 1, 128), dtype=torch.bfloat16, device="cuda")
    kn, kd = rows_of(rng, n, 1, 128, "bf16")
    k[base:] = kn
    mqa.kv_append(dev, k, k, starts)
    c.append(kd, kd, st)
    assert ref.same(c, dev) == []
    del k
    q = torch.zeros((base + n, 2, 128), dtype=torch.bfloat16, device="cuda")
    qn, qd = rows_of(rng, n, 2, 128, "bf16")
    q[base:] = qn
    sel = random_selection(rng, c, rows, 20)
    out = torch.zeros_like(q)
    for max_rows, s in ((None, None), (1, None), (None, sel)):
        wide = None
        if s is not None:
            wide = torch.zeros((base + n, 20), dtype=torch.int32, device="cuda")
            wide[base:] = ints(s)
        out.zero_()
        mqa.kv_attention(q, dev, starts, selected=wide, max_rows=max_rows, out=out)
        check(out[base:], None, c.attention(qd, st, 128 ** -0.5, "bf16", s))
        assert not out[:base].any() and mqa.kv_status(dev) == 0


def test_as_many_sequences_as_there_may_be(mqa):
    import torch
    rng = np.random.default_rng(79)
    n = 65536
    lens, rows = np.zeros(n, np.int64), np.zeros(n, np.int64)
    pick = rng.choice(n, 60, replace=False)
    pick[:2] = 0, n - 1
    lens[pick] = rng.integers(1, 90, 60)
    rows[pick] = np.minimum(lens[pick], rng.integers(1, 60, 60))
    lens[pick[5]], rows[pick[5]] = 700, 300
    c = ref.random_cache(rng, 600, 1, 16, 64, lens, 45)
    _, dev, _, st = attend(mqa, c, rng, rows, 4)
    attend(mqa, c, rng, rows, 4, "fp16", max_rows=2)
    attend(mqa, c, rng, rows, 4, selected=random_selection(rng, c, rows, 20))
    counts = np.zeros(n, np.int32)
    counts[pick] = rng.integers(0, 9, 60)
    mqa.kv_reserve(dev, ints(counts))
    assert c.reserve(counts) == 0 and mqa.kv_status(dev) == 0
    k, kd = rows_of(rng, int(counts.sum()), 1, 64, "fp32")
    st = starts_of(counts)
    mqa.kv_append(dev, k, k, ints(st))
    c.append(kd, kd, st)
    assert ref.same(c, dev) == []


def test_a_decode_step_in_a_graph(mqa):
    """Room, a token's keys and values and its attention, captured once on a stream of its own and replayed while the
    sequences grow over their pages; then a fork, a return and a packing, captured as well."""
    import torch
    rng = np.random.default_rng(80)
    c = ref.random_cache(rng, 60, 2, 16, 64, [14, 31, 0, 1], 8)
    dev = ref.to_device(c, mqa)
    counts = np.array([1, 1, 0, 2], np.int32)
    st = starts_of(counts)
    k, v, q = (torch.zeros((4, h, 64), dtype=torch.bfloat16, device="cuda") for h in (2, 2, 8))
    dcounts, dst = ints(counts), ints(st)
    ws, out = mqa.alloc_kv_workspace(dev, 4, 8), torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step, pages = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    mqa.kv_attention(q, dev, dst, workspace=ws, out=out, stream=side)
    side.synchronize()
    with torch.cuda.graph(step, stream=side):
        mqa.kv_reserve(dev, dcounts)
        mqa.kv_append(dev, k, v, dst)
        mqa.kv_attention(q, dev, dst, workspace=ws, out=out)
    parents, children, gone = ints([1]), ints([2]), ints([0])
    with torch.cuda.graph(pages, stream=side):
        mqa.kv_fork(dev, parents, children)
        mqa.kv_free(dev, gone)
        mqa.kv_compact(dev)
    torch.cuda.synchronize()
    for i in range(20):
        kn, vn, qn = (rows_of(rng, 4, h, 64, "bf16") for h in (2, 2, 8))
        for t, x in ((k, kn), (v, vn), (q, qn)):
            t.copy_(x[0])
        step.replay()
        torch.cuda.synchronize()
        assert c.reserve(counts) == 0
        c.append(kn[1], vn[1], st)
        assert ref.same(c, dev) == [], i
        check(out, None, c.attention(qn[1], st, 0.125, "bf16"), i)
    pages.replay()
    torch.cuda.synchronize()
    assert c.fork(np.array([1]), np.array([2])) == 0
    c.free([0])
    c.compact()
    assert ref.same(c, dev) == [] and mqa.kv_status(dev) == 0
