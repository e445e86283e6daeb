"""Norm and rotation of query and key heads on the GPU, against the formula in 64 bits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": 2.0 ** -24}  # half a step, relative
TINY = {"bfloat16": 2.0 ** -134, "float16": 2.0 ** -25, "float32": 2.0 ** -126}  # half the least step (fp32: flushed)


@pytest.fixture(scope="module")
def mqa():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_attention_indexer_relu_gb300 as m
    m.lib()
    return m


def plain(x, w, eps, norm, inv_freq, positions, interleaved, dtype):
    """(result, bound).  A head's factor: 13 fp32 sums, a product and a sum under a root (half their 2^-24 each), rsqrt
    (2^-22), two products: below 2^-20 of a component.  sin and cos: the angle rounded to 2^-25 of a half turn, then 2
    ulp: below 2^-22.  The turned pair: two products and a sum.  In all below 2^-19 of |a| + |b|."""
    x = x.astype(np.float64)
    y = x if not norm else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = y * w
    out, mag = y.copy(), np.abs(y)
    if inv_freq is not None:
        r = 2 * len(inv_freq)
        # the fraction of a turn, in whole numbers: positions are exact, frequencies are given in 64 bits
        angle = np.array([[float(np.remainder(np.longdouble(p) * np.longdouble(f), 2 * np.longdouble(np.pi)))
                           for f in inv_freq] for p in positions]).reshape(len(positions), -1)[:, None]
        cos, sin = np.cos(angle), np.sin(angle)
        a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
        out[..., a], out[..., b] = y[..., a] * cos - y[..., b] * sin, y[..., b] * cos + y[..., a] * sin
        mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, mag * 2.0 ** -19 + np.abs(out) * U[dtype] * 1.01 + TINY[dtype]


def run(mqa, rows, hq, hk, dim, rotary, dtype, interleaved=False, norm=True, weights=True, far=100000, eps=1e-6,
        weight_type=None, seed=0, scale=1.5):
    import torch
    rng = np.random.default_rng(seed + rows + dim)
    t = getattr(torch, dtype)
    qkv = (torch.from_numpy(rng.standard_normal((rows, hq + 2 * hk, dim))) * scale).to(t).cuda()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    wt = t if weight_type is None else getattr(torch, weight_type)
    w = [(torch.from_numpy(1 + 0.3 * rng.standard_normal(dim))).to(wt).cuda() if weights else None for _ in range(2)]
    inv = 500000.0 ** (-np.arange(0, rotary, 2) / max(rotary, 1)) if rotary else None
    turns = mqa.rope_turns(torch.from_numpy(inv)) if rotary else None
    pos = rng.integers(-far // 10, far, rows)
    positions = torch.from_numpy(pos.astype(np.int32)).cuda() if rotary else None
    before = qkv.clone()
    got = mqa.qk_norm_rope(q, k, turns, positions, w[0], w[1], eps=eps, norm=norm, interleaved=interleaved)
    assert torch.equal(qkv, before)
    for x, y, weight in zip((q, k), got, w):
        wd = 1.0 if weight is None else weight.double().cpu().numpy()
        out, tol = plain(x.double().cpu().numpy(), wd, eps, norm, inv, pos, interleaved, dtype)
        bad = np.abs(y.double().cpu().numpy() - out) > tol
        assert y.shape == x.shape and y.dtype == t
        assert not bad.any(), (np.argwhere(bad)[:4], y.double().cpu().numpy()[bad][:4], out[bad][:4], tol[bad][:4])
    return qkv, turns, positions, w, got


CASES = [  # rows, q heads, k heads, dim, rotary
    (1, 32, 8, 128, 128), (1, 1, 1, 64, 64), (3, 5, 1, 64, 32), (7, 4, 4, 256, 256), (33, 3, 2, 128, 16),
    (100, 1, 1, 64, 48), (257, 7, 1, 128, 96), (1000, 40, 8, 128, 64), (9, 6, 3, 256, 80), (50, 2, 1, 128, 0),
    (2049, 1, 1, 256, 16)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_and_rotation(mqa, case, dtype, interleaved):
    run(mqa, *case, dtype, interleaved)


@pytest.mark.parametrize("kw", [dict(norm=False), dict(weights=False), dict(norm=False, weights=False),
                                dict(weight_type="float32"), dict(weight_type="float16"), dict(eps=0.0), dict(eps=3.0)],
                         ids=str)
def test_forms(mqa, kw):
    run(mqa, 20, 6, 2, 128, 128, "bfloat16", **kw)


def test_far_positions(mqa):
    run(mqa, 64, 2, 1, 128, 128, "float32", far=2 ** 31 - 1)


@pytest.mark.parametrize("scale", [1e30, 1e-30, 2.0 ** -120])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_heads_whose_squares_leave_the_range(mqa, scale, eps):
    run(mqa, 9, 6, 2, 64, 64, "bfloat16", scale=scale, eps=eps)


def test_values_that_are_no_numbers_stay_in_their_head(mqa):
    import torch
    qkv, turns, pos, w, _ = run(mqa, 5, 6, 2, 128, 64, "bfloat16")
    clean = mqa.qk_norm_rope(qkv[:, :6], qkv[:, 6:8], turns, pos, *w)
    x = qkv.clone()
    x[1, 2, 7], x[3, 7, 100], x[4, 0] = float("nan"), float("inf"), 0
    q, k = mqa.qk_norm_rope(x[:, :6], x[:, 6:8], turns, pos, *w)
    assert q[1, 2].isnan().all() and k[3, 1, 100].isnan() and not q[4, 0].any()
    for a, b, skip in ((q, clean[0], [(1, 2), (4, 0)]), (k, clean[1], [(3, 1)])):
        keep = torch.ones(a.shape[:2], dtype=torch.bool)
        for s in skip:
            keep[s] = False
        assert torch.equal(a[keep], b[keep])


def test_in_place_strided_and_one_of_the_two(mqa):
    import torch
    qkv, turns, pos, w, (q, k) = run(mqa, 70, 6, 2, 128, 128, "bfloat16")
    x = qkv.clone()
    a, b = mqa.qk_norm_rope(x[:, :6], x[:, 6:8], turns, pos, *w, q_out=x[:, :6], k_out=x[:, 6:8])
    assert a.data_ptr() == x.data_ptr() and torch.equal(x[:, :6], q) and torch.equal(x[:, 6:8], k)
    assert torch.equal(x[:, 8:], qkv[:, 8:])  # the values are not touched
    only = mqa.qk_norm_rope(qkv[:, :6], qkv[:, :0], turns, pos, w[0])
    assert torch.equal(only[0], q) and only[1].shape == (70, 0, 128)
    only = mqa.qk_norm_rope(qkv[:, :0], qkv[:, 6:8], turns, pos, None, w[1])
    assert torch.equal(only[1], k)
    none = mqa.qk_norm_rope(qkv[:0, :6], qkv[:0, 6:8], turns, pos[:0], *w)
    assert none[0].shape == (0, 6, 128)


def test_on_a_side_stream_and_in_a_graph(mqa):
    import torch
    qkv, turns, pos, w, want = run(mqa, 70, 6, 2, 128, 128, "bfloat16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mqa.qk_norm_rope(qkv[:, :6], qkv[:, 6:8], turns, pos, *w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, p = torch.zeros_like(qkv), torch.zeros_like(pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mqa.qk_norm_rope(x[:, :6], x[:, 6:8], turns, p, *w)
    x.copy_(qkv)
    p.copy_(pos)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_rows_past_32_bits(mqa):
    """More than 2^32 bytes of rows: the last of them are read and written where they lie."""
    import torch
    rows, n = (1 << 20) + 5, 16
    x = torch.zeros((rows, n + 2, 128), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, n + 2, 128), device="cuda").bfloat16()
    turns = mqa.rope_turns(torch.tensor([1.0] * 64, dtype=torch.float64))
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    q, k = mqa.qk_norm_rope(x[:, :n], x[:, n:n + 1], turns, pos)
    few = mqa.qk_norm_rope(x[-3:, :n], x[-3:, n:n + 1], turns, pos[-3:])
    assert torch.equal(q[-3:], few[0]) and torch.equal(k[-3:], few[1]) and not q[:-3].any() and few[0].any()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("scale,weight", [(1e18, 1e21), (1e-25, 1e-20), (1.0, 1e37), (1e12, 1e-37)])
def test_weights_whose_products_with_rows_leave_the_range(mqa, dtype, scale, weight):
    """The norm's answer times the weight stays in fp32's range although row times weight does not."""
    import torch
    rng = np.random.default_rng(3)
    t = getattr(torch, dtype)
    q = (torch.from_numpy(rng.standard_normal((9, 6, 64))) * scale).to(t).cuda()
    k = q[:, :2].clone()
    w = [(torch.from_numpy(1 + 0.3 * rng.random(64)) * weight).to(t).cuda() for _ in range(2)]
    inv, pos = 10000.0 ** (-np.arange(0, 64, 2) / 64), np.arange(9) * 100
    turns, positions = mqa.rope_turns(torch.from_numpy(inv)), torch.from_numpy(pos.astype(np.int32)).cuda()
    got = mqa.qk_norm_rope(q, k, turns, positions, *w, eps=0.0)
    for x, y, v in zip((q, k), got, w):
        out, tol = plain(x.double().cpu().numpy(), v.double().cpu().numpy(), 0.0, True, inv, pos, False, dtype)
        assert np.abs(out).max() < 1e39 and (np.abs(y.double().cpu().numpy() - out) <= tol).all()


@pytest.mark.parametrize("eps", [1e-40, 2.0 ** -149, 1e-38, 1e-30])
def test_heads_of_zeros_under_the_least_eps(mqa, eps):
    """0 / sqrt(0 + eps) is 0 for every eps above 0, and heads of such sizes are divided as the formula has it."""
    import torch
    q = torch.zeros((5, 3, 64), device="cuda")
    q[1] = torch.from_numpy(np.random.default_rng(4).standard_normal((3, 64)) * eps ** 0.5).float().cuda()
    got, _ = mqa.qk_norm_rope(q, q[:, :1], None, None, eps=eps)
    eps = float(np.float32(eps))
    out, tol = plain(q.double().cpu().numpy(), 1.0, eps, True, None, None, False, "float32")
    assert (np.abs(got.double().cpu().numpy() - out) <= tol).all() and not got[0].any() and not got[2:].any()
    zeros = mqa.qk_norm_rope(q, q[:, :1], None, None, eps=0.0)[0]
    assert zeros[0].isnan().all() and zeros[1].isfinite().all()
