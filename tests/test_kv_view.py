"""Windows, trees, accepted rows and head rotation without a GPU: the plain forms, the C entries' refusals (found on the
host before any work, so fake addresses are safe), and the binding's."""
import ctypes
import math
import re

import numpy as np
import pytest

import kv_reference as ref
import sparse_attention_indexer_relu_gb300 as mqa
import view_reference as view
from sparse_attention_indexer_relu_gb300 import kv_cache as kv
from sparse_attention_indexer_relu_gb300 import qk_rope as qk
from test_kv_cache import BAD_CACHES, OnDevice, cache, fake_cache

torch = pytest.importorskip("torch")
P = ctypes.c_void_p


# ---------------------------------------------------------------- plain forms
def test_plain_views():
    rng = np.random.default_rng(1)
    c = ref.random_cache(rng, 9, 1, 16, 64, [37, 5], 4)
    st = np.array([0, 3, 8])
    assert view.window_seen(c, st, 4, 2)[0].tolist() == [0, 1, 31, 32, 33, 34]
    assert view.window_seen(c, st, 4, 2)[3].tolist()[:2] == [0, -1]
    parents = np.array([-1, 0, 0, -1, 0, 1, 1, 3], np.int32)
    mask, pos = view.tree_mask(c, st, parents, 1)
    assert mask[:, 0].tolist() == [1, 3, 5, 1, 3, 7, 11, 27] and pos.tolist() == [34, 35, 35, 0, 1, 2, 2, 3]
    assert view.tree_seen(c, st, mask)[2].tolist() == list(range(34)) + [34, 36]
    assert [t for t in view.tree_seen(c, st, mask)[7] if t >= 0] == [0, 1, 3, 4]


def test_plain_acceptance_keeps_values():
    rng = np.random.default_rng(2)
    c = ref.random_cache(rng, 9, 2, 16, 64, [37, 20], 4, spread=0)
    was = [c.values(0, h, "k").copy() for h in range(2)]
    view.accept(c, np.array([0, 8, 8]), np.array([3, 0]), np.array([1, 4, 7, 0, 0, 0, 0, 0]))
    assert c.lens.tolist() == [32, 20] and c.table[0, 2] == -1 and (c.refs[c.table[0, :2]] == 1).all()
    for h in range(2):
        assert np.array_equal(c.values(0, h, "k"), was[h][list(range(29)) + [30, 33, 36]])


# ---------------------------------------------------------------- refusals of the C entries
def call(c=None, q=0x1000, stride=4096, type=0, heads=32, starts=0x2000, rows=8, max_rows=0, window=0, sinks=0, tree=0,
         words=0, scale=0.1, out=0x3000, lse=0, ws=0x100000, ws_bytes=1 << 40, view=True):
    v = kv._View(window, sinks, tree, words)
    return mqa.lib().mqa_kv_attention_view(ctypes.byref(c or cache()), P(q), stride, type, heads, P(starts), rows, max_rows,
                                           ctypes.byref(v) if view else None, scale, P(out), P(lse), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(view=False), 1), (dict(window=-1), 1), (dict(window=5, sinks=-1), 1), (dict(sinks=4), 1),
    (dict(tree=0x5000), 1), (dict(tree=0x5000, words=-1), 1), (dict(words=2), 1),
    (dict(tree=0x5000, words=2, window=9), 1), (dict(tree=0x5002, words=2), 2), (dict(rows=-1, window=4), 1),
    (dict(type=2, window=4), 1), (dict(heads=30, window=4), 1), (dict(scale=0.0, window=4), 1), (dict(q=0, window=4), 1),
    (dict(stride=4100, window=4), 2), (dict(ws=0x100010, tree=0x5000, words=1), 2), (dict(rows=0, window=4), 0),
    (dict(rows=0, window=-4), 1), (dict(rows=0), 0)])
def test_view_refusals(kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_every_new_entry_refuses_a_bad_cache(change, code):
    L, c = mqa.lib(), cache(**change)
    r = ctypes.byref(c)
    assert call(c, window=5) == code and call(c, tree=0x5000, words=1) == code
    assert L.mqa_kv_tree_mask(r, P(0x1000), P(0x2000), 8, P(0x3000), 1, P(0x4000), None) == code
    assert L.mqa_kv_accept(r, P(0x1000), 8, P(0x2000), P(0x3000), None) == code


def test_mask_and_accept_refusals():
    L, r = mqa.lib(), ctypes.byref(cache())
    f = lambda parents=0x1000, st=0x2000, rows=8, mask=0x3000, words=1, pos=0x4000: L.mqa_kv_tree_mask(  # noqa: E731
        r, P(parents), P(st), rows, P(mask), words, P(pos), None)
    assert f(rows=-1) == 1 and f(words=0) == 1 and f(parents=0) == 1 and f(st=0) == 1 and f(mask=0) == 1
    assert f(parents=0x1002) == 2 and f(st=0x2001) == 2 and f(mask=0x3002) == 2 and f(pos=0x4001) == 2
    assert f(rows=0, parents=0, mask=0) == 0
    g = lambda st=0x1000, rows=8, counts=0x2000, acc=0x3000, c=r: L.mqa_kv_accept(  # noqa: E731
        c, P(st), rows, P(counts), P(acc), None)
    assert g(rows=-1) == 1 and g(st=0) == 1 and g(counts=0) == 1 and g(st=0x1001) == 2 and g(counts=0x2002) == 2
    assert g(acc=0x3002) == 2 and g(rows=0, st=0) == 0 and g(c=ctypes.byref(cache(refcounts=0))) == 1


def heads(at=0x1000, out=0x2000, weight=0, si=1024, so=1024, n=8):
    return qk._Heads(at, out, weight, si, so, n)


def rotate(q=None, k=None, rows=8, type=0, wt=0, dim=128, rotary=128, eps=1e-6, turns=0x3000, pos=0x4000):
    return mqa.lib().mqa_qk_norm_rope(ctypes.byref(q or heads()), ctypes.byref(k or heads()), rows, type, wt, dim, rotary, 0,
                                      1, eps, P(turns), P(pos), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(type=3), 1), (dict(type=-1), 1), (dict(wt=3), 1), (dict(dim=96), 1), (dict(dim=512), 1),
    (dict(rotary=8), 1), (dict(rotary=136), 1), (dict(rotary=144), 1), (dict(rotary=-16), 1), (dict(eps=-1.0), 1),
    (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(turns=0), 1), (dict(pos=0), 1), (dict(turns=0x3004), 2),
    (dict(pos=0x4002), 2), (dict(q=heads(at=0)), 1), (dict(k=heads(out=0)), 1), (dict(q=heads(n=-1)), 1),
    (dict(q=heads(n=65537)), 1), (dict(q=heads(si=1016)), 1), (dict(k=heads(so=1000)), 1), (dict(q=heads(si=1028)), 2),
    (dict(q=heads(at=0x1008)), 2), (dict(k=heads(out=0x2004)), 2), (dict(k=heads(weight=0x5008)), 2),
    (dict(rows=1 << 28), 1), (dict(rows=0), 0), (dict(q=heads(n=0), k=heads(n=0)), 0), (dict(rows=0, dim=96), 1)])
def test_rotation_refusals(kw, code):
    assert rotate(**kw) == code


def test_exports():
    text = open(mqa.HEADER_PATH.replace("mqatopk.h", "mqaqk.h")).read()
    names = set(re.findall(r"\b(mqa_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(qk.QK_EXPORTS)
    assert all(hasattr(ctypes.CDLL(mqa.LIB_PATH), n) for n in names)


# ---------------------------------------------------------------- the binding
def test_binding_refuses_views_that_do_not_go_together():
    i32, c = torch.int32, fake_cache()
    q, st = OnDevice(5, 2, 64, dtype=torch.bfloat16), OnDevice(4, dtype=i32)
    sel, tree = OnDevice(5, 7, dtype=i32), OnDevice(5, 1, dtype=i32)
    for kw in (dict(window=0), dict(window=-3), dict(window=2 ** 31), dict(sinks=4), dict(window=4, sinks=-1),
               dict(window=4, causal=False), dict(window=4, selected=sel), dict(tree=tree, selected=sel),
               dict(tree=tree, window=4), dict(tree=tree, sinks=1), dict(tree=tree, causal=False),
               dict(window=4, debug={}), dict(tree=OnDevice(4, 1, dtype=i32)), dict(tree=OnDevice(5, 0, dtype=i32)),
               dict(tree=OnDevice(5, dtype=i32))):
        with pytest.raises(ValueError):
            mqa.kv_attention(q, c, st, **kw)
    with pytest.raises(TypeError):
        mqa.kv_attention(q, c, st, tree=OnDevice(5, 1, dtype=torch.int64))
    q.requires_grad = True
    with pytest.raises(ValueError, match="requires a gradient"):
        mqa.kv_attention(q, c, st, window=4)


def test_binding_refuses_bad_lists():
    i32, c = torch.int32, fake_cache()
    st, counts, par = OnDevice(4, dtype=i32), OnDevice(3, dtype=i32), OnDevice(5, dtype=i32)
    for args, kw in (((c, par, st, 0), {}), ((c, par, OnDevice(3, dtype=i32), 4), {}),
                     ((c, par, st, 4), dict(mask=OnDevice(5, 2, dtype=i32))),
                     ((c, par, st, 4), dict(mask=OnDevice(5, 1, dtype=i32), positions=OnDevice(4, dtype=i32)))):
        with pytest.raises(ValueError):
            mqa.kv_tree_mask(*args, **kw)
    with pytest.raises(TypeError):
        mqa.kv_tree_mask(c, OnDevice(5, dtype=torch.int64), st, 4)
    for args, kw in (((c, st, counts), {}), ((c, st, OnDevice(4, dtype=i32), par), {}),
                     ((c, OnDevice(5, dtype=i32), counts, par), {}), ((c, st, counts, par), dict(rows=6))):
        with pytest.raises(ValueError):
            mqa.kv_accept(*args, **kw)


class Rows(OnDevice):
    def get_device(self):
        return 0

    def stride(self, i=None):
        return [self.shape[j + 1:].numel() for j in range(len(self.shape))] if i is None else super().stride(i)


def test_binding_refuses_bad_heads():
    bf, f32 = torch.bfloat16, torch.float32
    on = lambda *s, dtype=bf: Rows(*s, dtype=dtype)  # noqa: E731
    turns, pos = Rows(64, dtype=torch.int64), Rows(5, dtype=torch.int32)
    q, k = on(5, 4, 128), on(5, 2, 128)
    f = lambda q=q, k=k, t=turns, p=pos, **kw: mqa.qk_norm_rope(q, k, t, p, **kw)  # noqa: E731
    out = dict(q_out=on(5, 4, 128), k_out=on(5, 2, 128))
    for bad in (dict(q=on(5, 4, 96), k=on(5, 2, 96)), dict(k=on(4, 2, 128)), dict(k=on(5, 2, 64)), dict(t=None),
                dict(p=None), dict(p=Rows(4, dtype=torch.int32)), dict(q_weight=on(64)),
                dict(q_out=on(5, 3, 128), k_out=on(5, 2, 128))):
        with pytest.raises(ValueError):
            f(**{**out, **bad})
    for bad in (dict(q=on(5, 4, 128, dtype=torch.int32)), dict(k=on(5, 2, 128, dtype=f32)),
                dict(t=Rows(64, dtype=f32)), dict(p=Rows(5, dtype=torch.int64)),
                dict(q_weight=on(128), k_weight=on(128, dtype=f32)), dict(k_weight=on(128, dtype=torch.int32))):
        with pytest.raises(TypeError):
            f(**{**out, **bad})
    q.requires_grad = True
    with pytest.raises(ValueError, match="q requires a gradient"):
        f(**out)
    q.requires_grad = False
    w = on(128)
    w.requires_grad = True
    with pytest.raises(ValueError, match="k_weight requires a gradient"):
        f(k_weight=w, **out)
    host = torch.zeros((5, 4, 128), dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        mqa.qk_norm_rope(host, host, None, None)


def test_turns():
    """64-bit fractions of a turn: wraps, signs, and the angle of far positions."""
    f = torch.tensor([0.0, math.pi, 2 * math.pi, 1.0, 1e-6, -1.0], dtype=torch.float64)
    t = mqa.rope_turns(f, device="cpu").tolist()
    assert t[0] == 0 and abs(abs(t[1]) - 2 ** 63) < 2 ** 12 and abs(t[2]) < 2 ** 13 and abs(t[3] + t[5]) <= 1
    for p in (1, 1000, 2 ** 31 - 1):
        turn = (p * t[3]) % 2 ** 64 / 2 ** 64
        exact = (p * 0.159154943091895335768883763372514362) % 1.0
        assert abs(turn - exact) < 1e-6
    with pytest.raises(TypeError):
        mqa.rope_turns(torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        mqa.rope_turns(torch.zeros(4, 2))


@pytest.mark.parametrize("opt,code", [(dict(stall=3), 1), (dict(stall=-1), 1), (dict(wait_timeout_ms=10001), 1),
                                      (dict(wait_timeout_ms=-1), 1)])
def test_debug_options_of_views_are_checked(opt, code):
    v = kv._View(5, 0, None, 0)
    entry = lambda view: mqa.lib().mqa_kv_attention_view_debug(  # noqa: E731
        ctypes.byref(cache()), P(0x1000), 4096, 0, 32, P(0x2000), 8, 0, view, 0.1, P(0x3000), P(0), P(0x100000), 1 << 40,
        None, ctypes.byref(kv.KVDebugOptions(**opt)))
    assert entry(ctypes.byref(v)) == code and entry(None) == 1
