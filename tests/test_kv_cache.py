"""The paged 8-bit cache without a GPU: the plain forms against independent facts, the C entries' refusals (found on
the host before any work, so fake addresses are safe), and the binding's."""
import ctypes
import re

import numpy as np
import pytest

import kv_reference as ref
import sparse_attention_indexer_relu_gb300 as mqa
from sparse_attention_indexer_relu_gb300 import kv_cache as kv

torch = pytest.importorskip("torch")
P = ctypes.c_void_p


# ---------------------------------------------------------------- plain forms
def test_codes_round_as_torch_rounds():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * s for s in (0.001, 0.02, 1, 100, 300)] + [ref.E4M3[:127]])
    x = x.astype(np.float32).clip(-448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.round_e4m3(x), want)
    mid = (ref.E4M3[:126] + ref.E4M3[1:127]) / 2  # ties
    want = torch.from_numpy(mid.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.round_e4m3(mid), want)


@pytest.mark.parametrize("amax,want", [(448.0, 127), (448.0001, 128), (224.0, 126), (1.75, 119), (0.0, 7),
                                       (3.3e38, 247), (1e-40, 7), (896.0, 128)])
def test_needed_exponent(amax, want):
    assert ref.need_exp(amax) == want


def test_plain_attention_against_a_full_softmax():
    rng = np.random.default_rng(2)
    c = ref.random_cache(rng, 9, 2, 16, 64, [37, 0, 20], 4)
    q = rng.standard_normal((7, 4, 64))
    starts = np.array([0, 5, 5, 7])
    out, lse, tol, _ = c.attention(q, starts, 0.125, "bf16")
    k, v = c.values(0, 1, "k"), c.values(0, 1, "v")
    s = 0.125 * k[:35] @ q[2, 3]  # row 2 of 5 is position 34
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(out[2, 3], w @ v[:35], rtol=1e-12) and np.isclose(lse[2, 3], np.log(np.exp(s).sum()))
    assert (tol > 0).all()


# ---------------------------------------------------------------- refusals of the C entries
def test_exports_every_declared_symbol():
    text = open(mqa.HEADER_PATH.replace("mqatopk.h", "mqakv.h")).read()
    names = set(re.findall(r"\b(mqa_kv_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(kv.KV_EXPORTS)
    lib = ctypes.CDLL(mqa.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)


def cache(**kw):
    a = dict(k=0x10000, v=0x20000, k_exps=0x30000, v_exps=0x30100, page_table=0x40000, seq_lens=0x50000,
             refcounts=0x60000, scratch=0x70000, scratch_bytes=1 << 30, num_pages=100, page_size=64, kv_heads=8,
             head_dim=128, max_seqs=4, max_pages=16, n_extra=0)
    a.update(kw)
    return kv._Cache(**a)


BAD_CACHES = [(dict(num_pages=0), 1), (dict(page_size=48), 1), (dict(page_size=256), 1), (dict(kv_heads=0), 1),
              (dict(kv_heads=257), 1), (dict(head_dim=96), 1), (dict(max_seqs=0), 1), (dict(max_seqs=65537), 1),
              (dict(max_pages=0), 1), (dict(n_extra=5), 1), (dict(n_extra=-1), 1), (dict(n_extra=1), 1),
              (dict(num_pages=1 << 22), 1), (dict(max_pages=1 << 25), 1), (dict(k=0), 1), (dict(v_exps=0), 1),
              (dict(scratch=0), 1), (dict(k=0x10008), 2), (dict(scratch=0x70010), 2), (dict(scratch_bytes=300), 3)]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_every_entry_refuses_a_bad_cache(change, code):
    L, c = mqa.lib(), cache(**change)
    r = ctypes.byref(c)
    n = ctypes.c_size_t()
    assert L.mqa_kv_append(r, P(0x1000), P(0x2000), 1024, 1024, 0, P(0x3000), 8, None) == code
    assert L.mqa_kv_attention_workspace_bytes(0, r, 8, 32, ctypes.byref(n)) == code
    assert attention(c) == code
    assert L.mqa_kv_reserve(r, P(0x1000), None) == code
    assert L.mqa_kv_fork(r, P(0x1000), P(0x1000), 1, None) == code
    assert L.mqa_kv_free(r, P(0x1000), 1, None) == code
    assert L.mqa_kv_compact(r, None) == code
    assert L.mqa_kv_copy_pages(r, P(0x1000), P(0x1000), 1, None) == code


def attention(c=None, q=0x1000, stride=4096, type=0, heads=32, starts=0x2000, rows=8, max_rows=0, sel=0, nsel=0,
              scale=0.1, out=0x3000, lse=0, ws=0x100000, ws_bytes=1 << 40):
    c = c or cache()
    return mqa.lib().mqa_kv_attention(ctypes.byref(c), P(q), stride, type, heads, P(starts), rows, max_rows, P(sel),
                                      nsel, 1, scale, P(out), P(lse), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(type=2), 1), (dict(type=-1), 1), (dict(heads=30), 1), (dict(heads=0), 1),
    (dict(heads=1 << 17), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(scale=65537.0), 1), (dict(scale=-1.0), 1),
    (dict(nsel=-1, sel=0x1000), 1), (dict(nsel=5), 1), (dict(q=0), 1), (dict(out=0), 1), (dict(starts=0), 1),
    (dict(ws=0), 1), (dict(stride=4088), 1), (dict(stride=4100), 2), (dict(q=0x1008), 2), (dict(out=0x3004), 2),
    (dict(starts=0x2002), 2), (dict(sel=0x1002, nsel=5), 2), (dict(lse=0x1002), 2), (dict(ws=0x100010), 2)])
def test_attention_refusals(kw, code):
    assert attention(**kw) == code


def test_calls_without_work_are_no_ops():
    L, r = mqa.lib(), ctypes.byref(cache())
    assert attention(rows=0) == 0
    assert L.mqa_kv_append(r, None, None, 0, 0, 0, None, 0, None) == 0
    assert L.mqa_kv_fork(r, None, None, 0, None) == 0
    assert L.mqa_kv_free(r, None, 0, None) == 0
    assert L.mqa_kv_copy_pages(r, None, None, 0, None) == 0


def test_append_refusals():
    L, r = mqa.lib(), ctypes.byref(cache())
    f = lambda k=0x1000, v=0x2000, ks=1024, vs=1024, ty=0, st=0x3000, rows=8: L.mqa_kv_append(  # noqa: E731
        r, P(k), P(v), ks, vs, ty, P(st), rows, None)
    assert f(rows=-1) == 1 and f(ty=3) == 1 and f(ty=-1) == 1 and f(k=0) == 1 and f(v=0) == 1 and f(st=0) == 1
    assert f(ks=1016) == 1 and f(vs=0) == 1 and f(ks=1028) == 2 and f(k=0x1008) == 2 and f(st=0x3001) == 2
    assert f(ty=2, ks=1030) == 2


def test_page_operation_refusals():
    L, c = mqa.lib(), cache()
    r = ctypes.byref(c)
    assert L.mqa_kv_reserve(r, None, None) == 1 and L.mqa_kv_reserve(r, P(0x1001), None) == 2
    assert L.mqa_kv_fork(r, P(0x1000), P(0x1000), 5, None) == 1  # more children than sequences
    assert L.mqa_kv_fork(r, P(0x1000), P(0x1000), -1, None) == 1
    assert L.mqa_kv_fork(r, None, P(0x1000), 1, None) == 1 and L.mqa_kv_fork(r, P(0x1002), P(0x1000), 1, None) == 2
    assert L.mqa_kv_free(r, P(0x1000), -1, None) == 1 and L.mqa_kv_free(r, None, 1, None) == 1
    assert L.mqa_kv_copy_pages(r, P(0x1000), P(0x1000), 101, None) == 1
    assert L.mqa_kv_copy_pages(r, P(0x1000), None, 1, None) == 1
    for change in (dict(refcounts=0), dict(page_table=0), dict(seq_lens=0)):
        c2 = ctypes.byref(cache(**change))
        assert L.mqa_kv_reserve(c2, P(0x1000), None) == 1 and L.mqa_kv_compact(c2, None) == 1
        assert L.mqa_kv_free(c2, P(0x1000), 1, None) == 1
    assert L.mqa_kv_get_status(r, None, None) == 1


def test_scratch_bytes():
    n = ctypes.c_size_t()
    assert mqa.lib().mqa_kv_scratch_bytes(0, 1, ctypes.byref(n)) == 1
    assert mqa.lib().mqa_kv_scratch_bytes(1, 65537, ctypes.byref(n)) == 1
    assert mqa.lib().mqa_kv_scratch_bytes(1, 1, None) == 1
    assert mqa.kv_scratch_bytes(1000, 10) >= 256 + 3 * 4 * 1000 + 2 * 4 * 10


def test_binding_refuses_host_tensors():
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError):
        mqa.KVCache(z(4, 2, 16, 64), z(4, 2, 16, 64), z(4, 2), z(4, 2), z(2, 3, dtype=torch.int32),
                    z(2, dtype=torch.int32))


@pytest.mark.parametrize("opt,code", [(dict(stall=3), 1), (dict(stall=-1), 1), (dict(wait_timeout_ms=-1), 1),
                                      (dict(wait_timeout_ms=10001), 1), (dict(stall=2, wait_timeout_ms=10000), 0)])
def test_debug_options_are_checked(opt, code):
    rc = mqa.lib().mqa_kv_attention_debug(ctypes.byref(cache()), P(0x1000), 4096, 0, 32, P(0x2000), 0 if code == 0 else 8,
                                          0, None, 0, 1, 0.1, P(0x3000), None, P(0x100000), 1 << 40, None,
                                          ctypes.byref(kv.KVDebugOptions(**opt)))
    assert rc == code


class OnDevice:
    """What the binding reads of a CUDA tensor, at a made-up address."""
    is_cuda = True
    device = torch.device("cuda", 0)
    requires_grad = False

    def __init__(self, *shape, dtype=torch.uint8, at=0x10000):
        self.shape, self.dtype, self.at = torch.Size(shape), dtype, at

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return self.at

    def is_contiguous(self):
        return True

    def stride(self, i):
        return self.shape[i + 1:].numel()


def fake_cache(**kw):
    i32 = torch.int32
    a = dict(k=OnDevice(9, 2, 16, 64), v=OnDevice(9, 2, 16, 64), k_exps=OnDevice(9, 2), v_exps=OnDevice(9, 2),
             page_table=OnDevice(3, 4, dtype=i32), seq_lens=OnDevice(3, dtype=i32), refcounts=OnDevice(9, dtype=i32),
             scratch=OnDevice(mqa.kv_scratch_bytes(9, 3)))
    a.update(kw)
    return mqa.KVCache(**a)


def test_rows_that_require_a_gradient_are_refused():
    """The operators have no backward pass: an answer without history would lose the gradient silently."""
    c, starts = fake_cache(), OnDevice(4, dtype=torch.int32)
    x, y = (OnDevice(5, 2, 64, dtype=torch.bfloat16) for _ in range(2))
    y.requires_grad = True
    with pytest.raises(ValueError, match="q requires a gradient"):
        mqa.kv_attention(y, c, starts)
    for k, v, name in ((y, x, "k"), (x, y, "v")):
        with pytest.raises(ValueError, match=name + " requires a gradient"):
            mqa.kv_append(c, k, v, starts)
    with torch.no_grad():
        assert kv._rows(y, c, (torch.bfloat16,), None, "q") == (0x10000, 128)


def test_replace_without_refcounts():
    c = fake_cache()
    bare = c.replace(refcounts=None)
    assert bare.refcounts is None and bare._c.refcounts is None
    again = bare.replace(refcounts=OnDevice(9, dtype=torch.int32, at=0x80000))
    assert again._c.refcounts == 0x80000
    with pytest.raises(ValueError):
        bare.replace(refcounts=OnDevice(8, dtype=torch.int32))
    with pytest.raises((TypeError, ValueError, AttributeError)):
        c.replace(page_table=None)


def test_a_handle_keeps_the_tensors_it_was_made_of():
    """The C entries read the addresses taken when the handle was made: another tensor under a name of the handle would
    not be used, and the one in use could be freed."""
    c = fake_cache()
    for name in ("k", "v", "k_exps", "v_exps", "page_table", "seq_lens", "refcounts", "scratch", "extra", "device",
                 "num_pages", "max_pages"):
        with pytest.raises(AttributeError, match="replace"):
            setattr(c, name, getattr(c, name))
        with pytest.raises(AttributeError, match="replace"):
            delattr(c, name)
    other = c.replace(seq_lens=OnDevice(3, dtype=torch.int32, at=0x90000))
    assert other._c.seq_lens == 0x90000 == other.seq_lens.data_ptr() and c._c.seq_lens == 0x10000
    assert other._c.k == c._c.k and other._c.scratch == c._c.scratch
    with pytest.raises(AttributeError, match="replace"):
        other.seq_lens = c.seq_lens
    c.note = "a program's own attributes are its business"
    assert c.note
