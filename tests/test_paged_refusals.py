"""What the paged cache's calls refuse, before anything is enqueued (CPU only:
no kernel is launched; see test_abi.py for the fake addresses)."""
import ctypes as C

import pytest
import torch

A = 1 << 20  # aligned, never dereferenced
BIG = 1 << 40

cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation tests run only without a GPU")


@pytest.fixture(scope="module")
def lib():
    from long_context_gsa_b200 import build, load
    build.build_library()
    return load()


def _desc(**kw):
    from long_context_gsa_b200 import gsa_desc
    base = dict(batch=2, hq=8, hkv=2, d=128, chunk=16, n_max=64, t_max=64 * 16 + 16, topk=8, exclude_unselected=0,
                scale=0.0, dtype=1, out_dtype=0)
    base.update(kw)
    return gsa_desc(*[base[f] for f, _ in gsa_desc._fields_])


def _pdesc(**kw):
    from long_context_gsa_b200 import gsa_pdesc
    base = dict(cache_dtype=2, page=64, n_pages=100, max_pages=17)
    base.update(kw)
    return gsa_pdesc(*[base[f] for f, _ in gsa_pdesc._fields_])


def _adesc(**kw):
    from long_context_gsa_b200 import gsa_append_desc
    base = dict(n_tok=4, rot_dim=128, interleaved=0, advance=0, q_stride=0, k_stride=0, v_stride=0)
    base.update(kw)
    return gsa_append_desc(*[base[f] for f, _ in gsa_append_desc._fields_])


def _append(lib, d, p, a, nbytes=BIG, **ptr):
    names = ["q", "k", "v", "cu", "pos", "freq", "table", "n", "own", "kp", "vp", "ks", "vs", "qo", "ws"]
    v = {x: A for x in names}
    v["qo"] = A + 4096
    v.update(ptr)
    return lib.gsa_paged_append(C.byref(d), C.byref(p), C.byref(a), *[v[x] for x in names], nbytes, None)


def _calls(lib, d, p, ws=BIG, drop=None):
    """The status of each reading call, with pointer argument `drop` left out."""
    def ptrs(n):
        return [A if i != drop else None for i in range(n)]
    return dict(
        attend=lambda n_q=1: lib.gsa_paged_attend(C.byref(d), C.byref(p), n_q, *ptrs(10), A, ws, None),
        unfold=lambda prior=1: lib.gsa_paged_unfold(C.byref(d), C.byref(p), *ptrs(11), prior, A, None, A, ws, None),
        decode=lambda: lib.gsa_paged_decode(C.byref(d), C.byref(p), *ptrs(14), A, ws, None),
        gist_step=lambda: lib.gsa_paged_gist_step(C.byref(d), C.byref(p), *ptrs(14), A, ws, None))


def test_workspace(lib):
    from long_context_gsa_b200 import GSA_OP_DECODE, GSA_OP_GIST_STEP, GSA_OP_PAGED, gsa_workspace_bytes
    d = _desc()
    n = gsa_workspace_bytes(d, GSA_OP_PAGED)
    assert n > gsa_workspace_bytes(d, GSA_OP_DECODE) and n > gsa_workspace_bytes(d, GSA_OP_GIST_STEP) and n % 256 == 0
    assert gsa_workspace_bytes(_desc(d=96), GSA_OP_PAGED) == 0
    assert gsa_workspace_bytes(d, 7) == 0


@cpu_only
@pytest.mark.parametrize("bad,code", [
    (dict(page=40), 1), (dict(page=0), 1), (dict(n_pages=0), 1), (dict(max_pages=16), 1), (dict(cache_dtype=4), 1),
    (dict(cache_dtype=-1), 1), (dict(n_pages=1 << 30), 2),
])
def test_bad_page_descriptor(lib, bad, code):
    d, p = _desc(), _pdesc(**bad)
    assert _append(lib, d, p, _adesc()) == code
    for name, call in _calls(lib, d, p).items():
        assert call() == code, name


@cpu_only
def test_readers_take_8_bit_codes_only(lib):
    for dt in (0, 1):
        for name, call in _calls(lib, _desc(), _pdesc(cache_dtype=dt)).items():
            assert call() == 2, name
    assert _append(lib, _desc(), _pdesc(cache_dtype=0), _adesc()) == 2  # fp32 pages for bf16 tokens


@cpu_only
@pytest.mark.parametrize("bad,code", [
    (dict(n_tok=-1), 1), (dict(rot_dim=-16), 1), (dict(rot_dim=144), 1), (dict(rot_dim=24), 2),
    (dict(interleaved=2), 1), (dict(advance=-1), 1), (dict(q_stride=8 * 128 - 8), 1),
    (dict(k_stride=2 * 128 + 4), 1), (dict(v_stride=8), 1),
])
def test_bad_append_descriptor(lib, bad, code):
    assert _append(lib, _desc(), _pdesc(), _adesc(**bad)) == code


@cpu_only
def test_append_pointers(lib):
    d, p, a = _desc(), _pdesc(), _adesc()
    for name in ("k", "v", "freq", "table", "own", "kp", "vp", "ks", "vs", "qo", "ws"):
        assert _append(lib, d, p, a, **{name: None}) == 1, name
    for name in ("q", "k", "cu", "pos", "n", "ks"):
        assert _append(lib, d, p, a, **{name: A + 4}) == 1, name
    assert _append(lib, d, p, a, qo=A) == 1              # turned in place
    assert _append(lib, d, p, _adesc(n_tok=3), cu=None) == 1  # 3 tokens over 2 sequences
    assert _append(lib, d, p, a, nbytes=4096) == 3
    assert _append(lib, _desc(batch=9000), _pdesc(), a) == 2
    assert _append(lib, _desc(hq=1 << 16, hkv=1 << 13), _pdesc(), a) == 2
    assert _append(lib, d, p, _adesc(n_tok=0), k=None, v=None, q=None, qo=None) == 0  # nothing to do
    assert lib.gsa_paged_append(C.byref(d), None, C.byref(a), *[A] * 15, BIG, None) == 1
    assert lib.gsa_paged_append(C.byref(d), C.byref(p), None, *[A] * 15, BIG, None) == 1


@cpu_only
def test_reader_pointers_and_counts(lib):
    d, p = _desc(), _pdesc()
    for i in (0, 1, 2, 3, 4, 5, 7, 8):      # q, the cache, own_len, out
        assert _calls(lib, d, p, drop=i)["attend"]() == 1, i
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 9):   # q, the cache, n_gists, own_len, sel_idx
        assert _calls(lib, d, p, drop=i)["unfold"]() == 1, i
    ex = _desc(exclude_unselected=1)
    for i in (6, 10):                       # gist_v, sel_score of exclude mode
        assert _calls(lib, ex, p, drop=i)["unfold"](0) == 1, i
    for i in range(11):
        assert _calls(lib, d, p, drop=i)["decode"]() == 1, i
    for i in range(13):
        assert _calls(lib, d, p, drop=i)["gist_step"]() == 1, i
    assert _calls(lib, d, p)["unfold"](0) == 1 and _calls(lib, d, p)["unfold"](9) == 1
    assert _calls(lib, d, p)["attend"](0) == 1 and _calls(lib, d, p)["attend"](65) == 2
    for name, call in _calls(lib, d, p, ws=4096).items():
        assert call() == 3, name
    # steps are counted in 32 bits
    huge = _desc(batch=8192, t_max=1 << 28, n_max=1, chunk=64)
    assert _calls(lib, huge, _pdesc(page=1 << 20, max_pages=256))["attend"]() == 2


def test_binding_checks(lib):
    from long_context_gsa_b200 import _abi
    d, p = _desc(), _pdesc()
    short = torch.zeros(7, dtype=torch.bfloat16)
    t = torch.zeros(4)
    codes, scale = torch.zeros(100 * 64 * 2 * 128, dtype=torch.int8), torch.zeros(100 * 4 * 2)
    with pytest.raises(ValueError, match="q holds 7"):
        _abi.gsa_paged_attend(d, p, 1, short, codes, codes, scale, scale, t, None, t, t, t, t)
    with pytest.raises(ValueError, match="k_pages holds 4"):
        _abi._cache(d, p, t, codes, scale, scale, t, 0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        _abi._cache(d, p, codes, codes, scale, scale, t, 0)
    with pytest.raises(ValueError, match="must be"):
        _abi._rows(torch.zeros((3, 2, 128)), torch.float32, "k_new", 4, 2, 128, 0, 0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        _abi._rows(torch.zeros((4, 2, 128)), torch.float32, "k_new", 4, 2, 128, 0, 0)

    class Fake(torch.Tensor):  # a CUDA tensor's attributes
        is_cuda, where, strides = True, 0, None

        def get_device(self):
            return self.where

        def stride(self):
            return self.strides or super().stride()

        def data_ptr(self):
            return A

    def fake(shape=(4, 2, 128), strides=None, where=0, dtype=torch.float32):
        f = torch.zeros(shape, dtype=dtype).as_subclass(Fake)
        f.strides, f.where = strides, where
        return f

    def rows(strides=None, stride=0, dev=0, dtype=torch.float32):
        return _abi._rows(fake(strides=strides, dtype=dtype), torch.float32, "k", 4, 2, 128, stride, dev)

    assert rows() == A and rows((1024, 128, 1), 1024) == A
    for strides in ((1024, 128, 1), (256, 256, 1), (256, 128, 2)):
        with pytest.raises(ValueError, match="strides"):
            rows(strides)
    with pytest.raises(TypeError):
        rows(dtype=torch.bfloat16)
    # tensors on another device than the current one
    assert _abi._arg(fake(), torch.float32, "x", 1024, 0) == A
    for call in (lambda: rows(dev=1), lambda: _abi._arg(fake(), torch.float32, "x", 1024, 1),
                 lambda: _abi._tail(fake(), None, 1)):
        with pytest.raises(ValueError, match="current device"):
            call()
    with pytest.raises(ValueError, match="holds 1024"):
        _abi._arg(fake(), torch.float32, "x", 1025, 0)
    with pytest.raises(TypeError):
        _abi._arg(fake(), torch.int32, "x", 1, 0)
    assert _abi._arg(None, torch.int32, "x", 1, 0, True) is None
    with pytest.raises(ValueError, match="required"):
        _abi._arg(None, torch.int32, "x", 1, 0)
