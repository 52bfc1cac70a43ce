"""Host-side refusals of tv_token_logprobs and the tv_pages_* calls, without a GPU: stand-in device
addresses, and every call must return before anything touches them."""

import ctypes

import pytest
import torch

from tree_speculative_verify_gb300 import _lib, build as tvbuild


@pytest.fixture(scope="module")
def lib():
    tvbuild.build()
    return _lib.load()


OK = 1 << 20


def _pages_shape(**kw):
    base = dict(B=2, D=8, H=64, d=512, raw_cap=1024, c4_cap=256, c128_cap=8, page_tokens=512,
                max_pages=2, n_pool_pages=8)
    base.update(kw)
    s = _lib.make_shape(**base)
    s.page_table = OK
    return s


def _logprobs(lib, s=None, vocab=100, ld=100, dtype=_lib.TV_BF16, logits=OK, n_tok=8, tokens=OK,
              nodes=OK, scale=1.0, n_top=4, lse=OK, ent=OK, lps=OK, ids=OK, top=OK, target=OK, st=OK):
    s = s or _lib.make_shape(B=2, D=8, H=1, d=8, comp_mask=1)
    return lib.tv_token_logprobs(ctypes.byref(s), vocab, ld, dtype, logits, n_tok, tokens, nodes,
                                 scale, n_top, lse, ent, lps, ids, top, target, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(vocab=0), -2), (dict(vocab=-5), -2), (dict(vocab=(1 << 30) + 1, ld=1 << 31), -2), (dict(ld=99), -2),
    (dict(ld=(1 << 40) + 1), -2), (dict(dtype=2), -1), (dict(n_tok=-1), -2), (dict(n_tok=1025), -2),
    (dict(n_top=-1), -2), (dict(n_top=33), -2), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("inf")), -1), (dict(scale=float("nan")), -1), (dict(logits=None), -1),
    (dict(st=None), -1), (dict(tokens=None), -1), (dict(lps=None), -1), (dict(nodes=None, n_tok=9), -1),
    (dict(ids=None), -1), (dict(top=None), -1), (dict(logits=OK + 1), -1),
    (dict(logits=OK + 2, dtype=_lib.TV_F32), -1),
])
def test_logprobs_refuses(lib, kw, code):
    assert _logprobs(lib, **kw) == code
    assert lib.tv_last_error_string().startswith(b"tv_token_logprobs")


def test_empty_batches_are_no_ops(lib):
    s = _lib.make_shape(B=0, D=8, H=1, d=8, comp_mask=1)
    assert _logprobs(lib, s, logits=None, st=None) == 0
    s = _pages_shape(B=0)
    assert lib.tv_pages_workspace_size(ctypes.byref(s)) == 0
    assert lib.tv_pages_reserve(ctypes.byref(s), *([None] * 4), 0, None, None) == 0
    assert lib.tv_pages_fork(ctypes.byref(s), *([None] * 11), 0, None, 0, None, None) == 0
    assert lib.tv_pages_compact(ctypes.byref(s), *([None] * 11), 0, None, None) == 0


def _fork(lib, s, source=OK, keep=None, L=OK, refs=OK, pools=(OK,) * 6, keys=None, d_idx=0, ws=OK,
          ws_bytes=None, st=OK):
    n = lib.tv_pages_workspace_size(ctypes.byref(s)) if ws_bytes is None else ws_bytes
    return lib.tv_pages_fork(ctypes.byref(s), source, keep, L, refs, *pools, keys, d_idx, ws, n, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(source=None), -1), (dict(L=None), -1), (dict(refs=None), -1), (dict(st=None), -1),
    (dict(ws=None), -1), (dict(ws=OK + 128), -1), (dict(ws_bytes=100), -7),
    (dict(pools=(OK, None, OK, OK, OK, OK)), -1), (dict(pools=(OK, OK, OK, OK, OK, None)), -1),
    (dict(pools=(OK, OK, OK + 8, OK, OK, OK)), -1), (dict(keys=OK, d_idx=12), -2),
    (dict(keys=OK, d_idx=0), -2), (dict(keys=OK, d_idx=264), -2), (dict(keys=OK + 8, d_idx=64), -1),
])
def test_fork_refuses(lib, kw, code):
    assert _fork(lib, _pages_shape(), **kw) == code
    assert lib.tv_last_error_string().startswith(b"tv_pages_fork")


def test_pages_calls_need_pools_and_workspace(lib):
    plain = _lib.make_shape(B=2, D=8, H=64, d=512, raw_cap=1024, c4_cap=256, c128_cap=8)
    assert lib.tv_pages_workspace_size(ctypes.byref(plain)) == 0
    assert _fork(lib, plain, ws_bytes=1 << 20) == -2
    c128 = _pages_shape(comp_mask=_lib.TV_COMP_C128)
    assert _fork(lib, c128, pools=(OK, OK, None, None, OK, OK), keys=OK, d_idx=64) == -1   # no C4
    s = _pages_shape()
    n = lib.tv_pages_workspace_size(ctypes.byref(s))
    assert n > 0 and n % 256 == 0
    assert lib.tv_pages_reserve(ctypes.byref(s), OK, OK, OK, OK, n - 1, OK, None) == -7
    assert lib.tv_pages_reserve(ctypes.byref(s), None, OK, OK, OK, n, OK, None) == -1
    args = lambda remap=OK, live=OK, pools=(OK,) * 6: (OK, OK, *pools, remap, live, OK, n, OK, None)
    assert lib.tv_pages_compact(ctypes.byref(s), *args(remap=None)) == -1
    assert lib.tv_pages_compact(ctypes.byref(s), *args(live=None)) == -1
    assert lib.tv_pages_compact(ctypes.byref(s), *args(pools=(OK, OK, OK, OK, OK + 4, OK))) == -1
    big = _pages_shape(n_pool_pages=4000)
    assert lib.tv_pages_workspace_size(ctypes.byref(big)) > n


def test_binding_refuses_host_tensors(lib):
    s = _lib.make_shape(B=1, D=2, H=1, d=8, comp_mask=1)
    st = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        _lib.tv_token_logprobs(s, torch.zeros(1, 2, 10), None, None, 1.0, None, None, None, None, None,
                               None, st)
    with pytest.raises(ValueError):
        _lib.tv_pages_reserve(_pages_shape(), st, st, st, None, st)
    with pytest.raises(TypeError):
        _lib.tv_pages_reserve(_pages_shape(), st, [1, 2], st, None, st)


class _OnDevice:
    """Stands in for a tensor of another device, which a machine with one device cannot make."""
    is_cuda, dtype = True, torch.int32

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def numel(self):
        return 1 << 20

    def data_ptr(self):
        raise AssertionError("the address of a tensor on another device was taken")


def test_binding_refuses_another_device(monkeypatch):
    monkeypatch.setattr(_lib, "_here", lambda: 0)
    monkeypatch.setattr(_lib.torch, "Tensor", _OnDevice)
    t = _OnDevice()
    with pytest.raises(ValueError, match="another device"):
        _lib.tv_pages_reserve(_pages_shape(), t, t, t, t, t)


def test_managed_pool_maps_what_the_prefixes_cover(lib):
    from tree_speculative_verify_gb300 import engine, workloads
    wl = workloads.make_workload("pool", B=3, D=4, H=2, d=64, W=128, tail_mode="window", ms=(4, 128),
                                 dtype="f32", L=(100, 1300), k=2, steps=3, p_match=0.5, seed=3, kv_scale=0.5)
    wl.L[:] = (0, 512, 1025)
    shape, st = engine.alloc_pool(wl, 512, 6, device="cpu")
    G = shape.max_pages
    assert st.page_table.tolist() == [[-1] * G, [0] + [-1] * (G - 1), [1, 2, 3] + [-1] * (G - 3)]
    assert st.page_refs.tolist() == [1, 1, 1, 1, 0, 0]
    assert st.page_ws.numel() == lib.tv_pages_workspace_size(ctypes.byref(shape)) > 0
    assert torch.equal(st.rawK[3, :1], wl.rawK[2, 1024:1025]) and not st.rawK[3, 1:].any()
    with pytest.raises(ValueError):
        engine.alloc_pool(wl, 512, 3, device="cpu")


def test_copy_of_a_managed_pool_shares_nothing(lib):
    from dataclasses import fields
    from tree_speculative_verify_gb300 import engine, workloads
    wl = workloads.make_workload("pool", B=2, D=4, H=2, d=64, W=128, tail_mode="window", ms=(4, 128),
                                 dtype="f32", L=(100, 1300), k=2, steps=3, p_match=0.5, seed=3, kv_scale=0.5)
    wl.k_idx = torch.randn((2, wl.cap4, 64)).bfloat16()
    shape, st = engine.alloc_pool(wl, 512, 12, device="cpu")
    with pytest.raises(ValueError, match="clone_pool"):
        st.clone()
    cshape, copy = engine.clone_pool(shape, st)
    for f in fields(st):
        a, b = getattr(st, f.name), getattr(copy, f.name)
        assert a.untyped_storage().data_ptr() != b.untyped_storage().data_ptr(), f.name
        if f.name != "page_ws":
            assert torch.equal(a, b), f.name
    assert shape.page_table == st.page_table.data_ptr()
    assert cshape.page_table == copy.page_table.data_ptr()
    assert all(getattr(shape, n) == getattr(cshape, n) for n, _ in shape._fields_ if n != "page_table")
    # a state without counts keeps sharing what a round only reads
    pshape, paged = engine.alloc_paged(wl, 512, device="cpu")
    assert paged.clone().page_table is paged.page_table
