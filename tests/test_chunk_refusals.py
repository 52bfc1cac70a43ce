"""Host-side refusals of tv_chunk_append, tv_chunk_attn and tv_beam_select, without a GPU: stand-in device
addresses, and every call must return before anything touches them."""

import ctypes

import pytest
import torch

from tree_speculative_verify_gb300 import _lib, build as tvbuild

OK = 1 << 20


@pytest.fixture(scope="module")
def lib():
    tvbuild.build()
    return _lib.load()


def _shape(**kw):
    base = dict(B=2, D=1, H=4, d=64, W=128, raw_cap=1024, c4_cap=256, c128_cap=8)
    base.update(kw)
    return _lib.make_shape(**base)


def _append(lib, s=None, n=8, starts=OK, K=OK, V=OK, ld=64, Q=OK, rope=64, pairs=0, f=OK, g4=OK, g128=OK,
            Qr=OK, layers=(OK,) * 6, L=OK, st=OK):
    s = s or _shape()
    return lib.tv_chunk_append(ctypes.byref(s), n, starts, K, V, ld, Q, rope, pairs, f, g4, g128, Qr, *layers,
                               L, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -2), (dict(n=(1 << 30) + 1), -2), (dict(n=1 << 29), -2), (dict(starts=None), -1),
    (dict(K=None), -1), (dict(V=None), -1), (dict(ld=63), -2), (dict(ld=68), -2), (dict(ld=1 << 41), -2),
    (dict(Qr=None), -1), (dict(rope=63), -2), (dict(rope=66), -2), (dict(rope=-2), -2), (dict(pairs=2), -1),
    (dict(f=None), -1), (dict(g4=None), -1), (dict(g128=None), -1), (dict(L=None), -1), (dict(st=None), -1),
    (dict(layers=(OK, None, OK, OK, OK, OK)), -1), (dict(layers=(OK, OK, OK, None, OK, OK)), -1),
    (dict(layers=(OK, OK, OK, OK, None, OK)), -1), (dict(layers=(OK + 8, OK, OK, OK, OK, OK)), -1),
    (dict(K=OK + 8), -1), (dict(Q=OK + 2), -1), (dict(Qr=OK + 4), -1),
])
def test_append_refuses(lib, kw, code):
    assert _append(lib, **kw) == code
    assert lib.tv_last_error_string().startswith(b"tv_chunk_append")


def _attn(lib, s=None, n=8, starts=OK, Q=OK, layers=(OK,) * 6, L=OK, scale=0.1, O=OK, lse=OK, ws=OK,
          ws_bytes=None, st=OK):
    s = s or _shape()
    size = lib.tv_chunk_workspace_size(ctypes.byref(s), n) if ws_bytes is None else ws_bytes
    return lib.tv_chunk_attn(ctypes.byref(s), n, starts, Q, *layers, L, scale, O, lse, ws, size, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -2), (dict(n=1 << 29), -2), (dict(starts=None), -1), (dict(Q=None), -1), (dict(L=None), -1),
    (dict(O=None), -1), (dict(lse=None), -1), (dict(st=None), -1), (dict(ws=None), -1), (dict(ws=OK + 16), -1),
    (dict(ws_bytes=0), -7), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=-1.0), -1),
    (dict(Q=OK + 8), -1), (dict(O=OK + 8), -1), (dict(layers=(OK,) * 5 + (None,)), -1),
    (dict(layers=(None,) + (OK,) * 5), -1), (dict(layers=(OK,) * 5 + (OK + 4,)), -1),
    (dict(s=_shape(n_sel=16)), -1),
])
def test_attn_refuses(lib, kw, code):
    assert _attn(lib, **kw) == code
    assert lib.tv_last_error_string().startswith(b"tv_chunk_attn")


def test_outputs_that_overlap_the_queries_are_refused(lib):
    """8 rows of 4 heads (see _shape): the queries end 8 H d es bytes behind their start."""
    s = _shape()
    size = 8 * s.H * s.d * (2 if s.dtype == _lib.TV_BF16 else 4)
    for off in (0, 16, size - 16, 16 - size):
        assert _attn(lib, O=OK + size, Q=OK + size + off) == -1
        assert lib.tv_last_error_string() == b"tv_chunk_attn: O overlaps Q"
    for off in (16, size - 16, 16 - size):     # (Qr may be Q itself)
        assert _append(lib, Q=OK + size, Qr=OK + size + off) == -1
        assert lib.tv_last_error_string() == b"tv_chunk_append: Qr overlaps Q and is not Q"


def _beam(lib, B=6, width=3, vocab=100, ld=100, dtype=0, logits=OK, scores=OK, done=OK, eos=1, scale=1.0,
          source=OK, token=OK, new=OK, new_done=OK, rank=OK, ws=OK, ws_bytes=1 << 20, st=OK):
    s = _lib.make_shape(B=B, D=1, H=1, d=8, comp_mask=1)
    return lib.tv_beam_select(ctypes.byref(s), width, vocab, ld, dtype, logits, scores, done, eos, scale,
                              source, token, new, new_done, rank, ws, ws_bytes, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(width=0), -2), (dict(width=4), -2), (dict(width=33, B=33), -2), (dict(vocab=0), -2), (dict(ld=99), -2),
    (dict(vocab=(1 << 30) + 1, ld=1 << 31), -2), (dict(dtype=2), -1), (dict(scale=0.0), -1),
    (dict(scale=float("inf")), -1), (dict(logits=None), -1), (dict(scores=None), -1), (dict(source=None), -1),
    (dict(token=None), -1), (dict(new=None), -1), (dict(st=None), -1), (dict(ws=None), -1), (dict(ws=OK + 64), -1),
    (dict(ws_bytes=10), -7), (dict(logits=OK + 2), -1), (dict(logits=OK + 1, dtype=1), -1),
])
def test_beam_refuses(lib, kw, code):
    assert _beam(lib, **kw) == code
    assert lib.tv_last_error_string().startswith(b"tv_beam_select")


def test_empty_batches_are_no_ops(lib):
    s = _shape(B=0, raw_cap=0, c4_cap=0, c128_cap=0)
    none = (None,) * 6
    assert _append(lib, s, 0, None, None, None, 64, None, 0, 0, None, None, None, None, none, None, None) == 0
    assert lib.tv_chunk_workspace_size(ctypes.byref(s), 10) == 0
    assert _attn(lib, s, 0, None, None, none, None, 1.0, None, None, None, 0, None) == 0
    assert _attn(lib, _shape(), 0, OK, None, none, None, 1.0, None, None, None, 0, None) == 0
    assert _beam(lib, B=0, width=3, logits=None, scores=None, source=None, token=None, new=None, ws=None,
                 st=None) == 0


def test_bindings_check_their_tensors():
    s = _shape()
    with pytest.raises((ValueError, TypeError)):
        _lib.tv_chunk_append(s, torch.zeros(3, dtype=torch.int32), torch.zeros(4, 64), torch.zeros(4, 64),
                             None, 0, 0, None, *[None] * 10, None)
    with pytest.raises((ValueError, TypeError)):
        _lib.tv_chunk_attn(s, torch.zeros(3, dtype=torch.int32), torch.zeros(4, 4, 64), *[None] * 7, 1.0,
                           None, None, None, None)
    with pytest.raises(ValueError, match="logits"):
        _lib.tv_beam_select(s, 2, torch.zeros(3, 10), *[None] * 2, 0, 1.0, *[None] * 7)


@pytest.mark.parametrize("width", [0, 4, 33])
def test_beams_of_a_width_that_does_not_divide_the_slots_are_refused(lib, width):
    from tree_speculative_verify_gb300 import engine
    with pytest.raises(ValueError, match="width"):
        engine.alloc_beams(_shape(B=6), width, 2, device="cpu")
    assert engine.alloc_beams(_shape(B=6), 3, 2, device="cpu").scores.tolist() == [0.0, -float("inf"),
                                                                                  -float("inf")] * 2
    assert engine.alloc_beams(_shape(B=0, raw_cap=0, c4_cap=0, c128_cap=0), 4, 2, device="cpu").done.numel() == 0
