"""Host side of the cross-attention entry points, without a GPU: the C entries'
argument checks (fake pointers: every refusal here happens before any CUDA call)
and the binding's refusals."""
import ctypes
import struct

import pytest
import torch

import gated_deltanet_linear_chunked_b200 as gdn
from gated_deltanet_linear_chunked_b200 import _lib

BASE = 0x7F0000000000
ROWS = struct.Struct("Pqq")  # gdn_rows


def fake(i):
    return BASE + i * (256 << 20)


def rows(i, T=8, H=4, D=64, off=0, bs=None, ts=None):
    ts = H * D if ts is None else ts
    return ROWS.pack(fake(i) + off, T * ts if bs is None else bs, ts)


KV = dict(T=16, H=2)


def call(q=rows(0), k=rows(1, **KV), v=rows(2, **KV), mask=fake(3), mbs=16, out=fake(4), lse=fake(5), B=2, Tq=8,
         S=16, Hq=4, Hk=2, D=64, scale=0.125, dtype=_lib.GDN_BF16):
    return _lib.load().gdn_cross_attention(q, k, v, mask, mbs, out, lse, B, Tq, S, Hq, Hk, D, scale, dtype, None)


def back(q=rows(0), k=rows(1, **KV), v=rows(2, **KV), mask=fake(3), mbs=16, out=fake(4), lse=fake(5), do=fake(6),
         dq=fake(7), dk=fake(8), dv=fake(9), B=2, Tq=8, S=16, Hq=4, Hk=2, D=64, scale=0.125,
         dtype=_lib.GDN_BF16):
    return _lib.load().gdn_cross_attention_backward(q, k, v, mask, mbs, out, lse, do, dq, dk, dv, B, Tq, S, Hq, Hk,
                                                    D, scale, dtype, None)


REACHES_DEVICE = (_lib.GDN_ERR_CUDA, _lib.GDN_ERR_INVALID_ARG)


@pytest.mark.parametrize("f", [call, back])
def test_sizes_types_and_scale(f):
    for kw in ({"B": -1}, {"Tq": -1}, {"S": -1}, {"Hq": -4}, {"Hk": -2}, {"D": -16}, {"dtype": 7}, {"mbs": -1},
               {"Hq": 3}, {"Hk": 0}, {"scale": 0.0}, {"scale": -1.0}, {"scale": float("nan")},
               {"scale": float("inf")}, {"scale": 1e-40}, {"scale": 3e38}):
        assert f(**kw) == _lib.GDN_ERR_INVALID_ARG, kw
    for kw in ({"dtype": _lib.GDN_F32}, {"D": 8}, {"D": 72}, {"D": 144}, {"Hq": 258, "Hk": 2},
               {"Tq": (1 << 30) + 1}, {"B": 1 << 12, "Tq": 1 << 20}):
        assert f(**kw) == _lib.GDN_ERR_UNSUPPORTED, kw
    assert f(B=0) == _lib.GDN_OK
    assert f() in REACHES_DEVICE


def test_nothing_to_do():
    assert call(Tq=0, q=None, out=None) == _lib.GDN_OK
    assert call(Hq=0) == _lib.GDN_OK
    assert back(Hq=0, Hk=0) == _lib.GDN_OK
    assert back(Tq=0, S=0) == _lib.GDN_OK
    # gradients of what nothing attends to are still written
    assert back(Tq=0, q=None, out=None, lse=None, do=None, dq=None) in REACHES_DEVICE
    assert back(Tq=0, dk=None) == _lib.GDN_ERR_INVALID_ARG


def test_pointers_and_strides():
    for name, t in (("q", 8), ("k", 16), ("v", 16)):
        assert call(**{name: None}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(10, T=t, off=8)}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(10, T=t, ts=260)}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(10, T=t, ts=0)}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(10, T=t, ts=-256)}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(10, T=t, bs=1 << 37)}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(10, T=t, bs=0)}) in REACHES_DEVICE, name      # shared by the batch
    for name in ("out", "lse"):
        assert call(**{name: fake(10) + 8}) == _lib.GDN_ERR_INVALID_ARG, name
    assert call(out=None) == _lib.GDN_ERR_INVALID_ARG
    assert call(lse=None) in REACHES_DEVICE
    for name in ("out", "lse", "do", "dq", "dk", "dv"):
        assert back(**{name: None}) == _lib.GDN_ERR_INVALID_ARG, name
        assert back(**{name: fake(10) + 8}) == _lib.GDN_ERR_INVALID_ARG, name
    assert call(k=None, v=None, S=0) in REACHES_DEVICE


@pytest.mark.parametrize("stride", (3, 132, -128, -(1 << 62), 1 << 60))
@pytest.mark.parametrize("f", [call, back])
def test_unused_strides_are_not_looked_at(f, stride):
    """Strides whose extent is 1 are not used: such a call goes as far as one with plain ones."""
    one = dict(B=1)
    for name, t, n in (("q", 8, 0), ("k", 16, 1), ("v", 16, 2)):
        h = 4 if name == "q" else 2
        assert f(B=1, **{name: rows(n, T=t, H=h, bs=stride)}) == f(**one), name
    assert f(Tq=1, q=rows(0, bs=256, ts=stride)) == f(**one)
    assert f(S=1, k=rows(1, bs=128, ts=stride), v=rows(2, bs=128, ts=stride)) == f(**one)
    assert f(B=1, mbs=stride) == f(**one)


def test_overlaps():
    for i in (0, 1, 2, 3):
        assert call(out=fake(i) + 16) == _lib.GDN_ERR_ALIAS, i
        assert call(lse=fake(i)) == _lib.GDN_ERR_ALIAS, i
    assert call(lse=fake(4)) == _lib.GDN_ERR_ALIAS
    for name in ("dq", "dk", "dv"):
        for i in range(7):
            assert back(**{name: fake(i)}) == _lib.GDN_ERR_ALIAS, (name, i)
    assert back(dq=fake(8)) == _lib.GDN_ERR_ALIAS
    assert back(dv=fake(8)) == _lib.GDN_ERR_ALIAS
    assert call(v=rows(1, **KV)) in REACHES_DEVICE      # keys that are the values


def test_binding_refusals():
    q = torch.zeros(1, 4, 2, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        gdn.cross_attention(q, q, q)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        gdn.cross_attention_backward(q, q, q, q, q, q)
    with pytest.raises(TypeError, match="must be bfloat16"):
        gdn.cross_attention(q.float(), q, q)
    with pytest.raises(ValueError, match=r"\[B,Tq,Hq,D\]"):
        gdn.cross_attention(q[0], q, q)


def test_missing_binding_raises_instead_of_falling_back(monkeypatch, tmp_path):
    from gated_deltanet_linear_chunked_b200 import build as _build
    monkeypatch.setattr(_lib, "_bind", None)
    monkeypatch.setattr(_build, "BIND_PATH", str(tmp_path / "_gdn_torch.so"))

    def no_compiler(*a, **k):
        raise OSError("g++ not found")
    monkeypatch.setattr(_build, "build_bind", no_compiler)
    with pytest.raises(RuntimeError, match="_gdn_torch.so is missing"):
        _lib.bind()


def test_kernel_names():
    lib = _lib.load()
    names = [ctypes.string_at(lib.gdn_kernel_name(i)).decode() for i in range(14, 20)]
    assert names == ["gdn_cross_kernel", "gdn_cross_join_kernel", "gdn_cross_bwd_kernel",
                     "gdn_cross_grad_join_kernel", "gdn_cross_stat_kernel", "gdn_cross_few_kernel"]
    assert lib.gdn_kernel_name(20) == b"unknown"
