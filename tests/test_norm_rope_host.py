"""Host side of the norm / rotary entry points, without a GPU: the frequencies,
the binding's refusals, and the C entry's argument checks (fake pointers: every
refusal here happens before any CUDA call)."""
import ctypes
import math
import struct

import pytest
import torch

import gated_deltanet_linear_chunked_b200 as gdn
from gated_deltanet_linear_chunked_b200 import _lib

BASE = 0x7F0000000000
ROWS, ROTATION = struct.Struct("Pqq"), struct.Struct("PPqiiiiiiif")  # gdn_rows, gdn_rotation


def fake(i):
    return BASE + i * (256 << 20)


# ------------------------------------------------------------- frequencies
def test_plain_frequencies():
    f, a = gdn.rope_frequencies(8, base=16.0, device="cpu")
    assert f.dtype == torch.float64 and a == 1.0
    torch.testing.assert_close(f, torch.tensor([1.0, 0.5, 0.25, 0.125], dtype=torch.float64))
    f, _ = gdn.rope_frequencies(12, base=16.0, sections=(2, 4, 0), device="cpu")
    torch.testing.assert_close(f, torch.tensor([1, 0.25, 1, 0.5, 0.25, 0.125], dtype=torch.float64))


def test_stretched_frequencies():
    f, _ = gdn.rope_frequencies(64, device="cpu")
    lin, a = gdn.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    torch.testing.assert_close(lin, f / 4.0)
    assert a == 1.0
    ntk, a = gdn.rope_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert a == 1.0
    torch.testing.assert_close(ntk[0], f[0])                       # the fastest pair is kept
    torch.testing.assert_close(ntk[-1], f[-1] / 4.0)               # the slowest is stretched
    yarn, a = gdn.rope_frequencies(64, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    assert a == pytest.approx(0.1 * math.log(4.0) + 1.0)
    turns = 4096 * f / (2 * math.pi)
    torch.testing.assert_close(yarn[turns > 32], f[turns > 32])
    torch.testing.assert_close(yarn[turns < 1], f[turns < 1] / 4.0)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (yarn[mid] < f[mid]).all() and (yarn[mid] > f[mid] / 4.0).all()


@pytest.mark.parametrize("kw", [{"dim": 7}, {"scaling": "other"}, {"factor": 0.5}, {"scaling": "yarn"},
                                {"sections": (3,)}, {"sections": (5, -1)}])
def test_frequency_refusals(kw):
    kw = {"dim": 8, **kw}
    with pytest.raises(ValueError):
        gdn.rope_frequencies(device="cpu", **kw)


# ---------------------------------------------------------------- binding
def test_binding_refuses_cpu_tensors_and_other_types():
    q = torch.zeros(1, 4, 2, 32, dtype=torch.bfloat16)
    f = torch.ones(8, dtype=torch.float64)
    pos = torch.arange(4)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        gdn.rope(q, q, pos, f)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        gdn.qk_norm_rope(q, None)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        gdn.qk_norm_rope_backward(q, None, None, None, q, None)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        gdn.rope_backward(q, None, pos, f)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        gdn.qk_norm_rope(q.half(), None)
    with pytest.raises(ValueError, match=r"\[B,T,H,D\]"):
        gdn.qk_norm_rope(q[0], None)


# ------------------------------------------------------------------ C entry
def rows(i, H=2, D=64, T=8, off=0, bs=None, ts=None):
    ts = H * D if ts is None else ts
    return ROWS.pack(fake(i) + off, T * ts if bs is None else bs, ts)


def rot(pos=fake(20), freq=fake(21), bs=8, pb=8, axes=1, sec=(16, 0, 0), R=32, layout=0, amp=1.0):
    return ROTATION.pack(pos, freq, bs, pb, axes, *sec, R, layout, amp)


def call(q=rows(0), k=rows(1), wq=fake(2), wk=fake(3), r=rot(), qo=rows(4), ko=rows(5), B=2, T=8, Hq=2,
         Hk=2, D=64, eps=1e-6, dtype=_lib.GDN_BF16):
    return _lib.load().gdn_qk_norm_rope(q, k, wq, wk, r, qo, ko, B, T, Hq, Hk, D, eps, dtype, None)


def back(q=rows(0), k=rows(1), wq=fake(2), wk=fake(3), r=rot(), gq=rows(4), gk=rows(5), dq=rows(6),
         dk=rows(7), dwq=fake(8), dwk=fake(9), B=2, T=8, Hq=2, Hk=2, D=64, eps=1e-6,
         dtype=_lib.GDN_BF16):
    return _lib.load().gdn_qk_norm_rope_backward(q, k, wq, wk, r, gq, gk, dq, dk, dwq, dwk, B, T, Hq, Hk,
                                                 D, eps, dtype, None)


REACHES_DEVICE = (_lib.GDN_ERR_CUDA, _lib.GDN_ERR_INVALID_ARG)


def test_struct_sizes():
    assert ROWS.size == 24 and ROTATION.size == 56


def test_sizes_and_types():
    for kw in ({"B": -1}, {"T": -1}, {"Hq": -1}, {"Hk": -2}, {"dtype": 7}, {"eps": -1.0},
               {"eps": float("nan")}):
        assert call(**kw) == _lib.GDN_ERR_INVALID_ARG, kw
        assert back(**kw) == _lib.GDN_ERR_INVALID_ARG, kw
    for d in (0, 8, 24, 144):
        assert call(D=d) == _lib.GDN_ERR_UNSUPPORTED, d
    assert call(B=1 << 16, T=1 << 15) == _lib.GDN_ERR_UNSUPPORTED
    for kw in ({"B": 0}, {"T": 0}, {"Hq": 0, "Hk": 0}):
        assert call(**kw) == _lib.GDN_OK


def test_rotation_checks():
    for kw in ({"R": 80}, {"R": -16}, {"axes": 0}, {"axes": 4}, {"layout": 2}, {"sec": (15, 0, 0)},
               {"sec": (8, 8, 0)}, {"sec": (-1, 0, 0)}, {"pb": 2}, {"bs": -1}, {"pos": 0}, {"freq": 0},
               {"pos": fake(20) + 4}, {"freq": fake(21) + 4}):
        assert call(r=rot(**kw)) == _lib.GDN_ERR_INVALID_ARG, kw
    assert call(r=rot(R=24, sec=(12, 0, 0))) == _lib.GDN_ERR_UNSUPPORTED
    lib = _lib.load()
    assert lib.gdn_rope(rows(0), None, None, 0, rows(4), None, 2, 8, 2, 0, 64, _lib.GDN_BF16,
                        None) == _lib.GDN_ERR_INVALID_ARG


def test_pointers_and_strides():
    for name in ("q", "k", "qo", "ko"):
        assert call(**{name: None}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: ROWS.pack(0, 1024, 128)}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(9, off=8)}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(9, ts=132)}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(9, ts=-128)}) == _lib.GDN_ERR_INVALID_ARG, name
        assert call(**{name: rows(9, bs=1 << 41)}) == _lib.GDN_ERR_INVALID_ARG, name
    for name in ("wq", "wk"):
        assert call(**{name: fake(9) + 4}) == _lib.GDN_ERR_INVALID_ARG, name
    for name in ("gq", "gk", "dq", "dk"):
        assert back(**{name: None}) == _lib.GDN_ERR_INVALID_ARG, name


def test_overlaps():
    assert call(qo=rows(0)) in REACHES_DEVICE                       # in place
    assert call(qo=rows(0, off=256)) == _lib.GDN_ERR_ALIAS          # shifted by a row
    assert call(qo=rows(1)) == _lib.GDN_ERR_ALIAS                   # over k
    assert call(ko=rows(4)) == _lib.GDN_ERR_ALIAS                   # both outputs in one place
    assert call(qo=rows(4, ts=64)) == _lib.GDN_ERR_ALIAS            # rows of the output overlap
    assert call(qo=rows(4, bs=0)) == _lib.GDN_ERR_ALIAS             # one output for two batch rows
    assert call(qo=ROWS.pack(fake(2), 1024, 128)) == _lib.GDN_ERR_ALIAS   # over a weight
    assert call(qo=ROWS.pack(fake(20), 1024, 128)) == _lib.GDN_ERR_ALIAS  # over the positions
    # q, k side by side in one projection, in place
    p = dict(ts=384, bs=8 * 384)
    assert call(q=rows(0, **p), k=rows(0, off=256, **p), qo=rows(0, **p),
                ko=rows(0, off=256, **p)) in REACHES_DEVICE
    assert call(q=rows(0, **p), k=rows(0, off=128, **p), qo=rows(0, **p),
                ko=rows(0, off=128, **p)) == _lib.GDN_ERR_ALIAS
    # sequence first: tokens outside, batch rows inside
    assert call(qo=rows(4, bs=128, ts=256)) in REACHES_DEVICE
    assert back(dq=rows(4)) in REACHES_DEVICE                       # over its own output's gradient
    assert back(dq=rows(5)) == _lib.GDN_ERR_ALIAS
    assert back(dwq=fake(9)) == _lib.GDN_ERR_ALIAS
    assert back(dwk=fake(3)) == _lib.GDN_ERR_ALIAS
    assert back(dwq=fake(6)) == _lib.GDN_ERR_ALIAS
    assert back(dwq=fake(8) + 4) == _lib.GDN_ERR_INVALID_ARG


# Strides whose extent is 1 are not used: odd ones, negative ones, too large ones, and
# different ones of views that lie side by side.
UNUSED = (0, 3, 132, -128, -(1 << 62), 1 << 60)


@pytest.mark.parametrize("stride", UNUSED)
def test_unused_strides_are_not_looked_at(stride):
    def reaches(status):
        # the same call with strides that nothing can object to goes as far
        assert status == call(B=1, T=8), status

    for name in ("q", "k", "qo", "ko"):
        i = {"q": 0, "k": 1, "qo": 4, "ko": 5}[name]
        reaches(call(B=1, **{name: rows(i, bs=stride)}))
        reaches(call(T=1, **{name: rows(i, bs=128, ts=stride)}))
        reaches(call(B=1, T=1, **{name: rows(i, bs=stride, ts=stride)}))
    for name in ("gq", "gk", "dq", "dk"):
        i = {"gq": 4, "gk": 5, "dq": 6, "dk": 7}[name]
        reaches(back(B=1, **{name: rows(i, bs=stride)}))
        reaches(back(T=1, **{name: rows(i, bs=128, ts=stride)}))
    reaches(call(B=1, r=rot(bs=stride)))
    # side by side in one projection, in place, with different unused strides
    p = dict(ts=384)
    q, k = rows(0, bs=stride, **p), rows(0, off=256, bs=7, **p)
    reaches(call(B=1, q=q, k=k, qo=rows(0, bs=8 * 384, **p), ko=rows(0, off=256, bs=0, **p)))
    k = rows(0, off=128, bs=7, **p)
    assert call(B=1, q=q, k=k, qo=q, ko=k) == _lib.GDN_ERR_ALIAS


def test_kernel_names():
    lib = _lib.load()
    assert ctypes.string_at(lib.gdn_kernel_name(11)) == b"gdn_norm_rope_kernel"
    assert ctypes.string_at(lib.gdn_kernel_name(13)) == b"gdn_norm_rope_reduce_kernel"
