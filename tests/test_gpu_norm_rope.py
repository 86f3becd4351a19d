"""GPU parity of the query/key norm and rotary positions, and their gradients,
against the fp64 formulas.

Tolerances, element by element.  Every value is computed in fp32 from the stored
inputs and rounded once to the output's type, so it may be off by half a step of
that type, eps(type) / 2 of its size, plus the fp32 work: u = 2^-24 times
* forward: the pair's size A (|y_a| + |y_b|), for the row's sum of squares (at
  most 16 products in a lane and 4 sums across lanes: 20 u, halved by the root),
  its root (2 u), the two products with weight and r (2 u), the angle (reduced in
  fp64 to a fraction of a turn below 1/2, rounded to fp32: u / 2 turns = 3.2 u
  radians), sincospi (2 u), the amplitude (u) and the turn itself (3 u): 24 u, taken as 32;
* backward: r (|g w| of the pair + |x^| mean |g w x^|), the dot product adding the
  same 20 u and the turn of dy the same 10: 64 u;
* dweight: the sum over rows of |g x^|, each lane adding at most 64 rows in turn,
  5 + 8 sums across the block, 14 + 5 across blocks, and 30 u of each term: 128 u.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_chunked_b200 as gdn
from oracle import norm_rope as nr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def np64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Inputs of one call from a seed: numpy copies of what the tensors hold."""

    def __init__(self, B, T, Hq, Hk, D, R, dtype, layout, sections, seed, far=1000, packed=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = DT[dtype]
        n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        if packed:
            qkv = n(B, T, Hq + 2 * Hk, D).to(dt)
            self.q, self.k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        else:
            self.q, self.k = n(B, T, Hq, D).to(dt), n(B, T, Hk, D).to(dt)
        self.wq, self.wk = 1 + 0.3 * n(D), 1 + 0.3 * n(D)
        self.gq, self.gk = n(B, T, Hq, D).to(dt), n(B, T, Hk, D).to(dt)
        self.layout, self.sections, self.R = layout, sections, R
        self.pos = torch.randint(-far, far + 1, (B, T, len(sections)), generator=g, device="cuda")
        self.freq, _ = gdn.rope_frequencies(R, sections=sections)
        self.amp = 1.25
        self.angle = nr.angles(self.pos.cpu().numpy(), self.freq.cpu().numpy(), sections)
        self.turn = dict(sections=sections, layout=layout, amplitude=self.amp)

    def size(self, y):
        """Of every value, its pair's |y_a| + |y_b| times the amplitude; beyond R itself."""
        y = np.abs(y)
        a, b = nr.pair_indices(self.R, self.layout)
        m = y.copy()
        m[..., a] = m[..., b] = self.amp * (y[..., a] + y[..., b])
        return m

    def check_forward(self, out, x, w, eps=1e-6, norm=True):
        y = nr.norm(np64(x), None if w is None else np64(w), eps) if norm else np64(x)
        ref = nr.turn(y, self.angle, self.layout, self.amp)
        tol = HALF[out.dtype] * np.abs(ref) * (1 + 2 * HALF[out.dtype]) + 32 * U * self.size(y)
        err = np.abs(np64(out) - ref)
        assert out.shape == x.shape and (err <= tol).all(), float((err / (tol + 1e-300)).max())

    def check_backward(self, dx, dw, x, w, dy, eps=1e-6):
        X, W, DY = np64(x), np64(w), np64(dy)
        ref, refw = nr.norm_turn_backward(X, W, eps, DY, self.angle, self.layout, self.amp)
        r = 1 / np.sqrt(np.mean(X * X, -1, keepdims=True) + eps)
        hat = X * r
        g = nr.turn(DY, self.angle, self.layout, self.amp, inverse=True)
        gs = self.size(DY)
        gw = np.abs(g * W * hat).mean(-1, keepdims=True) + (gs * np.abs(W * hat)).mean(-1, keepdims=True)
        tol = HALF[dx.dtype] * np.abs(ref) * (1 + 2 * HALF[dx.dtype]) + \
            64 * U * r * (gs * np.abs(W) + np.abs(hat) * gw)
        err = np.abs(np64(dx) - ref)
        assert (err <= tol).all(), float((err / (tol + 1e-300)).max())
        assert dw.dtype == torch.float32
        tolw = 128 * U * np.sum(gs * np.abs(hat), (0, 1, 2)) + 1e-30
        assert (np.abs(np64(dw) - refw) <= tolw).all(), float((np.abs(np64(dw) - refw) / tolw).max())


CASES = [
    # B, T, Hq, Hk, D, R, dtype, layout, sections, packed
    (1, 1, 1, 1, 16, 16, "bf16", "half", (8,), False),
    (1, 1, 20, 20, 112, 112, "bf16", "half", (20, 18, 18), True),
    (2, 3, 5, 1, 32, 16, "bf16", "interleaved", (8,), False),
    (3, 7, 4, 2, 48, 48, "bf16", "half", (12, 12), False),
    (1, 33, 3, 3, 64, 32, "bf16", "half", (16,), True),
    (2, 129, 6, 2, 80, 80, "bf16", "interleaved", (20, 0, 20), True),
    (1, 65, 12, 4, 96, 64, "bf16", "half", (32,), False),
    (1, 700, 20, 20, 112, 112, "bf16", "half", (20, 18, 18), True),
    (4, 301, 16, 4, 128, 64, "bf16", "interleaved", (32,), False),
    (1, 1, 2, 1, 16, 16, "f32", "interleaved", (8,), False),
    (2, 19, 5, 5, 48, 32, "f32", "half", (16,), True),
    (1, 77, 3, 1, 80, 16, "f32", "interleaved", (3, 5), False),
    (2, 130, 20, 5, 112, 112, "f32", "half", (56,), True),
    (1, 257, 33, 8, 128, 128, "f32", "half", (64,), False),
]


@pytest.mark.parametrize("B,T,Hq,Hk,D,R,dtype,layout,sections,packed", CASES)
def test_forward_and_gradients(B, T, Hq, Hk, D, R, dtype, layout, sections, packed):
    c = Case(B, T, Hq, Hk, D, R, dtype, layout, sections, 10 * T + D, packed=packed)
    q0, k0 = c.q.clone(), c.k.clone()
    qo, ko = gdn.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.pos, c.freq, **c.turn)
    c.check_forward(qo, c.q, c.wq)
    c.check_forward(ko, c.k, c.wk)
    qo, ko = gdn.rope(c.q, c.k, c.pos, c.freq, **c.turn)
    c.check_forward(qo, c.q, None, norm=False)
    c.check_forward(ko, c.k, None, norm=False)
    g = gdn.qk_norm_rope_backward(c.q, c.k, c.wq, c.wk, c.gq, c.gk, c.pos, c.freq, **c.turn)
    c.check_backward(g["dq"], g["dq_weight"], c.q, c.wq, c.gq)
    c.check_backward(g["dk"], g["dk_weight"], c.k, c.wk, c.gk)
    again = gdn.qk_norm_rope_backward(c.q, c.k, c.wq, c.wk, c.gq, c.gk, c.pos, c.freq, **c.turn)
    assert all(torch.equal(g[n], again[n]) for n in g)          # the same bits
    assert torch.equal(c.q, q0) and torch.equal(c.k, k0)        # inputs untouched


def backward(c, **kw):
    return gdn.qk_norm_rope_backward(c.q, c.k, c.wq, c.wk, c.gq, c.gk, c.pos, c.freq, **c.turn, **kw)


@pytest.mark.parametrize("B,T,Hq,Hk,D,R,dtype,packed", [
    (1, 33, 5, 2, 64, 32, "f32", False),
    (1, 1, 1, 1, 16, 16, "bf16", False),
    (2, 301, 16, 4, 128, 64, "bf16", False),   # heads that the groups do not share evenly
    (1, 700, 20, 20, 112, 112, "bf16", True),  # a last tile with places for tokens that are none
    (3, 130, 7, 3, 48, 48, "f32", True),
])
def test_weight_gradients_without_eps(B, T, Hq, Hk, D, R, dtype, packed):
    """eps = 0: finite wherever no row is all zeros; places of a block that have no row
    (past the last token or head) add nothing."""
    c = Case(B, T, Hq, Hk, D, R, dtype, "half", (R // 2,), 3 * T + D, packed=packed)
    g = backward(c, eps=0.0)
    c.check_backward(g["dq"], g["dq_weight"], c.q, c.wq, c.gq, eps=0.0)
    c.check_backward(g["dk"], g["dk_weight"], c.k, c.wk, c.gk, eps=0.0)


@pytest.mark.parametrize("T,Hq,Hk,D", [(700, 20, 20, 112), (1000, 16, 4, 64), (300, 2, 2, 64), (5, 3, 1, 16)])
def test_weight_gradients_do_not_hold_what_another_call_left(T, Hq, Hk, D):
    """A rotation by NaN angles before it, which leaves them in the shared memory of
    every SM, changes no bit: the places of the last tile that have no token read none."""
    c = Case(1, T, Hq, Hk, D, D, "bf16", "half", (D // 2,), 5 * T + D)
    want = backward(c)
    c.check_backward(want["dq"], want["dq_weight"], c.q, c.wq, c.gq)
    x = torch.ones(1, 1 << 18, 1, 16, dtype=torch.bfloat16, device="cuda")
    at = torch.zeros(1 << 18, dtype=torch.int64, device="cuda")
    freq = torch.full((8,), float("nan"), dtype=torch.float64, device="cuda")
    for _ in range(5):
        assert gdn.rope(x, None, at, freq)[0].isnan().all()
        got = backward(c)
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_rope_backward_is_the_transposed_turn():
    """<rope(x), y> = <x, rope_backward(y)>: both are sums of fp32-exact turns rounded once."""
    c = Case(2, 37, 3, 2, 64, 32, "f32", "half", (16,), 6)
    qo, ko = gdn.rope(c.q, c.k, c.pos, c.freq, **c.turn)
    g = gdn.rope_backward(c.gq, c.gk, c.pos, c.freq, **c.turn)
    for x, y, o, d in ((c.q, c.gq, qo, g["dq"]), (c.k, c.gk, ko, g["dk"])):
        ref = nr.turn(np64(y), c.angle, c.layout, c.amp, inverse=True)
        assert (np.abs(np64(d) - ref) <= U * np.abs(ref) * 1.01 + 32 * U * c.size(np64(y))).all()
        size = np.sum(c.size(np64(x)) * np.abs(np64(y)))
        assert abs(np.sum(np64(o) * np64(y)) - np.sum(np64(x) * np64(d))) <= 80 * U * size


def test_gradients_match_differences():
    """The gradient of <out, dy> against central differences of the kernel's own
    forward in fp32.  A step h moves the loss by 2 h dL; rounding of the outputs is
    at most u (1 + 32) of their size each way, so |difference - gradient| is at most
    33 u sum |out dy| / h plus the third-order term, h^2 / 6 times the third
    derivative of a row of mean square 1: below 20 |dy| per row for |x| < 4 / r."""
    c = Case(1, 2, 2, 1, 16, 16, "f32", "interleaved", (8,), 8)
    g = gdn.qk_norm_rope_backward(c.q, c.k, c.wq, c.wk, c.gq, c.gk, c.pos, c.freq, **c.turn)

    def loss(q, w):
        out, _ = gdn.qk_norm_rope(q, None, w, None, c.pos, c.freq, **c.turn)
        return float((out.double() * c.gq.double()).sum()), float((out.double() * c.gq.double()).abs().sum())
    h = 2.0 ** -7
    third = h * h / 6 * 20 * float(c.gq.abs().sum())
    for t, h_, f in ((0, 0, 3), (1, 1, 0), (1, 0, 15)):
        up, dn = c.q.clone(), c.q.clone()
        up[0, t, h_, f] += h
        dn[0, t, h_, f] -= h
        (a, s), (b, _) = loss(up, c.wq), loss(dn, c.wq)
        step = float(up[0, t, h_, f].double() - dn[0, t, h_, f].double())
        assert abs((a - b) / step - float(g["dq"][0, t, h_, f])) <= 33 * U * s * 2 / step + third
    for f in (0, 9):
        up, dn = c.wq.clone(), c.wq.clone()
        up[f] += h
        dn[f] -= h
        (a, s), (b, _) = loss(c.q, up), loss(c.q, dn)
        step = float(up[f].double() - dn[f].double())
        assert abs((a - b) / step - float(g["dq_weight"][f])) <= 33 * U * s * 2 / step


def test_norm_alone_and_defaults():
    c = Case(2, 9, 3, 2, 96, 16, "bf16", "half", (8,), 11)
    q, k = gdn.qk_norm_rope(c.q, c.k)
    for x, o in ((c.q, q), (c.k, k)):
        ref = nr.norm(np64(x), None, 1e-6)
        assert (np.abs(np64(o) - ref) <= 2.0 ** -8 * 1.01 * np.abs(ref) + 32 * U * np.abs(ref)).all()
    q1, none = gdn.qk_norm_rope(c.q, None)
    assert none is None and torch.equal(q, q1)
    g = gdn.qk_norm_rope_backward(c.q, None, None, None, c.gq, None)
    assert g["dk"] is None and g["dk_weight"] is None
    ref, refw = nr.norm_turn_backward(np64(c.q), None, 1e-6, np64(c.gq))
    assert np.abs(np64(g["dq"]) - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
    assert np.abs(np64(g["dq_weight"]) - refw).max() <= 128 * U * 54 * 20


@pytest.mark.parametrize("form", ["T", "BT", "TA", "BTA", "int32", "expanded"])
def test_position_forms(form):
    sections = (10, 6) if form in ("TA", "BTA") else (16,)
    c = Case(3, 21, 2, 1, 48, 32, "f32", "half", sections, 12)
    if form in ("T", "TA", "expanded"):
        c.pos = c.pos[:1].expand(3, -1, -1)
        c.angle = nr.angles(c.pos.cpu().numpy(), c.freq.cpu().numpy(), sections)
    pos = {"T": c.pos[0, :, 0], "BT": c.pos[:, :, 0], "TA": c.pos[0], "BTA": c.pos, "int32": c.pos.int(),
           "expanded": c.pos[:1].contiguous().expand(3, -1, -1)}[form]
    if form in ("T", "BT"):
        pos = pos.contiguous()
    qo, ko = gdn.qk_norm_rope(c.q, c.k, c.wq, c.wk, pos, c.freq, **c.turn)
    c.check_forward(qo, c.q, c.wq)
    c.check_forward(ko, c.k, c.wk)


def test_far_positions_keep_their_angles():
    """Positions near +-2^31: the fp64 angle's own rounding, 3 half steps of at most
    2^31 / 2 pi turns, is 3 * 2^-53 * 3.5e8 = 1.2e-7 turns = 7.2e-7 rad = 12 u more than the
    near ones', within the 32 u of the tolerance's 24 + 12 rounded up to 36: checked with 48."""
    c = Case(1, 64, 2, 1, 32, 32, "f32", "half", (16,), 13, far=2 ** 31 - 1)
    qo, _ = gdn.rope(c.q, c.k, c.pos, c.freq, **c.turn)
    ref = nr.turn(np64(c.q), c.angle, c.layout, c.amp)
    # the oracle's own fp64 angle: half a step of 2^31 radians, 2^-53 * 2^31 = 2.4e-7 = 4 u, and its reduction
    assert (np.abs(np64(qo) - ref) <= U * np.abs(ref) * 1.01 + 48 * U * c.size(np64(c.q))).all()


def test_in_place_views_of_one_projection():
    c = Case(2, 50, 6, 2, 112, 64, "bf16", "half", (32,), 14, packed=True)
    want = gdn.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.pos, c.freq, **c.turn)
    base = c.q._base.clone()
    q, k, v = base[:, :, :6], base[:, :, 6:8], base[:, :, 8:].clone()
    got = gdn.qk_norm_rope(q, k, c.wq, c.wk, c.pos, c.freq, q_out=q, k_out=k, **c.turn)
    assert got[0] is q and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(base[:, :, 8:], v)                       # the values between the rows
    gq, gk = c.gq.clone(), c.gk.clone()
    ref = gdn.qk_norm_rope_backward(c.q, c.k, c.wq, c.wk, gq, gk, c.pos, c.freq, **c.turn)
    gdn.qk_norm_rope_backward(c.q, c.k, c.wq, c.wk, gq, gk, c.pos, c.freq, dq=gq, dk=gk, **c.turn)
    assert torch.equal(gq, ref["dq"]) and torch.equal(gk, ref["dk"])


def test_sequence_first_and_neighbours_untouched():
    c = Case(3, 20, 2, 2, 64, 32, "bf16", "interleaved", (16,), 15)
    want = gdn.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.pos, c.freq, **c.turn)
    pad = torch.full((20, 3, 5, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    qo, ko = pad[:, :, :2].transpose(0, 1), pad[:, :, 3:].transpose(0, 1)
    gdn.qk_norm_rope(c.q.transpose(0, 1).contiguous().transpose(0, 1), c.k, c.wq, c.wk, c.pos, c.freq,
                     q_out=qo, k_out=ko, **c.turn)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert (pad[:, :, 2] == 7).all()


def test_infinity_stays_in_its_place():
    """A feature that does not turn keeps its infinity from its neighbours."""
    c = Case(1, 4, 2, 1, 32, 16, "f32", "half", (8,), 16)
    for layout in ("half", "interleaved"):
        x = c.q.clone()
        x[..., 20] = float("inf")
        out, _ = gdn.rope(x, None, c.pos, c.freq, sections=(8,), layout=layout)
        assert torch.isinf(out[..., 20]).all()
        out[..., 20] = 0
        assert torch.isfinite(out).all()
        assert torch.equal(out[..., 21:], x[..., 21:])


def test_offsets_past_32_bits():
    """Tokens 2^30 elements apart: the third starts at element 2^31."""
    flat = torch.zeros((1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    q = flat.as_strided((1, 3, 1, 64), (0, 1 << 30, 64, 1))
    x = torch.randn(1, 3, 1, 64, device="cuda").bfloat16()
    q.copy_(x)
    pos = torch.arange(3, device="cuda") + 5
    f, _ = gdn.rope_frequencies(64)
    want, _ = gdn.qk_norm_rope(x, None, None, None, pos, f)
    got, _ = gdn.qk_norm_rope(q, None, None, None, pos, f)
    assert torch.equal(got, want)
    gdn.qk_norm_rope(q, None, None, None, pos, f, q_out=q)
    assert torch.equal(q, want)


def test_empty_calls():
    f, _ = gdn.rope_frequencies(32)
    for B, T, H in ((0, 3, 2), (2, 0, 2)):
        q = torch.zeros(B, T, H, 32, dtype=torch.bfloat16, device="cuda")
        pos = torch.zeros(B, T, dtype=torch.int64, device="cuda")
        out, _ = gdn.qk_norm_rope(q, q, None, None, pos, f)
        assert out.shape == q.shape
        g = gdn.qk_norm_rope_backward(q, q, None, None, q, q, pos, f)
        assert (g["dq_weight"] == 0).all() and (g["dk_weight"] == 0).all()


def test_another_stream_and_two_graphs():
    """Two backward calls captured on one stream, replayed at the same time on two
    others: each graph has its own scratch, so both give the eager call's bits."""
    cs = [Case(2, 900, 8, 4, 64, 64, "bf16", "half", (32,), s) for s in (17, 18)]

    def call(c, **kw):
        return gdn.qk_norm_rope_backward(c.q, c.k, c.wq, c.wk, c.gq, c.gk, c.pos, c.freq, **c.turn, **kw)
    want = [call(c) for c in cs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = [call(c, stream=s) for c in cs]
    torch.cuda.current_stream().wait_stream(s)
    for w, o in zip(want, other):
        assert all(torch.equal(w[n], o[n]) for n in w)
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(c))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for o in outs:
            for t in o.values():
                t.fill_(0)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(w[n], o[n]) for n in w)


def test_device_side_refusals():
    q = torch.zeros(1, 4, 2, 32, dtype=torch.bfloat16, device="cuda")
    f, _ = gdn.rope_frequencies(32)
    pos = torch.arange(4, device="cuda")
    with pytest.raises(ValueError):
        gdn.rope(q, None, pos.cpu(), f)
    with pytest.raises(ValueError):
        gdn.rope(q, None, pos, f, layout="other")
    with pytest.raises(ValueError):
        gdn.rope(q, None, pos[:3], f)
    with pytest.raises(TypeError):
        gdn.rope(q, None, pos, f.float())
    with pytest.raises(TypeError):
        gdn.rope(q, None, pos.float(), f)
    with pytest.raises(ValueError):
        gdn.rope(q.transpose(2, 3).contiguous().transpose(2, 3), None, pos, f)
    with pytest.raises(gdn.GDNError, match="ALIAS"):
        gdn.rope(q[:, :, :1], None, pos, f, q_out=q[:, :, :1].flip(1)[:, :1].expand(1, 4, 1, 32))
