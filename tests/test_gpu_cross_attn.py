"""GPU parity of the attention to an encoder's states against the fp64 formulas.

Tolerances, element by element, with u = 2^-24 and h = 2^-8 (half a step of bf16):
* a score's error: D products and sums in fp32 (the tensor core may drop the bits
  below its 24: 2 u per step), the scale and the subtraction of the maximum:
  d = 2 u (D + 4) * scale sum |q k|, its largest over the row; p = e^s is off by
  d relative, by 7.5e-5 where the polynomial forms it (2^-22 elsewhere), and P by h;
* out: (h + 8e-5 + 2 d) sum p |v| from P and the row sum, and h |out| from the
  rounding at the end;
* lse: 8e-5 + d + 4 u |lse|.
Gradients, from bounds on each factor carried through the products:
* P: e_P = d + 2^-22 + 4 u (|s| + |lse|) + the error of lse, relative; h more as an operand;
* dP: 2 u (D + 4) sum |dO v|;  delta: sum |dO| (the error of out) + 2 u (D + 4) sum |dO out|;
* dS: P ((h + e_P) |dP - delta| + both errors);
* dv: h |dv| + sum (h + e_P) P |dO|, dk, dq: h |.| + scale sum (error of dS) |q or k|; each sum
  in fp32 over n products adds 2 u (n + 4) of its absolute terms.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_chunked_b200 as gdn
from gated_deltanet_linear_chunked_b200 import _lib
from oracle import cross_attn as ca

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8


def np64(t):
    return t.detach().double().cpu().numpy()


class Case:
    def __init__(self, B, Tq, S, Hk, G, D, mask, seed, q_scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.q = (q_scale * n(B, Tq, Hk * G, D)).bfloat16()
        kv = n(B, S, 2, Hk, D)
        self.k, self.v = kv[:, :, 0], kv[:, :, 1]
        self.g = n(B, Tq, Hk * G, D)
        self.mask = None
        if mask == "tail":
            keep = torch.tensor([S - (b + 1) * S // (4 * B) for b in range(B)], device="cuda")
            self.mask = torch.arange(S, device="cuda")[None] < keep[:, None]
        elif mask == "holes":
            self.mask = torch.rand((B, S), generator=g, device="cuda") < 0.6
            if B > 1:
                self.mask[-1] = False
        elif mask == "far":  # one key, in the last tile
            self.mask = torch.zeros((B, S), dtype=torch.bool, device="cuda")
            self.mask[:, -1] = True
        self.np = {n: np64(getattr(self, n)) for n in ("q", "k", "v", "g")}
        self.npmask = None if self.mask is None else self.mask.cpu().numpy()

    def score_error(self):
        """d of every query row: [B, Hq, Tq]."""
        q, k = np.abs(self.np["q"]), np.abs(self.np["k"])
        B, Tq, Hq, D = q.shape
        d = np.zeros((B, Hq, Tq))
        if k.shape[1]:
            for b in range(B):
                for h in range(Hq):
                    d[b, h] = (q[b, :, h] @ k[b, :, h // (Hq // k.shape[2])].T).max(-1)
        return 2 * U * (D + 4) * d * D ** -0.5

    def check(self, out, lse=None):
        q, k, v = (self.np[n] for n in ("q", "k", "v"))
        ref, rlse = ca.forward(q, k, v, self.npmask)
        size, _ = ca.forward(q, k, np.abs(v), self.npmask)
        d = self.score_error()
        tol = H * np.abs(ref) + (H + 8e-5 + 2 * d.transpose(0, 2, 1)[..., None]) * size
        err = np.abs(np64(out) - ref)
        assert out.shape == ref.shape and (err <= tol).all(), float((err / (tol + 1e-300)).max())
        if lse is not None:
            got = np64(lse)
            assert lse.dtype == torch.float32 and lse.shape == rlse.shape
            none = np.isinf(rlse)
            assert (np.isneginf(got) == none).all()
            e = np.abs(got[~none] - rlse[~none])
            assert (e <= 8e-5 + d[~none] + 4 * U * np.abs(rlse[~none])).all(), e.max()


    def check_grads(self, got):
        q, k, v, g = (self.np[n] for n in ("q", "k", "v", "g"))
        B, Tq, Hq, D = q.shape
        S, Hk = k.shape[1:3]
        G, scale = Hq // Hk, D ** -0.5
        ref = dict(zip(("dq", "dk", "dv"), ca.backward(q, k, v, g, self.npmask)))
        out, lse = ca.forward(q, k, v, self.npmask)
        size, _ = ca.forward(q, k, np.abs(v), self.npmask)
        d = self.score_error()
        e_out = H * np.abs(out) + (H + 8e-5 + 2 * d.transpose(0, 2, 1)[..., None]) * size
        tol = {n: np.zeros_like(x) for n, x in ref.items()}
        for b in range(B):
            keep = np.arange(S) if self.npmask is None else np.flatnonzero(self.npmask[b])
            for h in range(Hq if len(keep) else 0):
                kh, vh = np.abs(k[b, keep, h // G]), np.abs(v[b, keep, h // G])
                s = scale * (q[b, :, h] @ k[b, keep, h // G].T)
                p = np.exp(s - lse[b, h][:, None])
                dp = g[b, :, h] @ v[b, keep, h // G].T
                delta = np.sum(g[b, :, h] * out[b, :, h], -1, keepdims=True)
                ga = np.abs(g[b, :, h])
                e_lse = 8e-5 + d[b, h][:, None] + 4 * U * np.abs(lse[b, h])[:, None]
                e_p = d[b, h][:, None] + 2.0 ** -22 + 4 * U * (np.abs(s) + np.abs(lse[b, h])[:, None]) + e_lse
                e_dp = 2 * U * (D + 4) * (ga @ vh.T)
                e_delta = np.sum(ga * e_out[b, :, h], -1, keepdims=True) * (1 + 2 * U * (D + 4)) + \
                    2 * U * (D + 4) * np.sum(ga * np.abs(out[b, :, h]), -1, keepdims=True)
                size_ds = p * np.abs(dp - delta)
                e_ds = p * ((H + e_p) * np.abs(dp - delta) + (1 + H + e_p) * (e_dp + e_delta))
                nq, nk = 2 * U * (Tq * G + 4), 2 * U * (S + 4)
                tol["dv"][b, keep, h // G] += ((H + e_p + nq) * p).T @ ga
                tol["dk"][b, keep, h // G] += scale * (e_ds + nq * size_ds).T @ np.abs(q[b, :, h])
                tol["dq"][b, :, h] = scale * (e_ds + nk * size_ds) @ kh
        for n, x in ref.items():
            err = np.abs(np64(got[n]) - x)
            t = H * np.abs(x) + tol[n] * (1 + H)
            assert got[n].dtype == torch.bfloat16 and got[n].shape == x.shape
            assert (err <= t).all(), (n, float((err / (t + 1e-300)).max()))
            if np.abs(x).max() > 0:   # and well within the type's accuracy as a whole
                assert np.linalg.norm(err) <= 2 * H * np.linalg.norm(x), (n, np.linalg.norm(err) / np.linalg.norm(x))


CASES = [
    # B, Tq, S, Hk, G, D, mask
    (1, 1, 1, 1, 1, 16, "none"),
    (1, 128, 128, 1, 1, 64, "none"),
    (1, 256, 256, 2, 1, 128, "none"),
    (2, 130, 129, 2, 1, 112, "none"),
    (1, 333, 77, 2, 3, 80, "holes"),
    (3, 100, 300, 1, 2, 96, "tail"),
    (2, 64, 500, 2, 8, 32, "holes"),
    (1, 17, 1000, 1, 16, 48, "tail"),
    (2, 5, 127, 1, 128, 16, "none"),
    (4, 1, 2000, 2, 4, 128, "tail"),
    (2, 3, 700, 3, 1, 112, "far"),
    (1, 700, 300, 4, 1, 112, "tail"),
    (2, 257, 64, 1, 5, 64, "holes"),
    (1, 129, 20000, 1, 1, 32, "holes"),
    (1, 300, 4000, 1, 1, 128, "none"),
    # at most 16 rows of a key head
    (2, 16, 50, 1, 1, 48, "holes"),
    (1, 1, 5000, 1, 16, 80, "none"),
    (3, 2, 333, 2, 7, 64, "tail"),
    (2, 5, 100, 1, 3, 32, "none"),
    (1, 4, 17, 2, 4, 96, "holes"),
    (9, 1, 700, 40, 1, 112, "tail"),
    (4, 513, 1000, 20, 1, 16, "holes"),   # most units whole, the last wave's split along the keys
    (4, 260, 2100, 20, 1, 32, "tail"),
    (5, 1, 4100, 8, 3, 64, "holes"),      # a cluster of CTAs a key head, more rows than CTAs or fewer
    (8, 2, 4100, 4, 8, 128, "tail"),
    (1, 1, 300, 30, 1, 80, "none"),
]


@pytest.mark.parametrize("B,Tq,S,Hk,G,D,mask", CASES)
def test_forward(B, Tq, S, Hk, G, D, mask):
    c = Case(B, Tq, S, Hk, G, D, mask, 7 * Tq + S + D)
    out, lse = gdn.cross_attention(c.q, c.k, c.v, c.mask, return_lse=True)
    torch.cuda.synchronize()
    assert gdn.device_error() == _lib.GDN_OK
    c.check(out, lse)
    assert torch.equal(gdn.cross_attention(c.q, c.k, c.v, c.mask), out)   # and the same bits again
    if mask == "none":
        full = torch.ones(B, S, dtype=torch.uint8, device="cuda")
        torch.testing.assert_close(gdn.cross_attention(c.q, c.k, c.v, full), out, rtol=0, atol=0)


def both(c, mask="own", **kw):
    mask = c.mask if isinstance(mask, str) else mask
    out, lse = gdn.cross_attention(c.q, c.k, c.v, mask, return_lse=True, **kw)
    return out, lse, gdn.cross_attention_backward(c.q, c.k, c.v, out, lse, c.g, mask, **kw)


@pytest.mark.parametrize("B,Tq,S,Hk,G,D,mask", [x for x in CASES if x[2] != 20000 and x[3] != 20] + [
    (1, 2000, 130, 1, 2, 64, "none"),      # many query tiles to few key tiles: shares of them
    (1, 128, 1, 1, 1, 32, "none"),
    (2, 40, 3000, 1, 3, 48, "far"),
    (2, 20, 2500, 2, 2, 64, "holes"),      # few query tiles to many key tiles: shares of those
    (1, 1, 9000, 1, 16, 32, "tail"),
])
def test_gradients(B, Tq, S, Hk, G, D, mask):
    c = Case(B, Tq, S, Hk, G, D, mask, 3 * Tq + S + D)
    out, lse, grads = both(c)
    torch.cuda.synchronize()
    assert gdn.device_error() == _lib.GDN_OK
    c.check_grads(grads)
    again = gdn.cross_attention_backward(c.q, c.k, c.v, out, lse, c.g, c.mask)
    assert all(torch.equal(grads[n], again[n]) for n in grads)          # the same bits
    if c.mask is not None:
        assert (grads["dk"][~c.mask] == 0).all() and (grads["dv"][~c.mask] == 0).all()


@pytest.mark.parametrize("Tq,S,G,D,mask", [(50, 2, 1, 64, "none"), (33, 5, 3, 80, "holes"), (1, 8, 4, 128, "none"),
                                           (70, 60, 2, 32, "tail")])
def test_gradients_of_few_keys(Tq, S, G, D, mask):
    """With few keys neither dS's rounding nor that of out is in dq and dk, only their
    own.  dS = P (dP - delta), delta = A = sum P dP: P is off by e_P = 7.5e-5 (the
    polynomial) + d + the error of lse (8e-5 + d), so P dP and P delta by P |dP| e_P and
    P sum(P |dP|) 2 e_P, dS's two terms by 2^-16, and out, from 9 keys on, by its
    rounding in delta: sum |dO| (H |out| + (H + 8e-5 + 2 d) sum P |v|)."""
    c = Case(2, Tq, S, 2, G, D, mask, 5 * S + Tq)
    _, _, grads = both(c)
    q, k, v, g = (c.np[n] for n in ("q", "k", "v", "g"))
    ref = dict(zip(("dq", "dk", "dv"), ca.backward(q, k, v, g, c.npmask)))
    out, lse = ca.forward(q, k, v, c.npmask)
    size, _ = ca.forward(q, k, np.abs(v), c.npmask)
    d, scale = c.score_error(), D ** -0.5
    tol = {n: np.zeros_like(x) for n, x in ref.items()}
    for b in range(2):
        keep = np.arange(S) if c.npmask is None else np.flatnonzero(c.npmask[b])
        for h in range(2 * G if len(keep) else 0):
            kh, vh = k[b, keep, h // G], v[b, keep, h // G]
            p = np.exp(scale * (q[b, :, h] @ kh.T) - lse[b, h][:, None])
            dp = np.abs(g[b, :, h] @ vh.T)
            e_p = 1.6e-4 + 2 * d[b, h][:, None]
            a = np.sum(p * dp, -1, keepdims=True)
            e = p * ((dp + 2 * a) * e_p + (dp + a) * 2.0 ** -16 + 4 * U * (D + 4) * (np.abs(g[b, :, h]) @ np.abs(vh).T))
            if S > 8:
                rounded = H * np.abs(out[b, :, h]) + (H + 8e-5 + 2 * d[b, h][:, None]) * size[b, :, h]
                e += p * np.sum(np.abs(g[b, :, h]) * rounded, -1, keepdims=True)
            tol["dq"][b, :, h] = scale * e @ np.abs(kh)
            tol["dk"][b, keep, h // G] += scale * e.T @ np.abs(q[b, :, h])
    for n in ("dq", "dk"):
        err = np.abs(np64(grads[n]) - ref[n])
        t = H * np.abs(ref[n]) + (1 + H) * tol[n]
        assert (err <= t).all(), (n, float((err / (t + 1e-300)).max()))


def test_gradients_along_a_direction():
    """<gradient, step> against central differences of the fp64 oracle's loss along a
    random step: the differences are exact to 1e-6, the gradients to 2 h of their
    norms, so the products differ by at most 2 h |gradient| |step|."""
    c = Case(2, 70, 150, 2, 2, 64, "holes", 31)
    _, _, grads = both(c)
    rng = np.random.default_rng(5)
    for n, name in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        step = rng.standard_normal(c.np[n].shape)

        def loss(e):
            x = dict(c.np)
            x[n] = x[n] + e * step
            return np.sum(x["g"] * ca.forward(x["q"], x["k"], x["v"], c.npmask)[0])
        slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
        d = np64(grads[name])
        assert abs(slope - np.sum(d * step)) <= 2 * H * np.linalg.norm(d) * np.linalg.norm(step) + 1e-5 * abs(slope)


@pytest.mark.parametrize("q_scale", [6.0, 40.0])
def test_sharp_softmax(q_scale):
    c = Case(1, 200, 900, 2, 1, 64, "holes", 5, q_scale=q_scale)
    out, lse, grads = both(c)
    c.check(out, lse)
    if q_scale < 10:
        c.check_grads(grads)


def test_growing_scores():
    """Scores that rise along the keys by far more than the headroom: every tile rescales."""
    c = Case(1, 130, 1200, 1, 1, 64, "none", 6)
    k = c.k.clone()
    k[..., 0] = torch.linspace(-60, 60, 1200, device="cuda")[None, :, None].bfloat16()
    q = c.q.clone()
    q[..., 0] = 20.0
    c.q, c.k = q, k
    c.np["q"], c.np["k"] = np64(q), np64(k)
    c.check(*gdn.cross_attention(c.q, c.k, c.v, None, return_lse=True))


@pytest.mark.parametrize("Tq,G", [(300, 1), (1, 4), (100, 3)])
def test_masked_places_hold_anything(Tq, G):
    """NaN, infinities and the type's largest values in masked keys and values
    change no bit, in tiles that are masked in part and in whole."""
    c = Case(2, Tq, 700, 2, G, 80, "holes", 9)
    c.mask[0, 128:300] = False
    want = both(c)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.3e38], device="cuda").bfloat16()
    k, v = c.k.clone(), c.v.clone()
    for x in (k, v):
        where = ~c.mask
        x[where] = bad[torch.arange(int(where.sum()), device="cuda") % 4][:, None, None]
    c.k, c.v = k, v
    got = both(c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isneginf(got[1][-1]).all() and (got[0][-1] == 0).all()
    assert all(torch.equal(got[2][n], want[2][n]) for n in want[2])
    assert (got[2]["dq"][-1] == 0).all()


@pytest.mark.parametrize("Tq,S,G", [(1, 40, 4), (1, 1000, 4), (1, 5000, 4), (300, 300, 1), (300, 4000, 1)])
def test_nan_is_not_hidden(Tq, S, G):
    """A query row of NaN gives NaN for that row, whichever way its parts are joined,
    and leaves the others' bits; a seen key of NaN reaches every row."""
    c = Case(1, Tq, S, 2, G, 64, "none", 17)
    out, lse, grads = both(c)
    t, h = Tq // 2, G // 2
    q = c.q.clone()
    q[0, t, h] = float("nan")
    o, l = gdn.cross_attention(q, c.k, c.v, return_lse=True)
    g = gdn.cross_attention_backward(q, c.k, c.v, o, l, c.g)
    other = torch.ones(Tq, 2 * G, dtype=torch.bool, device="cuda")
    other[t, h] = False
    assert o[0, t, h].isnan().all() and l[0, h, t].isnan()
    assert torch.equal(o[0][other], out[0][other]) and torch.equal(l[0].T[other], lse[0].T[other])
    assert g["dq"][0, t, h].isnan().all() and torch.equal(g["dq"][0][other], grads["dq"][0][other])
    for n in ("dk", "dv"):
        assert not g[n][0, :, 0].isfinite().any() and torch.equal(g[n][0, :, 1], grads[n][0, :, 1])
    k = c.k.clone()
    k[0, S // 32 * 16 + 14, 1] = float("nan")   # (a key whose exponential is the polynomial's)
    o, l = gdn.cross_attention(c.q, k, c.v, return_lse=True)
    g = gdn.cross_attention_backward(c.q, k, c.v, o, l, c.g)
    assert o[0, :, G:].isnan().all() and l[0, G:].isnan().all() and torch.equal(o[0, :, :G], out[0, :, :G])
    for n, x in (("dq", g["dq"][0, :, G:]), ("dk", g["dk"][0, :, 1]), ("dv", g["dv"][0, :, 1])):
        assert not x.isfinite().any(), n
    assert torch.equal(g["dk"][0, :, 0], grads["dk"][0, :, 0])


@pytest.mark.parametrize("Tq,S,G", [(1, 40, 4), (1, 1000, 4), (1, 5000, 4), (300, 300, 1), (300, 4000, 1),
                                    (40, 5000, 3), (2000, 2500, 1)])
def test_scores_of_minus_infinity(Tq, S, G):
    """Seen keys whose score is -inf have no weight, wherever they lie and however many
    query rows there are; a row that has no other scores gives 0 and -inf, as one that
    keeps no key."""
    c = Case(2, Tq, S, 2, G, 64, "none", 51)
    c.q = c.q.clone()
    c.q[..., 0] = 1.0
    c.np["q"] = np64(c.q)
    gone = torch.arange(S, device="cuda") % 3 == 1
    gone[:S // 2] = True
    k = c.k.clone()
    k[:, gone, :, 0] = -float("inf")
    c.npmask = (~gone)[None].expand(2, -1).cpu().numpy()
    c.check(*gdn.cross_attention(c.q, k, c.v, return_lse=True))
    k[1, ..., 0] = -float("inf")
    c.npmask = c.npmask.copy()
    c.npmask[1] = False
    c.check(*gdn.cross_attention(c.q, k, c.v, return_lse=True))


@pytest.mark.parametrize("Tq,S", [(1, 40), (1, 5000), (300, 300), (300, 2500)])
def test_scores_of_a_thousand_million(Tq, S):
    """Scores of +-2^30, exact in fp32: the one key that matches is all of the result."""
    c = Case(1, Tq, S, 1, 1, 16, "none", 52)
    q, k = torch.zeros_like(c.q), torch.zeros(1, S, 1, 16, dtype=torch.bfloat16, device="cuda")
    q[..., 0], k[..., 0] = 2.0 ** 15, -2.0 ** 15
    k[:, S // 2 + 9, :, 0] = 2.0 ** 15
    out, lse = gdn.cross_attention(q, k, c.v, scale=1.0, return_lse=True)
    v = np64(c.v)[:, S // 2 + 9]
    assert (np.abs(np64(out) - v[:, None]) <= 2 * H * np.abs(v[:, None])).all()
    assert (np.abs(np64(lse) - 2.0 ** 30) <= 8 * U * 2.0 ** 30).all()


@pytest.mark.parametrize("S", [131072, 140001])
def test_long_mask(S):
    """As many masked keys as one CTA lists, and more (each CTA then takes a part)."""
    c = Case(2, 40, S, 1, 1, 16, "holes", S)
    out, lse = gdn.cross_attention(c.q, c.k, c.v, c.mask, return_lse=True)
    c.check(out, lse)


def test_no_keys():
    q = torch.randn(2, 5, 4, 32, device="cuda").bfloat16()
    k = torch.empty(2, 0, 2, 32, device="cuda").bfloat16()
    out, lse = gdn.cross_attention(q, k, k, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    grads = gdn.cross_attention_backward(q, k, k, out, lse, q)
    assert (grads["dq"] == 0).all() and grads["dk"].shape == k.shape
    k1 = torch.randn(2, 9, 2, 32, device="cuda").bfloat16()
    e = q[:, :0]
    grads = gdn.cross_attention_backward(e, k1, k1, e, lse[:, :, :0].contiguous(), e)
    assert (grads["dk"] == 0).all() and (grads["dv"] == 0).all() and grads["dk"].shape == k1.shape
    assert gdn.cross_attention(q[:, :0], k, k).shape == (2, 0, 4, 32)
    assert gdn.cross_attention(q[:0], k[:0], k[:0]).shape == (0, 5, 4, 32)


@pytest.mark.parametrize("Tq,S,G", [(300, 0, 1), (1500, 0, 3), (300, 300, 1), (1500, 77, 3), (300, 2500, 1), (70, 4000, 5)])
def test_batch_rows_without_keys_in_tiles(Tq, S, G):
    """More than 16 query rows a key head and nothing to attend to, in CTAs of one query
    tile and of two and along split keys: zeros and -inf in every row, whenever the
    queries arrive; a row of the batch that sees keys keeps its bits."""
    c = Case(24, Tq, S, 2, G, 112, "none", 41)
    if S:
        c.mask = torch.zeros(24, S, dtype=torch.bool, device="cuda")
        c.mask[5] = True
        c.npmask = c.mask.cpu().numpy()
    first = None
    for _ in range(30):
        out = torch.full_like(c.q, 7.0)
        out, lse = gdn.cross_attention(c.q, c.k, c.v, c.mask, out=out, return_lse=True)
        if first is None:
            c.check(out, lse)
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert gdn.device_error() == _lib.GDN_OK


def test_views_and_broadcast():
    """Queries inside a wider projection, states shared by the batch, scale given."""
    wide = torch.randn(3, 70, 9, 48, device="cuda").bfloat16()
    q = wide[:, :, 2:6]
    kv = torch.randn(1, 150, 2, 2, 48, device="cuda").bfloat16().expand(3, -1, -1, -1, -1)
    k, v = kv[:, :, 0], kv[:, :, 1]
    mask = (torch.arange(150, device="cuda") % 5 != 0)[None].expand(3, -1)
    got = gdn.cross_attention(q, k, v, mask, scale=0.3)
    want = gdn.cross_attention(q.contiguous(), k.contiguous(), v.contiguous(), mask.contiguous(), scale=0.3)
    assert torch.equal(got, want)
    ref, _ = ca.forward(np64(q), np64(k), np64(v), mask.cpu().numpy(), scale=0.3)
    assert np.abs(np64(got) - ref).max() <= 2 * H * np.abs(np64(v)).max()
    out, lse = gdn.cross_attention(q, k, v, mask, scale=0.3, return_lse=True)
    g = torch.randn_like(out)
    grads = gdn.cross_attention_backward(q, k, v, out, lse, g, mask, scale=0.3)
    plain = gdn.cross_attention_backward(q.contiguous(), k.contiguous(), v.contiguous(), out, lse, g,
                                         mask.contiguous(), scale=0.3)
    assert all(torch.equal(grads[n], plain[n]) for n in grads)
    dq, dk, dv = ca.backward(np64(q), np64(k), np64(v), np64(g), mask.cpu().numpy(), scale=0.3)
    for n, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert np.linalg.norm(np64(grads[n]) - x) <= 2 * H * np.linalg.norm(x), n
    # sequence first
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(gdn.cross_attention(qt, k, v, mask, scale=0.3), want)


def test_out_rows_only():
    """An output inside a larger buffer: nothing around it changes."""
    c = Case(1, 130, 200, 2, 3, 80, "tail", 21)
    n = c.q.numel()
    buf = torch.full((n + 2048,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1024:1024 + n].view(c.q.shape)
    gdn.cross_attention(c.q, c.k, c.v, c.mask, out=out)
    c.check(out)
    assert (buf[:1024] == 5).all() and (buf[1024 + n:] == 5).all()


def test_expired_wait_reports_timeout_and_next_call_is_right():
    c = Case(1, 300, 500, 2, 1, 64, "tail", 22)
    assert gdn.device_error() == _lib.GDN_OK
    gdn.set_wait_limit(1)
    try:
        gdn.cross_attention(c.q, c.k, c.v, c.mask)
        torch.cuda.synchronize()
    finally:
        gdn.set_wait_limit(0)
    assert gdn.device_error() == _lib.GDN_ERR_TIMEOUT
    assert gdn.device_error() == _lib.GDN_OK
    out, lse, want = both(c)
    c.check(out)
    gdn.set_wait_limit(1)
    try:
        gdn.cross_attention_backward(c.q, c.k, c.v, out, lse, c.g, c.mask)
        torch.cuda.synchronize()
    finally:
        gdn.set_wait_limit(0)
    assert gdn.device_error() == _lib.GDN_ERR_TIMEOUT
    got = gdn.cross_attention_backward(c.q, c.k, c.v, out, lse, c.g, c.mask)
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_two_graphs_of_one_stream():
    """Split calls captured on one stream and replayed together on two others."""
    cs = [Case(1, 3, 6000, 2, 2, 64, "tail", s) for s in (23, 24)]
    want = [gdn.cross_attention(c.q, c.k, c.v, c.mask, return_lse=True) for c in cs]
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gdn.cross_attention(c.q, c.k, c.v, c.mask, return_lse=True))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])
            o[0].zero_()
            o[1].zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gdn.cross_attention(cs[0].q, cs[0].k, cs[0].v, cs[0].mask, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want[0][0])


def test_gradients_in_two_graphs_of_one_stream():
    """Forward and gradients in a graph each, replayed together: shares, row
    statistics and mask lists are each graph's own."""
    cs = [Case(1, 2500, 200, 2, 1, 64, "holes", s) for s in (26, 27)]
    want = [both(c) for c in cs]
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(c))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert torch.equal(w[0], o[0]) and all(torch.equal(w[2][n], o[2][n]) for n in w[2])
            for x in (o[0], o[1], *o[2].values()):
                x.zero_()


def test_refusals():
    c = Case(1, 8, 8, 2, 1, 32, "none", 25)
    with pytest.raises(gdn.GDNError, match="INVALID_ARG"):
        gdn.cross_attention(c.q[:, :, :1], c.k, c.v)
    with pytest.raises(gdn.GDNError, match="INVALID_ARG"):
        gdn.cross_attention(c.q, c.k, c.v, scale=-1.0)
    with pytest.raises(TypeError):
        gdn.cross_attention(c.q.float(), c.k, c.v)
    with pytest.raises(TypeError):
        gdn.cross_attention(c.q, c.k, c.v, torch.ones(1, 8, device="cuda"))
    with pytest.raises(ValueError):
        gdn.cross_attention(c.q, c.k, c.v, torch.ones(1, 7, device="cuda", dtype=torch.bool))
    with pytest.raises(gdn.GDNError, match="ALIAS"):
        gdn.cross_attention(c.q, c.k, c.v, out=c.q)
    out, lse = gdn.cross_attention(c.q, c.k, c.v, return_lse=True)
    with pytest.raises(TypeError):
        gdn.cross_attention_backward(c.q, c.k, c.v, out, lse.double(), c.g)
    with pytest.raises(ValueError):
        gdn.cross_attention_backward(c.q, c.k, c.v, out, lse, c.g[:, :4])
