"""GPU parity of the attention to an encoder's states against the fp64 formulas.

Tolerances, element by element, with u = 2^-24 and h = 2^-8 (half a step of bf16):
* a score's error: D products and sums in fp32 (the tensor core may drop the bits
  below its 24: 2 u per step), the scale and the subtraction of the maximum:
  d = 2 u (D + 4) * scale sum |q k|, its largest over the row; p = e^s is off by
  d relative, by 7.5e-5 where the polynomial forms it (2^-22 elsewhere), and P by h;
* out: (h + 8e-5 + 2 d) sum p |v| from P and the row sum, and h |out| from the
  rounding at the end;
* lse: 8e-5 + d + 4 u |lse|.
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


@pytest.mark.parametrize("q_scale", [6.0, 40.0])
def test_sharp_softmax(q_scale):
    c = Case(1, 200, 900, 2, 1, 64, "holes", 5, q_scale=q_scale)
    c.check(*gdn.cross_attention(c.q, c.k, c.v, c.mask, return_lse=True))


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
    want = gdn.cross_attention(c.q, c.k, c.v, c.mask, return_lse=True)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.3e38], device="cuda").bfloat16()
    k, v = c.k.clone(), c.v.clone()
    for x in (k, v):
        where = ~c.mask
        x[where] = bad[torch.arange(int(where.sum()), device="cuda") % 4][:, None, None]
    got = gdn.cross_attention(c.q, k, v, c.mask, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isneginf(got[1][-1]).all() and (got[0][-1] == 0).all()


def test_no_keys():
    q = torch.randn(2, 5, 4, 32, device="cuda").bfloat16()
    k = torch.empty(2, 0, 2, 32, device="cuda").bfloat16()
    out, lse = gdn.cross_attention(q, k, k, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert gdn.cross_attention(q[:, :0], k, k).shape == (2, 0, 4, 32)
    assert gdn.cross_attention(q[:0], k[:0], k[:0]).shape == (0, 5, 4, 32)


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
    c.check(gdn.cross_attention(c.q, c.k, c.v, c.mask))


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
