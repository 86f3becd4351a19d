"""The softmax block's operators in a row, as a block calls them: the projection's
queries and keys normalised and rotated (the keys straight into their cache slot),
attention over the sink and the window, then the normalised queries over the
encoder's normalised states, chunk after chunk; a training step back through the
norm and the attention to the encoder; and both inside a CUDA graph.

Every stage is held to its own oracle on the values it was given (what the stage
before stored), with that stage's own bar: the norm and rotation half a step of bf16
(2^-8) of each value and 2^-19 of its pair, the attention over the window 2e-2 of
the head's largest value, the one over the encoder 2^-7 of the sum of p |v| (P and
the result rounded to bf16) and 1e-3 for the scores' fp32 sums.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_chunked_b200 as gdn
from gated_deltanet_linear_chunked_b200 import _lib
from oracle import cross_attn as ca
from oracle import norm_rope as nr
from oracle import sink_window_attn as swa

from gdn_testlib import TOL, max_rel_per_head

pytestmark = pytest.mark.gpu

H = 2.0 ** -8


def np64(t):
    return t.detach().double().cpu().numpy()


class Block:
    def __init__(self, seed, Tc=330, heads=4, D=112, S=77, n_sink=1, window=2):
        self.Tc, self.heads, self.D, self.n_sink, self.window = Tc, heads, D, n_sink, window
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.wq, self.wk, self.wx, self.wy = (1 + 0.2 * self.normal(D) for _ in range(4))
        self.sections = (D // 2 - 2 * (D // 6), D // 6, D // 6)
        self.freq, self.amp = gdn.rope_frequencies(D, sections=self.sections)
        self.kc, self.vc = gdn.sink_window_cache(1, Tc, heads, D, n_sink, window)
        kv = self.normal(1, S, 2, heads, D).bfloat16()     # the encoder side's projection
        self.k_enc, self.v_enc = kv[:, :, 0], kv[:, :, 1]
        self.mask = torch.arange(S, device="cuda")[None] < S - 13
        self.kn_enc, _ = gdn.qk_norm_rope(self.k_enc, None, self.wy)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda")

    def positions(self, c):
        t = torch.arange(self.Tc, device="cuda")
        return torch.stack([3 * c + torch.div(t, 110, rounding_mode="floor"),
                            torch.div(t, 11, rounding_mode="floor") % 10, t % 11], -1)

    def turn(self):
        return dict(sections=self.sections, amplitude=self.amp)

    def chunk(self, c, qkv):
        """The block's calls for chunk c; returns what each stage stored."""
        h = self.heads
        slot = gdn.sink_window_slot(c, self.n_sink, self.window)
        q, _ = gdn.qk_norm_rope(qkv[:, :, :h], qkv[:, :, h:2 * h], self.wq, self.wk, self.positions(c), self.freq,
                                k_out=self.kc[:, slot], **self.turn())
        self.vc[:, slot].copy_(qkv[:, :, 2 * h:])
        a = gdn.sink_window_attention(q, self.kc[:, slot], self.vc[:, slot], self.kc, self.vc, c, self.n_sink,
                                      self.window)
        x, _ = gdn.qk_norm_rope(a, None, self.wx)
        return q, slot, a, x, gdn.cross_attention(x, self.kn_enc, self.v_enc, self.mask)


def close_norm(got, ref, pair):
    assert (np.abs(np64(got) - ref) <= 1.01 * H * np.abs(ref) + 2.0 ** -19 * pair).all()


def test_stream_of_chunks():
    b = Block(1)
    ks, vs = [], []
    for c in range(5):
        qkv = b.normal(1, b.Tc, 3 * b.heads, b.D).bfloat16()
        q, slot, a, x, out = b.chunk(c, qkv)
        torch.cuda.synchronize()
        assert gdn.device_error() == _lib.GDN_OK
        ang = nr.angles(b.positions(c)[None].cpu().numpy(), b.freq.cpu().numpy(), b.sections)
        h = b.heads
        for got, src, w in ((q, qkv[:, :, :h], b.wq), (b.kc[:, slot], qkv[:, :, h:2 * h], b.wk)):
            y = nr.norm(np64(src), np64(w), 1e-6)
            pair = np.abs(y).max(-1, keepdims=True) * 2
            close_norm(got, nr.turn(y, ang, "half", b.amp), pair)
        ks.append(np64(b.kc[:, slot]))
        vs.append(np64(qkv[:, :, 2 * h:]))
        ref = swa.chunk_output(np64(q), np.concatenate(ks, 1), np.concatenate(vs, 1), c, b.Tc, b.n_sink, b.window)
        assert max_rel_per_head(np64(a), ref, (0, 2)) <= TOL["bf16"], c
        y = nr.norm(np64(a), np64(b.wx), 1e-6)
        close_norm(x, y, np.abs(y).max(-1, keepdims=True))
        args = (np64(x), np64(b.kn_enc))
        m = b.mask.cpu().numpy()
        ref, _ = ca.forward(*args, np64(b.v_enc), m)
        size, _ = ca.forward(*args, np.abs(np64(b.v_enc)), m)
        assert (np.abs(np64(out) - ref) <= H * np.abs(ref) + (H + 1e-3) * size).all(), c


def test_captured_chunk_gives_the_same_bits():
    """One graph holds a chunk's five calls; replayed with new projections in its
    input it gives the eager calls' bits."""
    eager, graphed = Block(2), Block(2)
    inputs = [eager.normal(1, eager.Tc, 3 * eager.heads, eager.D).bfloat16() for _ in range(3)]
    static = inputs[0].clone()
    graphed.chunk(0, static)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = graphed.chunk(0, static)[-1]
    for x in inputs:
        want = eager.chunk(0, x)[-1]
        static.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(eager.kc, graphed.kc) and torch.equal(eager.vc, graphed.vc)


@pytest.mark.parametrize("captured", [False, True])
def test_training_step(captured):
    """Gradients of <out, g> through the attention to the encoder and the norms and
    rotations before it, against fp64 autograd of the whole.  On the way to each
    gradient at most ten values are rounded to bf16 (q, k, P and out going forward;
    P, dS, delta through out, the inner gradient and the result going back, and the
    scores' two operands again), each by at most h of its size: 10 h of the norm."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    B, T, S, Hk, G, D = 2, 150, 210, 2, 2, 64
    q, k, v = n(B, T, Hk * G, D).bfloat16(), n(B, S, Hk, D).bfloat16(), n(B, S, Hk, D).bfloat16()
    wq, wk = 1 + 0.2 * n(D), 1 + 0.2 * n(D)
    g = n(B, T, Hk * G, D).bfloat16()
    pos = torch.arange(T, device="cuda")
    freq, amp = gdn.rope_frequencies(32, scaling="yarn", factor=2.0, original_length=64)
    mask = torch.rand(B, S, generator=gen, device="cuda") < 0.8

    def step():
        qn, _ = gdn.qk_norm_rope(q, None, wq, None, pos, freq, amplitude=amp)
        kn, _ = gdn.qk_norm_rope(k, None, wk)
        out, lse = gdn.cross_attention(qn, kn, v, mask, return_lse=True)
        d = gdn.cross_attention_backward(qn, kn, v, out, lse, g, mask)
        dq = gdn.qk_norm_rope_backward(q, None, wq, None, d["dq"], None, pos, freq, amplitude=amp)
        dk = gdn.qk_norm_rope_backward(k, None, wk, None, d["dk"], None)
        return {"q": dq["dq"], "wq": dq["dq_weight"], "k": dk["dq"], "wk": dk["dq_weight"], "v": d["dv"]}

    if captured:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graph.replay()
        torch.cuda.synchronize()
    else:
        got = step()
    leaves = {"q": q, "k": k, "v": v, "wq": wq, "wk": wk}
    x = {name: t.double().cpu().requires_grad_() for name, t in leaves.items()}

    def norm(y, w):
        return y * w / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6)
    y = norm(x["q"], x["wq"])
    ang = (pos.double()[:, None] * freq).cpu()[None, :, None]
    c, s = amp * ang.cos(), amp * ang.sin()
    a, b = y[..., :16], y[..., 16:32]
    y = torch.cat([a * c - b * s, a * s + b * c, y[..., 32:]], -1)
    z = norm(x["k"], x["wk"]).repeat_interleave(G, 2)
    scores = torch.einsum("bthd,bshd->bhts", y, z) * D ** -0.5
    scores = scores.masked_fill(~mask.cpu()[:, None, None], -np.inf)
    out = torch.einsum("bhts,bshd->bthd", scores.softmax(-1), x["v"].repeat_interleave(G, 2))
    out.backward(g.double().cpu())
    for name, t in x.items():
        e = np.linalg.norm(np64(got[name]) - t.grad.numpy()) / np.linalg.norm(t.grad.numpy())
        assert e <= 10 * H, (name, e)


def test_two_threads_on_one_stream():
    """Two host threads call the C entries on one stream at once, which share its
    scratch (partial sums, row statistics, shares): every call's results are those of
    the same call alone."""
    import struct
    import threading
    lib = _lib.load()
    rows = lambda t: struct.pack("Pqq", t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    gen = torch.Generator(device="cuda").manual_seed(9)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    jobs = []
    for Tq, S in ((1500, 140), (2100, 260)):
        q, k, v, g = n(1, Tq, 4, 64), n(1, S, 2, 64), n(1, S, 2, 64), n(1, Tq, 4, 64)
        mask = torch.rand(1, S, generator=gen, device="cuda") < 0.7
        out, lse = gdn.cross_attention(q, k, v, mask, return_lse=True)
        want = gdn.cross_attention_backward(q, k, v, out, lse, g, mask)
        nwant = gdn.qk_norm_rope_backward(q, None, None, None, g, None)
        got = [torch.empty_like(x) for x in (q, k, v)]
        ngot = [torch.empty_like(q), torch.empty(64, device="cuda")]
        jobs.append((q, k, v, g, mask, out, lse, want, nwant, got, ngot))
    torch.cuda.synchronize()
    failed = []

    def work(j):
        q, k, v, g, mask, out, lse, _, _, (dq, dk, dv), (dx, dw) = jobs[j]
        for _ in range(200):
            st = lib.gdn_cross_attention_backward(
                rows(q), rows(k), rows(v), mask.data_ptr(), mask.stride(0), out.data_ptr(), lse.data_ptr(),
                g.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), 1, q.shape[1], k.shape[1], 4, 2, 64, 0.125,
                _lib.GDN_BF16, stream)
            st = st or lib.gdn_qk_norm_rope_backward(
                rows(q), None, None, None, None, rows(g), None, rows(dx), None, dw.data_ptr(), None, 1, q.shape[1], 4,
                0, 64, 1e-6, _lib.GDN_BF16, stream)
            if st:
                failed.append(st)
    for _ in range(3):
        threads = [threading.Thread(target=work, args=(j,)) for j in (0, 1)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed
        for *_, want, nwant, got, ngot in jobs:
            assert all(torch.equal(a, b) for a, b in zip(got, (want["dq"], want["dk"], want["dv"])))
            assert torch.equal(ngot[0], nwant["dq"]) and torch.equal(ngot[1], nwant["dq_weight"])


def test_lengths_that_creep_up():
    """Gradients for one prompt length after another: the stream's scratch is replaced by
    larger ones and freed under work in flight, and every result is that of the same call
    in a scratch that stays."""
    s = torch.cuda.Stream()
    gen = torch.Generator(device="cuda").manual_seed(12)
    n = lambda *z: torch.randn(z, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, g = n(1, 3000, 4, 128), n(1, 3000, 4, 128)
    kv = n(1, 3000, 2, 2, 128)
    lengths = range(200, 3000, 56)

    def run(S):
        k, v = kv[:, :S, 0], kv[:, :S, 1]
        out, lse = gdn.cross_attention(q, k, v, return_lse=True)
        return gdn.cross_attention_backward(q, k, v, out, lse, g)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        first = [run(S) for S in lengths]                       # growing
        again = [run(S) for S in reversed(lengths)][::-1]       # in the largest
    torch.cuda.synchronize()
    assert gdn.device_error(s) == _lib.GDN_OK
    for a, b in zip(first, again):
        assert all(torch.equal(a[x], b[x]) for x in a)


def test_threads_on_streams_of_their_own():
    """Three host threads on three streams at once, while a fourth frees what the streams
    hold between calls: every result is that of the call alone."""
    import threading
    gen = torch.Generator(device="cuda").manual_seed(13)
    n = lambda *z: torch.randn(z, generator=gen, device="cuda").bfloat16()  # noqa: E731
    jobs = []
    for Tq, S in ((1500, 140), (2100, 260), (40, 3000)):
        q, k, v, g = n(1, Tq, 4, 64), n(1, S, 2, 64), n(1, S, 2, 64), n(1, Tq, 4, 64)
        out, lse = gdn.cross_attention(q, k, v, return_lse=True)
        jobs.append((q, k, v, g, out, lse, gdn.cross_attention_backward(q, k, v, out, lse, g)))
    torch.cuda.synchronize()
    wrong, done = [], threading.Event()

    def work(q, k, v, g, out, lse, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(100):
                got = gdn.cross_attention_backward(q, k, v, out, lse, g)
                o, _ = gdn.cross_attention(q, k, v, return_lse=True)
                if not torch.equal(o, out) or not all(torch.equal(got[x], want[x]) for x in want):
                    wrong.append(q.shape)

    def release():
        while not done.wait(0.005):
            gdn.workspace_release()
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    other = threading.Thread(target=release)
    for t in (*threads, other):
        t.start()
    for t in threads:
        t.join()
    done.set()
    other.join()
    torch.cuda.synchronize()
    assert not wrong and gdn.device_error() == _lib.GDN_OK


SLOW_ENTRIES = r"""
#include <unistd.h>
#define SLOW(name) int name() { usleep(300000); return 0; }
SLOW(gdn_rope) SLOW(gdn_qk_norm_rope) SLOW(gdn_qk_norm_rope_backward) SLOW(gdn_cross_attention)
SLOW(gdn_cross_attention_backward)
"""


def test_other_threads_run_while_a_call_waits(tmp_path):
    """The binding connected to entries that take 0.3 s, as one does that waits for its
    stream: another thread's Python goes on meanwhile."""
    import ctypes
    import subprocess
    import threading
    import time
    (tmp_path / "slow.c").write_text(SLOW_ENTRIES)
    so = str(tmp_path / "slow.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", so, str(tmp_path / "slow.c")], check=True)
    slow, lib, bind = ctypes.CDLL(so), _lib.load(), _lib.bind()
    at = lambda x: {n: ctypes.cast(getattr(x, n), ctypes.c_void_p).value for n in _lib._BOUND}  # noqa: E731
    q = torch.zeros(1, 4, 2, 32, dtype=torch.bfloat16, device="cuda")
    pos, (freq, _) = torch.arange(4, device="cuda"), gdn.rope_frequencies(32)
    lse = torch.zeros(1, 2, 4, device="cuda")
    calls = [lambda: gdn.rope(q, q, pos, freq), lambda: gdn.qk_norm_rope(q, q),
             lambda: gdn.qk_norm_rope_backward(q, q, None, None, q, q), lambda: gdn.cross_attention(q, q, q),
             lambda: gdn.cross_attention_backward(q, q, q, q, lse, q)]
    bind.connect(at(slow))
    try:
        for call in calls:
            t = threading.Thread(target=call)
            start = time.monotonic()
            t.start()
            turns = 0
            while time.monotonic() - start < 0.15:
                time.sleep(0.005)
                turns += 1
            assert t.is_alive() and turns >= 3
            t.join()
    finally:
        bind.connect(at(lib))
    torch.cuda.synchronize()
