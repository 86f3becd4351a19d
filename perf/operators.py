"""The softmax blocks' operators around the attention, as cases to measure.

A softmax block of the hybrid diffusion Transformer normalises its queries and
keys per head, rotates them by their positions, attends to the streaming cache,
and then attends to the encoder's states (the prompt's, or the source clip's).
Four operators and their gradients:

  rope          rotary positions of queries and keys, no norm
  norm_rope     RMS norm per head and rotary positions in one pass
  norm_rope_bwd its gradients: inputs and norm weights
  cross         softmax attention of queries over an encoder's states of
                another length, some of them masked
  cross_train   the same with its gradients, as a training step makes them

``run`` computes them from elementary torch operations, or, where ``own`` is
true, with the package's calls.  Sizes are the streaming chunk's (2640 tokens
of 20 heads, 112 wide), the stress sweep's (16 heads, 64 and 128 wide, up to
65536 tokens) and generic ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # eight interactive streams, one token each, far into a long context:
        # half of each head rotates, frequencies stretched; latency counts
        {"name": "rope_token", "op": "rope", "B": 8, "T": 1, "Hq": 16, "Hk": 4, "D": 64, "R": 32,
         "dtype": "bf16", "layout": "interleaved", "axes": 1, "packed": False, "stretch": 8.0},
        # the longest stress length in fp32, whole heads, no norm
        {"name": "rope_long_f32", "op": "rope", "B": 1, "T": 65536, "Hq": 16, "Hk": 4, "D": 128, "R": 128,
         "dtype": "f32", "layout": "half", "axes": 1, "packed": False, "stretch": 1.0},
        # one token of the block: the smallest call
        {"name": "norm_rope_token", "op": "norm_rope", "B": 1, "T": 1, "Hq": 20, "Hk": 20, "D": 112, "R": 112,
         "dtype": "bf16", "layout": "half", "axes": 3, "packed": True, "stretch": 1.0},
        # the streaming chunk: frame, row and column positions, q and k views of the packed projection
        {"name": "norm_rope_chunk", "op": "norm_rope", "B": 1, "T": 2640, "Hq": 20, "Hk": 20, "D": 112, "R": 112,
         "dtype": "bf16", "layout": "half", "axes": 3, "packed": True, "stretch": 1.0},
        # the chunk's gradients
        {"name": "norm_rope_bwd_chunk", "op": "norm_rope_bwd", "B": 1, "T": 2640, "Hq": 20, "Hk": 20, "D": 112,
         "R": 112, "dtype": "bf16", "layout": "half", "axes": 3, "packed": True, "stretch": 1.0},
        # gradients of a training batch with fewer key heads and neighbouring pairs
        {"name": "norm_rope_bwd_batch", "op": "norm_rope_bwd", "B": 4, "T": 4096, "Hq": 16, "Hk": 4, "D": 128,
         "R": 64, "dtype": "bf16", "layout": "interleaved", "axes": 1, "packed": False, "stretch": 1.0},
        # one query of eight requests over long encoder states, key heads shared by four
        {"name": "cross_token", "op": "cross", "B": 8, "Tq": 1, "S": 4096, "Hk": 4, "G": 4, "D": 128, "mask": "tail"},
        # odd lengths, shared heads, scattered holes in the mask, and a row with no state at all
        {"name": "cross_ragged", "op": "cross", "B": 5, "Tq": 333, "S": 77, "Hk": 4, "G": 3, "D": 80,
         "mask": "holes"},
        # the streaming chunk over a prompt of 300 states, the last quarter padding
        {"name": "cross_chunk", "op": "cross", "B": 1, "Tq": 2640, "S": 300, "Hk": 20, "G": 1, "D": 112,
         "mask": "tail"},
        # the streaming chunk over the states of a source clip of three chunks
        {"name": "cross_source", "op": "cross", "B": 1, "Tq": 2640, "S": 7920, "Hk": 20, "G": 1, "D": 112,
         "mask": "none"},
        # a training step of the chunk over its prompt
        {"name": "cross_train_chunk", "op": "cross_train", "B": 1, "Tq": 2640, "S": 300, "Hk": 20, "G": 1,
         "D": 112, "mask": "tail"},
        # a training step of long odd lengths with shared key heads
        {"name": "cross_train_batch", "op": "cross_train", "B": 2, "Tq": 4095, "S": 2641, "Hk": 4, "G": 4,
         "D": 128, "mask": "tail"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "norm_rope_bwd", "cross", "cross_train"])
    D = 16 * rng.randint(1, 8)
    if op in ("rope", "norm_rope", "norm_rope_bwd"):
        B, G, Hk = rng.randint(1, 8), rng.choice([1, 1, 2, 3, 4]), rng.randint(1, 8)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        moved = (3 if op == "norm_rope_bwd" else 2) * SIZE[dtype] * B * (G + 1) * Hk * D
        T = _log_int(rng, 1, max(1, min(65536, int(1.0e9 / moved))))
        return {"op": op, "B": B, "T": T, "Hq": G * Hk, "Hk": Hk, "D": D, "R": 16 * rng.randint(1, D // 16),
                "dtype": dtype, "layout": rng.choice(["half", "interleaved"]), "axes": rng.choice([1, 3]),
                "packed": rng.random() < 0.5, "stretch": rng.choice([1.0, 4.0, 16.0])}
    B, G, Hk = rng.randint(1, 8), rng.choice([1, 1, 2, 3, 4, 8]), rng.randint(1, 8)
    Tq = _log_int(rng, 1, 4096)
    # products of at most about 1.5e11 operations forward, and 2.5 GB of 32-bit scores
    most = min(1.5e11 / (4.0 * B * G * Hk * Tq * D), 6.0e8 / (B * G * Hk * Tq))
    S = _log_int(rng, 1, int(max(1, min(8192, most))))
    return {"op": op, "B": B, "Tq": Tq, "S": S, "Hk": Hk, "G": G, "D": D,
            "mask": rng.choice(["none", "tail", "holes"])}


def _kept(case):
    """States that the mask keeps, over all batch rows (expected, for holes)."""
    B, S = case["B"], case["S"]
    if case["mask"] == "none":
        return B * S
    if case["mask"] == "tail":
        return sum(_tail(B, S, b) for b in range(B))
    return 0.75 * S * (B - 1 if B > 1 else 1)


def _tail(B, S, b):
    """Valid states of batch row b: three quarters to all of them."""
    return S - (b + 1) * S // (4 * B)


def work(case):
    D = case["D"]
    if case["op"] in ("rope", "norm_rope", "norm_rope_bwd"):
        rows = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        back = case["op"] == "norm_rope_bwd"
        per = {"rope": 3 * case["R"], "norm_rope": 4 * D + 3 * case["R"],
               "norm_rope_bwd": 12 * D + 3 * case["R"]}[case["op"]]
        return {"bytes": rows * D * SIZE[case["dtype"]] * (3 if back else 2)
                + case["B"] * case["T"] * case["axes"] * 8 + 4 * case["R"], "flops": rows * per}
    Hq, rows = case["G"] * case["Hk"], case["B"] * case["Tq"] * case["G"] * case["Hk"]
    kv, kept = 2 * case["Hk"] * D * 2, _kept(case)
    product = 2.0 * Hq * case["Tq"] * kept * D
    masks = 0 if case["mask"] == "none" else case["B"] * case["S"]
    forward = 2 * rows * D * 2 + kept * kv + masks
    if case["op"] == "cross":
        return {"bytes": forward, "flops": 2 * product}
    # out and lse, then d_out in, dq, dk and dv out; seven products: two forward, five back
    return {"bytes": forward + 4 * rows + 2 * rows * D * 2 + case["B"] * case["S"] * kv, "flops": 7 * product}


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    B, D = case["B"], case["D"]
    state = dict(case)
    if case["op"] in ("rope", "norm_rope", "norm_rope_bwd"):
        T, Hq, Hk, R = case["T"], case["Hq"], case["Hk"], case["R"]
        dt = DTYPES[case["dtype"]]
        if case["packed"]:  # views of the projection's one output, its values behind them
            qkv = normal(B, T, Hq + 2 * Hk, D, dtype=dt)
            state["q"], state["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        else:
            state["q"], state["k"] = normal(B, T, Hq, D, dtype=dt), normal(B, T, Hk, D, dtype=dt)
        t = torch.arange(T, device="cuda")
        first = torch.randint(0, 1000000 if case["axes"] == 1 else 1000, (B, 1), generator=gen, device="cuda")
        if case["axes"] == 1:
            state["positions"] = (first + t)[:, :, None]
        else:  # frame, row and column of a 40 x 22 latent frame
            frame = first + torch.div(t, 880, rounding_mode="floor")
            row = torch.div(t, 22, rounding_mode="floor").remainder(40).expand(B, T)
            state["positions"] = torch.stack([frame, row, t.remainder(22).expand(B, T)], -1).contiguous()
        pairs = R // 2
        side = pairs // 3
        state["sections"] = (pairs,) if case["axes"] == 1 else (pairs - 2 * side, side, side)
        state["inv_freq"] = torch.cat([
            10000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / max(n, 1))
            for n in state["sections"]]) / case["stretch"]
        state["axis"] = torch.cat([torch.full((n,), i, device="cuda") for i, n in enumerate(state["sections"])])
        state["amplitude"] = 1.0 + 0.1 * math.log(case["stretch"])
        if case["op"] != "rope":
            state["q_weight"] = 1.0 + 0.2 * normal(D)
            state["k_weight"] = 1.0 + 0.2 * normal(D)
        if case["op"] == "norm_rope_bwd":
            state["dq_out"], state["dk_out"] = normal(B, T, Hq, D, dtype=dt), normal(B, T, Hk, D, dtype=dt)
        return state
    Tq, S, Hk, Hq = case["Tq"], case["S"], case["Hk"], case["G"] * case["Hk"]
    state["q"] = normal(B, Tq, Hq, D, dtype=torch.bfloat16)
    kv = normal(B, S, 2, Hk, D, dtype=torch.bfloat16)  # the encoder side's one projection
    state["k"], state["v"] = kv[:, :, 0], kv[:, :, 1]
    state["key_mask"] = None
    if case["mask"] == "tail":
        lengths = torch.tensor([_tail(B, S, b) for b in range(B)], device="cuda")
        state["key_mask"] = torch.arange(S, device="cuda")[None] < lengths[:, None]
    elif case["mask"] == "holes":  # a quarter of the states dropped; the last of several rows keeps none
        keep = torch.rand((B, S), generator=gen, device="cuda") < 0.75
        if B > 1:
            keep[-1] = False
        state["key_mask"] = keep
    if case["op"] == "cross_train":
        state["d_out"] = normal(B, Tq, Hq, D, dtype=torch.bfloat16)
    return state


# -------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import gated_deltanet_linear_chunked_b200 as gdn
    op = state["op"]
    if op in ("rope", "norm_rope", "norm_rope_bwd"):
        turn = {"sections": state["sections"], "layout": state["layout"], "amplitude": state["amplitude"]}
        at = (state["positions"], state["inv_freq"])
        if op == "rope":
            return gdn.rope(state["q"], state["k"], *at, **turn)
        weights = (state["q_weight"], state["k_weight"])
        if op == "norm_rope":
            return gdn.qk_norm_rope(state["q"], state["k"], *weights, *at, eps=EPS, **turn)
        return gdn.qk_norm_rope_backward(state["q"], state["k"], *weights, state["dq_out"], state["dk_out"],
                                         *at, eps=EPS, **turn)
    if op == "cross":
        return gdn.cross_attention(state["q"], state["k"], state["v"], state["key_mask"])
    out, lse = gdn.cross_attention(state["q"], state["k"], state["v"], state["key_mask"], return_lse=True)
    grads = gdn.cross_attention_backward(state["q"], state["k"], state["v"], out, lse, state["d_out"],
                                         state["key_mask"])
    return {"out": out, "lse": lse, **grads}


def _run_plain(state):
    op = state["op"]
    if op == "rope":
        cos, sin = _angles(state)
        return (_rotate(state["q"].float(), cos, sin, state["layout"]).to(state["q"].dtype),
                _rotate(state["k"].float(), cos, sin, state["layout"]).to(state["k"].dtype))
    if op == "norm_rope":
        cos, sin = _angles(state)
        return (_norm_rotate(state["q"], state["q_weight"], cos, sin, state["layout"]),
                _norm_rotate(state["k"], state["k_weight"], cos, sin, state["layout"]))
    if op == "norm_rope_bwd":
        cos, sin = _angles(state)
        dq, dqw = _norm_rotate_back(state["q"], state["q_weight"], state["dq_out"], cos, sin, state["layout"])
        dk, dkw = _norm_rotate_back(state["k"], state["k_weight"], state["dk_out"], cos, sin, state["layout"])
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    return _cross_plain(state)


def _angles(state):
    """cos and sin of position x frequency, [B, T, 1, R/2]: 64 bits up to them."""
    angle = state["positions"].double()[:, :, state["axis"]] * state["inv_freq"]
    scale = state["amplitude"]
    return (angle.cos() * scale).float()[:, :, None], (angle.sin() * scale).float()[:, :, None]


def _rotate(x, cos, sin, layout):
    R = 2 * cos.shape[-1]
    head, rest = x[..., :R], x[..., R:]
    if layout == "half":
        a, b = head[..., :R // 2], head[..., R // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)


def _norm_rotate(x, weight, cos, sin, layout):
    f = x.float()
    f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * weight
    return _rotate(f, cos, sin, layout).to(x.dtype)


def _norm_rotate_back(x, weight, dy, cos, sin, layout):
    f, g = x.float(), _rotate(dy.float(), cos, -sin, layout)
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    hat, gw = f * r, g * weight
    dx = r * (gw - hat * (gw * hat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * hat).sum((0, 1, 2), dtype=torch.float64).float()


def _cross_plain(state):
    G, D = state["G"], state["D"]
    q, k, v = (state[n].float().transpose(1, 2) for n in ("q", "k", "v"))  # [B, H, rows, D]
    B, Hq, Tq, _ = q.shape
    scale = 1.0 / math.sqrt(D)
    q = q.reshape(B, Hq // G, G * Tq, D)  # the query heads of one key head, stacked
    s = (q @ k.transpose(2, 3)).mul_(scale)
    if state["key_mask"] is not None:
        s.masked_fill_(~state["key_mask"][:, None, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)  # a row that sees nothing
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = p @ v

    def back(x, H, T, dtype=torch.bfloat16):
        return x.reshape(B, H, T, -1).transpose(1, 2).to(dtype).contiguous()

    if state["op"] == "cross":
        return back(o, Hq, Tq)
    lse = (top + total.log()).reshape(B, Hq, Tq)
    do = state["d_out"].float().transpose(1, 2).reshape(B, Hq // G, G * Tq, D)
    ds = do @ v.transpose(2, 3)
    ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    S = k.shape[2]
    return {"out": back(o, Hq, Tq), "lse": lse, "dq": back((ds @ k).mul_(scale), Hq, Tq),
            "dk": back((ds.transpose(2, 3) @ q).mul_(scale), Hq // G, S),
            "dv": back(p.transpose(2, 3) @ do, Hq // G, S)}


# --------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "norm_rope", "norm_rope_bwd"):
        return _exact_rope(s)
    return _exact_cross(s)


def _turned(x, s):
    """The first R values of each head as complex numbers times amplitude e^(i angle)."""
    R, out = s["R"], x.clone()
    first, angles = 0, []
    for axis, n in enumerate(s["sections"]):
        angles.append(s["positions"][:, :, None, axis, None].double() * s["inv_freq"][first:first + n])
        first += n
    angle = torch.cat(angles, -1)
    turn = s["amplitude"] * torch.complex(torch.cos(angle), torch.sin(angle))
    even = slice(0, R // 2) if s["layout"] == "half" else slice(0, R, 2)
    odd = slice(R // 2, R) if s["layout"] == "half" else slice(1, R, 2)
    z = torch.complex(x[..., even], x[..., odd]) * turn
    out[..., even], out[..., odd] = z.real, z.imag
    return out


def _exact_rope(s):
    def forward(x, w):
        if w is not None:
            x = w * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        return _turned(x, s)

    if s["op"] != "norm_rope_bwd":
        return tuple(forward(s[n].double(), s[n + "_weight"].double() if s["op"] == "norm_rope" else None)
                     for n in ("q", "k"))
    got = {}
    for n in ("q", "k"):
        x = s[n].double().requires_grad_()
        w = s[n + "_weight"].double().requires_grad_()
        got["d" + n], got["d%s_weight" % n] = torch.autograd.grad(forward(x, w), (x, w),
                                                                   s["d%s_out" % n].double())
    return got


def _exact_cross(s):
    """One batch row and key head after another, its gradients by autograd."""
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    B, Tq, Hq, D = q.shape
    G, train = s["G"], s["op"] == "cross_train"
    out, lse = torch.zeros_like(q), q.new_full((B, Hq, Tq), -math.inf)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        seen = torch.arange(k.shape[1], device="cuda")
        seen = seen if s["key_mask"] is None else seen[s["key_mask"][b]]
        if not len(seen):
            continue
        for h in range(Hq // G):
            heads = slice(h * G, (h + 1) * G)
            qh, kh, vh = (x.clone().requires_grad_(train)
                          for x in (q[b, :, heads], k[b, seen, h], v[b, seen, h]))
            scores = torch.einsum("tgd,sd->gts", qh, kh) / D ** 0.5
            row = torch.logsumexp(scores, -1)
            o = torch.einsum("gts,sd->tgd", torch.exp(scores - row[..., None]), vh)
            out[b, :, heads], lse[b, heads] = o.detach(), row.detach()
            if train:
                g = torch.autograd.grad(o, (qh, kh, vh), s["d_out"][b, :, heads].double())
                dq[b, :, heads], dk[b, seen, h], dv[b, seen, h] = g
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else out
