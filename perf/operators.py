"""What the voxel-token operators are measured on: their cases, their inputs and their plain forms.

A batch of voxelized frames is a ragged sequence of tokens (one per pillar or
voxel, frames concatenated, coordinates (batch, z, y, x)).  Three operators
work on such sequences: per-head normalisation and rotation of queries and keys
by the voxel coordinates, attention inside each frame, and a gated linear
recurrence along each frame.

``run`` computes an operator in plain torch (32-bit arithmetic, rounded once at
the end) or, with ``own`` set, through this package's entry points.  A case
with ``train`` set is a forward pass and its backward pass.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
# Cells of a KITTI-shaped grid at 0.16 m along (z, y, x); one axis is the place in a sequence.
GRID = {1: (131072,), 2: (496, 432), 3: (20, 496, 432)}
EPS = 1e-6


def listed():
    return [
        # The newest token of a streaming decoder: nothing but launch latency.
        {"name": "rope_one", "op": "rope", "T": 1, "H": 8, "Hk": 2, "D": 64, "axes": 1, "dtype": "bf16", "train": False},
        # One KITTI-shaped frame of 3-D voxels, in the voxelizer's own 32-bit type.
        {"name": "rope_frame", "op": "rope", "T": 12345, "H": 4, "Hk": 4, "D": 32, "axes": 3, "dtype": "f32", "train": False},
        # A training batch of pillars: rotation by (y, x), forward and backward.
        {"name": "rope_batch_train", "op": "rope", "T": 96001, "H": 8, "Hk": 8, "D": 64, "axes": 2, "dtype": "bf16",
         "train": True},
        # One query in each of eight streams, each over its own long cache of keys and values, shared heads.
        {"name": "attn_one", "op": "attn", "frames": 8, "Lq": 1, "Lk": 20001, "H": 16, "Hk": 2, "D": 128, "axes": 0,
         "cap": 0.0, "causal": False, "prefix": 0, "empty": False, "dtype": "bf16", "train": False},
        # A detector's object queries over the pillars of four ragged frames, nearer pillars preferred.
        {"name": "attn_queries", "op": "attn", "frames": 4, "Lq": 200, "Lk": 16000, "H": 8, "Hk": 8, "D": 32, "axes": 2,
         "cap": 0.0, "causal": False, "prefix": 0, "empty": False, "dtype": "f16", "train": False},
        # The tiny cloud's pillars, capped scores.
        {"name": "attn_tiny", "op": "attn", "frames": 1, "Lq": 4071, "Lk": 4071, "H": 4, "Hk": 4, "D": 32, "axes": 0,
         "cap": 30.0, "causal": False, "prefix": 0, "empty": False, "dtype": "f16", "train": False},
        # A batch of eight ragged frames of pillars attending inside each frame, nearer pillars preferred.
        {"name": "attn_frames", "op": "attn", "frames": 8, "Lq": 6000, "Lk": 6000, "H": 8, "Hk": 8, "D": 64, "axes": 2,
         "cap": 0.0, "causal": False, "prefix": 0, "empty": False, "dtype": "bf16", "train": False},
        # One long frame generated token by token after a visible prefix, shared heads.
        {"name": "attn_long", "op": "attn", "frames": 1, "Lq": 24571, "Lk": 24571, "H": 8, "Hk": 2, "D": 128, "axes": 0,
         "cap": 0.0, "causal": True, "prefix": 1000, "empty": False, "dtype": "bf16", "train": False},
        # A training step on four ragged frames of pillars.
        {"name": "attn_frames_train", "op": "attn", "frames": 4, "Lq": 4000, "Lk": 4000, "H": 8, "Hk": 8, "D": 64,
         "axes": 2, "cap": 0.0, "causal": False, "prefix": 0, "empty": False, "dtype": "bf16", "train": True},
        # A training step on one long causal sequence, shared heads, capped scores.
        {"name": "attn_long_train", "op": "attn", "frames": 1, "Lq": 12289, "Lk": 12289, "H": 8, "Hk": 2, "D": 128,
         "axes": 0, "cap": 30.0, "causal": True, "prefix": 0, "empty": False, "dtype": "f16", "train": True},
        # One KITTI-shaped frame read from its last token to its first, in 32 bits.
        {"name": "scan_frame", "op": "scan", "frames": 1, "L": 12345, "C": 128, "reverse": True, "empty": False,
         "dtype": "f32", "train": False},
        # A training batch of 32 ragged frames.
        {"name": "scan_frames_train", "op": "scan", "frames": 32, "L": 9000, "C": 512, "reverse": False, "empty": False,
         "dtype": "bf16", "train": True},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "scan"])
    train = rng.random() < 0.5
    empty = rng.random() < 0.25
    if op == "rope":
        Hk = rng.choice([1, 2, 4, 8])
        return {"op": op, "T": _spread(rng, 1, 96001), "H": Hk * rng.choice([1, 1, 2, 4]) if Hk <= 2 else Hk, "Hk": Hk,
                "D": rng.choice([32, 48, 64]), "axes": rng.choice([1, 2, 3]), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "train": train}
    if op == "scan":
        frames = rng.choice([1, 2, 5, 8, 32])
        return {"op": op, "frames": frames, "L": _spread(rng, 1, 9000 if frames > 2 else 60000),
                "C": rng.choice([8, 40, 128, 256, 512]), "reverse": rng.random() < 0.5, "empty": empty and frames > 1,
                "dtype": rng.choice(["bf16", "f16", "f32"]), "train": train}
    frames = rng.choice([1, 1, 2, 4, 8])
    Hk = rng.choice([1, 2, 4, 8])
    most = 4000 if frames > 2 else 6000
    Lk = _spread(rng, 1, most)
    Lq = Lk if rng.random() < 0.5 else _spread(rng, 1, most)
    causal = rng.random() < 0.4
    return {"op": op, "frames": frames, "Lq": Lq, "Lk": Lk, "H": min(8, Hk * rng.choice([1, 2, 4])), "Hk": Hk,
            "D": rng.choice([32, 40, 64, 128]), "axes": rng.choice([0, 0, 1, 2, 3]), "cap": rng.choice([0.0, 0.0, 30.0]),
            "causal": causal, "prefix": _spread(rng, 1, 1000) if causal and rng.random() < 0.5 else 0,
            "empty": empty and frames > 1, "dtype": rng.choice(["bf16", "f16"]), "train": train}


def _offsets(frames, longest, empty):
    """Row offsets of ragged frames: the first is the longest, the others 40 % to 100 % of it; with `empty`, the second has none."""
    lens = [longest if b == 0 else max(1, round(longest * (1.0 - 0.6 * ((b * 0.6180339887) % 1.0)))) for b in range(frames)]
    if empty:
        lens[1] = 0
    return [sum(lens[:b]) for b in range(frames + 1)]


def _visible(case):
    """(query, key) pairs that the masks leave, over all frames."""
    qo, ko = (_offsets(case["frames"], case[x], case["empty"]) for x in ("Lq", "Lk"))
    pairs = 0
    for b in range(case["frames"]):
        nq, nk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        if case["causal"]:
            seen = np.clip(np.arange(nq, dtype=np.int64) + 1 + nk - nq, min(case["prefix"], nk), nk)
            pairs += int(np.maximum(seen, 0).sum())
        else:
            pairs += nq * nk
    return pairs


def work(case):
    size = SIZES[case["dtype"]]
    if case["op"] == "rope":
        rows = case["T"] * (case["H"] + case["Hk"])
        fwd = 2 * rows * case["D"] * size + 4 * case["T"] * case["axes"]
        bwd = (3 * rows * case["D"] * size + 4 * case["T"] * case["axes"]) if case["train"] else 0
        return {"bytes": fwd + bwd, "flops": rows * case["D"] * (8 + (22 if case["train"] else 0))}
    if case["op"] == "scan":
        T = _offsets(case["frames"], case["L"], case["empty"])[-1]
        return {"bytes": T * case["C"] * size * (8 if case["train"] else 3), "flops": T * case["C"] * (30 if case["train"] else 8)}
    Tq, Tk = (_offsets(case["frames"], case[x], case["empty"])[-1] for x in ("Lq", "Lk"))
    q, kv = Tq * case["H"] * case["D"] * size, 2 * Tk * case["Hk"] * case["D"] * size
    # Forward: q, k, v in, out out.  Backward: q, k, v, out and its gradient in, three gradients out.
    moved = 2 * q + kv + ((4 * q + 2 * kv) if case["train"] else 0)
    return {"bytes": moved, "flops": _visible(case) * case["H"] * case["D"] * (14 if case["train"] else 4)}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=gen, device=dev) * std + mean).to(dt)

    def cells(rows, axes):
        return torch.stack([torch.randint(0, n, (rows,), generator=gen, device=dev, dtype=torch.int32)
                            for n in GRID[axes]], 1)

    s = dict(case)
    if case["op"] == "rope":
        T, H, Hk, D, A = (case[x] for x in ("T", "H", "Hk", "D", "axes"))
        s["q"], s["k"] = normal(T, H, D, std=2.0), normal(T, Hk, D, std=2.0)
        s["wq"], s["wk"] = (1.0 + 0.1 * torch.randn((D,), generator=gen, device=dev) for _ in range(2))
        s["pos"] = cells(T, A)
        # Pair p turns with axis p mod A, from one turn in 2 pi cells to one in 10,000 times that.
        s["freq"] = torch.tensor([10000.0 ** (-(A * (p // A)) / (D / 2)) for p in range(D // 2)], dtype=torch.float32).to(dev)
        if case["train"]:
            s["dq"], s["dk"] = normal(T, H, D), normal(T, Hk, D)
        return s
    if case["op"] == "scan":
        s["off"] = _offsets(case["frames"], case["L"], case["empty"])
        # The first and the last row of every frame that has one, in the order of reading, and which frames those are.
        some = [b for b in range(case["frames"]) if s["off"][b + 1] > s["off"][b]]
        ends = [s["off"][b + (1 if case["reverse"] else 0)] - (1 if case["reverse"] else 0) for b in some], [
            s["off"][b + (0 if case["reverse"] else 1)] - (0 if case["reverse"] else 1) for b in some]
        s["some"], s["first"], s["last"] = (torch.tensor(i, device=dev) for i in (some, *ends))
        T, C, B = s["off"][-1], case["C"], case["frames"]
        s["x"], s["gate"] = normal(T, C), normal(T, C, std=1.5, mean=-2.0)
        s["h0"] = torch.randn((B, C), generator=gen, device=dev)
        if case["train"]:
            s["dh"] = normal(T, C)
            s["dlast"] = torch.randn((B, C), generator=gen, device=dev)
        return s
    H, Hk, D, A = (case[x] for x in ("H", "Hk", "D", "axes"))
    s["qo"], s["ko"] = (_offsets(case["frames"], case[x], case["empty"]) for x in ("Lq", "Lk"))
    s["qo_dev"], s["ko_dev"] = torch.tensor(s["qo"], device=dev), torch.tensor(s["ko"], device=dev)
    s["q"] = normal(s["qo"][-1], H, D, std=6.0 if case["cap"] else 1.0)
    s["k"], s["v"] = normal(s["ko"][-1], Hk, D), normal(s["ko"][-1], Hk, D)
    s["scale"] = D ** -0.5
    s["slopes"] = s["qpos"] = s["kpos"] = None
    if A:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32).to(dev)
        s["kpos"] = cells(s["ko"][-1], A)
        s["qpos"] = s["kpos"] if s["qo"] == s["ko"] else cells(s["qo"][-1], A)
    if case["train"]:
        s["dout"] = normal(s["qo"][-1], H, D)
    return s


# ---------------------------------------------------------------- plain forms


def _rotate(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _rope_plain(s):
    pair = torch.arange(s["D"] // 2, device=s["q"].device)
    angle = s["pos"][:, pair % s["axes"]].float() * s["freq"]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def forward(x, w):
        x = x.float()
        return _rotate(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w, cos, sin)

    def backward(dy, x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        g = _rotate(dy.float(), cos, -sin)
        n = x * r
        gw = g * w
        return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum((0, 1))

    dt = s["q"].dtype
    out = {"q": forward(s["q"], s["wq"]).to(dt), "k": forward(s["k"], s["wk"]).to(dt)}
    if s["train"]:
        dq, out["dwq"] = backward(s["dq"], s["q"], s["wq"])
        dk, out["dwk"] = backward(s["dk"], s["k"], s["wk"])
        out["dq"], out["dk"] = dq.to(dt), dk.to(dt)
    return out


def _scan_pairs(a, b):
    """h[t] = a[t] * h[t-1] + b[t] from h = 0, by halving: neighbouring steps are joined, the halves solved, the rest filled in."""
    n = a.shape[0]
    if n <= 1:
        return b
    m = n // 2
    odd = _scan_pairs(a[1:2 * m:2] * a[0:2 * m:2], a[1:2 * m:2] * b[0:2 * m:2] + b[1:2 * m:2])
    h = torch.empty_like(b)
    h[1:2 * m:2] = odd
    h[0] = b[0]
    h[2::2] = a[2::2] * odd[: (n - 1) // 2] + b[2::2]
    return h


def _scan_plain(s):
    dt = s["x"].dtype
    x, z = s["x"].float(), torch.sigmoid(s["gate"].float())
    some, first, last = s["some"], s["first"], s["last"]

    def turn(t):
        return t.flip(0) if s["reverse"] else t

    a, b = 1.0 - z, z * x
    b[first] += a[first] * s["h0"][some]
    a0 = a.clone()
    a0[first] = 0.0
    h = turn(_scan_pairs(turn(a0), turn(b)))
    end = s["h0"].clone()
    end[some] = h[last]
    out = {"h": h.to(dt), "last": end}
    if s["train"]:
        g = s["dh"].float()
        g[last] += s["dlast"][some]
        # The state's gradient runs the other way: e[t] = g[t] + a[t+1] * e[t+1], in the order of reading.
        nxt = torch.roll(turn(a0), -1, 0)
        e = turn(_scan_pairs(nxt.flip(0), turn(g).flip(0)).flip(0))
        before = turn(torch.roll(turn(h), 1, 0))
        before[first] = s["h0"][some]
        out["dx"] = (e * z).to(dt)
        out["dgate"] = (e * (x - before) * z * (1.0 - z)).to(dt)
        dh0 = s["dlast"].clone()
        dh0[some] = (e * a)[first]
        out["dh0"] = dh0
    return out


def _attn_plain(s):
    B, H, Hk, D, dt = s["frames"], s["H"], s["Hk"], s["D"], s["q"].dtype
    G = H // Hk
    Lq, Lk = (max(o[b + 1] - o[b] for b in range(B)) for o in (s["qo"], s["ko"]))
    dev = s["q"].device
    iq, ik = torch.arange(Lq, device=dev), torch.arange(Lk, device=dev)
    nq, nk = ((o[1:] - o[:-1])[:, None] for o in (s["qo_dev"], s["ko_dev"]))
    okq, okk = iq < nq, ik < nk
    rowq = torch.where(okq, s["qo_dev"][:-1, None] + iq, 0)
    rowk = torch.where(okk, s["ko_dev"][:-1, None] + ik, 0)

    def queries(t):  # [Tq, H, D] -> [B, Hk, G, Lq, D], rows past a frame's end zero
        t = torch.where(okq[:, :, None, None], t[rowq].float(), 0.0)
        return t.view(B, Lq, Hk, G, D).permute(0, 2, 3, 1, 4)

    def keys(t):
        t = torch.where(okk[:, :, None, None], t[rowk].float(), 0.0)
        return t.permute(0, 2, 1, 3)[:, :, None]

    def packed(t, off, rows):  # [B, L, ...] -> [rows, ...]
        row = torch.arange(rows, device=dev)
        frame = torch.bucketize(row, off[1:], right=True)
        return t[frame, row - off[frame]].to(dt)

    def back_q(t):
        return packed(t.permute(0, 3, 1, 2, 4).reshape(B, Lq, H, D), s["qo_dev"], s["q"].shape[0])

    def back_k(t):
        return packed(t.permute(0, 2, 1, 3), s["ko_dev"], s["k"].shape[0])

    q, k, v = queries(s["q"]), keys(s["k"]), keys(s["v"])
    c = torch.matmul(q * s["scale"], k.transpose(-1, -2))
    if s["cap"]:
        c = torch.tanh(c.div_(s["cap"]))
        p = c * s["cap"]
    else:
        p = c
    if s["slopes"] is not None:
        gap = (s["qpos"][rowq].float()[:, :, None] - s["kpos"][rowk].float()[:, None]).abs().sum(-1)
        p = p - s["slopes"].view(1, Hk, G, 1, 1) * gap[:, None, None]
    seen = okq[:, :, None] & okk[:, None]
    if s["causal"]:
        seen = seen & ((ik <= iq[:, None] + (nk - nq)[:, :, None]) | (ik < s["prefix"]))
    p = p.masked_fill(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True).clamp_min(-1e30)
    p = (p - top).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp_min(1e-30))
    o = torch.matmul(p, v)
    out = {"out": back_q(o)}
    if s["train"]:
        do = queries(s["dout"])
        out["dv"] = back_k(torch.matmul(p.transpose(-1, -2), do).sum(2))
        ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        if s["cap"]:
            ds = ds.mul_(1.0 - c * c)
        out["dq"] = back_q(torch.matmul(ds, k) * s["scale"])
        out["dk"] = back_k(torch.matmul(ds.transpose(-1, -2), q * s["scale"]).sum(2))
    return out


# ------------------------------------------------------------------- own calls


def _run_own(s):
    import lidar_point_cloud_gb300 as pv

    if s["op"] == "rope":
        q, k = pv.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], EPS)
        out = {"q": q, "k": k}
        if s["train"]:
            dq, dk, out["dwq"], out["dwk"] = pv.qk_norm_rope_backward(
                s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], EPS)
            out["dq"], out["dk"] = dq, dk
        return out
    if s["op"] == "scan":
        if not s["train"]:
            h, last = pv.gated_scan(s["x"], s["gate"], s["off"], s["h0"], reverse=s["reverse"])
            return {"h": h, "last": last}
        h, last, states = pv.gated_scan(s["x"], s["gate"], s["off"], s["h0"], reverse=s["reverse"], return_states=True)
        dx, dgate, dh0 = pv.gated_scan_backward(s["dh"], s["dlast"], s["x"], s["gate"], states, s["off"],
                                                reverse=s["reverse"])
        return {"h": h, "last": last, "dx": dx, "dgate": dgate, "dh0": dh0}
    how = dict(scale=s["scale"], cap=s["cap"], slopes=s["slopes"], q_positions=s["qpos"], k_positions=s["kpos"],
               causal=s["causal"], prefix=[s["prefix"]] * s["frames"] if s["prefix"] else None)
    if not s["train"]:
        return {"out": pv.attention(s["q"], s["k"], s["v"], s["qo"], s["ko"], **how)}
    o, lse = pv.attention(s["q"], s["k"], s["v"], s["qo"], s["ko"], return_lse=True, **how)
    dq, dk, dv = pv.attention_backward(s["dout"], s["q"], s["k"], s["v"], o, lse, s["qo"], s["ko"], **how)
    return {"out": o, "dv": dv, "dq": dq, "dk": dk}


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope_plain, "scan": _scan_plain, "attn": _attn_plain}[state["op"]](state)


# -------------------------------------------------------------- 64-bit values


def _rope_exact(s):
    D, A = s["D"], s["axes"]
    half = D // 2
    # The angle is by definition the 32-bit product of a cell and its frequency, as models' tables hold it.
    turn = (s["pos"].float()[:, [p % A for p in range(half)]] * s["freq"]).double()
    spin = torch.polar(torch.ones_like(turn), turn)[:, None]

    def unit(x):
        return x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()

    def forward(x, w):
        y = unit(x.double()) * w.double()
        z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * spin
        return torch.cat([z.real, z.imag], -1)

    def backward(dy, x, w):
        x, dy = x.double(), dy.double()
        z = torch.complex(dy[..., :half].contiguous(), dy[..., half:].contiguous()) * spin.conj()
        g = torch.cat([z.real, z.imag], -1)
        m = x.pow(2).sum(-1, keepdim=True) / D + EPS
        gw = g * w.double()
        dx = gw / m.sqrt() - x * (gw * x).sum(-1, keepdim=True) / (D * m.pow(1.5))
        return dx, (g * x / m.sqrt()).sum(0).sum(0)

    out = {"q": forward(s["q"], s["wq"]), "k": forward(s["k"], s["wk"])}
    if s["train"]:
        dq, out["dwq"] = backward(s["dq"], s["q"], s["wq"])
        dk, out["dwk"] = backward(s["dk"], s["k"], s["wk"])
        out["dq"], out["dk"] = dq, dk
    return out


def _scan_exact(s):
    x, gate, h0 = (s[n].double().cpu().numpy() for n in ("x", "gate", "h0"))
    z = 1.0 / (1.0 + np.exp(-gate))
    h, last, before = np.empty_like(x), h0.copy(), np.empty_like(x)
    dx, dgate = np.empty_like(x), np.empty_like(x)
    grads = s["train"]
    dh0 = s["dlast"].double().cpu().numpy() if grads else None
    dh = s["dh"].double().cpu().numpy() if grads else None
    for b in range(s["frames"]):
        steps = range(s["off"][b], s["off"][b + 1])
        steps = steps[::-1] if s["reverse"] else steps
        state = last[b]
        for t in steps:
            before[t] = state
            state = state + z[t] * (x[t] - state)
            h[t] = state
        last[b] = state
        if grads:
            e = dh0[b]
            for t in steps[::-1]:
                e = e + dh[t]
                dx[t] = e * z[t]
                dgate[t] = e * (x[t] - before[t]) * z[t] * (1.0 - z[t])
                e = e * (1.0 - z[t])
            dh0[b] = e
    out = {"h": torch.from_numpy(h), "last": torch.from_numpy(last)}
    if grads:
        out.update(dx=torch.from_numpy(dx), dgate=torch.from_numpy(dgate), dh0=torch.from_numpy(dh0))
    return out


def _attn_exact(s):
    H, Hk = s["H"], s["Hk"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out = torch.zeros_like(q)
    if s["train"]:
        do, dq, dk, dv = s["dout"].double(), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(s["frames"]):
        i0, i1, j0, j1 = s["qo"][b], s["qo"][b + 1], s["ko"][b], s["ko"][b + 1]
        if i1 == i0 or j1 == j0:
            continue
        hide = gap = None
        if s["causal"]:
            i, j = torch.arange(i1 - i0, device=q.device)[:, None], torch.arange(j1 - j0, device=q.device)
            hide = (j - (j1 - j0) > i - (i1 - i0)) & (j >= s["prefix"])
        if s["slopes"] is not None:
            gap = torch.cdist(s["qpos"][i0:i1].double(), s["kpos"][j0:j1].double(), p=1.0)
        for h in range(H):
            g = h * Hk // H
            w = (q[i0:i1, h] @ k[j0:j1, g].T) * s["scale"]
            slope = None
            if s["cap"]:
                w = torch.tanh(w / s["cap"])
                slope = 1.0 - w * w
                w *= s["cap"]
            if gap is not None:
                w -= float(s["slopes"][h]) * gap
            if hide is not None:
                w.masked_fill_(hide, -math.inf)
            w = torch.softmax(w, -1).nan_to_num_(nan=0.0)
            out[i0:i1, h] = w @ v[j0:j1, g]
            if s["train"]:
                dv[j0:j1, g] += w.T @ do[i0:i1, h]
                d = do[i0:i1, h] @ v[j0:j1, g].T
                d -= (do[i0:i1, h] * out[i0:i1, h]).sum(-1, keepdim=True)
                d *= w
                d *= s["scale"]
                if slope is not None:
                    d *= slope
                dq[i0:i1, h] = d @ k[j0:j1, g]
                dk[j0:j1, g] += d.T @ q[i0:i1, h]
    return {"out": out, "dv": dv, "dq": dq, "dk": dk} if s["train"] else {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope_exact, "scan": _scan_exact, "attn": _attn_exact}[case["op"]](s)
