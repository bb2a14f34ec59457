"""64-bit implementations of the token operators, and error bounds that follow
from where the library rounds.

Each function returns values and, beside them, the sums of magnitudes that
their rounding errors scale with.  With u half a unit in the last place of the
storage type (relative), an output is rounded once (u |value|), and inside
attention the probabilities and the scores' gradients are rounded to the
storage type before their products (u times the sum of magnitudes); 32-bit
sums add some 2^-23 of the same magnitudes, which the factors of two below
leave room for.
"""

from __future__ import annotations

import math

import torch

UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12, torch.float64: 0.0}


def within(got, want, slack, name):
    """|got - want| <= slack everywhere, and nothing that is not finite."""
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got.double()).all(), f"{name}: not finite"
    bad = (got.double() - want).abs() - slack
    assert got.numel() == 0 or bad.max().item() <= 0, (
        f"{name}: off by {(got.double() - want).abs().max().item():.3e}, over the bound by {bad.max().item():.3e}")


# ------------------------------------------------------------------- rotation


def turn(x, pos, freq, back=False):
    D = x.shape[-1]
    axis = torch.arange(D // 2, device=x.device) % pos.shape[1]
    angle = (pos.float()[:, axis] * freq).double()[:, None]  # by definition the 32-bit product
    c, s = angle.cos(), -angle.sin() if back else angle.sin()
    a, b = x[..., : D // 2], x[..., D // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def rope(x, w, pos, freq, eps):
    x, w = x.double(), w.double()
    n = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    y = turn(n * w, pos, freq)
    mag = (n * w).abs()
    D = x.shape[-1]
    pair = mag[..., : D // 2] + mag[..., D // 2:]
    return y, torch.cat([pair, pair], -1)


def rope_backward(dy, x, w, pos, freq, eps):
    x, w = x.double(), w.double()
    r = 1.0 / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    n = x * r
    g = turn(dy.double(), pos, freq, back=True)
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    mag = r * ((g * w).abs() + n.abs() * (g * w * n).abs().mean(-1, keepdim=True))
    D = x.shape[-1]
    gm = dy.double().abs()
    gm = gm[..., : D // 2] + gm[..., D // 2:]
    gm = torch.cat([gm, gm], -1)
    mag = mag + r * (gm * w.abs() + n.abs() * (gm * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, mag, (g * n).sum((0, 1)), (gm * n.abs()).sum((0, 1))


# ------------------------------------------------------------------ attention


def attention(q, k, v, qo, ko, scale, cap=0.0, slopes=None, qpos=None, kpos=None, causal=False, prefix=None, dout=None):
    """(out, lse, their magnitudes) and, with dout, the gradients and theirs."""
    unit = UNIT[q.dtype]
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    r = {"out": torch.zeros_like(q), "lse": torch.full((H, q.shape[0]), -math.inf, dtype=torch.float64, device=q.device)}
    names = ["out"]
    if dout is not None:
        dout = dout.double()
        r.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
        names += ["dq", "dk", "dv"]
    slack = {n: torch.zeros_like(r[n]) for n in names}
    for b in range(len(qo) - 1):
        i, j = slice(qo[b], qo[b + 1]), slice(ko[b], ko[b + 1])
        nq, nk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        if not nq or not nk:
            continue
        seen = torch.ones((nq, nk), dtype=torch.bool, device=q.device)
        if causal:
            x, y = torch.arange(nq, device=q.device)[:, None], torch.arange(nk, device=q.device)
            seen = (y <= x + nk - nq) | (y < (prefix[b] if prefix else 0))
        for h in range(H):
            g = h // G
            s = scale * q[i, h] @ k[j, g].T
            steep = torch.ones_like(s)
            if cap:
                t = torch.tanh(s / cap)
                steep, s = 1 - t * t, cap * t
            bias = 0.0
            if slopes is not None:
                bias = slopes[h].double() * (qpos[i].double()[:, None] - kpos[j].double()[None]).abs().sum(-1)
                s = s - bias
            # 32-bit scores: some 2^-22 of the sum of their terms' magnitudes.
            noise = 2.0 ** -22 * (scale * q[i, h].abs() @ k[j, g].abs().T + bias + 1.0)
            s = s.masked_fill(~seen, -math.inf)
            top = s.amax(-1, keepdim=True)
            top = top.masked_fill(top == -math.inf, 0.0)
            p = (s - top).exp()
            total = p.sum(-1, keepdim=True)
            lse = torch.where(total > 0, top + total.log(), -math.inf)
            r["lse"][h, i] = lse[:, 0]
            p = torch.where(seen, p / total.clamp_min(1e-300), 0.0)
            noise = torch.where(seen, noise, 0.0).amax(-1, keepdim=True)
            o = p @ v[j, g]
            r["out"][i, h] = o
            # Probabilities in the storage type: relative unit, and 2^-25 of the row's
            # largest where float16 runs out of exponent.
            pe = p * (2 * unit + 2 * noise) + (2.0 ** -24) * p.amax(-1, keepdim=True) * seen
            slack["out"][i, h] = pe @ v[j, g].abs() + 2 * unit * o.abs()
            if dout is None:
                continue
            do = dout[i, h]
            delta = (do * o).sum(-1, keepdim=True)
            dp = do @ v[j, g].T
            ds = p * (dp - delta) * steep * scale
            # The library's delta comes from the rounded out; each ds is rounded once.
            dde = (do.abs() * slack["out"][i, h]).sum(-1, keepdim=True) + 2.0 ** -22 * (do.abs() * o.abs()).sum(-1, keepdim=True)
            dpe = 2.0 ** -22 * do.abs() @ v[j, g].abs().T
            dse = scale * (p * steep * (dde + dpe) + pe * ((dp - delta).abs() + dde)) + 2 * unit * ds.abs()
            dse = dse + scale * p * (dp - delta).abs() * 2 * noise * (2.0 / cap if cap else 0.0)
            r["dq"][i, h] += ds @ k[j, g]
            slack["dq"][i, h] += dse @ k[j, g].abs()
            r["dk"][j, g] += ds.T @ q[i, h]
            slack["dk"][j, g] += dse.T @ q[i, h].abs()
            r["dv"][j, g] += p.T @ do
            slack["dv"][j, g] += pe.T @ do.abs()
    for n in names[1:]:
        slack[n] += 2 * unit * r[n].abs()
    # What float16 holds below its normal range, once per rounding.
    for n in names:
        slack[n] += 2.0 ** -24
    return r, slack


# ------------------------------------------------------------------ recurrence


def scan(x, gate, off, h0=None, reverse=False, dh=None, dlast=None):
    x, gate = x.double().cpu(), gate.double().cpu()
    B, C = len(off) - 1, x.shape[1]
    z = torch.sigmoid(gate)
    last = torch.zeros((B, C), dtype=torch.float64) if h0 is None else h0.double().cpu().clone()
    h, before = torch.empty_like(x), torch.empty_like(x)
    r = {"h": h, "last": last}
    if dh is not None:
        dh = dh.double().cpu()
        e_end = torch.zeros((B, C), dtype=torch.float64) if dlast is None else dlast.double().cpu().clone()
        r.update(dx=torch.empty_like(x), dgate=torch.empty_like(x), dh0=e_end)
    for b in range(B):
        steps = list(range(off[b], off[b + 1]))
        if reverse:
            steps.reverse()
        for t in steps:
            before[t] = last[b]
            last[b] = (1 - z[t]) * last[b] + z[t] * x[t]
            h[t] = last[b]
        if dh is not None:
            for t in reversed(steps):
                e = e_end[b] + dh[t]
                r["dx"][t] = e * z[t]
                r["dgate"][t] = e * (x[t] - before[t]) * z[t] * (1 - z[t])
                e_end[b] = (1 - z[t]) * e
    return r
