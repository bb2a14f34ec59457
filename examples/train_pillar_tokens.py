"""A network on voxel tokens, trained for a few steps on synthetic frames.

A batch of frames is voxelized in one launch; every pillar becomes a token.  One
block mixes the tokens of each frame twice: attention with queries and keys
normalised per head and rotated by the pillar's (y, x), nearer pillars preferred,
and a gated recurrence along the frame's pillars.  The network predicts each
pillar's mean intensity and height from its points' horizontal positions.

    python examples/train_pillar_tokens.py [--frames 4] [--steps 20]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lidar_point_cloud_gb300 as pv  # noqa: E402
from lidar_point_cloud_gb300 import synth  # noqa: E402


class NormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        return pv.qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq)

    @staticmethod
    def backward(ctx, dq, dk):
        return (*pv.qk_norm_rope_backward(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors), None, None)


class Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, offsets, slopes, positions):
        ctx.how = dict(slopes=slopes, q_positions=positions, k_positions=positions)
        ctx.offsets = offsets
        out, lse = pv.attention(q, k, v, offsets, offsets, return_lse=True, **ctx.how)
        ctx.save_for_backward(q, k, v, out, lse)
        return out

    @staticmethod
    def backward(ctx, dout):
        grads = pv.attention_backward(dout.contiguous(), *ctx.saved_tensors, ctx.offsets, ctx.offsets, **ctx.how)
        return (*grads, None, None, None)


class GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, offsets):
        h, _, states = pv.gated_scan(x, gate, offsets, return_states=True)
        ctx.offsets = offsets
        ctx.save_for_backward(x, gate, states)
        return h

    @staticmethod
    def backward(ctx, dh):
        x, gate, states = ctx.saved_tensors
        dx, dgate, _ = pv.gated_scan_backward(dh.contiguous(), None, x, gate, states, ctx.offsets)
        return dx, dgate, None


class PillarBlock(torch.nn.Module):
    """Weights in 32 bits, tokens between the operators in bfloat16."""

    def __init__(self, features: int, channels: int = 128, heads: int = 4, key_heads: int = 2):
        super().__init__()
        self.heads, self.key_heads, self.dim = heads, key_heads, channels // heads
        self.embed = torch.nn.Linear(features, channels)
        self.qkv = torch.nn.Linear(channels, (heads + 2 * key_heads) * self.dim)
        self.mix = torch.nn.Linear(channels, channels)
        self.scan_in = torch.nn.Linear(channels, 2 * channels)
        self.scan_out = torch.nn.Linear(channels, channels)
        self.head = torch.nn.Linear(channels, 2)
        self.q_weight = torch.nn.Parameter(torch.ones(self.dim))
        self.k_weight = torch.nn.Parameter(torch.ones(self.dim))
        self.register_buffer("inv_freq", pv.rope_frequencies(self.dim, axes=2))
        self.register_buffer("slopes", torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]))

    def forward(self, features, coords, offsets):
        x = self.embed(features)
        qkv = self.qkv(x).to(torch.bfloat16).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.heads, self.key_heads, self.key_heads], dim=1)  # slices, as they lie
        q, k = NormRope.apply(q, k, self.q_weight, self.k_weight, coords[:, 2:], self.inv_freq)
        o = Attention.apply(q, k, v, offsets, self.slopes, coords[:, 2:])
        x = x + self.mix(o.flatten(1).float())
        inputs, gate = self.scan_in(x).to(torch.bfloat16).chunk(2, dim=1)
        x = x + self.scan_out(GatedScan.apply(inputs, gate, offsets).float())
        return self.head(x)


def tokens_of(frames: int, device):
    """Features, coordinates, row offsets and targets of a batch of KITTI-shaped frames."""
    points, frame_offsets, P = synth.make_batch("kitti", frames)
    voxels, coords, counts = pv.voxelize_batch(torch.from_numpy(points).to(device), frame_offsets.tolist(),
                                               P.point_cloud_range, P.voxel_size, P.max_points, P.max_voxels)
    voxels = voxels.nan_to_num(0.0, 0.0, 0.0)  # an intensity is copied as it is, a NaN too
    n = counts.clamp_min(1)[:, None].float()
    mean = voxels.sum(1) / n
    spread = (voxels[..., :2].square().sum(1) / n - mean[:, :2].square()).clamp_min(0).sqrt()
    cell = coords[:, 2:].float() / torch.tensor([496.0, 432.0], device=device)
    features = torch.cat([mean[:, :2] / 40.0, spread, cell, n.log()], 1)
    rows = torch.bincount(coords[:, 0].long(), minlength=frames).tolist()
    offsets = [sum(rows[:b]) for b in range(frames + 1)]
    return features, coords, offsets, torch.stack([mean[:, 3], mean[:, 2] / 3.0], 1)


def main(argv=None) -> list:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--frames", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    device = torch.device("cuda")
    features, coords, offsets, target = tokens_of(args.frames, device)
    model = PillarBlock(features.shape[1]).to(device)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(args.steps):
        opt.zero_grad(set_to_none=True)
        loss = (model(features, coords, offsets) - target).square().mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    print(f"{offsets[-1]} pillars of {args.frames} frames: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {args.steps} steps")
    return losses


if __name__ == "__main__":
    main()
