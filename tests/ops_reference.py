"""Plain 64-bit forms of the layer's parts (dispatch, combine, linear, swiglu and their
gradients), on any device."""
from __future__ import annotations

import torch

BF16 = 2.0 ** -8       # half a step of bf16, relative
E4M3 = 2.0 ** -4       # of e4m3, in its normal range
E4M3_SUB = 2.0 ** -10  # half a step of e4m3's subnormals


def order(idx, n):
    """(starts, pair_of_slot, slot_of_pair), pair by pair."""
    flat = idx.flatten().tolist()
    rows = [[] for _ in range(n)]
    for p, e in enumerate(flat):
        if 0 <= e < n:
            rows[e].append(p)
    starts, pair, slot = [0], [-1] * len(flat), [-1] * len(flat)
    at = 0
    for r in rows:
        for p in r:
            pair[at], slot[p] = p, at
            at += 1
        starts.append(at)
    dev = idx.device
    return (torch.tensor(starts, dtype=torch.int32, device=dev),
            torch.tensor(pair, dtype=torch.int32, device=dev),
            torch.tensor(slot, dtype=torch.int32, device=dev).view(idx.shape))


def quantise(x):
    """fp32 rows -> (codes uint8, scales fp32): fp32 quotients (by IEEE division on the host)."""
    dev = x.device
    x = x.float().cpu()
    rows, width = x.shape
    codes, scales = [], []
    for c in range(0, width, 128):
        g = x[:, c:c + 128]
        amax = torch.where(g.isnan(), torch.zeros_like(g), g).abs().amax(dim=1)
        s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        q = (g / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.append(q)
        scales.append(s)
    return torch.cat(codes, 1).to(dev), torch.stack(scales, 1).to(dev)


def values(codes, scales):
    """The values of quantised rows, or of one group's weights [out, in], in 64 bits."""
    s = scales.double()
    if s.shape[0] != codes.shape[0]:
        s = s.repeat_interleave(128, dim=0)[:codes.shape[0]]
    s = s.repeat_interleave(128, dim=1)[:, :codes.shape[1]]
    return codes.view(torch.float8_e4m3fn).double() * s


def linear(x, codes, scales, starts, y, trans=False):
    """x (64-bit values of rows) by group into y; (results, sums of magnitudes)."""
    out, mag = y.double().clone(), torch.zeros_like(y, dtype=torch.float64)
    for g in range(codes.shape[0]):
        a, b = int(starts[g]), int(starts[g + 1])
        if b > a:
            w = values(codes[g], scales[g])
            w = w if trans else w.t()
            out[a:b] = x[a:b] @ w
            mag[a:b] = x[a:b].abs() @ w.abs()
    return out, mag


def combine(rows, slot, weights=None):
    """(y, sums of magnitudes)"""
    there = slot >= 0
    x = rows[slot.clamp(min=0).long()].double()
    x = torch.where(there[..., None], x, torch.zeros_like(x))
    if weights is not None:
        x = x * torch.where(there, weights.double(), torch.zeros_like(weights.double()))[..., None]
    return x.sum(1), x.abs().sum(1)


def swiglu(gate_up):
    g, u = gate_up.double().chunk(2, dim=1)
    return g * torch.sigmoid(g) * u


def swiglu_grad(dh, gate_up):
    g, u = gate_up.double().chunk(2, dim=1)
    s = torch.sigmoid(g)
    return torch.cat([dh.double() * u * s * (1 + g * torch.sigmoid(-g)),
                      dh.double() * g * s], dim=1)
