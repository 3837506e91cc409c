"""The norms around a block and their gradients in 64 bits (torch, CPU), and
bounds of what 32-bit arithmetic and one final rounding may change.

U is the largest relative error of one FP32 operation (half a unit in the last
place).  A sum over a row of H <= 16384 values runs over at most 16 values of a
thread and two butterflies of five steps, so its error is at most 30 U times
the sum of the terms' magnitudes, the products' own rounding included; a
factor 1 / sqrt(mean + eps) is within 20 U of its value."""
from __future__ import annotations

import torch

U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def rms_factor(x, eps):
    return 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)


def forward(y, h, post_w, gate, scale, pre_w, eps):
    """(h', z, b): b is what the block adds, scale * gate * post_w * u.
    Everything float64; h, post_w, gate, pre_w may be None; gate [H] or [rows, 1]."""
    b = y * rms_factor(y, eps) * post_w if post_w is not None else y
    b = b * scale
    if gate is not None:
        b = b * gate
    hp = b if h is None else h + b
    z = hp * rms_factor(hp, eps)
    return hp, z if pre_w is None else z * pre_w, b


def forward_bounds(y, h, post_w, gate, scale, pre_w, eps):
    """Largest errors of the unrounded h' and z computed in FP32."""
    hp, z, b = forward(y, h, post_w, gate, scale, pre_w, eps)
    # b: the factor (20 U) and the products with scale, gate, weights and y (6 U); the sum: U
    eh = 32 * U * b.abs() + 2 * U * hp.abs()
    r1 = rms_factor(hp, eps)
    # relative change of sum h'^2 from the errors of h', half of it in the factor
    rel = (hp.abs() * eh).sum(1, keepdim=True) / (hp * hp).sum(1, keepdim=True).clamp(min=1e-300)
    ez = eh * r1 * (1.0 if pre_w is None else pre_w.abs()) + z.abs() * (rel + 24 * U)
    return eh, ez


def backward(dz, dho, hp, y, post_w, gate, scale, pre_w, eps):
    """dict of dh, dy, dpre, dpost, dgate and the bounds e_* of their FP32 errors
    (before the final rounding of dh and dy)."""
    rows = y.shape[0]
    one = torch.ones(1, dtype=torch.float64)
    zero = torch.zeros_like(y)
    dz = zero if dz is None else dz
    dho = zero if dho is None else dho
    w1 = one if pre_w is None else pre_w
    g = one if gate is None else gate
    r1 = rms_factor(hp, eps)
    n = hp * r1
    dn = dz * w1
    m1 = (dn * n).mean(1, keepdim=True)
    dh = dho + r1 * (dn - n * m1)
    # r1 (20 U), the mean (30 U), the products
    e_dh = 80 * U * (r1 * dn.abs() + r1 * n.abs() * (dn * n).abs().mean(1, keepdim=True)) + 2 * U * (dho.abs() + dh.abs())
    r2 = rms_factor(y, eps) if post_w is not None else 1.0
    u = y * r2
    w2 = one if post_w is None else post_w
    du = scale * g * w2 * dh
    e_du = (scale * g * w2).abs() * e_dh + 6 * U * du.abs()
    if post_w is not None:
        dy = r2 * (du - u * (du * u).mean(1, keepdim=True))
        e_dy = r2 * (e_du + u.abs() * (e_du * u.abs()).mean(1, keepdim=True)
                     + 100 * U * (du.abs() + u.abs() * (du * u).abs().mean(1, keepdim=True)))
    else:
        dy, e_dy = du, e_du
    out = dict(dh=dh, dy=dy, e_dh=e_dh, e_dy=e_dy, dpre=None, dpost=None, dgate=None)
    # sums over rows: any order of `rows` terms adds at most `rows` roundings to a term
    if pre_w is not None:
        out["dpre"] = (dz * n).sum(0)
        out["e_dpre"] = (rows + 64) * U * (dz * n).abs().sum(0)
    if post_w is not None:
        t = scale * g * dh * u
        out["dpost"] = t.sum(0)
        out["e_dpost"] = (rows + 64) * U * t.abs().sum(0) + ((scale * g * u).abs() * e_dh).sum(0)
    if gate is not None:
        t = scale * w2 * dh * u
        over = 0 if gate.dim() == 1 else 1
        out["dgate"] = t.sum(over).view(gate.shape)
        out["e_dgate"] = ((rows + 64 if over == 0 else 64) * U * t.abs().sum(over)
                          + ((scale * w2 * u).abs() * e_dh).sum(over)).view(gate.shape)
    return out
