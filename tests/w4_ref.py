"""Weights in 4 bits and rows in 8, in 64 bits, from their definitions; shares no code with the
library.  What goes with them are worst cases of the library's arithmetic, as in
tests/expert_ref.py."""

import torch

from tests import expert_ref as X

U8 = 2.0 ** -4           # an e4m3 code is off by half a step: 2^-4 of the value, 2^-10 of the scale below 2^-6
# A scaled matrix instruction adds four neighbours along k with the bits cut off that lie more than 13
# below the largest one's power of two: each of the three others loses less than 2^-13 of the largest,
# which the four's magnitudes add up to at least.
CUT = 3 * 2.0 ** -13


def grid(m, bits, least):
    """Magnitudes on the grid with `bits` bits of fraction, even spacing below 2^least; ties to even."""
    step = torch.exp2(torch.floor(torch.log2(m.clamp_min(2.0 ** least))) - bits)
    return torch.round(m / step) * step


def power(top, most, floor):
    """The smallest power of two, 2^floor or more, that brings `top` to `most` or less."""
    p = torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-300) / most)).clamp_min(floor))
    return torch.where(top / p > most, p * 2, p)       # the logarithm's own rounding


def w4(m):
    """A matrix [rows, n] as the values of its 4-bit form."""
    rows, n = m.shape
    b = torch.nn.functional.pad(m.double(), (0, -n % 32)).view(rows, -1, 32)
    p = power(b.abs().amax(2, keepdim=True), 6.0, -126)
    v = torch.sign(b) * grid(b.abs() / p, 1, 0) * p
    v = torch.where(torch.isfinite(b).all(2, keepdim=True), v, torch.nan)
    return v.reshape(rows, -1)[:, :n]


def w4_slab(w, H, I):
    """An expert's slab [3*I*H] as the values of its 4-bit form."""
    return torch.cat([w4(w[:2 * I * H].view(2 * I, H)).reshape(-1), w4(w[2 * I * H:3 * I * H].view(H, I)).reshape(-1)])


def row_bytes(n):
    return (n + n // 32 + 15) // 16 * 16


def q8(x):
    """Rows as rows in 8 bits: codes, scales, zeros."""
    b = x.double().view(x.shape[0], -1, 32)
    p = power(b.abs().amax(2, keepdim=True), 448.0, -127)
    codes = (torch.sign(b) * grid(b.abs() / p, 3, -6)).float().to(torch.float8_e4m3fn).view(torch.uint8)
    out = torch.zeros(x.shape[0], row_bytes(x.shape[1]), dtype=torch.uint8, device=x.device)
    n = x.shape[1]
    out[:, :n] = codes.reshape(x.shape[0], n)
    out[:, n:n + n // 32] = (torch.log2(p[:, :, 0]) + 127).to(torch.uint8)
    return out


def q8_values(rows, n):
    """(values, the blocks' powers of two [rows, blocks]), 64 bits."""
    p = torch.exp2(rows[:, n:n + n // 32].double() - 127)
    v = rows[:, :n].contiguous().view(torch.float8_e4m3fn).double()
    return v * p.repeat_interleave(32, 1), p


def close_q8(rows, ref, bound, what):
    """Rows in 8 bits against what was rounded, known to `bound`: each value, the blocks' scales, the zeros."""
    n = ref.shape[1]
    v, p = q8_values(rows, n)
    p32 = p.repeat_interleave(32, 1)
    err = (v - ref).abs() - bound
    bad = ~(err <= torch.maximum(U8 * (ref.abs() + bound), 2.0 ** -10 * p32))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(err[bad].max()):.3g}"
    low = (ref.abs() - bound).view(len(ref), -1, 32).amax(2)
    high = (ref.abs() + bound).view(len(ref), -1, 32).amax(2)
    assert (low <= 448 * p).all(), f"{what}: a scale is too small"
    assert ((high > 224 * p) | (p <= 2.0 ** -127)).all(), f"{what}: a scale is too large"
    assert (rows[:, n + n // 32:] == 0).all(), f"{what}: the rows' ends must be zeros"


def gate_up8(x, w, H, I, kind):
    """expert_ref.gate_up with the scaled instructions' bounds."""
    z, v, h, dz, dv, _ = X.gate_up(x, w, H, I, kind)
    g, u, _ = X.slab(w, H, I)
    x = x.double().abs()
    dz, dv = dz + CUT * (x @ g.abs().T), dv + CUT * (x @ u.abs().T)
    a, _ = X.act(z, kind)
    dh = v.abs() * X.SLOPE_MAX * dz + a.abs() * dv + X.SLOPE_MAX * dz * dv + X.ACT_REL * (a * v).abs() + 1e-30
    return h, dh


def down8(h, w, H, I):
    y, d = X.down(h, w, H, I)
    return y, d + CUT * (h.double().abs() @ X.slab(w, H, I)[2].abs().T)
