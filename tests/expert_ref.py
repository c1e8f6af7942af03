"""The expert block in 64 bits, from its formulas: the gated feed-forward experts over a
plan's groups with their gradients, and the root-mean-square norm.  Plain torch on whatever
device the inputs are on; shares no code with the library.

`bound` values that go with the results are worst cases of the library's arithmetic: a sum
of n products in fp32, in any order, is off by at most n * 2^-24 times the sum of the
products' magnitudes, and a rounding to bf16 by at most 2^-8 of the value.
"""

import math

import torch

U32 = 2.0 ** -24
UB16 = torch.finfo(torch.bfloat16).eps / 2
# act in fp32: the hardware exponential is within 2 ulp, its argument z * log2(e) is rounded
# (|z| <= 88 beyond which the result is 0 or 1), a handful of roundings follow
ACT_REL = 96 * 2 * U32


def act(z, kind):
    """(activation, slope)"""
    if kind == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    c = math.sqrt(2 / math.pi)
    # (1 + tanh(u)) / 2 as sigmoid(2u): the sum would cancel for negative u, to 2^-53 of one
    p = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
    return z * p, p + 2 * z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)


SLOPE_MAX = 1.13         # of both activations (their slopes reach 1.0998 and 1.1290)


def groups(p):
    """(first row, rows, weight index, home expert) of each group of an oracle plan; the
    weight index counts the E home slabs, then the R * slots slot slabs."""
    sz = p.sz
    out = []
    for e in range(sz.E):
        if p.keep[e]:
            r = e // sz.E_loc
            out.append((r * sz.NvS + int(p.off[r, e - r * sz.E_loc]), int(p.keep[e]), e, e))
    for q in range(p.n_pieces):
        e, r, slot, n = (int(v) for v in p.pieces[q, :4])
        out.append((p.piece_row0(q), n, e if slot < 0 else sz.E + r * sz.slots + slot, e))
    return out


def slab(w, H, I):
    w = w.double()
    return w[:I * H].view(I, H), w[I * H:2 * I * H].view(I, H), w[2 * I * H:3 * I * H].view(H, I)


def gate_up(x, w, H, I, kind):
    """(gate, up, h, bound of gate, of up, of h) before any rounding to bf16 of the outputs."""
    x = x.double()
    g, u, _ = slab(w, H, I)
    z, v = x @ g.T, x @ u.T
    dz, dv = H * U32 * (x.abs() @ g.abs().T), H * U32 * (x.abs() @ u.abs().T)
    a, _ = act(z, kind)
    dh = v.abs() * SLOPE_MAX * dz + a.abs() * dv + SLOPE_MAX * dz * dv + ACT_REL * (a * v).abs() + 1e-30
    return z, v, a * v, dz, dv, dh


def down(h, w, H, I):
    """(y, bound) from h as the library stored it."""
    h = h.double()
    d = slab(w, H, I)[2]
    return h @ d.T, I * U32 * (h.abs() @ d.abs().T)


def back_gu(g_y, gu, w, H, I, kind):
    """(g_gate, g_up, bounds)"""
    d = slab(w, H, I)[2]
    g_y = g_y.double()
    g_h, dg = g_y @ d, H * U32 * (g_y.abs() @ d.abs())
    z, v = gu[:, :I].double(), gu[:, I:].double()
    a, s = act(z, kind)
    # the slope's terms cancel near its zero: its error is relative to their size, at most 2
    gg, gu_ = g_h * v * s, g_h * a
    return (gg, gu_, dg * (v * s).abs() + ACT_REL * (g_h * v).abs() * (1 + z.abs()).clamp_max(4) + 1e-30,
            dg * a.abs() + ACT_REL * gu_.abs() + 1e-30)


def back_rows(g_gu, w, H, I):
    g, u, _ = slab(w, H, I)
    gg, gu = g_gu[:, :I].double(), g_gu[:, I:].double()
    return gg @ g + gu @ u, 2 * I * U32 * (gg.abs() @ g.abs() + gu.abs() @ u.abs())


def close(got, ref, bound, rounding, what):
    """|got - ref| <= bound + rounding * (|ref| + bound), element by element."""
    got = got.double()
    bad = ~((got - ref).abs() <= bound + rounding * (ref.abs() + bound))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((got - ref).abs()[bad].max()):.3g} at value {float(ref[bad][0]):.3g}")
