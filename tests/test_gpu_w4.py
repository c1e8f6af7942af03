"""The experts in 4 bits on the GPU: packing bit for bit, the forward pass with rows in bf16 and in 8
bits against the formulas in 64 bits with bounds derived from the arithmetic (tests/w4_ref.py),
element by element, padding rows and unused slots untouched."""

import numpy as np
import pytest
import torch

import combine_top_id_amd as M
from gen import TINY, make_hidden
from tests import expert_ref as X
from tests import w4_ref as W
from tests.gpu_util import say
from tests.test_gpu_expert_ffn import Case, bf16
from tests.w4_tiles import TILES

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


# ----------------------------------------------------------------------------------------
# packing
# ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("n,H,I,more", [(1, 8, 8, 0), (3, 72, 40, 8), (2, 1000, 680, 0), (1, 128, 64, 16), (2, 264, 24, 24),
                                        (1, 24, 1000, 0), (5, 512, 256, 0), (1, 7168, 256, 0), (1, 16, 32768, 0),
                                        (1, 32768, 16, 0)])
def test_packing_against_64_bits(n, H, I, more):
    say(f"w4 pack n={n} H={H} I={I} pitch +{more}")
    el, need = 3 * I * H, M.moonep_w4_slab_bytes(H, I)
    w = torch.full((n, el + more), NAN, dtype=torch.bfloat16, device="cuda")
    w[:, :el] = bf16(n, el, seed=n + H + I) * torch.exp2(torch.randint(-8, 9, (n, el), device="cuda").float())
    w4 = torch.full((n, need + 2 * more), 0xA5, dtype=torch.uint8, device="cuda")
    assert M.moonep_w4_pack(w, H, I, out=w4) is w4
    assert (w4[:, need:] == 0xA5).all(), "the slab's tail must not be written"
    got = torch.full((n, el + more), NAN, dtype=torch.bfloat16, device="cuda")
    assert M.moonep_w4_unpack(w4, H, I, out=got) is got
    assert torch.isnan(got[:, el:]).all()
    for e in range(n):
        assert torch.equal(got[e, :el].double(), W.w4_slab(w[e], H, I))
    # what is of that form already is kept: its values are, while 6.3 is first 3 * 2 and then 6 * 1
    assert torch.equal(M.moonep_w4_unpack(M.moonep_w4_pack(got, H, I), H, I), got[:, :el])


def test_packing_of_borders_and_extremes():
    H, I = 64, 32
    w = torch.zeros(1, 3 * I * H, dtype=torch.bfloat16, device="cuda")
    rows = w[0, :2 * I * H].view(2 * I, H)
    ties = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 0.26, 4.97],
                        device="cuda")
    for r, e in enumerate((0, -20, 100, 124, -124, -126, -130, -133, 125)):
        rows[r, :17] = (ties.double() * 2.0 ** e).to(torch.bfloat16)       # near both ends of bf16's range
    rows[20, :2] = torch.tensor([3.38e38, -1e38], device="cuda")           # the largest
    rows[21, 3] = 2.0 ** -133                                              # the smallest
    rows[22, 5], rows[23, 40] = float("inf"), NAN                          # their group only
    rows[22, 40], rows[23, 5] = 3.0, -3.0
    got = M.moonep_w4_unpack(M.moonep_w4_pack(w, H, I), H, I)
    ref = W.w4_slab(w[0], H, I).to(torch.bfloat16).double()               # subnormals of bf16 are its own
    assert torch.equal(torch.nan_to_num(got[0].double(), nan=-77.0), torch.nan_to_num(ref, nan=-77.0))
    bad = torch.isnan(got[0, :2 * I * H].view(2 * I, H))
    assert bad.sum() == 64 and bad[22, :32].all() and bad[23, 32:].all()
    assert torch.isnan(got).sum() == 64


def test_packing_of_nothing():
    w = torch.empty(0, 3 * 64 * 32, dtype=torch.bfloat16, device="cuda")
    w4 = M.moonep_w4_pack(w, 64, 32)
    assert w4.shape == (0, M.moonep_w4_slab_bytes(64, 32)) and M.moonep_w4_unpack(w4, 64, 32).shape == w.shape


# ----------------------------------------------------------------------------------------
# the experts
# ----------------------------------------------------------------------------------------

class Case4(Case):
    """A routed batch with the weights in 4 bits: home_w is what they stand for."""

    def __init__(self, *args, more=0, **kw):
        super().__init__(*args, **kw)
        H, I = self.H, self.I
        self.home_w4 = torch.full((self.E, M.moonep_w4_slab_bytes(H, I) + more), 0xFF, dtype=torch.uint8, device="cuda")
        self.unrounded = self.home_w
        M.moonep_w4_pack(self.unrounded, H, I, out=self.home_w4)
        self.home_w = M.moonep_w4_unpack(self.home_w4, H, I)
        # a slot that nothing uses holds NaN
        self.slot_w4 = torch.full((self.R, self.slots, self.home_w4.shape[1]), 0xFF, dtype=torch.uint8, device="cuda")
        M.moonep_prefetch_weight(self.plan, self.home_w4.view(torch.bfloat16), self.slot_w4.view(torch.bfloat16))

    def check16(self, act):
        H, I = self.H, self.I
        y, h, gu = M.moonep_expert_ffn_w4(self.plan, self.recv, self.home_w4, self.slot_w4, I, act=act, h=self.empty(I),
                                          gu=self.empty(2 * I), y=self.empty(H))
        for r0, n, _, e in self.groups:
            w, s = self.home_w[e], slice(r0, r0 + n)
            z, v, hh, dz, dv, dh = X.gate_up(self.recv[s], w, H, I, act)
            X.close(gu[s, :I], z, dz, X.UB16, "gate")
            X.close(gu[s, I:], v, dv, X.UB16, "up")
            X.close(h[s], hh, dh, X.UB16, "h")
            ref, d = X.down(h[s], w, H, I)
            X.close(y[s], ref, d, X.UB16, "y")
        for t, what in ((y, "y"), (h, "h"), (gu, "gu")):
            self.untouched(t, what)
        y2, _, none = M.moonep_expert_ffn_w4(self.plan, self.recv, self.home_w4, self.slot_w4, I, act=act)
        assert none is None and torch.equal(y2[self.mapped], y[self.mapped])
        return y, h, gu

    def rows8(self):
        x = W.q8(torch.where(self.mapped[:, None], self.recv, torch.zeros_like(self.recv)))
        x[~self.mapped] = 0xFF                        # nothing may read them
        return x

    def check8(self, act, x=None):
        H, I = self.H, self.I
        x = self.rows8() if x is None else x
        h = torch.full((self.rows, W.row_bytes(I)), 0xA5, dtype=torch.uint8, device="cuda")
        y, h2 = M.moonep_expert_ffn_w4q8(self.plan, x, self.home_w4, self.slot_w4, H, I, act=act, h=h, y=self.empty(H))
        assert h2 is h
        for r0, n, _, e in self.groups:
            w, s = self.home_w[e], slice(r0, r0 + n)
            ref, d = W.gate_up8(W.q8_values(x[s], H)[0], w, H, I, act)
            W.close_q8(h[s], ref, d, "h")
            ref, d = W.down8(W.q8_values(h[s], I)[0], w, H, I)
            X.close(y[s], ref, d, X.UB16, "y")
        self.untouched(y, "y")
        assert (h[~self.mapped] == 0xA5).all(), "h: padding rows must not be written"
        again, _ = M.moonep_expert_ffn_w4q8(self.plan, x.view(torch.bfloat16), self.home_w4, self.slot_w4, H, I, act=act)
        assert torch.equal(again[self.mapped], y[self.mapped])
        return y, h


CASES = [
    # R, E, K, S, slots, H, I, maxvio
    (4, 16, 2, 64, 4, 128, 64, 2.0),         # the tiny workload
    (1, 1, 1, 1, 0, 8, 8, 0.0),              # one token, one expert, the smallest matrices
    (2, 4, 2, 1, 1, 72, 40, 0.5),            # one token a rank
    (3, 21, 3, 57, 1, 200, 136, 3.0),        # too few slots: fallback pieces; no size fills a tile
    (8, 64, 6, 20, 0, 264, 72, 4.0),         # no slots at all
    (2, 6, 3, 200, 2, 1000, 24, 1.0),        # a narrow expert
    (2, 6, 3, 200, 2, 24, 1000, 1.0),        # a wide one
    (4, 8, 2, 700, 2, 320, 456, 1.0),        # hundreds of rows to a group
    (2, 2, 1, 1500, 1, 512, 264, 0.4),       # over a thousand
    (16, 384, 8, 8, 4, 64, 32, 5.0),         # many experts, few rows
    (2, 6, 2, 180, 1, 136, 200, 1.0),        # around a hundred rows to an expert
    (8, 64, 4, 64, 2, 256, 1408, 0.8),       # tens of rows, many columns
    (8, 64, 8, 1, 3, 1024, 512, 1.0),        # a decode step
    (64, 1024, 2, 32, 256, 8, 8, 6.0),       # as many experts, ranks and slots as there can be
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("R,E,K,S,slots,H,I,mv", CASES)
def test_rows_in_bf16(R, E, K, S, slots, H, I, mv, act):
    say(f"w4 R={R} E={E} K={K} S={S} slots={slots} H={H} I={I} maxvio={mv} {act}")
    Case4(R, E, K, S, slots, H, I, mv, 140 + R + E + S, more=32 * (R % 2)).check16(act)
    torch.cuda.synchronize()


def up32(n):
    return (n + 31) // 32 * 32


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("R,E,K,S,slots,H,I,mv", CASES)
def test_rows_in_8_bits(R, E, K, S, slots, H, I, mv, act):
    H, I = up32(H), up32(I)
    say(f"w4q8 R={R} E={E} K={K} S={S} slots={slots} H={H} I={I} maxvio={mv} {act}")
    Case4(R, E, K, S, slots, H, I, mv, 240 + R + E + S, more=32 * (R % 2)).check8(act)
    torch.cuda.synchronize()


@pytest.mark.parametrize("sizes,q8,product,tile", TILES)
def test_every_tile(sizes, q8, product, tile):
    say(f"tile {tile} of {product}, rows in {8 if q8 else 16} bits: {sizes}")
    c = Case4(*sizes, 340 + sizes[3])
    assert M.moonep_expert_tile_w4(c.plan, c.H, c.I, q8, product) == tile
    (c.check8 if q8 else c.check16)("silu")
    torch.cuda.synchronize()


def test_the_whole_block():
    """Norm to 8 bits, dispatch of the 8-bit rows, experts, combine: as they are used together; and the bf16
    form with its gradient of the rows through the expanded weights."""
    w = TINY
    c = Case4(w.R, w.E, w.K, w.S, w.slots, w.H, 64, 2.0, 9)
    hid = make_hidden(w.T, w.H, 3, device="cuda")
    gamma = torch.ones(w.H, dtype=torch.bfloat16, device="cuda")
    rows, _, _ = M.moonep_rmsnorm_q8(hid, gamma)
    recv = torch.full((c.rows, rows.shape[1] // 2), NAN, dtype=torch.bfloat16, device="cuda")
    M.moonep_dispatch(c.plan, rows.view(torch.bfloat16), recv)
    y, h = c.check8("silu", x=recv.view(torch.uint8))
    out = M.moonep_combine(c.plan, y)
    dst = c.plan.dst_row.long()
    ref = (c.plan.weights.double()[:, :, None] * y.double()[dst]).sum(1)
    X.close(out, ref, w.K * X.U32 * 4 * ref.abs() + 1e-6, X.UB16, "out")

    # training of what is in front of frozen 4-bit experts
    _, h, gu = c.check16("silu")
    slot_w = torch.full((c.R, c.slots, c.home_w.shape[1]), NAN, dtype=torch.bfloat16, device="cuda")
    M.moonep_prefetch_weight(c.plan, c.home_w, slot_w)
    g_y = c.rows_of(c.H, 5, 0.1)
    g_recv, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, slot_w, c.I)
    for r0, n, _, e in c.groups:
        s = slice(r0, r0 + n)
        gg, gv, dg, dv = X.back_gu(g_y[s], gu[s], c.home_w[e], c.H, c.I, "silu")
        X.close(g_gu[s, :c.I], gg, dg, X.UB16, "g_gate")
        ref, d = X.back_rows(g_gu[s], c.home_w[e], c.H, c.I)
        X.close(g_recv[s], ref, d, X.UB16, "g_recv")


def test_captured_passes():
    c = Case4(4, 16, 2, 64, 4, 128, 64, 2.0, 21)
    x8 = c.rows8()
    y16, y8 = c.empty(c.H), c.empty(c.H)
    h16, h8 = c.empty(c.I), torch.zeros(c.rows, W.row_bytes(c.I), dtype=torch.uint8, device="cuda")

    def go():
        M.moonep_expert_ffn_w4(c.plan, c.recv, c.home_w4, c.slot_w4, c.I, h=h16, y=y16)
        M.moonep_expert_ffn_w4q8(c.plan, x8, c.home_w4, c.slot_w4, c.H, c.I, h=h8, y=y8)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for seed in range(3):
        c.recv.copy_(c.rows_of(c.H, 90 + seed))
        x8.copy_(c.rows8())
        y16.fill_(NAN), y8.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        a, b = y16.clone(), y8.clone()
        y16.fill_(NAN), y8.fill_(NAN)
        go()
        assert torch.equal(a[c.mapped], y16[c.mapped]) and torch.equal(b[c.mapped], y8[c.mapped])
        c.untouched(a, "y")


def test_on_the_stream_that_is_given():
    c = Case4(4, 16, 2, 64, 4, 128, 64, 2.0, 22)
    ref = M.moonep_expert_ffn_w4(c.plan, c.recv, c.home_w4, c.slot_w4, c.I)[0]
    x8 = c.rows8()
    ref8 = M.moonep_expert_ffn_w4q8(c.plan, x8, c.home_w4, c.slot_w4, c.H, c.I)[0]
    side = torch.cuda.Stream()
    late = torch.zeros_like(c.recv)
    late8 = torch.zeros_like(x8)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(c.recv)
        late8.copy_(x8)
        w4 = torch.zeros_like(c.home_w4)
    # of the same weights: 3 * 2 and 6 * 1 are one value, but not bit for bit the same in the scaled products
    M.moonep_w4_pack(c.unrounded, c.H, c.I, out=w4, stream=side)
    got = M.moonep_expert_ffn_w4(c.plan, late, w4, c.slot_w4, c.I, stream=side)[0]
    got8 = M.moonep_expert_ffn_w4q8(c.plan, late8, w4, c.slot_w4, c.H, c.I, stream=side)[0]
    back = M.moonep_w4_unpack(w4, c.H, c.I, stream=side)
    side.synchronize()
    assert torch.equal(got[c.mapped], ref[c.mapped]) and torch.equal(got8[c.mapped], ref8[c.mapped])
    assert torch.equal(back, c.home_w)


def test_two_plans_on_two_streams():
    cs = [Case4(4, 16, 2, 64, 4, 128, 64, 2.0, 31), Case4(3, 21, 3, 57, 1, 224, 160, 3.0, 32)]
    refs = [(M.moonep_expert_ffn_w4(c.plan, c.recv, c.home_w4, c.slot_w4, c.I)[0],
             M.moonep_expert_ffn_w4q8(c.plan, c.rows8(), c.home_w4, c.slot_w4, c.H, c.I)[0]) for c in cs]
    x8 = [c.rows8() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for c, x, s in zip(cs, x8, streams):
            got.append((M.moonep_expert_ffn_w4(c.plan, c.recv, c.home_w4, c.slot_w4, c.I, stream=s)[0],
                        M.moonep_expert_ffn_w4q8(c.plan, x, c.home_w4, c.slot_w4, c.H, c.I, stream=s)[0]))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        m = cs[i % 2].mapped
        assert torch.equal(g[0][m], refs[i % 2][0][m]) and torch.equal(g[1][m], refs[i % 2][1][m])


def test_slabs_further_apart_than_32_bits():
    # three slabs 2.2 GB apart: the last one's offset is past 2^32
    c = Case4(1, 3, 2, 40, 1, 128, 64, 0.5, 77)
    need, far = c.home_w4.shape[1], 2_200_000_000 // 256 * 256
    home, slot = (torch.empty(n, far, dtype=torch.uint8, device="cuda") for n in (3, 1))
    el = 3 * c.H * c.I
    wide = torch.empty(3, far // 2, dtype=torch.bfloat16, device="cuda")
    wide[:, :el] = c.unrounded
    M.moonep_w4_pack(wide, c.H, c.I, out=home)
    assert torch.equal(home[:, :need], c.home_w4)
    M.moonep_w4_unpack(home, c.H, c.I, out=wide)
    assert torch.equal(wide[:, :el], c.home_w)
    slot[0, :need] = c.slot_w4[0, 0]
    x = c.rows8()
    y = M.moonep_expert_ffn_w4(c.plan, c.recv, home, slot[None], c.I)[0]
    y8 = M.moonep_expert_ffn_w4q8(c.plan, x, home, slot[None], c.H, c.I)[0]
    assert torch.equal(y[c.mapped], M.moonep_expert_ffn_w4(c.plan, c.recv, c.home_w4, c.slot_w4, c.I)[0][c.mapped])
    assert torch.equal(y8[c.mapped], M.moonep_expert_ffn_w4q8(c.plan, x, c.home_w4, c.slot_w4, c.H, c.I)[0][c.mapped])


def test_an_invalid_plan_writes_nothing():
    ids = np.full((8, 2), 99, dtype=np.int32)
    plan = M.moonep_plan(torch.from_numpy(ids).cuda(), torch.ones(8, 2, device="cuda"), 2, 4, 2, 4, 1)
    n = plan.sz.recv_rows
    x = torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda")
    x8 = torch.zeros(n, W.row_bytes(64), dtype=torch.uint8, device="cuda")
    b = M.moonep_w4_slab_bytes(64, 32)
    home = torch.zeros(4, b, dtype=torch.uint8, device="cuda")
    slot = torch.zeros(2, 1, b, dtype=torch.uint8, device="cuda")
    y = torch.full((n, 64), NAN, dtype=torch.bfloat16, device="cuda")
    M.moonep_expert_ffn_w4(plan, x, home, slot, 32, y=y)
    M.moonep_expert_ffn_w4q8(plan, x8, home, slot, 64, 32, y=y)
    assert torch.isnan(y).all()
    assert M.moonep_plan_status(plan)["status"] == 1


@pytest.mark.parametrize("special", [NAN, float("inf"), -float("inf")])
def test_special_values_stay_in_their_row_and_column(special):
    c = Case4(2, 4, 2, 40, 1, 128, 64, 0.5, 41)
    r0, n, _, e = max(c.groups, key=lambda g: g[1])
    clean = M.moonep_expert_ffn_w4(c.plan, c.recv, c.home_w4, c.slot_w4, c.I)[0]
    c.recv[r0 + 1, 5] = special
    y, h, _ = M.moonep_expert_ffn_w4(c.plan, c.recv, c.home_w4, c.slot_w4, c.I)
    others = c.mapped.clone()
    others[r0 + 1] = False
    assert torch.equal(y[others], clean[others])
    assert not torch.isfinite(y[r0 + 1]).any()
    # a group of weights with a NaN: one output column of the expert's rows
    c.recv[r0 + 1, 5] = 0
    w = c.home_w.clone()
    w[e, 2 * c.I * c.H + 7 * c.I + 3] = special
    M.moonep_w4_pack(w, c.H, c.I, out=c.home_w4)
    M.moonep_prefetch_weight(c.plan, c.home_w4.view(torch.bfloat16), c.slot_w4.view(torch.bfloat16))
    for y in (M.moonep_expert_ffn_w4(c.plan, c.recv, c.home_w4, c.slot_w4, c.I)[0],
              M.moonep_expert_ffn_w4q8(c.plan, c.rows8(), c.home_w4, c.slot_w4, c.H, c.I)[0]):
        nan = torch.isnan(y[c.mapped])
        mine = torch.zeros(c.rows, dtype=torch.bool, device="cuda")
        for a, k, _, x in c.groups:
            if x == e:
                mine[a:a + k] = True
        assert nan[mine[c.mapped], 7].all() and nan.sum() == int(mine.sum())


def test_special_rows_in_8_bits():
    c = Case4(2, 4, 2, 40, 1, 128, 64, 0.5, 43)
    x = c.rows8()
    clean = M.moonep_expert_ffn_w4q8(c.plan, x, c.home_w4, c.slot_w4, c.H, c.I)[0]
    r0 = max(c.groups, key=lambda g: g[1])[0]
    x[r0 + 1, 5] = 0x7F                                # the code NaN
    x[r0 + 2, c.H + 1] = 0xFF                          # the scale NaN
    x[r0 + 3, :c.H] = 0                                # a row of zeros, with the smallest scales
    x[r0 + 3, c.H:] = 0
    y = M.moonep_expert_ffn_w4q8(c.plan, x, c.home_w4, c.slot_w4, c.H, c.I)[0]
    others = c.mapped.clone()
    others[r0 + 1:r0 + 4] = False
    assert torch.equal(y[others], clean[others])
    assert torch.isnan(y[r0 + 1:r0 + 3]).all() and (y[r0 + 3] == 0).all()
