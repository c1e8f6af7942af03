"""The experts at sizes that take their larger tiles (tests/expert_tiles.py): every element
against the formulas in 64 bits, in place, with padding rows that must not be read or
written, and rows that hold a NaN or an infinity."""

import pytest
import torch

import combine_top_id_amd as M
from tests import expert_tiles as T
from tests.gpu_util import say
from tests.test_gpu_expert_ffn import NAN, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("R,E,K,S,slots,H,I,mv", T.LARGE_CASES)
def test_large_tiles_against_64_bits(R, E, K, S, slots, H, I, mv, act):
    say(f"ffn tiles R={R} E={E} K={K} S={S} slots={slots} H={H} I={I} maxvio={mv} {act}")
    c = Case(R, E, K, S, slots, H, I, mv, 140 + R + E + S)
    if slots == 1 and E == 21:
        assert c.p.n_fallback > 0
    c.check(act, 177)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("R,E,K,S,slots,H,I,mv", T.LARGE_CASES)
def test_nonfinite_rows_stay_in_their_rows(R, E, K, S, slots, H, I, mv, act):
    """A NaN or an infinity in a group's first, last and middle rows, in both passes."""
    say(f"ffn tiles nonfinite R={R} E={E} S={S} H={H} I={I} {act}")
    c = Case(R, E, K, S, slots, H, I, mv, 150 + R + E + S)
    r0, n, _, _ = max(c.groups, key=lambda g: g[1])
    bad = sorted({r0, r0 + n // 2 + 1, r0 + n - 1})
    rest = c.mapped.clone()
    rest[bad] = False

    def forward():
        return M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, I, act=act, save=True)

    def backward():
        return M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, I, act=act)

    y0, h0, gu = forward()
    g_y = c.rows_of(H, 151)
    back0 = backward()
    x = c.recv.clone()
    for k, r in enumerate(bad):
        c.recv[r, (H - 1 - 9 * k)] = [NAN, float("inf"), NAN][k % 3]
    y, h, gu2 = forward()
    for got, want in ((y, y0), (h, h0), (gu2, gu)):
        assert torch.equal(got[rest], want[rest])
        assert not torch.isfinite(got[bad]).any()
    c.recv = x
    # the gradient: a NaN gate, a NaN up, a NaN output gradient
    gate, up, grad = (bad * 3)[:3]
    gu[gate, I - 1], gu[up, I + 3], g_y[grad, H - 2] = NAN, NAN, NAN
    g_recv, g_gu = backward()
    for got, want in zip((g_recv, g_gu), back0):
        assert torch.equal(got[rest], want[rest])
        assert torch.isnan(got[bad]).any(1).all()
    assert torch.isnan(g_recv[bad]).all()
    if len(bad) == 3:
        assert torch.isnan(g_gu[gate]).nonzero().flatten().tolist() == [I - 1, 2 * I - 1]
        assert torch.isnan(g_gu[up]).nonzero().flatten().tolist() == [3]
        assert torch.isnan(g_gu[grad]).all()
    torch.cuda.synchronize()
