"""The experts at the ends of what the header allows: the largest matrices, more rounds of
tiles than one look-up holds where the plan has few groups, and tokens that name an expert
twice."""

import numpy as np
import pytest
import torch

import combine_top_id_amd as M
from tests import expert_ref as X
from tests.gpu_util import say
from tests.test_gpu_expert_ffn import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


def test_largest_matrices():
    """Up rows that begin just below 2^31 bytes behind their gate rows, in the second of two
    experts; all of the forward pass and the rows' gradient, and the corners of the weights'."""
    H, I = 32768, 32504
    assert (I + 256) * H < 2 ** 30 <= (I + 264) * H
    say("ffn largest matrices")
    c = Case(1, 2, 1, 24, 0, H, I, 0.5, 211)
    _, h, gu = c.check_forward("silu")
    g_y, _, g_gu = c.check_rows_gradient("silu", gu, 212)
    home, _ = M.moonep_expert_ffn_bwd_weight(c.plan, c.recv, g_y, h, g_gu)
    torch.cuda.synchronize()
    for r0, n, e, _ in c.groups:
        s = slice(r0, r0 + n)
        x, gy, hh, gg = (t[s].double() for t in (c.recv, g_y, h, g_gu))
        gate_up, down = home[e][:2 * I * H].view(2 * I, H), home[e][2 * I * H:].view(H, I)
        for got, a, b in ((gate_up, gg, x), (down, gy, hh)):
            rows, cols = got.shape
            for p in (0, rows // 2 - 150, rows - 300):
                for q in (0, cols - 300):
                    u, v = a[:, p:p + 300].T, b[:, q:q + 300]
                    X.close(got[p:p + 300, q:q + 300], u @ v, n * X.U32 * (u.abs() @ v.abs()) + 1e-30, X.U32,
                            f"gradient of expert {e}")
    torch.cuda.synchronize()


def test_more_rounds_than_a_look_up_holds_with_few_groups():
    """Over 64 rounds of tiles of four experts, every row compared."""
    R, E, K, S, slots, H, I = 2, 4, 2, 9100, 1, 32768, 8
    say("ffn many rounds, few groups")
    c = Case(R, E, K, S, slots, H, I, 0.6, 213)
    for product in ("down", "g_rows"):
        wide, rows, _ = M.moonep_expert_tile(c.plan, H, I, product)
        assert (R * S * K // rows) * (H // wide) > 64 * 256 * (1 if wide == 256 else 2)
    recv = c.recv
    y, h, gu = M.moonep_expert_ffn(c.plan, recv, c.home_w, c.slot_w, I, save=True)
    g_y = c.rows_of(H, 214, 0.1)
    g_recv, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, I)
    for r0, n, _, e in c.groups:
        for k in range(r0, r0 + n, 4096):
            s, w = slice(k, min(k + 4096, r0 + n)), c.home_w[e]
            z, v, hh, dz, dv, dh = X.gate_up(recv[s], w, H, I, "silu")
            X.close(h[s], hh, dh, X.UB16, "h")
            X.close(gu[s], torch.cat([z, v], 1), torch.cat([dz, dv], 1), X.UB16, "gu")
            X.close(y[s], *X.down(h[s], w, H, I), X.UB16, "y")
            gg, gv, dg, du = X.back_gu(g_y[s], gu[s], w, H, I, "silu")
            X.close(g_gu[s], torch.cat([gg, gv], 1), torch.cat([dg, du], 1), X.UB16, "g_gu")
            X.close(g_recv[s], *X.back_rows(g_gu[s], w, H, I), X.UB16, "g_recv")
    torch.cuda.synchronize()


@pytest.mark.parametrize("slots", [0, 1])
def test_tokens_that_name_an_expert_twice(slots):
    R, E, K, S = 4, 8, 3, 70
    ids = np.random.default_rng(215).integers(0, E, (R * S, K)).astype(np.int32)
    ids[::3, 1] = ids[::3, 0]
    ids[::5, :] = 2
    say(f"ffn ids twice slots={slots}")
    Case(R, E, K, S, slots, 136, 72, 0, 216, ids=ids).check("gelu", 217)
