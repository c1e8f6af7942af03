"""Buffers of the experts' calls that lie next to each other in one allocation are taken, and
those that overlap are refused, through the binding."""

import pytest
import torch

import combine_top_id_amd as M
from tests.gpu_util import say
from tests.test_gpu_expert_ffn import NAN, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


def cut(flat, *shapes):
    out, at = [], 0
    for s in shapes:
        n = 1
        for d in s:
            n *= d
        out.append(flat[at:at + n].view(*s))
        at += n
    assert at == flat.numel()
    return out


def test_neighbours_are_taken_and_overlaps_refused():
    say("expert overlaps")
    c = Case(4, 16, 2, 64, 4, 64, 32, 2.0, 181)
    H, I, n, el = c.H, c.I, c.rows, 3 * c.H * c.I
    g_y = c.rows_of(H, 182)
    y, h, gu = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, I, save=True)
    back = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, I)
    home, rep = M.moonep_expert_ffn_bwd_weight(c.plan, c.recv, g_y, h, back[1])

    flat = torch.full((n * (2 * H + 3 * I),), NAN, dtype=torch.bfloat16, device="cuda")
    h2, x, gu2, y2 = cut(flat, (n, I), (n, H), (n, 2 * I), (n, H))
    x.copy_(c.recv)
    M.moonep_expert_ffn(c.plan, x, c.home_w, c.slot_w, I, h=h2, gu=gu2, y=y2)
    for a, b in ((y2, y), (h2, h), (gu2, gu)):
        assert torch.equal(a[c.mapped], b[c.mapped])
    flat = torch.full((n * (2 * H + 2 * I),), NAN, dtype=torch.bfloat16, device="cuda")
    r2, gg2, gy2 = cut(flat, (n, H), (n, 2 * I), (n, H))
    gy2.copy_(g_y)
    gg2.copy_(gu)
    M.moonep_expert_ffn_bwd_data(c.plan, gy2, gg2, c.home_w, c.slot_w, I, g_gu=gg2, g_recv=r2)
    assert torch.equal(r2[c.mapped], back[0][c.mapped]) and torch.equal(gg2[c.mapped], back[1][c.mapped])
    flat = torch.full(((c.E + c.R * c.slots) * el,), NAN, device="cuda")
    home2, rep2 = cut(flat, (c.E, el), (c.R, c.slots, el))
    M.moonep_expert_ffn_bwd_weight(c.plan, c.recv, g_y, h, back[1], home_grad=home2, rep_grad=rep2)
    assert torch.equal(home2, home)

    kept = [t.clone() for t in (c.recv, h, gu, g_y)]
    wide = torch.empty(n, 2 * H, dtype=torch.bfloat16, device="cuda").view(2 * n, H)
    for call in (lambda: M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, I, y=c.recv),
                 lambda: M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, I, gu=gu, h=gu.view(2 * n, I)[:n]),
                 lambda: M.moonep_expert_ffn(c.plan, wide[:n], c.home_w, c.slot_w, I, y=wide[n - 1:2 * n - 1]),
                 lambda: M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, I, g_recv=g_y),
                 lambda: M.moonep_expert_ffn_bwd_weight(c.plan, c.recv, g_y, h, back[1], home_grad=home, rep_grad=home)):
        with pytest.raises(M.MoonepError, match="invalid"):
            call()
    torch.cuda.synchronize()
    for a, b in zip((c.recv, h, gu, g_y), kept):
        assert torch.equal(a[c.mapped], b[c.mapped])
