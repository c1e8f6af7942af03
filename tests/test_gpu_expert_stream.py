"""Every call of the expert block runs on the stream that it is given: an input reaches its
buffer on that stream late, behind work that takes tens of milliseconds, and the call is made
from another stream without a wait.  Launched anywhere else it would read NaN."""

import pytest
import torch

import combine_top_id_amd as M
from tests.gpu_util import say
from tests.test_gpu_expert_ffn import NAN, Case, bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


def test_calls_run_on_the_stream_they_are_given():
    say("expert block on a given stream")
    c = Case(4, 16, 2, 64, 4, 128, 64, 2.0, 191)
    H, I, T = c.H, c.I, c.rows
    g_y, gamma = c.rows_of(H, 192), bf16(H, seed=193)
    x = bf16(T, H, seed=194)
    y, h, gu = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, I, save=True)
    _, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, I)
    rows, _, rstd = M.moonep_rmsnorm_q8(x, gamma)
    new = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    f32, u8 = torch.float32, torch.uint8
    el = 3 * H * I
    # the call from its late input, what it writes, and the rows that count
    calls = [
        ("ffn", c.recv, lambda b, o, s: M.moonep_expert_ffn(c.plan, b, c.home_w, c.slot_w, I, h=o[0], gu=o[1], y=o[2],
                                                            stream=s),
         lambda: [new(T, I), new(T, 2 * I), new(T, H)]),
        ("data", g_y, lambda b, o, s: M.moonep_expert_ffn_bwd_data(c.plan, b, gu, c.home_w, c.slot_w, I, g_gu=o[0],
                                                                   g_recv=o[1], stream=s),
         lambda: [new(T, 2 * I), new(T, H)]),
        ("weight", c.recv, lambda b, o, s: M.moonep_expert_ffn_bwd_weight(c.plan, b, g_y, h, g_gu, home_grad=o[0],
                                                                          rep_grad=o[1], stream=s),
         lambda: [new(c.E, el, t=f32), new(c.R, c.slots, el, t=f32)]),
        ("norm", x, lambda b, o, s: M.moonep_rmsnorm(b, gamma, out=o[0], h=o[1], rstd=o[2], stream=s),
         lambda: [new(T, H), new(T, H), new(T, t=f32)]),
        ("q8", x, lambda b, o, s: M.moonep_rmsnorm_q8(b, gamma, rows=o[0], h=o[1], rstd=o[2], stream=s),
         lambda: [new(T, M.moonep_q8_row_bytes(H), t=u8), new(T, H), new(T, t=f32)]),
        ("unpack", rows, lambda b, o, s: M.moonep_q8_unpack(b, H, out=o[0], stream=s), lambda: [new(T, H)]),
        ("norm bwd", x, lambda b, o, s: M.moonep_rmsnorm_bwd(x, b, gamma, rstd, g_x=o[0], g_gamma=o[1], workspace=ws,
                                                             stream=s),
         lambda: [new(T, H), new(H, t=f32)])]
    ws = torch.empty(M.lib().moonep_rmsnorm_bwd_workspace(T, H), dtype=u8, device="cuda")
    s = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    for name, late, call, outputs in calls:
        say(" ", name)
        want = outputs()
        call(late, want, None)
        got = outputs()
        buf = torch.full_like(late, NAN) if late.dtype is torch.bfloat16 else torch.full_like(late, 0x7F)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(30):
                torch.mm(a, a)
            buf.copy_(late)
            waiting = torch.cuda.Event()
            waiting.record()
        call(buf, got, s)
        assert not waiting.query(), "the input has to arrive after the call is made"
        s.synchronize()
        for g, w in zip(got, want):
            if g.shape[0] == T and g.dtype is torch.bfloat16 and name in ("ffn", "data"):
                g, w = g[c.mapped], w[c.mapped]
            assert torch.equal(g, w), name
    torch.cuda.synchronize()
