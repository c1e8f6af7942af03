"""The gated feed-forward experts on the GPU, forward and backward, against the formulas in
64 bits with bounds derived from the arithmetic (tests/expert_ref.py): every group of the
plan, element by element, padding rows and unused slots untouched."""

import numpy as np
import pytest
import torch

import combine_top_id_amd as M
from gen import TINY, make_routing, make_hidden
from oracle import moonep_oracle as O
from tests import expert_ref as X
from tests.gpu_util import say, to_dev_ids

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


def bf16(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


class Case:
    """A routed batch: the GPU plan, the oracle's, the weights and the dispatched rows."""

    def __init__(self, R, E, K, S, slots, H, I, mv, seed, ids=None, w_el=None):
        self.R, self.E, self.K, self.S, self.slots, self.H, self.I = R, E, K, S, slots, H, I
        if ids is None:
            t, wt, _, _ = make_routing(R, E, K, S, mv, seed)
            ids, wt = t.numpy(), wt.numpy()
        else:
            wt = np.full((R * S, K), 1.0 / K, dtype=np.float32)
        self.ids, self.wt = ids, wt
        self.plan = M.moonep_plan(*to_dev_ids(ids, wt), R, E, K, S, slots)
        self.p = O.plan(ids, R, E, K, S, slots)
        self.groups = X.groups(self.p)
        self.rows = self.plan.sz.recv_rows
        self.w_el = w_el or 3 * H * I
        self.home_w = bf16(E, self.w_el, seed=seed + 1, scale=H ** -0.5)
        self.slot_w = torch.full((R, slots, self.w_el), NAN, dtype=torch.bfloat16, device="cuda")
        M.moonep_prefetch_weight(self.plan, self.home_w, self.slot_w)
        self.mapped = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        for r0, n, _, _ in self.groups:
            self.mapped[r0:r0 + n] = True
        self.recv = self.rows_of(H, seed + 2)

    def rows_of(self, n, seed, scale=1.0):
        """Buffer rows whose padding holds NaN: nothing may read it."""
        t = bf16(self.rows, n, seed=seed, scale=scale)
        t[~self.mapped] = NAN
        return t

    def empty(self, n):
        return torch.full((self.rows, n), NAN, dtype=torch.bfloat16, device="cuda")

    def untouched(self, t, what):
        assert torch.isnan(t[~self.mapped]).all(), f"{what}: padding rows must not be written"

    def check_forward(self, act):
        H, I = self.H, self.I
        y, h, gu = M.moonep_expert_ffn(self.plan, self.recv, self.home_w, self.slot_w, I, act=act,
                                       h=self.empty(I), gu=self.empty(2 * I), y=self.empty(H))
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
        # nothing saved: the same y
        y2, _, none = M.moonep_expert_ffn(self.plan, self.recv, self.home_w, self.slot_w, I, act=act)
        assert none is None and torch.equal(y2[self.mapped], y[self.mapped])
        return y, h, gu

    def check_rows_gradient(self, act, gu, seed):
        H, I = self.H, self.I
        g_y = self.rows_of(H, seed, 0.1)
        g_recv, g_gu = M.moonep_expert_ffn_bwd_data(self.plan, g_y, gu, self.home_w, self.slot_w, I, act=act,
                                                    g_gu=self.empty(2 * I), g_recv=self.empty(H))
        for r0, n, _, e in self.groups:
            w, s = self.home_w[e], slice(r0, r0 + n)
            gg, gv, dg, dv = X.back_gu(g_y[s], gu[s], w, H, I, act)
            X.close(g_gu[s, :I], gg, dg, X.UB16, "g_gate")
            X.close(g_gu[s, I:], gv, dv, X.UB16, "g_up")
            ref, d = X.back_rows(g_gu[s], w, H, I)
            X.close(g_recv[s], ref, d, X.UB16, "g_recv")
        self.untouched(g_gu, "g_gu")
        self.untouched(g_recv, "g_recv")
        # in place
        over = gu.clone()
        r2, o2 = M.moonep_expert_ffn_bwd_data(self.plan, g_y, over, self.home_w, self.slot_w, I, act=act, g_gu=over)
        assert o2 is over and torch.equal(over[self.mapped], g_gu[self.mapped])
        assert torch.equal(r2[self.mapped], g_recv[self.mapped])
        return g_y, g_recv, g_gu

    def check_weights_gradient(self, g_y, h, g_gu):
        H, I = self.H, self.I
        el = 3 * H * I
        pitch = el + 4
        home = torch.full((self.E, pitch), NAN, device="cuda")
        rep = torch.full((self.R, self.slots, pitch), NAN, device="cuda")
        M.moonep_expert_ffn_bwd_weight(self.plan, self.recv, g_y, h, g_gu, home_grad=home, rep_grad=rep)
        refs = {}
        for r0, n, w, _ in self.groups:
            s = slice(r0, r0 + n)
            x, gy, hh, gg = (t[s].double() for t in (self.recv, g_y, h, g_gu))
            ref = torch.cat([(gg.T @ x).reshape(-1), (gy.T @ hh).reshape(-1)])
            mag = torch.cat([(gg.T.abs() @ x.abs()).reshape(-1), (gy.T.abs() @ hh.abs()).reshape(-1)])
            a, m, k = refs.get(w, (0, 0, 0))
            refs[w] = (a + ref, m + mag, k + n)
        zero = torch.zeros(el, dtype=torch.float64, device="cuda")
        flat = rep.view(-1, pitch)
        for w in range(self.E + self.R * self.slots):
            got = home[w] if w < self.E else flat[w - self.E]
            assert torch.isnan(got[el:]).all(), "the slab's tail must not be written"
            if w in refs:
                ref, mag, k = refs[w]
                X.close(got[:el], ref, k * X.U32 * mag + 1e-30, X.U32, f"gradient of weight {w}")
            elif w < self.E:
                assert (got[:el] == 0).all()
            else:
                assert torch.isnan(got).all(), "unused slots must not be written"
        # added to what is there
        base = torch.randn(self.E, pitch, device="cuda")
        more, again = base.clone(), torch.zeros_like(rep)
        M.moonep_expert_ffn_bwd_weight(self.plan, self.recv, g_y, h, g_gu, home_grad=more, rep_grad=again,
                                       accumulate=True)
        assert torch.equal(more[:, :el], base[:, :el] + home[:, :el])
        assert torch.equal(more[:, el:], base[:, el:])
        for w in refs:
            if w >= self.E:
                assert torch.equal(again.view(-1, pitch)[w - self.E][:el], flat[w - self.E][:el])
        return home, rep

    def check(self, act, seed):
        y, h, gu = self.check_forward(act)
        g_y, _, g_gu = self.check_rows_gradient(act, gu, seed)
        self.check_weights_gradient(g_y, h, g_gu)
        torch.cuda.synchronize()


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
    (8, 64, 4, 64, 2, 256, 1408, 0.8),       # tens of rows, many columns: the gate and up product's
    (8, 64, 4, 80, 2, 3584, 64, 0.8),        # and the down product's
    (64, 1024, 2, 32, 256, 8, 8, 6.0),       # as many experts, ranks and slots as there can be
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("R,E,K,S,slots,H,I,mv", CASES)
def test_against_64_bits(R, E, K, S, slots, H, I, mv, act):
    say(f"ffn R={R} E={E} K={K} S={S} slots={slots} H={H} I={I} maxvio={mv} {act}")
    Case(R, E, K, S, slots, H, I, mv, 40 + R + E + S).check(act, 77)


def test_more_tiles_than_a_look_up_holds():
    """Over 64 tiles to each workgroup: 256 experts and rows of 32768."""
    say("ffn many tiles")
    c = Case(2, 256, 2, 128, 2, 32768, 8, 0.5, 71)
    y, h, gu = c.check_forward("silu")
    c.check_rows_gradient("silu", gu, 72)
    torch.cuda.synchronize()


@pytest.mark.parametrize("slots", [0, 2])
def test_one_expert_takes_all(slots):
    """Every token to expert 1: the other experts have no rows, and their gradient is zero."""
    R, E, K, S, H, I = 4, 8, 1, 150, 96, 80
    ids = np.full((R * S, K), 1, dtype=np.int32)
    say(f"ffn one expert slots={slots}")
    Case(R, E, K, S, slots, H, I, 0, 5, ids=ids).check("silu", 6)


def test_slabs_with_a_pitch():
    say("ffn pitch")
    Case(2, 6, 2, 90, 1, 128, 72, 2.0, 11, w_el=3 * 128 * 72 + 40).check("gelu", 12)


def test_large_and_nonfinite_gates():
    """Gates far outside the activations' bend, and rows that hold an infinity or a NaN: they
    stay in their row."""
    say("ffn large gates")
    c = Case(2, 4, 2, 100, 2, 64, 48, 1.0, 21)
    c.recv *= 300
    c.check("silu", 22)
    c.check("gelu", 23)
    live = torch.nonzero(c.mapped).flatten()
    a, b = int(live[3]), int(live[77])
    clean = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, c.I)[0]
    c.recv[a, 5], c.recv[b, 7] = float("inf"), NAN
    y = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, c.I)[0]
    assert torch.isnan(y[b]).all() and not torch.isfinite(y[a]).any()
    rest = c.mapped.clone()
    rest[a] = rest[b] = False
    assert torch.equal(y[rest], clean[rest])
    torch.cuda.synchronize()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_nonfinite_rows_of_the_gradient(act):
    """A NaN gate, a NaN up and a NaN in g_y reach their row's gradients and no other row."""
    say(f"ffn nonfinite gradients {act}")
    c = Case(2, 4, 2, 100, 2, 64, 48, 1.0, 24)
    I = c.I
    _, _, gu = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, I, act=act, save=True)
    g_y = c.rows_of(c.H, 25)
    clean, g_clean = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, I, act=act)
    live = torch.nonzero(c.mapped).flatten()
    gate, up, grad = (int(live[k]) for k in (5, 90, 140))
    gu[gate, 3], gu[up, I + 4], g_y[grad, 7] = NAN, NAN, NAN
    g_recv, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, I, act=act)
    bad = torch.isnan(g_gu)
    assert bad[gate].nonzero().flatten().tolist() == [3, I + 3]
    assert bad[up].nonzero().flatten().tolist() == [4]
    assert bad[grad].all() and torch.isnan(g_recv[[gate, up, grad]]).all()
    rest = c.mapped.clone()
    rest[[gate, up, grad]] = False
    assert torch.equal(g_recv[rest], clean[rest]) and torch.equal(g_gu[rest], g_clean[rest])
    torch.cuda.synchronize()


def test_gradients_against_differences():
    """The library's gradients along random directions against central differences of the
    64-bit forward pass.  bf16 rounding of g_gate and g_up (2^-8 each, independent over
    thousands of terms) is what is left: 1% of the gradient's size."""
    say("ffn differences")
    c = Case(2, 4, 2, 60, 2, 64, 48, 1.0, 31)
    H, I = c.H, c.I
    _, h, gu = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, I, save=True)
    g_y = c.rows_of(H, 32)
    g_recv, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, I)
    home, rep = M.moonep_expert_ffn_bwd_weight(c.plan, c.recv, g_y, h, g_gu)
    M.moonep_reduce_grad(c.plan, home, rep)

    def loss(x, w):
        total = 0.0
        for r0, n, _, e in c.groups:
            s = slice(r0, r0 + n)
            g, u, d = X.slab(w[e], H, I)
            a, _ = X.act(x[s] @ g.T, "silu")
            total = total + (g_y[s].double() * ((a * (x[s] @ u.T)) @ d.T)).sum()
        return float(total)

    x0, w0 = torch.where(c.mapped[:, None], c.recv, 0).double(), c.home_w.double()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    for k in range(4):
        # directions along the gradient's own signs: no cancellation in the sum
        gx = torch.where(c.mapped[:, None], g_recv, 0).double()
        dx = gx.sign() * torch.rand(x0.shape, generator=gen, device="cuda", dtype=torch.float64)
        dw = home.double().sign() * torch.rand(w0.shape, generator=gen, device="cuda", dtype=torch.float64)
        eps = 1e-6
        num = (loss(x0 + eps * dx, w0) - loss(x0 - eps * dx, w0)) / (2 * eps)
        assert abs(num - float((gx * dx).sum())) <= 0.01 * num
        num = (loss(x0, w0 + eps * dw) - loss(x0, w0 - eps * dw)) / (2 * eps)
        assert abs(num - float((home.double() * dw).sum())) <= 0.01 * num
    torch.cuda.synchronize()


def test_invalid_plan_writes_nothing():
    """An expert id outside [0, E): the plan maps nothing."""
    say("ffn invalid plan")
    c = Case(4, 16, 2, 64, 4, 64, 32, 2.0, 41)
    ids = c.ids.copy()
    ids[7, 1] = 16
    M.moonep_plan(*to_dev_ids(ids, c.wt), c.R, c.E, c.K, c.S, c.slots, plan=c.plan)
    assert M.moonep_plan_status(c.plan)["status"] == 1
    y, h, gu = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, c.I, h=c.empty(32), gu=c.empty(64),
                                   y=c.empty(64))
    assert torch.isnan(y).all() and torch.isnan(h).all() and torch.isnan(gu).all()
    g_recv, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, c.recv, gu, c.home_w, c.slot_w, c.I, g_gu=c.empty(64),
                                                g_recv=c.empty(64))
    assert torch.isnan(g_recv).all() and torch.isnan(g_gu).all()
    rep = torch.full((4, 4, 3 * 64 * 32), NAN, device="cuda")
    home, _ = M.moonep_expert_ffn_bwd_weight(c.plan, c.recv, c.recv, h, g_gu, rep_grad=rep)
    assert (home == 0).all() and torch.isnan(rep).all()
    torch.cuda.synchronize()


def test_captured_training_pass_replays():
    """plan, forward and both gradients captured once, replayed on new routings, each replay
    against the eager calls, with eager work in between."""
    R, E, K, S, slots, H, I = 4, 16, 2, 96, 4, 128, 72
    say("ffn capture")
    T = R * S
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    wt = torch.empty(T, K, dtype=torch.float32, device="cuda")
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    home_w = bf16(E, 3 * H * I, seed=2, scale=H ** -0.5)

    def fill(k):
        a, b, _, _ = make_routing(R, E, K, S, [0.5, 3.0, 1.0][k % 3], 90 + k, device="cuda")
        ids.copy_(a)
        wt.copy_(b)
        x.copy_(make_hidden(T, H, 50 + k, device="cuda"))

    def step(plan, b):
        M.moonep_plan(ids, wt, R, E, K, S, slots, plan=plan)
        M.moonep_prefetch_weight(plan, home_w, b["slot_w"])
        M.moonep_dispatch(plan, x, b["recv"])
        M.moonep_expert_ffn(plan, b["recv"], home_w, b["slot_w"], I, h=b["h"], gu=b["gu"], y=b["y"])
        M.moonep_combine(plan, b["y"], b["out"])
        M.moonep_combine_bwd(plan, b["out"], b["y"], g_y=b["g_y"], dw=b["dw"])
        M.moonep_expert_ffn_bwd_data(plan, b["g_y"], b["gu"], home_w, b["slot_w"], I, g_gu=b["g_gu"],
                                     g_recv=b["g_recv"])
        M.moonep_expert_ffn_bwd_weight(plan, b["recv"], b["g_y"], b["h"], b["g_gu"], home_grad=b["home"],
                                       rep_grad=b["rep"])
        M.moonep_reduce_grad(plan, b["home"], b["rep"])
        M.moonep_dispatch_bwd(plan, b["g_recv"], b["g_x"])

    def buffers(n):
        z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        return dict(slot_w=z(R, slots, 3 * H * I), recv=z(n, H), h=z(n, I), gu=z(n, 2 * I), y=z(n, H),
                    out=z(T, H), g_y=z(n, H), dw=z(T, K, t=torch.float32), g_gu=z(n, 2 * I), g_recv=z(n, H),
                    home=z(E, 3 * H * I, t=torch.float32), rep=z(R, slots, 3 * H * I, t=torch.float32),
                    g_x=z(T, H))

    fill(0)
    plan = M.moonep_plan(ids, wt, R, E, K, S, slots)
    b, eager_plan = buffers(plan.sz.recv_rows), None
    step(plan, b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(plan, b)
    torch.cuda.synchronize()
    e = buffers(plan.sz.recv_rows)
    for k in range(1, 5):
        fill(k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: b[n].clone() for n in ("out", "g_x", "home", "dw")}
        eager_plan = M.moonep_plan(ids, wt, R, E, K, S, slots, plan=eager_plan)
        step(eager_plan, e)
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], e[n]), f"replay {k}: {n}"


def test_two_calls_at_once():
    """Two plans' calls on two streams at the same time give what each gives alone."""
    say("ffn two streams")
    cs = [Case(4, 16, 2, 200, 4, 256, 128, 2.0, 51), Case(2, 8, 2, 300, 2, 192, 160, 1.0, 52)]
    alone = [M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, c.I)[0] for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(5):
        for k, c in enumerate(cs):
            with torch.cuda.stream(streams[k]):
                outs[k].append(M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, c.I)[0])
    torch.cuda.synchronize()
    for k, c in enumerate(cs):
        for o in outs[k]:
            assert torch.equal(o[c.mapped], alone[k][c.mapped])


def test_stream_argument():
    """Calls given a stream run on it, in order, whatever the current stream is."""
    say("ffn stream argument")
    c = Case(4, 16, 2, 200, 4, 256, 128, 2.0, 53)
    g_y = c.rows_of(c.H, 54)

    def step(stream):
        y, h, gu = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, c.I, stream=stream, h=b[0], gu=b[1], y=b[2])
        g_recv, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, c.I, stream=stream,
                                                    g_gu=b[3], g_recv=b[4])
        home, rep = M.moonep_expert_ffn_bwd_weight(c.plan, c.recv, g_y, h, g_gu, stream=stream, home_grad=b[5],
                                                   rep_grad=b[6])
        return y[c.mapped], g_recv[c.mapped], home

    def buffers():
        el = 3 * c.H * c.I
        return [c.empty(c.I), c.empty(2 * c.I), c.empty(c.H), c.empty(2 * c.I), c.empty(c.H),
                torch.empty(c.E, el, device="cuda"), torch.empty(c.R, c.slots, el, device="cuda")]

    b = buffers()
    want = step(None)
    b = buffers()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(s)
    s.synchronize()
    for a, w in zip((b[2][c.mapped], b[4][c.mapped], b[5]), want):
        assert torch.equal(a, w)
    torch.cuda.synchronize()


def test_allocations_follow_the_stream():
    """What a call allocates belongs to the stream that it runs on: memory of the current
    stream could be handed to that one's next work while the call still uses it."""
    say("ffn allocations")
    c = Case(4, 16, 2, 64, 4, 128, 64, 2.0, 55)
    g_y = c.rows_of(c.H, 56)
    gamma = torch.ones(c.H, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    seen = []
    empty = torch.empty

    def watched(*shape, **kw):
        seen.append(torch.cuda.current_stream())
        return empty(*shape, **kw)

    torch.empty = watched
    try:
        y, h, gu = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, c.slot_w, c.I, save=True, stream=s)
        g_recv, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, c.I, stream=s)
        home, rep = M.moonep_expert_ffn_bwd_weight(c.plan, c.recv, g_y, h, g_gu, stream=s)
        out, _, rstd = M.moonep_rmsnorm(y, gamma, stream=s)
        rows, _, _ = M.moonep_rmsnorm_q8(y, gamma, stream=s)
        back = M.moonep_q8_unpack(rows, c.H, stream=s)
        g_x, g_gamma = M.moonep_rmsnorm_bwd(out, y, gamma, rstd, stream=s)
    finally:
        torch.empty = empty
    s.synchronize()
    assert seen and all(x == s for x in seen)
    held = [(b["address"], b["total_size"], b["stream"]) for b in torch.cuda.memory_snapshot()]
    for t in (y, h, gu, g_recv, g_gu, home, rep, out, rstd, rows, back, g_x, g_gamma):
        of = [st for a, n, st in held if a <= t.data_ptr() < a + n]
        assert of == [s.cuda_stream]


def test_rows_past_32_bits():
    """A buffer of more than 2^31 elements: the last rows of the last group, and all gradients of
    one expert's weights against those rows' alone."""
    say("ffn large buffer")
    R, E, K, S, H, I = 2, 2, 2, 76000, 7168, 8
    ids = np.tile(np.arange(2, dtype=np.int32), (R * S, 1))
    c = Case(R, E, K, S, 0, H, I, 0, 57, ids=ids)
    assert c.rows * H > 2 ** 31
    y, h, gu = M.moonep_expert_ffn(c.plan, c.recv, c.home_w, None, I, save=True)
    r0, n, _, e = max(c.groups)
    s = slice(r0 + n - 70, r0 + n)
    w = c.home_w[e]
    _, _, hh, _, _, dh = X.gate_up(c.recv[s], w, H, I, "silu")
    X.close(h[s], hh, dh, X.UB16, "h")
    ref, d = X.down(h[s], w, H, I)
    X.close(y[s], ref, d, X.UB16, "y")
    # only those rows have an output gradient
    g_y = torch.zeros_like(c.recv)
    g_y[s] = bf16(70, H, seed=58)
    g_recv, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, None, I)
    gg, gv, dg, dv = X.back_gu(g_y[s], gu[s], w, H, I, "silu")
    X.close(g_gu[s], torch.cat([gg, gv], 1), torch.cat([dg, dv], 1), X.UB16, "g_gu")
    ref, d = X.back_rows(g_gu[s], w, H, I)
    X.close(g_recv[s], ref, d, X.UB16, "g_recv")
    home, _ = M.moonep_expert_ffn_bwd_weight(c.plan, c.recv, g_y, h, g_gu)
    x, gy, hd, ggu = (t[s].double() for t in (c.recv, g_y, h, g_gu))
    ref = torch.cat([(ggu.T @ x).reshape(-1), (gy.T @ hd).reshape(-1)])
    mag = torch.cat([(ggu.T.abs() @ x.abs()).reshape(-1), (gy.T.abs() @ hd.abs()).reshape(-1)])
    X.close(home[e], ref, 70 * X.U32 * mag + 1e-30, X.U32, "weights' gradient")
    assert (home[1 - e] == 0).all()
    torch.cuda.synchronize()


def test_block_trains_as_without_replication():
    """norm -> 8-bit rows -> dispatch -> expand -> experts -> combine, and its backward pass,
    against each token's experts applied without any plan, in 64 bits."""
    R, E, K, S, slots, H, I = TINY.R, TINY.E, TINY.K, TINY.S, TINY.slots, 128, 64
    say("expert block")
    c = Case(R, E, K, S, slots, H, I, TINY.maxvio[0], 61)
    T = R * S
    x, res = bf16(T, H, seed=62), bf16(T, H, seed=63, scale=2.0)
    gamma = (1 + 0.1 * torch.randn(H, device="cuda")).to(torch.bfloat16)
    rows, stream, rstd = M.moonep_rmsnorm_q8(x, gamma, res=res)
    q = M.moonep_q8_unpack(rows, H)
    sent = M.moonep_dispatch(c.plan, rows.view(torch.bfloat16))
    recv = M.moonep_q8_unpack(sent, H)
    assert torch.equal(recv[c.plan.dst_row.long()], q[:, None].expand(T, K, H))
    y, h, gu = M.moonep_expert_ffn(c.plan, recv, c.home_w, c.slot_w, I, save=True)
    out = M.moonep_combine(c.plan, y)
    g_out = bf16(T, H, seed=64)
    g_y, dw = M.moonep_combine_bwd(c.plan, g_out, y)
    g_recv, g_gu = M.moonep_expert_ffn_bwd_data(c.plan, g_y, gu, c.home_w, c.slot_w, I)
    home, rep = M.moonep_expert_ffn_bwd_weight(c.plan, recv, g_y, h, g_gu)
    M.moonep_reduce_grad(c.plan, home, rep)
    g_q = M.moonep_dispatch_bwd(c.plan, g_recv)
    g_x, g_gamma = M.moonep_rmsnorm_bwd(g_q, stream, gamma, rstd, g_h=g_out)
    torch.cuda.synchronize()

    xs = q.double().requires_grad_()
    ws = c.home_w.double().requires_grad_()
    wt = torch.from_numpy(c.wt).cuda().double().requires_grad_()
    ids = torch.from_numpy(c.ids).cuda().long()
    ref = 0
    for k in range(K):
        w = ws[ids[:, k]]
        g, u, d = w[:, :I * H].view(T, I, H), w[:, I * H:2 * I * H].view(T, I, H), w[:, 2 * I * H:].view(T, H, I)
        a, _ = X.act((g * xs[:, None]).sum(2), "silu")
        hk = a * (u * xs[:, None]).sum(2)
        ref = ref + wt[:, k:k + 1] * (d * hk[:, None]).sum(2)
    ref.backward(g_out.double())

    def rel(a, b):
        return float((a.double() - b).norm() / b.norm())

    # each chain holds at most five roundings to bf16 of 2^-8 each at most; in the norm over
    # thousands of elements they add as squares: below sqrt(5) * 2^-8
    tol = 5 ** 0.5 * X.UB16
    assert rel(out, ref.detach()) <= tol
    assert rel(home, ws.grad) <= tol
    assert rel(dw, wt.grad) <= tol
    assert rel(g_q, xs.grad) <= tol
    # the norm's own backward, from what reached it
    hs = stream.double().requires_grad_()
    gm = gamma.double().requires_grad_()
    n = hs * (hs.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gm
    (n * g_q.double()).sum().backward()
    assert rel(g_x, hs.grad + g_out.double()) <= X.UB16
    assert rel(g_gamma, gm.grad) <= 1e-5
    assert torch.equal(stream, (x.float() + res.float()).to(torch.bfloat16))
