"""The router on the GPU, forward and backward, against the definition in 64 bits (tests/router_ref.py): ids exactly,
weights and gradients with bounds counted in roundings."""

import numpy as np
import pytest
import torch

import combine_top_id_amd as M
from tests import expert_ref as X
from tests import router_ref as R
from tests import w4_ref as W
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


def draw(T, E, dtype, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * scale).to(DT[dtype]).cuda()


def check(l, K, bias=None, score="softmax", groups=1, top_groups=1, normalize=True, scale=1.0):
    ids, w = M.moonep_router(l, K, bias=bias, score=score, groups=groups, top_groups=top_groups, normalize=normalize,
                             scale=scale)
    ln = l.float().cpu().numpy()
    ref = R.choose(ln, None if bias is None else bias.cpu().numpy(), score, K, groups, top_groups)
    got = ids.cpu().numpy()
    assert (got == ref).all(), f"ids differ in tokens {np.nonzero((got != ref).any(1))[0][:5]}"
    wr, d = R.weights(ln, ref, score, normalize, scale)
    err = np.abs(w.double().cpu().numpy() - wr)
    assert (err <= d).all(), f"weights off by {np.nanmax(err)}"
    check_bwd(l, ids, score, normalize, scale)
    return ids, w


def check_bwd(l, ids, score, normalize, scale, g=None):
    g = torch.randn(ids.shape, generator=torch.Generator().manual_seed(4)).cuda() if g is None else g
    out = torch.full_like(l, NAN)
    assert M.moonep_router_bwd(l, ids, g, score=score, normalize=normalize, scale=scale, g_logits=out) is out
    ref, d = R.gradient(l.float().cpu().numpy(), ids.cpu().numpy(), g.cpu().numpy(), score, normalize, scale)
    err = np.abs(out.double().cpu().numpy() - ref)
    u = X.UB16 if l.dtype == torch.bfloat16 else X.U32
    bad = ~(err <= d + u * (np.abs(ref) + d))
    assert not bad.any(), f"gradient: {bad.sum()} off, worst {err[bad].max() if bad.any() else 0}"
    return out


SHAPES = [(1, 1, 1), (3, 2, 1), (5, 3, 3), (130, 16, 2), (37, 17, 5), (64, 64, 6), (33, 65, 8), (20, 100, 32), (70, 256, 8),
          (9, 255, 32), (18, 257, 8), (50, 384, 8), (7, 385, 16), (6, 1000, 31), (5, 1024, 32), (1, 1024, 1)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_against_64_bits(score, normalize, dtype):
    for i, (T, E, K) in enumerate(SHAPES):
        say(f"router T={T} E={E} K={K} {score} {normalize} {dtype}")
        l = draw(T, E, dtype, 100 + i)
        check(l, K, score=score, normalize=normalize, scale=2.5)
        b = torch.randn(E, generator=torch.Generator().manual_seed(i)).cuda() * 0.1
        check(l, K, bias=b, score=score, normalize=normalize)


GROUPS = [(40, 256, 8, 8, 4), (9, 64, 6, 4, 2), (11, 64, 1, 64, 1), (13, 60, 7, 3, 2), (5, 1024, 32, 2, 1), (21, 21, 3, 7, 3),
          (8, 384, 8, 64, 5), (6, 1024, 16, 64, 1), (17, 12, 2, 12, 2), (10, 256, 8, 8, 8)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(score, dtype):
    for i, (T, E, K, n, top) in enumerate(GROUPS):
        say(f"router groups T={T} E={E} K={K} groups={n} top={top} {score} {dtype}")
        l = draw(T, E, dtype, 300 + i)
        check(l, K, score=score, groups=n, top_groups=top)
        b = torch.randn(E, generator=torch.Generator().manual_seed(i)).cuda() * 0.1
        check(l, K, bias=b, score=score, groups=n, top_groups=top, normalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_keys_go_to_the_lowest_index(score):
    for E, n, top in ((64, 1, 1), (256, 8, 3), (1000, 1, 1), (384, 4, 2)):
        l = draw(64, E, "bf16", E).sign() * 0.5
        l[0] = 0
        l[1, ::2], l[1, 1::2] = 0.0, -0.0
        check(l, 8, score=score, groups=n, top_groups=top)
        check(l, 8, score=score, groups=n, top_groups=top, bias=torch.zeros(E).cuda())
        check(l.float(), 8, score=score, bias=-0.0 * torch.ones(E).cuda(), groups=n, top_groups=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_keys_that_differ_by_less_than_32_bits_of_a_score_hold(score, bias):
    E = 256
    base = draw(64, 1, "fp32", 5).cpu()
    steps = torch.randint(-6, 7, (64, E), generator=torch.Generator().manual_seed(6))
    l = (base * (1 + steps * 2.0 ** -23)).cuda()                            # logits of a few ulp
    check(l, 8, score=score, bias=torch.full((E,), 0.25).cuda() if bias else None)
    check(l, 8, score=score, bias=torch.full((E,), 0.25).cuda() if bias else None, groups=8, top_groups=4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_masked_experts(score, normalize):
    for E, K, n, top in ((64, 6, 1, 1), (256, 8, 8, 4), (100, 32, 1, 1), (1024, 16, 4, 1)):
        l = draw(24, E, "fp32", 7 + E)
        mask = torch.rand(24, E, generator=torch.Generator().manual_seed(8)) < 0.5
        l[mask.cuda()] = -INF
        l[0] = -INF                                       # nothing left
        l[1] = NAN
        l[2, :] = -INF
        l[2, E - 1] = 0.3                                 # one expert
        l[3, :] = -INF
        l[3, 5:5 + K - 1] = 1.0                           # fewer than K
        l[4, 7] = INF
        l[5, 3], l[5, 9] = INF, INF
        l[6, :] = -INF
        l[6, 4] = INF
        l[7, 2] = NAN
        for b in (None, torch.linspace(-2, 3, E).cuda()):
            ids, w = check(l, K, bias=b, score=score, groups=n, top_groups=top, normalize=normalize)
            assert torch.isfinite(w).all() and (w[:2] == 0).all()


def test_biases_that_switch_experts_off_or_on():
    l = draw(16, 64, "fp32", 9)
    b = torch.zeros(64)
    b[3], b[10], b[20] = -INF, NAN, INF
    ids, _ = check(l, 8, bias=b.cuda(), score="sigmoid")
    assert (ids[:, 0] == 20).all() and not ((ids == 3) | (ids == 10)).any()
    ids, _ = check(l, 8, bias=torch.full((64,), NAN).cuda(), score="sigmoid")
    assert (ids == torch.arange(8, device="cuda", dtype=torch.int32)).all()


def test_scores_far_out():
    l = draw(32, 128, "fp32", 10, scale=40.0)
    for s in ("softmax", "sigmoid"):
        for shift in (0.0, -300.0, 300.0, -3e4):
            check(l + shift, 8, score=s)
        check(l, 8, score=s, normalize=False)


def test_of_no_tokens():
    ids, w = M.moonep_router(torch.empty(0, 64, device="cuda"), 8)
    assert ids.shape == (0, 8) and w.shape == (0, 8)
    assert M.moonep_router_bwd(torch.empty(0, 64, device="cuda"), ids, w).shape == (0, 64)


def test_ids_that_are_not_the_routers():
    l = draw(8, 64, "fp32", 11)
    ids = torch.randint(0, 64, (8, 6), dtype=torch.int32, generator=torch.Generator().manual_seed(12)).cuda()
    ids[0, 1] = ids[0, 0]                                 # named twice, three times, always
    ids[1, :3] = 5
    ids[2] = 63
    for s in ("softmax", "sigmoid"):
        for n in (True, False):
            check_bwd(l, ids, s, n, 1.5)
    ids[3, 2], ids[4, 0], ids[5] = -1, 64, 1 << 30        # outside
    for s in ("softmax", "sigmoid"):
        for n in (True, False):
            check_bwd(l, ids, s, n, 1.5)


def test_many_tokens():
    l = draw(40000, 64, "bf16", 13)
    ids, w = M.moonep_router(l, 6)
    for at in (0, 20000, 39990):
        a, b = M.moonep_router(l[at:at + 10].clone(), 6)
        assert torch.equal(ids[at:at + 10], a) and torch.equal(w[at:at + 10], b)
    key = l.float()
    top = torch.topk(key, 6, dim=1)[0]
    assert torch.equal(torch.gather(key, 1, ids.long()), top)
    g = M.moonep_router_bwd(l, ids, w)
    for at in (0, 20000, 39990):
        assert torch.equal(M.moonep_router_bwd(l[at:at + 10].clone(), ids[at:at + 10].clone(), w[at:at + 10].clone()), g[at:at + 10])


def test_logits_past_32_bits():
    T, E, K = 2_200_000, 1024, 4                       # 4.5 GB
    part = draw(1000, E, "bf16", 17)
    l = part.repeat(T // 1000, 1)
    for score, bias, groups, top in (("softmax", None, 1, 1), ("sigmoid", draw(1, E, "fp32", 18)[0], 4, 2)):
        kw = dict(bias=bias, score=score, groups=groups, top_groups=top)
        ids, w = M.moonep_router(l, K, **kw)
        a, b = M.moonep_router(part, K, **kw)
        assert torch.equal(ids.view(-1, 1000, K), a.expand(T // 1000, -1, -1))
        assert torch.equal(w.view(-1, 1000, K), b.expand(T // 1000, -1, -1))
        g = M.moonep_router_bwd(l, ids, w, score=score, normalize=False)
        assert torch.equal(g[-1000:], M.moonep_router_bwd(part, a, b, score=score, normalize=False))
        del g


def test_captured_and_on_another_stream():
    l, g = draw(300, 256, "fp32", 14), draw(300, 8, "fp32", 15)
    b = draw(1, 256, "fp32", 16)[0] * 0.1
    ids, w = torch.empty(300, 8, dtype=torch.int32, device="cuda"), torch.empty(300, 8, device="cuda")
    gl = torch.empty_like(l)

    def go(stream=None):
        M.moonep_router(l, 8, bias=b, score="sigmoid", groups=8, top_groups=4, ids=ids, w=w, stream=stream)
        M.moonep_router_bwd(l, ids, g, score="sigmoid", g_logits=gl, stream=stream)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for seed in range(3):
        l.copy_(draw(300, 256, "fp32", 40 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (ids, w, gl)]
        ids.fill_(-1), w.fill_(NAN), gl.fill_(NAN)
        go()
        assert all(torch.equal(x, y) for x, y in zip(got, (ids, w, gl)))
    new = draw(300, 256, "fp32", 50)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        l.copy_(new)
    go(side)
    side.synchronize()
    got = [t.clone() for t in (ids, w, gl)]
    go()
    assert all(torch.equal(x, y) for x, y in zip(got, (ids, w, gl)))


def test_a_layer_from_logits_to_their_gradient():
    """Router, plan, dispatch, experts in 4 bits, combine, and the gradient back to the logits."""
    Rk, E, K, S, slots, H, I = 4, 16, 2, 64, 4, 128, 64
    T = Rk * S
    l, x = draw(T, E, "fp32", 17), draw(T, H, "bf16", 18)
    w = draw(E, 3 * H * I, "bf16", 19, scale=H ** -0.5)
    ids, wt = M.moonep_router(l, K, score="sigmoid", scale=2.0)
    plan = M.moonep_plan(ids, wt, Rk, E, K, S, slots)
    recv = M.moonep_dispatch(plan, x)
    home = M.moonep_w4_pack(w, H, I)
    slot = M.moonep_prefetch_weight(plan, home.view(torch.bfloat16)).view(torch.uint8)
    y, _, _ = M.moonep_expert_ffn_w4(plan, recv, home, slot, I)
    out = M.moonep_combine(plan, y)
    assert M.moonep_plan_status(plan)["status"] == 0
    d_out = draw(T, H, "bf16", 20)
    _, dw = M.moonep_combine_bwd(plan, d_out, y, g_y=torch.empty_like(y))
    g = M.moonep_router_bwd(l, ids, dw, score="sigmoid", scale=2.0)
    # the same from the logits, each expert on each of its tokens, in 64 bits
    ln = l.cpu().double().requires_grad_(True)
    i = ids.cpu().long()
    s = torch.gather(torch.sigmoid(ln), 1, i)
    ww = 2.0 * s / s.sum(1, keepdim=True)
    dst = plan.dst_row.cpu().long()
    rows = y.cpu().double()[dst]
    ref = (ww[:, :, None] * rows).sum(1)
    X.close(out.cpu(), ref.detach(), 64 * X.U32 * (ww[:, :, None] * rows).abs().sum(1).detach(), X.UB16, "out")
    (ref * d_out.cpu().double()).sum().backward()
    mag = (rows.abs() * d_out.cpu().double().abs()[:, None]).sum((1, 2))[:, None] * 2.0
    X.close(g.cpu(), ln.grad, 512 * X.U32 * mag, X.U32, "logits' gradient")
    # and y, whose weights in 4 bits are what the experts multiplied
    for t in range(0, T, 37):
        for k in range(K):
            v = W.w4_slab(w[ids[t, k]].cpu(), H, I)
            _, _, h, _, _, dh = X.gate_up(x[t:t + 1].cpu(), v, H, I, "silu")
            yr, d = X.down(h, v, H, I)
            dd = X.slab(v, H, I)[2].abs()
            X.close(y[dst[t, k]].cpu()[None], yr, d + (dh + X.UB16 * (h.abs() + dh)) @ dd.T, X.UB16, "y")
