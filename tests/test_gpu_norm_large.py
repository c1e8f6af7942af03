"""The norm where its rows are more than the last-level cache holds and pass it by: random rows
with a residual (forward) and a gradient past the norm (backward), for each number of vectors
that a thread can hold.  A part of the rows alone takes the path through the caches, which
computes the same, bit for bit; the results of all are compared in 64 bits too.  Bounds as in
tests/test_gpu_norm.py."""

import pytest
import torch

import combine_top_id_amd as M
from tests import expert_ref as X
from tests.gpu_util import say
from tests.test_gpu_norm import U32, UB16, bf16, normed

pytestmark = pytest.mark.gpu
CACHE = 256 << 20

# 1, 2, 3, 4 and 8 vectors of 8 elements a thread, with threads that hold fewer
SHAPES = [(34000, 1000), (4800, 7136), (4100, 8456), (2900, 12296), (1100, 32768)]
SHAPES_Q8 = [(34300, 992), (4800, 7136), (4100, 8480), (2900, 12320), (1100, 32736)]
PARTS = 5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


def parts(T, H):
    """Row ranges whose calls stay in the cache."""
    assert T * H * 8 > CACHE and -(-T // PARTS) * H * 8 <= CACHE
    n = -(-T // PARTS)
    return [slice(k, min(k + n, T)) for k in range(0, T, n)]


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, res):
    say(f"norm past the caches T={T} H={H} res={res}")
    x, gamma = bf16(T, H, seed=21), bf16(H, seed=22)
    r = bf16(T, H, seed=23, scale=4.0) if res else None
    own = torch.empty_like(x)
    out, h, rstd = M.moonep_rmsnorm(x, gamma, 1e-5, res=r, h=own)
    assert h is own and torch.equal(h, (x.float() + r.float()).to(torch.bfloat16) if res else x)
    rel = (H + 8) * U32
    for s in parts(T, H):
        o, hs, rs = M.moonep_rmsnorm(x[s], gamma, 1e-5, res=r[s] if res else None)
        assert torch.equal(o, out[s]) and torch.equal(hs, h[s]) and torch.equal(rs, rstd[s])
        ref, rs = normed(h[s], gamma, 1e-5)
        X.close(rstd[s], rs, 0.0, rel, "rstd")
        X.close(out[s], ref, rel * ref.abs() + 1e-38, UB16, "out")
    if res:
        for over in (r.clone(), x.clone()):
            a, b = (x, over) if torch.equal(over, r) else (over, r)
            o2, h2, none = M.moonep_rmsnorm(a, gamma, 1e-5, res=b, h=over, stats=False)
            assert h2 is over and none is None and torch.equal(over, h) and torch.equal(o2, out)
    torch.cuda.synchronize()


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("T,H", SHAPES_Q8)
def test_eight_bits(T, H, res):
    say(f"norm q8 past the caches T={T} H={H} res={res}")
    x, gamma = bf16(T, H, seed=24), bf16(H, seed=25)
    r = bf16(T, H, seed=26, scale=3.0) if res else None
    rows, h, rstd = M.moonep_rmsnorm_q8(x, gamma, res=r, h=torch.empty_like(x))
    wide = M.moonep_q8_unpack(rows, H)
    assert torch.equal(h, (x.float() + r.float()).to(torch.bfloat16) if res else x)
    rel = (H + 8) * U32
    for s in parts(T, H):
        few, hs, rs = M.moonep_rmsnorm_q8(x[s], gamma, res=r[s] if res else None)
        assert torch.equal(few, rows[s]) and torch.equal(hs, h[s]) and torch.equal(rs, rstd[s])
        ref, rs = normed(h[s], gamma, 1e-6)
        X.close(rstd[s], rs, 0.0, rel, "rstd")
        scale = torch.exp2(rows[s, H:H + H // 32].double() - 127).repeat_interleave(32, 1)
        step = torch.maximum(ref.abs() * 2 ** -4, scale * 2 ** -10)
        assert ((wide[s].double() - ref).abs() <= step * (1 + 16 * rel) + rel * ref.abs()).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("more", [False, True])
@pytest.mark.parametrize("T,H", SHAPES)
def test_backward(T, H, more):
    say(f"norm bwd past the caches T={T} H={H} g_h={more}")
    h, gamma, g = bf16(T, H, seed=27, scale=2.0), bf16(H, seed=28), bf16(T, H, seed=29)
    g_h = bf16(T, H, seed=30) if more else None
    rstd = torch.cat([normed(h[s], gamma, 1e-6)[1].float() for s in parts(T, H)])
    g_x, g_gamma = M.moonep_rmsnorm_bwd(g, h, gamma, rstd, g_h=g_h)
    total, size = 0, 0
    for s in parts(T, H):
        few, _ = M.moonep_rmsnorm_bwd(g[s], h[s], gamma, rstd[s], g_h=g_h[s] if more else None)
        assert torch.equal(few, g_x[s])
        rs = rstd[s].double()[:, None]
        xhat, gg = h[s].double() * rs, g[s].double() * gamma.double()
        dot = (gg * xhat).mean(1, keepdim=True)
        ref = rs * (gg - xhat * dot)
        bound = rs * xhat.abs() * (gg * xhat).abs().mean(1, keepdim=True) * (H + 8) * U32 \
            + 8 * U32 * rs * (gg.abs() + (xhat * dot).abs()) + 1e-38
        if more:
            ref = ref + g_h[s].double()
        X.close(g_x[s], ref, bound + U32 * ref.abs(), UB16, "g_x")
        total = total + (g[s].double() * xhat).sum(0)
        size = size + (g[s].double() * xhat).abs().sum(0)
    X.close(g_gamma, total, (T + 4) * U32 * size + 1e-38, U32, "g_gamma")
    for k in range(3 if more else 2):
        a = [g.clone(), h.clone(), g_h.clone() if more else None]
        o, gm = M.moonep_rmsnorm_bwd(a[0], a[1], gamma, rstd, g_h=a[2], g_x=a[k])
        assert o is a[k] and torch.equal(o, g_x) and torch.equal(gm, g_gamma)
    torch.cuda.synchronize()
