"""The root-mean-square norm on the GPU: bf16 and 8-bit outputs, the expansion of 8-bit rows
and the backward pass, against the formulas in 64 bits.

Bounds: a sum of n terms in fp32 is off by at most n * 2^-24 of the terms' magnitudes, so
rstd is off by (n + 8) * 2^-24 of itself; the few products after it by 2^-24 each; a
rounding to bf16 by 2^-8 and to e4m3 by 2^-4 of the value (2^-10 of the block's scale below
the smallest normal number)."""

import pytest
import torch

import combine_top_id_amd as M
from tests import expert_ref as X
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
U32, UB16 = X.U32, X.UB16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


def bf16(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def normed(h, gamma, eps):
    v = h.double()
    rstd = (v.square().mean(1) + eps).rsqrt()
    return v * rstd[:, None] * gamma.double(), rstd


SHAPES = [(1, 8), (3, 64), (1, 7168), (64, 7168), (1001, 1000), (5, 520), (700, 2048), (2, 32768), (7, 12296),
          (3000, 128), (130, 4104), (9, 24576)]


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_against_64_bits(T, H, res):
    say(f"norm T={T} H={H} res={res}")
    x, gamma = bf16(T, H, seed=1), bf16(H, seed=2)
    r = bf16(T, H, seed=3, scale=4.0) if res else None
    out, h, rstd = M.moonep_rmsnorm(x, gamma, 1e-5, res=r)
    assert torch.equal(h, (x.float() + r.float()).to(torch.bfloat16) if res else x)
    ref, rs = normed(h, gamma, 1e-5)
    rel = (H + 8) * U32
    X.close(rstd, rs, 0.0, rel, "rstd")
    X.close(out, ref, rel * ref.abs() + 1e-38, UB16, "out")
    # without statistics; the stream over the residual, in place
    if res:
        over = r.clone()
        o2, h2, none = M.moonep_rmsnorm(x, gamma, 1e-5, res=over, h=over, stats=False)
        assert h2 is over and none is None and torch.equal(over, h) and torch.equal(o2, out)
        over = x.clone()
        o2, h2, _ = M.moonep_rmsnorm(over, gamma, 1e-5, res=r, h=over)
        assert torch.equal(over, h) and torch.equal(o2, out)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,H", [(1, 32), (64, 7168), (33, 96), (1000, 1024), (2, 32768), (5, 4128)])
def test_eight_bits(T, H):
    say(f"norm q8 T={T} H={H}")
    x, r = bf16(T, H, seed=4), bf16(T, H, seed=5, scale=3.0)
    gamma = bf16(H, seed=6)
    x[0, :32], r[0, :32] = 0, 0                      # a block of zeros
    if H > 64:
        gamma[32:64] *= 1e-4                          # a block with another scale
        gamma[40] = 0.0                               # and elements far below it
        gamma[41] *= 1e-3
    out, h, rstd = M.moonep_rmsnorm(x, gamma, res=r)
    rows, h8, rstd8 = M.moonep_rmsnorm_q8(x, gamma, res=r)
    rb = M.moonep_q8_row_bytes(H)
    assert rows.shape == (T, rb) and torch.equal(h8, h) and torch.equal(rstd8, rstd)
    ref, _ = normed(h, gamma, 1e-6)
    # exp2 in 64 bits is exact for whole numbers (torch.ldexp's power is not, on this device)
    scale = torch.exp2(rows[:, H:H + H // 32].double() - 127)
    assert (torch.frexp(scale).mantissa == 0.5).all()
    assert (rows[:, H + H // 32:] == 0).all()
    top = ref.view(T, -1, 32).abs().amax(2)
    rel = (H + 8) * U32
    assert (top <= 448 * scale * (1 + rel)).all()
    small = (top * 2 > 448 * scale * (1 - rel)) | (top == 0)      # half the scale would not do
    assert small.all()
    code = rows[:, :H].contiguous().view(torch.float8_e4m3fn).double().view(T, -1, 32)
    back = (code * scale[:, :, None]).view(T, H)
    step = torch.maximum(ref.abs() * 2 ** -4, (scale * 2 ** -10).repeat_interleave(32, 1))
    assert ((back - ref).abs() <= step * (1 + 16 * rel) + rel * ref.abs()).all()
    wide = M.moonep_q8_unpack(rows, H)
    assert torch.equal(wide.double(), back)            # exact
    assert torch.equal(M.moonep_q8_unpack(rows.view(torch.bfloat16), H), wide)
    torch.cuda.synchronize()


def test_every_code_and_scale_expands():
    """All 256 codes under a range of scales, against torch's own table of e4m3."""
    say("q8 expand")
    H = 256
    rb = M.moonep_q8_row_bytes(H)
    scales = list(range(20, 240, 20)) + [1, 127, 254]
    rows = torch.zeros(len(scales), rb, dtype=torch.uint8, device="cuda")
    rows[:, :H] = torch.arange(256, dtype=torch.uint8, device="cuda")
    for i, s in enumerate(scales):
        rows[i, H:H + H // 32] = s
    got = M.moonep_q8_unpack(rows, H).float()
    code = rows[:, :H].contiguous().view(torch.float8_e4m3fn).double()
    ref = code * torch.exp2(torch.tensor(scales, device="cuda", dtype=torch.float64)[:, None] - 127)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    ok = ~torch.isnan(ref)
    small = ref.abs() < 2.0 ** -126                    # below bf16's normal numbers: within its last step
    assert torch.equal(got.double()[ok & ~small & (ref.abs() < 3e38)], ref[ok & ~small & (ref.abs() < 3e38)])
    assert ((got.double() - ref).abs()[ok & small] <= 2.0 ** -133).all()
    torch.cuda.synchronize()


def test_special_rows():
    """Zero rows, a NaN, an infinity, and magnitudes whose squares are far from one: each stays
    in its row."""
    say("norm special")
    H = 1024
    x = bf16(6, H, seed=7)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 6] = float("inf")
    x[4] *= 1e15
    x[5] *= 1e-15
    gamma = bf16(H, seed=8)
    out, _, rstd = M.moonep_rmsnorm(x, gamma, 1e-6)
    wide = M.moonep_q8_unpack(M.moonep_rmsnorm_q8(x, gamma, 1e-6)[0], H)
    ref, _ = normed(x, gamma, 1e-6)
    for t in (0, 1, 4, 5):
        X.close(out[t], ref[t], (H + 8) * U32 * ref[t].abs() + 1e-38, UB16, f"row {t}")
        assert torch.isfinite(wide[t]).all()
    assert (out[1] == 0).all() and (wide[1] == 0).all() and abs(float(rstd[1]) - 1e3) < 1e-2
    assert torch.isnan(out[2]).all() and torch.isnan(wide[2]).all()
    assert torch.isnan(out[3, 6]) and (out[3, :6] == 0).all()       # everything else over an infinite norm
    assert torch.isnan(wide[3, 6]) and (wide[3, :6] == 0).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("more", [False, True])
@pytest.mark.parametrize("T,H", SHAPES)
def test_backward_against_64_bits(T, H, more):
    say(f"norm bwd T={T} H={H} g_h={more}")
    h, gamma, g = bf16(T, H, seed=9, scale=2.0), bf16(H, seed=10), bf16(T, H, seed=11)
    g_h = bf16(T, H, seed=12) if more else None
    rstd = normed(h, gamma, 1e-6)[1].float()
    g_x, g_gamma = M.moonep_rmsnorm_bwd(g, h, gamma, rstd, g_h=g_h)
    rs = rstd.double()[:, None]
    xhat, gg = h.double() * rs, g.double() * gamma.double()
    dot = (gg * xhat).mean(1, keepdim=True)
    ref = rs * (gg - xhat * dot)
    # the mean: H terms; each of the terms that follow has a few roundings of its own
    bound = rs * xhat.abs() * (gg * xhat).abs().mean(1, keepdim=True) * (H + 8) * U32 \
        + 8 * U32 * rs * (gg.abs() + (xhat * dot).abs()) + 1e-38
    if more:
        ref = ref + g_h.double()
    X.close(g_x, ref, bound + U32 * ref.abs(), UB16, "g_x")
    X.close(g_gamma, (g.double() * xhat).sum(0), (T + 4) * U32 * (g.double() * xhat).abs().sum(0) + 1e-38, U32,
            "g_gamma")
    # in place over each input, and with a workspace of the caller's
    ws = torch.empty(M.lib().moonep_rmsnorm_bwd_workspace(T, H), dtype=torch.uint8, device="cuda")
    for k in range(3 if more else 2):
        a = [g.clone(), h.clone(), g_h.clone() if more else None]
        o, gm = M.moonep_rmsnorm_bwd(a[0], a[1], gamma, rstd, g_h=a[2], g_x=a[k], workspace=ws)
        assert o is a[k] and torch.equal(o, g_x) and torch.equal(gm, g_gamma)
    torch.cuda.synchronize()


def test_backward_against_differences():
    """Central differences of the 64-bit norm along random directions; what is left is the
    rounding of g_x to bf16."""
    say("norm differences")
    T, H = 20, 256
    h, gamma, g = bf16(T, H, seed=13), bf16(H, seed=14), bf16(T, H, seed=15)
    _, _, rstd = M.moonep_rmsnorm(h, gamma, 1e-6)
    g_x, g_gamma = M.moonep_rmsnorm_bwd(g, h, gamma, rstd)
    f = lambda a, b: float((normed(a, b, 1e-6)[0] * g.double()).sum())  # noqa: E731
    dx, dg, e = g_x.double().sign(), g_gamma.double().sign(), 1e-6
    num = (f(h.double() + e * dx, gamma) - f(h.double() - e * dx, gamma)) / (2 * e)
    assert abs(num - float(g_x.double().abs().sum())) <= UB16 * num
    num = (f(h, gamma.double() + e * dg) - f(h, gamma.double() - e * dg)) / (2 * e)
    assert abs(num - float(g_gamma.double().abs().sum())) <= 1e-4 * num


def test_no_rows():
    say("norm T=0")
    gamma = bf16(64, seed=16)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    out, h, rstd = M.moonep_rmsnorm(x, gamma)
    assert out.shape == (0, 64) and rstd.numel() == 0
    rows, _, _ = M.moonep_rmsnorm_q8(x, gamma)
    assert M.moonep_q8_unpack(rows, 64).shape == (0, 64)
    g_gamma = torch.full((64,), float("nan"), device="cuda")
    g_x, g_gamma = M.moonep_rmsnorm_bwd(x, x, gamma, rstd, g_gamma=g_gamma)
    assert g_x.shape == (0, 64) and (g_gamma == 0).all()
    torch.cuda.synchronize()


def test_capture_and_another_stream():
    """The norm, both forms, and its backward captured and replayed on new inputs, on a stream
    of their own, against eager calls."""
    say("norm capture")
    T, H = 300, 1024
    x, r, g = (bf16(T, H, seed=k) for k in (17, 18, 19))
    gamma = bf16(H, seed=20)
    ws = torch.empty(M.lib().moonep_rmsnorm_bwd_workspace(T, H), dtype=torch.uint8, device="cuda")
    o = dict(out=torch.empty_like(x), h=torch.empty_like(x), rstd=torch.empty(T, device="cuda"),
             rows=torch.empty(T, M.moonep_q8_row_bytes(H), dtype=torch.uint8, device="cuda"),
             wide=torch.empty_like(x), g_x=torch.empty_like(x), g_gamma=torch.empty(H, device="cuda"))

    def step():
        M.moonep_rmsnorm(x, gamma, res=r, out=o["out"], h=o["h"], rstd=o["rstd"])
        M.moonep_rmsnorm_q8(x, gamma, res=r, rows=o["rows"], h=o["h"], rstd=o["rstd"])
        M.moonep_q8_unpack(o["rows"], H, out=o["wide"])
        M.moonep_rmsnorm_bwd(g, o["h"], gamma, o["rstd"], g_h=g, g_x=o["g_x"], g_gamma=o["g_gamma"], workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for k in range(3):
        x.copy_(bf16(T, H, seed=100 + k))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in o.items()}
        step()
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], o[n]), n


def test_rows_past_32_bits():
    """More than 2^31 elements: the last rows, as the same rows give alone, and gradients of
    those rows only."""
    say("norm large")
    T, H = 300000, 7168
    assert T * H > 2 ** 31
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-50:] = bf16(50, H, seed=81)
    gamma = bf16(H, seed=82)
    tail = x[-50:].contiguous()
    out, _, rstd = M.moonep_rmsnorm(x, gamma)
    few, _, few_rstd = M.moonep_rmsnorm(tail, gamma)
    assert torch.equal(out[-50:], few) and torch.equal(rstd[-50:], few_rstd) and (out[:-50] == 0).all()
    rows, _, _ = M.moonep_rmsnorm_q8(x, gamma)
    few_rows, _, _ = M.moonep_rmsnorm_q8(tail, gamma)
    assert torch.equal(rows[-50:], few_rows)
    back = M.moonep_q8_unpack(rows, H)
    assert torch.equal(back[-50:], M.moonep_q8_unpack(few_rows, H)) and (back[:-50] == 0).all()
    del rows, back
    g_x, g_gamma = M.moonep_rmsnorm_bwd(out, x, gamma, rstd)
    few_g, few_gamma = M.moonep_rmsnorm_bwd(few, tail, gamma, few_rstd)
    assert torch.equal(g_x[-50:], few_g) and (g_x[:-50] == 0).all()
    # the rows before add zeros, in another order of at most 50 nonzero terms each
    n = tail.double() * few_rstd.double()[:, None]
    mag = (few.double() * n).abs().sum(0)
    assert ((g_gamma.double() - few_gamma.double()).abs() <= 2 * 52 * 2.0 ** -24 * mag).all()
    torch.cuda.synchronize()
