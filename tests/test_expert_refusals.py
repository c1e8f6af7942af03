"""What the expert block's calls refuse, found on the host before anything is launched: the
C entries with addresses that are never followed, and the binding with CPU tensors.  Also
the 64-bit references of the GPU tests against differences."""

import ctypes
import inspect
import os

import pytest
import torch

import combine_top_id_amd as M
from combine_top_id_amd.moonep import PlanDesc
from tests import expert_ref as X

EINVAL, ELIMIT, EPLAN, EHIP, EALIGN = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        pytest.fail("libmoonep.so is not built (run __graft_entry__.build())")
    return M.lib()


@pytest.fixture
def desc(lib):
    d = PlanDesc()
    d.magic = 0x4D4F4E45
    d.dev = 256
    d.sz = M.moonep_query(4, 16, 2, 4, 4)
    return d


P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)


def ffn(lib, d, recv=P, H=64, I=32, act=0, home=P, slot=P, W_el=None, gu=None, h=P, y=P):
    return lib.moonep_expert_ffn(ctypes.byref(d) if d else None, recv, H, I, act, home, slot,
                                 3 * H * I if W_el is None else W_el, gu, h, y, None)


def data(lib, d, g_y=P, gu=P, H=64, I=32, act=0, home=P, slot=P, W_el=None, g_gu=P, g_recv=P):
    return lib.moonep_expert_ffn_bwd_data(ctypes.byref(d) if d else None, g_y, gu, H, I, act, home, slot,
                                          3 * H * I if W_el is None else W_el, g_gu, g_recv, None)


def weight(lib, d, recv=P, g_y=P, h=P, g_gu=P, H=64, I=32, home=P, rep=P, G_el=None, acc=0):
    return lib.moonep_expert_ffn_bwd_weight(ctypes.byref(d) if d else None, recv, g_y, h, g_gu, H, I, home, rep,
                                            3 * H * I if G_el is None else G_el, acc, None)


@pytest.mark.parametrize("call,ptrs", [
    (ffn, ["recv", "home", "slot", "h", "y"]),
    (data, ["g_y", "gu", "home", "slot", "g_gu", "g_recv"]),
    (weight, ["recv", "g_y", "h", "g_gu", "home", "rep"])])
def test_experts_refuse(lib, desc, call, ptrs):
    assert call(lib, None) == EPLAN
    assert call(lib, PlanDesc()) == EPLAN
    for p in ptrs:
        assert call(lib, desc, **{p: None}) == EINVAL, p
        assert call(lib, desc, **{p: ODD}) == EALIGN, p
    for bad in (dict(H=0), dict(H=-8), dict(H=60), dict(I=0), dict(I=12), dict(I=-16)):
        assert call(lib, desc, **bad) == EINVAL, bad
    assert call(lib, desc, H=32776) == ELIMIT
    assert call(lib, desc, I=32776) == ELIMIT
    assert call(lib, desc, H=32768, I=32768) == ELIMIT      # an expert's matrix beyond 31 bits of bytes
    pitch = "G_el" if call is weight else "W_el"
    assert call(lib, desc, **{pitch: 3 * 64 * 32 - 8}) == EINVAL
    assert call(lib, desc, **{pitch: 3 * 64 * 32 + 2}) == EINVAL
    if call is weight:
        assert call(lib, desc, acc=2) == EINVAL
    else:
        assert call(lib, desc, act=2) == EINVAL and call(lib, desc, act=-1) == EINVAL
    desc.sz.NvS += 16
    assert call(lib, desc) == EPLAN


def test_forward_refuses_a_misaligned_save_buffer(lib, desc):
    assert ffn(lib, desc, gu=ODD) == EALIGN


def test_more_tiles_than_32_bits(lib, desc):
    # a plan of 2^30 assignments and rows of 32768 columns
    desc.sz = M.moonep_query(64, 64, 1, 1 << 24, 0)
    assert ffn(lib, desc, H=32768, I=64, slot=None) == ELIMIT


def test_norm_refuses(lib):
    f = lambda x=P, res=None, g=P, eps=1e-6, T=4, H=64, out=P, h=None, rstd=None, n="moonep_rmsnorm": getattr(  # noqa
        lib, n)(x, res, g, eps, T, H, out, h, rstd, None)
    for n in ("moonep_rmsnorm", "moonep_rmsnorm_q8"):
        for p in ("x", "g", "out"):
            assert f(n=n, **{p: None}) == EINVAL
        for p in ("x", "res", "g", "out", "h"):
            assert f(n=n, **{p: ODD}) == EALIGN
        assert f(n=n, rstd=ctypes.c_void_p(258)) == EALIGN
        assert f(n=n, H=0) == EINVAL and f(n=n, H=-64) == EINVAL and f(n=n, H=36) == EINVAL
        assert f(n=n, T=-1) == EINVAL
        assert f(n=n, eps=-1e-6) == EINVAL and f(n=n, eps=float("nan")) == EINVAL
        assert f(n=n, H=32800) == ELIMIT and f(n=n, T=1 << 31) == ELIMIT
        assert f(n=n, x=None, g=None, out=None, T=0) == 0          # nothing to do
    assert f(n="moonep_rmsnorm_q8", H=72) == EINVAL                # not whole blocks
    u = lambda rows=P, N=4, H=64, out=P: lib.moonep_q8_unpack(rows, N, H, out, None)  # noqa: E731
    assert u(rows=None) == EINVAL and u(out=None) == EINVAL and u(N=-1) == EINVAL and u(H=40) == EINVAL
    assert u(rows=ODD) == EALIGN and u(out=ODD) == EALIGN
    assert u(H=32800) == ELIMIT and u(N=1 << 31) == ELIMIT and u(rows=None, N=0) == 0
    b = lambda g=P, h=P, gm=P, rs=P, gh=None, T=4, H=64, ws=P, gx=P, gg=P: lib.moonep_rmsnorm_bwd(  # noqa: E731
        g, h, gm, rs, gh, T, H, ws, gx, gg, None)
    for p in ("g", "h", "gm", "rs", "ws", "gx", "gg"):
        assert b(**{p: None}) == EINVAL, p
    for p in ("g", "h", "gm", "gh", "ws", "gx", "gg"):
        assert b(**{p: ODD}) == EALIGN, p
    assert b(rs=ctypes.c_void_p(258)) == EALIGN and b(ws=ctypes.c_void_p(272)) == EALIGN
    assert b(H=4) == EINVAL and b(T=-1) == EINVAL and b(H=32776) == ELIMIT and b(T=1 << 31) == ELIMIT


def test_sizes(lib):
    assert [M.moonep_q8_row_bytes(h) for h in (32, 512, 7168, 96)] == [48, 528, 7392, 112]
    for h in (32, 64, 96, 7168, 32768):
        b = M.moonep_q8_row_bytes(h)
        assert b % 16 == 0 and h + h // 32 <= b < h + h // 32 + 16
    for h in (0, -32, 8, 100):
        with pytest.raises(M.MoonepError, match="invalid"):
            M.moonep_q8_row_bytes(h)
    with pytest.raises(M.MoonepError, match="limits"):
        M.moonep_q8_row_bytes(32800)
    assert lib.moonep_rmsnorm_bwd_workspace(0, 64) == 0
    assert lib.moonep_rmsnorm_bwd_workspace(3, 64) >= 64 * 4
    assert lib.moonep_rmsnorm_bwd_workspace(-1, 64) == EINVAL
    assert lib.moonep_rmsnorm_bwd_workspace(1, 12) == EINVAL
    assert lib.moonep_rmsnorm_bwd_workspace(1, 32776) == ELIMIT


def test_binding_refuses_cpu_tensors(lib):
    x, g = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for f in (lambda: M.moonep_rmsnorm(x, g), lambda: M.moonep_rmsnorm_q8(x, g),
              lambda: M.moonep_q8_unpack(torch.zeros(4, 80, dtype=torch.uint8), 64),
              lambda: M.moonep_rmsnorm_bwd(x, x, g, torch.ones(4))):
        with pytest.raises(M.MoonepError, match="GPU tensor"):
            f()
    plan = M.Plan(M.moonep_query(4, 16, 2, 4, 4), torch.zeros(4, dtype=torch.int32), None)
    rows = plan.sz.recv_rows
    recv, w, s = torch.zeros(rows, 64, dtype=torch.bfloat16), torch.zeros(16, 6144, dtype=torch.bfloat16), \
        torch.zeros(4, 4, 6144, dtype=torch.bfloat16)
    for f in (lambda: M.moonep_expert_ffn(plan, recv, w, s, 32),
              lambda: M.moonep_expert_ffn_bwd_data(plan, recv, recv, w, s, 32),
              lambda: M.moonep_expert_ffn_bwd_weight(plan, recv, recv, recv[:, :32], recv)):
        with pytest.raises(M.MoonepError, match="GPU tensor"):
            f()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_reference_gradients_against_differences(kind):
    """The 64-bit gradients that the GPU tests compare with, against central differences."""
    torch.manual_seed(3)
    H, I, n = 6, 5, 7
    x, w, g_y = (torch.randn(*s, dtype=torch.float64) for s in ((n, H), (3 * H * I,), (n, H)))

    def loss(x, w):
        g, u, d = X.slab(w, H, I)
        a, _ = X.act(x @ g.T, kind)
        return float((((a * (x @ u.T)) @ d.T) * g_y).sum())

    z, v, h, *_ = X.gate_up(x, w, H, I, kind)
    gg, gu, *_ = X.back_gu(g_y, torch.cat([z, v], 1), w, H, I, kind)
    g_gu = torch.cat([gg, gu], 1)
    g_x, _ = X.back_rows(g_gu, w, H, I)
    g_w = torch.cat([(g_gu.T @ x).reshape(-1), (g_y.T @ h).reshape(-1)])
    e = 1e-6
    for t, g in ((x, g_x), (w, g_w)):
        for i in range(0, t.numel(), 5):
            d = torch.zeros_like(t).view(-1)
            d[i] = e
            d = d.view_as(t)
            num = (loss(x + d, w) - loss(x - d, w)) / (2 * e) if t is x else (loss(x, w + d) - loss(x, w - d)) / (2 * e)
            assert abs(num - float(g.reshape(-1)[i])) <= 1e-7 * (1 + abs(num))


def test_stream_is_given_by_name():
    # the binding allocates on it before anything else, so it has to know it from the rest
    for f in (M.moonep_expert_ffn, M.moonep_expert_ffn_bwd_data, M.moonep_expert_ffn_bwd_weight, M.moonep_rmsnorm,
              M.moonep_rmsnorm_q8, M.moonep_q8_unpack, M.moonep_rmsnorm_bwd):
        assert inspect.signature(f).parameters["stream"].kind is inspect.Parameter.KEYWORD_ONLY
