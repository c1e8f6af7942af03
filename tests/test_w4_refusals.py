"""What the calls of the experts in 4 bits refuse, found on the host before anything is launched, and the
64-bit references of their GPU tests against known values."""

import ctypes
import inspect
import os

import pytest
import torch

import combine_top_id_amd as M
from combine_top_id_amd.moonep import PlanDesc
from tests import w4_ref as W

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
    d.dev = 1 << 44
    d.sz = M.moonep_query(4, 16, 2, 4, 4)
    return d


def at(k):
    return ctypes.c_void_p(k << 40)           # never followed


ODD = ctypes.c_void_p((9 << 40) + 8)
H0, I0 = 64, 32


def f16(lib, d, recv=at(1), H=H0, I=I0, act=0, home=at(2), slot=at(3), pitch=None, gu=at(4), h=at(5), y=at(6)):
    pitch = lib.moonep_w4_slab_bytes(H0, I0) if pitch is None else pitch
    return lib.moonep_expert_ffn_w4(ctypes.byref(d) if d else None, recv, H, I, act, home, slot, pitch, gu, h, y, None)


def f8(lib, d, recv=at(1), H=H0, I=I0, act=0, home=at(2), slot=at(3), pitch=None, h=at(5), y=at(6)):
    pitch = lib.moonep_w4_slab_bytes(H0, I0) if pitch is None else pitch
    return lib.moonep_expert_ffn_w4q8(ctypes.byref(d) if d else None, recv, H, I, act, home, slot, pitch, h, y, None)


def test_slab_bytes(lib):
    f = lib.moonep_w4_slab_bytes
    # 64 rows times 128 k are 4352 bytes; gate and up fill up I to 32, down H to 64, k to 128
    assert f(128, 64) == (2 * 1 + 2 * 1) * 4352
    assert f(7168, 2048) == 3 * 7168 * 2048 * 17 // 32
    assert f(8, 8) == 2 * 4352
    assert f(1000, 680) == (22 * 8 + 16 * 6) * 4352
    for h, i in ((0, 8), (8, 0), (12, 8), (8, 12), (-8, 8), (8, -8)):
        assert f(h, i) == EINVAL
    assert f(32776, 8) == ELIMIT and f(8, 32776) == ELIMIT and f(32768, 32768) > 0
    with pytest.raises(M.MoonepError, match="invalid"):
        M.moonep_w4_slab_bytes(12, 8)


@pytest.mark.parametrize("call", ["moonep_w4_pack", "moonep_w4_unpack"])
def test_packing_refuses(lib, call):
    b = lib.moonep_w4_slab_bytes(H0, I0)
    el = 3 * H0 * I0

    def f(w=at(1), W_el=el, n=2, H=H0, I=I0, w4=at(2), pitch=b):
        if call == "moonep_w4_pack":
            return lib.moonep_w4_pack(w, W_el, n, H, I, w4, pitch, None)
        return lib.moonep_w4_unpack(w4, pitch, n, H, I, w, W_el, None)

    assert f(w=None) == EINVAL and f(w4=None) == EINVAL
    assert f(w=ODD) == EALIGN and f(w4=ODD) == EALIGN
    assert f(W_el=el - 8) == EINVAL and f(W_el=el + 4) == EINVAL
    assert f(pitch=b - 16) == EINVAL and f(pitch=b + 8) == EINVAL
    assert f(H=60) == EINVAL and f(I=0) == EINVAL and f(H=-8) == EINVAL and f(I=32776) == ELIMIT
    assert f(n=-1) == EINVAL and f(n=1 << 31) == ELIMIT and f(n=0, w=None, w4=None) == 0
    assert f(w4=at(1)) == EINVAL                                     # overlaps
    assert f(w4=ctypes.c_void_p((1 << 40) + el * 4 - 16)) == EINVAL  # with the last slab
    assert f(w=at(2), w4=ctypes.c_void_p((2 << 40) - b)) == EINVAL


@pytest.mark.parametrize("call,ptrs", [(f16, ["recv", "home", "slot", "h", "y"]), (f8, ["recv", "home", "slot", "h", "y"])])
def test_experts_refuse(lib, desc, call, ptrs):
    assert call(lib, None) == EPLAN
    assert call(lib, PlanDesc()) == EPLAN
    for p in ptrs:
        assert call(lib, desc, **{p: None}) == EINVAL, p
        assert call(lib, desc, **{p: ODD}) == EALIGN, p
    big = 1 << 40
    for bad in (dict(H=0), dict(H=-32), dict(H=60), dict(I=0), dict(I=12), dict(I=-32)):
        assert call(lib, desc, pitch=big, **bad) == EINVAL, bad
    assert call(lib, desc, H=32800, pitch=big) == ELIMIT
    assert call(lib, desc, I=32800, pitch=big) == ELIMIT
    b = lib.moonep_w4_slab_bytes(H0, I0)
    assert call(lib, desc, pitch=b - 16) == EINVAL and call(lib, desc, pitch=b + 8) == EINVAL
    assert call(lib, desc, pitch=0) == EINVAL and call(lib, desc, pitch=-16) == EINVAL
    assert call(lib, desc, act=2) == EINVAL and call(lib, desc, act=-1) == EINVAL
    # outputs over inputs, weights, the plan, each other
    for out, others in (("h", (1, 2, 3, 6, 16)), ("y", (1, 2, 3, 5, 16))):
        for o in others:
            assert call(lib, desc, **{out: at(o)}) == EINVAL, (out, o)
    assert call(lib, desc, h=ctypes.c_void_p((2 << 40) + 15 * b)) == EINVAL       # the last expert's slab
    assert call(lib, desc, y=ctypes.c_void_p((3 << 40) + 15 * b)) == EINVAL       # the last slot's
    desc.sz.NvS += 16
    assert call(lib, desc) == EPLAN


def test_saved_rows_are_checked(lib, desc):
    assert f16(lib, desc, gu=ODD) == EALIGN
    for o in (1, 2, 3, 5, 6, 16):
        assert f16(lib, desc, gu=at(o)) == EINVAL, o


def test_8_bit_rows_are_whole_blocks(lib, desc):
    assert f8(lib, desc, H=72, pitch=1 << 40) == EINVAL and f8(lib, desc, I=40, pitch=1 << 40) == EINVAL


def test_more_tiles_than_32_bits(lib, desc):
    desc.sz = M.moonep_query(64, 64, 1, 1 << 24, 0)          # 2^30 assignments
    assert f16(lib, desc, H=32768, I=64, slot=None, pitch=1 << 40) == ELIMIT
    assert f8(lib, desc, H=32768, I=64, slot=None, pitch=1 << 40) == ELIMIT


def test_binding_refuses(lib):
    w = torch.zeros(2, 3 * 64 * 32, dtype=torch.bfloat16)
    w4 = torch.zeros(16, M.moonep_w4_slab_bytes(64, 32), dtype=torch.uint8)
    for f in (lambda: M.moonep_w4_pack(w, 64, 32), lambda: M.moonep_w4_unpack(w4, 64, 32)):
        with pytest.raises(M.MoonepError, match="GPU tensor"):
            f()
    plan = M.Plan(M.moonep_query(4, 16, 2, 4, 4), torch.zeros(4, dtype=torch.int32), None)
    rows = plan.sz.recv_rows
    s4 = torch.zeros(4, 4, w4.shape[1], dtype=torch.uint8)
    for f in (lambda: M.moonep_expert_ffn_w4(plan, torch.zeros(rows, 64, dtype=torch.bfloat16), w4, s4, 32),
              lambda: M.moonep_expert_ffn_w4q8(plan, torch.zeros(rows, 80, dtype=torch.uint8), w4, s4, 64, 32)):
        with pytest.raises(M.MoonepError, match="GPU tensor"):
            f()
    for f in (M.moonep_w4_pack, M.moonep_w4_unpack, M.moonep_expert_ffn_w4, M.moonep_expert_ffn_w4q8):
        assert inspect.signature(f).parameters["stream"].kind is inspect.Parameter.KEYWORD_ONLY


def test_the_references_themselves():
    m = torch.tensor([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.3, 4.9, 5.1] + [0.0] * 20 + [7.0, 1.0]])
    want = [6, 0, 1, 1, 2, 2, 4, 4, 0, -0.5, 4, 6] + [0] * 20 + [8, 1]      # the short group: steps of 0.5, 1 (to 4), 2, 4 * 2
    assert W.w4(m)[0].tolist() == want
    assert W.w4(torch.zeros(1, 40))[0].tolist() == [0] * 40
    x = torch.randn(3, 96, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    v, p = W.q8_values(W.q8(x), 96)
    assert ((v - x).abs() <= torch.maximum(W.U8 * x.abs(), 2.0 ** -10 * p.repeat_interleave(32, 1))).all()
    W.close_q8(W.q8(x), x, torch.zeros_like(x), "itself")
    with pytest.raises(AssertionError):
        W.close_q8(W.q8(x * 1.2), x, torch.zeros_like(x), "another")
