"""Every tile of every product of the experts in 4 bits is among the sizes that the GPU tests compare: the library
says which tile the sizes of tests/w4_tiles.py take."""

import ctypes
import os

import pytest
import torch

import combine_top_id_amd as M
from tests.w4_tiles import TILES

EINVAL, ELIMIT, EPLAN = -1, -2, -3


def plan_of(R, E, K, S, slots):
    p = M.Plan(M.moonep_query(R, E, K, S, slots), torch.zeros(1, dtype=torch.int32), None)
    p.desc.magic, p.desc.dev, p.desc.sz = 0x4D4F4E45, 256, p.sz
    return p


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(M.LIB_PATH):
        pytest.fail("libmoonep.so is not built (run __graft_entry__.build())")


def test_the_tiles_are_those_that_are_meant():
    for sizes, q8, product, tile in TILES:
        p = plan_of(*sizes[:5])
        assert M.moonep_expert_tile_w4(p, sizes[5], sizes[6], q8, product) == tile, (sizes, q8, product)


def test_every_tile_is_taken():
    few = {(128, 16), (256, 32), (256, 64), (256, 128)}
    for q8, all_ in ((False, few), (True, {(128, 16), (128, 64), (256, 64), (256, 128), (256, 256)})):
        for product in ("gate_up", "down"):
            assert {t for _, q, pr, t in TILES if q == q8 and pr == product} == all_
        # and no other
        for R, E in ((1, 1), (8, 64), (64, 1024)):
            for S in (1, 16, 300, 20000):
                for H, I in ((32, 32), (7168, 2048), (1024, 4096), (32768, 32768)):
                    p = plan_of(R, E, min(E, 8), S, 1)
                    for product in ("gate_up", "down"):
                        assert M.moonep_expert_tile_w4(p, H, I, q8, product) in all_


def test_refusals():
    L = M.lib()
    t = (ctypes.c_int32 * 2)()
    p = plan_of(4, 16, 2, 4, 4)
    f = lambda d=p.desc, H=64, I=32, q8=0, pr=0, t=t: L.moonep_expert_tile_w4(ctypes.byref(d) if d else None, H, I, q8, pr, t)  # noqa: E731
    assert f() == 0 and f(d=None) == EPLAN and f(t=None) == EINVAL
    assert f(pr=2) == EINVAL and f(pr=-1) == EINVAL and f(q8=2) == EINVAL and f(q8=-1) == EINVAL
    assert f(H=60) == EINVAL and f(I=0) == EINVAL and f(H=32776) == ELIMIT
    assert f(H=72) == 0 and f(H=72, q8=1) == EINVAL and f(I=40, q8=1) == EINVAL
    big = plan_of(64, 64, 1, 1 << 24, 0)
    assert f(d=big.desc, H=32768) == ELIMIT
    with pytest.raises(M.MoonepError, match="product"):
        M.moonep_expert_tile_w4(p, 64, 32, False, "g_rows")
