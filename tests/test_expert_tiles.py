"""The tiles that the experts' products take, a choice made on the host: the GPU tests' sizes
meet each of them, so a change of the rule cannot leave a kernel without a test."""

import ctypes
import os

import pytest

import combine_top_id_amd as M
from combine_top_id_amd.moonep import PRODUCTS, PlanDesc
from tests import expert_tiles as T
from tests.test_gpu_expert_ffn import CASES

EINVAL, ELIMIT, EPLAN = -1, -2, -3


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(M.LIB_PATH):
        pytest.fail("libmoonep.so is not built (run __graft_entry__.build())")
    return M.lib()


def test_the_gpu_tests_meet_every_tile_of_every_product():
    seen = {p: set() for p in PRODUCTS}
    for case in CASES + T.LARGE_CASES:
        for p, t in T.tiles(*case[:7]).items():
            seen[p].add(t)
    assert seen == T.TILES


def test_the_largest_tiles_have_odd_sizes_and_several_rounds():
    """Of each product's 256-wide tiles: one case at least with columns and steps that end inside
    a tile, and more tiles than the 256 workgroups take in one round."""
    for product, wide, deep in (("gate_up", lambda H, I: 2 * I, lambda H, I: H), ("down", lambda H, I: H, lambda H, I: I),
                                ("g_gate_up", lambda H, I: I, lambda H, I: H),
                                ("g_rows", lambda H, I: H, lambda H, I: 2 * I)):
        for tile in ((256, 256, False), (256, 128, False)):
            assert any(T.tiles(R, E, K, S, slots, H, I)[product] == tile and wide(H, I) % 256 and deep(H, I) % 64 and
                       (R * S * K // tile[1]) * -(-wide(H, I) // 256) > 256
                       for R, E, K, S, slots, H, I, _ in T.LARGE_CASES), (product, tile)


def test_refusals(lib):
    d = PlanDesc()
    d.magic, d.dev, d.sz = 0x4D4F4E45, 256, M.moonep_query(4, 16, 2, 4, 4)
    out = (ctypes.c_int32 * 3)()
    f = lambda d=d, H=64, I=32, product=0, out=out: lib.moonep_expert_tile(  # noqa: E731
        ctypes.byref(d) if d else None, H, I, product, out)
    assert f() == 0 and f(product=4) == 0
    assert f(d=None) == EPLAN and f(d=PlanDesc()) == EPLAN
    assert f(H=0) == EINVAL and f(H=12) == EINVAL and f(I=-8) == EINVAL and f(I=4) == EINVAL
    assert f(H=32776) == ELIMIT and f(H=32768, I=32768) == ELIMIT
    assert f(product=-1) == EINVAL and f(product=5) == EINVAL and f(out=None) == EINVAL
    with pytest.raises(M.MoonepError, match="product"):
        M.moonep_expert_tile(None, 64, 32, "gate")
