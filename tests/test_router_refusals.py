"""What the router's calls refuse, found on the host before anything is launched, and the 64-bit gradients of their
GPU tests against differences."""

import ctypes
import inspect
import os

import numpy as np
import pytest
import torch

import combine_top_id_amd as M
from tests import router_ref as R

EINVAL, ELIMIT, EALIGN = -1, -2, -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        pytest.fail("libmoonep.so is not built (run __graft_entry__.build())")
    return M.lib()


def at(k, more=0):
    return ctypes.c_void_p((k << 40) + more)           # never followed


def fwd(lib, logits=at(1), dtype=0, bias=at(2), T=4, E=16, K=2, score=0, groups=1, top=1, norm=1, scale=1.0, ids=at(3), w=at(4)):
    return lib.moonep_router(logits, dtype, bias, T, E, K, score, groups, top, norm, scale, ids, w, None)


def bwd(lib, logits=at(1), dtype=0, ids=at(2), g_w=at(3), T=4, E=16, K=2, score=0, norm=1, scale=1.0, out=at(4)):
    return lib.moonep_router_bwd(logits, dtype, ids, g_w, T, E, K, score, norm, scale, out, None)


@pytest.mark.parametrize("call,ptrs,outs", [(fwd, ["logits", "ids", "w"], {"ids": (1, 2, 4), "w": (1, 2, 3)}),
                                            (bwd, ["logits", "ids", "g_w", "out"], {"out": (1, 2, 3)})])
def test_refuses(lib, call, ptrs, outs):
    for p in ptrs:
        assert call(lib, **{p: None}) == EINVAL, p
        assert call(lib, **{p: at(9, 2)}) == EALIGN, p
    assert call(lib, logits=at(9, 1), dtype=1) == EALIGN
    for bad in (dict(dtype=2), dict(dtype=-1), dict(score=2), dict(score=-1), dict(norm=2), dict(norm=-1), dict(T=-1), dict(E=0),
                dict(E=-16), dict(K=0), dict(K=-1), dict(K=17), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(lib, **bad) == EINVAL, bad
    assert call(lib, E=1025) == ELIMIT and call(lib, E=64, K=33) == ELIMIT and call(lib, T=1 << 31) == ELIMIT
    assert call(lib, T=0, **{p: None for p in ptrs}) == 0
    for out, others in outs.items():
        for o in others:
            assert call(lib, **{out: at(o)}) == EINVAL, (out, o)
    last = "ids" if call is fwd else "out"
    assert call(lib, **{last: at(1, 4 * 16 * 4 - 4)}) == EINVAL          # the last logit


def test_refuses_groups(lib):
    assert fwd(lib, bias=at(9, 2)) == EALIGN
    for g, top in ((0, 1), (-1, 1), (3, 1), (4, 0), (4, 5), (4, -1), (16, 1)):      # the last: fewer experts than K
        assert fwd(lib, groups=g, top=top) == EINVAL, (g, top)
    assert fwd(lib, E=128, groups=128, top=128) == ELIMIT


def test_binding_refuses(lib):
    l = torch.zeros(4, 16)
    for f in (lambda: M.moonep_router(l, 2), lambda: M.moonep_router_bwd(l, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))):
        with pytest.raises(M.MoonepError, match="GPU tensor"):
            f()
    for f in (M.moonep_router, M.moonep_router_bwd):
        assert inspect.signature(f).parameters["stream"].kind is inspect.Parameter.KEYWORD_ONLY


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_reference_gradient_against_differences(kind, normalize):
    rng = np.random.RandomState(3)
    l = rng.randn(3, 7)
    ids = np.array([[1, 4, 2], [6, 0, 3], [5, 1, 0]])
    g = rng.randn(3, 3)
    f = lambda v: float((R.weights(v, ids, kind, normalize, 1.7)[0] * g).sum())  # noqa: E731
    grad, _ = R.gradient(l, ids, g, kind, normalize, 1.7)
    e = 1e-5
    for t in range(3):
        for i in range(7):
            d = np.zeros_like(l)
            d[t, i] = e
            num = (f(l + d) - f(l - d)) / (2 * e)
            assert abs(num - grad[t, i]) <= 1e-8 * (1 + abs(num))


def test_reference_choice():
    l = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0, np.nan]])
    assert R.choose(l, None, "softmax", 6).tolist() == [[1, 2, 4, 0, 3, 5]]
    assert R.choose(l, np.array([9.0, 0, 0, 99, 0, 99]), "sigmoid", 4).tolist() == [[0, 1, 2, 4]]
    # groups (1, 3), (3, -), (2, -): the sum of two, of what is there
    assert R.choose(l, None, "sigmoid", 2, 3, 1).tolist() == [[1, 0]]
    w, _ = R.weights(l, np.array([[1, 2, 3]]), "softmax", True, 2.0)
    assert np.allclose(w, [[1, 1, 0]])
