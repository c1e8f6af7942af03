"""The norm's outputs and workspace overlapping anything but what the header allows are refused
on the host.  Addresses here are never followed: each call returns before a launch."""

import ctypes
import os

import pytest

import combine_top_id_amd as M

EINVAL = -1
T, H = 5, 64


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        pytest.fail("libmoonep.so is not built (run __graft_entry__.build())")
    return M.lib()


def bf16(name, lib, a):
    return lib.moonep_rmsnorm(a["x"], a["res"], a["gamma"], 1e-6, T, H, a["out"], a["h"], a["rstd"], None)


def q8(name, lib, a):
    return lib.moonep_rmsnorm_q8(a["x"], a["res"], a["gamma"], 1e-6, T, H, a["out"], a["h"], a["rstd"], None)


def unpack(name, lib, a):
    return lib.moonep_q8_unpack(a["rows"], T, H, a["out"], None)


def back(name, lib, a):
    return lib.moonep_rmsnorm_bwd(a["g_out"], a["h"], a["gamma"], a["rstd"], a["g_h"], T, H, a["ws"], a["g_x"],
                                  a["g_gamma"], None)


ROW, Q8_ROW = T * H * 2, T * 80
SIZES = dict(x=ROW, res=ROW, h=ROW, out=ROW, g_out=ROW, g_h=ROW, g_x=ROW, rows=Q8_ROW, gamma=H * 2, rstd=T * 4,
             g_gamma=H * 4)


@pytest.mark.parametrize("call,inputs,outputs,same", [
    (bf16, ["x", "res", "gamma"], ["out", "h", "rstd"], [("h", "x"), ("h", "res")]),
    (q8, ["x", "res", "gamma"], ["out", "h", "rstd"], [("h", "x"), ("h", "res")]),
    (unpack, ["rows"], ["out"], []),
    (back, ["g_out", "h", "gamma", "rstd", "g_h"], ["g_x", "ws", "g_gamma"],
     [("g_x", "g_out"), ("g_x", "h"), ("g_x", "g_h")])])
def test_overlaps(lib, call, inputs, outputs, same):
    size = dict(SIZES, ws=lib.moonep_rmsnorm_bwd_workspace(T, H))
    if call is q8:
        size["out"] = Q8_ROW
    apart = {k: (k0 + 1) << 40 for k0, k in enumerate(inputs + outputs)}
    tested = 0
    for out in outputs:
        step = {"ws": 256, "rstd": 4}.get(out, 16)
        for other in inputs + outputs:
            if other == out:
                continue
            for at in (apart[other] - (size[out] - 1) // step * step, apart[other] + (size[other] - 1) // step * step,
                       apart[other]):
                if (out, other) in same and at == apart[other]:
                    continue
                a = {k: ctypes.c_void_p(v) for k, v in dict(apart, **{out: at}).items()}
                assert call(None, lib, a) == EINVAL, (out, other, at - apart[other])
                tested += 1
    assert tested >= 3 * len(outputs)


def test_h_over_both_inputs_that_are_one(lib):
    """x, res and h at one address: allowed as h == x and h == res, so only `out` is at fault."""
    p = [ctypes.c_void_p(k << 40) for k in range(1, 4)]
    assert lib.moonep_rmsnorm(p[0], p[0], p[1], 1e-6, T, H, p[0], p[0], None, None) == EINVAL
