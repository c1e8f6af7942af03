"""The router's choice where two keys are nearly or exactly equal, or at the ends of fp32's range: what the comparison
by short keys has to hand on to the one in 64 bits.  Ids exactly, as in tests/test_gpu_router.py."""

import numpy as np
import pytest
import torch

import combine_top_id_amd as M
from tests import router_ref as R
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M.lib()


def same_ids(l, K, bias=None, score="softmax", groups=1, top_groups=1, normalize=True):
    """`l` fp32 [T, E] and `bias` fp32 [E], numpy."""
    ids, _ = M.moonep_router(torch.from_numpy(l).cuda(), K, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                             score=score, groups=groups, top_groups=top_groups, normalize=normalize)
    ref, got = R.choose(l, bias, score, K, groups, top_groups), ids.cpu().numpy()
    bad = np.nonzero((got != ref).any(1))[0]
    assert not len(bad), f"{len(bad)} of {len(l)} tokens differ, token {bad[0]}: {got[bad[0]]}, not {ref[bad[0]]}"


def rivals(score, T, E, seed, step=1e-5):
    """Logits and biases with pairs of experts, one with a score of 1e-6 to 1e-5 and one of about a tenth, whose keys
    differ by 1e-10 to 1e-7 only: two experts of every eight, each pair's keys `step` below the last's, all other keys far below."""
    rng = np.random.RandomState(seed)
    n = min(E // 4, 16) // 2                             # pairs
    eights = rng.permutation(E // 8)[:n]
    one, two = (np.array([rng.permutation(8)[:2] for _ in range(n)]) + 8 * eights[:, None]).T
    level = 2e-5 + step * np.arange(n)[::-1]
    bias = np.full(E, -2.0, np.float32)
    bias[one] = level - 10.0 ** rng.uniform(-6, -5, n)
    bias[two] = level - 0.9 / n * rng.uniform(0.5, 1.0, n)
    off = rng.randn(T, n) * 10.0 ** rng.uniform(-10, -7, (T, 1))
    small, large = level - bias[one].astype(np.float64) + 0 * off, level - bias[two].astype(np.float64) + off
    l = np.zeros((T, E))
    if score == "softmax":
        l[:] = np.log((1 - small.sum(1, keepdims=True) - large.sum(1, keepdims=True)) / (E - 2 * n))
        l[:, one], l[:, two] = np.log(small), np.log(large)
    else:
        l[:, one], l[:, two] = (np.log(s) - np.log1p(-s) for s in (small, large))
    return l.astype(np.float32), bias


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(64, 1), (64, 5), (64, 8), (256, 1), (256, 8), (256, 15), (512, 5), (256, 16), (1024, 5)])
def test_unlike_scores_with_nearly_equal_keys(score, E, K):
    for seed in range(4):
        say(f"router rivals E={E} K={K} {score} seed={seed}")
        l, b = rivals(score, 500, E, seed)
        same_ids(l, K, b, score)
        same_ids(l, min(K, 8), b, score, groups=8, top_groups=4, normalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,groups,top", [(64, 4, 8, 3), (64, 1, 8, 1), (64, 16, 8, 4), (128, 8, 16, 5), (512, 8, 64, 4), (1024, 6, 64, 3)])
def test_groups_with_nearly_equal_sums_of_unlike_scores(score, E, K, groups, top):
    for seed, step in enumerate((0.0, 1e-9, 1e-7, 4e-6)):
        say(f"router sums E={E} K={K} groups={groups} top={top} {score} step={step}")
        l, b = rivals(score, 200, E, seed, step)
        same_ids(l, K, b, score, groups, top)


def test_a_rounded_score_behind_a_tiny_bias():
    # key 1 is 1/25 less its rounding to fp32, which is more than 1e-30; in fp32 it is zero
    l, b = np.zeros((1, 26), np.float32), np.full(26, -1.0, np.float32)
    l[0, 0], b[0], b[1] = -200, 1e-30, -np.float32(1 / 25)
    assert R.choose(l, b, "softmax", 1)[0, 0] == 1
    same_ids(l, 1, b)
    same_ids(np.concatenate([l, l + 3]), 2, b)


def test_scores_below_the_smallest_normal_number():
    rng = np.random.RandomState(5)
    for E, K in ((64, 8), (384, 8), (1024, 16)):
        say(f"router tiny scores E={E} K={K}")
        l = (-86 - 20 * rng.rand(100, E)).astype(np.float32)
        l[:, 3] = 0                                      # the others' scores are between 2^-153 and 2^-124
        same_ids(l, K, np.zeros(E, np.float32))
        same_ids(l, K, (rng.randint(-3, 4, E) * 2.0 ** -149).astype(np.float32))
        same_ids(l, K, np.zeros(E, np.float32), groups=4, top_groups=2)


@pytest.mark.parametrize("E,K", [(64, 1), (64, 7), (300, 15), (600, 8), (1024, 31)])
def test_subnormal_logits(E, K):
    for seed, top in enumerate((25, 60, 1000, 1 << 22)):
        say(f"router subnormal logits E={E} K={K} up to {top} units")
        rng = np.random.RandomState(seed)
        l = (rng.randint(-top, top + 1, (200, E)) * 2.0 ** -149).astype(np.float32)
        same_ids(l, K)
        same_ids(l, K, score="sigmoid", normalize=False)
        l[rng.rand(200, E) < 0.9] = -1.0                 # few beside many that are far below
        same_ids(l, K)


def test_a_subnormal_logit_behind_two_smaller_ones():
    l = np.full((1, 64), -1.0, np.float32)
    l[0, [0, 1, 20]] = np.float32(2.0 ** -149) * np.array([3, 1, 20], np.float32)
    assert R.choose(l, None, "softmax", 1)[0, 0] == 20
    same_ids(l, 1)


MAX = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_with_biases_at_the_ends_of_the_range(score):
    for i, (T, E, K, groups, top) in enumerate([(20, 64, 6, 8, 3), (9, 256, 8, 8, 4), (7, 12, 2, 12, 2), (5, 1024, 16, 64, 8),
                                                (11, 64, 4, 2, 1), (6, 768, 8, 3, 1)]):
        rng = np.random.RandomState(40 + i)
        l = rng.randn(T, E).astype(np.float32)
        size = E // groups
        for what, values in dict(on=[np.inf, 0, 0, 0, 0], off=[-MAX, 0], on_and_off=[np.inf, -np.inf, 0, 0, 0, 0], ends=[MAX, -MAX],
                                 all=[np.inf, MAX, 3e38, 1.0, -1e38, -MAX, -np.inf], lowest=[-MAX, -np.inf, -3e38]).items():
            say(f"router biases {what} E={E} groups={groups} {score}")
            for _ in range(4):
                b = rng.choice(np.array(values, np.float32), E)
                same_ids(l, K, b, score, groups, top)
                # whole groups alike
                b = np.repeat(rng.choice(np.array(values, np.float32), groups), size)
                same_ids(l, K, b, score, groups, top)
        b = np.zeros(E, np.float32)
        b[E - 2] = np.inf                                # one expert that every token takes
        assert (R.choose(l, b, score, K, groups, top)[:, 0] == E - 2).all()
        same_ids(l, K, b, score, groups, top)


def test_a_group_of_lowest_biases_before_one_that_is_masked():
    l, b = np.zeros((3, 16), np.float32), np.zeros(16, np.float32)
    l[:, :8] = -np.inf                                   # nothing left in the first group
    b[8:] = -MAX
    assert (R.choose(l, b, "sigmoid", 2, 2, 1) == [8, 9]).all()
    same_ids(l, 2, b, "sigmoid", 2, 1)
    same_ids(l, 2, b, "softmax", 2, 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_at_the_ends_of_the_range(score):
    for E, K in ((64, 6), (384, 15), (700, 8)):
        rng = np.random.RandomState(E)
        l = rng.randint(-2, 3, (30, E)).astype(np.float32)
        for values in ([np.inf, MAX, 3e38, 0.0], [np.inf, 0, 0, 0, 0, 0, 0], [-MAX, -np.inf, -3e38, 1.0], [np.inf, MAX, -MAX, -np.inf]):
            say(f"router biases {values} E={E} {score}")
            same_ids(l, K, rng.choice(np.array(values, np.float32), E), score)
