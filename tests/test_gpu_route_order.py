"""Routing by scores: the order of chosen experts whose values a bias brings together, for the softmax, against 64 bits.

The pairs' distances are those that fp64 tells apart (1e-8 of the value and more, where fp64 is off by 1e-15), and lie below what
fp32 can: the rounding of x - max, by which a far score is off by up to 2^-24 |x - max| of itself, and the fp32 sum of the exponentials,
which moves all scores of a token by one factor that does not cancel against a bias."""
import math
import random

import pytest
import torch

from test_gpu_route_scored import DEV, check, scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


def _row(x):
    """fp32 logits of one token, and their softmax in 64 bits."""
    x = torch.tensor([x], dtype=torch.float32, device=DEV)
    return x, scores(x, "softmax")[0].tolist()


@pytest.mark.parametrize("far", [9.0, 17.0, 34.0, 60.0])
def test_a_pair_far_below_the_largest(far):
    """Two experts far below a third, their values within 3e-6 of one another."""
    for seed in range(250):
        rng = random.Random(seed)
        e, top = 64, 34.18254
        first, a, b = rng.sample(range(e), 3)
        x = [top - far - 5.0] * e
        x[first], x[a], x[b] = top, top - far + rng.uniform(-0.01, 0.01), top - far + rng.uniform(-0.01, 0.01)
        logits, s = _row(x)
        bias = [-1.0] * e
        bias[first], bias[a] = 0.0, 0.1 * s[a]
        bias[b] = (s[a] + bias[a]) * (1 + rng.choice((-1, 1)) * 10 ** rng.uniform(-6.5, -5.5)) - s[b]
        check(logits, 3, "softmax", torch.tensor(bias, dtype=torch.float32, device=DEV))


@pytest.mark.parametrize("e", [32, 128, 256, 512, 1024])
@pytest.mark.parametrize("groups", [1, 4])
def test_one_large_and_many_equal_logits(e, groups):
    """The largest score against a smaller one that its bias brings close to it, where the sum has many equal terms."""
    for seed in range(250):
        rng = random.Random(seed)
        first, second = rng.sample(range(e // groups), 2)
        x = [rng.uniform(-1, 1)] * e
        x[first] += math.log(e) + rng.uniform(-1, 2)
        logits, s = _row(x)
        bias = [-1.0] * e
        bias[first] = 0.0
        bias[second] = s[first] - s[second] + rng.choice((-1, 1)) * 10 ** rng.uniform(-8.5, -6.5)
        check(logits, 2, "softmax", torch.tensor(bias, dtype=torch.float32, device=DEV), groups, 1, 1)


def test_scores_below_the_smallest_normal_number():
    """A bias of zeros, and scores that fp32 holds with few bits or not at all: the order is the logits'."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.randn(64, 128, generator=g, device=DEV) * 0.02 - 95
    zero = torch.zeros(128, device=DEV)
    for k in (2, 9, 24):
        check(x, k, "sigmoid", zero)
        y = x.clone()
        y[:, 40] = 0.0
        check(y, k, "softmax", zero)
