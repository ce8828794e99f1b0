"""Routing by scores with logits that are NaN, -inf or the type's lowest value, and with experts that the bias shuts out, where groups are
valued by their best or their two best expert."""
import math

import pytest
import torch

from test_gpu_route_scored import DEV, DTYPES, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


def _inputs(e, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(200, e, generator=g, device=DEV) * 1.5).to(DTYPES[dtype]), torch.rand(200, e, generator=g, device=DEV), g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("part", [0.02, 0.3, 0.9])
@pytest.mark.parametrize("e,groups,kept,dtype", [(256, 8, 4, "fp32"), (160, 8, 3, "bf16"), (512, 16, 5, "fp16"), (64, 32, 9, "fp32"), (1024, 4, 1, "bf16"), (48, 2, 1, "fp32")])
def test_a_nan_stands_behind_all_numbers(score, top, part, e, groups, kept, dtype):
    """Also in its group's value, which is that of the numbers: the two best of a group with one number are no value at all."""
    x, where, g = _inputs(e, dtype, 60 + groups)
    x = x.masked_fill(where < part, math.nan)
    x[:, 0] = 1.0  # (a token of NaN alone has no softmax)
    for bias in (None, torch.zeros(e, device=DEV), torch.randn(e, generator=g, device=DEV) * 0.1):
        for renorm in (False, True):
            check(x, min(8, kept * (e // groups)), score, bias, groups, kept, top, renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("e,groups,kept,dtype", [(256, 8, 4, "fp32"), (160, 8, 3, "bf16"), (64, 32, 9, "fp16"), (96, 1, 1, "fp32")])
def test_masked_logits_and_shut_out_experts(score, top, e, groups, kept, dtype):
    x, where, g = _inputs(e, dtype, 70 + groups)
    k = min(8, kept * (e // groups))
    bias = torch.randn(e, generator=g, device=DEV) * 0.1
    y = x.masked_fill(where < 0.4, -math.inf)
    y[:, 0] = 1.0
    for b in (None, bias):
        if b is not None or top == 1:  # (without a bias vanished scores make sums that are the same for different groups)
            check(y, k, score, b, groups, kept, top)
    if top == 1:
        check(x.masked_fill(where < 0.4, torch.finfo(x.dtype).min), k, score, None, groups, kept, top)
    shut = bias.masked_fill(torch.rand(e, generator=g, device=DEV) < 0.3, -math.inf)
    check(x, k, score, shut, groups, kept, top)
