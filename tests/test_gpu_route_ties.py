"""Routing by scores: experts and groups whose values are exactly the same, with a bias that is not zero and with groups valued by
their two best.

Experts come in classes of one logit and one bias each, so that equal values are of equal inputs, in the kernel and in the reference
(two different sums that happen to be the same number would be rounded apart)."""
import pytest
import torch

from test_gpu_route_scored import DEV, DTYPES, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,kept", [(256, 8, 4), (256, 8, 2), (64, 4, 1), (160, 32, 9), (96, 2, 1), (1024, 16, 5), (33, 1, 1)])
@pytest.mark.parametrize("classes", [1, 2, 5, 12])
def test_classes_of_equal_experts(score, e, groups, kept, classes):
    g = torch.Generator(device=DEV)
    g.manual_seed(classes + e)
    of = torch.randint(0, classes, (e,), generator=g, device=DEV)
    for dtype in DTYPES.values():
        x = torch.randn(100, classes, generator=g, device=DEV).to(dtype)[:, of].contiguous()
        for bias in (None, torch.zeros(e, device=DEV), (torch.randn(classes, generator=g, device=DEV) * 0.1)[of].contiguous()):
            for top in (1, 2):
                for k in (1, 8, 20):
                    check(x, min(k, kept * (e // groups)), score, bias, groups, kept, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
def test_all_experts_equal(score, top):
    """Equal logits under an equal bias: the lowest experts of the lowest groups."""
    for bias in (None, torch.full((256,), 0.25, device=DEV)):
        x = torch.full((9, 256), 1.5, device=DEV)
        for groups, kept in ((1, 1), (8, 3), (32, 2)):
            ids, _ = check(x, 12, score, bias, groups, kept, top)
            assert torch.equal(ids, torch.arange(12, dtype=torch.int32, device=DEV).expand(9, 12))
