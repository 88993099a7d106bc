"""Group-limited routing on MI355X where experts are masked (logits or biases of -inf and NaN): ids, counts and rows
equal the fp64 oracle's, weights are within the bound of tests/test_gpu_layer.py."""
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_gpu_layer import check_route, gen

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_of_one_candidate(T, score):
    """One expert left in a group: its score is the group's, and a group with none comes last."""
    l = torch.full((T, 8), -INF)
    l[:, 1], l[:, 3], l[:, 6] = 0, 9, 3
    _, ids = check_route(l.cuda(), 2, 2 * T, score=score, n_groups=4, topk_groups=1, group_top=2)
    assert (ids == [3, -1]).all()
    bias = torch.full((8,), -INF)
    bias[3] = -5
    _, ids = check_route(torch.zeros(T, 8).cuda(), 2, 2 * T, bias=bias.cuda(), score=score, n_groups=4, topk_groups=1,
                         group_top=2)
    assert (ids == [3, -1]).all()


@pytest.mark.parametrize("keep", [0.02, 0.1, 0.5])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,n,top", [(1, 8, 2, 4, 1), (16, 64, 8, 32, 9), (40, 12, 3, 4, 2), (33, 256, 8, 8, 4),
                                         (17, 111, 4, 3, 1), (50, 592, 6, 16, 3), (24, 1024, 8, 64, 10), (70, 300, 6, 2, 1)])
def test_masked_groups(T, E, k, n, top, with_bias, keep):
    """Few experts left: most groups have none, one or two.  Groups on whole runs of lanes and off them."""
    g = gen(T + E + int(100 * keep))
    l = torch.randn(T, E, generator=g)
    l[torch.rand(T, E, generator=g) >= keep] = -INF
    l[T // 2, E // 2] = float("nan")
    bias = None
    if with_bias:
        bias = torch.randn(E, generator=g) * 0.5 - 0.5      # keys of either sign
        bias[torch.rand(E, generator=g) < 0.1] = -INF
        bias = bias.cuda()
    for score in ("softmax", "sigmoid"):
        for group_top in (1, 2):
            check_route(l.cuda(), k, T * k, bias=bias, score=score, n_groups=n, topk_groups=top, group_top=group_top)
