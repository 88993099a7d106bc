"""The z loss's gradient on MI355X where a logit is infinite."""
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_gpu_balance import BF16, F32, I32, buf, forward, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


@pytest.mark.parametrize("kind", [F32, BF16])
def test_z_gradient_of_infinite_logits(kind):
    """+inf is the largest number: its p is 1 and every other one of its token 0, whose gradients are 0."""
    T, E, k = 6, 70, 2
    l, ids, _ = inputs(T, E, k, 0, kind, 7)
    l[1, 3] = l[4, 69] = float("inf")
    off = torch.tensor([0, 1, 2, 6], dtype=I32)
    counts = forward(l, ids, off, "softmax")["counts"]
    for dz in (0.25, 3.0, 1000.0, 2.0 ** 127):
        d = buf((T, E), kind)
        mg.balance_loss_backward(l.cuda(), counts, torch.full((3,), 0.01).cuda(), d, k=k, d_z_loss=torch.full((3,), dz).cuda(),
                                 seq_offsets=off.cuda())
        d = d.cpu()
        for t, e in ((1, 3), (4, 69)):
            rest = torch.ones(E, dtype=torch.bool)
            rest[e] = False
            assert bool((d[t][rest] == 0).all()), (t, dz, d[t][rest].isnan().sum())
            assert float(d[t, e]) >= 2.0 ** 120
        if dz <= 1000:
            assert bool(d[[0, 2, 3, 5]].isfinite().all())
