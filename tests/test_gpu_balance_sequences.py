"""The router's balance loss and its gradient on MI355X with more sequences than a wave holds bounds of (64): sequences of one
token, so that a tile of tokens meets more than 63, and runs of empty ones in front, in between and behind.  Bounds as in
test_gpu_balance.py."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_gpu_balance import BF16, F32, I32, buf, check_backward, check_forward, code, forward, gen, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def offsets(T, S, plan, seed):
    """Bounds of S sequences of T tokens."""
    r = np.random.default_rng(seed)
    if plan == "one":                                        # of one token each, the last of the rest
        n = np.ones(S, dtype=np.int64)
    elif plan == "runs":                                     # empty in front, behind, and in the middle of those of one
        n = np.zeros(S, dtype=np.int64)
        n[S // 5:S // 5 + T // 3] = 1
        n[S // 2:S // 2 + T // 3] = 1
    else:                                                    # of any length
        n = r.multinomial(T - 1, np.ones(S) / S)
    o = np.minimum(np.concatenate([[0], np.cumsum(n)]), T)
    if plan == "one":
        o[-1] = T
    return torch.tensor(o, dtype=I32)


@pytest.mark.parametrize("T,E,k,S,plan", [
    (65, 8, 2, 65, "one"), (100, 130, 4, 65, "one"), (500, 16, 2, 65, "any"), (500, 300, 3, 500, "one"),
    (700, 8, 2, 500, "any"), (300, 40, 4, 1000, "runs"), (9000, 20, 2, 1000, "any"), (8300, 12, 2, 5000, "one"),
    (3000, 65, 2, 5000, "runs")])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_sequences(T, E, k, S, plan, score):
    print("CASE balance sequences", T, E, k, S, plan, score, flush=True)
    l, ids, _ = inputs(T, E, k, 0, F32 if T % 2 else BF16, T + S)
    off = offsets(T, S, plan, S)
    check_forward(l, ids, off, score)
    check_backward(l, ids, off, score, S)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_empty_sequences_change_no_bits(score):
    """65536 sequences, most of them empty, against the others alone."""
    T, E, k, S = 4100, 24, 3, 65536
    l, ids, _ = inputs(T, E, k, 0, F32, 3)
    n = np.random.default_rng(4).multinomial(T, np.ones(700) / 700)
    at = np.sort(np.random.default_rng(5).choice(np.arange(9000, S - 9000), 700, replace=False))
    few = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=I32)
    many = np.zeros(S, dtype=np.int64)
    many[at] = n
    many = torch.tensor(np.concatenate([[0], np.cumsum(many)]), dtype=I32)
    a = check_forward(l, ids, few, score)
    b = forward(l, ids, many, score, z=score == "softmax")
    there = torch.from_numpy(at).cuda()
    others = torch.ones(S, dtype=torch.bool, device="cuda")
    others[there] = False
    for name in a:
        if a[name] is not None:
            assert torch.equal(a[name], b[name][there]) and not bool(b[name][others].any()), name
    d = []
    for off, counts in ((few, a["counts"]), (many, b["counts"])):
        dl = torch.zeros(len(off) - 1)
        dl[torch.from_numpy(at) if len(dl) == S else slice(None)] = torch.randn(700, generator=gen(6))
        d.append(buf((T, E), F32))
        mg.balance_loss_backward(l.cuda(), counts, dl.cuda(), d[-1], k=k, seq_offsets=off.cuda(), score=code(score))
    assert torch.equal(*d)
