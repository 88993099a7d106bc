"""The fp64 oracle of the operators around the layer (oracle/block.py), pinned by hand-worked cases, closed forms and
differences (CPU only)."""
import numpy as np
import pytest

from oracle import block as ob


def rng(seed):
    return np.random.default_rng(seed)


def difference(f, x, h=1e-6):
    """Gradient of a scalar function by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


def test_norm_by_hand():
    v, r = ob.rms_norm(np.array([[3.0, -4.0], [0.0, 0.0]]), np.array([2.0, 10.0]), 12.5)
    assert np.allclose(r, [0.2, 12.5 ** -0.5])               # (9 + 16) / 2 + 12.5 = 25
    assert np.allclose(v, [[1.2, -8.0], [0.0, 0.0]])


def test_norm_does_not_see_a_rows_size():
    h, w = rng(1).normal(size=(3, 50)), rng(2).normal(size=50)
    assert np.allclose(ob.rms_norm(h * 1e6, w, 1e-30)[0], ob.rms_norm(h, w, 1e-30)[0])


def test_norm_gradient_by_differences():
    r = rng(3)
    h, w, dy, ds = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=(3, 7)), r.normal(size=(3, 7))
    eps = 0.1
    dx, dw = ob.rms_norm_backward(dy, h, w, ob.rms_norm(h, w, eps)[1], ds)
    assert np.allclose(dx, difference(lambda x: (dy * ob.rms_norm(x, w, eps)[0] + ds * x).sum(), h), atol=1e-8)
    assert np.allclose(dw, difference(lambda x: (dy * ob.rms_norm(h, x, eps)[0]).sum(), w), atol=1e-8)


def test_balance_by_hand():
    # two tokens, two experts, one assignment each: p = (3/4, 1/4) and (1/2, 1/2)
    logits = np.log(np.array([[3.0, 1.0], [1.0, 1.0]]))
    loss, z, counts, probs = ob.balance_loss(logits, np.array([[0], [0]]))
    assert counts.tolist() == [[2, 0]] and np.allclose(probs, [[0.625, 0.375]])
    assert np.allclose(loss, [2 / (1 * 2) * 2 * 0.625])
    assert np.allclose(z, [(np.log(4) ** 2 + np.log(2) ** 2) / 2])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_is_one_where_experts_are_alike(score):
    E, k, T = 8, 2, 12
    ids = np.array([[t % E, (t + 4) % E] for t in range(T)])
    loss, _, _, probs = ob.balance_loss(np.full((T, E), -1.7), ids, score=score)
    assert np.allclose(loss, 1.0) and np.allclose(probs, 1 / E)


def test_balance_of_sequences_is_that_of_each():
    r = rng(5)
    logits, ids = r.normal(size=(9, 6)), r.integers(-1, 7, size=(9, 3))
    whole = ob.balance_loss(logits, ids, [1, 4, 4, 8])       # token 0 and token 8 belong to none
    for s, (a, b) in enumerate([(1, 4), (4, 4), (4, 8)]):
        if a == b:
            assert all((v[s] == 0).all() for v in whole)
            continue
        for got, one in zip(whole, ob.balance_loss(logits[a:b], ids[a:b])):
            assert np.allclose(got[s], one[0])


def test_tokens_without_experts_and_infinities():
    logits = np.array([[-np.inf, np.nan, -np.inf], [np.inf, 0.0, -np.inf]])
    for score in ("softmax", "sigmoid"):
        p = ob.probabilities(logits, score)
        assert (p[0] == 0).all() and p[1, 2] == 0 and np.allclose(p[1].sum(), 1)
    assert ob.log_sum_exp(logits)[0] == 0


@pytest.mark.parametrize("score,z", [("softmax", False), ("softmax", True), ("sigmoid", False)])
def test_balance_gradient_by_differences(score, z):
    r = rng(7)
    T, E, k = 7, 5, 2
    logits, ids, off = r.normal(size=(T, E)), r.integers(0, E, size=(T, k)), [0, 3, 6]
    dl, dz = r.normal(size=2), r.normal(size=2) if z else None

    def total(l):
        loss, zz, _, _ = ob.balance_loss(l, ids, off, score)
        return (dl * loss).sum() + ((dz * zz).sum() if z else 0.0)
    counts = ob.balance_loss(logits, ids, off, score)[2]
    before = r.normal(size=(T, E))
    got = ob.balance_loss_backward(logits, counts, dl, k, dz, off, score, before)
    assert np.allclose(got - before, difference(total, logits), atol=1e-8)
    assert (got[6] == before[6]).all()                       # of no sequence


def test_lora_by_hand_and_as_a_dense_product():
    X, Y = np.array([[1.0, 2.0]]), np.array([[10.0, 20.0, 30.0]])
    A, B = np.array([[[3.0, 4.0]]]), np.array([[[1.0], [0.0], [-1.0]]])
    assert np.allclose(ob.lora(X, A, B, [0], Y, np.array([0.5])), [[15.5, 20.0, 24.5]])
    assert np.allclose(ob.lora(X, A, B, [-1], Y), Y) and np.allclose(ob.lora(X, A, B, [1], Y), Y)
    r = rng(9)
    X, Y, A, B = r.normal(size=(6, 4)), r.normal(size=(6, 5)), r.normal(size=(3, 2, 4)), r.normal(size=(3, 5, 2))
    who, sc = np.array([2, 0, -1, 2, 1, 7]), r.normal(size=3)
    dense = np.stack([Y[t] + (sc[a] * X[t] @ (B[a] @ A[a]).T if 0 <= a < 3 else 0) for t, a in enumerate(who)])
    assert np.allclose(ob.lora(X, A, B, who, Y, sc), dense)
