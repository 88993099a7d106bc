"""examples/moe_layer.py: a whole layer, forward and backward, against autograd in fp64 on the CPU.

The experts chosen are the layer's own.  Everything else is compared end to end, so the bar is that of e4m3: one
operand's rounding is off by up to 2^-4 of a value, 2.6 % in the 2-norm; a product of two rounded operands 3.7 %; two
products, SwiGLU's two factors and its rounded input and output in a chain at most sqrt(8) * 2.6 % = 7.4 % forward, and
twice as many roundings backward, 10.4 %.  Bars 0.1 and 0.15; a wrong row, scale or transpose is off by about 1."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def rel(got, ref):
    got, ref = got.detach().double().cpu(), ref.detach().double()
    return float((got - ref).norm() / ref.norm())


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (100, 8, 2), (333, 5, 3)])
def test_layer_against_autograd(T, E, k):
    from examples.moe_layer import MoELayer
    K, I = 512, 256
    g = torch.Generator()
    g.manual_seed(T)
    rnd = lambda *s, std: (torch.randn(*s, generator=g) * std).to(torch.bfloat16)   # noqa: E731
    router, w_gate, w_up = rnd(E, K, std=K ** -0.5), rnd(E, I, K, std=K ** -0.5), rnd(E, I, K, std=K ** -0.5)
    w_down, x, dout = rnd(E, K, I, std=I ** -0.5), rnd(T, K, std=1.0), rnd(T, K, std=1.0)
    layer = MoELayer(router.cuda(), w_gate.cuda(), w_up.cuda(), w_down.cuda(), k, T, scale=1.5)
    out, kept = layer.forward(x.cuda())
    grads = layer.backward(dout.cuda(), kept)
    few = layer.decode(x.cuda())

    ids = kept["ids"].cpu().long()
    p = [t.double().requires_grad_() for t in (x, router, w_gate, w_up, w_down)]
    X, R, Wg, Wu, Wd = p
    w = torch.softmax(torch.gather(X @ R.t(), 1, ids), 1) * 1.5
    ref = torch.zeros(T, K, dtype=torch.float64)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gate, up = X[t] @ Wg[e].t(), X[t] @ Wu[e].t()
        ref = ref.index_add(0, t, (torch.sigmoid(gate) * gate * up) @ Wd[e].t() * w[t, j][:, None])
    ref.backward(dout.double())
    dW1 = mg.interleave_gate_up(Wg.grad, Wu.grad).transpose(1, 2)
    errs = {"out": rel(out, ref), "decode": rel(few, ref)}
    back = {"x": rel(grads["x"], X.grad), "router": rel(grads["router"], R.grad), "W1": rel(grads["W1"], dW1),
            "W2": rel(grads["W2"], Wd.grad.transpose(1, 2))}
    print(errs, back, flush=True)
    assert all(v <= 0.1 for v in errs.values()), errs
    assert all(np.isfinite(v) and v <= 0.15 for v in back.values()), back
