"""examples/moe_block.py: norm, layer, balance loss and their gradients, and a projection with adapters, against autograd
in fp64 on the CPU.

The experts chosen are the block's own.  Bars as for the layer by itself: e4m3's rounding is 2.6 % in the 2-norm for each
operand, the chain of products at most 7.4 % forward (bar 0.1) and 10.4 % backward (bar 0.15).  The losses are bf16's: the
norm's output rounded (2^-8 of a value) in the logits' sum and once more as logits, whose errors e turn a probability by
e: the balance loss by 2 max e, ln sum e^l by max e."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def rel(got, ref):
    got, ref = got.detach().double().cpu(), ref.detach().double()
    return float((got - ref).norm() / ref.norm())


def norm64(h, w, eps):
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w


@pytest.mark.parametrize("T,E,k,cuts", [(1, 8, 2, [0, 1]), (100, 8, 2, [0, 30, 30, 100]), (333, 5, 3, [0, 1, 200, 333])])
def test_block_against_autograd(T, E, k, cuts):
    from examples.moe_block import MoEBlock
    from examples.moe_layer import MoELayer
    K, I, S = 512, 256, len(cuts) - 1
    g = torch.Generator()
    g.manual_seed(T)
    rnd = lambda *s, std: (torch.randn(*s, generator=g) * std).to(BF16)   # noqa: E731
    router, w_gate, w_up = rnd(E, K, std=K ** -0.5), rnd(E, I, K, std=K ** -0.5), rnd(E, I, K, std=K ** -0.5)
    w_down, x, r = rnd(E, K, I, std=I ** -0.5), rnd(T, K, std=2.0), rnd(T, K, std=1.0)
    dout, dh, nw = rnd(T, K, std=1.0), rnd(T, K, std=0.5), 1 + 0.2 * torch.randn(K, generator=g)
    layer = MoELayer(router.cuda(), w_gate.cuda(), w_up.cuda(), w_down.cuda(), k, T, scale=1.5)
    block = MoEBlock(layer, nw.cuda(), T, S, balance=20.0, z=5.0)         # large, so that their gradients count
    off = torch.tensor(cuts, dtype=I32).cuda()
    out, h, losses, kept = block.forward(x.cuda(), r.cuda(), off)
    grads = block.backward(dout.cuda(), dh.cuda(), kept)

    assert torch.equal(h.cpu(), (x.float() + r.float()).to(BF16))
    ids = kept["ids"].cpu().long()
    p = [t.double().requires_grad_() for t in (h.cpu(), router, w_gate, w_up, w_down, nw)]
    H, R, Wg, Wu, Wd, NW = p
    Y = norm64(H, NW, 1e-6)
    logits = Y @ R.t()
    w = torch.softmax(torch.gather(logits, 1, ids), 1) * 1.5
    ref = torch.zeros(T, K, dtype=torch.float64)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gate, up = Y[t] @ Wg[e].t(), Y[t] @ Wu[e].t()
        ref = ref.index_add(0, t, (torch.sigmoid(gate) * gate * up) @ Wd[e].t() * w[t, j][:, None])
    # an error of the logits: half a step for the norm's output in each term, half a step of the result
    e_logit = float((2.0 ** -8 * (Y.abs() @ R.abs().t() + logits.abs())).detach().max())
    total, probs = (ref * dout.double()).sum() + (H * dh.double()).sum(), torch.softmax(logits, 1)
    for s, (a, b) in enumerate(zip(cuts[:-1], cuts[1:])):
        if a == b:
            assert float(losses["balance"][s]) == float(losses["z"][s]) == 0
            continue
        c = torch.bincount(ids[a:b].reshape(-1), minlength=E)
        assert torch.equal(kept["counts"][s].cpu().long(), c)
        balance = E / (k * (b - a)) * (c * probs[a:b].mean(0)).sum()
        lse = torch.logsumexp(logits[a:b], 1)
        z = (lse ** 2).mean()
        b64, z64 = float(balance.detach()), float(z.detach())
        assert abs(float(losses["balance"][s]) - b64) <= 2.1 * e_logit * b64
        assert abs(float(losses["z"][s]) - z64) <= 1.05 * e_logit * float((2 * lse.detach().abs() + e_logit).mean())
        total = total + 20.0 / S * balance + 5.0 / S * z
    total.backward()
    dW1 = mg.interleave_gate_up(Wg.grad, Wu.grad).transpose(1, 2)
    back = {"x": rel(grads["x"], H.grad), "router": rel(grads["router"], R.grad), "norm": rel(grads["norm"], NW.grad),
            "W1": rel(grads["W1"], dW1), "W2": rel(grads["W2"], Wd.grad.transpose(1, 2))}
    print(rel(out, ref), back, flush=True)
    assert rel(out, ref) <= 0.1
    assert all(np.isfinite(v) and v <= 0.15 for v in back.values()), back


@pytest.mark.parametrize("T", [1, 70, 300])
def test_projection_with_adapters(T):
    """The shared product is off by 3.7 % in the 2-norm (two e4m3 operands), the adapters' by bf16's roundings of their
    input and of the sum, 2 * 2^-8 at most: of an adapter's part as large as the product's, 0.05 of the whole."""
    from examples.moe_block import Projection
    K, N, R, L = 512, 768, 16, 5
    g = torch.Generator()
    g.manual_seed(T)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF16)   # noqa: E731
    x, r, w, nw = rnd(T, K), rnd(T, K), rnd(N, K, std=K ** -0.5), rnd(K, std=0.2) + 1
    A, B, scale = rnd(L, R, K, std=K ** -0.5), rnd(L, N, R, std=R ** -0.5), 1 + torch.rand(L, generator=g)
    adapter = torch.randint(-1, L, (T,), generator=g).to(I32)
    proj = Projection(nw.cuda(), w.cuda(), A.cuda(), B.cuda(), scale.cuda(), T)
    out, h = proj(x.cuda(), r.cuda(), adapter.cuda())
    H = (x.float() + r.float()).to(BF16)
    assert torch.equal(h.cpu(), H)
    y = norm64(H.double(), nw.double(), 1e-6)
    ref = y @ w.double().t()
    for a in range(L):
        rows = adapter == a
        ref[rows] += scale[a].double() * (y[rows] @ A[a].double().t()) @ B[a].double().t()
    assert rel(out, ref) <= 0.05
    # and no row has another's adapter: with each row's own bar at three times that of all
    err = (out.double().cpu() - ref).norm(dim=1) / ref.norm(dim=1)
    assert float(err.max()) <= 0.15, float(err.max())


def test_two_calls_at_once_have_workspaces_of_their_own():
    """The same calls on two streams, each with its workspaces, give what they give one after the other."""
    T, K, N, R, L, E = 3000, 512, 640, 16, 7, 48
    g = torch.Generator()
    g.manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()        # noqa: E731
    sides = []
    for _ in range(2):
        s = dict(x=rnd(T, K), Y=rnd(T, N), A=rnd(L, R, K), B=rnd(L, N, R), dy=rnd(T, K), w=rnd(K), logits=rnd(T, E))
        s["adapter"] = torch.randint(-1, L, (T,), generator=g).to(I32).cuda()
        s["ids"] = torch.randint(0, E, (T, 4), generator=g).to(I32).cuda()
        s["ws"] = (mg.lora_workspace(T, K, R), mg.rms_norm_workspace(T, K), mg.balance_loss_workspace(T, E))
        sides.append(s)

    def step(s):
        new = lambda *shape, dtype=F32: torch.empty(shape, dtype=dtype, device="cuda")   # noqa: E731
        y, rstd, dx, dw, out = new(T, K, dtype=BF16), new(T), new(T, K, dtype=BF16), new(K), new(T, N, dtype=BF16)
        loss, counts = new(1), new(1, E, dtype=I32)
        mg.rms_norm(s["x"], s["w"], y=y, rstd=rstd)
        mg.lora(y, s["A"], s["B"], s["adapter"], s["Y"], out, s["ws"][0])
        mg.rms_norm_backward(s["dy"], s["x"], s["w"], rstd, dx, dw, s["ws"][1])
        mg.balance_loss(s["logits"], s["ids"], loss, counts, s["ws"][2])
        return y, out, dx, dw, loss, counts
    alone = [step(s) for s in sides]
    torch.cuda.synchronize()
    streams, both = [torch.cuda.Stream() for _ in sides], [[], []]
    for _ in range(3):
        for i, s in enumerate(sides):
            with torch.cuda.stream(streams[i]):
                both[i].append(step(s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in range(2) for run in both[i] for a, b in zip(run, alone[i]))


def test_tensors_of_another_device_than_the_current_one_are_refused(monkeypatch):
    """Launches go to the current device: without a stream the tensors have to be on it."""
    x, w, y = torch.zeros(2, 64, dtype=BF16).cuda(), torch.ones(64).cuda(), torch.zeros(2, 64, dtype=BF16).cuda()
    stream = torch.cuda.current_stream()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        mg.rms_norm(x, w, y=y)
    mg.rms_norm(x, w, y=y, stream=stream)
