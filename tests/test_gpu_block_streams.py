"""The block's calls with a stream given, on MI355X: the bits of the current stream's calls, and a stream of another device is
refused before anything is launched."""
from types import SimpleNamespace

import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_gpu_layer import gen

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def step(s, stream):
    new = lambda *shape, dtype=F32: torch.empty(shape, dtype=dtype, device="cuda")   # noqa: E731
    (T, K), E = s["x"].shape, s["logits"].shape[1]
    y, rstd, dx, dw, out = new(T, K, dtype=BF16), new(T), new(T, K, dtype=BF16), new(K), new(T, K, dtype=BF16)
    loss, counts, dl, ws = new(1), new(1, E, dtype=I32), new(T, E), s["ws"]
    mg.rms_norm(s["x"], s["w"], y=y, rstd=rstd, stream=stream)
    mg.rms_norm_backward(s["dy"], s["x"], s["w"], rstd, dx, dw, ws[0], stream=stream)
    mg.balance_loss(s["logits"], s["ids"], loss, counts, ws[1], stream=stream)
    mg.balance_loss_backward(s["logits"], counts, loss, dl, k=2, stream=stream)
    mg.lora(y, s["A"], s["B"], s["adapter"], s["dy"], out, ws[2], stream=stream)
    return y, rstd, dx, dw, loss, counts, dl, out


def state():
    T, K, E, R, L = 300, 512, 40, 16, 3
    g = gen(1)
    rnd = lambda *s, dtype=BF16: torch.randn(*s, generator=g).to(dtype).cuda()       # noqa: E731
    return dict(x=rnd(T, K), dy=rnd(T, K), w=rnd(K), logits=rnd(T, E, dtype=F32), A=rnd(L, R, K), B=rnd(L, K, R),
                ids=torch.randint(0, E, (T, 2), generator=g).to(I32).cuda(),
                adapter=torch.randint(-1, L, (T,), generator=g).to(I32).cuda(),
                ws=(mg.rms_norm_workspace(T, K), mg.balance_loss_workspace(T, E), mg.lora_workspace(T, K, R)))


def test_a_stream_given():
    s = state()
    want = step(s, None)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.default_stream(), torch.cuda.current_stream()):
        got = step(s, stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_stream_of_another_device_is_refused():
    for handle in (0, torch.cuda.Stream().cuda_stream):
        with pytest.raises(ValueError, match="tensors on cuda:0, stream of cuda:1"):
            step(state(), SimpleNamespace(device_index=1, cuda_stream=handle))
