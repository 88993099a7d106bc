"""What stands around the mixture-of-experts layer of moe_layer.py, out of the library's calls.

    python examples/moe_block.py [--tokens 4096 --experts 64 --top-k 8 --hidden 7168 --inter 2048 --steps 10]

MoEBlock is a training step: the residual's addition and the norm, the layer, and the router's balance and z loss of every
sequence, whose gradients meet those of the routing weights in the logits:

    h = x + residual;  out = layer(norm(h));  losses of the layer's logits

Projection is a projection that many requests share, in fp8, with each request's low-rank adapter: the norm writes its
e4m3 operand and the adapters' bf16 input in one pass.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_sizes_amd as mg  # noqa: E402
from examples.moe_layer import random_layer, quantize_weight, timed  # noqa: E402

E4M3, BF16, F32, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32


class MoEBlock:
    """norm_weight [hidden]; balance and z: what the two losses count for, over the mean of the sequences."""

    def __init__(self, layer, norm_weight, max_tokens: int, max_sequences: int, balance: float = 0.01, z: float = 0.001,
                 eps: float = 1e-6):
        self.layer, self.weight, self.eps = layer, norm_weight, eps
        self.balance, self.z = balance, z
        self.norm_ws = mg.rms_norm_workspace(max_tokens, layer.hidden, layer.dev)
        self.loss_ws = mg.balance_loss_workspace(max_tokens, layer.E, max_sequences, layer.dev)

    def forward(self, x, residual, offsets):
        """out and h bf16 [T, hidden], the losses fp32 [S] of the sequences offsets [S + 1] bound, and what backward
        needs."""
        new, T, S = self.layer._new, x.shape[0], offsets.numel() - 1
        h, y, rstd = torch.empty_like(x), torch.empty_like(x), new(T, dtype=F32)
        mg.rms_norm(x, self.weight, residual=residual, sum_out=h, y=y, rstd=rstd, eps=self.eps)
        out, kept = self.layer.forward(y)
        loss, z, counts = new(S, dtype=F32), new(S, dtype=F32), new(S, self.layer.E, dtype=I32)
        mg.balance_loss(kept["logits"], kept["ids"], loss, counts, self.loss_ws, z_loss=z, seq_offsets=offsets)
        return out, h, dict(balance=loss, z=z), dict(kept, h=h, rstd=rstd, counts=counts, offsets=offsets)

    def backward(self, dout, dh, kept):
        """The layer's gradients, with that of x and of the residual alike as x, and the norm's weight's."""
        S = kept["offsets"].numel() - 1
        d_loss, d_z = (torch.full((S,), v / S, device=dout.device) for v in (self.balance, self.z))

        def losses(d_logits):
            mg.balance_loss_backward(kept["logits"], kept["counts"], d_loss, d_logits, k=self.layer.k, d_z_loss=d_z,
                                     seq_offsets=kept["offsets"], before=d_logits)
        grads = self.layer.backward(dout, kept, losses)
        dx, d_weight = torch.empty_like(dout), torch.empty(dout.shape[1], device=dout.device)
        mg.rms_norm_backward(grads["x"], kept["h"], self.weight, kept["rstd"], dx, d_weight, self.norm_ws, d_sum=dh)
        return dict(grads, x=dx, norm=d_weight)


class Projection:
    """w [N, hidden] bf16, shared; adapters A [L, R, hidden], B [L, N, R] bf16 with fp32 scale [L]."""

    def __init__(self, norm_weight, w, A, B, scale, max_tokens: int, eps: float = 1e-6):
        self.norm, self.eps, self.A, self.B, self.scale = norm_weight, eps, A, B, scale
        self.W, self.W_scale = quantize_weight(w[None])
        self.ws = mg.workspace(1, max_tokens, w.device)
        self.lora_ws = mg.lora_workspace(max_tokens, w.shape[1], A.shape[1], w.device)

    def __call__(self, x, residual, adapter):
        """out bf16 [T, N] and h = x + residual; adapter int32 [T], -1 for a row without one."""
        T, K = x.shape
        h, y, dev = torch.empty_like(x), torch.empty_like(x), x.device
        q, q_scale = torch.empty(T, K, dtype=E4M3, device=dev), torch.empty(K // 128, T, device=dev)
        mg.rms_norm(x, self.norm, residual=residual, sum_out=h, y=y, q=q, q_scale=q_scale, eps=self.eps, scale_km=True)
        out = torch.empty(T, self.W.shape[1], dtype=BF16, device=dev)
        rows = torch.full((1,), T, dtype=I32, device=dev)
        mg.grouped_gemm_contiguous(q, self.W, out, rows, self.ws, q_scale, self.W_scale, b_layout=mg.B_NK, scale_km=True)
        mg.lora(y, self.A, self.B, adapter, out, out, self.lora_ws, scale=self.scale)
        return out, h


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--top-k", type=int, default=8)
    p.add_argument("--hidden", type=int, default=7168)
    p.add_argument("--inter", type=int, default=2048)
    p.add_argument("--steps", type=int, default=10)
    a = p.parse_args()
    T, K = a.tokens, a.hidden
    rnd = lambda *s: torch.randn(*s, device="cuda")          # noqa: E731
    block = MoEBlock(random_layer(a.experts, K, a.inter, a.top_k, T), torch.ones(K, device="cuda"), T, 4)
    x, residual, dout, dh = (rnd(T, K).to(BF16) for _ in range(4))
    offsets = torch.tensor([0, T // 8, T // 2, T // 2, T], dtype=I32, device="cuda")
    out, _, losses, kept = block.forward(x, residual, offsets)
    grads = block.backward(dout, dh, kept)
    print(f"out {list(out.shape)}, balance losses {losses['balance'].tolist()}, z losses {losses['z'].tolist()}")
    print(f"gradients {({n: list(v.shape) for n, v in grads.items()})}")
    print(f"forward {timed(lambda: block.forward(x, residual, offsets), a.steps):.3f} ms, "
          f"backward {timed(lambda: block.backward(dout, dh, kept), a.steps):.3f} ms", flush=True)
    L, R = 16, 16
    shared = Projection(torch.ones(K, device="cuda"), (rnd(4096, K) * K ** -0.5).to(BF16), (rnd(L, R, K) * K ** -0.5).to(BF16),
                        (rnd(L, 4096, R) * R ** -0.5).to(BF16), torch.ones(L, device="cuda"), T)
    for n in (96, T):
        adapter = (torch.arange(n, device="cuda") % (L + 1) - 1).to(I32)
        xs, rs = x[:n].contiguous(), residual[:n].contiguous()
        print(f"projection of {n} rows: {timed(lambda: shared(xs, rs, adapter), a.steps):.3f} ms", flush=True)


if __name__ == "__main__":
    main()
