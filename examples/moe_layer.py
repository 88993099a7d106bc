"""One mixture-of-experts layer on one GPU, from router logits to gradients, out of the library's calls.

    python examples/moe_layer.py [--tokens 4096 --experts 64 --top-k 8 --hidden 7168 --inter 2048 --steps 10]

MoELayer.forward / backward is a training step in fp8 (e4m3 operands with fp32 scales, [K/128, rows] for activations):

    route -> dispatch -> W1 product -> SwiGLU with an 8-bit checkpoint -> W2 product -> combine

What forward keeps for backward: the fp8 input rows (hidden + hidden / 32 bytes a row) and the fp8 gate/up columns
(2 inter + inter / 16), a little over half of what bf16 would take, plus the router's choice.  MoELayer.decode is
the same layer without a checkpoint for a few tokens: five calls that a graph can capture.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_sizes_amd as mg  # noqa: E402

E4M3, BF16, F32, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32


def quantize_weight(w: torch.Tensor):
    """[G, N, K] -> e4m3 [G, N, K] and fp32 scales [G, K/128, N/128] of 128x128 blocks."""
    G, N, K = w.shape
    b = w.float().reshape(G, N // 128, 128, K // 128, 128)
    s = b.abs().amax(dim=(2, 4)) / 448
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (b / s[:, :, None, :, None]).clamp(-448, 448).to(E4M3).reshape(G, N, K)
    return q, s.transpose(1, 2).contiguous()


class MoELayer:
    """router [E, hidden] bf16; W1 [E, 2 inter, hidden] (gate and up rows interleaved), W2 [E, hidden, inter]."""

    def __init__(self, router, w_gate, w_up, w_down, top_k: int, max_tokens: int, scale: float = 1.0):
        self.router, self.k, self.scale = router, top_k, scale
        self.E, self.inter, self.hidden = w_gate.shape
        self.W1, self.W1_scale = quantize_weight(mg.interleave_gate_up(w_gate, w_up))
        self.W2, self.W2_scale = quantize_weight(w_down)
        # the same weights as [G, K, N] operands of the input gradients' products
        self.W1_scale_t = self.W1_scale.transpose(1, 2).contiguous()
        self.W2_scale_t = self.W2_scale.transpose(1, 2).contiguous()
        dev = router.device
        self.ws = mg.workspace(self.E, max_tokens * top_k, dev)
        self.route_ws = mg.route_workspace(max_tokens, self.E, dev)
        self.dev = dev

    def _new(self, *shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.dev)

    def _fp8(self, rows, width):
        return self._new(rows, width, dtype=E4M3), self._new(width // 128, rows, dtype=F32)

    def _route(self, x):
        T = x.shape[0]
        logits = x @ self.router.t()
        r = dict(logits=logits, ids=self._new(T, self.k, dtype=I32), weights=self._new(T, self.k, dtype=F32),
                 m_sizes=self._new(self.E, dtype=I32), row_of=self._new(T, self.k, dtype=I32))
        mg.route(logits, r["ids"], r["weights"], r["m_sizes"], r["row_of"], self.route_ws, rows_total=T * self.k,
                 scale=self.scale)
        return r

    def forward(self, x):
        """out bf16 [T, hidden], and what backward needs."""
        rows, I, K = x.shape[0] * self.k, self.inter, self.hidden
        r = self._route(x)
        A, A_scale = self._fp8(rows, K)
        mg.dispatch(x, r["row_of"], A, A_scale, scale_km=True)
        mg.schedule(r["m_sizes"], rows, self.ws, N=2 * I)
        GU = self._new(rows, 2 * I, dtype=BF16)
        mg.grouped_gemm_contiguous_scheduled(A, self.W1, GU, self.E, self.ws, A_scale, self.W1_scale, b_layout=mg.B_NK,
                                             scale_km=True)
        H, H_scale = self._fp8(rows, I)
        ckpt, ckpt_scale = self._new(rows, 2 * I, dtype=E4M3), self._new(rows, 2 * I // 128, dtype=F32)
        mg.swiglu_checkpoint(GU, r["m_sizes"], H, ckpt, ckpt_scale, H_scale, scale_km=True)
        Y = self._new(rows, K, dtype=BF16)
        mg.grouped_gemm_contiguous_scheduled(H, self.W2, Y, self.E, self.ws, H_scale, self.W2_scale, b_layout=mg.B_NK,
                                             scale_km=True)
        out = self._new(x.shape[0], K, dtype=BF16)
        mg.combine(Y, r["row_of"], out, r["weights"])
        return out, dict(r, x=x, A=A, A_scale=A_scale, ckpt=ckpt, ckpt_scale=ckpt_scale, Y=Y)

    def backward(self, dout, kept, d_logits_of=None):
        """Gradients of x (bf16), the router (a bf16 product, as fp32) and the expert weights: W1 fp32 [E, hidden,
        2 inter] and W2 [E, inter, hidden], as the K-grouped product writes them.  d_logits_of: adds what else the logits
        get (of a balance loss) to their gradient, in place."""
        T, rows, I, K, E = dout.shape[0], dout.shape[0] * self.k, self.inter, self.hidden, self.E
        m, row_of = kept["m_sizes"], kept["row_of"]
        dY, dY_scale = self._fp8(rows, K)
        d_weights = self._new(T, self.k, dtype=F32)
        mg.combine_backward(dout, kept["Y"], kept["weights"], row_of, dY, d_weights, dY_scale, scale_km=True)
        dH = self._new(rows, I, dtype=BF16)
        mg.schedule(m, rows, self.ws, N=I)
        mg.grouped_gemm_contiguous_scheduled(dY, self.W2, dH, E, self.ws, dY_scale, self.W2_scale_t, b_layout=mg.B_KN,
                                             scale_km=True)
        S = rows // 128 + E                                # token groups of any histogram
        dGU, dGU_scale = self._fp8(rows, 2 * I)
        dGU_k, dGU_ks = self._new(rows, 2 * I, dtype=E4M3), self._new(S, 2 * I, dtype=F32)
        H_k, H_ks = self._new(rows, I, dtype=E4M3), self._new(S, I, dtype=F32)
        mg.swiglu_checkpoint_backward_fp8(dH, m, kept["ckpt"], kept["ckpt_scale"], dGU, dGU_scale, dGU_k, dGU_ks, H_k,
                                          H_ks, scale_km=True)
        dX = self._new(rows, K, dtype=BF16)
        mg.grouped_gemm_contiguous_scheduled(dGU, self.W1, dX, E, self.ws, dGU_scale, self.W1_scale_t, b_layout=mg.B_KN,
                                             scale_km=True)
        dx = self._new(T, K, dtype=BF16)
        mg.combine(dX, row_of, dx)
        # weight gradients, with scales along the tokens
        A_k, A_ks = self._new(rows, K, dtype=E4M3), self._new(S, K, dtype=F32)
        dY_k, dY_ks = self._new(rows, K, dtype=E4M3), self._new(S, K, dtype=F32)
        mg.checkpoint_to_k_groups(kept["A"], m, A_k, A_ks, kept["A_scale"], scale_km=True)
        mg.checkpoint_to_k_groups(dY, m, dY_k, dY_ks, dY_scale, scale_km=True)
        dW1, dW2 = self._new(E, K, 2 * I, dtype=F32), self._new(E, I, K, dtype=F32)
        mg.grouped_gemm_k_grouped(A_k, dGU_k, dW1, m, self.ws, A_ks, dGU_ks)
        mg.grouped_gemm_k_grouped(H_k, dY_k, dW2, m, self.ws, H_ks, dY_ks)
        d_logits = self._new(T, E, dtype=kept["logits"].dtype)
        mg.route_backward(kept["logits"], kept["ids"], d_weights, d_logits, scale=self.scale)
        if d_logits_of is not None:
            d_logits_of(d_logits)
        dx += d_logits @ self.router
        return dict(x=dx, router=(d_logits.t() @ kept["x"]).float(), W1=dW1, W2=dW2)

    def decode(self, x):
        """out bf16 [T, hidden] of a few tokens: both projections in one call, nothing kept."""
        rows = x.shape[0] * self.k
        r = self._route(x)
        A, A_scale = self._fp8(rows, self.hidden)
        mg.dispatch(x, r["row_of"], A, A_scale, scale_km=True)
        H, H_scale = self._fp8(rows, self.inter)
        Y, out = self._new(rows, self.hidden, dtype=BF16), self._new(x.shape[0], self.hidden, dtype=BF16)
        mg.expert_mlp_fused(A, self.W1, self.W2, H, Y, r["m_sizes"], self.ws, A_scale, self.W1_scale, self.W2_scale,
                            H_scale, scale_km=True)
        mg.combine(Y, r["row_of"], out, r["weights"])
        return out


def random_layer(experts, hidden, inter, top_k, max_tokens, seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rnd = lambda *s, std: (torch.randn(*s, generator=g, device=device) * std).to(BF16)   # noqa: E731
    return MoELayer(rnd(experts, hidden, std=hidden ** -0.5), rnd(experts, inter, hidden, std=hidden ** -0.5),
                    rnd(experts, inter, hidden, std=hidden ** -0.5), rnd(experts, hidden, inter, std=inter ** -0.5),
                    top_k, max_tokens)


def timed(f, steps):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(steps):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / steps


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--top-k", type=int, default=8)
    p.add_argument("--hidden", type=int, default=7168)
    p.add_argument("--inter", type=int, default=2048)
    p.add_argument("--steps", type=int, default=10)
    a = p.parse_args()
    layer = random_layer(a.experts, a.hidden, a.inter, a.top_k, a.tokens)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(BF16)
    dout = torch.randn(a.tokens, a.hidden, device="cuda").to(BF16)
    out, kept = layer.forward(x)
    grads = layer.backward(dout, kept)
    size = sum(kept[n].numel() * kept[n].element_size() for n in ("A", "A_scale", "ckpt", "ckpt_scale"))
    print(f"{a.tokens} tokens, {a.experts} experts, top {a.top_k}, hidden {a.hidden}, inter {a.inter}: "
          f"out {list(out.shape)}, gradients {({n: list(v.shape) for n, v in grads.items()})}")
    print(f"kept in 8 bits: {size / 2**20:.0f} MiB")
    print(f"forward {timed(lambda: layer.forward(x), a.steps):.3f} ms, "
          f"backward {timed(lambda: layer.backward(dout, kept), a.steps):.3f} ms", flush=True)
    few = x[:16].contiguous()
    layer.decode(few)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.decode(few)
    print(f"decode of 16 tokens: {timed(lambda: layer.decode(few), a.steps):.3f} ms, "
          f"as a graph {timed(graph.replay, a.steps):.3f} ms", flush=True)


if __name__ == "__main__":
    main()
