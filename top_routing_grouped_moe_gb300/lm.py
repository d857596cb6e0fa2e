"""A small language model around `MoELayer`, as a training step runs the
library: token embedding, blocks of (norm, MoE layer, norm and residual), the
vocabulary's cross entropy, their backward, and the clipping of all gradients by
their global norm.  Every step of it is a C-ABI call on one stream; this module
owns the buffers and holds no arithmetic of its own but the plain SGD update of
the example.

    python -m top_routing_grouped_moe_gb300.lm --steps 20

trains on synthetic token sequences (each token's successor is a fixed function
of it) and prints the loss and the gradient norm of every step."""
from __future__ import annotations

import argparse
import math

import torch

from . import _binding as B
from .layer import MoELayer

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


class MoELM:
    """Buffers and call sequence of one model shape.

    T tokens per step, vocabulary V, width d, `blocks` MoE layers of E experts,
    k per token, hidden width H (shared expert Hs).  tied: the head is the
    embedding table.  r_scale multiplies every block's branch."""

    def __init__(self, T, V, d, blocks, E, k, H, Hs, tied=True, r_scale=1.0, z_weight=0.0, max_norm=1.0,
                 device="cuda"):
        self.T, self.V, self.d, self.blocks, self.tied = T, V, d, blocks, tied
        self.scale, self.r_scale, self.z_weight, self.max_norm = math.sqrt(d), float(r_scale), z_weight, max_norm
        dev = self.device = torch.device(device)
        e = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        self.layers = [MoELayer(T, d, E, k, H, Hs, device=dev) for _ in range(blocks)]
        # the residual stream and the normed input of every block (and of the head)
        self.r = [e(T, d) for _ in range(blocks + 1)]
        self.x = [e(T, d) for _ in range(blocks + 1)]
        self.rstd_pre = [e(T, dt=F32) for _ in range(blocks + 1)]
        self.rstd_post = [e(T, dt=F32) for _ in range(blocks)]
        self.loss, self.lse = e(T, dt=F32), e(T, dt=F32)
        # gradients of the activations: two of the stream, in turn
        self.dr = [e(T, d), e(T, d)]
        self.dx, self.dy = e(T, d), e(T, d)
        # gradients of the weights, one tensor each
        self.grads = {"table": e(V, d)}
        if not tied:
            self.grads["head"] = e(V, d)
        for i, layer in enumerate(self.layers):
            self.grads[f"{i}.w_post"] = e(d, dt=F32)
            for name in ("W_r", "W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d"):
                g = getattr(layer, "d" + name)
                if g is not None:
                    self.grads[f"{i}.{name}"] = g
        for i in range(blocks + 1):
            self.grads[f"{i}.w_pre"] = e(d, dt=F32)
        self.norm, self.coef = e(1, dt=F32), e(1, dt=F32)
        self.clip = B.GradList(self.grads.values(), self.grads.values())
        self.ws_bytes = max(B.moe_cross_entropy_workspace(T, d, V), B.moe_embedding_workspace(T, V, d),
                            B.moe_residual_norm_workspace(T, d), B.moe_grad_clip_workspace(self.clip))
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)

    def init_weights(self, seed=0, std=0.02):
        """Random weights: {"table", "head" (untied), "i.w_pre", "i.w_post",
        "i.W_r", "i.W_g", ...}, bf16."""
        g = torch.Generator(device=self.device).manual_seed(seed)
        p = {}
        for name, grad in self.grads.items():
            if name.endswith(("w_pre", "w_post")):
                p[name] = torch.ones(self.d, dtype=BF16, device=self.device)
            else:
                w = torch.randn(*grad.shape, generator=g, device=self.device)
                p[name] = (w * (1.0 / math.sqrt(self.d) if name == "table" else std)).to(BF16)
        return p

    def _layer_weights(self, p, i):
        names = ("W_r", "W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d")
        return {n: p[f"{i}.{n}"] for n in names if f"{i}.{n}" in p}

    def forward(self, ids, targets, p, stream=None):
        """Per-token losses [T] fp32 (0 where the target is negative), for ids
        and targets [T] int32, contiguous (another type is refused).  A padding
        token (negative id) needs a negative target: its row is zero, whose norm
        has a gain of 1/sqrt(eps) per block in the backward, and a gradient of
        that size would take the range of the layer's fp16 gradient terms from
        the other tokens (they are scaled by the largest)."""
        T, V, d = self.T, self.V, self.d
        B.moe_embedding(p["table"], ids, T, V, d, self.scale, self.r[0], stream)
        B.moe_residual_norm(self.r[0], None, None, B.MOE_GATE_NONE, None, p["0.w_pre"], T, d, False, 1.0, EPS, None,
                            self.x[0], None, self.rstd_pre[0], stream)
        for i, layer in enumerate(self.layers):
            y = layer.forward(self.x[i], self._layer_weights(p, i), stream=stream)
            B.moe_residual_norm(self.r[i], y, None, B.MOE_GATE_NONE, p[f"{i}.w_post"], p[f"{i + 1}.w_pre"], T, d,
                                False, self.r_scale, EPS, self.r[i + 1], self.x[i + 1], self.rstd_post[i],
                                self.rstd_pre[i + 1], stream)
        B.moe_cross_entropy(self.x[-1], p["table" if self.tied else "head"], targets, T, d, V, self.z_weight,
                            self.loss, self.lse, self.ws, self.ws_bytes, stream)
        return self.loss

    def backward(self, ids, targets, dloss, p, stream=None):
        """Backward of the last forward for dloss [T] fp32: fills self.grads."""
        T, V, d, g, ws, n = self.T, self.V, self.d, self.grads, self.ws, self.ws_bytes
        head = "table" if self.tied else "head"
        B.moe_cross_entropy_bwd(self.x[-1], p[head], targets, self.lse, dloss, T, d, V, self.z_weight, 0, self.dx,
                                g[head], ws, n, stream)
        dx = self.dx  # gradient of the normed input, from the head and then from each layer's own buffer
        up = None  # gradient of the residual stream from the blocks above
        for i in reversed(range(self.blocks)):
            layer, dr = self.layers[i], self.dr[i & 1]
            B.moe_residual_norm_bwd(dx, up, layer.y, None, B.MOE_GATE_NONE, p[f"{i}.w_post"],
                                    p[f"{i + 1}.w_pre"], self.r[i + 1], self.rstd_post[i], self.rstd_pre[i + 1], T, d,
                                    False, self.r_scale, dr, self.dy, None, g[f"{i}.w_post"], g[f"{i + 1}.w_pre"], ws,
                                    n, stream)
            dx = layer.backward(self.x[i], self.dy, self._layer_weights(p, i), stream=stream)
            up = dr
        dr = self.dr[self.blocks & 1]
        B.moe_residual_norm_bwd(dx, up, None, None, B.MOE_GATE_NONE, None, p["0.w_pre"], self.r[0], None,
                                self.rstd_pre[0], T, d, False, 1.0, dr, None, None, None, g["0.w_pre"], ws, n, stream)
        B.moe_embedding_bwd(dr, ids, T, V, d, self.scale, self.tied, g["table"], ws, n, stream)
        return g

    def clip_gradients(self, stream=None):
        """Scales self.grads in place by min(1, max_norm / global norm)."""
        B.moe_grad_clip(self.clip, self.max_norm, self.norm, self.coef, self.ws, self.ws_bytes, stream)
        return self.norm


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--lr", type=float, default=0.5)
    a = ap.parse_args(argv)
    torch.cuda.set_device(0)
    m = MoELM(a.tokens, a.vocab, a.width, a.blocks, E=8, k=2, H=256, Hs=128, z_weight=1e-4)
    p = m.init_weights()
    gen = torch.Generator(device="cuda").manual_seed(1)
    dloss = torch.full((a.tokens,), 1.0 / a.tokens, device="cuda")
    losses = []
    for step in range(a.steps):
        ids = torch.randint(0, a.vocab, (a.tokens,), generator=gen, device="cuda", dtype=torch.int32)
        targets = (ids * 7 + 3) % a.vocab
        loss = m.forward(ids, targets, p).mean()
        m.backward(ids, targets, dloss, p)
        m.clip_gradients()
        for name, g in m.grads.items():
            p[name].add_(g.to(BF16), alpha=-a.lr)
        losses.append(float(loss))
        print(f"step {step}: loss {losses[-1]:.4f}, gradient norm {float(m.norm):.4f}", flush=True)
    status = B.moe_device_status()
    if status:
        raise RuntimeError(B.status_string(status))
    return losses


if __name__ == "__main__":
    main()
