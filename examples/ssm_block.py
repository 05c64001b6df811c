"""A selective state space block on the package's kernels: projection, short convolution, scan,
gated norm, projection; as a prompt, as single tokens that continue it, and as a training step.

    python examples/ssm_block.py

Between the projections (plain matrix products) the convolution reads a slice of the input projection
and the scan of a prompt slices of the convolution's output, without copies.  What the operators take
dense is copied: the norm's gate, a single token's v, k, q and a, and, in training, dv, dk and dq side
by side for the convolution's backward.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_state_nonlinear_gb300 as m2  # noqa: E402


class Block:
    """``D`` model channels, ``N`` heads of ``V`` values, ``G`` shared q, k heads of ``K``."""

    def __init__(self, D=256, N=6, G=2, K=64, V=64, seed=0, device="cuda"):
        self.N, self.G, self.K, self.V = N, G, K, V
        self.C = N * V + 2 * G * K              # channels of the convolution: v, k, q
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s, scale=1.0, dtype=torch.float32: (  # noqa: E731
            torch.randn(s, generator=gen) * scale).to(dtype).to(device)
        # rows: gate of the norm, channels of the convolution, logits of the scan (to a multiple of 8)
        self.rows = N * V + self.C + (N + 7) // 8 * 8
        self.p = dict(
            w_in=rand(self.rows, D, scale=D ** -0.5, dtype=torch.bfloat16),
            w_out=rand(D, N * V, scale=(N * V) ** -0.5, dtype=torch.bfloat16),
            conv_w=rand(self.C, 4, scale=0.5), conv_b=rand(self.C, scale=0.1),
            alpha=torch.exp(rand(N, scale=0.5)), beta=rand(N), w_r=rand(N, V),
            norm_w=1.0 + rand(N * V, scale=0.1), norm_b=rand(N * V, scale=0.1))

    def cache(self, B):
        """What a sequence carries from call to call, zero before its first token."""
        dev = self.p["alpha"].device
        return dict(window=torch.zeros(B, 3, self.C, dtype=torch.bfloat16, device=dev),
                    H=torch.zeros(B, self.N, self.K, self.V, device=dev))

    def _project(self, x):
        z = x @ self.p["w_in"].T
        nv = self.N * self.V
        return z[..., :nv], z[..., nv:nv + self.C], z[..., nv + self.C:nv + self.C + self.N]

    def _heads(self, c):
        """v, k, q as slices of the convolution's output."""
        nv, gk = self.N * self.V, self.G * self.K
        return (c[..., :nv].unflatten(-1, (self.N, self.V)), c[..., nv:nv + gk].unflatten(-1, (self.G, self.K)),
                c[..., nv + gk:].unflatten(-1, (self.G, self.K)))

    def _scan_inputs(self, c, a, H0):
        v, k, q = self._heads(c)
        return dict(q=q, k=k, v=v, a=a, H0=H0, **{n: self.p[n] for n in ("alpha", "beta", "w_r")})

    def prompt(self, x, cache):
        """x [B, T, D] bf16 -> [B, T, D]; the cache moves on by T tokens, in place."""
        p = self.p
        gate, u, a = self._project(x)
        c, _ = m2.conv_silu_window(u, p["conv_w"], p["conv_b"], cache["window"], window_out=cache["window"])
        y, _ = m2.ssm_forward(self._scan_inputs(c, a, cache["H"]), H_T=cache["H"])
        o = m2.gate_groupnorm(y.flatten(2), gate.contiguous(), p["norm_w"], p["norm_b"], self.N)
        return o @ p["w_out"].T

    def token(self, x, cache):
        """x [B, D] bf16 -> [B, D]; the cache moves on by one token, in place."""
        p = self.p
        gate, u, a = self._project(x)
        c, _ = m2.conv_silu_step(u, p["conv_w"], p["conv_b"], cache["window"])
        v, k, q = (t.contiguous() for t in self._heads(c))
        y, _ = m2.ssm_step(q, k, v, a.contiguous(), p["alpha"], p["beta"], p["w_r"], cache["H"])
        o = m2.gate_groupnorm(y.flatten(1), gate.contiguous(), p["norm_w"], p["norm_b"], self.N)
        return o @ p["w_out"].T

    def train(self, x, dout):
        """Output and gradients (a dict by parameter, and ``x``) of a loss with gradient ``dout``
        at the output of a sequence from its beginning."""
        p = self.p
        gate, u, a = self._project(x)
        gate = gate.contiguous()
        c, _ = m2.conv_silu_window(u, p["conv_w"], p["conv_b"])
        s = self._scan_inputs(c, a, None)
        y, _, Hs = m2.ssm_forward_train(s)
        y = y.flatten(2)
        o = m2.gate_groupnorm(y, gate, p["norm_w"], p["norm_b"], self.N)
        out = o @ p["w_out"].T

        g = {"w_out": dout.flatten(0, 1).T @ o.flatten(0, 1)}
        n = m2.gate_groupnorm_backward(y, gate, p["norm_w"], p["norm_b"], dout @ p["w_out"], self.N)
        d = m2.ssm_backward(s, Hs, n["dy"].unflatten(-1, (self.N, self.V)))
        dc = torch.cat([d["dv"].flatten(2), d["dk"].flatten(2), d["dq"].flatten(2)], -1)
        e = m2.conv_silu_backward(u, p["conv_w"], p["conv_b"], dc)
        dz = torch.cat([n["dg_pre"], e["dx"], d["da"],
                        d["da"].new_zeros(*x.shape[:2], self.rows - self.N * self.V - self.C - self.N)], -1)
        g.update(w_in=dz.flatten(0, 1).T @ x.flatten(0, 1), conv_w=e["dw"], conv_b=e["dbias"], alpha=d["dalpha"],
                 beta=d["dbeta"], w_r=d["dw_r"], norm_w=n["dw"], norm_b=n["dbias"], x=dz @ p["w_in"])
        return out, g


def check(steps=5):
    """A prompt in two parts and single tokens against one call (the largest difference over the
    largest output), and the losses of a few steps of descent towards a random target."""
    block = Block()
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(2, 300, 256, generator=gen).to(torch.bfloat16).cuda()
    whole, cache = block.prompt(x, block.cache(2)), block.cache(2)
    parts = [block.prompt(x[:, :157], cache), block.prompt(x[:, 157:290], cache)]
    parts += [block.token(x[:, t], cache)[:, None] for t in range(290, 300)]
    split = float((torch.cat(parts, 1).float() - whole.float()).abs().max() / whole.float().abs().max())

    target = torch.randn(2, 300, 256, generator=gen).cuda()
    losses = []
    for _ in range(steps):
        out = block.prompt(x, block.cache(2)).float()
        losses.append(float(((out - target) ** 2).sum() / 2))
        _, g = block.train(x, (out - target).to(torch.bfloat16))
        for n, p in block.p.items():  # a thousandth of each parameter's size
            if p.dtype is torch.float32:
                p.sub_(g[n], alpha=1e-3 * float(p.norm() / g[n].norm()))
    if m2.stream_status() != 0:
        raise RuntimeError("a kernel's wait ran out")
    return split, losses


if __name__ == "__main__":
    split, losses = check()
    print(f"prompt in parts and tokens against one call: {split:.1e} of the largest output")
    print("loss of each step:", " ".join(f"{x:.0f}" for x in losses))
    if not (split < 2.0 ** -5 and all(b < a for a, b in zip(losses, losses[1:]))):
        raise SystemExit("the parts disagree, or a step did not lower the loss")
