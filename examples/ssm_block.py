"""A selective state space block on the package's kernels: projection, short convolution, scan,
gated norm, projection; as a prompt, as single tokens that continue it, and as a training step.  And a
stack of such blocks on a residual stream: the norm in front of each with the residual's addition, the
projections in 8 bits for serving, the clipping of a training step's gradients.

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
        self.w8 = None                          # 8-bit copies of the projections

    def cache(self, B):
        """What a sequence carries from call to call, zero before its first token."""
        dev = self.p["alpha"].device
        return dict(window=torch.zeros(B, 3, self.C, dtype=torch.bfloat16, device=dev),
                    H=torch.zeros(B, self.N, self.K, self.V, device=dev))

    def quantise(self):
        """From now on prompts and tokens go through 8-bit copies of the projections; training does not."""
        self.w8 = {n: m2.quantise_weight_fp8(self.p[n]) for n in ("w_in", "w_out")}
        return self

    def _out(self, o):
        return o @ self.p["w_out"].T if self.w8 is None else m2.linear_fp8(o, None, *self.w8["w_out"])

    def _project(self, x):
        """x [..., D] bf16, or in 8 bits with its scales (a pair)."""
        if self.w8 is None:
            z = x @ self.p["w_in"].T
        else:
            z = m2.linear_fp8(*(x if isinstance(x, tuple) else (x, None)), *self.w8["w_in"])
        return self._split(z)

    def _split(self, z):
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
        return self._out(self._mix(*self._project(x), cache))

    def forward(self, x, cache):
        """``prompt`` as ``train`` computes it: through the projections that it returns gradients of."""
        return self._mix(*self._split(x @ self.p["w_in"].T), cache) @ self.p["w_out"].T

    def _mix(self, gate, u, a, cache):
        p = self.p
        c, _ = m2.conv_silu_window(u, p["conv_w"], p["conv_b"], cache["window"], window_out=cache["window"])
        y, _ = m2.ssm_forward(self._scan_inputs(c, a, cache["H"]), H_T=cache["H"])
        return m2.gate_groupnorm(y.flatten(2), gate.contiguous(), p["norm_w"], p["norm_b"], self.N)

    def token(self, x, cache):
        """x [B, D] bf16 -> [B, D]; the cache moves on by one token, in place."""
        p = self.p
        gate, u, a = self._project(x)
        c, _ = m2.conv_silu_step(u, p["conv_w"], p["conv_b"], cache["window"])
        v, k, q = (t.contiguous() for t in self._heads(c))
        y, _ = m2.ssm_step(q, k, v, a.contiguous(), p["alpha"], p["beta"], p["w_r"], cache["H"])
        o = m2.gate_groupnorm(y.flatten(1), gate.contiguous(), p["norm_w"], p["norm_b"], self.N)
        return self._out(o)

    def train(self, x, dout):
        """Output and gradients (a dict by parameter, and ``x``) of a loss with gradient ``dout``
        at the output of a sequence from its beginning."""
        p = self.p
        gate, u, a = self._split(x @ p["w_in"].T)
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


class Stack:
    """``depth`` blocks on a float32 residual stream of D channels, a norm in front of each and one at the end."""

    def __init__(self, depth=2, D=256, seed=0, device="cuda", **kw):
        self.blocks = [Block(D=D, seed=seed + i, device=device, **kw) for i in range(depth)]
        gen = torch.Generator().manual_seed(seed + 100)
        self.norms = [(1.0 + 0.1 * torch.randn(D, generator=gen)).to(device) for _ in range(depth + 1)]

    def cache(self, B):
        return [b.cache(B) for b in self.blocks]

    def quantise(self):
        for b in self.blocks:
            b.quantise()
        return self

    def _serve(self, x, caches, form):
        h, y = None, x
        for b, w, c in zip(self.blocks, self.norms, caches):
            if b.w8 is None:
                n, h = m2.add_rmsnorm(y, h, w)
            else:
                q, scales, h = m2.add_rmsnorm_fp8(y, h, w)
                n = (q, scales)
            y = getattr(b, form)(n, c)
        return m2.add_rmsnorm(y, h, self.norms[-1])[0]

    def prompt(self, x, caches):
        """x [B, T, D] float32 -> [B, T, D] bf16; the caches move on by T tokens, in place."""
        return self._serve(x, caches, "prompt")

    def token(self, x, caches):
        """x [B, D] float32 -> [B, D] bf16; the caches move on by one token, in place."""
        return self._serve(x, caches, "token")

    def train(self, x, dout, max_norm=None):
        """Output and gradients (a dict by parameter, and ``x``) of a loss with gradient ``dout`` (bf16) at the
        output; with ``max_norm`` the parameters' gradients are clipped and their norm is returned as well.
        A block's forward runs again in its backward, from the norm's output."""
        h, y, kept = None, x, []
        for b, w in zip(self.blocks, self.norms):
            n, h = m2.add_rmsnorm(y, h, w)
            kept.append((n, h))
            y = b.forward(n, b.cache(x.shape[0]))
        out, h = m2.add_rmsnorm(y, h, self.norms[-1])
        d = m2.add_rmsnorm_backward(h, self.norms[-1], dout)
        grads = {f"norm{len(self.blocks)}": d["dw"]}
        for i in range(len(self.blocks) - 1, -1, -1):
            n, h = kept[i]
            _, g = self.blocks[i].train(n, d["dx"])
            d = m2.add_rmsnorm_backward(h, self.norms[i], g.pop("x"), d["dresidual"])
            grads.update({f"block{i}.{k}": t for k, t in g.items()}, **{f"norm{i}": d["dw"]})
        norm = None if max_norm is None else m2.clip_grad_norm(grads, max_norm)
        return out, dict(grads, x=d["dresidual"]), norm


def check_stack():
    """A prompt in two parts and single tokens against one call, in bf16 and with 8-bit projections (the largest
    difference over the largest output), the 8-bit prompt's distance from the bf16 one (2-norms), and the
    gradients' norm after a clip over the norm it was to have."""
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(2, 200, 256, generator=gen).cuda()
    found, wholes = [], []
    for stack in (Stack(), Stack().quantise()):
        whole, caches = stack.prompt(x, stack.cache(2)), stack.cache(2)
        parts = [stack.prompt(x[:, :95].contiguous(), caches), stack.prompt(x[:, 95:192].contiguous(), caches)]
        parts += [stack.token(x[:, t].contiguous(), caches)[:, None] for t in range(192, 200)]
        found.append(float((torch.cat(parts, 1).float() - whole.float()).abs().max() / whole.float().abs().max()))
        wholes.append(whole.float())
    far = float((wholes[1] - wholes[0]).norm() / wholes[0].norm())
    dout = torch.randn(2, 200, 256, generator=gen).to(torch.bfloat16).cuda()
    _, g, norm = Stack().train(x, dout, max_norm=1.0)
    clipped = float(m2.grad_norm([t for n, t in g.items() if n != "x"]))
    if m2.stream_status() != 0:
        raise RuntimeError("a kernel's wait ran out")
    return found, far, clipped if float(norm) > 1.0 else None


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
    parts, far, clipped = check_stack()
    print(f"stack: parts against one call {parts[0]:.1e} (bf16), {parts[1]:.1e} (8 bits); 8 bits against bf16 {far:.1e}; "
          f"norm after the clip {clipped}")
