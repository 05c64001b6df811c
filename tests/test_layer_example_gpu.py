"""The norms, 8-bit projections and the clip together, as the stack of the example uses them.

The gradients are compared with those of the same stack in 64 bits, made by automatic differentiation of the
definitions.  A token's part of a gradient passes about 8 roundings to bf16 per block forwards and 8 backwards,
of 2^-9 of the value in the mean square each at most; 32 of them in two blocks are 1.1e-2, held to 2^-5.  A
parameter's gradient is the sum of the tokens' parts, which may cancel where their errors, of independent
roundings, do not: it is held to 2^-5 of the 2-norm of all parts together.  To see the parts, every parameter
is given to the reference once per token.
8-bit operands are off by up to 2^-4, in the mean square 2^-5.3 (uniform within a step of a binade); a product
of two 2^-4.8, and its sum over K independent terms the same of the terms' 2-norm.  Four such products in a
row, the residual stream between them: 2^-2 holds.
"""
import numpy as np
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from examples.ssm_block import Stack, check_stack
from test_layer_gpu import built  # noqa: F401

pytestmark = pytest.mark.gpu


def test_check_stack():
    parts, far, clipped = check_stack()
    # bf16: one call and parts differ by bf16 roundings of the scan's operands, 2^-5 of the largest output; 8 bits: a
    # value next to a border of e4m3 may fall on either side, 2^-3 of it
    assert parts[0] < 2.0 ** -5 and parts[1] < 2.0 ** -2 and far < 2.0 ** -2
    # clipped matrices are bf16: each value within 2^-8 of it
    assert abs(clipped - 1.0) < 2.0 ** -8 + 2.0 ** -20


def silu(x):
    return x * torch.sigmoid(x)


def block64(b, p, n):
    """One block in 64 bits from its parameters of each token, token by token."""
    B, T, _ = n.shape
    nv, gk = b.N * b.V, b.G * b.K
    apply = lambda w, x: torch.einsum("btoi,bti->bto", w, x)  # noqa: E731
    z = apply(p["w_in"], n)
    gate, u, a = z[..., :nv], z[..., nv:nv + b.C], z[..., nv + b.C:nv + b.C + b.N]
    X = torch.cat([u.new_zeros(B, 3, b.C), u], 1)
    c = silu(sum(X[:, j:j + T] * p["conv_w"][..., j] for j in range(4)) + p["conv_b"])
    v, k, q = (t.unflatten(-1, (h, -1)) for t, h in ((c[..., :nv], b.N), (c[..., nv:nv + gk], b.G), (c[..., nv + gk:], b.G)))
    k, q = k.repeat_interleave(b.N // b.G, 2), q.repeat_interleave(b.N // b.G, 2)
    d = torch.nn.functional.softplus(a + p["beta"], threshold=1e9)
    f = torch.exp(-p["alpha"] * d)
    H, y = n.new_zeros(B, b.N, b.K, b.V), []
    for t in range(T):
        H = f[:, t, :, None, None] * H + (d[:, t, :, None] * k[:, t]).unsqueeze(3) * v[:, t].unsqueeze(2)
        y.append((q[:, t].unsqueeze(3) * H).sum(2) + p["w_r"][:, t] * v[:, t])
    y = torch.stack(y, 1)
    m = (y - y.mean(-1, keepdim=True)) / torch.sqrt(y.var(-1, unbiased=False, keepdim=True) + 1e-5)
    o = (m.flatten(2) * p["norm_w"] + p["norm_b"]) * silu(gate)
    return apply(p["w_out"], o)


def test_gradients_of_a_stack():
    B, T = 2, 40
    stack = Stack(depth=2, D=128, N=2, G=1, K=32, V=64, seed=3)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(B, T, 128, generator=gen).cuda()
    dout = torch.randn(B, T, 128, generator=gen).to(torch.bfloat16).cuda()
    out, g, _ = stack.train(x, dout)

    each = lambda t: t.double().expand(B, T, *t.shape).clone().requires_grad_()  # noqa: E731
    leaves = {"x": x.double().requires_grad_()}
    for i, b in enumerate(stack.blocks):
        leaves.update({f"block{i}.{n}": each(t) for n, t in b.p.items()})
    leaves.update({f"norm{i}": each(w) for i, w in enumerate(stack.norms)})
    norm = lambda h, w: h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-5) * w  # noqa: E731
    h = leaves["x"]
    for i, b in enumerate(stack.blocks):
        h = h + block64(b, {n: leaves[f"block{i}.{n}"] for n in b.p}, norm(h, leaves[f"norm{i}"]))
    want = norm(h, leaves["norm2"])
    assert float((out.double() - want.detach()).norm() / want.detach().norm()) < 2.0 ** -5
    parts = torch.autograd.grad(want, list(leaves.values()), dout.double())
    assert set(g) == set(leaves)
    off = {n: float((g[n].double() - (p if n == "x" else p.sum((0, 1)))).norm() / p.norm()) for n, p in zip(leaves, parts)}
    assert max(off.values()) < 2.0 ** -5, off


def test_clip_in_a_step():
    """Clipped gradients are the unclipped ones times max_norm / norm, within their types' rounding."""
    stack = Stack(depth=1, D=128, N=2, G=1, K=32, V=64, seed=5)
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(1, 70, 128, generator=gen).cuda()
    dout = torch.randn(1, 70, 128, generator=gen).to(torch.bfloat16).cuda()
    _, g, _ = stack.train(x, dout)
    _, c, norm = stack.train(x, dout, max_norm=0.25)
    n = np.sqrt(sum(float(t.double().square().sum()) for k, t in g.items() if k != "x"))
    assert abs(float(norm) - n) < 2.0 ** -20 * n and n > 0.25
    assert torch.equal(c["x"], g["x"])
    for k in g:
        if k != "x":
            want = g[k].double() * (0.25 / n)
            half = 2.0 ** -8 if g[k].dtype is torch.bfloat16 else 2.0 ** -24
            assert float(((c[k].double() - want).abs() - (half + 2.0 ** -19) * want.abs()).max()) <= 1e-38, k
    assert pkg.stream_status() == 0
