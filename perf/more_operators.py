"""The measured cases of what stands around a recurrent block in a stack: the residual's addition with
its RMS norm (bf16 out, 8 bits out, training), the 8-bit projection with a scale for each block of 128,
and the clipping of a step's gradients by their global norm.  ``run`` computes them in plain torch
operations in 32 bits, or, with ``own`` set, through this package's kernels; ``exact`` is the definition
in 64 bits."""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-5
BLOCK = 128      # values that share a scale
E4M3_MAX = 448.0
BF16, F32, FP8, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # Serving: one token for each of 64 requests, a bf16 residual stream.
        dict(name="norm token x64", op="norm", rows=64, D=2048, f32=False, residual=True, pad=0),
        # The last norm of a stack over a long prompt, on a 32-bit stream.
        dict(name="norm last 32k", op="norm", rows=32768, D=2048, f32=True, residual=False, pad=0),
        # A ragged prompt whose norm feeds 8-bit projections; x is a slice of a wider projection.
        dict(name="norm8 prompt 8191", op="norm8", rows=8191, D=4096, f32=True, residual=True, pad=512),
        # Serving: 8 requests, the norm in front of an 8-bit projection.
        dict(name="norm8 token x8", op="norm8", rows=8, D=1000, f32=False, residual=True, pad=0),
        # A training step's norm, forward and backward, with the stream's own gradient arriving.
        dict(name="norm train 64k", op="norm_train", rows=65536, D=2048, f32=False, residual=True, pad=0),
        # Serving one request: the input projection of a block of 32 heads of 64 over one k and q of 128
        # (gate, conv channels and logits side by side).
        dict(name="linear token x1", op="linear", M=1, K=2048, N=4384, f32=False),
        # Serving 64 requests of a wider model.
        dict(name="linear token x64", op="linear", M=64, K=4096, N=8192, f32=False),
        # A ragged prompt through the output projection, onto a 32-bit stream.
        dict(name="linear prompt 1021", op="linear", M=1021, K=2048, N=2000, f32=True),
        # A batch of long prompts.
        dict(name="linear prompt 16k", op="linear", M=16384, K=4096, N=8192, f32=False),
        # A layer's way in: residual, norm, 8 bits, input projection.
        dict(name="norm linear prompt 8k", op="norm_linear", M=8192, K=2048, N=4384, f32=False),
        # The gradients of a small block, 32 bits.
        dict(name="clip block", op="clip", layers=1, D=256, heads=6, wide=False, clips=True),
        # The gradients of a stack, matrices in bf16 and vectors in 32 bits.
        dict(name="clip stack", op="clip", layers=32, D=2048, heads=32, wide=True, clips=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm8", "norm8", "norm_train", "norm_train", "linear", "linear", "linear", "norm_linear",
                     "clip", "clip"])
    if op in ("norm", "norm8", "norm_train"):
        D = _log(rng, 96, 8192)
        D = D if rng.random() < 0.3 else (D + 7) // 8 * 8
        return dict(op=op, rows=_log(rng, 1, max(2, 2 ** 27 // D if op == "norm_train" else 2 ** 26 // D)), D=D,
                    f32=rng.random() < 0.5, residual=op == "norm_train" or rng.random() < 0.75,
                    pad=rng.choice([0, 0, 8 * rng.randint(1, 64)]))
    if op in ("linear", "norm_linear"):
        K, N = _log(rng, 128, 8192), _log(rng, 128, 8192)
        if rng.random() < 0.7:
            K, N = (K + 15) // 16 * 16, (N + 7) // 8 * 8
        M = _log(rng, 1, 256) if rng.random() < 0.5 else _log(rng, 64, 16384)
        return dict(op=op, M=min(M, 2 ** 39 // (K * N)), K=K, N=N, f32=op == "linear" and rng.random() < 0.3)
    layers, heads = _log(rng, 1, 48), rng.choice([1, 3, 6, 8, 16, 32])
    D = _log(rng, 64, 2048) if layers < 16 else _log(rng, 64, 1024)
    return dict(op=op, layers=layers, D=D, heads=heads, wide=rng.random() < 0.5, clips=rng.random() < 0.75)


# ------------------------------------------------------------------------------ their inputs
def _layer_sizes(D, heads):
    """(values, is a matrix) of each of a block's parameters, one shared k and q of 128, heads of 64."""
    nv = 64 * heads
    C = nv + 256
    return [((nv + C + heads) * D, True), (D * nv, True), (4 * C, False), (C, False), (heads, False), (heads, False),
            (nv, False), (nv, False), (nv, False), (D, False)]


def _gradient_sizes(case):
    return _layer_sizes(case["D"], case["heads"]) * case["layers"]


def _views(flat, sizes):
    """Consecutive parts of a flat buffer."""
    return list(flat.split(sizes))


def _e4m3_weights(w):
    """w [N, K] in blocks of 128 x 128: e4m3 values, rows 16 bytes aligned, and a power of two for each block."""
    N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    big = torch.zeros(nb * BLOCK, kb * BLOCK, device=DEV)
    big[:N, :K] = w
    big = big.view(nb, BLOCK, kb, BLOCK)
    scales = _power(big.abs().amax((1, 3)))
    q = (big / scales[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:N, :K].to(FP8)
    room = torch.zeros(N, (K + 15) // 16 * 16, dtype=torch.uint8, device=DEV)
    room[:, :K] = q.view(torch.uint8)
    return room.view(FP8)[:, :K], scales.to(E8M0)


def _inputs(case, seed):
    """The call's inputs (a dict of tensors and None), from the seed alone."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=BF16):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    def activations(rows, D, dtype, pad=0):
        """Channels of unequal sizes, a few of them large, and rows of unequal sizes."""
        channel = torch.exp(0.5 * torch.randn(D + pad, generator=g, device=DEV))
        channel[:: 97] *= 12.0
        row = torch.exp(0.3 * torch.randn(rows, 1, generator=g, device=DEV))
        return (torch.randn(rows, D + pad, generator=g, device=DEV) * channel * row).to(dtype)[:, :D]

    op = case["op"]
    if op == "clip":
        sizes = _gradient_sizes(case)
        wide = [n for n, matrix in sizes if matrix or not case["wide"]]
        rest = [n for n, matrix in sizes if case["wide"] and not matrix]
        size = torch.exp(torch.randn(len(wide), generator=g, device=DEV))
        flat = torch.randn(sum(wide), generator=g, device=DEV)
        for t, s in zip(_views(flat, wide), size):
            t.mul_(s)
        s = dict(flat=(flat * 1e-3).to(BF16 if case["wide"] else F32), sizes=wide,
                 more=randn(sum(rest), scale=1e-3, dtype=F32), more_sizes=rest)
        total = math.sqrt(sum(wide) + sum(rest)) * 1e-3
        return dict(s, max_norm=total * (0.5 if case["clips"] else 100.0))
    if op in ("linear", "norm_linear"):
        M, K, N = case["M"], case["K"], case["N"]
        s = dict(zip(("wq", "ws"), _e4m3_weights(randn(N, K, scale=K ** -0.5, dtype=F32))))
        if op == "linear":
            return dict(s, x=activations(M, K, BF16))
        return dict(s, x=activations(M, K, BF16), residual=activations(M, K, BF16), w=1.0 + randn(K, scale=0.1, dtype=F32))
    R, D = case["rows"], case["D"]
    stream = F32 if case["f32"] else BF16
    s = dict(x=activations(R, D, BF16 if case["residual"] else stream, case["pad"]), w=1.0 + randn(D, scale=0.1, dtype=F32),
             residual=activations(R, D, stream).contiguous() if case["residual"] else None)
    if op == "norm_train":
        s["dout"], s["dh"] = randn(R, D), randn(R, D, dtype=stream)
    return s


def prepare(case, seed):
    s = dict(case=case, **_inputs(case, seed))
    if case["op"] == "clip":  # the tensors of a step, and where their clipped values go
        s["out"], s["more_out"] = torch.empty_like(s["flat"]), torch.empty_like(s["more"])
        s["grads"] = _views(s["flat"], s["sizes"]) + _views(s["more"], s["more_sizes"])
        s["outs"] = _views(s["out"], s["sizes"]) + _views(s["more_out"], s["more_sizes"])
    return s


# --------------------------------------------------------------------- plain forms, 32 bits
def _power(amax):
    """The least power of two s with amax / s <= 448 (2^-126 at the least)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    e = torch.clamp(e - 9 + (m > 0.875), min=-126)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, -126))


def _blocks(x):
    """x [R, D] -> [R, blocks, 128], zeros behind the last channel."""
    R, D = x.shape
    nb = -(-D // BLOCK)
    return torch.nn.functional.pad(x, (0, nb * BLOCK - D)).view(R, nb, BLOCK)


def _e4m3(x):
    """x [R, D] float32 -> e4m3 values and the power of two of each 128 of them."""
    b = _blocks(x)
    scales = _power(b.abs().amax(2))
    return (b / scales.unsqueeze(2)).flatten(1)[:, :x.shape[1]].to(FP8), scales.to(E8M0)


def _values(q, scales):
    """What 8-bit activations stand for, in 32 bits."""
    return (_blocks(q.float()) * scales.float().unsqueeze(2)).flatten(1)[:, :q.shape[1]]


def _weight_values(q, scales):
    N, K = q.shape
    s = scales.float().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return q.float() * s


def _sum_plain(s):
    """The stream after the addition, rounded to its type."""
    return s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)


def _norm_plain(h, w):
    h = h.float()
    return h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * w


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        h = _sum_plain(s)
        out = _norm_plain(h, s["w"]).to(BF16)
        return dict(out=out) if s["residual"] is None else dict(out=out, h=h)
    if op == "norm8":
        h = _sum_plain(s)
        q, scales = _e4m3(_norm_plain(h, s["w"]))
        return dict(q=q, scales=scales) if s["residual"] is None else dict(q=q, scales=scales, h=h)
    if op == "norm_train":
        h = _sum_plain(s)
        leaf, w = h.float().requires_grad_(True), s["w"].clone().requires_grad_(True)
        out = _norm_plain(leaf, w)
        d, dw = torch.autograd.grad(out, (leaf, w), s["dout"].float())
        d = d + s["dh"].float()
        return dict(out=out.detach().to(BF16), h=h, dx=d.to(BF16), dresidual=d.to(h.dtype), dw=dw)
    if op == "linear":
        out = _values(*_e4m3(s["x"].float())) @ _weight_values(s["wq"], s["ws"]).T
        return dict(out=out.to(F32 if case["f32"] else BF16))
    if op == "norm_linear":
        h = _sum_plain(s)
        out = _values(*_e4m3(_norm_plain(h, s["w"]))) @ _weight_values(s["wq"], s["ws"]).T
        return dict(out=out.to(F32 if case["f32"] else BF16), h=h)
    norm = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum().sqrt().float()
    by = torch.clamp(s["max_norm"] / norm, max=1.0)
    clipped = [(t.float() * by).to(t.dtype) for t in s["grads"]]
    n = len(s["sizes"])
    return dict(norm=norm, out=torch.cat(clipped[:n]), more=torch.cat(clipped[n:]) if clipped[n:] else s["more"])


# ----------------------------------------------------------------------- this package's calls
def _run_own(s):
    import matrix_state_nonlinear_gb300 as m2
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        out, h = m2.add_rmsnorm(s["x"], s["residual"], s["w"], EPS)
        return dict(out=out) if s["residual"] is None else dict(out=out, h=h)
    if op == "norm8":
        q, scales, h = m2.add_rmsnorm_fp8(s["x"], s["residual"], s["w"], EPS)
        return dict(q=q, scales=scales) if s["residual"] is None else dict(q=q, scales=scales, h=h)
    if op == "norm_train":
        out, h = m2.add_rmsnorm(s["x"], s["residual"], s["w"], EPS)
        g = m2.add_rmsnorm_backward(h, s["w"], s["dout"], s["dh"], EPS)
        return dict(out=out, h=h, dx=g["dx"], dresidual=g["dresidual"], dw=g["dw"])
    if op == "linear":
        return dict(out=m2.linear_fp8(s["x"], None, s["wq"], s["ws"], out_dtype=F32 if case["f32"] else BF16))
    if op == "norm_linear":
        q, scales, h = m2.add_rmsnorm_fp8(s["x"], s["residual"], s["w"], EPS)
        return dict(out=m2.linear_fp8(q, scales, s["wq"], s["ws"], out_dtype=F32 if case["f32"] else BF16), h=h)
    norm = m2.clip_grad_norm(s["grads"], s["max_norm"], out=s["outs"])
    return dict(norm=norm, out=s["out"], more=s["more_out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------- the floors
def work(case):
    """Each input read once, each output written once."""
    op = case["op"]
    if op == "clip":
        matrices = sum(n for n, matrix in _gradient_sizes(case) if matrix)
        n = sum(n for n, _ in _gradient_sizes(case))
        return dict(bytes=2 * ((2 if case["wide"] else 4) * matrices + 4 * (n - matrices)), flops=3 * n)
    if op in ("linear", "norm_linear"):
        M, K, N = case["M"], case["K"], case["N"]
        out = M * N * (4 if case["f32"] else 2)
        return dict(bytes=(2 if op == "linear" else 6) * M * K + N * K + out, flops=2 * M * N * K + (0 if op == "linear" else 5 * M * K))
    n, stream = case["rows"] * case["D"], 4 if case["f32"] else 2
    read = 2 + 2 * stream if case["residual"] else stream
    if op == "norm":
        return dict(bytes=n * (read + 2), flops=5 * n)
    if op == "norm8":
        return dict(bytes=n * (read + 1) + n // BLOCK, flops=8 * n)
    # forward; then h, dout and dh in, dx and (where the stream is wider) dresidual out
    return dict(bytes=n * (read + 2) + n * (stream + 2 + stream + (6 if case["f32"] else 2)), flops=20 * n)


# ------------------------------------------------------------ the definitions, in 64 bits
def _exact_scale(v):
    """Per 128 channels of v [R, D]: 2^ceil(log2(max |v| / 448)), at least 2^-126, for every channel."""
    R, D = v.shape
    out, e = torch.empty_like(v), []
    for c in range(0, D, BLOCK):
        a = v[:, c:c + BLOCK].abs().amax(1)
        k = torch.ceil(torch.log2(a / E4M3_MAX))
        k = torch.where(torch.exp2(k - 1) * E4M3_MAX >= a, k - 1, k)  # a logarithm next to a whole number
        k = torch.where(torch.exp2(k) * E4M3_MAX < a, k + 1, k)
        e.append(torch.exp2(torch.clamp(k, min=-126.0)))
        out[:, c:c + BLOCK] = e[-1].unsqueeze(1)
    return out, torch.stack(e, 1)


def _exact_round(v):
    """The nearest e4m3 value: three bits below the leading one, steps of 2^-9 below 2^-6, ties to even."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs())), min=-6.0) - 3)
    return torch.round(v / step) * step


def _exact_weights(s):
    N, K = s["wq"].shape
    n, k = torch.arange(N, device=DEV) // BLOCK, torch.arange(K, device=DEV) // BLOCK
    return s["wq"].double() * s["ws"].double()[n][:, k]


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "clip":
        a, b = s["flat"].double(), s["more"].double()
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(a), torch.linalg.vector_norm(b)]))
        by = min(1.0, s["max_norm"] / float(norm))
        return dict(norm=norm, out=a * by, more=b * by)
    x = s["x"].double()
    if op != "linear":
        h = x if s["residual"] is None else x + s["residual"].double()
        kept = h if s["residual"] is None else h.to(s["residual"].dtype).double()  # the stream as its type holds it
        inv = 1 / torch.sqrt((kept ** 2).mean(1, keepdim=True) + EPS)
        n = kept * inv * s["w"].double()
    if op in ("linear", "norm_linear"):
        v = x if op == "linear" else n
        each, _ = _exact_scale(v)
        out = (_exact_round(v / each) * each) @ _exact_weights(s).T
        return dict(out=out) if op == "linear" else dict(out=out, h=h)
    if op == "norm8":
        each, scales = _exact_scale(n)
        res = dict(q=n / each, scales=scales)
        return res if s["residual"] is None else dict(res, h=h)
    res = dict(out=n) if s["residual"] is None else dict(out=n, h=h)
    if op == "norm":
        return res
    dout = s["dout"].double()
    dn = dout * s["w"].double()
    d = inv * dn - kept * inv ** 3 * (dn * kept).mean(1, keepdim=True) + s["dh"].double()
    return dict(res, dx=d, dresidual=d, dw=(dout * kept * inv).sum(0))
