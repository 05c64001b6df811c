"""The measured cases of the selective state space block's operators: the short causal
convolution with its carried window, the selective scan and the gated group norm, each for
prompts, single tokens and training.  ``run`` computes them in plain torch operations in
32 bits, or, with ``own`` set, through this package's kernels; ``exact`` is the definition
in 64 bits."""
import math

import torch

own = False
DEV = "cuda"
TAPS = 4
CHUNK = 64  # tokens per chunk of the plain scan


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # Serving, one token for each of 256 requests: the block's conv on its v, k and q channels.
        dict(name="conv token x256", op="conv_step", B=256, C=1152, bias=True),
        # A short ragged prompt that continues an earlier one: x is a slice of a wider projection.
        dict(name="conv prompt 1021", op="conv", B=2, T=1021, C=1152, pad=1024, bias=True, window=True),
        # A training step's conv, forward and backward (16 heads of 128 beside one k and q of 128).
        dict(name="conv train 64k", op="conv_train", B=8, T=8192, C=2304, pad=0, bias=True, window=False),
        # A short prompt, where latency counts.
        dict(name="scan prompt 77", op="scan", B=1, T=77, N=8, G=8, K=64, V=64, h0=False, fused=False),
        # The 16K-context shape this package quotes its recurrence on.
        dict(name="scan prompt 8x16k", op="scan", B=8, T=16384, N=16, G=16, K=64, V=64, h0=False, fused=False),
        # One long sequence, q and k shared by all heads, continuing from a state, operands sliced
        # out of the conv's output.
        dict(name="scan prompt 64k", op="scan", B=1, T=65536, N=16, G=1, K=64, V=128, h0=True, fused=True),
        # A small training step with q and k for every head.
        dict(name="scan train 4x2k", op="scan_train", B=4, T=2048, N=8, G=8, K=64, V=64, h0=False, fused=False),
        # A large training step: 32 heads of 64 over one shared q and k of 128.
        dict(name="scan train 4x8k", op="scan_train", B=4, T=8192, N=32, G=1, K=128, V=64, h0=False, fused=True),
        # Serving, one token for each of 1024 requests.
        dict(name="scan token x1024", op="scan_step", B=1024, N=16, G=16, K=64, V=64),
        # Serving a few requests, where latency counts.
        dict(name="scan token x4", op="scan_step", B=4, N=32, G=1, K=128, V=64),
        # A training step's norm over 16 heads of 64, forward and backward.
        dict(name="norm train 128k", op="norm_train", rows=131072, D=1024, groups=16, f32=False, gate=True, bias=False),
        # Serving: one token for each of 256 requests, on the recurrence's 32-bit readout.
        dict(name="norm token x256", op="norm", rows=256, D=1024, groups=16, f32=True, gate=True, bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _not(n, step):
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(["conv_step", "conv", "conv_train", "scan", "scan", "scan_train", "scan_train",
                     "scan_step", "norm", "norm_train"])
    if op.startswith("conv"):
        C = _log(rng, 40, 2304)
        C = _not(C if rng.random() < 0.25 else (C + 7) // 8 * 8, 8)
        if op == "conv_step":
            return dict(op=op, B=_log(rng, 1, 1024), C=C, bias=rng.random() < 0.5)
        B = _log(rng, 1, 8)
        pad = _not(C + rng.choice([0, 8 * rng.randint(1, 128)]), 8) - C
        return dict(op=op, B=B, T=_not(_log(rng, 2, 65536 // B), 1), C=C, pad=pad, bias=rng.random() < 0.5,
                    window=rng.random() < 0.5)
    if op.startswith("scan"):
        K, V = rng.choice([16, 32, 40, 64, 64, 112, 128, 128]), rng.choice([32, 48, 64, 64, 80, 128])
        N = rng.choice([1, 2, 4, 6, 8, 12, 16, 32])
        G = rng.choice([g for g in (1, 2, 4, N) if N % g == 0])
        if op == "scan_step":
            return dict(op=op, B=_log(rng, 1, max(2, 2 ** 26 // (N * K * V))), N=N, G=G, K=K, V=V)
        # Token-heads such that the case costs no more than the largest listed one.
        most = (2 ** 21 if op == "scan" else 2 ** 19) * 4096 // max(4096, K * V)
        B = _log(rng, 1, 8)
        return dict(op=op, B=B, T=_not(_log(rng, 1, max(2, min(65536, most // (B * N)))), 1), N=N, G=G, K=K, V=V,
                    h0=rng.random() < 0.5, fused=rng.random() < 0.5 and N * V + 2 * G * K != 3072)
    groups = rng.choice([1, 4, 8, 16, 32])
    D = groups * (rng.choice([32, 64, 125, 128]) if groups > 1 else rng.choice([1000, 1024, 2048, 4096]))
    return dict(op=op, rows=_not(_log(rng, 1, 2 ** 27 // D), 1), D=D, groups=groups, f32=rng.random() < 0.5,
                gate=rng.random() < 0.75, bias=rng.random() < 0.5)


# ------------------------------------------------------------------------------ their inputs
def _inputs(case, seed):
    """The call's inputs (a dict of tensors and None), from the seed alone."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device=DEV) * (hi - lo) + lo

    op, f32 = case["op"], torch.float32
    if op.startswith("conv"):
        B, C = case["B"], case["C"]
        s = dict(w=randn(C, TAPS, scale=0.5, dtype=f32), bias=randn(C, scale=0.1, dtype=f32) if case["bias"] else None)
        if op == "conv_step":
            return dict(s, x=randn(B, C), window=randn(B, TAPS - 1, C))
        T = case["T"]
        s["x"] = randn(B, T, C + case["pad"])[:, :, :C]
        s["window"] = randn(B, TAPS - 1, C) if case["window"] else None
        if op == "conv_train":
            s["dout"] = randn(B, T, C)
        return s
    if op.startswith("scan"):
        B, N, G, K, V = (case[n] for n in ("B", "N", "G", "K", "V"))
        # The gate of a trained layer: decay rates over the heads from slow to fast, step sizes
        # that the token chooses.
        s = dict(alpha=torch.exp(uniform(math.log(0.1), math.log(2.0), N)), beta=uniform(-4.0, 1.0, N),
                 w_r=randn(N, V, dtype=f32))
        if op == "scan_step":
            return dict(s, q=randn(B, G, K, scale=K ** -0.5), k=randn(B, G, K, scale=K ** -0.5), v=randn(B, N, V),
                        a=randn(B, N), H=randn(B, N, K, V, scale=0.3, dtype=f32))
        T = case["T"]
        if case["fused"]:  # v, k, q side by side, as one conv call writes them
            x = randn(B, T, N * V + 2 * G * K)
            x[:, :, N * V:] *= K ** -0.5
            s["v"] = x[:, :, :N * V].unflatten(2, (N, V))
            s["k"] = x[:, :, N * V:N * V + G * K].unflatten(2, (G, K))
            s["q"] = x[:, :, N * V + G * K:].unflatten(2, (G, K))
        else:
            s["q"], s["k"] = randn(B, T, G, K, scale=K ** -0.5), randn(B, T, G, K, scale=K ** -0.5)
            s["v"] = randn(B, T, N, V)
        s["a"] = randn(B, T, N)
        s["H0"] = randn(B, N, K, V, scale=0.3, dtype=f32) if case["h0"] else None
        if op == "scan_train":
            s["dy"] = randn(B, T, N, V)
        return s
    R, D = case["rows"], case["D"]
    s = dict(y=randn(R, D, dtype=f32 if case["f32"] else torch.bfloat16), g_pre=randn(R, D) if case["gate"] else None,
             w=1.0 + randn(D, scale=0.1, dtype=f32), bias=randn(D, scale=0.1, dtype=f32) if case["bias"] else None)
    if op == "norm_train":
        s["dout"] = randn(R, D)
    return s


def prepare(case, seed):
    return dict(case=case, **_inputs(case, seed))


# --------------------------------------------------------------------- plain forms, 32 bits
def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _f32(t):
    return None if t is None else t.float()


def _conv_plain(x, w, bias, window):
    """x [B, T, C], window [B, 3, C] -> pre-rounding output; all in 32 bits."""
    T = x.shape[1]
    X = torch.cat([window, x], 1)
    pre = X[:, 0:T] * w[:, 0] + X[:, 1:T + 1] * w[:, 1] + X[:, 2:T + 2] * w[:, 2] + X[:, 3:T + 3] * w[:, 3]
    return _silu(pre if bias is None else pre + bias)


def _window(s):
    x = s["x"]
    return x.new_zeros(x.shape[0], TAPS - 1, x.shape[2]) if s["window"] is None else s["window"]


def _scan_plain(q, k, v, a, alpha, beta, w_r, H0):
    """All in 32 bits: y [B, T, N, V] and H_T [B, N, K, V], in chunks of CHUNK tokens."""
    B, T, N, V = v.shape
    G, K = q.shape[2:]
    L, C = CHUNK, (T + CHUNK - 1) // CHUNK
    x = a + beta
    d = torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))

    def chunks(t):  # [B, T, H, ...] -> [B, H, C, L, ...], zeros after the last token
        pad = t.new_zeros(B, C * L - T, *t.shape[2:])
        return torch.cat([t, pad], 1).unflatten(1, (C, L)).movedim(3, 1)

    d, logf = chunks(d), chunks(-alpha * d)
    rep = N // G
    kc, qc, vc = (chunks(t) for t in (k, q, v))
    kh, qh = kc.repeat_interleave(rep, 1), qc.repeat_interleave(rep, 1)
    cum = torch.cumsum(logf, 3)
    low = torch.ones(L, L, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp(torch.where(low, cum.unsqueeze(4) - cum.unsqueeze(3), -math.inf))
    scores = (qc @ kc.transpose(3, 4)).repeat_interleave(rep, 1)
    dv = d.unsqueeze(4) * vc
    y = (scores * decay) @ dv
    # Each chunk's own contribution to the state, then the states before each chunk: sums over the
    # earlier chunks, their decays summed from the later end so that near ones stay exact.
    own_part = kh.transpose(3, 4) @ (torch.exp(cum[:, :, :, -1:] - cum).unsqueeze(4) * dv)
    total = cum[:, :, :, -1]
    c = torch.arange(C + 1, device=q.device)
    between = torch.where(c[:, None] > c[None, 1:], torch.cat([total.new_zeros(B, N, 1), total], 2).unsqueeze(3), 0.0)
    between = torch.where(c[:, None] >= c[None, 1:], torch.cumsum(between, 2), -math.inf)  # [B, N, C + 1, C]
    states = torch.exp(between) @ own_part.flatten(3)
    if H0 is not None:
        whole = torch.cat([total.new_zeros(B, N, 1), torch.cumsum(total, 2)], 2)
        states = states + torch.exp(whole).unsqueeze(3) * H0.flatten(2).unsqueeze(2)
    states = states.unflatten(3, (K, V))
    y = y + torch.exp(cum).unsqueeze(4) * (qh @ states[:, :, :-1])
    y = y.movedim(1, 3).flatten(1, 2)[:, :T]
    return y + w_r * v, states[:, :, -1]


def _scan_step_plain(q, k, v, a, alpha, beta, w_r, H):
    N = v.shape[1]
    rep = N // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    x = a + beta
    d = torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))
    f = torch.exp(-alpha * d)
    H = f[..., None, None] * H + (d[..., None] * k).unsqueeze(3) * v.unsqueeze(2)
    return (q.unsqueeze(3) * H).sum(2) + w_r * v, H


def _norm_plain(y, g_pre, w, bias, groups, eps=1e-5):
    z = y.unflatten(1, (groups, -1))
    z = z - z.mean(2, keepdim=True)
    z = z / torch.sqrt((z * z).mean(2, keepdim=True) + eps)
    p = z.flatten(1) * w
    p = p if bias is None else p + bias
    return _silu(p) if g_pre is None else p * _silu(g_pre)


def _with_grads(f, inputs, names, dout):
    """f's output and the gradients of <out, dout> at inputs[name]; leaves in 32 bits."""
    leaves = {n: _f32(t) for n, t in inputs.items()}
    wanted = [n for n in names if leaves[n] is not None]
    for n in wanted:
        leaves[n] = leaves[n].detach().requires_grad_(True)
    out, extra = f(leaves)
    grads = torch.autograd.grad(out, [leaves[n] for n in wanted], dout.float())
    return out.detach(), extra, {n: g.to(inputs[n].dtype) for n, g in zip(wanted, grads)}


def _run_plain(s):
    case, op, bf = s["case"], s["case"]["op"], torch.bfloat16
    if op == "conv_step":
        out = _conv_plain(s["x"].float().unsqueeze(1), s["w"], s["bias"], s["window"].float())
        return dict(out=out.squeeze(1).to(bf), window=torch.cat([s["window"], s["x"].unsqueeze(1)], 1)[:, 1:])
    if op == "conv":
        out = _conv_plain(s["x"].float(), s["w"], s["bias"], _window(s).float())
        return dict(out=out.to(bf), window=torch.cat([_window(s), s["x"]], 1)[:, -(TAPS - 1):])
    if op == "conv_train":
        ins = dict(x=s["x"], w=s["w"], bias=s["bias"], window=s["window"])
        out, _, g = _with_grads(lambda t: (_conv_plain(t["x"], t["w"], t["bias"], _f32(_window(s)) if t["window"] is None
                                                       else t["window"]), None), ins, list(ins), s["dout"])
        return dict(out=out.to(bf), **{"d" + n: x for n, x in g.items()})
    if op == "scan":
        y, H = _scan_plain(*(_f32(s[n]) for n in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H0")))
        return dict(y=y.to(bf), H_T=H)
    if op == "scan_train":
        ins = {n: s[n] for n in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H0")}
        y, H, g = _with_grads(lambda t: _scan_plain(**t), ins, list(ins), s["dy"])
        return dict(y=y.to(bf), H_T=H.detach(), **{"d" + n: x for n, x in g.items()})
    if op == "scan_step":
        y, H = _scan_step_plain(*(_f32(s[n]) for n in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H")))
        return dict(y=y.to(bf), H=H)
    if op == "norm":
        return dict(out=_norm_plain(*(_f32(s[n]) for n in ("y", "g_pre", "w", "bias")), case["groups"]).to(bf))
    ins = {n: s[n] for n in ("y", "g_pre", "w", "bias")}
    out, _, g = _with_grads(lambda t: (_norm_plain(**t, groups=case["groups"]), None), ins, list(ins), s["dout"])
    return dict(out=out.to(bf), **{"d" + n: x for n, x in g.items()})


# ----------------------------------------------------------------------- this package's calls
def _run_own(s):
    import matrix_state_nonlinear_gb300 as m2
    case, op = s["case"], s["case"]["op"]
    if op == "conv_step":
        out, window = m2.conv_silu_step(s["x"], s["w"], s["bias"], s["window"], window_out=torch.empty_like(s["window"]))
        return dict(out=out, window=window)
    if op == "conv":
        out, window = m2.conv_silu_window(s["x"], s["w"], s["bias"], s["window"])
        return dict(out=out, window=window)
    if op == "conv_train":
        out, _ = m2.conv_silu_window(s["x"], s["w"], s["bias"], s["window"])
        g = m2.conv_silu_backward(s["x"], s["w"], s["bias"], s["dout"], s["window"])
        return dict(out=out, **{n: g[n] for n in ("dx", "dw", "dbias", "dwindow") if s[n[1:]] is not None})
    if op == "scan":
        y, H = m2.ssm_forward(s)
        return dict(y=y, H_T=H)
    if op == "scan_train":
        y, H, Hs = m2.ssm_forward_train(s)
        g = m2.ssm_backward(s, Hs, s["dy"])
        return dict(y=y, H_T=H, **{"d" + n: g["d" + n] for n in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H0")
                                   if s[n] is not None})
    if op == "scan_step":
        y, H = m2.ssm_step(*(s[n] for n in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H")), H_out=torch.empty_like(s["H"]))
        return dict(y=y, H=H)
    out = m2.gate_groupnorm(s["y"], s["g_pre"], s["w"], s["bias"], case["groups"], 1e-5)
    if op == "norm":
        return dict(out=out)
    g = m2.gate_groupnorm_backward(s["y"], s["g_pre"], s["w"], s["bias"], s["dout"], case["groups"], 1e-5)
    return dict(out=out, **{"d" + n: g["d" + n] for n in ("y", "g_pre", "w", "bias") if s[n] is not None})


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------- the floors
def work(case):
    """Each input read once, each output written once; the operations of the recurrent form
    (of a training pass: its forward, and the two products of each in the backward)."""
    op = case["op"]
    if op.startswith("conv"):
        n = case["B"] * case.get("T", 1) * case["C"]
        if op == "conv_step":
            return dict(bytes=2 * n * (1 + 1 + 3 + 3), flops=12 * n)
        edge = 4 * 3 * case["B"] * case["C"]
        return dict(bytes=4 * n + edge, flops=12 * n) if op == "conv" else dict(bytes=(4 + 6) * n + edge, flops=40 * n)
    if op.startswith("scan"):
        B, N, G, K, V = (case[n] for n in ("B", "N", "G", "K", "V"))
        T = case.get("T", 1)
        heads, state = B * T * N, 4 * B * N * K * V
        ins, out = 4 * B * T * G * K + heads * (2 * V + 2), 2 * heads * V
        if op == "scan_step":
            return dict(bytes=ins + out + 2 * state, flops=5 * heads * K * V)
        if op == "scan":
            return dict(bytes=ins + out + state * (1 + case["h0"]), flops=5 * heads * K * V)
        return dict(bytes=(ins + out) + (ins + out) + ins + state * (1 + 2 * case["h0"]), flops=15 * heads * K * V)
    n = case["rows"] * case["D"]
    y, g = 4 if case["f32"] else 2, 2 if case["gate"] else 0
    forward = n * (y + g + 2)
    return dict(bytes=forward, flops=15 * n) if op == "norm" else dict(bytes=forward + n * (y + g + 2 + y + g), flops=50 * n)


# ------------------------------------------------------------ the definitions, in 64 bits
def _f64(s):
    return {n: t.double() if isinstance(t, torch.Tensor) else t for n, t in s.items()}


def _exact_conv(s, T):
    """Tap by tap, from the convolution's definition."""
    x, w = s["x"], s["w"]
    B, _, C = x.shape
    before = s["window"] if s["window"] is not None else torch.zeros(B, 3, C, dtype=torch.float64, device=DEV)
    X = torch.cat([before, x], 1)
    taps = X.unfold(1, TAPS, 1)  # [B, T, C, 4]
    pre = torch.einsum("btcj,cj->btc", taps, w)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    sig = torch.sigmoid(pre)
    res = dict(out=pre * sig)
    if "dout" not in s:
        res["window"] = X[:, T:]
        return res
    dpre = s["dout"] * (sig + pre * sig * (1 - sig))
    dX = torch.zeros_like(X)
    for j in range(TAPS):
        dX[:, j:j + T] += dpre * w[:, j]
    res["dx"], res["dw"] = dX[:, 3:], torch.einsum("btc,btcj->cj", dpre, taps)
    if s["bias"] is not None:
        res["dbias"] = dpre.sum((0, 1))
    if s["window"] is not None:
        res["dwindow"] = dX[:, :3]
    return res


def _exact_scan(s, T):
    """Token by token, from the recurrence and its reverse."""
    B, _, N, V = s["v"].shape
    G, K = s["q"].shape[2:]
    rep = N // G
    x = s["a"] + s["beta"]
    d = torch.nn.functional.softplus(x, threshold=1e9)
    f = torch.exp(-s["alpha"] * d)
    H = s["H0"].clone() if s.get("H0") is not None else torch.zeros(B, N, K, V, dtype=torch.float64, device=DEV)
    y = torch.empty(B, T, N, V, dtype=torch.float64, device=DEV)
    every, kept = 64, []
    head = lambda t: t.repeat_interleave(rep, 1)  # noqa: E731

    def forward(H, t):
        kd = head(s["k"][:, t]) * d[:, t, :, None]
        return H.mul(f[:, t, :, None, None]).addcmul_(kd.unsqueeze(3), s["v"][:, t].unsqueeze(2))

    for t in range(T):
        if t % every == 0:
            kept.append(H)
        H = forward(H, t)
        y[:, t] = torch.matmul(head(s["q"][:, t]).unsqueeze(2), H).squeeze(2)
    res = dict(y=y + s["w_r"] * s["v"], H_T=H)
    if "dy" not in s:
        return res
    dy, Gs = s["dy"], torch.zeros_like(H)
    dq, dkk = (torch.empty(B, T, N, K, dtype=torch.float64, device=DEV) for _ in range(2))
    dv, g, kGv = torch.empty_like(y), torch.empty_like(x), torch.empty_like(x)
    for c in range(len(kept) - 1, -1, -1):
        states = [kept[c]]
        for t in range(c * every, min(T, (c + 1) * every)):
            states.append(forward(states[-1], t))
        for t in range(min(T, (c + 1) * every) - 1, c * every - 1, -1):
            Hb, Ha = states[t - c * every], states[t - c * every + 1]
            Gs = Gs.addcmul(head(s["q"][:, t]).unsqueeze(3), dy[:, t].unsqueeze(2))
            dq[:, t] = torch.matmul(Ha, dy[:, t].unsqueeze(3)).squeeze(3)
            Gv = torch.matmul(Gs, s["v"][:, t].unsqueeze(3)).squeeze(3)
            kh = head(s["k"][:, t])
            dkk[:, t] = d[:, t, :, None] * Gv
            kGv[:, t] = (kh * Gv).sum(2)
            dv[:, t] = d[:, t, :, None] * torch.matmul(kh.unsqueeze(2), Gs).squeeze(2)
            g[:, t] = f[:, t] * (Gs * Hb).sum((2, 3))
            Gs = Gs * f[:, t, :, None, None]
    da = torch.sigmoid(x) * (kGv - s["alpha"] * g)
    res.update(dq=dq.unflatten(2, (G, rep)).sum(3), dk=dkk.unflatten(2, (G, rep)).sum(3), dv=dv + s["w_r"] * dy, da=da,
               dalpha=-(g * d).sum((0, 1)), dbeta=da.sum((0, 1)), dw_r=(dy * s["v"]).sum((0, 1)))
    if s.get("H0") is not None:
        res["dH0"] = Gs
    return res


def _exact_norm(s, groups):
    y = s["y"]
    E = y.shape[1] // groups
    z = y.view(-1, groups, E)
    var, mean = torch.var_mean(z, 2, correction=0, keepdim=True)
    inv = (var + 1e-5).rsqrt()
    n = ((z - mean) * inv).view_as(y)
    p = n * s["w"] if s["bias"] is None else n * s["w"] + s["bias"]
    at = p if s["g_pre"] is None else s["g_pre"]
    sig = torch.sigmoid(at)
    slope = sig * (1 + at * (1 - sig))
    res = dict(out=at * sig if s["g_pre"] is None else p * at * sig)
    if "dout" not in s:
        return res
    dp = s["dout"] * (slope if s["g_pre"] is None else at * sig)
    if s["g_pre"] is not None:
        res["dg_pre"] = s["dout"] * p * slope
    dn = (dp * s["w"]).view(-1, groups, E)
    nz = n.view(-1, groups, E)
    res["dy"] = (inv * (dn - dn.mean(2, keepdim=True) - nz * (dn * nz).mean(2, keepdim=True))).view_as(y)
    res["dw"] = (dp * n).sum(0)
    if s["bias"] is not None:
        res["dbias"] = dp.sum(0)
    return res


def exact(case, seed):
    s = _f64(_inputs(case, seed))
    op = case["op"]
    if op == "conv_step":
        r = _exact_conv(dict(s, x=s["x"].unsqueeze(1)), 1)
        return dict(out=r["out"].squeeze(1), window=r["window"])
    if op.startswith("conv"):
        return _exact_conv(s, case["T"])
    if op == "scan_step":
        one = {n: s[n].unsqueeze(1) for n in ("q", "k", "v", "a")}
        r = _exact_scan(dict(s, **one, H0=s["H"]), 1)
        return dict(y=r["y"].squeeze(1), H=r["H_T"])
    if op.startswith("scan"):  # a token at a time: too slow for a long training pass
        return None if op == "scan_train" and case["T"] > 16384 else _exact_scan(s, case["T"])
    return _exact_norm(s, case["groups"])
