"""The residual RMS norm, the 8-bit values and their product, and the clipping of gradients on the GPU
against the fp64 oracle.

Tolerances, derived from the arithmetic (eps / 2 of a type: bf16 2^-8, e4m3 2^-4, float32 2^-24):
 * float32 arithmetic before a rounding: a row's sum of squares adds at most 32 terms per thread, then 5 + 4
   levels: within 2^-18 of itself (all terms are positive), its root and three products add 2^-22.
   A result of the norm is therefore within 2^-17 of itself, and its bf16 rounding within 2^-8 + 2^-17.
 * Gradients: every term of d within 2^-17 of its magnitude, the mean of g h within 2^-17 of the mean of |g h|;
   dw sums rows in at most 2^7 steps per thread and as many blocks: 2^-15 of the terms' magnitudes.
 * e4m3: half a step, 2^-4 of the value or (below 2^-6 of the scale) 2^-10 of the scale, plus 2^-17 of the value.
   A scale may be the neighbouring power only where max / 448 is within 2^-17 of a power of two.
 * Products: 8-bit values multiply exactly; the tensor cores add 32 products to a float32 at a time, each
   addition within 2^-23 of the sum of magnitudes so far: 2^-23 (K / 32 + 2) A, A the sum of all terms' magnitudes.
 * The gradients' norm: exact sums of float32 sums of at most 64 squares, in at most 12 roundings each: 12 2^-25 of
   the norm, below 2^-21; clipped values 2^-22 more, and their type's rounding.
"""
import numpy as np
import pytest
import torch

import __graft_entry__
import matrix_state_nonlinear_gb300 as pkg
from matrix_state_nonlinear_gb300 import m2rnn as binding
from oracle import layer as ol

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, FP8, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    pkg.load_library()


def rand(shape, seed, scale=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def f64(t):
    return t.double().cpu().numpy()


def within(got, want, tol, what=""):
    over = np.abs(f64(got) - want) - tol
    assert np.isfinite(f64(got)).all() and float(over.max(initial=-1.0)) <= 0.0, (what, float(over.max()))


# ---------------------------------------------------------------- 8-bit values
def values(rows, D, seed, dtype=BF16):
    """Rows and channels of unequal sizes, a row of zeros, one of very small and one of very large values."""
    x = rand((rows, D), seed, 1.0, F32) * torch.exp(2 * rand((rows, 1), seed + 1, 1.0, F32))
    x[:, ::13] *= 50
    if rows > 3:
        x[1] = 0
        x[2] *= 1e-37
        x[3] *= 1e35
    return x.to(dtype)


@pytest.mark.parametrize("rows,D", [(1, 1), (1, 128), (5, 7), (4, 127), (7, 129), (33, 1000), (6, 2048), (300, 257)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_quantise_rows(rows, D, dtype, pad):
    x = values(rows, D + pad, 3, dtype)[:, :D]
    q, s = pkg.quantise_fp8(x)
    want, scales = ol.quantise(f64(x))
    assert q.dtype is FP8 and s.dtype is E8M0
    assert np.array_equal(f64(s), scales) and np.array_equal(f64(q), want)


@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 127), (200, 300), (256, 1024), (77, 16)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantise_weight(N, K, dtype):
    w = values(N, K, 5, dtype)
    q, s = pkg.quantise_weight_fp8(w)
    want, scales = ol.quantise_weight(f64(w))
    assert np.array_equal(f64(s), scales) and np.array_equal(f64(q), want)
    assert q.stride(0) % 16 == 0


def test_quantise_infinities():
    x = rand((4, 300), 6)
    x[0, 5], x[1, 200], x[2, 299] = float("inf"), float("-inf"), float("nan")
    q, s = pkg.quantise_fp8(x)
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert torch.equal(s.float().isnan().cpu(), bad)
    assert torch.equal(q.float().isnan().cpu(), bad.repeat_interleave(128, 1)[:, :300])


# ---------------------------------------------------------------- residual norm
# rows, D: one channel, odd widths, one and several threads' chunks, wide rows, many rows
NORM = [(1, 1), (3, 7), (2, 8), (5, 129), (9, 1000), (4, 1001), (64, 2048), (3, 4104), (2, 8192), (2, 16384), (2, 16383),
        (2600, 264), (2500, 2100), (2701, 96), (5003, 128), (3001, 134), (2439, 505), (2433, 1001), (2600, 1032), (40, 200)]


def norm_case(rows, D, f32, residual, seed=0, pad=0):
    stream = F32 if f32 else BF16
    x = rand((rows, D + pad), seed, 1.5, BF16 if residual else stream)[:, :D]
    r = rand((rows, D + pad), seed + 1, 2.0, stream)[:, :D] if residual else None
    return x, r, 1 + rand((D,), seed + 2, 0.2, F32)


def check_h(h, x, residual):
    if residual is None:
        assert h is x
    elif h.dtype is F32:
        assert torch.equal(h, x.float() + residual)
    else:
        assert torch.equal(h, (x.float() + residual.float()).to(BF16))


@pytest.mark.parametrize("rows,D", NORM)
@pytest.mark.parametrize("f32,residual,pad", [(False, True, 0), (True, True, 8), (False, False, 0), (True, False, 3)])
def test_norm(rows, D, f32, residual, pad):
    x, r, w = norm_case(rows, D, f32, residual, pad=pad)
    out, h = pkg.add_rmsnorm(x, r, w, 1e-5)
    check_h(h, x, r)
    want = ol.rmsnorm(f64(h), f64(w), 1e-5)
    within(out, want, (2.0 ** -8 + 2.0 ** -17) * np.abs(want))


def check_quantised(q, s, v):
    """8-bit values against values known to 2^-17."""
    want, got = ol.row_scales(v), f64(s)
    blocks = np.repeat(np.maximum.reduceat(np.abs(v), np.arange(0, v.shape[1], 128), axis=1), 1, 1)
    near = np.exp2(np.round(np.log2(np.maximum(blocks, 1e-300) / 448)))
    edge = np.abs(blocks / 448 - near) <= 2.0 ** -17 * near
    assert ((got == want) | (edge & ((got == 2 * want) | (got == want / 2)))).all()
    each = np.repeat(got, 128, 1)[:, :v.shape[1]]
    over = np.abs(f64(q) * each - v) - ((2.0 ** -4 + 2.0 ** -17) * np.abs(v) + 2.0 ** -10 * each)
    assert np.isfinite(f64(q)).all() and over.max() <= 0, over.max()


@pytest.mark.parametrize("rows,D", NORM)
@pytest.mark.parametrize("f32,residual,pad", [(False, True, 8), (True, True, 0), (True, False, 3)])
def test_norm_in_8_bits(rows, D, f32, residual, pad):
    x, r, w = norm_case(rows, D, f32, residual, seed=7, pad=pad)
    q, s, h = pkg.add_rmsnorm_fp8(x, r, w, 1e-5)
    check_h(h, x, r)
    check_quantised(q, s, ol.rmsnorm(f64(h), f64(w), 1e-5))
    assert q.stride(0) % 16 == 0 and s.shape == (rows, (D + 127) // 128)


def test_norm_rows_of_zeros_and_infinities():
    x, r, w = norm_case(6, 384, True, True)
    x[0], r[0] = 0, 0
    x[2, 100], r[3, 200], r[4, 300] = float("inf"), float("-inf"), float("nan")
    r[5] *= 1e22  # its square leaves float32
    out, h = pkg.add_rmsnorm(x, r, w)
    assert (out[0] == 0).all() and out[1].isfinite().all() and (out[5] == 0).all()
    assert out[2, 100].isnan() and out[3, 200].isnan() and out[4].isnan().all()
    q, s, _ = pkg.add_rmsnorm_fp8(x, r, w)
    assert (q[0].float() == 0).all() and (s[0].float() == 2.0 ** -126).all()
    assert s[4].float().isnan().all() and q[4].float().isnan().all() and q[1].float().isfinite().all()


def test_norm_in_place_and_batches():
    x, r, w = norm_case(60, 256, True, True)
    want, h = pkg.add_rmsnorm(x, r, w)
    y, kept = x.view(3, 20, 256), r.clone().view(3, 20, 256)
    out, same = pkg.add_rmsnorm(y, kept, w, h=kept)
    assert same is kept and torch.equal(kept.view(60, 256), h) and torch.equal(out.view(60, 256), want)
    out, g = pkg.add_rmsnorm(y[:, :0], kept[:, :0], w)
    assert out.shape == (3, 0, 256) and g.shape == (3, 0, 256)
    one, _ = pkg.add_rmsnorm(x[7], r[7], w)
    assert torch.equal(one, want[7])


@pytest.mark.parametrize("rows,D", NORM)
@pytest.mark.parametrize("f32,with_dh", [(False, True), (True, True), (False, False)])
def test_norm_backward(rows, D, f32, with_dh):
    _, h, w = norm_case(rows, D, f32, True, seed=20)
    dout = rand((rows, D), 25)
    dh = rand((rows, D), 26, 1.0, h.dtype) if with_dh else None
    g = pkg.add_rmsnorm_backward(h.contiguous(), w, dout, dh, 1e-5)
    d, dw, size, wsize = ol.rmsnorm_backward(f64(h), f64(w), f64(dout), None if dh is None else f64(dh), 1e-5)
    within(g["dx"], d, 2.0 ** -8 * np.abs(d) + 2.0 ** -16 * size, "dx")
    within(g["dresidual"], d, (0 if f32 else 2.0 ** -8) * np.abs(d) + 2.0 ** -16 * size, "dresidual")
    within(g["dw"], dw, 2.0 ** -15 * wsize, "dw")
    assert f32 or g["dresidual"] is g["dx"]


@pytest.mark.parametrize("scale", [2.0 ** -50, 2.0 ** 50])
@pytest.mark.parametrize("D,f32", [(384, True), (1001, True), (520, False)])
def test_norm_backward_over_the_range(scale, D, f32):
    """Streams whose 1 / sqrt(mean(h^2)) has a cube outside float32; every result is inside."""
    _, h, w = norm_case(40, D, f32, True, seed=36)
    h, dout = h.contiguous() * scale, rand((40, D), 37)
    g = pkg.add_rmsnorm_backward(h, w, dout, None, 0.0)
    d, dw, size, wsize = ol.rmsnorm_backward(f64(h), f64(w), f64(dout), None, 0.0)
    within(g["dx"], d, 2.0 ** -8 * np.abs(d) + 2.0 ** -16 * size, "dx")
    within(g["dresidual"], d, (0 if f32 else 2.0 ** -8) * np.abs(d) + 2.0 ** -16 * size, "dresidual")
    within(g["dw"], dw, 2.0 ** -15 * wsize, "dw")


@pytest.mark.parametrize("rows,D", [(3, 1001), (5, 9), (3000, 37), (2500, 1340), (2, 8), (17, 8187)])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_rows_keep_to_themselves(rows, D, f32):
    """Rows side by side at any offset: a row of NaN changes no other, and nothing around a result is written."""
    _, h, w = norm_case(rows, D, f32, True, seed=90)
    x, r, dout, dh = rand((rows, D), 91), h.contiguous(), rand((rows, D), 92), rand((rows, D), 93, 1.0, h.dtype)

    def room(dtype):
        flat = torch.full((rows * D + 64,), 7.0, dtype=dtype, device=DEV)
        return flat, flat[32:32 + rows * D].view(rows, D)

    def call(x, dout):
        flats, places = zip(*(room(k) for k in (BF16, h.dtype, BF16, h.dtype)))
        pkg.add_rmsnorm(x, r, w, out=places[0], h=places[1])
        g = pkg.add_rmsnorm_backward(r, w, dout, dh, grads=dict(dx=places[2], dresidual=places[3]))
        for flat in flats:
            assert (flat[:32] == 7).all() and (flat[32 + rows * D:] == 7).all()
        return (*places, g["dw"])

    want = call(x, dout)
    for bad in {0, rows // 2, rows - 1}:
        y, d = x.clone(), dout.clone()
        y[bad] = d[bad] = float("nan")
        got = call(y, d)
        rest = torch.arange(rows, device=DEV) != bad
        for a, b in zip(got[:4], want[:4]):
            assert torch.equal(a[rest], b[rest]) and a[bad].isnan().all()
        assert got[4].isnan().all()


@pytest.mark.parametrize("rows,D", [(3, 1001), (5, 9), (3000, 37), (2500, 1340), (17, 8187), (40, 200)])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_rows_in_8_bits_keep_to_themselves(rows, D, f32):
    """The same in 8 bits: the bytes between rows stay as they were."""
    _, h, w = norm_case(rows, D, f32, True, seed=95)
    x, r, row = rand((rows, D), 96), h.contiguous(), (D + 15) // 16 * 16 + 16

    def call(x):
        flat = torch.full((rows + 1, row), 0x55, dtype=torch.uint8, device=DEV)
        q, s, h = pkg.add_rmsnorm_fp8(x, r, w, out=flat.view(torch.float8_e4m3fn)[:rows, :D])
        assert (flat[:rows, D:] == 0x55).all() and (flat[rows] == 0x55).all()
        return q.view(torch.uint8), s.view(torch.uint8), h

    want = call(x)
    check_quantised(want[0].view(torch.float8_e4m3fn), want[1].view(torch.float8_e8m0fnu),
                    ol.rmsnorm(f64(want[2]), f64(w), 1e-5))
    for bad in {0, rows // 2, rows - 1}:
        y = x.clone()
        y[bad] = float("nan")
        got = call(y)
        rest = torch.arange(rows, device=DEV) != bad
        assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got, want))
        assert (got[1][bad] == 255).all() and (got[0][bad] & 0x7f == 0x7f).all()


def test_norm_rows_of_one_infinity():
    """An infinity leaves the rest of its row zero, in 8 bits but for its block, and other rows as they are."""
    x, r, w = norm_case(4, 384, True, True)
    want, _ = pkg.add_rmsnorm(x, r, w)
    eight, scales, _ = pkg.add_rmsnorm_fp8(x, r, w)
    r[2, 200] = float("inf")
    out, _ = pkg.add_rmsnorm(x, r, w)
    q, s, _ = pkg.add_rmsnorm_fp8(x, r, w)
    rest = torch.arange(384, device=out.device) != 200
    assert out[2, 200].isnan() and (out[2][rest] == 0).all()
    assert s[2].float().isnan().tolist() == [False, True, False] and (q[2].float()[:128] == 0).all()
    assert (q[2].float()[256:] == 0).all() and q[2].float()[128:256].isnan().all()
    others = [0, 1, 3]
    assert torch.equal(out[others], want[others]) and torch.equal(s[others].float(), scales[others].float())
    assert torch.equal(q[others].float(), eight[others].float())


def test_norm_backward_against_differences():
    """The gradients against central differences of the oracle at the same point."""
    rows, D, step = 4, 136, 1e-6
    _, h, w = norm_case(rows, D, True, True, seed=30)
    h = h.contiguous()
    dout = rand((rows, D), 31)
    g = pkg.add_rmsnorm_backward(h, w, dout, None, 1e-5)
    H, W, O = f64(h), f64(w), f64(dout)
    for name, which, at in (("dresidual", 0, H), ("dw", 1, W)):
        v = np.random.default_rng(0).standard_normal(at.shape)
        a, b = [H, W], [H, W]
        a[which], b[which] = at + step * v, at - step * v
        slope = (np.sum(ol.rmsnorm(*a, 1e-5) * O) - np.sum(ol.rmsnorm(*b, 1e-5) * O)) / (2 * step)
        got = np.sum(f64(g[name]) * v)
        assert abs(got - slope) <= 2.0 ** -15 * np.sum(np.abs(f64(g[name]) * v)) + 1e-6


def test_norm_backward_repeats_and_empty():
    _, h, w = norm_case(3000, 520, False, True, seed=33)
    h, dout = h.contiguous(), rand((3000, 520), 34)
    a, b = (pkg.add_rmsnorm_backward(h, w, dout, dout) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
    kept = dout.clone()  # dx may take dh's place
    c = pkg.add_rmsnorm_backward(h, w, dout, kept, grads=dict(dx=kept))
    assert c["dx"] is kept and all(torch.equal(a[n], c[n]) for n in a)
    e = pkg.add_rmsnorm_backward(h[:0], w, dout[:0])
    assert (e["dw"] == 0).all() and e["dx"].shape == (0, 520)


# ---------------------------------------------------------------- product of 8-bit values
# M, N, K: single tokens, odd widths, the edges of tiles and of scale blocks, long sums
LINEAR = [(1, 1, 1), (1, 128, 128), (1, 2000, 1000), (2, 129, 127), (3, 8, 4096), (7, 256, 384), (16, 200, 144), (17, 130, 513),
          (33, 96, 2048), (64, 520, 640), (65, 128, 256), (100, 4384, 300), (127, 127, 127), (129, 257, 129), (200, 300, 1300),
          (255, 384, 96), (257, 136, 8192), (520, 1000, 520), (1021, 264, 200), (3, 5, 20000),
          (20, 6400, 1700), (86, 6381, 1500), (100, 3200, 3000), (60, 2700, 2600), (9, 2500, 4100), (2100, 2200, 300), (4000, 1300, 1280), (260, 16500, 2180), (2500, 2001, 700), (3000, 1158, 1821), (2049, 2052, 4000),
          (5000, 1000, 7), (20000, 100, 129), (19500, 1, 200), (2560, 1024, 640), (2432, 1024, 640), (129, 9800, 1040)]


def linear_case(M, N, K, seed=0):
    return (*pkg.quantise_fp8(values(M, K, seed).float().clamp(-1e4, 1e4)), *pkg.quantise_weight_fp8(rand((N, K), seed + 2, 1.0, F32)))


def check_linear(out, x, sx, w, sw):
    want, size = ol.linear(f64(x), f64(sx), f64(w), f64(sw))
    tol = 2.0 ** -23 * (x.shape[-1] / 32 + 2) * size
    within(out, want, tol + (2.0 ** -8 * np.abs(want) if out.dtype is BF16 else 0) + 1e-38)


@pytest.mark.parametrize("M,N,K", LINEAR)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear(M, N, K, dtype):
    args = linear_case(M, N, K)
    out = pkg.linear_fp8(*args, out_dtype=dtype)
    assert pkg.stream_status() == 0
    assert out.dtype is dtype and out.shape == (M, N)
    check_linear(out, *args)


@pytest.mark.parametrize("M,N,K", [(1, 384, 1000), (9, 200, 257), (70, 256, 2048), (300, 136, 130)])
def test_linear_quantises(M, N, K):
    """bf16 and float32 activations: the same bits as the two calls."""
    x, w = values(M, K, 3), pkg.quantise_weight_fp8(rand((N, K), 9, 0.1))
    for v in (x, x.float(), values(M, K + 5, 3)[:, :K]):
        assert torch.equal(pkg.linear_fp8(v, None, *w), pkg.linear_fp8(*pkg.quantise_fp8(v), *w))


def test_linear_leaves_what_is_not_its_own():
    """Rows behind the last one and values around a slice stay as they were; a wider row stride is taken."""
    M, N, K = 45, 136, 272
    args = linear_case(M, N, K, 4)
    room = torch.full((M + 40, N), 7.0, dtype=BF16, device=DEV)
    want = pkg.linear_fp8(*args)
    pkg.linear_fp8(*args, out=room[:M])
    assert torch.equal(room[:M], want) and (room[M:] == 7).all()
    wide = torch.empty((M, 512), dtype=torch.uint8, device=DEV).fill_(0x7f).view(FP8)  # NaN around the values
    wide[:, 16:16 + K].copy_(args[0])
    assert torch.equal(pkg.linear_fp8(wide[:, 16:16 + K], *args[1:]), want)


@pytest.mark.parametrize("K", [1300, 5000])
@pytest.mark.parametrize("first", [1, 2, 3])
def test_linear_of_some_tokens(K, first):
    """Scales of an odd number to a row, from any row on: whatever lies around the part does not count."""
    x, sx, w, sw = linear_case(300, 2100 if K == 1300 else 200, K, 3)
    want = pkg.linear_fp8(x, sx, w, sw)
    s = torch.full((302, sx.shape[1]), 255, dtype=torch.uint8, device=DEV).view(E8M0)  # NaN around it
    s.view(torch.uint8)[1:301] = sx.view(torch.uint8)
    for last in (300, 299, 270):
        out = pkg.linear_fp8(x[first:last], s[1 + first:1 + last], w, sw)
        assert torch.equal(out, want[first:last])
    M = 2400  # and the pairs' kernel
    x, sx, w, sw = linear_case(M, 2100, K, 4)
    want = pkg.linear_fp8(x, sx, w, sw)
    assert torch.equal(pkg.linear_fp8(x[first:], sx[first:], w, sw), want[first:])
    assert torch.equal(pkg.linear_fp8(x[:-first], sx[:-first], w, sw), want[:-first])


@pytest.mark.parametrize("M,N,K", [(1, 264, 1000), (40, 264, 1000), (2100, 2200, 300)])
@pytest.mark.parametrize("large", ["x", "w"])
def test_linear_scales_far_apart(M, N, K, large):
    """Activations and weights near opposite ends of float32, whose products are near one."""
    up, down = 2.0 ** 112, 2.0 ** -112
    x, w = rand((M, K), 80, up if large == "x" else down, F32), rand((N, K), 81, down if large == "x" else up, F32)
    args = (*pkg.quantise_fp8(x), *pkg.quantise_weight_fp8(w))
    check_linear(pkg.linear_fp8(*args, out_dtype=F32), *args)
    x = x.to(BF16)
    assert torch.equal(pkg.linear_fp8(x, None, *args[2:]), pkg.linear_fp8(*pkg.quantise_fp8(x), *args[2:]))


def test_linear_nan_stays_in_its_row_and_block():
    M, N, K = 40, 300, 400
    x, sx, w, sw = linear_case(M, N, K, 8)
    v = rand((M, K), 1)
    v[11, 399] = float("nan")
    out = pkg.linear_fp8(v, None, w, sw)
    bad = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    bad[11] = True
    assert torch.equal(out.isnan(), bad)
    u = rand((N, K), 2, 1.0, F32)
    u[130, 7] = float("inf")
    out = pkg.linear_fp8(x, sx, *pkg.quantise_weight_fp8(u))
    bad[:] = False
    bad[:, 128:256] = True
    assert torch.equal(out.isnan(), bad)


def test_linear_batches_and_repeats():
    x, sx, w, sw = linear_case(60, 264, 256)
    want = pkg.linear_fp8(x, sx, w, sw)
    out = pkg.linear_fp8(x.view(3, 20, 256), sx.view(3, 20, 2), w, sw)
    assert out.shape == (3, 20, 264) and torch.equal(out.view(60, 264), want)
    assert pkg.linear_fp8(x[:0], sx[:0], w, sw).shape == (0, 264)


# ---------------------------------------------------------------- gradients
def tensors(sizes, seed, kinds, scale=1.0):
    return [rand((n,), seed + i, scale, k) for i, (n, k) in enumerate(zip(sizes, kinds))]


SIZES = {
    "one": [1], "odd": [1, 2, 3, 7, 8, 9, 15, 17], "chunks": [8191, 8192, 8193, 16384, 16385, 50000],
    "many": [5 + 3 * i for i in range(300)], "launches": [1 + i % 4 for i in range(2100)], "empty": [0, 5, 0], "none": [0],
}


def check_clip(grads, most, got, norm):
    n, want = ol.clip([f64(g) for g in grads], most)
    # 2^-150: half a step of float32 below 2^-126, where its steps are 2^-149.  From 2^128 on the nearest float32
    # is infinity (the largest finite one is 2^128 - 2^104); the clipping goes by the 64-bit norm.
    assert float(norm) == np.inf if n >= 2.0 ** 128 else abs(float(norm) - n) <= 2.0 ** -21 * n + 2.0 ** -150
    for g, w in zip(got, want):
        half = 2.0 ** -8 if g.dtype is BF16 else 2.0 ** -24
        within(g, w, (half + 2.0 ** -20) * np.abs(w) + (2.0 ** -134 if g.dtype is BF16 else 2.0 ** -150))


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("mixed", [0, 1, 2])
@pytest.mark.parametrize("most", [0.5, 1e6])
def test_clip(name, mixed, most):
    sizes = SIZES[name]
    kinds = [F32 if mixed == 0 or mixed == 2 and i % 2 else BF16 for i in range(len(sizes))]
    grads = tensors(sizes, 40, kinds)
    before = [g.clone() for g in grads]
    out = [torch.empty_like(g) for g in grads]
    norm = pkg.clip_grad_norm(grads, most, out=out)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    check_clip(before, most, out, norm)
    again = pkg.clip_grad_norm(grads, most)
    assert torch.equal(norm, again) and all(torch.equal(a, b) for a, b in zip(grads, out))
    assert torch.equal(pkg.grad_norm(before), norm)


@pytest.mark.parametrize("off,to", [(1, 1), (3, 0), (0, 5), (2, 7)])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_clip_unaligned(off, to, kind):
    """Gradients in flat buffers: any boundary of their type, and outputs on another one."""
    flat, room = rand((40000,), 50, 1.0, kind), torch.full((40100,), 9.0, dtype=kind, device=DEV)
    sizes = [off, 9001, 3, 20000] if off else [9001, 3, 20000]
    grads = [t for t in flat[:sum(sizes)].split(sizes)][1 if off else 0:]
    out = list(room[to:to + sum(t.numel() for t in grads)].split([t.numel() for t in grads]))
    norm = pkg.clip_grad_norm(grads, 3.0, out=out)
    check_clip(grads, 3.0, out, norm)
    n = to + sum(t.numel() for t in grads)
    assert (room[:to] == 9).all() and (room[n:] == 9).all()


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-20, 1e15, 1e25, 1e37])
def test_clip_over_the_range(kind, scale):
    """Squares that leave float32's range on either side, beside zeros and values of another size."""
    grads = tensors([1000, 37, 9000], 60, [kind] * 3, scale)
    grads[1].zero_()
    grads[2][::3] *= 1e-4
    out = [torch.empty_like(g) for g in grads]
    most = scale  # far below the norm
    check_clip(grads, float(np.float32(most)), out, pkg.clip_grad_norm(grads, most, out=out))


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("scale", [2e18, 1e17])
def test_clip_sums_that_leave_the_range_together(kind, scale):
    """Squares whose sums over a part of a thread's values stay below 2^128, those over all of its values not."""
    grads = tensors([12_000_001], 61, [kind], scale)
    out = [torch.empty_like(g) for g in grads]
    check_clip(grads, 1.0, out, pkg.clip_grad_norm(grads, 1.0, out=out))


def test_clip_zero_and_not_finite():
    grads = tensors([100, 9], 70, [F32, BF16])
    before = [g.clone() for g in grads]
    for bad in (float("inf"), float("nan")):
        grads[1][4] = bad
        norm = pkg.clip_grad_norm(grads, 1.0)
        assert not norm.isfinite() and torch.equal(grads[0], before[0])
        out = [torch.empty_like(g) for g in grads]
        pkg.clip_grad_norm(grads, 1.0, out=out)
        assert torch.equal(out[0], before[0]) and torch.equal(out[1][:4], before[1][:4])
    grads = [torch.zeros(1000, device=DEV), torch.zeros(3, dtype=BF16, device=DEV)]
    assert float(pkg.clip_grad_norm(grads, 1.0)) == 0 and (grads[0] == 0).all()
    grads = tensors([100, 9], 70, [F32, BF16])
    pkg.clip_grad_norm(dict(a=grads[0], b=grads[1]), 0.0)
    assert all((g == 0).all() for g in grads)


def test_clip_refuses_shared_memory():
    flat = torch.ones(100, device=DEV)
    for grads, out in (([flat, flat], None), ([flat[:60], flat[50:]], None), ([flat[:50]], [flat[10:60]]),
                       ([flat[:50], flat[50:]], [flat[50:], flat[:50]])):
        with pytest.raises(binding.M2RNNError):
            pkg.clip_grad_norm(grads, 1.0, out=out)
    assert (flat == 1).all()
    assert float(pkg.grad_norm([flat, flat])) == pytest.approx(200 ** 0.5)
    with pytest.raises(binding.M2RNNError):
        pkg.clip_grad_norm([flat], -1.0)
    with pytest.raises(binding.M2RNNError):
        pkg.clip_grad_norm([flat], float("nan"))
